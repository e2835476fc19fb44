"""Routed experts on the bounds-checked build: wrong places and offsets -- which every build keeps inside the arrays --
are reported as SPX_ERR_INDEX_RANGE by spx_last_device_error; right ones are not, and give the product build's bits."""
import pytest
import torch

from csr_bsr_spmv_gb300 import spx

pytestmark = pytest.mark.gpu

INDEX_RANGE = -2
T, K_SLOTS, E, H, N = 300, 2, 5, 64, 128
S = T * K_SLOTS


def operands():
    g = torch.Generator(device="cuda")
    g.manual_seed(3)
    ids = torch.randint(-1, E, (T, K_SLOTS), device="cuda", generator=g)

    def normal(*shape):
        return torch.randn(*shape, device="cuda", generator=g)

    return ids, normal(T, H).bfloat16(), normal(E, N, H).bfloat16(), normal(T, K_SLOTS)


def every_call(r, X, W, w):
    """The outputs of every call that reads places or offsets, in every form that reads them in its own way."""
    Xs = spx.spx_route_gather(r, X)
    C = spx.spx_gemm_grouped(r.offsets, Xs, W)
    out = [Xs, C, spx.spx_route_combine(r, C, w), *spx.spx_route_combine_grad(r, X, Xs, w)]
    out += [spx.spx_gemm_grouped(r.offsets, Xs[:, 1:], W[:, :, 1:]),  # off 16 bytes: the CUDA cores
            spx.spx_gemm_grouped_wgrad(r.offsets, C, Xs), spx.spx_gemm_grouped_wgrad(r.offsets, C[:, 1:], Xs)]
    q, s = spx.spx_quant_rows_i8(Xs)
    W8, ws = W.to(torch.int8), torch.ones(E, N, device="cuda")
    out += [spx.spx_gemm_i8(q, s, W8, ws, offsets=r.offsets), spx.spx_gemm_i8(q[:, 1:], s, W8[:, :, 1:], ws, offsets=r.offsets)]
    return out


def test_valid_routing_is_bitwise_the_product_build():
    ids, X, W, w = operands()
    want = every_call(spx.spx_route_build(ids, E), X, W, w)
    with spx.checked_build():
        got = every_call(spx.spx_route_build(ids, E), X, W, w)
        assert spx.spx_last_device_error() == 0
    assert all(torch.equal(a, b) for a, b in zip(got, want))


@pytest.mark.parametrize("value", [-2, S, 2 ** 30])
@pytest.mark.parametrize("call", ["gather", "combine", "grad"])
def test_wrong_places_are_reported(value, call):
    ids, X, W, w = operands()
    with spx.checked_build():
        r = spx.spx_route_build(ids, E)
        Ys = torch.ones(S, H, device="cuda", dtype=torch.bfloat16)
        pos = r.pos.clone()
        pos[S // 2] = value
        bad = spx.Route(T, K_SLOTS, E, r.offsets, r.slot, pos)
        run = {"gather": lambda x: spx.spx_route_gather(x, X), "combine": lambda x: spx.spx_route_combine(x, Ys, w),
               "grad": lambda x: spx.spx_route_combine_grad(x, X, Ys, w)}[call]
        run(bad)
        assert spx.spx_last_device_error() == INDEX_RANGE
        run(r)
        assert spx.spx_last_device_error() == 0


@pytest.mark.parametrize("bad", [[0, 500, 100, 200, 300, 400], [-7, 3, 200, 210, 220, 230], [0, 1, 2, 3, 4, S + 1]])
@pytest.mark.parametrize("form", ["product", "gradient", "cores", "cores' gradient", "few rows", "widened", "copied"])
def test_wrong_offsets_are_reported(bad, form):
    ids, X, W, w = operands()
    with spx.checked_build():
        A = torch.ones(S, H, device="cuda", dtype=torch.bfloat16)
        G = torch.ones(S, N, device="cuda", dtype=torch.bfloat16)
        W8, ws = W.to(torch.int8), torch.ones(E, N, device="cuda")
        q, s = spx.spx_quant_rows_i8(A)
        run = {"product": lambda o: spx.spx_gemm_grouped(o, A, W),
               "gradient": lambda o: spx.spx_gemm_grouped_wgrad(o, G, A),
               "cores": lambda o: spx.spx_gemm_grouped(o, A[:, 1:], W[:, :, 1:]),
               "cores' gradient": lambda o: spx.spx_gemm_grouped_wgrad(o, G[:, 1:], A),
               "few rows": lambda o: spx.spx_gemm_i8(q[:40], s[:40], W8, ws, offsets=o),
               "widened": lambda o: spx.spx_gemm_i8(q, s, W8, ws, offsets=o),
               "copied": lambda o: spx.spx_gemm_i8(q[:, 1:], s, W8[:, :, 1:], ws, offsets=o)}[form]
        run(torch.tensor(bad, dtype=torch.int32, device="cuda"))
        assert spx.spx_last_device_error() == INDEX_RANGE
        rows = 40 if form == "few rows" else S
        run(torch.tensor([0, 5, 5, 20, 30, rows], dtype=torch.int32, device="cuda"))
        assert spx.spx_last_device_error() == 0


def test_the_end_of_the_sorted_rows_is_tested():
    ids, X, W, w = operands()
    with spx.checked_build():
        r = spx.spx_route_build(ids, E)
        for end in (-1, S + 1):
            off = r.offsets.clone()
            off[E] = end
            bad = spx.Route(T, K_SLOTS, E, off, r.slot, r.pos)
            spx.spx_route_gather(bad, X)
            assert spx.spx_last_device_error() == INDEX_RANGE
            spx.spx_route_combine_grad(bad, X)
            assert spx.spx_last_device_error() == INDEX_RANGE
