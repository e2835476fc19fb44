"""Chains of routed-expert calls on one stream, whose kernels are launched before the ones ahead of them end."""
import ctypes

import numpy as np
import pytest
import torch

from csr_bsr_spmv_gb300 import spx

pytestmark = pytest.mark.gpu


def ptr(t):
    return ctypes.c_void_p(t.data_ptr())


@pytest.mark.parametrize("T,k,E,H", [(8, 2, 4, 64), (300, 2, 8, 128), (3000, 4, 16, 96), (9000, 2, 32, 64)])
@pytest.mark.parametrize("graph", [False, True])
def test_back_to_back_calls_see_the_arrays_of_their_own_turn(T, k, E, H, graph):
    """Sort, return and gradient over the same arrays again and again, the ids of each turn written by a gather right
    before the sort that reads them, nothing else on the stream and no wait on the host: every turn's places, sums
    and gradients are those of its own ids.  Whole numbers with small sums, so they are exact."""
    turns = 12
    rng = np.random.default_rng(T + E)
    tables = rng.integers(-1, E, (turns, T, k)).astype(np.int32)
    lib = spx._lib()
    # row t of `all_ids` holds token t's ids of every turn; a turn's gather copies its columns, bits unchanged
    all_ids = torch.from_numpy(np.ascontiguousarray(tables.transpose(1, 0, 2)).reshape(T, turns * k)).cuda()
    same = spx.spx_route_build(torch.zeros(T, 1, dtype=torch.int32, device="cuda"), 1)
    Ys = torch.from_numpy(rng.integers(-3, 4, (T * k, H)).astype(np.float32)).cuda()
    w = torch.from_numpy(rng.integers(-2, 3, (T, k)).astype(np.float32)).cuda()
    dev = dict(device="cuda", dtype=torch.int32)
    ids, off, slot, pos = (torch.empty(n, **dev) for n in (T * k, E + 1, T * k, T * k))
    need = lib.spx_route_scratch_bytes(T, k, E)
    scratch = torch.empty(max(need, 4) // 4, **dev)
    Y = torch.zeros(turns, T, H, device="cuda")
    dYs = torch.zeros(turns, T * k, H, device="cuda")
    dw = torch.zeros(turns, T, k, device="cuda")
    places = torch.zeros(turns, T * k, **dev)
    torch.cuda.synchronize()

    def chain():
        st = torch.cuda.current_stream().cuda_stream
        for i in range(turns):
            spx._check(lib.spx_route_gather(T, 1, k, 0, ptr(same.pos), ctypes.c_void_p(same.offsets.data_ptr() + 4),
                                            ctypes.c_void_p(all_ids.data_ptr() + 4 * k * i), turns * k, ptr(ids), k, st), "ids")
            spx._check(lib.spx_route_build(T, k, E, ptr(ids), 4, k, ptr(off), ptr(slot), ptr(pos), ptr(scratch), need, st),
                       "build")
            end = ctypes.c_void_p(off.data_ptr() + 4 * E)
            spx._check(lib.spx_route_combine(T, k, H, 0, ptr(pos), ptr(w), ptr(Ys), H, ptr(Y[i]), H, st), "combine")
            spx._check(lib.spx_route_combine_grad(T, k, H, 0, ptr(pos), end, ptr(w), ptr(Y[i]), H, ptr(Ys), H, ptr(dYs[i]), H,
                                                  ptr(dw[i]), st), "grad")
            spx._check(lib.spx_route_gather(1, 1, T * k, 0, ptr(same.pos), ctypes.c_void_p(same.offsets.data_ptr() + 4),
                                            ptr(pos), T * k, ptr(places[i]), T * k, st), "places")

    if graph:
        chain()
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            chain()
        run = g.replay
    else:
        run = chain
    ysn, wn = Ys.cpu().numpy().astype(np.float64), w.cpu().numpy().astype(np.float64).reshape(-1)
    for _ in range(4):
        run()
    torch.cuda.synchronize()
    for i in range(turns):
        x = tables[i].reshape(-1)
        kept = np.nonzero(x >= 0)[0]
        order = kept[np.argsort(x[kept], kind="stable")]
        at = np.full(T * k, -1)
        at[order] = np.arange(order.size)
        assert np.array_equal(places[i].cpu().numpy(), at), i
        rows = np.where(at[:, None] >= 0, ysn[np.maximum(at, 0)], 0.0)
        y = (rows * wn[:, None]).reshape(T, k, H).sum(1)
        assert np.array_equal(Y[i].cpu().numpy(), y), i
        g_rows = np.repeat(y, k, axis=0)
        want = np.zeros((T * k, H))
        want[at[kept]] = (g_rows * wn[:, None])[kept]
        assert np.array_equal(dYs[i].cpu().numpy(), want), i
        assert np.array_equal(dw[i].cpu().numpy().reshape(-1), (g_rows * rows).sum(1)), i


def test_back_to_back_products_see_the_arrays_of_their_own_turn():
    """Quantise, 8-bit product, 16-bit product and gradient over the same buffers, the input of each turn written by a
    gather just before: few rows (straight from memory), more (widened on the way) and many (widened first)."""
    lib = spx._lib()
    for S, N, K in ((2, 64, 256), (12, 96, 256), (60, 160, 384), (700, 160, 384)):
        turns = 8
        rng = np.random.default_rng(S)
        X = torch.from_numpy(rng.integers(-3, 4, (S, turns * K)).astype(np.float32)).cuda()
        X[:, ::K] = 127.0  # every row's scale is 1, its codes are its values
        W = torch.from_numpy(rng.integers(-3, 4, (N, K)).astype(np.float32)).cuda()
        W8, one = W.to(torch.int8), torch.ones(N, device="cuda")
        W16 = W.half()
        same = spx.spx_route_build(torch.zeros(S, 1, dtype=torch.int32, device="cuda"), 1)
        cols = torch.empty(S, K, device="cuda")
        q, s = torch.empty(S, K, dtype=torch.int8, device="cuda"), torch.empty(S, device="cuda")
        out = [torch.empty(S, N, device="cuda") for _ in range(turns)]
        scratch = torch.empty(max(256, lib.spx_gemm_i8_scratch_bytes(1, S, N, K, 1)), dtype=torch.uint8, device="cuda")
        G = torch.from_numpy(rng.integers(-1, 2, (S, N)).astype(np.float32)).cuda().half()
        X16 = X.half()
        prod = [torch.empty(S, N, device="cuda") for _ in range(turns)]
        dW = [torch.empty(1, N, K, device="cuda") for _ in range(turns)]
        h = torch.empty(S, K, dtype=torch.float16, device="cuda")
        torch.cuda.synchronize()
        for _ in range(3):
            for i in range(turns):
                spx.spx_route_gather(same, X[:, i * K:(i + 1) * K], cols)
                spx.spx_quant_rows_i8(cols, q, s)
                spx.spx_gemm_i8(q, s, W8, one, C=out[i], scratch=scratch)
                spx.spx_route_gather(same, X16[:, i * K:(i + 1) * K], h)
                spx.spx_gemm_grouped(same.offsets, h, W16[None], prod[i])
                spx.spx_gemm_grouped_wgrad(same.offsets, G, h, dW[i])
        torch.cuda.synchronize()
        assert spx.spx_last_device_error() == 0
        for i in range(turns):
            x = X[:, i * K:(i + 1) * K].double()
            assert torch.equal(out[i].double(), x @ W.double().T), (S, i)
            assert torch.equal(prod[i].double(), x @ W.double().T), (S, i)
            assert torch.equal(dW[i][0].double(), G.double().T @ x), (S, i)
