"""Sizes past 32 bits, which the library's int32 arguments cannot hold, are refused by the bindings of the norm, the gated
products and the embedding (no GPU: the operands are stand-ins).  So is no id beyond them taken for another one."""
import pytest
import torch

from csr_bsr_spmv_gb300 import spx
from test_block_devices import current  # noqa: F401  (fixture)
from test_experts_devices import BF16, F32, I32, Far, Library

BIG = [2 ** 31, 2 ** 32 + 3]


def calls(n):
    """Every binding with a size of n in one place."""
    def m(shape, dtype=BF16):
        return Far(shape, dtype, 0)

    off = m((4,), I32)
    return {
        "norm rows": lambda: spx.spx_rms_norm(m((n, 8)), Y=m((n, 8))),
        "norm columns": lambda: spx.spx_rms_norm(m((1, n)), Y=m((1, n))),
        "norm to 8 bits": lambda: spx.spx_rms_norm_i8(m((n, 8)), Q=m((n, 8), torch.int8), scale=m((n,), F32)),
        "norm gradient": lambda: spx.spx_rms_norm_grad(m((n, 8)), m((n, 8)), m((n,), F32), dX=m((n, 8)), dweight=False),
        "gated rows": lambda: spx.spx_gemm_grouped_gated(off, m((n, 8)), m((3, 16, 8)), C=m((n, 8))),
        "gated weights": lambda: spx.spx_gemm_grouped_gated(off, m((4, 8)), m((3, 2 * n, 8)), C=m((4, n))),
        "gated weights of one": lambda: spx.spx_gemm_grouped_gated(None, m((4, 8)), m((2 * n, 8)), C=m((4, n))),
        "gate's gradient": lambda: spx.spx_gemm_grouped_gated_grad(off, m((n, 8)), m((3, 8, 16)), m((n, 32)), dH=m((n, 32)),
                                                                   product=False),
        "table": lambda: spx.spx_embed(m((4,), I32), m((n, 8)), Y=m((4, 8))),
        "tokens": lambda: spx.spx_embed(m((n,), I32), m((40, 8)), Y=m((n, 8))),
        "table's gradient": lambda: spx.spx_embed_grad(m((4,), I32), m((4, 8)), n, dW=m((n, 8)), scratch=m((64,), torch.uint8)),
        "its tokens": lambda: spx.spx_embed_grad(m((n,), I32), m((n, 8)), 40, dW=m((40, 8)), scratch=m((64,), torch.uint8)),
    }


@pytest.mark.parametrize("name", calls(0))
@pytest.mark.parametrize("n", BIG)
def test_sizes_past_32_bits_are_refused(current, name, n):  # noqa: F811
    before = Library.calls
    with pytest.raises(ValueError):
        calls(n)[name]()
    assert Library.calls == before


@pytest.mark.parametrize("padding,passed", [(None, -1), (3, 3), (0, 0), (39, 39), (40, -1), (-100, -1), (2 ** 32 + 3, -1), (-2 ** 32 + 3, -1)])
def test_padding_beyond_the_table_is_no_id(current, monkeypatch, padding, passed):  # noqa: F811
    seen = []

    class Seen(Library):
        def __getattr__(self, name):
            if name == "spx_embed_grad":
                return lambda *a: seen.append(a[6]) or 0
            return super().__getattr__(name)

    monkeypatch.setattr(spx, "_lib", Seen)
    spx.spx_embed_grad(Far((4,), I32, 0), Far((4, 8), BF16, 0), 40, padding=padding, dW=Far((40, 8), BF16, 0),
                       scratch=Far((64,), torch.uint8, 0))
    assert seen == [passed]
