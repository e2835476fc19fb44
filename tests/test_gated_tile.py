"""The tile rule for the gated products (plain host arithmetic, compiled here with the host compiler): that the sizes of
the GPU tests reach every form of the kernels on 152 SMs, and what the rule may choose for the gate's gradient."""
import pytest

import gated_forms
from test_experts_tile import PRODUCT, SIZES, rule  # noqa: F401  (the fixture)

BACK = 3
SHARED = {(tn, 1, split) for tn in (32, 64, 128) for split in (1, 2, 4, 8)}
LARGE = {(256, 1, 1), (128, 2, 1), (256, 2, 1)}


def test_the_gpu_tests_reach_every_form(rule):  # noqa: F811
    assert {rule(PRODUCT, E, S, 2 * F, 0, K)[:3] for E, S, F, K in gated_forms.GATE} == SHARED | LARGE
    assert {rule(BACK, E, S, F, 0, N)[:3] for E, S, F, N in gated_forms.BACK} == SHARED | LARGE


@pytest.mark.parametrize("E", [1, 8, 300])
def test_every_choice_is_one_the_kernel_has(rule, E):  # noqa: F811
    for F in SIZES:
        for S in SIZES:
            for N in (1, 64, 777, 4096, 40000):
                tn, cg, split, red = rule(BACK, E, S, F, 0, N)
                assert (tn, cg, split) in SHARED | LARGE and (cg == 1 or F > 128)
                assert tn == 32 or tn == 64 or tn / 2 < S
                assert red % 64 == 0 and red * split >= N
