"""The tile rule of the experts' products (plain host arithmetic, compiled here with the host compiler): what it may
choose for any size, and that the sizes of the GPU tests reach every form of the kernel on 152 SMs."""
import ctypes
import os
import subprocess

import pytest

import experts_forms

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "csr_bsr_spmv_gb300", "csrc")
PRODUCT, GRADIENT, CODES = 0, 1, 2
SMS = 152


@pytest.fixture(scope="module")
def rule(tmp_path_factory):
    d = tmp_path_factory.mktemp("tile")
    src, lib = d / "tile.cpp", d / "libtile.so"
    src.write_text('#include "spx_experts_tile.h"\n'
                   'extern "C" void tile(int kind, int E, int S, int NL, int NC, int NR, int sms, int* out) {\n'
                   '    const spx_exp::Tile t = spx_exp::choose_tile(static_cast<spx_exp::Kind>(kind), E, S, NL, NC, NR, sms);\n'
                   '    out[0] = t.tn, out[1] = t.cg, out[2] = t.split, out[3] = t.split_red;\n}\n')
    subprocess.run(["g++", "-std=c++17", "-O1", "-shared", "-fPIC", "-I", CSRC, str(src), "-o", str(lib)], check=True)
    f = ctypes.CDLL(str(lib)).tile

    def choose(kind, E, S, NL, NC, NR):
        out = (ctypes.c_int * 4)()
        f(kind, E, S, NL, NC, NR, SMS, out)
        return tuple(out)

    return choose


SIZES = (1, 2, 8, 31, 64, 65, 100, 128, 129, 200, 256, 257, 700, 2048, 5000)


@pytest.mark.parametrize("E", [1, 2, 8, 64, 300])
def test_every_choice_is_one_the_kernel_has(rule, E):
    for NL in SIZES:
        for m in SIZES:
            for R in (1, 64, 777, 4096, 40000):
                for kind in (PRODUCT, CODES):
                    tn, cg, split, red = rule(kind, E, m, NL, 0, R)
                    assert tn in ((32, 64, 128) if kind == CODES else (32, 64, 128, 256)) and split in (1, 2, 4, 8)
                    assert cg == 1 or (kind == PRODUCT and cg == 2 and NL > 128 and split == 1 and tn >= 128)
                    assert split == 1 or tn <= 128
                    assert tn == 32 or tn == 64 or tn / 2 < m  # no tile that a smaller one would hold
                    unit = 128 if kind == CODES else 64
                    assert red % unit == 0 and red * split >= R and (split == 1 or red * (split - 1) < R + split * unit)
                tn, cg, split, _ = rule(GRADIENT, E, R, NL, m, 0)
                assert tn in (128, 256) and split == 1 and (cg == 1 or NL > 128), (E, R, NL, m)
                assert tn == 128 or m > 128, "a gradient of few rows on a tile that is mostly empty"


def forms(rule, kind, cases):
    if kind == GRADIENT:
        return {rule(kind, E, S, K, N, 0)[:3] for _, E, S, N, K in cases}
    return {rule(kind, E, S, N, 0, K)[:3] for _, E, S, N, K in cases}


def test_the_gpu_tests_reach_every_form(rule):
    shared = {(tn, 1, split) for tn in (32, 64, 128) for split in (1, 2, 4, 8)}
    pairs = {(128, 2, 1), (256, 2, 1)}
    assert forms(rule, PRODUCT, experts_forms.PRODUCTS) == shared | pairs | {(256, 1, 1)}
    assert forms(rule, GRADIENT, experts_forms.GRADIENTS) == pairs | {(128, 1, 1), (256, 1, 1)}
    assert forms(rule, CODES, experts_forms.WIDENED) == shared
    assert forms(rule, PRODUCT, experts_forms.COPIED) >= pairs | {(tn, 1, s) for tn in (64, 128) for s in (1, 2, 4)}
    assert all(S > 128 * E for _, E, S, _, _ in experts_forms.COPIED)
    assert all(16 * E < S <= 128 * E for _, E, S, _, _ in experts_forms.WIDENED)
