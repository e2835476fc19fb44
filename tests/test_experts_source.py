"""What the routed-expert kernels' sources have to keep to, read as text (no GPU): faults that would show on
hardware only once in a long while, or by hanging it, are refused here."""
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "csr_bsr_spmv_gb300", "csrc")
FILES = ["spx_route.cu", "spx_int8.cu", "spx_experts.cu", "spx_experts.cuh", "spx_experts_simt.cu", "spx_experts_tc.cu"]


def code(name):
    """The file without its comments."""
    text = open(os.path.join(CSRC, name)).read()
    return re.sub(r"//[^\n]*|/\*.*?\*/", "", text, flags=re.S)


@pytest.mark.parametrize("name", FILES)
def test_kernels_launched_early_read_no_memory_as_read_only(name):
    """A kernel launched with programmatic serialisation is resident while the calls before it write its inputs,
    and the read-only path is defined only for memory that nobody writes during the kernel's life."""
    assert not re.search(r"\b__ldg\b|\b__restrict__\b|ld\.global\.nc", code(name))


def test_every_kernel_launched_early_waits_before_it_reads():
    for name in FILES:
        text = code(name)
        for k in re.findall(r"__global__.*?\n}", text, flags=re.S):
            assert "wait_for_previous();" in k, k[:200]
            first = re.search(r"\bload(_once)?(<[^;(]*>)?\(|\bexpert_rows\(|\bwarp_find_tile\(", k)
            assert first is None or k.index("wait_for_previous();") < first.start(), k[:200]


def test_addresses_are_taken_behind_the_wait():
    """A load whose address is known at the kernel's start may be moved above the wait: every pointer that a kernel
    reads through passes behind_wait() first, parameters right after the wait."""
    for name in FILES:
        text = code(name)
        for k in re.findall(r"__global__.*?\n}", text, flags=re.S):
            params, body = k[:k.index("{")], k[k.index("wait_for_previous();"):]
            for p in re.findall(r"const [\w:<> ]+\* (\w+)", params):
                assert re.search(r"\b%s = behind_wait\(%s\)" % (p, p), body), (name, p, params[:200])
            for field in re.findall(r"\bload(?:_once)?\((a\.\w+|g\.\w+|x\.p)", body):
                assert "%s = behind_wait(%s)" % (field, field) in body, (name, field)
        for field in re.findall(r"\bload(?:_once)?\((a\.\w+)", text):
            assert "%s = behind_wait(%s)" % (field, field) in text, (name, field)


def test_the_abort_flag_is_read_in_a_vote():
    """Lanes of a warp may read the flag at different times: unless they vote on it, part of a warp can leave a loop
    whose next whole-warp instruction the rest then waits at for ever."""
    text = code("spx_experts_tc.cu")
    reads = [m.start() for m in re.finditer(r"!\s*s_abort", text)]
    assert reads
    for at in reads:
        statement = text[max(text.rfind(c, 0, at) for c in ";{}"):at]
        vote = statement.rfind("__all_sync(")
        assert vote >= 0 and statement[vote:].count("(") > statement[vote:].count(")"), statement
