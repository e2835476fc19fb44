"""What the sources of the norm, the gates and the embedding have to keep to, read as text (no GPU): a kernel launched with
programmatic serialisation is resident while the calls before it write its inputs."""
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "csr_bsr_spmv_gb300", "csrc")
FILES = ["spx_norm.cu", "spx_embed.cu", "spx_gated.cu", "spx_rows.cuh", "spx_act.cuh"]


def code(name):
    text = open(os.path.join(CSRC, name)).read()
    return re.sub(r"//[^\n]*|/\*.*?\*/", "", text, flags=re.S)


@pytest.mark.parametrize("name", FILES)
def test_no_memory_is_read_as_read_only(name):
    assert not re.search(r"\b__ldg\b|\b__restrict__\b|ld\.global\.nc", code(name))


@pytest.mark.parametrize("name", ["spx_norm.cu", "spx_embed.cu"])
def test_every_kernel_waits_before_it_reads_and_lets_the_next_start(name):
    kernels = re.findall(r"__global__.*?\n}", code(name), flags=re.S)
    assert len(kernels) >= 4
    for k in kernels:
        assert "let_next_start();" in k and "wait_for_previous();" in k, k[:200]
        start = k[:k.index("wait_for_previous();")]
        assert not re.search(r"\b(load|load_once|read|read_any|copy_piece|copy_near|fetch|weights)(<[^;(]*>)?\(", start), k[:200]


@pytest.mark.parametrize("name", ["spx_norm.cu", "spx_embed.cu"])
def test_addresses_are_taken_behind_the_wait(name):
    """Every pointer that a kernel reads through passes behind_wait(): arguments and the fields of its argument struct."""
    for k in re.findall(r"__global__.*?\n}", code(name), flags=re.S):
        params, body = k[:k.index("{")], k[k.index("wait_for_previous();"):]
        for p in re.findall(r"const [\w:<> ]+\* (\w+)", params):
            assert re.search(r"\b%s = behind_wait\(%s\)" % (p, p), body), (name, p)
        for field in re.findall(r"static_cast<const \w+\*>\((a\.\w+)\)", body):
            assert "behind_wait(static_cast<const" in body and re.search(r"behind_wait\(static_cast<const \w+\*>\(%s\)\)" % re.escape(field), body), field
        for field in re.findall(r"\bload(?:_once)?\((a\.\w+)", body):
            raise AssertionError(field)
