"""Rules of the kernels that start before the stream's previous kernel has ended
(csrc/dependent_launch.cuh), read off their sources: nothing is loaded before the wait, and
no load goes through the read-only path, which is for data that nothing writes while the
kernel runs, or through another function whose loads the compiler may move over the wait."""

import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "block_sparse_attention_48_b200", "csrc")
KERNELS = ("rope.cu", "paged_decode.cu", "shared_prefix.cu")
HEADERS = ("paged_decode_impl.cuh", "paged_walk.cuh", "shared_walk.cuh", "rope.cuh", "dependent_launch.cuh")


def _code(name):
    with open(os.path.join(CSRC, name)) as f:
        return re.sub(r"//[^\n]*|/\*.*?\*/", "", f.read(), flags=re.S)


@pytest.mark.parametrize("name", KERNELS + HEADERS)
def test_no_read_only_loads(name):
    found = re.findall(r"\b__ld\w+|ld\.global\.nc|\bldg_\w+|__restrict__", _code(name))
    assert not found, f"{name}: {found}"


@pytest.mark.parametrize("name", KERNELS)
def test_nothing_is_read_before_the_wait(name):
    code = _code(name)
    kernels = re.findall(r"__global__[^;{]*\{", code)
    assert kernels
    for head in kernels:
        body = code[code.index(head) + len(head):]
        assert "wait_prerequisites();" in body, head
        before = body[:body.index("wait_prerequisites();")]
        # any pointer of the parameters, a load of any kind, or a function that is given them
        found = re.findall(r"p\.(?:seq_lens|page_table|prefix_row|positions|cache_lens|new_lens|q\b|lse|slopes|inv_freq|"
                           r"split|part_ml|part_o|own_ml|own_o|o\b|status|tm_k|tm_v)|ld\.global|"
                           r"scan_lengths|tma_load\w*|\bg\.x\b", before)
        assert not found, f"{name}, before the wait in {head.split('(')[0].split()[-1]}: {found}"


def test_every_dependent_launch_is_of_such_a_kernel():
    """launch_after is used in these files alone."""
    for name in sorted(os.listdir(CSRC)):
        if name.endswith((".cu", ".cuh", ".cpp")) and name not in KERNELS + ("dependent_launch.cuh",):
            assert "launch_after(" not in _code(name), name
