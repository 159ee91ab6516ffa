"""The serving calls' rules that need no GPU: what a workspace is sized for, soft caps that
fp32 cannot work with, and how many teams a call gets (csrc/serving_rules.h, built for the
host)."""

import ctypes
import math
import os
import random
import subprocess

import pytest

import block_sparse_attention_48_b200 as fa

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
BUILD = os.path.join(ROOT, "tests", "host", "_build")


@pytest.fixture(scope="module")
def rules():
    os.makedirs(BUILD, exist_ok=True)
    out = os.path.join(BUILD, "libservingrules.so")
    subprocess.check_call(["g++", "-O2", "-std=c++17", "-shared", "-fPIC", "-I",
                           os.path.join(ROOT, "block_sparse_attention_48_b200", "csrc"),
                           os.path.join(ROOT, "tests", "host", "serving_rules.cpp"), "-o", out])
    L, i64 = ctypes.CDLL(out), ctypes.c_int64
    L.fa_host_segment_pages.argtypes, L.fa_host_segment_pages.restype = [i64] * 3, i64
    L.fa_host_teams.argtypes = L.fa_host_once.argtypes = [i64] * 5
    return L


@pytest.mark.parametrize("shape", [
    # B, Hq, Hkv, q_len, D: shapes that the calls refuse
    (1, 8, 1, 1024, 64), (1, 4096, 1, 1, 64), (2, 34, 2, 1, 128), (2, 8, 2, 5, 64), (2, 8, 3, 1, 64), (2, 8, 2, 1, 96),
    (2, 8, 2, 1, 10 ** 6), (65536, 8, 2, 1, 64), (1, 65536, 65536, 1, 64), (1, 1, 1, 2 ** 62, 64),
    (1, 2 ** 62, 1, 4, 64), (2 ** 40, 0, 1, 1, 64), (-1, 8, 2, 1, 64), (1, 8, 2, -1, 64)])
def test_no_workspace_for_refused_shapes(shape):
    lib = fa.library()
    assert lib.fa_decode_paged_workspace_size(*shape) == 0
    for prefix in (0, 128, 2 ** 31 - 256):
        assert lib.fa_decode_shared_workspace_size(*shape, prefix) == 0


def test_workspaces_of_taken_shapes():
    lib = fa.library()
    for B, Hq, Hkv, n, D in ((1, 16, 1, 1, 64), (65535, 4, 4, 1, 128), (3, 12, 4, 5, 64)):
        paged = lib.fa_decode_paged_workspace_size(B, Hq, Hkv, n, D)
        assert paged > 256 and lib.fa_decode_shared_workspace_size(B, Hq, Hkv, n, D, 0) == paged
    # nothing to do: the status word
    for B, Hq, n in ((0, 8, 1), (2, 0, 1), (2, 64, 0)):
        assert lib.fa_decode_paged_workspace_size(B, Hq, 2, n, 64) == 256
        assert lib.fa_decode_shared_workspace_size(B, Hq, 2, n, 64, 2 ** 31 - 256) == 256
    # a prefix's work list of 2^31 entries is refused
    assert lib.fa_decode_shared_workspace_size(65535, 16, 1, 1, 64, 2 ** 31 - 256) == 0


@pytest.mark.parametrize("shared", [False, True])
def test_soft_caps_beyond_fp32_are_refused(shared):
    """The kernels multiply by scale / cap and by cap log2(e): both must be finite, or every
    output would be NaN."""
    lib = fa.library()

    def tensor(dims, data=4096):
        t = fa.TensorDesc()
        t.data = data
        for i in range(4):
            t.dims[i], t.strides[i] = dims[i], math.prod(dims[i + 1:])
        return t
    q, pool = tensor([2, 8, 1, 64]), tensor([5, 2, 128, 64])
    sm = fa.ScoreModDesc()
    sm.kind = fa.SCORE["softcap"]

    def call(cap, scale):
        sm.softcap = cap
        fn = lib.fa_decode_shared if shared else lib.fa_decode_paged
        return fn(q, pool, pool, 4096, 3, 3, 4096, 128 if shared else -1, sm, scale, q, None, 4096, 1 << 30, None)
    for cap, scale in ((math.inf, 0.0), (math.nan, 0.0), (3e38, 0.0), (1e-40, 0.0), (1e-30, 1e10), (-1.0, 0.0)):
        assert call(cap, scale) == fa.FA_ERR_INVALID_ARG


def test_pages_of_a_segment(rules):
    """No segment has more pages than the rule says, and some segment has as many: by the
    pages that the keys of a window touch, at every length."""
    rng = random.Random(5)
    for _ in range(300):
        width, n = rng.randint(0, 40), rng.randint(1, 16)
        window = rng.choice([-1, 0, 1, 126, 127, 128, 129, 500, rng.randint(0, 6000), 2 ** 62])
        most = 0
        for length in range(0, 128 * width + 1):
            first = length - n - window if 0 <= window and length - n > window else 0
            most = max(most, (length + 127) // 128 - first // 128)
        got = rules.fa_host_segment_pages(width, window, n)
        assert got == most, (width, window, n)


def test_teams_that_pay(rules):
    """All teams, or as many for every segment, each with a whole page at least; a window's
    segments count as what they read."""
    rng = random.Random(6)
    for _ in range(3000):
        segments, pages = rng.choice([1, 2, 3, 8, 9, 40, 600]), rng.randint(0, 4000)
        rows, D, most = rng.randint(1, 16), rng.choice([64, 128]), rng.choice([2, 296])
        n = rules.fa_host_teams(segments, pages, rows, D, most)
        assert n == most or (n % segments == 0 and segments <= n < most and n // segments <= pages)
    # one sequence behind a window: as with a table of the pages that it reads
    reads = rules.fa_host_segment_pages(600, 16384, 1)
    assert reads == 129
    for rows in (4, 8, 16):
        n = rules.fa_host_teams(1, reads, rows, 128, 296)
        assert n <= reads // 2 and n < rules.fa_host_teams(1, 600, rows, 128, 296)


def test_where_a_prefix_is_taken_once(rules):
    """By the pages that would be read again: more of them, of any of the sizes, never turn it
    back; both sides of each threshold."""
    def once(B, Hkv, rows, D, pages):
        return bool(rules.fa_host_once(B, Hkv, rows, D, pages))
    for B, Hkv, rows, D, least in ((33, 1, 8, 128, 4096), (33, 1, 8, 64, 6144), (33, 1, 4, 64, 6144), (33, 1, 9, 64, 2048),
                                   (33, 1, 16, 128, 256), (13, 1, 16, 128, 256), (11, 1, 16, 128, 1024),
                                   (3, 8, 16, 128, 1024)):
        pages = -(-least // ((B - 1) * Hkv))
        assert once(B, Hkv, rows, D, pages) and not once(B, Hkv, rows, D, pages - 1), (B, rows, D)
    assert not once(65, 2, 16, 128, 4) and once(65, 2, 16, 128, 5)  # 512 and 640 pages
    assert not once(2, 8, 16, 128, 10 ** 4) and once(2, 8, 16, 64, 10 ** 4)
    assert not any(once(1, 8, r, D, 10 ** 5) or once(9, 8, r, D, 0) for r in (1, 16) for D in (64, 128))
    rng = random.Random(8)
    for _ in range(2000):
        x = [rng.randint(3, 200), rng.randint(1, 16), rng.randint(1, 16), rng.choice([64, 128]), rng.randint(1, 300)]
        if once(*x):
            for i in (0, 1, 4):
                y = list(x)
                y[i] += rng.randint(1, 50)
                assert once(*y)
