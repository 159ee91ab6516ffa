"""The paged decode kernels' walk (csrc/paged_walk.cuh, built for the host) as their CTAs do it:
two teams a CTA, 320 threads that scan the lengths, or 352 beside a shared prefix, and up to
296 teams.  Every page of every (sequence, kv head) segment goes to one team, in order; the
teams that hold a segment's pieces are those its join counts; partial results are distinct."""

import ctypes
import os
import random
import subprocess

import numpy as np
import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
BUILD = os.path.join(ROOT, "tests", "host", "_build")
I32P = ctypes.POINTER(ctypes.c_int32)
TEAMS = 2  # of a CTA


@pytest.fixture(scope="module")
def lib():
    os.makedirs(BUILD, exist_ok=True)
    out = os.path.join(BUILD, "libservingwalk.so")
    subprocess.check_call(["g++", "-O2", "-std=c++17", "-shared", "-fPIC", "-I",
                           os.path.join(ROOT, "block_sparse_attention_48_b200", "csrc"),
                           os.path.join(ROOT, "tests", "host", "paged_walk.cpp"), "-o", out])
    L = ctypes.CDLL(out)
    i32, i64 = ctypes.c_int32, ctypes.c_longlong
    L.fa_host_pd_range.argtypes = [i32, i32, i64, i32, i32, I32P]
    L.fa_host_pd_walk.argtypes = [i32, i32, i32, i32, i64, i32, I32P, i64, ctypes.c_int, ctypes.c_int, ctypes.c_int,
                                  I32P]
    L.fa_host_pd_walk.restype = i64
    L.fa_host_pd_holder.argtypes = [i64, i64, ctypes.c_int]
    return L


@pytest.mark.parametrize("threads", [320, 352])
@pytest.mark.parametrize("seed", range(25))
def test_walk_of_two_teams_a_cta(lib, threads, seed):
    rng = random.Random(1000 * threads + seed)
    sms = 148
    B, Hkv, q_len = rng.choice([1, 2, 9, 40, 319, 321, 353, 800]), rng.randint(1, 4), rng.randint(1, 5)
    width = rng.choice([1, 3, 12, 60])
    window = rng.choice([-1, -1, 100, 500])
    prefix = rng.randint(1, width) if window < 0 and threads == 352 else 0
    ctas = rng.choice([1, sms, rng.randint(1, sms)]) if threads == 352 else min(B * Hkv * width, sms)
    teams = rng.choice([TEAMS * sms, rng.randint(1, TEAMS * sms)])  # the cap that the host sets
    lens = [rng.choice([0, 0, 1, rng.randint(0, 128 * width), 128 * width + 5, -3]) for _ in range(B)]
    entries, spans = [], []
    r = (ctypes.c_int32 * 4)()
    for b, raw in enumerate(lens):
        lib.fa_host_pd_range(q_len, width, window, prefix, raw, r)
        for hk in range(Hkv):
            if r[2]:
                spans.append((len(entries), r[2]))
            entries += [(b, hk, t) for t in range(r[2])]
    T = len(entries)
    used = min(T, TEAMS * ctas, teams)
    # the first teams of all CTAs come before the second ones; every team below `used` exists
    numbered = sorted(block + ctas * t for block in range(ctas) for t in range(TEAMS))
    assert numbered == list(range(TEAMS * ctas)) and used <= len(numbered)
    arr, out = np.array(lens, np.int32), np.zeros(3 * (T + 1), np.int32)
    walked, held = [], []
    for c in range(used):
        n = lib.fa_host_pd_walk(B, Hkv, q_len, width, window, prefix, arr.ctypes.data_as(I32P), T, c, used, threads,
                                out.ctypes.data_as(I32P))
        assert n > 0
        walked += [tuple(x) for x in out[:3 * n].reshape(n, 3).tolist()]
        held += [c] * n
    assert walked == entries
    taken = set()
    for at, n in spans:
        c0, c1 = lib.fa_host_pd_holder(T, at, used), lib.fa_host_pd_holder(T, at + n - 1, used)
        assert sorted(set(held[at:at + n])) == list(range(c0, c1 + 1))
        if c0 != c1:
            parts = {2 * c + (c == c0) for c in range(c0, c1 + 1)}
            assert not parts & taken and max(parts) < 2 * TEAMS * sms
            taken |= parts
