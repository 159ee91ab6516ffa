"""The rotary and paged-cache entry points without a GPU: frequencies, refusals before
any CUDA call, and the paged decode kernel's walk over its work list
(csrc/paged_walk.cuh, built for the host): every page of every (sequence, kv head)
segment goes to exactly one CTA, in order, and the CTAs that hold a segment's pieces are
those that the join counts."""

import ctypes
import math
import os
import random
import subprocess

import numpy as np
import pytest
import torch

import block_sparse_attention_48_b200 as fa

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
BUILD = os.path.join(ROOT, "tests", "host", "_build")
I32P = ctypes.POINTER(ctypes.c_int32)
THREADS = 288  # a CTA: eight compute warps and the producer warp


# ------------------------------------------------------------------ frequencies

def _freq(rotary, base, scaling=None):
    f, amp = fa.rope_frequencies(rotary, base, scaling, device="cpu")
    assert f.dtype == torch.float64 and f.shape == (rotary // 2,)
    return f.tolist(), amp


@pytest.mark.parametrize("rotary", [2, 16, 64, 128])
def test_frequencies_unscaled_linear_and_base(rotary):
    plain = [10000.0 ** (-2 * j / rotary) for j in range(rotary // 2)]
    got, amp = _freq(rotary, 10000.0)
    assert amp == 1.0 and np.allclose(got, plain, rtol=1e-14, atol=0)
    assert np.allclose(_freq(rotary, 10000.0, ("linear", 4.0))[0], np.array(plain) / 4, rtol=1e-14, atol=0)
    if rotary > 2:
        got = _freq(rotary, 10000.0, ("base", 4.0))[0]
        assert got[0] == 1.0 and math.isclose(got[-1], plain[-1] / 4, rel_tol=1e-12)
        assert all(p / 4 <= g * (1 + 1e-12) and g <= p for g, p in zip(got, plain))


def test_frequencies_bands_and_yarn():
    rotary, base, n, lo, hi, s = 128, 500000.0, 8192.0, 1.0, 4.0, 8.0
    plain = [base ** (-2 * j / rotary) for j in range(rotary // 2)]
    got, amp = _freq(rotary, base, ("bands", s, n, lo, hi))
    assert amp == 1.0
    for g, f in zip(got, plain):
        turns = n * f / (2 * math.pi)
        if turns >= hi:
            want = f
        elif turns <= lo:
            want = f / s
        else:
            keep = (turns - lo) / (hi - lo)
            want = f * keep + f / s * (1 - keep)
        assert math.isclose(g, want, rel_tol=1e-12)
    got, amp = _freq(rotary, base, ("yarn", s, n, lo, hi))
    assert math.isclose(amp, 0.1 * math.log(s) + 1, rel_tol=1e-6)

    def index(turns):
        return rotary * math.log(n / (turns * 2 * math.pi)) / (2 * math.log(base))
    a, b = max(0, math.floor(index(hi))), min(rotary - 1, math.ceil(index(lo)))
    for j, (g, f) in enumerate(zip(got, plain)):
        share = min(1.0, max(0.0, (j - a) / (b - a)))
        assert math.isclose(g, f / s * share + f * (1 - share), rel_tol=1e-12)


def test_frequencies_refusals():
    for args in ((0, 1e4, None), (7, 1e4, None), (16, 1.0, None), (16, float("inf"), None),
                 (16, 1e4, ("linear", 0.5)), (16, 1e4, ("linear", float("nan"))), (2, 1e4, ("base", 2.0)),
                 (16, 1e4, ("bands", 2.0, 0.0, 1.0, 4.0)), (16, 1e4, ("bands", 2.0, 8192, 4.0, 4.0)),
                 (16, 1e4, ("yarn", 2.0, 8192, 0.0, 4.0)), (-4, 1e4, None)):
        with pytest.raises(fa.FlexAttnError):
            fa.rope_frequencies(*args, device="cpu")
    for scaling in (("dynamic", 2.0), ("linear", 1.0, 2.0), ("yarn", 2.0)):
        with pytest.raises(ValueError):
            fa.rope_frequencies(16, 1e4, scaling, device="cpu")
    bad = fa.RopeScalingDesc(9, 2.0, 1.0, 1.0, 2.0)
    assert fa.library().fa_rope_frequencies(16, 1e4, bad, (ctypes.c_double * 8)(), None) == fa.FA_ERR_INVALID_ARG
    assert fa.library().fa_rope_frequencies(16, 1e4, None, None, None) == fa.FA_ERR_INVALID_ARG


# ------------------------------------------------------------------ refusals of the C ABI

def _tensor(dims, data=4096):
    t = fa.TensorDesc()
    t.data = data
    st = [dims[1] * dims[2] * dims[3], dims[2] * dims[3], dims[3], 1]
    for i in range(4):
        t.dims[i], t.strides[i] = dims[i], st[i]
    return t


def _rope(rotary=64, data=4096, amplitude=1.0):
    return fa.RopeDesc(data, rotary, 0, amplitude)


def test_rope_apply_refusals():
    q, k = _tensor([2, 4, 8, 64]), _tensor([2, 2, 8, 64])

    def call(q=q, k=k, rope=_rope(), qo=q, ko=k, stride=0, offset=0):
        return fa.library().fa_rope_apply(q, k, rope, None, stride, offset, 0, qo, ko, None)
    INVALID, UNSUPPORTED = fa.FA_ERR_INVALID_ARG, fa.FA_ERR_UNSUPPORTED
    assert call(rope=None) == INVALID
    assert call(q=None, qo=None, k=None, ko=None) == INVALID
    assert call(qo=None) == INVALID and call(ko=None) == INVALID
    assert call(rope=_rope(80)) == INVALID and call(rope=_rope(-16)) == INVALID
    assert call(rope=_rope(24)) == UNSUPPORTED
    assert call(rope=_rope(data=0)) == INVALID
    for amp in (-1.0, float("nan"), float("inf")):
        assert call(rope=_rope(amplitude=amp)) == INVALID
    assert call(ko=_tensor([2, 2, 9, 64])) == INVALID
    k9 = _tensor([2, 2, 9, 64])
    assert call(k=k9, ko=k9) == INVALID
    k3 = _tensor([3, 2, 8, 64])
    assert call(k=k3, ko=k3) == INVALID
    q32 = _tensor([2, 4, 8, 32])
    assert call(q=q32, qo=q32, k=None, ko=None, rope=_rope(32)) == UNSUPPORTED
    assert call(stride=-1) == INVALID and call(offset=2 ** 40) == INVALID
    odd = _tensor([2, 4, 8, 64], data=4098)
    assert call(q=odd) == INVALID and call(qo=odd) == INVALID
    flat = _tensor([2, 4, 8, 64])
    flat.strides[1] = 0
    assert call(q=flat) == INVALID
    big = _tensor([65536, 1, 1, 64])
    assert call(q=big, qo=big, k=None, ko=None) == INVALID
    none = _tensor([2, 4, 0, 64])
    assert call(q=none, qo=none, k=None, ko=None) == fa.FA_OK


def test_paged_append_refusals():
    k, pool = _tensor([2, 2, 8, 64]), _tensor([5, 2, 128, 64])
    q = _tensor([2, 4, 8, 64])

    def call(k=k, v=None, q=q, rope=_rope(), lens=4096, table=4096, stride=3, width=3, kp=pool, vp=None, qo=q, ws=4096,
             size=256):
        return fa.library().fa_paged_append(k, v or k, q, rope, lens, None, table, stride, width, kp, vp or kp, qo, ws,
                                            size, None)
    INVALID, UNSUPPORTED = fa.FA_ERR_INVALID_ARG, fa.FA_ERR_UNSUPPORTED
    assert call(v=_tensor([2, 2, 9, 64])) == INVALID
    assert call(vp=_tensor([6, 2, 128, 64])) == INVALID
    assert call(kp=_tensor([5, 3, 128, 64])) == INVALID
    assert call(kp=_tensor([5, 2, 64, 64])) == INVALID
    assert call(qo=None) == INVALID and call(q=None) == INVALID
    assert call(q=_tensor([2, 4, 9, 64])) == INVALID
    assert call(rope=_rope(40)) == UNSUPPORTED and call(rope=_rope(128)) == INVALID
    assert call(lens=0) == INVALID and call(table=0) == INVALID
    assert call(stride=2) == INVALID and call(width=-1) == INVALID
    assert call(ws=0) == INVALID and call(size=8) == INVALID and call(ws=4100) == INVALID
    none = _tensor([2, 2, 0, 64])
    assert call(k=none, q=None, qo=None) == fa.FA_OK


@pytest.mark.parametrize("shared", [False, True])
def test_decode_paged_refusals(shared):
    lib = fa.library()
    q, pool = _tensor([2, 8, 1, 64]), _tensor([5, 2, 128, 64])

    def call(q=q, kp=pool, vp=None, o=None, table=4096, stride=3, width=3, lens=4096, sm=None, ws=4096, size=1 << 30,
             prefix=128):
        fn = lib.fa_decode_shared if shared else lib.fa_decode_paged
        return fn(q, kp, vp or kp, table, stride, width, lens, prefix if shared else -1, sm, 0.0, o or q, None, ws,
                  size, None)
    INVALID, UNSUPPORTED = fa.FA_ERR_INVALID_ARG, fa.FA_ERR_UNSUPPORTED
    assert call(o=_tensor([2, 8, 2, 64])) == INVALID
    assert call(vp=_tensor([4, 2, 128, 64])) == INVALID
    assert call(q=_tensor([2, 7, 1, 64])) == INVALID
    assert call(kp=_tensor([5, 2, 128, 128])) == INVALID
    assert call(kp=_tensor([5, 2, 256, 64])) == INVALID
    assert call(q=_tensor([2, 34, 1, 64])) == UNSUPPORTED and call(q=_tensor([2, 8, 5, 64])) == UNSUPPORTED
    assert call(q=_tensor([2, 8, 1, 96]), kp=_tensor([5, 2, 128, 96])) == UNSUPPORTED
    assert call(table=0) == INVALID and call(lens=0) == INVALID
    assert call(stride=2) == INVALID and call(width=-1) == INVALID and call(width=1 << 25) == INVALID
    assert call(ws=0) == INVALID and call(ws=4104) == INVALID
    sm = fa.ScoreModDesc()
    for kind, rc in (("bias", UNSUPPORTED), ("bias_softcap", UNSUPPORTED), ("alibi", INVALID), ("softcap", INVALID)):
        sm.kind = fa.SCORE[kind]
        assert call(sm=sm) == rc, kind
    sm.kind = 17
    assert call(sm=sm) == INVALID
    none = _tensor([0, 8, 1, 64])
    assert call(q=none) == fa.FA_OK
    if shared:
        for prefix in (-128, 1, 127, 512):
            assert call(prefix=prefix) == INVALID


# ------------------------------------------------------------------ the walk

@pytest.fixture(scope="module")
def lib():
    os.makedirs(BUILD, exist_ok=True)
    out = os.path.join(BUILD, "libpagedwalk.so")
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
    L.fa_host_pd_page.argtypes = [ctypes.c_int, ctypes.c_int, I32P]
    L.fa_host_sp_geom.argtypes = [i64, i32, I32P]
    L.fa_host_sp_pieces.argtypes = [i64, i32, i32, ctypes.c_int, ctypes.c_int, I32P]
    return L


def _range(lib, q_len, width, window, prefix, length):
    out = (ctypes.c_int32 * 4)()
    bad = lib.fa_host_pd_range(q_len, width, window, prefix, length, out)
    return tuple(out), bool(bad)


def test_ranges(lib):
    rng = random.Random(1)
    for _ in range(4000):
        q_len, width = rng.randint(1, 16), rng.choice([0, 1, 2, 9, 400, 16777214])
        window = rng.choice([-1, -1, 0, 1, 127, 128, 129, rng.randint(0, 60000), 2 ** 31 - 256])
        prefix = rng.randint(0, min(width, 20)) if window < 0 else 0
        raw = rng.choice([-2 ** 31, -1, 0, 1, 127, 128, 129, width * 128 if width < 1 << 24 else 5, 2 ** 31 - 1,
                          rng.randint(0, 60000)])
        (length, lo, n, shared), bad = _range(lib, q_len, width, window, prefix, raw)
        assert bad == (raw < 0 or raw > 128 * width)
        assert length == min(max(raw, 0), 128 * width)
        assert 0 <= lo and lo + n == (length + 127) // 128 and n >= 0
        if length:
            assert n > 0
            first = length - q_len  # the first row's position
            if shared:
                assert lo == prefix > 0 and first >= 128 * prefix
            elif window >= 0:
                # every attended key's page is in the range, and its first page holds one
                assert 128 * lo <= max(0, first - window)
                assert lo == 0 or 128 * (lo + 1) > first - window
            else:
                assert lo == 0 and (prefix == 0 or first < 128 * prefix)


@pytest.mark.parametrize("seed", range(60))
def test_walk_covers_every_page_once(lib, seed):
    rng = random.Random(seed)
    B, Hkv, q_len = rng.choice([1, 2, 7, 40, 288, 300, 700]), rng.randint(1, 4), rng.randint(1, 5)
    width = rng.choice([1, 3, 12])
    window = rng.choice([-1, -1, 100, 500])
    prefix = rng.randint(0, width) if window < 0 else 0
    lens = [rng.choice([0, 0, 1, rng.randint(0, 128 * width), 128 * width + 5, -3]) for _ in range(B)]
    entries, spans = [], []
    for b, raw in enumerate(lens):
        n = _range(lib, q_len, width, window, prefix, raw)[0][2]
        for hk in range(Hkv):
            if n:
                spans.append((len(entries), n))
            entries += [(b, hk, t) for t in range(n)]
    T = len(entries)
    grid = min(148, B * Hkv * width)
    used = min(T, grid)
    arr = np.array(lens, np.int32)
    walked, held = [], []
    out = np.zeros(3 * (T + 1), np.int32)
    for c in range(used):
        n = lib.fa_host_pd_walk(B, Hkv, q_len, width, window, prefix, arr.ctypes.data_as(I32P), T, c, used, THREADS,
                                out.ctypes.data_as(I32P))
        assert n > 0
        walked += [tuple(int(x) for x in out[3 * i:3 * i + 3]) for i in range(n)]
        held += [c] * n
    assert walked == entries
    # a split segment's pieces: its first is the last piece of CTA c0's share, the others
    # the first of theirs, so the partial results 2 c0 + 1 and 2 c are distinct
    taken = set()
    for at, n in spans:
        c0, c1 = lib.fa_host_pd_holder(T, at, used), lib.fa_host_pd_holder(T, at + n - 1, used)
        assert held[at] == c0 and held[at + n - 1] == c1
        assert sorted(set(held[at:at + n])) == list(range(c0, c1 + 1))
        if c0 != c1:
            parts = {2 * c + (c == c0) for c in range(c0, c1 + 1)}
            assert not parts & taken and max(parts) < 2 * grid
            taken |= parts


def test_pages_are_clamped(lib):
    bad = ctypes.c_int32()
    for page, num, want in ((0, 1, 0), (4, 5, 4), (5, 5, 4), (-1, 5, 0), (2 ** 31 - 1, 7, 6), (-2 ** 31, 7, 0)):
        assert lib.fa_host_pd_page(page, num, ctypes.byref(bad)) == want
        assert bad.value == (page < 0 or page >= num)


@pytest.mark.parametrize("R", [1, 16, 127, 128, 129, 255, 256, 257, 384, 385, 512, 2048, 2100])
@pytest.mark.parametrize("pages", [1, 2, 3, 8, 41])
@pytest.mark.parametrize("Hkv", [1, 3])
def test_shared_prefix_work_list(lib, R, pages, Hkv):
    """Every tile of rows meets every page of the prefix once, in order, and the partial
    results of a column are those of the CTAs from the holder of its first entry to the
    holder of its last."""
    geom = np.zeros(3, np.int32)
    lib.fa_host_sp_geom(R, pages, geom.ctypes.data_as(I32P))
    pairs, single, per_head = geom.tolist()
    tiles = (R + 127) // 128
    assert 2 * pairs + single in (tiles, tiles + 1) and 256 * pairs + 128 * single >= R
    T = Hkv * per_head
    for used in {1, min(T, 7), min(T, 148)}:
        seen, slots, holders = {}, set(), {}
        out = np.zeros(7 * (T + 1), np.int32)
        for c in range(used):
            n = lib.fa_host_sp_pieces(R, pages, Hkv, c, used, out.ctypes.data_as(I32P))
            assert n > 0
            for hk, col, e0, m, one, t0, t1 in out[:7 * n].reshape(n, 7).tolist():
                assert m > 0
                for s in (0, 1):
                    slot = 2 * (hk * (pairs + single) + col + c) + s
                    assert slot not in slots and slot < 2 * (Hkv * (pairs + single) + used)
                    slots.add(slot)
                holders.setdefault((hk, col), []).append(c)
                for s, t in ((0, t0), (1, t1)):
                    for e in range(e0, e0 + t):
                        tile, page = (2 * col, 2 * e + s) if one else (2 * col + s, e)
                        seen.setdefault((hk, tile), []).append(page)
        for hk in range(Hkv):
            for tile in range(tiles):
                # a column of one tile alternates between its streams within a piece
                got = seen[(hk, tile)]
                assert sorted(got) == list(range(pages))
                if tile < 2 * pairs:
                    assert got == sorted(got)
            for col in range(pairs + single):
                start = hk * per_head + col * pages
                n = pages if col < pairs else (pages + 1) // 2
                c0 = lib.fa_host_pd_holder(T, start, used)
                c1 = lib.fa_host_pd_holder(T, start + n - 1, used)
                assert holders[(hk, col)] == list(range(c0, c1 + 1))


@pytest.mark.parametrize("cost", [16, 32])
def test_split_of_the_sms(lib, cost):
    """Both lists get an SM whatever their sizes; whatever an entry costs."""
    for entries in (1, 5, 576, 10 ** 6):
        for columns in (1, 4, 48, 300):
            for pages, segments in ((0, 0), (1, 1), (1024, 1024), (10 ** 6, 10)):
                for sms in (2, 7, 148):
                    n = lib.fa_host_sp_split(entries, columns, pages, segments, sms, cost)
                    assert 1 <= n <= sms - 1 and n <= max(entries, 1)


def test_workspace_sizes():
    lib = fa.library()
    assert lib.fa_decode_paged_workspace_size(0, 8, 2, 1, 64) == 256
    assert lib.fa_decode_paged_workspace_size(2, 8, 0, 1, 64) == 0
    assert lib.fa_decode_shared_workspace_size(2, 8, 2, 1, 64, -1) == 0
    assert lib.fa_decode_shared_workspace_size(2, 8, 2, 1, 64, 256) >= lib.fa_decode_paged_workspace_size(2, 8, 2, 1, 64)
