"""Decoding against a paged cache (fa_decode_paged) and behind a shared prefix
(fa_decode_shared) against their 64-bit form."""

import pytest
import torch

from paged_reference import PAGE, assert_decode, decode_ref, paged_case

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda", 0)


def _fa():
    import block_sparse_attention_48_b200 as fa
    return fa


def _score(kind, Hq):
    if kind == "alibi":
        return ("alibi", torch.tensor([2.0 ** (-8 * (h + 1) / Hq) for h in range(Hq)], dtype=torch.float32))
    return ("softcap", 5.0) if kind == "softcap" else None


def _gpu(score):
    return (score[0], score[1].cuda()) if score is not None and score[0] == "alibi" else score


CASES = [
    # lens, q_len, Hq, Hkv, D, window, score
    ([1], 1, 1, 1, 64, None, None),
    ([128], 1, 4, 4, 128, None, None),
    ([129, 0, 1, 127], 1, 8, 2, 64, None, "alibi"),
    ([0, 0, 300, 0], 1, 8, 8, 128, None, None),
    ([0, 0], 2, 4, 2, 64, None, None),
    ([2, 700, 3, 1], 5, 3, 1, 64, None, "softcap"),
    ([640, 513, 2000], 4, 16, 4, 128, None, None),
    ([640, 513, 2000], 4, 16, 4, 128, 0, None),
    ([640, 127, 2000, 5], 4, 8, 4, 64, 1, "alibi"),
    ([1500, 257, 64, 900], 2, 16, 2, 128, 300, "softcap"),
    ([3000, 20], 3, 4, 2, 64, 128, None),
    ([5000], 1, 16, 1, 128, None, "alibi"),
    ([37 * i + 1 for i in range(33)], 1, 4, 2, 64, None, None),
    ([11 * (i % 7) for i in range(300)], 1, 2, 1, 64, 50, None),
]


@pytest.mark.parametrize("filler", [0.0, float("inf"), float("nan")])
@pytest.mark.parametrize("case", CASES, ids=lambda c: "-".join(str(x) for x in c)[:60])
def test_decode_paged_matches_the_formula(case, filler):
    fa = _fa()
    lens, n, Hq, Hkv, D, window, kind = case
    q, k, v, table, sl = paged_case(lens, n, Hq, Hkv, D, seed=len(lens) + D, filler=filler)
    score = _score(kind, Hq)
    got = fa.flex_decode_paged(q.cuda(), k.cuda(), v.cuda(), table.cuda(), sl.cuda(), window=window,
                               score_mod=_gpu(score))
    torch.cuda.synchronize()
    assert fa.device_status(ws=fa.paged_workspace(DEV)) == 0
    assert_decode(got, decode_ref(q, k, v, table, lens, window, score))


def test_decode_paged_infinite_values_stay_with_their_rows():
    """Drafted tokens: an infinite or NaN value that only later query tokens attend does
    not reach the earlier ones."""
    fa = _fa()
    lens, n, Hq, Hkv, D = [200, 40], 3, 4, 2, 64
    q, k, v, table, sl = paged_case(lens, n, Hq, Hkv, D, seed=5)
    clean = fa.flex_decode_paged(q.cuda(), k.cuda(), v.cuda(), table.cuda(), sl.cuda())[0]
    last = int(table[0, 1])
    v[last, :, 199 - 128, 3], k[last, :, 199 - 128, 5] = float("nan"), float("inf")
    v[last, :, 198 - 128, 7] = float("inf")
    o, lse = fa.flex_decode_paged(q.cuda(), k.cuda(), v.cuda(), table.cuda(), sl.cuda())
    assert torch.equal(o[0, :, 0], clean[0, :, 0]) and torch.equal(o[1], clean[1])
    keep = [d for d in range(D) if d != 7]
    assert torch.equal(o[0, :, 1][:, keep], clean[0, :, 1][:, keep])
    assert bool(torch.isinf(o[0, :, 1, 7]).all()) and not bool(torch.isfinite(o[0, :, 2, 3]).any())


def test_decode_paged_views_scale_and_outputs():
    """Token-major queries, outputs and pools, a table wider than needed with rows apart,
    an explicit scale, outputs given; the workspace serves other shapes in turn; the same
    call gives the same bits."""
    fa = _fa()
    lens, n, Hq, Hkv, D = [300, 1000, 17], 2, 8, 4, 128
    q, k, v, table, sl = paged_case(lens, n, Hq, Hkv, D, seed=9, width=11)
    ref = decode_ref(q, k, v, table, lens, scale=0.03)
    qt = q.transpose(1, 2).contiguous().cuda().transpose(1, 2)
    pool = torch.stack([k.transpose(1, 2), v.transpose(1, 2)], dim=3).contiguous().cuda()  # [p, 128, H, 2, D]
    kp, vp = pool[:, :, :, 0].transpose(1, 2), pool[:, :, :, 1].transpose(1, 2)
    wide = torch.full((3, 20), -9, dtype=torch.int32, device="cuda")
    wide[:, :11] = table.cuda()
    out = torch.full((3, n, Hq, D), 5.0, dtype=torch.bfloat16, device="cuda").transpose(1, 2)
    lse = torch.zeros((3, Hq, n), device="cuda")
    ws = torch.zeros(1 << 22, dtype=torch.uint8, device="cuda")
    for _ in range(3):
        got = fa.flex_decode_paged(qt, kp, vp, wide[:, :11], sl.cuda(), scale=0.03, out=out, lse=lse, ws=ws)
        assert got[0] is out and got[1] is lse
        assert_decode(got, ref)
        bits = out.clone()
        other = paged_case([4000, 9], 1, 2, 2, 64, seed=3)
        assert_decode(fa.flex_decode_paged(*[t.cuda() for t in other], ws=ws), decode_ref(*other))
        fa.flex_decode_paged(qt, kp, vp, wide[:, :11], sl.cuda(), scale=0.03, out=out, lse=lse, ws=ws)
        assert torch.equal(bits, out)
    assert fa.device_status(ws=ws) == 0


def test_decode_paged_far_pages():
    """Pages whose elements lie past 2^31 from the pool's start."""
    fa = _fa()
    lens, n, Hq, Hkv, D = [260, 100], 1, 8, 8, 128
    q, k, v, table, sl = paged_case(lens, n, Hq, Hkv, D, seed=13)
    num = 2 ** 31 // (Hkv * PAGE * D) + 40
    kp = torch.empty((num, Hkv, PAGE, D), dtype=torch.bfloat16, device="cuda")
    vp = torch.empty((num, Hkv, PAGE, D), dtype=torch.bfloat16, device="cuda")
    far = num - k.shape[0]
    kp[far:], vp[far:] = k.cuda(), v.cuda()
    got = fa.flex_decode_paged(q.cuda(), kp, vp, (table + far).cuda(), sl.cuda())
    assert_decode(got, decode_ref(q, k, v, table, lens))
    # and appended to
    x = torch.ones((2, Hkv, 1, D), dtype=torch.bfloat16, device="cuda")
    fa.paged_append(x, 2 * x, kp, vp, (table + far).cuda(), (sl - 1).cuda())
    p0 = int(table[0, 2]) + far
    assert bool((kp[p0, :, 3] == 1).all()) and bool((vp[p0, :, 3] == 2).all())
    assert torch.equal(kp[p0, :, 2].cpu(), k[p0 - far, :, 2])
    assert fa.device_status(ws=fa.paged_workspace(DEV)) == 0


@pytest.mark.parametrize("shape", [(8, 8, 128, 1), (8, 8, 64, 2), (32, 8, 128, 4)])
@pytest.mark.parametrize("shared", [False, True])
def test_decode_with_many_pages_a_cta(shape, shared):
    """Shares of 20 and more pages a CTA that run over several segments, and an odd number
    of shared pages: the rings of tiles go round many times; calls one after another give
    the same bits."""
    fa = _fa()
    Hq, Hkv, D, n = shape
    prefix = 301 * PAGE if shared else 0
    lens = [prefix + 11000, prefix + 300] if shared else [47003, 2, 5100]
    q, k, v, table, sl = paged_case(lens, n, Hq, Hkv, D, seed=77, prefix=prefix, filler=float("nan"))
    args = [t.cuda() for t in (q, k, v, table, sl)]
    call = (lambda: fa.flex_decode_shared(*args, prefix)) if shared else (lambda: fa.flex_decode_paged(*args))
    got = call()
    assert_decode(got, decode_ref(q, k, v, table, lens))
    for _ in range(20):
        again = call()
        assert torch.equal(again[0], got[0]) and torch.equal(again[1], got[1])
    assert fa.device_status(ws=fa.paged_workspace(DEV)) == 0


@pytest.mark.parametrize("shape", [(8, 8, 128, 1, None, None), (8, 8, 64, 2, None, "softcap"),
                                   (32, 8, 128, 4, 30000, "alibi")])
def test_decode_of_long_lists_on_streams(shape):
    """A dozen pages and more a team: calls one after another, on one workspace and on two
    streams at once, give the same bits."""
    fa = _fa()
    Hq, Hkv, D, n, window, kind = shape
    lens = [47003, 2, 13000, 0, 130, 36000]
    q, k, v, table, sl = paged_case(lens, n, Hq, Hkv, D, seed=78, filler=float("nan"))
    score = _score(kind, Hq)
    args = [t.cuda() for t in (q, k, v, table, sl)]
    kw = dict(window=window, score_mod=_gpu(score))
    got = fa.flex_decode_paged(*args, **kw)
    assert_decode(got, decode_ref(q, k, v, table, lens, window, score))
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    outs = []
    for i in range(40):
        outs.append(fa.flex_decode_paged(*args, **kw) if i % 4 == 0 else
                    fa.flex_decode_paged(*args, stream=streams[i % 2], **kw))
    torch.cuda.synchronize()
    for o, lse in outs:
        assert torch.equal(o, got[0]) and torch.equal(lse, got[1])
    assert fa.device_status(ws=fa.paged_workspace(DEV)) == 0


@pytest.mark.parametrize("shared", [False, True])
@pytest.mark.parametrize("what", ["page", "negative page", "length", "negative length"])
def test_decode_paged_reports_bad_tables_and_lengths(what, shared):
    """Bad entries are clamped (no read outside the pools) and reported; the other
    sequences' rows are right."""
    fa = _fa()
    lens, n, Hq, Hkv, D = [600, 500, 450], 1, 8, 4, 64
    q, k, v, table, sl = paged_case(lens, n, Hq, Hkv, D, seed=21, prefix=256)
    ref = decode_ref(q, k, v, table, lens)
    tab, ln = table.clone(), sl.clone()
    if what == "page":
        tab[1, 3] = k.shape[0]
    elif what == "negative page":
        tab[1, 3] = -1
    elif what == "length":
        ln[1] = 2 ** 31 - 1
    else:
        ln[1] = -7
    ws = torch.zeros(1 << 23, dtype=torch.uint8, device="cuda")
    call = (lambda *a, **kw: fa.flex_decode_shared(*a, 256, **kw)) if shared else fa.flex_decode_paged
    o, lse = call(q.cuda(), k.cuda(), v.cuda(), tab.cuda(), ln.cuda(), ws=ws)
    torch.cuda.synchronize()
    assert fa.device_status(ws=ws) == fa.FA_ERR_BAD_BLOCKMASK
    assert fa.device_status(ws=ws) == 0
    keep = [0, 2]
    assert_decode((o[keep], lse[keep]), tuple(t[keep] for t in ref))
    if what == "negative length":
        assert not bool(o[1].any()) and bool(torch.isneginf(lse[1]).all())


def test_decode_paged_without_pages():
    fa = _fa()
    q = torch.ones((2, 4, 1, 64), dtype=torch.bfloat16, device="cuda")
    pool = torch.zeros((0, 2, PAGE, 64), dtype=torch.bfloat16, device="cuda")
    table = torch.zeros((2, 0), dtype=torch.int32, device="cuda")
    lens = torch.zeros(2, dtype=torch.int32, device="cuda")
    for o, lse in (fa.flex_decode_paged(q, pool, pool, table, lens),
                   fa.flex_decode_shared(q, pool, pool, table, lens, 0)):
        assert not bool(o.any()) and bool(torch.isneginf(lse).all())


# ------------------------------------------------------------------ shared prefix

SHARED = [
    # own lengths behind the prefix, prefix, q_len, Hq, Hkv, D, score
    ([1], 128, 1, 1, 1, 64, None),
    ([5, 130, 1], 256, 1, 8, 2, 128, None),
    ([40, 2, 3, 700], 1024, 2, 16, 4, 64, "alibi"),
    ([3, 128, 129], 640, 3, 8, 8, 128, "softcap"),
    ([17 + i for i in range(20)], 384, 1, 32, 4, 128, None),
    ([9 + i % 5 for i in range(40)], 512, 4, 8, 2, 64, "alibi"),
    ([1 + 3 * i for i in range(70)], 256, 4, 8, 2, 128, "softcap"),
    ([10, 20], 0, 1, 4, 4, 64, None),
    ([2 + i % 3 for i in range(129)], 128, 2, 2, 1, 64, None),
    ([2], 5120, 1, 16, 1, 128, None),
]


@pytest.mark.parametrize("case", SHARED, ids=lambda c: "-".join(str(x) for x in c)[-60:])
def test_decode_shared_matches_the_formula(case):
    fa = _fa()
    own, prefix, n, Hq, Hkv, D, kind = case
    lens = [prefix + x for x in own]
    q, k, v, table, sl = paged_case(lens, n, Hq, Hkv, D, seed=len(own) + D, prefix=prefix, filler=float("nan"))
    score = _score(kind, Hq)
    got = fa.flex_decode_shared(q.cuda(), k.cuda(), v.cuda(), table.cuda(), sl.cuda(), prefix, score_mod=_gpu(score))
    torch.cuda.synchronize()
    assert fa.device_status(ws=fa.paged_workspace(DEV)) == 0
    assert_decode(got, decode_ref(q, k, v, table, lens, None, score))
    bits = fa.flex_decode_shared(q.cuda(), k.cuda(), v.cuda(), table.cuda(), sl.cuda(), prefix, score_mod=_gpu(score))
    assert torch.equal(bits[0], got[0]) and torch.equal(bits[1], got[1])


@pytest.mark.parametrize("case", [
    # lens, q_len, Hq, Hkv, D, score: few segments of many pages, whose pieces one team joins
    ([21000], 1, 1, 1, 64, None),
    ([30011], 1, 16, 1, 128, "softcap"),
    ([12345, 9000], 2, 8, 1, 128, None),
    ([25000, 1, 0, 3100], 5, 6, 2, 64, "alibi"),
    ([16500, 12], 3, 5, 1, 128, None),
], ids=lambda c: "-".join(str(x) for x in c)[:60])
def test_decode_of_few_long_sequences(case):
    """Every row's pieces of a long sequence, joined by one team, with a table of just the
    pages and one that is much wider; the same bits every time."""
    fa = _fa()
    lens, n, Hq, Hkv, D, kind = case
    score, pages = _score(kind, Hq), (max(lens) + PAGE - 1) // PAGE
    for width in (None, 4 * pages):
        q, k, v, table, sl = paged_case(lens, n, Hq, Hkv, D, seed=len(lens) + D, width=width, filler=float("nan"))
        args = [t.cuda() for t in (q, k, v, table, sl)]
        got = fa.flex_decode_paged(*args, score_mod=_gpu(score))
        assert_decode(got, decode_ref(q, k, v, table, lens, None, score))
        for _ in range(5):
            again = fa.flex_decode_paged(*args, score_mod=_gpu(score))
            assert torch.equal(again[0], got[0]) and torch.equal(again[1], got[1])
    assert fa.device_status(ws=fa.paged_workspace(DEV)) == 0


def test_decode_shared_with_short_sequences():
    """Sequences that end inside the prefix, or whose first query tokens lie in it, are
    taken from their own rows (which may name other pages); empty ones give zeros."""
    fa = _fa()
    prefix, n, Hq, Hkv, D = 512, 3, 8, 2, 64
    lens = [700, 512, 100, 0, 514, 515, 2, 1000]
    q, k, v, table, sl = paged_case(lens, n, Hq, Hkv, D, seed=3, prefix=prefix, filler=float("nan"))
    table[2, 0] = int(table[0, 4])  # a short sequence with a page of its own
    ref = decode_ref(q, k, v, table, lens, None, ("softcap", 5.0))
    got = fa.flex_decode_shared(q.cuda(), k.cuda(), v.cuda(), table.cuda(), sl.cuda(), prefix,
                                score_mod=("softcap", 5.0))
    torch.cuda.synchronize()
    assert fa.device_status(ws=fa.paged_workspace(DEV)) == 0
    assert_decode(got, ref)


def test_decode_shared_reads_the_prefix_from_row_zero():
    """Every long sequence's prefix is that of row 0 of the table."""
    fa = _fa()
    lens = [300, 400]
    q, k, v, table, sl = paged_case(lens, 1, 4, 2, 64, seed=8, prefix=256)
    ref = decode_ref(q, k, v, table, lens)
    tab = table.clone()
    tab[1, :2] = 0
    assert_decode(fa.flex_decode_shared(q.cuda(), k.cuda(), v.cuda(), tab.cuda(), sl.cuda(), 256), ref)


def test_decode_shared_large_scores():
    """Scores that grow along the prefix by far more than one rescaling step, at an
    explicit scale."""
    fa = _fa()
    lens, prefix, D = [1100 + i for i in range(9)], 1024, 64
    q, k, v, table, sl = paged_case(lens, 1, 8, 2, D, seed=15, prefix=prefix)
    q[:] = 1.0
    g = torch.Generator().manual_seed(4)
    for t in range(8):
        k[int(table[0, t])] = (0.25 * t + 0.001 * torch.randn((2, PAGE, D), generator=g)).to(torch.bfloat16)
    k[int(table[0, 5]), :, 64:] = -3.0
    got = fa.flex_decode_shared(q.cuda(), k.cuda(), v.cuda(), table.cuda(), sl.cuda(), prefix, scale=1.0)
    assert_decode(got, decode_ref(q, k, v, table, lens, scale=1.0))


# Prefixes that are taken once (the sizes above are taken page by page): one tile of rows,
# pairs of tiles with a full and a partial second one and with a single one behind them,
# odd numbers of pages, fewer columns than CTAs and more.
ONCE = [
    # batch, own lengths (cycled), prefix pages, q_len, Hq, Hkv, D, score
    (49, (1, 130, 7), 17, 1, 8, 8, 128, None),
    (40, (4, 300, 129), 79, 4, 8, 2, 64, "alibi"),
    (70, (9, 128, 40, 5), 45, 4, 8, 2, 128, "softcap"),
    (129, (2, 3, 200), 48, 2, 4, 1, 64, None),
    (17, (60, 1), 385, 1, 16, 1, 128, "alibi"),
    (2, (1, 2), 768, 1, 8, 8, 64, None),
    (200, (1, 50), 4, 1, 8, 8, 64, "softcap"),
    (4, (11000, 300, 7), 301, 4, 32, 8, 128, None),
    (700, (1, 2, 140), 3, 1, 8, 8, 64, None),
]


def _once(own, B, pages):
    return [PAGE * pages + own[i % len(own)] for i in range(B)]


def _assert_taken_once(fa, q, k, prefix):
    lib, B, Hkv = fa.library(), q.shape[0], k.shape[1]
    assert lib.fa_decode_shared_workspace_size(B, q.shape[1], Hkv, q.shape[2], q.shape[3], prefix) > \
        lib.fa_decode_paged_workspace_size(B, q.shape[1], Hkv, q.shape[2], q.shape[3])


@pytest.mark.parametrize("case", ONCE, ids=lambda c: f"b{c[0]}-p{c[2]}-n{c[3]}-h{c[4]}-{c[5]}-d{c[6]}-{c[7]}")
def test_decode_shared_prefix_taken_once(case):
    fa = _fa()
    B, own, pages, n, Hq, Hkv, D, kind = case
    lens, prefix = _once(own, B, pages), PAGE * pages
    q, k, v, table, sl = paged_case(lens, n, Hq, Hkv, D, seed=B + D, prefix=prefix, filler=float("nan"))
    _assert_taken_once(fa, q, k, prefix)
    score = _score(kind, Hq)
    args = [t.cuda() for t in (q, k, v, table, sl)]
    tab = args[3].clone()
    tab[1:, :pages] = 0  # the shared entries are those of row 0
    got = fa.flex_decode_shared(*args[:3], tab, args[4], prefix, score_mod=_gpu(score))
    assert_decode(got, decode_ref(q, k, v, table, lens, None, score))
    for _ in range(10):
        again = fa.flex_decode_shared(*args, prefix, score_mod=_gpu(score))
        assert torch.equal(again[0], got[0]) and torch.equal(again[1], got[1])
    assert fa.device_status(ws=fa.paged_workspace(DEV)) == 0


def test_decode_shared_once_with_short_sequences():
    """Sequences that end in the prefix (with pages of their own), reach only just past it,
    or are empty, among those that share it."""
    fa = _fa()
    B, pages, n, Hq, Hkv, D = 200, 4, 3, 16, 8, 64
    prefix = PAGE * pages
    lens = [(700, 512, 100, 0, 514, 515, 2, 1000)[i % 8] for i in range(B)]
    q, k, v, table, sl = paged_case(lens, n, Hq, Hkv, D, seed=3, prefix=prefix, filler=float("nan"))
    _assert_taken_once(fa, q, k, prefix)
    table[2, 0] = int(table[0, 4])
    got = fa.flex_decode_shared(q.cuda(), k.cuda(), v.cuda(), table.cuda(), sl.cuda(), prefix,
                                score_mod=("softcap", 5.0))
    assert_decode(got, decode_ref(q, k, v, table, lens, None, ("softcap", 5.0)))
    none = torch.zeros_like(sl)
    o, lse = fa.flex_decode_shared(q.cuda(), k.cuda(), v.cuda(), table.cuda(), none.cuda(), prefix)
    assert not bool(o.any()) and bool(torch.isneginf(lse).all())
    assert fa.device_status(ws=fa.paged_workspace(DEV)) == 0


@pytest.mark.parametrize("D", [64, 128])
def test_decode_shared_once_large_and_infinite_scores(D):
    """Scores that grow along the prefix by many rescaling steps; then keys of the prefix
    that are minus infinity for every row, and an infinite value."""
    fa = _fa()
    B, pages, Hq, Hkv = 60, 14, 8, 8
    prefix = PAGE * pages
    lens = _once((5, 140), B, pages)
    q, k, v, table, sl = paged_case(lens, 1, Hq, Hkv, D, seed=15, prefix=prefix)
    _assert_taken_once(fa, q, k, prefix)
    q[:] = 1.0
    g = torch.Generator().manual_seed(4)
    for t in range(pages):
        k[int(table[0, t])] = (0.25 * (t % 9) + 0.001 * torch.randn((Hkv, PAGE, D), generator=g)).to(torch.bfloat16)
    k[int(table[0, 5]), :, 64:] = -3.0
    got = fa.flex_decode_shared(q.cuda(), k.cuda(), v.cuda(), table.cuda(), sl.cuda(), prefix, scale=1.0)
    assert_decode(got, decode_ref(q, k, v, table, lens, scale=1.0))
    k[int(table[0, 2]), :, :70] = float("-inf")
    k[int(table[0, 0])] = float("-inf")
    got = fa.flex_decode_shared(q.cuda(), k.cuda(), v.cuda(), table.cuda(), sl.cuda(), prefix, scale=1.0)
    ref = decode_ref(q, k, v, table, lens, scale=1.0)
    ref = ref[0], ref[1], ref[2].nan_to_num(0.0), ref[3]
    # the bound of a score's own error is infinite there; 2^-7 covers P's rounding and 2 e of
    # the finite scores (|x| <= 2.1 D: e <= D 2^-23 2.1 D + 2^-16 < 2^-7.8)
    v_size = v.abs().max().double()
    assert bool(((got[0].cpu().double() - ref[0]).abs() <= (2 ** -8 + 2 * 2 ** -7.8 + 2 ** -8) * v_size).all())
    v[int(table[0, 9]), 3, 17, 5] = float("inf")
    got = fa.flex_decode_shared(q.cuda(), k.cuda(), v.cuda(), table.cuda(), sl.cuda(), prefix)
    assert bool(torch.isinf(got[0][:, 3, 0, 5]).all())
    rest = torch.ones_like(got[0], dtype=torch.bool)
    rest[:, 3, 0, 5] = False
    assert bool(torch.isfinite(got[0][rest]).all())


def test_decode_shared_once_views_and_reports():
    """Token-major queries and outputs, a bad page in the prefix (clamped and reported),
    and the next call on the same workspace clean."""
    fa = _fa()
    B, pages, n, Hq, Hkv, D = 52, 30, 2, 8, 4, 128
    prefix = PAGE * pages
    lens = _once((9, 1, 300), B, pages)
    lens = [x + 1 for x in lens]
    q, k, v, table, sl = paged_case(lens, n, Hq, Hkv, D, seed=5, prefix=prefix)
    kp, vp, tab, ln = k.cuda(), v.cuda(), table.cuda(), sl.cuda()
    qt = q.transpose(1, 2).contiguous().cuda().transpose(1, 2)
    out = torch.full((B, n, Hq, D), 5.0, dtype=torch.bfloat16, device="cuda").transpose(1, 2)
    size = fa.library().fa_decode_shared_workspace_size(B, Hq, Hkv, n, D, prefix)
    ws = torch.zeros(int(size), dtype=torch.uint8, device="cuda")
    bad = tab.clone()
    bad[0, 3], bad[0, 11] = -4, k.shape[0] + 9
    fa.flex_decode_shared(qt, kp, vp, bad, ln, prefix, out=out, ws=ws)
    assert fa.device_status(ws=ws) == fa.FA_ERR_BAD_BLOCKMASK
    got = fa.flex_decode_shared(qt, kp, vp, tab, ln, prefix, scale=0.05, out=out, ws=ws)
    assert fa.device_status(ws=ws) == 0 and got[0] is out
    assert_decode(got, decode_ref(q, k, v, table, lens, scale=0.05))
    with pytest.raises(fa.FlexAttnError):
        fa.flex_decode_shared(qt, kp, vp, tab, ln, prefix, ws=ws[:-16])


def test_decode_shared_once_in_graphs_and_on_streams():
    """Two captured calls replayed on two streams at once beside an eager one, their
    lengths changed in place (and with them the kernel's split of the SMs)."""
    fa = _fa()
    cases = []
    for B, pages, Hq, Hkv, D in ((49, 17, 8, 8, 64), (30, 55, 8, 4, 128)):
        lens = _once((700, 3, 90), B, pages)
        c = paged_case(lens, 1, Hq, Hkv, D, seed=B, prefix=PAGE * pages)
        cases.append((c, [t.cuda() for t in c], PAGE * pages))
    graphs, outs = [], []
    for c, d, prefix in cases:
        fa.flex_decode_shared(*d, prefix)
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(fa.flex_decode_shared(*d, prefix))
        graphs.append(g)
    streams = [torch.cuda.Stream() for _ in range(3)]
    for step in range(3):
        lens = []
        for c, d, prefix in cases:
            x = c[4].clone()
            if step:
                x[::step] = prefix + 1 + step  # most sequences' own parts shrink
            d[4].copy_(x)
            lens.append(x.tolist())
        torch.cuda.synchronize()
        for _ in range(4):
            for g, s in zip(graphs, streams):
                with torch.cuda.stream(s):
                    g.replay()
            eager = fa.flex_decode_shared(*cases[0][1], cases[0][2], stream=streams[2])
        torch.cuda.synchronize()
        for (c, d, prefix), o, x in zip(cases, outs, lens):
            assert_decode(o, decode_ref(*c[:4], x), f"step {step}")
        assert_decode(eager, decode_ref(*cases[0][0][:4], lens[0]), f"eager, step {step}")


# ------------------------------------------------------------------ streams, graphs, refusals

def test_decode_calls_on_two_streams_at_once():
    fa = _fa()
    cases = [paged_case([4000 + i, 30, 900], 1, 8, 2, 128, seed=i, prefix=0) for i in range(2)]
    streams = [torch.cuda.Stream() for _ in cases]
    dev = [[t.cuda() for t in c] for c in cases]
    torch.cuda.synchronize()
    outs = [[], []]
    for _ in range(5):
        for i, s in enumerate(streams):
            outs[i].append(fa.flex_decode_paged(*dev[i], stream=s))
    torch.cuda.synchronize()
    for i, c in enumerate(cases):
        ref = decode_ref(*c)
        for got in outs[i]:
            assert_decode(got, ref)
        with torch.cuda.stream(streams[i]):
            assert fa.device_status(ws=fa.paged_workspace(DEV)) == 0


def test_decode_graphs_replayed_with_new_lengths():
    """Two captured graphs of different shapes, replayed in turn and on two streams,
    their lengths and queries changed in place."""
    fa = _fa()
    a = paged_case([900, 1, 400], 1, 8, 2, 64, seed=1)
    b = paged_case([300, 700], 2, 8, 4, 128, seed=2, prefix=256)
    da, db = [t.cuda() for t in a], [t.cuda() for t in b]
    calls = [lambda: fa.flex_decode_paged(*da), lambda: fa.flex_decode_shared(*db, 256)]
    graphs, outs = [], []
    for call in calls:
        call()
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(call())
        graphs.append(g)
    for lens_a, lens_b in (([900, 1, 400], [300, 700]), ([10, 0, 512], [258, 400])):
        da[4].copy_(torch.tensor(lens_a, dtype=torch.int32))
        db[4].copy_(torch.tensor(lens_b, dtype=torch.int32))
        torch.cuda.synchronize()
        streams = [torch.cuda.Stream(), torch.cuda.Stream()]
        for _ in range(3):
            for g, s in zip(graphs, streams):
                with torch.cuda.stream(s):
                    g.replay()
        torch.cuda.synchronize()
        assert_decode(outs[0], decode_ref(*a[:4], lens_a))
        assert_decode(outs[1], decode_ref(*b[:4], lens_b))


def test_decode_of_a_large_batch():
    """More sequences than a CTA has threads, many of them empty, and a table far wider
    than any sequence needs."""
    fa = _fa()
    lens = [(i * 7) % 260 if i % 3 else 0 for i in range(5000)]
    q, k, v, table, sl = paged_case(lens, 1, 2, 1, 64, seed=6, width=200)
    got = fa.flex_decode_paged(q.cuda(), k.cuda(), v.cuda(), table.cuda(), sl.cuda())
    assert_decode(got, decode_ref(q, k, v, table, lens))
    with pytest.raises(fa.FlexAttnError):  # a work list of 2^31 pages
        wide = torch.zeros((1, 1), dtype=torch.int32, device="cuda").expand(1, 2 ** 24 - 2)
        many = torch.zeros((1, 256, 1, 64), dtype=torch.bfloat16, device="cuda")
        pool = torch.zeros((1, 256, PAGE, 64), dtype=torch.bfloat16, device="cuda")
        fa.flex_decode_paged(many, pool, pool, wide.contiguous(), sl[:1].cuda())


@pytest.mark.parametrize("captured", [False, True])
def test_append_and_decode_chained_over_streams(captured):
    """Each step appends on one stream and decodes on another, ordered by events, the
    lengths advanced on the device in between: kernels that start before the stream's
    previous kernel has ended still see everything before them.  Eagerly, and as one
    captured graph that is replayed."""
    fa = _fa()
    B, Hq, Hkv, D, steps = 3, 8, 2, 64, 4
    g = torch.Generator().manual_seed(12)
    table = torch.randperm(24, generator=g)[:B * 4].view(B, 4).to(torch.int32).contiguous()
    new = [[torch.randn((B, h, 1, D), generator=g).to(torch.bfloat16) for h in (Hq, Hkv, Hkv)] for _ in range(steps)]
    start = [126, 3, 250]
    kp0, vp0 = [torch.randn((24, Hkv, PAGE, D), generator=g).to(torch.bfloat16) for _ in range(2)]
    f = 10000.0 ** (-torch.arange(0, D, 2, dtype=torch.float64) / D)
    kp, vp, tab, fd = kp0.cuda(), vp0.cuda(), table.cuda(), f.cuda()
    dev = [[t.cuda() for t in step] for step in new]
    have = torch.tensor(start, dtype=torch.int32, device="cuda")
    ws = [torch.zeros(1 << 23, dtype=torch.uint8, device="cuda") for _ in range(2)]
    main, side = torch.cuda.Stream(), torch.cuda.Stream()

    def run():
        outs = []
        for q, k, v in dev:
            qr = fa.paged_append(k, v, kp, vp, tab, have, q=q, inv_freq=fd, ws=ws[0])
            have.add_(1)
            side.wait_stream(main)
            with torch.cuda.stream(side):
                outs.append((qr, *fa.flex_decode_paged(qr, kp, vp, tab, have, ws=ws[1])))
            main.wait_stream(side)
        return outs
    torch.cuda.synchronize()
    with torch.cuda.stream(main):
        if captured:
            run()
            torch.cuda.synchronize()
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph, stream=main):
                outs = run()
            kp.copy_(kp0)
            vp.copy_(vp0)
            have.copy_(torch.tensor(start, dtype=torch.int32))
            graph.replay()
        else:
            outs = run()
    torch.cuda.synchronize()
    assert fa.device_status(ws=ws[0]) == 0 and fa.device_status(ws=ws[1]) == 0
    assert have.tolist() == [x + steps for x in start]
    kc, vc = kp.cpu(), vp.cpu()
    for i, (qr, o, lse) in enumerate(outs):
        # later steps' keys lie behind this step's lengths
        want = decode_ref(qr.cpu(), kc, vc, table, [x + i + 1 for x in start])
        assert_decode((o, lse), want, f"step {i}")


def test_decode_paged_refusals():
    fa = _fa()
    q, k, v, table, sl = [t.cuda() for t in paged_case([300, 20], 1, 8, 2, 64, seed=1)]
    ok = dict(q=q, k_pages=k, v_pages=v, page_table=table, seq_lens=sl)

    def call(shared=False, prefix=128, **change):
        kw = {**ok, **change}
        first = kw.pop("q")
        return fa.flex_decode_shared(first, prefix_len=prefix, **kw) if shared else fa.flex_decode_paged(first, **kw)
    many = torch.zeros((2, 34, 1, 64), dtype=torch.bfloat16, device="cuda")
    for shared in (False, True):
        for bad in (dict(q=many), dict(score_mod=("bias", torch.zeros((2, 8, 1, 304), dtype=torch.bfloat16,
                                                                      device="cuda"))),
                    dict(k_pages=k[:1]), dict(k_pages=k[:, :, :64], v_pages=v[:, :, :64]),
                    dict(q=q[:, :7].contiguous()), dict(score_mod=("softcap", 0.0)),
                    dict(ws=torch.zeros(256, dtype=torch.uint8, device="cuda")),
                    dict(page_table=table[:1].expand(2, -1))):
            with pytest.raises(fa.FlexAttnError):
                call(shared, **bad)
        for bad in (dict(seq_lens=sl.long()), dict(seq_lens=sl[:1]), dict(page_table=table.long()),
                    dict(page_table=table[:1]), dict(q=q.half()), dict(lse=torch.zeros((2, 8, 2), device="cuda")),
                    dict(score_mod=("alibi", torch.zeros(7, device="cuda")))):
            with pytest.raises(TypeError):
                call(shared, **bad)
    for prefix in (-128, 100, 128 * (table.shape[1] + 1)):
        with pytest.raises(fa.FlexAttnError):
            call(True, prefix)
    with pytest.raises(ValueError):
        call(window=-1)
    torch.cuda.synchronize()
    assert fa.device_status(ws=fa.paged_workspace(DEV)) == 0


# ------------------------------------------------------------------ the operators as they are used together

@pytest.mark.parametrize("shared", [False, True])
def test_serving_run_prompts_then_steps(shared):
    """A batch of prompts appended in two chunks behind a (shared) prefix, prefilled
    through flex_attention_paged, then decoding steps of one and of two tokens: after
    every call the attention equals the 64-bit form over everything appended so far."""
    fa = _fa()
    B, Hq, Hkv, D, prefix = 3, 8, 2, 64, 256 if shared else 0
    g = torch.Generator().manual_seed(2)
    inv_freq, amp = fa.rope_frequencies(32, scaling=("yarn", 4.0, 512, 1.0, 32.0))
    width = 8
    num = 2 + B * width
    table = torch.randperm(num, generator=g)[:2 + B * (width - 2)].to(torch.int32)
    table = torch.cat([table[:2].expand(B, 2), table[2:].view(B, width - 2)], dim=1).contiguous() if shared else \
        torch.randperm(num, generator=g)[:B * width].view(B, width).to(torch.int32).contiguous()
    kp, vp = [torch.full((num, Hkv, PAGE, D), 8.0, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    tab, have = table.cuda(), torch.zeros(B, dtype=torch.int32, device="cuda")
    cached = [0] * B

    def put(S, new, rows=slice(None)):
        q, k, v = [torch.randn((B, S, h, D), generator=g).to(torch.bfloat16).cuda().transpose(1, 2)
                   for h in (Hq, Hkv, Hkv)]
        fresh = torch.tensor(new, dtype=torch.int32, device="cuda")
        qr = fa.paged_append(k, v, kp, vp, tab, have, new_lens=fresh, q=q, inv_freq=inv_freq, amplitude=amp)
        have.add_(fresh)
        for b in range(B):
            cached[b] += new[b]
        return qr
    if shared:  # the prefix once, by the first sequence
        put(prefix, [prefix] + [0] * (B - 1))
        have.fill_(prefix)
        cached[:] = [prefix] * B
    qr = put(200, [200] * B)
    bm = fa.create_block_mask("and", [("causal",)], 1, 1, 200, prefix + 200, q_offset=prefix)
    o, lse = fa.flex_attention_paged(qr, kp, vp, tab, bm)
    rows = [0, 7, 199]
    for r in rows:
        want = decode_ref(qr[:, :, r:r + 1].cpu(), kp.cpu(), vp.cpu(), table, [prefix + r + 1] * B)
        assert_decode((o[:, :, r:r + 1], lse[:, :, r:r + 1]), want, f"prefill row {r}")
    put(90, [90, 0, 31])
    for step in range(3):
        n = 1 + step % 2
        qr = put(n, [n] * B)
        if shared:
            got = fa.flex_decode_shared(qr, kp, vp, tab, have, prefix)
        else:
            got = fa.flex_decode_paged(qr, kp, vp, tab, have)
        assert_decode(got, decode_ref(qr.cpu(), kp.cpu(), vp.cpu(), table, cached), f"step {step}")
    assert have.tolist() == cached
    assert fa.device_status(ws=fa.paged_workspace(DEV)) == 0 and fa.device_status() == 0
