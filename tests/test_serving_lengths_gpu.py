"""Decoding with lengths that the other tests do not have: out of range behind a shared prefix
that is taken once, and few long sequences with a window or of unequal lengths."""

import pytest
import torch

from paged_reference import PAGE, assert_decode, decode_ref, paged_case

pytestmark = pytest.mark.gpu


def _fa():
    import block_sparse_attention_48_b200 as fa
    return fa


def _assert_taken_once(fa, q, k, prefix):
    lib, B, Hkv = fa.library(), q.shape[0], k.shape[1]
    assert lib.fa_decode_shared_workspace_size(B, q.shape[1], Hkv, q.shape[2], q.shape[3], prefix) > \
        lib.fa_decode_paged_workspace_size(B, q.shape[1], Hkv, q.shape[2], q.shape[3])


@pytest.mark.parametrize("kind", [None, "alibi", "softcap"])
def test_shared_prefix_once_with_bad_lengths(kind):
    """Lengths below zero and beyond the table count as the nearest length that the table
    has, in the prefix's part as in the own one, and are reported; the other sequences' rows
    are right."""
    fa = _fa()
    B, pages, n, Hq, Hkv, D = 52, 30, 2, 8, 4, 128
    prefix = PAGE * pages
    lens = [prefix + (9, 2, 300)[i % 3] for i in range(B)]
    q, k, v, table, sl = paged_case(lens, n, Hq, Hkv, D, seed=5, prefix=prefix)
    _assert_taken_once(fa, q, k, prefix)
    most = PAGE * table.shape[1]
    for b, raw in ((1, 2 ** 31 - 1), (4, most + 3), (7, -7), (12, -2 ** 31), (20, most)):
        sl[b], lens[b] = raw, min(max(raw, 0), most)
    slopes = torch.tensor([2.0 ** (-8 * (h + 1) / Hq) for h in range(Hq)], dtype=torch.float32)
    score = {None: None, "alibi": ("alibi", slopes), "softcap": ("softcap", 5.0)}[kind]
    on_gpu = ("alibi", slopes.cuda()) if kind == "alibi" else score
    ws = torch.zeros(1 << 25, dtype=torch.uint8, device="cuda")
    got = fa.flex_decode_shared(q.cuda(), k.cuda(), v.cuda(), table.cuda(), sl.cuda(), prefix, score_mod=on_gpu, ws=ws)
    assert fa.device_status(ws=ws) == fa.FA_ERR_BAD_BLOCKMASK
    assert_decode(got, decode_ref(q, k, v, table, lens, None, score))


@pytest.mark.parametrize("case", [
    # batch, own lengths (cycled), prefix pages, q_len, Hq, Hkv, score
    (33, (1, 130, 7), 8, 1, 16, 1, None),
    (12, (40, 300, 129, 4), 6, 4, 16, 4, "softcap"),
    (20, (5, 2000), 14, 5, 6, 2, "alibi"),
], ids=lambda c: f"b{c[0]}-p{c[2]}-n{c[3]}-h{c[4]}-{c[5]}-{c[6]}")
def test_shared_prefix_once_of_few_pages(case):
    """More than eight rows per kv head, D = 128, behind a short prefix."""
    fa = _fa()
    B, own, pages, n, Hq, Hkv, kind = case
    prefix = PAGE * pages
    lens = [prefix + own[i % len(own)] for i in range(B)]
    q, k, v, table, sl = paged_case(lens, n, Hq, Hkv, 128, seed=B, prefix=prefix, filler=float("nan"))
    _assert_taken_once(fa, q, k, prefix)
    slopes = torch.tensor([2.0 ** (-8 * (h + 1) / Hq) for h in range(Hq)], dtype=torch.float32)
    score = {None: None, "alibi": ("alibi", slopes), "softcap": ("softcap", 5.0)}[kind]
    args = [t.cuda() for t in (q, k, v, table, sl)]
    kw = dict(score_mod=("alibi", slopes.cuda()) if kind == "alibi" else score,
              ws=torch.zeros(1 << 25, dtype=torch.uint8, device="cuda"))
    got = fa.flex_decode_shared(*args, prefix, **kw)
    assert_decode(got, decode_ref(q, k, v, table, lens, None, score))
    for _ in range(5):
        again = fa.flex_decode_shared(*args, prefix, **kw)
        assert torch.equal(again[0], got[0]) and torch.equal(again[1], got[1])
    assert fa.device_status(ws=kw["ws"]) == 0


@pytest.mark.parametrize("case", [
    # lens, q_len, Hq, Hkv, D, window, score
    ([30000], 1, 16, 1, 128, 16384, None),
    ([20000, 3000, 9100], 2, 8, 1, 128, 4096, "softcap"),
    ([25000, 14], 5, 6, 2, 64, 9000, None),
    ([1200, 2500, 1700, 2111, 1500], 1, 16, 1, 128, None, None),
    ([2000, 5700, 130, 4100], 2, 4, 2, 64, None, "softcap"),
    ([2500, 2500, 2500], 1, 8, 1, 128, None, None),
], ids=lambda c: "-".join(str(x) for x in c)[:60])
def test_decode_of_few_segments(case):
    """Few segments, alike and not, with a window and without: right whatever the number of
    teams that take them, and the same bits every time; tables of just the pages and much
    wider ones."""
    fa = _fa()
    lens, n, Hq, Hkv, D, window, kind = case
    score = ("softcap", 5.0) if kind else None
    for width in (None, 3 * ((max(lens) + PAGE - 1) // PAGE)):
        q, k, v, table, sl = paged_case(lens, n, Hq, Hkv, D, seed=len(lens) + D, width=width, filler=float("nan"))
        args = [t.cuda() for t in (q, k, v, table, sl)]
        ws = torch.zeros(1 << 23, dtype=torch.uint8, device="cuda")
        got = fa.flex_decode_paged(*args, window=window, score_mod=score, ws=ws)
        assert_decode(got, decode_ref(q, k, v, table, lens, window, score))
        for _ in range(5):
            again = fa.flex_decode_paged(*args, window=window, score_mod=score, ws=ws)
            assert torch.equal(again[0], got[0]) and torch.equal(again[1], got[1])
        assert fa.device_status(ws=ws) == 0


@pytest.mark.parametrize("shape", [(3, 8, 8, 128, 1), (4, 8, 8, 64, 2), (3, 32, 8, 128, 4)])
def test_shared_prefix_once_over_long_lists(shape):
    """Few sequences behind an odd number of shared pages, taken once, and shares of 20 and
    more own pages that run over several segments; calls one after another give the same
    bits."""
    fa = _fa()
    B, Hq, Hkv, D, n = shape
    prefix = 301 * PAGE
    lens = [prefix + (11000, 300, 4001, 2 * n)[i] for i in range(B)]
    q, k, v, table, sl = paged_case(lens, n, Hq, Hkv, D, seed=79, prefix=prefix, filler=float("nan"))
    _assert_taken_once(fa, q, k, prefix)
    args = [t.cuda() for t in (q, k, v, table, sl)]
    ws = torch.zeros(1 << 25, dtype=torch.uint8, device="cuda")
    got = fa.flex_decode_shared(*args, prefix, ws=ws)
    assert_decode(got, decode_ref(q, k, v, table, lens))
    for _ in range(20):
        again = fa.flex_decode_shared(*args, prefix, ws=ws)
        assert torch.equal(again[0], got[0]) and torch.equal(again[1], got[1])
    assert fa.device_status(ws=ws) == 0


@pytest.mark.parametrize("B", [6, 40])
def test_shared_prefix_with_an_empty_first_sequence(B):
    """Sequence 0 empty, or ending in the prefix: its row still names the shared pages, and the
    others read them there (page by page and taken once)."""
    fa = _fa()
    pages, n, Hq, Hkv, D = 30, 1, 8, 4, 128
    prefix = PAGE * pages
    for first in (0, 200):
        lens = [first] + [prefix + 5 + 31 * i for i in range(1, B)]
        q, k, v, table, sl = paged_case(lens, n, Hq, Hkv, D, seed=B, prefix=prefix, filler=float("nan"))
        if B == 40:
            _assert_taken_once(fa, q, k, prefix)
        tab = table.clone()
        tab[1:, :pages] = -1
        ws = torch.zeros(1 << 25, dtype=torch.uint8, device="cuda")
        got = fa.flex_decode_shared(q.cuda(), k.cuda(), v.cuda(), tab.cuda(), sl.cuda(), prefix, ws=ws)
        assert fa.device_status(ws=ws) == 0
        assert_decode(got, decode_ref(q, k, v, table, lens))
