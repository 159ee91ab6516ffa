"""Decoding behind a shared prefix that is taken once: lengths out of range, and long
lists with an odd number of shared pages."""

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
