"""Arguments of the serving calls in the forms that a program gives them."""

import pytest
import torch

from paged_reference import paged_case

pytestmark = pytest.mark.gpu


def _fa():
    import block_sparse_attention_48_b200 as fa
    return fa


def test_tensors_by_name_on_a_stream():
    """stream= with every tensor given by name."""
    fa = _fa()
    q, k, v, table, sl = [t.cuda() for t in paged_case([300, 20], 1, 8, 2, 64, seed=1)]
    new = torch.ones((2, 2, 1, 64), dtype=torch.bfloat16, device="cuda")
    f = torch.ones(32, dtype=torch.float64, device="cuda")
    s = torch.cuda.Stream()
    want, have = (fa.rope_apply(q, None, f, offset=3)[0], fa.flex_decode_paged(q, k, v, table, sl)), sl - 1
    torch.cuda.synchronize()
    got = fa.rope_apply(q=q, k=None, inv_freq=f, offset=3, stream=s)[0]
    paged = fa.flex_decode_paged(q=q, k_pages=k, v_pages=v, page_table=table, seq_lens=sl, stream=s)
    shared = fa.flex_decode_shared(q=q, k_pages=k, v_pages=v, page_table=table, seq_lens=sl, prefix_len=0, stream=s)
    fa.paged_append(k=new, v=new, k_pages=k, v_pages=v, page_table=table, cache_lens=have, stream=s)
    torch.cuda.synchronize()
    assert torch.equal(got, want[0]) and torch.equal(k[table[1, 0].item(), :, 19], new[1, :, 0])
    for o in (paged, shared):
        assert torch.equal(o[0], want[1][0]) and torch.equal(o[1], want[1][1])
