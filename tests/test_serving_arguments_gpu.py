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


def test_tensors_written_in_place_are_marked():
    """A tensor that autograd saved and a call then wrote over raises in the backward pass,
    as with torch's own in-place operators, instead of giving another gradient."""
    fa = _fa()
    f = torch.ones(32, dtype=torch.float64, device="cuda")
    x = torch.zeros((1, 2, 3, 64), dtype=torch.bfloat16, device="cuda", requires_grad=True)
    y = x.exp()  # saves its result
    fa.rope_apply(y, None, f, out=(y, None))
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        y.sum().backward()
    q, k, v, table, sl = [t.cuda() for t in paged_case([300, 20], 1, 8, 2, 64, seed=1)]
    new = torch.ones((2, 2, 1, 64), dtype=torch.bfloat16, device="cuda")
    q_out, out, lse = torch.zeros_like(q), torch.zeros_like(q), torch.zeros((2, 8, 1), device="cuda")
    seen = [t._version for t in (k, v, q_out, out, lse)]
    fa.paged_append(new, new, k, v, table, sl - 1, q=q, q_out=q_out)
    fa.flex_decode_paged(q, k, v, table, sl, out=out, lse=lse)
    assert all(t._version > n for t, n in zip((k, v, q_out, out, lse), seen))
    # tensors without such a count
    with torch.inference_mode():
        k2, out2 = torch.zeros_like(k), torch.zeros_like(q)
    fa.paged_append(new, new, k2, k2.clone(), table, sl - 1)
    fa.flex_decode_paged(q, k, v, table, sl, out=out2)
    assert torch.equal(out2, out)


def test_an_amplitude_that_fp32_rounds_to_zero_is_refused():
    """An amplitude of 0 means 1 to the C ABI: what becomes 0 in fp32 must not turn into it."""
    fa = _fa()
    f = torch.ones(32, dtype=torch.float64, device="cuda")
    q = torch.ones((1, 2, 3, 64), dtype=torch.bfloat16, device="cuda")
    for amp in (1e-50, 0.0, -1.0, float("nan")):
        with pytest.raises(ValueError):
            fa.rope_apply(q, None, f, amplitude=amp)
    small = fa.rope_apply(q, None, f, amplitude=1e-30)[0]
    assert float(small.abs().max()) < 2e-30
