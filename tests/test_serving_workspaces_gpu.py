"""The serving calls' default workspaces: what is held as a batch grows, and after refused calls."""

import pytest
import torch

from paged_reference import PAGE, assert_decode, decode_ref, paged_case

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda", 0)
LEAST = 1 << 22  # the smallest default workspace


def _fa():
    import block_sparse_attention_48_b200 as fa
    return fa


def _held(before):
    torch.cuda.synchronize()
    return torch.cuda.memory_allocated() - before


def test_workspace_of_a_growing_batch():
    """A batch that grows by a sequence at a time: at most twice the last call's need is
    held, a status from before a growth is still there after it, and the results are those
    of a workspace of the caller's own."""
    fa = _fa()
    pages, n, Hq, Hkv, D, top = 32, 1, 32, 8, 128, 40
    prefix = PAGE * pages
    lens = [prefix + 1 + 5 * i for i in range(top)]
    q, k, v, table, sl = paged_case(lens, n, Hq, Hkv, D, seed=6, prefix=prefix)
    q, k, v, table, sl = [t.cuda() for t in (q, k, v, table, sl)]
    lib = fa.library()

    def need(B):
        return lib.fa_decode_shared_workspace_size(B, Hq, Hkv, n, D, prefix)
    own = torch.zeros(need(top), dtype=torch.uint8, device="cuda")
    want = fa.flex_decode_shared(q, k, v, table, sl, prefix, ws=own)
    bad = table[:16].clone()
    bad[3, pages] = -1
    torch.cuda.synchronize()
    before = torch.cuda.memory_allocated()
    with torch.cuda.stream(torch.cuda.Stream()):  # which has no workspace yet
        for B in range(8, top + 1):
            if B == 16:
                fa.flex_decode_shared(q[:B], k, v, bad, sl[:B], prefix)
            got = fa.flex_decode_shared(q[:B], k, v, table[:B], sl[:B], prefix)
        for a, b in zip(got, want):
            assert torch.equal(a, b)
        got = a = b = None
        assert _held(before) <= max(LEAST, 2 * need(top))
        ws = fa.paged_workspace(DEV)
        assert need(top) <= ws.numel()
        assert fa.device_status(ws=ws) == fa.FA_ERR_BAD_BLOCKMASK
        assert fa.device_status(ws=ws) == 0


@pytest.mark.parametrize("shared", [False, True])
def test_refused_calls_get_no_workspace(shared):
    """A call that is refused for its shape does not first take the memory that such a shape
    would need, let alone keep it."""
    fa = _fa()
    pool = torch.zeros((3, 1, PAGE, 64), dtype=torch.bfloat16, device="cuda")
    table = torch.zeros((1, 2), dtype=torch.int32, device="cuda")
    lens = torch.full((1,), 200, dtype=torch.int32, device="cuda")
    call = (lambda q: fa.flex_decode_shared(q, pool, pool, table, lens, PAGE)) if shared else \
        (lambda q: fa.flex_decode_paged(q, pool, pool, table, lens))
    for shape in ((1, 8, 1024, 64), (1, 4096, 1, 64)):
        q = torch.zeros(shape, dtype=torch.bfloat16, device="cuda")
        torch.cuda.synchronize()
        before = torch.cuda.memory_allocated()
        torch.cuda.reset_peak_memory_stats()
        with torch.cuda.stream(torch.cuda.Stream()):
            with pytest.raises(fa.FlexAttnError):
                call(q)
        assert _held(before) <= LEAST
        # the outputs may have been made: of q's size and its rows in fp32
        assert torch.cuda.max_memory_allocated() - before <= LEAST + 2 * q.numel() * 2 + 1024
