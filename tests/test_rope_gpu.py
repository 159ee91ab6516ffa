"""Rotary positions (fa_rope_apply) and the paged append (fa_paged_append) against their
64-bit forms: layouts, part of the head, far positions, ragged batches, views, refused
and reported inputs."""

import pytest
import torch

from paged_reference import PAGE, assert_rope, rope_ref

pytestmark = pytest.mark.gpu


def _fa():
    import block_sparse_attention_48_b200 as fa
    return fa


def _randn(shape, seed):
    return torch.randn(shape, generator=torch.Generator().manual_seed(seed)).to(torch.bfloat16)


def _freq(rotary, base=10000.0):
    return base ** (-torch.arange(0, rotary, 2, dtype=torch.float64) / max(rotary, 1))


CASES = [
    # B, Hq, Hk, S, D, rotary, interleaved, far, amplitude, token-major
    (1, 1, 1, 1, 64, 64, False, 0, 1.0, False),
    (1, 1, 1, 1, 64, 16, True, 7, 1.0, False),
    (3, 5, 2, 17, 64, 48, False, 1000000, 1.1, True),
    (2, 32, 8, 1, 128, 128, False, 1000000, 1.0, True),
    (2, 8, 8, 333, 128, 64, True, 40000, 1.0, False),
    (1, 17, 1, 70, 128, 112, True, 100, 0.5, True),
    (4, 16, 16, 257, 64, 64, True, 0, 1.0, False),
    (2, 3, 3, 40, 128, 0, False, 0, 1.0, True),
    (1, 40, 20, 2000, 128, 128, False, 2000000000, 1.0, False),
]


@pytest.mark.parametrize("case", CASES, ids=lambda c: "-".join(str(x) for x in c))
@pytest.mark.parametrize("inverse", [False, True])
def test_rope_matches_the_formula(case, inverse):
    fa = _fa()
    B, Hq, Hk, S, D, rotary, inter, far, amp, tm = case
    if tm:
        qkv = _randn((B, S, Hq + Hk, D), 1).cuda().transpose(1, 2)
        q, k = qkv[:, :Hq], qkv[:, Hq:]
    else:
        q, k = _randn((B, Hq, S, D), 1).cuda(), _randn((B, Hk, S, D), 2).cuda()
    g = torch.Generator().manual_seed(3)
    pos = (torch.randint(0, far + 1, (B, 1), generator=g) + torch.arange(S)).to(torch.int32)
    f = _freq(rotary)
    before = q.clone(), k.clone()
    qo, ko = fa.rope_apply(q, k, f.cuda(), positions=pos.cuda(), interleaved=inter, amplitude=amp, inverse=inverse)
    torch.cuda.synchronize()
    assert_rope(qo, q.cpu(), pos, f, inter, amp, inverse)
    assert_rope(ko, k.cpu(), pos, f, inter, amp, inverse)
    assert torch.equal(q, before[0]) and torch.equal(k, before[1])


def test_rope_positions_forms_and_in_place():
    fa = _fa()
    B, H, S, D = 3, 4, 50, 64
    q, f = _randn((B, H, S, D), 5).cuda(), _freq(64).cuda()
    shared = torch.randint(0, 5000, (S,), generator=torch.Generator().manual_seed(1)).to(torch.int32)
    by_row = fa.rope_apply(q, None, f, positions=shared.expand(B, S).contiguous().cuda())[0]
    assert torch.equal(fa.rope_apply(q, None, f, positions=shared.cuda())[0], by_row)
    # a column range of a wider tensor of positions
    wide = torch.cat([shared.expand(B, S) + 1, shared.expand(B, S)], dim=1).contiguous().cuda()
    assert torch.equal(fa.rope_apply(q, None, f, positions=wide[:, S:])[0], by_row)
    at = (11 + torch.arange(S)).expand(B, S).to(torch.int32).contiguous().cuda()
    want = fa.rope_apply(q, None, f, positions=at)[0]
    assert torch.equal(fa.rope_apply(q, None, f, offset=11)[0], want)
    x = q.clone()
    got, none = fa.rope_apply(x, None, f, offset=11, out=(x, None))
    assert got is x and none is None and torch.equal(x, want)
    # an expanded input and one whose start is not 16-byte aligned are read through a copy
    assert torch.equal(fa.rope_apply(q[:1].expand(B, H, S, D), None, f, offset=11)[0],
                       fa.rope_apply(q[:1].repeat(B, 1, 1, 1), None, f, offset=11)[0])
    flat = torch.zeros(q.numel() + 1, dtype=torch.bfloat16, device="cuda")
    odd = flat[1:].view(B, H, S, D).copy_(q)
    assert torch.equal(fa.rope_apply(odd, None, f, offset=11)[0], want)
    # other strides of the input's are kept apart from the output's
    out = torch.full((B, S, H, D), 7.0, dtype=torch.bfloat16, device="cuda").transpose(1, 2)
    assert torch.equal(fa.rope_apply(q, None, f, offset=11, out=(out, None))[0], want)


@pytest.mark.parametrize("shape", [(0, 4, 8, 64), (2, 4, 0, 64), (2, 0, 8, 64)])
def test_rope_of_nothing(shape):
    fa = _fa()
    q = torch.zeros(shape, dtype=torch.bfloat16, device="cuda")
    assert fa.rope_apply(q, None, _freq(64).cuda())[0].shape == shape


@pytest.mark.parametrize("inter", [False, True])
def test_rope_gradients(inter):
    """backward() against the formula (the transposed rotation) and against differences:
    the operator is linear, so <g, R(x + d) - R(x)> = <R^T g, d> up to the roundings."""
    fa = _fa()
    B, Hq, Hk, S, D, rotary, amp = 2, 4, 2, 60, 128, 96, 1.25
    q, k = _randn((B, Hq, S, D), 1).cuda().requires_grad_(), _randn((B, Hk, S, D), 2).cuda().requires_grad_()
    gq, gk = _randn((B, Hq, S, D), 3), _randn((B, Hk, S, D), 4)
    f = _freq(rotary)
    pos = (torch.arange(S) + 900).expand(B, S).to(torch.int32).contiguous()
    qo, ko = fa.rope_autograd(q, k, f.cuda(), positions=pos.cuda(), interleaved=inter, amplitude=amp)
    torch.autograd.backward([qo, ko], [gq.cuda(), gk.cuda()])
    assert_rope(q.grad, gq, pos, f, inter, amp, True)
    assert_rope(k.grad, gk, pos, f, inter, amp, True)
    d = _randn((B, Hq, S, D), 6)
    x = q.detach().cpu().double()
    step = rope_ref(x + d.double(), pos, f, inter, amp) - rope_ref(x, pos, f, inter, amp)
    left, right = (gq.double() * step).sum(), (q.grad.cpu().double() * d.double()).sum()
    # q.grad's entries are off by half a bf16 step each, whatever their signs
    assert abs(left - right) <= 2 ** -8 * (q.grad.cpu().double() * d.double()).abs().sum() + 1e-6
    # a broadcast gradient (the sum's) and one without k
    x = q.detach().clone().requires_grad_()
    y, none = fa.rope_autograd(x, None, f.cuda(), positions=pos.cuda(), interleaved=inter)
    assert none is None
    y.sum().backward()
    assert_rope(x.grad, torch.ones_like(gq), pos, f, inter, 1.0, True)


def test_rope_training_step_in_a_graph():
    """Forward and backward captured and replayed on new contents of the same buffers."""
    fa = _fa()
    q, f = _randn((2, 4, 64, 64), 1).cuda(), _freq(64).cuda()
    g = _randn((2, 4, 64, 64), 2).cuda()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        x = q.clone().requires_grad_()
        torch.autograd.grad(fa.rope_autograd(x, None, f, offset=3)[0], x, g)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            y = fa.rope_autograd(x, None, f, offset=3)[0]
            grad, = torch.autograd.grad(y, x, g)
    with torch.no_grad():
        x.copy_(_randn((2, 4, 64, 64), 8).cuda())
    g.copy_(_randn((2, 4, 64, 64), 9).cuda())
    graph.replay()
    torch.cuda.synchronize()
    pos = (3 + torch.arange(64)).expand(2, 64)
    assert_rope(y.detach(), x.detach().cpu(), pos, f.cpu(), False)
    assert_rope(grad, g.cpu(), pos, f.cpu(), False, inverse=True)


def test_rope_refusals():
    fa = _fa()
    q, f = _randn((1, 2, 8, 64), 1).cuda(), _freq(64).cuda()
    for bad in (dict(inv_freq=_freq(128).cuda()), dict(inv_freq=_freq(24).cuda())):
        with pytest.raises(fa.FlexAttnError):
            fa.rope_apply(q, None, **bad)
    with pytest.raises(fa.FlexAttnError):
        fa.rope_apply(q[..., :32].contiguous(), None, _freq(32).cuda())
    with pytest.raises(TypeError):
        fa.rope_apply(q, None, f.float())
    with pytest.raises(TypeError):
        fa.rope_apply(q, None, f, positions=torch.zeros(9, dtype=torch.int32, device="cuda"))
    with pytest.raises(TypeError):
        fa.rope_apply(q, None, f, positions=torch.zeros(8, dtype=torch.int64, device="cuda"))
    with pytest.raises(TypeError):
        fa.rope_apply(q.float(), None, f)
    with pytest.raises(TypeError):
        fa.rope_apply(q.cpu(), None, f)
    with pytest.raises(ValueError):
        fa.rope_apply(q, None, f, amplitude=0.0)
    with pytest.raises(fa.FlexAttnError):  # k of another length
        fa.rope_apply(q, _randn((1, 2, 9, 64), 1).cuda(), f)
    x = q.clone().requires_grad_()
    y = fa.rope_autograd(x, None, f)[0]
    gx, = torch.autograd.grad(y, x, q.clone().requires_grad_(), create_graph=True)
    with pytest.raises(RuntimeError):  # no second derivative
        gx.sum().backward()


# ------------------------------------------------------------------ append

APPENDS = [
    # cache_lens, new_lens, S, Hq, Hkv, D, rotary, interleaved
    ([0], [1], 1, 4, 4, 64, 64, False),
    ([127, 128, 5, 0], [1, 1, 0, 1], 1, 8, 2, 128, 128, False),
    ([100, 0, 250, 128], [300, 257, 3, 0], 300, 16, 8, 128, 64, True),
    ([3, 77], [40, 13], 40, 3, 1, 64, 16, False),
    ([1, 2, 3], [5, 5, 5], 5, 2, 2, 64, 0, False),
]


def _append_inputs(cache, S, Hq, Hkv, D, seed=0):
    B = len(cache)
    counts = [(c + S + PAGE - 1) // PAGE for c in cache]
    num = sum(counts) + 2
    g = torch.Generator().manual_seed(seed)
    order = torch.randperm(num, generator=g).to(torch.int32)
    table = torch.full((B, max(counts)), -5, dtype=torch.int32)
    at = 0
    for b, n in enumerate(counts):
        table[b, :n] = order[at:at + n]
        at += n
    kp = torch.randn((num, Hkv, PAGE, D), generator=g).to(torch.bfloat16)
    vp = torch.randn((num, Hkv, PAGE, D), generator=g).to(torch.bfloat16)
    qkv = torch.randn((B, S, Hq + 2 * Hkv, D), generator=g).to(torch.bfloat16).transpose(1, 2)
    return table, kp, vp, qkv[:, :Hq], qkv[:, Hq:Hq + Hkv], qkv[:, Hq + Hkv:]


def _expect_append(kp, vp, qo, q, k, v, table, cache, new, f, inter):
    """64-bit pools and q_out after the call, and where they were written."""
    B, _, S, _ = k.shape
    pos = torch.tensor(cache)[:, None] + torch.arange(S)
    kr, qr = rope_ref(k, pos, f, inter), rope_ref(q, pos, f, inter)
    ek, ev, eq = kp.double(), vp.double(), qo.double()
    for b in range(B):
        for s in range(new[b]):
            page, slot = int(table[b, int(pos[b, s]) // PAGE]), int(pos[b, s]) % PAGE
            ek[page, :, slot], ev[page, :, slot], eq[b, :, s] = kr[b, :, s], v[b, :, s].double(), qr[b, :, s]
    return ek, ev, eq


@pytest.mark.parametrize("case", APPENDS, ids=lambda c: "-".join(str(x) for x in c))
def test_append_matches_the_formula(case):
    fa = _fa()
    cache, new, S, Hq, Hkv, D, rotary, inter = case
    table, kp, vp, q, k, v = _append_inputs(cache, S, Hq, Hkv, D)
    f = _freq(rotary)
    kpd, vpd = kp.cuda(), vp.cuda()
    qo = torch.full(q.shape, 9.0, dtype=torch.bfloat16, device="cuda")
    lens = torch.tensor(cache, dtype=torch.int32, device="cuda")
    qkv = torch.cat([q, k, v], dim=1).transpose(1, 2).contiguous().cuda().transpose(1, 2)
    got = fa.paged_append(qkv[:, Hq:Hq + Hkv], qkv[:, Hq + Hkv:], kpd, vpd, table.cuda(), lens,
                          new_lens=torch.tensor(new, dtype=torch.int32, device="cuda"), q=qkv[:, :Hq], q_out=qo,
                          inv_freq=f.cuda(), interleaved=inter)
    torch.cuda.synchronize()
    assert fa.device_status(ws=fa.paged_workspace(torch.device("cuda", 0))) == 0
    assert got is qo and lens.tolist() == cache
    ek, ev, eq = _expect_append(kp, vp, torch.full(q.shape, 9.0), q, k, v, table, cache, new, f, inter)
    assert torch.equal(vpd.cpu().double(), ev)
    # a rotated element is at most |a| + |b| <= 12 here: half a bf16 step of it, and 2^-19 of 12
    for out, ref, was in ((kpd, ek, kp), (qo, eq, torch.full(q.shape, 9.0, dtype=torch.bfloat16))):
        err = (out.cpu().double() - ref).abs()
        assert bool((err <= 2 ** -8 * ref.abs() + 12 * 2 ** -19).all())
        untouched = ref == was.double()
        assert torch.equal(out.cpu()[untouched], was[untouched])


def test_append_without_queries_lengths_or_rotation():
    fa = _fa()
    cache, S = [5, 130], 9
    table, kp, vp, q, k, v = _append_inputs(cache, S, 2, 2, 64)
    kpd, vpd = kp.cuda(), vp.cuda()
    lens = torch.tensor(cache, dtype=torch.int32, device="cuda")
    assert fa.paged_append(k.cuda(), v.cuda(), kpd, vpd, table.cuda(), lens) is None
    ek, ev, _ = _expect_append(kp, vp, q.clone(), q, k, v, table, cache, [S, S], _freq(0), False)
    assert torch.equal(kpd.cpu().double(), ek) and torch.equal(vpd.cpu().double(), ev)
    # a q_out made by the call is zero behind a sequence's new tokens
    new = torch.tensor([4, 0], dtype=torch.int32, device="cuda")
    out = fa.paged_append(k.cuda(), v.cuda(), kpd, vpd, table.cuda(), lens, new_lens=new, q=q.cuda())
    assert torch.equal(out[0, :, :4].cpu(), q[0, :, :4]) and not out[0, :, 4:].any() and not out[1].any()
    assert fa.device_status(ws=fa.paged_workspace(torch.device("cuda", 0))) == 0


@pytest.mark.parametrize("what", ["page", "negative page", "past the table", "cache_lens", "new_lens", "new_lens above"])
def test_append_reports_what_it_leaves_out(what):
    """Bad pages and lengths write nothing, and the sequences beside them are appended."""
    fa = _fa()
    cache, new, S = [130, 40], [7, 7], 7
    table, kp, vp, q, k, v = _append_inputs(cache, S, 2, 2, 64, seed=4)
    ws = torch.zeros(1 << 12, dtype=torch.uint8, device="cuda")
    tab, lens, fresh = table.clone(), list(cache), list(new)
    done = [0, 7]
    if what == "page":
        tab[0, 1] = kp.shape[0]
    elif what == "negative page":
        tab[0, 1] = -1
    elif what == "past the table":
        lens[0] = 2 ** 31 - 3
    elif what == "cache_lens":
        lens[0] = -1
    elif what == "new_lens":
        fresh[0] = -1
    else:
        fresh[0], done[0] = 8, 7
    kpd, vpd = kp.cuda(), vp.cuda()
    qo = q.cuda().contiguous().clone()
    i32 = dict(dtype=torch.int32, device="cuda")
    fa.paged_append(k.cuda(), v.cuda(), kpd, vpd, tab.cuda(), torch.tensor(lens, **i32),
                    new_lens=torch.tensor(fresh, **i32), q=q.cuda(), q_out=qo, inv_freq=_freq(0).cuda(), ws=ws)
    torch.cuda.synchronize()
    assert fa.device_status(ws=ws) == fa.FA_ERR_BAD_BLOCKMASK
    assert fa.device_status(ws=ws) == 0
    ek, ev, _ = _expect_append(kp, vp, q.clone(), q, k, v, table, cache, done, _freq(0), False)
    assert torch.equal(kpd.cpu().double(), ek) and torch.equal(vpd.cpu().double(), ev)
