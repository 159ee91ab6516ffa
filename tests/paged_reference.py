"""Plain 64-bit forms of the rotary, append and paged-decode operators, and the error
bounds their bf16 / fp32 kernels are held to (CPU tensors)."""

import math

import torch

PAGE = 128
HALF_BF16 = torch.finfo(torch.bfloat16).eps / 2  # one rounding to bf16, relative


def rope_ref(x, positions, inv_freq, interleaved, amplitude=1.0, inverse=False):
    """x [B,H,S,D] (any type) -> fp64, the pairs of the first 2 len(inv_freq) elements
    turned by positions [B,S] * inv_freq."""
    y = x.double().clone()
    n = inv_freq.numel()
    if n == 0:
        return y
    ang = positions.double()[:, None, :, None] * inv_freq.double()
    c, s = torch.cos(ang) * amplitude, torch.sin(ang) * amplitude * (-1 if inverse else 1)
    i = torch.arange(n)
    i, j = (2 * i, 2 * i + 1) if interleaved else (i, i + n)
    a, b = x.double()[..., i], x.double()[..., j]
    y[..., i], y[..., j] = a * c - b * s, b * c + a * s
    return y


def rope_tol(x, n, interleaved, amplitude=1.0):
    """Elementwise bound on a rotated element: half a bf16 step of the result (its size
    is at most A (|a| + |b|)), and 2^-19 of A (|a| + |b|) for cosine, sine, the reduced
    angle in 32 bits (2^-24 turns, times 2 pi) and three fp32 roundings."""
    y = torch.zeros_like(x, dtype=torch.float64)
    if n:
        i = torch.arange(n)
        i, j = (2 * i, 2 * i + 1) if interleaved else (i, i + n)
        size = amplitude * (x.double()[..., i].abs() + x.double()[..., j].abs())
        y[..., i], y[..., j] = size, size
    return y * 2.0 ** -19


def assert_rope(got, x, positions, inv_freq, interleaved, amplitude=1.0, inverse=False):
    ref = rope_ref(x, positions, inv_freq, interleaved, amplitude, inverse)
    tol = HALF_BF16 * ref.abs() + rope_tol(x, inv_freq.numel(), interleaved, amplitude)
    err = (got.cpu().double() - ref).abs()
    assert bool((err <= tol).all()), f"max error {err.max():.3e}, worst excess {(err - tol).max():.3e}"
    rest = 2 * inv_freq.numel()
    assert torch.equal(got.cpu()[..., rest:], x[..., rest:].cpu())


def decode_ref(q, k_pages, v_pages, table, lens, window=None, score=None, scale=None):
    """fp64 (o, lse, tol_o, tol_lse).  Bounds: a score's 32-bit error e is at most
    D 2^-23 of the products' summed size (truncating adds) plus 2^-16 for the score_mod
    and the exponent's argument; a weight is then off by e, the sum of the row by e, and
    P's rounding to bf16 by half a step: |dO| <= (half + 2 e + 2^-18) sum p |v| +
    half |O|, |dLSE| <= e + 2^-18."""
    B, Hq, n, D = q.shape
    Hkv = k_pages.shape[1]
    G = Hq // Hkv
    scale = 1 / math.sqrt(D) if scale is None else scale
    o = torch.zeros((B, Hq, n, D), dtype=torch.float64)
    lse = torch.full((B, Hq, n), -math.inf, dtype=torch.float64)
    to, tl = torch.zeros_like(o), torch.zeros_like(lse)
    for b in range(B):
        L = int(lens[b])
        if L == 0:
            continue
        pages = table[b, :(L + PAGE - 1) // PAGE].long()
        k = k_pages[pages].double().permute(1, 0, 2, 3).reshape(Hkv, -1, D)[:, :L]
        v = v_pages[pages].double().permute(1, 0, 2, 3).reshape(Hkv, -1, D)[:, :L]
        for i in range(n):
            pos = L - n + i
            lo = 0 if window is None else max(0, pos - window)
            if pos < 0:
                continue
            for h in range(Hq):
                kk, vv, qq = k[h // G, lo:pos + 1], v[h // G, lo:pos + 1], q[b, h, i].double()
                x = scale * (kk @ qq)
                e = D * 2.0 ** -23 * scale * float((kk.abs() @ qq.abs()).max()) + 2.0 ** -16
                if score is not None and score[0] == "alibi":
                    x = x + float(score[1][h]) * (torch.arange(lo, pos + 1) - pos).double()
                elif score is not None and score[0] == "softcap":
                    x = score[1] * torch.tanh(x / score[1])
                p = torch.softmax(x, 0)
                o[b, h, i] = p @ vv
                lse[b, h, i] = torch.logsumexp(x, 0)
                to[b, h, i] = (HALF_BF16 + 2 * e + 2.0 ** -18) * (p @ vv.abs()) + HALF_BF16 * o[b, h, i].abs()
                tl[b, h, i] = e + 2.0 ** -18
    return o, lse, to, tl


def assert_decode(got, ref, what=""):
    o, lse = got[0].cpu().double(), got[1].cpu().double()
    ro, rl, to, tl = ref
    err = (o - ro).abs()
    assert bool((err <= to).all()), f"{what}: O off by {err.max():.3e}, worst excess {(err - to).max():.3e}"
    empty = torch.isinf(rl)
    assert torch.equal(torch.isneginf(lse), empty), f"{what}: rows with LSE = -inf differ"
    lerr = (lse - rl).abs()[~empty]
    assert bool((lerr <= tl[~empty]).all()), f"{what}: LSE off by {lerr.max():.3e}"


def paged_case(lens, q_len, Hq, Hkv, D, seed, width=None, prefix=0, filler=0.0):
    """Inputs of a paged decode (CPU): q, k_pages, v_pages, table, lens.  Every sequence's
    first `prefix` keys (whole pages) are the same pages; slots behind the last key hold
    `filler`, table entries behind the last page an arbitrary page of the pool."""
    g = torch.Generator().manual_seed(seed)
    B, first = len(lens), prefix // PAGE
    own = [max(0, (n + PAGE - 1) // PAGE - first) for n in lens]
    width = max([first + n for n in own] + [width or 0])
    num = sum(own) + first + 3
    order = torch.randperm(num, generator=g).to(torch.int32)
    table = torch.randint(0, num, (B, width), generator=g).to(torch.int32)
    k = torch.randn((num, Hkv, PAGE, D), generator=g).to(torch.bfloat16)
    v = torch.randn((num, Hkv, PAGE, D), generator=g).to(torch.bfloat16)
    at = first
    for b in range(B):
        table[b, :first] = order[:first]
        table[b, first:first + own[b]] = order[at:at + own[b]]
        at += own[b]
        if own[b] and lens[b] % PAGE:
            last = int(table[b, first + own[b] - 1])
            k[last, :, lens[b] % PAGE:] = filler
            v[last, :, lens[b] % PAGE:] = filler
    for p in order[at:].tolist():
        k[p], v[p] = filler, filler
    q = torch.randn((B, Hq, q_len, D), generator=g).to(torch.bfloat16)
    return q, k, v, table, torch.tensor(lens, dtype=torch.int32)
