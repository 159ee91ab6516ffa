"""Measured cases of the serving and rotary operators.

Four operators that belong together around a paged key / value cache:

  rope    rotary positions on Q and K (half and interleaved pairs, part of the
          head, frequencies of long contexts), and the rotation of their gradients
  append  new keys and values of a ragged batch into the page pools, K (and Q)
          rotated on the way
  decode  a few query tokens per sequence against the paged cache, every sequence
          with its own length
  shared  the same for a batch whose sequences share their first pages: the
          prefix is taken once for all

Cases are dicts of plain values.  `run` computes a case in its plain form
(elementary torch operations, in 32 bits, angles in 64) or, where `own` is true,
through the package's entry points; `exact` computes it from the definition in
64 bits.  Sequence lengths are a fixed ragged pattern between the case's bounds,
dealt to the batch by the seed, so `work` can count them.
"""

import math

import torch

own = False

PAGE = 128


# ---------------------------------------------------------------- cases

def listed():
    return [
        # one decoding step's Q and K at far positions of a long context (frequencies
        # divided by a factor): latency
        dict(name="rope_step_b8_h32", op="rope", B=8, Hq=32, Hkv=8, S=1, D=128, rotary=128, interleaved=False,
             token_major=True, far=1000000, factor=8.0, amplitude=1.0, grad=False),
        # training: the headline attention workload's Q and K with interleaved pairs,
        # forward and the gradients' way back
        dict(name="rope_train_b4_h16_s2048", op="rope", B=4, Hq=16, Hkv=16, S=2048, D=64, rotary=64, interleaved=True,
             token_major=False, far=0, factor=1.0, amplitude=1.0, grad=True),
        # a long prompt, half of every head rotated, Q and K as a projection leaves them
        # (token-major), an odd length
        dict(name="rope_long_s16383", op="rope", B=1, Hq=32, Hkv=8, S=16383, D=128, rotary=64, interleaved=False,
             token_major=True, far=100000, factor=4.0, amplitude=1.1, grad=False),
        # one decoding step: every sequence appends one token and rotates its query
        dict(name="append_step_b8", op="append", B=8, Hq=32, Hkv=8, S=1, D=128, rotary=128, interleaved=False,
             new_min=1, cache_min=100, cache_max=1900),
        # a ragged batch of prompts appended behind caches that end inside a page
        dict(name="append_prompts_s4000", op="append", B=4, Hq=32, Hkv=8, S=4000, D=128, rotary=128,
             interleaved=False, new_min=777, cache_min=1, cache_max=300),
        # a single short conversation: latency
        dict(name="decode_one_kv700", op="decode", B=1, Hq=16, Hkv=16, q_len=1, D=64, kv_min=700, kv_max=700,
             window=0, score="alibi"),
        # a serving batch of very unequal lengths, one slot of it empty
        dict(name="decode_ragged_b16", op="decode", B=16, Hq=32, Hkv=8, q_len=1, D=128, kv_min=0, kv_max=8191,
             window=0, score="none"),
        # four drafted tokens a step, a sliding window and soft-capped scores
        dict(name="decode_draft_window", op="decode", B=24, Hq=16, Hkv=8, q_len=4, D=64, kv_min=500, kv_max=16384,
             window=4096, score="softcap"),
        # the longest caches: bound by reading them
        dict(name="decode_long_b8_kv32k", op="decode", B=8, Hq=32, Hkv=8, q_len=1, D=128, kv_min=24001, kv_max=32768,
             window=0, score="none"),
        # a few requests behind one short system prompt
        dict(name="shared_b4_p512", op="shared", B=4, Hq=16, Hkv=4, q_len=1, D=64, prefix=512, kv_min=1, kv_max=130,
             score="none"),
        # a serving batch behind a document of 4096 tokens
        dict(name="shared_b32_p4096", op="shared", B=32, Hq=32, Hkv=8, q_len=1, D=128, prefix=4096, kv_min=17,
             kv_max=600, score="none"),
        # many samples of one long prompt: the prefix is a matrix product
        dict(name="shared_b128_p16384", op="shared", B=128, Hq=32, Hkv=8, q_len=1, D=128, prefix=16384, kv_min=128,
             kv_max=777, score="none"),
    ]


def _log(rng, lo, hi):
    """A whole number between lo and hi, spread over its logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["rope", "append", "decode", "decode", "shared", "shared"])
    D = rng.choice([64, 128])
    Hkv = rng.choice([1, 2, 4, 8, 16])
    G = rng.choice([1, 2, 4, 8])
    Hq = Hkv * G if Hkv * G <= 32 else 32
    if op == "rope":
        B = _log(rng, 1, 8)
        S = _log(rng, 1, max(1, 655320 // (B * (Hq + Hkv))))
        return dict(op=op, B=B, Hq=Hq, Hkv=Hkv, S=S, D=D, rotary=16 * rng.randint(1, D // 16),
                    interleaved=rng.random() < 0.5, token_major=rng.random() < 0.5, far=rng.choice([0, 5000, 1000000]),
                    factor=rng.choice([1.0, 4.0, 32.0]), amplitude=rng.choice([1.0, 1.1]),
                    grad=S < 6000 and rng.random() < 0.4)
    if op == "append":
        B = _log(rng, 1, 32)
        S = _log(rng, 1, max(1, 600000 // (B * (Hq + 2 * Hkv))))
        lo = rng.randint(0, 200)
        return dict(op=op, B=B, Hq=Hq, Hkv=Hkv, S=S, D=D, rotary=16 * rng.randint(0, D // 16),
                    interleaved=rng.random() < 0.5, new_min=rng.randint(0, S), cache_min=lo,
                    cache_max=lo + rng.randint(0, 1500))
    G = Hq // Hkv
    q_len = rng.randint(1, max(1, min(5, 16 // G)))
    score = rng.choice(["none", "none", "alibi", "softcap"])
    if op == "decode":
        B = _log(rng, 1, 64)
        top = _log(rng, 20, min(65536, 220000000 // (B * Hkv * D)))
        return dict(op=op, B=B, Hq=Hq, Hkv=Hkv, q_len=q_len, D=D, kv_min=rng.randint(0, top), kv_max=top,
                    window=rng.choice([0, 0, 0, _log(rng, 1, 4096)]), score=score)
    B = _log(rng, 2, 128)
    top = _log(rng, q_len, 700)
    most = min(128, 128 * 32 * 128 * 128 // (B * Hq * q_len * D))  # pages of the prefix
    return dict(op=op, B=B, Hq=Hq, Hkv=Hkv, q_len=q_len, D=D, prefix=PAGE * _log(rng, 1, most),
                kv_min=rng.randint(q_len, top), kv_max=top, score=score)


def _lengths(n, lo, hi):
    """n lengths between lo and hi, both among them, unequal in between."""
    if n == 1:
        return [hi]
    frac = [(0.6180339887498949 * i) % 1.0 for i in range(n - 2)]
    return [lo, hi] + [lo + int((hi - lo) * f) for f in frac]


def _pages(n):
    return (n + PAGE - 1) // PAGE


# ---------------------------------------------------------------- inputs

def _inv_freq(rotary, factor, device):
    j = torch.arange(0, rotary, 2, dtype=torch.float64, device=device)
    return 10000.0 ** (-j / max(rotary, 1)) / factor


def _heads(gen, B, H, S, D, token_major, device):
    """bf16 N(0, 1), [B, H, S, D]: contiguous, or a view of a token-major tensor."""
    if token_major:
        return torch.randn((B, S, H, D), generator=gen, device=device).to(torch.bfloat16).transpose(1, 2)
    return torch.randn((B, H, S, D), generator=gen, device=device).to(torch.bfloat16)


def _table(gen, counts, width, device):
    """Page table int32 [B, width] over a shuffled pool: the first counts[b] entries of
    row b are its pages, the others 0.  Returns it and the pool's size."""
    total = sum(counts)
    num = total + max(1, total // 16)
    order = torch.randperm(num, generator=gen, device=device).to(torch.int32)
    table = torch.zeros((len(counts), width), dtype=torch.int32, device=device)
    at = 0
    for b, n in enumerate(counts):
        table[b, :n] = order[at:at + n]
        at += n
    return table, num, order[at:]


def _dealt(values, seed):
    """The values in an order of the seed's."""
    order = torch.randperm(len(values), generator=torch.Generator().manual_seed(seed + 77)).tolist()
    return [values[i] for i in order]


def _i32(values, device):
    return torch.tensor(values, dtype=torch.int32, device=device)


def _score(case, device):
    if case["score"] == "alibi":
        H = case["Hq"]
        return ("alibi", torch.tensor([2.0 ** (-8.0 * (h + 1) / H) for h in range(H)], dtype=torch.float32,
                                      device=device))
    return ("softcap", 30.0) if case["score"] == "softcap" else None


def prepare(case, seed):
    device = torch.device("cuda")
    gen = torch.Generator(device=device).manual_seed(seed)
    B, Hq, Hkv, D = case["B"], case["Hq"], case["Hkv"], case["D"]
    s = {"case": case}
    if case["op"] == "rope":
        S, tm = case["S"], case["token_major"]
        s["q"], s["k"] = _heads(gen, B, Hq, S, D, tm, device), _heads(gen, B, Hkv, S, D, tm, device)
        if case["grad"]:
            s["gq"], s["gk"] = _heads(gen, B, Hq, S, D, tm, device), _heads(gen, B, Hkv, S, D, tm, device)
        first = torch.randint(0, case["far"] + 1, (B, 1), generator=gen, device=device)
        s["positions"] = (first + torch.arange(S, device=device)).to(torch.int32)
        s["inv_freq"] = _inv_freq(case["rotary"], case["factor"], device)
        return s
    if case["op"] == "append":
        S = case["S"]
        # the projection's output: Q, K and V of a token side by side
        qkv = torch.randn((B, S, Hq + 2 * Hkv, D), generator=gen, device=device).to(torch.bfloat16).transpose(1, 2)
        s["q"], s["k"], s["v"] = qkv[:, :Hq], qkv[:, Hq:Hq + Hkv], qkv[:, Hq + Hkv:]
        s["q_out"] = torch.zeros((B, Hq, S, D), dtype=torch.bfloat16, device=device)
        cache = _dealt(_lengths(B, case["cache_min"], case["cache_max"]), seed)
        s["cache_lens"] = _i32(cache, device)
        s["new_lens"] = _i32(_dealt(_lengths(B, case["new_min"], S), seed + 1), device)
        counts = [_pages(c + S) for c in cache]
        s["page_table"], num, _ = _table(gen, counts, max(counts), device)
        s["inv_freq"] = _inv_freq(case["rotary"], 1.0, device)
    else:
        q_len = case["q_len"]
        lens = _dealt(_lengths(B, case["kv_min"], case["kv_max"]), seed)
        first = case.get("prefix", 0)
        counts = [max(1, _pages(n)) for n in lens]
        table, num, spare = _table(gen, counts, max(counts), device)
        if first:
            shared = torch.arange(num, num + first // PAGE, dtype=torch.int32, device=device)
            shared = shared[torch.randperm(first // PAGE, generator=gen, device=device)]
            table = torch.cat([shared.expand(B, -1), table], dim=1).contiguous()
            num += first // PAGE
        s["page_table"] = table
        s["seq_lens"] = _i32([first + n for n in lens], device)
        s["q"] = _heads(gen, B, Hq, q_len, D, True, device)
        s["score_mod"] = _score(case, device)
    s["k_pages"] = torch.randn((num, Hkv, PAGE, D), generator=gen, device=device).to(torch.bfloat16)
    s["v_pages"] = torch.randn((num, Hkv, PAGE, D), generator=gen, device=device).to(torch.bfloat16)
    return s


# ---------------------------------------------------------------- one pass

def run(s):
    return {"rope": _rope, "append": _append, "decode": _decode, "shared": _shared}[s["case"]["op"]](s)


def _cos_sin(positions, inv_freq, amplitude):
    """fp32 [B, 1, S, rotary / 2], from angles in 64 bits."""
    angle = positions.to(torch.float64)[:, None, :, None] * inv_freq
    return (amplitude * torch.cos(angle)).float(), (amplitude * torch.sin(angle)).float()


def _rotate(x, cos, sin, interleaved):
    """Rotated bf16 x [B, H, S, D]: pairs of the first 2 * cos.shape[-1] elements."""
    half = cos.shape[-1]
    r, rest = x[..., :2 * half].float(), x[..., 2 * half:]
    a, b = (r[..., 0::2], r[..., 1::2]) if interleaved else (r[..., :half], r[..., half:])
    lo, hi = a * cos - b * sin, b * cos + a * sin
    y = torch.stack([lo, hi], dim=-1).flatten(-2) if interleaved else torch.cat([lo, hi], dim=-1)
    return torch.cat([y.to(x.dtype), rest], dim=-1)


def _rope(s):
    c = s["case"]
    if own:
        import block_sparse_attention_48_b200 as fa
        opts = dict(positions=s["positions"], interleaved=c["interleaved"], amplitude=c["amplitude"])
        out = fa.rope_apply(s["q"], s["k"], s["inv_freq"], **opts)
        if c["grad"]:
            out = out + fa.rope_apply(s["gq"], s["gk"], s["inv_freq"], inverse=True, **opts)
        return out
    cos, sin = _cos_sin(s["positions"], s["inv_freq"], c["amplitude"])
    out = _rotate(s["q"], cos, sin, c["interleaved"]), _rotate(s["k"], cos, sin, c["interleaved"])
    if c["grad"]:
        out = out + (_rotate(s["gq"], cos, -sin, c["interleaved"]), _rotate(s["gk"], cos, -sin, c["interleaved"]))
    return out


def _append(s):
    c = s["case"]
    if own:
        import block_sparse_attention_48_b200 as fa
        fa.paged_append(s["k"], s["v"], s["k_pages"], s["v_pages"], s["page_table"], s["cache_lens"],
                        new_lens=s["new_lens"], q=s["q"], q_out=s["q_out"], inv_freq=s["inv_freq"],
                        interleaved=c["interleaved"])
        return s["q_out"], s["k_pages"], s["v_pages"]
    new = torch.arange(c["S"], device=s["q"].device)
    pos = s["cache_lens"][:, None].long() + new
    valid = (new < s["new_lens"][:, None])[:, :, None, None]
    cos, sin = _cos_sin(pos, s["inv_freq"], 1.0)
    s["q_out"].copy_(torch.where(valid.transpose(1, 2), _rotate(s["q"], cos, sin, c["interleaved"]), s["q_out"]))
    page, slot = s["page_table"].long().gather(1, pos // PAGE), pos % PAGE
    for pages, x in ((s["k_pages"], _rotate(s["k"], cos, sin, c["interleaved"])), (s["v_pages"], s["v"])):
        pages[page, :, slot] = torch.where(valid, x.transpose(1, 2), pages[page, :, slot])
    return s["q_out"], s["k_pages"], s["v_pages"]


def _modified(x, score_mod, kv, pos):
    """score_mod of scores x [B, Hkv, G, q_len, keys] at key positions kv and query positions pos."""
    if score_mod is None:
        return x
    if score_mod[0] == "softcap":
        return score_mod[1] * torch.tanh(x / score_mod[1])
    slopes = score_mod[1].view(1, x.shape[1], x.shape[2], 1, 1)
    return x + slopes * (kv - pos).to(x.dtype)[:, None, None]


def _own_keys(pages, table):
    """fp32 [B, Hkv, keys, D] of the pages that the table's rows name."""
    x = pages[table.long()].float()
    return x.transpose(1, 2).flatten(2, 3)


def _softmax_pv(x, v_of):
    """Rows' softmax of x (masked places -inf; a row with nothing else gives 0), its
    product with the values and the natural-log sum."""
    m = x.amax(dim=-1, keepdim=True)
    e = torch.exp(x - torch.where(torch.isinf(m), torch.zeros_like(m), m))
    z = e.sum(dim=-1, keepdim=True)
    o = v_of(e) / torch.where(z > 0, z, torch.ones_like(z))
    return o, (m + torch.log(z)).squeeze(-1)


def _decode(s):
    c = s["case"]
    if own:
        import block_sparse_attention_48_b200 as fa
        return fa.flex_decode_paged(s["q"], s["k_pages"], s["v_pages"], s["page_table"], s["seq_lens"],
                                    window=c["window"] or None, score_mod=s["score_mod"])
    B, Hq, Hkv, n, D = c["B"], c["Hq"], c["Hkv"], c["q_len"], c["D"]
    q = s["q"].float().reshape(B, Hkv, Hq // Hkv * n, D)
    k, v = _own_keys(s["k_pages"], s["page_table"]), _own_keys(s["v_pages"], s["page_table"])
    kv = torch.arange(k.shape[2], device=q.device)
    pos = (s["seq_lens"][:, None].long() - n + torch.arange(n, device=q.device))[:, :, None]
    x = (torch.matmul(q, k.transpose(2, 3)) / math.sqrt(D)).view(B, Hkv, Hq // Hkv, n, -1)
    x = _modified(x, s["score_mod"], kv, pos)
    seen = kv <= pos
    if c["window"]:
        seen = seen & (pos - kv <= c["window"])
    x = torch.where(seen[:, None, None], x, float("-inf"))
    o, lse = _softmax_pv(x.flatten(2, 3), lambda e: torch.matmul(e, v))
    return o.reshape(B, Hq, n, D).to(torch.bfloat16), lse.reshape(B, Hq, n)


def _shared(s):
    c = s["case"]
    if own:
        import block_sparse_attention_48_b200 as fa
        return fa.flex_decode_shared(s["q"], s["k_pages"], s["v_pages"], s["page_table"], s["seq_lens"], c["prefix"],
                                     score_mod=s["score_mod"])
    B, Hq, Hkv, n, D, P = c["B"], c["Hq"], c["Hkv"], c["q_len"], c["D"], c["prefix"]
    G, first = Hq // Hkv, c["prefix"] // PAGE
    q = s["q"].float().reshape(B, Hkv, G * n, D)
    # the prefix once, its rows those of every sequence
    k0 = _own_keys(s["k_pages"], s["page_table"][:1, :first])[0]
    v0 = _own_keys(s["v_pages"], s["page_table"][:1, :first])[0]
    k1, v1 = _own_keys(s["k_pages"], s["page_table"][:, first:]), _own_keys(s["v_pages"], s["page_table"][:, first:])
    x0 = torch.matmul(q.transpose(0, 1).reshape(Hkv, B * G * n, D), k0.transpose(1, 2))
    x0 = x0.view(Hkv, B, G * n, P).transpose(0, 1)
    x = (torch.cat([x0, torch.matmul(q, k1.transpose(2, 3))], dim=-1) / math.sqrt(D)).view(B, Hkv, G, n, -1)
    kv = torch.arange(x.shape[-1], device=q.device)
    pos = (s["seq_lens"][:, None].long() - n + torch.arange(n, device=q.device))[:, :, None]
    x = torch.where((kv <= pos)[:, None, None], _modified(x, s["score_mod"], kv, pos), float("-inf"))

    def values(e):
        e0 = e[..., :P].transpose(0, 1).reshape(Hkv, B * G * n, P)
        return torch.matmul(e0, v0).view(Hkv, B, G * n, D).transpose(0, 1) + torch.matmul(e[..., P:], v1)
    o, lse = _softmax_pv(x.flatten(2, 3), values)
    return o.reshape(B, Hq, n, D).to(torch.bfloat16), lse.reshape(B, Hq, n)


# ---------------------------------------------------------------- what a pass cannot do without

def work(case):
    B, Hq, Hkv, D = case["B"], case["Hq"], case["Hkv"], case["D"]
    if case["op"] == "rope":
        rows = B * case["S"] * (Hq + Hkv) * (2 if case["grad"] else 1)
        return {"bytes": rows * D * 4 + B * case["S"] * 4, "flops": rows * case["rotary"] * 3}
    if case["op"] == "append":
        new = sum(_lengths(B, case["new_min"], case["S"]))
        return {"bytes": new * (Hq + 2 * Hkv) * D * 4 + new / PAGE * 4, "flops": new * (Hq + Hkv) * case["rotary"] * 3}
    n, first, window = case["q_len"], case.get("prefix", 0), case.get("window", 0)
    keys, pairs = first, 0
    for own_len in _lengths(B, case["kv_min"], case["kv_max"]):
        end = first + own_len
        keys += own_len if not window else min(own_len, window + n)
        for i in range(n):
            pos = end - n + i
            if pos >= 0:
                pairs += pos + 1 if not window else min(pos, window) + 1
    return {"bytes": keys * Hkv * D * 4 + B * Hq * n * (D * 4 + 4), "flops": 4 * D * Hq * pairs}


# ---------------------------------------------------------------- the definition in 64 bits

def exact(case, seed):
    s = prepare(case, seed)
    f = torch.float64
    if case["op"] in ("rope", "append"):
        positions = s["positions"] if case["op"] == "rope" else \
            s["cache_lens"][:, None] + torch.arange(case["S"], device=s["q"].device)
        rot = case["rotary"]
        # the pairs (i, j) of the head's elements, each turned by position * inv_freq
        i = torch.arange(rot // 2, device=s["q"].device)
        i, j = (2 * i, 2 * i + 1) if case["interleaved"] else (i, i + rot // 2)
        turn = torch.polar(torch.full((1,), case.get("amplitude", 1.0), dtype=f, device=i.device),
                           positions.to(f).unsqueeze(-1) * s["inv_freq"]).unsqueeze(1)

        def turned(x, way):
            y = x.to(f)
            z = torch.complex(y[..., i], y[..., j]) * (turn if way > 0 else turn.conj())
            y[..., i], y[..., j] = z.real, z.imag
            return y
        if case["op"] == "rope":
            out = turned(s["q"], 1), turned(s["k"], 1)
            return out + (turned(s["gq"], -1), turned(s["gk"], -1)) if case["grad"] else out
        q, k = turned(s["q"], 1), turned(s["k"], 1)
        q_out, kp, vp = s["q_out"].to(f), s["k_pages"].to(f), s["v_pages"].to(f)
        cache, new, table = s["cache_lens"].tolist(), s["new_lens"].tolist(), s["page_table"].tolist()
        for b in range(case["B"]):
            q_out[b, :, :new[b]] = q[b, :, :new[b]]
            t = 0
            while t < new[b]:  # page by page
                at = (cache[b] + t) % PAGE
                n = min(PAGE - at, new[b] - t)
                page = table[b][(cache[b] + t) // PAGE]
                kp[page, :, at:at + n] = k[b, :, t:t + n]
                vp[page, :, at:at + n] = s["v"][b, :, t:t + n].to(f)
                t += n
        return q_out, kp, vp
    B, Hq, Hkv, n, D = case["B"], case["Hq"], case["Hkv"], case["q_len"], case["D"]
    G = Hq // Hkv
    out = torch.zeros((B, Hq, n, D), dtype=f, device=s["q"].device)
    lse = torch.full((B, Hq, n), -math.inf, dtype=f, device=s["q"].device)
    lens = s["seq_lens"].tolist()
    for b in range(B):
        L = lens[b]
        pages = s["page_table"][b, :_pages(L)].long()
        k = s["k_pages"][pages].to(f).permute(1, 0, 2, 3).reshape(Hkv, -1, D)[:, :L]
        v = s["v_pages"][pages].to(f).permute(1, 0, 2, 3).reshape(Hkv, -1, D)[:, :L]
        for t in range(n):
            pos = L - n + t
            lo = max(0, pos - case["window"]) if case.get("window") else 0
            if pos < 0:
                continue
            x = torch.einsum("hgd,hkd->hgk", s["q"][b, :, t].to(f).view(Hkv, G, D), k[:, lo:pos + 1]) / math.sqrt(D)
            if case["score"] == "softcap":
                x = 30.0 * torch.tanh(x / 30.0)
            elif case["score"] == "alibi":
                slopes = s["score_mod"][1].to(f).view(Hkv, G, 1)
                x = x + slopes * (torch.arange(lo, pos + 1, device=x.device) - pos).to(f)
            out[b, :, t] = torch.einsum("hgk,hkd->hgd", torch.softmax(x, dim=-1), v[:, lo:pos + 1]).reshape(Hq, D)
            lse[b, :, t] = torch.logsumexp(x, dim=-1).reshape(Hq)
    return out, lse
