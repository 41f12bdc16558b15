"""Rotary positions, the append that applies them, and the paged 4-bit cache.

Five operators of a serving step over a pool of cache pages:

  * angles: cosine and sine of every new token's rotary angles, once a step for
    all layers, frequencies scaled for long contexts;
  * rotate: queries or keys turned by those angles, half and interleaved
    layouts, all or a part of the head;
  * append: new keys and values into E4M3 pages, the keys (and the step's
    queries) rotated on the way;
  * append4: the same into 4-bit pages (for each token, kv head and group of 32
    channels a step and a minimum in fp16, and 4-bit codes), and the new tokens
    read back as the values that their codes stand for;
  * attention4: attention over the 4-bit pages, for one or a few new tokens of
    each request ("decode") and for prompts and chunks of prompts.

Frequencies are whole numbers: the part of a turn that a pair of channels moves
in one position, in units of 2^-64 turns, so that a position times a frequency
modulo 2^64 is the exact angle, however far the position.
"""
import math
import random

import numpy as np
import torch

own = False

TYPES = {"fp16": torch.float16, "bf16": torch.bfloat16}
MIN_EXP, MAX_EXP = -15, 40  # exponents of the smallest and largest scale of an E4M3 page
GROUP = 32  # channels of a 4-bit group


# ---------------------------------------------------------------- cases

def listed():
    return [
        # a decode step's angles, every request at its own place, far into its context: latency counts
        dict(name="angles-decode-b64", op="angles", tokens=64, rot=128, scaled=False, max_pos=131072, lens=1),
        # the angles of every position of a long context, frequencies scaled for it
        dict(name="angles-131072", op="angles", tokens=131072, rot=128, scaled=True, max_pos=131072, lens=0),
        # the queries of a decode step
        dict(name="rotate-decode-b64", op="rotate", tokens=64, heads=32, dim=128, rot=128, inter=False, scaled=False,
             dtype="fp16", max_pos=131072, lens=1),
        # the queries of a prefill step, half of the head, interleaved pairs
        dict(name="rotate-prompts-part", op="rotate", tokens=16003, heads=40, dim=128, rot=64, inter=True, scaled=True,
             dtype="bf16", max_pos=32768, lens=2),
        # a large decode batch: the new token of every request, with its queries
        dict(name="append-decode-t256", op="append", batch=256, q_heads=32, kv_heads=8, dim=128, rot=128, inter=False,
             scaled=False, page=64, dtype="fp16", max_ctx=2048, max_new=1, lens=3),
        # the prompts of one prefill step
        dict(name="append-prompts-bf16", op="append", batch=8, q_heads=32, kv_heads=8, dim=128, rot=128, inter=False,
             scaled=True, page=64, dtype="bf16", max_ctx=0, max_new=7001, lens=4),
        # a decode batch into 4-bit pages
        dict(name="append4-decode-t64", op="append4", batch=64, q_heads=32, kv_heads=8, dim=128, rot=128, inter=False,
             scaled=False, page=64, dtype="fp16", max_ctx=8192, max_new=1, lens=5),
        # ragged chunks behind earlier tokens, narrow heads, small pages, a quarter of the head rotated
        dict(name="append4-chunks-d64", op="append4", batch=7, q_heads=32, kv_heads=32, dim=64, rot=16, inter=True,
             scaled=False, page=16, dtype="bf16", max_ctx=777, max_new=1003, lens=6),
        # the smallest attention: one short request, two heads
        dict(name="decode4-tiny", op="attention4", batch=1, q_heads=2, kv_heads=2, dim=64, page=16, dtype="fp16",
             max_ctx=256, max_new=1, window=0, lens=0),
        # a ragged serving batch with shared heads
        dict(name="decode4-b64-gqa4", op="attention4", batch=64, q_heads=32, kv_heads=8, dim=128, page=32,
             dtype="bf16", max_ctx=2047, max_new=1, window=0, lens=7),
        # one long sequence
        dict(name="decode4-131072", op="attention4", batch=1, q_heads=32, kv_heads=8, dim=128, page=128,
             dtype="fp16", max_ctx=131071, max_new=1, window=0, lens=0),
        # a chunk of a long prompt behind what is cached already
        dict(name="chunk4-2048-of-34816", op="attention4", batch=1, q_heads=32, kv_heads=8, dim=128, page=64,
             dtype="fp16", max_ctx=32768, max_new=2048, window=0, lens=0),
    ]


def _between(rng, lo, hi):
    """A whole number of [lo, hi], spread over its logarithm."""
    return max(lo, min(hi, int(math.exp(rng.uniform(math.log(lo), math.log(hi + 1))))))


def draw(rng):
    lens = rng.randrange(1, 1 << 30)
    op = rng.choice(("angles", "rotate", "append", "append4", "append4", "attention4", "attention4", "attention4"))
    dtype = rng.choice(("fp16", "bf16"))
    if op == "angles":
        return dict(op=op, tokens=_between(rng, 1, 131072), rot=2 * _between(rng, 1, 64), scaled=rng.random() < 0.5,
                    max_pos=_between(rng, 1, 1 << 20), lens=lens)
    if op == "rotate":
        while True:
            tokens, heads, dim = _between(rng, 1, 65536), _between(rng, 1, 64), rng.choice((64, 80, 96, 128, 256))
            if tokens * heads * dim <= 16003 * 40 * 128:
                rot = rng.choice((dim, dim, dim // 2, 2 * rng.randint(1, dim // 2)))
                return dict(op=op, tokens=tokens, heads=heads, dim=dim, rot=rot, inter=rng.random() < 0.5,
                            scaled=rng.random() < 0.5, dtype=dtype, max_pos=_between(rng, 1, 1 << 20), lens=lens)
    dim, page, kv = rng.choice((64, 128)), rng.choice((16, 32, 64, 128)), rng.choice((1, 2, 3, 4, 8, 12, 32))
    heads = kv * rng.choice((1, 2, 4, 5, 8))
    while True:
        batch, ctx = _between(rng, 1, 256), _between(rng, 1, 65536)
        new = rng.choice((1, 1, _between(rng, 2, 8), _between(rng, 9, 4096)))
        if rng.random() < 0.2:
            ctx = 0
        if op != "attention4":
            # as many bytes as the largest listed append at most, and a pool of a few GB
            if batch * new * (heads + 2 * kv) * dim <= 16e7 and batch * (ctx + new) * kv * dim <= 1 << 29:
                rot = rng.choice((dim, dim, dim // 2, 2 * rng.randint(1, dim // 2)))
                return dict(op=op, batch=batch, q_heads=heads, kv_heads=kv, dim=dim, rot=rot,
                            inter=rng.random() < 0.5, scaled=rng.random() < 0.5, page=page, dtype=dtype, max_ctx=ctx,
                            max_new=new, lens=lens)
            continue
        window = rng.choice((0, 0, 0, _between(rng, 16, 4096)))
        # the scores of the largest listed case at most, and a cache of a few GB
        if batch * heads * new * (ctx + new) <= 32 * 2048 * 34816 and batch * (ctx + new) * kv * dim <= 3e8 \
                and batch * new * heads * dim <= 1e8:
            return dict(op=op, batch=batch, q_heads=heads, kv_heads=kv, dim=dim, page=page, dtype=dtype, max_ctx=ctx,
                        max_new=new, window=window, lens=lens)


def _lengths(case):
    """Cached and new tokens of each request: all the largest where `lens` is
    0, else ragged (the first request takes the largest)."""
    B, ctx, new = case["batch"], case["max_ctx"], case["max_new"]
    if case["lens"] == 0:
        return [ctx] * B, [new] * B
    r = random.Random(case["lens"])
    cs = [ctx] + [r.randint(ctx // 8, ctx) for _ in range(B - 1)]
    ns = [new] + [r.randint(min(new, 1 + new // 8), new) for _ in range(B - 1)]
    return cs, ns


def work(case):
    if case["op"] == "angles":
        return {"bytes": 4 * case["tokens"] * (1 + case["rot"]) + 4 * case["rot"], "flops": 0}
    if case["op"] == "rotate":
        n = case["tokens"] * case["heads"]
        return {"bytes": 4 * n * case["dim"] + 4 * case["tokens"] * case["rot"], "flops": 3 * n * case["rot"]}
    cs, ns = _lengths(case)
    T, h, d, q = sum(ns), case["kv_heads"], case["dim"], case["q_heads"]
    if case["op"] != "attention4":
        turned = 4 * T * q * d + 4 * T + 4 * T * case["rot"]  # queries in and out, slots, angles
        flops = 3 * T * (q + h) * case["rot"] + 4 * T * h * d
        if case["op"] == "append":
            pages = sum(-(-(c + n) // case["page"]) - c // case["page"] for c, n in zip(cs, ns))
            return {"bytes": turned + T * h * d * 2 * (2 + 1) + 8 * pages * h, "flops": flops}
        # 16-bit keys and values in, 5 bits a value written, read back, and 16 bits out
        return {"bytes": turned + 4 * T + T * h * d * 2 * (2 + 0.625 + 0.625 + 2), "flops": flops + 4 * T * h * d}
    w = case["window"] or 1 << 60
    pairs = seen = 0
    for c, n in zip(cs, ns):
        lo = max(0, c + 1 - w)
        seen += c + n - lo
        full = min(n, max(0, w - c))  # new tokens whose window is not full yet: c + 1, c + 2, ... keys
        pairs += full * (c + 1) + full * (full - 1) // 2 + (n - full) * min(w, c + n)
    return {"bytes": seen * h * d * 2 * 0.625 + 4 * T * q * d, "flops": 4 * d * q * pairs}


# ---------------------------------------------------------------- inputs

def _normal(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda", dtype=torch.float32)


def _turns(rot, scaled):
    """Frequencies base^(-2i / rot) in turns a position, units of 2^-64.  Scaled:
    eight times slower where a pair makes at most one turn in 8192 positions,
    as they are above 32 turns, between the two in between."""
    f = 10000.0 ** (-2.0 * np.arange(rot // 2) / rot)
    if scaled:
        keep = np.clip((8192 * f / (2 * math.pi) - 1.0) / 31.0, 0.0, 1.0)
        f = f * (keep + (1.0 - keep) / 8.0)
    return torch.tensor([round(x * 2.0 ** 64 / (2 * math.pi)) for x in f.tolist()], dtype=torch.int64, device="cuda")


def _magnitude(case):
    return 1.0 + 0.1 * math.log(8.0) if case["scaled"] else 1.0


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    ints = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
    s = dict(op=case["op"])
    if case["op"] in ("angles", "rotate"):
        start = torch.randint(case["max_pos"], (case["tokens"],), generator=g, device="cuda")
        if case["tokens"] > 256:  # prompts, one after the other; else a decode step, every request at its own place
            start = (start[:1] + torch.arange(case["tokens"], device="cuda")) % case["max_pos"]
        pos, turns = start.to(torch.int32), _turns(case["rot"], case["scaled"])
        if case["op"] == "angles":
            s["positions"], s["turns"], s["magnitude"] = pos, turns, _magnitude(case)
            return s
    dt = TYPES[case["dtype"]]
    if case["op"] == "rotate":
        s["x"] = _normal(g, case["tokens"], case["heads"], case["dim"]).to(dt)
        s["angles"], s["inter"] = _angles(pos, turns, _magnitude(case)), case["inter"]
        return s
    cs, ns = _lengths(case)
    ps, T, h, d, q = case["page"], sum(ns), case["kv_heads"], case["dim"], case["q_heads"]
    need = [-(-(c + n) // ps) for c, n in zip(cs, ns)]
    width, total = max(need), sum(need)
    n_pages = total + 8
    order = torch.randperm(n_pages, generator=g, device="cuda").to(torch.int32)
    col = torch.arange(width, device="cuda")[None, :]
    first = ints([0] + need).cumsum(0)[:-1, None]
    table = torch.where(col < ints(need)[:, None], order[(first + col).clamp(max=n_pages - 1)], -1).to(torch.int32)
    cu = ints([0] + ns).cumsum(0).to(torch.int32)
    seq = ints([c + n for c, n in zip(cs, ns)])
    # four key channels are larger at every token, as in real key caches
    loud = torch.ones(h, d, device="cuda")
    loud.scatter_(1, torch.rand(h, d, generator=g, device="cuda").argsort(1)[:, :4], 4.0)
    # the pool holds what earlier steps stored: N(0, 1) values, a different size for each page and head
    amp = torch.exp2(torch.rand(n_pages, h, 1, 1, generator=g, device="cuda") - 0.5)
    kf = _normal(g, n_pages, h, ps, d) * loud[:, None, :] * amp
    if case["op"] == "append":
        s["k_scale"] = _scale_of(kf.abs().amax((2, 3)))
        s["k_pages"] = (kf / s["k_scale"][..., None, None]).to(torch.float8_e4m3fn)
    else:
        s["k_codes"], s["k_meta"] = _packed(kf.half(), True)
    del kf
    vf = _normal(g, n_pages, h, ps, d) * amp
    if case["op"] == "append":
        s["v_scale"] = _scale_of(vf.abs().amax((2, 3)))
        s["v_pages"] = (vf / s["v_scale"][..., None, None]).to(torch.float8_e4m3fn)
    else:
        s["v_codes"], s["v_meta"] = _packed(vf.half(), False)
    del vf
    if case["op"] == "attention4":
        s["block_table"], s["cu_new"], s["seq_len"] = table, cu, seq
        s["max_new"], s["max_len"] = max(ns), max(c + n for c, n in zip(cs, ns))
        s["q"] = _normal(g, T, q, d).to(dt)
        s["softmax_scale"], s["window"] = d ** -0.5, case["window"]
        return s
    # q, k and v as slices of one projection's output
    fused = torch.empty(T, q + 2 * h, d, dtype=dt, device="cuda")
    fused[:, :q] = _normal(g, T, q, d).to(dt)
    fused[:, q:q + h] = (_normal(g, T, h, d) * loud).to(dt)
    fused[:, q + h:] = _normal(g, T, h, d).to(dt)
    s["q"], s["k"], s["v"] = fused[:, :q], fused[:, q:q + h], fused[:, q + h:]
    t = torch.arange(T, device="cuda")
    b = torch.searchsorted(cu[1:].long(), t, right=True)
    pos = seq.long()[b] - cu.long()[b + 1] + t
    s["slots"] = (table.long()[b, pos // ps] * ps + pos % ps).to(torch.int32)
    s["angles"], s["inter"] = _angles(pos, _turns(case["rot"], case["scaled"]), _magnitude(case)), case["inter"]
    return s


# ---------------------------------------------------------------- one pass

def run(s):
    if s["op"] == "angles":
        return _angles_own(s) if own else _angles(s["positions"], s["turns"], s["magnitude"])
    if s["op"] == "rotate":
        return _rotate_own(s) if own else _rotate(s, s["x"])
    if s["op"] == "append":
        return _append_own(s) if own else _append(s)
    if s["op"] == "append4":
        return _append4_own(s) if own else _append4(s)
    return _attention4_own(s) if own else _attention4(s)


def _angles_own(s):
    from bit_kv_cache_11_gb300 import kvq
    return kvq.kvq_rotary_angles(s["positions"], s["turns"], magnitude=s["magnitude"])


def _rotate_own(s):
    from bit_kv_cache_11_gb300 import kvq
    return kvq.kvq_rotate(s["x"], s["angles"], interleaved=s["inter"])


def _append_own(s):
    from bit_kv_cache_11_gb300 import kvq
    q = kvq.kvq_paged_append(s["k"], s["v"], s["slots"], s["k_pages"], s["v_pages"], s["k_scale"], s["v_scale"],
                             s["angles"], interleaved=s["inter"], q=s["q"])
    return {"q": q, **{n: s[n] for n in ("k_pages", "v_pages", "k_scale", "v_scale")}}


def _append4_own(s):
    from bit_kv_cache_11_gb300 import kvq
    pool = (s["k_codes"], s["v_codes"], s["k_meta"], s["v_meta"])
    q = kvq.kvq_paged4_append(s["k"], s["v"], s["slots"], *pool, s["angles"], interleaved=s["inter"], q=s["q"])
    k, v = kvq.kvq_paged4_read(s["slots"], *pool)
    return {"q": q, "k": k, "v": v}


def _attention4_own(s):
    from bit_kv_cache_11_gb300 import kvq
    return kvq.kvq_paged4_attention(s["q"], s["k_codes"], s["v_codes"], s["k_meta"], s["v_meta"], s["block_table"],
                                    s["cu_new"], s["seq_len"], max_new=s["max_new"],
                                    softmax_scale=s["softmax_scale"], window=s["window"])


def _angles(pos, turns, magnitude):
    """[tokens][rot / 2][2] cosines and sines; whole turns drop out of the wrapping product."""
    angle = (pos.long()[:, None] * turns).double() * (2 * math.pi / 2.0 ** 64)
    return (torch.stack([angle.cos(), angle.sin()], -1) * magnitude).float()


def _rotate(s, x):
    """x [tokens][heads][dim] turned by its tokens' angles."""
    c, n = s["angles"][:, None, :, 0], s["angles"][:, None, :, 1]
    xf, r = x.float(), 2 * s["angles"].shape[1]
    out = xf.clone()
    if s["inter"]:
        a, b = slice(0, r, 2), slice(1, r, 2)
    else:
        a, b = slice(0, r // 2), slice(r // 2, r)
    out[..., a] = xf[..., a] * c - xf[..., b] * n
    out[..., b] = xf[..., b] * c + xf[..., a] * n
    return out.to(x.dtype)


def _scale_of(amax):
    """The smallest power of two of the exponents' range that brings amax to
    448 (E4M3's largest) or below."""
    m, e = torch.frexp(amax / 448.0)
    e = torch.where(m == 0.5, e - 1, e)
    return torch.ldexp(torch.ones_like(amax), e.clamp(MIN_EXP, MAX_EXP))


def _codes(x):
    """Nearest E4M3 values (ties to even) of x, at most 448 in magnitude; 0 for NaN."""
    return torch.nan_to_num(x, nan=0.0, posinf=448.0, neginf=-448.0).clamp(-448.0, 448.0).to(torch.float8_e4m3fn)


def _append(s):
    ps, slots = s["k_pages"].shape[2], s["slots"].long()
    page, row = slots // ps, slots % ps
    n_pages = s["k_pages"].shape[0]
    first = torch.full((n_pages,), ps, device=slots.device).scatter_reduce(0, page, row, "amin")
    touched = first < ps
    partly = (touched & (first > 0)).nonzero()[:, 0]  # pages that hold older rows
    older = torch.arange(ps, device=slots.device)[None, :] < first[partly][:, None]
    for x, pages, scale in ((_rotate(s, s["k"]), s["k_pages"], s["k_scale"]), (s["v"], s["v_pages"], s["v_scale"])):
        x = x.float()
        size = torch.where(torch.isfinite(x), x.abs(), 0.0).amax(2)
        amax = torch.zeros_like(scale).scatter_reduce(0, page[:, None].expand_as(size), size, "amax")
        was = torch.where((first > 0)[:, None], scale, 0.0)
        now = torch.where(touched[:, None], torch.maximum(_scale_of(amax), was), scale)
        bits = pages.view(torch.uint8)
        old = pages[partly].float() * (scale[partly] / now[partly])[..., None, None]
        bits[partly] = torch.where(older[:, None, :, None], _codes(old).view(torch.uint8), bits[partly])
        bits[page, :, row] = _codes(x / now[page][..., None]).view(torch.uint8)
        scale.copy_(now)
    return {"q": _rotate(s, s["q"]), **{n: s[n] for n in ("k_pages", "v_pages", "k_scale", "v_scale")}}


def _packed(x, key):
    """fp16 x [..., dim] as bytes of two codes [..., dim / 2] and {step, minimum}
    pairs [..., dim / 32, 2].  The eight codes of a word lie one after the other,
    lowest bits first, in keys the four even channels before the four odd ones."""
    xg = x.unflatten(-1, (-1, GROUP)).float()
    mn = xg.amin(-1, keepdim=True)
    step = ((xg.amax(-1, keepdim=True) - mn) / 15.0).half()
    c = ((xg - mn) / torch.where(step > 0, step, 1.0).float()).round().clamp(0, 15)
    c = torch.where(step > 0, c, 0.0).to(torch.uint8).flatten(-2)
    if key:
        c = c.unflatten(-1, (-1, 4, 2)).transpose(-1, -2).flatten(-3)
    return c[..., 0::2] | (c[..., 1::2] << 4), torch.cat([step, mn.half()], -1)


def _values(codes, meta, key):
    """fp16 values [..., dim] of packed codes: code * step + minimum."""
    c = torch.stack([codes & 15, codes >> 4], -1).flatten(-2)
    if key:
        c = c.unflatten(-1, (-1, 2, 4)).transpose(-1, -2).flatten(-3)
    m = meta.float()
    return (c.unflatten(-1, (-1, GROUP)).float() * m[..., :1] + m[..., 1:]).half().flatten(-2)


def _append4(s):
    ps, slots = s["k_codes"].shape[2], s["slots"].long()
    page, row = slots // ps, slots % ps
    out = {"q": _rotate(s, s["q"])}
    for n, x in (("k", _rotate(s, s["k"])), ("v", s["v"])):
        codes, meta = _packed(x.clamp(-65408.0, 65408.0).half(), n == "k")
        s[n + "_codes"][page, :, row] = codes
        s[n + "_meta"][page, :, row] = meta
        out[n] = _values(s[n + "_codes"][page, :, row], s[n + "_meta"][page, :, row], n == "k")
    return out


def _gather(codes, meta, table, length, key):
    """[B][heads][length][D] fp32 values of the first `length` tokens of each request."""
    at = table[:, : -(-length // codes.shape[2])].long().clamp(min=0)
    x = _values(codes[at], meta[at], key).float().permute(0, 2, 1, 3, 4)  # [B][heads][pages][ps][D]
    return x.reshape(x.shape[0], x.shape[1], -1, x.shape[4])[:, :, :length]


def _attention4(s):
    q, table, cu, seq = s["q"].float(), s["block_table"], s["cu_new"].long(), s["seq_len"].long()
    T, Hq, D = q.shape
    B, N, L = table.shape[0], s["max_new"], s["max_len"]
    k = _gather(s["k_codes"], s["k_meta"], table, L, True)
    v = _gather(s["v_codes"], s["v_meta"], table, L, False)
    H = k.shape[1]
    j = torch.arange(N, device=q.device)
    n = cu[1:] - cu[:-1]
    at = (cu[:-1, None] + j).clamp(max=T - 1)
    qb = q[at].reshape(B, N, H, Hq // H, D).permute(0, 2, 3, 1, 4).reshape(B, H, -1, D)
    z = (qb * s["softmax_scale"]) @ k.transpose(2, 3)  # [B][H][R * N][L]
    t = torch.arange(L, device=q.device)
    pos = (seq - n)[:, None] + j
    see = t <= pos[..., None]
    if s["window"]:
        see &= t > pos[..., None] - s["window"]
    z = z.view(B, H, Hq // H, N, L).masked_fill_(~see[:, None, None], -math.inf)
    top = z.amax(-1, keepdim=True)
    p = z.sub_(torch.where(torch.isfinite(top), top, 0.0)).exp_()
    total = p.sum(-1, keepdim=True)
    live = see.any(1)  # tokens that some new token sees; what lies in the others' places does not count
    o = p.view(B, H, -1, L) @ torch.where(live[:, None, :, None], v, 0.0)
    o = o.view(B, H, Hq // H, N, D) / torch.where(total > 0, total, 1.0)
    i = torch.arange(T, device=q.device)
    b = torch.searchsorted(cu[1:], i, right=True)
    return o.permute(0, 3, 1, 2, 4).reshape(B, N, Hq, D)[b, i - cu[b]].to(s["q"].dtype)


# ---------------------------------------------------------------- in 64 bits

def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "rotate":
        return _exact_rotate(s, s["x"])
    return {"angles": _exact_angles, "append": _exact_append, "append4": _exact_append4,
            "attention4": _exact_attention4}[case["op"]](s)


def _exact_angles(s):
    pos, turns = s["positions"].cpu().numpy().astype(np.uint64), s["turns"].cpu().numpy().astype(np.uint64)
    unit = s["magnitude"] * np.exp(1j * ((pos[:, None] * turns[None, :]).astype(np.float64) * (2 * np.pi / 2.0 ** 64)))
    return torch.view_as_real(torch.from_numpy(unit))


def _exact_rotate(s, x):
    """Pairs of channels as complex numbers times those of the angles."""
    unit = torch.view_as_complex(s["angles"].double())[:, None, :]
    y, r = x.double(), 2 * s["angles"].shape[1]
    first, second = (y[..., 0:r:2], y[..., 1:r:2]) if s["inter"] else (y[..., : r // 2], y[..., r // 2:r])
    z = torch.complex(first.contiguous(), second.contiguous()) * unit
    turned = torch.stack([z.real, z.imag], -1).flatten(-2) if s["inter"] else torch.cat([z.real, z.imag], -1)
    return torch.cat([turned, y[..., r:]], -1)


def _nearest_e4m3(x):
    """The E4M3 value nearest to x (ties to even), written out: steps of
    2^(e - 3) for 2^e <= |x| < 2^(e + 1), of 2^-9 below 2^-6, at most 448."""
    e = torch.frexp(x)[1].double() - 1
    step = torch.exp2(torch.clamp(e, min=-6.0) - 3)
    return (torch.round(x / step) * step).clamp(-448.0, 448.0)


def _exact_append(s):
    out = {"q": _exact_rotate(s, s["q"])}
    slots = s["slots"].long()
    ps = s["k_pages"].shape[2]
    for name in ("k", "v"):
        # a rotated key is held in its own type before it is stored
        x = _exact_rotate(s, s["k"]).to(s["k"].dtype).double() if name == "k" else s["v"].double()
        values, scale = s[name + "_pages"].double(), s[name + "_scale"].double()
        page = slots // ps
        runs, where = torch.unique(page, return_inverse=True)
        first = torch.full_like(runs, ps).scatter_reduce(0, where, slots % ps, "amin")
        top = torch.zeros(runs.numel(), x.shape[1], dtype=torch.double, device=x.device)
        top = top.scatter_reduce(0, where[:, None].expand(-1, x.shape[1]), x.abs().amax(2), "amax")
        power = torch.exp2(torch.ceil(torch.log2((top / 448.0).clamp(min=2.0 ** MIN_EXP))).clamp(max=MAX_EXP))
        held = (first > 0)[:, None]
        power = torch.where(held & (scale[runs] > power), scale[runs], power)
        grown = _nearest_e4m3(values[runs] * (scale[runs] / power)[..., None, None])
        old = (torch.arange(ps, device=x.device)[None, :] < first[:, None])[:, None, :, None]
        values[runs] = torch.where(old, grown, values[runs])
        scale[runs] = power
        values[page, :, slots % ps] = _nearest_e4m3(x / power[where][..., None])
        out[name + "_pages"], out[name + "_scale"] = values, scale
    return out


def _exact_append4(s):
    out = {"q": _exact_rotate(s, s["q"])}
    for name in ("k", "v"):
        x = _exact_rotate(s, s["k"]).to(s["k"].dtype).double() if name == "k" else s["v"].double()
        y = x.reshape(x.shape[0], x.shape[1], -1, GROUP)
        low, high = y.min(-1, keepdim=True).values, y.max(-1, keepdim=True).values
        step = ((high - low) / 15).half().double()
        level = torch.where(step > 0, (y - low) / torch.where(step > 0, step, 1.0), 0.0)
        out[name] = (torch.round(level).clamp(0, 15) * step + low).reshape(x.shape)
    return out


def _exact_attention4(s):
    q, table, cu, seq = s["q"].double(), s["block_table"].tolist(), s["cu_new"].tolist(), s["seq_len"].tolist()
    H, D = s["k_codes"].shape[1], q.shape[2]
    ps, R = s["k_codes"].shape[2], q.shape[1] // H
    # channel c of a key: word c / 8, nibble (c % 8) / 2 of the even channels or of the odd ones behind them
    c = torch.arange(D, device=q.device)
    nibble = {"k": c // 8 * 8 + c % 8 // 2 + 4 * (c % 2), "v": c}

    def read(name, ids, h, length):
        codes = s[name + "_codes"][ids, h].reshape(-1, D // 2)[:length]
        meta = s[name + "_meta"][ids, h].reshape(-1, D // GROUP, 2)[:length].double()
        at = nibble[name]
        code = (codes[:, at // 2] >> (at % 2 * 4).to(torch.uint8)) & 15
        return (code.double() * meta[:, c // GROUP, 0] + meta[:, c // GROUP, 1]).half().double()

    out = torch.zeros_like(q)
    for b, length in enumerate(seq):
        n = cu[b + 1] - cu[b]
        ids = torch.tensor(table[b][: -(-length // ps)], device=q.device)
        pos = torch.arange(length - n, length, device=q.device)[:, None]
        t = torch.arange(length, device=q.device)[None, :]
        hidden = t > pos
        if s["window"]:
            hidden = hidden | (pos - t >= s["window"])
        for h in range(H):
            k, v = read("k", ids, h, length), read("v", ids, h, length)
            for r in range(R):
                z = (q[cu[b]:cu[b + 1], h * R + r] @ k.T * s["softmax_scale"]).masked_fill(hidden, -math.inf)
                out[cu[b]:cu[b + 1], h * R + r] = torch.softmax(z, -1) @ v
    return out
