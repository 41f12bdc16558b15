"""The paged cache's operators in numpy and 64 bits, for the tests: plain loops
over requests, pages and heads, from the definitions in include/kvq.h."""
import numpy as np

E4M3 = np.array([(-1.0) ** (c >> 7) * (((c >> 3 & 15) and (1 + (c & 7) / 8) * 2.0 ** ((c >> 3 & 15) - 7))
                                       or (c & 7) * 2.0 ** -9) if c & 127 != 127 else np.nan
                 for c in range(256)])


def e4m3_code(x):
    """Codes (uint8) of the E4M3 values nearest to x, ties to the even code,
    saturating; 0 for NaN."""
    x = np.asarray(x, np.float64)
    grid = E4M3[:127]
    a = np.minimum(np.abs(np.nan_to_num(x, nan=0.0, posinf=1e9, neginf=-1e9)), 448.0)
    hi = np.clip(np.searchsorted(grid, a), 0, 126)
    lo = np.maximum(hi - 1, 0)
    down, up = a - grid[lo], grid[hi] - a
    c = np.where((down < up) | ((down == up) & (lo % 2 == 0)), lo, hi)
    c = np.where(grid[hi] == a, hi, c)
    return (c | np.where(np.signbit(x) & ~np.isnan(x), 128, 0)).astype(np.uint8)


def page_scale(amax):
    for e in range(-15, 41):
        if amax <= 448.0 * 2.0 ** e:
            return 2.0 ** e
    return 2.0 ** 40


def plan(ctx, new, table, free, n_free, ps, n_tokens):
    table = table.copy()
    B, width = table.shape
    cu, seq, slots = [0], [], np.full(n_tokens, -1, np.int32)
    ahead, left = 0, n_free
    for b in range(B):
        n = max(int(new[b]), 0)
        have, tot = -(-int(ctx[b]) // ps), -(-int(ctx[b] + new[b]) // ps)
        ok = ctx[b] >= 0 and new[b] >= 0 and tot <= width
        need = tot - have if ok else 0
        ahead += need
        ok = ok and (need == 0 or ahead <= n_free)
        if ok:
            for j in range(need):
                table[b, have + j] = free[n_free - 1 - (ahead - need) - j]
            left -= need
            for j in range(n):
                pos = int(ctx[b]) + j
                if cu[b] + j < n_tokens:
                    slots[cu[b] + j] = table[b, pos // ps] * ps + pos % ps
        seq.append(int(ctx[b]) + n if ok else int(ctx[b]))
        cu.append(cu[b] + n)
    return table, np.array(cu), np.array(seq), slots, left


def store(x, slots, codes, scale, ps):
    """x: float64 [T][H][D]; codes: uint8 [pages][H][ps][D]; scale: [pages][H].
    Returns new codes and scales."""
    codes, scale = codes.copy(), scale.copy()
    by_page = {}
    for t, s in enumerate(slots):
        if s >= 0:
            by_page.setdefault(int(s) // ps, []).append((int(s) % ps, t))
    for page, rows in by_page.items():
        first = min(r for r, _ in rows)
        tok = [t for _, t in rows]
        for h in range(x.shape[1]):
            v = x[tok, h]
            fin = np.abs(v[np.isfinite(v)])
            sc = page_scale(fin.max() if fin.size else 0.0)
            old = scale[page, h]
            if first > 0:
                sc = max(sc, old)
                if sc > old:
                    codes[page, h, :first] = e4m3_code(E4M3[codes[page, h, :first]] * (old / sc))
            for r, t in rows:
                codes[page, h, r] = e4m3_code(x[t, h] / sc)
            scale[page, h] = sc
    return codes, scale


def attention(q, kc, vc, ks, vs, table, cu, seq, ps, scale, window=0):
    """Returns (out, size, reach): the attention, sum p |v| per output (the size
    that weight errors scale with) and the largest scale * sum |q k| per row."""
    T, Hq, D = q.shape
    H = kc.shape[1]
    R = Hq // H
    out, size, reach = np.zeros(q.shape), np.zeros(q.shape), np.zeros((T, Hq))
    for b in range(len(seq)):
        n = cu[b + 1] - cu[b]
        for j in range(n):
            pos = seq[b] - n + j
            lo = max(0, pos - window + 1) if window else 0
            t = np.arange(lo, pos + 1)
            if t.size == 0:
                continue
            pg, row = table[b][t // ps], t % ps
            for h in range(H):
                k = E4M3[kc[pg, h, row]] * ks[pg, h][:, None]
                v = E4M3[vc[pg, h, row]] * vs[pg, h][:, None]
                for r in range(R):
                    x = q[cu[b] + j, h * R + r]
                    z = k @ x * scale
                    p = np.exp(z - z.max())
                    p /= p.sum()
                    out[cu[b] + j, h * R + r] = p @ v
                    size[cu[b] + j, h * R + r] = p @ np.abs(v)
                    reach[cu[b] + j, h * R + r] = (np.abs(k) @ np.abs(x)).max() * abs(scale)
    return out, size, reach


def tolerance(out, size, reach, half_step, n_tokens, vmax):
    """Largest error of an output.  Weights are rounded to fp16 (half a step:
    2^-11 of a weight, 2^-25 of the largest below fp16's normal range); a
    score is an fp32 sum of D products, whose additions (rounded or cut, a
    step each) err by at most D * 2^-23 * sum |q k|, twice in the quotient;
    exponentials, sums and the division take 2^-18 at most; the output is
    rounded by half a step."""
    D = out.shape[-1]
    err = size * (2.0 ** -11 + 2 * D * 2.0 ** -23 * reach[..., None] + 2.0 ** -18)
    err = err + n_tokens * 2.0 ** -25 * vmax
    return err + half_step * (np.abs(out) + err) + 2.0 ** -25


# The kernels' weights are fp16 numbers 2^15 (decode) and 2^7 (prompt) times the
# share p * scale of the row's largest: half a step of fp16 is 2^-11 of a number
# of at least 2^-14 and 2^-25 below.
WEIGHT_LOG2 = {"decode": 15, "prompt": 7}


def row(q, k, v, sv, scale, log2, half_step):
    """Attention of one query over the tokens it sees, k and v [n][D] with v's page
    scales sv [n]: (out, bound, parts).  `bound` is the largest error of an
    output of the kernel: weights rounded to fp16, scores whose D products are
    summed in fp32 (D * 2^-23 of sum |q k|, a step each) and scaled, exponentials
    and logarithms of 22 bits, sums in fp32 of 16 tokens at a time (a step each),
    and the output's rounding.  An error d of a score moves a weight by d of it
    in the numerator and in the sum below.  parts: every token's p * v."""
    n, D = k.shape
    z = k @ q * scale
    p = np.exp(z - z.max())
    p /= p.sum()
    out = p @ v
    w = p * sv
    rounded = np.where(w >= 2.0 ** (-14 - log2) * w.max(), 2.0 ** -11 * w, 2.0 ** (-25 - log2) * w.max()) / sv
    score = D * 2.0 ** -23 * (np.abs(k) @ np.abs(q)) * abs(scale) + (np.abs(z) + 64) * 2.0 ** -23
    other = score + 2.0 ** -20 + (n / 16 + 32) * 2.0 ** -23
    err = rounded @ np.abs(v) + (p * other) @ np.abs(v) + (p @ other) * np.abs(out)
    return out, err + half_step * (np.abs(out) + err) + 2.0 ** -25, p[:, None] * v


def rows(q, kc, vc, ks, vs, table, cu, seq, ps, scale, window, log2, half_step, each=None):
    """(out, bound) of all new tokens; `each(b, j, hq, parts, out, bound)` sees every row."""
    T, Hq, D = q.shape
    R = Hq // kc.shape[1]
    out, bound = np.zeros(q.shape), np.full(q.shape, 2.0 ** -25)
    for b in range(len(seq)):
        n = int(cu[b + 1] - cu[b])
        t = np.arange(seq[b])
        pg, r = table[b][t // ps], t % ps
        for h in range(kc.shape[1] if n else 0):
            k, v = E4M3[kc[pg, h, r]] * ks[pg, h][:, None], E4M3[vc[pg, h, r]] * vs[pg, h][:, None]
            for j in range(n):
                pos = int(seq[b]) - n + j
                lo = max(0, pos - window + 1) if window else 0
                if pos < lo:
                    continue
                s = slice(lo, pos + 1)
                for hq in range(h * R, h * R + R):
                    o, e, parts = row(q[cu[b] + j, hq], k[s], v[s], vs[pg[s], h], scale, log2, half_step)
                    out[cu[b] + j, hq], bound[cu[b] + j, hq] = o, e
                    if each:
                        each(b, j, hq, parts, o, e)
    return out, bound


# page size, head_dim, kv heads, query heads a kv head, type, cached, new, window, kernel
SHARES = [
    (64, 128, 2, 4, "fp16", [5000], [1], 0, "decode"),         # an item over many CTAs
    (16, 64, 1, 1, "bf16", [3000, 2, 90], [1] * 3, 0, "decode"),
    (128, 128, 1, 2, "fp16", [5300], [1], 0, "decode"),
    (16, 64, 1, 8, "fp16", [2500, 700], [5, 3], 0, "decode"),  # three groups of rows
    (32, 128, 1, 2, "bf16", [3000, 40], [4, 9], 1500, "decode"),
    (32, 64, 2, 2, "fp16", list(range(100, 900, 50)), [1] * 16, 0, "decode"),
    (64, 128, 1, 1, "fp16", [2000, 5], [130, 40], 0, "prompt"),
    (16, 64, 1, 2, "bf16", [700], [70], 0, "prompt"),
    (128, 64, 1, 1, "fp16", [900, 0], [60, 100], 300, "prompt"),
]


def shares_case(case):
    """Numbers of a case of SHARES: values of about 1, scales 2^-9 .. 2^-4; rows that
    hold no token are NaN codes in `stale`.  Requests without tokens follow in the
    prompt kernel's cases (a large batch: many rows go to that kernel)."""
    import torch
    ps, D, H, R, dtype, ctx, new, window, kernel = case
    idle = 140 if kernel == "prompt" else 0
    ctx, new = list(ctx) + [0] * idle, list(new) + [0] * idle
    rng = np.random.default_rng(ps + D + H + R + sum(ctx) + sum(new) + window)
    seq = np.array(ctx) + np.array(new)
    need = -(-seq // ps)
    n_pages = int(need.sum()) + 2
    scale = [2.0 ** rng.integers(-9, -3, (n_pages, H)).astype(np.float64) for _ in range(2)]
    codes = [e4m3_code(rng.standard_normal((n_pages, H, ps, D)) / s[..., None, None]) for s in scale]
    table = np.full((len(seq), int(need.max()) + 1), -1, np.int32)
    ids, at = rng.permutation(n_pages), 0
    used = np.zeros((n_pages, ps), bool)
    for b, n in enumerate(need):
        table[b, :n] = ids[at:at + n]
        for i in range(n):
            used[ids[at + i], :max(0, min(ps, seq[b] - i * ps))] = True
        at += n
    stale = [c.copy() for c in codes]
    for c in stale:
        c.transpose(0, 2, 1, 3)[~used] = 0x7F
    q = torch.from_numpy(rng.standard_normal((sum(new), H * R, D))).to({"fp16": torch.float16, "bf16": torch.bfloat16}[dtype])
    return dict(ps=ps, codes=codes, stale=stale, scale=scale, table=table, cu=np.concatenate([[0], np.cumsum(new)]),
                seq=seq, q=q, max_new=max(new), window=window, softmax_scale=D ** -0.5, kernel=kernel,
                half_step={"fp16": 2.0 ** -11, "bf16": 2.0 ** -8}[dtype])


def shares_want(s, each=None):
    return rows(s["q"].double().numpy(), *s["codes"], *s["scale"], s["table"], s["cu"], s["seq"], s["ps"],
                s["softmax_scale"], s["window"], WEIGHT_LOG2[s["kernel"]], s["half_step"], each)
