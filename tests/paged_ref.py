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
