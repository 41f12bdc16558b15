"""Cases of the 4-bit pages' attention for the tests: paged_ref.SHARES over pages of
values that 4 bits hold, with the bound of paged_ref.row at each kernel's own weights."""
import numpy as np

import paged4_ref
import paged_ref


def held(x):
    """Codes, steps, minima and values of x [pages][H][ps][D]."""
    codes, step, mn = paged4_ref.quantize(x.astype(np.float16))
    return codes, step, mn, paged4_ref.values(codes, step, mn)


def pool(k, v, unused=None):
    """A pool's buffers (numpy) of what `held` gave for keys and values; rows of `unused`
    [pages][ps] hold NaN steps and infinite minima."""
    sides = []
    for side, key in ((k, True), (v, False)):
        codes, step, mn, _ = side
        step, mn = step.copy(), mn.copy()
        if unused is not None:
            step.transpose(0, 2, 1, 3)[unused] = np.nan
            mn.transpose(0, 2, 1, 3)[unused] = -np.inf
        sides.append((paged4_ref.pack(codes, key), np.stack([step, mn], -1)))
    return [sides[0][0], sides[1][0], sides[0][1], sides[1][1]]


def shares_case(case):
    """paged_ref.shares_case over 4-bit pages: keys and values of about 1."""
    s = paged_ref.shares_case(case)
    rng = np.random.default_rng(sum(s["seq"]) + s["ps"])
    shape = s["codes"][0].shape
    k, v = (held(rng.standard_normal(shape)) for _ in "kv")
    used = np.zeros((shape[0], s["ps"]), bool)
    for b, n in enumerate(s["seq"]):
        t = np.arange(n)
        used[s["table"][b][t // s["ps"]], t % s["ps"]] = True
    return {**s, "k": k, "v": v, "pool": pool(k, v, ~used)}


def shares_want(s, each=None):
    """(out, bound) of all new tokens, as paged_ref.rows."""
    q, seq, cu, ps, window = s["q"].double().numpy(), s["seq"], s["cu"], s["ps"], s["window"]
    R = q.shape[1] // s["k"][3].shape[1]
    out, bound = np.zeros(q.shape), np.full(q.shape, 2.0 ** -25)
    for b in range(len(seq)):
        n = int(cu[b + 1] - cu[b])
        t = np.arange(seq[b])
        pg, r = s["table"][b][t // ps], t % ps
        for hq in range(q.shape[1] if n else 0):
            k, v = s["k"][3][pg, hq // R, r], s["v"][3][pg, hq // R, r]
            for j in range(n):
                pos = int(seq[b]) - n + j
                lo = max(0, pos - window + 1) if window else 0
                if pos < lo:
                    continue
                at = slice(lo, pos + 1)
                o, e, parts = paged_ref.row(q[cu[b] + j, hq], k[at], v[at], np.ones(pos + 1 - lo), s["softmax_scale"],
                                            paged_ref.WEIGHT_LOG2[s["kernel"]], s["half_step"])
                out[cu[b] + j, hq], bound[cu[b] + j, hq] = o, e
                if each:
                    each(b, j, hq, parts, o, e)
    return out, bound


def one_before_many(D, n, kernel):
    """A token whose weight is 2^23 times another's, but whose value is 0, before 4096
    others; (keys, values, q, T, page size, out, bound)."""
    rng = np.random.default_rng(D + n)
    ps, T = 64, 4096 + n
    k = np.zeros((-(-T // ps), 1, ps, D))
    k[..., 0], k[..., 1] = -16.0, -rng.uniform(0.5, 1.5, k.shape[:3])
    k[0, 0, 0] = 0.0
    v = rng.uniform(0.5, 1.0, k.shape)
    v[0, 0, 0] = 0.0
    k, v = held(k), held(v)
    q = np.zeros((n, 1, D))
    q[..., :2] = 1.0
    kk, vv = k[3].reshape(-1, D), v[3].reshape(-1, D)
    out, bound = np.zeros(q.shape), np.zeros(q.shape)
    for j in range(n):
        m = T - n + j + 1
        out[j, 0], bound[j, 0], _ = paged_ref.row(q[j, 0], kk[:m], vv[:m], np.ones(m), 1.0, paged_ref.WEIGHT_LOG2[kernel],
                                                  2.0 ** -11)
    return k, v, q, T, ps, out, bound
