"""64-bit forms of the paged cache, decode attention, routing by scores and
sampling, in numpy, from their definitions (include/lora.h), with bounds of
what fp32 sums may lose."""
import numpy as np

E4M3_MAX = 448.0


def e4m3_nearest(x):
    """The value E4M3 keeps of each x (64-bit): half-way cases to the even step,
    past 448 the largest."""
    x = np.asarray(x, np.float64)
    with np.errstate(invalid="ignore"):
        y = np.clip(x, -E4M3_MAX, E4M3_MAX)
        _, e = np.frexp(np.where(np.isnan(y), 0.0, y))
        step = np.ldexp(1.0, np.maximum(e - 4, -9))
        return np.rint(y / step) * step


def e4m3_values():
    """The value of each code 0..255: sign, 4 bits of exponent (bias 7), 3 of mantissa."""
    c = np.arange(256)
    e, m = (c >> 3) & 15, (c & 7).astype(np.float64)
    v = np.where(e == 0, np.ldexp(m, -9), np.ldexp(8 + m, e - 10))
    v = np.where((c & 127) == 127, np.nan, v)
    return np.where(c >> 7, -v, v)


def attention(q, k, v, scale):
    """One request: q [heads, D], k and v [n, kv heads, D] (its attended
    positions). (out, lse, bound): `bound` is what fp32 sums may lose of out.

    A score is D products summed in fp32 and scaled: off by at most d =
    (D + 4) 2^-24 scale sum |q k|; p = exp of the difference of two such scores,
    so off by 2 d relative, by 2^-21 for the exponential and its argument's
    rounding (|argument| up to 2^3 before p no longer counts, 2^-24 each and as
    much for the base-2 form) and by 2^-16 where p is carried as two 16-bit
    halves; sums of n terms add n 2^-24 each, for the numerator and the
    denominator."""
    heads, D = q.shape
    n, kv = k.shape[:2]
    out = np.zeros((heads, D))
    lse = np.full(heads, -np.inf)
    bound = np.zeros((heads, D))
    lse_bound = np.zeros(heads)
    if n == 0:
        return out, lse, bound, lse_bound
    for h in range(heads):
        hk = h // (heads // kv)
        s = scale * (k[:, hk] @ q[h])
        d = (D + 4) * 2.0 ** -24 * abs(scale) * (np.abs(k[:, hk]) @ np.abs(q[h]))
        top = s.max()
        p = np.exp(s - top)
        p_sum = p.sum()
        lse[h] = top + np.log(p_sum)
        p /= p_sum
        out[h] = p @ v[:, hk]
        near = p > 2.0 ** -40  # the others are lost with less than the sums lose
        worst = d[near].max()
        bound[h] = (p @ np.abs(v[:, hk])) * (4 * worst + 2.0 ** -16 + 2.0 ** -20 + 2 * (n + 16) * 2.0 ** -24)
        lse_bound[h] = worst + (n + 16) * 2.0 ** -24 + 4 * 2.0 ** -24 * (abs(top) + np.log(n) + 1)
    return out, lse, bound, lse_bound


def _key(c):
    """NaN below every number."""
    return np.where(np.isnan(c), -np.inf, c), ~np.isnan(c)


def _falling(c):
    """Indices of c in falling order, equal values by index, NaN last."""
    val, num = _key(c)
    return np.lexsort((np.arange(len(c)), -val, ~num))


def route(x, router, k, score, bias, groups, top_groups, group_best, renorm, scale):
    z = x @ router.T
    T, E = z.shape
    ids, w = np.zeros((T, k), np.int32), np.zeros((T, k))
    n = E // groups
    with np.errstate(over="ignore", invalid="ignore"):
        for t in range(T):
            if score == "sigmoid":
                s = 1.0 / (1.0 + np.exp(-z[t]))
            else:
                e = np.exp(z[t] - (np.nanmax(z[t]) if not np.isnan(z[t]).all() else np.nan))
                s = e / e.sum()
            c = s if bias is None else s + bias
            left = np.ones(E, bool)
            if groups > 1:
                value = np.array([c[g * n:(g + 1) * n][_falling(c[g * n:(g + 1) * n])][:group_best].sum()
                                  for g in range(groups)])
                kept = _falling(value)[:top_groups]
                left = np.isin(np.arange(E) // n, kept)
            order = [e for e in _falling(c) if left[e]][:k]
            ids[t] = order
            w[t] = s[order] / (s[order].sum() if renorm else 1.0) * scale
    return ids, w


def sample(logits, u, t, k, p, least):
    """One request: (id, probability)."""
    x = np.asarray(logits, np.float64)
    cand = np.flatnonzero(~np.isnan(x) & (x > -np.inf))
    if cand.size == 0:
        return -1, 0.0
    order = cand[np.lexsort((cand, -x[cand]))]
    if not t > 0:
        return int(order[0]), 1.0
    top = x[order[0]]
    with np.errstate(invalid="ignore", over="ignore"):
        w = (x[order] == top).astype(float) if np.isinf(top) else np.exp((x[order] - top) / t)
    n = len(order) if k < 1 else min(k, len(order))
    if p < 1:
        run = np.cumsum(w[:n])
        n = min(n, max(1, int(np.searchsorted(run, max(p, 0) * run[-1])) + 1))
    keep = np.arange(n)
    if least > 0:
        keep = keep[(w[:n] >= least) | (keep == 0)]
    by = np.argsort(order[keep])
    idx, wi = order[keep][by], w[keep][by]
    run = np.cumsum(wi)
    i = min(int(np.searchsorted(run, u * run[-1], side="right")), int(np.flatnonzero(wi > 0)[-1]))
    return int(idx[i]), wi[i] / run[-1]
