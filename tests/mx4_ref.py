"""Plain 64-bit forms of the MXFP4, mixed-adapter and mixture-of-experts
operators, from their definitions, for the tests."""
import numpy as np

MAGNITUDES = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])


def quantize(v):
    """(codes [rows, 16 nb] uint8, scale bytes [rows, nb] uint8) of fp64 rows
    that came from bf16 or fp32 values."""
    v = np.asarray(v, np.float64)
    rows, K = v.shape
    nb = -(-K // 32)
    p = np.zeros((rows, nb * 32))
    p[:, :K] = v
    p = p.reshape(rows, nb, 32)
    bad = ~np.isfinite(p).all(axis=2)
    p = np.where(bad[:, :, None], 0.0, p)
    top = np.abs(p).max(axis=2)
    e = np.frexp(np.where(top > 0, top, 1.0))[1] - 1 - 2  # floor(log2) - 2
    e = np.where(top > 0, np.maximum(e, -127), -127)
    q = p / np.ldexp(1.0, e)[:, :, None]
    # nearest magnitude, a tie to the code with mantissa bit 0 (even codes)
    m = np.minimum(np.abs(q), 6.0)
    d = np.abs(m[..., None] - MAGNITUDES)
    lo = d.argmin(axis=-1)
    hi = 7 - d[..., ::-1].argmin(axis=-1)
    code = np.where(lo == hi, lo, np.where(lo % 2 == 0, lo, hi)).astype(np.uint8)
    code |= (np.signbit(q) * 8).astype(np.uint8)
    code[bad] = 0
    code = code.reshape(rows, nb * 16, 2)
    return code[:, :, 0] | code[:, :, 1] << 4, np.where(bad, 255, e + 127).astype(np.uint8)


def values(codes, byte, K):
    """fp64 values of codes and scale bytes in row order."""
    rows, nb = byte.shape
    c = np.stack([codes & 15, codes >> 4], axis=2).reshape(rows, nb, 32)
    s = np.where(byte == 255, np.nan, np.ldexp(1.0, byte.astype(np.int64) - 127))
    v = MAGNITUDES[c & 7] * np.where(c & 8, -1.0, 1.0) * s[:, :, None]
    return v.reshape(rows, nb * 32)[:, :K]


def tiles(byte):
    """Scale bytes in row order -> the tiles of 64 rows x 8 blocks."""
    rows, nb = byte.shape
    gt, kt = -(-rows // 64), -(-nb // 8)
    out = np.zeros((gt, kt, 512), np.uint8)
    for r in range(rows):
        for b in range(nb):
            q, c = r % 64, b % 8
            out[r // 64, b // 8, 4 * (2 * (16 * (c % 4) + q % 16) + c // 4) + q // 16] = byte[r, b]
    return out.reshape(-1)


def linear(x, W, ids, A, B, alpha, base_x=None):
    """(y, error scale) of the mixed-adapter layer in 64 bits: A[s], B[s] None
    for empty slots. The error scale is what fp32 sums can lose: gamma times
    the sums of magnitudes, plus the 16 bits kept of scale * h."""
    bx = x if base_x is None else base_x
    K = x.shape[1]
    gamma = 2 * (K + 64) * 2.0 ** -24
    y, lost = bx @ W.T, gamma * (np.abs(bx) @ np.abs(W).T)
    for s in range(len(A)):
        rows = np.flatnonzero(ids == s)
        if A[s] is None or rows.size == 0:
            continue
        sc = alpha[s] / A[s].shape[0]
        y[rows] += sc * (x[rows] @ A[s].T) @ B[s].T
        lost[rows] += (gamma + 2.0 ** -15) * abs(sc) * (np.abs(x[rows]) @ np.abs(A[s]).T) @ np.abs(B[s]).T
    return y, lost


def route(x, router, k, renorm):
    logits = x @ router.T
    ids = np.argsort(-logits, axis=1, kind="stable")[:, :k]
    p = np.exp(logits - logits.max(axis=1, keepdims=True))
    w = np.take_along_axis(p, ids, 1)
    return ids.astype(np.int32), w / (w.sum(axis=1, keepdims=True) if renorm else p.sum(axis=1, keepdims=True))


def experts(x, ids, w, gate, up, down):
    """(y, error scale) of the experts' part; gate, up, down fp64 [E, ...]."""
    T, H = x.shape
    E, I = gate.shape[:2]
    eps = 2.0 ** -24
    y, lost = np.zeros((T, H)), np.zeros((T, H))
    for t in range(T):
        for j in range(ids.shape[1]):
            e = ids[t, j]
            if not 0 <= e < E:
                continue
            g, u = gate[e] @ x[t], up[e] @ x[t]
            dg = 2 * (H + 16) * eps * (np.abs(gate[e]) @ np.abs(x[t]))
            du = 2 * (H + 16) * eps * (np.abs(up[e]) @ np.abs(x[t]))
            sg = 1.0 / (1.0 + np.exp(-g))
            a = g * sg * u
            # |silu'| <= 1.1; the function itself in fp32; 16 bits kept of a
            da = 1.1 * dg * (np.abs(u) + du) + np.abs(g * sg) * du + np.abs(a) * (2.0 ** -15 + 16 * eps)
            y[t] += w[t, j] * (down[e] @ a)
            lost[t] += abs(w[t, j]) * (np.abs(down[e]) @ (da + 2 * (I + 16) * eps * np.abs(a)))
    return y, lost + 16 * eps * np.abs(y)
