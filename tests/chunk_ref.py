"""The chunk step written out in float64 with loops, straight from its formulas, and the
error bounds the kernels are held to.

Roundings are counted as at most half a step of the type: bf16 2^-8, fp32 2^-24, E4M3 2^-4
(2^-10 absolute below its smallest normal number), each relative to the rounded value.
"""
import numpy as np

PAGE = 128
U32 = 2.0 ** -24
HALF_STEP = {"f32": 2.0 ** -24, "bf16": 2.0 ** -8}


def chunk_map(lens, cu, rows, capacity, table=None, held=None, free=None, taken=0, n_pages=0):
    """Sequential plan of a step. Returns slots, positions, kv_lens, table, held, taken."""
    B = len(lens)
    paged = table is not None
    table = table.copy() if paged else None
    held = list(held) if paged else [0] * B
    slots, positions, kv = [-1] * rows, [-1] * rows, [0] * B
    asked, got_all = 0, 0
    for b in range(B):
        lo, hi = int(cu[b]), int(cu[b + 1])
        if lo < 0 or hi < lo or hi > rows:
            continue
        total = int(lens[b]) + hi - lo
        if lens[b] < 0 or total > capacity:
            continue
        if paged:
            need = max(0, -(-total // PAGE) - held[b])
            first = taken + asked
            asked += need
            if need and taken + asked > len(free):
                continue
            for i in range(need):
                table[b, held[b] + i] = free[first + i]
            held[b] += need
            got_all += need
        kv[b] = total
        for r in range(lo, hi):
            p = int(lens[b]) + r - lo
            if paged:
                page = int(table[b, p // PAGE])
                if not 0 <= page < n_pages:
                    continue
                slots[r] = page * PAGE + p % PAGE
            else:
                slots[r] = b * capacity + p
            positions[r] = p
    return slots, positions, kv, table, held, taken + got_all


def rope_angles(pos, d_h, theta=1e6):
    i = np.arange(d_h // 2)
    return pos * theta ** (-2.0 * i / d_h)


def norm_rope(x, gamma, pos, eps=1e-6, rope=True):
    """RMSNorm over the last axis (gamma None: none), then the rotation of pairs (i, i + d/2).
    Returns the values and the sum of the two products' magnitudes behind each of them."""
    x = np.asarray(x, np.float64)
    d = x.shape[-1]
    if gamma is not None:
        x = x / np.sqrt((x * x).mean(-1, keepdims=True) + eps) * np.asarray(gamma, np.float64)
    if not rope:
        return x, np.abs(x)
    a, b = x[..., :d // 2], x[..., d // 2:]
    c, s = np.cos(rope_angles(pos, d)), np.sin(rope_angles(pos, d))
    y = np.concatenate((a * c - b * s, b * c + a * s), -1)
    mag = np.concatenate((np.abs(a * c) + np.abs(b * s), np.abs(b * c) + np.abs(a * s)), -1)
    return y, mag


def append_bound(y, mag, d_h, out):
    """fp32: the mean of squares sums d_h terms (d_h + 2 roundings), the root and the scaling
    4 more, the angle's table entries 1 each, products and sum 3; then the stored rounding."""
    fp32 = mag * (d_h + 12) * U32
    if out == "e4m3":
        return fp32 + (np.abs(y) + fp32) * 2.0 ** -4 + 2.0 ** -10
    return fp32 + (np.abs(y) + fp32) * HALF_STEP[out]


def attention(q, k, v, kv_len, n, G, window, scaling):
    """q [n][n_h][d], k / v [kv_len][n_kv][d]: out [n][n_h][d], sum of p |v| (same shape), the
    largest sum of |q_i k_i| scaling, and the number of keys."""
    n_h, d = q.shape[1:]
    out, mag = np.zeros((n, n_h, d)), np.zeros((n, n_h, d))
    big = 0.0
    for i in range(n):
        p = kv_len - n + i
        lo = max(0, p - window + 1) if window > 0 else 0
        if p < 0 or kv_len == 0:
            continue
        for h in range(n_h):
            K, V = k[lo:p + 1, h // G], v[lo:p + 1, h // G]
            s = K @ q[i, h] * scaling
            w = np.exp(s - s.max())
            w /= w.sum()
            out[i, h] = w @ V
            mag[i, h] = w @ np.abs(V)
            big = max(big, float((np.abs(K) @ np.abs(q[i, h])).max()) * scaling)
    return out, mag, big, kv_len


def attention_bound(out, mag, big, keys, d, dtype):
    """A score's dot product is off by at most d half-steps of its magnitude sum (and the
    exponent's argument by a few half-steps of its size, under the same sum), an exponential
    by 2^-21 relative; both enter numerator and denominator. Sums over the keys: `keys`
    half-steps each (a tile's sum, then one addition per tile or split). bf16: weights are
    rounded to bf16 once for the product with V, the output once.

    An E4M3 cache is held to the bf16 bound: its weights are rounded to f16 (2^-11), which leaves
    2^-8 - 2^-11 for the queries, whose two codes are off by at most 2^-17 of the row's largest
    power of two: scores by 2^-17 max|q| sum|k| scaling, weights (numerator and denominator) by
    twice that. So max|q| sum|k| scaling <= (2^-8 - 2^-11) 2^16 = 224 is asked of the inputs: a
    normed query of 128 dims has no element above sqrt(128) 1.8 = 20.4, normal keys average below
    0.9 in magnitude, and 20.4 * 128 * 0.9 * 128^-0.5 = 208."""
    rel = 2 * ((d + 8) * U32 * max(big, 1.0) + 2.0 ** -21 + keys * U32)
    err = mag * rel
    if dtype == "f32":
        return err + np.abs(out) * U32 + 1e-37
    err = err + mag * (1 + rel) * HALF_STEP["bf16"]
    return err + (np.abs(out) + err) * HALF_STEP["bf16"] + 1e-37
