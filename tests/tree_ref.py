"""Trees and beams written out in float64 with loops, straight from their formulas, and the error
bounds the kernels are held to."""
import numpy as np

import chunk_ref as R


def random_tree(rng, n, width=4):
    """Parents of n nodes: 0 the root, each later one below one of the last 2 * width."""
    return [-1] + [int(rng.integers(max(0, i - 2 * width), i)) for i in range(1, n)]


def tree_map(cu, kv_lens, parents, before, depths, masks, max_nodes):
    """positions by row, nodes, and the depths and masks (bit sets as whole numbers, one list per
    sequence), continued from what the earlier nodes have; refused sequences are None."""
    pos, nodes = {}, list(before)
    depths, masks = [list(d) for d in depths], [list(m) for m in masks]
    refused = []
    for b, t0 in enumerate(before):
        lo, hi = int(cu[b]), int(cu[b + 1])
        n, kv = hi - lo, kv_lens[b]
        par = [int(u) for u in parents[lo:hi]]
        if n and (kv == 0 or t0 + n > max_nodes or kv < t0 + n or any(not -1 <= u < t0 + i for i, u in enumerate(par))):
            refused.append(b)
            continue
        for i, u in enumerate(par):
            depths[b].append(0 if u < 0 else depths[b][u] + 1)
            masks[b].append((1 << (t0 + i)) | (0 if u < 0 else masks[b][u]))
            pos[lo + i] = kv - n - t0 + depths[b][t0 + i]
        nodes[b] = t0 + n
    return pos, nodes, depths, masks, refused


def words(mask, max_nodes):
    """A bit set as int32 words."""
    return np.frombuffer(mask.to_bytes(max_nodes // 8, "little"), dtype=np.int32)


def visible(kv, nodes, node, depths, mask, window):
    """Cache rows that a node sees."""
    ctx = kv - nodes
    p = ctx + depths[node]
    keys = [j for j in range(ctx) if not window or p - j < window]
    return keys + [ctx + u for u in range(node + 1) if mask >> u & 1 and (not window or depths[node] - depths[u] < window)]


def attention(q, k, v, keys, G, scaling):
    """q [n][n_h][d], k / v [rows][n_kv][d], keys: the rows each query sees. As chunk_ref.attention."""
    n, n_h, d = q.shape
    out, mag, big, most = np.zeros((n, n_h, d)), np.zeros((n, n_h, d)), 0.0, 0
    for i in range(n):
        most = max(most, len(keys[i]))
        if not keys[i]:
            continue
        for h in range(n_h):
            K, V = k[keys[i], h // G], v[keys[i], h // G]
            s = K @ q[i, h] * scaling
            w = np.exp(s - s.max())
            w /= w.sum()
            out[i, h] = w @ V
            mag[i, h] = w @ np.abs(V)
            big = max(big, float((np.abs(K) @ np.abs(q[i, h])).max()) * scaling)
    return out, mag, big, most


attention_bound = R.attention_bound


def accept(parents, tokens, posterior, max_path):
    """Path from node 0 and the anchor behind it."""
    path = [0]
    while len(path) < max_path:
        u = path[-1]
        kids = [i for i in range(u + 1, len(parents)) if parents[i] == u and tokens[i] == posterior[u]]
        if not kids:
            break
        path.append(kids[0])
    return path, posterior[path[-1]]


def beam_select(logits, scores, k):
    """logits [beams][vocab], scores [beams] float64: tokens, beams, scores of the k best."""
    beams, V = logits.shape
    out = np.full((beams, V), -np.inf)
    for i in range(beams):
        x = logits[i]
        m = np.max(x) if not np.isnan(x).any() else np.nan
        if not np.isfinite(m) or not np.isfinite(scores[i]):
            continue
        with np.errstate(divide="ignore"):
            out[i] = scores[i] + ((x - m) - np.log(np.exp(x - m).sum()))
    flat = out.reshape(-1)
    order = np.lexsort((np.arange(flat.size), -flat))[:k]
    return order % V, order // V, flat[order]


def beam_bound(score):
    """The result is rounded to fp32 once. Of the log-sum: a term e^d is off by d's own rounding
    (2^-24 |d|, weighted by e^d: at most log V < 13 of them on average), 2^f by 2^-22 and f by two
    roundings below 1 (2^-24 each), so the sum, relative, and its logarithm, absolute, by 13 2^-24 +
    2^-22 + 2^-23 < 2^-19."""
    return np.abs(score) * 2.0 ** -24 + 2.0 ** -19
