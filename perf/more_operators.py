"""Speculative trees and beams over a KV cache, as measured workloads.

A round that verifies a tree of drafted tokens, or a step of a beam search that keeps its
hypotheses as a tree behind one committed prefix, makes these calls next to the chunk step's:

  select  the k best of beams x vocabulary by accumulated log-probability: a level of a drafted
          tree, a beam search's step, the target's greedy choice per node (dflash_beam_select)
  map     positions, depths and ancestor masks of a step's rows, the newest nodes of their
          sequences' trees (dflash_tree_map)
  attn    attention of those rows over the committed rows and their own ancestors, with an
          optional sliding window (dflash_tree_attn)
  accept  the path of nodes that the target agrees with (dflash_tree_accept)
  commit  that path's K and V rows moved up behind the committed ones, in every layer
          (dflash_tree_commit)

Where ``own`` is false the operators run in their plain form, elementary torch operations in 32
bits (select in 64: near ties between beams are decided there). Where it is true they are the
library's calls.
"""

import math
import random

import torch

own = False

PAGE = 128      # rows of a cache page
DEEP = 16       # nodes of the longest path of a verified tree (the root and a block of 15 drafts)


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------

def _select(name, dtype, batch, beams, vocab, k, shared=False, base=0, ban=False, dead=0):
    return {"name": name, "op": "select", "dtype": dtype, "batch": batch, "beams": beams, "vocab": vocab,
            "k": k, "shared": shared, "base": base, "ban": ban, "dead": dead}


def _map(name, batch, rows, before=(0, 0), width=8, max_nodes=128, ctx=(256, 4096), pad=0, lens=1):
    return {"name": name, "op": "map", "batch": batch, "rows_lo": rows[0], "rows_hi": rows[1],
            "before_lo": before[0], "before_hi": before[1], "width": width, "max_nodes": max_nodes,
            "ctx_lo": ctx[0], "ctx_hi": ctx[1], "pad": pad, "lens": lens}


def _attn(name, kv, batch, rows, ctx, before=(0, 0), width=8, max_nodes=128, heads=(32, 8, 128), window=0, lens=1):
    return dict(_map(name, batch, rows, before, width, max_nodes, ctx, 0, lens), op="attn", kv=kv,
                n_h=heads[0], n_kv=heads[1], d_h=heads[2], window=window)


def _accept(name, batch, rows, width=8, agree=0.8, pad=0, lens=1):
    return dict(_map(name, batch, rows, (0, 0), width, 0, (0, 4096), pad, lens), op="accept", agree=agree)


def _commit(name, kv, batch, rows, path, layers, ctx, heads=(32, 8, 128), lens=1):
    return dict(_map(name, batch, rows, (0, 0), 8, 0, ctx, 0, lens), op="commit", kv=kv, path_lo=path[0],
                path_hi=path[1], layers=layers, n_h=heads[0], n_kv=heads[1], d_h=heads[2])


def listed():
    return [
        # one level of a drafted tree for one sequence: eight beams over one row of block marginals
        _select("select_level_b1", "bf16", 1, 8, 32000, 8, shared=True, base=1),
        # a beam search's step of a serving batch
        _select("select_beams_b32", "bf16", 32, 8, 131072, 16),
        # float32 logits of an odd vocabulary, with banned tokens and finished beams
        _select("select_f32_b64", "f32", 64, 4, 50001, 8, ban=True, dead=1),
        # the tree of a verification round: 64 nodes each
        _map("map_verify_b32", 32, (64, 64)),
        # a beam search's step behind hundreds of nodes that are in the cache already
        _map("map_beams_b64", 64, (9, 16), before=(200, 900), width=16, max_nodes=1024),
        # one sequence, a small tree: nothing but latency
        _attn("tree_b1", "bf16", 1, (16, 16), (1023, 1023)),
        # verification of 64-node trees at the serving lengths
        _attn("tree_verify_b32", "bf16", 32, (64, 64), (256, 4096)),
        # beams of a long generation on the one-byte cache, in a layer with a sliding window
        _attn("tree_beams_fp8_b16", "fp8", 16, (9, 16), (1024, 8192), before=(100, 500), width=16,
              max_nodes=1024, window=4096),
        # acceptance of the round above
        _accept("accept_b32", 32, (64, 64)),
        # the same for a large ragged batch
        _accept("accept_b512", 512, (17, 200), width=20, pad=9),
        # a draft model's two layers after the round
        _commit("commit_b32", "bf16", 32, (64, 64), (1, 8), 2, (256, 1024)),
        # a deeper model's sixteen, many sequences with short contexts
        _commit("commit_b64", "bf16", 64, (40, 128), (4, 16), 16, (0, 120)),
    ]


def _log(rng, lo, hi):
    """A whole number in [lo, hi], spread over its logarithm."""
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def draw(rng):
    op = rng.choice(("select", "select", "map", "attn", "attn", "attn", "accept", "commit"))
    lens = rng.randrange(1 << 20)
    if op == "select":
        dtype = rng.choice(("bf16", "bf16", "f32"))
        vocab = _log(rng, 100, 200000)
        most = 32000000 if dtype == "bf16" else 12000000
        beams = _log(rng, 1, 16)
        batch = _log(rng, 1, max(1, min(256, most // (vocab * beams))))
        c = _select("", dtype, batch, beams, vocab, _log(rng, 1, min(64, vocab)),
                    shared=rng.random() < 0.25, base=rng.choice((0, 1, 17)), ban=rng.random() < 0.4,
                    dead=rng.choice((0, 0, rng.randint(0, beams - 1))))
    elif op == "map" or op == "accept":
        batch = _log(rng, 1, 256)
        hi = _log(rng, 1, max(1, min(300, 40000 // batch)))
        rows, width = (rng.randint(1, hi), hi), _log(rng, 1, 24)
        if op == "accept":
            c = _accept("", batch, rows, width, rng.choice((0.3, 0.8, 0.95)), rng.randint(0, 5), lens)
        else:
            before = rng.choice((0, _log(rng, 1, 700)))
            c = _map("", batch, rows, (before // 2, before), width, rng.choice((1024, 1024, 2048)),
                     (0, _log(rng, 1, 8192)), rng.randint(0, 5), lens)
    elif op == "attn":
        kv = rng.choice(("bf16", "bf16", "bf16", "fp8", "fp8", "f32"))
        if kv == "f32":
            heads = rng.choice(((8, 8, 64), (4, 2, 80), (8, 1, 128), (6, 2, 32)))
        else:
            heads = rng.choice(((32, 8, 128), (32, 8, 128), (16, 16, 128), (20, 4, 128), (14, 2, 128),
                                (8, 1, 128), (64, 4, 128)))
        n_h, n_kv, d_h = heads
        batch = _log(rng, 1, 32)
        before = rng.choice((0, 0, _log(rng, 1, 500)))
        # bounds: the plain form's padded scores, the cache rows read
        per = (3.0e8 if kv != "f32" else 1.0e8) / (batch * n_h)
        ctx = _log(rng, 1, max(1, min(32768, 100000000 // (batch * n_kv * d_h))))
        hi = _log(rng, 1, max(1, min(256, int(per / (ctx + before + 256)))))
        c = _attn("", kv, batch, (rng.randint(1, hi), hi), (rng.randint(0, ctx), ctx), (before // 2, before),
                  _log(rng, 1, 24), 1024, heads, rng.choice((0, 0, _log(rng, 1, 4096))), lens)
    else:
        kv = rng.choice(("bf16", "fp8", "f32"))
        heads = rng.choice(((32, 8, 128), (8, 2, 128))) if kv != "f32" else rng.choice(((8, 8, 64), (4, 2, 80)))
        hi = _log(rng, 2, 200)
        path = rng.randint(1, max(1, min(16, hi // 2)))
        batch = _log(rng, 1, 64)
        ctx = _log(rng, 1, 400)
        layers = _log(rng, 1, max(1, min(16, 2000000 // (batch * heads[1] * (ctx + hi + PAGE)))))
        c = _commit("", kv, batch, (rng.randint(2 * path, max(2 * path, hi)), max(2 * path, hi)),
                    (rng.randint(1, path), path), layers, (0, ctx), heads, lens)
    del c["name"]
    return c


# ---------------------------------------------------------------------------
# lengths and trees: the same for every seed of a case
# ---------------------------------------------------------------------------

def _lengths(case):
    """New nodes, nodes already in the cache and committed rows of every sequence."""
    r = random.Random(case["lens"])
    B = case["batch"]
    rows = [r.randint(case["rows_lo"], case["rows_hi"]) for _ in range(B)]
    before = [r.randint(case["before_lo"], case["before_hi"]) for _ in range(B)]
    ctx = [r.randint(case["ctx_lo"], case["ctx_hi"]) for _ in range(B)]
    return rows, before, ctx


def _tree(r, n, width, deep):
    """Parents of n nodes: node 0 the root, later ones below one of the last 2 * width, the
    likelier the earlier it is (the better drafts have more children), no path longer than deep."""
    parents, depth = [-1], [1]
    for i in range(1, n):
        lo = max(0, i - 2 * width)
        p = lo + int((i - lo) * r.random() ** 2)
        while depth[p] >= deep:
            p = parents[p]
        parents.append(p)
        depth.append(depth[p] + 1)
    return parents


def _depths(parents):
    d = []
    for p in parents:
        d.append(0 if p < 0 else d[p] + 1)
    return d


def _trees(case, seed=0):
    """Parents of every sequence's nodes, those in the cache first."""
    rows, before, _ = _lengths(case)
    r = random.Random(case["lens"] * 1000003 + seed)
    deep = DEEP if case["op"] == "accept" else 1 << 30
    return [_tree(r, n + t, case["width"], deep) for n, t in zip(rows, before)]


def _scales(kv):
    return (0.03125, 0.0078125) if kv == "fp8" else (1.0, 1.0)


# ---------------------------------------------------------------------------
# what a program has in hand before the call
# ---------------------------------------------------------------------------

def _i32(v, dev="cuda"):
    return torch.tensor(v, dtype=torch.int32, device=dev)


def _starts(rows):
    cu = [0]
    for n in rows:
        cu.append(cu[-1] + n)
    return cu


def _masks(parents, max_nodes, dev):
    """Ancestor bits (a node's own among them) [batch][max_nodes][max_nodes / 32] and depths
    [batch][max_nodes] of whole trees; the bits as int32 words, bit u of word u / 32 for node u."""
    B, W = len(parents), max_nodes // 32
    words = torch.zeros((B, max_nodes, W), dtype=torch.int32)
    depths = torch.zeros((B, max_nodes), dtype=torch.int32)
    for b, par in enumerate(parents):
        bits = []
        for i, p in enumerate(par):
            bits.append((1 << i) | (bits[p] if p >= 0 else 0))
        if par:
            raw = bytearray(b"".join(v.to_bytes(4 * W, "little") for v in bits))
            words[b, :len(par)] = torch.frombuffer(raw, dtype=torch.int32).reshape(len(par), W)
            depths[b, :len(par)] = torch.tensor(_depths(par), dtype=torch.int32)
    return words.to(dev), depths.to(dev)


def _prepare_select(case, seed):
    dev = "cuda"
    g = torch.Generator(device=dev).manual_seed(int(seed))
    B, beams, V = case["batch"], case["beams"], case["vocab"]
    dt = torch.float32 if case["dtype"] == "f32" else torch.bfloat16
    shape = (B, 1 if case["shared"] else beams, V)
    x = torch.randn(shape, generator=g, device=dev) * 2.0
    # a few likely tokens per row
    likely = torch.randint(0, V, shape[:2] + (12,), generator=g, device=dev)
    x.scatter_add_(2, likely, 9.0 * torch.rand(likely.shape, generator=g, device=dev))
    if case["ban"]:
        x.masked_fill_(torch.rand(shape, generator=g, device=dev) < 0.02, float("-inf"))
    x = x.to(dt)
    scores = -3.0 * torch.rand((B, beams), generator=g, device=dev)
    if case["dead"]:
        scores[:, beams - case["dead"]:] = float("-inf")
    s = {"op": "select", "logits": x.expand(B, beams, V) if case["shared"] else x, "scores": scores,
         "k": case["k"], "base": case["base"], "batch": B, "beams": beams, "vocab": V}
    s["tokens"], s["parents"] = (torch.zeros((B, case["k"]), dtype=torch.int32, device=dev) for _ in range(2))
    s["out"] = torch.zeros((B, case["k"]), dtype=torch.float32, device=dev)
    if own:
        from speculative_decoding_draft_dflash_gb300 import dflash
        s["ws"] = torch.empty(dflash.dflash_beam_workspace_bytes(B, beams, V, case["k"]), dtype=torch.uint8, device=dev)
    return s


def _prepare_map(case, seed):
    dev = "cuda"
    rows, before, ctx = _lengths(case)
    trees = _trees(case, int(seed))
    N = case["max_nodes"]
    cu = _starts(rows)
    M = cu[-1] + case["pad"]
    # the nodes in the cache have their masks and depths; those of the step are to come
    masks, depths = _masks([t[:k] for t, k in zip(trees, before)], N, dev)
    new = [p for t, k in zip(trees, before) for p in t[k:]] + [0] * case["pad"]
    total = [c + k + n for c, k, n in zip(ctx, before, rows)]
    s = {"op": "map", "batch": case["batch"], "rows": M, "n_rows": max(rows), "max_nodes": N, "cu_rows": _i32(cu),
         "parents": _i32(new), "before": _i32(before), "nodes": _i32([0] * len(rows)), "masks": masks,
         "depths": depths, "kv_lens": _i32(total), "slots": _i32([0] * cu[-1] + [-1] * case["pad"]),
         "positions": _i32([-1] * M), "depth_max": max(max(_depths(t)) for t in trees)}
    if own:
        from speculative_decoding_draft_dflash_gb300 import dflash
        s["plan"] = dflash.ChunkPlan(s["cu_rows"], M, s["kv_lens"], s["slots"], s["positions"])
        s["tree"] = dflash.Tree(case["batch"], N, nodes=s["nodes"], depths=depths, masks=masks)
    return s


def _cache(case, total, seed, layers):
    """Paged cache rows (contiguous for f32): K, V of every layer and the block table."""
    dev = "cuda"
    g = torch.Generator(device=dev).manual_seed(int(seed))
    kv, n_kv, d_h, B = case["kv"], case["n_kv"], case["d_h"], case["batch"]
    pps = max(1, -(-max(total) // PAGE))
    n_pages = sum(-(-t // PAGE) for t in total) + 3
    table = torch.zeros((B, pps), dtype=torch.int32, device=dev)
    used = torch.arange(pps, device=dev)[None] < ((_i32(total)[:, None] + PAGE - 1) // PAGE)
    table[used] = torch.randperm(n_pages, generator=g, device=dev).int()[:n_pages - 3]
    paged = kv != "f32"
    shape = (n_pages, n_kv, PAGE, d_h) if paged else (B, n_kv, pps * PAGE, d_h)
    dt = {"f32": torch.float32, "bf16": torch.bfloat16, "fp8": torch.uint8}[kv]
    K, V = (torch.empty((layers,) + shape, dtype=dt, device=dev) for _ in range(2))
    for l in range(layers):
        for t, scale, size in ((K, _scales(kv)[0], 1.0), (V, _scales(kv)[1], 0.25)):
            x = torch.randn(shape, generator=g, device=dev)
            if kv == "fp8":
                x = (x * size / scale).clamp_(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
            t[l].copy_(x)
    return K, V, table, paged, pps, n_pages, g


def _own_cache(s, case):
    from speculative_decoding_draft_dflash_gb300 import dflash
    dt = torch.float32 if case["kv"] == "f32" else torch.bfloat16
    L = s["k"].shape[0]
    c = dflash.KVCache(L, case["batch"], case["n_kv"], s["pps"] * PAGE, case["d_h"], dt, "cuda",
                       page_table=s["table"] if s["paged"] else None, n_pages=s["n_pages"] if s["paged"] else None,
                       kv="fp8" if case["kv"] == "fp8" else "bf16", kv_scales=[_scales(case["kv"])] * L)
    c.k.copy_(s["k"])
    c.v.copy_(s["v"])
    s["cache"], s["k"], s["v"] = c, c.k, c.v
    s["dims"] = dflash.make_dims(case["n_h"] * case["d_h"], case["n_h"], case["n_kv"], case["d_h"], 1, 1, 1e-6, dt)
    return dflash


def _prepare_attn(case, seed):
    dev = "cuda"
    rows, before, ctx = _lengths(case)
    total = [c + k + n for c, k, n in zip(ctx, before, rows)]
    K, V, table, paged, pps, n_pages, g = _cache(case, total, seed, 1)
    masks, depths = _masks(_trees(case), case["max_nodes"], dev)
    cu = _starts(rows)
    M = cu[-1]
    dt = torch.float32 if case["kv"] == "f32" else torch.bfloat16
    s = dict(op="attn", kv=case["kv"], batch=case["batch"], n_h=case["n_h"], n_kv=case["n_kv"], d_h=case["d_h"],
             window=case["window"], scales=_scales(case["kv"]), M=M, rows_max=max(rows), kv_max=max(total), k=K, v=V,
             table=table, paged=paged, pps=pps, n_pages=n_pages, masks=masks, depths=depths, cu_rows=_i32(cu),
             kv_lens=_i32(total), nodes=_i32([k + n for k, n in zip(before, rows)]), max_nodes=case["max_nodes"],
             slots=_i32([-1] * M), positions=_i32([-1] * M))
    s["q"] = torch.randn((M, s["n_h"] * s["d_h"]), generator=g, device=dev).to(dt)
    s["out"] = torch.zeros_like(s["q"])
    if own:
        dflash = _own_cache(s, case)
        s["plan"] = dflash.ChunkPlan(s["cu_rows"], M, s["kv_lens"], s["slots"], s["positions"])
        s["tree"] = dflash.Tree(case["batch"], case["max_nodes"], nodes=s["nodes"], depths=depths, masks=masks)
        s["ws"] = torch.empty(dflash.dflash_chunk_workspace_bytes(s["dims"]), dtype=torch.uint8, device=dev)
    return s


def _prepare_accept(case, seed):
    dev = "cuda"
    rows, _, ctx = _lengths(case)
    trees = _trees(case, int(seed))
    r = random.Random(int(seed))
    cu = _starts(rows)
    M = cu[-1] + case["pad"]
    tokens, posterior = [], []
    for par in trees:
        tok = [r.randrange(32000) for _ in par]
        kids = [[] for _ in par]
        for i, p in enumerate(par):
            if p >= 0:
                kids[p].append(i)
        tokens += tok
        # the target agrees with one of a node's children, or says something else
        posterior += [tok[r.choice(c)] if c and r.random() < case["agree"] else r.randrange(32000) for c in kids]
    pad = [0] * case["pad"]
    B = case["batch"]
    s = {"op": "accept", "batch": B, "rows": M, "width": DEEP, "n_rows": max(rows), "cu_rows": _i32(cu),
         "parents": _i32([p for t in trees for p in t] + pad), "tokens": _i32(tokens + pad),
         "posterior": _i32(posterior + pad), "ctx_len": _i32(ctx), "kv_lens": _i32([c + n for c, n in zip(ctx, rows)]),
         "slots": _i32([0] * M), "positions": _i32([0] * M),
         "accept_len": _i32([0] * B), "path": torch.zeros((B, DEEP), dtype=torch.int32, device=dev),
         "next_cu_rows": _i32([0] * (B + 1)), "ctx_next": _i32([0] * B), "next_anchor": _i32([0] * B)}
    if own:
        from speculative_decoding_draft_dflash_gb300 import dflash
        s["plan"] = dflash.ChunkPlan(s["cu_rows"], M, s["kv_lens"], s["slots"], s["positions"])
    return s


def _paths(case):
    """Accepted paths (node numbers, node 0 first). A path stays among its own first numbers or
    leaves them for good, so that a pass may be repeated on the rows that it left."""
    rows, _, _ = _lengths(case)
    r = random.Random(case["lens"] + 7)
    out = []
    for n in rows:
        a = min(r.randint(case["path_lo"], case["path_hi"]) - 1, (n - 1) // 2)
        keep = r.randint(0, a) if r.random() < 0.3 else 0
        out.append(list(range(keep + 1)) + sorted(r.sample(range(a + 1, n), a - keep)))
    return out


def _prepare_commit(case, seed):
    rows, _, ctx = _lengths(case)
    paths = _paths(case)
    K, V, table, paged, pps, n_pages, _ = _cache(case, [c + n for c, n in zip(ctx, rows)], seed, case["layers"])
    w = max(len(p) for p in paths)
    s = dict(op="commit", kv=case["kv"], batch=case["batch"], k=K, v=V, table=table, paged=paged, pps=pps,
             n_pages=n_pages, layers=case["layers"], ctx_len=_i32(ctx), nodes=_i32(rows), width=w,
             path=_i32([p + [-1] * (w - len(p)) for p in paths]), accept_len=_i32([len(p) - 1 for p in paths]),
             lens=_i32([[c + n for c, n in zip(ctx, rows)]] * case["layers"]))
    if own:
        dflash = _own_cache(s, case)
        s["cache"].lens.copy_(s["lens"])
        s["lens"] = s["cache"].lens
        s["tree"] = dflash.Tree(case["batch"], -(-max(rows) // 32) * 32, nodes=s["nodes"])
    return s


def prepare(case, seed):
    return {"select": _prepare_select, "map": _prepare_map, "attn": _prepare_attn, "accept": _prepare_accept,
            "commit": _prepare_commit}[case["op"]](case, seed)


# ---------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------

def run(s):
    return (_OWN if own else _PLAIN)[s["op"]](s)


def _value(s, t):
    return t.view(torch.float8_e4m3fn) if s["kv"] == "fp8" else t


def _own_select(s):
    from speculative_decoding_draft_dflash_gb300 import dflash
    dflash.dflash_beam_select(s["logits"], s["scores"], s["k"], s["tokens"], s["parents"], s["out"], s["ws"],
                              parent_base=s["base"])
    return {"tokens": s["tokens"], "parents": s["parents"], "scores": s["out"]}


def _own_map(s):
    from speculative_decoding_draft_dflash_gb300 import dflash
    dflash.dflash_tree_map(s["plan"], s["tree"], s["parents"], s["before"])
    return {k: s[k] for k in ("positions", "nodes", "depths", "masks")}


def _own_attn(s):
    from speculative_decoding_draft_dflash_gb300 import dflash
    dflash.dflash_tree_attn(s["dims"], s["cache"], 0, s["plan"], s["tree"], s["q"], s["window"], 0.0, s["out"], s["ws"])
    return s["out"]


def _own_accept(s):
    from speculative_decoding_draft_dflash_gb300 import dflash
    dflash.dflash_tree_accept(s["plan"], s["parents"], s["tokens"], s["posterior"], s["ctx_len"], s["accept_len"],
                              s["path"], s["next_cu_rows"], s["ctx_next"], s["next_anchor"])
    return {k: s[k] for k in ("accept_len", "path", "next_cu_rows", "ctx_next", "next_anchor")}


def _own_commit(s):
    from speculative_decoding_draft_dflash_gb300 import dflash
    dflash.dflash_tree_commit(s["dims"], s["cache"], s["tree"], s["ctx_len"], s["path"], s["accept_len"])
    return {"k": _value(s, s["k"]), "v": _value(s, s["v"]), "lens": s["lens"]}


def _plain_select(s):
    x = s["logits"].double()
    m = x.amax(-1, keepdim=True)
    total = (x - m).exp().sum(-1, keepdim=True)
    score = s["scores"].double()[..., None] + ((x - m) - total.log())
    # a row without a probability gives its beam no candidate; -inf candidates rank by their place
    low, used = -1e300, float("-inf")
    score = torch.where(torch.isfinite(score) & torch.isfinite(total), score, low)
    flat = score.reshape(s["batch"], -1)
    at, best = [], []
    for _ in range(s["k"]):
        v, i = flat.max(-1, keepdim=True)
        best.append(v)
        at.append(i)
        flat.scatter_(1, i, used)
    at, best = torch.cat(at, 1), torch.cat(best, 1)
    V = s["vocab"]
    return {"tokens": (at % V).int(), "parents": (at // V + s["base"]).int(),
            "scores": torch.where(best > low, best, used).float()}


def _plain_map(s):
    N, B = s["max_nodes"], s["batch"]
    dev = s["masks"].device
    cu, before = s["cu_rows"].long(), s["before"].long()
    n = cu[1:] - cu[:-1]
    r = torch.arange(s["rows"], device=dev)
    b = (torch.searchsorted(cu, r, right=True) - 1).clamp(max=B - 1)
    live = r < cu[-1]
    node = before[b] + r - cu[b]
    up = torch.where(live, s["parents"].long(), -1)
    seen = torch.zeros((s["rows"], N), dtype=torch.bool, device=dev)
    seen[r[live], node[live]] = True
    depth = torch.zeros_like(r)
    old = torch.full_like(r, -1)            # the ancestor that was in the cache before
    for _ in range(s["depth_max"] + 1):
        mine = up >= before[b]
        old = torch.where((up >= 0) & ~mine, up, old)
        seen[r[mine], up[mine]] = True
        depth += mine
        nxt = s["parents"].long()[(cu[b] + up - before[b]).clamp(0, s["rows"] - 1)]
        up = torch.where(mine, nxt, -1)
    depth = torch.where(old >= 0, depth + 1 + s["depths"][b, old.clamp(min=0)], depth)
    bits = seen.reshape(s["rows"], N // 32, 32).long() << torch.arange(32, device=dev)
    words = bits.sum(-1)
    words = torch.where(words >= 1 << 31, words - (1 << 32), words).int()
    words |= torch.where(old[:, None] >= 0, s["masks"][b, old.clamp(min=0)], 0)
    s["masks"][b[live], node[live]] = words[live]
    s["depths"][b[live], node[live]] = depth[live].int()
    ctx = s["kv_lens"].long() - n - before
    return {"positions": torch.where(live, ctx[b] + depth, -1).int(), "nodes": (before + n).int(),
            "depths": s["depths"], "masks": s["masks"]}


def _visible(s, b_rows):
    """[B][rows][keys]: which cache rows the new nodes of every sequence see."""
    dev = s["q"].device
    cu, kv, nodes = s["cu_rows"].long(), s["kv_lens"].long(), s["nodes"].long()
    n = cu[1:] - cu[:-1]
    ctx = kv - nodes
    j = torch.arange(s["kv_max"], device=dev)
    node = ((nodes - n)[:, None] + b_rows).clamp(max=s["max_nodes"] - 1)
    at = torch.arange(s["batch"], device=dev)[:, None]
    u = (j[None] - ctx[:, None]).clamp(0, s["max_nodes"] - 1)             # node of a key
    word = s["masks"][at[..., None], node[..., None], (u // 32)[:, None]]
    bit = (word >> (u % 32)[:, None]) & 1
    seen = (j < ctx[:, None])[:, None] | ((bit != 0) & (j < kv[:, None])[:, None])
    if s["window"] > 0:
        pos = ctx[:, None] + s["depths"].long()[at, node]
        kpos = torch.where(j < ctx[:, None], j, ctx[:, None] + s["depths"].long()[at, u])
        seen &= pos[..., None] - kpos[:, None] < s["window"]
    return seen


def _plain_attn(s):
    B, n_h, n_kv, d_h, G = s["batch"], s["n_h"], s["n_kv"], s["d_h"], s["n_h"] // s["n_kv"]
    cu = s["cu_rows"].long()
    n = cu[1:] - cu[:-1]
    i = torch.arange(s["rows_max"], device=s["q"].device)
    at = (cu[:-1, None] + i).clamp(max=s["M"] - 1)
    q = s["q"].reshape(s["M"], n_kv, G, d_h)[at].float().permute(0, 2, 1, 3, 4).reshape(B, n_kv, -1, d_h)
    j = torch.arange(s["kv_max"], device=s["q"].device)

    def rows(t):
        if s["paged"]:
            page = s["table"].long()[:, j // PAGE]
            return _value(s, t[0][page, :, (j % PAGE)[None]]).float().permute(0, 2, 1, 3)
        return t[0][:, :, :s["kv_max"]].float()

    x = q @ rows(s["k"]).transpose(-1, -2)
    x *= d_h ** -0.5 * s["scales"][0]
    hidden = ~_visible(s, i)[:, None, :, None, :].expand(B, 1, s["rows_max"], G, s["kv_max"])
    x.masked_fill_(hidden.reshape(B, 1, -1, s["kv_max"]), float("-inf"))
    x -= x.amax(-1, keepdim=True).clamp(min=-3e38)
    x.exp_()
    total = x.sum(-1, keepdim=True)
    o = (x @ rows(s["v"])) * (s["scales"][1] / total.clamp(min=1e-37))
    o = o.reshape(B, n_kv, s["rows_max"], G, d_h).permute(0, 2, 1, 3, 4)
    return o[i[None] < n[:, None]].reshape(s["M"], n_h * d_h).to(s["q"].dtype)


def _plain_accept(s):
    B, W = s["batch"], s["width"]
    cu = s["cu_rows"].long()
    n = cu[1:] - cu[:-1]
    i = torch.arange(s["n_rows"], device=cu.device)
    inside = i[None] < n[:, None]
    at = (cu[:-1, None] + i).clamp(max=s["rows"] - 1)
    parents = torch.where(inside, s["parents"][at], -2)
    tokens, posterior = s["tokens"][at], s["posterior"][at]
    path = torch.full((B, W), -1, dtype=torch.int32, device=cu.device)
    cur = torch.zeros((B, 1), dtype=torch.long, device=cu.device)
    path[:, 0] = 0
    length = torch.zeros((B, 1), dtype=torch.int32, device=cu.device)
    alive = torch.ones((B, 1), dtype=torch.bool, device=cu.device)
    for step in range(1, W):
        hit = (parents == cur) & (tokens == posterior.gather(1, cur)) & alive
        first = torch.where(hit, i[None], s["n_rows"]).amin(-1, keepdim=True)
        alive = first < s["n_rows"]
        cur = torch.where(alive, first, cur)
        path[:, step] = torch.where(alive, first, -1).int()[:, 0]
        length += alive
    a = length[:, 0]
    nxt = torch.cat((torch.zeros_like(a[:1]), (a + 1).cumsum(0).int()))
    return {"accept_len": a, "path": path, "next_cu_rows": nxt, "ctx_next": s["ctx_len"] + a + 1,
            "next_anchor": posterior.gather(1, cur)[:, 0]}


def _plain_commit(s):
    i = torch.arange(s["width"], device=s["path"].device)
    ctx, a = s["ctx_len"].long(), s["accept_len"].long()
    b, i = torch.nonzero(i[None] <= a[:, None], as_tuple=True)
    src, dst = ctx[b] + s["path"].long()[b, i], ctx[b] + i
    for t in (s["k"], s["v"]):
        if s["paged"]:
            page = s["table"].long()
            x = t[:, page[b, src // PAGE], :, src % PAGE]
            t[:, page[b, dst // PAGE], :, dst % PAGE] = x
        else:
            x = t[:, b, :, src]
            t[:, b, :, dst] = x
    s["lens"][:] = (ctx + a + 1).int()
    return {"k": _value(s, s["k"]), "v": _value(s, s["v"]), "lens": s["lens"]}


_OWN = {"select": _own_select, "map": _own_map, "attn": _own_attn, "accept": _own_accept, "commit": _own_commit}
_PLAIN = {"select": _plain_select, "map": _plain_map, "attn": _plain_attn, "accept": _plain_accept,
          "commit": _plain_commit}


# ---------------------------------------------------------------------------
# what a pass cannot do without
# ---------------------------------------------------------------------------

def work(case):
    B = case["batch"]
    if case["op"] == "select":
        n = B * (1 if case["shared"] else case["beams"]) * case["vocab"]
        return {"bytes": n * (4 if case["dtype"] == "f32" else 2) + 4 * B * (case["beams"] + 3 * case["k"]), "flops": 4 * n}
    rows, before, ctx = _lengths(case)
    M = sum(rows)
    if case["op"] == "map":
        # parents in; position, depth and mask words out; masks of the old nodes that rows hang below
        words = case["max_nodes"] // 32
        old = sum(min(n, k) for n, k in zip(rows, before))
        return {"bytes": M * (12 + 4 * words) + old * (4 + 4 * words) + 16 * B, "flops": M * words}
    if case["op"] == "accept":
        return {"bytes": 12 * M + 4 * 6 * B, "flops": M}
    e = {"f32": 4, "bf16": 2, "fp8": 1}[case["kv"]] * case["d_h"] * case["n_kv"]
    if case["op"] == "commit":
        moved = sum(i != p for path in _paths(case) for i, p in enumerate(path))
        return {"bytes": case["layers"] * moved * 4 * e + sum(4 * len(p) for p in _paths(case)) + 4 * B * (2 + case["layers"]),
                "flops": 0}
    pairs = keys = 0
    for n, k, c, tree in zip(rows, before, ctx, _trees(case)):
        deep = _depths(tree)
        w = case["window"] or 1 << 30
        pairs += sum(min(d + 1, w) + max(0, min(c, w - 1 - d)) for d in deep[k:])
        # keys that some row sees: committed ones in the widest window, and the rows' ancestors
        used = set()
        for i in range(k, k + n):
            p, left = i, w
            while p >= 0 and p not in used and left > 0:
                used.add(p)
                p, left = tree[p], left - 1
        keys += max(0, min(c, w - 1 - min(deep[k:]))) + len(used)
    q = 4 if case["kv"] == "f32" else 2
    return {"bytes": 2 * M * case["n_h"] * case["d_h"] * q + 2 * keys * e, "flops": 4 * pairs * case["n_h"] * case["d_h"]}


# ---------------------------------------------------------------------------
# the definition, in 64 bits
# ---------------------------------------------------------------------------

def exact(case, seed):
    if case["op"] in ("map", "accept"):
        return None                            # whole numbers only
    s = prepare(case, seed)
    f64 = torch.float64
    if case["op"] == "commit":
        lens = s["lens"].clone()
        out = {"k": s["k"].clone(), "v": s["v"].clone()}
        for b, path in enumerate(_paths(case)):
            c = int(s["ctx_len"][b])
            for i, p in enumerate(path):
                for t in ("k", "v"):
                    if s["paged"]:
                        to, fr = (int(s["table"][b, x // PAGE]) for x in (c + i, c + p))
                        out[t][:, to, :, (c + i) % PAGE] = s[t][:, fr, :, (c + p) % PAGE]
                    else:
                        out[t][:, b, :, c + i] = s[t][:, b, :, c + p]
            lens[:, b] = c + len(path)
        return {"k": _value(s, out["k"]).to(f64), "v": _value(s, out["v"]).to(f64), "lens": None}
    if case["op"] == "select":
        best = []
        for b in range(case["batch"]):
            x = s["logits"][b].to(f64)
            p = s["scores"][b].to(f64)[:, None] + torch.log_softmax(x, -1)
            best.append(torch.sort(p.nan_to_num(nan=float("-inf")).flatten(), descending=True).values[:case["k"]])
        return {"tokens": None, "parents": None, "scores": torch.stack(best)}
    n_h, n_kv, d_h, G = s["n_h"], s["n_kv"], s["d_h"], s["n_h"] // s["n_kv"]
    rows, before, ctx = _lengths(case)
    if 4 * sum(n * (c + k + n) for n, k, c in zip(rows, before, ctx)) * n_h * d_h > 6e12:
        return None                            # too long in 64 bits
    sk, sv = s["scales"]
    out = torch.zeros((s["M"], n_h, d_h), dtype=f64, device=s["q"].device)
    lo = 0
    for b, tree in enumerate(_trees(case)):
        n, k, c = rows[b], before[b], ctx[b]
        L, deep = c + k + n, _depths(tree)
        keep = torch.zeros((n, L), dtype=torch.bool)
        for i in range(n):
            pos, p = c + deep[k + i], k + i
            first = max(0, pos - case["window"] + 1) if case["window"] else 0
            keep[i, first:c] = True
            while p >= 0 and c + deep[p] >= first:
                keep[i, c + p] = True
                p = tree[p]
        keep = keep.to(out.device)
        t = torch.arange(L, device=out.device)
        for h in range(n_kv):
            if s["paged"]:
                pg = s["table"][b, t // PAGE].long()
                kk, vv = s["k"][0][pg, h, t % PAGE], s["v"][0][pg, h, t % PAGE]
            else:
                kk, vv = s["k"][0][b, h, :L], s["v"][0][b, h, :L]
            kk, vv = _value(s, kk).to(f64) * sk, _value(s, vv).to(f64) * sv
            for g in range(h * G, (h + 1) * G):
                a = s["q"][lo:lo + n, g * d_h:(g + 1) * d_h].to(f64) @ kk.T / d_h ** 0.5
                out[lo:lo + n, g] = torch.softmax(a.masked_fill(~keep, float("-inf")), -1) @ vv
        lo += n
    return out.reshape(s["M"], n_h * d_h)
