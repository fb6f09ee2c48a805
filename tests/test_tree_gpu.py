"""Trees over a cache (map, attention, acceptance, commit) against their formulas in float64."""
import numpy as np
import pytest
import torch

import chunk_ref as R
import tree_ref as T
from test_chunk_gpu import DEV, HEADS, D, Step, i32, np64  # noqa: F401  (D is the fixture)

pytestmark = pytest.mark.gpu


def rng_of(seed):
    return np.random.Generator(np.random.PCG64(seed))


# ---------------------------------------------------------------------------
# map
# ---------------------------------------------------------------------------

class Trees:
    """Node arrays of a batch on the device, and the same as whole numbers."""

    def __init__(self, D, before, max_nodes, seed=0, width=4):
        r = rng_of(seed)
        self.max_nodes, self.before = max_nodes, list(before)
        B = len(before)
        par = [T.random_tree(r, n, width) if n else [] for n in before]
        cu = np.concatenate(([0], np.cumsum(before)))
        flat = [u for p in par for u in p]
        _, _, self.depths, self.masks, _ = T.tree_map(cu, [10 ** 6] * B, flat, [0] * B, [[]] * B, [[]] * B, max_nodes)
        self.tree = D.Tree(B, max_nodes, DEV)
        self.tree.masks.fill_(-1)              # what no node has is noise
        self.tree.depths.fill_(-7)
        self.upload(self.depths, self.masks)
        self.tree.nodes.fill_(-5)

    def upload(self, depths, masks):
        for b, (d, m) in enumerate(zip(depths, masks)):
            if d:
                self.tree.depths[b, :len(d)] = i32(d)
                self.tree.masks[b, :len(m)] = i32(np.stack([T.words(x, self.max_nodes) for x in m]))


def _check_map(D, tr, plan, cu, kv, parents, want_bits=0):
    pos, nodes, depths, masks, refused = T.tree_map(cu, kv, parents, tr.before, tr.depths, tr.masks, tr.max_nodes)
    got_pos, got_slot = plan.positions.tolist(), plan.slots.tolist()
    for b in range(len(nodes)):
        for row in range(int(cu[b]), int(cu[b + 1])):
            assert got_pos[row] == (-1 if b in refused else pos[row]), (b, row)
            assert (got_slot[row] == -1) == (b in refused)
    assert tr.tree.nodes.tolist() == nodes
    assert plan.kv_lens.tolist() == [0 if b in refused else k for b, k in enumerate(kv)]
    got_d, got_m = tr.tree.depths.cpu().numpy(), tr.tree.masks.cpu().numpy()
    for b, n in enumerate(nodes):
        assert got_d[b, :n].tolist() == depths[b]
        assert (got_d[b, n:] == -7).all() and (got_m[b, n:] == -1).all()     # nothing behind the last node
        for t in range(n):
            assert (got_m[b, t] == T.words(masks[b][t], tr.max_nodes)).all(), (b, t)
    assert D.dflash_status_get() == want_bits


@pytest.mark.parametrize("rows,before,max_nodes,pad", [
    ([1], [0], 32, 0), ([32, 0, 5], [0, 3, 27], 32, 2), ([64] * 5, [0] * 5, 64, 0), ([129, 400, 1], [300, 0, 511], 1024, 3),
    ([16] * 40, list(range(40)), 1024, 0), ([1000, 7], [1000, 2041], 2048, 1), ([4096, 300], [0, 3000], 4096, 0)])
def test_map(D, rows, before, max_nodes, pad):
    r = rng_of(max_nodes + len(rows))
    tr = Trees(D, before, max_nodes, seed=len(rows))
    cu = np.concatenate(([0], np.cumsum(rows)))
    M = int(cu[-1]) + pad
    parents = []
    for n, t in zip(rows, before):
        parents += [int(r.integers(max(-1, t + i - 9), t + i)) for i in range(n)]
    parents += [10 ** 8] * pad                       # padding is not looked at
    kv = [int(r.integers(0, 5000)) + n + t for n, t in zip(rows, before)]
    plan = D.ChunkPlan(i32(cu), M, kv_lens=i32(kv), slots=i32([5] * M), positions=i32([-77] * M))
    D.dflash_tree_map(plan, tr.tree, i32(parents), i32(before))
    _check_map(D, tr, plan, cu, kv, parents)
    assert plan.positions[int(cu[-1]):].tolist() == [-77] * pad and plan.slots[int(cu[-1]):].tolist() == [5] * pad


@pytest.mark.parametrize("shape", ["chain", "star", "comb"])
def test_map_of_extreme_trees(D, shape):
    n = 700
    parents = {"chain": [i - 1 for i in range(n)], "star": [-1] + [0] * (n - 1), "comb": [-1] * n}[shape]
    tr = Trees(D, [0, 0], 1024)
    plan = D.ChunkPlan(i32([0, n, 2 * n]), 2 * n, kv_lens=i32([n, n + 9]), slots=i32([0] * (2 * n)))
    D.dflash_tree_map(plan, tr.tree, i32(parents * 2))               # no nodes before
    _check_map(D, tr, plan, [0, n, 2 * n], [n, n + 9], parents * 2)


def test_map_refuses(D):
    rows, before = [3, 3, 3, 3, 2, 0, 2], [2, 0, 62, 1, 4, 9, 0]
    cu = np.concatenate(([0], np.cumsum(rows)))
    parents = [1, 2, 5] + [-1, -2, 0] + [1, 2, 3] + [0, 1, 1] + [0, 4] + [-1, 0]
    kv = [9, 9, 90, 3, 0, 12, 2]
    # 0: parent 5 of node 4; 1: -2; 2: 65 nodes of 64; 3: four nodes, three rows held; 4: refused by
    # the chunk map; 5: no new rows; 6: fine
    tr = Trees(D, before, 64)
    plan = D.ChunkPlan(i32(cu), int(cu[-1]), kv_lens=i32(kv), slots=i32([3] * int(cu[-1])))
    D.dflash_tree_map(plan, tr.tree, i32(parents), i32(before))
    assert T.tree_map(cu, kv, parents, before, tr.depths, tr.masks, 64)[4] == [0, 1, 2, 3, 4]
    _check_map(D, tr, plan, cu, kv, parents, D.DEV_TREE)
    # a negative count, and rows that run backwards (their sequence is refused, the others are not)
    tr = Trees(D, [0, 0, 0], 64)
    plan = D.ChunkPlan(i32([0, 4, 2, 6]), 6, kv_lens=i32([9, 9, 9]), slots=i32([3] * 6))
    D.dflash_tree_map(plan, tr.tree, i32([-1, 0, -1, 0, 1, 2]), i32([-1, 0, 0]))
    assert D.dflash_status_get() == D.DEV_TREE | D.DEV_ROWS
    assert plan.kv_lens.tolist() == [0, 0, 9] and tr.tree.nodes.tolist() == [-1, 0, 4]


def test_map_in_place_over_three_steps(D):
    tr = Trees(D, [0, 0], 64)
    tr.tree.nodes.zero_()
    parents, depths, masks = [[-1, 0], [-1, 0, 0]], [[], []], [[], []]
    before = [0, 0]
    for step in range(3):
        cu = [0, 2, 5]
        kv = [10 + 2 * (step + 1), 3 * (step + 1)]
        plan = D.ChunkPlan(i32(cu), 5, kv_lens=i32(kv), slots=i32([0] * 5))
        flat = [max(-1, before[b] + p - 1) for b in range(2) for p in parents[b]]
        pos, nodes, depths, masks, _ = T.tree_map(cu, kv, flat, before, depths, masks, 64)
        D.dflash_tree_map(plan, tr.tree, i32(flat), tr.tree.nodes)
        assert plan.positions.tolist() == [pos[r] for r in range(5)] and tr.tree.nodes.tolist() == nodes
        before = nodes
    for b in range(2):
        got = tr.tree.masks[b, :before[b]].cpu().numpy()
        assert all((got[t] == T.words(masks[b][t], 64)).all() for t in range(before[b]))


# ---------------------------------------------------------------------------
# attention
# ---------------------------------------------------------------------------

class TreeStep(Step):
    """A step whose rows are the newest nodes of trees that have `before` nodes in the cache."""

    def __init__(self, D, kv, heads, ctx, before, rows, max_nodes=512, masks=None, seed=0, width=4, **kw):
        super().__init__(D, kv, heads, [c + t for c, t in zip(ctx, before)], rows, seed=seed, **kw)
        r = rng_of(seed)
        self.committed, self.max_nodes = ctx, max_nodes
        par = [T.random_tree(r, t + n, width) if t + n else [] for t, n in zip(before, rows)]
        self.par = par
        B = len(ctx)
        whole = np.concatenate(([0], np.cumsum([len(p) for p in par])))
        _, self.nodes, self.depths, self.masks, _ = T.tree_map(whole, [10 ** 6] * B, [u for p in par for u in p],
                                                              [0] * B, [[]] * B, [[]] * B, max_nodes)
        self.tree = D.Tree(B, max_nodes, DEV)
        self.tree.masks.fill_(-1), self.tree.depths.fill_(99)
        for b in range(B):
            if before[b]:
                self.tree.depths[b, :before[b]] = i32(self.depths[b][:before[b]])
                self.tree.masks[b, :before[b]] = i32(np.stack([T.words(m, max_nodes) for m in self.masks[b][:before[b]]]))
        self.parents = i32([u for p, t in zip(par, before) for u in p[t:]] + [0] * kw.get("pad", 0))
        self.before = i32(before)

    def tree_map(self):
        self.D.dflash_tree_map(self.plan, self.tree, self.parents, self.before)

    def set_masks(self, masks):
        """Other masks for the step's nodes (whole numbers per sequence, all nodes)."""
        self.masks = masks
        for b, m in enumerate(masks):
            if m:
                self.tree.masks[b, :len(m)] = i32(np.stack([T.words(x, self.max_nodes) for x in m]))

    def tree_attn(self, q, out, window=0, scaling=0.0):
        self.D.dflash_tree_attn(self.dims, self.cache, self.layer, self.plan, self.tree, q, window, scaling, out, self.ws)

    def keys(self, b, window):
        n = self.rows[b]
        kv = self.committed[b] + self.nodes[b]
        return [T.visible(kv, self.nodes[b], t, self.depths[b], self.masks[b][t], window)
                for t in range(self.nodes[b] - n, self.nodes[b])]

    def check_tree(self, q, out, window=0, scaling=None, skip=()):
        sc = scaling or self.d ** -0.5
        qn, on = np64(q).reshape(self.M, self.n_h, self.d), np64(out).reshape(self.M, self.n_h, self.d)
        for b in range(self.B):
            lo, hi = int(self.cu[b]), int(self.cu[b + 1])
            if hi == lo or b in skip:
                continue
            k, v = self.cached(b, self.committed[b] + self.nodes[b])
            ref, mag, big, most = T.attention(qn[lo:hi], k, v, self.keys(b, window), self.G, sc)
            tol = T.attention_bound(ref, mag, big, max(most, 1), self.d, "f32" if self.kv == "f32" else "bf16")
            err = np.abs(on[lo:hi] - ref)
            assert np.isfinite(on[lo:hi]).all(), f"sequence {b}: not finite"
            worst = np.unravel_index(np.argmax(err - tol), err.shape)
            assert (err <= tol).all(), (f"sequence {b}: row, head, dim {worst}: {on[lo:hi][worst]} "
                                        f"against {ref[worst]}, bound {tol[worst]}")


# (committed, nodes before, new rows): a tree from nothing, page and tile ends inside the tree, an
# item's border, earlier nodes, a tree across several tiles, a long axis that is cut
SHAPES = {
    "small": ([0, 1, 126, 128, 700, 5], [0] * 6, [1, 7, 16, 16, 16, 0]),
    "grown": ([0, 100, 250, 1023, 40], [31, 5, 33, 200, 64], [4, 16, 1, 8, 33]),
    "wide": ([77, 0, 301], [0, 130, 0], [129, 70, 201]),
    "long": ([9000, 3], [40, 0], [9, 2]),
}


@pytest.mark.parametrize("shape", list(SHAPES))
@pytest.mark.parametrize("window", [0, 1, 3, 100, 300])
@pytest.mark.parametrize("kv,heads,paged", HEADS)
def test_attn(D, kv, heads, paged, window, shape):
    ctx, before, rows = SHAPES[shape]
    s = TreeStep(D, kv, heads, ctx, before, rows, paged=paged, pad=3, seed=window + len(ctx))
    s.map()
    s.tree_map()
    assert s.tree.nodes.tolist() == s.nodes
    q = torch.empty((s.M, s.n_h * s.d), dtype=s.q.dtype, device=DEV)
    s.append(q)
    out = torch.full_like(q, 5.0)
    s.tree_attn(q, out, window)
    assert D.dflash_status_get() == 0
    s.check_tree(q, out, window)
    assert (out[int(s.cu[-1]):] == 5.0).all()       # padding rows: as they were


@pytest.mark.parametrize("kv,heads,paged", [("bf16", (8, 2, 128), True), ("fp8", (8, 2, 128), True), ("f32", (4, 2, 64), False)])
@pytest.mark.parametrize("window", [0, 2, 90])
def test_attn_any_masks_and_rows_that_see_nothing(D, kv, heads, paged, window):
    """Masks that no tree has: random bits, bits of later nodes, none at all."""
    ctx, before, rows = [0, 0, 300, 60], [0, 150, 20, 0], [40, 40, 70, 3]
    s = TreeStep(D, kv, heads, ctx, before, rows, paged=paged, seed=12)
    s.map()
    s.tree_map()
    r = rng_of(13)
    masks = [[int.from_bytes(r.bytes(s.max_nodes // 8), "little") for _ in range(n)] for n in s.nodes]
    for b in range(4):
        for t in range(0, s.nodes[b], 3):
            masks[b][t] = 0
        masks[b][s.nodes[b] - 1] = 1                  # node 0 alone
    s.set_masks(masks)
    q = torch.empty((s.M, s.n_h * s.d), dtype=s.q.dtype, device=DEV)
    s.append(q)
    out = torch.full_like(q, 5.0)
    s.tree_attn(q, out, window)
    assert D.dflash_status_get() == 0
    s.check_tree(q, out, window)
    assert any(not k for k in s.keys(0, window)) and (out[0] == 0).all()


@pytest.mark.parametrize("kv,heads,paged", [("bf16", (8, 2, 128), True), ("fp8", (4, 1, 128), True), ("f32", (4, 2, 64), False)])
@pytest.mark.parametrize("value", [float("nan"), float("inf")])
def test_attn_hidden_keys_never_enter(D, kv, heads, paged, value):
    """A node's K and V are not finite: the rows that do not see it are as without it, those
    that do are not finite."""
    s = TreeStep(D, kv, heads, [200, 0], [9, 0], [30, 20], paged=paged, seed=21)
    s.map()
    s.tree_map()
    q = torch.empty((s.M, s.n_h * s.d), dtype=s.q.dtype, device=DEV)
    s.append(q)
    clean = torch.empty_like(q)
    s.tree_attn(q, clean)
    bad = [12, 3]                                     # nodes of sequences 0 and 1
    for b in range(2):
        at = s.committed[b] + bad[b]
        K, V = (s.cache.rows(w, 0, b, 0, s.committed[b] + s.nodes[b], codes=True).clone() for w in "kv")
        if kv == "fp8":
            K, V = (x.to(torch.float8_e4m3fn).view(torch.uint8) for x in (K, V))
            V[:, at] = 0x7F
            K[:, at] = 0x7F
        else:
            V[:, at], K[:, at] = value, value
        s.cache.set_rows(0, b, K, V)
    out = torch.empty_like(q)
    s.tree_attn(q, out)
    assert D.dflash_status_get() == 0
    hit = 0
    for b in range(2):
        for i in range(s.rows[b]):
            t = s.nodes[b] - s.rows[b] + i
            row = int(s.cu[b]) + i
            if s.masks[b][t] >> bad[b] & 1:
                hit += 1
                assert not torch.isfinite(out[row]).all(), (b, i)
            else:
                assert torch.equal(out[row], clean[row]), (b, i)
    assert hit > 2


@pytest.mark.parametrize("kv,heads,paged", [("bf16", (8, 2, 128), True), ("fp8", (32, 8, 128), True), ("f32", (8, 8, 64), False)])
@pytest.mark.parametrize("window", [0, 200])
def test_attn_of_chains_is_the_causal_attention(D, kv, heads, paged, window):
    ctx, rows = [0, 77, 300, 3000], [50, 64, 201, 1]
    s = TreeStep(D, kv, heads, ctx, [0] * 4, rows, paged=paged, seed=5)
    s.parents = i32([i - 1 for n in rows for i in range(n)])
    s.map()
    want = s.plan.positions.clone()
    s.tree_map()
    assert torch.equal(want, s.plan.positions)
    q = torch.empty((s.M, s.n_h * s.d), dtype=s.q.dtype, device=DEV)
    s.append(q)
    a, b = torch.empty_like(q), torch.empty_like(q)
    s.tree_attn(q, a, window)
    s.attn(q, b, window)
    s.check_attn(q, a, window)
    if window == 0:                                   # the same items, the same keys
        assert torch.equal(a, b)
    assert D.dflash_status_get() == 0


@pytest.mark.parametrize("kv,heads,paged", [("bf16", (4, 2, 128), True), ("f32", (4, 2, 64), False)])
def test_attn_refused_sequences(D, kv, heads, paged):
    s = TreeStep(D, kv, heads, [10, 10, 10, 10, 10], [2] * 5, [5] * 5, paged=paged, seed=6, max_nodes=32)
    s.map()
    s.tree_map()
    q = torch.empty((s.M, s.n_h * s.d), dtype=s.q.dtype, device=DEV)
    s.append(q)
    s.plan.kv_lens[0] = 0                             # refused by a map
    s.tree.nodes[1] = 4                               # fewer nodes than new rows
    s.tree.nodes[2] = 33                              # more than there can be
    s.tree.nodes[3] = 18                              # more than rows held
    out = torch.full_like(q, 5.0)
    s.tree_attn(q, out)
    assert D.dflash_status_get() == D.DEV_TREE
    assert (out[:20] == 0).all()
    s.check_tree(q, out, skip=(0, 1, 2, 3))


@pytest.mark.parametrize("kv", ["bf16", "f32"])
def test_attn_scores_of_minus_infinity(D, kv):
    """A row whose keys all score minus infinity is NaN, one that sees no key is zero."""
    s = TreeStep(D, kv, (2, 1, 128) if kv == "bf16" else (2, 1, 64), [0, 200], [0, 0], [3, 3], paged=kv == "bf16", seed=7)
    s.map()
    s.tree_map()
    s.set_masks([[1, 0, 4], [1, 0, 4]])
    q = torch.empty((s.M, s.n_h * s.d), dtype=s.q.dtype, device=DEV)
    s.append(q)
    big = 3e38
    q.fill_(big)
    for b in range(2):
        n = s.committed[b] + 3
        K = torch.full((1, n, s.d), -big, dtype=s.cache.k.dtype, device=DEV)
        s.cache.set_rows(0, b, K, torch.ones_like(K))
    out = torch.empty_like(q)
    s.tree_attn(q, out)
    o = out.float().cpu()
    assert o[0].isnan().all() and (o[1] == 0).all() and o[2].isnan().all()
    assert o[3:].isnan().all()
    assert D.dflash_status_get() == 0


def test_attn_repeats_bit_for_bit_on_another_stream(D):
    s = TreeStep(D, "bf16", (32, 8, 128), [3000, 500], [0, 0], [64, 33], seed=8)
    s.map()
    s.tree_map()
    q = torch.empty((s.M, s.n_h * s.d), dtype=s.q.dtype, device=DEV)
    s.append(q)
    a, b = torch.empty_like(q), torch.empty_like(q)
    s.tree_attn(q, a)
    torch.cuda.synchronize()
    st = torch.cuda.Stream()
    with torch.cuda.stream(st):
        s.tree_attn(q, b)
    st.synchronize()
    assert torch.equal(a, b)


# ---------------------------------------------------------------------------
# acceptance
# ---------------------------------------------------------------------------

def _accept(D, rows, parents, tokens, posterior, max_path, kv=None, pad=0, ctx=None, cu=None):
    B = len(rows)
    cu = np.concatenate(([0], np.cumsum(rows))) if cu is None else cu
    M = sum(rows) + pad
    plan = D.ChunkPlan(i32(cu), M, kv_lens=i32([9] * B if kv is None else kv))
    ctx = [100 + b for b in range(B)] if ctx is None else ctx
    o = {"path": i32(np.full((B, max_path), -9)), "a": i32([-9] * B), "cu": i32([-9] * (B + 1)), "ctx": i32(ctx),
         "anchor": i32([-9] * B)}
    z = [0] * pad
    D.dflash_tree_accept(plan, i32(parents + z), i32(tokens + z), i32(posterior + z), o["ctx"], o["a"], o["path"],
                         o["cu"], o["ctx"], o["anchor"])        # ctx_next in place
    return {k: v.tolist() for k, v in o.items()}, ctx


def _check_accept(got, ctx, rows, parents, tokens, posterior, max_path, refused=()):
    lo, total = 0, 0
    assert got["cu"][0] == 0
    for b, n in enumerate(rows):
        par, tok, post = (x[lo:lo + n] for x in (parents, tokens, posterior))
        path, anchor = ([], -1) if n == 0 or b in refused else T.accept(par, tok, post, max_path)
        assert got["path"][b] == path + [-1] * (max_path - len(path)), b
        assert got["a"][b] == len(path) - 1 and got["anchor"][b] == anchor
        total += len(path)
        assert got["cu"][b + 1] == total and got["ctx"][b] == ctx[b] + len(path)
        lo += n


@pytest.mark.parametrize("rows,max_path,pad", [([1], 1, 0), ([64] * 33, 16, 3), ([0, 5, 700, 0, 513, 512], 40, 1), ([9] * 300, 5, 0),
                                               ([17] * 2049, 9, 0)])
def test_accept(D, rows, max_path, pad):
    r = rng_of(len(rows))
    parents, tokens, posterior = [], [], []
    for n in rows:
        par = T.random_tree(r, n, 5) if n else []
        tok = [int(x) for x in r.integers(0, 4, size=n)]       # siblings share tokens now and then
        parents, tokens = parents + par, tokens + tok
        posterior += [int(x) for x in r.integers(0, 4, size=n)]
    got, ctx = _accept(D, rows, parents, tokens, posterior, max_path, pad=pad)
    _check_accept(got, ctx, rows, parents, tokens, posterior, max_path)
    assert D.dflash_status_get() == 0


def test_accept_chain_is_the_block_acceptance(D):
    r = rng_of(3)
    B, bs = 70, 16
    block = r.integers(0, 2, size=(B, bs))
    post = r.integers(0, 2, size=(B, bs))
    post[0, :-1] = block[0, 1:]                                  # all accepted
    got, ctx = _accept(D, [bs] * B, [i - 1 for _ in range(B) for i in range(bs)], block.ravel().tolist(), post.ravel().tolist(), bs)
    a, cu, nxt, anchor = i32([0] * B), i32([0] * (B + 1)), i32([0] * B), i32([0] * B)
    D.dflash_accept(i32(block), i32(post), i32(ctx), a, cu, nxt, anchor)
    assert got["a"] == a.tolist() and got["cu"] == cu.tolist() and got["ctx"] == nxt.tolist() and got["anchor"] == anchor.tolist()


def test_accept_refused_sequences_and_bad_rows(D):
    rows = [3, 3, 3]
    parents, tokens, posterior = [-1, 0, 1] * 3, [1, 2, 3] * 3, [2, 3, 7] * 3
    got, ctx = _accept(D, rows, parents, tokens, posterior, 4, kv=[9, 0, 9])
    _check_accept(got, ctx, rows, parents, tokens, posterior, 4, refused=(1,))
    got, ctx = _accept(D, rows, parents, tokens, posterior, 4, cu=[0, 5, 3, 9])
    assert got["a"] == [2, -1, 2] and got["path"][1] == [-1] * 4 and got["cu"] == [0, 3, 3, 6]
    assert D.dflash_status_get() == D.DEV_ROWS
    # parents that point nowhere (a later node, themselves, below -1) are nobody's children
    got, _ = _accept(D, [4], [5, 1, -3, 0], [1] * 4, [1] * 4, 4)
    assert got["path"] == [[0, 3, -1, -1]]


# ---------------------------------------------------------------------------
# commit
# ---------------------------------------------------------------------------

def _raw(cache):
    return [t.view(torch.uint8).clone() for t in (cache.k, cache.v)]


def _commit_case(D, kv, heads, paged, ctx, nodes, layers, seed=0):
    n_h, n_kv, d = heads
    dt = torch.float32 if kv == "f32" else torch.bfloat16
    cap = -(-max(c + n for c, n in zip(ctx, nodes)) // 128) * 128 + 128
    c = D.KVCache(layers, len(ctx), n_kv, cap, d, dt, DEV, paged=paged, seed=seed, kv="fp8" if kv == "fp8" else "bf16")
    for t in (c.k, c.v):
        x = t.view(torch.uint8)
        x.copy_(torch.randint(0, 256, x.shape, generator=torch.Generator().manual_seed(seed), dtype=torch.uint8))
    c.lens.copy_(i32([a + b for a, b in zip(ctx, nodes)])[None])
    return c, D.make_dims(64, n_h, n_kv, d, 1, 1, 1e-6, dt), D.Tree(len(ctx), -(-max(max(nodes), 1) // 32) * 32, nodes=i32(nodes))


def _slot(c, b, s):
    """Index of a sequence's row in a layer: (unit, row)."""
    return (int(c.block_table[b, s // 128]), s % 128) if c.paged else (b, s)


@pytest.mark.parametrize("kv,heads,paged", [("bf16", (32, 8, 128), True), ("bf16", (2, 1, 128), False), ("fp8", (8, 8, 128), True),
                                            ("fp8", (4, 2, 128), False), ("f32", (4, 2, 80), False), ("f32", (3, 3, 6), False),
                                            ("f32", (2, 1, 256), False), ("f32", (1, 1, 2), False)])
@pytest.mark.parametrize("layers", [1, 3])
def test_commit(D, kv, heads, paged, layers):
    r = rng_of(layers)
    ctx, nodes = [0, 127, 250, 64, 5, 3], [1, 20, 300, 8, 130, 40]
    c, dims, tree = _commit_case(D, kv, heads, paged, ctx, nodes, layers, seed=layers)
    # the first node alone; an overlapping ascent; 100 of 300; a prefix (nothing moves); nothing; the last node
    paths = [[0], [0, 1, 3, 4, 5, 9, 10, 11, 12, 13, 19], sorted(r.choice(300, 100, replace=False).tolist()), list(range(8)),
             [], [0, 39]]
    W = 101
    path = np.full((6, W), -1)
    for b, p in enumerate(paths):
        path[b, :len(p)] = p
    want, lens = _raw(c), c.lens.clone()
    shape = c.k.shape[:-1] + (-1,)
    before = [w.view(shape).clone() for w in want]
    for w, old in zip(want, before):
        w = w.view(shape)
        for b, p in enumerate(paths):
            for i, u in enumerate(p):
                (pu, ru), (pi, ri) = _slot(c, b, ctx[b] + u), _slot(c, b, ctx[b] + i)
                w[:, pi, :, ri] = old[:, pu, :, ru]
    for b, p in enumerate(paths):
        if p:
            lens[:, b] = ctx[b] + len(p)
    D.dflash_tree_commit(dims, c, tree, i32(ctx), i32(path), i32([len(p) - 1 for p in paths]))
    assert D.dflash_status_get() == 0
    assert torch.equal(c.lens, lens)
    for now, w in zip(_raw(c), want):
        assert torch.equal(now, w)


@pytest.mark.parametrize("paged", [True, False])
def test_commit_refuses(D, paged):
    ctx, nodes = [10, 10, 10, 10, 10, 250, -1, 10], [8, 8, 8, 8, 8, 8, 8, -1]
    c, dims, tree = _commit_case(D, "bf16", (2, 1, 128), paged, [10] * 8, [8] * 8, 2)
    tree = D.Tree(8, 32, nodes=i32(nodes))
    cap = c.capacity
    ctx[5] = cap - 7                                              # nodes beyond the capacity
    path = [[0, 1, 1, -1], [0, 8, -1, -1], [-1, 0, -1, -1], [0, 1, 2, 3], [0, 1, 2, 3], [0, 2, -1, -1], [0, 2, -1, -1], [0, 2, -1, -1]]
    a = [2, 1, 1, 4, -2, 1, 1, 1]
    before, lens = _raw(c), c.lens.clone()
    D.dflash_tree_commit(dims, c, tree, i32(ctx), i32(path), i32(a))
    assert D.dflash_status_get() == D.DEV_TREE
    assert torch.equal(c.lens, lens) and all(torch.equal(x, y) for x, y in zip(_raw(c), before))


def test_commit_bad_page(D):
    c, dims, tree = _commit_case(D, "bf16", (2, 1, 128), True, [120], [40], 2)
    keep = int(c.block_table[0, 1])
    c.block_table[0, 1] = 10 ** 6
    before = _raw(c)
    D.dflash_tree_commit(dims, c, tree, i32([120]), i32([[0, 3, 20, 30]]), i32([3]))
    assert D.dflash_status_get() == D.DEV_PAGE
    c.block_table[0, 1] = keep
    for now, old in zip(_raw(c), before):                         # the move inside the good page alone
        old.view(c.k.shape[:-1] + (-1,))[:, int(c.block_table[0, 0]), :, 121] = \
            old.view(c.k.shape[:-1] + (-1,))[:, int(c.block_table[0, 0]), :, 123]
        assert torch.equal(now, old)
    assert c.lens.tolist() == [[124], [124]]
