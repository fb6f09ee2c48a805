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


@pytest.mark.parametrize("kv", [-2 ** 31, -2 ** 31 + 1, -1, 2, 2 ** 31 - 1])
def test_map_of_any_length(D, kv):
    """Three new rows: fewer rows held, also so few that the difference wraps, are refused."""
    tr = Trees(D, [0], 32)
    plan = D.ChunkPlan(i32([0, 3]), 3, kv_lens=i32([kv]), slots=i32([3] * 3))
    D.dflash_tree_map(plan, tr.tree, i32([-1, 0, 0]))
    good = kv >= 3
    assert D.dflash_status_get() == (0 if good else D.DEV_TREE)
    assert plan.positions.tolist() == ([kv - 3, kv - 2, kv - 2] if good else [-1] * 3)
    assert plan.kv_lens.tolist() == [kv if good else 0] and tr.tree.nodes.tolist() == [3 if good else 0]


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


# ---------------------------------------------------------------------------
# together: rounds of drafted trees, a beam search
# ---------------------------------------------------------------------------

@pytest.mark.parametrize("kv,paged", [("bf16", True), ("bf16", False), ("fp8", True), ("f32", False)])
@pytest.mark.parametrize("graph", [False, True])
def test_rounds_of_trees_leave_the_accepted_rows_in_the_cache(D, kv, paged, graph):
    """Map, tree map, append, attention, greedy posterior, acceptance and commit, round after round on
    the device (captured: one graph, replayed): what each round decides, then the cache against rows made from
    the accepted nodes' projections."""
    B, layers, n, width = 3, 2, 24, 8
    n_h, n_kv, d = (8, 2, 128) if kv != "f32" else (4, 2, 64)
    dt = torch.float32 if kv == "f32" else torch.bfloat16
    cap, V = 384, 40
    r = rng_of(17)
    c = D.KVCache(layers, B, n_kv, cap, d, dt, DEV, paged=paged, kv="fp8" if kv == "fp8" else "bf16",
                  kv_scales=[[0.05, 0.02]] * layers if kv == "fp8" else None)
    dims = D.make_dims(64, n_h, n_kv, d, 1, 1, 1e-6, dt)
    pool = D.PagePool(i32([0] * B), c.block_table.flatten().clone(), i32([0])) if paged else None
    M = B * n
    cu = [b * n for b in range(B + 1)]
    plan, tree = D.ChunkPlan(i32(cu), M), D.Tree(B, 32, DEV)
    widths = (n_h * d, n_kv * d, n_kv * d)
    x = torch.zeros((layers, M, sum(widths)), dtype=dt, device=DEV)
    parents, tokens = i32([0] * M), i32([0] * M)
    logits = torch.zeros((M, 1, V), dtype=torch.float32, device=DEV)
    posterior = torch.zeros((M, 1), dtype=torch.int32, device=DEV)
    ctx, acc, path = i32([0] * B), i32([0] * B), i32(np.zeros((B, 8)))
    ncu, nxt, anchor = i32([0] * (B + 1)), i32([0] * B), i32([0] * B)
    table = torch.empty((cap, d // 2, 2), dtype=torch.float32, device=DEV)
    D.dflash_rope_table_build(1e6, d, cap, table)
    gk = (1 + 0.1 * torch.randn(d, generator=torch.Generator().manual_seed(1))).to(DEV, dt)
    q = [torch.zeros((M, n_h * d), dtype=dt, device=DEV) for _ in range(layers)]
    out = [torch.zeros_like(t) for t in q]
    ws = torch.empty(D.dflash_chunk_workspace_bytes(dims), dtype=torch.uint8, device=DEV)
    bws = torch.empty(D.dflash_beam_workspace_bytes(M, 1, V, 1), dtype=torch.uint8, device=DEV)

    def round_():
        D.dflash_chunk_map(c, 0, plan, pool)
        D.dflash_tree_map(plan, tree, parents)
        for l in range(layers):
            a, b, v = x[l].split(widths, dim=1)
            D.dflash_chunk_append(dims, c, l, plan, a, b, v, gk, gk, table, cap, q[l])
            D.dflash_tree_attn(dims, c, l, plan, tree, q[l], 0, 0.0, out[l], ws)
        D.dflash_beam_select(logits, None, 1, posterior, None, None, bws)
        D.dflash_tree_accept(plan, parents, tokens, posterior, ctx, acc, path, ncu, nxt, anchor)
        D.dflash_tree_commit(dims, c, tree, ctx, path, acc)
        ctx.copy_(nxt)

    g = None
    if graph:                                        # capture (nothing runs)
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            round_()
    kept = [[[] for _ in range(B)] for _ in range(layers)]      # (k, v) projections of the accepted rows
    moved = 0
    for step in range(5):
        host = r.standard_normal((layers, M, sum(widths))).astype(np.float32)
        x.copy_(torch.from_numpy(host).to(dt))
        par, tok, post = [], [], []
        for b in range(B):
            p = T.random_tree(r, n, width // 2)
            t = r.integers(0, V, size=n).tolist()
            kids = [[i for i in range(n) if p[i] == u] for u in range(n)]
            par, tok = par + p, tok + t
            post += [t[int(r.choice(k))] if k and r.random() < 0.85 else int(r.integers(0, V)) for k in kids]
        parents.copy_(i32(par)), tokens.copy_(i32(tok))
        lg = torch.randn((M, 1, V), generator=torch.Generator().manual_seed(step))
        lg[torch.arange(M), 0, torch.tensor(post)] = 9.0
        logits.copy_(lg)
        before = ctx.tolist()
        g.replay() if graph else round_()
        assert D.dflash_status_get() == 0
        assert posterior[:, 0].tolist() == post
        xn = np64(x.reshape(layers * M, -1)).reshape(layers, M, -1)
        for b in range(B):
            lo = b * n
            want, last = T.accept(par[lo:lo + n], tok[lo:lo + n], post[lo:lo + n], 8)
            assert path[b].tolist() == want + [-1] * (8 - len(want)) and int(anchor[b]) == last
            assert int(ctx[b]) == before[b] + len(want) and c.lens[:, b].tolist() == [int(ctx[b])] * layers
            moved += sum(i != u for i, u in enumerate(want))
            for l in range(layers):
                kept[l][b] += [xn[l, lo + u, n_h * d:] for u in want]
    assert moved > 10
    scales = c.scales
    for l in range(layers):
        for b in range(B):
            m = int(ctx[b])
            assert m == len(kept[l][b])
            got = [np64(c.rows(w, l, b, 0, m, codes=True)).transpose(1, 0, 2) for w in "kv"]
            for i in range(m):
                k, v = kept[l][b][i][:n_kv * d].reshape(n_kv, d), kept[l][b][i][n_kv * d:].reshape(n_kv, d)
                y, mag = R.norm_rope(k, np64(gk), i)
                how = {"f32": "f32", "bf16": "bf16", "fp8": "e4m3"}[kv]
                sk, sv = (scales[l] if kv == "fp8" else (1.0, 1.0))
                assert (np.abs(got[0][i] - np.clip(y / sk, -448, 448)) <= R.append_bound(y / sk, mag / sk, d, how)).all(), (l, b, i)
                assert (np.abs(got[1][i] - np.clip(v / sv, -448, 448)) <= R.append_bound(v / sv, np.abs(v / sv), d, how)).all()


def test_beam_search_over_one_cache(D):
    """A beam search on a small random model: hypotheses are paths of one tree behind the prompt, and
    nothing of the cache moves. Tokens, parents and scores against the same search with every hypothesis
    recomputed from its start in float64."""
    n_h, n_kv, d, V, beams, steps, B = 4, 2, 32, 60, 3, 7, 2
    g = torch.Generator().manual_seed(31)
    emb = torch.randn((V, 48), generator=g, dtype=torch.float64)
    Wq, Wk, Wv = (torch.randn((48, h * d), generator=g, dtype=torch.float64) * 0.3 for h in (n_h, n_kv, n_kv))
    Wo = torch.randn((n_h * d, V), generator=g, dtype=torch.float64) * 0.4
    emb, Wq, Wk, Wv, Wo = (t.float() for t in (emb, Wq, Wk, Wv, Wo))
    prompts = [[3, 17, 41, 8], [55, 2, 9, 30]]
    P = len(prompts[0])
    cap = 128
    c = D.KVCache(1, B, n_kv, cap, d, "f32", DEV)
    dims = D.make_dims(64, n_h, n_kv, d, 1, 1, 1e-6, "f32")
    table = torch.empty((cap, d // 2, 2), dtype=torch.float32, device=DEV)
    D.dflash_rope_table_build(1e6, d, cap, table)
    ws = torch.empty(D.dflash_chunk_workspace_bytes(dims), dtype=torch.uint8, device=DEV)
    dev = [t.to(DEV) for t in (emb, Wq, Wk, Wv, Wo)]

    def step(plan, tree, tokens):
        h = dev[0][tokens.long()]
        q, k, v = h @ dev[1], h @ dev[2], h @ dev[3]
        qo, out = torch.empty_like(q), torch.empty_like(q)
        D.dflash_chunk_append(dims, c, 0, plan, q, k, v, None, None, table, cap, qo)
        if tree is None:
            D.dflash_chunk_attn(dims, c, 0, plan, qo, 0, 0.0, out, ws)
        else:
            D.dflash_tree_attn(dims, c, 0, plan, tree, qo, 0, 0.0, out, ws)
        return out @ dev[4]

    def exact(seq):
        """Next-token logits of a whole sequence in float64."""
        e = emb.double().numpy()[seq]
        q, k, v = ((e @ w.double().numpy()).reshape(len(seq), -1, d) for w in (Wq, Wk, Wv))
        k = np.stack([R.norm_rope(k[i], None, i)[0] for i in range(len(seq))])
        q1 = R.norm_rope(q[-1], None, len(seq) - 1)[0][None]
        o, _, _, _ = R.attention(q1, k, v, len(seq), 1, n_h // n_kv, 0, d ** -0.5)
        return o.reshape(-1) @ Wo.double().numpy()

    torch.backends.cuda.matmul.allow_tf32 = False
    plan = D.ChunkPlan(i32([0, P, 2 * P]), 2 * P)
    D.dflash_chunk_map(c, 0, plan)
    logits = step(plan, None, i32(sum(prompts, [])))
    ref = [[(p, 0.0)] for p in prompts]
    tree = D.Tree(B, 64, DEV)
    nodes = 0
    scores = None
    last = logits.view(B, P, V)[:, -1:, :]                     # one beam: the prompt
    for s in range(steps):
        n_in = last.shape[1]
        tok, par = (torch.zeros((B, beams), dtype=torch.int32, device=DEV) for _ in range(2))
        new = torch.zeros((B, beams), dtype=torch.float32, device=DEV)
        bws = torch.empty(D.dflash_beam_workspace_bytes(B, n_in, V, beams), dtype=torch.uint8, device=DEV)
        base = max(0, nodes - n_in) if s else 0
        D.dflash_beam_select(last.contiguous(), scores, beams, tok, par, new, bws, parent_base=base)
        scores = new
        for b in range(B):
            x = np.stack([exact(h) for h, _ in ref[b]])
            t, i, v = T.beam_select(x, np.array([w for _, w in ref[b]]), beams)
            assert tok[b].tolist() == t.tolist() and (par[b] - base).tolist() == i.tolist(), (s, b)
            # scores: fp32 projections, attention and sums of up to 48, 64 and 128 terms, a step's error adding
            # to the last's
            assert np.abs(np64(new[b]) - v).max() <= (s + 1) * 2e-4
            ref[b] = [(ref[b][j][0] + [int(u)], float(w)) for j, u, w in zip(i, t, v)]
        parents = par if s else torch.full_like(par, -1)       # the first hypotheses follow the prompt
        plan = D.ChunkPlan(i32([0, beams, 2 * beams]), 2 * beams)
        D.dflash_chunk_map(c, 0, plan)
        D.dflash_tree_map(plan, tree, parents.contiguous(), tree.nodes)
        nodes += beams
        assert plan.positions.tolist() == [P + s] * (2 * beams) and tree.nodes.tolist() == [nodes] * B
        last = step(plan, tree, tok.flatten()).view(B, beams, V)
    assert D.dflash_status_get() == 0
    # keep the best hypothesis: its path becomes the cache's rows
    paths = []
    for b in range(B):
        masks = tree.masks[b].cpu().numpy().astype(np.uint32)
        m = int(masks[nodes - beams, 0]) | int(masks[nodes - beams, 1]) << 32
        paths.append([u for u in range(nodes) if m >> u & 1])
    assert all(len(p) == steps for p in paths)
    D.dflash_tree_commit(dims, c, tree, i32([P] * B), i32(paths), i32([steps - 1] * B))
    assert c.lens.tolist() == [[P + steps] * B] and D.dflash_status_get() == 0
    for b in range(B):
        seq = ref[b][0][0]
        k = (emb.double().numpy()[seq] @ Wk.double().numpy()).reshape(len(seq), n_kv, d)
        got = np64(c.rows("k", 0, b, 0, P + steps)).transpose(1, 0, 2)
        for i in range(P + steps):
            y, mag = R.norm_rope(k[i], None, i)
            assert (np.abs(got[i] - y) <= 48 * 2.0 ** -22 * (np.abs(emb.numpy()[seq[i]])[:, None] * np.abs(Wk.numpy())).sum(0).max()
                    + R.append_bound(y, mag, d, "f32")).all()


# ---------------------------------------------------------------------------
# sizes
# ---------------------------------------------------------------------------

def test_steps_without_rows(D):
    plan = D.ChunkPlan(i32([0, 0, 0]), 3, kv_lens=i32([5, 0]), slots=i32([-1] * 3), positions=i32([-7] * 3))
    tree = D.Tree(2, 32, DEV)
    tree.nodes.fill_(9)
    D.dflash_tree_map(plan, tree, i32([7] * 3), i32([2, 3]))
    assert tree.nodes.tolist() == [2, 3] and plan.positions.tolist() == [-7] * 3 and plan.kv_lens.tolist() == [5, 0]
    got, ctx = _accept(D, [0, 0], [], [], [], 3, pad=3, kv=[5, 5])
    _check_accept(got, ctx, [0, 0], [], [], [], 3)
    s = TreeStep(D, "bf16", (4, 2, 128), [10], [0], [4], seed=1)
    s.map(), s.tree_map()
    plan = D.ChunkPlan(i32([0, 0]), 0, kv_lens=i32([10]))
    out = torch.full((1, 512), 3.0, dtype=torch.bfloat16, device=DEV)
    D.dflash_tree_attn(s.dims, s.cache, 0, plan, s.tree, out, 0, 0.0, out, s.ws)
    assert (out == 3.0).all() and D.dflash_status_get() == 0


def test_map_beyond_32_bit_offsets(D):
    """Masks of 1100 sequences of 4096 nodes: 2.3 GB."""
    B, N = 1100, 4096
    tree = D.Tree(B, N, DEV)
    n = 5
    plan = D.ChunkPlan(i32([n * b for b in range(B + 1)]), n * B, kv_lens=i32([n + 4000 + b for b in range(B)]), slots=i32([1] * n * B))
    par = [-1, 0, 0, 2, 1]
    D.dflash_tree_map(plan, tree, i32(par * B))
    D.dflash_tree_map(plan, tree, i32([4, 5, 5, 7, 8] * B), tree.nodes)
    assert D.dflash_status_get() == 0 and tree.nodes.unique().tolist() == [10]
    for b in (0, 1023, 1024, 1099):
        want = T.tree_map([0, 5], [10 ** 6], par, [0], [[]], [[]], N)
        want = T.tree_map([0, 5], [10 ** 6], [4, 5, 5, 7, 8], want[1], want[2], want[3], N)
        got = tree.masks[b, :10].cpu().numpy()
        assert all((got[t] == T.words(want[3][0][t], N)).all() for t in range(10))
        assert tree.depths[b, :10].tolist() == want[2][0]


def test_attn_and_commit_beyond_32_bit_offsets(D):
    """The second layer of a pool of 9000 pages begins 2.4 GB on."""
    n_h, n_kv, d, pages = 16, 8, 128, 9000
    table = torch.tensor([[8999, 4500, 17]], dtype=torch.int32)
    c = D.KVCache(2, 1, n_kv, 384, d, "bf16", DEV, page_table=table, n_pages=pages)
    dims = D.make_dims(64, n_h, n_kv, d, 1, 1, 1e-6, "bf16")
    g = torch.Generator().manual_seed(2)
    ctx, n = 120, 40
    K, V = (torch.randn((n_kv, ctx + n, d), generator=g).to(DEV, torch.bfloat16) for _ in range(2))
    c.set_rows(1, 0, K, V)
    plan = D.ChunkPlan(i32([0, n]), n, kv_lens=i32([ctx + n]), slots=i32([0] * n))
    tree = D.Tree(1, 64, DEV)
    par = T.random_tree(rng_of(3), n)
    D.dflash_tree_map(plan, tree, i32(par))
    q = torch.randn((n, n_h * d), generator=g).to(DEV, torch.bfloat16)
    out = torch.zeros_like(q)
    ws = torch.empty(D.dflash_chunk_workspace_bytes(dims), dtype=torch.uint8, device=DEV)
    D.dflash_tree_attn(dims, c, 1, plan, tree, q, 0, 0.0, out, ws)
    _, nodes, depths, masks, _ = T.tree_map([0, n], [10 ** 6], par, [0], [[]], [[]], 64)
    keys = [T.visible(ctx + n, n, t, depths[0], masks[0][t], 0) for t in range(n)]
    kn, vn = np64(K).transpose(1, 0, 2), np64(V).transpose(1, 0, 2)
    ref, mag, big, most = T.attention(np64(q).reshape(n, n_h, d), kn, vn, keys, 2, d ** -0.5)
    assert (np.abs(np64(out).reshape(n, n_h, d) - ref) <= T.attention_bound(ref, mag, big, most, d, "bf16")).all()
    D.dflash_tree_commit(dims, c, tree, i32([ctx]), i32([[0, 5, 20, 39]]), i32([3]))
    for i, u in enumerate((0, 5, 20, 39)):
        assert torch.equal(c.rows("k", 1, 0, ctx + i, ctx + i + 1)[:, 0], K[:, ctx + u])
        assert torch.equal(c.rows("v", 1, 0, ctx + i, ctx + i + 1)[:, 0], V[:, ctx + u])
    assert D.dflash_status_get() == 0 and c.lens.tolist() == [[ctx + 4]] * 2


@pytest.mark.parametrize("kv", ["bf16", "fp8", "f32"])
def test_attn_many_sequences(D, kv):
    """4096 sequences of a node or two."""
    B = 4096
    n_h, n_kv, d = (2, 1, 128) if kv != "f32" else (2, 1, 32)
    r = rng_of(5)
    ctx, rows = r.integers(0, 4, size=B).tolist(), r.integers(0, 3, size=B).tolist()
    s = TreeStep(D, kv, (n_h, n_kv, d), ctx, [0] * B, rows, max_nodes=32, paged=False, seed=5)
    s.map(), s.tree_map()
    q = torch.empty((s.M, n_h * d), dtype=s.q.dtype, device=DEV)
    s.append(q)
    out = torch.empty_like(q)
    s.tree_attn(q, out)
    assert D.dflash_status_get() == 0
    s.check_tree(q, out, skip=set(range(B)) - set(range(0, B, 41)) - {B - 1})


@pytest.mark.parametrize("kv", ["bf16", "fp8"])
def test_attn_that_gives_up_leaves_a_working_gpu(D, kv):
    """With a limit of 1 ns the roles of the kernel stop at their first longer wait; the next call is
    right. (The warp that checks the tiles of the tree first waits for tens of microseconds.)"""
    s = TreeStep(D, kv, (32, 8, 128), [100_000], [0], [64], seed=9)
    s.map(), s.tree_map()
    q = torch.empty((s.M, s.n_h * s.d), dtype=s.q.dtype, device=DEV)
    s.append(q)
    out, want = torch.empty_like(q), torch.empty_like(q)
    s.tree_attn(q, want)
    assert D.dflash_status_get() == 0
    st = 0
    try:
        D.dflash_test_wait_limit(1)
        for _ in range(3):
            s.tree_attn(q, out)
            st |= D.dflash_status_get()
            if st & D.DEV_TIMEOUT:
                break
    finally:
        D.dflash_test_wait_limit(0)
    assert st == D.DEV_TIMEOUT
    out.fill_(float("nan"))
    s.tree_attn(q, out)
    assert D.dflash_status_get() == 0
    assert torch.equal(out, want)


def test_launches_and_trace_kinds(D):
    s = TreeStep(D, "bf16", (8, 2, 128), [300], [0], [20], seed=10)
    s.map()
    q = torch.empty((s.M, s.n_h * s.d), dtype=s.q.dtype, device=DEV)
    out = torch.empty_like(q)
    kinds = ["tree_map", "chunk_append", "chunk_attn", "chunk_merge", "tree_accept", "tree_commit"]
    n = D.dflash_launch_count()
    D.dflash_trace_start(kinds, 16)
    s.tree_map(), s.append(q), s.tree_attn(q, out)
    o = [i32([0]), i32([[0] * 4]), i32([0, 0]), i32([0]), i32([0])]
    D.dflash_tree_accept(s.plan, s.parents, s.parents, s.parents, i32([300]), *o)
    D.dflash_tree_commit(s.dims, s.cache, s.tree, i32([300]), o[1], o[0])
    assert [k for k, _ in D.dflash_trace_stop()] == kinds
    assert D.dflash_launch_count() == n + len(kinds) and D.dflash_status_get() == 0


@pytest.mark.parametrize("graph", [False, True])
def test_calls_wait_for_a_stream_that_was_joined(D, graph):
    """Inputs that another stream writes late, after long products; the calling stream waits for its event only.
    What the calls read before that would be other inputs, whose results differ."""
    r = rng_of(21)
    n, B, path = 64, 30, 12
    parents = [u for _ in range(B) for u in T.random_tree(r, n, 5)]
    tokens, posterior = ([int(x) for x in r.integers(0, 3, size=n * B)] for _ in range(2))
    right = [i32(parents), i32(tokens), i32(posterior)]
    wrong = [i32([i - 1 for _ in range(B) for i in range(n)]), torch.zeros_like(right[1]), torch.ones_like(right[2])]
    logits = torch.randn(4, 2, 40000, device=DEV)
    ins = [w.clone() for w in wrong] + [torch.zeros_like(logits)]
    cu, kv = i32(np.arange(B + 1) * n), [n] * B
    plan = D.ChunkPlan(cu, n * B, kv_lens=i32(kv))
    tree = D.Tree(B, n, DEV)
    ctx = i32(range(B))
    o = [i32([0] * B), i32([[0] * path] * B), i32([0] * (B + 1)), i32([0] * B), i32([0] * B)]
    sel = [torch.zeros((4, 3), dtype=t, device=DEV) for t in (torch.int32, torch.int32, torch.float32)]
    ws = torch.empty(D.dflash_beam_workspace_bytes(4, 2, 40000, 3), dtype=torch.uint8, device=DEV)
    side = torch.cuda.Stream()
    big = torch.randn(4096, 4096, device=DEV)
    out = torch.empty_like(big)

    def step():
        main = torch.cuda.current_stream()
        side.wait_stream(main)
        with torch.cuda.stream(side):
            for _ in range(3):
                torch.mm(big, big, out=out)
            for i, t in zip(ins, right + [logits]):
                i.copy_(t)
        D.dflash_beam_select(ins[3], None, 2, sel[0][:, :2], sel[1][:, :2], sel[2][:, :2], ws)   # of the zeros, or of both
        main.wait_stream(side)
        D.dflash_tree_accept(plan, *ins[:3], ctx, *o)
        D.dflash_beam_select(ins[3], None, 3, *sel, ws)
        D.dflash_tree_map(plan, tree, ins[0])

    torch.mm(big, big, out=out)
    if graph:
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            step()
    for _ in range(3):
        for i, t in zip(ins, wrong):
            i.copy_(t)
        ins[3].zero_()
        [t.fill_(-3) for t in o + sel]
        g.replay() if graph else step()
        torch.cuda.synchronize()
        got = dict(zip(("a", "path", "cu", "ctx", "anchor"), (t.tolist() for t in o)))
        _check_accept(got, list(range(B)), [n] * B, parents, tokens, posterior, path)
        for b in range(4):
            t, i, _ = T.beam_select(np64(logits)[b], np.zeros(2), 3)
            assert sel[0][b].tolist() == t.tolist() and sel[1][b].tolist() == i.tolist()
        _, _, depths, masks, _ = T.tree_map(np.arange(B + 1) * n, kv, parents, [0] * B, [[]] * B, [[]] * B, n)
        assert tree.depths.tolist() == [list(d) for d in depths]
        got = tree.masks.cpu().numpy()
        assert all((got[b, t] == T.words(masks[b][t], n)).all() for b in range(B) for t in range(n))
    assert D.dflash_status_get() == 0


@pytest.mark.parametrize("kv,heads,paged", [("bf16", (8, 1, 128), True), ("fp8", (8, 2, 128), True), ("f32", (2, 1, 64), False)])
@pytest.mark.parametrize("ctx,before,rows", [([30000], [0], [1]), ([20001], [100], [16]), ([9000], [0], [130]),
                                             ([5000, 0, 300], [7, 0, 0], [3, 40, 1])])
def test_attn_few_heads_over_long_contexts(D, kv, heads, paged, ctx, before, rows):
    """One item cut into many pieces, of more than a tile each."""
    s = TreeStep(D, kv, heads, ctx, before, rows, paged=paged, pad=1, seed=31)
    s.map(), s.tree_map()
    q = torch.empty((s.M, s.n_h * s.d), dtype=s.q.dtype, device=DEV)
    out = torch.empty_like(q)
    s.append(q)
    for window in (0, 4000):
        s.tree_attn(q, out, window)
        s.check_tree(q, out, window)
    assert D.dflash_status_get() == 0


@pytest.mark.parametrize("kv", ["bf16", "fp8", "f32"])
@pytest.mark.parametrize("batch", [1, 2, 3, 4, 5, 8, 9, 16, 17, 31, 32, 33, 64])
def test_attn_any_number_of_sequences(D, kv, batch):
    """Both ways of finding a share of the work; empty sequences, one of several items, refused ones between."""
    r = rng_of(batch)
    rows = [int(n) for n in r.integers(0, 20, size=batch)]
    rows[batch // 2] = 150
    ctx = [int(c) for c in r.integers(0, 500, size=batch)]
    s = TreeStep(D, kv, (4, 2, 64 if kv == "f32" else 128), ctx, [0] * batch, rows, paged=kv != "f32", seed=batch)
    s.map(), s.tree_map()
    q = torch.empty((s.M, s.n_h * s.d), dtype=s.q.dtype, device=DEV)
    out = torch.full_like(q, float("nan"))
    s.append(q)
    refused = [b for b in range(batch) if rows[b] and b % 5 == 4 and b != batch // 2]
    for b in refused:
        s.plan.kv_lens[b] = 0
    s.tree_attn(q, out)
    s.check_tree(q, out, skip=refused)
    for b in refused:
        assert (out[int(s.cu[b]):int(s.cu[b + 1])] == 0).all()
    assert D.dflash_status_get() == 0


@pytest.mark.parametrize("kv", ["bf16", "fp8"])
def test_attn_hidden_keys_of_a_window(D, kv):
    """A value that is not finite behind chains of 128 nodes: with a window too, only the rows that see it are not
    finite, and the masks are not looked up key by key (a window takes keys away; it took 2.6 times as long)."""
    n, ctx, B, bad = 128, 1000, 8, 100
    s = TreeStep(D, kv, (32, 8, 128), [ctx] * B, [0] * B, [n] * B, seed=3, max_nodes=n)
    s.parents = i32([i - 1 for _ in range(B) for i in range(n)])
    s.map(), s.tree_map()
    q = torch.empty((s.M, s.n_h * s.d), dtype=s.q.dtype, device=DEV)
    s.append(q)
    clean, out, took = {}, torch.empty_like(q), {}
    for window in (0, 20):
        clean[window] = torch.empty_like(q)
        s.tree_attn(q, clean[window], window)
    for b in range(B):
        K, V = (s.cache.rows(w, 0, b, 0, ctx + n, codes=True).clone() for w in "kv")
        if kv == "fp8":
            K, V = (x.to(torch.float8_e4m3fn).view(torch.uint8) for x in (K, V))
        V[:, ctx + bad] = 0x7F if kv == "fp8" else float("nan")
        s.cache.set_rows(0, b, K, V)
    for window in (0, 20):
        times = []
        for _ in range(9):
            at = [torch.cuda.Event(enable_timing=True) for _ in range(2)]
            at[0].record()
            s.tree_attn(q, out, window)
            at[1].record()
            torch.cuda.synchronize()
            times.append(at[0].elapsed_time(at[1]))
        took[window] = sorted(times)[4]
        o, c = out.view(B, n, -1), clean[window].view(B, n, -1)
        sees = torch.tensor([t >= bad and (not window or t - bad < window) for t in range(n)], device=DEV)
        assert o[:, sees].isnan().all() and torch.equal(o[:, ~sees], c[:, ~sees])
    assert D.dflash_status_get() == 0
    assert took[20] < 1.5 * took[0], took
