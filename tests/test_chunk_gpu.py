"""The chunk step (map, append, causal attention) against its formulas in float64."""
import numpy as np
import pytest
import torch

import chunk_ref as R

pytestmark = pytest.mark.gpu

DEV = "cuda"
TORCH = {"f32": torch.float32, "bf16": torch.bfloat16, "fp8": torch.bfloat16}


@pytest.fixture(scope="module")
def D():
    from speculative_decoding_draft_dflash_gb300 import dflash
    return dflash


def i32(x):
    return torch.tensor(np.asarray(x), dtype=torch.int32, device=DEV)


def np64(t):
    return t.detach().float().cpu().numpy().astype(np.float64)


# ---------------------------------------------------------------------------
# map
# ---------------------------------------------------------------------------

def _map_case(D, lens, rows, capacity, held_extra, n_free, pad=0, seed=0, taken=0, in_place=False,
              n_pages=None):
    rng = np.random.Generator(np.random.PCG64(seed))
    B, pps = len(lens), capacity // R.PAGE
    cu = np.concatenate(([0], np.cumsum(rows))).astype(np.int64)
    M = int(cu[-1]) + pad
    held = [min(pps, -(-max(0, n) // R.PAGE) + int(e)) for n, e in zip(lens, held_extra)]
    n_pages = n_pages or sum(held) + n_free + taken + 3
    perm = rng.permutation(n_pages)
    table = rng.integers(0, n_pages, size=(B, pps))     # what lies behind the held pages is noise
    k = 0
    for b in range(B):
        table[b, :held[b]] = perm[k:k + held[b]]
        k += held[b]
    free = perm[k:k + n_free + taken]
    want = R.chunk_map(lens, cu, M, capacity, table, held, free, taken, n_pages)
    cache = D.KVCache(1, B, 1, capacity, 128, "bf16", DEV, page_table=i32(table), n_pages=n_pages)
    cache.lens.copy_(i32(lens)[None])
    plan = D.ChunkPlan(i32(cu), M)
    plan.slots.fill_(-77), plan.positions.fill_(-77), plan.kv_lens.fill_(-77)
    pool = (D.PagePool(i32(held), i32(free), i32([taken])) if in_place else
            D.PagePool(i32(held), i32(free), i32([taken]), i32([0] * B), i32([0])))
    return cache, plan, pool, want


def _check_map(cache, plan, pool, want):
    slots, positions, kv, table, held, taken = want
    assert plan.slots.tolist() == list(slots)
    assert plan.positions.tolist() == list(positions)
    assert plan.kv_lens.tolist() == list(kv)
    assert cache.block_table.cpu().numpy().tolist() == table.tolist()
    assert pool.pages_held_out.tolist() == list(held)
    assert pool.taken_out.tolist() == [taken]


@pytest.mark.parametrize("B,hi,pad,in_place", [(1, 1, 0, False), (1, 0, 3, True), (37, 5, 2, True),
                                               (130, 300, 7, False), (1025, 3, 0, True), (3, 4000, 1, False)])
def test_map(D, B, hi, pad, in_place):
    rng = np.random.Generator(np.random.PCG64(B))
    lens = rng.integers(0, 600, size=B)
    rows = rng.integers(0, hi + 1, size=B)
    cap = int(-(-(lens + rows).max() // 128) * 128 + 128)
    args = _map_case(D, lens, rows, cap, rng.integers(0, 2, size=B), 4 * B + int(rows.sum()) // 64, pad, B, 2, in_place)
    D.dflash_chunk_map(args[0], 0, args[1], args[2])
    _check_map(*args)
    assert D.dflash_status_get() == 0
    if not in_place:   # the same inputs again: the same results
        D.dflash_chunk_map(args[0], 0, args[1], args[2])
        _check_map(*args)


def test_map_refuses_by_capacity_and_by_pages(D):
    lens, rows = [100, 500, 127, 384, 10, 128], [30, 20, 1, 1, 200, 128]
    # sequence 1 outgrows 512; two free pages: 0 and 4 take them, 5 gets none; 2 and 3 need none
    args = _map_case(D, lens, rows, 512, [0, 0, 0, 1, 0, 0], 2)
    D.dflash_chunk_map(args[0], 0, args[1], args[2])
    _check_map(*args)
    assert args[1].kv_lens.tolist() == [130, 0, 128, 385, 210, 0]
    assert D.dflash_status_get() == D.DEV_CAPACITY


def test_map_once_short_refuses_every_later_sequence_that_needs_a_page(D):
    # 0 takes one of two pages, 1 asks two (short); 2 would fit in the one left, but comes
    # after; 3 needs none
    args = _map_case(D, [100, 10, 120, 5], [30, 300, 20, 3], 512, [0, 0, 0, 0], 2)
    D.dflash_chunk_map(args[0], 0, args[1], args[2])
    _check_map(*args)
    assert args[1].kv_lens.tolist() == [130, 0, 0, 8]
    assert D.dflash_status_get() == D.DEV_CAPACITY


def test_map_bad_row_ranges_and_pages(D):
    args = _map_case(D, [10, 20, 30], [4, 5, 6], 256, [0, 0, 0], 9)
    cache, plan, pool, _ = args
    plan.cu_rows.copy_(i32([0, 9, 5, 15]))          # sequence 1 runs backwards
    D.dflash_chunk_map(cache, 0, plan, pool)
    assert plan.kv_lens.tolist() == [19, 0, 40]
    assert D.dflash_status_get() == D.DEV_ROWS
    cache, plan, pool, want = _map_case(D, [128, 5], [3, 2], 256, [0, 0], 4)
    pool.free_pages.copy_(i32([10 ** 6] * 4))       # ids outside the pool
    D.dflash_chunk_map(cache, 0, plan, pool)
    assert plan.slots.tolist()[:3] == [-1] * 3 and plan.slots.tolist()[3:] == want[0][3:]
    assert D.dflash_status_get() == D.DEV_PAGE


def test_map_contiguous(D):
    lens, rows, cap = [3, 0, 70, 90], [5, 0, 1, 11], 100
    cu = np.concatenate(([0], np.cumsum(rows)))
    cache = D.KVCache(2, 4, 2, cap, 64, "f32", DEV)
    cache.lens[1] = i32(lens)
    plan = D.ChunkPlan(i32(cu), 20)
    D.dflash_chunk_map(cache, 1, plan)
    want = R.chunk_map(lens, cu, 20, cap)
    assert plan.slots.tolist() == want[0] and plan.positions.tolist() == want[1]
    assert plan.kv_lens.tolist() == [8, 0, 71, 0]
    assert D.dflash_status_get() == D.DEV_CAPACITY


# ---------------------------------------------------------------------------
# a step on random data
# ---------------------------------------------------------------------------

class Step:
    """A cache with random rows, a mapped plan and projected rows, and their float64 copies."""

    def __init__(self, D, kv, heads, ctx, rows, paged=True, layers=1, layer=0, pad=0, seed=0,
                 fused=True, d_scale=1.0, spare=128):
        self.D, self.kv, self.layer, self.pad = D, kv, layer, pad
        self.n_h, self.n_kv, self.d = heads
        self.G = self.n_h // self.n_kv
        dt = TORCH[kv]
        g = torch.Generator().manual_seed(seed)
        B = len(ctx)
        self.B, self.ctx, self.rows = B, ctx, rows
        cap = -(-max(c + n for c, n in zip(ctx, rows)) // 128) * 128 + spare
        self.cap = cap
        self.scales = np.array([[0.5 + l, 0.25 / (1 + l)] for l in range(layers)]) if kv == "fp8" else None
        self.dims = D.make_dims(self.n_h * self.d, self.n_h, self.n_kv, self.d, 1, 1, 1e-6, dt)
        self.cache = D.KVCache(layers, B, self.n_kv, cap, self.d, dt, DEV, paged=paged, seed=seed,
                               kv="fp8" if kv == "fp8" else "bf16", kv_scales=self.scales,
                               n_pages=B * (cap // 128) + 2 if paged else None)
        c = self.cache
        self.nan = float("nan")
        # every slot starts as NaN; the cached rows get values
        if kv == "fp8":
            c.k.fill_(0x7F), c.v.fill_(0x7F)
        else:
            c.k.fill_(self.nan), c.v.fill_(self.nan)
        for l in range(layers):
            for b in range(B):
                rows_ = [torch.randn((self.n_kv, ctx[b], self.d), generator=g) for _ in range(2)]
                if kv == "fp8":
                    rows_ = [x.to(torch.float8_e4m3fn).view(torch.uint8) for x in rows_]
                c.set_rows(l, b, rows_[0].to(DEV, c.k.dtype), rows_[1].to(DEV, c.v.dtype))
            c.lens[l] = i32(ctx)
        self.cu = np.concatenate(([0], np.cumsum(rows))).astype(np.int64)
        self.M = int(self.cu[-1]) + pad
        self.plan = D.ChunkPlan(i32(self.cu), self.M)
        widths = (self.n_h * self.d, self.n_kv * self.d, self.n_kv * self.d)
        if fused:
            x = torch.randn((self.M, sum(widths)), generator=g).to(DEV, dt)
            self.q, self.k, self.v = x.split(widths, dim=1)
        else:
            self.q, self.k, self.v = (torch.randn((self.M, w), generator=g).to(DEV, dt) for w in widths)
        self.gq = (1 + 0.2 * torch.randn(self.d, generator=g)).to(DEV, dt)
        self.gk = (1 + 0.2 * torch.randn(self.d, generator=g)).to(DEV, dt)
        self.table = torch.empty((cap, self.d // 2, 2), dtype=torch.float32, device=DEV)
        D.dflash_rope_table_build(1e6, self.d, cap, self.table)
        self.ws = torch.full((D.dflash_chunk_workspace_bytes(self.dims),), 0xFF, dtype=torch.uint8, device=DEV)
        if paged:
            held = [-(-x // 128) for x in ctx]
            # each sequence's own next pages are the free list's, in the order they are asked for
            free = [int(c.block_table[b, i]) for b in range(B)
                    for i in range(held[b], -(-(ctx[b] + rows[b]) // 128))]
            self.pool = D.PagePool(i32(held), i32(free or [0]), i32([0]))
        else:
            self.pool = None

    def map(self):
        self.D.dflash_chunk_map(self.cache, self.layer, self.plan, self.pool)

    def append(self, q_out):
        self.D.dflash_chunk_append(self.dims, self.cache, self.layer, self.plan, self.q, self.k, self.v,
                                   self.gq, self.gk, self.table, self.cap, q_out)

    def attn(self, q, out, window=0, scaling=0.0):
        self.D.dflash_chunk_attn(self.dims, self.cache, self.layer, self.plan, q, window, scaling, out, self.ws)

    def cached(self, b, n):
        """float64 K, V rows 0 .. n-1 of sequence b as stored: [n][n_kv][d]."""
        return tuple(np64(self.cache.rows(w, self.layer, b, 0, n)).transpose(1, 0, 2) for w in "kv")

    def check_attn(self, q, out, window=0, scaling=None, kv_lens=None, skip=()):
        sc = scaling or self.d ** -0.5
        qn, on = np64(q).reshape(self.M, self.n_h, self.d), np64(out).reshape(self.M, self.n_h, self.d)
        kvl = self.plan.kv_lens.tolist() if kv_lens is None else kv_lens
        for b in range(self.B):
            lo, hi = int(self.cu[b]), int(self.cu[b + 1])
            if hi == lo or b in skip:
                continue
            k, v = self.cached(b, kvl[b])
            ref, mag, big, keys = R.attention(qn[lo:hi], k, v, kvl[b], hi - lo, self.G, window, sc)
            tol = R.attention_bound(ref, mag, big, keys, self.d, "f32" if self.kv == "f32" else "bf16")
            err = np.abs(on[lo:hi] - ref)
            assert np.isfinite(on[lo:hi]).all(), f"sequence {b}: not finite"
            worst = np.unravel_index(np.argmax(err - tol), err.shape)
            assert (err <= tol).all(), (f"sequence {b}: row, head, dim {worst}: {on[lo:hi][worst]} "
                                        f"against {ref[worst]}, bound {tol[worst]}")


# ---------------------------------------------------------------------------
# append
# ---------------------------------------------------------------------------

APPEND = [("bf16", (32, 8, 128), True), ("bf16", (5, 1, 128), False), ("fp8", (8, 8, 128), True),
          ("fp8", (14, 2, 128), False), ("f32", (8, 8, 64), False), ("f32", (6, 2, 80), False),
          ("f32", (3, 3, 256), False), ("f32", (4, 1, 2), False)]


@pytest.mark.parametrize("kv,heads,paged", APPEND)
@pytest.mark.parametrize("fused", [True, False])
def test_append(D, kv, heads, paged, fused):
    s = Step(D, kv, heads, [0, 130, 250, 7], [3, 1, 17, 0], paged, layers=2, layer=1, pad=2, seed=3, fused=fused)
    s.map()
    before = [t.clone() for t in (s.cache.k, s.cache.v)]
    q_out = torch.full((s.M, s.n_h * s.d), 7.0, dtype=s.q.dtype, device=DEV)
    s.append(q_out)
    assert D.dflash_status_get() == 0
    assert s.cache.lens.tolist() == [s.ctx, [3, 131, 267, 7]]
    pos = s.plan.positions.tolist()
    for b in range(s.B):
        for r in range(int(s.cu[b]), int(s.cu[b + 1])):
            for name, x, gamma, n in (("q", s.q, s.gq, s.n_h), ("k", s.k, s.gk, s.n_kv), ("v", s.v, None, s.n_kv)):
                y, mag = R.norm_rope(np64(x[r]).reshape(n, s.d), None if gamma is None else np64(gamma),
                                     pos[r], rope=name != "v")
                out = "f32" if kv == "f32" else "bf16"
                if name == "q":
                    got = np64(q_out[r]).reshape(n, s.d)
                else:
                    got = np64(s.cache.rows(name, 1, b, pos[r], pos[r] + 1, codes=True))[:, 0]
                    if kv == "fp8":
                        sc, out = s.scales[1][0 if name == "k" else 1], "e4m3"
                        y, mag = y / sc, mag / sc
                assert (np.abs(got - y) <= R.append_bound(y, mag, s.d, out)).all(), (b, r, name)
    assert (q_out[int(s.cu[-1]):] == 7.0).all()     # padding rows: as they were
    # nothing but the new rows' slots changed
    unit = 128 if paged else s.cap
    for now, old in zip((s.cache.k, s.cache.v), before):
        for t in s.plan.slots.tolist():
            if t >= 0:
                now[1, t // unit, :, t % unit] = old[1, t // unit, :, t % unit]
        assert torch.equal(now.view(torch.uint8), old.view(torch.uint8))


def test_append_without_q_norm_and_rotation(D):
    s = Step(D, "bf16", (4, 2, 128), [5, 100], [9, 60], seed=4)
    s.map()
    D.dflash_chunk_append(s.dims, s.cache, 0, s.plan, None, s.k, s.v, None, None, None, 0, None)
    for b in range(2):
        lo, hi = s.ctx[b], s.ctx[b] + s.rows[b]
        for w, x in (("k", s.k), ("v", s.v)):
            want = x[int(s.cu[b]):int(s.cu[b + 1])].reshape(s.rows[b], 2, 128).permute(1, 0, 2)
            assert torch.equal(s.cache.rows(w, 0, b, lo, hi), want)
    assert D.dflash_status_get() == 0


def test_append_in_place_and_numpy_like_views(D):
    s = Step(D, "bf16", (8, 2, 128), [64, 3], [70, 1], seed=5, fused=False)
    s.map()
    apart = torch.empty_like(s.q)
    s.append(apart)
    q = s.q.clone()
    D.dflash_chunk_append(s.dims, s.cache, 0, s.plan, q.view(s.M, 8, 128), s.k.view(s.M, 2, 128), s.v, s.gq, s.gk,
                          s.table, s.cap, q)
    assert torch.equal(q, apart)


@pytest.mark.parametrize("kv", ["bf16", "f32"])
def test_append_skips_bad_slots_and_positions(D, kv):
    s = Step(D, kv, (2, 1, 128), [0, 40], [4, 4], paged=kv == "bf16", seed=6)
    s.map()
    keep = s.plan.slots.clone()
    s.plan.slots[1] = -5
    s.plan.slots[6] = 2 ** 31 - 1
    before = s.cache.k.clone()
    q_out = torch.full_like(s.q, 3.0)
    s.append(q_out)
    assert D.dflash_status_get() == D.DEV_PAGE
    assert (q_out[1] == 3.0).all() and (q_out[6] == 3.0).all() and not (q_out[0] == 3.0).any()
    s.cache.k.copy_(before)
    s.cache.lens.copy_(i32(s.ctx)[None])
    s.plan.slots.copy_(keep)
    D.dflash_chunk_append(s.dims, s.cache, 0, s.plan, s.q, s.k, s.v, s.gq, s.gk, s.table, 42, q_out.fill_(3.0))
    assert D.dflash_status_get() == D.DEV_ROPE       # positions 42 and 43 are beyond the table
    assert (q_out[6:8] == 3.0).all() and not (q_out[5] == 3.0).any()
    assert s.cache.lens[0].tolist() == [4, 40]


# ---------------------------------------------------------------------------
# attention
# ---------------------------------------------------------------------------

# (ctx, rows): single tokens, blocks, ragged chunks, empty sequences, page ends inside and at
# tile borders, an item's border, a long axis that is cut over many CTAs
SHAPES = {
    "token": ([0, 1, 126, 127, 128, 129, 700], [1] * 7),
    "block": ([250, 0, 1023, 128, 5, 300], [16, 16, 16, 16, 0, 7]),
    "chunk": ([0, 77, 300], [129, 64, 201]),
    "long": ([9000, 3], [2, 1]),
}
HEADS = [("bf16", (32, 8, 128), True), ("bf16", (8, 8, 128), False), ("bf16", (14, 2, 128), True),
         ("bf16", (128, 1, 128), True), ("fp8", (32, 8, 128), True), ("fp8", (20, 4, 128), False),
         ("fp8", (2, 2, 128), True), ("f32", (8, 8, 64), False), ("f32", (6, 2, 80), False),
         ("f32", (3, 3, 256), False), ("f32", (70, 1, 32), False)]


@pytest.mark.parametrize("shape", list(SHAPES))
@pytest.mark.parametrize("window", [0, 1, 100, 300])
@pytest.mark.parametrize("kv,heads,paged", HEADS)
def test_attn(D, kv, heads, paged, window, shape):
    ctx, rows = SHAPES[shape]
    s = Step(D, kv, heads, ctx, rows, paged, pad=3, seed=window + len(ctx))
    s.map()
    q = torch.empty((s.M, s.n_h * s.d), dtype=s.q.dtype, device=DEV)
    s.append(q)
    out = torch.full_like(q, 5.0)
    s.attn(q, out, window)
    assert D.dflash_status_get() == 0
    s.check_attn(q, out, window)
    assert (out[int(s.cu[-1]):] == 5.0).all()       # padding rows: as they were


@pytest.mark.parametrize("kv,heads,paged", [("bf16", (4, 2, 128), True), ("fp8", (4, 1, 128), True),
                                            ("f32", (2, 2, 64), False)])
def test_attn_strided_queries_scaling_and_second_layer(D, kv, heads, paged):
    s = Step(D, kv, heads, [40, 500], [33, 2], paged, layers=3, layer=2, seed=9)
    s.map()
    s.append(torch.empty((s.M, s.n_h * s.d), dtype=s.q.dtype, device=DEV))
    out = torch.empty((s.M, s.n_h * s.d), dtype=s.q.dtype, device=DEV)
    s.attn(s.q, out, 0, 0.03)                        # rows of a fused projection, not dense
    s.check_attn(s.q, out, 0, 0.03)
    assert D.dflash_status_get() == 0


@pytest.mark.parametrize("kv", ["bf16", "fp8", "f32"])
@pytest.mark.parametrize("value", [float("nan"), float("inf")])
def test_attn_hidden_keys_never_enter(D, kv, value):
    """A later row's K and V (and rows below the window) hold NaN or infinity: earlier rows of
    the same chunk do not see them."""
    if kv == "fp8" and value == float("inf"):
        pytest.skip("E4M3 has no infinity")
    s = Step(D, kv, (4, 2, 128), [200, 128], [150, 5], paged=kv != "f32", seed=10)
    s.map()
    q = torch.empty((s.M, s.n_h * s.d), dtype=s.q.dtype, device=DEV)
    s.append(q)
    want = torch.empty_like(q)
    s.attn(q, want, 120)
    s.check_attn(q, want, 120)
    bad = 0x7F if kv == "fp8" else value
    hurt = {0: (260, 40), 1: (131, None)}            # a key inside the chunk, one below the window
    for b, (late, early) in hurt.items():
        for t in (s.cache.k, s.cache.v):
            for pos in (late, early):
                if pos is None:
                    continue
                if s.cache.paged:
                    t[0, s.cache.block_table[b, pos // 128].item(), :, pos % 128] = bad
                else:
                    t[0, b, :, pos] = bad
    out = torch.empty_like(q)
    s.attn(q, out, 120)
    for b, (late, _) in hurt.items():
        lo, first = int(s.cu[b]), late - s.ctx[b]
        assert torch.equal(out[lo:lo + first], want[lo:lo + first]), b      # rows before it
        seen = out[lo + first:int(s.cu[b + 1])]
        sees = min(seen.shape[0], 120)
        assert not torch.isfinite(seen[:sees].float()).any()
        assert torch.equal(seen[120:], want[lo + first + 120:int(s.cu[b + 1])])  # past the window
    assert D.dflash_status_get() == 0


@pytest.mark.parametrize("kv", ["bf16", "fp8", "f32"])
def test_attn_refused_sequences_and_rows_without_keys(D, kv):
    s = Step(D, kv, (4, 2, 128), [60, 200, 10], [4, 150, 3], paged=kv != "f32", seed=11)
    s.map()
    q = torch.empty((s.M, s.n_h * s.d), dtype=s.q.dtype, device=DEV)
    s.append(q)
    s.plan.kv_lens[0] = 0                            # refused
    s.plan.kv_lens[1] = 100                          # fewer rows held than new ones: 50 see none
    out = torch.full_like(q, float("nan"))
    s.attn(q, out)
    assert (out[:4] == 0).all() and (out[4:54] == 0).all()
    s.check_attn(q, out)
    assert D.dflash_status_get() == 0
    s.plan.kv_lens[2] = s.cap + 1
    s.plan.kv_lens[0] = -1
    s.attn(q, out.fill_(float("nan")))
    assert D.dflash_status_get() == D.DEV_CAPACITY
    assert (out[:4] == 0).all() and (out[154:] == 0).all()
    s.check_attn(q, out, skip=(0, 2))


def test_attn_bad_row_ranges_are_skipped(D):
    s = Step(D, "bf16", (4, 2, 128), [60, 200, 10], [4, 6, 3], seed=12)
    s.map()
    q = torch.empty((s.M, s.n_h * s.d), dtype=s.q.dtype, device=DEV)
    s.append(q)
    s.plan.cu_rows.copy_(i32([0, 4, 2, 999]))
    out = torch.full_like(q, 9.0)
    s.attn(q, out)
    assert D.dflash_status_get() == D.DEV_ROWS
    assert (out[4:] == 9.0).all() and not (out[:4] == 9.0).any()


@pytest.mark.parametrize("kv", ["bf16", "fp8"])
def test_attn_bad_pages_read_as_zeros(D, kv):
    s = Step(D, kv, (4, 2, 128), [300], [5], seed=13)
    s.map()
    q = torch.empty((s.M, s.n_h * s.d), dtype=s.q.dtype, device=DEV)
    s.append(q)
    out, want = torch.empty_like(q), torch.empty_like(q)
    page = s.cache.block_table[0, 1].item()
    s.cache.k[0, page].zero_()
    s.cache.v[0, page].zero_()
    s.attn(q, want)
    for bad in (-1, s.cache.n_pages, 2 ** 31 - 1, -2 ** 31):
        s.cache.block_table[0, 1] = bad
        s.attn(q, out)
        assert D.dflash_status_get() == D.DEV_PAGE
        assert torch.equal(out, want)


@pytest.mark.parametrize("kv,heads", [("bf16", (32, 8, 128)), ("fp8", (32, 8, 128)), ("f32", (8, 8, 64))])
def test_attn_repeats_bit_for_bit(D, kv, heads):
    s = Step(D, kv, heads, [4000, 100, 0], [16, 300, 40], paged=kv != "f32", seed=14)
    s.map()
    q = torch.empty((s.M, s.n_h * s.d), dtype=s.q.dtype, device=DEV)
    s.append(q)
    outs = []
    for fill in (0.0, 1.0, float("nan")):
        out = torch.full_like(q, fill)
        s.ws.fill_(0xFF if fill else 0)
        s.attn(q, out)
        outs.append(out)
    assert torch.equal(outs[0], outs[1]) and torch.equal(outs[0], outs[2])


# ---------------------------------------------------------------------------
# together
# ---------------------------------------------------------------------------

@pytest.mark.parametrize("graph", [False, True])
@pytest.mark.parametrize("kv", ["bf16", "fp8"])
def test_rounds_with_acceptance_and_crop(D, kv, graph):
    """Verification rounds as a server runs them: map, two layers of append and attention,
    acceptance, crop; lengths, pages and offsets stay on the device, and the same step runs
    as a captured graph. The cache is compared with rows rebuilt from the accepted tokens."""
    B, bs, L, n_h, n_kv, d, cap = 5, 6, 2, 8, 2, 128, 384
    g = torch.Generator().manual_seed(1)
    dt = torch.bfloat16
    dims = D.make_dims(n_h * d, n_h, n_kv, d, 1, bs, 1e-6, dt)
    n_pages = B * (cap // 128)
    cache = D.KVCache(L, B, n_kv, cap, d, dt, DEV, page_table=torch.full((B, cap // 128), -1), n_pages=n_pages,
                      kv="fp8" if kv == "fp8" else "bf16", kv_scales=[[0.5, 0.25]] * L)
    pool = D.PagePool(i32([0] * B), i32(np.random.default_rng(3).permutation(n_pages)), i32([0]))
    cu, M = i32(np.arange(B + 1) * bs), B * bs
    plan = D.ChunkPlan(cu, M)
    table = torch.empty((cap, d // 2, 2), dtype=torch.float32, device=DEV)
    D.dflash_rope_table_build(1e6, d, cap, table)
    ones = torch.ones(d, dtype=dt, device=DEV)
    ws = torch.empty(D.dflash_chunk_workspace_bytes(dims), dtype=torch.uint8, device=DEV)
    x = [torch.zeros((M, (n_h + 2 * n_kv) * d), dtype=dt, device=DEV) for _ in range(L)]
    q = torch.empty((M, n_h * d), dtype=dt, device=DEV)
    out = [torch.empty_like(q) for _ in range(L)]
    ids, post = (torch.zeros((B, bs), dtype=torch.int32, device=DEV) for _ in range(2))
    start = cache.lens[0].clone()
    acc, nxt, anchor = (torch.zeros(B, dtype=torch.int32, device=DEV) for _ in range(3))
    ncu = torch.zeros(B + 1, dtype=torch.int32, device=DEV)

    def step():
        start.copy_(cache.lens[0])
        D.dflash_chunk_map(cache, 0, plan, pool)
        for l in range(L):
            a, b, c = x[l].split((n_h * d, n_kv * d, n_kv * d), 1)
            D.dflash_chunk_append(dims, cache, l, plan, a, b, c, ones, ones, table, cap, q)
            D.dflash_chunk_attn(dims, cache, l, plan, q, 0 if l == 0 else 50, 0.0, out[l], ws)
        D.dflash_accept(ids, post, start, acc, ncu, nxt, anchor)
        D.dflash_cache_crop(cache, nxt)

    if graph:
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            step()                                   # warm-up, then back to the empty cache
        torch.cuda.current_stream().wait_stream(side)
        cache.lens.zero_(), pool.pages_held.zero_(), pool.taken.zero_(), cache.block_table.fill_(-1)
        gr = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gr):
            step()
    held_rows = [[[] for _ in range(B)] for _ in range(L)]   # accepted (k, v) rows in float64
    want_lens = [0] * B
    for rnd in range(40):
        for l in range(L):
            x[l].copy_(torch.randn(x[l].shape, generator=g))
        ids.copy_(torch.randint(0, 3, (B, bs), generator=g))
        post.copy_(torch.randint(0, 3, (B, bs), generator=g))
        gr.replay() if graph else step()
        torch.cuda.synchronize()
        a = acc.tolist()
        for b in range(B):
            want_lens[b] += a[b] + 1
        assert cache.lens.tolist() == [want_lens] * L
        assert pool.pages_held.tolist() == [-(-(n - a[b] - 1 + bs) // 128) for b, n in enumerate(want_lens)]
        if rnd % 13 == 12:
            for l in range(L):
                qn = np.zeros((M, n_h, d))
                for b in range(B):
                    n0 = want_lens[b] - a[b] - 1
                    for i in range(bs):
                        qn[b * bs + i] = R.norm_rope(np64(x[l][b * bs + i])[:n_h * d].reshape(n_h, d), np.ones(d), n0 + i)[0]
                    k, v = (np64(cache.rows(w, l, b, 0, n0 + bs)).transpose(1, 0, 2) for w in "kv")
                    qr = np64(torch.tensor(qn[b * bs:(b + 1) * bs]).to(dt))
                    ref, mag, big, keys = R.attention(qr, k, v, n0 + bs, bs, n_h // n_kv, 0 if l == 0 else 50, d ** -0.5)
                    # q as rounded here may sit one step from the kernel's: scores move by at
                    # most 2^-7 of sum |q k| scaling of the few elements at a rounding border;
                    # held to a tenth of that for all of them together
                    tol = R.attention_bound(ref, mag, big, keys, d, "bf16") + mag * big * 2.0 ** -7 * 0.1
                    got = np64(out[l][b * bs:(b + 1) * bs]).reshape(bs, n_h, d)
                    assert (np.abs(got - ref) <= tol).all(), (rnd, l, b)
    # the table names each held page once
    pages = [int(cache.block_table[b, i]) for b in range(B) for i in range(int(pool.pages_held[b]))]
    assert len(set(pages)) == len(pages) == int(pool.taken[0])
    assert D.dflash_status_get() == 0


def test_two_streams_with_their_own_workspaces(D):
    steps = [Step(D, "bf16", (32, 8, 128), [3000, 50], [20, 300], seed=20 + i) for i in range(2)]
    qs = []
    for s in steps:
        s.map()
        q = torch.empty((s.M, s.n_h * s.d), dtype=s.q.dtype, device=DEV)
        s.append(q)
        qs.append(q)
    want = [torch.empty_like(q) for q in qs]
    for s, q, o in zip(steps, qs, want):
        s.attn(q, o)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in steps]
    outs = [torch.empty_like(q) for q in qs]
    for _ in range(20):
        for s, q, o, st in zip(steps, qs, outs, streams):
            D.dflash_chunk_attn(s.dims, s.cache, 0, s.plan, q, 0, 0.0, o, s.ws, stream=st)
    torch.cuda.synchronize()
    for o, w in zip(outs, want):
        assert torch.equal(o, w)


def test_launches_and_trace_kinds(D):
    s = Step(D, "bf16", (8, 2, 128), [100], [20], seed=30)
    q = torch.empty((s.M, s.n_h * s.d), dtype=s.q.dtype, device=DEV)
    out = torch.empty_like(q)
    D.dflash_trace_start(("chunk_map", "chunk_append", "chunk_attn", "chunk_merge"), 16)
    n0 = D.dflash_launch_count()
    s.map(), s.append(q), s.attn(q, out)
    assert D.dflash_launch_count() - n0 == 4
    assert [k for k, _ in D.dflash_trace_stop()] == ["chunk_map", "chunk_append", "chunk_attn", "chunk_merge"]


# ---------------------------------------------------------------------------
# calls at the edges of what the documentation allows
# ---------------------------------------------------------------------------

@pytest.mark.parametrize("n_free,short", [(1024, False), (40, True)])   # about 100 pages are asked for
def test_map_most_sequences(D, n_free, short):
    B = 8192
    rng = np.random.Generator(np.random.PCG64(5))
    lens, rows = rng.integers(0, 300, size=B), rng.integers(0, 4, size=B)
    args = _map_case(D, lens, rows, 512, [0] * B, n_free, 5, 6, 1)
    D.dflash_chunk_map(args[0], 0, args[1], args[2])
    _check_map(*args)
    assert D.dflash_status_get() == (D.DEV_CAPACITY if short else 0)


@pytest.mark.parametrize("kv", ["bf16", "f32"])
def test_append_of_one_slot_twice_stores_elements_of_the_two_rows(D, kv):
    s = Step(D, kv, (4, 2, 128), [10], [300], paged=kv != "f32", seed=40)
    s.map()
    q = torch.empty((s.M, s.n_h * s.d), dtype=s.q.dtype, device=DEV)
    s.append(q)
    rows = [[x[:, 10 + i].clone() for x in (s.cache.rows(w, 0, 0, 0, 310) for w in "kv")] for i in (7, 290)]
    at = [int(s.plan.slots[i]) for i in (7, 290)]
    pos = s.plan.positions.clone()
    s.plan.slots[290] = at[0]
    s.append(q)
    assert torch.equal(s.plan.positions, pos)
    got = [x[:, 17] for x in (s.cache.rows(w, 0, 0, 0, 310) for w in "kv")]
    for w in range(2):   # (no order among the rows' heads is promised)
        assert ((got[w] == rows[0][w]) | (got[w] == rows[1][w])).all()
    assert D.dflash_status_get() == 0


@pytest.mark.parametrize("kv", ["bf16", "fp8", "f32"])
def test_attn_many_sequences(D, kv):
    rng = np.random.Generator(np.random.PCG64(41))
    B = 1500
    ctx, rows = rng.integers(0, 140, size=B).tolist(), rng.integers(0, 4, size=B).tolist()
    s = Step(D, kv, (4, 2, 128), ctx, rows, paged=kv != "f32", pad=2, seed=41, spare=0)
    s.map()
    q = torch.empty((s.M, s.n_h * s.d), dtype=s.q.dtype, device=DEV)
    s.append(q)
    out = torch.full_like(q, 5.0)
    s.attn(q, out)
    assert D.dflash_status_get() == 0
    s.check_attn(q, out)
    assert (out[int(s.cu[-1]):] == 5.0).all()


@pytest.mark.parametrize("kv", ["bf16", "fp8", "f32"])
def test_step_without_new_rows(D, kv):
    """Padding only: nothing is written, the lengths stay."""
    s = Step(D, kv, (4, 2, 128), [5, 130], [0, 0], paged=kv != "f32", pad=3, seed=42)
    s.map()
    assert s.plan.kv_lens.tolist() == [5, 130] and s.plan.slots.tolist() == [-1] * 3
    before = s.cache.k.clone()
    q = torch.full((s.M, s.n_h * s.d), 2.0, dtype=s.q.dtype, device=DEV)
    s.append(q)
    out = torch.full_like(q, 5.0)
    s.attn(q, out)
    assert (q == 2.0).all() and (out == 5.0).all() and s.cache.lens[0].tolist() == [5, 130]
    assert torch.equal(s.cache.k.view(torch.uint8), before.view(torch.uint8))
    assert D.dflash_status_get() == 0


@pytest.mark.parametrize("heads", [(4, 1, 2), (4, 1, 130), (4, 4, 254)])
def test_attn_f32_widths(D, heads):
    s = Step(D, "f32", heads, [0, 70, 300], [20, 1, 90], paged=False, seed=43)
    s.map()
    q = torch.empty((s.M, s.n_h * s.d), dtype=s.q.dtype, device=DEV)
    s.append(q)
    out = torch.empty_like(q)
    s.attn(q, out)
    s.check_attn(q, out)


@pytest.mark.parametrize("kv", ["bf16", "fp8"])
def test_attn_out_at_16_bytes(D, kv):
    s = Step(D, kv, (8, 2, 128), [3000, 50], [20, 300], seed=44)
    s.map()
    q = torch.empty((s.M, s.n_h * s.d), dtype=s.q.dtype, device=DEV)
    s.append(q)
    want = torch.empty_like(q)
    s.attn(q, want)
    flat = torch.full((q.numel() + 16,), 5.0, dtype=q.dtype, device=DEV)
    out = flat[8:8 + q.numel()].view_as(q)
    assert out.data_ptr() % 32 == 16
    s.attn(q, out)
    assert torch.equal(out, want)
    assert (flat[:8] == 5.0).all() and (flat[8 + q.numel():] == 5.0).all()


@pytest.mark.parametrize("kv", ["bf16", "fp8", "f32"])
@pytest.mark.parametrize("power", [-60, 60])
def test_attn_queries_of_any_size(D, kv, power):
    """Queries 2^60 larger or smaller with a scaling that makes up for it: the same scores, so
    the same bits."""
    s = Step(D, kv, (4, 2, 128), [200, 0], [3, 150], paged=kv != "f32", seed=45)
    s.map()
    q = torch.empty((s.M, s.n_h * s.d), dtype=s.q.dtype, device=DEV)
    s.append(q)
    out, want = torch.empty_like(q), torch.empty_like(q)
    s.attn(q, want, 0, 0.125)
    s.attn(q * 2.0 ** power, out, 0, 0.125 * 2.0 ** -power)
    assert torch.equal(out, want)
    s.check_attn(q, out, 0, 0.125)


@pytest.mark.parametrize("kv", ["bf16", "fp8", "f32"])
def test_step_beyond_32_bit_offsets(D, kv):
    """Rows more than 2^32 bytes into K and V."""
    if kv == "f32":
        s = Step(D, kv, (8, 8, 64), [5, 700], [3, 40], paged=False, seed=46, spare=2_200_064)
        assert s.cap * 8 * 64 * 4 > 2 ** 32
    else:
        s = Step(D, kv, (32, 8, 128), [700], [40], seed=46, spare=128 * (40000 if kv == "bf16" else 80000))
        page_bytes = 8 * 128 * 128 * (2 if kv == "bf16" else 1)
        assert int(s.cache.block_table[0, :6].max()) * page_bytes > 2 ** 32
    s.map()
    q = torch.empty((s.M, s.n_h * s.d), dtype=s.q.dtype, device=DEV)
    s.append(q)
    out = torch.empty_like(q)
    s.attn(q, out)
    assert D.dflash_status_get() == 0
    s.check_attn(q, out)
    k, _ = s.cached(len(s.ctx) - 1, s.ctx[-1] + s.rows[-1])
    assert np.isfinite(k).all() and (k[s.ctx[-1]:] != 0).any()


def test_two_graphs_with_their_own_workspaces(D):
    steps = [Step(D, "bf16", (32, 8, 128), [3000, 50], [20, 300], seed=50 + i) for i in range(2)]
    graphs, outs, want = [], [], []
    for s in steps:
        s.map()
        q = torch.empty((s.M, s.n_h * s.d), dtype=s.q.dtype, device=DEV)
        s.append(q)
        want.append(torch.empty_like(q))
        s.attn(q, want[-1])
        outs.append(torch.empty_like(q))
        torch.cuda.synchronize()
        gr = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gr):
            s.attn(q, outs[-1])
        graphs.append((gr, q))
    streams = [torch.cuda.Stream() for _ in steps]
    for _ in range(10):
        for (gr, _), st in zip(graphs, streams):
            with torch.cuda.stream(st):
                gr.replay()
    torch.cuda.synchronize()
    for o, w in zip(outs, want):
        assert torch.equal(o, w)
    assert D.dflash_status_get() == 0


@pytest.mark.parametrize("kv", ["bf16", "fp8"])
def test_attn_that_gives_up_leaves_a_working_gpu(D, kv):
    """With a limit of 1 ns the roles of the kernel stop at their first wait. Copies and MMAs
    in flight are waited for and tensor memory is freed; the next call is right."""
    # the warp that checks the tiles at the mask's edge first waits for tens of microseconds
    s = Step(D, kv, (32, 8, 128), [100_000], [64], seed=60)
    s.map()
    q = torch.empty((s.M, s.n_h * s.d), dtype=s.q.dtype, device=DEV)
    s.append(q)
    out, want = torch.empty_like(q), torch.empty_like(q)
    s.attn(q, want)
    assert D.dflash_status_get() == 0
    st = 0
    try:
        D.dflash_test_wait_limit(1)
        for _ in range(3):
            s.attn(q, out)
            st |= D.dflash_status_get()
            if st & D.DEV_TIMEOUT:
                break
    finally:
        D.dflash_test_wait_limit(0)
    assert st == D.DEV_TIMEOUT
    out.fill_(float("nan"))
    s.attn(q, out)
    assert D.dflash_status_get() == 0
    assert torch.equal(out, want)
