"""The chunk step at the edges that its first tests leave out: weights and queries of extreme
spread, values that are not finite, large steps, what a round leaves in the cache."""
import numpy as np
import pytest
import torch

import chunk_ref as R
from test_chunk_gpu import DEV, D, Step, _check_map, _map_case, i32, np64  # noqa: F401  (D is the fixture)

pytestmark = pytest.mark.gpu


# ---------------------------------------------------------------------------
# attention: spread of the weights and of a query's elements
# ---------------------------------------------------------------------------

@pytest.mark.parametrize("B,heads,ctx,n", [(40, (8, 8, 128), 8191, 1), (2, (2, 2, 128), 4000, 300)])
@pytest.mark.parametrize("bits", [25.5, 31.0])
def test_attn_fp8_long_tail_behind_a_strong_key(D, B, heads, ctx, n, bits):
    """One key of weight 1 whose value is 0, and a long tail of keys of weight 2^-bits each: the
    output is the tail's. Weights are rounded to f16 for the product with V. They carry a factor
    2^7, so the rounding is relative (2^-11) down to 2^-21 of the row's reference weight and
    absolute below: half a step of f16's smallest numbers, 2^-25, over 2^7. The sum of a row's weights
    is at least that reference, so the output moves by at most keys 2^-32 max|V| on top of
    the ordinary bound."""
    s = Step(D, "fp8", heads, [ctx] * B, [n] * B, seed=70)
    s.map()
    g = torch.Generator().manual_seed(70)
    for b in range(B):
        K = torch.zeros((s.n_kv, ctx + n, 128))
        K[:, 0] = 1.0
        V = 1 + 0.25 * torch.rand((s.n_kv, ctx + n, 128), generator=g)
        V[:, 0] = 0.0
        s.cache.set_rows(0, b, *(x.to(torch.float8_e4m3fn).view(torch.uint8).to(DEV) for x in (K, V)))
    q = torch.ones((s.M, s.n_h * 128), dtype=torch.bfloat16, device=DEV)
    out = torch.empty_like(q)
    scaling = bits * float(np.log(2.0)) / (128 * s.scales[0][0])   # the strong key's score: bits ln 2
    s.attn(q, out, 0, scaling)
    assert D.dflash_status_get() == 0
    qn, on = np64(q).reshape(s.M, s.n_h, 128), np64(out).reshape(s.M, s.n_h, 128)
    for b in range(B):
        lo, hi = int(s.cu[b]), int(s.cu[b + 1])
        k, v = s.cached(b, ctx + n)
        ref, mag, big, keys = R.attention(qn[lo:hi], k, v, ctx + n, n, s.G, 0, scaling)
        tol = R.attention_bound(ref, mag, big, keys, 128, "bf16") + keys * 2.0 ** -32 * np.abs(v).max()
        # a tail that was lost would be off by ref: the bound is at most 4300 / 4001 / 2 1.25 / 1.12 of it
        assert (ref > 0).all() and (tol < 0.75 * ref).all()
        assert (np.abs(on[lo:hi] - ref) <= tol).all(), b


@pytest.mark.parametrize("n", [1, 40, 150])
@pytest.mark.parametrize("power", [4, 8, 10])
def test_attn_fp8_queries_with_outliers(D, n, power):
    """Query rows with two elements 2^power above the rest, whose keys are small. A query next to
    an E4M3 cache is two codes, each element off by at most 2^-17 of its row's largest power of
    two: scores by e = 2^-17 max|q| sum|k| scaling, and a weight, relative, by exp(2 e) - 1 (its own
    score and the sum's). The rest of the bound is the ordinary one."""
    s = Step(D, "fp8", (8, 2, 128), [300, 0, 77], [n, n, n], seed=71)
    s.map()
    far = [5, 100]
    for b in range(s.B):
        tot = s.ctx[b] + n
        K = torch.randn((2, tot, 128), generator=torch.Generator().manual_seed(b))
        K[:, :, far] *= 2.0 ** -power
        V = torch.randn((2, tot, 128), generator=torch.Generator().manual_seed(9 + b))
        s.cache.set_rows(0, b, *(x.to(torch.float8_e4m3fn).view(torch.uint8).to(DEV) for x in (K, V)))
    q = torch.randn((s.M, s.n_h, 128), generator=torch.Generator().manual_seed(72))
    q[:, :, far] *= 2.0 ** power
    q = q.reshape(s.M, -1).to(DEV, torch.bfloat16)
    out = torch.empty_like(q)
    s.attn(q, out)
    assert D.dflash_status_get() == 0
    qn, on = np64(q).reshape(s.M, s.n_h, 128), np64(out).reshape(s.M, s.n_h, 128)
    sc = 128 ** -0.5
    for b in range(s.B):
        lo, hi = int(s.cu[b]), int(s.cu[b + 1])
        k, v = s.cached(b, s.ctx[b] + n)
        ref, mag, big, keys = R.attention(qn[lo:hi], k, v, s.ctx[b] + n, n, s.G, 0, sc)
        e = 2.0 ** -17 * np.abs(qn[lo:hi]).max(-1) * np.abs(k).sum(-1).max() * sc      # [n][n_h]
        tol = R.attention_bound(ref, mag, big, keys, 128, "bf16") + 1.01 * mag * np.expm1(2 * e)[..., None]
        assert (np.abs(on[lo:hi] - ref) <= tol).all(), b


@pytest.mark.parametrize("n", [1, 150])
@pytest.mark.parametrize("k_scale,scaling", [(1e-12, 0.125), (0.5, 1e-30)])
def test_attn_fp8_scores_below_the_smallest_float(D, n, k_scale, scaling):
    """Scores that vanish (a query of zeros next to a small scale): every visible key counts the
    same, and masked keys still nothing."""
    s = Step(D, "fp8", (4, 2, 128), [200, 3], [n, n], seed=73)
    s.map()
    s.append(torch.empty((s.M, 512), dtype=torch.bfloat16, device=DEV))
    s.cache._scales_c[0] = s.cache.scales[0, 0] = k_scale
    q = torch.randn((s.M, 512), generator=torch.Generator().manual_seed(1)).to(DEV, torch.bfloat16)
    q[:, :256] = 0
    q[:, 256:384] *= 2.0 ** -100
    out = torch.empty_like(q)
    s.attn(q, out, 0, scaling)
    assert D.dflash_status_get() == 0
    s.check_attn(q, out, 0, scaling)


@pytest.mark.parametrize("kv", ["bf16", "fp8", "f32"])
@pytest.mark.parametrize("window", [0, 40])
def test_attn_rows_whose_scores_all_overflow(D, kv, window):
    """Rows that see keys, all at a score of minus infinity, have no softmax: NaN, not the zeros
    of a row that sees none. (Next to an E4M3 cache a query of infinities is NaN by itself.)"""
    s = Step(D, kv, (4, 2, 128), [700, 0, 9], [3, 150, 4], paged=kv != "f32", seed=74)
    s.map()
    q = torch.ones((s.M, 512), dtype=s.q.dtype, device=DEV)
    s.append(torch.empty_like(q))
    # every key has a positive first element (the sign of V does not matter)
    for b in range(s.B):
        K, V = (s.cache.rows(w, 0, b, 0, s.ctx[b] + s.rows[b]) for w in "kv")
        K, V = K.float().clone(), V.float().clone()
        K[:, :, 0] = 1.0
        if kv == "fp8":
            K, V = (x.to(torch.float8_e4m3fn).view(torch.uint8) for x in (K, V))
        s.cache.set_rows(0, b, K.to(s.cache.k.dtype), V.to(s.cache.v.dtype))
    plain = torch.empty_like(q)
    s.attn(q, plain, window)
    hurt = [0, 2, 3, 60, 152, 154]
    q[hurt, 0] = -float("inf")                       # head 0 only
    s.plan.kv_lens[2] = 2                            # rows 153 and 154 see no key
    out = torch.empty_like(q)
    s.attn(q, out, window)
    seen = [r for r in hurt if r < 153]
    assert torch.isnan(out[seen, :128]).all()
    assert (out[153:155] == 0).all()
    rest = [r for r in range(153) if r not in hurt]
    assert torch.equal(out[rest], plain[rest]) and torch.equal(out[seen, 128:], plain[seen, 128:])
    assert D.dflash_status_get() == 0


@pytest.mark.parametrize("kv", ["bf16", "f32"])
@pytest.mark.parametrize("ctx,n", [(9000, 3), (700, 150)])
def test_attn_some_keys_at_minus_infinity(D, kv, ctx, n):
    """Visible keys at a score of minus infinity weigh nothing, also where they are all that a piece
    of the key axis has."""
    s = Step(D, kv, (4, 2, 128), [ctx], [n], paged=kv != "f32", seed=78)
    s.map()
    s.append(torch.empty((s.M, 512), dtype=s.q.dtype, device=DEV))
    K, V = (s.cache.rows(w, 0, 0, 0, ctx + n).clone() for w in "kv")
    K[:, :300, 0] = float("inf")
    s.cache.set_rows(0, 0, K, V)
    q = s.q.reshape(s.M, 4, 128).clone()
    q[:, :, 0] = -1.0
    q = q.reshape(s.M, 512)
    out = torch.empty_like(q)
    s.attn(q, out)
    assert D.dflash_status_get() == 0
    k, v = s.cached(0, ctx + n)
    ref, mag, big, keys = R.attention(np64(q).reshape(s.M, 4, 128), k[300:], v[300:], ctx + n - 300, n, 2, 0, 128 ** -0.5)
    tol = R.attention_bound(ref, mag, big, keys, 128, kv)
    assert (np.abs(np64(out).reshape(s.M, 4, 128) - ref) <= tol).all()


@pytest.mark.parametrize("kv", ["bf16", "fp8", "f32"])
@pytest.mark.parametrize("window", [2 ** 31 - 1, 2 ** 31 - 64, 1000, 384, 383])
def test_attn_windows_as_long_as_the_cache_and_longer(D, kv, window):
    """Also where a sequence holds fewer rows than it has new ones, so that the first are at negative
    positions and see nothing."""
    s = Step(D, kv, (4, 2, 128), [0, 100], [150, 130], paged=kv != "f32", pad=1, seed=79, spare=0 if kv != "f32" else 128)
    s.map()
    q = torch.empty((s.M, 512), dtype=s.q.dtype, device=DEV)
    s.append(q)
    s.plan.kv_lens[0] = 98
    out = torch.full_like(q, 5.0)
    s.attn(q, out, window)
    assert D.dflash_status_get() == 0
    assert (out[:52] == 0).all() and (out[280:] == 5.0).all()
    s.check_attn(q, out, window)


@pytest.mark.parametrize("kv", ["bf16", "fp8", "f32"])
@pytest.mark.parametrize("ctx,rows,spare", [([40], [9], -79), ([0, 130], [1, 70], -55), ([0], [1], -127)])
def test_attn_contiguous_capacities_that_end_inside_a_tile(D, kv, ctx, rows, spare):
    """One KV head, so that the last tile reaches past the end of the cache."""
    s = Step(D, kv, (4, 1, 128), ctx, rows, paged=False, seed=80, spare=spare)
    assert s.cap == max(c + n for c, n in zip(ctx, rows)) + (0 if spare != -55 else 1)
    s.map()
    q = torch.empty((s.M, 512), dtype=s.q.dtype, device=DEV)
    s.append(q)
    out = torch.empty_like(q)
    for window in (0, 5):
        s.attn(q, out, window)
        s.check_attn(q, out, window)
    assert D.dflash_status_get() == 0


# ---------------------------------------------------------------------------
# append
# ---------------------------------------------------------------------------

@pytest.mark.parametrize("kv", ["bf16", "f32"])
@pytest.mark.parametrize("rows", [[9, 60], [900, 700]])
@pytest.mark.parametrize("norm", [False, True])
def test_append_without_rotation_keeps_infinities_apart(D, kv, rows, norm):
    """No rotation: an element that is not finite does not reach its partner d_h / 2 away. Without
    a norm either the rows go through as they are."""
    s = Step(D, kv, (64, 8, 128), [5, 100], rows, paged=kv != "f32", seed=75)
    s.map()
    for x in (s.q, s.k):
        x[3, 7], x[5, 64 + 9], x[6, 128 + 1] = float("inf"), -float("inf"), float("nan")
        x[8] *= -0.0
    q_out = torch.empty((s.M, s.n_h * 128), dtype=s.q.dtype, device=DEV)
    gq, gk = (s.gq, s.gk) if norm else (None, None)
    D.dflash_chunk_append(s.dims, s.cache, 0, s.plan, s.q, s.k, s.v, gq, gk, None, 0, q_out)
    assert D.dflash_status_get() == 0
    k_out = torch.cat([s.cache.rows("k", 0, b, s.ctx[b], s.ctx[b] + rows[b]) for b in range(2)], 1)
    for x, got, gamma, n in ((s.q, q_out.view(s.M, -1, 128), gq, s.n_h), (s.k, k_out.permute(1, 0, 2), gk, s.n_kv)):
        x = x.reshape(s.M, n, 128)
        if not norm:
            same = (got == x) | (torch.isnan(got) & torch.isnan(x))
            assert same.all() and torch.equal(torch.signbit(got[8]), torch.signbit(x[8]))
            continue
        with np.errstate(invalid="ignore"):
            y, mag = R.norm_rope(np64(x), np64(gamma), 0, rope=False)
        g = np64(got)
        assert (np.isnan(g) == np.isnan(y)).all()
        fin = np.isfinite(y)
        assert (np.abs(g - y)[fin] <= R.append_bound(y, mag, 128, "f32" if kv == "f32" else "bf16")[fin]).all()


@pytest.mark.parametrize("norm", [False, True])
@pytest.mark.parametrize("rows", [[9, 60], [900, 700]])
def test_append_fp8_without_rotation(D, norm, rows):
    """E4M3 codes of rows that are not rotated; an infinity saturates, its partner is untouched."""
    s = Step(D, "fp8", (64, 8, 128), [5, 100], rows, seed=81)
    s.map()
    s.v[3, 7], s.v[4, 70] = float("inf"), -float("inf")
    if not norm:
        s.k[3, 7], s.k[4, 70] = float("inf"), -float("inf")
    q_out = torch.empty((s.M, s.n_h * 128), dtype=s.q.dtype, device=DEV)
    gq, gk = (s.gq, s.gk) if norm else (None, None)
    D.dflash_chunk_append(s.dims, s.cache, 0, s.plan, s.q, s.k, s.v, gq, gk, None, 0, q_out)
    assert D.dflash_status_get() == 0
    for w, x, gamma in (("k", s.k, gk), ("v", s.v, None)):
        got = np64(torch.cat([s.cache.rows(w, 0, b, s.ctx[b], s.ctx[b] + rows[b], codes=True) for b in range(2)], 1)
                   .permute(1, 0, 2))
        y, mag = R.norm_rope(np64(x).reshape(s.M, 8, 128), None if gamma is None else np64(gamma), 0, rope=False)
        sc = s.scales[0]["kv".index(w)]
        y, mag = np.clip(y / sc, -448, 448), np.clip(mag / sc, 0, 448)
        assert (np.abs(got - y) <= R.append_bound(y, mag, 128, "e4m3")).all(), w
    y, mag = R.norm_rope(np64(s.q).reshape(s.M, 64, 128), None if gq is None else np64(gq), 0, rope=False)
    assert (np.abs(np64(q_out).reshape(s.M, 64, 128) - y) <= R.append_bound(y, mag, 128, "bf16")).all()


LARGE = [("bf16", (32, 8), True, True), ("bf16", (5, 1), False, False), ("bf16", (14, 2), True, True),
         ("bf16", (64, 4), True, False), ("bf16", (128, 1), False, True), ("fp8", (32, 8), True, True),
         ("fp8", (5, 1), True, False), ("fp8", (64, 4), False, True), ("fp8", (128, 1), True, True)]


@pytest.mark.parametrize("kv,heads,paged,fused", LARGE)
@pytest.mark.parametrize("mode", ["apart", "in place", "no queries"])
def test_append_of_a_large_step(D, kv, heads, paged, fused, mode):
    """Steps of more than 768 heads per SM (150,000 of up to 160 SMs): a warp takes several heads of
    a row, across the ends of Q, K and V, with an odd number of heads and short last units too."""
    n_h, n_kv = heads
    if mode == "no queries":
        n_h = n_kv
    total = (0 if mode == "no queries" else n_h) + 2 * n_kv
    M = -(-150_000 // total)
    rows = [M // 2 - 3, 1, 0, M - M // 2 + 2]
    if mode == "in place":
        fused = False
    s = Step(D, kv, (n_h, n_kv, 128), [0, 130, 9, 77], rows, paged, layers=2, layer=1, pad=5, seed=76, fused=fused)
    s.map()
    q, q_out = s.q, torch.full((s.M, n_h * 128), 7.0, dtype=s.q.dtype, device=DEV)
    if mode == "no queries":
        q = q_out = None
    elif mode == "in place":
        q = q_out = s.q.clone()
    D.dflash_chunk_append(s.dims, s.cache, 1, s.plan, q, s.k, s.v, s.gq, s.gk, s.table, s.cap, q_out)
    assert D.dflash_status_get() == 0
    assert s.cache.lens.tolist() == [s.ctx, [c + n for c, n in zip(s.ctx, rows)]]
    pos = s.plan.positions.tolist()
    rng = np.random.Generator(np.random.PCG64(76))
    cached = [[np64(s.cache.rows(w, 1, b, 0, s.ctx[b] + rows[b], codes=True)) for w in "kv"] for b in range(s.B)]
    for b in range(s.B):
        lo, hi = int(s.cu[b]), int(s.cu[b + 1])
        # V goes through unchanged: all rows; Q and K: a sample of rows, the first and the last
        for r in sorted({lo, hi - 1, *rng.integers(lo, max(lo + 1, hi), size=300).tolist()}) if hi > lo else []:
            for name, x, gamma, n in (("q", q, s.gq, n_h), ("k", s.k, s.gk, n_kv), ("v", s.v, None, n_kv)):
                if x is None:
                    continue
                src = s.q if name == "q" else x
                y, mag = R.norm_rope(np64(src[r]).reshape(n, 128), None if gamma is None else np64(gamma),
                                     pos[r], rope=name != "v")
                out = "bf16"
                if name == "q":
                    got = np64(q_out[r]).reshape(n, 128)
                else:
                    got = cached[b]["kv".index(name)][:, pos[r]]
                    if kv == "fp8":
                        sc, out = s.scales[1]["kv".index(name)], "e4m3"
                        y, mag = y / sc, mag / sc
                assert (np.abs(got - y) <= R.append_bound(y, mag, 128, out)).all(), (b, r, name)
    if mode == "apart":
        assert (q_out[int(s.cu[-1]):] == 7.0).all()
    if kv == "bf16":
        for b in range(s.B):
            want = s.v[int(s.cu[b]):int(s.cu[b + 1])].reshape(-1, n_kv, 128).permute(1, 0, 2)
            assert torch.equal(s.cache.rows("v", 1, b, s.ctx[b], s.ctx[b] + rows[b]), want)


@pytest.mark.parametrize("kv", ["bf16", "fp8", "f32"])
def test_padding_rows_are_readable_and_never_used(D, kv):
    """Rows behind the last sequence belong to the arrays of a call; what they hold changes nothing."""
    outs = []
    for fill in (0.0, float("nan"), float("inf")):
        s = Step(D, kv, (8, 2, 128), [200, 3], [40, 70], paged=kv != "f32", pad=40, seed=77, fused=False)
        s.map()
        e = int(s.cu[-1])
        for x in (s.q, s.k, s.v):
            x[e:] = fill
        q = torch.zeros_like(s.q)
        s.append(q)
        q[e:] = fill
        out = torch.full_like(q, 5.0)
        s.attn(q, out, 100)
        assert (out[e:] == 5.0).all()
        outs.append((q[:e].clone(), out[:e], s.cache.k.view(torch.uint8), s.cache.v.view(torch.uint8)))
    for o in outs[1:]:
        for a, b in zip(outs[0], o):
            assert torch.equal(a, b)
    with pytest.raises(ValueError):
        D.dflash_chunk_attn(s.dims, s.cache, 0, s.plan, q[:e], 0, 0.0, out, s.ws)
    with pytest.raises(ValueError):
        D.dflash_chunk_append(s.dims, s.cache, 0, s.plan, s.q, s.k[:e], s.v, s.gq, s.gk, s.table, s.cap, q)
    assert D.dflash_status_get() == 0


# ---------------------------------------------------------------------------
# map
# ---------------------------------------------------------------------------

@pytest.mark.parametrize("rows", [1, 2500, 4500, 5500, 7000, 8192, 8193, 70_000])
def test_map_in_place_of_any_size(D, rows):
    """Outputs in place of the inputs (a PagePool's default): one to eight CTAs wait for one
    another, and more rows than they have threads."""
    rng = np.random.Generator(np.random.PCG64(rows))
    B = 1 if rows == 1 else 256
    lens = rng.integers(0, 2000, size=B)
    n = rng.multinomial(rows - 1, [1 / B] * B) if B > 1 else np.array([rows])
    args = _map_case(D, lens, n, 2560, rng.integers(0, 2, size=B), 6 * B, rows - int(n.sum()), rows, 3, True)
    D.dflash_chunk_map(args[0], 0, args[1], args[2])
    _check_map(*args)
    assert D.dflash_status_get() == 0


# ---------------------------------------------------------------------------
# rounds
# ---------------------------------------------------------------------------

@pytest.mark.parametrize("graph", [False, True])
@pytest.mark.parametrize("kv", ["bf16", "fp8"])
def test_rounds_leave_the_accepted_rows_in_the_cache(D, kv, graph):
    """Map, append, attention, acceptance and crop over many rounds, call by call and as a graph.
    After each round the cache holds the rows of the accepted tokens, made in float64 from
    their projections at their positions, and nothing that was rejected; the attention is
    compared with one over those rows."""
    B, bs, L, n_h, n_kv, d, cap = 5, 6, 2, 8, 2, 128, 384
    g = torch.Generator().manual_seed(2)
    dt = torch.bfloat16
    fp8 = kv == "fp8"
    scales = [[0.5, 0.25], [0.125, 0.0625]]
    dims = D.make_dims(n_h * d, n_h, n_kv, d, 1, bs, 1e-6, dt)
    n_pages = B * (cap // 128)
    cache = D.KVCache(L, B, n_kv, cap, d, dt, DEV, page_table=torch.full((B, cap // 128), -1), n_pages=n_pages,
                      kv="fp8" if fp8 else "bf16", kv_scales=scales if fp8 else None)
    pool = D.PagePool(i32([0] * B), i32(np.random.default_rng(4).permutation(n_pages)), i32([0]))
    M = B * bs
    plan = D.ChunkPlan(i32(np.arange(B + 1) * bs), M)
    table = torch.empty((cap, d // 2, 2), dtype=torch.float32, device=DEV)
    D.dflash_rope_table_build(1e6, d, cap, table)
    gq, gk = ((1 + 0.2 * torch.randn(d, generator=g)).to(DEV, dt) for _ in range(2))
    ws = torch.empty(D.dflash_chunk_workspace_bytes(dims), dtype=torch.uint8, device=DEV)
    x = [torch.zeros((M, (n_h + 2 * n_kv) * d), dtype=dt, device=DEV) for _ in range(L)]
    q = [torch.empty((M, n_h * d), dtype=dt, device=DEV) for _ in range(L)]
    out = [torch.empty_like(q[0]) for _ in range(L)]
    ids, post = (torch.zeros((B, bs), dtype=torch.int32, device=DEV) for _ in range(2))
    start = cache.lens[0].clone()
    acc, nxt, anchor = (torch.zeros(B, dtype=torch.int32, device=DEV) for _ in range(3))
    ncu = torch.zeros(B + 1, dtype=torch.int32, device=DEV)

    def step():
        start.copy_(cache.lens[0])
        D.dflash_chunk_map(cache, 0, plan, pool)
        for l in range(L):
            a, b, c = x[l].split((n_h * d, n_kv * d, n_kv * d), 1)
            D.dflash_chunk_append(dims, cache, l, plan, a, b, c, gq, gk, table, cap, q[l])
            D.dflash_chunk_attn(dims, cache, l, plan, q[l], 0 if l == 0 else 50, 0.0, out[l], ws)
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
    gk64 = np64(gk)
    # accepted rows in float64, [layer][sequence] -> list of (K, bound, V) of one row [n_kv][d]
    held = [[[] for _ in range(B)] for _ in range(L)]

    def block(l, b, start_pos):
        """K, its bound, and V of the block's rows, in the cache's units (E4M3: codes' values)."""
        rows = np64(x[l][b * bs:(b + 1) * bs])[:, n_h * d:].reshape(bs, 2, n_kv, d)
        res = []
        for i in range(bs):
            y, mag = R.norm_rope(rows[i, 0], gk64, start_pos + i)
            v = rows[i, 1]
            if fp8:
                y, mag, v = y / scales[l][0], mag / scales[l][0], v / scales[l][1]
            vb = R.append_bound(v, np.abs(v), d, "e4m3") if fp8 else 0.0 * v
            res.append((y, R.append_bound(y, mag, d, "e4m3" if fp8 else "bf16"), v, vb))
        return res

    for rnd in range(40):
        for l in range(L):
            x[l].copy_(torch.randn(x[l].shape, generator=g))
        ids.copy_(torch.randint(0, 3, (B, bs), generator=g))
        post.copy_(torch.randint(0, 3, (B, bs), generator=g))
        gr.replay() if graph else step()
        torch.cuda.synchronize()
        a = acc.tolist()
        check = rnd % 13 == 12 or rnd == 0
        for l in range(L):
            for b in range(B):
                n0 = len(held[l][b])
                rows = block(l, b, n0)
                # what the attention saw: all rows of the block, the cache's older rows
                now = held[l][b] + rows
                K, V = (np64(cache.rows(w, l, b, 0, n0 + bs, codes=True)).transpose(1, 0, 2) for w in "kv")
                assert (np.abs(K - np.stack([r[0] for r in now])) <= np.stack([r[1] for r in now])).all(), (rnd, l, b)
                assert (np.abs(V - np.stack([r[2] for r in now])) <= np.stack([r[3] for r in now])).all(), (rnd, l, b)
                held[l][b] += rows[:a[b] + 1]
                if not check:
                    continue
                # (K and V as stored: they have just been held to the rows)
                sk, sv = scales[l] if fp8 else (1.0, 1.0)
                qr = np64(q[l][b * bs:(b + 1) * bs]).reshape(bs, n_h, d)
                ref, mag, big, keys = R.attention(qr, K * sk, V * sv, n0 + bs, bs, n_h // n_kv, 0 if l == 0 else 50,
                                                  d ** -0.5)
                got = np64(out[l][b * bs:(b + 1) * bs]).reshape(bs, n_h, d)
                assert (np.abs(got - ref) <= R.attention_bound(ref, mag, big, keys, d, "bf16")).all(), (rnd, l, b)
        assert cache.lens.tolist() == [[len(held[0][b]) for b in range(B)]] * L
    assert D.dflash_status_get() == 0
