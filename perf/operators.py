"""The chunk step of a paged KV cache: mapping, append and causal attention, as measured workloads.

A serving round that runs a target model over new tokens (a prompt's chunk, the rows of a
speculative block to verify, a single token per sequence) makes three calls per step:

  map     once: from every sequence's length and its number of new rows, the pages it still
          needs (taken from a free list), each new row's cache slot and position, and the
          lengths after the step (dflash_chunk_map)
  append  per layer: per-head RMSNorm of Q and K, RoPE at the rows' positions, K and V stored
          at their slots in the cache's element type (dflash_chunk_append)
  attn    per layer: causal grouped-query attention of the new rows over everything their
          sequences hold, with an optional sliding window (dflash_chunk_attn)

Where ``own`` is false the operators run in their plain form, elementary torch operations in
32 bits. Where it is true they are the library's calls.
"""

import math
import random

import torch

own = False

PAGE = 128      # rows of a cache page
EPS = 1e-6      # RMSNorm epsilon
THETA = 1e6     # RoPE base


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------

def _map(name, batch, rows, ctx, singles=0, over=0, lens=1):
    return {"name": name, "op": "map", "batch": batch, "rows_lo": rows[0], "rows_hi": rows[1],
            "ctx_lo": ctx[0], "ctx_hi": ctx[1], "singles": singles, "over": over, "lens": lens}


def _append(name, kv, batch, rows, ctx, heads=(32, 8, 128), singles=0, lens=1):
    return {"name": name, "op": "append", "kv": kv, "batch": batch, "rows_lo": rows[0],
            "rows_hi": rows[1], "ctx_lo": ctx[0], "ctx_hi": ctx[1], "singles": singles,
            "n_h": heads[0], "n_kv": heads[1], "d_h": heads[2], "lens": lens}


def _attn(name, kv, batch, rows, ctx, heads=(32, 8, 128), singles=0, window=0, lens=1):
    return dict(_append(name, kv, batch, rows, ctx, heads, singles, lens), op="attn", window=window)


def listed():
    return [
        # a verification round: 32 sequences, a block of 16 rows each
        _map("map_verify_b32", 32, (16, 16), (256, 4096)),
        # admission of many ragged prompts next to running sequences, two of which do not fit
        _map("map_admit_b256", 256, (1, 700), (0, 2048), singles=64, over=2),
        # the verification round's rows in one layer
        _append("append_verify_b32", "bf16", 32, (16, 16), (256, 4096)),
        # a step of ragged prompt chunks
        _append("append_prompt_b9", "bf16", 9, (200, 1900), (0, 3000)),
        # the same on the one-byte cache
        _append("append_prompt_fp8_b5", "fp8", 5, (333, 1400), (0, 2000)),
        # one sequence, one token: nothing but latency
        _attn("token_b1", "bf16", 1, (1, 1), (1023, 1023)),
        # a decoding batch on the one-byte cache
        _attn("token_fp8_b64", "fp8", 64, (1, 1), (1024, 8192)),
        # verification of 16-row blocks at the serving lengths
        _attn("verify_b32", "bf16", 32, (16, 16), (256, 4096)),
        # few sequences with long caches: the long axis has to be shared out
        _attn("long_ctx_b4", "bf16", 4, (16, 16), (32768, 32768)),
        # prompt chunks next to decoding sequences, in a layer with a sliding window
        _attn("mixed_window_b16", "bf16", 16, (300, 700), (1000, 5000), singles=10, window=2048),
        # one long prompt from its start
        _attn("prompt_8k", "bf16", 1, (8192, 8192), (0, 0)),
        # float32 layer of the small walkthrough model: eight heads of 64
        _attn("prompt_f32_b6", "f32", 6, (65, 600), (0, 900), heads=(8, 8, 64)),
    ]


def _log(rng, lo, hi):
    """A whole number in [lo, hi], spread over its logarithm."""
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def draw(rng):
    op = rng.choice(("map", "append", "append", "attn", "attn", "attn"))
    lens = rng.randrange(1 << 20)
    if op == "map":
        batch = _log(rng, 1, 256)
        hi = _log(rng, 1, max(1, min(4000, 90000 // batch)))
        ctx = _log(rng, 1, 8192)
        c = _map("", batch, (rng.randint(1, hi), hi), (rng.randint(0, ctx), ctx),
                 singles=rng.randint(0, batch - 1), over=rng.randint(0, min(3, batch - 1)), lens=lens)
        del c["name"]
        return c
    kv = rng.choice(("bf16", "bf16", "bf16", "fp8", "fp8", "f32"))
    if kv == "f32":
        heads = rng.choice(((8, 8, 64), (4, 2, 80), (8, 1, 128), (3, 3, 256), (6, 2, 32)))
    else:
        heads = rng.choice(((32, 8, 128), (32, 8, 128), (16, 16, 128), (20, 4, 128), (14, 2, 128),
                            (8, 1, 128), (64, 4, 128)))
    n_h, n_kv, d_h = heads
    batch = _log(rng, 1, 64)
    if op == "append":
        hi = _log(rng, 1, max(1, 60000000 // ((n_h + 2 * n_kv) * d_h * batch)))
        ctx = _log(rng, 1, max(1, 60000 // batch))
        c = _append("", kv, batch, (rng.randint(1, hi), hi), (rng.randint(0, ctx), ctx), heads,
                    singles=rng.randint(0, batch - 1), lens=lens)
    else:
        # bounds: the plain form's padded scores, the cache rows read, the query rows
        per = (2.0e9 if kv != "f32" else 2.5e8) / (batch * n_h)
        ctx = _log(rng, 1, max(1, min(32768, 150000000 // (batch * n_kv * d_h))))
        top = min((math.sqrt(ctx * ctx + 4 * per) - ctx) / 2, 6.0e7 / (batch * n_h * d_h))
        hi = _log(rng, 1, max(1, int(top)))
        c = _attn("", kv, batch, (rng.randint(1, hi), hi), (rng.randint(0, ctx), ctx), heads,
                  singles=rng.choice((0, rng.randint(0, batch - 1))),
                  window=rng.choice((0, 0, _log(rng, 1, 4096))), lens=lens)
    del c["name"]
    return c


def _lengths(case):
    """New rows and cached rows of every sequence: the same for every seed of a case."""
    r = random.Random(case["lens"])
    B = case["batch"]
    rows = [1 if b < case["singles"] else r.randint(case["rows_lo"], case["rows_hi"]) for b in range(B)]
    ctx = [r.randint(case["ctx_lo"], case["ctx_hi"]) for _ in range(B)]
    r.shuffle(rows)
    return rows, ctx


def _pages_per_seq(case):
    rows, ctx = _lengths(case)
    return max(-(-(n + c) // PAGE) for n, c in zip(rows, ctx))


def _scales(kv):
    return (0.03125, 0.0078125) if kv == "fp8" else (1.0, 1.0)


# ---------------------------------------------------------------------------
# what a program has in hand before the call
# ---------------------------------------------------------------------------

def _i32(v, dev):
    return torch.tensor(v, dtype=torch.int32, device=dev)


def _rope_table(n, d_h, dev):
    """float32 [n][d_h / 2][2]: cosine and sine of p * THETA^(-2 i / d_h)."""
    i = torch.arange(d_h // 2, dtype=torch.float64, device=dev)
    a = torch.arange(n, dtype=torch.float64, device=dev)[:, None] * THETA ** (-2.0 * i / d_h)
    return torch.stack((a.cos(), a.sin()), -1).float()


def prepare(case, seed):
    dev = "cuda"
    g = torch.Generator(device=dev).manual_seed(int(seed))
    rows, ctx = _lengths(case)
    B = len(rows)
    cu = [0]
    for n in rows:
        cu.append(cu[-1] + n)
    s = {"op": case["op"], "batch": B, "rows_max": max(rows), "kv_max": max(n + c for n, c in zip(rows, ctx)),
         "cu_rows": _i32(cu, dev), "lens": _i32(ctx, dev), "M": cu[-1], "pps": _pages_per_seq(case)}
    pps = s["pps"]
    if case["op"] == "map":
        # pages held: those of the cached rows, sometimes one more (after a crop); the free
        # list holds what the step needs, but for the last `over` sequences' rows that grow
        # past the capacity
        r = random.Random(case["lens"] + 1)
        held = [min(pps, -(-c // PAGE) + r.randint(0, 1)) for c in ctx]
        lens = list(ctx)
        for b in r.sample(range(B), case["over"]):
            lens[b] = pps * PAGE - rows[b] + 1 + r.randint(0, PAGE)
            lens[b] = min(lens[b], pps * PAGE)
            held[b] = -(-lens[b] // PAGE)
        n_pages = B * pps + 7
        perm = torch.randperm(n_pages, generator=g, device=dev).int()
        n_held = sum(held)
        table = torch.zeros((B, pps), dtype=torch.int32, device=dev)
        h = _i32(held, dev)
        mine = torch.arange(pps, device=dev)[None] < h[:, None]
        table[mine] = perm[:n_held]
        s.update(lens=_i32(lens, dev), held=h, held_out=torch.zeros_like(h), table=table,
                 free=perm[n_held:].contiguous(), taken=_i32([3], dev), taken_out=_i32([0], dev),
                 n_pages=n_pages, rows=cu[-1] + 5)
        # five rows of padding behind the last sequence
        M = s["rows"]
        s.update(slots=_i32([0] * M, dev), positions=_i32([0] * M, dev), kv_lens=_i32([0] * B, dev))
        if own:
            from speculative_decoding_draft_dflash_gb300 import dflash
            s["cache"] = dflash.KVCache(1, B, 1, pps * PAGE, 128, "bf16", dev, page_table=table,
                                        n_pages=n_pages)
            s["table"] = s["cache"].block_table
            s["cache"].lens.copy_(s["lens"][None])
            s["plan"] = dflash.ChunkPlan(s["cu_rows"], M, s["kv_lens"], s["slots"], s["positions"])
            s["pool"] = dflash.PagePool(s["held"], s["free"], s["taken"], s["held_out"], s["taken_out"])
        return s

    kv, n_h, n_kv, d_h = case["kv"], case["n_h"], case["n_kv"], case["d_h"]
    dt = torch.float32 if kv == "f32" else torch.bfloat16
    paged = kv != "f32"
    total = [n + c for n, c in zip(rows, ctx)]
    cap = pps * PAGE
    M = cu[-1]
    s.update(kv=kv, n_h=n_h, n_kv=n_kv, d_h=d_h, scales=_scales(kv), paged=paged, cap=cap, rows=M,
             kv_lens=_i32(total, dev), window=case.get("window", 0))
    # pages of every sequence: a seeded permutation of the pool
    n_pages = sum(-(-t // PAGE) for t in total) + 3
    table = torch.zeros((B, pps), dtype=torch.int32, device=dev)
    used = torch.arange(pps, device=dev)[None] < ((s["kv_lens"][:, None] + PAGE - 1) // PAGE)
    perm = torch.randperm(n_pages, generator=g, device=dev).int()
    table[used] = perm[:n_pages - 3]
    s["table"] = table
    shape = (n_pages, n_kv, PAGE, d_h) if paged else (B, n_kv, cap, d_h)
    K = torch.randn(shape, generator=g, device=dev, dtype=torch.float32)
    V = torch.randn(shape, generator=g, device=dev, dtype=torch.float32)
    if kv == "fp8":
        K = (K / s["scales"][0]).clamp_(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
        V = (V * 0.25 / s["scales"][1]).clamp_(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
    else:
        K, V = K.to(dt), V.to(dt)
    s.update(k=K, v=V)
    # rows -> slots and positions, as the map operator leaves them
    cu64 = s["cu_rows"].long()
    r = torch.arange(M, device=dev)
    b = torch.searchsorted(cu64, r, right=True) - 1
    pos = s["lens"].long()[b] + r - cu64[b]
    slot = table.long()[b, pos // PAGE] * PAGE + pos % PAGE if paged else b * cap + pos
    s.update(slots=slot.int(), positions=pos.int())
    if case["op"] == "append":
        W = (n_h + 2 * n_kv) * d_h     # the rows of a fused Q/K/V projection
        qkv = torch.randn((M, W), generator=g, device=dev, dtype=torch.float32).to(dt)
        s.update(q=qkv[:, :n_h * d_h], k_new=qkv[:, n_h * d_h:(n_h + n_kv) * d_h], v_new=qkv[:, (n_h + n_kv) * d_h:],
                 gamma_q=(1 + 0.1 * torch.randn(d_h, generator=g, device=dev)).to(dt),
                 gamma_k=(1 + 0.1 * torch.randn(d_h, generator=g, device=dev)).to(dt),
                 rope=_rope_table(s["kv_max"], d_h, dev), q_out=torch.zeros((M, n_h * d_h), dtype=dt, device=dev))
    else:
        s["q"] = torch.randn((M, n_h * d_h), generator=g, device=dev, dtype=torch.float32).to(dt)
        s["out"] = torch.zeros((M, n_h * d_h), dtype=dt, device=dev)
    if own:
        from speculative_decoding_draft_dflash_gb300 import dflash
        s["dims"] = dflash.make_dims(n_h * d_h, n_h, n_kv, d_h, 1, 1, EPS, dt)
        s["cache"] = dflash.KVCache(1, B, n_kv, cap, d_h, dt, dev, page_table=table if paged else None,
                                    n_pages=n_pages if paged else None, kv="fp8" if kv == "fp8" else "bf16",
                                    kv_scales=[s["scales"]])
        s["cache"].k[0].copy_(K)
        s["cache"].v[0].copy_(V)
        s["cache"].lens.copy_(s["lens"][None])
        s["k"], s["v"] = s["cache"].k[0], s["cache"].v[0]
        s["plan"] = dflash.ChunkPlan(s["cu_rows"], M, s["kv_lens"], s["slots"], s["positions"])
        s["ws"] = torch.empty(dflash.dflash_chunk_workspace_bytes(s["dims"]), dtype=torch.uint8, device=dev)
    return s


# ---------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------

def run(s):
    if own:
        return {"map": _own_map, "append": _own_append, "attn": _own_attn}[s["op"]](s)
    return {"map": _plain_map, "append": _plain_append, "attn": _plain_attn}[s["op"]](s)


def _map_out(s):
    return {"slots": s["slots"], "positions": s["positions"], "kv_lens": s["kv_lens"], "table": s["table"],
            "held": s["held_out"], "taken": s["taken_out"]}


def _append_out(s):
    e = (lambda t: t.view(torch.float8_e4m3fn)) if s["kv"] == "fp8" else (lambda t: t)
    return {"q": s["q_out"], "k": e(s["k"]), "v": e(s["v"])}


def _own_map(s):
    from speculative_decoding_draft_dflash_gb300 import dflash
    dflash.dflash_chunk_map(s["cache"], 0, s["plan"], s["pool"])
    return _map_out(s)


def _own_append(s):
    from speculative_decoding_draft_dflash_gb300 import dflash
    dflash.dflash_chunk_append(s["dims"], s["cache"], 0, s["plan"], s["q"], s["k_new"], s["v_new"], s["gamma_q"],
                               s["gamma_k"], s["rope"], s["kv_max"], s["q_out"])
    return _append_out(s)


def _own_attn(s):
    from speculative_decoding_draft_dflash_gb300 import dflash
    dflash.dflash_chunk_attn(s["dims"], s["cache"], 0, s["plan"], s["q"], s["window"], 0.0, s["out"], s["ws"])
    return s["out"]


def _plain_map(s):
    cu, lens, held, table = s["cu_rows"].long(), s["lens"].long(), s["held"].long(), s["table"]
    cap = s["pps"] * PAGE
    total = lens + cu[1:] - cu[:-1]
    fits = total <= cap
    need = torch.where(fits, ((total + PAGE - 1) // PAGE - held).clamp(min=0), 0)
    end = need.cumsum(0)                       # pages asked for by this sequence and those before it
    first = s["taken"].long()
    ok = fits & ((need == 0) | (end <= s["free"].numel() - first))
    got = torch.where(ok, need, 0)
    # page p of sequence b, for held <= p < held + got, is the free list's entry of its rank
    p = torch.arange(s["pps"], device=table.device)[None]
    new = (p >= held[:, None]) & (p < (held + got)[:, None])
    at = (first + (end - need)[:, None] + p - held[:, None]).clamp(0, s["free"].numel() - 1)
    table.copy_(torch.where(new, s["free"][at], table))
    r = torch.arange(s["rows"], device=table.device)
    b = (torch.searchsorted(cu, r, right=True) - 1).clamp(max=s["batch"] - 1)
    pos = lens[b] + r - cu[b]
    live = (r < cu[-1]) & ok[b]
    page = table.long()[b, torch.where(live, pos // PAGE, 0)]
    return {"slots": torch.where(live, page * PAGE + pos % PAGE, -1).int(), "positions": torch.where(live, pos, -1).int(),
            "kv_lens": torch.where(ok, total, 0).int(), "table": table, "held": (held + got).int(),
            "taken": (first + got.sum()).int()}


def _plain_rows(x, gamma, cs):
    """RMSNorm over the head dimension, then the rotation of (i, i + d_h / 2) pairs."""
    x = x.float()
    x = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS) * gamma.float()
    a, b = x.chunk(2, -1)
    c, d = cs[:, None, :, 0], cs[:, None, :, 1]
    return torch.cat((a * c - b * d, b * c + a * d), -1)


def _plain_append(s):
    M, d_h = s["M"], s["d_h"]
    cs = s["rope"][s["positions"].long()]
    q = _plain_rows(s["q"].reshape(M, s["n_h"], d_h), s["gamma_q"], cs)
    k = _plain_rows(s["k_new"].reshape(M, s["n_kv"], d_h), s["gamma_k"], cs)
    v = s["v_new"].reshape(M, s["n_kv"], d_h).float()
    s["q_out"].copy_(q.reshape(M, -1))
    slot = s["slots"].long()
    unit = PAGE if s["paged"] else s["cap"]
    for name, x, scale in (("k", k, s["scales"][0]), ("v", v, s["scales"][1])):
        if s["kv"] == "fp8":
            x = (x / scale).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
        s[name][slot // unit, :, slot % unit] = x.to(s[name].dtype)
    return _append_out(s)


def _plain_attn(s):
    B, n_h, n_kv, d_h, G = s["batch"], s["n_h"], s["n_kv"], s["d_h"], s["n_h"] // s["n_kv"]
    dev = s["q"].device
    cu, kv = s["cu_rows"].long(), s["kv_lens"].long()
    n = cu[1:] - cu[:-1]
    # queries, padded: [B][n_kv][rows * G][d_h], row i of sequence b at position kv - n + i
    i = torch.arange(s["rows_max"], device=dev)
    at = (cu[:-1, None] + i).clamp(max=s["M"] - 1)
    q = s["q"].reshape(s["M"], n_kv, G, d_h)[at].float().permute(0, 2, 1, 3, 4).reshape(B, n_kv, -1, d_h)
    pos = (kv - n)[:, None] + i
    # keys and values, padded: [B][n_kv][keys][d_h]
    j = torch.arange(s["kv_max"], device=dev)
    value = (lambda t: t.view(torch.float8_e4m3fn)) if s["kv"] == "fp8" else (lambda t: t)

    def rows(t):
        if s["paged"]:
            page = s["table"].long()[:, j // PAGE]
            return value(t[page, :, (j % PAGE)[None]]).float().permute(0, 2, 1, 3)
        return t[:, :, :s["kv_max"]].float()

    x = q @ rows(s["k"]).transpose(-1, -2)
    x *= d_h ** -0.5 * s["scales"][0]
    seen = (j <= pos[..., None]) & (j < kv[:, None, None])
    if s["window"] > 0:
        seen &= pos[..., None] - j < s["window"]
    hidden = ~seen[:, None, :, None, :].expand(B, 1, s["rows_max"], G, s["kv_max"]).reshape(B, 1, -1, s["kv_max"])
    x.masked_fill_(hidden, float("-inf"))
    x -= x.amax(-1, keepdim=True).clamp(min=-3e38)
    x.exp_()
    total = x.sum(-1, keepdim=True)
    o = (x @ rows(s["v"])) * (s["scales"][1] / total.clamp(min=1e-37))
    o = o.reshape(B, n_kv, s["rows_max"], G, d_h).permute(0, 2, 1, 3, 4)
    return o[i[None] < n[:, None]].reshape(s["M"], n_h * d_h).to(s["q"].dtype)


# ---------------------------------------------------------------------------
# what a pass cannot do without
# ---------------------------------------------------------------------------

def work(case):
    rows, ctx = _lengths(case)
    B, M = len(rows), sum(rows)
    if case["op"] == "map":
        new = sum(-(-(n + c) // PAGE) - -(-c // PAGE) for n, c in zip(rows, ctx))
        return {"bytes": 4 * (2 * M + 5 * B + 2 * new), "flops": 2 * M}
    n_h, n_kv, d_h = case["n_h"], case["n_kv"], case["d_h"]
    e = 4 if case["kv"] == "f32" else 2
    ce = 1 if case["kv"] == "fp8" else e
    if case["op"] == "append":
        per = (2 * n_h + 2 * n_kv) * d_h * e + 2 * n_kv * d_h * ce + 8
        positions = len({c + i for n, c in zip(rows, ctx) for i in range(n)})
        return {"bytes": M * per + positions * d_h * 4, "flops": M * (n_h + n_kv) * d_h * 7}
    w = case["window"]
    pairs = keys = 0
    for n, c in zip(rows, ctx):
        # row i (0-based) sees min(c + i + 1, window) keys
        if w:
            short = max(0, min(n, w - c))              # rows whose window is not full yet
            pairs += short * c + short * (short + 1) // 2 + (n - short) * w
            keys += min(c + n, w + n - 1)
        else:
            pairs += n * c + n * (n + 1) // 2
            keys += c + n
    return {"bytes": 2 * M * n_h * d_h * e + 2 * keys * n_kv * d_h * ce, "flops": 4 * pairs * n_h * d_h}


# ---------------------------------------------------------------------------
# the definition, in 64 bits
# ---------------------------------------------------------------------------

def exact(case, seed):
    if case["op"] == "map":
        return None                            # whole numbers only
    s = prepare(case, seed)
    n_h, n_kv, d_h, G = s["n_h"], s["n_kv"], s["d_h"], s["n_h"] // s["n_kv"]
    sk, sv = s["scales"]
    cu = s["cu_rows"].tolist()
    f64 = torch.float64
    if case["op"] == "append":
        pos = s["positions"].to(f64)
        i = torch.arange(d_h // 2, dtype=f64, device=pos.device)
        ang = pos[:, None] * (THETA ** (-2.0 * i / d_h))
        rot = torch.polar(torch.ones_like(ang), ang)[:, None]

        def head(x, gamma, heads):
            x = x.to(f64).reshape(-1, heads, d_h)
            x = x / (x.square().sum(-1, keepdim=True) / d_h + EPS).sqrt() * gamma.to(f64)
            z = torch.complex(x[..., :d_h // 2].contiguous(), x[..., d_h // 2:].contiguous()) * rot
            return torch.cat((z.real, z.imag), -1)

        q = head(s["q"], s["gamma_q"], n_h).reshape(-1, n_h * d_h)
        code = (lambda t: t.view(torch.float8_e4m3fn).to(f64)) if s["kv"] == "fp8" else (lambda t: t.to(f64))
        K, V = code(s["k"]), code(s["v"])
        unit = PAGE if s["paged"] else s["cap"]
        top = 448.0 if s["kv"] == "fp8" else float("inf")
        slot = s["slots"].long()
        K[slot // unit, :, slot % unit] = (head(s["k_new"], s["gamma_k"], n_kv) / sk).clamp(-top, top)
        V[slot // unit, :, slot % unit] = (s["v_new"].to(f64).reshape(-1, n_kv, d_h) / sv).clamp(-top, top)
        return {"q": q, "k": K, "v": V}
    if 2 * sum((b - a) * s["kv_max"] for a, b in zip(cu, cu[1:])) * n_h * d_h * 2 > 1.2e13:
        return None                            # too long in 64 bits
    out = torch.zeros((s["M"], n_h, d_h), dtype=f64, device=s["q"].device)
    for b, (lo, hi) in enumerate(zip(cu, cu[1:])):
        L = int(s["kv_lens"][b])
        if hi == lo:
            continue
        t = torch.arange(L, device=out.device)
        p = torch.arange(L - (hi - lo), L, device=out.device)
        keep = t[None] <= p[:, None]
        if s["window"] > 0:
            keep &= t[None] > p[:, None] - s["window"]
        for h in range(n_kv):
            if s["paged"]:
                pg = s["table"][b, t // PAGE].long()
                k, v = s["k"][pg, h, t % PAGE], s["v"][pg, h, t % PAGE]
            else:
                k, v = s["k"][b, h, :L], s["v"][b, h, :L]
            if s["kv"] == "fp8":
                k, v = k.view(torch.float8_e4m3fn), v.view(torch.float8_e4m3fn)
            k, v = k.to(f64) * sk, v.to(f64) * sv
            for g in range(h * G, (h + 1) * G):
                a = s["q"][lo:hi, g * d_h:(g + 1) * d_h].to(f64) @ k.T / d_h ** 0.5
                out[lo:hi, g] = torch.softmax(a.masked_fill(~keep, float("-inf")), -1) @ v
    return out.reshape(s["M"], n_h * d_h)
