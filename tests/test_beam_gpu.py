"""Beam selection against its formula in float64."""
import numpy as np
import pytest
import torch

import tree_ref as T
from test_chunk_gpu import DEV, D, i32  # noqa: F401  (D is the fixture)

pytestmark = pytest.mark.gpu

TORCH = {"f32": torch.float32, "bf16": torch.bfloat16}


def np64(t):
    return t.detach().double().cpu().numpy()


def select(D, logits, scores, k, base=0, ws=None, pad=0):
    batch, beams, vocab = logits.shape
    n = D.dflash_beam_workspace_bytes(batch, beams, vocab, k)
    ws = torch.full((n,), 0xFF, dtype=torch.uint8, device=DEV) if ws is None else ws
    out = [torch.full((batch, k + pad), -9, dtype=t, device=DEV) for t in (torch.int32, torch.int32, torch.float32)]
    D.dflash_beam_select(logits, scores, k, *(o[:, pad:] for o in out), ws, parent_base=base)
    assert all((o[:, :pad] == -9).all() for o in out)
    return [o[:, pad:] for o in out]


def check(D, logits, scores, k, base=0, **kw):
    """All three outputs against float64. Whole numbers are equal: no two scores of these cases are
    nearer than the log-sum's error, but for those that are equal."""
    tok, par, out = select(D, logits, scores, k, base, **kw)
    s = np.zeros(logits.shape[:2]) if scores is None else np64(scores)
    x = np64(logits)
    for b in range(logits.shape[0]):
        t, i, v = T.beam_select(x[b], s[b], k)
        assert tok[b].tolist() == t.tolist(), b
        assert par[b].tolist() == (i + base).tolist(), b
        got = np64(out[b])
        fin = np.isfinite(v)
        assert (np.isneginf(got) == ~fin).all()
        assert (np.abs(got[fin] - v[fin]) <= T.beam_bound(v[fin])).all(), b
    return tok, par, out


def random(dtype, batch, beams, vocab, seed=0, spread=2.0):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn((batch, beams, vocab), generator=g) * spread
    s = -4 * torch.rand((batch, beams), generator=g)
    return x.to(DEV, TORCH[dtype]), s.to(DEV)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("batch,beams,vocab,k", [
    (1, 1, 1, 1), (3, 4, 7, 28), (2, 3, 1000, 17), (2, 8, 32000, 8), (3, 2, 50001, 128), (2, 128, 300, 128), (5, 1, 8193, 1),
    (1, 5, 131072, 33), (300, 2, 2047, 3), (1, 1, 100003, 1), (4, 3, 9, 5), (2, 2, 64, 128)])
def test_select(D, dtype, batch, beams, vocab, k):
    x, s = random(dtype, batch, beams, vocab, seed=vocab)
    check(D, x, s, k, base=7)
    if vocab > 9000:                                  # as peaked as a language model's
        x[..., ::997] += 12 * torch.rand_like(x[..., ::997])
        check(D, x, s, k)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("vocab,first,ld", [(50001, 1, 50003), (33000, 3, 33007), (32000, 0, 32000), (700, 5, 705)])
def test_select_strides_and_alignments(D, dtype, vocab, first, ld):
    """Rows inside wider ones, at every alignment; beams before sequences; a row for all beams."""
    x, s = random(dtype, 3, 4, ld, seed=first)
    v = x[:, :, first:first + vocab]
    check(D, v, s, 9)
    check(D, v.transpose(0, 1), s.t().contiguous(), 9)
    check(D, v[:, :1].expand(3, 4, vocab), s, 9, pad=3)       # (and outputs inside wider rows)
    check(D, v[:1].expand(3, 4, vocab), s, 9)
    check(D, v[:, 1:3], None, 5)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("shift", [0, 1])
def test_select_ties_go_to_the_lowest_place(D, dtype, shift):
    """Few distinct values, and beams that are copies of one another at other alignments."""
    g = torch.Generator().manual_seed(4)
    V = 20000 + shift
    row = torch.randint(0, 6, (V,), generator=g).float()
    x = torch.zeros((2, 5, V + 3))
    x[:, :, :V] = row                                 # equal beams
    x[1, 2, :V] = 1.0                                 # a constant row
    x = x.to(DEV, TORCH[dtype])[:, :, :V]
    s = torch.zeros((2, 5), device=DEV)
    check(D, x, s, 100)
    s[0] = torch.tensor([-1.0, -0.5, -0.5, -3, -0.5])
    check(D, x, s, 64)
    const = torch.full((1, 3, 30000), -2.5, dtype=TORCH[dtype], device=DEV)
    check(D, const, None, 128)
    zeros = torch.zeros((1, 1, 9000), dtype=TORCH[dtype], device=DEV)
    zeros[..., ::2] = -0.0                            # minus zero is zero
    tok, _, _ = select(D, zeros, None, 40)
    assert tok[0].tolist() == list(range(40))


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_select_banned_tokens_and_dead_beams(D, dtype):
    inf = float("inf")
    x, s = random(dtype, 9, 3, 12000, seed=2)
    low = torch.finfo(TORCH[dtype]).min
    x[0] = -inf                                       # nothing left: the lowest places, minus infinity
    x[1, :, 5:] = -inf                                # fewer candidates than asked for
    x[2, 0, 77] = float("nan")
    x[2, 1, 11999] = inf
    x[3] = low                                        # masked with the lowest value: uniform
    x[4, :, :11990] = low                             # ten tokens left
    x[5, 0, :9000] = -inf                             # whole tiles banned
    x[5, 1, 3000:] = -inf
    s[6] = torch.tensor([-inf, 1.0, -inf])
    s[7] = torch.tensor([float("nan"), inf, -2.0])
    s[8] = -inf
    x[8, 1, 5] = float("nan")
    for k in (1, 20, 128):
        check(D, x, s, k)
    # NaN behind a tile of banned tokens, and in a row of nothing else
    y, _ = random(dtype, 2, 2, 40000, seed=3)
    y[0, 0, :20000], y[0, 0, 100] = -inf, float("nan")
    y[1, 0] = float("nan")
    check(D, y, None, 12)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("vocab", [20000, 131072])
def test_select_rows_in_ascending_order(D, dtype, vocab):
    """Every logit beats those before it, and the reference of the sum moves again and again."""
    up = torch.arange(vocab, dtype=torch.float32).floor()
    for scale, k in ((1e-3, 50), (0.05, 128), (3.0, 7)):
        x = torch.stack((up * scale, -up * scale, up.flip(0) * scale * 0.5))[None].to(DEV, TORCH[dtype])
        check(D, x, torch.tensor([[0.0, -0.25, -0.5]], device=DEV), k)


def test_select_large_offsets(D):
    """A common offset of a row changes nothing but its logits' own roundings."""
    x, s = random("f32", 2, 3, 30000, seed=9)
    x = (x * 8).round() / 8
    base = select(D, x, s, 30)
    for off in (512.0, -100000.0):
        got = check(D, x + off, s, 30)
        assert all(torch.equal(a, b) for a, b in zip(base, got))


def test_select_repeats_and_runs_side_by_side(D):
    """The same bits again, from a graph, and from two streams with their own workspaces."""
    x, s = random("bf16", 8, 4, 60001, seed=5)
    y, t = random("f32", 3, 8, 20000, seed=6)
    want, want_y = select(D, x, s, 24), select(D, y, t, 24)
    torch.cuda.synchronize()
    outs = [[torch.empty_like(o) for o in w] for w in (want, want_y)]
    ws = [torch.empty(D.dflash_beam_workspace_bytes(*v.shape, 24), dtype=torch.uint8, device=DEV) for v in (x, y)]
    streams = [torch.cuda.Stream() for _ in range(2)]
    for _ in range(20):
        for st, v, u, o, w in zip(streams, (x, y), (s, t), outs, ws):
            with torch.cuda.stream(st):
                D.dflash_beam_select(v, u, 24, *o, w)
    torch.cuda.synchronize()
    for a, b in zip(outs[0] + outs[1], want + want_y):
        assert torch.equal(a, b)
    for o in outs[0]:
        o.zero_()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        D.dflash_beam_select(x, s, 24, *outs[0], ws[0])
    for _ in range(3):
        g.replay()
    torch.cuda.synchronize()
    for a, b in zip(outs[0], want):
        assert torch.equal(a, b)


def test_select_optional_outputs_and_launches(D):
    x, s = random("bf16", 2, 3, 5000, seed=8)
    want = select(D, x, s, 6)
    tok = torch.zeros((2, 6), dtype=torch.int32, device=DEV)
    ws = torch.empty(D.dflash_beam_workspace_bytes(2, 3, 5000, 6), dtype=torch.uint8, device=DEV)
    n = D.dflash_launch_count()
    D.dflash_trace_start(["beam_scan", "beam_merge"], 8)
    D.dflash_beam_select(x, s, 6, tok, None, None, ws)
    assert [k for k, _ in D.dflash_trace_stop()] == ["beam_scan", "beam_merge"]
    assert D.dflash_launch_count() == n + 2
    assert torch.equal(tok, want[0])
    with pytest.raises(ValueError, match="workspace|rows|tokens"):
        D.dflash_beam_select(x, s, 6, tok[:, ::2], None, None, ws)
    with pytest.raises(D.DFlashError):
        D.dflash_beam_select(x, s, 6, tok, None, None, ws[:100].clone())


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_select_rows_beyond_32_bit_offsets(D, dtype):
    far = 2 ** 31 + 8
    t = torch.zeros(far + 4096, dtype=TORCH[dtype], device=DEV)
    x, s = random(dtype, 2, 1, 4001, seed=11)
    t[:4001], t[far:far + 4001] = x[0, 0], x[1, 0]
    check(D, t.as_strided((2, 1, 4001), (far, 4001, 1)), s, 20)
    check(D, t.as_strided((1, 2, 4001), (far, far, 1)), s.t().contiguous(), 20)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_select_clustered_maxima(D, dtype):
    """The best logits side by side in one run, in one lane's runs of every tile, and in the last elements."""
    V = 70001
    for place in ("run", "lane", "end"):
        x, s = random(dtype, 2, 2, V, seed=12)
        at = {"run": torch.arange(33000, 33100), "lane": torch.arange(0, V - 32, 8192)[:, None] + torch.arange(12),
              "end": torch.arange(V - 90, V)}[place].flatten()
        x[..., at] = (30 + torch.arange(at.numel()).float() * 0.125).to(DEV, TORCH[dtype])
        for k in (3, 40, 128):
            check(D, x, s, k)


def test_select_many_rows_and_beams(D):
    x, s = random("bf16", 3000, 1, 100, seed=13)
    check(D, x, s, 1)
    x, s = random("f32", 2, 128, 5000, seed=14)
    check(D, x, s, 128)
    check(D, x[:, :1].expand(2, 128, 5000), s, 128)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("high", [11.9, 12.5, 39.0, 90.0])
def test_select_sums_whose_terms_err_one_way(D, dtype, high):
    """A few low logits, then one value over and over, so that no term's error makes up for another's. Of the
    values near `high` the one whose product with log2 e rounds the furthest."""
    v = torch.linspace(high - 0.5, high, 4001).to(TORCH[dtype])
    t = v.float() * np.float32(np.log2(np.e))
    err = (np64(t) - np64(v) * np.log2(np.e)) * (np64(v) < high)
    x = torch.zeros((2, 2, 60000), dtype=TORCH[dtype])
    for b, worst in enumerate((v[int(err.argmax())], v[int(err.argmin())])):
        x[b, :, 9000:] = worst
        x[b, 1, 9000:20000] -= 3
    check(D, x.to(DEV), torch.tensor([[-1.0, -1.125], [0.0, 0.0]], device=DEV), 5)
