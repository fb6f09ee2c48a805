"""Beam selection of so many rows that each is one piece of eight tiles and more, where a lane's notes fill up:
equal, few-valued, clipped and masked logits, against the formula in float64."""
import numpy as np
import pytest
import torch

import tree_ref as T
from test_beam_gpu import TORCH, np64, select
from test_chunk_gpu import DEV, D  # noqa: F401  (D is the fixture)

pytestmark = pytest.mark.gpu

INF = float("inf")
TILE = {"f32": 4096, "bf16": 8192}  # elements of a tile
# (a row in one piece of 16, 8 and 13 tiles)
ROWS = [("bf16", 256, 131072), ("f32", 256, 32000), ("f32", 256, 50001)]


def expect(logits, scores, k):
    """tree_ref.beam_select of every sequence, on the device."""
    x = logits.double()
    m = x.amax(-1, keepdim=True)                      # (NaN where the row has one)
    s = torch.zeros(x.shape[:2], dtype=torch.float64, device=DEV) if scores is None else scores.double()
    v = s[..., None] + ((x - m) - torch.log(torch.exp(x - m).sum(-1, keepdim=True)))
    v = torch.where(torch.isfinite(m) & torch.isfinite(s)[..., None], v, -INF).flatten(1)
    best, at = torch.sort(v, dim=1, descending=True, stable=True)
    at = at[:, :k]
    return at % logits.shape[2], at // logits.shape[2], np64(best[:, :k])


def check(D, logits, scores, k, base=0):
    """Every place is written (the buffers held -9), with what float64 gives. Beams with rows of their own may change
    places where their scores are nearer than the errors of their two log-sums: each is within 2 10^-6, so that
    the order of the scores is sure from 4 10^-6 on ("high in one lane": rows that differ in noise, 10^-13 of their
    sums). The tokens of one beam keep their order."""
    batch, beams, vocab = logits.shape
    got = select(D, logits, scores, k, base)
    tok, par, want = expect(logits, scores, k)
    t, i = got[0].long(), got[1].long() - base
    if beams > 1 and logits.stride(1) != 0 and not (torch.equal(t, tok) and torch.equal(i, par)):
        assert ((t >= 0) & (t < vocab) & (i >= 0) & (i < beams)).all()
        whole = expect(logits, scores, beams * k)            # (k of a beam are among them, or minus infinity)
        for b in (~((t == tok) & (i == par)).all(1)).nonzero().flatten().tolist():
            ranked = list(zip(whole[1][b].tolist(), whole[0][b].tolist()))
            score = dict(zip(ranked, whole[2][b]))
            mine = list(zip(i[b].tolist(), t[b].tolist()))
            for j, (place, v) in enumerate(zip(mine, want[b])):
                assert place == ranked[j] or (place[0] != ranked[j][0] and abs(score[place] - v) <= 4e-6), (b, j)
            for beam in range(beams):
                own = [p for p in mine if p[0] == beam]
                assert own == [p for p in ranked if p[0] == beam][:len(own)], (b, beam)
    else:
        assert torch.equal(t, tok) and torch.equal(i, par)
    out, fin = np64(got[2]), np.isfinite(want)
    assert (np.isneginf(out) == ~fin).all()
    assert (np.abs(out[fin] - want[fin]) <= T.beam_bound(want[fin])).all()
    return got


def allowed(dtype, batch, beams, vocab, n, fill):
    """n random tokens of each beam, the others masked."""
    g = torch.Generator().manual_seed(n)
    x = torch.full((batch, beams, vocab), fill, dtype=TORCH[dtype])
    at = torch.randint(0, vocab, (batch, beams, n), generator=g)
    x.scatter_(2, at, torch.randn((batch, beams, n), generator=g).to(TORCH[dtype]))
    return x.to(DEV), (-4 * torch.rand((batch, beams), generator=g)).to(DEV)


@pytest.mark.parametrize("dtype,batch,beams,vocab,k", [("bf16", 32, 8, 131072, 16), ("f32", 64, 4, 50001, 8)])
def test_one_token_allowed_a_beam_keeps_every_beam(D, dtype, batch, beams, vocab, k):
    """A constrained search: the allowed tokens come first, and no place keeps what the buffer held."""
    x, s = allowed(dtype, batch, beams, vocab, 1, -INF)
    tok, par, out = select(D, x, s, k, base=3)
    t, p, v = expect(x, s, k)
    assert torch.equal(tok[:, :beams].long(), t[:, :beams]) and torch.equal(par[:, :beams].long(), p[:, :beams] + 3)
    assert (np.abs(np64(out[:, :beams]) - v[:, :beams]) <= T.beam_bound(v[:, :beams])).all()
    assert (out[:, beams:] == -INF).all()
    assert ((tok >= 0) & (tok < vocab)).all() and ((par >= 3) & (par < 3 + beams)).all()


def high_in_one_lane(x, tile):
    """Falling logits in the same lane's run of every tile, so that this lane alone has notes to spare; the last
    of them have bare mantissas."""
    x[..., 5::tile] = 39.0 - torch.arange(len(range(5, x.shape[-1], tile)), dtype=torch.float32)
    x[..., 70] = 15.0


KINDS = {
    "equal": lambda x, tile: x.fill_(-2.5),
    "zeros": lambda x, tile: x.zero_(),
    "three values": lambda x, tile: x.copy_((x > 1.0).float() - (x < -1.0).float()),
    "clipped": lambda x, tile: x.clamp_(-3.0, 3.0),                            # (1.5 standard deviations)
    "clipped at 2": lambda x, tile: x.clamp_(-4.0, 4.0),
    "one top value": lambda x, tile: x[..., ::11].fill_(20.0),                 # 3000 to 12000 elements
    "top behind": lambda x, tile: x[..., x.shape[-1] // 2:].fill_(11.0),
    "rounded": lambda x, tile: x.round_(),
    "high in one lane": high_in_one_lane,
    "ascending in steps": lambda x, tile: x.copy_((torch.arange(x.shape[-1]) // 700).float() * 0.125),
}


@pytest.mark.parametrize("dtype,batch,vocab", ROWS)
@pytest.mark.parametrize("kind", KINDS)
def test_rows_with_more_notes_than_a_lane_holds(D, dtype, batch, vocab, kind):
    g = torch.Generator().manual_seed(21)
    x = torch.randn((4, 1, vocab), generator=g) * 2
    KINDS[kind](x, TILE[dtype])
    x = x.to(DEV, TORCH[dtype]).repeat(batch // 4, 1, 1)
    for k in (1, 8, 16, 128):
        check(D, x, None, k)
    s = torch.linspace(-1, 0, batch, device=DEV).view(-1, 4)                    # as four beams of a sequence
    s[:, 2] = s[:, 1]
    check(D, x.view(-1, 4, vocab), s.contiguous(), 8, base=1)


@pytest.mark.parametrize("dtype,batch,vocab", ROWS)
@pytest.mark.parametrize("n", [1, 5, 40])
@pytest.mark.parametrize("lowest", [False, True])
def test_rows_masked_to_a_few_tokens(D, dtype, batch, vocab, n, lowest):
    """Fewer allowed tokens than asked for: the lowest of the others follow."""
    x, s = allowed(dtype, batch, 1, vocab, n, torch.finfo(TORCH[dtype]).min if lowest else -INF)
    for k in (1, 8, 128):
        check(D, x, s, k)
    check(D, x.view(-1, 8, vocab), s.view(-1, 8), 16)


def test_one_token_allowed_a_beam(D):
    for dtype, batch, beams, vocab, k in [("bf16", 32, 8, 131072, 16), ("f32", 64, 4, 50001, 8)]:
        x, s = allowed(dtype, batch, beams, vocab, 1, -INF)
        check(D, x, s, k)


@pytest.mark.parametrize("dtype,vocab", [("bf16", 131072), ("bf16", 65601), ("f32", 50001)])
def test_a_row_for_all_beams_of_many_sequences(D, dtype, vocab):
    """A level of as many trees, masked and clipped."""
    for kind in ("clipped", "high in one lane", "zeros"):
        x = torch.randn((4, 1, vocab), generator=torch.Generator().manual_seed(5)) * 2
        KINDS[kind](x, TILE[dtype])
        x = x.to(DEV, TORCH[dtype]).repeat(64, 1, 1)
        s = -4 * torch.rand((256, 3), generator=torch.Generator().manual_seed(6)).to(DEV)
        check(D, x.expand(256, 3, vocab), s, 20)
    x, _ = allowed(dtype, 256, 1, vocab, 5, -INF)
    check(D, x.expand(256, 3, vocab), s, 20)


def test_the_same_bits_again_where_notes_fill_up(D):
    x = (torch.randn((256, 1, 131072), generator=torch.Generator().manual_seed(8)) * 2).clamp(-3, 3).to(DEV, torch.bfloat16)
    want = select(D, x, None, 16)
    for _ in range(20):
        assert all(torch.equal(a, b) for a, b in zip(select(D, x, None, 16), want))


@pytest.mark.parametrize("dtype,batch,vocab", ROWS + [("bf16", 6, 131072), ("f32", 3, 50001)])
@pytest.mark.parametrize("nan,high,value", [(5, 31000, 200.0), (5, 31000, 90.0), (31990, 70, 300.0), (20000, 31000, 81.0)])
def test_rows_with_nan_next_to_a_much_larger_logit(D, dtype, batch, vocab, nan, high, value):
    """The row has no probability, however far above the NaN's neighbours another logit lies. In the larger
    calls a row is one piece, in the others several."""
    x = (torch.randn((batch, 1, vocab), generator=torch.Generator().manual_seed(9)) * 2).to(DEV, TORCH[dtype])
    x[::2, :, nan] = float("nan")
    x[:, :, high] = value
    for k in (1, 8):
        check(D, x, None, k)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("batch,vocab", [(1, 131072), (2, 50001), (40, 20000), (256, 65601), (3, 700)])
def test_scores_that_64_bits_do_not_tell_apart(D, dtype, batch, vocab):
    """Tiny logits, and logits next to a far larger score or logit: a beam's tokens still come in the order of their
    logits, equal ones lowest first, in however many pieces its row is."""
    g = torch.Generator().manual_seed(12)
    noise = torch.randn((batch, 1, vocab), generator=g)
    tiny, far = (noise * 1e-20).to(DEV, TORCH[dtype]), noise.to(DEV, TORCH[dtype])
    spiked = far.clone()
    spiked[..., vocab // 3] = 3e38
    s = torch.full((batch, 1), -1e30, device=DEV)
    for x, scores in ((tiny, None), (far, s), (spiked, None), (tiny, s)):
        rank = torch.sort(x[:, 0].double(), dim=1, descending=True, stable=True)[1]
        for k in (1, 8, 100):
            tok, par, _ = select(D, x, scores, k, base=2)
            assert torch.equal(tok.long(), rank[:, :k]) and (par == 2).all()
    # two beams alike: the first one's tokens, in order, before the second one's
    two = tiny.expand(batch, 2, vocab)
    for x in (two, two.contiguous()):
        tok, par, _ = select(D, x, torch.cat((s, s), 1), 60)
        assert (par == 0).all() and torch.equal(tok.long(), torch.sort(tiny[:, 0].double(), dim=1, descending=True,
                                                                        stable=True)[1][:, :60])
