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
    """Every place is written (the buffers held -9), with what float64 gives."""
    got = select(D, logits, scores, k, base)
    tok, par, want = expect(logits, scores, k)
    assert torch.equal(got[0].long(), tok)
    assert torch.equal(got[1].long(), par + base)
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
