"""The chunk step at the edges that its first tests leave out: weights and queries of extreme
spread, values that are not finite, large steps, what a round leaves in the cache."""
import ctypes

import numpy as np
import pytest
import torch

import chunk_ref as R
from test_chunk_gpu import DEV, D, Step, i32, np64  # noqa: F401  (D is the module's fixture)

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
