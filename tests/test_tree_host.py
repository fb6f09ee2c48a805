"""Host-side refusals of the tree and beam calls: nothing is launched, so no GPU is needed."""
import ctypes

import pytest

from test_chunk_host import INVALID, UNSUPPORTED, WORKSPACE, D, _cache, _chunk, _dims  # noqa: F401

r = ctypes.byref


def _tree(D, **kw):
    base = dict(nodes=64, depths=128, masks=256, batch=4, max_nodes=64)
    base.update(kw)
    return D.dflash_tree(*(base[n] for n, _ in D.dflash_tree._fields_))


BAD_TREES = [dict(nodes=None), dict(nodes=66), dict(batch=3), dict(max_nodes=0), dict(max_nodes=33), dict(max_nodes=-32)]
BAD_MASKS = [dict(depths=None), dict(depths=129), dict(masks=None), dict(masks=258)]


def _map(D, chunk=None, tree=None, parents=512, before=None):
    return D._lib.dflash_tree_map(r(chunk or _chunk(D)), r(tree or _tree(D)), parents, before, None)


@pytest.mark.parametrize("kw", BAD_TREES + BAD_MASKS)
def test_map_and_attn_refuse_a_bad_tree(D, kw):
    assert _map(D, tree=_tree(D, **kw)) == INVALID
    assert _attn(D, tree=_tree(D, **kw)) == INVALID


@pytest.mark.parametrize("kw", [dict(cu_rows=None), dict(kv_lens=None), dict(slots=None), dict(positions=None),
                                dict(cu_rows=514), dict(slots=770), dict(batch=0), dict(rows=-1)])
def test_map_refuses_a_bad_plan(D, kw):
    assert _map(D, chunk=_chunk(D, **kw)) == INVALID


def test_map_refuses_other_arguments(D):
    assert _map(D, parents=None) == INVALID and _map(D, parents=513) == INVALID
    assert _map(D, before=66) == INVALID
    assert D._lib.dflash_tree_map(None, r(_tree(D)), 512, None, None) == INVALID
    assert D._lib.dflash_tree_map(r(_chunk(D)), None, 512, None, None) == INVALID
    assert _map(D, tree=_tree(D, max_nodes=4128)) == UNSUPPORTED
    assert _map(D, chunk=_chunk(D, batch=4097), tree=_tree(D, batch=4097)) == UNSUPPORTED


def _attn(D, dims=None, cache=None, chunk=None, tree=None, layer=0, **kw):
    a = dict(q=4096, ld_q=4096, window=0, scaling=0.0, out=32768, ws=65536, wsb=1 << 30)
    a.update(kw)
    return D._lib.dflash_tree_attn(r(dims or _dims(D)), r(cache or _cache(D)), layer, r(chunk or _chunk(D)),
                                   r(tree or _tree(D)), a["q"], a["ld_q"], a["window"], a["scaling"], a["out"],
                                   a["ws"], a["wsb"], None)


def test_attn_refuses(D):
    for kw in (dict(q=None), dict(q=4104), dict(ld_q=4088), dict(out=None), dict(ws=None), dict(window=-1), dict(layer=7),
               dict(scaling=float("nan"))):
        assert _attn(D, **kw) == INVALID, kw
    assert _attn(D, wsb=1 << 20) == WORKSPACE
    assert _attn(D, tree=_tree(D, max_nodes=4128)) == UNSUPPORTED
    assert _attn(D, cache=_cache(D, batch=4097), chunk=_chunk(D, batch=4097), tree=_tree(D, batch=4097)) == UNSUPPORTED
    assert D._lib.dflash_tree_attn(r(_dims(D)), r(_cache(D)), 0, r(_chunk(D)), None, 4096, 4096, 0, 0.0, 32768, 65536,
                                   1 << 30, None) == INVALID
    assert _attn(D, chunk=_chunk(D, rows=0)) == 0


def _accept(D, chunk=None, **kw):
    a = dict(parents=64, tokens=128, posterior=256, ctx_len=512, max_path=8, path=640, accept_len=768, cu=896, ctx=1024,
             anchor=1152)
    a.update(kw)
    return D._lib.dflash_tree_accept(r(chunk or _chunk(D)), *a.values(), None)


@pytest.mark.parametrize("name", ["parents", "tokens", "posterior", "ctx_len", "path", "accept_len", "cu", "ctx", "anchor"])
def test_accept_refuses(D, name):
    assert _accept(D, **{name: None}) == INVALID
    assert _accept(D, **{name: 66}) == INVALID


def test_accept_refuses_sizes(D):
    assert _accept(D, max_path=0) == INVALID
    assert _accept(D, chunk=_chunk(D, batch=0)) == INVALID
    assert _accept(D, chunk=_chunk(D, cu_rows=None)) == INVALID
    assert _accept(D, chunk=_chunk(D, batch=8193)) == UNSUPPORTED


def _commit(D, dims=None, cache=None, tree=None, **kw):
    a = dict(ctx_len=64, path=128, max_path=8, accept_len=256)
    a.update(kw)
    return D._lib.dflash_tree_commit(r(dims or _dims(D)), r(cache or _cache(D)), r(tree or _tree(D)), *a.values(), None)


def test_commit_refuses(D):
    for kw in (dict(ctx_len=None), dict(path=None), dict(accept_len=None), dict(ctx_len=66), dict(path=130),
               dict(accept_len=257), dict(max_path=0)):
        assert _commit(D, **kw) == INVALID, kw
    for kw in BAD_TREES:
        assert _commit(D, tree=_tree(D, **kw)) == INVALID, kw
    assert _commit(D, cache=_cache(D, page_size=64)) == INVALID
    assert _commit(D, dims=_dims(D, d_h=64)) == UNSUPPORTED
    assert _commit(D, cache=_cache(D, n_layers=32768)) == UNSUPPORTED


def test_commit_refuses_inputs_that_are_the_lengths(D):
    """2 layers of 4 sequences from 1024 on: 32 bytes, which the call writes while it reads the others."""
    cache = _cache(D, lens=1024, block_table=4096)
    for at in (1024, 1040, 1052, 1012):
        for name in ("ctx_len", "accept_len", "path"):
            assert _commit(D, cache=cache, **{name: at}) == INVALID, (name, at)
        assert _commit(D, cache=cache, tree=_tree(D, nodes=at)) == INVALID, at
    assert _commit(D, cache=cache, path=1024 - 4 * 4 * 8 + 4) == INVALID     # (its last element)


def _select(D, dtype=1, **kw):
    a = dict(logits=4096, ld_seq=1000, ld_beam=100, scores=64, batch=2, beams=4, vocab=100, k=8, base=0, tokens=128,
             parents=192, out=256, ld_out=8, ws=65536, wsb=1 << 30)
    a.update(kw)
    return D._lib.dflash_beam_select(dtype, *a.values(), None)


@pytest.mark.parametrize("kw", [dict(logits=None), dict(logits=4097), dict(dtype=0, logits=4098), dict(ld_seq=-1),
                                dict(ld_beam=-1), dict(scores=66), dict(batch=0), dict(beams=0), dict(vocab=0), dict(k=0),
                                dict(k=9, beams=2, vocab=4, ld_out=9), dict(base=-1), dict(base=2 ** 31 - 2),
                                dict(tokens=None), dict(tokens=130), dict(parents=193), dict(out=257), dict(ld_out=7),
                                dict(ws=None), dict(ws=65664)])
def test_select_refuses(D, kw):
    assert _select(D, **kw) == INVALID


def test_select_refuses_sizes(D):
    assert _select(D, dtype=2) == UNSUPPORTED
    assert _select(D, beams=129) == UNSUPPORTED
    assert _select(D, k=129, ld_out=129) == UNSUPPORTED
    assert _select(D, vocab=1 << 29) == UNSUPPORTED
    assert _select(D, batch=1 << 19) == UNSUPPORTED
    assert _select(D, wsb=100) == WORKSPACE
    assert D.dflash_beam_workspace_bytes(2, 4, 100, 8) > 0
    assert D.dflash_beam_workspace_bytes(2, 129, 100, 8) == 0


def test_binding_refuses_host_and_mismatched_tensors(D):
    import types

    import torch
    i32 = torch.int32
    with pytest.raises(ValueError, match="CUDA"):
        D.Tree(2, 64, device="cpu")
    for bad in (0, 33):
        with pytest.raises(ValueError, match="max_nodes"):
            D.Tree(2, bad, device="cpu")
    plan = types.SimpleNamespace(batch=2, rows=4, device=3, ref=None)
    for tree in (types.SimpleNamespace(batch=3, device=3, ref=None), types.SimpleNamespace(batch=2, device=1, ref=None)):
        with pytest.raises(ValueError, match="tree"):
            D._tree(tree, plan)
    with pytest.raises(ValueError, match="logits"):
        D.dflash_beam_select(torch.zeros(1, 2, 8), None, 2, None, None, None, None)
    t = torch.zeros(2, 6, dtype=i32)
    assert D._k_rows(t[:, 1:4], "tokens", i32, 2, 3, -1) == (t[:, 1:4].data_ptr(), 6)
    assert D._k_rows(None, "parents", i32, 2, 3, -1) == (None, None)
    for bad in (t.float(), t[:1], t[:, :2], t.t().contiguous().t(), t[0]):
        with pytest.raises(ValueError, match="tokens"):
            D._k_rows(bad, "tokens", i32, 2, 3, -1)


def _beam_bytes(batch, beams, vocab, k, sms):
    """The selection's workspace, with every number of pieces of a row tried: the least of turns of CTAs x (units of a
    piece + 27) + candidates / 128, of equal ones the fewest pieces."""
    slots, units, fit = 3 * sms, -(-vocab // 2048), 8192 // (beams * k)

    def pieces(rows):
        cost = {}
        for s in range(1, units + 1):
            if (s > 1 and s > fit) or rows * (s - 1) >= 8 * slots:
                break
            per = -(-units // s)
            n = -(-units // per)
            cost.setdefault(-(-rows * n // slots) * (per + 27) + beams * n * k / 128, n)
        return rows * cost[min(cost)]

    most = max(pieces(batch * beams), pieces(batch))
    return sum(-(-most * size // 256) * 256 for size in (8 * k, 16))


def test_select_cuts_rows_at_the_least_cost_in_little_host_time(D):
    """Few rows of a long vocabulary may have thousands of pieces: not every number of them is tried in a call (it took
    13 times as long for a row of 2^24 as for one of 131072)."""
    import random
    import time

    r = random.Random(3)
    sizes = [(1, 1, 1, 1), (1, 1, 2 ** 24, 1), (3, 128, 5 * 10 ** 6, 128), (1, 1, 2 ** 28, 1), (1, 1, 2 ** 28 - 2047, 2)]
    for _ in range(300):
        beams = r.choice((1, 1, 2, 5, 8, 33))
        vocab = int(2 ** r.uniform(0, 23))
        sizes.append((int(2 ** r.uniform(0, 9)), beams, vocab, min(r.choice((1, 2, 8, 50, 128)), beams * vocab)))
    for size in sizes:
        got = D.dflash_beam_workspace_bytes(*size)
        assert got in (_beam_bytes(*size, 148), _beam_bytes(*size, 152)), size   # (148: no device to ask)

    def best(*size):
        took = []
        for _ in range(200):
            t = time.perf_counter()
            D.dflash_beam_workspace_bytes(*size)
            took.append(time.perf_counter() - t)
        return min(took)

    assert best(1, 1, 2 ** 24, 1) < 6 * best(1, 1, 131072, 1)
