"""Host-side refusals of the chunk step's calls: nothing is launched, so no GPU is needed."""
import ctypes

import pytest

OK, INVALID, UNSUPPORTED, WORKSPACE = 0, 1, 2, 3
P = ctypes.c_void_p


@pytest.fixture(scope="module")
def D():
    from speculative_decoding_draft_dflash_gb300 import build
    build.build()
    from speculative_decoding_draft_dflash_gb300 import dflash
    return dflash


def _dims(D, **kw):
    base = dict(d=4096, n_h=32, n_kv=8, d_h=128, k_layers=1, block_size=1, eps=1e-6, dtype=D.DFLASH_BF16)
    base.update(kw)
    return D.dflash_dims(*(base[n] for n, _ in D.dflash_dims._fields_))


def _cache(D, paged=True, **kw):
    base = dict(k=4096, v=8192, lens=256, n_layers=2, batch=4, capacity=512,
                block_table=1024 if paged else None, page_size=128 if paged else 0,
                n_pages=64 if paged else 0, kv_dtype=0, kv_scales=None)
    base.update(kw)
    return D.dflash_kv_cache(*(base[n] for n, _ in D.dflash_kv_cache._fields_))


def _chunk(D, **kw):
    base = dict(cu_rows=512, kv_lens=640, slots=768, positions=896, batch=4, rows=10)
    base.update(kw)
    return D.dflash_chunk(*(base[n] for n, _ in D.dflash_chunk._fields_))


def _pool(D, **kw):
    base = dict(block_table=1024, pages_held=64, pages_held_out=64, free_pages=128, n_free=8, taken=192, taken_out=192)
    base.update(kw)
    return D.dflash_page_pool(*(base[n] for n, _ in D.dflash_page_pool._fields_))


def _map(D, cache=None, chunk=None, pool=None, layer=0, no_pool=False):
    r = ctypes.byref
    pool = None if no_pool else r(pool or _pool(D))
    return D._lib.dflash_chunk_map(r(cache or _cache(D)), layer, r(chunk or _chunk(D)), pool, None)


@pytest.mark.parametrize("kw", [dict(cu_rows=None), dict(kv_lens=None), dict(slots=None), dict(positions=None),
                                dict(cu_rows=513), dict(kv_lens=642), dict(slots=769), dict(positions=898),
                                dict(batch=3), dict(rows=-1)])
def test_map_refuses_a_bad_plan(D, kw):
    assert _map(D, chunk=_chunk(D, **kw)) == INVALID


@pytest.mark.parametrize("kw", [dict(block_table=2048), dict(block_table=None), dict(pages_held=None),
                                dict(pages_held_out=None), dict(free_pages=None), dict(n_free=-1), dict(taken=None),
                                dict(taken_out=None), dict(taken=193), dict(free_pages=130)])
def test_map_refuses_a_bad_pool(D, kw):
    assert _map(D, pool=_pool(D, **kw)) == INVALID


def test_map_refuses_other_arguments(D):
    assert _map(D, no_pool=True) == INVALID                            # paged without a pool
    assert _map(D, layer=2) == INVALID and _map(D, layer=-1) == INVALID
    assert _map(D, cache=_cache(D, page_size=64)) == INVALID
    assert _map(D, chunk=_chunk(D, kv_lens=256)) == INVALID            # the cache's own lengths
    assert _map(D, chunk=_chunk(D, kv_lens=272), layer=1) == INVALID
    assert _map(D, cache=_cache(D, capacity=500)) == INVALID           # not whole pages
    assert _map(D, cache=_cache(D, n_pages=1 << 24)) == UNSUPPORTED    # 2^31 slots
    assert _map(D, cache=_cache(D, batch=8193), chunk=_chunk(D, batch=8193)) == UNSUPPORTED
    assert _map(D, cache=_cache(D, paged=False, batch=4, capacity=1 << 29)) == UNSUPPORTED


def _append(D, dims=None, cache=None, chunk=None, layer=0, **kw):
    a = dict(q=4096, ld_q=4096, k=8192, ld_k=1024, v=16384, ld_v=1024, gq=256, gk=512, rope=768, tl=64, out=32768)
    a.update(kw)
    r = ctypes.byref
    return D._lib.dflash_chunk_append(r(dims or _dims(D)), r(cache or _cache(D)), layer, r(chunk or _chunk(D)),
                                      *(a[n] for n in ("q", "ld_q", "k", "ld_k", "v", "ld_v", "gq", "gk", "rope", "tl",
                                                       "out")), None)


@pytest.mark.parametrize("kw", [dict(k=None), dict(v=None), dict(q=None), dict(out=None), dict(q=4104), dict(k=8194),
                                dict(ld_q=4095), dict(ld_q=4100), dict(ld_k=1023), dict(ld_v=1020), dict(gq=264),
                                dict(gk=520), dict(rope=776), dict(rope=None), dict(tl=-1), dict(layer=2),
                                dict(out=4096, ld_q=8192), dict(out=32776)])
def test_append_refuses(D, kw):
    assert _append(D, **kw) == INVALID


def test_append_refuses_layouts_and_accepts_no_rows(D):
    f32 = _dims(D, dtype=D.DFLASH_F32, d_h=64, n_h=8, n_kv=8, d=512)
    assert _append(D, dims=f32) == UNSUPPORTED                          # f32 has no paged layout
    assert _append(D, dims=f32, cache=_cache(D, paged=False, kv_dtype=2)) == UNSUPPORTED
    assert _append(D, dims=_dims(D, d_h=64)) == UNSUPPORTED
    assert _append(D, chunk=_chunk(D, rows=0, slots=None, positions=None)) == OK


def _attn(D, dims=None, cache=None, chunk=None, layer=0, **kw):
    a = dict(q=4096, ld_q=4096, window=0, scaling=0.0, out=32768, ws=65536, wsb=1 << 30)
    a.update(kw)
    r = ctypes.byref
    return D._lib.dflash_chunk_attn(r(dims or _dims(D)), r(cache or _cache(D)), layer, r(chunk or _chunk(D)), a["q"],
                                    a["ld_q"], a["window"], a["scaling"], a["out"], a["ws"], a["wsb"], None)


@pytest.mark.parametrize("kw", [dict(q=None), dict(q=4104), dict(ld_q=4088), dict(ld_q=4100), dict(out=None),
                                dict(out=32776), dict(ws=None), dict(ws=65552), dict(window=-1), dict(layer=7),
                                dict(scaling=float("nan")), dict(scaling=float("inf"))])
def test_attn_refuses(D, kw):
    assert _attn(D, **kw) == INVALID


def test_attn_refuses_sizes(D):
    assert _attn(D, wsb=1 << 20) == WORKSPACE
    assert _attn(D, chunk=_chunk(D, batch=5)) == INVALID
    assert _attn(D, chunk=_chunk(D, kv_lens=None)) == INVALID
    assert _attn(D, chunk=_chunk(D, rows=0)) == OK
    assert _attn(D, cache=_cache(D, n_pages=1 << 21)) == UNSUPPORTED    # 2^31 key rows of a layer
    assert _attn(D, dims=_dims(D, n_h=136, n_kv=1)) == UNSUPPORTED      # more than 128 query heads a KV head
    one = dict(batch=1, paged=False)
    assert _attn(D, dims=_dims(D, n_h=8, n_kv=1), cache=_cache(D, capacity=(1 << 28) + 1, **one),
                 chunk=_chunk(D, batch=1)) == UNSUPPORTED
    assert _attn(D, chunk=_chunk(D, rows=(1 << 28) + 1)) == UNSUPPORTED   # 2^30 stacked rows
    assert _attn(D, cache=_cache(D, batch=8193), chunk=_chunk(D, batch=8193)) == UNSUPPORTED
    assert D.dflash_chunk_workspace_bytes(_dims(D)) > 0
    assert D.dflash_chunk_workspace_bytes(_dims(D, d_h=64)) == 0


def test_binding_refuses_host_and_mismatched_tensors(D):
    import torch
    cu = torch.zeros(5, dtype=torch.int32)
    with pytest.raises(ValueError):
        D.ChunkPlan(cu, 3)                                              # host memory
    with pytest.raises(ValueError):
        D.ChunkPlan(torch.zeros(1, dtype=torch.int32), 3)               # no sequence
    with pytest.raises(ValueError):
        D.PagePool(torch.zeros(4), torch.zeros(4), torch.zeros(1))
    with pytest.raises(ValueError):
        D._rows(torch.zeros(4, 8, dtype=torch.bfloat16), "q", torch.bfloat16, 4, 8)


def test_binding_refuses_other_devices(D):
    """What belongs to a step lies on the plan's device. (A plan of device 3 stands in, and what
    it meets lies in host memory, which is no device.)"""
    import types

    import torch
    plan = types.SimpleNamespace(batch=2, rows=4, device=3, ref=None)
    cache = D.KVCache(1, 2, 2, 128, 64, "f32", device="cpu")
    with pytest.raises(ValueError, match="cache"):
        D.dflash_chunk_map(cache, 0, plan)
    pool = types.SimpleNamespace(batch=2, device=-1)
    with pytest.raises(ValueError, match="page pool"):
        D.dflash_chunk_map(cache, 0, plan, pool)
    for t in (torch.zeros(4), torch.zeros(8, dtype=torch.int32)[::2]):
        with pytest.raises(ValueError):
            D._array(t, "out", torch.float32, 4, 3)
    assert D._array(None, "out", torch.float32, 4, 3) is None and D._array(64, "out", torch.float32, 4, 3) == 64
