"""The chunk step's Python binding on the host: what it hands to the library."""
import types

import pytest


@pytest.fixture(scope="module")
def D():
    from speculative_decoding_draft_dflash_gb300 import build
    build.build()
    from speculative_decoding_draft_dflash_gb300 import dflash
    return dflash


def test_map_calls_that_share_a_pool_keep_their_own_block_tables(D, monkeypatch):
    """A second call with another cache begins while the first is in the library (two threads;
    here it is made from inside): each call passes its own cache's block table, and the pool's
    descriptor stays as it was."""
    desc = D.dflash_page_pool(None, 64, 64, 128, 8, 192, 192)
    pool = types.SimpleNamespace(batch=2, device=-1, desc=desc)
    plan = types.SimpleNamespace(batch=2, rows=4, device=-1, ref=None)
    caches = [D.dflash_kv_cache(4096, 8192, 256, 1, 2, 128, table, 128, 4) for table in (1024, 2048)]
    seen = []

    def call(cache, layer, chunk, own, stream):
        if not seen:
            seen.append(None)
            D.dflash_chunk_map(caches[1], 0, plan, pool, stream=0)
        seen.append(own._obj.block_table)
        assert (own._obj.pages_held, own._obj.free_pages, own._obj.n_free, own._obj.taken) == (64, 128, 8, 192)
        return D.OK

    monkeypatch.setattr(D, "_lib", types.SimpleNamespace(dflash_chunk_map=call))
    monkeypatch.setattr(D, "_current_device", lambda: -1)
    D.dflash_chunk_map(caches[0], 0, plan, pool, stream=0)
    assert seen[1:] == [2048, 1024]
    assert desc.block_table is None
