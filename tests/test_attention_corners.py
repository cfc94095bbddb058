"""Corners of the attention entry points' checks (CPU)."""
import expert_cache_host_router_b200 as moe
from test_attention_refusals import INVALID, P, lib, pool, rows, table  # noqa: F401


def test_one_table_row_for_all_sequences(lib):
    """A row stride of 0 where pages are read or written row by row; not for the pages that an eviction fills."""
    c, t = pool(), table(row_stride=0)
    assert lib.moe_kv_store(c, t, P, None, rows(), rows(), 0, 0, None) == moe.MOE_OK
    assert lib.moe_kv_load(c, t, P, None, rows(), rows(), 0, 0, None) == moe.MOE_OK
    for bad in (-1, -4, 1, 3):
        assert lib.moe_kv_store(c, table(row_stride=bad), P, None, rows(), rows(), 0, 0, None) == INVALID
    s = moe.KvScore(P, 512, 256)
    assert lib.moe_kv_evict(c, t, P, 100, s, 16, 4, table(table_dev=2 * P, row_stride=0), 3 * P, P, P, None) == INVALID


def test_stalls_asked_for(lib):
    assert lib.moe_debug_stall_attention(-1) == INVALID and lib.moe_debug_stall_attention(0) == moe.MOE_OK
