"""How calls over shared pages are cut, on the host without a GPU."""
import ctypes

import pytest

from block_quantized_weight_dequant_gb300 import _lib

from test_cache_host import attention, cache, lib  # noqa: F401
from test_shared_host import groups


def needs(lib, x, c, *pairs):  # noqa: F811
    """Workspace bytes over the groups, and of the ordinary call, which is one pass."""
    return (lib.bq_paged_prefix_attention_workspace_bytes(c, x, *groups(*pairs)),
            lib.bq_paged_attention_workspace_bytes(c, x))


@pytest.mark.parametrize("kind", [_lib.BQ_F16, _lib.BQ_BF16, _lib.BQ_Q8_0])
def test_groups_of_one_request_read_nothing_again(lib, kind):  # noqa: F811
    """However long, they are one pass of the ordinary kernel, alone or beside each other;
    two requests that share as much are not, and then they alone count."""
    c = cache(kind, kv_heads=8, head_dim=128, slot_stride=128, head_stride=2048, page_stride=16384)
    width = 8192
    one = attention(requests=1, heads=16, table_width=width, table_stride=width)
    shared, whole = needs(lib, one, c, (1, width * 16))
    assert shared == whole
    many = attention(requests=64, heads=16, table_width=width, table_stride=width)
    shared, whole = needs(lib, many, c, *[(1, 100000 + 16 * i) for i in range(64)])
    assert shared == whole
    shared, whole = needs(lib, many, c, *[(1, 100000)] * 62, (2, 100000))
    assert shared != whole
    # 2 * 8 * 128 values a position, read once more: 16 M of them
    shared, whole = needs(lib, many, c, *[(1, 100000)] * 62, (2, 8192))
    assert shared == whole


def test_the_type_of_the_queries_does_not_move_the_workspace(lib):  # noqa: F811
    """paged_prefix_attention_workspace may be asked without it."""
    limit = lib.bq_internal_prefix_whole_limit
    limit.restype, limit.argtypes = ctypes.c_int64, [ctypes.c_int64]
    limit(0)
    try:
        for kind in (_lib.BQ_F16, _lib.BQ_BF16, _lib.BQ_Q8_0):
            c = cache(kind, kv_heads=8, head_dim=128, slot_stride=128, head_stride=2048, page_stride=16384)
            need = {lib.bq_paged_prefix_attention_workspace_bytes(
                c, attention(requests=96, heads=32, dtype=dtype, table_width=4000, table_stride=4000), *groups((96, 32801)))
                for dtype in (_lib.BQ_F32, _lib.BQ_F16, _lib.BQ_BF16)}
            assert len(need) == 1 and need.pop() > 0
    finally:
        limit(-1)


def test_whole_numbers_of_any_kind_say_what_is_shared():
    """numpy's among them; others are refused, not cut to whole ones."""
    import numpy as np

    from block_quantized_weight_dequant_gb300.cache import _groups, _shared

    def told(shared, requests):
        counts, positions, n = _groups(_shared(shared), requests)
        return list(zip(counts, positions))

    for one in (40, np.int64(40), np.int32(40), np.array([40])[0]):
        assert told(one, 3) == [(3, 40)]
    pairs = np.array([[2, 40], [1, 0]])
    for several in (pairs, pairs.tolist(), [(np.int32(2), 40), (1, np.int64(0))], (p for p in pairs)):
        assert told(several, 3) == [(2, 40), (1, 0)]
    for bad in (40.0, 40.5, [(2, 40.5), (1, 0)], [(2.0, 40), (1, 0)], "40", [40, 1], None):
        with pytest.raises((TypeError, ValueError)):
            told(bad, 3)
