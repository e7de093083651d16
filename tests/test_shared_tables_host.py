"""SharedBlockTables on the host, without a GPU: the buffers that its calls hand over."""
import pytest
import torch

import block_quantized_weight_dequant_gb300 as bq
from block_quantized_weight_dequant_gb300 import cache


@pytest.mark.parametrize("pages", [1, 2, 41])
def test_compact_keeps_its_buffers(monkeypatch, pages):
    """A graph that captured a compaction holds the addresses of its lists and of
    `moved`: calls with other max_moves take the same ones, none is given back."""
    seen = []
    monkeypatch.setattr(cache, "kv_compact", lambda *a: seen.append(a[6:10]))
    t = bq.SharedBlockTables(3, 4, pages, 16, 8, device="cpu")
    room = pages // 2
    for most in (None, 3, 0, None, pages, room):
        moved = t.compact() if most is None else t.compact(most)
        src, dst, count, given = seen[-1]
        assert moved is given and given.numel() == pages and count.numel() == 1
        # half the pool is all there can be
        assert src.numel() == dst.numel() == (room if most is None else min(most, room))
    first = seen[0]
    for later in seen[1:]:
        for a, b in zip(first, later):
            assert a.untyped_storage().data_ptr() == b.untyped_storage().data_ptr()
            assert a.storage_offset() == b.storage_offset() == 0
    with pytest.raises(ValueError, match="max_moves"):
        t.compact(-1)


def test_the_hook_of_held_barriers_takes_those_that_there_are():
    """What a GPU test of the bounded waits is made with (not in the public header)."""
    import ctypes

    from block_quantized_weight_dequant_gb300 import _lib

    hook = _lib.lib.bq_internal_prefix_hold
    hook.restype, hook.argtypes = ctypes.c_int, [ctypes.c_int, ctypes.c_ulonglong]
    assert hook(-1, 0) == -1 and hook(10, 0) == -1
    assert hook(9, 1000) == 0 and hook(0, 0) == 0
