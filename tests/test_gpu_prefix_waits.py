"""The bounded waits of the attention over shared pages: one that nothing ends runs out
within its limit, the kernel says so and returns, and the next call is as before."""
import ctypes

import pytest
import torch

import block_quantized_weight_dequant_gb300 as bq
from block_quantized_weight_dequant_gb300 import _lib

from test_gpu_cache import BF16, DEV, F16, F32, filled_cache, healthy, normal, rng  # noqa: F401
from test_gpu_prefix_attention import pages_needed, shared_table

pytestmark = pytest.mark.gpu

HOLDS = dict(queries=1, full=2, empty=3, mask=4, scores=5, weights=6, reference=7, flushed=8, end=9)


@pytest.fixture
def hold():
    """hold(barrier, limit): barrier 0 is none, limit 0 the ordinary one."""
    whole, call = _lib.lib.bq_internal_prefix_whole_limit, _lib.lib.bq_internal_prefix_hold
    whole.restype, whole.argtypes = ctypes.c_int64, [ctypes.c_int64]
    call.restype, call.argtypes = ctypes.c_int, [ctypes.c_int, ctypes.c_ulonglong]
    whole(0)
    yield call
    assert call(0, 0) == 0
    whole(-1)


@pytest.mark.parametrize("kind,dtype,page", [("f16", F16, 16), ("f16", F32, 7), ("bf16", BF16, 16), ("bf16", F32, 64),
                                             ("q8_0", F32, 16), ("q8_0", BF16, 24)])
def test_waits_run_out_and_are_reported(hold, kind, dtype, page):
    """Copies by tensor maps and by 16 bytes, and codes put into parts: as many kv heads as
    the GPU has places, so that a chunk is all 2048 positions and every barrier is used."""
    g = rng("waits", kind, str(dtype))
    requests, kv, D, shared = 40, 152, 64, 2048 // page * page
    lens = [shared + 1 + b % 5 for b in range(requests)]
    pages = pages_needed(lens, [(requests, shared)], page)
    cache = filled_cache(g, kind, pages, page, kv, D)
    table = shared_table(g, lens, [(requests, shared)], page, pages)
    q = normal(g, (requests, kv, D), dtype)
    at = torch.tensor(lens, dtype=torch.int32, device=DEV)
    want = bq.paged_prefix_attention(cache, q, table, at, shared)
    assert bq.device_status(clear=True) == 0
    for name, barrier in HOLDS.items():
        assert hold(barrier, 2_000_000) == 0
        bq.paged_prefix_attention(cache, q, table, at, shared)
        assert bq.device_status(clear=True) == _lib.BQ_DEVERR_WAIT, name
        assert hold(0, 0) == 0
        assert torch.equal(bq.paged_prefix_attention(cache, q, table, at, shared), want), name
        assert bq.device_status(clear=True) == 0
