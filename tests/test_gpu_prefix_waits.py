"""The waits of the attention over shared pages: a bounded one that nothing ends runs out
within its limit, the kernel says so and returns, and the next call is as before; calls of
two threads on one stream."""
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


@pytest.mark.parametrize("kind,dtype", [("f16", F16), ("bf16", BF16), ("q8_0", F32)])
def test_two_threads_on_one_stream(hold, kind, dtype):
    """Steps of two caches, each appended and attended by a thread of its own on the same
    stream: launches of the one come between those of the other's calls."""
    import threading

    g = rng("threads", kind)
    requests, heads, kv, D, page, shared, steps = 40, 8, 2, 128, 16, 1040, 30
    whole, stream = shared // page, torch.cuda.Stream()
    sides = []
    for side in range(2):
        cache = filled_cache(g, kind, whole + 4 * requests, page, kv, D)
        table = torch.arange(whole, dtype=torch.int32).expand(requests, -1)
        table = torch.cat([table, whole + torch.arange(4 * requests, dtype=torch.int32).view(requests, 4)], 1).to(DEV)
        k, v = (normal(g, (steps, requests, kv, D), dtype) for _ in range(2))
        q = normal(g, (steps, requests, heads, D), dtype)
        slots = [table[:, (shared + i) // page].long() * page + (shared + i) % page for i in range(steps)]
        lens = [torch.full((requests,), shared + i + 1, dtype=torch.int32, device=DEV) for i in range(steps)]
        room = torch.empty(bq.paged_prefix_attention_workspace(cache, requests, 1, heads, whole + 4, shared, dtype),
                           dtype=torch.uint8, device=DEV)
        out = torch.empty(2, steps, requests, heads, D, dtype=dtype, device=DEV)
        sides.append((cache, table, k, v, q, slots, lens, room, out))

    def run(side, turn, wait):
        cache, table, k, v, q, slots, lens, room, out = sides[side]
        with torch.cuda.stream(stream):
            for i in range(steps):
                bq.kv_append(cache, k[i], v[i], slots[i])
                wait()
                bq.paged_prefix_attention(cache, q[i], table, lens[i], shared, out=out[turn, i], workspace=room)
                wait()

    torch.cuda.synchronize()
    for side in range(2):
        run(side, 0, torch.cuda.synchronize)
    threads = [threading.Thread(target=run, args=(side, 1, lambda: None)) for side in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    for side in sides:
        assert torch.equal(side[-1][0], side[-1][1])
