"""Lengths at their ends in attention over shared pages."""
import pytest
import torch

import block_quantized_weight_dequant_gb300 as bq

from test_gpu_cache import BF16, DEV, F16, F32, filled_cache, healthy, normal, rng  # noqa: F401
from test_gpu_prefix_attention import limit, pages_needed, shared_table  # noqa: F401

pytestmark = pytest.mark.gpu
KINDS = [("f16", F32, 4), ("bf16", BF16, 4), ("q8_0", F32, 4), ("q8_0", BF16, 40), ("f16", F16, 40)]


@pytest.mark.parametrize("kind,dtype,heads", KINDS)
@pytest.mark.parametrize("rows", [1, 2, 6])
@pytest.mark.parametrize("bad", [-(1 << 31), -(1 << 31) + 4, -1])
def test_a_length_below_zero_is_none_whatever_its_size(kind, dtype, heads, rows, bad):
    """It counts as 0: its request gives zeros, and the shared pages are not looked up in
    its row, although it is the group's first."""
    g = rng("below", kind, heads, rows)
    page, shared = 16, 320
    lens = [0, shared + rows, shared + rows + 9]
    pages = pages_needed(lens, [(3, shared)], page)
    cache = filled_cache(g, kind, pages, page, 1, 64)
    table = shared_table(g, lens, [(3, shared)], page, pages)
    q = normal(g, (3 * rows, heads, 64), dtype)
    at = torch.tensor(lens, dtype=torch.int32, device=DEV)
    want = bq.paged_prefix_attention(cache, q, table, at, shared, rows=rows)
    assert bq.device_status(clear=True) == 0 and (want[:rows] == 0).all()
    at[0] = bad
    got = bq.paged_prefix_attention(cache, q, table, at, shared, rows=rows)
    assert bq.device_status(clear=True) == 0x200
    assert torch.equal(got, want)
