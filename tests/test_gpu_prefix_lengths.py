"""Lengths at their ends in attention over shared pages: out of range, and shorter than
the call's rows."""
import pytest
import torch

import block_quantized_weight_dequant_gb300 as bq

from test_gpu_cache import BF16, DEV, F16, F32, filled_cache, healthy, normal, rng  # noqa: F401
from test_gpu_prefix_attention import case, limit, pages_needed, shared_table  # noqa: F401

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


@pytest.mark.parametrize("kind,dtype,heads", KINDS)
@pytest.mark.parametrize("rows", [2, 4, 6])
def test_requests_shorter_than_the_rows_where_no_page_is_shared(kind, dtype, heads, rows):
    """With nothing shared there is nothing to see: the last rows have their positions, as
    in the ordinary call, and nothing is reported."""
    for shared in (0, 15, [(2, 0), (0, 64), (3, 15), (2, 0)], [(2, 0), (3, 320), (2, 9)]):
        lens = [1, rows, 0, rows - 1, 3, 2, 1]
        if shared == [(2, 0), (3, 320), (2, 9)]:
            lens[2:5] = [0, 320 + rows, 340]
        g = rng("short", kind, heads, rows)
        case(g, kind, dtype, lens, shared, 16, heads, 1, 64, rows=rows, width=23)  # (groups share no more than it holds)
        assert bq.device_status(clear=True) == 0
