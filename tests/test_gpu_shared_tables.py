"""SharedBlockTables and the calls on shared pages at their ends: captured calls beside
others, caches that do not fit, pools beyond what one pass keeps in mind."""
import numpy as np
import pytest
import torch

import block_quantized_weight_dequant_gb300 as bq

import pages_plain
from test_gpu_cache import DEV, healthy, rng  # noqa: F401

pytestmark = pytest.mark.gpu
I32 = dict(dtype=torch.int32, device=DEV)


def cuda(x, dtype=torch.int32):
    return torch.as_tensor(np.asarray(x), dtype=dtype, device=DEV)


def test_a_captured_compaction_after_eager_ones_of_fewer_moves():
    """A graph of a compaction goes on after calls with other max_moves: it finds its
    lists, and writes nothing that was allocated since."""
    def made():
        caches = [bq.PagedKVCache.zeros(64, 4, 1, 32) for _ in range(2)]
        for c in caches:
            c.k.copy_(torch.arange(64, device=DEV).view(64, 1, 1, 1).expand_as(c.k))
        return bq.SharedBlockTables(5, 12, 64, 4, 64, caches)

    t, twin = made(), made()
    t.compact()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        moved = t.compact()
    for most in (3, 0, 32):
        t.compact(most)
    others = [torch.full((n,), 7, **I32) for n in (32, 32, 1, 64) * 8]
    for lens in ([40, 9, 20, 0, 31], [0, 9, 20, 14, 0], [3, 0, 24, 14, 9], [0, 0, 0, 0, 40]):
        t.resize(cuda(lens))
        twin.resize(cuda(lens))
        graph.replay()
        assert torch.equal(twin.compact(), moved)
        for a in ("lens", "table", "free_pages", "free_count", "refs"):
            assert torch.equal(getattr(t, a), getattr(twin, a)), a
        assert all(torch.equal(a.k, b.k) for a, b in zip(t.caches, twin.caches))
    assert all((x == 7).all() for x in others)


def test_caches_that_a_step_could_not_copy_in_are_refused_when_the_tables_are_made():
    good = bq.PagedKVCache.zeros(20, 4, 2, 64)
    other = [bq.PagedKVCache.zeros(20, 4, 1, 64), bq.PagedKVCache.zeros(20, 4, 2, 32),
             bq.PagedKVCache.zeros(20, 4, 2, 64, "bf16"),
             bq.PagedKVCache(*[torch.zeros(20, 4, 2, 64, dtype=torch.float16, device=DEV).transpose(1, 2) for _ in "kv"])]
    for bad in other:
        with pytest.raises(bq.BQError):
            bq.SharedBlockTables(3, 4, 20, 4, 16, [good, bad])
    with pytest.raises(TypeError):
        bq.SharedBlockTables(3, 4, 20, 4, 16, [good, None])
    t = bq.SharedBlockTables(3, 4, 20, 4, 16, [good, bq.PagedKVCache.zeros(20, 4, 2, 64)])
    assert int(t.resize(cuda([5, 0, 1]))) == 0


@pytest.mark.parametrize("pool", [2048 * 32 * 16, 2048 * 32 * 16 + 1, 1300003])
@pytest.mark.parametrize("used", [0.3, 0.97])
def test_compaction_of_pools_beyond_the_bits_it_keeps(pool, used):
    """Beyond 2048 pages for each warp of 16 CTAs the counts are read again in place of bits
    kept of them: all moves, few of them, and no page left in its place."""
    g = rng("large", pool, int(used * 100))
    count, page = int(used * pool), 2
    order = g.permutation(pool)
    cut = [0, count // 2, count - 5, count]
    table = np.full((3, count // 2 + 9), -1, np.int32)
    lens, refs = np.zeros(3, np.int32), np.zeros(pool, np.int32)
    for b in range(3):
        row = order[cut[b]:cut[b + 1]]
        table[b, :row.size], lens[b] = row, 2 * row.size - 1
        refs[row] += 1
    refs[order[:7]] += 1  # some are held twice
    free = np.full(pool, -1, np.int32)
    free[:pool - count] = order[count:]
    for room in (pool // 9, pool // 2, 3):
        want = pages_plain.compact(lens, table, free, refs, page, room)
        t, f, r = cuda(table), cuda(free), cuda(refs)
        src, dst, moved = (torch.empty(k, **I32) for k in (room, room, pool))
        copies, left = torch.empty(1, **I32), torch.empty(1, **I32)
        bq.kv_compact(cuda(lens), t, f, cuda([pool - count]), r, page, src, dst, copies, moved, free_count_out=left)
        assert bq.device_status(clear=True) == 0
        n = len(want[4])
        assert int(copies) == n and int(left) == want[3]
        assert torch.equal(torch.stack([src, dst]), cuda(np.array(want[4] + [(-1, -1)] * (room - n)).T))
        for got, told in ((t, want[0]), (f, want[1]), (r, want[2]), (moved, want[5])):
            assert torch.equal(got, cuda(told))
        table, free, refs = want[0], want[1], want[2]
    assert (refs[:count] > 0).all() and (refs[count:] == 0).all()
