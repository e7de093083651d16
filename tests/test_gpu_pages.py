"""Pages that requests share: steps with forks against a plain form, copies in all
layers, compaction, and a server's life of them together, whose requests must read
back their own tokens."""
import ctypes

import numpy as np
import pytest
import torch

import block_quantized_weight_dequant_gb300 as bq

import pages_plain as plain
from test_gpu_cache import DEV, F16, F32, filled_cache, healthy, normal, rng  # noqa: F401

pytestmark = pytest.mark.gpu
I32 = dict(dtype=torch.int32, device=DEV)


def cuda(x, dtype=torch.int32):
    return torch.from_numpy(np.ascontiguousarray(x)).to(dtype).to(DEV)


class State:
    """The host's picture of a server's tables beside the GPU's."""

    def __init__(self, n, width, pool, page, order=None):
        self.page = page
        self.lens, self.table = np.zeros(n, np.int32), np.full((n, width), -1, np.int32)
        self.free = (np.arange(pool)[::-1] if order is None else order).astype(np.int32)
        self.count, self.refs = pool, np.zeros(pool, np.int32)

    def step(self, new, parents=None, room=4096, in_place=True, stride=None):
        n, pool = self.lens.size, self.refs.size
        par = np.full(n, -1, np.int32) if parents is None else np.asarray(parents, np.int32)
        new = np.asarray(new, np.int32)
        want = plain.shared_tables(self.lens, new, par, self.table, self.free, self.count, self.refs, self.page, room)
        lens, table, free, refs = cuda(self.lens), cuda(self.table), cuda(self.free), cuda(self.refs)
        if stride:
            wide = torch.full((n, stride), 77, **I32)
            wide[:, :table.shape[1]] = table
            table = wide[:, :table.shape[1]]
        count = torch.tensor([self.count], **I32)
        slots, positions = torch.full((room,), 7, dtype=torch.int64, device=DEV), torch.full((room,), 7, **I32)
        starts = torch.full((n + 1,), 7, **I32)
        lens_out, count_out = (lens, count) if in_place else (torch.empty_like(lens), torch.empty_like(count))
        src, dst, copies = torch.full((n,), 7, **I32), torch.full((n,), 7, **I32), torch.full((1,), 7, **I32)
        refused = bq.kv_shared_tables(lens, cuda(new), table, free, count, refs, self.page, slots, positions, starts, src,
                                      dst, copies, parents=None if parents is None else cuda(par),
                                      lens_out=None if in_place else lens_out,
                                      free_count_out=None if in_place else count_out)
        pairs = want[9] + [(-1, -1)] * (n - len(want[9]))
        got = (table, free, refs, slots, positions, starts, lens_out, count_out, refused, src, dst, copies)
        expected = want[:7] + ([want[7]], [want[8]], [a for a, _ in pairs], [b for _, b in pairs], [len(want[9])])
        names = "table free refs slots positions starts lens count refused src dst copies".split()
        for name, g, w in zip(names, got, expected):
            g = g.cpu().numpy()
            assert np.array_equal(g, np.asarray(w).reshape(g.shape)), (name, g, w)
        if not in_place:
            assert np.array_equal(lens.cpu().numpy(), self.lens) and int(count) == self.count
        if stride:
            assert (wide[:, self.table.shape[1]:] == 77).all()
        self.table, self.free, self.refs, self.lens, self.count = want[0], want[1], want[2], want[6], want[7]
        self.consistent()
        return want

    def consistent(self):
        held = [self.table[b, j] for b in range(self.lens.size) for j in range(-(-int(self.lens[b]) // self.page))]
        counts = np.bincount(np.asarray(held, np.int64), minlength=self.refs.size)
        assert np.array_equal(counts, self.refs)
        free = np.sort(self.free[:self.count])
        assert np.array_equal(free, np.flatnonzero(self.refs == 0))

    def compact(self, room):
        want = plain.compact(self.lens, self.table, self.free, self.refs, self.page, room)
        pool = self.refs.size
        table, free, refs = cuda(self.table), cuda(self.free), cuda(self.refs)
        count = torch.tensor([self.count], **I32)
        src, dst, copies = torch.full((room,), 7, **I32), torch.full((room,), 7, **I32), torch.full((1,), 7, **I32)
        moved = torch.full((pool,), 7, **I32)
        bq.kv_compact(cuda(self.lens), table, free, count, refs, self.page, src, dst, copies, moved)
        pairs = want[4] + [(-1, -1)] * (room - len(want[4]))
        for name, g, w in (("table", table, want[0]), ("free", free, want[1]), ("refs", refs, want[2]),
                           ("count", count, [want[3]]), ("src", src, [a for a, _ in pairs]),
                           ("dst", dst, [b for _, b in pairs]), ("copies", copies, [len(want[4])]), ("moved", moved, want[5])):
            g = g.cpu().numpy()
            assert np.array_equal(g, np.asarray(w).reshape(g.shape)), (name, g, w)
        self.table, self.free, self.refs, self.count = want[:4]
        self.consistent()
        return want


@pytest.mark.parametrize("page", [1, 4, 16, 33])
def test_forks_grow_part_and_end(page):
    """One request forked at its length, below it, at page borders and to nothing; the
    forks part, shrink into what they share and end one by one."""
    s = State(8, 40, 400, page, order=rng("order", page).permutation(400))
    none = [-1] * 8
    s.step([3 * page + 1, 0, 0, 0, 0, 0, 0, 2])
    # of request 0: at its length, one position on, at a border, below one, at nothing, far on
    s.step([3 * page + 2, 3 * page + 1, 3 * page + 2, 2 * page, max(1, page - 1), 0, 6 * page, 2],
           [-1, 0, 0, 0, 0, 0, 0, -1])
    s.step(s.lens + 1, none)
    s.step(s.lens + 1)
    s.step(np.maximum(s.lens - page, 0))  # back into shared pages
    s.step(s.lens + 1)
    for b in (0, 3, 1):
        new = s.lens + 1
        new[b] = 0
        s.step(new)
    s.step([0] * 8)
    assert s.count == 400


def test_a_fork_of_a_request_that_ends_or_shrinks_in_the_same_step():
    s = State(6, 10, 60, 4)
    s.step([11, 9, 0, 0, 0, 0])
    s.step([0, 3, 11, 12, 9, 2], [-1, -1, 0, 0, 1, 1])
    s.step([0, 3, 0, 0, 0, 0])
    s.step([0, 0, 0, 0, 0, 0])
    assert s.count == 60


def test_all_holders_of_a_page_part_at_once():
    s = State(5, 6, 30, 8)
    s.step([5, 0, 0, 0, 0])
    s.step([5, 5, 5, 5, 5], [-1, 0, 0, 0, 0])
    assert s.refs.max() == 5
    want = s.step([6, 6, 6, 6, 6])
    assert len(want[9]) == 5 and s.refs.max() == 1  # the page that they held is free again


def test_refusals_keep_what_there_was():
    s = State(6, 8, 10, 4)
    s.step([17, 0, 0, 0, 0, 6])
    # 5 + 2 pages held, 3 free: the fork that grows asks for 2 (its copy and one page), the next for 2
    want = s.step([17, 21, 21, 17, 9, 6], [-1, 0, 0, 0, -1, -1])
    assert want[8] >= 1 and s.lens[2] == 0
    s.step([18, 22, 2, 17, 0, 0], [-1, -1, 5, -1, -1, -1])
    before = s.lens.copy()
    # forks of itself, of a fork, of nobody, over a request that holds pages; lengths out of range
    s.lens = before
    want = s.step([17, 22, 33, 17, -1, 3], [-1, -1, 2, 9, -1, 4])
    assert want[8] >= 3
    # rows beyond the room
    s.step([0] * 6)
    want = s.step([9, 9, 9, 0, 0, 0], room=20)
    assert want[8] == 1 and list(want[6]) == [9, 9, 0, 0, 0, 0]
    want = s.step([9, 9, 0, 12, 0, 0], [-1, -1, -1, 0, -1, -1], room=2)
    assert want[8] == 1 and s.lens[3] == 0


@pytest.mark.parametrize("n,width,page,pool,room", [(1, 1, 1, 1, 1), (3, 7, 2, 40, 8), (40, 30, 8, 700, 600),
                                                    (700, 50, 16, 9000, 6000), (130, 400, 4, 60000, 4096)])
def test_random_steps(n, width, page, pool, room):
    """A server at random: prompts, decode, forks, rollbacks, ends, pools that run out."""
    g = rng("steps", n, width)
    s = State(n, width, pool, page, order=g.permutation(pool))
    most = width * page
    for step in range(14):
        kind = g.random(n)
        new = s.lens + 1
        parents = np.full(n, -1, np.int32)
        empty = np.flatnonzero(s.lens == 0)
        alive = np.flatnonzero(s.lens > 0)
        for b in empty:
            if alive.size and kind[b] < 0.5:
                parents[b] = g.choice(alive)
                new[b] = max(0, int(s.lens[parents[b]]) + int(g.integers(-3 * page, 2 * page)))
            else:
                new[b] = int(g.integers(0, max(2, most // 3)))
        for b in alive:
            if kind[b] < 0.12:
                new[b] = 0
            elif kind[b] < 0.25:
                new[b] = max(0, int(s.lens[b]) - int(g.integers(0, 3 * page)))
            elif kind[b] > 0.9:
                new[b] = min(most, int(s.lens[b]) + int(g.integers(0, 2 * page)))
        s.step(np.minimum(new, most), parents if step % 3 else None if step == 0 else parents, room=room,
               in_place=step % 2 == 0, stride=width + 5 if step % 4 == 1 else None)
        if step % 5 == 4:
            s.compact([max(1, pool // 2), 3, pool][step // 5 % 3])


@pytest.mark.parametrize("pool", [1, 2, 31, 32, 33, 1000, 4097, 100003])
@pytest.mark.parametrize("used", [0.0, 0.1, 0.5, 0.9, 1.0])
def test_compaction(pool, used):
    g = rng("compact", pool, int(used * 10))
    count = int(used * pool)
    order = g.permutation(pool)
    n = 3
    s = State(n, pool + 1, pool, 2)
    cut = [0, count // 3, count // 2, count]
    for b in range(n):
        row = order[cut[b]:cut[b + 1]]
        s.table[b, :row.size] = row
        s.lens[b] = max(0, 2 * row.size - (b == 1 and row.size > 0))
        s.refs[row] += 1
    if cut[2] > cut[1]:  # request 0 holds some of request 1's pages too
        both = s.table[1, :min(5, cut[2] - cut[1])]
        s.table[0, cut[1]:cut[1] + both.size] = both
        s.lens[0] += 2 * both.size
        s.refs[both] += 1
    rest = np.setdiff1d(np.arange(pool), order[:count])
    s.free[:rest.size], s.count = g.permutation(rest), rest.size
    limited = s.compact(max(1, pool // 7))
    s.compact(max(1, pool // 2))
    assert (s.refs[:count] > 0).all() and (s.refs[count:] == 0).all()
    assert len(limited[4]) <= max(1, pool // 7)
    assert len(s.compact(0)[4]) == 0


@pytest.mark.parametrize("kind", ["f16", "bf16", "q8_0"])
@pytest.mark.parametrize("layout", ["hs", "sh", "kv"])
@pytest.mark.parametrize("page,kv,D", [(16, 8, 128), (1, 1, 32), (7, 3, 96), (24, 2, 256), (64, 5, 64)])
def test_copies(kind, layout, page, kv, D):
    g = rng("copy", kind, layout, page)
    caches = [filled_cache(g, kind, 21, page, kv, D, layout) for _ in range(3)]
    if kind == "q8_0" and caches[0].v_scale.data_ptr() % 8:  # refused, as by every call on a cache
        with pytest.raises(bq.BQError):
            bq.kv_copy_pages(caches, cuda([1]), cuda([2]))
        return
    order = g.permutation(21)
    src, dst = order[:9].copy(), order[9:18].copy()
    src[2], dst[4] = -1, -5  # skipped
    dst[6] = src[6]  # as it is
    kept = [[t.clone() for t in (c.k, c.v) + (() if c.k_scale is None else (c.k_scale, c.v_scale))] for c in caches]
    for count in (None, 4, 0, 100, -3):
        n = 9 if count is None else min(9, max(0, count))
        for planes in kept:
            for t in planes:
                for a, b in zip(src[:n], dst[:n]):
                    if a >= 0 and b >= 0:
                        t[b] = t[a].clone()
        bq.kv_copy_pages(caches, cuda(src), cuda(dst), None if count is None else torch.tensor([count], **I32))
        for c, planes in zip(caches, kept):
            now = (c.k, c.v) + (() if c.k_scale is None else (c.k_scale, c.v_scale))
            assert all(torch.equal(a.view(torch.uint8) if a.is_contiguous() else a, b.view(torch.uint8) if a.is_contiguous()
                                   else b) for a, b in zip(now, planes))
    bq.kv_copy_pages(caches[0], cuda([order[18]]), cuda([order[19]]))
    assert torch.equal(caches[0].k[order[19]], caches[0].k[order[18]])
    bq.kv_copy_pages(caches, cuda([]), cuda([]))
    bq.kv_copy_pages([], cuda([]), cuda([]))


def test_copies_of_many_layers_and_of_any_bits():
    """More caches than one launch takes; NaNs and both zeros stay as they are."""
    caches = [bq.PagedKVCache.zeros(4, 8, 1, 64) for _ in range(200)]
    for i, c in enumerate(caches):
        c.k[1] = i
        c.v.view(torch.int16)[2] = torch.arange(512, device=DEV, dtype=torch.int32).to(torch.int16).view(1, 8, 64) * 128 - i
    bq.kv_copy_pages(caches, cuda([1, 2]), cuda([0, 3]))
    for i, c in enumerate(caches):
        assert (c.k[0] == i).all() and torch.equal(c.v.view(torch.int16)[3], c.v.view(torch.int16)[2])


def test_pages_outside_the_pool_are_reported():
    caches = [bq.PagedKVCache.zeros(4, 8, 1, 64)]
    caches[0].k[1] = 5
    bq.kv_copy_pages(caches, cuda([1, 9, 1]), cuda([0, 2, 4]))
    assert bq.device_status(clear=True) == 0x100
    assert (caches[0].k[0] == 5).all() and (caches[0].k[2:] == 0).all()
    # a row whose entries are not pages, shared and given up; a free count out of range
    t = bq.SharedBlockTables(3, 4, 20, 4, 16)
    t.resize(cuda([9, 0, 0]))
    t.table[0, 1] = 99
    t.resize(cuda([9, 10, 0]), cuda([-1, 0, -1]))
    assert bq.device_status(clear=True) == 0x100
    t.resize(cuda([0, 10, 0]))
    assert bq.device_status(clear=True) == 0x100
    moved = t.compact()
    assert bq.device_status(clear=True) == 0x100
    assert moved.numel() == 20
    t.free_count.fill_(21)
    t.resize(cuda([0, 10, 0]))
    assert bq.device_status(clear=True) == 0x800


@pytest.mark.parametrize("kind", ["f16", "q8_0"])
def test_a_server_of_forks_reads_back_its_tokens(kind):
    """Prompts, forks, decode, rollback, compaction, over two layers: what attention
    reads through the tables is what each request appended, whoever else shares it,
    and attention over the shared prefix agrees with attention of each request."""
    g = rng("server", kind)
    kv, D, heads, page, pool, n = 2, 64, 4, 8, 300, 7
    caches = [bq.PagedKVCache.zeros(pool, page, kv, D, kind) for _ in range(2)]
    t = bq.SharedBlockTables(n, 40, pool, page, 512, caches)
    twin = bq.PagedKVCache.zeros(n * 40, page, kv, D, kind)  # every request by itself
    own = torch.arange(n * 40, **I32).view(n, 40)
    lens = np.zeros(n, np.int64)

    def step(new, parents=None):
        new = np.asarray(new)
        old = lens.copy()
        assert int(t.resize(cuda(new), None if parents is None else cuda(parents))) == 0
        for b in range(n):
            p = -1 if parents is None else parents[b]
            if p >= 0:  # the twin's fork holds copies of everything
                for x in (twin.k, twin.v) + (() if kind == "f16" else (twin.k_scale, twin.v_scale)):
                    x[own[b].long()] = x[own[p].long()]
                old[b] = min(lens[p], new[b])
        rows = int(np.maximum(new - old, 0).sum())
        k, v = normal(g, (rows, kv, D)), normal(g, (rows, kv, D))
        for i, c in enumerate(caches):
            bq.kv_append(c, k * (i + 1), v, t.slots[:rows])
        at = np.concatenate([np.arange(a, max(a, z)) + b * 40 * page for b, (a, z) in enumerate(zip(old, new))])
        bq.kv_append(twin, k, v, cuda(at, torch.int64))
        lens[:] = new

    def same():
        q = normal(g, (n, heads, D))
        at = cuda(lens)
        want = bq.paged_attention(twin, q, own, at)
        assert torch.equal(bq.paged_attention(caches[0], q, t.table, t.lens), want)
        assert torch.equal(bq.paged_attention(caches[1], q / 2, t.table, t.lens), want)
        shared = 60  # of requests 0 to 4 since the first forks
        if (lens[:5] > shared).all():
            got = bq.paged_prefix_attention(caches[0], q, t.table, t.lens, [(5, shared), (2, 0)])
            # both forms are within 2^-13 of a mean of |v| (below 1.5) of the exact value
            assert float((got - want).abs().max()) <= 2.0 ** -12 * 1.5

    step([61, 0, 0, 0, 0, 30, 0])
    same()
    step([62, 62, 62, 70, 61, 31, 0], [-1, 0, 0, 0, 0, -1, -1])
    same()
    for _ in range(9):
        step(lens + (lens > 0))
        same()
    step([71, 63, 66, 75, 70, 0, 66], [-1, -1, -1, -1, -1, -1, 2])  # rollbacks, an end, a fork of a fork
    same()
    t.compact()
    same()
    step(lens + (lens > 0))
    same()
    t.compact(3)
    step([0, 64, 67, 0, 71, 9, 67])
    t.compact()
    step(lens + (lens > 0))
    same()
    step([0] * n)
    assert int(t.free_count) == pool and (t.refs == 0).all()


@pytest.mark.parametrize("limit", [0, -1])
def test_a_decode_of_forks_over_their_shared_prefix(limit):
    """A prompt, three forks of it and steps of all four with the prefix given: the
    logits of steps that know nothing of it."""
    from block_quantized_weight_dequant_gb300 import _lib, workloads as wl
    from test_gpu_paged_decode import HIDDEN, decoder

    hook = _lib.lib.bq_internal_prefix_whole_limit
    hook.restype, hook.argtypes = ctypes.c_int64, [ctypes.c_int64]
    h = wl.normal_torch((48, HIDDEN), 1.0, seed=3, stream=14, device=DEV)
    out = []
    for shared in (None, 20):
        one, four = decoder("q8_0", "f16"), decoder("q8_0", "f16", rows=4)
        four.caches = one.caches
        t = bq.SharedBlockTables(4, 8, 12, 16, 8, one.caches)
        for i in range(20):
            t.resize(cuda([i + 1, 0, 0, 0]))
            one.step(h[i:i + 1], t.slots[:1], t.positions[:1], t.table[:1], t.lens[:1])
        hook(limit)
        try:
            for i in range(7):
                parents = cuda([-1, 0, 0, 0]) if i == 0 else None
                assert int(t.resize(cuda([21 + i] * 4), parents)) == 0
                rows = h[20 + 4 * i:24 + 4 * i]
                out.append(four.step(rows, t.slots[:4], t.positions[:4], t.table, t.lens, shared=shared).clone())
        finally:
            hook(-1)
    a, b = torch.stack(out[:7]), torch.stack(out[7:])
    if limit:  # so little is read again that the ordinary kernel serves the call: the same bits
        assert torch.equal(a, b)
    # else the attention outputs differ in the last bits of fp32 (2^-13 of them at most) and
    # keys or values next to a rounding border of the fp16 cache by 2^-11: as in the decoder's
    # own test that moves a logit by less than 2^-12 * 16 of their rms
    assert float((a - b).abs().max()) <= 2.0 ** -12 * 16 * float(a.square().mean().sqrt())


def test_captured_steps():
    """A step with forks, its copies and a compaction in one graph, replayed over new
    lengths and parents, against the same calls made one by one."""
    def made():
        caches = [bq.PagedKVCache.zeros(64, 4, 1, 32) for _ in range(3)]
        for c in caches:
            c.k.copy_(torch.arange(64, device=DEV).view(64, 1, 1, 1).expand_as(c.k))
        return bq.SharedBlockTables(5, 12, 64, 4, 64, caches)

    steps = [([13, 0, 0, 2, 0], [-1] * 5), ([14, 14, 13, 3, 0], [-1, 0, 0, -1, -1]), ([15, 2, 14, 0, 3], [-1, -1, -1, -1, 3]),
             ([0, 3, 15, 9, 4], [-1, -1, -1, 1, -1])]
    eager, t = made(), made()
    new, parents = torch.zeros(5, **I32), torch.full((5,), -1, **I32)
    t.resize(new, parents)  # (nothing: the first call outside the capture)
    t.compact()
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        t.resize(new, parents)
        moved = t.compact()
    for z, p in steps:
        new.copy_(cuda(z))
        parents.copy_(cuda(p))
        graph.replay()
        eager.resize(cuda(z), cuda(p))
        assert torch.equal(eager.compact(), moved)
        for a in ("lens", "table", "free_pages", "free_count", "refs", "copy_src", "copy_dst", "copy_count", "slots"):
            assert torch.equal(getattr(t, a), getattr(eager, a)), a
        assert all(torch.equal(a.k, b.k) for a, b in zip(t.caches, eager.caches))


def test_limits_of_a_step():
    """The most requests, a slot map of its own kernel, nothing at all."""
    n = 4096
    s = State(n, 3, 9000, 4)
    lens = np.zeros(n, np.int32)
    lens[::2] = 7
    s.step(lens, room=16000)
    parents = np.full(n, -1, np.int32)
    parents[1::2] = np.arange(0, n, 2)
    s.step(np.where(parents >= 0, 8, lens), parents, room=9000)
    s.step(np.where(np.arange(n) % 3 == 0, 0, s.lens), room=0)
    empty = torch.zeros(0, **I32)
    starts = torch.zeros(1, **I32)
    count, copies = torch.tensor([3], **I32), torch.full((1,), 9, **I32)
    out = bq.kv_shared_tables(empty, empty, torch.zeros(0, 4, **I32), torch.zeros(3, **I32), count, torch.zeros(3, **I32), 4,
                              torch.zeros(0, dtype=torch.int64, device=DEV), empty, starts, empty, empty, copies)
    assert int(out) == 0 and int(copies) == 0 and int(count) == 3


def test_refusals():
    t = bq.SharedBlockTables(3, 4, 20, 4, 16)
    good = (t.lens, t.lens.clone(), t.table, t.free_pages, t.free_count, t.refs, 4, t.slots, t.positions, t.starts, t.copy_src,
            t.copy_dst, t.copy_count)
    for i, bad in ((1, t.lens[:2]), (2, t.table[:2]), (5, t.refs[:5]), (10, t.copy_src[:1]), (12, t.lens)):
        with pytest.raises(ValueError):
            bq.kv_shared_tables(*good[:i], bad, *good[i + 1:])
    for more in (dict(parents=t.lens[:1]), dict(parents=t.lens.long())):
        with pytest.raises((ValueError, TypeError)):
            bq.kv_shared_tables(*good, **more)
    with pytest.raises(bq.BQError):
        bq.kv_shared_tables(*good[:6], 0, *good[7:])
    new = t.lens.clone()
    with pytest.raises(bq.BQError):
        bq.kv_shared_tables(t.lens, new, *good[2:], lens_out=new)
    caches = [bq.PagedKVCache.zeros(4, 8, 1, 64), bq.PagedKVCache.zeros(5, 8, 1, 64)]
    one = torch.zeros(1, **I32)
    with pytest.raises(bq.BQError):
        bq.kv_copy_pages(caches, one, one)
    with pytest.raises(TypeError):
        bq.kv_copy_pages([None], one, one)
    with pytest.raises(ValueError):
        bq.kv_copy_pages(caches[0], one, torch.zeros(2, **I32))
    with pytest.raises(ValueError):
        bq.kv_copy_pages(caches[0], one, one, count=torch.zeros(2, **I32))
    with pytest.raises(ValueError):
        bq.SharedBlockTables(3, 4, 20, 4, 16, caches)
    with pytest.raises(ValueError):
        bq.kv_compact(t.lens, t.table, t.free_pages, t.free_count, t.refs, 4, one, torch.zeros(2, **I32), one.clone(), t.refs)


def test_the_readmes_example_of_a_shared_prompt():
    import os
    import re

    import paged_plain

    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    with open(os.path.join(root, "README.md")) as f:
        first, second = re.findall(r"```python\n(.*?)```", f.read(), flags=re.S)[:2]
    said = {}
    exec(first + second, said)
    n, lens = said["requests"], [said["prompt"] + 1] * said["requests"]
    table, cache, q = said["shared"].table.cpu(), said["cache"], said["q"]
    want, mag, top = paged_plain.attention(*paged_plain.values(cache), q.cpu(), table, lens, 1, cache.head_dim ** -0.5)
    bound = paged_plain.attention_bound(want, mag, top, F32, False)
    assert ((said["out"].cpu().double() - want).abs() <= bound).all()
    # 40 positions in 2 whole pages and a half: the forks share two and have one of their own
    assert int(said["shared"].refs.max()) == n and int(said["shared"].free_count) == 64 - 2 - n
