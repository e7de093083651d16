"""The calls around the paged key-value cache and the block norms on the host,
without a GPU: every refusal of the C ABI and of the binding, the division by a
launch constant, and how attention calls are cut."""
import ctypes
import gc
import os
import re
import threading
import weakref

import pytest
import torch

import block_quantized_weight_dequant_gb300 as bq
from block_quantized_weight_dequant_gb300 import _lib

A = 0x10000  # a well-aligned fake device address; validation must not dereference it
OK, NULL, SHAPE, ALIGN, QTYPE = (_lib.BQ_OK, _lib.BQ_ERR_NULL, _lib.BQ_ERR_SHAPE, _lib.BQ_ERR_ALIGN,
                                 _lib.BQ_ERR_QTYPE)
INF, NAN = float("inf"), float("nan")


@pytest.fixture(scope="module")
def lib():
    return _lib.get()


def cache(kind=_lib.BQ_F16, **over):
    c = dict(type=kind, kv_heads=4, head_dim=128, page_size=16, pages=10, page_stride=8192, head_stride=2048,
             slot_stride=128, k=A, v=A, k_scale=A, v_scale=A)
    c.update(over)
    s = _lib.BqKvCache()
    for n, v in c.items():
        setattr(s, n, v)
    return s


def tables(**over):
    c = dict(requests=0, page_size=16, table_width=8, pool=100, table_stride=8, max_tokens=64, lens=A, new_lens=A + 256,
             table=A, free_pages=A, free_count=A, slots=A, positions=A, starts=A, lens_out=A, free_count_out=A,
             refused=A)
    c.update(over)
    s = _lib.BqKvTables()
    for n, v in c.items():
        setattr(s, n, v)
    return s


def append(**over):
    c = dict(dtype=_lib.BQ_F32, heads=16, rot=128, axes=1, interleaved=0, tokens=0, k=A, v=A, q=A, q_out=A,
             k_token_stride=512, k_head_stride=128, v_token_stride=512, v_head_stride=128, q_token_stride=2048,
             q_head_stride=128, q_out_token_stride=2048, q_out_head_stride=128, slots=A, positions=A,
             position_stride=4, freq=A)
    sections = over.pop("sections", (64, 0, 0))
    c.update(over)
    s = _lib.BqKvAppendArgs()
    for n, v in c.items():
        setattr(s, n, v)
    s.sections[:] = sections
    return s


def attention(**over):
    c = dict(dtype=_lib.BQ_F32, requests=0, rows=1, heads=16, table_width=8, scale=0.1, table_stride=8,
             q_row_stride=2048, q_head_stride=128, out_row_stride=2048, out_head_stride=128, q=A, out=A, table=A,
             lens=A)
    c.update(over)
    s = _lib.BqAttentionArgs()
    for n, v in c.items():
        setattr(s, n, v)
    return s


def sandwich(**over):
    c = dict(dtype=_lib.BQ_F32, h_dtype=_lib.BQ_F32, rows=0, width=64, y=A, h=A, gate=A, post=A, pre=A, h_out=A, x=A,
             y_stride=64, h_stride=64, gate_stride=0, h_out_stride=64, x_stride=64, alpha=1.0, beta=1.0, eps=1e-6)
    c.update(over)
    s = _lib.BqSandwichArgs()
    for n, v in c.items():
        setattr(s, n, v)
    return s


# requests / tokens / rows are 0 in the accepted calls, so nothing is launched
CACHE_BAD = [(dict(type=2), QTYPE), (dict(type=_lib.BQ_F32), QTYPE), (dict(head_dim=0), SHAPE),
             (dict(head_dim=12), SHAPE), (dict(head_dim=264), SHAPE), (dict(kv_heads=0), SHAPE),
             (dict(kv_heads=1025), SHAPE), (dict(page_size=0), SHAPE), (dict(page_size=65537), SHAPE),
             (dict(pages=0), SHAPE), (dict(pages=1 << 31), SHAPE), (dict(page_stride=-8), SHAPE),
             (dict(slot_stride=4), SHAPE), (dict(head_stride=1 << 31), SHAPE),
             (dict(kind=_lib.BQ_Q8_0, head_dim=48), SHAPE), (dict(kind=_lib.BQ_Q8_0, slot_stride=64), SHAPE)]


@pytest.mark.parametrize("over,status", CACHE_BAD)
def test_cache_layouts_are_refused(lib, over, status):
    c = cache(**over)
    assert lib.bq_kv_append(c, append(), None) == status
    assert lib.bq_paged_attention(c, attention(), None, 0, None) == status
    assert lib.bq_paged_attention_workspace_bytes(c, attention()) == -1


@pytest.mark.parametrize("over,status", [
    (dict(dtype=8), QTYPE), (dict(tokens=-1), SHAPE), (dict(tokens=1 << 31), SHAPE), (dict(heads=0), SHAPE),
    (dict(heads=4097), SHAPE), (dict(k_token_stride=-1), SHAPE), (dict(v_head_stride=1 << 31), SHAPE),
    (dict(q_out_head_stride=-1), SHAPE), (dict(rot=8, sections=(4, 0, 0)), SHAPE),
    (dict(rot=24, sections=(12, 0, 0)), SHAPE), (dict(rot=144, sections=(72, 0, 0)), SHAPE), (dict(axes=0), SHAPE),
    (dict(axes=4), SHAPE), (dict(sections=(60, 0, 0)), SHAPE), (dict(axes=3, sections=(80, -16, 0)), SHAPE),
    (dict(position_stride=-1), SHAPE), (dict(tokens=2, k=None), NULL), (dict(tokens=2, v=None), NULL),
    (dict(tokens=2, slots=None), NULL), (dict(tokens=2, q_out=None), NULL), (dict(tokens=2, positions=None), NULL),
    (dict(tokens=2, k=A + 2), ALIGN), (dict(tokens=2, q=A + 1), ALIGN), (dict(tokens=2, slots=A + 4), ALIGN),
    (dict(tokens=2, freq=A + 4), ALIGN), (dict(), OK), (dict(q=None, heads=0, q_out=None), OK),
    (dict(freq=None, rot=3, axes=9, positions=None), OK), (dict(axes=3, sections=(16, 24, 24)), OK)])
def test_append_arguments(lib, over, status):
    assert lib.bq_kv_append(cache(), append(**over), None) == status


def test_append_needs_its_structs_and_the_cache_pointers(lib):
    assert lib.bq_kv_append(None, append(), None) == NULL
    assert lib.bq_kv_append(cache(), None, None) == NULL
    assert lib.bq_kv_append(cache(k=None), append(tokens=1), None) == NULL
    assert lib.bq_kv_append(cache(v=A + 8), append(tokens=1), None) == ALIGN
    assert lib.bq_kv_append(cache(kind=_lib.BQ_Q8_0, k_scale=None), append(tokens=1), None) == NULL
    assert lib.bq_kv_append(cache(kind=_lib.BQ_Q8_0, v_scale=A + 2), append(tokens=1), None) == ALIGN


@pytest.mark.parametrize("over,status", [
    (dict(dtype=2), QTYPE), (dict(requests=-1), SHAPE), (dict(requests=4097), SHAPE), (dict(rows=0), SHAPE),
    (dict(rows=7), SHAPE), (dict(heads=0), SHAPE), (dict(heads=18), SHAPE), (dict(heads=4100), SHAPE),
    (dict(table_width=0), SHAPE), (dict(table_width=(1 << 19) + 1, table_stride=1 << 20), SHAPE),
    (dict(table_stride=7), SHAPE), (dict(scale=NAN), SHAPE), (dict(scale=INF), SHAPE), (dict(q_row_stride=-1), SHAPE),
    (dict(requests=1, q=None), NULL), (dict(requests=1, out=None), NULL), (dict(requests=1, table=None), NULL),
    (dict(requests=1, lens=None), NULL), (dict(requests=1, q=A + 2), ALIGN), (dict(requests=1, lens=A + 1), ALIGN),
    (dict(), OK)])
def test_attention_arguments(lib, over, status):
    assert lib.bq_paged_attention(cache(), attention(**over), None, 0, None) == status


def test_attention_workspace(lib):
    one = attention(requests=1)  # 8 pages of 16: one unit, nothing to join
    assert lib.bq_paged_attention_workspace_bytes(cache(), one) == 0
    long = attention(requests=1, table_width=4096, table_stride=4096)
    need = lib.bq_paged_attention_workspace_bytes(cache(), long)
    assert need > 0
    assert lib.bq_paged_attention(cache(), long, None, 0, None) == NULL
    assert lib.bq_paged_attention(cache(), long, A + 8, need, None) == ALIGN
    assert lib.bq_paged_attention(cache(), long, A, need - 1, None) == SHAPE
    assert lib.bq_paged_attention_workspace_bytes(cache(), attention(rows=9)) == -1
    assert lib.bq_paged_attention_workspace_bytes(None, one) == -1


@pytest.mark.parametrize("requests,kv_heads,width", [(1, 4, 8), (1, 4, 64), (1, 4, 100), (1, 8, 4096), (3, 8, 70),
                                                     (48, 8, 800), (256, 1, 20), (4096, 2, 9)])
@pytest.mark.parametrize("kind", [_lib.BQ_F16, _lib.BQ_BF16, _lib.BQ_Q8_0])
def test_the_cut_does_not_depend_on_the_query_rows(lib, requests, kv_heads, width, kind):
    """A row's bits may not depend on the rows beside it, so neither may the
    chunks and the way they are joined; and the chunks cover the table."""
    c = cache(kind, kv_heads=kv_heads)
    cuts = set()
    for rows in range(1, 7):
        for group in (1, 4, 7):
            out = (ctypes.c_int * 4)()
            x = attention(requests=requests, rows=rows, heads=group * kv_heads, table_width=width, table_stride=width)
            assert lib.bq_internal_attention_plan(ctypes.byref(c), ctypes.byref(x), out) == OK
            chunk, chunks, cluster, tiles = out
            cuts.add((chunk, chunks, cluster))
            assert chunk % 64 == 0 and (chunks - 1) * chunk < width * 16 <= chunks * chunk
            assert tiles * 32 >= rows * group and (not cluster or 2 <= chunks <= 8)
    assert len(cuts) == 1


@pytest.mark.parametrize("over", [dict(requests=(1 << 32) + 1), dict(rows=(1 << 32) + 1), dict(heads=(1 << 32) + 16),
                                  dict(width=(1 << 32) + 8), dict(rows=1 << 31)])
def test_sizes_beyond_32_bits_are_not_cut_short(lib, over):
    class Held:
        _c = cache()
        _ref = ctypes.byref(_c)

    assert bq.paged_attention_workspace(Held, 1, 1, 16, 4096) > 0
    with pytest.raises(ValueError):
        bq.paged_attention_workspace(Held, **dict(dict(requests=1, rows=1, heads=16, width=8), **over))


def test_fast_division(lib):
    f = lib.bq_internal_fast_div
    f.restype, f.argtypes = ctypes.c_uint, [ctypes.c_uint, ctypes.c_uint]
    top = (1 << 31) - 1
    for d in [1, 2, 3, 5, 7, 8, 15, 16, 17, 24, 100, 127, 128, 129, 255, 1000, 4095, 65535, 65536]:
        for n in [0, 1, d - 1, d, d + 1, 2 * d - 1, 2 * d, 12345, 99991 * d % top, top // d * d, top // d * d - 1, top - 1,
                  top]:
            assert f(n, d) == n // d, (n, d)


@pytest.mark.parametrize("over,status", [
    (dict(requests=-1), SHAPE), (dict(requests=4097), SHAPE), (dict(page_size=0), SHAPE),
    (dict(page_size=65537), SHAPE), (dict(table_width=0), SHAPE), (dict(table_stride=7), SHAPE),
    (dict(max_tokens=-1), SHAPE), (dict(max_tokens=(1 << 31) - 1), SHAPE), (dict(pool=0), SHAPE),
    (dict(pool=(1 << 31) - 1), SHAPE), (dict(free_pages=None), NULL), (dict(free_count=None), NULL),
    (dict(starts=None), NULL), (dict(free_count_out=None), NULL), (dict(refused=None), NULL),
    (dict(requests=1, lens=None), NULL), (dict(requests=1, new_lens=None), NULL), (dict(requests=1, table=None), NULL),
    (dict(requests=1, lens_out=None), NULL), (dict(slots=None), NULL), (dict(positions=None), NULL),
    (dict(table=A + 2), ALIGN), (dict(slots=A + 4), ALIGN), (dict(requests=1, lens_out=A, new_lens=A, lens=A + 64), SHAPE)])
def test_block_table_arguments(lib, over, status):
    assert lib.bq_kv_block_tables(tables(**over), None) == status


@pytest.mark.parametrize("over,status", [
    (dict(dtype=8), QTYPE), (dict(h_dtype=8), QTYPE), (dict(dtype=_lib.BQ_F16, h_dtype=_lib.BQ_BF16), QTYPE),
    (dict(dtype=_lib.BQ_F32, h_dtype=_lib.BQ_F16), QTYPE), (dict(rows=-1), SHAPE), (dict(rows=1 << 31), SHAPE),
    (dict(width=0), SHAPE), (dict(width=16385), SHAPE), (dict(y_stride=-1), SHAPE), (dict(x_stride=1 << 31), SHAPE),
    (dict(eps=-1.0), SHAPE), (dict(eps=NAN), SHAPE), (dict(alpha=INF), SHAPE), (dict(beta=NAN), SHAPE),
    (dict(rows=1, y=None), NULL), (dict(rows=1, h=None), NULL), (dict(rows=1, h_out=None), NULL),
    (dict(rows=1, pre=None), NULL), (dict(rows=1, y=A + 2), ALIGN), (dict(rows=1, post=A + 2), ALIGN),
    (dict(rows=1, h_out=A + 1), ALIGN), (dict(), OK), (dict(y=None, h=None, h_out=None, pre=None), OK)])
def test_sandwich_arguments(lib, over, status):
    assert lib.bq_sandwich_norm(sandwich(**over), None) == status
    assert lib.bq_sandwich_norm(None, None) == NULL


def test_sandwich_outputs_are_apart(lib):
    """The same address for both outputs, as `h_out=y, x_out=y` gives it."""
    assert lib.bq_sandwich_norm(sandwich(rows=1, h_out=A + 4096, x=A + 4096), None) == SHAPE


def test_structs_match_the_header():
    """Field names and order of the ctypes structs are those of the header."""
    text = open(os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "include", "bqgemv.h")).read()
    text = re.sub(r"/\*.*?\*/", "", text, flags=re.S)
    for name, cls in (("bq_kv_cache", _lib.BqKvCache), ("bq_kv_tables", _lib.BqKvTables),
                      ("bq_kv_append_args", _lib.BqKvAppendArgs), ("bq_attention_args", _lib.BqAttentionArgs),
                      ("bq_sandwich_args", _lib.BqSandwichArgs)):
        body = next(b for b, n in re.findall(r"typedef struct \{([^}]*)\} (\w+);", text) if n == name)
        fields = []
        for line in body.split(";"):
            m = re.match(r"\s*(?:const\s+)?(\w+)\s+(.*)", line.strip(), flags=re.S)
            if m:
                kind = m.group(1)
                for f in m.group(2).split(","):
                    f = f.strip()
                    pointer = "*" in f
                    f = f.replace("*", "").strip()
                    size = 8 if pointer else {"int32_t": 4, "float": 4, "int64_t": 8}[kind]
                    if "[" in f:
                        f, n = f[:-1].split("[")
                        size *= int(n)
                    fields.append((f, size))
        assert fields == [(n, ctypes.sizeof(t)) for n, t in cls._fields_], name


# ---- the binding has no CPU path and reaches no library with CPU tensors ----
def cpu_calls():
    f, i, l = torch.zeros, dict(dtype=torch.int32), dict(dtype=torch.int64)
    return {
        "PagedKVCache": lambda: bq.PagedKVCache(f(2, 1, 4, 32, dtype=torch.float16),
                                                f(2, 1, 4, 32, dtype=torch.float16)),
        "PagedKVCache.zeros": lambda: bq.PagedKVCache.zeros(2, 4, 1, 32, device="cpu"),
        "Rope": lambda: bq.Rope(f(16, dtype=torch.float64)),
        "Rope.from_theta": lambda: bq.Rope.from_theta(32, device="cpu"),
        "kv_block_tables": lambda: bq.kv_block_tables(f(1, **i), f(1, **i), f(1, 4, **i), f(4, **i), f(1, **i), 16,
                                                      f(4, **l), f(4, **i), f(2, **i)),
        "BlockTables": lambda: bq.BlockTables(1, 4, 8, 16, 8, device="cpu").resize(f(1, **i)),
        "sandwich_norm": lambda: bq.sandwich_norm(f(1, 8), f(1, 8), torch.ones(8)),
    }


@pytest.mark.parametrize("name", sorted(cpu_calls()))
def test_cpu_tensors_are_refused(monkeypatch, name):
    from block_quantized_weight_dequant_gb300 import cache as mod

    class Untouchable:
        def __getattr__(self, entry):
            raise AssertionError(f"library entry point {entry} reached with CPU tensors")

    monkeypatch.setattr(mod, "lib", Untouchable())
    with pytest.raises(ValueError, match="no CPU path"):
        cpu_calls()[name]()


def test_other_objects_are_refused():
    with pytest.raises(TypeError, match="PagedKVCache"):
        bq.kv_append(None, None, None, None)
    with pytest.raises(TypeError, match="PagedKVCache"):
        bq.paged_attention("cache", None, None, None)
    with pytest.raises(TypeError, match="torch.Tensor"):
        bq.sandwich_norm([1.0], [1.0])
    with pytest.raises(TypeError, match="fp16, bf16 or int8|CUDA|torch"):
        bq.PagedKVCache([[1]], [[1]])
    with pytest.raises(ValueError, match="kind"):
        bq.PagedKVCache.zeros(2, 4, 1, 32, kind="q4_0")


# ---- workspaces, with CPU tensors in place of the GPU's and no launch ----
def host_attention(monkeypatch, call):
    """A paged_attention call that needs a workspace, `call` in place of the
    library's (it gets the workspace's address)."""
    from block_quantized_weight_dequant_gb300 import cache as mod
    for name in ("_dense", "_first", "_activation", "_result"):
        monkeypatch.setattr(mod, name, lambda *a, **k: None)
    monkeypatch.setattr(mod, "_table", lambda t, n, device: (t.shape[1], t.shape[1]))
    monkeypatch.setattr(mod, "_raw_stream", lambda index: 0)  # one stream for all calls
    monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: False)  # (of the current device)
    monkeypatch.setattr(mod, "_call", lambda fn, what, device, cache, args, ws, nbytes: call(ws))
    c = object.__new__(bq.PagedKVCache)
    c.device, c.kv_heads, c.head_dim, c._scale, c._workspace = torch.device("cpu"), 4, 128, 0.1, {}
    c._c = cache()
    c._ref = ctypes.byref(c._c)
    q, table = torch.zeros(1, 16, 128), torch.zeros(1, 4096, dtype=torch.int32)
    return lambda: bq.paged_attention(c, q, table, torch.ones(1, dtype=torch.int32))


def test_calls_of_two_threads_at_once_have_workspaces_of_their_own(monkeypatch):
    """Both may launch on one stream, their kernels in turn."""
    both, seen = threading.Barrier(2, timeout=30), []

    def call(ws):
        if threading.current_thread() is not threading.main_thread():
            seen.append(ws)
            both.wait()

    attend = host_attention(monkeypatch, call)
    attend()
    threads = [threading.Thread(target=attend) for _ in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert len(seen) == 2 and None not in seen and seen[0] != seen[1]


def test_no_workspace_outlives_its_call(monkeypatch):
    """A kept one would be shared by whatever comes under the same stream handle:
    a captured call beside eager ones, a stream made after another's end, the
    threads' default streams."""
    made, empty = [], torch.empty

    def record(*a, **k):
        t = empty(*a, **k)
        if t.dtype == torch.uint8:
            made.append(weakref.ref(t))
        return t

    monkeypatch.setattr(torch, "empty", record)
    host_attention(monkeypatch, lambda ws: None)()
    gc.collect()
    assert len(made) == 1 and made[0]() is None
