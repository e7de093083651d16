"""Normed appends, attention over shared pages and the calls on shared pages on the
host, without a GPU: refusals of the C ABI and of the binding, struct layouts and
how calls over shared pages are cut."""
import ctypes
import os
import re

import pytest
import torch

import block_quantized_weight_dequant_gb300 as bq
from block_quantized_weight_dequant_gb300 import _lib

from test_cache_host import A, ALIGN, INF, NAN, NULL, OK, QTYPE, SHAPE, append, attention, cache, lib, tables  # noqa: F401


def fill(cls, base, over):
    s = cls()
    for n, v in dict(base, **over).items():
        setattr(s, n, v)
    return s


def norm(**over):
    return fill(_lib.BqKvNormArgs, dict(q_gain=A, k_gain=A, eps=1e-6), over)


def sharing(**over):
    return fill(_lib.BqKvSharing, dict(parents=A, refs=A, copy_src=A, copy_dst=A, copy_count=A), over)


def compact(**over):
    return fill(_lib.BqKvCompactArgs, dict(requests=0, page_size=16, table_width=8, pool=100, table_stride=8, max_moves=50,
                                           lens=A, table=A, free_pages=A, refs=A, copy_src=A, copy_dst=A, copy_count=A,
                                           moved=A, free_count_out=A), over)


def groups(*pairs):
    n = len(pairs)
    array = ctypes.c_int32 * max(n, 1)
    return array(*[p[0] for p in pairs]), array(*[p[1] for p in pairs]), n


def test_structs_match_the_header():
    text = open(os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "include", "bqgemv.h")).read()
    text = re.sub(r"/\*.*?\*/", "", text, flags=re.S)
    for name, cls in (("bq_kv_norm_args", _lib.BqKvNormArgs), ("bq_kv_sharing", _lib.BqKvSharing),
                      ("bq_kv_compact_args", _lib.BqKvCompactArgs)):
        body = next(b for b, n in re.findall(r"typedef struct \{([^}]*)\} (\w+);", text) if n == name)
        fields = []
        for line in body.split(";"):
            m = re.match(r"\s*(?:const\s+)?(\w+)\s+(.*)", line.strip(), flags=re.S)
            for f in m.group(2).split(",") if m else ():
                f = f.strip()
                size = 8 if "*" in f else {"int32_t": 4, "float": 4, "int64_t": 8}[m.group(1)]
                fields.append((f.replace("*", "").strip(), size))
        assert fields == [(n, ctypes.sizeof(t)) for n, t in cls._fields_], name
    for name in ("PAGE", "LENGTH", "SLOT", "POOL", "WAIT"):
        value = re.search(rf"#define BQ_DEVERR_{name} (0x[0-9a-f]+)u", text).group(1)
        assert getattr(_lib, f"BQ_DEVERR_{name}") == int(value, 16)
    assert int(re.search(r"#define BQ_PREFIX_MAX_GROUPS (\d+)", text).group(1)) == _lib.BQ_PREFIX_MAX_GROUPS


@pytest.mark.parametrize("over,status", [
    (dict(eps=-1.0), SHAPE), (dict(eps=NAN), SHAPE), (dict(eps=INF), SHAPE), (dict(eps=0.0), OK),
    (dict(q_gain=None, k_gain=None), OK)])
def test_append_norm_arguments(lib, over, status):
    assert lib.bq_kv_append_norm(cache(), append(), norm(**over), None) == status


def test_append_norm_pointers_and_the_appends_own_checks(lib):
    assert lib.bq_kv_append_norm(cache(), append(), None, None) == NULL
    assert lib.bq_kv_append_norm(None, append(), norm(), None) == NULL
    assert lib.bq_kv_append_norm(cache(), append(dtype=2), norm(), None) == QTYPE
    assert lib.bq_kv_append_norm(cache(), append(rot=24, sections=(12, 0, 0)), norm(), None) == SHAPE
    assert lib.bq_kv_append_norm(cache(), append(tokens=1), norm(q_gain=A + 2), None) == ALIGN
    assert lib.bq_kv_append_norm(cache(), append(tokens=1), norm(k_gain=A + 1), None) == ALIGN
    assert lib.bq_kv_append_norm(cache(), append(tokens=1, k=None), norm(), None) == NULL


@pytest.mark.parametrize("pairs,status", [
    ([(3, 64), (1, 0)], None), ([], SHAPE), ([(5, 64)], SHAPE), ([(3, 64)], SHAPE), ([(5, 64), (-1, 0)], SHAPE),
    ([(4, -1)], SHAPE), ([(4, 129)], SHAPE), ([(4, 128)], None), ([(1, 16)] * 4 + [(0, 999)], SHAPE),
    ([(1, 16)] * 4 + [(0, 5)] * 61, SHAPE), ([(1, 16)] * 4 + [(0, 5)] * 60, None)])
def test_groups(lib, pairs, status):
    x = attention(requests=4)
    need = lib.bq_paged_prefix_attention_workspace_bytes(cache(), x, *groups(*pairs))
    assert (need >= 0) == (status is None)
    if status is not None:
        assert lib.bq_paged_prefix_attention(cache(), x, *groups(*pairs), A, 1 << 40, None) == status


@pytest.mark.parametrize("over,status", [
    (dict(dtype=2), QTYPE), (dict(rows=7), SHAPE), (dict(heads=18), SHAPE), (dict(scale=NAN), SHAPE),
    (dict(table_stride=7), SHAPE), (dict(q=None), NULL), (dict(out=None), NULL), (dict(table=None), NULL),
    (dict(lens=None), NULL), (dict(q=A + 2), ALIGN), (dict(lens=A + 1), ALIGN)])
def test_prefix_attention_arguments(lib, over, status):
    x = attention(requests=2, **over)
    assert lib.bq_paged_prefix_attention(cache(), x, *groups((2, 64)), A, 1 << 40, None) == status
    assert lib.bq_paged_prefix_attention(cache(), attention(), *groups((0, 64)), None, 0, None) == OK  # no requests
    assert lib.bq_paged_prefix_attention(cache(), attention(requests=2), None, None, 1, A, 1 << 40, None) == NULL


@pytest.fixture
def shared_always(lib):
    lib.bq_internal_prefix_whole_limit.restype = ctypes.c_int64
    lib.bq_internal_prefix_whole_limit.argtypes = [ctypes.c_int64]
    lib.bq_internal_prefix_whole_limit(0)
    yield
    lib.bq_internal_prefix_whole_limit(-1)


def test_prefix_attention_workspace(lib, shared_always):
    x, g = attention(requests=2, table_width=512, table_stride=512), groups((2, 4096))
    need = lib.bq_paged_prefix_attention_workspace_bytes(cache(), x, *g)
    assert need > 0
    assert lib.bq_paged_prefix_attention(cache(), x, *g, None, 0, None) == NULL
    assert lib.bq_paged_prefix_attention(cache(), x, *g, A + 8, need, None) == ALIGN
    assert lib.bq_paged_prefix_attention(cache(), x, *g, A, need - 1, None) == SHAPE
    assert lib.bq_paged_prefix_attention_workspace_bytes(None, x, *g) == -1


@pytest.mark.parametrize("kind,dim", [(_lib.BQ_F16, 128), (_lib.BQ_BF16, 64), (_lib.BQ_F16, 256), (_lib.BQ_Q8_0, 128)])
@pytest.mark.parametrize("requests,kv_heads,heads,shared,width", [
    (1, 1, 1, 16, 1), (2, 8, 16, 700, 60), (96, 8, 32, 32801, 2100), (4096, 4, 32, 1000, 80), (4096, 1024, 4096, 48, 4),
    (1, 1, 8, 1 << 23, 1 << 19), (300, 2, 14, 100000, 6400)])
def test_any_geometry_has_a_plan(lib, shared_always, kind, dim, requests, kv_heads, heads, shared, width):
    """The most and the fewest of everything: a plan, and a workspace that a GPU may have."""
    c = cache(kind, kv_heads=kv_heads, head_dim=dim, slot_stride=dim, head_stride=16 * dim,
              page_stride=min(16 * dim * kv_heads, 1 << 30))
    for rows in (1, 6):
        x = attention(requests=requests, rows=rows, heads=heads, table_width=width, table_stride=width)
        need = lib.bq_paged_prefix_attention_workspace_bytes(c, x, *groups((requests, shared)))
        assert 0 < need < 1 << 40


@pytest.mark.parametrize("over,status", [
    (dict(refs=None), NULL), (dict(copy_count=None), NULL), (dict(copy_src=None), NULL), (dict(copy_dst=None), NULL),
    (dict(refs=A + 2), ALIGN), (dict(parents=A + 1), ALIGN), (dict(copy_src=A + 2), ALIGN)])
def test_shared_table_arguments(lib, over, status):
    assert lib.bq_kv_shared_tables(tables(requests=1), sharing(**over), None) == status


@pytest.mark.parametrize("over,status", [
    (dict(requests=4097), SHAPE), (dict(page_size=0), SHAPE), (dict(pool=0), SHAPE), (dict(free_pages=None), NULL),
    (dict(slots=A + 4), ALIGN), (dict(requests=1, lens_out=A, new_lens=A, lens=A + 64), SHAPE)])
def test_shared_tables_check_their_tables(lib, over, status):
    assert lib.bq_kv_shared_tables(tables(**over), sharing(), None) == status
    assert lib.bq_kv_shared_tables(None, sharing(), None) == NULL
    assert lib.bq_kv_shared_tables(tables(), None, None) == NULL


@pytest.mark.parametrize("over,status", [
    (dict(requests=-1), SHAPE), (dict(requests=4097), SHAPE), (dict(page_size=0), SHAPE), (dict(page_size=65537), SHAPE),
    (dict(table_width=0), SHAPE), (dict(table_stride=7), SHAPE), (dict(pool=0), SHAPE), (dict(pool=(1 << 31) - 1), SHAPE),
    (dict(max_moves=-1), SHAPE), (dict(max_moves=(1 << 31) - 1), SHAPE), (dict(free_pages=None), NULL),
    (dict(refs=None), NULL), (dict(copy_count=None), NULL), (dict(moved=None), NULL), (dict(free_count_out=None), NULL),
    (dict(requests=1, lens=None), NULL), (dict(requests=1, table=None), NULL), (dict(copy_src=None), NULL),
    (dict(copy_dst=None), NULL), (dict(moved=A + 2), ALIGN), (dict(refs=A + 1), ALIGN)])
def test_compact_arguments(lib, over, status):
    assert lib.bq_kv_compact(compact(**over), None) == status
    assert lib.bq_kv_compact(None, None) == NULL


def copy(lib, caches, src=A, dst=A, count=None, pairs=1):
    array = (ctypes.c_void_p * max(1, len(caches)))(*[None if c is None else ctypes.addressof(c) for c in caches])
    return lib.bq_kv_copy_pages(array, len(caches), src, dst, count, pairs, None)


def test_copy_arguments(lib):
    one = cache()
    assert copy(lib, []) == OK
    assert copy(lib, [one], pairs=0) == OK
    assert copy(lib, [one], pairs=-1) == SHAPE and copy(lib, [one], pairs=1 << 31) == SHAPE
    assert copy(lib, [one, None]) == NULL and copy(lib, [None]) == NULL
    assert copy(lib, [one], src=None) == NULL and copy(lib, [one], dst=None) == NULL
    assert copy(lib, [one], src=A + 2) == ALIGN and copy(lib, [one], count=A + 1) == ALIGN
    assert copy(lib, [cache(k=None)]) == NULL and copy(lib, [cache(v=A + 8)]) == ALIGN
    assert copy(lib, [cache(kind=_lib.BQ_Q8_0, v_scale=A + 2)]) == ALIGN
    for other in (dict(pages=11), dict(kv_heads=2), dict(page_size=8), dict(page_stride=16384), dict(kind=_lib.BQ_BF16)):
        assert copy(lib, [one, cache(**other)]) == SHAPE
    big = cache(kv_heads=1024, page_size=65536, head_dim=128, page_stride=0, head_stride=128, slot_stride=128)
    assert copy(lib, [big], pairs=0) == SHAPE  # its accesses are counted in 32 bits


def cpu_calls():
    i, l = dict(dtype=torch.int32), dict(dtype=torch.int64)
    z = torch.zeros
    return {
        "kv_shared_tables": lambda: bq.kv_shared_tables(z(1, **i), z(1, **i), z(1, 4, **i), z(4, **i), z(1, **i), z(4, **i),
                                                        16, z(4, **l), z(4, **i), z(2, **i), z(1, **i), z(1, **i), z(1, **i)),
        "kv_compact": lambda: bq.kv_compact(z(1, **i), z(1, 4, **i), z(4, **i), z(1, **i), z(4, **i), 16, z(2, **i),
                                            z(2, **i), z(1, **i), z(4, **i)),
        "SharedBlockTables": lambda: bq.SharedBlockTables(1, 4, 8, 16, 8, device="cpu").resize(z(1, **i)),
    }


@pytest.mark.parametrize("name", sorted(cpu_calls()))
def test_no_cpu_path(name):
    with pytest.raises(ValueError, match="CUDA"):
        cpu_calls()[name]()


def test_arguments_that_are_no_caches():
    for call in (lambda: bq.paged_prefix_attention("cache", None, None, None, 0), lambda: bq.kv_copy_pages([None], None, None),
                 lambda: bq.kv_copy_pages("x", None, None)):
        with pytest.raises(TypeError, match="PagedKVCache"):
            call()
    assert bq.kv_copy_pages([], None, None) is None
