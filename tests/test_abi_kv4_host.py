"""Argument checks of the 4-bit cache's entry points (no GPU needed): status codes before any HIP call."""
from __future__ import annotations

import ctypes
import os

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
LIB = os.environ.get("NM_SPMV_LIB") or os.path.join(ROOT, "bitmask_spmv_amd", "libnmspmv.so")
OK, NULL, SHAPE, PATTERN, ALIGN, WORKSPACE, HIP = range(7)
A = 0x10000  # never read: the call is refused first
ODD = 0x10001
HALF = 0x10008

i64, p, i32, sz, f32 = ctypes.c_int64, ctypes.c_void_p, ctypes.c_int, ctypes.c_size_t, ctypes.c_float
BATCH = [("cache", p, A), ("num_pages", i64, 4), ("page_table", p, A), ("ld_table", i64, 80), ("kv_len", p, A),
         ("q_start", p, A), ("S", i64, 3), ("T", i64, 5), ("table_cols", i32, 80), ("page_size", i32, 64), ("n_kv", i32, 2),
         ("head_dim", i32, 128)]
BOOK = [("page_table", p, A), ("ld_table", i64, 8), ("kv_len", p, A), ("S", i64, 3), ("refcount", p, A),
        ("num_pages", i64, 40000), ("table_cols", i32, 8), ("page_size", i32, 64)]
WS = [("workspace", p, A), ("workspace_bytes", sz, 1 << 40), ("stream", p, None)]


def rows(n):
    return ("rows " + n, [(n, p, A), ("ld" + n, i64, 1024), ("hd" + n, i64, 128)])


# an argument: (name, type, value), or (name, fields) of a struct that is passed by address
CALLS = {
    "nm_kv4_append": [("batch", BATCH), rows("k"), rows("v"), ("stream", p, None)],
    "nm_kv4_unpack": [("batch", BATCH), rows("k"), rows("v"), ("stream", p, None)],
    "nm_kv4_attention": [("batch", BATCH), rows("q"), ("n_heads", i32, 8), ("max_q_len", i64, 1), ("scale", f32, 0.1),
                         ("window", i64, 0), rows("o"), ("lse", p, A), ("ld_lse", i64, 8), *WS],
    "nm_kv_resize": [("book", BOOK), ("new_len", p, A), ("moves", p, A), ("missing", p, A), *WS],
    "nm_kv_fork": [("book", BOOK), ("parent", p, A), ("child", p, A), ("n", i64, 2), ("moves", p, A), ("missing", p, A), *WS],
    "nm_kv_compact": [("book", BOOK), ("moves", p, A), ("max_moves", i64, 9), ("used", p, A), *WS],
    "nm_kv_copy_pages": [("cache", p, A), ("num_pages", i64, 4), ("page_bytes", i64, 64), ("layers", i64, 2),
                         ("layer_stride", i64, 256), ("moves", p, A), ("n", i64, 3), ("stream", p, None)],
}


def fields(name):
    return [f for a in CALLS[name] for f in (a[1] if len(a) == 2 else [a])]


@pytest.fixture(scope="module")
def L():
    lib = ctypes.CDLL(LIB)
    lib.nm_last_error.restype = ctypes.c_char_p
    for name, args in CALLS.items():
        getattr(lib, name).argtypes = [p if len(a) == 2 else a[1] for a in args]
    lib.nm_kv4_page_bytes.argtypes, lib.nm_kv4_page_bytes.restype = [i32] * 3, i64
    lib.nm_kv4_attention_workspace_bytes.argtypes = [i64, i64, i32, i32, i32, i64, i64]
    lib.nm_kv4_attention_workspace_bytes.restype = sz
    lib.nm_kv_pages_workspace_bytes.argtypes, lib.nm_kv_pages_workspace_bytes.restype = [i64, i64, i64, i32], sz
    return lib


def call(L, name, **bad):
    assert not set(bad) - {f[0] for f in fields(name)} - {a[0] for a in CALLS[name]}
    args, keep = [], []
    for a in CALLS[name]:
        if len(a) == 3:
            args.append(bad.get(a[0], a[2]))
        elif a[0] in bad:
            args.append(bad[a[0]])
        else:
            S = type("S", (ctypes.Structure,), {"_fields_": [(n, t) for n, t, _ in a[1]]})
            keep.append(S(*[bad.get(n, v) for n, _, v in a[1]]))
            args.append(ctypes.addressof(keep[-1]))
    return getattr(L, name)(*args)


def test_python_packs_the_structs_as_c_does():
    """The binding's struct formats have the sizes of the C structs."""
    import struct

    for fmt, fl in (("@PqPqPPqq4i", BATCH), ("@Pqq", rows("k")[1]), ("@PqPqPq2i", BOOK)):
        S = type("S", (ctypes.Structure,), {"_fields_": [(n, t) for n, t, _ in fl]})
        assert struct.calcsize(fmt) == sum(ctypes.sizeof(t) for _, t, _ in fl) <= ctypes.sizeof(S)
        text = open(os.path.join(ROOT, "bitmask_spmv_amd", "__init__.py")).read()
        assert f'struct.Struct("{fmt}")' in text


OPTIONAL = {"stream", "lse"}


@pytest.mark.parametrize("name", sorted(CALLS))
def test_null_pointers_and_odd_addresses(L, name):
    for a in CALLS[name]:
        if len(a) == 2:
            assert call(L, name, **{a[0]: None}) == NULL, a[0]
    for arg, kind, _ in fields(name):
        if kind is not p or arg in OPTIONAL:
            continue
        st = call(L, name, **{arg: None})
        if arg == "workspace":
            need = L.nm_kv4_attention_workspace_bytes(5, 3, 8, 2, 128, 1, 80 * 64) if name == "nm_kv4_attention" else 1
            if need:
                assert st == WORKSPACE, arg
                assert call(L, name, workspace=HALF) == WORKSPACE
            continue
        assert st == NULL, arg
        assert name.encode() in L.nm_last_error()
        assert call(L, name, **{arg: ODD}) == ALIGN, arg


BAD_BATCH = [dict(head_dim=96), dict(head_dim=256), dict(head_dim=0), dict(page_size=16), dict(page_size=96),
             dict(page_size=1024), dict(n_kv=0), dict(n_kv=257), dict(T=-1), dict(T=(1 << 24) + 1), dict(S=0), dict(S=-1),
             dict(S=(1 << 20) + 1), dict(num_pages=0), dict(num_pages=1 << 31), dict(table_cols=0), dict(ld_table=7)]


@pytest.mark.parametrize("name", ["nm_kv4_append", "nm_kv4_unpack", "nm_kv4_attention"])
@pytest.mark.parametrize("bad", BAD_BATCH)
def test_sizes_of_a_batch(L, name, bad):
    assert call(L, name, **bad) == SHAPE


@pytest.mark.parametrize("name,bad,want", [
    ("nm_kv4_append", dict(ldk=120), SHAPE), ("nm_kv4_append", dict(hdv=64), SHAPE), ("nm_kv4_append", dict(ldk=1028), ALIGN),
    ("nm_kv4_append", dict(k=HALF), ALIGN), ("nm_kv4_append", dict(cache=HALF), ALIGN), ("nm_kv4_unpack", dict(hdk=132), ALIGN),
    ("nm_kv4_unpack", dict(ldv=-8), SHAPE), ("nm_kv4_attention", dict(n_heads=7), SHAPE),
    ("nm_kv4_attention", dict(n_heads=0), SHAPE), ("nm_kv4_attention", dict(n_heads=2048), SHAPE),
    ("nm_kv4_attention", dict(window=-1), SHAPE), ("nm_kv4_attention", dict(max_q_len=0), SHAPE),
    ("nm_kv4_attention", dict(scale=float("nan")), SHAPE), ("nm_kv4_attention", dict(scale=float("inf")), SHAPE),
    ("nm_kv4_attention", dict(ldo=100), SHAPE), ("nm_kv4_attention", dict(hdq=124), SHAPE),
    ("nm_kv4_attention", dict(hdo=129), ALIGN), ("nm_kv4_attention", dict(ld_lse=7), SHAPE),
    ("nm_kv4_attention", dict(lse=0x10002), ALIGN),
    # rows and launches are numbered in 32 bits
    ("nm_kv4_attention", dict(T=(1 << 24) - 7, n_heads=256, n_kv=2, ldo=32768, ldq=32768, ld_lse=256), SHAPE),
    ("nm_kv4_attention", dict(S=1 << 20, n_heads=8, n_kv=8), SHAPE)])
def test_rows_heads_and_scales(L, name, bad, want):
    assert call(L, name, **bad) == want


@pytest.mark.parametrize("name", ["nm_kv_resize", "nm_kv_fork", "nm_kv_compact"])
@pytest.mark.parametrize("bad,want", [
    (dict(page_size=32), SHAPE), (dict(S=0), SHAPE), (dict(S=(1 << 20) + 1), SHAPE), (dict(num_pages=0), SHAPE),
    (dict(num_pages=(1 << 30) + 1), SHAPE), (dict(table_cols=0), SHAPE), (dict(ld_table=5), SHAPE),
    (dict(S=1 << 20, table_cols=2048, ld_table=2048), SHAPE), (dict(workspace_bytes=8), WORKSPACE)])
def test_page_keeping(L, name, bad, want):
    assert call(L, name, **bad) == want


@pytest.mark.parametrize("name,bad,want", [
    ("nm_kv_fork", dict(n=0), SHAPE), ("nm_kv_fork", dict(n=(1 << 16) + 1), SHAPE), ("nm_kv_compact", dict(max_moves=0), SHAPE),
    ("nm_kv_compact", dict(max_moves=(1 << 29) + 1), SHAPE), ("nm_kv_copy_pages", dict(page_bytes=24), ALIGN),
    ("nm_kv_copy_pages", dict(page_bytes=0), SHAPE), ("nm_kv_copy_pages", dict(layers=0), SHAPE),
    ("nm_kv_copy_pages", dict(layer_stride=240), SHAPE), ("nm_kv_copy_pages", dict(layer_stride=264), ALIGN),
    ("nm_kv_copy_pages", dict(n=-1), SHAPE), ("nm_kv_copy_pages", dict(num_pages=0), SHAPE)])
def test_lists(L, name, bad, want):
    assert call(L, name, **bad) == want


def test_nothing_to_do_is_not_an_error(L):
    assert call(L, "nm_kv4_append", T=0, k=None, v=None) == OK
    assert call(L, "nm_kv4_unpack", T=0, S=0, k=None, v=None) == OK
    assert call(L, "nm_kv4_attention", T=0, q=None, o=None, lse=None) == OK
    assert call(L, "nm_kv_copy_pages", n=0, moves=None) == OK


def test_size_queries(L):
    assert L.nm_kv4_page_bytes(64, 8, 128) == 69632
    assert L.nm_kv4_page_bytes(512, 1, 64) == 512 * 2 * 34
    for bad in ((0, 8, 128), (48, 8, 128), (64, 0, 128), (64, 8, 80), (64, 300, 128)):
        assert L.nm_kv4_page_bytes(*bad) == 0
    assert L.nm_kv4_attention_workspace_bytes(5, 3, 8, 2, 128, 1, 4096) > 0
    assert L.nm_kv4_attention_workspace_bytes(5, 3, 8, 2, 128, 1, 1024) == 0  # one workgroup to each row tile
    for bad in ((-1, 1, 8, 2, 128, 1, 4096), (5, 3, 7, 2, 128, 1, 4096), (5, 3, 8, 2, 96, 1, 4096),
                (5, 3, 8, 2, 128, 0, 4096), (5, 3, 8, 2, 128, 1, 0)):
        assert L.nm_kv4_attention_workspace_bytes(*bad) == 0
    for bad in ((0, 0, 5, 1), (1, 0, 0, 1), (1, -1, 5, 1), (1, 0, 5, 0)):
        assert L.nm_kv_pages_workspace_bytes(*bad) == 0
    assert L.nm_kv_pages_workspace_bytes(8, 8, 4096, 64) == 0  # one workgroup
    for big in ((8, 8, 16385, 64), (257, 0, 100, 4), (8, 65, 100, 4), (256, 0, 100, 257)):
        assert L.nm_kv_pages_workspace_bytes(*big) > 0
    assert L.nm_kv_pages_workspace_bytes(4, 100, 50000, 8) >= L.nm_kv_pages_workspace_bytes(4, 0, 50000, 8)
