"""Argument checks of the 8-bit cache's entry points (no GPU needed): status codes before any HIP call."""
from __future__ import annotations

import ctypes
import os
import struct

import pytest

from tests.test_abi_kv4_host import A, ALIGN, BAD_BATCH, BATCH, HALF, LIB, NULL, ODD, OK, ROOT, SHAPE, WORKSPACE, WS, f32, i32, i64, p, rows, sz

ROTATION = [("cos_sin", p, A), ("ld_turn", i64, 128), ("positions", i64, 80 * 64), ("rotary_dim", i32, 128), ("interleaved", i32, 0)]
CALLS = {
    "nm_kv8_append": [("batch", BATCH), rows("k"), rows("v"), ("rotation", ROTATION), rows("q"), ("n_heads", i32, 8), rows("o"),
                      ("stream", p, None)],
    "nm_kv8_unpack": [("batch", BATCH), rows("k"), rows("v"), ("stream", p, None)],
    "nm_kv8_select": [("batch", BATCH), rows("q"), ("n_heads", i32, 8), ("top", i32, 12), ("first", i32, 1), ("last", i32, 2),
                      ("selected", p, A), ("ld_selected", i64, 24), *WS],
    "nm_kv8_attention": [("batch", BATCH), rows("q"), ("n_heads", i32, 8), ("max_q_len", i64, 1), ("scale", f32, 0.1),
                         ("window", i64, 0), ("selected", p, A), ("ld_selected", i64, 24), ("top", i32, 12), rows("o"), ("lse", p, A),
                         ("ld_lse", i64, 8), *WS],
}


def fields(name):
    return [f for a in CALLS[name] for f in (a[1] if len(a) == 2 else [a])]


@pytest.fixture(scope="module")
def L():
    lib = ctypes.CDLL(LIB)
    lib.nm_last_error.restype = ctypes.c_char_p
    for name, args in CALLS.items():
        getattr(lib, name).argtypes = [p if len(a) == 2 else a[1] for a in args]
    lib.nm_kv8_page_bytes.argtypes, lib.nm_kv8_page_bytes.restype = [i32] * 3, i64
    lib.nm_kv8_attention_workspace_bytes.argtypes = [i64, i64, i32, i32, i32, i64, i64, i32]
    lib.nm_kv8_attention_workspace_bytes.restype = sz
    lib.nm_kv8_select_workspace_bytes.argtypes, lib.nm_kv8_select_workspace_bytes.restype = [i64, i64, i32, i64], sz
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


def test_python_packs_the_rotation_as_c_does():
    S = type("S", (ctypes.Structure,), {"_fields_": [(n, t) for n, t, _ in ROTATION]})
    assert struct.calcsize("@Pqq2i") == ctypes.sizeof(S)
    assert 'struct.Struct("@Pqq2i")' in open(os.path.join(ROOT, "bitmask_spmv_amd", "__init__.py")).read()


OPTIONAL = {"stream", "lse", "selected"}


@pytest.mark.parametrize("name", sorted(CALLS))
def test_null_pointers_and_odd_addresses(L, name):
    for a in CALLS[name]:
        if len(a) == 2 and a[0] != "rotation":
            assert call(L, name, **{a[0]: None}) == NULL, a[0]
    for arg, kind, _ in fields(name):
        if kind is not p or (arg in OPTIONAL and (name, arg) != ("nm_kv8_select", "selected")):
            continue
        if arg == "workspace":  # asked of calls that need one
            long = dict(table_cols=8000, ld_table=8000)
            if name == "nm_kv8_attention":
                long["selected"] = None
            assert call(L, name, workspace=None, **long) == WORKSPACE and call(L, name, workspace=HALF, **long) == WORKSPACE
            assert call(L, name, workspace_bytes=8, **long) == WORKSPACE
            continue
        assert call(L, name, **{arg: None}) == NULL, arg
        assert name.encode() in L.nm_last_error()
        assert call(L, name, **{arg: ODD}) == ALIGN, arg


@pytest.mark.parametrize("name", sorted(CALLS))
@pytest.mark.parametrize("bad", BAD_BATCH)
def test_sizes_of_a_batch(L, name, bad):
    assert call(L, name, **bad) == SHAPE


@pytest.mark.parametrize("name,bad,want", [
    ("nm_kv8_append", dict(ldk=120), SHAPE), ("nm_kv8_append", dict(hdv=64), SHAPE), ("nm_kv8_append", dict(ldk=1028), ALIGN),
    ("nm_kv8_append", dict(k=HALF), ALIGN), ("nm_kv8_append", dict(cache=HALF), ALIGN), ("nm_kv8_append", dict(ldq=100), SHAPE),
    ("nm_kv8_append", dict(hdo=130), ALIGN), ("nm_kv8_append", dict(n_heads=7), SHAPE), ("nm_kv8_append", dict(n_heads=0), SHAPE),
    ("nm_kv8_append", dict(rotation=None), NULL), ("nm_kv8_append", dict(cos_sin=HALF), ALIGN), ("nm_kv8_append", dict(ld_turn=130), ALIGN),
    ("nm_kv8_append", dict(ld_turn=124), SHAPE), ("nm_kv8_append", dict(ld_turn=-4), SHAPE), ("nm_kv8_append", dict(positions=80 * 64 - 1), SHAPE),
    ("nm_kv8_append", dict(rotary_dim=0), SHAPE), ("nm_kv8_append", dict(rotary_dim=24), SHAPE), ("nm_kv8_append", dict(rotary_dim=144), SHAPE),
    ("nm_kv8_append", dict(T=1 << 24, n_kv=32, n_heads=32, ldk=4096, ldv=4096), SHAPE), ("nm_kv8_append", dict(S=1 << 20, n_kv=4), SHAPE),
    ("nm_kv8_unpack", dict(hdk=132), ALIGN), ("nm_kv8_unpack", dict(ldv=-8), SHAPE), ("nm_kv8_unpack", dict(S=1 << 20, n_kv=4), SHAPE),
    ("nm_kv8_select", dict(n_heads=7), SHAPE), ("nm_kv8_select", dict(top=0), SHAPE), ("nm_kv8_select", dict(top=1 << 15), SHAPE),
    ("nm_kv8_select", dict(first=-1), SHAPE), ("nm_kv8_select", dict(last=-1), SHAPE), ("nm_kv8_select", dict(first=2, last=11), SHAPE),
    ("nm_kv8_select", dict(first=2**31 - 1, last=2**31 - 1), SHAPE), ("nm_kv8_select", dict(ld_selected=23), SHAPE),
    ("nm_kv8_select", dict(table_cols=16385, ld_table=16385), SHAPE), ("nm_kv8_select", dict(table_cols=2049, ld_table=2049, page_size=512), SHAPE),
    ("nm_kv8_select", dict(T=(1 << 20) + 1), SHAPE), ("nm_kv8_select", dict(hdq=124), SHAPE),
    ("nm_kv8_attention", dict(n_heads=7), SHAPE), ("nm_kv8_attention", dict(n_heads=2048), SHAPE), ("nm_kv8_attention", dict(window=-1), SHAPE),
    ("nm_kv8_attention", dict(max_q_len=0), SHAPE), ("nm_kv8_attention", dict(scale=float("nan")), SHAPE),
    ("nm_kv8_attention", dict(scale=float("inf")), SHAPE), ("nm_kv8_attention", dict(scale=2.0**61), SHAPE),
    ("nm_kv8_attention", dict(scale=-(2.0**-61)), SHAPE), ("nm_kv8_attention", dict(ldo=100), SHAPE),
    ("nm_kv8_attention", dict(hdo=129), ALIGN), ("nm_kv8_attention", dict(ld_lse=7), SHAPE), ("nm_kv8_attention", dict(lse=0x10002), ALIGN),
    ("nm_kv8_attention", dict(selected=ODD), ALIGN), ("nm_kv8_attention", dict(top=0), SHAPE), ("nm_kv8_attention", dict(top=-1), SHAPE),
    ("nm_kv8_attention", dict(ld_selected=23), SHAPE), ("nm_kv8_attention", dict(top=(1 << 20) + 1, ld_selected=1 << 40), SHAPE),
    ("nm_kv8_attention", dict(T=(1 << 20) + 1), SHAPE),
    ("nm_kv8_attention", dict(T=(1 << 24) - 7, n_heads=256, n_kv=2, ldo=32768, ldq=32768, ld_lse=256, selected=None), SHAPE),
    ("nm_kv8_attention", dict(S=1 << 20, n_heads=8, n_kv=8), SHAPE)])
def test_rows_heads_and_sizes(L, name, bad, want):
    assert call(L, name, **bad) == want


def test_nothing_to_do_is_not_an_error(L):
    assert call(L, "nm_kv8_append", T=0, k=None, v=None, q=None, o=None) == OK
    assert call(L, "nm_kv8_unpack", T=0, S=0, k=None, v=None) == OK
    assert call(L, "nm_kv8_select", T=0, q=None, selected=None) == OK
    assert call(L, "nm_kv8_attention", T=0, q=None, o=None, lse=None, selected=None) == OK


def test_size_queries(L):
    assert L.nm_kv8_select_workspace_bytes(16, 16, 8, 1 << 18) == 16 * 8 * (4096 + 16 + 1) * 4
    assert L.nm_kv8_select_workspace_bytes(16, 16, 8, 65536) == 0  # short contexts
    assert L.nm_kv8_select_workspace_bytes(512, 1, 8, 65536) == 0  # rows of a sequence go by sixteen
    assert L.nm_kv8_select_workspace_bytes(2000, 2000, 8, 1 << 20) == 0  # rows enough for the machine
    for bad in ((-1, 1, 8, 65536), (16, 16, 0, 65536), (16, 16, 8, 0), (16, 16, 8, (1 << 20) + 1)):
        assert L.nm_kv8_select_workspace_bytes(*bad) == 0
    assert L.nm_kv8_page_bytes(64, 8, 128) == 133248  # 8 blocks of 16384 + 256 + 4, to a multiple of 128
    assert L.nm_kv8_page_bytes(512, 1, 64) == 66688
    for bad in ((0, 8, 128), (48, 8, 128), (64, 0, 128), (64, 8, 80), (64, 300, 128)):
        assert L.nm_kv8_page_bytes(*bad) == 0
    assert L.nm_kv8_attention_workspace_bytes(5, 3, 8, 2, 128, 1, 1 << 20, 0) > 0
    assert L.nm_kv8_attention_workspace_bytes(5, 3, 8, 2, 128, 1, 1024, 0) == 0  # one workgroup to each row tile
    assert L.nm_kv8_attention_workspace_bytes(5, 3, 8, 2, 128, 1, 1 << 20, 512) > 0
    assert L.nm_kv8_attention_workspace_bytes(4000, 3, 8, 2, 128, 2000, 1 << 20, 12) == 0  # rows enough for the machine
    for bad in ((-1, 1, 8, 2, 128, 1, 4096, 0), (5, 3, 7, 2, 128, 1, 4096, 0), (5, 3, 8, 2, 96, 1, 4096, 0),
                (5, 3, 8, 2, 128, 0, 4096, 0), (5, 3, 8, 2, 128, 1, 0, 0), (5, 3, 8, 2, 128, 1, 4096, -1)):
        assert L.nm_kv8_attention_workspace_bytes(*bad) == 0
