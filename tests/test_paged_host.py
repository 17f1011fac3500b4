"""The paged cache on the host: the struct, sizes and refusals before any CUDA call."""
import ctypes
import os
import re

import pytest

from sliding_window_attention_device_gb300 import bdattn, build

HEADER = os.path.join(os.path.dirname(bdattn.__file__), "..", "include", "bdattn.h")


@pytest.fixture(scope="module")
def lib():
    build.build()
    return bdattn.load()


def test_struct_matches_header():
    fields = re.search(r"typedef struct \{([^}]*)\} bd_paged;", open(HEADER).read()).group(1)
    assert re.findall(r"\b(?:int|float)\s+(\w+);", fields) == [n for n, _ in bdattn.Paged._fields_]


BASE = dict(B=4, Hq=8, Hkv=2, D=128, n_pages=100, page_size=16, max_pages=200)


@pytest.mark.parametrize("bad", [
    dict(B=0), dict(B=70000), dict(Hq=6, Hkv=4), dict(Hkv=0), dict(D=96), dict(D=0), dict(n_pages=0),
    dict(page_size=0), dict(max_pages=0), dict(n_sink=-1), dict(scale=float("nan")),
    dict(max_pages=1 << 20, page_size=1 << 11), dict(n_pages=1 << 28, page_size=4), dict(B=60000, Hq=128),
])
def test_bad_geometry(lib, bad):
    g = bdattn.paged_geom(**{**BASE, **bad})
    P, E = ctypes.c_void_p, bdattn.BD_ERR_ARG
    assert lib.bd_attn_paged_decode_workspace_bytes(ctypes.byref(g)) == 0
    with pytest.raises(ValueError):
        bdattn.paged_decode_workspace_bytes(g)
    assert lib.bd_attn_paged_decode(*[P(256)] * 5, ctypes.byref(g), *[P(256)] * 4, None) == E
    assert lib.bd_attn_paged_append(*[P(256)] * 5, ctypes.byref(g), 4, *[P(256)] * 3, None) == E


def test_bad_pointers(lib):
    g = bdattn.paged_geom(**BASE)
    P, E = ctypes.c_void_p, bdattn.BD_ERR_ARG
    base = [P(256)] * 5 + [ctypes.byref(g)] + [P(256)] * 4 + [None]
    for i in (0, 1, 2, 3, 4, 5, 6, 7, 8, 9):
        a = list(base)
        a[i] = None
        assert lib.bd_attn_paged_decode(*a) == E
    for i in (0, 1, 2, 6, 8):
        a = list(base)
        a[i] = P(264)
        assert lib.bd_attn_paged_decode(*a) == E
    base = [P(256)] * 5 + [ctypes.byref(g), 4] + [P(256)] * 3 + [None]
    for i in (0, 1, 2, 3, 4, 5, 7, 8, 9):
        a = list(base)
        a[i] = None
        assert lib.bd_attn_paged_append(*a) == E
    for i, v in ((6, -1), (0, P(8)), (8, P(8))):
        a = list(base)
        a[i] = v
        assert lib.bd_attn_paged_append(*a) == E


@pytest.mark.parametrize("D", [64, 128, 256, 512])
@pytest.mark.parametrize("G", [1, 3, 8, 9, 16, 40])
def test_workspace(lib, D, G):
    n = bdattn.paged_decode_workspace_bytes(bdattn.paged_geom(**{**BASE, "D": D, "Hq": 2 * G}))
    assert n % 16 == 0 and 0 < n < 64 << 20
