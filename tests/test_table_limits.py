"""Geometries at the tables' size limit, on the host: a table has fewer than 2^31 words, else the geometry is
refused before anything is laid out with wrapped offsets."""
import ctypes

import pytest

from sliding_window_attention_device_gb300 import bdattn, build


@pytest.fixture(scope="module")
def lib():
    build.build()
    return bdattn.load()


def words(B, L, S_kv):
    """The table's words without its regions' padding."""
    nqt, nkt = -(-L // 128), -(-S_kv // 128)
    return B * (32 + 2 * (L + 1) + L + 2 * nqt + 2 * nkt + nqt * -(-nkt // 32) + nqt + nkt) + 8


@pytest.mark.parametrize("B,L,S_kv", [(1, 1 << 24, 1 << 27), (1, 1 << 24, 1 << 26), (4, 1 << 22, 1 << 25),
                                      (1, 1 << 20, 1 << 28), (1, 50_000_000, 200_000_000), (1, 1 << 23, 1 << 26),
                                      (2, 1000, 5000), (1, 1, 1)])
def test_table_size(lib, B, L, S_kv):
    g = bdattn.geom(B, 2, 1, 64, S_kv, L, 0, 0, S_kv, 1024)
    n = int(lib.bd_attn_seg_bytes(ctypes.byref(g)))
    ns = int(lib.bd_attn_sink_seg_bytes(ctypes.byref(g), 4))
    if words(B, L, S_kv) >= 2 ** 31 or B * (L + 1) * 4 + B * S_kv > 2 ** 29:
        assert n == 0 and ns == 0
        with pytest.raises(ValueError):
            bdattn.seg_bytes(g)
    else:
        assert 0 <= n // 4 - words(B, L, S_kv) < 64 and ns > n
