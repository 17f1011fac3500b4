"""Numbers that do not fit the C structs' 32 bits, on the host: refused instead of wrapped; a window of any size
is one beyond every distance."""
import pytest

from sliding_window_attention_device_gb300 import bdattn, build

GEOM = dict(B=1, Hq=2, Hkv=1, D=64, S_full=256, L=64, row_offset=0, kv_offset=0, S_kv=256)
PAGED = dict(B=4, Hq=8, Hkv=2, D=128, n_pages=100, page_size=16, max_pages=200)


@pytest.mark.parametrize("name", list(GEOM))
@pytest.mark.parametrize("add", [2 ** 32, -2 ** 32, 2 ** 63])
def test_geom(name, add):
    with pytest.raises(ValueError, match=name):
        bdattn.geom(**{**GEOM, name: GEOM[name] + add})


@pytest.mark.parametrize("name", list(PAGED))
@pytest.mark.parametrize("add", [2 ** 32, -2 ** 32, 2 ** 63])
def test_paged(name, add):
    with pytest.raises(ValueError, match=name):
        bdattn.paged_geom(**{**PAGED, name: PAGED[name] + add})


@pytest.mark.parametrize("window,want", [(2 ** 32 + 5, 2 ** 31 - 1), (2 ** 63 - 1, 2 ** 31 - 1), (2 ** 31 - 1, 2 ** 31 - 1),
                                         (100, 100), (0, 0), (-1, -1), (-2 ** 40, -1)])
def test_window(window, want):
    for g in (bdattn.geom(**GEOM, window=window), bdattn.paged_geom(**PAGED, window=window)):
        assert g.window == want


def test_sinks():
    build.build()
    g = bdattn.geom(**GEOM, window=32)
    for n in (2 ** 32 + 4, -2 ** 32, 129, -1):
        with pytest.raises(ValueError):
            bdattn.sink_seg_bytes(g, n)
        with pytest.raises(ValueError):
            bdattn.sink_bwd_workspace_bytes(g, n)
    assert bdattn.paged_geom(**PAGED, window=3, n_sink=2 ** 40).n_sink == 2 ** 31 - 1  # all of them
    with pytest.raises(ValueError, match="n_sink"):
        bdattn.paged_geom(**PAGED, n_sink=-2 ** 40)


@pytest.mark.parametrize("name,values", [("pairing", (64, 2 ** 32, 100)), ("pairing", (64, -2 ** 32 + 1, 100)),
                                         ("n_pos", (0, 0, 2 ** 32 + 5))])
def test_rope(name, values):
    with pytest.raises(ValueError, match=name):
        bdattn._rope(*values, 0, 0, 0)
    assert bdattn._rope(64, 1, 100, 512, 256, 2 ** 31).v_stride == 2 ** 31
