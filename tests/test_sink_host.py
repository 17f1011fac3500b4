"""Attention sinks on the host: sizes, refusals before any CUDA call, and the
plain form the GPU tests compare with, by brute force."""
import ctypes
import math

import pytest
import torch

from helpers import make_case
from sink_ref import reference, visible
from sliding_window_attention_device_gb300 import bdattn, build, synth


@pytest.fixture(scope="module")
def lib():
    build.build()
    return bdattn.load()


@pytest.mark.parametrize("window", [0, 1, 100, 128, 1024])
@pytest.mark.parametrize("D", [64, 128, 256, 512])
def test_sizes(lib, D, window):
    g = bdattn.geom(2, 4, 2, D, 4096, 1024, 2048, 0, 4096, window)
    for n in (0, 1, 4, 128):
        assert bdattn.sink_seg_bytes(g, n) > bdattn.seg_bytes(g) and bdattn.sink_seg_bytes(g, n) % 16 == 0
        extra = bdattn.sink_bwd_workspace_bytes(g, n) - bdattn.bwd_workspace_bytes(g)
        assert (extra == 0) if (window == 0 or n == 0) else extra > 0
    for n in (-1, 129, 1 << 20):
        assert lib.bd_attn_sink_seg_bytes(ctypes.byref(g), n) == 0
        assert lib.bd_attn_sink_bwd_workspace_bytes(ctypes.byref(g), n) == 0
        with pytest.raises(ValueError):
            bdattn.sink_seg_bytes(g, n)
    g.D = 96
    assert lib.bd_attn_sink_seg_bytes(ctypes.byref(g), 4) == 0


def test_arguments(lib):
    g = bdattn.geom(1, 2, 1, 64, 256, 64, 128, 0, 256, 32)
    P, G, E = ctypes.c_void_p, ctypes.byref(g), bdattn.BD_ERR_ARG
    ok = P(256)
    assert lib.bd_attn_sink_seg_build(None, G, 4, 0, ok, ok, None) == E
    assert lib.bd_attn_sink_seg_build(ok, G, 4, 2, ok, ok, None) == E
    assert lib.bd_attn_sink_seg_build(ok, G, 129, 0, ok, ok, None) == E
    assert lib.bd_attn_sink_seg_build(ok, G, 4, 0, P(264), ok, None) == E
    assert lib.bd_attn_sink_seg_build(ok, None, 4, 0, ok, ok, None) == E
    for f in (lib.bd_attn_sink_fwd, lib.bd_attn_sink_fwd_merge):
        for n in (-1, 129):
            assert f(ok, ok, ok, ok, G, n, ok, ok, ok, None) == E
        for i in (0, 1, 2, 3, 6, 7, 8):
            a = [ok, ok, ok, ok, G, 4, ok, ok, ok, None]
            a[i] = None
            assert f(*a) == E
        assert f(P(8), ok, ok, ok, G, 4, ok, ok, ok, None) == E
    for f in (lib.bd_attn_sink_bwd, lib.bd_attn_sink_bwd_deterministic):
        base = [ok] * 7 + [G, 4, 0, ok, ok, ok, ok, ok, None]
        for i in (0, 1, 2, 3, 4, 5, 6, 10, 11, 12, 13, 14):
            a = list(base)
            a[i] = None
            assert f(*a) == E
        for i, v in ((8, -1), (8, 129), (9, 2), (13, P(128))):
            a = list(base)
            a[i] = v
            assert f(*a) == E
    base = [ok] * 6 + [G, 4, 0, ok, ok, ok, ok, None]
    for i, v in ((0, None), (7, -1), (8, 2), (11, P(16)), (11, None)):
        a = list(base)
        a[i] = v
        assert lib.bd_attn_sink_bwd_main(*a) == E


def test_header_constant():
    import os
    import re
    text = open(os.path.join(os.path.dirname(bdattn.__file__), "..", "include", "bdattn.h")).read()
    assert int(re.search(r"#define BD_SINK_MAX (\d+)", text).group(1)) == bdattn.SINK_MAX


def test_plain_form_by_hand():
    """Two documents of 5 and 3 tokens, window 2, one sink: the visible keys written out."""
    doc = torch.tensor([[1, 1, 1, 1, 1, 2, 2, 2, 0]])
    want = [[0], [0, 1], [0, 1, 2], [0, 2, 3], [0, 3, 4], [5], [5, 6], [5, 6, 7], []]
    m = visible(doc, 0, 9, 0, 9, 2, 1)[0]
    assert [torch.nonzero(r).flatten().tolist() for r in m] == want
    # a window as long as the document, no sinks and sinks without a window: plain causal
    for args in ((5, 0), (5, 3), (0, 1)):
        m = visible(doc, 0, 9, 0, 9, *args)[0]
        assert [len(torch.nonzero(r)) for r in m] == [1, 2, 3, 4, 5, 1, 2, 3, 0]


def test_plain_form_gradients_against_differences():
    w = synth.Workload("s", "s", B=1, Hq=2, Hkv=1, D=64, S=40, cp_size=2, layout=("explicit", (5, 30), 5), window=6)
    c = make_case(w, 1)
    ref = reference(c, 3)
    gen = torch.Generator().manual_seed(1)
    for key, grad in (("q", "dq"), ("k", "dk"), ("v", "dv")):
        u = torch.randn(c[key].shape, generator=gen, dtype=torch.float64)
        f = []
        for s in (1e-5, -1e-5):
            cc = dict(c)
            cc[key] = c[key].double() + s * u
            f.append((reference(cc, 3)["out"] * c["do"].double()).sum())
        want = (f[0] - f[1]) / 2e-5
        assert math.isclose(float((ref[grad] * u).sum()), float(want), rel_tol=1e-6, abs_tol=1e-6)
