"""Sink tables on the GPU: a table belongs to the heads its units were cut for."""
import numpy as np
import pytest
import torch

from helpers import gpu_geom, make_case
from sliding_window_attention_device_gb300 import bdattn, synth

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda")


def case(B, Hq, Hkv, D, S, window, layout):
    w = synth.Workload("s", "s", B=B, Hq=Hq, Hkv=Hkv, D=D, S=S, cp_size=1, layout=layout, window=window)
    return make_case(w, 0, seed=3)


# name, D, Hkv, built for G, used with G, rows: tables of one size
OTHER_HEADS = [
    ("coarse", 512, 8, 4, 8, 1024, 256),
    ("coarse_fewer", 512, 8, 8, 4, 1024, 256),
    ("fine", 128, 1, 4, 8, 1024, 256),
]


@pytest.mark.parametrize("name,D,Hkv,G0,G1,S,W", OTHER_HEADS, ids=[c[0] for c in OTHER_HEADS])
def test_table_of_other_heads_is_reported(name, D, Hkv, G0, G1, S, W):
    """The units name query heads of the group they were cut for; a backward with another group reports it
    and writes nothing."""
    n = 4
    c = case(1, Hkv * G1, Hkv, D, S, W, ("explicit", (S - 40,), 40))
    g1 = gpu_geom(c)
    g0 = bdattn.geom(1, Hkv * G0, Hkv, D, S, S, 0, 0, S, W)
    assert bdattn.sink_seg_bytes(g0, n) == bdattn.sink_seg_bytes(g1, n)  # else the size check would do
    doc = torch.from_numpy(c["doc"]).to(DEV)
    q, k, v, do = (c[x].to(DEV) for x in ("q", "k", "v", "do"))
    seg1, status = bdattn.bd_attn_sink_seg_build(doc, g1, n)
    out, lse = bdattn.bd_attn_sink_fwd(q, k, v, seg1, g1, n, status)
    assert int(status.item()) == 0
    seg0, status = bdattn.bd_attn_sink_seg_build(doc, g0, n)
    assert int(status.item()) == 0
    ws = torch.zeros(bdattn.sink_bwd_workspace_bytes(g1, n), dtype=torch.uint8, device=DEV)
    for f in (bdattn.bd_attn_sink_bwd, bdattn.bd_attn_sink_bwd_deterministic):
        for dt in (torch.float32, torch.bfloat16):
            s = bdattn.new_status(DEV)
            dk, dv = (torch.full(k.shape, 7.0, dtype=dt, device=DEV) for _ in range(2))
            f(do, q, k, v, out, lse, seg0, g1, n, s, dt, dk=dk, dv=dv, workspace=ws)
            assert int(s.item()) == bdattn.STATUS_BOUNDS
            assert (dk == 7).all() and (dv == 7).all()
    s = bdattn.new_status(DEV)
    dk, dv = (torch.full(k.shape, 7.0, device=DEV) for _ in range(2))
    bdattn.bd_attn_bwd_prep(do, out, g1, s, ws[:bdattn.bwd_workspace_bytes(g1)])
    bdattn.bd_attn_sink_bwd_main(do, q, k, v, lse, seg0, g1, n, s, ws, dk, dv)
    assert int(s.item()) == bdattn.STATUS_BOUNDS
    assert (dk == 7).all() and (dv == 7).all()
    # the forward's part of a table does not depend on the heads
    s = bdattn.new_status(DEV)
    o, l = bdattn.bd_attn_sink_fwd(q, k, v, seg0, g1, n, s)
    assert int(s.item()) == 0 and torch.equal(o, out) and torch.equal(l, lse)
