"""How the sink backward's work is cut, on the GPU: cases sized from the rule, the cut read back from the table
and asserted, the gradients against the plain 64-bit form.

Coarse: a tile's first unit and units of the rows behind it, the sinks' key rows through slots, the other rows
written by the first unit. Fine (tiles for half the SMs or fewer): rows and query heads cut alike, whole tiles
through slots."""
import dataclasses

import pytest
import torch

from helpers import gpu_geom, make_case, oracle_geom
from sink_ref import check, reference
from sliding_window_attention_device_gb300 import bdattn, synth

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda")


def case(B, Hkv, G, D, S, layout, window, seed=4):
    w = synth.Workload("s", "s", B=B, Hq=Hkv * G, Hkv=Hkv, D=D, S=S, cp_size=1, layout=layout, window=window)
    return make_case(w, 0, seed=seed)


def of_kv_head(c, hk):
    """The case of one kv head and its group (heads are independent)."""
    w = c["w"]
    G = w.Hq // w.Hkv
    sub = dict(c, w=dataclasses.replace(w, Hq=G, Hkv=1))
    for n, h in (("q", G), ("do", G), ("k", 1), ("v", 1)):
        sub[n] = c[n][:, hk * h:(hk + 1) * h]
    return sub


def cut(seg, g):
    """Units by tile, [(q_begin, q_end, primary, slot, rbase, head0, heads)], and the key rows of a slot."""
    a = seg.cpu().tolist()
    at = (bdattn.seg_layout(g)["total"] + 3) // 4 * 4
    B, G, _, rows = a[28:32]
    assert (B, G) == (g.B, g.Hq // g.Hkv)
    tiles = {}
    for u in range(a[at]):
        w = a[at + 8 + 8 * u:at + 16 + 8 * u]
        tiles.setdefault(w[0], []).append(tuple(w[1:]))
    return tiles, rows


def run(c, n, g, seg, status, grad_dtype, det):
    q, k, v, do = (c[x].to(DEV) for x in ("q", "k", "v", "do"))
    out, lse = bdattn.bd_attn_sink_fwd(q, k, v, seg, g, n, status)
    nan = lambda like: torch.full(like.shape, float("nan"), dtype=grad_dtype, device=DEV)
    ws = torch.full((bdattn.sink_bwd_workspace_bytes(g, n),), 255, dtype=torch.uint8, device=DEV)
    f = bdattn.bd_attn_sink_bwd_deterministic if det else bdattn.bd_attn_sink_bwd
    dq, dk, dv = f(do, q, k, v, out, lse, seg, g, n, status, grad_dtype, dq=nan(q), dk=nan(k), dv=nan(v), workspace=ws)
    assert int(status.item()) == 0
    return dict(out=out, dq=dq, dk=dk, dv=dv)


def compare(res, c, n, heads, grad_dtype, og=None):
    G = c["w"].Hq // c["w"].Hkv
    for hk in heads:
        ref = reference(of_kv_head(c, hk), n, og)
        for x in ("out", "dq", "dk", "dv"):
            h = G if x in ("out", "dq") else 1
            check(f"{x} kv head {hk}", res[x][:, hk * h:(hk + 1) * h], ref, x, x == "out" or grad_dtype == torch.bfloat16)


COARSE = [
    # name, B, Hkv, G, D, window, n_sink
    ("d64_g3", 2, 4, 3, 64, 130, 5),
    ("d128_g2", 2, 4, 2, 128, 130, 4),
    ("d128_g8", 1, 8, 8, 128, 200, 4),
    ("d128_70_sinks", 2, 4, 2, 128, 200, 70),
    ("d64_short_window", 2, 4, 2, 64, 9, 128),
    ("d256_g2", 1, 8, 2, 256, 130, 4),
    ("d512_g2", 1, 2, 2, 512, 130, 16),
]


@pytest.mark.parametrize("grad_dtype", [torch.float32, torch.bfloat16], ids=["f32", "bf16"])
@pytest.mark.parametrize("name,B,Hkv,G,D,W,n", COARSE, ids=[c[0] for c in COARSE])
def test_coarse(name, B, Hkv, G, D, W, n, grad_dtype):
    c = case(B, Hkv, G, D, 1500, ("explicit", (60, 1380), 60), W)
    g = gpu_geom(c)
    seg, status = bdattn.bd_attn_sink_seg_build(torch.from_numpy(c["doc"]).to(DEV), g, n)
    tiles, rows = cut(seg, g)
    assert rows == n
    several = {t: u for t, u in tiles.items() if len(u) > 1}
    assert several and any(len(u) == 1 for u in tiles.values())
    for t, u in several.items():
        assert sum(x[2] for x in u) == 1 and all(x[5:] == (0, G) and x[3] >= 0 for x in u)
        edges = sorted(x[:2] for x in u)
        assert all(a[1] == b[0] for a, b in zip(edges, edges[1:]))
    compare(run(c, n, g, seg, status, grad_dtype, False), c, n, (0, Hkv - 1), grad_dtype)
    if grad_dtype == torch.bfloat16:
        compare(run(c, n, g, seg, status, grad_dtype, True), c, n, (Hkv // 2,), grad_dtype)


@pytest.mark.parametrize("D", [64, 128])
def test_coarse_dropout_and_token_major(D):
    c = case(2, 4, 2, D, 1500, ("explicit", (60, 1380), 60), 130)
    c.update(dropout_p=0.25, drop_seed=77)
    g = gpu_geom(c)
    g.kv_layout = bdattn.KV_SBHD
    seg, status = bdattn.bd_attn_sink_seg_build(torch.from_numpy(c["doc"]).to(DEV), g, 6)
    assert any(len(u) > 1 for u in cut(seg, g)[0].values()) and cut(seg, g)[1] == 6
    t = dict(c, k=c["k"].permute(2, 0, 1, 3).contiguous(), v=c["v"].permute(2, 0, 1, 3).contiguous())
    res = run(t, 6, g, seg, status, torch.bfloat16, False)
    for x in ("dk", "dv"):
        res[x] = res[x].permute(1, 2, 0, 3)
    compare(res, c, 6, (0,), torch.bfloat16, oracle_geom(c))


@pytest.mark.parametrize("D,Hkv", [(64, 8), (256, 8)])
def test_coarse_chunks(D, Hkv):
    """K/V in two chunks, each coarse with several units in the first; gradients of the exact out."""
    n, W = 6, 130
    c = case(2, Hkv, 2, D, 1500, ("explicit", (60, 1380), 60), W)
    w = c["w"]
    doc = torch.from_numpy(c["doc"]).to(DEV)
    q, k, v, do = (c[x].to(DEV) for x in ("q", "k", "v", "do"))
    gw = gpu_geom(c)
    seg, status = bdattn.bd_attn_sink_seg_build(doc, gw, n)
    out, lse = bdattn.bd_attn_sink_fwd(q, k, v, seg, gw, n, status)
    parts = []
    for a, e in ((0, 800), (800, 1500)):
        g = bdattn.geom(w.B, w.Hq, w.Hkv, D, w.S, w.L, 0, a, e - a, W)
        s, _ = bdattn.bd_attn_sink_seg_build(doc, g, n, kv_chunk=True, status=status)
        assert cut(s, g)[1] == n and any(len(u) > 1 for u in cut(s, g)[0].values()) == (a == 0)
        parts.append((g, s, k[:, :, a:e].contiguous(), v[:, :, a:e].contiguous()))
    ws = torch.full((max(bdattn.sink_bwd_workspace_bytes(p[0], n) for p in parts),), 255, dtype=torch.uint8, device=DEV)
    head = ws[:bdattn.bwd_workspace_bytes(gw)]
    bdattn.bd_attn_bwd_prep(do, out, gw, status, head)
    grads = []
    for g, s, kc, vc in parts:
        dk, dv = (torch.full_like(kc, float("nan")) for _ in range(2))
        bdattn.bd_attn_sink_bwd_main(do, q, kc, vc, lse, s, g, n, status, ws, dk, dv)
        grads.append((dk, dv))
    dq = torch.empty_like(q)
    bdattn.bd_attn_bwd_finalize(gw, status, head, dq)
    assert int(status.item()) == 0
    dk, dv = (torch.cat([x[i] for x in grads], 2) for i in range(2))
    compare(dict(out=out, dq=dq, dk=dk, dv=dv), c, n, (0, Hkv - 1), torch.bfloat16)


FINE = [
    # name, G, D, rows, heads of a unit
    ("d64", 7, 64, 1664, 2),
    ("d128", 7, 128, 1664, 2),
    ("d256", 7, 256, 1664, 2),
    ("d512", 7, 512, 1024, 4),
]


@pytest.mark.parametrize("grad_dtype", [torch.float32, torch.bfloat16], ids=["f32", "bf16"])
@pytest.mark.parametrize("name,G,D,S,heads", FINE, ids=[c[0] for c in FINE])
def test_fine_head_groups(name, G, D, S, heads, grad_dtype):
    """Units of several heads whose number does not divide the group's."""
    c = case(1, 1, G, D, S, ("explicit", (50, S - 90), 40), 200)
    g = gpu_geom(c)
    n = 4
    seg, status = bdattn.bd_attn_sink_seg_build(torch.from_numpy(c["doc"]).to(DEV), g, n)
    tiles, rows = cut(seg, g)
    assert rows == 128
    groups = {(h, min(heads, G - h)) for h in range(0, G, heads)}
    assert all({x[5:] for x in u} == groups for u in tiles.values()) and any(x[1] < heads for x in groups)
    assert any(len(u) > len(groups) for u in tiles.values())  # rows are cut too
    compare(run(c, n, g, seg, status, grad_dtype, False), c, n, (0,), grad_dtype)
    compare(run(c, n, g, seg, status, grad_dtype, True), c, n, (0,), grad_dtype)
