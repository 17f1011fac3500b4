"""Attention sinks on the GPU against the plain 64-bit form: forward, backward
(both accumulation orders, both gradient types), K/V chunks, token-major K/V,
dropout, and the tables, at the sizes and masks where they can go wrong."""
import numpy as np
import pytest
import torch

import oracle
from helpers import gpu_geom, make_case, oracle_geom
from sink_ref import check, check_lse, reference
from sliding_window_attention_device_gb300 import bdattn, synth

pytestmark = pytest.mark.gpu


def W(B, Hq, Hkv, D, S, cp, layout, window, kv="full"):
    return synth.Workload("s", "s", B=B, Hq=Hq, Hkv=Hkv, D=D, S=S, cp_size=cp, layout=layout, window=window,
                          ranks=tuple(range(cp)), kv=kv)


# name, workload, n_sink, ranks
CASES = [
    ("d64_small", W(1, 2, 1, 64, 256, 4, ("explicit", (100, 90, 50), 16), 32), 4, (0, 2, 3)),
    ("d64_odd", W(2, 6, 2, 64, 999, 3, ("uniform", 20, 500, 13), 77), 5, (0, 1, 2)),
    ("d64_window1", W(1, 2, 2, 64, 512, 2, ("uniform", 3, 200, 5), 1), 1, (0, 1)),
    ("d64_tiny_window_tiny_docs", W(2, 2, 1, 64, 640, 2, ("uniform", 1, 40, 17), 7), 3, (0, 1)),
    ("d64_long_doc", W(1, 2, 1, 64, 4096, 2, ("single",), 130), 4, (1,)),
    ("d128_far_straddle", W(1, 4, 2, 128, 2048, 4, ("single",), 200), 4, (0, 2, 3)),
    ("d128_sinks_cross_tile", W(1, 2, 1, 128, 1536, 2, ("explicit", (100, 1000, 400), 36), 150), 60, (0, 1)),
    ("d128_128_sinks", W(1, 2, 1, 128, 1536, 3, ("explicit", (70, 1300, 100), 66), 129), 128, (0, 1, 2)),
    ("d128_sinks_meet_window", W(1, 4, 1, 128, 900, 2, ("explicit", (333, 500), 67), 128), 90, (0, 1)),
    ("d128_window_over_all", W(1, 2, 1, 128, 640, 2, ("uniform", 100, 300, 9), 5000), 4, (0, 1)),
    ("d128_no_window", W(1, 2, 1, 128, 640, 2, ("uniform", 100, 300, 9), 0), 4, (1,)),
    ("d128_all_pad_shard", W(1, 2, 1, 128, 1024, 4, ("explicit", (300, 200), 524), 60), 4, (1, 2, 3)),
    ("d128_one_row", W(1, 2, 1, 128, 200, 200, ("single",), 20), 3, (0, 3, 22, 199)),
    ("d128_many_long_docs", W(2, 4, 2, 128, 2560, 2, ("uniform", 300, 700, 40), 128), 17, (0, 1)),
    ("d256_far_straddle", W(1, 4, 2, 256, 1536, 3, ("uniform", 400, 1500, 20), 128), 4, (0, 1, 2)),
    ("d256_small_window", W(1, 2, 2, 256, 600, 2, ("uniform", 30, 300, 11), 9), 33, (0, 1)),
    ("d512_far_straddle", W(1, 4, 2, 512, 1280, 4, ("uniform", 400, 1200, 20), 140), 16, (1, 3)),
    ("d512_small_window", W(1, 2, 1, 512, 500, 2, ("uniform", 30, 300, 11), 9), 4, (0, 1)),
]


def run(c, n_sink, grad_dtype=torch.float32, det=False, layout=bdattn.KV_BHSD, stream=None):
    g = gpu_geom(c)
    g.kv_layout = layout
    dev = torch.device("cuda")
    q, k, v, do = (c[n].to(dev) for n in ("q", "k", "v", "do"))
    if layout == bdattn.KV_SBHD:
        k, v = (t.permute(2, 0, 1, 3).contiguous() for t in (k, v))
    seg, status = bdattn.bd_attn_sink_seg_build(torch.from_numpy(c["doc"]).to(dev), g, n_sink)
    nan = lambda *s, dt: torch.full(s, float("nan"), dtype=dt, device=dev)  # what a call leaves unwritten shows
    out, lse = bdattn.bd_attn_sink_fwd(q, k, v, seg, g, n_sink, status, out=nan(*q.shape, dt=torch.bfloat16),
                                       lse=nan(*q.shape[:3], dt=torch.float32))
    f = bdattn.bd_attn_sink_bwd_deterministic if det else bdattn.bd_attn_sink_bwd
    ws = torch.full((bdattn.sink_bwd_workspace_bytes(g, n_sink),), 255, dtype=torch.uint8, device=dev)
    dq, dk, dv = f(do, q, k, v, out, lse, seg, g, n_sink, status, grad_dtype, dq=nan(*q.shape, dt=grad_dtype),
                   dk=nan(*k.shape, dt=grad_dtype), dv=nan(*k.shape, dt=grad_dtype), workspace=ws)
    torch.cuda.synchronize()
    assert int(status.item()) == 0, f"status {int(status.item()):#x}"
    if layout == bdattn.KV_SBHD:
        dk, dv = (t.permute(1, 2, 0, 3).contiguous() for t in (dk, dv))
    return dict(out=out, lse=lse, dq=dq, dk=dk, dv=dv)


def check_all(name, res, ref, grad_dtype=torch.float32):
    check(f"{name} out", res["out"], ref, "out", True)
    check_lse(name, res["lse"], ref)
    for n in ("dq", "dk", "dv"):
        check(f"{name} {n}", res[n], ref, n, grad_dtype == torch.bfloat16)


@pytest.mark.parametrize("name,w,n,ranks", CASES, ids=[c[0] for c in CASES])
def test_parity(name, w, n, ranks):
    for r in ranks:
        c = make_case(w, r, seed=r + 1)
        check_all(f"{name} r{r}", run(c, n), reference(c, n))


@pytest.mark.parametrize("det", [False, True])
@pytest.mark.parametrize("D,Hkv", [(64, 8), (128, 8), (256, 8), (512, 2)])
def test_long_documents_over_many_tiles(D, Hkv, det):
    """Tiles for most SMs, so that only the rows behind a sink tile's first unit are cut off, and bf16
    gradients, which end in one launch."""
    c = make_case(W(1, Hkv, Hkv, D, 2304, 3, ("explicit", (1000, 1250), 54), 130), 2, seed=6)
    ref = reference(c, 5)
    check_all("coarse", run(c, 5, torch.bfloat16, det=det), ref, torch.bfloat16)
    c = make_case(W(1, Hkv, Hkv, D, 1800, 1, ("explicit", (20, 1700), 80), 200), 0, seed=7)
    ref = reference(c, 70)
    check_all("coarse 70", run(c, 70, det=det), ref)


@pytest.mark.parametrize("D", [64, 128, 256, 512])
def test_bf16_gradients_and_token_major(D):
    c = make_case(W(2, 4, 2, D, 900, 2, ("uniform", 50, 600, 30), 140), 1, seed=3)
    ref = reference(c, 6)
    check_all("bf16", run(c, 6, torch.bfloat16), ref, torch.bfloat16)
    check_all("token-major", run(c, 6, torch.bfloat16, layout=bdattn.KV_SBHD), ref, torch.bfloat16)


@pytest.mark.parametrize("D", [64, 128, 256, 512])
def test_deterministic(D):
    """Twice the same bits, with other calls in between, and the right ones."""
    c = make_case(W(1, 4, 2, D, 1300, 2, ("explicit", (90, 1100), 110), 130), 1, seed=5)
    ref = reference(c, 20)
    a = run(c, 20, det=True)
    check_all("det", a, ref)
    run(make_case(c["w"], 0, seed=6), 20, det=True)
    b = run(c, 20, det=True)
    for n in a:
        assert torch.equal(a[n], b[n]), n
    # dk / dv add their partials in a fixed order in the other backward too
    x, y = run(c, 20), run(c, 20)
    assert torch.equal(x["dk"], y["dk"]) and torch.equal(x["dv"], y["dv"])


@pytest.mark.parametrize("D", [64, 128, 256, 512])
def test_dropout(D):
    c = make_case(W(1, 4, 2, D, 700, 2, ("explicit", (90, 500), 110), 100), 1, seed=7)
    c.update(dropout_p=0.25, drop_seed=1234567890123)
    ref = reference(c, 9, oracle_geom(c))
    check_all("dropout", run(c, 9), ref)
    check_all("dropout det", run(c, 9, det=True), ref)


@pytest.mark.parametrize("D,n,window", [(64, 4, 100), (128, 70, 130), (256, 4, 9), (512, 16, 128)])
def test_chunks(D, n, window):
    """K/V in chunks that cut documents and sinks: merged forward, summed backward."""
    w = W(2, 4, 2, D, 1100, 2, ("explicit", (70, 900), 130), window)
    c = make_case(w, 1, seed=11)
    ref = reference(c, n)
    dev = torch.device("cuda")
    doc = torch.from_numpy(c["doc"]).to(dev)
    q, k, v, do = (c[x].to(dev) for x in ("q", "k", "v", "do"))
    edges = [0, 75, 130, 640, 641, c["S_kv"]]
    status = bdattn.new_status(dev)
    out = torch.full(q.shape, float("nan"), dtype=torch.bfloat16, device=dev)
    lse = torch.full(q.shape[:3], float("-inf"), device=dev)
    parts = []
    for a, e in zip(edges, edges[1:]):
        g = bdattn.geom(w.B, w.Hq, w.Hkv, D, w.S, w.L, c["row_offset"], a, e - a, window)
        seg, _ = bdattn.bd_attn_sink_seg_build(doc, g, n, kv_chunk=True, status=status)
        kc, vc = k[:, :, a:e].contiguous(), v[:, :, a:e].contiguous()
        bdattn.bd_attn_sink_fwd_merge(q, kc, vc, seg, g, n, status, out, lse)
        parts.append((g, seg, kc, vc))
    check_lse("chunks", lse, ref)
    g0 = parts[0][0]
    ws = torch.empty(max(bdattn.sink_bwd_workspace_bytes(p[0], n) for p in parts), dtype=torch.uint8, device=dev)
    head = ws[:bdattn.bwd_workspace_bytes(g0)]
    # the gradients of the exact out, so that only the backward's own roundings count
    o_exact = ref["out"].to(torch.bfloat16).to(dev)
    l_exact = ref["lse"].float().to(dev)
    bdattn.bd_attn_bwd_prep(do, o_exact, g0, status, head)
    dks, dvs = [], []
    for g, seg, kc, vc in parts:
        dk, dv = torch.full_like(kc, float("nan"), dtype=torch.float32), torch.full_like(vc, float("nan"), dtype=torch.float32)
        bdattn.bd_attn_sink_bwd_main(do, q, kc, vc, l_exact, seg, g, n, status, ws, dk, dv)
        dks.append(dk)
        dvs.append(dv)
    dq = torch.empty(q.shape, dtype=torch.float32, device=dev)
    bdattn.bd_attn_bwd_finalize(g0, status, head, dq)
    assert int(status.item()) == 0
    # every merge rounds the running out once more, as each of the up to five chunks may
    ref["e_out"], ref["r_out"] = 5 * ref["e_out"], 25 * ref["r_out"]
    check("chunks out", out, ref, "out", True)
    check("chunks dq", dq, ref, "dq", False)
    check("chunks dk", torch.cat(dks, 2), ref, "dk", False)
    check("chunks dv", torch.cat(dvs, 2), ref, "dv", False)


@pytest.mark.parametrize("D", [64, 128, 256, 512])
def test_no_sinks_is_the_plain_window(D):
    """n_sink 0, or sinks without a window: the bits of the ordinary forward."""
    for window, n in ((60, 0), (0, 7)):
        c = make_case(W(1, 4, 2, D, 600, 2, ("uniform", 50, 300, 30), window), 1, seed=2)
        g = gpu_geom(c)
        dev = torch.device("cuda")
        q, k, v, do = (c[x].to(dev) for x in ("q", "k", "v", "do"))
        doc = torch.from_numpy(c["doc"]).to(dev)
        seg, st = bdattn.bd_attn_seg_build(doc, g)
        out, lse = bdattn.bd_attn_fwd(q, k, v, seg, g, st)
        dq, dk, dv = bdattn.bd_attn_bwd_deterministic(do, q, k, v, out, lse, seg, g, st)
        res = run(c, n, det=True)
        for a, b in ((out, "out"), (lse, "lse"), (dq, "dq"), (dk, "dk"), (dv, "dv")):
            assert torch.equal(a, res[b]), b


def test_gradients_against_differences():
    """(f(x + e) - f(x - e)) / 2e of sum(out dO) along random directions, in 64 bits of the plain form."""
    c = make_case(W(1, 2, 1, 64, 300, 2, ("explicit", (30, 250), 20), 40), 1, seed=4)
    n, eps = 5, 1e-4
    res = run(c, n)
    gen = torch.Generator().manual_seed(0)
    for key, grad in (("q", "dq"), ("k", "dk"), ("v", "dv")):
        u = torch.randn(c[key].shape, generator=gen, dtype=torch.float64)
        f = []
        for s in (eps, -eps):
            cc = dict(c)
            cc[key] = c[key].double() + s * u
            f.append((reference(cc, n)["out"] * c["do"].double()).sum())
        want = (f[0] - f[1]) / (2 * eps)
        ref = reference(c, n)
        got = (res[grad].double().cpu() * u).sum()
        # the bound of every element along the direction, its rms part taken as independent
        lim = (ref["r_" + grad] * u ** 2).sum().sqrt() * 4 + 1e-3
        assert abs(got - want) <= lim, (key, float(got), float(want), float(lim))


def test_graph_replay_and_other_stream():
    """Captured once, replayed on new inputs; and the same on a side stream, eagerly."""
    w, n = W(1, 4, 2, 128, 800, 2, ("explicit", (50, 700), 50), 130), 4
    c1, c2 = make_case(w, 1, seed=1), make_case(w, 1, seed=2)
    c2["doc"] = c1["doc"]
    dev = torch.device("cuda")
    g = gpu_geom(c1)
    x = {k: c1[k].to(dev) for k in ("q", "k", "v", "do")}
    doc = torch.from_numpy(c1["doc"]).to(dev)
    status = bdattn.new_status(dev)

    def step(stream=None):
        seg, _ = bdattn.bd_attn_sink_seg_build(doc, g, n, status=status, stream=stream)
        out, lse = bdattn.bd_attn_sink_fwd(x["q"], x["k"], x["v"], seg, g, n, status, stream=stream)
        return (out, lse) + bdattn.bd_attn_sink_bwd(x["do"], x["q"], x["k"], x["v"], out, lse, seg, g, n, status,
                                                    torch.bfloat16, stream=stream)

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        res = step()
    for k in x:
        x[k].copy_(c2[k])
    graph.replay()
    torch.cuda.synchronize()
    ref = reference(c2, n)
    names = ("out", "lse", "dq", "dk", "dv")
    check_all("replay", dict(zip(names, res)), ref, torch.bfloat16)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    res2 = step(side)
    side.synchronize()
    check_all("side stream", dict(zip(names, res2)), ref, torch.bfloat16)
    assert int(status.item()) == 0


def test_table_belongs_to_its_n_sink():
    w = W(1, 2, 1, 128, 600, 2, ("explicit", (50, 500), 50), 130)
    c = make_case(w, 1)
    dev = torch.device("cuda")
    g = gpu_geom(c)
    q, k, v, do = (c[x].to(dev) for x in ("q", "k", "v", "do"))
    doc = torch.from_numpy(c["doc"]).to(dev)
    seg, status = bdattn.bd_attn_sink_seg_build(doc, g, 4)
    assert bdattn.read_seg(seg, g)["rows"][0]["kv_need_lo"] == 50
    mark = lambda: torch.full(q.shape, 7.0, dtype=torch.bfloat16, device=dev)
    out, lse = bdattn.bd_attn_sink_fwd(q, k, v, seg, g, 4, status)
    assert int(status.item()) == 0
    for call in (lambda s, o: bdattn.bd_attn_fwd(q, k, v, seg[:bdattn.seg_bytes(g) // 4], g, s, out=o),
                 lambda s, o: bdattn.bd_attn_sink_fwd(q, k, v, seg, g, 5, s, out=o)):
        s, o = bdattn.new_status(dev), mark()
        call(s, o)
        assert int(s.item()) & bdattn.STATUS_BOUNDS and (o == 7).all()
    # an ordinary table in a buffer of a sink table's size
    plain = torch.zeros_like(seg)
    bdattn.bd_attn_seg_build(doc, g, seg=plain[:bdattn.seg_bytes(g) // 4])
    s, o = bdattn.new_status(dev), mark()
    dk = torch.full(k.shape, 7.0, device=dev)
    bdattn.bd_attn_sink_bwd(do, q, k, v, out, lse, plain, g, 4, s, dk=dk)
    assert int(s.item()) & bdattn.STATUS_BOUNDS and (dk == 7).all()


def test_missing_sinks_are_reported():
    """A K/V buffer that holds the window but not the straddling document's sinks."""
    w = W(1, 2, 1, 128, 1024, 2, ("single",), 100)
    dev = torch.device("cuda")
    doc = torch.ones(1, 1024, dtype=torch.int32, device=dev)
    g = bdattn.geom(1, 2, 1, 128, 1024, 512, 512, 400, 624, 100)
    seg, status = bdattn.bd_attn_sink_seg_build(doc, g, 4)
    assert int(status.item()) == bdattn.STATUS_KV_RANGE
    seg, status = bdattn.bd_attn_sink_seg_build(doc, g, 4, kv_chunk=True)
    assert int(status.item()) == 0


def test_refusals():
    dev = torch.device("cuda")
    g = bdattn.geom(1, 2, 1, 128, 512, 256, 256, 0, 512, 100)
    doc = torch.ones(1, 512, dtype=torch.int32, device=dev)
    for n in (-1, 129):
        with pytest.raises(ValueError):
            bdattn.bd_attn_sink_seg_build(doc, g, n)
    with pytest.raises(ValueError):
        bdattn.bd_attn_sink_seg_build(doc.cpu(), g, 4)
    with pytest.raises(ValueError):
        bdattn.bd_attn_sink_seg_build(doc.long(), g, 4)
    seg, status = bdattn.bd_attn_sink_seg_build(doc, g, 4)
    q = torch.zeros(1, 2, 256, 128, dtype=torch.bfloat16, device=dev)
    k = torch.zeros(1, 1, 512, 128, dtype=torch.bfloat16, device=dev)
    for bad in (q.half(), q[:, :1], q.transpose(2, 3).contiguous().transpose(2, 3)):
        with pytest.raises(ValueError):
            bdattn.bd_attn_sink_fwd(bad, k, k, seg, g, 4, status)
    with pytest.raises(ValueError):
        bdattn.bd_attn_sink_fwd(q, k, k, seg[:-4], g, 4, status)
    with pytest.raises(ValueError):
        bdattn.bd_attn_sink_bwd(q, q, k, k, q, torch.zeros(1, 2, 256, device=dev), seg, g, 4, status, torch.float16)
    with pytest.raises(ValueError):
        bdattn.bd_attn_sink_fwd_merge(q, k, k, seg, g, 4, status, None, None)


@pytest.mark.parametrize("D", [64, 128, 256, 512])
def test_scale(D):
    """A softmax scale of its own: the reference with q scaled by scale / D^-0.5 (a power of two, so exactly)."""
    c = make_case(W(1, 2, 1, D, 500, 2, ("explicit", (40, 420), 40), 60), 1, seed=8)
    g = gpu_geom(c)
    g.scale = 0.5 * D ** -0.5
    dev = torch.device("cuda")
    q, k, v, do = (c[x].to(dev) for x in ("q", "k", "v", "do"))
    seg, status = bdattn.bd_attn_sink_seg_build(torch.from_numpy(c["doc"]).to(dev), g, 4)
    out, lse = bdattn.bd_attn_sink_fwd(q, k, v, seg, g, 4, status)
    dq, dk, dv = bdattn.bd_attn_sink_bwd(do, q, k, v, out, lse, seg, g, 4, status)
    assert int(status.item()) == 0
    cc = dict(c)
    cc["q"] = (c["q"].float() * 0.5).bfloat16()
    ref = reference(cc, 4)
    for x in ("dq", "e_dq"):  # d/dq of f(q / 2)
        ref[x] = ref[x] * 0.5
    ref["r_dq"] = ref["r_dq"] * 0.25
    check_all("scale", dict(out=out, lse=lse, dq=dq, dk=dk, dv=dv), ref)


def test_ids_in_any_order():
    """Document ids that fall from one document to the next, and every id negative or repeated refused."""
    c = make_case(W(2, 2, 1, 64, 700, 2, ("uniform", 60, 300, 30), 50), 1, seed=3)
    c["doc"] = np.where(c["doc"] > 0, 1000 - c["doc"], 0).astype(np.int32)
    check_all("falling ids", run(c, 4), reference(c, 4))
    g = gpu_geom(c)
    doc = c["doc"].copy()
    doc[0, :20] = doc[0, 500]  # a local document's id before its run
    _, status = bdattn.bd_attn_sink_seg_build(torch.from_numpy(doc).cuda(), g, 4)
    assert int(status.item()) == bdattn.STATUS_LAYOUT


@pytest.mark.parametrize("D", [64, 128, 256, 512])
def test_window_of_any_size(D):
    """A window of 2^31 - 1: position + window must not wrap, with sinks and without."""
    c = make_case(W(1, 2, 1, D, 500, 2, ("explicit", (40, 420), 40), 2 ** 31 - 1), 1, seed=8)
    cc = dict(c)
    cc["window"] = 0
    ref = reference(cc, 0)
    check_all("sinks", run(c, 4), ref)
    check_all("none", run(c, 0), ref)
    g = gpu_geom(c)
    dev = torch.device("cuda")
    q, k, v, do = (c[x].to(dev) for x in ("q", "k", "v", "do"))
    seg, status = bdattn.bd_attn_seg_build(torch.from_numpy(c["doc"]).to(dev), g)
    out, lse = bdattn.bd_attn_fwd(q, k, v, seg, g, status)
    dq, dk, dv = bdattn.bd_attn_bwd(do, q, k, v, out, lse, seg, g, status)
    assert int(status.item()) == 0
    check_all("ordinary", dict(out=out, lse=lse, dq=dq, dk=dk, dv=dv), ref)
