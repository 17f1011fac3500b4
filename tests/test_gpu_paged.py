"""The paged cache on the GPU: append against indexing, decode against a plain
64-bit form, and a prompt and its continuation through both next to the sink
attention of the whole sequence.

Decode rounds the weights P to bf16 and then out: |error| <= 2^-8 (sum P |v| +
|out|), plus 1e-4 of those magnitudes for fp32 sums and exponentials; over a
tensor the roundings are held to the root of their summed squares. lse as in the
forward, 2e-4."""
import math

import pytest
import torch

from sink_ref import H, LSE_ABS, SLACK
from sliding_window_attention_device_gb300 import bdattn

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda")


def cache(lens, Hkv, D, page, seed=0, spare=3, extra_pages=0):
    """Pages in random order; table entries and places behind a sequence's end hold what must not be read."""
    gen = torch.Generator().manual_seed(seed)
    need = [-(-n // page) for n in lens]
    n_pages = sum(need) + spare
    order = torch.randperm(n_pages, generator=gen).tolist()
    max_pages = max(1, max(need)) + extra_pages
    table = torch.full((len(lens), max_pages), 1 << 30, dtype=torch.int32)
    k = torch.full((n_pages, Hkv, page, D), float("nan"), dtype=torch.bfloat16)
    v = torch.full((n_pages, Hkv, page, D), float("nan"), dtype=torch.bfloat16)
    at, rows = 0, []
    for b, n in enumerate(lens):
        ids = order[at:at + need[b]]
        at += need[b]
        table[b, :need[b]] = torch.tensor(ids, dtype=torch.int32)
        kk = torch.randn(n, Hkv, D, generator=gen).bfloat16()
        vv = torch.randn(n, Hkv, D, generator=gen).bfloat16()
        for i, pg in enumerate(ids):
            m = min(page, n - i * page)
            k[pg, :, :m] = kk[i * page:i * page + m].transpose(0, 1)
            v[pg, :, :m] = vv[i * page:i * page + m].transpose(0, 1)
        rows.append((kk, vv))
    return table, k, v, rows


def visible(n, window, n_sink):
    s = torch.arange(n)
    return (s >= n - window) | (s < n_sink) if window > 0 else torch.ones(n, dtype=torch.bool)


def plain(q, rows, window, n_sink, scale=None):
    B, Hq, D = q.shape
    out, e, r2 = (torch.zeros(B, Hq, D, dtype=torch.float64) for _ in range(3))
    lse = torch.full((B, Hq), -math.inf, dtype=torch.float64)
    for b, (k, v) in enumerate(rows):
        if len(k) == 0:
            continue
        see = visible(len(k), window, n_sink)
        G = Hq // k.shape[1]
        for h in range(Hq):
            kk, vv = k[see, h // G].double(), v[see, h // G].double()
            x = kk @ q[b, h].double() * (scale or D ** -0.5)
            lse[b, h] = torch.logsumexp(x, 0)
            p = torch.exp(x - lse[b, h])
            out[b, h] = p @ vv
            e[b, h] = (H + SLACK) * (p @ vv.abs()) + H * out[b, h].abs()
            r2[b, h] = H ** 2 * (p ** 2 @ vv ** 2 + out[b, h] ** 2)
    return out, lse, e, r2


def check(got, got_lse, want):
    out, lse, e, r2 = want
    d, dl = got.double().cpu(), got_lse.double().cpu()
    none = torch.isinf(lse)
    assert torch.equal(dl[none], lse[none]) and (d[none] == 0).all()
    assert torch.isfinite(d).all()
    if (~none).any():
        assert (dl - lse)[~none].abs().max() <= LSE_ABS
    err = (d - out).abs()
    assert (err <= e + 1e-7).all(), float((err - e).max())
    assert err.pow(2).mean().sqrt() <= r2.mean().sqrt() + SLACK * out.pow(2).mean().sqrt() + 1e-7


def decode(lens, Hq, Hkv, D, page, window=0, n_sink=0, seed=0, scale=0.0, stream=None, extra_pages=0):
    table, k, v, rows = cache(lens, Hkv, D, page, seed, extra_pages=extra_pages)
    q = torch.randn(len(lens), Hq, D, generator=torch.Generator().manual_seed(seed + 1)).bfloat16()
    pg = bdattn.paged_geom(len(lens), Hq, Hkv, D, k.shape[0], page, table.shape[1], window, n_sink, scale)
    status = bdattn.new_status(DEV)
    out = torch.full(q.shape, float("nan"), dtype=torch.bfloat16, device=DEV)
    lse = torch.full(q.shape[:2], float("nan"), device=DEV)
    ws = torch.full((bdattn.paged_decode_workspace_bytes(pg),), 255, dtype=torch.uint8, device=DEV)
    bdattn.bd_attn_paged_decode(q.to(DEV), k.to(DEV), v.to(DEV), table.to(DEV),
                                torch.tensor(lens, dtype=torch.int32, device=DEV), pg, status, out, lse, ws, stream)
    torch.cuda.synchronize()
    assert int(status.item()) == 0, f"status {int(status.item()):#x}"
    check(out, lse, plain(q, rows, window, n_sink, scale or None))
    return out, lse


DECODE = [
    # name, lens, Hq, Hkv, D, page, window, n_sink
    ("one_key", [1], 1, 1, 64, 16, 0, 0),
    ("lengths_0_to_33", list(range(34)), 2, 1, 64, 16, 0, 0),
    ("all_empty", [0, 0, 0], 4, 2, 128, 16, 0, 0),
    ("page_of_one", [5, 40], 4, 2, 128, 1, 0, 0),
    ("odd_page", [5, 300, 77], 6, 2, 128, 7, 0, 0),
    ("page_200", [199, 200, 201, 650], 8, 2, 128, 200, 0, 0),
    ("groups_of_3", [100, 513], 9, 3, 128, 32, 0, 0),
    ("groups_of_8", [1000, 17, 0, 255], 16, 2, 128, 16, 0, 0),
    ("groups_of_12", [300, 90], 24, 2, 128, 16, 0, 0),
    ("groups_of_20", [300, 90], 20, 1, 64, 16, 0, 0),
    ("groups_of_16_d256", [400, 31], 32, 2, 256, 32, 0, 0),
    ("groups_of_20_d512", [400, 31], 20, 1, 512, 32, 0, 0),
    ("window", [1, 99, 100, 101, 900], 4, 2, 128, 16, 100, 0),
    ("window_sinks", [1, 4, 5, 99, 104, 105, 900], 4, 2, 128, 16, 100, 4),
    ("window1", [1, 2, 50], 2, 2, 64, 16, 1, 0),
    ("window1_sink1", [1, 2, 50], 2, 2, 64, 16, 1, 1),
    ("sinks_past_window", [50, 300, 1000], 4, 2, 128, 16, 64, 200),
    ("window_and_sinks_of_any_size", [50, 700], 4, 2, 128, 16, 2 ** 31 - 1, 2 ** 31 - 1),
    ("sinks_of_any_size", [50, 700], 4, 2, 128, 16, 60, 2 ** 31 - 1),
    ("d256", [2000, 0, 700, 1], 8, 4, 256, 16, 512, 4),
    ("d512", [900, 33, 16], 8, 2, 512, 64, 0, 0),
    ("long_split", [20011], 8, 1, 128, 64, 0, 0),
    ("long_split_d64", [30000, 1], 8, 2, 64, 128, 0, 0),
    ("long_split_d512", [9000], 2, 1, 512, 64, 0, 0),
    ("many_short", [(7 * i) % 50 for i in range(300)], 4, 2, 64, 16, 0, 0),
    ("many_mixed", [(131 * i) % 700 for i in range(140)], 8, 4, 128, 16, 256, 4),
]


@pytest.mark.parametrize("name,lens,Hq,Hkv,D,page,window,n", DECODE, ids=[c[0] for c in DECODE])
def test_decode(name, lens, Hq, Hkv, D, page, window, n):
    decode(lens, Hq, Hkv, D, page, window, n, seed=len(name))


def test_decode_scale_and_spare_table():
    decode([300, 20], 4, 2, 128, 16, scale=0.3, extra_pages=37)


def test_decode_large_scores():
    """Keys whose scores grow along the sequence: the running maximum is raised again and again."""
    lens, D = [3000], 64
    table, k, v, rows = cache(lens, 1, D, 16)
    q = torch.ones(1, 2, D).bfloat16()
    ramp = (torch.arange(3000) / 8).bfloat16()[:, None, None].expand(3000, 1, D).contiguous()
    rows = [(ramp, rows[0][1])]
    for i in range(table.shape[1]):
        m = min(16, 3000 - 16 * i)
        k[table[0, i], :, :m] = ramp[16 * i:16 * i + m].transpose(0, 1)
    pg = bdattn.paged_geom(1, 2, 1, D, k.shape[0], 16, table.shape[1])
    status = bdattn.new_status(DEV)
    out, lse = bdattn.bd_attn_paged_decode(q.to(DEV), k.to(DEV), v.to(DEV), table.to(DEV),
                                           torch.tensor(lens, dtype=torch.int32, device=DEV), pg, status)
    want = plain(q, rows, 0, 0)
    # scores up to 3000: a score is off by 2^-23 of itself, so the weights by 4e-4 and lse by 4e-4
    out_w, lse_w, e, r2 = want
    assert (lse.double().cpu() - lse_w).abs().max() <= 3000 * 2.0 ** -22
    assert ((out.double().cpu() - out_w).abs() <= e + 3000 * 2.0 ** -22 * 4).all()


def test_decode_repeats_bitwise():
    lens = [5000, 12, 0, 900]
    a = decode(lens, 8, 2, 128, 16, seed=3)
    decode([3], 8, 2, 128, 16, seed=4)
    b = decode(lens, 8, 2, 128, 16, seed=3)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


def test_decode_graph_and_stream():
    """Captured at one set of lengths, replayed at others; and on a side stream."""
    Hq, Hkv, D, page = 8, 2, 128, 16
    table, k, v, rows = cache([4000, 700, 300], Hkv, D, page, seed=9)
    pg = bdattn.paged_geom(3, Hq, Hkv, D, k.shape[0], page, table.shape[1], 1024, 4)
    k, v, table = k.to(DEV), v.to(DEV), table.to(DEV)
    q = torch.randn(3, Hq, D, generator=torch.Generator().manual_seed(1)).bfloat16()
    qd, status = q.to(DEV), bdattn.new_status(DEV)
    lens = torch.tensor([1, 1, 1], dtype=torch.int32, device=DEV)
    bdattn.bd_attn_paged_decode(qd, k, v, table, lens, pg, status)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out, lse = bdattn.bd_attn_paged_decode(qd, k, v, table, lens, pg, status)
    for now in ([4000, 0, 300], [17, 700, 1]):
        lens.copy_(torch.tensor(now, dtype=torch.int32))
        graph.replay()
        torch.cuda.synchronize()
        cut = [(kk[:n], vv[:n]) for (kk, vv), n in zip(rows, now)]
        check(out, lse, plain(q, cut, 1024, 4))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    out2, lse2 = bdattn.bd_attn_paged_decode(qd, k, v, table, lens, pg, status, stream=side)
    side.synchronize()
    assert torch.equal(out2, out) and torch.equal(lse2, lse) and int(status.item()) == 0


APPEND = [
    # name, new tokens, earlier tokens, Hkv, D, page, padding rows
    ("single_tokens", [1] * 9, [0, 1, 15, 16, 17, 100, 31, 32, 33], 2, 128, 16, 0),
    ("prompts", [100, 1, 0, 333, 16], [0, 5, 9, 20, 16], 4, 64, 16, 7),
    ("odd_page", [50, 3], [3, 11], 3, 256, 7, 1),
    ("d512", [20, 40], [0, 0], 1, 512, 32, 0),
    ("page_of_one", [3, 5], [2, 0], 2, 64, 1, 0),
    ("many_tokens", [5000, 4000], [0, 77], 1, 64, 64, 3),
    ("nothing_new", [0, 0], [4, 0], 1, 64, 16, 0),
]


@pytest.mark.parametrize("name,new,old,Hkv,D,page,pad", APPEND, ids=[c[0] for c in APPEND])
def test_append(name, new, old, Hkv, D, page, pad):
    lens = [n + o for n, o in zip(new, old)]
    table, k, v, _ = cache(lens, Hkv, D, page, seed=2)
    k, v = torch.full_like(k, 7.0), torch.full_like(v, 7.0)
    T, B = sum(new) + pad, len(new)
    gen = torch.Generator().manual_seed(3)
    kn, vn = (torch.randn(T, Hkv, D, generator=gen).bfloat16() for _ in range(2))
    cu = torch.tensor([sum(new[:i]) for i in range(B + 1)], dtype=torch.int32)
    want_k, want_v = k.clone(), v.clone()
    for b in range(B):
        for i in range(new[b]):
            pos = old[b] + i
            pg, off = int(table[b, pos // page]), pos % page
            want_k[pg, :, off] = kn[int(cu[b]) + i]
            want_v[pg, :, off] = vn[int(cu[b]) + i]
    g = bdattn.paged_geom(B, Hkv, Hkv, D, k.shape[0], page, table.shape[1])
    kd, vd, status = k.to(DEV), v.to(DEV), bdattn.new_status(DEV)
    bdattn.bd_attn_paged_append(kn.to(DEV), vn.to(DEV), cu.to(DEV), torch.tensor(lens, dtype=torch.int32, device=DEV),
                                table.to(DEV), g, kd, vd, status)
    torch.cuda.synchronize()
    assert int(status.item()) == 0
    assert torch.equal(kd.cpu(), want_k) and torch.equal(vd.cpu(), want_v)


def test_append_drops_tokens_without_a_page():
    table = torch.tensor([[-1, 2, 0]], dtype=torch.int32, device=DEV)
    g = bdattn.paged_geom(1, 1, 1, 64, 3, 4, 3)
    k = torch.full((3, 1, 4, 64), 7.0, dtype=torch.bfloat16, device=DEV)
    v, status = k.clone(), bdattn.new_status(DEV)
    new = torch.arange(10, device=DEV).bfloat16()[:, None, None].expand(10, 1, 64).contiguous()
    i32 = lambda *x: torch.tensor(x, dtype=torch.int32, device=DEV)
    bdattn.bd_attn_paged_append(new, new, i32(0, 10), i32(10), table, g, k, v, status)
    assert int(status.item()) == 0
    assert k[:, 0, :, 0].tolist() == [[8, 9, 7, 7], [7, 7, 7, 7], [4, 5, 6, 7]] and torch.equal(k, v)


@pytest.mark.parametrize("what", ["page_high", "page_negative", "length_high", "length_negative"])
def test_bad_places_are_reported_and_not_touched(what):
    """What the table or the lengths name outside the cache sets a status bit; the rest of the cache stays."""
    g = bdattn.paged_geom(2, 2, 1, 64, 4, 4, 2)
    i32 = lambda *x: torch.tensor(x, dtype=torch.int32, device=DEV)
    table, lens = i32(0, 1, 2, 3).reshape(2, 2), i32(8, 5)
    if what == "page_high":
        table[1, 1] = 4
    elif what == "page_negative":
        table[1, 1] = -2
    elif what == "length_high":
        lens[1] = 9
    else:
        lens[1] = -1
    k = torch.full((4, 1, 4, 64), 7.0, dtype=torch.bfloat16, device=DEV)
    v, status = k.clone(), bdattn.new_status(DEV)
    new = torch.ones(2, 1, 64, dtype=torch.bfloat16, device=DEV)
    bdattn.bd_attn_paged_append(new, new, i32(0, 1, 2), lens, table, g, k, v, status)
    assert int(status.item()) == bdattn.STATUS_BOUNDS
    assert (k[2:] == 7).all() and (k[0] == 7).all()
    q = torch.ones(2, 2, 64, dtype=torch.bfloat16, device=DEV)
    status = bdattn.new_status(DEV)
    bdattn.bd_attn_paged_decode(q, k, v, table, lens, g, status)
    assert int(status.item()) == bdattn.STATUS_BOUNDS
    # and nothing is done once a bit is set
    out = torch.full((2, 2, 64), 7.0, dtype=torch.bfloat16, device=DEV)
    before = k.clone()
    bdattn.bd_attn_paged_decode(q, k, v, table, lens, g, status, out=out)
    bdattn.bd_attn_paged_append(new * 3, new * 3, i32(0, 1, 2), i32(8, 5), i32(0, 1, 2, 3).reshape(2, 2), g, k, v,
                                status)
    assert (out == 7).all() and torch.equal(k, before)


def test_append_offsets_are_checked():
    g = bdattn.paged_geom(2, 1, 1, 64, 4, 4, 2)
    i32 = lambda *x: torch.tensor(x, dtype=torch.int32, device=DEV)
    table = i32(0, 1, 2, 3).reshape(2, 2)
    new = torch.ones(2, 1, 64, dtype=torch.bfloat16, device=DEV)
    for cu in (i32(0, 1, 3), i32(1, 1, 2), i32(0, 1, -1)):
        k = torch.zeros(4, 1, 4, 64, dtype=torch.bfloat16, device=DEV)
        status = bdattn.new_status(DEV)
        bdattn.bd_attn_paged_append(new, new, cu, i32(8, 5), table, g, k, k.clone(), status)
        assert int(status.item()) == bdattn.STATUS_BOUNDS


@pytest.mark.parametrize("D,window,n_sink", [(64, 0, 0), (128, 100, 4), (256, 64, 1)])
def test_prompt_then_tokens(D, window, n_sink):
    """Prefill by the sink attention, the prompt appended, then tokens one by one:
    each one's out and lse are the sink attention's rows of the whole sequence."""
    Hq, Hkv, page, n0, steps = 4, 2, 16, 150, 3
    lens = [n0, 90]
    total = [n + steps for n in lens]
    gen = torch.Generator().manual_seed(D)
    S = sum(total)
    q, k, v = (torch.randn(1, h, S, D, generator=gen).bfloat16().to(DEV) for h in (Hq, Hkv, Hkv))
    doc = torch.repeat_interleave(torch.arange(1, 3), torch.tensor(total)).int()[None].to(DEV)
    g = bdattn.geom(1, Hq, Hkv, D, S, S, 0, 0, S, window)
    seg, status = bdattn.bd_attn_sink_seg_build(doc, g, n_sink)
    out, lse = bdattn.bd_attn_sink_fwd(q, k, v, seg, g, n_sink, status)
    pages = [-(-n // page) for n in total]
    table = torch.full((2, max(pages)), -1, dtype=torch.int32)
    ids = torch.randperm(sum(pages), generator=gen).int()
    table[0, :pages[0]], table[1, :pages[1]] = ids[:pages[0]], ids[pages[0]:]
    table = table.to(DEV)
    pg = bdattn.paged_geom(2, Hq, Hkv, D, sum(pages), page, max(pages), window, n_sink)
    kp = torch.full((sum(pages), Hkv, page, D), float("nan"), dtype=torch.bfloat16, device=DEV)
    vp = kp.clone()
    start = [0, total[0]]
    i32 = lambda *x: torch.tensor(x, dtype=torch.int32, device=DEV)
    rows = torch.cat([torch.arange(s, s + n) for s, n in zip(start, lens)]).to(DEV)
    tok = lambda t, r: t[0][:, r].transpose(0, 1).contiguous()
    bdattn.bd_attn_paged_append(tok(k, rows), tok(v, rows), i32(0, lens[0], sum(lens)), i32(*lens), table, pg, kp, vp,
                                status)
    for i in range(steps):
        at = torch.tensor([s + n + i for s, n in zip(start, lens)], device=DEV)
        now = i32(*[n + i + 1 for n in lens])
        bdattn.bd_attn_paged_append(tok(k, at), tok(v, at), i32(0, 1, 2), now, table, pg, kp, vp, status)
        o, l = bdattn.bd_attn_paged_decode(tok(q, at), kp, vp, table, now, pg, status)
        assert int(status.item()) == 0
        want, lw = tok(out, at).double(), lse[0][:, at].transpose(0, 1).double()
        assert (l.double() - lw).abs().max() <= 2 * LSE_ABS
        # both sides round P and out: twice 2^-8 of sum P |v| + |out|, sum P |v| <= max |v|
        lim = 2 * (H + SLACK) * (max(1.0, float(v.abs().max())) + want.abs())
        assert ((o.double() - want).abs() <= lim).all()


def test_refusals():
    pg = bdattn.paged_geom(2, 4, 2, 64, 8, 16, 4)
    k = torch.zeros(8, 2, 16, 64, dtype=torch.bfloat16, device=DEV)
    table = torch.zeros(2, 4, dtype=torch.int32, device=DEV)
    lens, status = torch.ones(2, dtype=torch.int32, device=DEV), bdattn.new_status(DEV)
    q = torch.zeros(2, 4, 64, dtype=torch.bfloat16, device=DEV)
    new, cu = torch.zeros(3, 2, 64, dtype=torch.bfloat16, device=DEV), torch.zeros(3, dtype=torch.int32, device=DEV)
    D, A = bdattn.bd_attn_paged_decode, bdattn.bd_attn_paged_append
    for args in ((q.half(), k, k, table, lens), (q[:, :2], k, k, table, lens), (q, k[:4], k, table, lens),
                 (q, k, k.transpose(1, 2), table, lens), (q, k, k, table.long(), lens), (q, k, k, table[:, :3], lens),
                 (q, k, k, table, lens[:1]), (q.cpu(), k, k, table, lens)):
        with pytest.raises(ValueError):
            D(*args, pg, status)
    with pytest.raises(ValueError):
        D(q, k, k, table, lens, pg, status, workspace=torch.empty(8, dtype=torch.uint8, device=DEV))
    with pytest.raises(ValueError):
        D(q, k, k, table, lens, bdattn.paged_geom(2, 4, 2, 96, 8, 16, 4), status)
    for args in ((new.float(), new, cu), (new, new[:2], cu), (new, new, cu[:2]), (new.cpu(), new, cu)):
        with pytest.raises(ValueError):
            A(*args, lens, table, pg, k, k, status)


def test_cache_beyond_32_bit_offsets():
    """Pages whose elements lie past 2^32: appended to, and read back by decode."""
    D, page, Hkv, n_pages = 128, 16, 2, (1 << 20) + 40  # 2^32 elements and a little, 8.6 GB each
    k = torch.empty(n_pages, Hkv, page, D, dtype=torch.bfloat16, device=DEV)
    v = torch.empty_like(k)
    lens = [70, 33]
    ids = [[n_pages - 1, 3, 1 << 19, n_pages - 7, (1 << 19) + 1], [n_pages - 2, 0, n_pages - 30]]
    table = torch.full((2, 5), -1, dtype=torch.int32)
    table[0, :5], table[1, :3] = torch.tensor(ids[0]), torch.tensor(ids[1])
    gen = torch.Generator().manual_seed(0)
    kn, vn = (torch.randn(sum(lens), Hkv, D, generator=gen).bfloat16() for _ in range(2))
    q = torch.randn(2, 4, D, generator=gen).bfloat16()
    i32 = lambda *x: torch.tensor(x, dtype=torch.int32, device=DEV)
    pg = bdattn.paged_geom(2, 4, Hkv, D, n_pages, page, 5)
    status = bdattn.new_status(DEV)
    bdattn.bd_attn_paged_append(kn.to(DEV), vn.to(DEV), i32(0, 70, 103), i32(*lens), table.to(DEV), pg, k, v, status)
    for b, s in enumerate((0, 70)):
        for pos in range(lens[b]):
            assert torch.equal(k[ids[b][pos // page], :, pos % page].cpu(), kn[s + pos])
    out, lse = bdattn.bd_attn_paged_decode(q.to(DEV), k, v, table.to(DEV), i32(*lens), pg, status)
    assert int(status.item()) == 0
    check(out, lse, plain(q, [(kn[:70], vn[:70]), (kn[70:], vn[70:])], 0, 0))


def test_shared_pages():
    """Two sequences on one prefix, and one place of the batch listed twice: pages are only read."""
    table, k, v, rows = cache([64, 20], 2, 128, 16, seed=5)
    n_pages = k.shape[0]
    t2 = torch.full((3, 4), -1, dtype=torch.int32)
    t2[0], t2[1, :4], t2[2, :2] = table[0], table[0], table[1, :2]
    t2[1, 2:] = table[1, :2]  # the first 32 tokens of sequence 0, then sequence 1's
    second = tuple(torch.cat([a[:32], c]) for a, c in zip(rows[0], rows[1]))
    q = torch.randn(3, 4, 128, generator=torch.Generator().manual_seed(8)).bfloat16()
    pg = bdattn.paged_geom(3, 4, 2, 128, n_pages, 16, 4)
    status = bdattn.new_status(DEV)
    out, lse = bdattn.bd_attn_paged_decode(q.to(DEV), k.to(DEV), v.to(DEV), t2.to(DEV),
                                           torch.tensor([64, 52, 20], dtype=torch.int32, device=DEV), pg, status)
    assert int(status.item()) == 0
    check(out, lse, plain(q, [rows[0], second, rows[1]], 0, 0))


def test_decode_joins_a_running_result():
    """A cache in two parts: each part's (out, lse) merged by bd_attn_merge is the whole's."""
    D, Hq, Hkv, n = 128, 4, 2, 500
    table, k, v, rows = cache([n], Hkv, D, 16, seed=6)
    q = torch.randn(1, Hq, D, generator=torch.Generator().manual_seed(9)).bfloat16().to(DEV)
    k, v, table = k.to(DEV), v.to(DEV), table.to(DEV)
    status = bdattn.new_status(DEV)
    i32 = lambda *x: torch.tensor(x, dtype=torch.int32, device=DEV)
    cut = 12  # pages
    res = []
    for t, m in ((table[:, :cut].contiguous(), cut * 16), (table[:, cut:].contiguous(), n - cut * 16)):
        pg = bdattn.paged_geom(1, Hq, Hkv, D, k.shape[0], 16, t.shape[1])
        res.append(bdattn.bd_attn_paged_decode(q, k, v, t, i32(m), pg, status))
    g = bdattn.geom(1, Hq, Hkv, D, 1, 1, 0, 0, 1)
    out, lse = (x.reshape(1, Hq, 1, -1).contiguous() for x in res[0])
    oc, lc = (x.reshape(1, Hq, 1, -1).contiguous() for x in res[1])
    lse, lc = lse.reshape(1, Hq, 1), lc.reshape(1, Hq, 1)
    bdattn.bd_attn_merge(out, lse, oc, lc, g, status)
    assert int(status.item()) == 0
    o, l, e, r2 = plain(q.cpu(), rows, 0, 0)
    # the parts' roundings and the merge's own: three bounds of one
    check(out.reshape(1, Hq, D), lse.reshape(1, Hq), (o, l, 3 * e, 9 * r2))
