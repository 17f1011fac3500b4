"""4-bit decode's rounding: out is the softmax's weighted sum rounded to bf16 once, and little more.

The cache's values are exact in the products, q is scaled by a power of two, and the weights P enter the product with V
as two fp16 numbers, the second of what the first left: off by 2^-11 of 2^-11 of P at most, or by 2^-32 of the largest
weight where they are as small as that. A score is a sum of D exact products in fp32, off by D 2^-23 sum |q k| scale at
most, and its weight by the same, relative; the running sum and the quotient likewise. Exponentials, products with
powers and the sums over n keys add a few 2^-22 and n 2^-23 (each warp sums n / 8 at most). So with d the largest of the
scores' bounds
  |out error| <= half a step of bf16 at out + (2 d + 2^-22 + 8 * 2^-22 + n 2^-23) sum P |v| + n 2^-32 max |v|.
The softmax scale is small, so that d is: one fp16 number per weight would be off by 2^-11, some 20 times that."""
import pytest
import torch

import paged4_ref as ref
from sliding_window_attention_device_gb300 import bdattn
from test_gpu_paged4_decode import fill, i32, on_gpu

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda")

CASES = [
    # name, lens, Hq, Hkv, D, window, n_sink, spare table entries (0: whole rows)
    ("one_head", list(range(1, 41)), 2, 2, 64, 0, 0, 0),
    ("four_heads", list(range(1, 41)), 8, 2, 64, 0, 0, 0),
    ("four_heads_cut", list(range(1, 41)), 4, 1, 128, 0, 0, 2000),
    ("five_heads", list(range(1, 41)), 10, 2, 128, 0, 0, 0),
    ("eight_heads_cut", list(range(1, 41)), 8, 1, 64, 0, 0, 2000),
    ("eight_heads_d256", [2, 9, 33, 60], 16, 2, 256, 0, 0, 0),
    ("two_heads_d256", [2, 9, 33, 60], 4, 2, 256, 0, 0, 0),
    ("sixteen_heads", [3, 17, 60, 40], 32, 2, 128, 0, 0, 0),
    ("sixteen_heads_d64", [3, 17, 60, 40], 16, 1, 64, 0, 0, 0),
    ("twelve_heads_d256", [3, 17, 60, 40], 24, 2, 256, 0, 0, 0),
    ("window_sinks", [5, 30, 70, 90], 8, 4, 256, 20, 4, 0),
    ("d512", [2, 9, 33, 60], 4, 2, 512, 0, 0, 0),
    ("d512_seven_heads", [2, 9, 33, 60], 7, 1, 512, 0, 0, 0),
    ("d512_ten_heads_cut", [2, 9, 33, 60], 10, 1, 512, 0, 0, 1000),
]


@pytest.mark.parametrize("name,lens,Hq,Hkv,D,window,n,spare", CASES, ids=[c[0] for c in CASES])
def test_out_is_rounded_once(name, lens, Hq, Hkv, D, window, n, spare):
    table, cache, values = fill(lens, Hkv, D, 16, (0.5, 0.37), seed=len(name), extra_pages=spare)
    q = torch.randn(len(lens), Hq, D, generator=torch.Generator().manual_seed(1)).bfloat16()
    scale = 0.25 / D
    pg = bdattn.paged_geom(len(lens), Hq, Hkv, D, cache.k_codes.shape[0], 16, table.shape[1], window, n, scale)
    status = bdattn.new_status(DEV)
    out, _ = bdattn.bd_attn_paged4_decode(q.to(DEV), on_gpu(cache), table.to(DEV), i32(*lens), pg, status)
    assert int(status.item()) == 0
    got, scale = out.double().cpu(), float(torch.tensor(scale, dtype=torch.float32))
    for b, (k, v) in enumerate(values):
        s = torch.arange(len(k))
        see = (s >= len(k) - window) | (s < n) if window > 0 else torch.ones(len(k), dtype=torch.bool)
        for h in range(Hq):
            kk, vv, qq = k[see, h // (Hq // Hkv)], v[see, h // (Hq // Hkv)], q[b, h].double()
            p = torch.softmax(kk @ qq * scale, 0)
            want, d = p @ vv, float((kk.abs() @ qq.abs()).max()) * scale * D * 2.0 ** -23
            e = (2 * d + 9 * 2.0 ** -22 + len(kk) * 2.0 ** -23) * (p @ vv.abs()) + len(kk) * 2.0 ** -32 * vv.abs().amax(0)
            assert float(d) < 2e-5
            step = torch.exp2(torch.floor(torch.log2(want.abs().clamp(min=1e-30))) - 7)
            assert ((got[b, h] - want).abs() <= step / 2 + e).all(), (b, h)
