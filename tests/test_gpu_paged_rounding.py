"""Decode's rounding on the GPU: out is off by its own rounding to bf16 and little more.

The weights P enter the product as two bf16 numbers, the second of what the first left: off by 2^-8 of 2^-8 of
P at most. So |error| <= 2^-8 |out| + (2^-16 + 1e-4) sum P |v|, the 1e-4 for fp32 sums and exponentials."""
import pytest
import torch

from sink_ref import H, SLACK
from sliding_window_attention_device_gb300 import bdattn
from test_gpu_paged import cache, plain, visible

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda")

CASES = [
    # name, lens, Hq, Hkv, D, window, n_sink, spare table entries (0: whole rows)
    ("few_keys", list(range(1, 41)), 4, 2, 64, 0, 0, 0),
    ("few_keys_cut", list(range(1, 41)), 4, 2, 128, 0, 0, 2000),
    ("groups_of_16", [3, 17, 90, 400], 32, 2, 128, 0, 0, 0),
    ("window_sinks", [5, 30, 700, 900], 8, 4, 256, 20, 4, 0),
    ("d512", [2, 9, 100, 300], 4, 2, 512, 0, 0, 0),
    ("split", [3000], 8, 2, 128, 0, 0, 1000),
]


@pytest.mark.parametrize("name,lens,Hq,Hkv,D,window,n,spare", CASES, ids=[c[0] for c in CASES])
def test_out_is_rounded_once(name, lens, Hq, Hkv, D, window, n, spare):
    table, k, v, rows = cache(lens, Hkv, D, 16, seed=len(name), extra_pages=spare)
    q = torch.randn(len(lens), Hq, D, generator=torch.Generator().manual_seed(1)).bfloat16()
    pg = bdattn.paged_geom(len(lens), Hq, Hkv, D, k.shape[0], 16, table.shape[1], window, n)
    status = bdattn.new_status(DEV)
    out, _ = bdattn.bd_attn_paged_decode(q.to(DEV), k.to(DEV), v.to(DEV), table.to(DEV),
                                         torch.tensor(lens, dtype=torch.int32, device=DEV), pg, status)
    assert int(status.item()) == 0
    want = plain(q, rows, window, n)[0]
    weight = torch.zeros_like(want)
    for b, (kk, vv) in enumerate(rows):
        see = visible(len(kk), window, n)
        for h in range(Hq):
            x = kk[see, h // (Hq // Hkv)].double() @ q[b, h].double() * D ** -0.5
            weight[b, h] = torch.softmax(x, 0) @ vv[see, h // (Hq // Hkv)].double().abs()
    err = (out.double().cpu() - want).abs()
    assert (err <= H * want.abs() + (2.0 ** -16 + SLACK) * weight + 1e-7).all()
