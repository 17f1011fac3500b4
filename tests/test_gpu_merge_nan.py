"""The merge of two forward results on the GPU keeps a NaN of either side, in out and in lse."""
import math

import pytest
import torch

from sliding_window_attention_device_gb300 import bdattn

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda")
INF, NAN = math.inf, math.nan


@pytest.mark.parametrize("D", [64, 128, 256, 512])
@pytest.mark.parametrize("nan_in", ["running", "chunk", "both"])
@pytest.mark.parametrize("other_empty", [False, True])
def test_merge_keeps_a_nan(nan_in, other_empty, D):
    """Rows 0 and 2 have a NaN lse and out on the named side, rows 1 and 3 are finite and stay so."""
    g = bdattn.geom(1, 2, 1, D, 4, 4, 0, 0, 4)
    gen = torch.Generator().manual_seed(D)
    out, out_c = (torch.randn(1, 2, 4, D, generator=gen).bfloat16() for _ in range(2))
    lse, lse_c = (torch.randn(1, 2, 4, generator=gen) for _ in range(2))
    want_lse = torch.logaddexp(lse.double(), lse_c.double())
    want = (torch.exp(lse - want_lse)[..., None] * out.double() + torch.exp(lse_c - want_lse)[..., None] * out_c.double())
    for side, (o, l) in (("running", (out, lse)), ("chunk", (out_c, lse_c))):
        if nan_in in (side, "both"):
            o[:, :, ::2], l[:, :, ::2] = NAN, NAN
        elif other_empty:
            o[:, :, ::2], l[:, :, ::2] = 0, -INF
    out, lse, status = out.to(DEV), lse.to(DEV), bdattn.new_status(DEV)
    bdattn.bd_attn_merge(out, lse, out_c.to(DEV), lse_c.to(DEV), g, status)
    assert int(status.item()) == 0
    o, l = out.double().cpu(), lse.double().cpu()
    assert torch.isnan(o[:, :, ::2]).all() and torch.isnan(l[:, :, ::2]).all()
    # a bf16 rounding of out, and fp32 exponentials and logarithms of numbers below 8
    assert ((o - want)[:, :, 1::2].abs() <= 2.0 ** -8 * want[:, :, 1::2].abs() + 1e-5).all()
    assert ((l - want_lse)[:, :, 1::2].abs() <= 1e-5).all()
