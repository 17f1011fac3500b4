"""Decode on infinities and NaN: out and lse are those of softmax over the visible keys, so a NaN shows in
both, a score of -inf weighs nothing, and what no new token sees has no effect.

The expected values come from the formula in 64 bits: x the scores, m their maximum (0 where all are -inf),
out = sum exp(x - m) v / sum exp(x - m), lse = m + log(sum); rows without a weight have out 0, lse -inf."""
import math

import pytest
import torch

from sink_ref import H, LSE_ABS, SLACK
from sliding_window_attention_device_gb300 import bdattn

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda")
INF, NAN = math.inf, math.nan
PAGE = 16
# whole rows per CTA; a row cut over CTAs (one sequence, table of 20,000 tokens)
FORMS = [("whole", 200, 13), ("cut", 3000, 1250)]


def formula(q, k, v):
    """out [Hq, D], lse [Hq], bound of out of one sequence: q [Hq, D], k and v [n, Hkv, D]."""
    Hq, D = q.shape
    G = Hq // k.shape[1]
    out, bound, lse = torch.zeros(Hq, D, dtype=torch.float64), torch.zeros(Hq, D, dtype=torch.float64), []
    for h in range(Hq):
        x = (k[:, h // G].double() @ q[h].double()) * D ** -0.5
        m = x.max() if not torch.isnan(x).any() else torch.tensor(NAN, dtype=torch.float64)
        m = torch.where(m == -INF, 0.0, m)
        e = torch.exp(x - m)
        s = e.sum()
        lse.append(m + torch.log(s))
        p = e / torch.where(s == 0, 1.0, s)
        vv = v[:, h // G].double()
        out[h] = p @ vv
        bound[h] = (H + SLACK) * (p @ vv.abs()) + H * out[h].abs() + 1e-7
    return out, torch.stack(lse), bound


def decode(q, k, v, max_pages):
    n, Hkv, D = k.shape
    pages = -(-n // PAGE)
    kp = torch.full((pages, Hkv, PAGE, D), NAN, dtype=torch.bfloat16)
    vp = torch.full((pages, Hkv, PAGE, D), NAN, dtype=torch.bfloat16)
    for i in range(pages):
        m = min(PAGE, n - i * PAGE)
        kp[i, :, :m] = k[i * PAGE:i * PAGE + m].transpose(0, 1)
        vp[i, :, :m] = v[i * PAGE:i * PAGE + m].transpose(0, 1)
    table = torch.full((1, max_pages), -1, dtype=torch.int32)
    table[0, :pages] = torch.arange(pages)
    pg = bdattn.paged_geom(1, q.shape[0], Hkv, D, pages, PAGE, max_pages)
    status = bdattn.new_status(DEV)
    out, lse = bdattn.bd_attn_paged_decode(q[None].to(DEV), kp.to(DEV), vp.to(DEV), table.to(DEV),
                                           torch.tensor([n], dtype=torch.int32, device=DEV), pg, status)
    assert int(status.item()) == 0
    return out[0].double().cpu(), lse[0].double().cpu()


def compare(got, want):
    out, lse = got
    o, l, bound = want
    assert torch.equal(torch.isnan(lse), torch.isnan(l)), (lse, l)
    fin = torch.isfinite(l)
    assert torch.equal(lse[~fin & ~torch.isnan(l)], l[~fin & ~torch.isnan(l)])
    assert ((lse - l)[fin].abs() <= LSE_ABS).all()
    assert torch.equal(torch.isnan(out), torch.isnan(o))
    ok = ~torch.isnan(o)
    assert ((out - o).abs()[ok] <= bound[ok]).all()


@pytest.mark.parametrize("D", [64, 128, 256, 512])
@pytest.mark.parametrize("form,n,max_pages", FORMS, ids=[f[0] for f in FORMS])
@pytest.mark.parametrize("what", ["nan_in_q", "nan_in_k", "first_scores_minus_inf", "all_scores_minus_inf",
                                  "some_scores_minus_inf", "score_plus_inf", "nan_behind_the_sequence"])
def test_nonfinite(what, form, n, max_pages, D):
    Hq, Hkv = 4, 2
    gen = torch.Generator().manual_seed(D + n)
    q = torch.randn(Hq, D, generator=gen).bfloat16()
    k, v = (torch.randn(n, Hkv, D, generator=gen).bfloat16() for _ in range(2))
    # infinite scores without NaN: one column of K infinite, q positive there
    q[:, 0] = q[:, 0].abs() + 0.5
    if what == "nan_in_q":
        q[1, 5] = NAN  # one head; the others stay
    elif what == "nan_in_k":
        k[n // 2, 1, 3] = NAN  # the second kv head's heads
    elif what == "first_scores_minus_inf":
        k[:16 * 9, 0, 0] = -INF  # whole steps of each warp
    elif what == "all_scores_minus_inf":
        k[:, 0, 0] = -INF
    elif what == "some_scores_minus_inf":
        k[::3, 1, 0] = -INF
    elif what == "score_plus_inf":
        k[n - 3, 0, 0] = INF
    got = decode(q, k, v, max_pages)
    compare(got, formula(q, k, v))
