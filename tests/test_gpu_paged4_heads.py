"""4-bit decode with 1 to 20 query heads to a key/value head, whose weights' second parts lie in columns of their own or
in a second product: the heads of a row have sizes of their own, and what one of them meets changes no other."""
import math

import pytest
import torch

from sliding_window_attention_device_gb300 import bdattn
from test_gpu_paged4_decode import fill, i32, on_gpu

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda")
H, EPS = 2.0 ** -8, 2.0 ** -22
FORMS = [(64, 1), (64, 4), (64, 5), (64, 12), (64, 16), (128, 3), (128, 8), (128, 9), (128, 20), (256, 2), (256, 6),
         (256, 16), (512, 4), (512, 7), (512, 12)]


def decode(q, cache, table, lens, scale):
    pg = bdattn.paged_geom(len(lens), q.shape[1], cache.k_codes.shape[1], q.shape[2], cache.k_codes.shape[0], 16,
                           table.shape[1], scale=scale)
    status = bdattn.new_status(DEV)
    out, lse = bdattn.bd_attn_paged4_decode(q.to(DEV), on_gpu(cache), table.to(DEV), i32(*lens), pg, status)
    assert int(status.item()) == 0
    return out.double().cpu(), lse.double().cpu()


def plain(q, k, v, scale):
    """out, lse of one head, and what each may be off by. A score is a sum of D exact products in fp32 and two more
    products, off by d = (D / 2 + 2) 2^-22 sum |q k| scale at most, a weight by d and lse by d; the running sums, the
    rescaling and the exponentials by (n + 16) 2^-22, relative; log2 and its product by 2^-22 of lse; the fp16 parts by
    2^-32 of the largest weight; out by half a step."""
    x = k @ q.double() * scale
    lse = torch.logsumexp(x, 0)
    p = torch.exp(x - lse)
    d = float((k.abs() @ q.double().abs()).max()) * scale * (q.shape[0] / 2 + 2) * EPS
    out, n = p @ v, len(k)
    e = (2 * d + (n + 16) * EPS) * (p @ v.abs()) + n * 2.0 ** -32 * v.abs().amax(0) + H * out.abs()
    return out, lse, e, d + (n + 16) * EPS + 4 * EPS * abs(float(lse)) + 1e-6


@pytest.mark.parametrize("spare", [0, 1000], ids=["whole", "cut"])
@pytest.mark.parametrize("D,G", FORMS)
def test_scores_that_grow_along_the_sequence(D, G, spare):
    """Each head's maximum rises again and again, at steps of its own, by a factor of its own."""
    lens, gen = [250, 900 if spare else 400], torch.Generator().manual_seed(D + G)
    rows = [tuple(torch.randn(n, 2, D, generator=gen) for _ in range(2)) for n in lens]
    for (k, _), n in zip(rows, lens):
        k *= (0.05 + torch.arange(n) / n * 3)[:, None, None]
    table, cache, values = fill(lens, 2, D, 16, seed=G, rows=rows, extra_pages=spare)
    q = torch.randn(2, 2 * G, D, generator=gen) * torch.exp2(torch.arange(2 * G) % 7 - 3.0)[None, :, None]
    q, scale = q.bfloat16(), float(torch.tensor(D ** -0.5, dtype=torch.float32))
    out, lse = decode(q, cache, table, lens, scale)
    for b, (k, v) in enumerate(values):
        for h in range(2 * G):
            o, l, e, el = plain(q[b, h], k[:, h // G], v[:, h // G], scale)
            assert abs(float(lse[b, h] - l)) <= el, (b, h)
            assert ((out[b, h] - o).abs() <= e + 1e-7).all(), (b, h)


@pytest.mark.parametrize("spare", [0, 1000], ids=["whole", "cut"])
@pytest.mark.parametrize("D,G", FORMS)
def test_a_head_of_infinities_or_nan_among_others(D, G, spare):
    """Head 0's scores are all -inf, the last one's are NaN, the ones between are as if alone; a NaN value makes its
    block's numbers NaN in every head that has weights."""
    n, gen = 300, torch.Generator().manual_seed(D + G)
    k, v = (torch.randn(n, 1, D, generator=gen) for _ in range(2))
    k[:, 0, 5] = -2.0
    v[n // 2, 0, 20] = math.nan
    table, cache, values = fill([n], 1, D, 16, rows=[(k, v)], extra_pages=spare)
    assert (values[0][0][:, 0, 5] < 0).all()
    q = torch.randn(1, G, D, generator=gen).bfloat16()
    q[0, 0, 5] = math.inf
    if G > 1:
        q[0, G - 1, 9] = math.nan
    scale = float(torch.tensor(D ** -0.5, dtype=torch.float32))
    out, lse = decode(q, cache, table, [n], scale)
    rest = torch.ones(D, dtype=torch.bool)
    rest[16:32] = False
    assert (out[0, 0, rest] == 0).all() and float(lse[0, 0]) == -math.inf
    if G > 1:
        assert torch.isnan(out[0, G - 1]).all() and torch.isnan(lse[0, G - 1])
    clean = torch.nan_to_num(values[0][1][:, 0])
    for h in range(1, G - 1):
        assert torch.isnan(out[0, h, ~rest]).all()
        o, l, e, el = plain(q[0, h], values[0][0][:, 0], clean, scale)
        assert abs(float(lse[0, h] - l)) <= el, h
        assert ((out[0, h] - o).abs() <= e + 1e-7)[rest].all(), h
