"""Very long rows on the GPU: tables whose work lists have more lengths than the sort's histogram has bins."""
import pytest
import torch

from sliding_window_attention_device_gb300 import bdattn

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda")


@pytest.mark.parametrize("n_sink", [None, 4])
def test_800000_rows(n_sink):
    """Forward and backward of documents of 1,000 tokens in one row, a few documents compared in 64 bits."""
    S, doc_len, D, W = 800_000, 1000, 64, 128
    g = bdattn.geom(1, 1, 1, D, S, S, 0, 0, S, W)
    doc = (torch.arange(S, dtype=torch.int32, device=DEV) // doc_len + 1)[None].contiguous()
    gen = torch.Generator(device=DEV)
    gen.manual_seed(0)
    q, k, v, do = (torch.randn(1, 1, S, D, generator=gen, device=DEV).bfloat16() for _ in range(4))
    if n_sink is None:
        seg, status = bdattn.bd_attn_seg_build(doc, g)
        out, lse = bdattn.bd_attn_fwd(q, k, v, seg, g, status)
        grads = bdattn.bd_attn_bwd(do, q, k, v, out, lse, seg, g, status)
    else:
        seg, status = bdattn.bd_attn_sink_seg_build(doc, g, n_sink)
        out, lse = bdattn.bd_attn_sink_fwd(q, k, v, seg, g, n_sink, status)
        grads = bdattn.bd_attn_sink_bwd(do, q, k, v, out, lse, seg, g, n_sink, status)
    assert int(status.item()) == 0
    i = torch.arange(doc_len, device=DEV)
    far = i[:, None] - i
    sees = (far >= 0) & ((far < W) | (i < (n_sink or 0)))
    for a in (0, 397_000, S - doc_len):
        r = slice(a, a + doc_len)
        x = [t[0, 0, r].double().requires_grad_() for t in (q, k, v)]
        s = (x[0] @ x[1].T * D ** -0.5).masked_fill(~sees, float("-inf"))
        ref = torch.softmax(s, 1) @ x[2]
        (ref * do[0, 0, r].double()).sum().backward()
        assert (torch.logsumexp(s, 1) - lse[0, 0, r].double()).abs().max() <= 2e-4
        # the rounding of P (2^-8 of weights that sum to 1, |v| below 6) and of out
        assert ((out[0, 0, r].double() - ref).abs() <= 2.0 ** -8 * (6 + ref.abs())).all()
        for got, t in zip(grads, x):
            # root mean square: P, dS and the saved out are rounded to bf16, 2^-8 each at most
            assert (got[0, 0, r].double() - t.grad).norm() <= 3 * 2.0 ** -8 * t.grad.norm()
