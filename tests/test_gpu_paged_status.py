"""Decode while a status bit is being set, on the GPU: a row is written whole or not at all."""
import pytest
import torch

from sliding_window_attention_device_gb300 import bdattn

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda")


@pytest.mark.parametrize("bad", [-1, 49, 2 ** 31 - 1])
@pytest.mark.parametrize("D,max_pages", [(64, 3), (128, 3), (512, 3), (128, 4000)], ids=["d64", "d128", "d512", "cut"])
def test_rows_are_whole(D, max_pages, bad):
    """One sequence of 300 has a length that is out of range: its row stays as it was, and every other row is
    either as it was or what the call gives without that sequence."""
    B, Hq, Hkv, page = 300, 4, 2, 16
    if max_pages == 4000 and bad == 49:
        bad = 64001  # past this table's end
    gen = torch.Generator().manual_seed(D)
    k, v = (torch.randn(8, Hkv, page, D, generator=gen).bfloat16().to(DEV) for _ in range(2))
    table = torch.randint(0, 8, (B, max_pages), generator=gen, dtype=torch.int32).to(DEV)
    q = torch.randn(B, Hq, D, generator=gen).bfloat16().to(DEV)
    pg = bdattn.paged_geom(B, Hq, Hkv, D, 8, page, max_pages)
    lens = torch.randint(0, 49, (B,), generator=gen, dtype=torch.int32).to(DEV)
    status = bdattn.new_status(DEV)
    want, want_lse = bdattn.bd_attn_paged_decode(q, k, v, table, lens, pg, status)
    assert int(status.item()) == 0
    for at in (0, 150, 299):
        now = lens.clone()
        now[at] = bad
        for _ in range(10):
            out, lse = torch.full_like(want, 7.0), torch.full_like(want_lse, 7.0)
            status.zero_()
            bdattn.bd_attn_paged_decode(q, k, v, table, now, pg, status, out=out, lse=lse)
            assert int(status.item()) == bdattn.STATUS_BOUNDS
            kept = (out == 7).all(2) & (lse == 7)
            done = (out == want).all(2) & (lse == want_lse)
            assert (kept | done).all()
            assert kept[at].all()
