"""Append's offsets on the GPU: one out of range or out of order is reported and no cached token is lost by it."""
import pytest
import torch

from sliding_window_attention_device_gb300 import bdattn

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda")
PAGE, PAGES = 4, 40


def i32(*x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


def append(cu, lens, n_tokens):
    """Cache of 7s, appended to with 1s; returns (status, cache [B, PAGES * PAGE])."""
    B = len(lens)
    g = bdattn.paged_geom(B, 1, 1, 64, B * PAGES, PAGE, PAGES)
    table = torch.arange(B * PAGES, dtype=torch.int32, device=DEV).reshape(B, PAGES)
    k = torch.full((B * PAGES, 1, PAGE, 64), 7.0, dtype=torch.bfloat16, device=DEV)
    v, status = k.clone(), bdattn.new_status(DEV)
    new = torch.ones(n_tokens, 1, 64, dtype=torch.bfloat16, device=DEV)
    bdattn.bd_attn_paged_append(new, new, i32(*cu), i32(*lens), table, g, k, v, status)
    torch.cuda.synchronize()
    assert torch.equal(k, v)
    return int(status.item()), k[:, 0, :, 0].reshape(B, PAGES * PAGE).cpu()


BAD = [
    ("interior_past_the_end", [0, 100, 4], [104, 4], 4),
    ("interior_falls", [0, 3, 2, 4], [10, 10, 10], 4),
    ("interior_negative", [0, -5, 4], [10, 10], 4),
    ("falls_to_zero", [0, 4, 0, 4], [10, 10, 10], 4),
    ("far_from_the_first", [0] + list(range(1, 300)) + [298, 300], [20] * 301, 300),
    ("no_tokens_but_an_end", [0, 0, 3], [5, 5], 0),
    ("no_tokens_but_a_start", [2, 2, 2], [5, 5], 0),
    ("end_past_the_tokens", [0, 1, 3], [8, 5], 2),
]


@pytest.mark.parametrize("name,cu,lens,n", BAD, ids=[c[0] for c in BAD])
def test_bad_offsets_are_reported(name, cu, lens, n):
    status, cache = append(cu, lens, n)
    assert status == bdattn.STATUS_BOUNDS
    # whatever was stored went to places its sequence's own offsets call new
    for b, m in enumerate(lens):
        new = min(max(cu[b + 1] - cu[b], 0), n)
        old = cache[b].clone()
        old[m - new:m] = 7
        assert (old == 7).all(), b


GOOD = [
    ("single_tokens", list(range(301)), [20] * 300, 300),
    ("empty_ones_between", [0, 0, 2, 2, 2, 5, 5], [3, 9, 1, 8, 30, 2], 9),
    ("no_tokens", [0, 0, 0], [5, 0], 0),
    ("all_padding", [0, 0, 0], [5, 0], 6),
]


@pytest.mark.parametrize("name,cu,lens,n", GOOD, ids=[c[0] for c in GOOD])
def test_good_offsets_are_not(name, cu, lens, n):
    status, cache = append(cu, lens, n)
    assert status == 0
    for b, m in enumerate(lens):
        want = torch.full_like(cache[b], 7)
        want[m - (cu[b + 1] - cu[b]):m] = 1
        assert torch.equal(cache[b], want), b
