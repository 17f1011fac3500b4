"""The rotating append's and the 4-bit read's offsets: with wrong ones the call reports BOUNDS, and whatever it wrote is
a token's own, at a place that its sequence's own offsets give it; no other byte changes.

Among offsets that fall, a token may lie in the ranges of several sequences, or of none. A range that begins below 0 or
ends past the last offset or past the new tokens is no sequence's."""
import random

import pytest
import torch

import paged4_ref as ref
from sliding_window_attention_device_gb300 import bdattn

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda")
BF16, U8 = torch.bfloat16, torch.uint8
PAGE, PAGES, D, Hq = 4, 8, 64, 2
CAP = PAGE * PAGES


def i32(*x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


def owners(cu, lens, n):
    """token -> {(sequence, position)} that the offsets call it."""
    of = {t: set() for t in range(n)}
    for b, m in enumerate(lens):
        begin, end = cu[b], cu[b + 1]
        if begin < 0 or end > min(cu[-1], n):
            continue
        for t in range(begin, end):
            if 0 <= m - (end - t) < CAP:
                of[t].add((b, m - (end - t)))
    return of


def counted(new):
    cu = [0]
    for x in new:
        cu.append(cu[-1] + x)
    return cu


def changed(cu, at, by):
    return cu[:at] + [cu[at] + by] + cu[at + 1:]


RAGGED = counted([1 + (5 * i) % 4 for i in range(70)])  # 175 tokens
SINGLE = counted([1] * 1100)
MIXED = RAGGED[:]
random.Random(3).shuffle(MIXED)
WILD = [random.Random(i).choice((-2 ** 31, -7, 0, 5, 80, 174, 175, 176, 2 ** 31 - 1)) for i in range(71)]

BAD = [
    # name, offsets, new tokens
    ("past_the_tokens", [0, 1, 3], 2),
    ("not_from_0", [1, 1, 2], 2),
    ("falls", [0, 2, 1], 2),
    ("falls_and_rises", [0, 3, 1, 4], 4),
    ("one_raised_among_70", changed(RAGGED, 40, 9), RAGGED[-1]),
    ("one_lowered_among_70", changed(RAGGED, 33, -20), RAGGED[-1]),
    ("one_below_0_among_70", changed(RAGGED, 50, -200), RAGGED[-1]),
    ("the_last_one_lowered", changed(RAGGED, 70, -30), RAGGED[-1]),
    ("more_than_the_tokens", RAGGED, RAGGED[-1] - 10),
    ("in_no_order", MIXED, RAGGED[-1]),
    ("anything", WILD, RAGGED[-1]),
    ("one_raised_among_1100", changed(SINGLE, 700, 9), 1100),
    ("many_lowered_among_1100", SINGLE[:300] + [x - 40 for x in SINGLE[300:]], 1100),
]


def call_append(four, cu, lens, n, seed=1):
    B = len(lens)
    pg = bdattn.paged_geom(B, Hq, 1, D, B * PAGES, PAGE, PAGES)
    table = torch.randperm(B * PAGES, generator=torch.Generator().manual_seed(seed)).int().reshape(B, PAGES)
    gen = torch.Generator().manual_seed(seed + 1)
    q, k, v = (torch.randn(n, h, D, generator=gen).bfloat16() for h in (Hq, 1, 1))
    cs, status = ref.table(CAP, D), bdattn.new_status(DEV)
    q_out, k_out = (torch.full(x.shape, 7.0, dtype=BF16, device=DEV) for x in (q, k))
    args = (q.to(DEV), k.to(DEV), v.to(DEV), cs.to(DEV), i32(*cu), i32(*lens), table.to(DEV), pg)
    if four:
        cache = bdattn.paged4_cache(pg, DEV)
        for x in cache[:4]:
            x.view(U8).fill_(0x5a)
        bdattn.bd_attn_paged4_append(*args, cache, status, q_out=q_out, k_out=k_out)
        state = [x.view(U8).cpu() for x in cache[:4]]
    else:
        kp = torch.full((B * PAGES, 1, PAGE, D), 7.0, dtype=BF16, device=DEV)
        vp = kp.clone()
        bdattn.bd_attn_paged_append_rope(*args, kp, vp, status, q_out=q_out, k_out=k_out)
        state = [kp.cpu(), vp.cpu()]
    return int(status.item()), table, cs, (q, k, v), (q_out.cpu(), k_out.cpu()), state


@pytest.mark.parametrize("four", [False, True], ids=["bf16", "4bit"])
@pytest.mark.parametrize("name,cu,n", BAD, ids=[c[0] for c in BAD])
def test_append_writes_its_own_or_nothing(name, cu, n, four):
    B = len(cu) - 1
    lens = [min(CAP, max(0, min(cu[b + 1] - cu[b], CAP)) + b % 9) for b in range(B)]
    status, table, cs, (q, k, v), (q_out, k_out), state = call_append(four, cu, lens, n)
    assert status == bdattn.STATUS_BOUNDS
    of = owners(cu, lens, n)
    # every place of every sequence that is not as it was holds a token that the offsets put there
    rows = [x.view(U8).reshape(B * PAGES, PAGE, -1) if four else x.view(torch.int16).reshape(B * PAGES, PAGE, -1)
            for x in state]
    fill = 0x5a if four else torch.tensor(7.0, dtype=BF16).view(torch.int16).item()
    put = torch.stack([(x != fill).any(-1) for x in rows]).any(0)
    back = {int(p): (b, i) for b in range(B) for i, p in enumerate(table[b])}
    token_of = {}
    for t, places in of.items():
        for place in places:
            token_of.setdefault(place, []).append(t)
    for page, off in put.nonzero().tolist():
        b, i = back[page]
        pos = i * PAGE + off
        assert (b, pos) in token_of, (b, pos)
        fits = []
        for t in token_of[(b, pos)]:
            kt = ref.rotate(k[t:t + 1], cs[pos:pos + 1], ref.HALVES)
            if four:
                (kc, ks), (vc, vs) = ref.to4(kt), ref.to4(v[t:t + 1].float())
                want = [kc, vc, ks.view(U8), vs.view(U8)]
            else:
                want = [kt.bfloat16().view(torch.int16), v[t:t + 1].view(torch.int16)]
            fits.append(all(torch.equal(w.reshape(-1), x[page, off]) for w, x in zip(want, rows)))
        assert any(fits), (b, pos)
    # rows of the outputs: untouched, or turned by one of the token's positions
    for x, y in ((q, q_out), (k, k_out)):
        for t in range(n):
            if not (y[t] == 7).all():
                assert any(torch.equal(y[t], ref.rotate(x[t:t + 1], cs[p:p + 1], ref.HALVES).bfloat16()[0])
                           for _, p in of[t]), t
    if name in ("falls", "not_from_0", "past_the_tokens"):  # who is left: nobody, and the other one's token
        left = {"falls": [], "not_from_0": [1], "past_the_tokens": [0]}[name]
        assert [t for t in range(n) if (q_out[t] != 7).any()] == left
        assert int(put.sum()) == len(left)


@pytest.mark.parametrize("name,cu,n", BAD, ids=[c[0] for c in BAD])
def test_read_gives_its_own_or_nothing(name, cu, n):
    B = len(cu) - 1
    lens = [min(CAP, max(0, min(cu[b + 1] - cu[b], CAP)) + b % 9) for b in range(B)]
    pg = bdattn.paged_geom(B, Hq, 1, D, B * PAGES, PAGE, PAGES)
    gen = torch.Generator().manual_seed(1)
    table = torch.randperm(B * PAGES, generator=gen).int().reshape(B, PAGES)
    host = [ref.to4(torch.randn(B * PAGES, 1, PAGE, D, generator=gen)) for _ in range(2)]
    cache = bdattn.Cache4(*(c.to(DEV) for c, _ in host), *(s.view(U8).to(DEV).view(ref.E4M3) for _, s in host))
    out = [torch.full((n, 1, D), 7.0, dtype=BF16, device=DEV) for _ in range(2)]
    status = bdattn.new_status(DEV)
    bdattn.bd_attn_paged4_read(cache, i32(*cu), i32(*lens), table.to(DEV), pg, n, status, *out)
    assert int(status.item()) == bdattn.STATUS_BOUNDS
    of = owners(cu, lens, n)
    values = [ref.bf16_of(c, s) for c, s in host]
    for got, val in zip((x.cpu() for x in out), values):
        for t in range(n):
            if not (got[t] == 7).all():
                assert any(torch.equal(got[t], val[int(table[b, p // PAGE]), :, p % PAGE]) for b, p in of[t]), t
    if name == "falls":
        assert all((x == 7).all() for x in out)
