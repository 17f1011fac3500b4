"""Document ids in every order on the GPU: which rows a table build reports, row by row, against the rule
applied position by position, and the segments of the rows that are in order."""
import numpy as np
import pytest
import torch

import oracle
from sliding_window_attention_device_gb300 import bdattn

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda")


def bad_layout(row, ro, L):
    """A negative id, a document behind padding, or a local document whose id occurs before its own run."""
    S = len(row)
    if any(row[p] < 0 or (p > 0 and row[p] != 0 and row[p - 1] == 0) for p in range(S)):
        return True
    for p in range(ro, ro + L):
        if row[p] == 0:
            break
        at = p
        while at > 0 and row[at - 1] == row[p]:
            at -= 1
        if (row[:at] == row[p]).any():
            return True
    return False


def rows(rng, B, S, ro, L, mean, kind):
    """`kind`: how the ids of the runs are drawn."""
    out = np.zeros((B, S), np.int32)
    for b in range(B):
        cuts, at = [], 0
        while at < S:
            n = int(min(S - at, 1 + rng.integers(0, 2 * mean)))
            cuts.append((at, at + n))
            at += n
        n = len(cuts)
        if kind == "rising":
            ids = np.arange(1, n + 1)
        elif kind == "falling":
            ids = np.arange(n, 0, -1)
        elif kind == "any_order":
            ids = rng.permutation(n) + 1
        elif kind == "restart_behind":  # small ids again behind the shard
            k = next((i for i, c in enumerate(cuts) if c[0] >= ro + L), n)
            ids = np.concatenate([np.arange(k) + 5, np.arange(n - k) % 7 + 1])
        elif kind == "falling_before":  # any order before the shard, all below its ids
            k = next((i for i, c in enumerate(cuts) if c[1] > ro), n)
            ids = np.concatenate([rng.permutation(k) + 1, np.arange(n - k) + k + 1])
        elif kind == "few":  # repeats almost surely
            ids = rng.integers(1, max(2, n), n)
        else:  # one repeat in a rising row
            ids = np.arange(1, n + 1) * 2
            if n > 2:
                i, j = sorted(rng.choice(n, 2, replace=False))
                ids[j] = ids[i]
        for (a, e), x in zip(cuts, ids):
            out[b, a:e] = x
        if rng.integers(0, 2):
            out[b, S - int(rng.integers(0, S // 2 + 1)):] = 0
        if rng.integers(0, 8) == 0:
            out[b, int(rng.integers(0, S))] = (0, -3)[int(rng.integers(0, 2))]
    return out


KINDS = ["rising", "falling", "any_order", "restart_behind", "falling_before", "few", "one_repeat"]
SHAPES = [(300, 0, 300, 1), (300, 100, 90, 3), (513, 128, 257, 20), (1000, 999, 1, 40), (1000, 0, 1, 40),
          (4000, 1300, 1500, 60), (70, 33, 37, 2), (3000, 400, 2000, 1)]  # (the last: more than 512 segments)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("S,ro,L,mean", SHAPES, ids=[f"S{s[0]}_ro{s[1]}_L{s[2]}" for s in SHAPES])
def test_reports(kind, S, ro, L, mean):
    B = 24
    rng = np.random.default_rng(S + ro + KINDS.index(kind))
    doc = rows(rng, B, S, ro, L, mean, kind)
    g = bdattn.geom(B, 2, 1, 64, S, L, ro, 0, S, 0)
    seg, status = bdattn.bd_attn_seg_build(torch.from_numpy(doc).to(DEV), g)
    got = bdattn.read_seg(seg, g)["rows"]
    want = [bad_layout(r, ro, L) for r in doc]
    assert [bool(r["row_status"] & bdattn.STATUS_LAYOUT) for r in got] == want
    assert bool(int(status.item()) & bdattn.STATUS_LAYOUT) == any(want)
    good = [b for b in range(B) if not want[b]]
    if good:
        og1 = oracle.geom(len(good), 2, 1, 64, S, L, ro, 0, S, 0)
        for b, ref in zip(good, oracle.segments(doc[good], og1)):
            assert got[b]["cu_q"].tolist() == ref["cu_q"].tolist() and got[b]["cu_k"].tolist() == ref["cu_k"].tolist()
            assert got[b]["s_first"] == ref["s_first"] or got[b]["n_real"] == 0
