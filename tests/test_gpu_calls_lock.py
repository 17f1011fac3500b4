"""The native calls and the interpreter's lock: another Python thread runs on while a call waits for the GPU's queue.

A kernel that takes a second is put on a stream, and calls behind it until the queue of launches is full: the call that
finds it full returns only when that kernel is done. A thread that writes down the time meanwhile must not stand still
for as long."""
import threading
import time

import pytest
import torch

import paged4_ref as ref
from sliding_window_attention_device_gb300 import bdattn

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda")
SECONDS = 1.0


def i32(*x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


@pytest.mark.parametrize("what", ["append_rope", "append4", "read4", "decode4"])
def test_other_threads_run_while_a_call_waits(what):
    pg = bdattn.paged_geom(1, 2, 1, 64, 4, 16, 4)
    cache, status = bdattn.paged4_cache(pg, DEV), bdattn.new_status(DEV)
    for x in cache[:4]:
        x.view(torch.uint8).zero_()
    kp = torch.zeros(4, 1, 16, 64, dtype=torch.bfloat16, device=DEV)
    vp, q = kp.clone(), torch.zeros(1, 2, 64, dtype=torch.bfloat16, device=DEV)
    k, table, lens, cu, cs = q[:, :1], i32(0, 1, 2, 3)[None], i32(20), i32(0, 1), ref.table(64, 64).to(DEV)
    q_out, k_row = torch.empty_like(q), torch.empty(1, 1, 64, dtype=torch.bfloat16, device=DEV)
    v_row, lse = k_row.clone(), torch.empty(1, 2, device=DEV)
    new = (q, k, k, cs, cu, lens, table, pg)
    call = {"append_rope": lambda: bdattn.bd_attn_paged_append_rope(*new, kp, vp, status, q_out=q_out),
            "append4": lambda: bdattn.bd_attn_paged4_append(*new, cache, status, q_out=q_out),
            "read4": lambda: bdattn.bd_attn_paged4_read(cache, cu, lens, table, pg, 1, status, k_row, v_row),
            "decode4": lambda: bdattn.bd_attn_paged4_decode(q, cache, table, lens, pg, status, q_out, lse)}[what]
    call()
    assert bdattn._calls is not None
    torch.cuda.synchronize()
    # cycles of a second: counted on this GPU
    torch.cuda._sleep(1000)
    torch.cuda.synchronize()
    a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    a.record()
    torch.cuda._sleep(10_000_000)
    b.record()
    torch.cuda.synchronize()
    cycles = int(10_000_000 * SECONDS * 1e3 / a.elapsed_time(b))

    ticks, stop = [], threading.Event()

    def tick():
        while not stop.is_set():
            ticks.append(time.perf_counter())
            time.sleep(0.001)

    other = threading.Thread(target=tick)
    other.start()
    try:
        torch.cuda._sleep(cycles)
        begin = time.perf_counter()
        waited = start = end = 0.0
        while waited < SECONDS / 4 and time.perf_counter() - begin < 2 * SECONDS:
            t = time.perf_counter()
            call()
            now = time.perf_counter()
            if now - t > waited:
                waited, start, end = now - t, t, now
        torch.cuda.synchronize()
    finally:
        stop.set()
        other.join()
    assert waited >= SECONDS / 4, "no call had to wait"
    inside = [start] + [t for t in ticks if start < t < end] + [end]
    assert max(y - x for x, y in zip(inside, inside[1:])) < waited / 2
    assert int(status.item()) == 0
