"""ctypes binding of libbdattn.so (declared in include/bdattn.h).

Argument marshalling only: every computation runs in the CUDA kernels behind
the C ABI. Tensors are PyTorch CUDA tensors (PyTorch provides the device
memory and the current stream); outputs the caller does not pass are
allocated here with torch. Small calls of the rotating append and the 4-bit cache go
through _calls, a module built with the library, which does the same and without which
they go through the functions here. There is no CPU fallback: without the compiled
library, or without a GPU, these functions raise.
"""
from __future__ import annotations

import ctypes
import importlib.util
import os
import threading
import warnings
from typing import NamedTuple

import torch

from .build import calls_path

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libbdattn.so")

# return codes
BD_OK, BD_ERR_ARG, BD_ERR_CUDA, BD_ERR_UNSUPPORTED = 0, 1, 2, 3
# device status bits
STATUS_LAYOUT, STATUS_KV_RANGE, STATUS_BOUNDS, STATUS_TIMEOUT = 0x1, 0x2, 0x4, 0x8
# gradient dtypes
BD_DTYPE_F32, BD_DTYPE_BF16 = 0, 1
# per-row header fields of the segment table
HDR_FIELDS = ("n_real", "n_seg", "s_first", "real_end", "max_q", "max_k", "first_q", "first_k", "max_tail",
              "kv_need_lo", "row_status")
HDR_WORDS = 32
# region indices of the segment table (BD_SEG_OFF_*)
REGIONS = ("hdr", "cu_q", "cu_k", "row_lo", "qt_krange", "kt_qrange", "full_bits", "fwd_work", "bwd_work",
           "counts", "total")

EXPORTS = ("bd_attn_seg_bytes", "bd_attn_seg_layout", "bd_attn_seg_build", "bd_attn_seg_build_chunk",
           "bd_attn_fwd", "bd_attn_fwd_merge", "bd_attn_merge",
           "bd_attn_bwd_workspace_bytes", "bd_attn_bwd", "bd_attn_bwd_deterministic", "bd_attn_bwd_prep",
           "bd_attn_bwd_main",
           "bd_attn_bwd_finalize", "bd_attn_bwd_prep_dq", "bd_attn_bwd_main_dq",
           "bd_attn_bwd_noalloc", "bd_attn_plan_bytes", "bd_attn_plan_layout", "bd_attn_exchange_plan",
           "bd_attn_needed_gather", "bd_attn_needed_scatter_add", "bd_attn_strerror",
           "bd_attn_sink_seg_bytes", "bd_attn_sink_seg_build", "bd_attn_sink_fwd", "bd_attn_sink_fwd_merge",
           "bd_attn_sink_bwd_workspace_bytes", "bd_attn_sink_bwd", "bd_attn_sink_bwd_deterministic",
           "bd_attn_sink_bwd_main", "bd_attn_paged_append", "bd_attn_paged_decode_workspace_bytes",
           "bd_attn_paged_decode", "bd_attn_paged_append_rope", "bd_attn_paged4_append", "bd_attn_paged4_read",
           "bd_attn_paged4_decode_workspace_bytes", "bd_attn_paged4_decode",
           "bd_attn_selftest_wait_timeout")

# exchange plan: header fields (BD_PLAN_*) and regions (BD_PLAN_OFF_*)
PLAN_HDR_FIELDS = ("magic", "cp_size", "L", "rank", "B", "use_halo", "halo_size", "total_send", "total_recv")
PLAN_HDR_WORDS = 16
PLAN_REGIONS = ("hdr", "s_first", "real_end", "back", "halo_send", "counts", "in_splits", "out_splits", "send_off",
                "recv_off", "send_index", "row_range", "total")
PLAN_MAGIC = 0x62647870


class Geom(ctypes.Structure):
    _fields_ = [("B", ctypes.c_int), ("Hq", ctypes.c_int), ("Hkv", ctypes.c_int), ("D", ctypes.c_int),
                ("S_full", ctypes.c_int), ("L", ctypes.c_int), ("row_offset", ctypes.c_int),
                ("kv_offset", ctypes.c_int), ("S_kv", ctypes.c_int), ("window", ctypes.c_int),
                ("scale", ctypes.c_float), ("kv_layout", ctypes.c_int), ("dropout_p", ctypes.c_float),
                ("seed_lo", ctypes.c_uint32), ("seed_hi", ctypes.c_uint32)]

    def __repr__(self):
        return "Geom(" + ", ".join(f"{n}={getattr(self, n)}" for n, _ in self._fields_) + ")"


class Paged(ctypes.Structure):
    _fields_ = [("B", ctypes.c_int), ("Hq", ctypes.c_int), ("Hkv", ctypes.c_int), ("D", ctypes.c_int),
                ("n_pages", ctypes.c_int), ("page_size", ctypes.c_int), ("max_pages", ctypes.c_int),
                ("window", ctypes.c_int), ("n_sink", ctypes.c_int), ("scale", ctypes.c_float)]

    def __repr__(self):
        return "Paged(" + ", ".join(f"{n}={getattr(self, n)}" for n, _ in self._fields_) + ")"


class Rope(ctypes.Structure):
    _fields_ = [("rot_dim", ctypes.c_int), ("pairing", ctypes.c_int), ("n_pos", ctypes.c_int),
                ("q_stride", ctypes.c_int64), ("k_stride", ctypes.c_int64), ("v_stride", ctypes.c_int64)]


class _Cache4(ctypes.Structure):
    _fields_ = [("k_codes", ctypes.c_void_p), ("v_codes", ctypes.c_void_p), ("k_blocks", ctypes.c_void_p),
                ("v_blocks", ctypes.c_void_p), ("k_gain", ctypes.c_float), ("v_gain", ctypes.c_float)]


class Cache4(NamedTuple):
    """A paged cache held in 4 bits: codes uint8 [n_pages, Hkv, page_size, D / 2] and block scales float8_e4m3fn
    [n_pages, Hkv, page_size, D / 16] of keys and values, and their gains (value = code * scale * gain)."""
    k_codes: torch.Tensor
    v_codes: torch.Tensor
    k_blocks: torch.Tensor
    v_blocks: torch.Tensor
    k_gain: float = 1.0
    v_gain: float = 1.0


ROPE_HALVES, ROPE_ADJACENT = 0, 1  # which numbers of a head turn together: (i, i + rot / 2) or (2 i, 2 i + 1)
KV_BHSD, KV_SBHD = 0, 1  # K/V layouts: [B, Hkv, S_kv, D] or token-major [S_kv, B, Hkv, D]


_INT_MAX = 2 ** 31 - 1


def _fit(struct, values):
    """Refuses what does not fit the struct's C ints, which ctypes would wrap."""
    if max(values) > _INT_MAX or min(values) < -_INT_MAX:
        for (name, _), x in zip(struct._fields_, values):
            if not -_INT_MAX <= x <= _INT_MAX:
                raise ValueError(f"{name}={x} does not fit 32 bits")


def _c_window(window) -> int:
    """Beyond every distance, or none."""
    return _INT_MAX if window > _INT_MAX else -1 if window < 0 else int(window)


def geom(B, Hq, Hkv, D, S_full, L, row_offset, kv_offset, S_kv, window=0, scale=0.0, kv_layout=KV_BHSD,
         dropout_p=0.0, seed=0) -> Geom:
    """Geometry of one query shard: local rows [row_offset, row_offset+L) of a
    padded sequence of S_full positions, K/V buffer rows = positions
    [kv_offset, kv_offset+S_kv). scale <= 0 means D**-0.5; window <= 0: none;
    kv_layout: KV_BHSD or KV_SBHD (token-major k, v, dk, dv); dropout_p > 0:
    attention dropout drawn from the 64-bit `seed` (the same p and seed in the
    forward and the backward of a step)."""
    seed = int(seed) & 0xFFFFFFFFFFFFFFFF
    v = (int(B), int(Hq), int(Hkv), int(D), int(S_full), int(L), int(row_offset), int(kv_offset), int(S_kv))
    _fit(Geom, v)
    return Geom(*v, _c_window(window), float(scale or 0.0), int(kv_layout), float(dropout_p), seed & 0xFFFFFFFF,
                seed >> 32)


def kv_shape(g: Geom) -> tuple:
    """Shape of k, v, dk, dv for the geometry's K/V layout."""
    return (g.S_kv, g.B, g.Hkv, g.D) if g.kv_layout == KV_SBHD else (g.B, g.Hkv, g.S_kv, g.D)


_lock = threading.Lock()
_lib = None
_calls = None  # the module behind which small calls are made without Python (csrc/calls.cpp)


def _native_calls():
    """The module _calls of this torch and Python, or None, with a warning, where it cannot be loaded: no operator
    needs it."""
    try:
        spec = importlib.util.spec_from_file_location(f"{__package__}._calls", calls_path())
        calls = importlib.util.module_from_spec(spec)
        spec.loader.exec_module(calls)
    except ImportError as e:
        warnings.warn(f"_calls cannot be loaded ({e}): small calls of the paged operators take some 10 us more of the "
                      "host's time; `python -m sliding_window_attention_device_gb300.build` builds it",
                      RuntimeWarning, stacklevel=3)
        return None
    calls.setup(Paged)
    return calls


def load() -> ctypes.CDLL:
    """Load libbdattn.so (raises if it has not been built)."""
    global _lib, _calls
    if _lib is not None:
        return _lib
    with _lock:
        if _lib is not None:
            return _lib
        if not os.path.exists(LIB_PATH):
            raise ImportError(f"{LIB_PATH} is missing: build it with "
                              "`python -m sliding_window_attention_device_gb300.build`")
        lib = ctypes.CDLL(LIB_PATH)
        P, G = ctypes.c_void_p, ctypes.POINTER(Geom)
        lib.bd_attn_seg_bytes.argtypes = [G]
        lib.bd_attn_seg_bytes.restype = ctypes.c_size_t
        lib.bd_attn_seg_layout.argtypes = [G, P]
        lib.bd_attn_seg_layout.restype = ctypes.c_int
        lib.bd_attn_bwd_workspace_bytes.argtypes = [G]
        lib.bd_attn_bwd_workspace_bytes.restype = ctypes.c_size_t
        lib.bd_attn_seg_build.argtypes = [P, G, P, P, P]
        lib.bd_attn_seg_build.restype = ctypes.c_int
        lib.bd_attn_seg_build_chunk.argtypes = [P, G, P, P, P]
        lib.bd_attn_seg_build_chunk.restype = ctypes.c_int
        lib.bd_attn_merge.argtypes = [P, P, P, P, G, P, P]
        lib.bd_attn_merge.restype = ctypes.c_int
        lib.bd_attn_fwd.argtypes = [P, P, P, P, G, P, P, P, P]
        lib.bd_attn_fwd.restype = ctypes.c_int
        lib.bd_attn_fwd_merge.argtypes = [P, P, P, P, G, P, P, P, P]
        lib.bd_attn_fwd_merge.restype = ctypes.c_int
        lib.bd_attn_bwd.argtypes = [P, P, P, P, P, P, P, G, ctypes.c_int, P, P, P, P, P, P]
        lib.bd_attn_bwd.restype = ctypes.c_int
        lib.bd_attn_bwd_deterministic.argtypes = [P, P, P, P, P, P, P, G, ctypes.c_int, P, P, P, P, P, P]
        lib.bd_attn_bwd_deterministic.restype = ctypes.c_int
        lib.bd_attn_bwd_prep.argtypes = [P, P, G, P, P, P]
        lib.bd_attn_bwd_prep.restype = ctypes.c_int
        lib.bd_attn_bwd_main.argtypes = [P, P, P, P, P, P, G, ctypes.c_int, P, P, P, P, P]
        lib.bd_attn_bwd_main.restype = ctypes.c_int
        lib.bd_attn_bwd_finalize.argtypes = [G, ctypes.c_int, P, P, P, P]
        lib.bd_attn_bwd_finalize.restype = ctypes.c_int
        lib.bd_attn_bwd_prep_dq.argtypes = [P, P, G, P, P, P, P]
        lib.bd_attn_bwd_prep_dq.restype = ctypes.c_int
        lib.bd_attn_bwd_main_dq.argtypes = [P, P, P, P, P, P, G, ctypes.c_int, P, P, P, P, P, P]
        lib.bd_attn_bwd_main_dq.restype = ctypes.c_int
        I = ctypes.c_int
        lib.bd_attn_plan_bytes.argtypes = [I, I, I]
        lib.bd_attn_plan_bytes.restype = ctypes.c_size_t
        lib.bd_attn_plan_layout.argtypes = [I, I, I, P]
        lib.bd_attn_plan_layout.restype = I
        lib.bd_attn_exchange_plan.argtypes = [P, I, I, I, I, P, P, P]
        lib.bd_attn_exchange_plan.restype = I
        lib.bd_attn_needed_gather.argtypes = [P, P, I, I, I, I, I, P, I, P, P]
        lib.bd_attn_needed_gather.restype = I
        lib.bd_attn_needed_scatter_add.argtypes = [P, P, I, I, I, I, I, P, I, P, P]
        lib.bd_attn_needed_scatter_add.restype = I
        for name in ("bd_attn_sink_seg_bytes", "bd_attn_sink_bwd_workspace_bytes"):
            getattr(lib, name).argtypes = [G, I]
            getattr(lib, name).restype = ctypes.c_size_t
        lib.bd_attn_sink_seg_build.argtypes = [P, G, I, I, P, P, P]
        lib.bd_attn_sink_fwd.argtypes = [P, P, P, P, G, I, P, P, P, P]
        lib.bd_attn_sink_fwd_merge.argtypes = [P, P, P, P, G, I, P, P, P, P]
        lib.bd_attn_sink_bwd.argtypes = [P, P, P, P, P, P, P, G, I, I, P, P, P, P, P, P]
        lib.bd_attn_sink_bwd_deterministic.argtypes = [P, P, P, P, P, P, P, G, I, I, P, P, P, P, P, P]
        lib.bd_attn_sink_bwd_main.argtypes = [P, P, P, P, P, P, G, I, I, P, P, P, P, P]
        for name in ("seg_build", "fwd", "fwd_merge", "bwd", "bwd_deterministic", "bwd_main"):
            getattr(lib, "bd_attn_sink_" + name).restype = I
        PG = ctypes.POINTER(Paged)
        lib.bd_attn_paged_append.argtypes = [P, P, P, P, P, PG, I, P, P, P, P]
        lib.bd_attn_paged_append.restype = I
        lib.bd_attn_paged_decode_workspace_bytes.argtypes = [PG]
        lib.bd_attn_paged_decode_workspace_bytes.restype = ctypes.c_size_t
        lib.bd_attn_paged_decode.argtypes = [P, P, P, P, P, PG, P, P, P, P, P]
        lib.bd_attn_paged_decode.restype = I
        RP, C4 = ctypes.POINTER(Rope), ctypes.POINTER(_Cache4)
        lib.bd_attn_paged_append_rope.argtypes = [P, P, P, P, RP, P, P, P, PG, I, P, P, P, P, P, P]
        lib.bd_attn_paged_append_rope.restype = I
        lib.bd_attn_paged4_append.argtypes = [P, P, P, P, RP, P, P, P, PG, I, P, P, C4, P, P]
        lib.bd_attn_paged4_append.restype = I
        lib.bd_attn_paged4_read.argtypes = [C4, P, P, P, PG, I, P, P, P, P]
        lib.bd_attn_paged4_read.restype = I
        lib.bd_attn_paged4_decode_workspace_bytes.argtypes = [PG]
        lib.bd_attn_paged4_decode_workspace_bytes.restype = ctypes.c_size_t
        lib.bd_attn_paged4_decode.argtypes = [P, C4, P, P, PG, P, P, P, P, P]
        lib.bd_attn_paged4_decode.restype = I
        _calls = _native_calls()
        lib.bd_attn_strerror.argtypes = [ctypes.c_int]
        lib.bd_attn_strerror.restype = ctypes.c_char_p
        lib.bd_attn_selftest_wait_timeout.argtypes = [P, ctypes.c_uint64, P]
        lib.bd_attn_selftest_wait_timeout.restype = ctypes.c_int
        _lib = lib
        return lib


def strerror(code: int) -> str:
    return load().bd_attn_strerror(int(code)).decode()


def _check(rc: int, what: str):
    if rc != BD_OK:
        raise RuntimeError(f"{what} failed: {strerror(rc)} (code {rc})")


def _stream(stream):
    s = torch.cuda.current_stream() if stream is None else stream
    return ctypes.c_void_p(s.cuda_stream)


def _ptr(t: torch.Tensor):
    return ctypes.c_void_p(t.data_ptr())


def _need(t: torch.Tensor, name: str, dtype, shape, device):
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dtype != dtype:
        raise ValueError(f"{name}: dtype {t.dtype}, expected {dtype}")
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name}: shape {tuple(t.shape)}, expected {tuple(shape)}")
    if not t.is_cuda or (device is not None and t.device != device):
        raise ValueError(f"{name} must be on {device or 'a CUDA device'}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")


def seg_bytes(g: Geom) -> int:
    n = load().bd_attn_seg_bytes(ctypes.byref(g))
    if n == 0:
        raise ValueError(f"invalid geometry {g}")
    return int(n)


def seg_layout(g: Geom) -> dict:
    arr = (ctypes.c_int32 * (len(REGIONS) + 3))()
    _check(load().bd_attn_seg_layout(ctypes.byref(g), arr), "bd_attn_seg_layout")
    d = {name: int(arr[i]) for i, name in enumerate(REGIONS)}
    d["nqt"], d["nkt"], d["nkw"] = int(arr[len(REGIONS)]), int(arr[len(REGIONS) + 1]), int(arr[len(REGIONS) + 2])
    return d


def bwd_workspace_bytes(g: Geom) -> int:
    n = load().bd_attn_bwd_workspace_bytes(ctypes.byref(g))
    if n == 0:
        raise ValueError(f"invalid geometry {g}")
    return int(n)


def new_status(device) -> torch.Tensor:
    return torch.zeros(1, dtype=torch.int32, device=device)


def bd_attn_seg_build(doc_ids: torch.Tensor, g: Geom, seg: torch.Tensor | None = None,
                      status: torch.Tensor | None = None, stream=None):
    """Segment table of the shard (device); returns (seg, status)."""
    dev = doc_ids.device
    _need(doc_ids, "doc_ids", torch.int32, (g.B, g.S_full), None)
    if seg is None:
        seg = torch.empty(seg_bytes(g) // 4, dtype=torch.int32, device=dev)
    if status is None:
        status = new_status(dev)
    _need(seg, "seg", torch.int32, (seg_bytes(g) // 4,), dev)
    _need(status, "status", torch.int32, (1,), dev)
    _check(load().bd_attn_seg_build(_ptr(doc_ids), ctypes.byref(g), _ptr(seg), _ptr(status), _stream(stream)),
           "bd_attn_seg_build")
    return seg, status


def bd_attn_seg_build_chunk(doc_ids: torch.Tensor, g: Geom, seg: torch.Tensor | None = None,
                            status: torch.Tensor | None = None, stream=None):
    """Segment table for one chunk of the K/V range (no K/V range requirement); returns (seg, status)."""
    dev = doc_ids.device
    _need(doc_ids, "doc_ids", torch.int32, (g.B, g.S_full), None)
    if seg is None:
        seg = torch.empty(seg_bytes(g) // 4, dtype=torch.int32, device=dev)
    if status is None:
        status = new_status(dev)
    _need(seg, "seg", torch.int32, (seg_bytes(g) // 4,), dev)
    _need(status, "status", torch.int32, (1,), dev)
    _check(load().bd_attn_seg_build_chunk(_ptr(doc_ids), ctypes.byref(g), _ptr(seg), _ptr(status),
                                          _stream(stream)), "bd_attn_seg_build_chunk")
    return seg, status


def bd_attn_merge(out, lse, out_chunk, lse_chunk, g: Geom, status, stream=None):
    """Merge a K/V chunk's (out, lse) into the running (out, lse), in place."""
    dev = out.device
    for name, t in (("out", out), ("out_chunk", out_chunk)):
        _need(t, name, torch.bfloat16, (g.B, g.Hq, g.L, g.D), dev)
    for name, t in (("lse", lse), ("lse_chunk", lse_chunk)):
        _need(t, name, torch.float32, (g.B, g.Hq, g.L), dev)
    _need(status, "status", torch.int32, (1,), dev)
    _check(load().bd_attn_merge(_ptr(out), _ptr(lse), _ptr(out_chunk), _ptr(lse_chunk), ctypes.byref(g),
                                _ptr(status), _stream(stream)), "bd_attn_merge")


def bd_attn_fwd(q, k, v, seg, g: Geom, status, out=None, lse=None, stream=None):
    """out [B,Hq,L,D] bf16 and lse [B,Hq,L] fp32 (natural log; -inf on padding rows)."""
    dev = q.device
    _need(q, "q", torch.bfloat16, (g.B, g.Hq, g.L, g.D), dev)
    _need(k, "k", torch.bfloat16, kv_shape(g), dev)
    _need(v, "v", torch.bfloat16, kv_shape(g), dev)
    _need(seg, "seg", torch.int32, (seg_bytes(g) // 4,), dev)
    _need(status, "status", torch.int32, (1,), dev)
    if out is None:
        out = torch.empty(g.B, g.Hq, g.L, g.D, dtype=torch.bfloat16, device=dev)
    if lse is None:
        lse = torch.empty(g.B, g.Hq, g.L, dtype=torch.float32, device=dev)
    _need(out, "out", torch.bfloat16, (g.B, g.Hq, g.L, g.D), dev)
    _need(lse, "lse", torch.float32, (g.B, g.Hq, g.L), dev)
    _check(load().bd_attn_fwd(_ptr(q), _ptr(k), _ptr(v), _ptr(seg), ctypes.byref(g), _ptr(out), _ptr(lse),
                              _ptr(status), _stream(stream)), "bd_attn_fwd")
    return out, lse


def bd_attn_fwd_merge(q, k, v, seg, g: Geom, status, out, lse, stream=None):
    """Forward over one K/V chunk merged into the running (out, lse), in place."""
    dev = q.device
    _need(q, "q", torch.bfloat16, (g.B, g.Hq, g.L, g.D), dev)
    _need(k, "k", torch.bfloat16, kv_shape(g), dev)
    _need(v, "v", torch.bfloat16, kv_shape(g), dev)
    _need(seg, "seg", torch.int32, (seg_bytes(g) // 4,), dev)
    _need(status, "status", torch.int32, (1,), dev)
    _need(out, "out", torch.bfloat16, (g.B, g.Hq, g.L, g.D), dev)
    _need(lse, "lse", torch.float32, (g.B, g.Hq, g.L), dev)
    _check(load().bd_attn_fwd_merge(_ptr(q), _ptr(k), _ptr(v), _ptr(seg), ctypes.byref(g), _ptr(out), _ptr(lse),
                                    _ptr(status), _stream(stream)), "bd_attn_fwd_merge")
    return out, lse


def bd_attn_bwd(dout, q, k, v, out, lse, seg, g: Geom, status, grad_dtype=torch.float32, dq=None, dk=None,
                dv=None, workspace=None, stream=None, _fn="bd_attn_bwd"):
    """dq [B,Hq,L,D], dk / dv [B,Hkv,S_kv,D] (summed over each GQA group) in grad_dtype."""
    dev = q.device
    if grad_dtype not in (torch.float32, torch.bfloat16):
        raise ValueError("grad_dtype must be torch.float32 or torch.bfloat16")
    for name, t in (("dout", dout), ("q", q), ("out", out)):
        _need(t, name, torch.bfloat16, (g.B, g.Hq, g.L, g.D), dev)
    _need(k, "k", torch.bfloat16, kv_shape(g), dev)
    _need(v, "v", torch.bfloat16, kv_shape(g), dev)
    _need(lse, "lse", torch.float32, (g.B, g.Hq, g.L), dev)
    _need(seg, "seg", torch.int32, (seg_bytes(g) // 4,), dev)
    _need(status, "status", torch.int32, (1,), dev)
    if dq is None:
        dq = torch.empty(g.B, g.Hq, g.L, g.D, dtype=grad_dtype, device=dev)
    if dk is None:
        dk = torch.empty(kv_shape(g), dtype=grad_dtype, device=dev)
    if dv is None:
        dv = torch.empty(kv_shape(g), dtype=grad_dtype, device=dev)
    if workspace is None:
        workspace = torch.empty(bwd_workspace_bytes(g), dtype=torch.uint8, device=dev)
    _need(dq, "dq", grad_dtype, (g.B, g.Hq, g.L, g.D), dev)
    _need(dk, "dk", grad_dtype, kv_shape(g), dev)
    _need(dv, "dv", grad_dtype, kv_shape(g), dev)
    _need(workspace, "workspace", torch.uint8, (bwd_workspace_bytes(g),), dev)
    code = BD_DTYPE_BF16 if grad_dtype == torch.bfloat16 else BD_DTYPE_F32
    _check(getattr(load(), _fn)(_ptr(dout), _ptr(q), _ptr(k), _ptr(v), _ptr(out), _ptr(lse), _ptr(seg),
                                ctypes.byref(g), code, _ptr(dq), _ptr(dk), _ptr(dv), _ptr(workspace), _ptr(status),
                                _stream(stream)), _fn)
    return dq, dk, dv


def bd_attn_bwd_deterministic(dout, q, k, v, out, lse, seg, g: Geom, status, grad_dtype=torch.float32, dq=None,
                              dk=None, dv=None, workspace=None, stream=None):
    """bd_attn_bwd with bitwise reproducible results (dq by a fixed-order pass)."""
    return bd_attn_bwd(dout, q, k, v, out, lse, seg, g, status, grad_dtype, dq, dk, dv, workspace, stream,
                       _fn="bd_attn_bwd_deterministic")


def bd_attn_bwd_prep(dout, out, g: Geom, status, workspace, stream=None):
    """Stage 1 of bd_attn_bwd: delta and a zeroed dq accumulator in `workspace`."""
    dev = out.device
    _need(dout, "dout", torch.bfloat16, (g.B, g.Hq, g.L, g.D), dev)
    _need(out, "out", torch.bfloat16, (g.B, g.Hq, g.L, g.D), dev)
    _need(workspace, "workspace", torch.uint8, (bwd_workspace_bytes(g),), dev)
    _need(status, "status", torch.int32, (1,), dev)
    _check(load().bd_attn_bwd_prep(_ptr(dout), _ptr(out), ctypes.byref(g), _ptr(workspace), _ptr(status),
                                   _stream(stream)), "bd_attn_bwd_prep")


def bd_attn_bwd_main(dout, q, k, v, lse, seg, g: Geom, status, workspace, dk, dv, stream=None):
    """Stage 2 of bd_attn_bwd: dk, dv (dtype of dk) and the dq accumulation."""
    dev = q.device
    gd = dk.dtype
    if gd not in (torch.float32, torch.bfloat16):
        raise ValueError("dk / dv must be float32 or bfloat16")
    for name, t in (("dout", dout), ("q", q)):
        _need(t, name, torch.bfloat16, (g.B, g.Hq, g.L, g.D), dev)
    _need(k, "k", torch.bfloat16, kv_shape(g), dev)
    _need(v, "v", torch.bfloat16, kv_shape(g), dev)
    _need(lse, "lse", torch.float32, (g.B, g.Hq, g.L), dev)
    _need(seg, "seg", torch.int32, (seg_bytes(g) // 4,), dev)
    _need(dk, "dk", gd, kv_shape(g), dev)
    _need(dv, "dv", gd, kv_shape(g), dev)
    _need(workspace, "workspace", torch.uint8, (bwd_workspace_bytes(g),), dev)
    _need(status, "status", torch.int32, (1,), dev)
    code = BD_DTYPE_BF16 if gd == torch.bfloat16 else BD_DTYPE_F32
    _check(load().bd_attn_bwd_main(_ptr(dout), _ptr(q), _ptr(k), _ptr(v), _ptr(lse), _ptr(seg), ctypes.byref(g),
                                   code, _ptr(dk), _ptr(dv), _ptr(workspace), _ptr(status), _stream(stream)),
           "bd_attn_bwd_main")


def bd_attn_bwd_finalize(g: Geom, status, workspace, dq, stream=None):
    """Stage 3 of bd_attn_bwd: dq = the (already scaled) accumulator, in the dtype of dq."""
    dev = dq.device
    if dq.dtype not in (torch.float32, torch.bfloat16):
        raise ValueError("dq must be float32 or bfloat16")
    _need(dq, "dq", dq.dtype, (g.B, g.Hq, g.L, g.D), dev)
    _need(workspace, "workspace", torch.uint8, (bwd_workspace_bytes(g),), dev)
    _need(status, "status", torch.int32, (1,), dev)
    code = BD_DTYPE_BF16 if dq.dtype == torch.bfloat16 else BD_DTYPE_F32
    _check(load().bd_attn_bwd_finalize(ctypes.byref(g), code, _ptr(dq), _ptr(workspace), _ptr(status),
                                       _stream(stream)), "bd_attn_bwd_finalize")


def bd_attn_bwd_prep_dq(dout, out, g: Geom, status, workspace, dq, stream=None):
    """Stage 1 with the fp32 dq as accumulator: delta in `workspace`, dq zeroed."""
    dev = out.device
    _need(dout, "dout", torch.bfloat16, (g.B, g.Hq, g.L, g.D), dev)
    _need(out, "out", torch.bfloat16, (g.B, g.Hq, g.L, g.D), dev)
    _need(workspace, "workspace", torch.uint8, (bwd_workspace_bytes(g),), dev)
    _need(dq, "dq", torch.float32, (g.B, g.Hq, g.L, g.D), dev)
    _need(status, "status", torch.int32, (1,), dev)
    _check(load().bd_attn_bwd_prep_dq(_ptr(dout), _ptr(out), ctypes.byref(g), _ptr(workspace), _ptr(dq),
                                      _ptr(status), _stream(stream)), "bd_attn_bwd_prep_dq")


def bd_attn_bwd_main_dq(dout, q, k, v, lse, seg, g: Geom, status, workspace, dq, dk, dv, stream=None):
    """Stage 2 with the fp32 dq as accumulator: dk, dv (dtype of dk) and dq += scale * dS K."""
    dev = q.device
    gd = dk.dtype
    if gd not in (torch.float32, torch.bfloat16):
        raise ValueError("dk / dv must be float32 or bfloat16")
    for name, t in (("dout", dout), ("q", q)):
        _need(t, name, torch.bfloat16, (g.B, g.Hq, g.L, g.D), dev)
    _need(k, "k", torch.bfloat16, kv_shape(g), dev)
    _need(v, "v", torch.bfloat16, kv_shape(g), dev)
    _need(lse, "lse", torch.float32, (g.B, g.Hq, g.L), dev)
    _need(seg, "seg", torch.int32, (seg_bytes(g) // 4,), dev)
    _need(dq, "dq", torch.float32, (g.B, g.Hq, g.L, g.D), dev)
    _need(dk, "dk", gd, kv_shape(g), dev)
    _need(dv, "dv", gd, kv_shape(g), dev)
    _need(workspace, "workspace", torch.uint8, (bwd_workspace_bytes(g),), dev)
    _need(status, "status", torch.int32, (1,), dev)
    code = BD_DTYPE_BF16 if gd == torch.bfloat16 else BD_DTYPE_F32
    _check(load().bd_attn_bwd_main_dq(_ptr(dout), _ptr(q), _ptr(k), _ptr(v), _ptr(lse), _ptr(seg), ctypes.byref(g),
                                      code, _ptr(dq), _ptr(dk), _ptr(dv), _ptr(workspace), _ptr(status),
                                      _stream(stream)), "bd_attn_bwd_main_dq")


def selftest_wait_timeout(limit_ns: int, status: torch.Tensor, stream=None):
    _need(status, "status", torch.int32, (1,), None)
    _check(load().bd_attn_selftest_wait_timeout(_ptr(status), int(limit_ns), _stream(stream)),
           "bd_attn_selftest_wait_timeout")


def read_seg(seg: torch.Tensor, g: Geom) -> dict:
    """Copy the segment table to the host and decode it (synchronises; tests and tools only)."""
    lay = seg_layout(g)
    a = seg.cpu().numpy()
    L, B, nqt, nkt, nkw = g.L, g.B, lay["nqt"], lay["nkt"], lay["nkw"]
    rows = []
    for b in range(B):
        h = a[lay["hdr"] + b * HDR_WORDS: lay["hdr"] + (b + 1) * HDR_WORDS]
        d = {name: int(h[i]) for i, name in enumerate(HDR_FIELDS)}
        n = d["n_seg"]
        cq = a[lay["cu_q"] + b * (L + 1): lay["cu_q"] + (b + 1) * (L + 1)]
        ck = a[lay["cu_k"] + b * (L + 1): lay["cu_k"] + (b + 1) * (L + 1)]
        d["cu_q"] = cq[:n + 1].copy()
        d["cu_k"] = ck[:n + 1].copy()
        d["row_lo"] = a[lay["row_lo"] + b * L: lay["row_lo"] + (b + 1) * L].copy()
        d["qt_krange"] = a[lay["qt_krange"] + b * nqt * 2: lay["qt_krange"] + (b + 1) * nqt * 2].reshape(nqt, 2).copy()
        d["kt_qrange"] = a[lay["kt_qrange"] + b * nkt * 2: lay["kt_qrange"] + (b + 1) * nkt * 2].reshape(nkt, 2).copy()
        d["full_bits"] = a[lay["full_bits"] + b * nqt * nkw: lay["full_bits"] + (b + 1) * nqt * nkw].reshape(nqt, nkw).copy()
        rows.append(d)
    return {"rows": rows,
            "fwd_work": a[lay["fwd_work"]: lay["fwd_work"] + B * nqt].copy(),
            "bwd_work": a[lay["bwd_work"]: lay["bwd_work"] + B * nkt].copy(),
            "counts": a[lay["counts"]: lay["counts"] + 4].copy(),
            "layout": lay}


# ------------------------------------------------------------ attention sinks
SINK_MAX = 128  # BD_SINK_MAX


def _want(dev, *tensors):
    """_need for every (tensor, name, dtype, shape); one test each when nothing is wrong, as small calls are
    bound by the host."""
    i = dev.index
    for t, name, dtype, shape in tensors:
        if not (isinstance(t, torch.Tensor) and t.dtype is dtype and t.get_device() == i and t.shape == shape
                and t.is_contiguous()):
            _need(t, name, dtype, shape, dev)


def _cuda_device(t, name):
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    return t.device


def _elsewhere(dev, stream):
    """The context in which a call on `stream` (None: the current one of `dev`) runs -- its device and stream
    current, so that what the call allocates belongs to that stream -- or None when it is that already."""
    if stream is not None:
        if stream.device != dev:
            raise ValueError(f"the stream is on {stream.device}, the tensors are on {dev}")
        return torch.cuda.stream(stream)
    return None if dev.index == torch.cuda.current_device() else torch.cuda.device(dev)


# the current stream's handle without making a Stream object of it, where torch offers that
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _current(dev) -> int:
    return torch.cuda.current_stream(dev).cuda_stream if _raw_stream is None else _raw_stream(dev.index)


_BF16, _F32, _I32, _U8 = torch.bfloat16, torch.float32, torch.int32, torch.uint8


def sink_seg_bytes(g: Geom, n_sink: int) -> int:
    n = load().bd_attn_sink_seg_bytes(ctypes.byref(g), int(n_sink)) if 0 <= n_sink <= SINK_MAX else 0
    if n == 0:
        raise ValueError(f"invalid geometry {g} or n_sink={n_sink} (0 to {SINK_MAX})")
    return int(n)


def sink_bwd_workspace_bytes(g: Geom, n_sink: int) -> int:
    n = load().bd_attn_sink_bwd_workspace_bytes(ctypes.byref(g), int(n_sink)) if 0 <= n_sink <= SINK_MAX else 0
    if n == 0:
        raise ValueError(f"invalid geometry {g} or n_sink={n_sink} (0 to {SINK_MAX})")
    return int(n)


def bd_attn_sink_seg_build(doc_ids: torch.Tensor, g: Geom, n_sink: int, kv_chunk: bool = False,
                           seg: torch.Tensor | None = None, status: torch.Tensor | None = None, stream=None):
    """Table of the shard with the first `n_sink` tokens of every document
    visible past the window; `kv_chunk`: of one chunk of the K/V range. Returns
    (seg, status); `seg` serves every bd_attn_sink_* call of this geometry and n_sink."""
    dev = _cuda_device(doc_ids, "doc_ids")
    if (ctx := _elsewhere(dev, stream)) is not None:
        with ctx:
            return bd_attn_sink_seg_build(doc_ids, g, n_sink, kv_chunk, seg, status)
    n = sink_seg_bytes(g, n_sink) // 4
    if seg is None:
        seg = torch.empty(n, dtype=torch.int32, device=dev)
    if status is None:
        status = new_status(dev)
    _want(dev, (doc_ids, "doc_ids", _I32, (g.B, g.S_full)), (seg, "seg", _I32, (n,)), (status, "status", _I32, (1,)))
    _check(load().bd_attn_sink_seg_build(doc_ids.data_ptr(), ctypes.byref(g), int(n_sink), int(bool(kv_chunk)),
                                         seg.data_ptr(), status.data_ptr(), _current(dev)), "bd_attn_sink_seg_build")
    return seg, status


def bd_attn_sink_fwd(q, k, v, seg, g: Geom, n_sink: int, status, out=None, lse=None, stream=None,
                     _fn="bd_attn_sink_fwd"):
    """bd_attn_fwd with the documents' first n_sink tokens visible past the window."""
    dev = _cuda_device(q, "q")
    if (ctx := _elsewhere(dev, stream)) is not None:
        with ctx:
            return bd_attn_sink_fwd(q, k, v, seg, g, n_sink, status, out, lse, None, _fn)
    rows, kv = (g.B, g.Hq, g.L, g.D), kv_shape(g)
    if out is None:
        out = torch.empty_like(q)
    if lse is None:
        lse = torch.empty(rows[:3], dtype=_F32, device=dev)
    _want(dev, (q, "q", _BF16, rows), (k, "k", _BF16, kv), (v, "v", _BF16, kv),
          (seg, "seg", _I32, (sink_seg_bytes(g, n_sink) // 4,)), (status, "status", _I32, (1,)),
          (out, "out", _BF16, rows), (lse, "lse", _F32, rows[:3]))
    _check(getattr(load(), _fn)(q.data_ptr(), k.data_ptr(), v.data_ptr(), seg.data_ptr(), ctypes.byref(g),
                                int(n_sink), out.data_ptr(), lse.data_ptr(), status.data_ptr(), _current(dev)), _fn)
    return out, lse


def bd_attn_sink_fwd_merge(q, k, v, seg, g: Geom, n_sink: int, status, out, lse, stream=None):
    """bd_attn_sink_fwd over one K/V chunk merged into the running (out, lse), in place."""
    if out is None or lse is None:
        raise ValueError("out and lse hold the running result")
    return bd_attn_sink_fwd(q, k, v, seg, g, n_sink, status, out, lse, stream, _fn="bd_attn_sink_fwd_merge")


def bd_attn_sink_bwd(dout, q, k, v, out, lse, seg, g: Geom, n_sink: int, status, grad_dtype=torch.float32, dq=None,
                     dk=None, dv=None, workspace=None, stream=None, _fn="bd_attn_sink_bwd"):
    """Gradients of bd_attn_sink_fwd: dq [B,Hq,L,D], dk / dv in k's layout (summed over each GQA group)."""
    dev = _cuda_device(q, "q")
    if (ctx := _elsewhere(dev, stream)) is not None:
        with ctx:
            return bd_attn_sink_bwd(dout, q, k, v, out, lse, seg, g, n_sink, status, grad_dtype, dq, dk, dv,
                                    workspace, None, _fn)
    if grad_dtype not in (torch.float32, torch.bfloat16):
        raise ValueError("grad_dtype must be torch.float32 or torch.bfloat16")
    rows, kv = (g.B, g.Hq, g.L, g.D), kv_shape(g)
    n = sink_bwd_workspace_bytes(g, n_sink)
    if dq is None:
        dq = torch.empty_like(q, dtype=grad_dtype)
    if dk is None:
        dk = torch.empty_like(k, dtype=grad_dtype)
    if dv is None:
        dv = torch.empty_like(v, dtype=grad_dtype)
    if workspace is None:
        workspace = torch.empty(n, dtype=torch.uint8, device=dev)
    _want(dev, (dout, "dout", _BF16, rows), (q, "q", _BF16, rows), (out, "out", _BF16, rows), (k, "k", _BF16, kv),
          (v, "v", _BF16, kv), (lse, "lse", _F32, rows[:3]), (seg, "seg", _I32, (sink_seg_bytes(g, n_sink) // 4,)),
          (status, "status", _I32, (1,)), (dq, "dq", grad_dtype, rows), (dk, "dk", grad_dtype, kv),
          (dv, "dv", grad_dtype, kv), (workspace, "workspace", _U8, (n,)))
    code = BD_DTYPE_BF16 if grad_dtype == torch.bfloat16 else BD_DTYPE_F32
    _check(getattr(load(), _fn)(dout.data_ptr(), q.data_ptr(), k.data_ptr(), v.data_ptr(), out.data_ptr(),
                                lse.data_ptr(), seg.data_ptr(), ctypes.byref(g), int(n_sink), code, dq.data_ptr(),
                                dk.data_ptr(), dv.data_ptr(), workspace.data_ptr(), status.data_ptr(),
                                _current(dev)), _fn)
    return dq, dk, dv


def bd_attn_sink_bwd_deterministic(dout, q, k, v, out, lse, seg, g: Geom, n_sink: int, status,
                                   grad_dtype=torch.float32, dq=None, dk=None, dv=None, workspace=None, stream=None):
    """bd_attn_sink_bwd with bitwise reproducible results (dq by a fixed-order pass)."""
    return bd_attn_sink_bwd(dout, q, k, v, out, lse, seg, g, n_sink, status, grad_dtype, dq, dk, dv, workspace,
                            stream, _fn="bd_attn_sink_bwd_deterministic")


def bd_attn_sink_bwd_main(dout, q, k, v, lse, seg, g: Geom, n_sink: int, status, workspace, dk, dv, stream=None):
    """bd_attn_bwd_main with sinks, for K/V chunks: dk, dv (dtype of dk) of the chunk and its dq share, between
    bd_attn_bwd_prep and bd_attn_bwd_finalize. `workspace`: uint8, at least sink_bwd_workspace_bytes of every
    chunk; the other two stages take its first bwd_workspace_bytes(g) bytes."""
    dev = _cuda_device(q, "q")
    if (ctx := _elsewhere(dev, stream)) is not None:
        with ctx:
            return bd_attn_sink_bwd_main(dout, q, k, v, lse, seg, g, n_sink, status, workspace, dk, dv)
    _cuda_device(dk, "dk"), _cuda_device(workspace, "workspace")
    gd = dk.dtype
    if gd not in (torch.float32, torch.bfloat16):
        raise ValueError("dk / dv must be float32 or bfloat16")
    rows, kv = (g.B, g.Hq, g.L, g.D), kv_shape(g)
    _want(dev, (dout, "dout", _BF16, rows), (q, "q", _BF16, rows), (k, "k", _BF16, kv), (v, "v", _BF16, kv),
          (lse, "lse", _F32, rows[:3]), (seg, "seg", _I32, (sink_seg_bytes(g, n_sink) // 4,)), (dk, "dk", gd, kv),
          (dv, "dv", gd, kv), (workspace, "workspace", _U8, (workspace.numel(),)), (status, "status", _I32, (1,)))
    n = sink_bwd_workspace_bytes(g, n_sink)
    if workspace.numel() < n:
        raise ValueError(f"workspace: {workspace.numel()} bytes, {n} needed")
    code = BD_DTYPE_BF16 if gd == torch.bfloat16 else BD_DTYPE_F32
    _check(load().bd_attn_sink_bwd_main(dout.data_ptr(), q.data_ptr(), k.data_ptr(), v.data_ptr(), lse.data_ptr(),
                                        seg.data_ptr(), ctypes.byref(g), int(n_sink), code, dk.data_ptr(),
                                        dv.data_ptr(), workspace.data_ptr(), status.data_ptr(), _current(dev)),
           "bd_attn_sink_bwd_main")


# ------------------------------------------------------------ paged K/V cache
def paged_geom(B, Hq, Hkv, D, n_pages, page_size, max_pages, window=0, n_sink=0, scale=0.0) -> Paged:
    """Geometry of a paged cache [n_pages, Hkv, page_size, D] and the B sequences
    in it (page table [B, max_pages]); window <= 0: none; n_sink: first tokens
    that stay visible past the window; scale <= 0 means D**-0.5."""
    v = (int(B), int(Hq), int(Hkv), int(D), int(n_pages), int(page_size), int(max_pages),
         window if window.__class__ is int and -1 < window <= _INT_MAX else _c_window(window),
         int(n_sink) if n_sink <= _INT_MAX else _INT_MAX)
    _fit(Paged, v)
    return Paged(*v, float(scale or 0.0))


def paged_decode_workspace_bytes(pg: Paged) -> int:
    n = load().bd_attn_paged_decode_workspace_bytes(ctypes.byref(pg))
    if n == 0:
        raise ValueError(f"invalid geometry {pg}")
    return int(n)


def bd_attn_paged_append(k_new, v_new, cu_new, seq_lens, page_table, pg: Paged, k_pages, v_pages, status,
                         stream=None):
    """Write k_new, v_new [T, Hkv, D] (sequence b's tokens at [cu_new[b], cu_new[b+1]), the last one at position
    seq_lens[b] - 1) into k_pages, v_pages in place."""
    dev = _cuda_device(k_pages, "k_pages")
    if (ctx := _elsewhere(dev, stream)) is not None:
        with ctx:
            return bd_attn_paged_append(k_new, v_new, cu_new, seq_lens, page_table, pg, k_pages, v_pages, status)
    _cuda_device(k_new, "k_new")
    n, B = k_new.shape[0] if k_new.dim() else 0, pg.B
    cache, new = (pg.n_pages, pg.Hkv, pg.page_size, pg.D), (n, pg.Hkv, pg.D)
    _want(dev, (k_new, "k_new", _BF16, new), (v_new, "v_new", _BF16, new), (cu_new, "cu_new", _I32, (B + 1,)),
          (seq_lens, "seq_lens", _I32, (B,)), (page_table, "page_table", _I32, (B, pg.max_pages)),
          (k_pages, "k_pages", _BF16, cache), (v_pages, "v_pages", _BF16, cache), (status, "status", _I32, (1,)))
    _check(load().bd_attn_paged_append(k_new.data_ptr(), v_new.data_ptr(), cu_new.data_ptr(), seq_lens.data_ptr(),
                                       page_table.data_ptr(), ctypes.byref(pg), n, k_pages.data_ptr(),
                                       v_pages.data_ptr(), status.data_ptr(), _current(dev)), "bd_attn_paged_append")


def bd_attn_paged_decode(q, k_pages, v_pages, page_table, seq_lens, pg: Paged, status, out=None, lse=None,
                         workspace=None, stream=None):
    """out [B, Hq, D] bf16 and lse [B, Hq] fp32 of one new token per sequence (q [B, Hq, D], at position
    seq_lens[b] - 1) over its cached keys; out 0 and lse -inf for a sequence of length 0."""
    dev = _cuda_device(q, "q")
    if (ctx := _elsewhere(dev, stream)) is not None:
        with ctx:
            return bd_attn_paged_decode(q, k_pages, v_pages, page_table, seq_lens, pg, status, out, lse, workspace)
    rows, cache = (pg.B, pg.Hq, pg.D), (pg.n_pages, pg.Hkv, pg.page_size, pg.D)
    n = paged_decode_workspace_bytes(pg)
    if out is None:
        out = torch.empty_like(q)
    if lse is None:
        lse = torch.empty(rows[:2], dtype=_F32, device=dev)
    if workspace is None and n > 16:  # 16: the call needs none
        workspace = torch.empty(n, dtype=_U8, device=dev)
    _want(dev, (q, "q", _BF16, rows), (k_pages, "k_pages", _BF16, cache), (v_pages, "v_pages", _BF16, cache),
          (page_table, "page_table", _I32, (rows[0], pg.max_pages)), (seq_lens, "seq_lens", _I32, rows[:1]),
          (status, "status", _I32, (1,)), (out, "out", _BF16, rows), (lse, "lse", _F32, rows[:2]))
    if workspace is not None:
        _want(dev, (workspace, "workspace", _U8, (n,)))
    _check(load().bd_attn_paged_decode(q.data_ptr(), k_pages.data_ptr(), v_pages.data_ptr(), page_table.data_ptr(),
                                       seq_lens.data_ptr(), ctypes.byref(pg), out.data_ptr(), lse.data_ptr(),
                                       workspace.data_ptr() if workspace is not None else None, status.data_ptr(),
                                       _current(dev)), "bd_attn_paged_decode")
    return out, lse


# ------------------------------- rotation on the way in, and pages held in 4 bits
# Small calls are bound by the host, so each function first hands its arguments to its namesake in _calls, which
# makes the call where all is as it should be and returns None, having done nothing, where something is not. What
# follows then does the same in Python: it finds what is wrong (_want, which raises), changes to the tensors' device
# or the stream, or makes the call.
_E4M3 = torch.float8_e4m3fn
_empty = torch.empty
_device_now = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)


def paged4_cache(pg: Paged, device, k_gain: float = 1.0, v_gain: float = 1.0) -> Cache4:
    """An empty cache of the geometry, held in 4 bits. The gains bring keys and values into the range that 4-bit
    blocks hold, 0.006 to 2688 times the gain."""
    pages = (pg.n_pages, pg.Hkv, pg.page_size)
    codes = [torch.empty(*pages, pg.D // 2, dtype=_U8, device=device) for _ in range(2)]
    blocks = [torch.empty(*pages, pg.D // 16, dtype=_E4M3, device=device) for _ in range(2)]
    return Cache4(*codes, *blocks, float(k_gain), float(v_gain))


def paged4_decode_workspace_bytes(pg: Paged) -> int:
    n = load().bd_attn_paged4_decode_workspace_bytes(ctypes.byref(pg))
    if n == 0:
        raise ValueError(f"invalid geometry {pg}")
    return int(n)


def _cache4(dev, i: int, cache: Cache4, pages, Hkv: int, page: int, D: int) -> _Cache4:
    kc, vc, kb, vb, kg, vg = cache
    codes, blocks = (pages, Hkv, page, D // 2), (pages, Hkv, page, D // 16)
    try:
        ok = (kc.dtype is _U8 and vc.dtype is _U8 and kb.dtype is _E4M3 and vb.dtype is _E4M3
              and kc.shape == codes and vc.shape == codes and kb.shape == blocks and vb.shape == blocks
              and kc.get_device() == i and vc.get_device() == i and kb.get_device() == i and vb.get_device() == i
              and kc.is_contiguous() and vc.is_contiguous() and kb.is_contiguous() and vb.is_contiguous())
    except AttributeError:
        ok = False
    if not ok:
        _want(dev, (kc, "k_codes", _U8, codes), (vc, "v_codes", _U8, codes), (kb, "k_blocks", _E4M3, blocks),
              (vb, "v_blocks", _E4M3, blocks))
    return _Cache4(kc.data_ptr(), vc.data_ptr(), kb.data_ptr(), vb.data_ptr(), float(kg), float(vg))


def _places_ok(i: int, cu, seq_lens, page_table, status, B: int, max_pages: int) -> bool:
    try:
        return (cu.dtype is _I32 and seq_lens.dtype is _I32 and page_table.dtype is _I32 and status.dtype is _I32
                and cu.shape == (B + 1,) and seq_lens.shape == (B,) and page_table.shape == (B, max_pages)
                and status.shape == (1,) and cu.get_device() == i and seq_lens.get_device() == i
                and page_table.get_device() == i and status.get_device() == i and cu.is_contiguous()
                and seq_lens.is_contiguous() and page_table.is_contiguous())
    except AttributeError:
        return False


def _token_rows(t, name, i: int, T: int, heads: int, D: int) -> int:
    """The stride from token to token of bf16 [T, heads, D], whose heads lie one after the other."""
    if isinstance(t, torch.Tensor) and t.dtype is _BF16 and t.get_device() == i and t.shape == (T, heads, D):
        s, h, e = t.stride()
        dense = heads * D
        if T < 2:  # (one row's stride says nothing)
            s = dense
        if e == 1 and (h == D or heads == 1) and s >= dense and not s & 7 or t.numel() == 0:
            return s if T > 1 else dense
        raise ValueError(f"{name}: strides {t.stride()}; a token's heads must lie one after the other, tokens a "
                         "multiple of 8 elements apart")
    what = f"{t.dtype} {tuple(t.shape)} on {t.device}" if isinstance(t, torch.Tensor) else type(t)
    raise ValueError(f"{name}: {what}, expected bfloat16 [{T}, {heads}, {D}] on cuda:{i}")


def _rope(rot, pairing, n_pos, q_stride, k_stride, v_stride) -> Rope:
    _fit(Rope, (rot, pairing, n_pos))
    return Rope(rot, pairing, n_pos, q_stride, k_stride, v_stride)


def _append_rope(fn, q_new, k_new, v_new, cos_sin, cu_new, seq_lens, page_table, pg: Paged, status, pairing, q_out,
                 k_out, dev, i, T, B, Hkv, D, cache):
    k_stride, v_stride = _token_rows(k_new, "k_new", i, T, Hkv, D), _token_rows(v_new, "v_new", i, T, Hkv, D)
    q_stride, q_at, q_to, k_to = 0, None, None, None
    if q_new is not None:
        Hq = pg.Hq
        q_stride = _token_rows(q_new, "q_new", i, T, Hq, D)
        if q_out is None:
            q_out = _empty((T, Hq, D), dtype=_BF16, device=dev)
        else:
            _want(dev, (q_out, "q_out", _BF16, (T, Hq, D)))
        q_at, q_to = q_new.data_ptr(), q_out.data_ptr()
    elif q_out is not None:
        raise ValueError("q_out without q_new")
    n_pos = rot = 0
    angles = None
    if cos_sin is not None:
        if not isinstance(cos_sin, torch.Tensor) or cos_sin.dim() != 2:
            raise ValueError("cos_sin must be [positions, rotated numbers]")
        n_pos, rot = cos_sin.shape
        if rot > D or rot % 16:
            raise ValueError(f"cos_sin: {rot} rotated numbers, a multiple of 16 up to {D} expected")
        if not (cos_sin.dtype is _F32 and cos_sin.get_device() == i and cos_sin.is_contiguous()):
            _want(dev, (cos_sin, "cos_sin", _F32, (n_pos, rot)))
        angles = cos_sin.data_ptr()
    if k_out is not None:
        _want(dev, (k_out, "k_out", _BF16, (T, Hkv, D)))
        k_to = k_out.data_ptr()
    if not _places_ok(i, cu_new, seq_lens, page_table, status, B, pg.max_pages):
        _want(dev, (cu_new, "cu_new", _I32, (B + 1,)), (seq_lens, "seq_lens", _I32, (B,)),
              (page_table, "page_table", _I32, (B, pg.max_pages)), (status, "status", _I32, (1,)))
    rc = fn(q_at, k_new.data_ptr(), v_new.data_ptr(), angles, _rope(rot, pairing, n_pos, q_stride, k_stride, v_stride),
            cu_new.data_ptr(), seq_lens.data_ptr(), page_table.data_ptr(), pg, T, q_to, k_to, *cache,
            status.data_ptr(), _current(dev))
    if rc:
        _check(rc, "bd_attn_paged4_append" if len(cache) == 1 else "bd_attn_paged_append_rope")
    return q_out


def bd_attn_paged_append_rope(q_new, k_new, v_new, cos_sin, cu_new, seq_lens, page_table, pg: Paged, k_pages, v_pages,
                              status, pairing: int = ROPE_HALVES, q_out=None, k_out=None, stream=None):
    """bd_attn_paged_append with queries and keys turned by their tokens' positions: row p of cos_sin, fp32
    [positions, rot], holds the cosines of rot / 2 pairs, then their sines (None: nothing turns). q_new [T, Hq, D]
    (or None), k_new, v_new [T, Hkv, D] may be parts of one projection's output. Returns the turned queries, and
    writes the turned keys to k_out [T, Hkv, D] as well where it is given; q_out may be q_new where that is dense."""
    if stream is None and _calls is not None:
        done = _calls.append_rope(q_new, k_new, v_new, cos_sin, cu_new, seq_lens, page_table, pg, (k_pages, v_pages),
                                  status, pairing, q_out, k_out)
        if done is not None:
            return done[0]
    dev = _cuda_device(k_pages, "k_pages")
    i = dev.index
    if (stream is not None or i != _device_now()) and (ctx := _elsewhere(dev, stream)) is not None:
        with ctx:
            return bd_attn_paged_append_rope(q_new, k_new, v_new, cos_sin, cu_new, seq_lens, page_table, pg, k_pages,
                                             v_pages, status, pairing, q_out, k_out)
    _cuda_device(k_new, "k_new")
    Hkv, D = pg.Hkv, pg.D
    pages = (pg.n_pages, Hkv, pg.page_size, D)
    _want(dev, (k_pages, "k_pages", _BF16, pages), (v_pages, "v_pages", _BF16, pages))
    return _append_rope((_lib or load()).bd_attn_paged_append_rope, q_new, k_new, v_new, cos_sin, cu_new, seq_lens,
                        page_table, pg, status, pairing, q_out, k_out, dev, i, k_new.shape[0] if k_new.dim() else 0,
                        pg.B, Hkv, D, (k_pages.data_ptr(), v_pages.data_ptr()))


def bd_attn_paged4_append(q_new, k_new, v_new, cos_sin, cu_new, seq_lens, page_table, pg: Paged, cache: Cache4,
                          status, pairing: int = ROPE_HALVES, q_out=None, k_out=None, stream=None):
    """bd_attn_paged_append_rope into a cache held in 4 bits."""
    if stream is None and _calls is not None:
        done = _calls.append4(q_new, k_new, v_new, cos_sin, cu_new, seq_lens, page_table, pg, cache, status, pairing,
                              q_out, k_out)
        if done is not None:
            return done[0]
    dev = _cuda_device(cache[0], "k_codes")
    i = dev.index
    if (stream is not None or i != _device_now()) and (ctx := _elsewhere(dev, stream)) is not None:
        with ctx:
            return bd_attn_paged4_append(q_new, k_new, v_new, cos_sin, cu_new, seq_lens, page_table, pg, cache,
                                         status, pairing, q_out, k_out)
    _cuda_device(k_new, "k_new")
    Hkv, D = pg.Hkv, pg.D
    c = _cache4(dev, i, cache, pg.n_pages, Hkv, pg.page_size, D)
    return _append_rope((_lib or load()).bd_attn_paged4_append, q_new, k_new, v_new, cos_sin, cu_new, seq_lens,
                        page_table, pg, status, pairing, q_out, k_out, dev, i, k_new.shape[0] if k_new.dim() else 0,
                        pg.B, Hkv, D, (c,))


def bd_attn_paged4_read(cache: Cache4, cu, seq_lens, page_table, pg: Paged, n_tokens: int, status, k_out=None,
                        v_out=None, stream=None):
    """The values of cached tokens as bf16 [n_tokens, Hkv, D]: of sequence b its last cu[b+1] - cu[b] tokens, at rows
    [cu[b], cu[b+1]). Returns (k_out, v_out)."""
    if stream is None and _calls is not None:
        done = _calls.read4(cache, cu, seq_lens, page_table, pg, n_tokens, status, k_out, v_out)
        if done is not None:
            return done
    dev = _cuda_device(cache[0], "k_codes")
    i = dev.index
    if (stream is not None or i != _device_now()) and (ctx := _elsewhere(dev, stream)) is not None:
        with ctx:
            return bd_attn_paged4_read(cache, cu, seq_lens, page_table, pg, n_tokens, status, k_out, v_out)
    T, B, Hkv, D = int(n_tokens), pg.B, pg.Hkv, pg.D
    c = _cache4(dev, i, cache, pg.n_pages, Hkv, pg.page_size, D)
    if not 0 <= T <= _INT_MAX:
        raise ValueError(f"n_tokens={n_tokens}")
    rows = (T, Hkv, D)
    if k_out is None:
        k_out = _empty(rows, dtype=_BF16, device=dev)
    else:
        _want(dev, (k_out, "k_out", _BF16, rows))
    if v_out is None:
        v_out = _empty(rows, dtype=_BF16, device=dev)
    else:
        _want(dev, (v_out, "v_out", _BF16, rows))
    if not _places_ok(i, cu, seq_lens, page_table, status, B, pg.max_pages):
        _want(dev, (cu, "cu", _I32, (B + 1,)), (seq_lens, "seq_lens", _I32, (B,)),
              (page_table, "page_table", _I32, (B, pg.max_pages)), (status, "status", _I32, (1,)))
    rc = (_lib or load()).bd_attn_paged4_read(c, cu.data_ptr(), seq_lens.data_ptr(), page_table.data_ptr(), pg, T,
                                              k_out.data_ptr(), v_out.data_ptr(), status.data_ptr(), _current(dev))
    if rc:
        _check(rc, "bd_attn_paged4_read")
    return k_out, v_out


def bd_attn_paged4_decode(q, cache: Cache4, page_table, seq_lens, pg: Paged, status, out=None, lse=None,
                          workspace=None, stream=None):
    """bd_attn_paged_decode over a cache held in 4 bits."""
    if stream is None and _calls is not None:
        done = _calls.decode4(q, cache, page_table, seq_lens, pg, status, out, lse, workspace)
        if done is not None:
            return done
    dev = _cuda_device(q, "q")
    i = dev.index
    if (stream is not None or i != _device_now()) and (ctx := _elsewhere(dev, stream)) is not None:
        with ctx:
            return bd_attn_paged4_decode(q, cache, page_table, seq_lens, pg, status, out, lse, workspace)
    lib = _lib or load()
    B, Hq, D, max_pages = pg.B, pg.Hq, pg.D, pg.max_pages
    rows = (B, Hq, D)
    n = lib.bd_attn_paged4_decode_workspace_bytes(pg)
    if n == 0:
        raise ValueError(f"invalid geometry {pg}")
    c = _cache4(dev, i, cache, pg.n_pages, pg.Hkv, pg.page_size, D)
    try:
        ok = (q.dtype is _BF16 and page_table.dtype is _I32 and seq_lens.dtype is _I32 and status.dtype is _I32
              and q.shape == rows and page_table.shape == (B, max_pages) and seq_lens.shape == (B,)
              and status.shape == (1,) and page_table.get_device() == i and seq_lens.get_device() == i
              and status.get_device() == i and q.is_contiguous() and page_table.is_contiguous()
              and seq_lens.is_contiguous())
    except AttributeError:
        ok = False
    if not ok:
        _want(dev, (q, "q", _BF16, rows), (page_table, "page_table", _I32, (B, max_pages)),
              (seq_lens, "seq_lens", _I32, (B,)), (status, "status", _I32, (1,)))
    if out is None:
        out = _empty(rows, dtype=_BF16, device=dev)
    else:
        _want(dev, (out, "out", _BF16, rows))
    if lse is None:
        lse = _empty((B, Hq), dtype=_F32, device=dev)
    else:
        _want(dev, (lse, "lse", _F32, (B, Hq)))
    at = None
    if workspace is not None:
        _want(dev, (workspace, "workspace", _U8, (n,)))
        at = workspace.data_ptr()
    elif n > 16:  # 16: the call needs none
        workspace = _empty(n, dtype=_U8, device=dev)
        at = workspace.data_ptr()
    rc = lib.bd_attn_paged4_decode(q.data_ptr(), c, page_table.data_ptr(), seq_lens.data_ptr(), pg, out.data_ptr(),
                                   lse.data_ptr(), at, status.data_ptr(), _current(dev))
    if rc:
        _check(rc, "bd_attn_paged4_decode")
    return out, lse


# ------------------------------------------------------------ exchange plans
def plan_bytes(B: int, cp_size: int, L: int) -> int:
    n = load().bd_attn_plan_bytes(int(B), int(cp_size), int(L))
    if n == 0:
        raise ValueError(f"invalid plan size B={B} cp_size={cp_size} L={L}")
    return int(n)


def plan_layout(B: int, cp_size: int, L: int) -> dict:
    arr = (ctypes.c_int32 * len(PLAN_REGIONS))()
    _check(load().bd_attn_plan_layout(int(B), int(cp_size), int(L), arr), "bd_attn_plan_layout")
    return {name: int(arr[i]) for i, name in enumerate(PLAN_REGIONS)}


def bd_attn_exchange_plan(doc_ids: torch.Tensor, cp_size: int, rank: int, plan: torch.Tensor | None = None,
                          status: torch.Tensor | None = None, stream=None):
    """Exchange plan of `rank` from the replicated doc ids [B, S] (device); returns (plan, status)."""
    dev = doc_ids.device
    B, S = doc_ids.shape
    _need(doc_ids, "doc_ids", torch.int32, (B, S), None)
    if S % cp_size:
        raise ValueError("the sequence must split into cp_size equal chunks")
    n = plan_bytes(B, cp_size, S // cp_size) // 4
    if plan is None:
        plan = torch.empty(n, dtype=torch.int32, device=dev)
    if status is None:
        status = new_status(dev)
    _need(plan, "plan", torch.int32, (n,), dev)
    _need(status, "status", torch.int32, (1,), dev)
    _check(load().bd_attn_exchange_plan(_ptr(doc_ids), int(B), int(S), int(cp_size), int(rank), _ptr(plan),
                                        _ptr(status), _stream(stream)), "bd_attn_exchange_plan")
    return plan, status


def _dtype_code(t: torch.Tensor) -> int:
    if t.dtype == torch.bfloat16:
        return BD_DTYPE_BF16
    if t.dtype == torch.float32:
        return BD_DTYPE_F32
    raise ValueError("bfloat16 or float32 expected")


def bd_attn_needed_gather(x_local: torch.Tensor, plan: torch.Tensor, send: torch.Tensor, status, stream=None):
    """send [max_rows, B, C, D] (token-major) from x_local [B, C, L, D] by the plan's send_index."""
    B, C, L, D = x_local.shape
    max_rows = send.shape[0]
    _need(x_local, "x_local", x_local.dtype, (B, C, L, D), None)
    _need(send, "send", x_local.dtype, (max_rows, B, C, D), x_local.device)
    _need(status, "status", torch.int32, (1,), x_local.device)
    _check(load().bd_attn_needed_gather(_ptr(x_local), _ptr(plan), B, C, L, D, _dtype_code(x_local), _ptr(send),
                                        int(max_rows), _ptr(status), _stream(stream)), "bd_attn_needed_gather")
    return send


def bd_attn_needed_scatter_add(grad_send: torch.Tensor, plan: torch.Tensor, grad_local: torch.Tensor, status,
                               stream=None):
    """grad_local [B, C, L, D] = the index-add of grad_send [max_rows, B, C, D] (token-major)."""
    B, C, L, D = grad_local.shape
    max_rows = grad_send.shape[0]
    _need(grad_local, "grad_local", grad_local.dtype, (B, C, L, D), None)
    _need(grad_send, "grad_send", grad_local.dtype, (max_rows, B, C, D), grad_local.device)
    _need(status, "status", torch.int32, (1,), grad_local.device)
    _check(load().bd_attn_needed_scatter_add(_ptr(grad_send), _ptr(plan), B, C, L, D, _dtype_code(grad_local),
                                             _ptr(grad_local), int(max_rows), _ptr(status), _stream(stream)),
           "bd_attn_needed_scatter_add")
    return grad_local


def read_plan(plan: torch.Tensor, B: int, cp_size: int, L: int) -> dict:
    """Copy a plan to the host and decode it (synchronises; tests and tools only)."""
    lay = plan_layout(B, cp_size, L)
    a = plan.cpu().numpy()
    W = cp_size
    h = a[lay["hdr"]: lay["hdr"] + PLAN_HDR_WORDS]
    d = {name: int(h[i]) for i, name in enumerate(PLAN_HDR_FIELDS)}
    for name in ("s_first", "real_end", "back", "halo_send", "in_splits", "out_splits", "send_off", "recv_off"):
        d[name] = [int(x) for x in a[lay[name]: lay[name] + W]]
    d["counts"] = [[int(x) for x in a[lay["counts"] + s * W: lay["counts"] + (s + 1) * W]] for s in range(W)]
    d["send_index"] = [int(x) for x in a[lay["send_index"]: lay["send_index"] + max(0, d["total_send"])]]
    return d
