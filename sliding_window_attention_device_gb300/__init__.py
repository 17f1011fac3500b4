"""Per-document causal (block-diagonal) attention for one context-parallel shard, GB300-native.

The compute lives in ``libbdattn.so`` (hand-written CUDA for sm_103a behind a C
ABI, declared in ``include/bdattn.h``); :mod:`.bdattn` is its thin ctypes
binding and :mod:`.synth` draws seeded synthetic inputs.
"""
from importlib import import_module

_ENTRIES = ("bd_attn_seg_build", "bd_attn_fwd", "bd_attn_bwd", "bd_attn_sink_seg_build", "bd_attn_sink_fwd",
            "bd_attn_sink_bwd", "bd_attn_paged_append", "bd_attn_paged_decode")
__all__ = ["bdattn", "synth", *_ENTRIES]


def __getattr__(name):
    if name in ("bdattn", "synth"):
        return import_module(f"{__name__}.{name}")
    if name in _ENTRIES:
        return getattr(import_module(f"{__name__}.bdattn"), name)
    raise AttributeError(name)
