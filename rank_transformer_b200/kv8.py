"""Owner of one layer's 8-bit key/value cache (include/flashsvd.h, "8-bit
key/value cache"): the tensors, and the flashsvd_kv8 struct that points at
them.  All work on it is done by the library (flashsvd.kv8_store,
kv8_decode_attn, kv8_evict, layer_forward_kv8).
"""
from __future__ import annotations

import torch

from . import flashsvd as fs

FORMATS = {"int8": fs.KV8_INT8, "e4m3": fs.KV8_E4M3}
_CODES = {"int8": torch.int8, "e4m3": torch.float8_e4m3fn}


class KV8Cache:
    """k, v [B, H_kv, S_max, D] codes (torch.int8 or torch.float8_e4m3fn),
    k_scale, v_scale [B, H_kv, S_max / 64] float32 and k_tail, v_tail
    [B, H_kv, 64, D] bfloat16, all contiguous on one device."""

    def __init__(self, B: int, H_kv: int, D: int, S_max: int, fmt: str = "int8", device="cuda"):
        if fmt not in FORMATS:
            raise ValueError(f"fmt is one of {sorted(FORMATS)}, not {fmt!r}")
        if S_max <= 0 or S_max % fs.KV8_BLOCK:
            raise ValueError(f"S_max is a multiple of {fs.KV8_BLOCK}, not {S_max}")
        codes = lambda: torch.zeros((B, H_kv, S_max, D), dtype=torch.int8,  # noqa: E731
                                    device=device).view(_CODES[fmt])
        scale = lambda: torch.zeros((B, H_kv, S_max // fs.KV8_BLOCK), device=device)  # noqa: E731
        tail = lambda: torch.zeros((B, H_kv, fs.KV8_BLOCK, D), dtype=torch.bfloat16,  # noqa: E731
                                   device=device)
        self._hold(codes(), codes(), scale(), scale(), tail(), tail())

    @classmethod
    def from_tensors(cls, k, v, k_scale, v_scale, k_tail, v_tail) -> "KV8Cache":
        self = cls.__new__(cls)
        self._hold(k, v, k_scale, v_scale, k_tail, v_tail)
        return self

    def _hold(self, k, v, k_scale, v_scale, k_tail, v_tail):
        fmt = {d: n for n, d in _CODES.items()}.get(k.dtype)
        if fmt is None:
            raise ValueError(f"codes are int8 or float8_e4m3fn, not {k.dtype}")
        B, G, S, D = k.shape
        for name, t, shape, dtype in (
                ("k", k, (B, G, S, D), k.dtype), ("v", v, (B, G, S, D), k.dtype),
                ("k_scale", k_scale, (B, G, S // fs.KV8_BLOCK), torch.float32),
                ("v_scale", v_scale, (B, G, S // fs.KV8_BLOCK), torch.float32),
                ("k_tail", k_tail, (B, G, fs.KV8_BLOCK, D), torch.bfloat16),
                ("v_tail", v_tail, (B, G, fs.KV8_BLOCK, D), torch.bfloat16)):
            if tuple(t.shape) != shape or t.dtype != dtype or not t.is_contiguous() \
                    or t.device != k.device:
                raise ValueError(f"{name}: contiguous {dtype} {shape} on {k.device} wanted, got "
                                 f"{t.dtype} {tuple(t.shape)} on {t.device}")
        self.fmt, self.B, self.H_kv, self.S_max, self.D = fmt, B, G, S, D
        self.k, self.v = k, v
        self.k_scale, self.v_scale = k_scale, v_scale
        self.k_tail, self.v_tail = k_tail, v_tail
        self.struct = fs.Kv8(FORMATS[fmt], B, G, D, S, *(fs.ptr(t) for t in (
            k, v, k_scale, v_scale, k_tail, v_tail)))

    def tensors(self):
        return (self.k, self.v, self.k_scale, self.v_scale, self.k_tail, self.v_tail)

    def bytes(self) -> int:
        return sum(t.numel() * t.element_size() for t in self.tensors())
