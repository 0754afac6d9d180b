"""The operators around the target model's forward pass: cache tables, rotary
positions with the cache write, shared-prefix attention and logit adjustments.

Like the rest of the binding these functions only marshal arguments; layouts,
rules and status bits are in ``include/spec.h``.  Tensors that a call makes for
itself belong to the stream it runs on.  Tensors and streams have to be of the
current device, where the kernels are launched.
"""
from __future__ import annotations

import contextlib
import ctypes
import math
import struct
from typing import Optional

import torch

from . import SPEC_BF16, SPEC_F32, _check, _dev, _dtype_code, _P, lib

_I, _L, _F = ctypes.c_int, ctypes.c_int64, ctypes.c_float


class CacheReserveArgs(ctypes.Structure):
    _fields_ = [("R", _I), ("rows", _I), ("page_size", _I), ("n_pages", _I), ("max_pages", _I),
                ("kv_len", _P), ("row_off", _P), ("pos_base", _P), ("block_table", _P), ("ring", _P),
                ("ring_pos", _P), ("ring_out", _P), ("new_len", _P), ("position", _P),
                ("request", _P), ("slot", _P), ("status", _P)]


class CacheCommitArgs(ctypes.Structure):
    _fields_ = [("R", _I), ("page_size", _I), ("n_pages", _I), ("max_pages", _I), ("kv_len", _P),
                ("new_len", _P), ("keep", _P), ("block_table", _P), ("ring", _P), ("ring_pos", _P),
                ("ring_out", _P), ("kv_out", _P), ("status", _P)]


class RopeCacheArgs(ctypes.Structure):
    _fields_ = [("rows", _I), ("Hq", _I), ("Hk", _I), ("D", _I), ("rot", _I), ("dtype", _I),
                ("layout", _I), ("scale", _F), ("q", _P), ("k", _P), ("v", _P), ("q_row", _L),
                ("q_head", _L), ("k_row", _L), ("k_head", _L), ("v_row", _L), ("v_head", _L),
                ("q_out", _P), ("q_out_row", _L), ("q_out_head", _L), ("k_cache", _P),
                ("v_cache", _P), ("n_slots", _L), ("freq", _P), ("position", _P), ("slot", _P),
                ("status", _P)]


class PrefixAttentionArgs(ctypes.Structure):
    _fields_ = [("R", _I), ("rows", _I), ("Hq", _I), ("Hk", _I), ("D", _I), ("dtype", _I),
                ("page_size", _I), ("n_pages", _I), ("max_pages", _I), ("G", _I),
                ("max_prefix_pages", _I), ("scale", _F), ("q", _P), ("q_row", _L), ("q_head", _L),
                ("k_cache", _P), ("v_cache", _P), ("row_off", _P), ("kv_len", _P),
                ("block_table", _P), ("group_off", _P), ("prefix_len", _P), ("prefix_table", _P),
                ("out", _P), ("out_row", _L), ("out_head", _L), ("lse", _P), ("workspace", _P),
                ("workspace_bytes", ctypes.c_size_t), ("status", _P)]


class NormRopeArgs(ctypes.Structure):
    _fields_ = [("rows", _I), ("Hq", _I), ("Hk", _I), ("D", _I), ("rot", _I), ("dtype", _I),
                ("layout", _I), ("cache", _I), ("page_size", _I), ("scale", _F), ("eps", _F), ("q", _P), ("k", _P), ("v", _P),
                ("q_row", _L), ("q_head", _L), ("k_row", _L), ("k_head", _L), ("v_row", _L), ("v_head", _L),
                ("q_out", _P), ("q_out_row", _L), ("q_out_head", _L), ("k_cache", _P),
                ("v_cache", _P), ("k_scale", _P), ("v_scale", _P), ("n_slots", _L), ("q_weight", _P), ("k_weight", _P),
                ("freq", _P), ("position", _P), ("slot", _P), ("status", _P)]


class CacheReadPackedArgs(ctypes.Structure):
    _fields_ = [("rows", _I), ("Hk", _I), ("D", _I), ("page_size", _I), ("dtype", _I), ("k_cache", _P), ("v_cache", _P),
                ("k_scale", _P), ("v_scale", _P), ("n_slots", _L), ("slot", _P), ("k", _P), ("v", _P), ("status", _P)]


class PrefixAttentionPackedArgs(ctypes.Structure):
    """spec_prefix_attention_packed_args with the fields of its first member in its place."""
    _fields_ = PrefixAttentionArgs._fields_ + [("k_scale", _P), ("v_scale", _P)]


class LogitsArgs(ctypes.Structure):
    _fields_ = [("R", _I), ("V", _I), ("rows", _I), ("rows_per_request", _I), ("dtype", _I),
                ("logits", _P), ("ld", _L), ("out", _P), ("out_ld", _L), ("row_off", _P),
                ("tokens", _P), ("tokens_ld", _L), ("prompt_len", _P), ("length", _P), ("x", _P),
                ("x_ld", _L), ("tokens_cols", _I), ("x_cols", _I), ("n_bias", _I), ("repetition", _P), ("frequency", _P),
                ("presence", _P), ("bias_off", _P), ("bias_tok", _P), ("bias_val", _P),
                ("mask", _P), ("mask_ld", _L), ("mask_row", _P), ("n_masks", _I), ("status", _P)]


class _Call:
    """An entry point whose argument struct is packed straight into bytes: these calls run once a
    layer, and filling a ctypes structure field by field took longer than the small kernels do."""

    def __init__(self, name: str, cls):
        self.name, self.cls, self.f = name, cls, None
        codes = {_I: "i", _F: "f", _L: "q", _P: "Q", ctypes.c_size_t: "Q"}
        fmt, at = "=", 0
        for field, kind in cls._fields_:
            gap = getattr(cls, field).offset - at
            fmt += (f"{gap}x" if gap else "") + codes[kind]
            at += gap + ctypes.sizeof(kind)
        self.pack = struct.Struct(fmt + f"{ctypes.sizeof(cls) - at}x").pack

    def bind(self, L: ctypes.CDLL) -> None:
        f = getattr(L, self.name)
        f.argtypes, f.restype = [ctypes.POINTER(self.cls), _P], ctypes.c_int
        self.f = L[self.name]  # another handle of the same function
        self.f.argtypes, self.f.restype = [ctypes.c_char_p, _P], ctypes.c_int

    def __call__(self, stream: int, *values) -> None:
        if self.f is None:
            lib()
        rc = self.f(self.pack(*values), stream)
        if rc:
            _check(rc, self.name)


_RESERVE = _Call("spec_cache_reserve", CacheReserveArgs)
_COMMIT = _Call("spec_cache_commit", CacheCommitArgs)
_ROPE = _Call("spec_rope_cache", RopeCacheArgs)
_ATTENTION = _Call("spec_prefix_attention", PrefixAttentionArgs)
_LOGITS = _Call("spec_adjust_logits", LogitsArgs)
_NORM_ROPE = _Call("spec_norm_rope_cache", NormRopeArgs)
_READ_PACKED = _Call("spec_cache_read_packed", CacheReadPackedArgs)
_ATTENTION_PACKED = _Call("spec_prefix_attention_packed", PrefixAttentionPackedArgs)


def _bind(L: ctypes.CDLL) -> None:
    """Prototypes of this module's entry points (called once by ``lib``)."""
    for call in (_RESERVE, _COMMIT, _ROPE, _ATTENTION, _LOGITS, _NORM_ROPE, _READ_PACKED, _ATTENTION_PACKED):
        call.bind(L)
    for f in (L.spec_attention_workspace_bytes, L.spec_attention_packed_workspace_bytes):
        f.argtypes, f.restype = [_I] * 4, ctypes.c_size_t


_i32, _i64, _f32, _f64, _u8 = torch.int32, torch.int64, torch.float32, torch.float64, torch.uint8
_Tensor = torch.Tensor
_codes = {torch.float32: SPEC_F32, torch.bfloat16: SPEC_BF16}


def _device() -> int:
    """The current device, which every launch goes to."""
    return torch._C._cuda_getDevice()


def _here(t: torch.Tensor, name: str) -> None:
    """Raise unless t is a tensor of the current device."""
    if not isinstance(t, _Tensor) or not t.is_cuda:
        raise TypeError(f"{name} must be a CUDA tensor")
    if t.get_device() != _device():
        raise ValueError(f"{name} must lie on the current device")


def _t(t: torch.Tensor, name: str, dtype: torch.dtype, numel: int = 0, dev: Optional[int] = None) -> int:
    """Address of a contiguous tensor of the current device (``dev``, where the caller has asked for it), of this dtype
    (and at least numel entries)."""
    # (a host tensor's device is -1)
    if isinstance(t, _Tensor) and t.get_device() == (_device() if dev is None else dev) and t.dtype is dtype and t.is_contiguous():
        if not numel or t.numel() >= numel:
            return t.data_ptr()
    _here(t, name)
    _dev(t, name)
    if t.dtype is not dtype:
        raise TypeError(f"{name} must be {dtype}")
    raise ValueError(f"{name} must have {numel} entries")


def _opt(t: Optional[torch.Tensor], name: str, dtype: torch.dtype, numel: int = 0, dev: Optional[int] = None) -> int:
    return 0 if t is None else _t(t, name, dtype, numel, dev)


def _code(t: torch.Tensor) -> int:
    return _codes[t.dtype] if t.dtype in _codes else _dtype_code(t)


def _on(stream, t: torch.Tensor) -> int:
    """Handle of the stream to launch on: the given one, or the current one of t's device, which the check
    of t makes the current device."""
    if stream is not None:
        if stream.device.index != _device():
            raise ValueError("stream must be one of the current device")
        return stream.cuda_stream
    return torch._C._cuda_getCurrentRawStream(t.get_device())


_HERE = contextlib.nullcontext()


def _made(stream):
    """The call's own tensors are memory of the stream it runs on."""
    return _HERE if stream is None else torch.cuda.stream(stream)


# ------------------------------------------------------------- cache tables --
def cache_tables(R: int, n_pages: int, page_size: int, max_pages: int, device="cuda") -> dict:
    """An empty cache's bookkeeping: lengths 0, every page free.  Keys: "kv_len" [R],
    "block_table" [R, max_pages], "ring" [n_pages] int32, "ring_pos" [2] int64 and "page_size"."""
    return {"kv_len": torch.zeros(R, dtype=torch.int32, device=device),
            "block_table": torch.full((R, max_pages), -1, dtype=torch.int32, device=device),
            "ring": torch.arange(n_pages, dtype=torch.int32, device=device),
            "ring_pos": torch.tensor([0, n_pages], dtype=torch.int64, device=device),
            "page_size": page_size}


def cache_reserve(cache: dict, row_off: torch.Tensor, rows: int, *,
                  pos_base: Optional[torch.Tensor] = None, out: Optional[dict] = None,
                  status: Optional[torch.Tensor] = None, stream=None) -> dict:
    """spec_cache_reserve: pages, positions and slots for row_off[R] new tokens.

    ``cache`` is the dict of ``cache_tables``; its "block_table" gets the new pages.  ``rows`` is
    the capacity of the row arrays (row_off[R] at least; the rest is -1).  Returns {"new_len" [R],
    "position", "request", "slot" [rows] int32, "ring_pos" [2] int64}, which ``cache_commit`` takes."""
    table, ring = cache["block_table"], cache["ring"]
    R, width = table.shape
    if out is None:  # (tensors of their own: views of one cost twice as much to make)
        dev = table.device
        with _made(stream):
            new = torch.empty(R, dtype=_i32, device=dev)
            position = torch.empty(rows, dtype=_i32, device=dev)
            request = torch.empty(rows, dtype=_i32, device=dev)
            slot = torch.empty(rows, dtype=_i32, device=dev)
            pos = torch.empty(2, dtype=_i64, device=dev)
        out = {"new_len": new, "position": position, "request": request, "slot": slot, "ring_pos": pos}
        made = pos.data_ptr(), new.data_ptr(), position.data_ptr(), request.data_ptr(), slot.data_ptr()
    else:
        made = (_t(out["ring_pos"], "out ring_pos", _i64, 2), _t(out["new_len"], "new_len", _i32, R),
                _t(out["position"], "position", _i32, rows), _t(out["request"], "request", _i32, rows),
                _t(out["slot"], "slot", _i32, rows))
    _RESERVE(_on(stream, table), R, rows, cache["page_size"], ring.numel(), width,
             _t(cache["kv_len"], "kv_len", _i32, R), _t(row_off, "row_off", _i32, R + 1),
             _opt(pos_base, "pos_base", _i32, R), _t(table, "block_table", _i32), _t(ring, "ring", _i32),
             _t(cache["ring_pos"], "ring_pos", _i64, 2), *made, _opt(status, "status", _i32, 1))
    return out


def cache_commit(cache: dict, reserved: dict, keep: torch.Tensor, *, out: Optional[dict] = None,
                 status: Optional[torch.Tensor] = None, stream=None) -> dict:
    """spec_cache_commit: keep the first keep[r] new tokens of each request (verify's n_out; a
    negative entry ends the request) and give the other pages back to cache["ring"].

    Returns {"kv_len" [R], "ring_pos" [2]}; ``cache.update(...)`` with it makes it the next
    round's state (both rounds' dicts can serve in turn as ``out``)."""
    table, ring = cache["block_table"], cache["ring"]
    R, width = table.shape
    if out is None:
        with _made(stream):
            kv = torch.empty(R, dtype=_i32, device=table.device)
            pos = torch.empty(2, dtype=_i64, device=table.device)
        out = {"kv_len": kv, "ring_pos": pos}
        made = pos.data_ptr(), kv.data_ptr()
    else:
        made = _t(out["ring_pos"], "out ring_pos", _i64, 2), _t(out["kv_len"], "out kv_len", _i32, R)
    _COMMIT(_on(stream, table), R, cache["page_size"], ring.numel(), width,
            _t(cache["kv_len"], "kv_len", _i32, R), _t(reserved["new_len"], "new_len", _i32, R),
            _t(keep, "keep", _i32, R), _t(table, "block_table", _i32), _t(ring, "ring", _i32),
            _t(reserved["ring_pos"], "ring_pos", _i64, 2), *made, _opt(status, "status", _i32, 1))
    return out


# --------------------------------------------------------- rotary positions --
def rope_frequencies(rot: int, base: float = 10000.0, *, scaling: str = "none", factor: float = 1.0,
                     trained: int = 0, low: float = 1.0, high: float = 32.0, device="cuda"):
    """Frequencies [rot / 2] float64 (radians per position) and the attention factor for ``rope_cache``.

    f_i = base^(-2 i / rot), then for contexts ``factor`` times as long as the trained ones:
      "none"    as they are
      "linear"  f_i / factor (positions interpolated)
      "base"    base * factor^(rot / (rot - 2)): the highest frequency kept, the lowest divided by factor
      "ramp"    f_i where a head turns more than ``high`` times over ``trained`` positions, f_i / factor
                where it turns less than ``low`` times, linear in the turns' pair index between; attention
                factor 0.1 ln(factor) + 1
      "band"    the same two ends, linear in the number of turns between; attention factor 1
    """
    if rot < 2 or rot % 2:
        raise ValueError("rot must be even and positive")
    if not factor >= 1.0 or (scaling in ("ramp", "band") and (trained < 1 or not 0 < low < high)):
        raise ValueError("factor must be 1 or more; ramp and band need trained > 0 and 0 < low < high")
    i = torch.arange(0, rot, 2, dtype=torch.float64)
    if scaling == "base":
        if rot < 4:
            raise ValueError("base scaling needs rot >= 4")
        base = base * factor ** (rot / (rot - 2))
    f = base ** (-i / rot)
    scale = 1.0
    if scaling == "linear":
        f = f / factor
    elif scaling in ("ramp", "band"):
        if scaling == "band":
            share = (trained * f / (2 * math.pi) - low) / (high - low)
        else:
            at = [rot * math.log(trained / (2 * math.pi * t)) / (2 * math.log(base)) for t in (high, low)]
            first, last = max(0, math.floor(at[0])), min(rot - 1, math.ceil(at[1]))
            share = 1 - (i / 2 - first) / max(last - first, 1e-3)
            scale = 0.1 * math.log(factor) + 1.0
        share = share.clamp(0, 1)
        f = f * share + f / factor * (1 - share)
    elif scaling not in ("none", "base"):
        raise ValueError(f"unknown scaling {scaling!r}")
    return f.to(device), scale


def _strided(t: torch.Tensor, name: str, dtype: torch.dtype, shape: tuple, dev: Optional[int] = None) -> tuple:
    """Address and the row and head strides of [rows, heads, D] whose last dimension is dense."""
    if not isinstance(t, _Tensor) or t.get_device() != (_device() if dev is None else dev):
        _here(t, name)
    if t.dtype is not dtype:
        raise TypeError(f"{name} must be {dtype}")
    if t.shape != shape:
        raise ValueError(f"{name} must be {list(shape)}")
    row, head, one = t.stride()
    if one != 1 and shape[2] > 1:
        raise ValueError(f"{name}'s last dimension must be dense")
    return t.data_ptr(), row, head


def rope_cache(q: torch.Tensor, k: Optional[torch.Tensor], v: Optional[torch.Tensor],
               freq: torch.Tensor, position: torch.Tensor, slot: Optional[torch.Tensor],
               k_cache: Optional[torch.Tensor], v_cache: Optional[torch.Tensor], *,
               interleaved: bool = False, scale: float = 1.0, q_out: Optional[torch.Tensor] = None,
               status: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """spec_rope_cache: turn q [rows, Hq, D] and k [rows, Hk, D] by their positions, write k and v
    to their slots of the caches [pages, page_size, Hk, D]; returns the turned queries (``q_out``,
    which may be ``q`` itself).  2 * freq.numel() elements of each head turn.  q, k and v may be
    parts of one wider tensor; with k None only the queries turn."""
    rows, Hq, D = shape = q.shape
    dt = q.dtype
    qp, qr, qh = _strided(q, "q", dt, shape)
    if q_out is None:
        with _made(stream):
            q_out = torch.empty(shape, dtype=dt, device=q.device)
        op, orow, oh = q_out.data_ptr(), Hq * D, D
    else:
        op, orow, oh = _strided(q_out, "q_out", dt, shape)
    if k is None:
        Hk = n_slots = sp = kc = vc = kp = vp = kr = kh = vr = vh = 0
    else:
        Hk = k.shape[1]
        kp, kr, kh = _strided(k, "k", dt, (rows, Hk, D))
        vp, vr, vh = _strided(v, "v", dt, (rows, Hk, D))
        if k_cache.dim() != 4 or k_cache.shape[2:] != (Hk, D) or v_cache.shape != k_cache.shape:
            raise ValueError("k_cache and v_cache must both be [pages, page_size, Hk, D]")
        kc, vc = _t(k_cache, "k_cache", dt), _t(v_cache, "v_cache", dt)
        n_slots, sp = k_cache.shape[0] * k_cache.shape[1], _t(slot, "slot", _i32, rows)
    _ROPE(_on(stream, q), rows, Hq, Hk, D, 2 * freq.numel(), _code(q), int(interleaved), scale, qp, kp, vp,
          qr, qh, kr, kh, vr, vh, op, orow, oh, kc, vc, n_slots, _t(freq, "freq", _f64),
          _t(position, "position", _i32, rows), sp, _opt(status, "status", _i32, 1))
    return q_out


# ------------------------------------------- head norms, caches in 4 bits --
def packed_cache(n_pages: int, page_size: int, Hk: int, D: int, device="cuda") -> tuple:
    """An empty cache in 4 bits for keys or values: data [n_pages, Hk, D / 32, page_size, 16] and scales
    [n_pages, Hk, page_size, D / 32], both uint8, D a multiple of 32 (zeros stand for -8 * 2^-20)."""
    if D < 1 or D % 32:
        raise ValueError("D must be a multiple of 32")
    return (torch.zeros(n_pages, Hk, D // 32, page_size, 16, dtype=_u8, device=device),
            torch.zeros(n_pages, Hk, page_size, D // 32, dtype=_u8, device=device))


def _packed(cache: tuple, name: str, Hk: Optional[int], D: int, dev: int) -> tuple:
    """Addresses of a packed cache's data and scales, and its pages, page size and key heads."""
    data, scale = cache
    if not isinstance(data, _Tensor) or not isinstance(scale, _Tensor):
        raise TypeError(f"{name} must be a pair of tensors")
    shape = data.shape
    if len(shape) == 5:
        n, heads, groups, P, width = shape
        if groups * 32 == D and width == 16 and (Hk is None or heads == Hk) and scale.shape == (n, heads, P, groups):
            return _t(data, name, _u8, 0, dev), _t(scale, f"{name} scales", _u8, 0, dev), n, P, heads
    raise ValueError(f"{name} must be the data [pages, Hk, D / 32, page_size, 16] and scales [pages, Hk, page_size, D / 32]")


def norm_rope_cache(q: torch.Tensor, k: Optional[torch.Tensor], v: Optional[torch.Tensor],
                    freq: torch.Tensor, position: torch.Tensor, slot: Optional[torch.Tensor], k_cache, v_cache, *,
                    q_weight: Optional[torch.Tensor] = None, k_weight: Optional[torch.Tensor] = None, eps: float = 1e-6,
                    interleaved: bool = False, scale: float = 1.0, q_out: Optional[torch.Tensor] = None,
                    status: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """spec_norm_rope_cache: ``rope_cache`` after a norm of each head of queries and keys (divided by its root mean
    square, times ``q_weight`` and ``k_weight`` [D] float32; None: no norm).  The caches are tensors [pages, page_size,
    Hk, D] as there, or both pairs of ``packed_cache``: then keys and values are stored in 4 bits."""
    rows, Hq, D = shape = q.shape
    dt, dev = q.dtype, _device()
    qp, qr, qh = _strided(q, "q", dt, shape, dev)
    if q_out is None:
        with _made(stream):
            q_out = torch.empty(shape, dtype=dt, device=q.device)
        op, orow, oh = q_out.data_ptr(), Hq * D, D
    else:
        op, orow, oh = _strided(q_out, "q_out", dt, shape, dev)
    Hk = P = n_slots = sp = kc = vc = ks = vs = kp = vp = kr = kh = vr = vh = kind = 0
    if k is not None:
        Hk = k.shape[1]
        kp, kr, kh = _strided(k, "k", dt, (rows, Hk, D), dev)
        vp, vr, vh = _strided(v, "v", dt, (rows, Hk, D), dev)
        if not isinstance(k_cache, (tuple, _Tensor)) or not isinstance(v_cache, (tuple, _Tensor)):
            raise TypeError("k_cache and v_cache must be tensors or pairs of packed_cache")
        if isinstance(k_cache, tuple) != isinstance(v_cache, tuple):
            raise ValueError("k_cache and v_cache must be of one kind")
        if isinstance(k_cache, tuple):
            kind = 1
            kc, ks, n, P, _ = _packed(k_cache, "k_cache", Hk, D, dev)
            vc, vs, n2, P2, _ = _packed(v_cache, "v_cache", Hk, D, dev)
            if (n, P) != (n2, P2):
                raise ValueError("k_cache and v_cache must have the same pages")
            n_slots = n * P
        else:
            if k_cache.dim() != 4 or k_cache.shape[2:] != (Hk, D) or v_cache.shape != k_cache.shape:
                raise ValueError("k_cache and v_cache must both be [pages, page_size, Hk, D]")
            kc, vc = _t(k_cache, "k_cache", dt, 0, dev), _t(v_cache, "v_cache", dt, 0, dev)
            n_slots = k_cache.shape[0] * k_cache.shape[1]
        sp = _t(slot, "slot", _i32, rows, dev)
    _NORM_ROPE(_on(stream, q), rows, Hq, Hk, D, 2 * freq.numel(), _code(q), int(interleaved), kind, P, scale, eps,
               qp, kp, vp, qr, qh, kr, kh, vr, vh, op, orow, oh, kc, vc, ks, vs, n_slots,
               _opt(q_weight, "q_weight", _f32, D, dev), _opt(k_weight, "k_weight", _f32, D, dev), _t(freq, "freq", _f64, 0, dev),
               _t(position, "position", _i32, rows, dev), sp, _opt(status, "status", _i32, 1, dev))
    return q_out


def cache_read_packed(k_cache: tuple, v_cache: tuple, slot: torch.Tensor, *, dtype: torch.dtype = torch.bfloat16,
                    out: Optional[tuple] = None, status: Optional[torch.Tensor] = None, stream=None) -> tuple:
    """spec_cache_read_packed: what the slots of two ``packed_cache`` pairs stand for, (k, v) [rows, Hk, D] of ``dtype``
    (exact in bfloat16 and float32), zeros where a slot is negative or past the cache."""
    rows, dev = slot.numel(), _device()
    D = k_cache[0].shape[2] * 32 if isinstance(k_cache[0], _Tensor) and k_cache[0].dim() == 5 else 0
    kc, ks, n, P, Hk = _packed(k_cache, "k_cache", None, D, dev)
    vc, vs, n2, P2, _ = _packed(v_cache, "v_cache", Hk, D, dev)
    if (n, P) != (n2, P2):
        raise ValueError("k_cache and v_cache must have the same pages")
    at = _t(slot, "slot", _i32, 0, dev)
    if out is None:
        if dtype not in _codes:
            raise TypeError("dtype must be float32 or bfloat16")
        with _made(stream):
            k = torch.empty((rows, Hk, D), dtype=dtype, device=slot.device)
            v = torch.empty((rows, Hk, D), dtype=dtype, device=slot.device)
        kp, vp = k.data_ptr(), v.data_ptr()
    else:
        k, v = out
        if k.dtype is not v.dtype or k.shape != (rows, Hk, D) or v.shape != k.shape:
            raise ValueError("out must be two tensors [rows, Hk, D] of one dtype")
        kp, vp = _t(k, "out k", k.dtype, 0, dev), _t(v, "out v", v.dtype, 0, dev)
    _READ_PACKED(_on(stream, slot), rows, Hk, D, P, _code(k), kc, vc, ks, vs, n * P, at, kp, vp, _opt(status, "status", _i32, 1, dev))
    return k, v


# -------------------------------------------------- shared-prefix attention --
def attention_workspace_bytes(rows: int, R: int, Hq: int, D: int) -> int:
    """spec_attention_workspace_bytes: workspace of ``prefix_attention``."""
    return int(lib().spec_attention_workspace_bytes(rows, R, Hq, D))


def attention_packed_workspace_bytes(rows: int, R: int, Hq: int, D: int) -> int:
    """spec_attention_packed_workspace_bytes: workspace of ``prefix_attention_packed``."""
    return int(lib().spec_attention_packed_workspace_bytes(rows, R, Hq, D))


def _prefixes(group_off, prefix_len, prefix_table) -> tuple:
    """Groups, pages of a prefix table and the addresses of an attention call's prefixes."""
    if prefix_len is None or prefix_len.numel() == 0:
        return 0, 0, 0, 0, 0
    G = prefix_len.numel()
    if group_off is None or prefix_table is None or prefix_table.dim() != 2 or prefix_table.shape[0] != G:
        raise ValueError("prefixes need group_off [G + 1], prefix_len [G] and prefix_table [G, pages]")
    return (G, prefix_table.shape[1], _t(group_off, "group_off", _i32, G + 1), _t(prefix_len, "prefix_len", _i32),
            _t(prefix_table, "prefix_table", _i32))


def prefix_attention(q: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor,
                     row_off: torch.Tensor, kv_len: torch.Tensor, block_table: torch.Tensor, *,
                     scale: Optional[float] = None, group_off: Optional[torch.Tensor] = None,
                     prefix_len: Optional[torch.Tensor] = None,
                     prefix_table: Optional[torch.Tensor] = None, want_lse: bool = False,
                     out: Optional[torch.Tensor] = None, lse: Optional[torch.Tensor] = None,
                     workspace: Optional[torch.Tensor] = None,
                     status: Optional[torch.Tensor] = None, stream=None):
    """spec_prefix_attention: attention of the packed rows q [rows, Hq, D] over a paged cache
    [pages, page_size, Hk, D]: each request's own ``kv_len`` keys in its ``block_table`` pages
    (causal over its rows) and, for requests ``group_off[g]`` .. ``group_off[g + 1]``, the
    ``prefix_len[g]`` keys in ``prefix_table[g]``.  ``scale`` defaults to D^-1/2.  Returns out
    [rows, Hq, D], or (out, lse [rows, Hq]) with ``want_lse``."""
    rows, Hq, D = shape = q.shape
    dt = q.dtype
    if k_cache.dim() != 4 or k_cache.shape[3] != D or v_cache.shape != k_cache.shape:
        raise ValueError("k_cache and v_cache must both be [pages, page_size, Hk, D]")
    n_pages, P, Hk, _ = k_cache.shape
    R, width = block_table.shape
    G, pages, go, pl, pt = _prefixes(group_off, prefix_len, prefix_table)
    strides = _strided(q, "q", dt, shape)
    dev = q.device

    if workspace is not None:
        _here(workspace, "workspace")
    with _made(stream):
        made = out is None
        if made:
            out = torch.empty(shape, dtype=dt, device=dev)
        if want_lse and lse is None:
            lse = torch.empty((rows, Hq), dtype=_f32, device=dev)
        if workspace is None:
            workspace = torch.empty(attention_workspace_bytes(rows, R, Hq, D), dtype=torch.uint8, device=dev)
    _ATTENTION(_on(stream, q), R, rows, Hq, Hk, D, _code(q), P, n_pages, width, G, pages,
               D ** -0.5 if scale is None else scale, *strides, _t(k_cache, "k_cache", dt),
               _t(v_cache, "v_cache", dt), _t(row_off, "row_off", _i32, R + 1), _t(kv_len, "kv_len", _i32, R),
               _t(block_table, "block_table", _i32), go, pl, pt,
               *((out.data_ptr(), Hq * D, D) if made else _strided(out, "out", dt, shape)),
               _opt(lse, "lse", _f32, rows * Hq), _dev(workspace, "workspace").data_ptr(),
               workspace.numel() * workspace.element_size(), _opt(status, "status", _i32, 1))
    return (out, lse) if want_lse else out


def prefix_attention_packed(q: torch.Tensor, k_cache: tuple, v_cache: tuple, row_off: torch.Tensor, kv_len: torch.Tensor,
                          block_table: torch.Tensor, *, scale: Optional[float] = None,
                          group_off: Optional[torch.Tensor] = None, prefix_len: Optional[torch.Tensor] = None,
                          prefix_table: Optional[torch.Tensor] = None, want_lse: bool = False,
                          out: Optional[torch.Tensor] = None, lse: Optional[torch.Tensor] = None,
                          workspace: Optional[torch.Tensor] = None, status: Optional[torch.Tensor] = None, stream=None):
    """spec_prefix_attention_packed: ``prefix_attention`` over two ``packed_cache`` pairs."""
    rows, Hq, D = shape = q.shape
    dt, dev = q.dtype, _device()
    kc, ks, n_pages, P, Hk = _packed(k_cache, "k_cache", None, D, dev)
    vc, vs, n2, P2, _ = _packed(v_cache, "v_cache", Hk, D, dev)
    if (n_pages, P) != (n2, P2):
        raise ValueError("k_cache and v_cache must have the same pages")
    R, width = block_table.shape
    G, pages, go, pl, pt = _prefixes(group_off, prefix_len, prefix_table)
    strides = _strided(q, "q", dt, shape, dev)
    if workspace is not None:
        _here(workspace, "workspace")
    with _made(stream):
        made = out is None
        if made:
            out = torch.empty(shape, dtype=dt, device=q.device)
        if want_lse and lse is None:
            lse = torch.empty((rows, Hq), dtype=_f32, device=q.device)
        if workspace is None:
            workspace = torch.empty(attention_packed_workspace_bytes(rows, R, Hq, D), dtype=_u8, device=q.device)
    _ATTENTION_PACKED(_on(stream, q), R, rows, Hq, Hk, D, _code(q), P, n_pages, width, G, pages,
                      D ** -0.5 if scale is None else scale, *strides, kc, vc, _t(row_off, "row_off", _i32, R + 1, dev),
                      _t(kv_len, "kv_len", _i32, R, dev), _t(block_table, "block_table", _i32, 0, dev), go, pl, pt,
                      *((out.data_ptr(), Hq * D, D) if made else _strided(out, "out", dt, shape, dev)),
                      _opt(lse, "lse", _f32, rows * Hq, dev), _dev(workspace, "workspace").data_ptr(),
                      workspace.numel() * workspace.element_size(), _opt(status, "status", _i32, 1, dev), ks, vs)
    return (out, lse) if want_lse else out


# -------------------------------------------------------- logit adjustments --
def _matrix(t: torch.Tensor, name: str, dtype: torch.dtype) -> tuple:
    """Address and row stride of a matrix with dense rows on the current device."""
    _here(t, name)
    if t.dtype is not dtype:
        raise TypeError(f"{name} must be {dtype}")
    if t.dim() != 2 or (t.shape[1] > 1 and t.stride(1) != 1):
        raise ValueError(f"{name} must be a matrix with dense rows")
    return t.data_ptr(), (t.stride(0) if t.shape[0] > 1 else t.shape[1])


def adjust_logits(logits: torch.Tensor, tokens: Optional[torch.Tensor] = None,
                  prompt_len: Optional[torch.Tensor] = None, length: Optional[torch.Tensor] = None, *,
                  row_off: Optional[torch.Tensor] = None, rows_per_request: int = 1,
                  x: Optional[torch.Tensor] = None, repetition: Optional[torch.Tensor] = None,
                  frequency: Optional[torch.Tensor] = None, presence: Optional[torch.Tensor] = None,
                  bias: Optional[tuple] = None, mask: Optional[torch.Tensor] = None,
                  mask_row: Optional[torch.Tensor] = None, out: Optional[torch.Tensor] = None,
                  status: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """spec_adjust_logits: penalties, biases and grammar masks on the rows of ``logits`` [rows, V].

    ``row_off`` [R + 1] int32 packs the rows (schedule's row_off); without it each request has
    ``rows_per_request``.  ``tokens`` [R, n] int32 are each request's prompt and output so far
    (``length`` [R] of them, the first ``prompt_len`` [R] the prompt); row j counts the first j
    drafted tokens of ``x`` [R, gamma] too.  ``bias`` = (offsets [R + 1], tokens, values),
    ``mask`` [n, ceil(V / 32)] int32 bits with ``mask_row`` [rows] (negative: no mask).
    ``out`` may be ``logits``.  Rows outside every request's are left as they are in ``out``."""
    dt = logits.dtype
    lp, ld = _matrix(logits, "logits", dt)
    rows, V = shape = logits.shape
    if out is None:
        with _made(stream):
            out = torch.empty(shape, dtype=dt, device=logits.device)
        op, old = out.data_ptr(), V
    else:
        op, old = _matrix(out, "out", dt)
        if out.shape != shape:
            raise ValueError("out must have the shape of logits")
    if row_off is not None:
        R = row_off.numel() - 1
    else:
        R = length.numel() if length is not None else rows // max(rows_per_request, 1)
    tp = tl = tc = xp = xl = xc = bo = bt = bv = nb = mp = ml = nm = 0
    if tokens is not None:
        tp, tl = _matrix(tokens, "tokens", _i32)
        tc = tokens.shape[1]
        if tokens.shape[0] < R:
            raise ValueError("tokens must have a row for each request")
    if x is not None:
        xp, xl = _matrix(x, "x", _i32)
        xc = x.shape[1]
        if x.shape[0] < R:
            raise ValueError("x must have a row for each request")
    if bias is not None and bias[1].numel() > 0:
        nb = bias[1].numel()
        bo, bt, bv = (_t(bias[0], "bias offsets", _i32, R + 1), _t(bias[1], "bias tokens", _i32),
                      _t(bias[2], "bias values", _f32, nb))
    if mask is not None:
        mp, ml = _matrix(mask, "mask", _i32)
        nm = mask.shape[0]
        if mask.shape[1] * 32 < V:
            raise ValueError("mask rows must have ceil(V / 32) words")
    _LOGITS(_on(stream, logits), R, V, rows, rows_per_request, _code(logits), lp, ld, op, old,
            _opt(row_off, "row_off", _i32, 1), tp, tl, _opt(prompt_len, "prompt_len", _i32, R),
            _opt(length, "length", _i32, R), xp, xl, tc, xc, nb, _opt(repetition, "repetition", _f32, R),
            _opt(frequency, "frequency", _f32, R), _opt(presence, "presence", _f32, R), bo, bt, bv, mp, ml,
            _opt(mask_row, "mask_row", _i32, rows), nm, _opt(status, "status", _i32, 1))
    return out
