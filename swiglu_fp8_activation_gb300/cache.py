"""A paged key-value cache and the attention that reads it (include/sgq_cache.h),
with the same entry-point names: rotary positions, new rows into the cache
(16-bit, or FP8 with a scale a row), rows of it back, and attention of one new token
a sequence.

Argument marshalling only, as in `binding` and `grouped`: checks, output
allocation, the call. Every tensor of a call has to be on one CUDA device; the call runs
on that device and on `stream` (default: its current stream), and what it allocates
belongs to that stream. For inference: autograd records none of them (rope's
gradient is rope with inverse=True).

A cache is two tensors k and v [pages, heads, page_size, D] of the same strides, their last axis
contiguous: bfloat16 or float16 with fmt="none", or uint8 E4M3 with fmt="per_token" and
the rows' scales, float32 [pages, heads, page_size], beside each. A cache that keeps a token's heads side by
side, [pages, page_size, heads, D], is passed as its .transpose(1, 2). The slot of a token
is page * page_size + its place in the page.
"""
from __future__ import annotations

import ctypes as C
import functools
import math
import struct

import torch

from . import binding
from .binding import F_FP16, SgqError, _act_dtype, _check, library
from .grouped import _device, _here, _need, _raw_stream, _there

F_ROPE_INTERLEAVED, F_ROPE_INVERSE = 64, 128
MAX_HEAD = 256
MAX_HEADS = 1024
MAX_PAGE = 65536
MAX_SEQUENCES = 65536
MAX_WINDOW = (1 << 31) - 1      # no sequence is longer
#: The cache's formats.
CACHE_FORMATS = {"none": 3, "per_token": 2}
ROPE_LAYOUTS = {"half": 0, "interleaved": F_ROPE_INTERLEAVED}
_bound = None
_bf16, _f16, _f32, _i32, _i64, _u8 = torch.bfloat16, torch.float16, torch.float32, torch.int32, torch.int64, torch.uint8


class Heads(C.Structure):
    """sgq_heads_t: heads of some tokens."""
    _fields_ = [("p", C.c_void_p), ("heads", C.c_int64), ("token_stride", C.c_int64), ("head_stride", C.c_int64)]


class KvCache(C.Structure):
    """sgq_kv_cache_t: a paged cache."""
    _fields_ = [("pages", C.c_int64), ("page_size", C.c_int64), ("heads", C.c_int64), ("D", C.c_int64),
                ("page_stride", C.c_int64), ("head_stride", C.c_int64), ("token_stride", C.c_int64),
                ("k", C.c_void_p), ("v", C.c_void_p), ("k_scale", C.c_void_p), ("v_scale", C.c_void_p)]


class Rope(C.Structure):
    """sgq_rope_t: rotary positions."""
    _fields_ = [("R", C.c_int64), ("freqs", C.c_void_p), ("positions", C.c_void_p), ("position_bytes", C.c_int), ("factor", C.c_float)]


# The same as bytes: a third of the time of filling a ctypes structure.
_heads_bytes = struct.Struct("@P3q").pack
_cache_bytes = struct.Struct("@7q4P").pack
_rope_bytes = struct.Struct("@q2Pif").pack


def _lib() -> C.CDLL:
    global _bound
    if _bound is not None and _bound is binding._lib:
        return _bound
    L = library()
    if _bound is not L:
        vp, i64, u32, i32 = C.c_void_p, C.c_int64, C.c_uint32, C.c_int
        L.rope.restype = i32
        L.rope.argtypes = [u32, i64, i64, vp, vp, vp, vp]
        L.cache_write.restype = i32
        L.cache_write.argtypes = [i32, u32, i64, vp, vp, vp, vp, vp, vp, vp, i32, vp]
        L.cache_read.restype = i32
        L.cache_read.argtypes = [i32, u32, i64, vp, vp, i32, vp, vp, vp]
        L.paged_attention.restype = i32
        L.paged_attention.argtypes = [i32, u32, i64, vp, vp, vp, i64, vp, C.c_float, i64, vp, vp, vp, vp, vp]
        L.sgq_attention_workspace_bytes.restype = i64
        L.sgq_attention_workspace_bytes.argtypes = [i32] + [i64] * 7
        _bound = L
    return L


def rope_turns(radians, device="cuda") -> torch.Tensor:
    """Frequencies for rope: radians a position (numbers, or a tensor of them) as 2^-64 of a turn, int64."""
    values = radians.double().tolist() if isinstance(radians, torch.Tensor) else radians
    whole = 1 << 64
    turns = [int(math.ldexp(float(f) / (2 * math.pi), 64)) % whole for f in values]
    return torch.tensor([t - whole if t >= whole >> 1 else t for t in turns], dtype=torch.int64, device=device)


def rope_frequencies(R: int, base: float = 10000.0, *, scaling: str | None = None, stretch: float = 1.0,
                     trained: int | None = None, fast: float = 32.0, slow: float = 1.0, device="cuda"):
    """(frequencies, factor) of rope for R rotated columns: base^(-2i/R) radians a
    position for pair i, and for a context `stretch` times as long as the trained one

      "linear"  every frequency divided by stretch
      "ntk"     the base raised to base * stretch^(R / (R - 2)): the slowest pair
                stretched by stretch, the fastest not at all
      "yarn"    pairs that turn more than `fast` times within `trained` positions kept, those
                that turn less than `slow` times divided by stretch, the ones between
                blended; factor 0.1 ln(stretch) + 1

    Computed in 64 bits; factor is 1 but with "yarn".
    """
    if R < 16 or R % 16:
        raise SgqError(f"R: a multiple of 16, got {R}", 2)
    if scaling not in (None, "linear", "ntk", "yarn"):
        raise SgqError(f"unknown scaling {scaling!r}")
    if not (stretch >= 1.0 and math.isfinite(stretch) and base > 1.0 and math.isfinite(base)):
        raise SgqError(f"stretch: at least 1, got {stretch}; base: above 1, got {base}")
    factor = 1.0
    if scaling == "ntk":
        base = base * stretch ** (R / (R - 2))
    inv = [base ** (-2 * i / R) for i in range(R // 2)]
    if scaling == "linear":
        inv = [f / stretch for f in inv]
    if scaling == "yarn":
        if trained is None or trained < 1:
            raise SgqError("yarn: the trained length is missing")
        pair = lambda turns: R * math.log(trained / (turns * 2 * math.pi)) / (2 * math.log(base))  # noqa: E731
        lo, hi = max(0, math.floor(pair(fast))), min(R - 1, math.ceil(pair(slow)))
        slowness = [min(1.0, max(0.0, (i - lo) / max(hi - lo, 0.001))) for i in range(R // 2)]
        inv = [f * (1 - s) + f / stretch * s for f, s in zip(inv, slowness)]
        factor = 0.1 * math.log(stretch) + 1
    return rope_turns(inv, device), factor


def _heads(t: torch.Tensor, dtype, name: str, shape) -> bytes:
    """sgq_heads_t of t, which has to have this shape [T, heads, D]."""
    if t.dtype is not dtype or t.shape != shape or len(shape) != 3:
        raise SgqError(f"{name}: expected {dtype} {tuple(shape) if len(shape) == 3 else '[T, heads, D]'}, got {t.dtype} {tuple(t.shape)}")
    ts, hs, one = t.stride()
    if one != 1 and shape[2] > 1:
        raise SgqError(f"{name}: the values of a head have to lie side by side")
    return _heads_bytes(t.data_ptr(), shape[1], ts, hs)


def _cache(k: torch.Tensor, v: torch.Tensor, fmt: str, k_scale, v_scale, dtype):
    """(sgq_kv_cache_t of the caches, their shape, the format's code)."""
    code = CACHE_FORMATS.get(fmt)
    if code is None:
        raise SgqError(f"unknown cache format {fmt!r}")
    want = dtype if code == 3 else torch.uint8
    shape, strides = k.shape, k.stride()
    if k.dtype is not want or v.dtype is not want or len(shape) != 4 or v.shape != shape:
        raise SgqError(f"{fmt}: expected two {want} caches [pages, heads, page_size, D], got {k.dtype} {tuple(shape)}, {v.dtype} {tuple(v.shape)}")
    if strides != v.stride() or strides[3] != 1:
        raise SgqError(f"the caches have to share their strides, the last one 1: got {strides}, {v.stride()}")
    if code == 3:
        if k_scale is not None or v_scale is not None:
            raise SgqError("k_scale, v_scale: of no use with format 'none'")
        ks = vs = 0
    else:
        if k_scale is None or v_scale is None:
            raise SgqError(f"k_scale, v_scale: missing with format {fmt!r}")
        _need(k_scale, shape[:3], torch.float32, "k_scale")
        _need(v_scale, shape[:3], torch.float32, "v_scale")
        ks, vs = k_scale.data_ptr(), v_scale.data_ptr()
    return (_cache_bytes(shape[0], shape[2], shape[1], shape[3], strides[0], strides[1], strides[2], k.data_ptr(), v.data_ptr(), ks, vs),
            shape, code)


def _index(t: torch.Tensor, n: int, name: str) -> int:
    """Bytes of an index of n int32 or int64."""
    dt = t.dtype
    if (dt is not torch.int64 and dt is not torch.int32) or t.shape != (n,) or not t.is_contiguous():
        raise SgqError(f"{name}: expected contiguous int32 or int64 [{n}], got {t.dtype} {tuple(t.shape)}")
    return 8 if dt is torch.int64 else 4


def _turn(freqs: torch.Tensor, positions: torch.Tensor, T: int, layout: str, factor: float):
    """(sgq_rope_t, the layout's flag)."""
    flag = ROPE_LAYOUTS.get(layout)
    if flag is None:
        raise SgqError(f"unknown order of pairs {layout!r}")
    if not abs(factor) <= 3.4e38:
        raise SgqError(f"factor: expected a finite number, got {factor}")
    if freqs.dim() != 1 or freqs.dtype is not torch.int64 or not freqs.is_contiguous():
        raise SgqError(f"freqs: expected contiguous int64 [R / 2], got {freqs.dtype} {tuple(freqs.shape)}")
    return _rope_bytes(2 * len(freqs), freqs.data_ptr(), positions.data_ptr(), _index(positions, T, "positions"), factor), flag


def rope(x: torch.Tensor, positions: torch.Tensor, freqs: torch.Tensor, *, layout: str = "half", factor: float = 1.0,
         inverse: bool = False, out: torch.Tensor | None = None, stream=None):
    """Rotary positions on heads (one kernel launch): pair i of the first R
    columns of x[t] turned by positions[t] * freqs[i] and multiplied by factor.

    x [T, heads, D] bfloat16 or float16, its tokens and heads at any strides that are
    multiples of 8 (a part of a projection's rows). positions [T] int32 or int64;
    freqs [R/2] int64 (rope_frequencies, rope_turns). layout: pairs are columns
    (i, i + R/2), "half", or (2i, 2i + 1), "interleaved"; columns from R on are
    passed on. inverse=True turns the other way: the gradient. Returns out
    [T, heads, D] of x's type, contiguous where it is not given; out=x rotates in place.
    """
    dt, shape = x.dtype, x.shape
    if dt is not _bf16 and dt is not _f16:
        _act_dtype(x, "x")
    src = _heads(x, dt, "x", shape)
    T, _, D = shape
    turn, flags = _turn(freqs, positions, T, layout, factor)
    d = x.get_device()
    if stream is None and d >= 0 and positions.get_device() == freqs.get_device() == d == _device() and (out is None or out.get_device() == d):
        at = _raw_stream(d)
    else:
        at = _here(stream, "rope", x, positions, freqs, out)
    if at is None:
        with _there(stream, x):
            return rope(x, positions, freqs, layout=layout, factor=factor, inverse=inverse, out=out)
    if out is None:
        out = torch.empty(shape, dtype=dt, device=x.device)
    if inverse:
        flags |= F_ROPE_INVERSE
    if dt is torch.float16:
        flags |= F_FP16
    st = _lib().rope(flags, T, D, turn, src, _heads(out, dt, "out", shape), at)
    if st:
        _check(st, "rope")
    return out


def cache_write(k: torch.Tensor, v: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor, slots: torch.Tensor, *,
                fmt: str = "none", k_scale: torch.Tensor | None = None, v_scale: torch.Tensor | None = None,
                q: torch.Tensor | None = None, q_out: torch.Tensor | None = None, positions: torch.Tensor | None = None,
                freqs: torch.Tensor | None = None, layout: str = "half", factor: float = 1.0, stream=None):
    """New rows into the cache (one kernel launch): token t's keys, rotated where
    positions and freqs are given, and values go to slots[t]; q, if given, is
    rotated to q_out in the same launch.

    k and v [T, heads, D] and q [T, Hq, D]: bfloat16 or float16, strided as in
    rope. k_cache, v_cache, k_scale, v_scale: see the module; written. slots [T]
    int32 or int64: all different; a token whose slot is outside the cache (-1) is not
    written (its q is rotated all the same). "per_token" quantises each row by
    quantize_fp8's rule, keys from their 32-bit rotation. Returns q_out
    (allocated where it is not given; q itself to rotate in place), or None without q.
    """
    dt = k.dtype
    if dt is not _bf16 and dt is not _f16:
        _act_dtype(k, "k")
    ck, laid, code = _cache(k_cache, v_cache, fmt, k_scale, v_scale, dt)
    T, D = k.shape[0], laid[3]
    shape = (T, laid[1], D)
    hk, hv = _heads(k, dt, "k", shape), _heads(v, dt, "v", shape)
    slot_bytes = _index(slots, T, "slots")
    turn, flags, hq = None, 0, None
    if positions is not None and freqs is not None:
        turn, flags = _turn(freqs, positions, T, layout, factor)
    elif positions is not None or freqs is not None:
        raise SgqError("positions and freqs go together")
    if q is not None:
        if turn is None:
            raise SgqError("q: of no use without positions")
        qshape = q.shape
        hq = _heads(q, dt, "q", (T, qshape[1], D) if len(qshape) == 3 else (T, 1, D))
    elif q_out is not None:
        raise SgqError("q_out: of no use without q")
    d = k.get_device()
    if (stream is None and d >= 0 and d == _device() == v.get_device() == k_cache.get_device() == v_cache.get_device() == slots.get_device()
            and (k_scale is None or d == k_scale.get_device() == v_scale.get_device()) and (turn is None or d == positions.get_device() == freqs.get_device())
            and (q is None or q.get_device() == d) and (q_out is None or q_out.get_device() == d)):
        at = _raw_stream(d)
    else:
        at = _here(stream, "cache_write", k, v, k_cache, v_cache, slots, k_scale, v_scale, q, q_out, positions, freqs)
    if at is None:
        with _there(stream, k):
            return cache_write(k, v, k_cache, v_cache, slots, fmt=fmt, k_scale=k_scale, v_scale=v_scale, q=q, q_out=q_out,
                               positions=positions, freqs=freqs, layout=layout, factor=factor)
    ho = None
    if q is not None:
        if q_out is None:
            q_out = torch.empty(qshape, dtype=dt, device=q.device)
        ho = _heads(q_out, dt, "q_out", qshape)
    if dt is torch.float16:
        flags |= F_FP16
    st = _lib().cache_write(code, flags, T, ck, turn, hq, ho, hk, hv, slots.data_ptr(), slot_bytes, at)
    if st:
        _check(st, "cache_write")
    return q_out


def cache_read(k_cache: torch.Tensor, v_cache: torch.Tensor, slots: torch.Tensor, *, fmt: str = "none",
               k_scale: torch.Tensor | None = None, v_scale: torch.Tensor | None = None, dtype: torch.dtype | None = None,
               k_out: torch.Tensor | None = None, v_out: torch.Tensor | None = None, stream=None):
    """Rows of the cache as 16-bit values (one kernel launch): k and v
    [S, heads, D] of the tokens at slots [S] (int32 or int64, any order, any
    number of times; zeros where a slot is outside the cache).

    dtype: bfloat16 (default with "per_token") or float16; the cache's own with "none".
    """
    own = k_cache.dtype if fmt == "none" else None
    dt = dtype or own or (k_out.dtype if k_out is not None else torch.bfloat16)
    if (dt is not torch.bfloat16 and dt is not torch.float16) or (own is not None and dt is not own):
        raise SgqError(f"rows of a {k_cache.dtype} cache as {dt}")
    ck, laid, code = _cache(k_cache, v_cache, fmt, k_scale, v_scale, dt)
    S = slots.shape[0] if slots.dim() == 1 else -1
    slot_bytes = _index(slots, S, "slots")
    shape = (S, laid[1], laid[3])
    for t, name in ((k_out, "k_out"), (v_out, "v_out")):
        if t is not None:
            _need(t, shape, dt, name)
    d = slots.get_device()
    if (stream is None and d >= 0 and d == _device() == k_cache.get_device() == v_cache.get_device()
            and (k_scale is None or d == k_scale.get_device() == v_scale.get_device()) and k_out is None and v_out is None):
        at = _raw_stream(d)
    else:
        at = _here(stream, "cache_read", k_cache, v_cache, slots, k_scale, v_scale, k_out, v_out)
    if at is None:
        with _there(stream, k_cache):
            return cache_read(k_cache, v_cache, slots, fmt=fmt, k_scale=k_scale, v_scale=v_scale, dtype=dt, k_out=k_out, v_out=v_out)
    if k_out is None:
        k_out = torch.empty(shape, dtype=dt, device=k_cache.device)
    if v_out is None:
        v_out = torch.empty(shape, dtype=dt, device=k_cache.device)
    st = _lib().cache_read(code, F_FP16 if dt is torch.float16 else 0, S, ck, slots.data_ptr(), slot_bytes,
                           k_out.data_ptr(), v_out.data_ptr(), at)
    if st:
        _check(st, "cache_read")
    return k_out, v_out


@functools.lru_cache(maxsize=1024)
def _workspace(lib, *sizes) -> int:
    return lib.sgq_attention_workspace_bytes(*sizes)


def attention_workspace_bytes(fmt: str, B: int, Hq: int, heads: int, D: int, width: int, page_size: int, window: int = 0) -> int:
    """Bytes of paged_attention's workspace (0 where it needs none, or out of range)."""
    if fmt not in CACHE_FORMATS:
        raise SgqError(f"unknown cache format {fmt!r}")
    return _workspace(_lib(), CACHE_FORMATS[fmt], B, Hq, heads, D, width, page_size, max(-1, min(window, MAX_WINDOW)))


def paged_attention(q: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor, pages: torch.Tensor, lengths: torch.Tensor, *,
                    fmt: str = "none", k_scale: torch.Tensor | None = None, v_scale: torch.Tensor | None = None,
                    scale: float | None = None, window: int = 0, sinks: torch.Tensor | None = None,
                    out: torch.Tensor | None = None, lse: bool | torch.Tensor = False,
                    workspace: torch.Tensor | None = None, stream=None):
    """Attention of one new token a sequence over its pages (one kernel launch, or
    two): softmax(scale * q[b] . keys) . values over tokens t < lengths[b], in fp32.

    q [B, Hq, D] bfloat16 or float16, strided as in rope; head h of q reads head
    h // (Hq / heads) of the cache. pages [B, width] int32: token t of b is at
    place t % page_size of page pages[b, t // page_size] (a page outside the cache
    masks its tokens); lengths [B] int32, on the device, the new token counted where its row is
    in the cache. scale: 1/sqrt(D) by default. window: only the last `window`
    tokens (0: all). sinks [Hq] float32: a logit a head that joins the softmax without a
    value. Returns out [B, Hq, D], zeros where a sequence has no token; with
    lse=True, or a float32 [B, Hq] to write, (out, the log of the softmax's sum).
    workspace: uint8 [attention_workspace_bytes(fmt, B, Hq, heads, D, width, page_size,
    window)] or None (allocated where one is needed). Waits inside the kernel are limited: see
    wait_timeouts.
    """
    dt, shape = q.dtype, q.shape
    if dt is not _bf16 and dt is not _f16:
        _act_dtype(q, "q")
    ck, laid, code = _cache(k_cache, v_cache, fmt, k_scale, v_scale, dt)
    _, heads, page_size, D = laid
    B, Hq, _ = shape if len(shape) == 3 else (0, 0, 0)
    hq = _heads(q, dt, "q", (B, Hq, D))
    wide = pages.shape
    width = wide[1] if len(wide) == 2 else 0
    if pages.dtype is not _i32 or wide != (B, width) or not pages.is_contiguous():
        _need(pages, (B, width), _i32, "pages")
    if lengths.dtype is not _i32 or lengths.shape != (B,) or not lengths.is_contiguous():
        _need(lengths, (B,), _i32, "lengths")
    if sinks is not None:
        _need(sinks, (Hq,), torch.float32, "sinks")
    if out is not None:
        _need(out, shape, dt, "out")
    if not 0 <= window <= MAX_WINDOW:        # an argument of 64 bits would cut what they do not hold
        if window < 0:
            raise SgqError(f"window: expected 0 (none) or more, got {window}", 1)
        window = MAX_WINDOW
    L = _lib()
    room = _workspace(L, code, B, Hq, heads, D, width, page_size, window)
    if workspace is not None:
        _need(workspace, (room,), torch.uint8, "workspace")
    told = None
    if lse is not False and lse is not True:
        told = lse
        _need(told, (B, Hq), torch.float32, "lse")
    d = q.get_device()
    if (stream is None and d >= 0 and d == _device() == k_cache.get_device() == v_cache.get_device() == pages.get_device() == lengths.get_device()
            and (k_scale is None or d == k_scale.get_device() == v_scale.get_device()) and (sinks is None or sinks.get_device() == d)
            and out is None and told is None and workspace is None):
        at = _raw_stream(d)
    else:
        at = _here(stream, "paged_attention", q, k_cache, v_cache, pages, lengths, k_scale, v_scale, sinks, out, told, workspace)
    if at is None:
        with _there(stream, q):
            return paged_attention(q, k_cache, v_cache, pages, lengths, fmt=fmt, k_scale=k_scale, v_scale=v_scale, scale=scale,
                                   window=window, sinks=sinks, out=out, lse=lse, workspace=workspace)
    device = q.device
    if out is None:
        out = torch.empty(shape, dtype=dt, device=device)
    if lse is True:
        told = torch.empty((B, Hq), dtype=torch.float32, device=device)
    if workspace is None and room:
        workspace = torch.empty((room,), dtype=torch.uint8, device=device)
    st = L.paged_attention(code, F_FP16 if dt is torch.float16 else 0, B, ck, hq, pages.data_ptr(), width, lengths.data_ptr(),
                           D ** -0.5 if scale is None else scale, window, None if sinks is None else sinks.data_ptr(), out.data_ptr(),
                           None if told is None else told.data_ptr(), None if workspace is None else workspace.data_ptr(), at)
    if st:
        _check(st, "paged_attention")
    return out if told is None else (out, told)
