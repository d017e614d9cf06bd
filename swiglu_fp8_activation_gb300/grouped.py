"""Products over ragged groups of rows (include/sgq_group.h), with the same
entry-point names: the routing of an expert layer, its grouped matrix products
on FP8 or 16-bit rows, its weighted sum, and the low-rank adapters of many
requests beside a shared projection.

Argument marshalling only, as in `binding`: checks, output allocation, the
call. Every tensor of a call has to be on one CUDA device; the call runs on
that device and on `stream` (default: its current stream), and what it
allocates belongs to that stream. Like the rest of the library these are for
inference: autograd records none of them, lora_add's update of y included.
"""
from __future__ import annotations

import ctypes as C

import torch

from .binding import F_FP16, FORMATS, GROUP, SgqError, _act_dtype, _check, library

MAX_GROUPS = 1024
MAX_RANK = 128
#: grouped_gemm's formats: the FP8 formats, and "none" for 16-bit rows and weights.
GEMM_FORMATS = {**FORMATS, "none": 3}
_bound = None


def _lib() -> C.CDLL:
    global _bound
    L = library()
    if _bound is not L:
        vp, i64, u32 = C.c_void_p, C.c_int64, C.c_uint32
        L.group_rows.restype = C.c_int
        L.group_rows.argtypes = [C.c_int, i64, i64, i64, vp, vp, vp, vp, vp]
        L.grouped_gemm.restype = C.c_int
        L.grouped_gemm.argtypes = [C.c_int, u32, i64, i64, i64, i64, i64, vp, vp, vp, vp, vp, vp, vp, vp]
        L.combine_rows.restype = C.c_int
        L.combine_rows.argtypes = [u32, i64, i64, i64, i64, vp, vp, vp, vp, vp]
        L.lora_add.restype = C.c_int
        L.lora_add.argtypes = [u32, i64, i64, i64, i64, i64, i64] + [vp] * 10
        L.sgq_wait_timeouts.restype = C.c_int
        L.sgq_wait_timeouts.argtypes = [C.POINTER(C.c_uint32)]
        L.sgq_lora_workspace_bytes.restype = i64
        L.sgq_lora_workspace_bytes.argtypes = [i64, i64, i64]
        _bound = L
    return L


def _dims(t: torch.Tensor, n: int, name: str):
    if t.dim() != n:
        raise SgqError(f"{name}: expected {n} dimensions, got {tuple(t.shape)}")
    return t.shape


_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (lambda d: torch.cuda.current_stream(d).cuda_stream)


def _need(t: torch.Tensor, shape, dtype, name: str):
    if t.dtype != dtype or t.shape != shape:
        raise SgqError(f"{name}: expected {dtype} {tuple(shape)}, got {t.dtype} {tuple(t.shape)}")
    if not t.is_contiguous():
        raise SgqError(f"{name}: must be contiguous")


def _here(stream, what: str, *tensors):
    """The current stream's handle, where every tensor (or None) is on the
    current CUDA device and no other stream is asked for; else None."""
    d = tensors[0].get_device()
    for t in tensors:
        if t is not None and t.get_device() != d:
            raise SgqError(f"{what}: a tensor on {t.device}, another on {tensors[0].device}")
    if d < 0:
        raise SgqError(f"{what}: expected CUDA tensors, got {tensors[0].device}")
    if stream is not None:
        if stream.device != tensors[0].device:
            raise SgqError(f"{what}: a stream of {stream.device}, tensors on {tensors[0].device}")
        return None
    return _raw_stream(d) if d == torch.cuda.current_device() else None


def _there(stream, t: torch.Tensor):
    """Makes t's device the current one and `stream` (default: that device's
    current stream) its current stream: what a call allocates inside belongs to it."""
    return torch.cuda.stream(torch.cuda.current_stream(t.device) if stream is None else stream)


def _at(t: torch.Tensor | None):
    return None if t is None else t.data_ptr()


def group_rows(ids: torch.Tensor, groups: int, *, offsets_out: torch.Tensor | None = None,
               rows_out: torch.Tensor | None = None, slots_out: torch.Tensor | None = None, stream=None):
    """Rows in group order (one kernel launch): the routing of an expert layer,
    or the adapters of a batch's requests.

    ids [T, k] (or [T], k = 1) int32 or int64: the group of each of a token's
    k rows; an id outside [0, groups) takes no slot. Returns (offsets
    [groups+1], rows [T*k], slots like ids), all int32: group g has the slots
    offsets[g] to offsets[g+1]; slot s holds token rows[s] (-1 behind the last
    group); ids[t, j] has slot slots[t, j] (-1 where it has none). Ids of one
    group keep their order.
    """
    if ids.dim() not in (1, 2):
        raise SgqError(f"ids: expected [T, k] or [T], got {tuple(ids.shape)}")
    if ids.dtype not in (torch.int32, torch.int64):
        raise SgqError(f"ids: expected int32 or int64, got {ids.dtype}")
    if not ids.is_contiguous():
        raise SgqError("ids: must be contiguous")
    shape = ids.shape
    T, k = shape[0], shape[1] if len(shape) == 2 else 1
    groups = int(groups)
    if not 1 <= groups <= MAX_GROUPS or k < 1:
        raise SgqError(f"groups: 1 to {MAX_GROUPS}, got {groups}; ids a token: at least 1, got {k}")
    if offsets_out is not None:
        _need(offsets_out, (groups + 1,), torch.int32, "offsets_out")
    if rows_out is not None:
        _need(rows_out, (T * k,), torch.int32, "rows_out")
    if slots_out is not None:
        _need(slots_out, shape, torch.int32, "slots_out")
    at = _here(stream, "group_rows", ids, offsets_out, rows_out, slots_out)
    if at is None:
        with _there(stream, ids):
            return group_rows(ids, groups, offsets_out=offsets_out, rows_out=rows_out, slots_out=slots_out)
    if offsets_out is None:
        offsets_out = torch.empty((groups + 1,), dtype=torch.int32, device=ids.device)
    if rows_out is None:
        rows_out = torch.empty((T * k,), dtype=torch.int32, device=ids.device)
    if slots_out is None:
        slots_out = torch.empty(shape, dtype=torch.int32, device=ids.device)
    st = _lib().group_rows(ids.element_size(), T, k, groups, ids.data_ptr(), offsets_out.data_ptr(), rows_out.data_ptr(),
                           slots_out.data_ptr(), at)
    if st:
        _check(st, "group_rows")
    return offsets_out, rows_out, slots_out


def gemm_scale_shapes(fmt: str, x_rows: int, groups: int, N: int, K: int):
    """(shape of x_scale, shape of w_scale, their dtype) of grouped_gemm; None for "none"."""
    if fmt == "none":
        return None, None, None
    if fmt == "mxfp8":
        return (x_rows, K // 32), (groups, -(-N // 128) * 128, -(-(K // 32) // 4) * 4), torch.uint8
    if fmt == "block128":
        return (x_rows, K // 128), (groups, -(-N // 128), K // 128), torch.float32
    return (x_rows, 1), (groups, N), torch.float32


def grouped_gemm(x: torch.Tensor, w: torch.Tensor, offsets: torch.Tensor, *, fmt: str = "mxfp8",
                 x_scale: torch.Tensor | None = None, w_scale: torch.Tensor | None = None,
                 rows: torch.Tensor | None = None, out: torch.Tensor | None = None,
                 out_dtype: torch.dtype | None = None, stream=None):
    """Matrix products grouped by ragged sets of rows (one kernel launch):
    out[s] = x[rows[s]] @ w[g].T for the slots s of group g, summed in fp32.

    x [X, K] and w [groups, N, K]: uint8 E4M3 with the scales of an FP8 format,
    or bfloat16 / float16 with fmt="none". x_scale is what the library's
    quantisation writes row-major; w_scale: "mxfp8" uint8 [groups, N up to 128,
    K/32 up to 4] (each group's scales in the swizzled layout), "block128"
    float32 [groups, ceil(N/128), K/128], "per_token" float32 [groups, N].
    offsets [groups+1] int32; rows [S] int32 or None (slot s reads x[s], S = X).
    A row index outside x reads zeros. Returns out [S, N] (bfloat16, float16 by
    out_dtype or `out`, x's type with "none"); slots of no group keep what out
    held. Waits inside the kernel are limited: see wait_timeouts.
    """
    if fmt not in GEMM_FORMATS:
        raise SgqError(f"unknown format {fmt!r}")
    X, K = _dims(x, 2, "x")
    groups, N, _ = _dims(w, 3, "w")
    dt = _act_dtype(x, "x") if fmt == "none" else torch.uint8
    _need(x, (X, K), dt, "x")
    _need(w, (groups, N, K), dt, "w")
    unit = {"per_token": 16, "none": 8, **GROUP}[fmt]
    if K < 1 or K % unit or N < 1 or N % 8:
        raise SgqError(f"{fmt}: K has to be a multiple of {unit} and N of 8, got K = {K}, N = {N}", 2)
    xshape, wshape, sdt = gemm_scale_shapes(fmt, X, groups, N, K)
    for t, shape, name in ((x_scale, xshape, "x_scale"), (w_scale, wshape, "w_scale")):
        if (t is None) != (shape is None):
            raise SgqError(f"{name}: {'missing' if t is None else 'of no use'} with format {fmt!r}")
        if t is not None:
            _need(t, shape, sdt, name)
    _need(offsets, (groups + 1,), torch.int32, "offsets")
    S = X
    if rows is not None:
        S, = _dims(rows, 1, "rows")
        _need(rows, (S,), torch.int32, "rows")
    odt = out_dtype or (out.dtype if out is not None else dt if fmt == "none" else torch.bfloat16)
    if odt not in (torch.bfloat16, torch.float16) or (fmt == "none" and odt != dt):
        raise SgqError(f"out: {odt} does not go with x of {x.dtype}")
    if out is not None:
        _need(out, (S, N), odt, "out")
    at = _here(stream, "grouped_gemm", x, w, offsets, x_scale, w_scale, rows, out)
    if at is None:
        with _there(stream, x):
            return grouped_gemm(x, w, offsets, fmt=fmt, x_scale=x_scale, w_scale=w_scale, rows=rows, out=out, out_dtype=odt)
    if out is None:
        out = torch.empty((S, N), dtype=odt, device=x.device)
    st = _lib().grouped_gemm(GEMM_FORMATS[fmt], F_FP16 if odt == torch.float16 else 0, S, groups, N, K, X, x.data_ptr(),
                             _at(x_scale), w.data_ptr(), _at(w_scale), offsets.data_ptr(), _at(rows), out.data_ptr(), at)
    if st:
        _check(st, "grouped_gemm")
    return out


def combine_rows(y: torch.Tensor, slots: torch.Tensor, weights: torch.Tensor | None = None, *,
                 out: torch.Tensor | None = None, stream=None):
    """The weighted sum of each token's rows (one kernel launch):
    out[t] = sum_j weights[t, j] * y[slots[t, j]], in fp32 in order of j.

    y [S, N] bfloat16 or float16; slots [T, k] int32 (a slot outside [0, S)
    adds nothing); weights [T, k] float32 or None (ones). Returns out [T, N] of
    y's type.
    """
    S, N = _dims(y, 2, "y")
    T, k = _dims(slots, 2, "slots")
    dt = _act_dtype(y, "y")
    _need(y, (S, N), dt, "y")
    _need(slots, (T, k), torch.int32, "slots")
    if weights is not None:
        _need(weights, (T, k), torch.float32, "weights")
    if out is not None:
        _need(out, (T, N), dt, "out")
    at = _here(stream, "combine_rows", y, slots, weights, out)
    if at is None:
        with _there(stream, y):
            return combine_rows(y, slots, weights, out=out)
    if out is None:
        out = torch.empty((T, N), dtype=dt, device=y.device)
    st = _lib().combine_rows(F_FP16 if dt == torch.float16 else 0, T, k, S, N, y.data_ptr(), slots.data_ptr(), _at(weights),
                             out.data_ptr(), at)
    if st:
        _check(st, "combine_rows")
    return out


def wait_timeouts() -> int:
    """Launches of grouped_gemm and lora_add on the current device in which a
    wait inside the kernel ran out of time (some seconds without progress). Such
    a launch ends, its call having returned, and leaves its outputs unspecified:
    this count is where it shows. Waits for the device; not during graph capture."""
    n = C.c_uint32(0)
    _check(_lib().sgq_wait_timeouts(C.byref(n)), "sgq_wait_timeouts")
    return n.value


def lora_workspace_bytes(S: int, groups: int, R: int) -> int:
    """Bytes of lora_add's workspace (0 where it needs none, or out of range)."""
    return _lib().sgq_lora_workspace_bytes(int(S), int(groups), int(R))


def lora_add(x: torch.Tensor, a: torch.Tensor, b: torch.Tensor, y: torch.Tensor, offsets: torch.Tensor, *,
             rows: torch.Tensor | None = None, slots: torch.Tensor | None = None,
             scaling: torch.Tensor | None = None, workspace: torch.Tensor | None = None, stream=None):
    """The low-rank adapters of many requests, added in place to a shared
    projection's output (one kernel launch, or two): for slot s of adapter g with
    t = rows[s], y[t] += scaling[g] * (x[t] @ a[g].T) @ b[g].T, in fp32.

    x [T, K], a [groups, R, K], b [groups, N, R] and y [T, N]: all bfloat16 or
    all float16. offsets, rows, slots: group_rows of the requests' adapters
    ([T] ids, -1 for none); rows and slots both None where the rows of x
    already are in adapter order (slot s is row s). scaling [groups] float32 or
    None (ones). workspace: uint8 [lora_workspace_bytes(S, groups, R)]
    or None (allocated where one is needed). Rows without an
    adapter stay as they are. Returns y. Waits inside the kernels are limited:
    see wait_timeouts.
    """
    T, K = _dims(x, 2, "x")
    groups, R, _ = _dims(a, 3, "a")
    _, N = _dims(y, 2, "y")
    dt = _act_dtype(x, "x")
    _need(x, (T, K), dt, "x")
    _need(a, (groups, R, K), dt, "a")
    _need(b, (groups, N, R), dt, "b")
    _need(y, (T, N), dt, "y")
    _need(offsets, (groups + 1,), torch.int32, "offsets")
    if (rows is None) != (slots is None):
        raise SgqError("rows and slots go together")
    S = T
    if rows is not None:
        S, = _dims(rows, 1, "rows")
        _need(rows, (S,), torch.int32, "rows")
        _need(slots, (T, 1) if slots.dim() == 2 else (T,), torch.int32, "slots")
    if scaling is not None:
        _need(scaling, (groups,), torch.float32, "scaling")
    room = _lib().sgq_lora_workspace_bytes(S, groups, R)
    if workspace is not None:
        _need(workspace, (room,), torch.uint8, "workspace")
    at = _here(stream, "lora_add", x, a, b, y, offsets, rows, slots, scaling, workspace)
    if at is None:
        with _there(stream, x):
            return lora_add(x, a, b, y, offsets, rows=rows, slots=slots, scaling=scaling, workspace=workspace)
    if workspace is None and room:
        workspace = torch.empty((room,), dtype=torch.uint8, device=x.device)
    st = _lib().lora_add(F_FP16 if dt == torch.float16 else 0, T, S, groups, R, K, N, x.data_ptr(), a.data_ptr(), b.data_ptr(),
                      _at(scaling), offsets.data_ptr(), _at(rows), _at(slots), y.data_ptr(), _at(workspace), at)
    if st:
        _check(st, "lora_add")
    return y
