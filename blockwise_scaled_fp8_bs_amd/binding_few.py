"""Thin Python binding of the C ABI's entry points that serve few tokens from
quantized weights (include/bs.h): the MXFP4 quantizer, the product of few rows,
and the gated experts of few routed tokens.

Conventions of ``binding_block``: argument marshalling only, ``ValueError`` for
tensors in the wrong layout, outputs and workspaces from the pool of the stream
that is passed (the current one without), a workspace of its own for each call.
Tensors may be on another GPU than the current one, all on the same.

Weights [N, K] by kind, codes as uint8 with contiguous rows:

* BS_WEIGHT_E4M3_128X128: [N, K] and float32 scales [K/128, >= N/128];
* BS_WEIGHT_MXFP8: [N, K] and uint8 scales [K/32, >= N];
* BS_WEIGHT_MXFP4: [N, K/2] (two codes a byte) and uint8 scales [K/32, >= N].
"""

import ctypes

import torch

from . import _lib
from .binding import _check, _mat
from .binding_block import _DT, _first, _flat, _matrix, _new, _optional, _stream_of

BS_WEIGHT_E4M3_128X128 = 0
BS_WEIGHT_MXFP8 = 1
BS_WEIGHT_MXFP4 = 2

#: by kind: codes a byte, contraction and rows of a scale, type of the scales
_KINDS = {
    BS_WEIGHT_E4M3_128X128: (1, 128, 128, torch.float32),
    BS_WEIGHT_MXFP8: (1, 32, 1, torch.uint8),
    BS_WEIGHT_MXFP4: (2, 32, 1, torch.uint8),
}


def _call(fn, index, *args):
    """Calls the library with the GPU of the tensors as the current one."""
    call = getattr(_lib.load(), fn)
    if torch._C._cuda_getDevice() == index:
        status = call(*args)
    else:
        with torch.cuda.device(index):
            status = call(*args)
    if status:
        _check(status, fn)


def _other_gpu(t, name, index):
    raise ValueError(f"{name} is on {t.device}, x on cuda:{index}: all tensors must be on one GPU")


def _rows_of(t, name, dtype, R, C, index):
    """(address, row stride) of a row-major [R, C] matrix on GPU `index` whose
    rows need no alignment; (None, 0) for None."""
    if t is None:
        return None, 0
    p, ld = _matrix(t, name, dtype, R, C)
    if t.get_device() != index:
        _other_gpu(t, name, index)
    return p, ld if R > 1 else C


def _fail_weight(q, s, names, kind, shape, scales, dtype, index):
    """Says what is wrong with weights that _weight did not take."""
    _mat(q, names[0], torch.uint8, len(shape))
    if q.shape != shape:
        raise ValueError(f"{names[0]} must be {list(shape)}, got {list(q.shape)}")
    _mat(s, names[1], dtype, len(shape))
    if s.shape[:-1] != scales[:-1] or s.shape[-1] < scales[-1]:
        raise ValueError(f"{names[1]} must be {list(scales[:-1])} x >= {scales[-1]} (K-major), got {list(s.shape)}")
    _other_gpu(*((q, names[0]) if q.get_device() != index else (s, names[1])), index)


def _weight(q, s, names, kind, N, K, index):
    """Codes of weights [N, K], their row stride, scales and theirs.  Strides of
    dimensions with one entry say nothing."""
    how = _KINDS.get(kind)
    if how is None:
        _fail_kind(kind)
    per, block, rows, dtype = how
    row, blocks, cols = K // per, K // block, N // rows
    if q is None or s is None or q.dtype is not torch.uint8 or s.dtype is not dtype or q.shape != (N, row) \
            or s.dim() != 2 or q.get_device() != index or s.get_device() != index:
        _fail_weight(q, s, names, kind, (N, row), (blocks, cols), dtype, index)
    (ld, unit), (ld_s, unit_s), (have, width) = q.stride(), s.stride(), s.shape
    if unit != 1 or (unit_s != 1 and width > 1) or have != blocks or width < cols:
        _fail_weight(q, s, names, kind, (N, row), (blocks, cols), dtype, index)
    if N == 1:
        ld = (row + 15) // 16 * 16
    if blocks == 1:
        ld_s = width if rows == 1 else (cols + 15) // 16 * 16
    return q.data_ptr(), ld, s.data_ptr(), ld_s


def _experts(q, s, names, kind, E, N, K, index):
    """The same of E experts' weights [E, N, K], strides between experts first."""
    how = _KINDS.get(kind)
    if how is None:
        _fail_kind(kind)
    per, block, rows, dtype = how
    row, blocks, cols = K // per, K // block, N // rows
    if q is None or s is None or q.dtype is not torch.uint8 or s.dtype is not dtype or q.shape != (E, N, row) \
            or s.dim() != 3 or q.get_device() != index or s.get_device() != index:
        _fail_weight(q, s, names, kind, (E, N, row), (E, blocks, cols), dtype, index)
    (each, ld, unit), (each_s, ld_s, unit_s), (experts, have, width) = q.stride(), s.stride(), s.shape
    if unit != 1 or (unit_s != 1 and width > 1) or have != blocks or width < cols or experts != E:
        _fail_weight(q, s, names, kind, (E, N, row), (E, blocks, cols), dtype, index)
    if blocks == 1:
        ld_s = width if rows == 1 else (cols + 15) // 16 * 16
    if E == 1:
        each = each_s = 0
    return q.data_ptr(), each, ld, s.data_ptr(), each_s, ld_s


def _fail_kind(kind):
    raise ValueError(f"kind must be BS_WEIGHT_E4M3_128X128, BS_WEIGHT_MXFP8 or BS_WEIGHT_MXFP4, got {kind!r}")


def _empty(x, stream, shape, dtype):
    """A tensor for the call from the pool of its stream, on x's GPU."""
    if stream is None:
        return x.new_empty(shape) if dtype is torch.bfloat16 else x.new_empty(shape, dtype=dtype)
    return _new(stream, shape, dtype, x.device)


def bs_mx4_quant_1x32(x, q, s, y=None, stream=None):
    """MXFP4 quantizer of weights: x [R, C] bf16 -> q [R, C/2] uint8 (column 2j
    in the low four bits of byte j), s [C/32, >= R] uint8 (empty_mx_scales)
    and, if given, y [R, C] bf16, the values that the codes stand for."""
    bf16 = torch.bfloat16
    R, C = _first(x, "x", bf16)
    p, ld = _matrix(x, "x", bf16, R, C)
    index = x.get_device()
    if s is None or s.dtype is not torch.uint8 or s.dim() != 2 or s.shape[0] != C // 32 or s.shape[1] < R \
            or s.stride(1) != 1:
        _mat(s, "s", torch.uint8)
        raise ValueError(f"s must be [{C // 32}, >= {R}], got {list(s.shape)}")
    p_q, ld_q = _matrix(q, "q", torch.uint8, R, C // 2)
    p_y, ld_y = _optional(y, "y", bf16, R, C)
    for t, name in ((q, "q"), (s, "s"), (y, "y")):
        if t is not None and t.get_device() != index:
            _mat(t, name, t.dtype)
            _other_gpu(t, name, index)
    _call("bs_mx4_quant_1x32", index, p, R, C, ld, p_q, ld_q, s.data_ptr() or None,
          s.stride(0) if C > 32 else max(s.shape[1], (R + 15) // 16 * 16) // 16 * 16, p_y, ld_y, _stream_of(x, stream))


def bs_few_mm(x, w, s, kind, residual=None, out=None, out_dtype=torch.bfloat16, stream=None):
    """out [T, N] = residual + x [T, K] w^T for few rows x (bf16), w and s
    weights [N, K] of the given kind; residual [T, N] bf16; out bf16 or fp32."""
    bf16 = torch.bfloat16
    T, K = _first(x, "x", bf16)
    p_x, ld_x = _matrix(x, "x", bf16, T, K)
    index = x.get_device()
    if w is None or w.dim() != 2:
        _mat(w, "w", torch.uint8)
    N = w.shape[0]
    weight = _weight(w, s, ("w", "s"), kind, N, K, index)
    if out is None:
        if out_dtype not in _DT:
            raise ValueError(f"out_dtype must be bfloat16 or float32, got {out_dtype}")
        out = _empty(x, stream, (T, N), out_dtype)
        p_out, ld_out = out.data_ptr() or None, N
    else:
        if out.dtype not in _DT:
            raise ValueError(f"out must be bfloat16 or float32, got {out.dtype}")
        p_out, ld_out = _rows_of(out, "out", out.dtype, T, N, index)
    p_res, ld_res = _rows_of(residual, "residual", bf16, T, N, index)
    _call("bs_few_mm", index, kind, T, N, K, p_x, ld_x, *weight, p_res, ld_res, p_out, ld_out, _DT[out.dtype],
          _stream_of(x, stream))
    return out


def bs_moe_few(x, idx, w, w12, s12, out_proj, s_out, kind, residual=None, out=None, stream=None):
    """out [T, D] = residual + sum_j w[t, j] out_e(silu(a) b), [a | b] = w12_e x,
    e = idx[t, j]: the gated experts of few tokens, x [T, D] bf16.

    idx [T, k] int32 (outside [0, E): not routed) and w [T, k] float32 (None:
    ones), as bs_moe_route gives them; with idx None every token takes the only
    expert.  w12 [E, 2H, D] and out_proj [E, D, H] with scales s12 and s_out of
    the given kind; residual [T, D] bf16; out bf16.  Up to 8 tokens the
    activations between the two products are kept in two bf16 parts.
    """
    bf16 = torch.bfloat16
    T, D = _first(x, "x", bf16)
    p_x, ld_x = _matrix(x, "x", bf16, T, D)
    index = x.get_device()
    if w12 is None or w12.dim() != 3 or w12.shape[1] % 2 != 0:
        raise ValueError(f"w12 must be [E, 2H, D], got {None if w12 is None else list(w12.shape)}")
    E, H = w12.shape[0], w12.shape[1] // 2
    k, p_idx, p_w = 1, None, None
    if idx is not None:
        if idx.dim() != 2 or idx.shape[0] != T:
            raise ValueError(f"idx must be [{T}, k], got {list(idx.shape)}")
        k, p_idx = idx.shape[1], _flat(idx, "idx", torch.int32, idx.shape)
        if idx.get_device() != index:
            _other_gpu(idx, "idx", index)
    elif E != 1:
        raise ValueError(f"idx is required with {E} experts")
    if w is not None:
        p_w = _flat(w, "w", torch.float32, (T, k))
        if w.get_device() != index:
            _other_gpu(w, "w", index)
    up = _experts(w12, s12, ("w12", "s12"), kind, E, 2 * H, D, index)
    down = _experts(out_proj, s_out, ("out_proj", "s_out"), kind, E, D, H, index)
    p_res, ld_res = _rows_of(residual, "residual", bf16, T, D, index)
    if out is None:
        out = _empty(x, stream, (T, D), bf16)
        p_out, ld_out = out.data_ptr() or None, D
    else:
        p_out, ld_out = _rows_of(out, "out", bf16, T, D, index)
    nbytes = _lib.load().bs_moe_few_full_workspace_bytes(T, D, H, E, k)
    workspace = _empty(x, stream, (nbytes // 2,), bf16)
    _call("bs_moe_few", index, kind, T, D, H, E, k, p_x, ld_x, p_idx, p_w, *up, *down, p_res, ld_res, p_out, ld_out,
          workspace.data_ptr() or None, nbytes, _stream_of(x, stream))
    return out


def _plan(fn, names, *sizes):
    values = (ctypes.c_int64 * len(names))()
    _check(getattr(_lib.load(), fn)(*sizes, ctypes.addressof(values)), fn)
    return dict(zip(names, values))


def bs_diag_few_mm_plan(kind, T, N, K):
    """What bs_few_mm runs for these sizes (host only): rows of x and tiles of 16
    columns of a workgroup, workgroups along the columns, threads of one."""
    return _plan("bs_diag_few_mm_plan", ("rows", "tiles", "workgroups", "threads"), kind, T, N, K)


def bs_diag_moe_few_plan(kind, T, D, H, E, k):
    """What bs_moe_few runs for these sizes (host only): tokens of an item and
    items of 64 tokens, at most; tiles of h that a wave streams at a time (0: a
    workgroup's waves share one) and the waves that they are spread over; tiles
    of the output of a workgroup and workgroups that share them."""
    return _plan("bs_diag_moe_few_plan", ("tokens", "items", "up_tiles", "up_waves", "out_tiles", "splits"), kind, T, D, H, E, k)
