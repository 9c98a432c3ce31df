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

import torch

from . import _lib
from .binding import BS_OUT_BF16, _check, _mat, _require
from .binding_block import _DT, _first, _flat, _matrix, _new, _optional, _scales, _stream_of

BS_WEIGHT_E4M3_128X128 = 0
BS_WEIGHT_MXFP8 = 1
BS_WEIGHT_MXFP4 = 2

_KINDS = (BS_WEIGHT_E4M3_128X128, BS_WEIGHT_MXFP8, BS_WEIGHT_MXFP4)


def _call(fn, device, *args):
    """Calls the library with the tensors' device as the current one."""
    call = getattr(_lib.load(), fn)
    if torch._C._cuda_getDevice() == device.index:
        _check(call(*args), fn)
    else:
        with torch.cuda.device(device):
            _check(call(*args), fn)


def _one_device(device, **tensors):
    for name, t in tensors.items():
        if t is not None and t.device != device:
            raise ValueError(f"{name} is on {t.device}, x on {device}: all tensors must be on one GPU")


def _out_matrix(t, name, dtype, R, C):
    """(address, row stride) of a row-major matrix whose rows need no alignment."""
    p, ld = _matrix(t, name, dtype, R, C)
    return p, ld if R > 1 else C


def _weight(q, s, name, s_name, kind, N, K, experts=None):
    """C arguments of weights [N, K] (or [experts, N, K]): codes, their
    strides, scales and theirs."""
    if kind not in _KINDS:
        raise ValueError(f"kind must be one of BS_WEIGHT_E4M3_128X128, BS_WEIGHT_MXFP8 and BS_WEIGHT_MXFP4, got {kind!r}")
    row = K // 2 if kind == BS_WEIGHT_MXFP4 else K
    blocks, cols, dtype = (K // 128, N // 128, torch.float32) if kind == BS_WEIGHT_E4M3_128X128 else (K // 32, N, torch.uint8)
    lead = () if experts is None else (experts,)
    _mat(q, name, torch.uint8, len(lead) + 2)
    _require(tuple(q.shape) == lead + (N, row), f"{name} must be {list(lead + (N, row))}, got {list(q.shape)}")
    _mat(s, s_name, dtype, len(lead) + 2)
    _require(tuple(s.shape[:-1]) == lead + (blocks,) and s.shape[-1] >= cols,
             f"{s_name} must be {list(lead + (blocks,))} x >= {cols} (K-major), got {list(s.shape)}")
    # strides of dimensions with one entry say nothing
    ld = q.stride(-2) if N > 1 else (row + 15) // 16 * 16
    ld_s = s.stride(-2) if blocks > 1 else s.shape[-1]
    p, p_s = q.data_ptr() or None, s.data_ptr() or None
    if experts is None:
        return p, ld, p_s, ld_s
    many = experts > 1
    return p, (q.stride(0) if many else 0), ld, p_s, (s.stride(0) if many else 0), ld_s


def bs_mx4_quant_1x32(x, q, s, y=None, stream=None):
    """MXFP4 quantizer of weights: x [R, C] bf16 -> q [R, C/2] uint8 (column 2j
    in the low four bits of byte j), s [C/32, >= R] uint8 (empty_mx_scales)
    and, if given, y [R, C] bf16, the values that the codes stand for."""
    bf16 = torch.bfloat16
    R, C = _first(x, "x", bf16)
    _one_device(x.device, q=q, s=s, y=y)
    _mat(s, "s", torch.uint8)
    _require(s.shape[0] == C // 32 and s.shape[1] >= R, f"s must be [{C // 32}, >= {R}], got {list(s.shape)}")
    ld_s = s.stride(0) if s.shape[0] > 1 else s.shape[1] // 16 * 16 if s.shape[1] // 16 * 16 >= R else s.stride(0)
    _call("bs_mx4_quant_1x32", x.device, *_first_args(x, R, C), *_matrix(q, "q", torch.uint8, R, C // 2),
          s.data_ptr() or None, ld_s, *_optional(y, "y", bf16, R, C), _stream_of(x, stream))


def _first_args(x, R, C):
    p, ld = _matrix(x, "x", torch.bfloat16, R, C)
    return p, R, C, ld


def bs_few_mm(x, w, s, kind, residual=None, out=None, out_dtype=torch.bfloat16, stream=None):
    """out [T, N] = residual + x [T, K] w^T for few rows x (bf16), w and s
    weights [N, K] of the given kind; residual [T, N] bf16; out bf16 or fp32."""
    bf16 = torch.bfloat16
    T, K = _first(x, "x", bf16)
    if w is None or w.dim() != 2:
        _mat(w, "w", torch.uint8)
    N = w.shape[0]
    if out is None:
        if out_dtype not in _DT:
            raise ValueError(f"out_dtype must be bfloat16 or float32, got {out_dtype}")
        out = _new(stream, (T, N), out_dtype, x.device)
    elif out.dtype not in _DT:
        raise ValueError(f"out must be bfloat16 or float32, got {out.dtype}")
    _one_device(x.device, w=w, s=s, residual=residual, out=out)
    p_x, ld_x = _matrix(x, "x", bf16, T, K)
    _call("bs_few_mm", x.device, kind, T, N, K, p_x, ld_x, *_weight(w, s, "w", "s", kind, N, K),
          *((None, 0) if residual is None else _out_matrix(residual, "residual", bf16, T, N)),
          *_out_matrix(out, "out", out.dtype, T, N), _DT[out.dtype], _stream_of(x, stream))
    return out


def bs_moe_few(x, idx, w, w12, s12, out_proj, s_out, kind, residual=None, out=None, stream=None):
    """out [T, D] = residual + sum_j w[t, j] out_e(silu(a) b), [a | b] = w12_e x,
    e = idx[t, j]: the gated experts of few tokens, x [T, D] bf16.

    idx [T, k] int32 (outside [0, E): not routed) and w [T, k] float32 (None:
    ones), as bs_moe_route gives them; with idx None every token takes the only
    expert.  w12 [E, 2H, D] and out_proj [E, D, H] with scales s12 and s_out of
    the given kind; residual [T, D] bf16; out bf16.
    """
    bf16 = torch.bfloat16
    T, D = _first(x, "x", bf16)
    if w12 is None or w12.dim() != 3 or w12.shape[1] % 2 != 0:
        raise ValueError(f"w12 must be [E, 2H, D], got {None if w12 is None else list(w12.shape)}")
    E, H = w12.shape[0], w12.shape[1] // 2
    if idx is None:
        k, p_idx = 1, None
        _require(E == 1, f"idx is required with {E} experts")
    else:
        _require(idx.dim() == 2 and idx.shape[0] == T, f"idx must be [{T}, k], got {list(idx.shape)}")
        k, p_idx = idx.shape[1], _flat(idx, "idx", torch.int32, idx.shape)
    if out is None:
        out = _new(stream, (T, D), bf16, x.device)
    _one_device(x.device, idx=idx, w=w, w12=w12, s12=s12, out_proj=out_proj, s_out=s_out, residual=residual, out=out)
    p_x, ld_x = _matrix(x, "x", bf16, T, D)
    nbytes = _lib.load().bs_moe_few_workspace_bytes(T, k, H)
    h = _new(stream, nbytes, torch.uint8, x.device)
    _call("bs_moe_few", x.device, kind, T, D, H, E, k, p_x, ld_x, p_idx,
          None if w is None else _flat(w, "w", torch.float32, (T, k)), *_weight(w12, s12, "w12", "s12", kind, 2 * H, D, E),
          *_weight(out_proj, s_out, "out_proj", "s_out", kind, D, H, E),
          *((None, 0) if residual is None else _out_matrix(residual, "residual", bf16, T, D)),
          *_out_matrix(out, "out", bf16, T, D), h.data_ptr() or None, nbytes, _stream_of(x, stream))
    return out
