"""Thin Python binding of the C ABI's entry points around the experts' products
of an MoE block (include/bs.h): router, dispatch, combine, residual norms, and
the gated activation with an 8-bit checkpoint.

Same conventions as ``binding``: argument marshalling only, tensors in the
wrong layout raise ``ValueError`` instead of being copied.  Outputs that are
not passed are allocated; workspaces are allocated per call, so that calls on
different streams never share one.  Both come from the pool of the stream that
is passed, the current one without.
"""

from collections import namedtuple

import torch

from . import _lib
from .binding import BS_OUT_BF16, BS_OUT_F32, _check, _mat, _require, _scale

BS_SCORE_SOFTMAX = 0
BS_SCORE_SIGMOID = 1

_DT = {torch.bfloat16: BS_OUT_BF16, torch.float32: BS_OUT_F32}


class MoEPlan(namedtuple("MoEPlan", ["group_end", "counts", "slot_row", "row_slot"])):
    """group_end, counts [E]; slot_row [T, k]; row_slot [M] -- int32, see
    bs_moe_plan.  ``align``: the rows that each group is padded to a multiple
    of (None where that is not known); no element of the tuple."""

    align = None

    def __new__(cls, group_end, counts, slot_row, row_slot, align=None):
        plan = super().__new__(cls, group_end, counts, slot_row, row_slot)
        plan.align = align
        return plan


#: gradients of bs_resid_norm; None for what was not asked for
ResidNormGrads = namedtuple("ResidNormGrads", ["dx", "du", "dw_pre", "dw_post", "dgate"])


# The helpers below return what the C call takes (addresses as integers, row
# strides) and keep the common case to one comparison of the tensor's type,
# device, shape and strides: a single token's call costs as much on the host
# as on the GPU, so a message is only put together once a check has failed.

def _stream_of(t, stream):
    """Raw stream: the given one, or the current one of t's device."""
    return torch._C._cuda_getCurrentRawStream(t.get_device()) if stream is None else stream.cuda_stream


def _new(stream, shape, dtype, device, zero=False):
    """A tensor from the pool of the stream that the kernel will run on, so
    that its memory is not handed out again before the kernel is through."""
    make = torch.zeros if zero else torch.empty
    if stream is None:
        return make(shape, dtype=dtype, device=device)
    with torch.cuda.stream(stream):
        return make(shape, dtype=dtype, device=device)


def _fail_matrix(t, name, dtype, R, C):
    _mat(t, name, dtype)
    raise ValueError(f"{name} must be [{R}, {C}], got {list(t.shape)}")


def _matrix(t, name, dtype, R, C):
    """(address, row stride) of a row-major [R, C] GPU matrix."""
    if t is None or t.dtype is not dtype or not t.is_cuda or t.shape != (R, C):
        _fail_matrix(t, name, dtype, R, C)
    ld, unit = t.stride()
    if unit != 1 and C > 1 and R > 0:
        _mat(t, name, dtype)
    # the strides of no row, and that of an only one, say nothing: its length stands for it
    return t.data_ptr() or None, ld if R > 1 else (C + 15) // 16 * 16


def _optional(t, name, dtype, R, C):
    return (None, 0) if t is None else _matrix(t, name, dtype, R, C)


def _first(t, name, dtype):
    """Shape of the matrix that gives a call its sizes."""
    if t is None or t.dtype is not dtype or not t.is_cuda or t.dim() != 2:
        _mat(t, name, dtype)
    return t.shape


def _fail_flat(t, name, dtype, shape):
    _require(t is not None, f"{name} is required")
    _require(t.dtype == dtype, f"{name} must be {dtype}, got {t.dtype}")
    _require(t.is_cuda, f"{name} must be a GPU tensor")
    _require(t.shape == shape, f"{name} must have shape {list(shape)}, got {list(t.shape)}")
    raise ValueError(f"{name} must be contiguous; got strides {t.stride()}")


def _flat(t, name, dtype, shape):
    """Address of a contiguous GPU tensor of the given shape."""
    if t is None or t.dtype is not dtype or not t.is_cuda or t.shape != shape or not t.is_contiguous():
        _fail_flat(t, name, dtype, shape)
    return t.data_ptr() or None


def _index(t, name, dims):
    """Shape and address of a contiguous int32 GPU tensor."""
    _require(t is not None, f"{name} is required")
    if t.dim() != dims:
        raise ValueError(f"{name} must be {'[T, k]' if dims == 2 else '1-D'}, got {list(t.shape)}")
    return t.shape, _flat(t, name, torch.int32, t.shape)


def _scales(t, name, nkb, count):
    """(address, row stride) of a K-major scale tensor [nkb, >= count]."""
    if t is None or t.dtype is not torch.float32 or not t.is_cuda or t.dim() != 2 or t.shape[0] != nkb \
            or t.shape[1] < count or t.stride(1) != 1:
        _scale(t, name, nkb, count)
    return t.data_ptr() or None, t.stride(0)


def _codes(R, C, q_row, s_row, q_col, s_col):
    """C arguments of the row and column outputs of an [R, C] matrix."""
    u8 = torch.uint8
    row = col = (None, 0, None, 0)
    if q_row is not None or s_row is not None:
        row = _matrix(q_row, "q_row", u8, R, C) + _scales(s_row, "s_row", C // 128, R)
    if q_col is not None or s_col is not None:
        col = _matrix(q_col, "q_col", u8, C, R) + _scales(s_col, "s_col", R // 128, C)
    return row + col


# ----------------------------------------------------------------------------
# router
# ----------------------------------------------------------------------------

def _logits(t, name):
    if t is None or t.dtype not in _DT:
        raise ValueError(f"{name} must be bfloat16 or float32")
    T, E = _first(t, name, t.dtype)
    return (T, E) + _matrix(t, name, t.dtype, T, E)


def bs_moe_route(logits, k, bias=None, score=BS_SCORE_SOFTMAX, n_group=1, topk_group=1, group_best=1,
                 renormalize=True, scale=1.0, idx=None, w=None, stream=None):
    """k experts per token and their weights: (idx [T, k] int32, w [T, k] float32).

    logits [T, E] bf16 or fp32 (-inf masks an expert); bias [E] fp32 enters the
    choice only.  n_group groups of consecutive experts, of which the topk_group
    with the largest sum of their group_best best scores stay.  idx is -1 and w
    0 where no expert is left to choose.
    """
    T, E, p, ld = _logits(logits, "logits")
    if k < 1:
        raise ValueError(f"k={k} must be >= 1")
    if idx is None:
        idx = _new(stream, (T, k), torch.int32, logits.device)
    if w is None:
        w = _new(stream, (T, k), torch.float32, logits.device)
    _check(_lib.load().bs_moe_route(
        p, _DT[logits.dtype], T, E, ld, None if bias is None else _flat(bias, "bias", torch.float32, (E,)), score, k,
        n_group, topk_group, group_best, int(renormalize), scale, _flat(idx, "idx", torch.int32, (T, k)),
        _flat(w, "w", torch.float32, (T, k)), _stream_of(logits, stream)), "bs_moe_route")
    return idx, w


def bs_moe_route_bwd(logits, idx, w, dw, score=BS_SCORE_SOFTMAX, renormalize=True, scale=1.0, out=None, stream=None):
    """dlogits [T, E] (the type of logits) from the gradient dw [T, k] of the weights."""
    T, E, p, ld = _logits(logits, "logits")
    (_, k), p_idx = _index(idx, "idx", 2)
    shape = (T, k)
    if out is None:
        out = _new(stream, (T, E), logits.dtype, logits.device)
    if idx.shape[0] != T:
        _fail_flat(idx, "idx", torch.int32, shape)
    _check(_lib.load().bs_moe_route_bwd(
        p, _DT[logits.dtype], T, E, ld, score, k, int(renormalize), scale, p_idx,
        _flat(w, "w", torch.float32, shape), _flat(dw, "dw", torch.float32, shape),
        *_matrix(out, "out", logits.dtype, T, E), _stream_of(logits, stream)), "bs_moe_route_bwd")
    return out


# ----------------------------------------------------------------------------
# dispatch and combine
# ----------------------------------------------------------------------------

def bs_moe_plan_rows(T, k, E, align=128):
    """Rows that hold every group padded to ``align``, whatever the routing."""
    return _lib.load().bs_moe_plan_rows(T, k, E, align)


def bs_moe_plan(idx, E, align=128, M=None, stream=None):
    """Sort of the slots (token, choice) by expert: a MoEPlan of device tensors.

    idx [T, k] int32, values outside [0, E) are not routed.  M: rows of the
    expert-ordered matrices, bs_moe_plan_rows by default.
    """
    (T, k), p_idx = _index(idx, "idx", 2)
    lib = _lib.load()
    if M is None:
        M = lib.bs_moe_plan_rows(T, k, E, align)
    if E < 1 or M < 0:
        raise ValueError(f"E={E} must be >= 1 and M={M} >= 0")
    # one allocation: the workspace, then the four arrays
    nbytes = lib.bs_moe_plan_workspace_bytes(T, k, E)
    n, nw = T * k, nbytes // 4
    buf = _new(stream, nw + 2 * E + n + M, torch.int32, idx.device)
    base = buf.data_ptr()
    at = base + nbytes
    _check(lib.bs_moe_plan(p_idx, T, k, E, align, M, at, at + 4 * E, at + 8 * E, at + 8 * E + 4 * n,
                           base if nbytes else None, nbytes, _stream_of(idx, stream)), "bs_moe_plan")
    _, group_end, counts, slot_row, row_slot = buf.split_with_sizes([nw, E, E, n, M])
    return MoEPlan(group_end, counts, slot_row.view(T, k), row_slot, align)


def bs_moe_gather_quant_1x128(x, row_slot, k, w=None, y=None, q_row=None, s_row=None, q_col=None, s_col=None,
                              stream=None):
    """Rows of x [T, D] in expert order, times w [T, k] if given: bf16 rows y
    [M, D] and/or their 1x128 codes along rows and transposed columns, outputs
    as in bs_quant_1x128."""
    bf16 = torch.bfloat16
    T, D = _first(x, "x", bf16)
    (M,), p_slot = _index(row_slot, "row_slot", 1)
    p, ld = _matrix(x, "x", bf16, T, D)
    _check(_lib.load().bs_moe_gather_quant_1x128(
        p, T, D, ld, k, p_slot, M, None if w is None else _flat(w, "w", torch.float32, (T, k)),
        *_optional(y, "y", bf16, M, D), *_codes(M, D, q_row, s_row, q_col, s_col), _stream_of(x, stream)),
        "bs_moe_gather_quant_1x128")


def bs_moe_combine(y, slot_row, w=None, residual=None, out=None, stream=None):
    """out [T, D] = residual + sum over the slots of w [T, k] (ones if None)
    times the rows slot_row [T, k] of y [M, D]; fp32 sum, bf16 out."""
    bf16 = torch.bfloat16
    M, D = _first(y, "y", bf16)
    (T, k), p_row = _index(slot_row, "slot_row", 2)
    if out is None:
        out = _new(stream, (T, D), bf16, y.device)
    p, ld = _matrix(y, "y", bf16, M, D)
    _check(_lib.load().bs_moe_combine(
        p, M, D, ld, p_row, None if w is None else _flat(w, "w", torch.float32, (T, k)), T, k,
        *_optional(residual, "residual", bf16, T, D), *_matrix(out, "out", bf16, T, D), _stream_of(y, stream)),
        "bs_moe_combine")
    return out


def bs_moe_combine_dw(dout, y, slot_row, dw=None, stream=None):
    """dw [T, k] = <dout [T, D] of the token, row slot_row of y [M, D]>, fp32."""
    bf16 = torch.bfloat16
    M, D = _first(y, "y", bf16)
    (T, k), p_row = _index(slot_row, "slot_row", 2)
    if dw is None:
        dw = _new(stream, (T, k), torch.float32, y.device)
    p_dout, ld_dout = _matrix(dout, "dout", bf16, T, D)
    p, ld = _matrix(y, "y", bf16, M, D)
    _check(_lib.load().bs_moe_combine_dw(p_dout, T, D, ld_dout, p, M, ld, p_row, k,
                                         _flat(dw, "dw", torch.float32, (T, k)), _stream_of(y, stream)),
           "bs_moe_combine_dw")
    return dw


# ----------------------------------------------------------------------------
# residual norms
# ----------------------------------------------------------------------------

def _norm_params(R, D, w_pre, w_post, gate):
    """(address of w_pre, of w_post, of gate, ld_gate, rows_per_gate, type)."""
    some = w_pre if w_pre is not None else w_post if w_post is not None else gate
    if some is None:
        return None, None, None, 0, R, BS_OUT_F32
    dt = some.dtype
    if dt not in _DT:
        raise ValueError(f"w_pre, w_post and gate must be bfloat16 or float32, got {dt}")
    p_gate, ld_gate, per = None, 0, R
    if gate is not None:
        B = _first(gate, "gate", dt)[0]
        p_gate, ld_gate = _matrix(gate, "gate", dt, B, D)
        if R % B != 0 if B else R != 0:
            raise ValueError(f"the {R} rows must be a multiple of the gate's {B}")
        per = max(R // B, 1) if B else 1
    return (None if w_pre is None else _flat(w_pre, "w_pre", dt, (D,)),
            None if w_post is None else _flat(w_post, "w_post", dt, (D,)), p_gate, ld_gate, per, _DT[dt])


def bs_resid_norm(x, w_pre=None, u=None, w_post=None, gate=None, alpha=1.0, eps=1e-6, r=None, h=None, rstd_u=None,
                  rstd_r=None, q_row=None, s_row=None, q_col=None, s_col=None, stream=None):
    """r = x + alpha gate N(u) w_post and h = N(r) w_pre (r = x without u), into
    the outputs given: r, h [R, D] bf16, rstd_u, rstd_r [R] fp32, and the 1x128
    codes of h as in bs_quant_1x128.

    x, u [R, D] bf16; w_pre, w_post [D] and gate [B, D] of one type, bf16 or
    fp32; consecutive R / B rows share a row of the gate.
    """
    bf16, f32 = torch.bfloat16, torch.float32
    R, D = _first(x, "x", bf16)
    p_pre, p_post, p_gate, ld_gate, per, dt = _norm_params(R, D, w_pre, w_post, gate)
    p_x, ld_x = _matrix(x, "x", bf16, R, D)
    p_u, ld_u = _optional(u, "u", bf16, R, D)
    _check(_lib.load().bs_resid_norm(
        p_x, p_u, R, D, ld_x, ld_u, p_post, p_gate, ld_gate, per, p_pre, dt, alpha, eps,
        *_optional(r, "r", bf16, R, D), None if rstd_u is None else _flat(rstd_u, "rstd_u", f32, (R,)),
        None if rstd_r is None else _flat(rstd_r, "rstd_r", f32, (R,)), *_optional(h, "h", bf16, R, D),
        *_codes(R, D, q_row, s_row, q_col, s_col), _stream_of(x, stream)), "bs_resid_norm")


def bs_resid_norm_bwd(r, rstd_r, w_pre, dh, dr=None, u=None, rstd_u=None, w_post=None, gate=None, alpha=1.0,
                      stream=None):
    """ResidNormGrads from dh [R, D] and dr [R, D] (None: zeros): dx, du [R, D]
    bf16, dw_pre, dw_post [D] and dgate [B, D] fp32.  r: the saved r (x without
    u).  Without w_pre (no norm of r) r, rstd_r and dh are None."""
    bf16, f32 = torch.bfloat16, torch.float32
    some = dr if r is None else r
    R, D = _first(some, "dr" if r is None else "r", bf16)
    p_pre, p_post, p_gate, ld_gate, per, dt = _norm_params(R, D, w_pre, w_post, gate)
    dev = some.device
    dx = _new(stream, (R, D), bf16, dev)
    du = _new(stream, (R, D), bf16, dev) if u is not None else None
    none = R == 0     # no rows: the sums are zero
    dw_pre = _new(stream, D, f32, dev, none) if w_pre is not None else None
    dw_post = _new(stream, D, f32, dev, none) if w_post is not None else None
    dgate = _new(stream, (gate.shape[0], D), f32, dev, none) if gate is not None else None
    grads = ResidNormGrads(dx, du, dw_pre, dw_post, dgate)
    if none:
        return grads
    lib = _lib.load()
    nbytes = lib.bs_resid_norm_bwd_workspace_bytes(R, D, per)
    ws = _new(stream, max(nbytes, 16), torch.uint8, dev)
    p_r, ld_r = _optional(r, "r", bf16, R, D)
    p_u, ld_u = _optional(u, "u", bf16, R, D)
    p_dh, ld_dh = _optional(dh, "dh", bf16, R, D)
    p_dr, ld_dr = _optional(dr, "dr", bf16, R, D)
    ptr = lambda t: None if t is None else t.data_ptr()  # noqa: E731
    _check(lib.bs_resid_norm_bwd(
        p_r, p_u, p_dh, p_dr, R, D, ld_r, ld_u, ld_dh, ld_dr, p_post, p_gate, ld_gate, per, p_pre, dt, alpha,
        None if w_post is None else _flat(rstd_u, "rstd_u", f32, (R,)),
        None if w_pre is None else _flat(rstd_r, "rstd_r", f32, (R,)), dx.data_ptr(), D, ptr(du), D if u is not None else 0,
        ptr(dw_pre), ptr(dw_post), ptr(dgate), ws.data_ptr(), nbytes, _stream_of(some, stream)), "bs_resid_norm_bwd")
    return grads


# ----------------------------------------------------------------------------
# gated activation with an 8-bit checkpoint
# ----------------------------------------------------------------------------

def bs_swiglu_quant_1x128_ckpt(a, b, ck, s_ck, q_row=None, s_row=None, q_col=None, s_col=None, stream=None):
    """bs_swiglu_quant_1x128 that also writes the 1x128 row codes of a and b
    for the backward: ck [R, 2C] uint8 (a then b), s_ck [2C/128, >= R]."""
    bf16 = torch.bfloat16
    R, C = _first(a, "a", bf16)
    p_a, ld_a = _matrix(a, "a", bf16, R, C)
    p_b, ld_b = _matrix(b, "b", bf16, R, C)
    _check(_lib.load().bs_swiglu_quant_1x128_ckpt(
        p_a, p_b, R, C, ld_a, ld_b, *_matrix(ck, "ck", torch.uint8, R, 2 * C), *_scales(s_ck, "s_ck", 2 * C // 128, R),
        *_codes(R, C, q_row, s_row, q_col, s_col), _stream_of(a, stream)), "bs_swiglu_quant_1x128_ckpt")


def bs_swiglu_bwd_quant_1x128_ckpt(ck, s_ck, dh, q_row=None, s_row=None, q_col=None, s_col=None, stream=None):
    """bs_swiglu_bwd_quant_1x128 from the checkpoint (ck, s_ck): the codes of
    [da | db] [R, 2C], rows and/or transposed columns."""
    bf16 = torch.bfloat16
    R, C = _first(dh, "dh", bf16)
    p_ck, ld_ck = _matrix(ck, "ck", torch.uint8, R, 2 * C)
    _check(_lib.load().bs_swiglu_bwd_quant_1x128_ckpt(
        p_ck, R, C, ld_ck, *_scales(s_ck, "s_ck", 2 * C // 128, R), *_matrix(dh, "dh", bf16, R, C),
        *_codes(R, 2 * C, q_row, s_row, q_col, s_col), _stream_of(dh, stream)), "bs_swiglu_bwd_quant_1x128_ckpt")
