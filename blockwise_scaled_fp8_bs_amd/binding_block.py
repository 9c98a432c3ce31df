"""Thin Python binding of the C ABI's entry points around the experts' products
of an MoE block (include/bs.h): router, dispatch, combine, residual norms, and
the gated activation with an 8-bit checkpoint.

Same conventions as ``binding``: argument marshalling only, tensors in the
wrong layout raise ``ValueError`` instead of being copied.  Outputs that are
not passed are allocated; workspaces are allocated per call, so that calls on
different streams never share one.
"""

from collections import namedtuple

import torch

from . import _lib
from .binding import BS_OUT_BF16, BS_OUT_F32, _check, _ld, _mat, _ptr, _require, _scale, _stream

BS_SCORE_SOFTMAX = 0
BS_SCORE_SIGMOID = 1

_DT = {torch.bfloat16: BS_OUT_BF16, torch.float32: BS_OUT_F32}

#: group_end, counts [E]; slot_row [T, k]; row_slot [M] -- int32, see bs_moe_plan
MoEPlan = namedtuple("MoEPlan", ["group_end", "counts", "slot_row", "row_slot"])

#: gradients of bs_resid_norm; None for what was not asked for
ResidNormGrads = namedtuple("ResidNormGrads", ["dx", "du", "dw_pre", "dw_post", "dgate"])


def _flat(t, name, dtype, shape):
    """A contiguous GPU tensor of the given type and shape (None in the shape: any)."""
    _require(t is not None, f"{name} is required")
    _require(t.dtype == dtype, f"{name} must be {dtype}, got {t.dtype}")
    _require(t.is_cuda, f"{name} must be a GPU tensor")
    _require(t.dim() == len(shape) and all(n is None or n == m for n, m in zip(shape, t.shape)),
             f"{name} must have shape {list(shape)}, got {list(t.shape)}")
    _require(t.is_contiguous(), f"{name} must be contiguous; got strides {t.stride()}")
    return t


def _bf16(t, name, R, D):
    _mat(t, name, torch.bfloat16)
    _require(tuple(t.shape) == (R, D), f"{name} must be [{R}, {D}], got {list(t.shape)}")
    # the stride of an only row says nothing: its length stands for it
    return _ld(t) if R > 1 else (D + 7) // 8 * 8


def _codes(R, C, q_row, s_row, q_col, s_col):
    """C arguments of the row and column outputs of an [R, C] matrix."""
    args = [None, 0, None, 0, None, 0, None, 0]
    if q_row is not None or s_row is not None:
        _mat(q_row, "q_row", torch.uint8)
        _require(tuple(q_row.shape) == (R, C), f"q_row must be [{R}, {C}]")
        args[0:4] = [_ptr(q_row), _ld(q_row), _ptr(s_row), _scale(s_row, "s_row", C // 128, R)]
    if q_col is not None or s_col is not None:
        _mat(q_col, "q_col", torch.uint8)
        _require(tuple(q_col.shape) == (C, R), f"q_col must be the transpose [{C}, {R}]")
        args[4:8] = [_ptr(q_col), _ld(q_col), _ptr(s_col), _scale(s_col, "s_col", R // 128, C)]
    return args


# ----------------------------------------------------------------------------
# router
# ----------------------------------------------------------------------------

def _logits(t, name):
    _require(t is not None and t.dtype in _DT, f"{name} must be bfloat16 or float32")
    _mat(t, name, t.dtype)
    T, E = t.shape
    return T, E, _ld(t) if T > 1 else E


def bs_moe_route(logits, k, bias=None, score=BS_SCORE_SOFTMAX, n_group=1, topk_group=1, group_best=1,
                 renormalize=True, scale=1.0, idx=None, w=None, stream=None):
    """k experts per token and their weights: (idx [T, k] int32, w [T, k] float32).

    logits [T, E] bf16 or fp32 (-inf masks an expert); bias [E] fp32 enters the
    choice only.  n_group groups of consecutive experts, of which the topk_group
    with the largest sum of their group_best best scores stay.  idx is -1 and w
    0 where no expert is left to choose.
    """
    T, E, ld = _logits(logits, "logits")
    if bias is not None:
        _flat(bias, "bias", torch.float32, (E,))
    idx = torch.empty((T, k), dtype=torch.int32, device=logits.device) if idx is None else \
        _flat(idx, "idx", torch.int32, (T, k))
    w = torch.empty((T, k), dtype=torch.float32, device=logits.device) if w is None else \
        _flat(w, "w", torch.float32, (T, k))
    _check(_lib.load().bs_moe_route(_ptr(logits), _DT[logits.dtype], T, E, ld, _ptr(bias), score, k, n_group,
                                    topk_group, group_best, int(renormalize), scale, _ptr(idx), _ptr(w),
                                    _stream(stream)), "bs_moe_route")
    return idx, w


def bs_moe_route_bwd(logits, idx, w, dw, score=BS_SCORE_SOFTMAX, renormalize=True, scale=1.0, out=None, stream=None):
    """dlogits [T, E] (the type of logits) from the gradient dw [T, k] of the weights."""
    T, E, ld = _logits(logits, "logits")
    _require(idx is not None and idx.dim() == 2, "idx must be [T, k]")
    k = idx.shape[1]
    _flat(idx, "idx", torch.int32, (T, k))
    _flat(w, "w", torch.float32, (T, k))
    _flat(dw, "dw", torch.float32, (T, k))
    if out is None:
        out = torch.empty((T, E), dtype=logits.dtype, device=logits.device)
    _mat(out, "out", logits.dtype)
    _require(tuple(out.shape) == (T, E), f"out must be [{T}, {E}]")
    _check(_lib.load().bs_moe_route_bwd(_ptr(logits), _DT[logits.dtype], T, E, ld, score, k, int(renormalize), scale,
                                        _ptr(idx), _ptr(w), _ptr(dw), _ptr(out),
                                        _ld(out) if T > 1 else E, _stream(stream)), "bs_moe_route_bwd")
    return out


# ----------------------------------------------------------------------------
# dispatch and combine
# ----------------------------------------------------------------------------

def bs_moe_plan_rows(T, k, E, align=128):
    """Rows that hold every group padded to ``align``, whatever the routing."""
    return int(_lib.load().bs_moe_plan_rows(T, k, E, align))


def bs_moe_plan(idx, E, align=128, M=None, stream=None):
    """Sort of the slots (token, choice) by expert: a MoEPlan of device tensors.

    idx [T, k] int32, values outside [0, E) are not routed.  M: rows of the
    expert-ordered matrices, bs_moe_plan_rows by default.
    """
    _require(idx is not None and idx.dim() == 2, "idx must be [T, k]")
    _flat(idx, "idx", torch.int32, (None, None))
    T, k = idx.shape
    lib = _lib.load()
    if M is None:
        M = int(lib.bs_moe_plan_rows(T, k, E, align))
    _require(E >= 1 and M >= 0, f"E={E} must be >= 1 and M={M} >= 0")
    dev, i32 = idx.device, torch.int32
    # one allocation for the four arrays; each starts 16-byte aligned
    sizes = [(E + 3) // 4 * 4, (E + 3) // 4 * 4, (T * k + 3) // 4 * 4, M]
    buf = torch.empty(sum(sizes), dtype=i32, device=dev)
    ends, counts, slots, rows = torch.split(buf, sizes)
    plan = MoEPlan(ends[:E], counts[:E], slots[:T * k].view(T, k), rows)
    nbytes = int(lib.bs_moe_plan_workspace_bytes(T, k, E))
    ws = torch.empty(nbytes, dtype=torch.uint8, device=dev) if nbytes else None
    _check(lib.bs_moe_plan(_ptr(idx), T, k, E, align, M, _ptr(plan.group_end), _ptr(plan.counts),
                           _ptr(plan.slot_row), _ptr(plan.row_slot), _ptr(ws), nbytes, _stream(stream)),
           "bs_moe_plan")
    return plan


def bs_moe_gather_quant_1x128(x, row_slot, k, w=None, y=None, q_row=None, s_row=None, q_col=None, s_col=None,
                              stream=None):
    """Rows of x [T, D] in expert order, times w [T, k] if given: bf16 rows y
    [M, D] and/or their 1x128 codes along rows and transposed columns, outputs
    as in bs_quant_1x128."""
    _mat(x, "x", torch.bfloat16)
    T, D = x.shape
    ld_x = _bf16(x, "x", T, D)
    _flat(row_slot, "row_slot", torch.int32, (None,))
    M = row_slot.shape[0]
    if w is not None:
        _flat(w, "w", torch.float32, (T, k))
    _check(_lib.load().bs_moe_gather_quant_1x128(_ptr(x), T, D, ld_x, k, _ptr(row_slot), M, _ptr(w), _ptr(y),
                                                 0 if y is None else _bf16(y, "y", M, D),
                                                 *_codes(M, D, q_row, s_row, q_col, s_col), _stream(stream)),
           "bs_moe_gather_quant_1x128")


def bs_moe_combine(y, slot_row, w=None, residual=None, out=None, stream=None):
    """out [T, D] = residual + sum over the slots of w [T, k] (ones if None)
    times the rows slot_row [T, k] of y [M, D]; fp32 sum, bf16 out."""
    _mat(y, "y", torch.bfloat16)
    M, D = y.shape
    _flat(slot_row, "slot_row", torch.int32, (None, None))
    T, k = slot_row.shape
    if w is not None:
        _flat(w, "w", torch.float32, (T, k))
    if out is None:
        out = torch.empty((T, D), dtype=torch.bfloat16, device=y.device)
    _check(_lib.load().bs_moe_combine(_ptr(y), M, D, _bf16(y, "y", M, D), _ptr(slot_row), _ptr(w), T, k,
                                      _ptr(residual), 0 if residual is None else _bf16(residual, "residual", T, D),
                                      _ptr(out), _bf16(out, "out", T, D), _stream(stream)), "bs_moe_combine")
    return out


def bs_moe_combine_dw(dout, y, slot_row, dw=None, stream=None):
    """dw [T, k] = <dout [T, D] of the token, row slot_row of y [M, D]>, fp32."""
    _mat(dout, "dout", torch.bfloat16)
    _mat(y, "y", torch.bfloat16)
    M, D = y.shape
    _flat(slot_row, "slot_row", torch.int32, (None, None))
    T, k = slot_row.shape
    if dw is None:
        dw = torch.empty((T, k), dtype=torch.float32, device=y.device)
    _flat(dw, "dw", torch.float32, (T, k))
    _check(_lib.load().bs_moe_combine_dw(_ptr(dout), T, D, _bf16(dout, "dout", T, D), _ptr(y), M,
                                         _bf16(y, "y", M, D), _ptr(slot_row), k, _ptr(dw), _stream(stream)),
           "bs_moe_combine_dw")
    return dw


# ----------------------------------------------------------------------------
# residual norms
# ----------------------------------------------------------------------------

def _norm_params(R, D, w_pre, w_post, gate):
    """Checked (dtype, ld_gate, rows_per_gate) of the parameters."""
    dt = None
    for t, name in ((w_pre, "w_pre"), (w_post, "w_post"), (gate, "gate")):
        if t is None:
            continue
        _require(t.dtype in _DT, f"{name} must be bfloat16 or float32, got {t.dtype}")
        _require(dt is None or dt == t.dtype, "w_pre, w_post and gate must have one type")
        dt = t.dtype
        if t is gate:
            _mat(t, name, dt)
            _require(t.shape[1] == D, f"gate must be [B, {D}], got {list(t.shape)}")
        else:
            _flat(t, name, dt, (D,))
    if gate is None:
        return dt, 0, R
    B = gate.shape[0]
    _require(B >= 1 and R % B == 0, f"the {R} rows must be a multiple of the gate's {B}")
    return dt, _ld(gate) if B > 1 else (D + 7) // 8 * 8, R // B


def bs_resid_norm(x, w_pre=None, u=None, w_post=None, gate=None, alpha=1.0, eps=1e-6, r=None, h=None, rstd_u=None,
                  rstd_r=None, q_row=None, s_row=None, q_col=None, s_col=None, stream=None):
    """r = x + alpha gate N(u) w_post and h = N(r) w_pre (r = x without u), into
    the outputs given: r, h [R, D] bf16, rstd_u, rstd_r [R] fp32, and the 1x128
    codes of h as in bs_quant_1x128.

    x, u [R, D] bf16; w_pre, w_post [D] and gate [B, D] of one type, bf16 or
    fp32; consecutive R / B rows share a row of the gate.
    """
    _mat(x, "x", torch.bfloat16)
    R, D = x.shape
    dt, ld_gate, per = _norm_params(R, D, w_pre, w_post, gate)
    for t, name in ((rstd_u, "rstd_u"), (rstd_r, "rstd_r")):
        if t is not None:
            _flat(t, name, torch.float32, (R,))
    ld = lambda t, name: 0 if t is None else _bf16(t, name, R, D)  # noqa: E731
    _check(_lib.load().bs_resid_norm(_ptr(x), _ptr(u), R, D, ld(x, "x"), ld(u, "u"), _ptr(w_post), _ptr(gate),
                                     ld_gate, per, _ptr(w_pre), _DT.get(dt, BS_OUT_F32), alpha, eps, _ptr(r),
                                     ld(r, "r"), _ptr(rstd_u), _ptr(rstd_r), _ptr(h), ld(h, "h"),
                                     *_codes(R, D, q_row, s_row, q_col, s_col), _stream(stream)), "bs_resid_norm")


def bs_resid_norm_bwd(r, rstd_r, w_pre, dh, dr=None, u=None, rstd_u=None, w_post=None, gate=None, alpha=1.0,
                      stream=None):
    """ResidNormGrads from dh [R, D] and dr [R, D] (None: zeros): dx, du [R, D]
    bf16, dw_pre, dw_post [D] and dgate [B, D] fp32.  r: the saved r (x without
    u).  Without w_pre (no norm of r) r, rstd_r and dh are None."""
    some = dr if r is None else r
    _mat(some, "dr" if r is None else "r", torch.bfloat16)
    R, D = some.shape
    dt, ld_gate, per = _norm_params(R, D, w_pre, w_post, gate)
    dev, f32 = some.device, torch.float32
    for t, name, need in ((rstd_r, "rstd_r", w_pre), (rstd_u, "rstd_u", w_post)):
        if need is not None:
            _flat(t, name, f32, (R,))
    ld = lambda t, name: 0 if t is None else _bf16(t, name, R, D)  # noqa: E731
    dx = torch.empty((R, D), dtype=torch.bfloat16, device=dev)
    du = torch.empty((R, D), dtype=torch.bfloat16, device=dev) if u is not None else None
    make = torch.empty if R > 0 else torch.zeros     # no rows: the sums are zero
    dw_pre = make(D, dtype=f32, device=dev) if w_pre is not None else None
    dw_post = make(D, dtype=f32, device=dev) if w_post is not None else None
    dgate = make((R // per if R else gate.shape[0], D), dtype=f32, device=dev) if gate is not None else None
    if R == 0:
        return ResidNormGrads(dx, du, dw_pre, dw_post, dgate)
    lib = _lib.load()
    nbytes = int(lib.bs_resid_norm_bwd_workspace_bytes(R, D, per))
    ws = torch.empty(max(nbytes, 16), dtype=torch.uint8, device=dev)
    _check(lib.bs_resid_norm_bwd(_ptr(r), _ptr(u), _ptr(dh), _ptr(dr), R, D, ld(r, "r"), ld(u, "u"), ld(dh, "dh"),
                                 ld(dr, "dr"), _ptr(w_post), _ptr(gate), ld_gate, per, _ptr(w_pre),
                                 _DT.get(dt, BS_OUT_F32), alpha, _ptr(rstd_u), _ptr(rstd_r), _ptr(dx), ld(dx, "dx"),
                                 _ptr(du), ld(du, "du"), _ptr(dw_pre), _ptr(dw_post), _ptr(dgate), _ptr(ws),
                                 ws.numel(), _stream(stream)), "bs_resid_norm_bwd")
    return ResidNormGrads(dx, du, dw_pre, dw_post, dgate)


# ----------------------------------------------------------------------------
# gated activation with an 8-bit checkpoint
# ----------------------------------------------------------------------------

def _ckpt(ck, s_ck, R, C):
    _mat(ck, "ck", torch.uint8)
    _require(tuple(ck.shape) == (R, 2 * C), f"ck must be [{R}, {2 * C}]")
    return _ld(ck) if R > 1 else max(_ld(ck), 2 * C), _scale(s_ck, "s_ck", 2 * C // 128, R)


def bs_swiglu_quant_1x128_ckpt(a, b, ck, s_ck, q_row=None, s_row=None, q_col=None, s_col=None, stream=None):
    """bs_swiglu_quant_1x128 that also writes the 1x128 row codes of a and b
    for the backward: ck [R, 2C] uint8 (a then b), s_ck [2C/128, >= R]."""
    _mat(a, "a", torch.bfloat16)
    R, C = a.shape
    ld_ck, ld_sck = _ckpt(ck, s_ck, R, C)
    _check(_lib.load().bs_swiglu_quant_1x128_ckpt(_ptr(a), _ptr(b), R, C, _bf16(a, "a", R, C), _bf16(b, "b", R, C),
                                                  _ptr(ck), ld_ck, _ptr(s_ck), ld_sck,
                                                  *_codes(R, C, q_row, s_row, q_col, s_col), _stream(stream)),
           "bs_swiglu_quant_1x128_ckpt")


def bs_swiglu_bwd_quant_1x128_ckpt(ck, s_ck, dh, q_row=None, s_row=None, q_col=None, s_col=None, stream=None):
    """bs_swiglu_bwd_quant_1x128 from the checkpoint (ck, s_ck): the codes of
    [da | db] [R, 2C], rows and/or transposed columns."""
    _mat(dh, "dh", torch.bfloat16)
    R, C = dh.shape
    ld_ck, ld_sck = _ckpt(ck, s_ck, R, C)
    _check(_lib.load().bs_swiglu_bwd_quant_1x128_ckpt(_ptr(ck), R, C, ld_ck, _ptr(s_ck), ld_sck, _ptr(dh),
                                                      _bf16(dh, "dh", R, C),
                                                      *_codes(R, 2 * C, q_row, s_row, q_col, s_col), _stream(stream)),
           "bs_swiglu_bwd_quant_1x128_ckpt")
