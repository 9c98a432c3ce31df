"""MoE block around the grouped FP8 GEMMs: router, dispatch, combine and the
residual norms with autograd, and the expert FFN that fuses them with the
quantizers.

(The grouped scaled GEMMs of MoE training: "[not for land] float8 blockwise
scaling training prototype using deep_gemm", description; "[mxfp8 moe
training] use new 3d colwise quantization kernel", summary.)

The pieces work with any experts, for instance ``mx_grouped_mm``:

    idx, w = moe_route(logits, k)              # differentiable in the logits
    plan   = bs_moe_plan(idx, E)               # sort by expert, on the device
    xs     = moe_dispatch(x, plan, k)          # rows in expert order
    ys     = mx_grouped_mm(xs, weight, plan.group_end)
    y      = moe_combine(ys, plan, w, residual)

``Float8BlockwiseMoE`` runs the gated experts in blockwise FP8 and stores
fewer tensors: the gathered rows exist only as FP8 codes (rows for the forward
GEMM, transposed columns for the weight gradient), h = silu(a) b only as its
codes, the weighted gradient rows only as theirs, and [a | b], the largest
tensor kept for the backward, as 1x128 codes (``checkpoint="fp8"``) or bf16.

  forward   gather + quantize x; [a | b] = xs [w1; w2]_e^T (GROUP_M);
            h = silu(a) b quantized, a and b kept in 8 bits (one kernel);
            ys = h out_e^T (GROUP_M); out = residual + sum w ys
  backward  dw = <dout, ys>; gather + weight + quantize dout;
            dh = dys out_e, dout_e = dys^T h (GROUP_K);
            [da | db] quantized from the 8-bit a, b and dh (one kernel);
            dxs = [da | db] [w1; w2]_e, d[w1; w2]_e = [da | db]^T xs;
            dx = sum dxs

Nothing here waits for the device, so a forward, and a training step with its
backward, can be captured into a HIP graph (no eager autograd graph of the same
parameters may be alive while a backward is captured).

Rows of the expert-ordered matrices past the last group (padding, and slots
that were not routed) are computed by the elementwise kernels but read by no
GEMM, and combined into no token.
"""

import torch
from torch.autograd.function import once_differentiable

from . import binding as _b
from . import binding_block as _k
from . import binding_few as _f
from . import serving as _s


def _rows(t, name):
    """A [..., D] contiguous bf16 GPU tensor as [R, D]."""
    if t.dtype != torch.bfloat16:
        raise ValueError(f"{name} must be bfloat16, got {t.dtype}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous (row-major); pass a contiguous tensor")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a GPU tensor")
    return t.view(-1, t.shape[-1])


def _bf16_grad(t):
    return t.to(torch.bfloat16).contiguous()


# ----------------------------------------------------------------------------
# router
# ----------------------------------------------------------------------------

_SCORES = {"softmax": _k.BS_SCORE_SOFTMAX, "sigmoid": _k.BS_SCORE_SIGMOID}


class _RouteFn(torch.autograd.Function):
    @staticmethod
    def forward(ctx, logits, bias, k, score, n_group, topk_group, group_best, renormalize, scale):
        idx, w = _k.bs_moe_route(logits, k, bias=bias, score=score, n_group=n_group, topk_group=topk_group,
                                 group_best=group_best, renormalize=renormalize, scale=scale)
        ctx.save_for_backward(logits, idx, w)
        ctx.how = (score, renormalize, scale)
        ctx.mark_non_differentiable(idx)
        return idx, w

    @staticmethod
    @once_differentiable
    def backward(ctx, _, dw):
        logits, idx, w = ctx.saved_tensors
        score, renormalize, scale = ctx.how
        d = _k.bs_moe_route_bwd(logits, idx, w, dw.contiguous(), score=score, renormalize=renormalize, scale=scale)
        return (d,) + (None,) * 8


def moe_route(logits, k, bias=None, score="softmax", n_group=1, topk_group=1, group_best=1, renormalize=True,
              scale=1.0):
    """(idx [T, k] int32, w [T, k] float32) of bs_moe_route, w differentiable
    in the logits.  The bias takes part in the choice only and gets no gradient."""
    if score not in _SCORES:
        raise ValueError(f"score must be one of {sorted(_SCORES)}, got {score!r}")
    return _RouteFn.apply(logits, bias, k, _SCORES[score], n_group, topk_group, group_best, renormalize, scale)


# ----------------------------------------------------------------------------
# dispatch and combine in bf16
# ----------------------------------------------------------------------------

class _DispatchFn(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x2, slot_row, row_slot):
        k = slot_row.shape[1]
        y = torch.empty((row_slot.shape[0], x2.shape[1]), dtype=torch.bfloat16, device=x2.device)
        _k.bs_moe_gather_quant_1x128(x2, row_slot, k, y=y)
        ctx.save_for_backward(slot_row)
        return y

    @staticmethod
    @once_differentiable
    def backward(ctx, dy):
        (slot_row,) = ctx.saved_tensors
        return _k.bs_moe_combine(_bf16_grad(dy), slot_row), None, None


def moe_dispatch(x, plan, k=None):
    """Rows of x [T, D] in the plan's expert order [M, D] bf16, zeros where a
    row belongs to no slot.  D a multiple of 128."""
    x2 = _rows(x, "x")
    if x2.shape[0] != plan.slot_row.shape[0] or (k is not None and k != plan.slot_row.shape[1]):
        raise ValueError(f"the plan is for {list(plan.slot_row.shape)} slots, x has {x2.shape[0]} tokens")
    return _DispatchFn.apply(x2, plan.slot_row, plan.row_slot)


class _CombineFn(torch.autograd.Function):
    @staticmethod
    def forward(ctx, y, w, residual, slot_row, row_slot):
        ctx.save_for_backward(y, w, slot_row, row_slot)
        return _k.bs_moe_combine(y, slot_row, w=w, residual=residual)

    @staticmethod
    @once_differentiable
    def backward(ctx, dout):
        y, w, slot_row, row_slot = ctx.saved_tensors
        dout = _bf16_grad(dout)
        dy = dw = None
        if ctx.needs_input_grad[0]:
            dy = torch.empty_like(y)
            _k.bs_moe_gather_quant_1x128(dout, row_slot, slot_row.shape[1], w=w, y=dy)
        if ctx.needs_input_grad[1]:
            dw = _k.bs_moe_combine_dw(dout, y, slot_row)
        return dy, dw, (dout if ctx.needs_input_grad[2] else None), None, None


def moe_combine(y, plan, w, residual=None):
    """residual + sum over each token's slots of w times its rows of y [M, D],
    in token order [T, D] bf16; differentiable in y, w and the residual."""
    if tuple(w.shape) != tuple(plan.slot_row.shape):
        raise ValueError(f"w must be {list(plan.slot_row.shape)} like the plan's slots, got {list(w.shape)}")
    y2 = _rows(y, "y")
    if y2.shape[0] != plan.row_slot.shape[0]:
        raise ValueError(f"y must have the plan's {plan.row_slot.shape[0]} rows, got {y2.shape[0]}")
    if y2.shape[1] % 128 != 0:
        raise ValueError(f"y has {y2.shape[1]} columns: they must be a multiple of 128 (its gradient's tiles)")
    r2 = None if residual is None else _rows(residual, "residual")
    out = _CombineFn.apply(y2, w, r2, plan.slot_row, plan.row_slot)
    return out if residual is None else out.view(residual.shape)


# ----------------------------------------------------------------------------
# residual norms
# ----------------------------------------------------------------------------

class _ResidNormFn(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, u, w_post, gate, w_pre, alpha, eps):
        R, dev = x.shape[0], x.device
        new = lambda want: torch.empty(R, dtype=torch.float32, device=dev) if want else None  # noqa: E731
        r = torch.empty_like(x) if u is not None else None
        h = torch.empty_like(x) if w_pre is not None else None
        rstd_u, rstd_r = new(w_post is not None), new(w_pre is not None)
        _k.bs_resid_norm(x, w_pre, u=u, w_post=w_post, gate=gate, alpha=alpha, eps=eps, r=r, h=h, rstd_u=rstd_u,
                         rstd_r=rstd_r)
        ctx.save_for_backward(x if u is None else r, u, w_post, gate, w_pre, rstd_u, rstd_r)
        ctx.alpha = alpha
        ctx.set_materialize_grads(False)
        return r, h

    @staticmethod
    @once_differentiable
    def backward(ctx, dr, dh):
        r, u, w_post, gate, w_pre, rstd_u, rstd_r = ctx.saved_tensors
        dr = None if dr is None else _bf16_grad(dr)
        dh = None if dh is None else _bf16_grad(dh)
        if dr is None and dh is None:
            return (None,) * 7
        pre = dh is not None
        g = _k.bs_resid_norm_bwd(r if pre else None, rstd_r if pre else None, w_pre if pre else None, dh, dr=dr, u=u,
                                 rstd_u=rstd_u, w_post=w_post, gate=gate, alpha=ctx.alpha)
        to = lambda d, p: None if d is None else d.to(p.dtype)  # noqa: E731
        return g.dx, g.du, to(g.dw_post, w_post), to(g.dgate, gate), to(g.dw_pre, w_pre), None, None


def resid_norm(x, w_pre=None, u=None, w_post=None, gate=None, alpha=1.0, eps=1e-6):
    """(r, h): r = x + alpha gate N(u) w_post and h = N(r) w_pre, N(v) = v /
    sqrt(mean(v^2) + eps); without u r is x, without w_pre h is None, without
    w_post u is added as it is.

    x, u [..., D] bf16; w_pre, w_post [D] and gate [B, D] of one type (bf16 or
    fp32), consecutive rows / B rows sharing a row of the gate.
    """
    if u is None and w_pre is None:
        raise ValueError("nothing to compute: neither u nor w_pre is given")
    if u is not None and u.shape != x.shape:
        raise ValueError(f"u must be {list(x.shape)} like x, got {list(u.shape)}")
    if u is None and (w_post is not None or gate is not None):
        raise ValueError("w_post and gate need u")
    x2 = _rows(x, "x")
    r, h = _ResidNormFn.apply(x2, None if u is None else _rows(u, "u"), w_post, gate, w_pre, alpha, eps)
    return (x if r is None else r.view(x.shape)), (None if h is None else h.view(x.shape))


# ----------------------------------------------------------------------------
# gated experts in blockwise FP8
# ----------------------------------------------------------------------------

def _codes(R, C, cols, dev):
    """Empty outputs of a 1x128 quantization of [R, C]."""
    q = dict(q_row=torch.empty((R, C), dtype=torch.uint8, device=dev), s_row=_b.empty_scales(C // 128, R, dev))
    if cols:
        q.update(q_col=torch.empty((C, R), dtype=torch.uint8, device=dev), s_col=_b.empty_scales(R // 128, C, dev))
    return q


def _expert_weights(w):
    """Codes of w [E, N, K] in 128x128 tiles, per expert: forward operand
    [E, N, K] with scales [E, K/128, N/128], transposed operand [E, K, N] with
    scales [E, N/128, >= K/128]."""
    E, N, K = w.shape
    dev = w.device
    q = torch.empty((E * N, K), dtype=torch.uint8, device=dev)
    s = _b.empty_scales(K // 128, E * N // 128, dev)
    qt = torch.empty((E, K, N), dtype=torch.uint8, device=dev)
    st = torch.empty((E, N // 128, _b._round4(K // 128)), dtype=torch.float32, device=dev)
    _b.bs_quant_128x128_both(w, q, s, qt, st)
    return q.view(E, N, K), torch.as_strided(s, (E, K // 128, N // 128), (N // 128, s.stride(0), 1)), qt, st


def _group_m(ends, q, w, s, zeros=False):
    """Rows of q times w[e]^T.  The rows past the last group are not written:
    zeros for a result that goes through an elementwise kernel, where what
    uninitialised memory holds can need the float64 path, an element at a time
    (8192 tokens of 4 slots, 16 experts of 1024: the forward activation takes
    121 us over garbage, 69 over zeros, which cost 20)."""
    new = torch.zeros if zeros else torch.empty
    out = new((q["q_row"].shape[0], w.shape[1]), dtype=torch.bfloat16, device=w.device)
    return _b.bs_grouped_scaled_mm(_b.BS_GROUP_M, ends, q["q_row"], q["s_row"], w, s, _b.BS_SCALE_128X128, out=out)


def _group_k(ends, a, b):
    """Per-expert a^T b over the tokens, from the transposed column codes of both."""
    return _b.bs_grouped_scaled_mm(_b.BS_GROUP_K, ends, a["q_col"], a["s_col"], b["q_col"], b["s_col"],
                                   _b.BS_SCALE_1X128, out_dtype=torch.bfloat16)


class _MoEFFNFn(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x2, w, w12, wo, residual, ends, slot_row, row_slot, fp8_checkpoint):
        E, H2, D = w12.shape
        H, M, dev = H2 // 2, row_slot.shape[0], x2.device
        if x2.shape[0] == 0:
            ctx.save_for_backward(w, w12, wo)
            return torch.empty_like(x2)
        qx = _codes(M, D, True, dev)
        _k.bs_moe_gather_quant_1x128(x2, row_slot, slot_row.shape[1], **qx)
        q12, s12, q12t, s12t = _expert_weights(w12)
        ab = _group_m(ends, qx, q12, s12, zeros=True)
        del qx["q_row"], qx["s_row"], q12  # (memory that the rest of the pass can have)
        qh = _codes(M, H, True, dev)
        if fp8_checkpoint:
            kept = (torch.empty((M, H2), dtype=torch.uint8, device=dev), _b.empty_scales(H2 // 128, M, dev))
            _k.bs_swiglu_quant_1x128_ckpt(ab[:, :H], ab[:, H:], *kept, **qh)
        else:
            kept = (ab, None)
            _b.bs_swiglu_quant_1x128(ab[:, :H], ab[:, H:], None, **qh)
        del ab
        qo, so, qot, sot = _expert_weights(wo)
        y = _group_m(ends, qh, qo, so)
        ctx.save_for_backward(w, ends, slot_row, row_slot, qx["q_col"], qx["s_col"], q12t, s12t, *kept, qh["q_col"],
                              qh["s_col"], qot, sot, y)
        return _k.bs_moe_combine(y, slot_row, w=w, residual=residual)

    @staticmethod
    @once_differentiable
    def backward(ctx, dout):
        need = ctx.needs_input_grad
        if dout.shape[0] == 0:
            d = [torch.zeros_like(t) if n else None for t, n in zip((dout, *ctx.saved_tensors, dout), need)]
            return (*d, None, None, None, None)
        (w, ends, slot_row, row_slot, qxt, sxt, q12t, s12t, kept, kept_s, qht, sht, qot, sot, y) = ctx.saved_tensors
        dout = _bf16_grad(dout)
        M, H2, dev = y.shape[0], q12t.shape[2], y.device
        H, D = H2 // 2, y.shape[1]
        dw = _k.bs_moe_combine_dw(dout, y, slot_row) if need[1] else None
        qd = _codes(M, D, True, dev)
        _k.bs_moe_gather_quant_1x128(dout, row_slot, slot_row.shape[1], w=w, **qd)
        dwo = _group_k(ends, qd, dict(q_col=qht, s_col=sht)) if need[3] else None
        dx = dw12 = None
        if need[0] or need[2]:
            dh = _group_m(ends, qd, qot, sot, zeros=True)
            del qd
            qab = _codes(M, H2, True, dev)
            if kept_s is not None:
                _k.bs_swiglu_bwd_quant_1x128_ckpt(kept, kept_s, dh, **qab)
            else:
                _b.bs_swiglu_bwd_quant_1x128(kept[:, :H], kept[:, H:], dh, None, **qab)
            del dh
            if need[2]:
                dw12 = _group_k(ends, qab, dict(q_col=qxt, s_col=sxt))
            if need[0]:
                dx = _k.bs_moe_combine(_group_m(ends, qab, q12t, s12t), slot_row)
        return dx, dw, dw12, dwo, (dout if need[4] else None), None, None, None, None


def _check_plan(plan, slots, E):
    """The weight gradients contract whole 128-row blocks of each group, so that
    a group that ends inside one would lose rows or take another expert's."""
    M, need, align = plan.row_slot.shape[0], _k.bs_moe_plan_rows(*slots, E), getattr(plan, "align", None)
    if tuple(plan.slot_row.shape) != tuple(slots) or plan.group_end.shape[0] != E or M % 128 != 0 or M < need \
            or align is None or align % 128 != 0:
        raise ValueError(f"the plan is for {list(plan.slot_row.shape)} slots, {plan.group_end.shape[0]} experts and {M} "
                         f"rows in groups of a multiple of {align}: this needs {list(slots)}, {E} and groups padded to "
                         f"128 rows (at least {need}; a MoEPlan made by hand says so by its align)")


def float8_blockwise_moe_ffn(x, idx, w, w12, out_proj, residual=None, checkpoint="fp8", plan=None):
    """residual + sum_j w_j out_e(silu(a) b), [a | b] = x [w1; w2]_e^T, over the
    experts e = idx[t, j] of each token, every GEMM in blockwise FP8.

    x [..., D] bf16 (T tokens); idx [T, k] int32 (-1: not routed) and w [T, k]
    fp32, as moe_route gives them; w12 [E, 2H, D] (w1's rows, then w2's) and
    out_proj [E, D, H] bf16; D and H multiples of 128.  checkpoint: how [a | b]
    is kept for the backward, "fp8" (1x128 codes) or "bf16".  plan: that of
    bs_moe_plan(idx, E), every group padded to 128 rows or a multiple (made
    here if None).
    """
    if checkpoint not in ("fp8", "bf16"):
        raise ValueError(f'checkpoint must be "fp8" or "bf16", got {checkpoint!r}')
    if w12.dim() != 3 or w12.shape[1] % 2 != 0:
        raise ValueError(f"w12 must be [E, 2H, D], got {list(w12.shape)}")
    E, H2, D = w12.shape
    H = H2 // 2
    if tuple(out_proj.shape) != (E, D, H):
        raise ValueError(f"out_proj must be [{E}, {D}, {H}], got {list(out_proj.shape)}")
    if D % 128 != 0 or H % 128 != 0:
        raise ValueError(f"dim = {D} and hidden = {H} must be multiples of 128 for blockwise FP8")
    for name, t in (("w12", w12), ("out_proj", out_proj)):
        if t.dtype != torch.bfloat16 or not t.is_contiguous() or not t.is_cuda:
            raise ValueError(f"{name} must be a contiguous bfloat16 GPU tensor")
    if x.shape[-1] != D:
        raise ValueError(f"x has {x.shape[-1]} features, the experts expect {D}")
    x2 = _rows(x, "x")
    if idx.dim() != 2 or idx.shape[0] != x2.shape[0] or w.shape != idx.shape:
        raise ValueError(f"idx and w must be [{x2.shape[0]}, k], got {list(idx.shape)} and {list(w.shape)}")
    if plan is None:
        plan = _k.bs_moe_plan(idx, E)
    _check_plan(plan, idx.shape, E)
    r2 = None if residual is None else _rows(residual, "residual")
    y = _MoEFFNFn.apply(x2, w, w12, out_proj, r2, plan.group_end, plan.slot_row, plan.row_slot, checkpoint == "fp8")
    return y.view(x.shape)


class Float8BlockwiseMoE(_s.ServedWeights, torch.nn.Module):
    """Bias-free gated experts in blockwise FP8 behind a top-k router.

    router [experts, dim], w12 [experts, 2 hidden, dim], out_proj
    [experts, dim, hidden] (bf16 parameters) and balance [experts], the bias of
    the choice (a buffer that a training loop moves by the loads in
    ``last_counts``, fp32 also where the module is cast).  forward(x, residual)
    returns residual + experts(x).  The logits are a bf16 product: experts
    whose logits round to the same value tie, and the lowest is taken.
    checkpoint: how [a | b] is kept for the backward, in 8 bits by default.

    For serving, ``prepare_serving()`` lays the weights out once in FP8; while
    that layout is there (see ``ServedWeights``) and gradients are off, forward
    takes it: the rows are sorted without padding and quantized along rows
    only.  With ``prepare_serving(few_tokens=...)`` passes of up to that many
    tokens take the experts in two kernels instead, tokens in bf16, and
    ``last_counts`` is None after them.  Other weights than those laid out are
    quantized by the forward that they are there for.  ``ServedWeights`` says
    until when a pass captured into a graph may be replayed.
    """

    _served_names = ("w12", "out_proj")

    def __init__(self, dim, hidden, experts, top_k, score="sigmoid", n_group=1, topk_group=1, group_best=1,
                 renormalize=True, scale=1.0, checkpoint="fp8", device=None):
        super().__init__()
        if dim % 128 != 0 or hidden % 128 != 0:
            raise ValueError(f"dim = {dim} and hidden = {hidden} must be multiples of 128 for blockwise FP8")
        if not 1 <= top_k <= min(experts, 32):
            raise ValueError(f"top_k = {top_k} must be in [1, min(experts, 32)]")
        self.dim, self.hidden, self.experts, self.top_k = dim, hidden, experts, top_k
        self.checkpoint = checkpoint
        self.how = dict(score=score, n_group=n_group, topk_group=topk_group, group_best=group_best,
                        renormalize=renormalize, scale=scale)
        new = lambda *shape: torch.nn.Parameter(torch.empty(shape, device=device, dtype=torch.bfloat16))  # noqa: E731
        self.router, self.w12 = new(experts, dim), new(experts, 2 * hidden, dim)
        self.out_proj = new(experts, dim, hidden)
        self.register_buffer("balance", torch.zeros(experts, device=device))
        with torch.no_grad():
            for p in (self.router, self.w12, self.out_proj):
                p.uniform_(-p.shape[-1] ** -0.5, p.shape[-1] ** -0.5)
        self.last_counts = None

    def prepare_serving(self, weights="fp8", few_tokens=None):
        """Quantizes the expert weights for the forward; call again after they
        change.  Not for inference tensors, whose changes nothing counts.

        weights: "fp8" (the 128x128 blocks of the training forward) or "mxfp4"
        (4 bits, for half the traffic of few tokens; passes of more tokens take
        the 4-bit values in FP8, which are kept too: half as much memory again).
        few_tokens: tokens up to which a pass takes bs_moe_few; by default none
        with "fp8", whose passes then give the training forward's bits, and
        FEW_TOKENS with "mxfp4".  With 0 the 4-bit codes, which no pass would
        read, are not kept.
        """
        if few_tokens is None:
            few_tokens = _s.FEW_TOKENS if weights == "mxfp4" else 0
        _s.check_formats(weights, few_tokens, ("fp8", "mxfp4"))

        def layout(w12, out_proj):
            few = ()
            if weights == "mxfp4":
                q12, s12, w12 = _s.experts_mx4(w12)
                qo, so, out_proj = _s.experts_mx4(out_proj)
                few = (q12, s12, qo, so, _f.BS_WEIGHT_MXFP4) if few_tokens else ()
            gemm = _expert_weights(w12)[:2] + _expert_weights(out_proj)[:2]
            return gemm + (few or gemm + (_f.BS_WEIGHT_E4M3_128X128,)) + (few_tokens,)

        return self._lay_out(layout)

    def _apply(self, fn, *args, **kw):
        balance = self.balance
        super()._apply(fn, *args, **kw)
        if self.balance.dtype != torch.float32:  # the module was cast: the weights' type is not the bias's
            self.balance = balance.to(self.balance.device)
        return self

    def _serve(self, layout, x2, idx, w, residual):
        q12, s12, qo, so = layout[:4]
        plan = _k.bs_moe_plan(idx, self.experts, align=1)
        M, H, dev = plan.row_slot.shape[0], self.hidden, x2.device
        qx = _codes(M, self.dim, False, dev)
        _k.bs_moe_gather_quant_1x128(x2, plan.row_slot, self.top_k, **qx)
        ab = _group_m(plan.group_end, qx, q12, s12, zeros=True)
        qh = _codes(M, H, False, dev)
        _b.bs_swiglu_quant_1x128(ab[:, :H], ab[:, H:], None, **qh)
        return plan, _k.bs_moe_combine(_group_m(plan.group_end, qh, qo, so), plan.slot_row, w=w, residual=residual)

    def forward(self, x, residual=None):
        x2 = _rows(x, "x")
        if x2.shape[1] != self.dim:
            raise ValueError(f"x has {x2.shape[1]} features, the experts expect {self.dim}")
        logits = torch.nn.functional.linear(x2, self.router)
        idx, w = moe_route(logits, self.top_k, bias=self.balance, **self.how)
        layout = None if x2.shape[0] == 0 else self._layout_for(x, residual)
        if layout is not None:
            r2 = None if residual is None else _rows(residual, "residual")
            if x2.shape[0] <= layout[-1]:
                self.last_counts = None
                return _f.bs_moe_few(x2, idx, w, *layout[4:9], residual=r2).view(x.shape)
            plan, y = self._serve(layout, x2, idx, w, r2)
            y = y.view(x.shape)
        else:
            plan = _k.bs_moe_plan(idx, self.experts)
            y = float8_blockwise_moe_ffn(x, idx, w, self.w12, self.out_proj, residual=residual,
                                         checkpoint=self.checkpoint, plan=plan)
        self.last_counts = plan.counts
        return y

    def extra_repr(self):
        return (f"dim={self.dim}, hidden={self.hidden}, experts={self.experts}, top_k={self.top_k}, blockwise fp8, "
                f"checkpoint={self.checkpoint}")
