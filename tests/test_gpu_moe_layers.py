"""Autograd layers of the MoE block: against the calls they make, against a
float64 implementation of the same layer on the quantized values, and against
differences."""

import importlib.util
import os

import numpy as np
import pytest
import torch

import blockwise_scaled_fp8_bs_amd as bs
from blockwise_scaled_fp8_bs_amd import inputs
from gpu_support import need_gpu
from oracle import block

pytestmark = pytest.mark.gpu


def _rel(a, b):
    a, b = a.detach().double().cpu(), b.detach().double().cpu()
    return float((a - b).norm() / b.norm())


def _setup(T, k, E, D, seed=0):
    g = torch.Generator().manual_seed(seed)
    logits = torch.randn((T, E), generator=g)
    if T > 3:
        logits[2] = -float("inf")
    return inputs.bf16_normal((T, D), 1.0, seed + 1).cuda(), logits.cuda(), g


def test_route_gradient_through_autograd_equals_differences():
    """Of the float64 oracle's forward: the layer's gradient is its Jacobian."""
    need_gpu()
    T, E, k = 6, 16, 3
    logits = torch.randn((T, E), generator=torch.Generator().manual_seed(1))
    g = torch.randn((T, k), generator=torch.Generator().manual_seed(2))
    for kind, name in ((block.SOFTMAX, "softmax"), (block.SIGMOID, "sigmoid")):
        l = logits.cuda().requires_grad_(True)
        idx, w = bs.moe_route(l, k, score=name, n_group=4, topk_group=2, group_best=2, scale=1.5)
        (w * g.cuda()).sum().backward()
        assert not idx.requires_grad
        L = logits.double().numpy()
        kw = dict(kind=kind, n_group=4, topk_group=2, group_best=2, scale=1.5)
        want = np.zeros((T, E))
        for t in range(T):
            for e in range(E):
                ends = []
                for h in (1e-6, -1e-6):
                    m = L.copy()
                    m[t, e] += h
                    ends.append((block.route(m, k, **kw)[1] * g.numpy()).sum())
                want[t, e] = (ends[0] - ends[1]) / 2e-6
        assert np.abs(l.grad.cpu().numpy() - want).max() < 1e-5


def row_slot_of(plan):
    """(rows that hold a slot, their slots)."""
    r = (plan.row_slot >= 0).nonzero()[:, 0]
    return r, plan.row_slot[r].long()


@pytest.mark.parametrize("T,k,E,D", [(50, 2, 4, 256), (300, 4, 16, 384), (1, 2, 8, 128)])
def test_dispatch_and_combine_with_mx_experts(T, k, E, D):
    """The bf16 pieces around mx_grouped_mm: outputs and gradients equal those
    of a loop over the experts on the same rows."""
    need_gpu()
    x, logits, g = _setup(T, k, E, D)
    wt = (torch.randn((E, 256, D), generator=g) * 0.05).to(torch.bfloat16).cuda()
    x.requires_grad_(True), logits.requires_grad_(True), wt.requires_grad_(True)
    idx, w = bs.moe_route(logits, k)
    plan = bs.bs_moe_plan(idx, E)
    print(f"mx experts T={T} k={k} E={E} D={D}", flush=True)
    xs = bs.moe_dispatch(x, plan, k)
    ys = bs.mx_grouped_mm(xs, wt, plan.group_end)
    out = bs.moe_combine(ys, plan, w)
    dout = inputs.bf16_normal((T, 256), 1.0, 9).cuda()
    out.backward(dout)
    # the same in float32 from the layer's own expert outputs
    rows = plan.slot_row.long().clamp_min(0)
    on = (plan.slot_row >= 0)
    picked = ys.detach()[rows].float() * on[..., None]
    want = (picked * w.detach()[..., None]).sum(1)
    # one rounding of the sum to bf16 and k in fp32
    assert ((out.float() - want).abs() <= want.abs() * 2.0 ** -8 + (picked.abs() * w.detach()[..., None]).sum(1) * 2.0 ** -20).all()
    dw = (picked * dout.float()[:, None]).sum(2)
    dl = block.route_bwd(logits.detach().double().cpu().numpy(), idx.cpu().numpy(), dw.double().cpu().numpy())
    assert _rel(logits.grad, torch.from_numpy(dl)) < 1e-4
    # x and the weights: the products' own gradients of the gathered rows, in expert order
    held = row_slot_of(plan)
    xr, wr = xs.detach().clone().requires_grad_(True), wt.detach().clone().requires_grad_(True)
    dys = torch.zeros_like(ys)
    dys[held[0]] = (w.detach().reshape(-1, 1)[held[1]] * dout[held[1] // k].float()).to(torch.bfloat16)
    bs.mx_grouped_mm(xr, wr, plan.group_end).backward(dys)
    assert torch.equal(wt.grad.view(torch.int16), wr.grad.view(torch.int16))
    terms = xr.grad[rows].float() * on[..., None]
    bound = terms.sum(1).abs() * 2.0 ** -8 + terms.abs().sum(1) * 2.0 ** -20
    assert ((x.grad.float() - terms.sum(1)).abs() <= bound).all()


def _experts_f32(x, idx, w, w12, wo, residual):
    H = wo.shape[2]
    out = residual.float()
    for j in range(idx.shape[1]):
        for e in range(w12.shape[0]):
            m = idx[:, j] == e
            ab = x[m].float() @ w12[e].float().t()
            h = torch.nn.functional.silu(ab[:, :H]) * ab[:, H:]
            out = out.index_add(0, m.nonzero()[:, 0], w[m, j][:, None] * (h @ wo[e].float().t()))
    return out


def _deq_rows(q, s):
    """1x128 row codes [R, C] with K-major scales, in float64."""
    v = q.view(torch.float8_e4m3fn).double()
    return v * s[:, :q.shape[0]].double().t().repeat_interleave(128, 1)


def _deq_tiles(q, s):
    """Per-expert 128x128 codes [E, N, K] with scales [E, K/128, >= N/128], in float64."""
    v = q.view(torch.float8_e4m3fn).double()
    n = s[:, :, :q.shape[1] // 128].double().transpose(1, 2)
    return v * n.repeat_interleave(128, 1).repeat_interleave(128, 2)


def _products(ends, a, w):
    """Rows of a times w[e]^T over each expert's rows, rounded to bf16; zeros past the last."""
    out = torch.zeros((a.shape[0], w.shape[1]), dtype=torch.bfloat16, device=a.device)
    lo = 0
    for e, hi in enumerate(ends):
        out[lo:hi] = (a[lo:hi] @ w[e].t()).to(torch.bfloat16)
        lo = hi
    return out


def _weight_grads(ends, a, b):
    lo, out = 0, []
    for hi in ends:
        out.append(a[:, lo:hi] @ b[:, lo:hi].t())
        lo = hi
    return torch.stack(out)


@pytest.mark.parametrize("checkpoint", ["fp8", "bf16"])
@pytest.mark.parametrize("T,k,E,D,H", [(200, 2, 4, 256, 384), (513, 4, 8, 384, 128), (3, 1, 4, 128, 256)])
def test_fp8_experts_equal_float64_products_of_the_codes(T, k, E, D, H, checkpoint):
    """The layer's sequence with every grouped product in float64 on the dequantized codes."""
    need_gpu()
    from blockwise_scaled_fp8_bs_amd.moe import _codes, _expert_weights

    x, logits, g = _setup(T, k, E, D, seed=5)
    w12 = (torch.randn((E, 2 * H, D), generator=g) * D ** -0.5).to(torch.bfloat16).cuda()
    wo = (torch.randn((E, D, H), generator=g) * H ** -0.5).to(torch.bfloat16).cuda()
    res, dout = inputs.bf16_normal((T, D), 1.0, 7).cuda(), inputs.bf16_normal((T, D), 1.0, 8).cuda()
    idx, w = bs.bs_moe_route(logits, k, score=bs.BS_SCORE_SIGMOID)
    plan = bs.bs_moe_plan(idx, E)
    ends, M = plan.group_end.tolist(), plan.row_slot.shape[0]
    leaves = [t.clone().requires_grad_(True) for t in (x, w, w12, wo, res)]
    print(f"experts T={T} k={k} E={E} D={D} H={H} {checkpoint}", flush=True)
    out = bs.float8_blockwise_moe_ffn(leaves[0], idx, leaves[1], leaves[2], leaves[3], residual=leaves[4],
                                      checkpoint=checkpoint)
    out.backward(dout)

    qx, qh, qd, qab = (_codes(M, c, True, x.device) for c in (D, H, D, 2 * H))
    bs.bs_moe_gather_quant_1x128(x, plan.row_slot, k, **qx)
    q12, s12, q12t, s12t = _expert_weights(w12)
    qo, so, qot, sot = _expert_weights(wo)
    ab = _products(ends, _deq_rows(qx["q_row"], qx["s_row"]), _deq_tiles(q12, s12))
    ck, s_ck = torch.empty((M, 2 * H), dtype=torch.uint8, device="cuda"), bs.empty_scales(2 * H // 128, M, "cuda")
    bs.bs_swiglu_quant_1x128_ckpt(ab[:, :H], ab[:, H:], ck, s_ck, **qh)
    y = _products(ends, _deq_rows(qh["q_row"], qh["s_row"]), _deq_tiles(qo, so))
    rows, on = plan.slot_row.long().clamp_min(0), plan.slot_row >= 0
    yt = y[rows].double() * on[..., None]
    bs.bs_moe_gather_quant_1x128(dout, plan.row_slot, k, w=w, **qd)
    dh = _products(ends, _deq_rows(qd["q_row"], qd["s_row"]), _deq_tiles(qot, sot))
    if checkpoint == "fp8":
        bs.bs_swiglu_bwd_quant_1x128_ckpt(ck, s_ck, dh, **qab)
    else:
        bs.bs_swiglu_bwd_quant_1x128(ab[:, :H], ab[:, H:], dh, None, **qab)
    dxs = _products(ends, _deq_rows(qab["q_row"], qab["s_row"]), _deq_tiles(q12t, s12t))
    cols = lambda q: _deq_rows(q["q_col"], q["s_col"])  # noqa: E731
    # A bf16 rounding of a product in fp32 instead of float64 moves an element by at most 2^-7 and few elements at all;
    # a code that flips by it moves by 2^-3 of an element.  2^-7 of the norm holds both.
    tol = 2.0 ** -7
    assert _rel(out, res.double() + (yt * w.double()[..., None]).sum(1)) < tol
    assert _rel(leaves[0].grad, (dxs[rows].double() * on[..., None]).sum(1)) < tol
    assert _rel(leaves[2].grad, _weight_grads(ends, cols(qab), cols(qx))) < tol
    assert _rel(leaves[3].grad, _weight_grads(ends, cols(qd), cols(qh))) < tol
    dw = (yt * dout.double()[:, None]).sum(2)
    assert ((leaves[1].grad - dw).abs() <= tol * yt.norm(dim=2) * dout.double().norm(dim=1)[:, None]).all()
    assert torch.equal(leaves[4].grad.view(torch.int16), dout.view(torch.int16))


@pytest.mark.parametrize("T,k,E,D,H", [(200, 2, 4, 256, 384), (513, 4, 8, 384, 128)])
def test_fp8_experts_against_float32_and_checkpoints(T, k, E, D, H):
    need_gpu()
    x, logits, g = _setup(T, k, E, D, seed=5)
    w12 = (torch.randn((E, 2 * H, D), generator=g) * D ** -0.5).to(torch.bfloat16).cuda()
    wo = (torch.randn((E, D, H), generator=g) * H ** -0.5).to(torch.bfloat16).cuda()
    res = inputs.bf16_normal((T, D), 1.0, 7).cuda()
    dout = inputs.bf16_normal((T, D), 1.0, 8).cuda()
    idx, w = bs.bs_moe_route(logits, k, score=bs.BS_SCORE_SIGMOID)
    got = {}
    for mode in ("fp8", "bf16", "f32"):
        leaves = [t.clone().requires_grad_(True) for t in (x, w, w12, wo, res)]
        print(f"experts T={T} k={k} E={E} D={D} H={H} {mode}", flush=True)
        a, b, c, d, r = leaves
        out = _experts_f32(a, idx, b, c, d, r) if mode == "f32" else \
            bs.float8_blockwise_moe_ffn(a, idx, b, c, d, residual=r, checkpoint=mode)
        out.backward(dout.to(out.dtype))
        got[mode] = [out] + [t.grad for t in leaves]
    # the forward does not depend on how [a | b] is kept
    assert torch.equal(got["fp8"][0].view(torch.int16), got["bf16"][0].view(torch.int16))
    for name, i, tol in (("out", 0, 0.08), ("x", 1, 0.12), ("w", 2, 0.08), ("w12", 3, 0.12), ("out_proj", 4, 0.08)):
        # e4m3 products err by about 3.7 % of their norm each (two operands of 2^-4 / sqrt(6) and the activation's
        # sensitivity); the 8-bit a and b add as much once more to da and db
        for mode in ("fp8", "bf16"):
            assert _rel(got[mode][i], got["f32"][i]) < tol, (name, mode)
    for mode in ("fp8", "bf16"):
        assert torch.equal(got[mode][5].view(torch.int16), dout.view(torch.int16))


@pytest.mark.parametrize("post,gated,pre", [(1, 1, 1), (0, 1, 1), (1, 0, 0), (None, 0, 1)])
def test_resid_norm_layer(post, gated, pre):
    need_gpu()
    B, S, D = 2, 9, 264
    g = torch.Generator().manual_seed(3)
    x = inputs.bf16_normal((B, S, D), 1.0, 1).cuda().requires_grad_(True)
    u = None if post is None else inputs.bf16_normal((B, S, D), 1.0, 2).cuda().requires_grad_(True)
    new = lambda *s: torch.randn(s, generator=g).cuda().requires_grad_(True)  # noqa: E731
    w_post, gate, w_pre = (new(D) if post else None), (new(B, D) if gated else None), (new(D) if pre else None)
    r, h = bs.resid_norm(x, w_pre, u=u, w_post=w_post, gate=gate, alpha=0.5, eps=1e-5)
    assert (h is None) == (not pre) and r.shape == x.shape and (u is not None or r is x)
    cr, ch = inputs.bf16_normal((B, S, D), 1.0, 4).cuda(), inputs.bf16_normal((B, S, D), 1.0, 5).cuda()
    loss = (r.float() * cr).sum() + ((h.float() * ch).sum() if pre else 0.0)
    loss.backward()
    # autograd of the plain formula in float64
    f = lambda t: None if t is None else t.detach().double().requires_grad_(True)  # noqa: E731
    X, U, WQ, G, WP = f(x), f(u), f(w_post), f(gate), f(w_pre)
    n = lambda v: v / torch.sqrt(v.square().mean(-1, keepdim=True) + 1e-5)  # noqa: E731
    R = X if U is None else X + 0.5 * (1.0 if G is None else G[:, None]) * (U if WQ is None else n(U) * WQ)
    want = (R * cr).sum() + ((n(R) * WP * ch).sum() if pre else 0.0)
    want.backward()
    for a, b in ((x, X), (u, U), (w_post, WQ), (gate, G), (w_pre, WP)):
        if a is not None:
            # bf16 values of r, dr and dh (2^-9 each, at random) against exact ones
            assert _rel(a.grad, b.grad) < 2.0 ** -7
    assert _rel(r, R) < 2.0 ** -8


def _example():
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "moe_block.py")
    spec = importlib.util.spec_from_file_location("moe_block_example", path)
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


def test_example_block_trains_and_serves():
    need_gpu()
    ex = _example()
    torch.manual_seed(0)
    b = ex.MoEBlock(256, 128, 8, 2)
    new = lambda n: torch.randn(n, 256, device="cuda").to(torch.bfloat16)  # noqa: E731
    x, u, target = new(700), new(700), new(700)
    losses = ex.train(b, x, u, target, 8)
    assert losses[-1] < losses[0] and all(np.isfinite(losses))
    assert int(b.moe.last_counts.sum()) == 700 * 2 and b.moe.balance.abs().max() > 0
    # serving: weights laid out once, rows unpadded and quantized along rows only: the same codes, so the same bits
    b.eval()
    with torch.no_grad():
        for n in (700, 33, 1):
            plain = b(x[:n].contiguous(), u[:n].contiguous())
            b.moe.prepare_serving()
            served = b(x[:n].contiguous(), u[:n].contiguous())
            b.moe._serving = None
            assert torch.equal(plain.view(torch.int16), served.view(torch.int16)), n


def test_serving_layout_follows_the_weights():
    need_gpu()
    m = bs.Float8BlockwiseMoE(128, 128, 4, 2, device="cuda").eval()
    x = torch.randn(5, 128, device="cuda").to(torch.bfloat16)
    with torch.no_grad():
        m.prepare_serving()
        m.w12.mul_(2.0)
        with pytest.raises(RuntimeError, match="call it again"):
            m(x)
        m.prepare_serving()
        y = m(x)
        state = {n: v * 0.5 if n == "w12" else v.clone() for n, v in m.state_dict().items()}
        m.load_state_dict(state)
        assert m._serving is None and not torch.equal(m(x), y)
    m.prepare_serving().train()
    assert m._serving is None
    # gradients on: the layout is not taken
    m.eval().prepare_serving()
    assert m(x).requires_grad


def test_no_tokens():
    need_gpu()
    m = bs.Float8BlockwiseMoE(128, 256, 4, 2, device="cuda")
    x = torch.empty((0, 128), dtype=torch.bfloat16, device="cuda", requires_grad=True)
    y = m(x, residual=x)
    y.sum().backward()
    assert y.shape == (0, 128) and x.grad.shape == (0, 128)
    for p in (m.w12, m.out_proj):
        assert (p.grad == 0).all()
    m.eval().prepare_serving()
    with torch.no_grad():
        assert m(x).shape == (0, 128)


def test_serving_pass_replays_from_a_graph():
    """Captured once; every replay equals the eager pass on the same inputs."""
    need_gpu()
    ex = _example()
    torch.manual_seed(1)
    b = ex.MoEBlock(256, 256, 16, 4).eval()
    b.moe.prepare_serving()
    new = lambda: torch.randn(3, 256, device="cuda").to(torch.bfloat16)  # noqa: E731
    x, u = new(), new()
    with torch.no_grad():
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            b(x, u)
        torch.cuda.current_stream().wait_stream(side)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            y = b(x, u)
        for _ in range(4):
            x.copy_(new()), u.copy_(new())
            want = b(x, u)
            graph.replay()
            torch.cuda.synchronize()
            assert torch.equal(y.view(torch.int16), want.view(torch.int16))


def test_training_step_replays_from_a_graph():
    """Forward and backward of the block captured once; every replay equals the
    eager step of a copy on the same inputs.  (The copy, so that no eager graph
    of the captured leaves lives while the backward is captured.)"""
    need_gpu()
    import copy

    ex = _example()
    torch.manual_seed(2)
    b = ex.MoEBlock(256, 128, 8, 2)
    eager = copy.deepcopy(b)
    new = lambda: torch.randn(300, 256, device="cuda").to(torch.bfloat16)  # noqa: E731
    x, u, dy = new(), new(), new()

    def step(m):
        y = m(x, u)
        return [y.detach()] + list(torch.autograd.grad(y, list(m.parameters()), dy))

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step(b)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step(b)
    for i in range(4):
        print(f"training step replay {i}", flush=True)
        for t in (x, u, dy):
            t.copy_(new())
        want = step(eager)
        graph.replay()
        torch.cuda.synchronize()
        for a, w in zip(got, want):
            assert torch.equal(a, w)
        del want


def test_layer_refusals():
    need_gpu()
    x = torch.zeros((4, 256), dtype=torch.bfloat16, device="cuda")
    idx = torch.zeros((4, 2), dtype=torch.int32, device="cuda")
    w = torch.zeros((4, 2), device="cuda")
    w12 = torch.zeros((2, 256, 256), dtype=torch.bfloat16, device="cuda")
    wo = torch.zeros((2, 256, 128), dtype=torch.bfloat16, device="cuda")
    for match, kw in (("checkpoint", dict(checkpoint="int4")), ("out_proj", dict(out_proj=wo[:1])),
                      ("features", dict(x=x[:, :128].contiguous())), ("contiguous", dict(x=torch.zeros((4, 512), dtype=torch.bfloat16, device="cuda")[:, :256])),
                      ("idx and w", dict(idx=idx[:3])), ("bfloat16", dict(w12=w12.float()))):
        args = dict(x=x, idx=idx, w=w, w12=w12, out_proj=wo)
        args.update(kw)
        with pytest.raises(ValueError, match=match):
            bs.float8_blockwise_moe_ffn(**args)
    for wrong in (bs.bs_moe_plan(idx, 2, align=1), bs.bs_moe_plan(idx, 3), bs.bs_moe_plan(idx[:3], 2)):
        with pytest.raises(ValueError, match="the plan is for"):
            bs.float8_blockwise_moe_ffn(x, idx, w, w12, wo, plan=wrong)
    plan = bs.bs_moe_plan(idx, 2)
    with pytest.raises(ValueError, match="slots"):
        bs.moe_dispatch(x[:3], plan)
    with pytest.raises(ValueError, match="rows"):
        bs.moe_combine(x, plan, w)
    with pytest.raises(ValueError, match="score"):
        bs.moe_route(torch.zeros((4, 8), device="cuda"), 2, score="relu")
    with pytest.raises(ValueError, match="need u"):
        bs.resid_norm(x, torch.ones(256, device="cuda"), gate=torch.ones((1, 256), device="cuda"))
    with pytest.raises(ValueError, match="nothing"):
        bs.resid_norm(x)
    with pytest.raises(ValueError, match="multiples of 128"):
        bs.Float8BlockwiseMoE(100, 128, 4, 2)
