"""GPU router against the float64 oracle: choices equal, weights and
gradients within their rounding."""

import numpy as np
import pytest
import torch

import blockwise_scaled_fp8_bs_amd as bs
from gpu_support import need_gpu
from oracle import block

pytestmark = pytest.mark.gpu

# (T, E, k, n_group, topk_group, group_best)
SHAPES = [
    (1, 256, 8, 8, 4, 2), (37, 256, 8, 8, 4, 2), (70, 8, 2, 1, 1, 1), (300, 8, 8, 4, 2, 1), (1, 1, 1, 1, 1, 1),
    (33, 5, 3, 1, 1, 1), (50, 9, 4, 3, 2, 2), (40, 32, 6, 4, 1, 2), (40, 33, 32, 1, 1, 1), (40, 64, 6, 1, 1, 1),
    (21, 100, 7, 10, 3, 2), (20, 128, 8, 128, 9, 1), (18, 200, 8, 4, 4, 2), (9, 257, 8, 1, 1, 1), (9, 512, 16, 16, 4, 2),
    (7, 1000, 32, 8, 8, 1), (5, 1024, 8, 1024, 10, 2), (6, 256, 8, 256, 12, 2),
]


def _logits(T, E, dtype, seed, grid=None):
    rng = np.random.default_rng(seed)
    l = torch.from_numpy(rng.standard_normal((T, E)).astype(np.float32) * 1.5)
    if grid:                       # few distinct values: many ties
        l = (l * grid).round() / grid
    if T > 4:
        l[3] = -float("inf")                      # nothing to choose
        l[4, E // 2:] = -float("inf")             # masked experts, maybe fewer than k left
        l[4, 0] = torch.finfo(torch.float32).min if dtype == torch.float32 else torch.finfo(torch.bfloat16).min
    return l.to(dtype)


def _f64(t):
    return t.double().numpy()


def _weights_close(w, want):
    # float64 arithmetic and one rounding to fp32 (2^-24), doubled; the softmax without a bias sums in fp32:
    # at most 16 + 6 additions and the exponentials of a row, each off by 2^-24 or 2^-23
    assert (np.abs(w - want) <= np.abs(want) * 2.0 ** -19 + 1e-38).all()


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16], ids=["f32", "bf16"])
@pytest.mark.parametrize("kind", [block.SOFTMAX, block.SIGMOID], ids=["softmax", "sigmoid"])
@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_route_and_gradient(shape, kind, dtype):
    need_gpu()
    T, E, k, G, tg, gb = shape
    for bias_kind, renorm, grid in (("none", True, None), ("normal", True, None), ("zero", False, 4), ("none", False, 2)):
        print(f"route {shape} kind={kind} {dtype} bias={bias_kind} renorm={renorm}", flush=True)
        l = _logits(T, E, dtype, seed=E + k, grid=grid)
        bias = None if bias_kind == "none" else torch.zeros(E)
        if bias_kind == "normal":
            bias = torch.from_numpy(np.random.default_rng(1).standard_normal(E).astype(np.float32) * 0.05)
        kw = dict(n_group=G, topk_group=tg, group_best=gb)
        scale = 2.5
        want_idx, want_w = block.route(_f64(l), k, bias=None if bias is None else _f64(bias), kind=kind, renorm=renorm,
                                       scale=scale, **kw)
        gl = l.cuda()
        idx, w = bs.bs_moe_route(gl, k, bias=None if bias is None else bias.cuda(), score=kind, renormalize=renorm,
                                 scale=scale, **kw)
        torch.cuda.synchronize()
        assert np.array_equal(idx.cpu().numpy(), want_idx)
        _weights_close(w.cpu().double().numpy(), want_w)
        # gradient: k products of fp32 values and their difference, then s (1 - s): about 16 roundings of 2^-24
        g = torch.from_numpy(np.random.default_rng(2).standard_normal((T, k)).astype(np.float32))
        want = block.route_bwd(_f64(l), want_idx, g.numpy(), kind=kind, renorm=renorm, scale=scale)
        d = bs.bs_moe_route_bwd(gl, idx, w, g.cuda(), score=kind, renormalize=renorm, scale=scale)
        torch.cuda.synchronize()
        got = d.cpu().double().numpy()
        s = block.scores(_f64(l), kind)
        mag = np.zeros((T, E))
        for t in range(T):
            on = want_idx[t] >= 0
            e, c = want_idx[t][on], s[t, want_idx[t][on]]
            tot = c.sum() + (1e-20 if kind == block.SIGMOID else 0) if renorm and on.any() else 1.0
            mix = (np.abs(g.numpy()[t][on]) * c / tot).sum()
            if kind == block.SOFTMAX and not renorm:
                mag[t] = scale * s[t] * mix
            mag[t, e] += scale * c / tot * (np.abs(g.numpy()[t][on]) + mix)
        half = 2.0 ** -24 if dtype == torch.float32 else 2.0 ** -8
        assert (np.abs(got - want) <= np.abs(want) * half + mag * 2.0 ** -19 + 1e-38).all()


@pytest.mark.parametrize("E", [8, 64, 256])
def test_route_strided_and_unaligned_rows(E):
    need_gpu()
    for dtype in (torch.float32, torch.bfloat16):
        base = _logits(23, E + 7, dtype, seed=5).cuda()
        base[3:5] = 0.5
        for off in (0, 1, 3):
            l = base[:, off:off + E]
            print(f"route strides E={E} {dtype} off={off}", flush=True)
            a = bs.bs_moe_route(l, 4, score=bs.BS_SCORE_SIGMOID)
            b = bs.bs_moe_route(l.contiguous(), 4, score=bs.BS_SCORE_SIGMOID)
            assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
            dw = torch.ones_like(a[1]) * torch.arange(1, 5, device="cuda")
            full = torch.full((23, E + 7), 7.0, dtype=dtype, device="cuda")
            out = full[:, off:off + E]
            bs.bs_moe_route_bwd(l, *a, dw, score=bs.BS_SCORE_SIGMOID, out=out)
            ref = bs.bs_moe_route_bwd(l.contiguous(), *a, dw, score=bs.BS_SCORE_SIGMOID)
            assert torch.equal(out, ref)
            rest = torch.ones(E + 7, dtype=torch.bool)
            rest[off:off + E] = False
            assert (full[:, rest.cuda()] == 7.0).all()


def test_route_non_finite_logits():
    need_gpu()
    inf, nan = float("inf"), float("nan")
    l = torch.tensor([[0.0, nan, 1.0, 2.0, -inf, 0.5, 0.1, 0.2],
                      [inf, 0.0, 1.0, 2.0, -inf, 0.5, 0.1, 0.2]])
    for kind in (bs.BS_SCORE_SOFTMAX, bs.BS_SCORE_SIGMOID):
        for bias in (None, torch.zeros(8, device="cuda")):
            idx, w = bs.bs_moe_route(l.cuda(), 3, bias=bias, score=kind)
            idx, w = idx.cpu(), w.cpu()
            assert ((idx >= 0) & (idx < 8)).all() and (idx != 4).all()
            assert all(len(set(r.tolist())) == 3 for r in idx)
            assert idx[1, 0] == 0
            assert torch.isnan(w[0]).all()
            if kind == bs.BS_SCORE_SIGMOID:
                assert idx[0, 0] == 1
                assert torch.allclose(w[1], torch.sigmoid(l[1])[idx[1].long()] / torch.sigmoid(l[1])[idx[1].long()].sum())
            else:
                assert torch.isnan(w[1]).any()


def test_route_empty_batch_and_far_scores():
    need_gpu()
    idx, w = bs.bs_moe_route(torch.empty((0, 16), device="cuda"), 2)
    assert idx.shape == (0, 2) and w.shape == (0, 2)
    # sigmoid scores that underflow in fp32 keep their ratios in float64
    l = torch.full((1, 8), -30.0, device="cuda")
    idx, w = bs.bs_moe_route(l, 2, score=bs.BS_SCORE_SIGMOID)
    assert idx.cpu().tolist() == [[0, 1]] and torch.allclose(w.cpu(), torch.tensor([[0.5, 0.5]]), atol=1e-6)
    l = torch.full((1, 8), -80.0, device="cuda")     # sum far below 1e-20: the weights vanish, nothing is NaN
    _, w = bs.bs_moe_route(l, 2, score=bs.BS_SCORE_SIGMOID)
    assert (w.cpu() < 1e-10).all() and not torch.isnan(w).any()


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16], ids=["f32", "bf16"])
@pytest.mark.parametrize("kind", [block.SOFTMAX, block.SIGMOID], ids=["softmax", "sigmoid"])
@pytest.mark.parametrize("E,G", [(64, 1), (256, 8), (128, 1), (512, 4), (32, 4), (48, 3)])
def test_route_choices_next_to_one_another(E, G, kind, dtype):
    """A bias that brings the choice values within about an fp32 step of a few
    levels: only float64 tells them apart."""
    need_gpu()
    T, k = 24, min(8, E // G)
    l = _logits(T, E, dtype, seed=77)
    l[3:5] = 0.25
    s = block.scores(_f64(l), kind)
    for row, level in ((0, 0.75), (7, 0.125), (11, -0.5)):
        want = np.where(np.arange(E) % 3 == 0, level, level + 0.01)
        bias = torch.from_numpy((want - s[row]).astype(np.float32))
        kw = dict(n_group=G, topk_group=max(1, G // 2), group_best=2)
        print(f"route near ties E={E} G={G} kind={kind} {dtype} row={row}", flush=True)
        want_idx, want_w = block.route(_f64(l), k, bias=_f64(bias), kind=kind, **kw)
        idx, w = bs.bs_moe_route(l.cuda(), k, bias=bias.cuda(), score=kind, **kw)
        assert np.array_equal(idx.cpu().numpy(), want_idx)
        _weights_close(w.cpu().double().numpy(), want_w)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16], ids=["f32", "bf16"])
@pytest.mark.parametrize("kind", [block.SOFTMAX, block.SIGMOID], ids=["softmax", "sigmoid"])
@pytest.mark.parametrize("E,G,best", [(16, 4, 2), (16, 8, 2), (12, 4, 1), (24, 24, 1), (40, 8, 2), (160, 8, 2), (360, 9, 2),
                                      (513, 27, 2), (6, 2, 2)])
def test_route_groups_of_any_size(E, G, best, kind, dtype):
    """Groups that are no whole lanes: far apart, next to one another, tied."""
    need_gpu()
    T, k = 67, min(4, E // G * max(1, G // 2))
    kw = dict(n_group=G, topk_group=max(1, G // 2), group_best=best)
    for grid, biased in ((None, True), (2, True), (None, False), (2, False)):
        l = _logits(T, E, dtype, seed=E + G, grid=grid)
        bias = None
        if biased:
            level = np.where(np.arange(E) % 3 == 0, 0.5, 0.51)
            bias = torch.from_numpy((level - block.scores(_f64(l), kind)[0]).astype(np.float32))
        print(f"route groups E={E} G={G} kind={kind} {dtype} grid={grid} bias={biased}", flush=True)
        want_idx, want_w = block.route(_f64(l), k, bias=None if bias is None else _f64(bias), kind=kind, **kw)
        idx, w = bs.bs_moe_route(l.cuda(), k, bias=None if bias is None else bias.cuda(), score=kind, **kw)
        assert np.array_equal(idx.cpu().numpy(), want_idx)
        _weights_close(w.cpu().double().numpy(), want_w)


@pytest.mark.parametrize("E,G", [(16, 1), (16, 4), (64, 8), (256, 1)])
def test_route_bias_that_masks_experts(E, G):
    """An expert whose bias is -inf is never chosen, even where too few are left."""
    need_gpu()
    l = _logits(19, E, torch.float32, seed=2)
    bias = torch.zeros(E)
    bias[:E - 3] = -float("inf")
    for kind in (block.SOFTMAX, block.SIGMOID):
        kw = dict(kind=kind, n_group=G, topk_group=max(1, G // 2), group_best=2)
        want_idx, want_w = block.route(_f64(l), 6 if E > 16 else 4, bias=_f64(bias), **kw)
        print(f"route masking bias E={E} G={G} kind={kind}", flush=True)
        kw["score"] = kw.pop("kind")
        idx, w = bs.bs_moe_route(l.cuda(), 6 if E > 16 else 4, bias=bias.cuda(), **kw)
        assert (want_idx[:, 3:] == -1).all() and (want_idx[0, :3] >= E - 3).all()
        assert np.array_equal(idx.cpu().numpy(), want_idx)
        _weights_close(w.cpu().double().numpy(), want_w)


@pytest.mark.parametrize("E,G", [(64, 1), (24, 24), (256, 8)])
def test_route_tie_at_the_last_place_next_to_a_better_expert(E, G):
    """The k-th and (k+1)-th by fp32 tie, and a third, better by less than fp32
    tells, comes after them: ties that are real must not hide it."""
    need_gpu()
    T = 40
    l = torch.full((T, E), -4.0)
    l[:, :3] = torch.tensor([4.0, 3.0, 2.0])
    bias = torch.zeros(E)
    bias[E - 1] = 0.5 - 1.0 / (1.0 + float(np.exp(-0.25)))  # a score of 0.5, plus its rounding
    for step in (0, 1, 2):
        b = bias.clone()
        for _ in range(step):
            b[E - 1] = torch.nextafter(b[E - 1], torch.tensor(1.0))
        l[:, 5] = l[:, 9] = 0.0
        l[:, E - 1] = 0.25
        kw = dict(n_group=G, topk_group=G, group_best=1)
        print(f"route hidden tie E={E} G={G} step={step}", flush=True)
        want_idx, _ = block.route(_f64(l), 4, bias=_f64(b), kind=block.SIGMOID, **kw)
        idx, _ = bs.bs_moe_route(l.cuda(), 4, bias=b.cuda(), score=bs.BS_SCORE_SIGMOID, **kw)
        assert np.array_equal(idx.cpu().numpy(), want_idx)


@pytest.mark.parametrize("E", [8, 64, 256])
def test_route_gradient_where_one_expert_has_all_the_weight(E):
    """g_j - sum p_i g_i is 0 for k = 1 and tiny for an expert with nearly the
    whole sum: no rounding of the terms may stand for it."""
    need_gpu()
    T = 33
    rng = np.random.default_rng(E)
    l = torch.from_numpy(rng.standard_normal((T, E)).astype(np.float32))
    g = torch.from_numpy(rng.standard_normal((T, 3)).astype(np.float32))
    for kind in (block.SOFTMAX, block.SIGMOID):
        print(f"route gradient E={E} kind={kind} k=1", flush=True)
        idx, w = bs.bs_moe_route(l.cuda(), 1, score=kind, scale=2.5)
        d = bs.bs_moe_route_bwd(l.cuda(), idx, w, g[:, :1].contiguous().cuda(), score=kind, scale=2.5).cpu()
        # the sigmoid's 1e-20 leaves scale g 1e-20 (1 - s) / s, s >= sigmoid(-6) = 2^-8.7
        assert d.abs().max() <= 2.5 * 6 * 1e-20 * 2.0 ** 9
    # softmax over the chosen: dl_j = scale p_j sum p_i (g_j - g_i), which does not cancel
    l[:, 5] += 30.0
    print(f"route gradient E={E} one expert dominates", flush=True)
    idx, w = bs.bs_moe_route(l.cuda(), 3, scale=2.5)
    d = bs.bs_moe_route_bwd(l.cuda(), idx, w, g.cuda(), scale=2.5).cpu().double().numpy()
    for t in range(T):
        e = idx[t].cpu().numpy()
        p = np.exp(_f64(l)[t, e] - _f64(l)[t, e].max())
        p /= p.sum()
        gt = g[t].double().numpy()
        diff = gt[:, None] - gt[None]
        want, mag = 2.5 * p * (p * diff).sum(1), 2.5 * p * (p * np.abs(diff)).sum(1)
        # expf of differences up to 36 (2^-24 of them each) and a few roundings; differences of g are exact to 2^-24
        # of their terms, which two shares enter at most
        mag += 2.5 * p * p.max() * np.abs(gt).max() * (p < 0.5) + 2.5 * p * (1 - p) * np.abs(gt).max()
        assert (np.abs(d[t, e] - want) <= mag * 2.0 ** -17 + 1e-30).all()


def test_route_gradient_of_scores_as_small_as_the_added_term():
    """Sigmoid scores about 1e-20: the term added to their sum takes part."""
    need_gpu()
    l = torch.tensor([[-46.0, -47.0, -60.0, -50.0], [-44.0, -44.0, -70.0, -46.0], [-90.0, -91.0, -92.0, -93.0]])
    g = torch.tensor([[1.0, -0.5], [2.0, 0.25], [0.5, 3.0]])
    print("route gradient of tiny scores", flush=True)
    idx, w = bs.bs_moe_route(l.cuda(), 2, score=block.SIGMOID, scale=2.0)
    d = bs.bs_moe_route_bwd(l.cuda(), idx, w, g.cuda(), score=block.SIGMOID, scale=2.0).cpu().double().numpy()
    want = block.route_bwd(_f64(l), idx.cpu().numpy(), g.numpy(), kind=block.SIGMOID, scale=2.0)
    want_idx, want_w = block.route(_f64(l), 2, kind=block.SIGMOID, scale=2.0)
    assert np.array_equal(idx.cpu().numpy(), want_idx)
    _weights_close(w.cpu().double().numpy(), want_w)
    # expf of numbers up to 93 and about 16 more roundings of terms as large as f (|g| + sum p |g|) s
    s = block.scores(_f64(l), block.SIGMOID)
    e = idx.cpu().numpy()
    c = np.take_along_axis(s, e, 1)
    mag = np.zeros_like(want)
    np.put_along_axis(mag, e, 2.0 * c / (c.sum(1, keepdims=True) + 1e-20) * 2 * np.abs(g.numpy()).max(1, keepdims=True), 1)
    assert (np.abs(d - want) <= mag * 2.0 ** -19 + 1e-37).all()
