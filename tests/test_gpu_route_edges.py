"""GPU router where fp32 alone would answer wrongly: ties hidden behind ties,
and gradients that are what is left of a cancellation."""

import numpy as np
import pytest
import torch

import blockwise_scaled_fp8_bs_amd as bs
from gpu_support import need_gpu
from oracle import block

pytestmark = pytest.mark.gpu


def _f64(t):
    return t.double().numpy()


@pytest.mark.parametrize("E,G,tg", [(64, 4, 2), (256, 8, 2), (24, 8, 4), (40, 8, 3)])
def test_route_hidden_tie_after_the_groups_are_chosen(E, G, tg):
    """As test_route_tie_at_the_last_place_next_to_a_better_expert, with groups
    dropped: groups of whole lanes (64, 256) and of other sizes."""
    need_gpu()
    l = torch.full((40, E), -4.0)
    l[:, :3] = torch.tensor([4.0, 3.0, 2.0])
    l[:, 5] = l[:, 9] = 0.0
    l[:, E - 1] = 0.25
    assert len({e // (E // G) for e in (0, 1, 2, 5, 9, E - 1)}) == tg < G
    bias = torch.zeros(E)
    bias[E - 1] = 0.5 - 1.0 / (1.0 + float(np.exp(-0.25)))  # a score of 0.5, plus its rounding
    seen = set()
    for step in range(-2, 3):
        b = bias.clone()
        for _ in range(abs(step)):
            b[E - 1] = torch.nextafter(b[E - 1], torch.tensor(float(np.sign(step))))
        kw = dict(n_group=G, topk_group=tg, group_best=1)
        print(f"route hidden tie in groups E={E} G={G} step={step}", flush=True)
        want_idx, want_w = block.route(_f64(l), 4, bias=_f64(b), kind=block.SIGMOID, **kw)
        idx, w = bs.bs_moe_route(l.cuda(), 4, bias=b.cuda(), score=bs.BS_SCORE_SIGMOID, **kw)
        assert np.array_equal(idx.cpu().numpy(), want_idx)
        # fp32 exponentials, k additions and a quotient
        assert (np.abs(w.cpu().double().numpy() - want_w) <= want_w * 2.0 ** -19).all()
        seen.add(int(want_idx[0, 3]))
    assert seen == {5, E - 1}  # both sides of the tie were met


@pytest.mark.parametrize("lead", [0.0, 4.0, 12.0, 16.0, 20.0, 30.0, 60.0])
@pytest.mark.parametrize("E,k", [(8, 1), (8, 3), (64, 6), (256, 8), (1000, 32)])
def test_route_gradient_of_plain_softmax_where_one_expert_has_all_the_weight(E, k, lead):
    """dl_j = scale p_j sum_e p_e (G_j - G_e), G_e = dw of a chosen expert and 0
    of the others: the term of j itself is 0, and with a lead p_j (1 - p_j) is
    far below the rounding of p_j."""
    need_gpu()
    T, scale = 19, 2.5
    rng = np.random.default_rng(E + k)
    l = rng.standard_normal((T, E)).astype(np.float32)
    ahead = rng.integers(0, E, T)
    l[np.arange(T), ahead] = l.max(axis=1) + np.float32(lead)
    if E > 2 * k:
        l[1, :E // 2] = -np.inf
    l = torch.from_numpy(l)
    g = torch.from_numpy(rng.standard_normal((T, k)).astype(np.float32))
    g[2] = 0.7
    print(f"route plain softmax gradient E={E} k={k} lead={lead}", flush=True)
    idx, w = bs.bs_moe_route(l.cuda(), k, renormalize=False, scale=scale)
    d = bs.bs_moe_route_bwd(l.cuda(), idx, w, g.cuda(), renormalize=False, scale=scale).cpu().double().numpy()
    L, at = _f64(l), idx.cpu().numpy()
    p = np.exp(L - L.max(axis=1, keepdims=True))
    p /= p.sum(axis=1, keepdims=True)
    G = np.zeros((T, E))
    np.put_along_axis(G, at, g.double().numpy(), 1)
    diff = G[:, :, None] - G[:, None, :]
    want = scale * p * (p[:, None, :] * diff).sum(axis=2)
    # Terms that the kernel adds: (1 - p_j) G_j and p_e G_e of the others.  Relative errors in units of 2^-24: a share
    # has lead + 5 from its exponent, 2 from the exponential, 25 from the sum and 5 from products and quotients; there
    # are two in a term, and up to 40 additions: 2 (65 + 37) + 40 < 256.
    others = np.ones((E, E)) - np.eye(E)
    mag = scale * p * (np.abs(G) * (p @ others) + (p * np.abs(G)) @ others)
    assert (np.abs(d - want) <= mag * 2.0 ** -16 + 1e-36).all()


@pytest.mark.parametrize("kind", [block.SOFTMAX, block.SIGMOID], ids=["softmax", "sigmoid"])
def test_route_gradient_of_plain_weights_equals_differences(kind):
    """Of the float64 oracle's forward, one logit of a token ahead of the others."""
    need_gpu()
    T, E, k = 5, 16, 3
    rng = np.random.default_rng(8)
    l = rng.standard_normal((T, E)).astype(np.float32)
    l[np.arange(T), 3] += np.float32(2.0) * np.arange(T, dtype=np.float32)
    g = rng.standard_normal((T, k)).astype(np.float32)
    gl = torch.from_numpy(l).cuda()
    print(f"route plain gradient against differences, kind {kind}", flush=True)
    idx, w = bs.bs_moe_route(gl, k, score=kind, renormalize=False, scale=1.5)
    d = bs.bs_moe_route_bwd(gl, idx, w, torch.from_numpy(g).cuda(), score=kind, renormalize=False, scale=1.5).cpu().numpy()
    want, h = np.zeros((T, E)), 1e-6
    for t in range(T):
        for e in range(E):
            ends = []
            for step in (h, -h):
                m = l.astype(np.float64)
                m[t, e] += step
                ends.append((block.route(m, k, kind=kind, renorm=False, scale=1.5)[1] * g).sum())
            want[t, e] = (ends[0] - ends[1]) / (2 * h)
    # differences: float64's 2^-52 of sums of about 10, over 2e-6, and the third derivative's h^2; the kernel's fp32
    assert np.abs(d - want).max() < 1e-5
