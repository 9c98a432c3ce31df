"""GPU residual norms against the float64 oracle: r bit for bit (a float64
value rounded once), h, codes and gradients within their roundings."""

import numpy as np
import pytest
import torch

import blockwise_scaled_fp8_bs_amd as bs
from blockwise_scaled_fp8_bs_amd import inputs
from gpu_support import bits16, check_canaries, check_scale_canaries, guarded, need_gpu, scale_buffer, u8
from oracle import block, swiglu

pytestmark = pytest.mark.gpu

EPS, ALPHA = 1e-6, 0.375


def _case(B, S, D, post, gated, dtype, seed=0):
    R = B * S
    c = {"x": inputs.bf16_normal((R, D), 2.0, seed), "dh": inputs.bf16_normal((R, D), 0.1, seed + 1),
         "dr": inputs.bf16_normal((R, D), 0.1, seed + 2)}
    g = torch.Generator().manual_seed(seed + 3)
    c["w_pre"] = (1 + 0.2 * torch.randn(D, generator=g)).to(dtype)
    c["u"] = inputs.bf16_normal((R, D), 0.7, seed + 4) if post is not None else None
    c["w_post"] = (1 + 0.2 * torch.randn(D, generator=g)).to(dtype) if post else None
    c["gate"] = torch.randn((B, D), generator=g).to(dtype) if gated else None
    return c


def _np(t):
    return None if t is None else t.double().numpy()


def _gpu(t, pad=0):
    if t is None:
        return None
    if not pad:
        return t.cuda()
    full = torch.full((t.shape[0], t.shape[1] + pad), 3.0, dtype=t.dtype, device="cuda")
    full[:, :t.shape[1]] = t.cuda()
    return full[:, :t.shape[1]]


CASES = [  # B, S, D, post (None: no u, 0: u without a norm), gate, type of the parameters, quantized
    (1, 1, 4096, 1, 1, torch.bfloat16, ""), (1, 1, 8, 1, 1, torch.float32, ""), (3, 5, 40, 1, 1, torch.float32, ""),
    (1, 7, 520, 1, 0, torch.float32, ""), (5, 1, 1032, 1, 1, torch.bfloat16, ""), (2, 33, 2048, 1, 1, torch.float32, ""),
    (1, 9, 2056, 0, 1, torch.float32, ""), (1, 37, 1024, None, 0, torch.float32, ""),
    (1, 130, 640, 1, 1, torch.float32, "rows"), (4, 19, 5120, 1, 1, torch.bfloat16, "rows"),
    (1, 3, 16384, 1, 1, torch.float32, "rows"), (1, 5, 8192, None, 0, torch.bfloat16, "rows"),
    (1, 128, 256, 1, 1, torch.float32, "both"), (2, 192, 512, 1, 1, torch.float32, "both"),
    (1, 256, 4096, None, 0, torch.float32, "both"), (1, 128, 6144, 0, 0, torch.bfloat16, "both"),
    (1, 1300, 128, 1, 1, torch.float32, "rows"), (700, 3, 64, 1, 1, torch.float32, ""),
]


@pytest.mark.parametrize("case", CASES, ids=str)
def test_forward_and_backward(case):
    need_gpu()
    B, S, D, post, gated, dtype, quantized = case
    R = B * S
    c = _case(B, S, D, post, gated, dtype)
    X, U, WQ, G, WP, DH, DR = (_np(c[n]) for n in ("x", "u", "w_post", "gate", "w_pre", "dh", "dr"))
    has_u = c["u"] is not None
    x, u = _gpu(c["x"], 16), _gpu(c["u"], 8)
    gate = _gpu(c["gate"], 8)
    rf, r = guarded(R, D, torch.bfloat16)
    hf, h = guarded(R, D, torch.bfloat16)
    rstd_u = torch.full((R,), 7.0, device="cuda") if post else None
    rstd_r = torch.full((R,), 7.0, device="cuda")
    out = {}
    if quantized:
        qf, q = guarded(R, D, torch.uint8)
        sf, s = scale_buffer(D // 128, R)
        out.update(q_row=q, s_row=s)
        if quantized == "both":
            cf, cc = guarded(D, R, torch.uint8)
            tf, t = scale_buffer(R // 128, D)
            out.update(q_col=cc, s_col=t)
    print(f"norm {case}", flush=True)
    params = dict(u=u, w_post=_gpu(c["w_post"]), gate=gate, alpha=ALPHA)
    bs.bs_resid_norm(x, _gpu(c["w_pre"]), **params, eps=EPS, r=r if has_u else None, h=h, rstd_u=rstd_u,
                     rstd_r=rstd_r, **out)
    torch.cuda.synchronize()
    rb = bits16(c["x"])
    if has_u:
        rb = swiglu.round_to_bf16(block.resid(X, U, WQ, G, ALPHA, float(np.float32(EPS))))
        assert np.array_equal(bits16(r), rb)
        check_canaries(rf, R, D)
    RR = block.f64(rb)
    eps32 = float(np.float32(EPS))
    want_rstd = block.rstd(RR, eps32)
    assert (np.abs(rstd_r.cpu().double().numpy() - want_rstd) <= want_rstd * 2.0 ** -23).all()
    if post:
        wu = block.rstd(U, eps32)
        assert (np.abs(rstd_u.cpu().double().numpy() - wu) <= wu * 2.0 ** -23).all()
    H = block.norm(RR, WP, eps32)
    # rstd rounded once, two products: 3 x 2^-24
    assert (np.abs(block.f64(bits16(h)) - H) <= np.abs(H) * (2.0 ** -8 + 2.0 ** -21) + 1e-38).all()
    check_canaries(hf, R, D)
    if quantized:
        assert max(block.check_codes(u8(q), s.cpu().numpy()[:, :R].T, H, 2.0 ** -22)) <= 1
        check_canaries(qf, R, D), check_scale_canaries(sf, D // 128, R)
    if quantized == "both":
        assert max(block.check_codes(u8(cc), t.cpu().numpy()[:, :D].T, H.T.copy(), 2.0 ** -22)) <= 1
        check_canaries(cf, D, R), check_scale_canaries(tf, R // 128, D)

    # backward, with and without the residual's gradient
    for with_dr in (True, False):
        g = bs.bs_resid_norm_bwd(r if has_u else x, rstd_r, _gpu(c["w_pre"]), _gpu(c["dh"], 24),
                                 dr=_gpu(c["dr"], 8) if with_dr else None, rstd_u=rstd_u, **params)
        torch.cuda.synchronize()
        dr = DR if with_dr else None
        want = block.norm_bwd(RR, WP, DH, dr, U, WQ, G, ALPHA, eps32)
        _check_grads(g, want, RR, WP, DH, dr, U, WQ, G, eps32, R, D, B)


def _check_grads(g, want, RR, WP, DH, dr, U, WQ, G, eps, R, D, B):
    # magnitudes whose roundings reach each gradient; sums over a row: at most 64 additions one after another
    # (8 chunks of 8, 6 exchanges, 2), sums over rows: those of one workgroup, then float64
    u24, depth = 2.0 ** -24, 96
    s = block.rstd(RR, eps)[:, None]
    n = np.abs(RR * s)
    q = np.abs(DH * WP)
    m_dr = s * (q + n * (q * n).mean(axis=1, keepdims=True)) + (0 if dr is None else np.abs(dr))
    close = lambda a, w, mag, half: (np.abs(a - w) <= np.abs(w) * half + mag * depth * u24 + 1e-37).all()  # noqa: E731
    assert close(g.dx.cpu().double().numpy(), want["dx"], m_dr, 2.0 ** -8)
    assert close(g.dw_pre.cpu().double().numpy(), want["dw_pre"], (np.abs(DH) * n).sum(axis=0), u24)
    if U is None:
        assert g.du is None and g.dw_post is None and g.dgate is None
        return
    gg = 1.0 if G is None else np.repeat(np.abs(G), R // B, axis=0)
    dp = ALPHA * gg * m_dr
    if WQ is None:
        assert g.dw_post is None
        assert close(g.du.cpu().double().numpy(), want["du"], dp, 2.0 ** -8)
        m, wq = np.abs(U), 1.0
    else:
        su = block.rstd(U, eps)[:, None]
        m, wq = np.abs(U * su), np.abs(WQ)
        dm = dp * wq
        assert close(g.du.cpu().double().numpy(), want["du"], su * (dm + m * (dm * m).mean(axis=1, keepdims=True)),
                     2.0 ** -8)
        assert close(g.dw_post.cpu().double().numpy(), want["dw_post"], (dp * m).sum(axis=0), u24)
    if G is not None:
        mag = (ALPHA * m_dr * m * wq).reshape(B, R // B, D).sum(axis=1)
        assert close(g.dgate.cpu().double().numpy(), want["dgate"], mag, u24)


@pytest.mark.parametrize("post,gated", [(1, 1), (0, 1), (1, 0)])
def test_residual_alone(post, gated):
    """No norm of r: r only, and its backward from dr."""
    need_gpu()
    B, S, D = 3, 11, 264
    c = _case(B, S, D, post, gated, torch.float32, seed=3)
    X, U, WQ, G, DR = (_np(c[n]) for n in ("x", "u", "w_post", "gate", "dr"))
    r = torch.empty((B * S, D), dtype=torch.bfloat16, device="cuda")
    ru = torch.empty(B * S, device="cuda") if post else None
    params = dict(u=_gpu(c["u"]), w_post=_gpu(c["w_post"]), gate=_gpu(c["gate"]), alpha=ALPHA)
    print(f"norm residual alone post={post} gate={gated}", flush=True)
    bs.bs_resid_norm(_gpu(c["x"]), **params, eps=EPS, r=r, rstd_u=ru)
    eps = float(np.float32(EPS))
    assert np.array_equal(bits16(r), swiglu.round_to_bf16(block.resid(X, U, WQ, G, ALPHA, eps)))
    g = bs.bs_resid_norm_bwd(None, None, None, None, dr=_gpu(c["dr"]), rstd_u=ru, **params)
    want = block.norm_bwd(None, None, None, DR, U, WQ, G, ALPHA, eps)
    assert g.dw_pre is None and torch.equal(g.dx.cpu().view(torch.int16), c["dr"].view(torch.int16))
    got = g.du.cpu().double().numpy()
    assert (np.abs(got - want["du"]) <= np.abs(want["du"]) * 2.0 ** -7 + 1e-5).all()
    for n in ("dw_post", "dgate"):
        v = getattr(g, n)
        assert (v is None) == (n not in want)
        if v is not None:
            assert np.allclose(v.cpu().double().numpy(), want[n], rtol=1e-5, atol=1e-5)


def test_extreme_rows_in_place_and_many_rows():
    need_gpu()
    D = 512
    x = inputs.bf16_normal((6, D), 1.0, 1)
    x[0] = 0
    x[1] = 3e38                     # squares leave fp32's range
    x[2] = 1e-30
    x[3] = torch.finfo(torch.bfloat16).tiny
    x[4, 0] = -3e38
    w = torch.ones(D)
    h = torch.empty((6, D), dtype=torch.bfloat16, device="cuda")
    bs.bs_resid_norm(x.cuda(), w.cuda(), eps=1e-6, h=h)
    X = x.double().numpy()
    want = block.norm(X, np.ones(D), float(np.float32(1e-6)))
    got = h.cpu().double().numpy()
    # rstd of the largest rows is a subnormal fp32 of about 20 bits
    assert (np.abs(got - want) <= np.abs(want) * 2.0 ** -7 + 1e-37).all()
    assert not got[0].any()
    # r written over x
    c = _case(1, 6, D, 1, 1, torch.float32, seed=9)
    a, b = c["x"].cuda(), torch.empty((6, D), dtype=torch.bfloat16, device="cuda")
    params = dict(u=_gpu(c["u"]), w_post=_gpu(c["w_post"]), gate=_gpu(c["gate"]), alpha=ALPHA)
    bs.bs_resid_norm(a, **params, r=b)
    bs.bs_resid_norm(a, **params, r=a)
    assert torch.equal(a.view(torch.int16), b.view(torch.int16))
    # more rows than workgroups of the backward pass, twice the same bits
    R = 5000
    c = _case(1, R, D, 1, 1, torch.float32, seed=10)
    params = {n: _gpu(c[n]) for n in ("u", "w_post", "gate")}
    r, ru, rr = torch.empty((R, D), dtype=torch.bfloat16, device="cuda"), torch.empty(R, device="cuda"), torch.empty(R, device="cuda")
    bs.bs_resid_norm(c["x"].cuda(), c["w_pre"].cuda(), **params, alpha=ALPHA, eps=EPS, r=r, rstd_u=ru, rstd_r=rr)
    runs = [bs.bs_resid_norm_bwd(r, rr, c["w_pre"].cuda(), c["dh"].cuda(), dr=c["dr"].cuda(), rstd_u=ru, alpha=ALPHA, **params)
            for _ in range(2)]
    for p, q in zip(*runs):
        assert torch.equal(p, q)
    want = block.norm_bwd(block.f64(bits16(r)), _np(c["w_pre"]), _np(c["dh"]), _np(c["dr"]), _np(c["u"]),
                          _np(c["w_post"]), _np(c["gate"]), ALPHA, float(np.float32(EPS)))
    _check_grads(runs[0], want, block.f64(bits16(r)), _np(c["w_pre"]), _np(c["dh"]), _np(c["dr"]), _np(c["u"]),
                 _np(c["w_post"]), _np(c["gate"]), float(np.float32(EPS)), R, D, 1)


@pytest.mark.parametrize("case", [(6, 300, 256, 1, 1, torch.float32, ""), (9, 1000, 64, 1, 1, torch.bfloat16, ""),
                                  (1, 5000, 72, 1, 1, torch.float32, ""), (2, 9000, 40, 1, 1, torch.float32, ""),
                                  (1, 4100, 1040, 1, 0, torch.float32, "")], ids=str)
def test_many_partial_sums(case):
    """More workgroups than parts of a column sum, a number of gate segments that fills no whole workgroup."""
    test_forward_and_backward(case)
