"""GPU gated activation with an 8-bit checkpoint: codes of h and of [a | b]
bit for bit, and the backward from them bit for bit against the float64
formula at the kept values."""

import numpy as np
import pytest
import torch

import blockwise_scaled_fp8_bs_amd as bs
from gpu_support import (bits16, check_canaries, check_scale_canaries, f32bits, guarded, need_gpu, scale_buffer, u8)
from oracle import block, quant, swiglu
from test_gpu_swiglu import _inputs

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("R,C,cols", [(256, 512, True), (128, 128, True), (384, 640, True), (1, 128, False),
                                      (200, 256, False)])
def test_forward_and_backward(R, C, cols):
    need_gpu()
    a, b = _inputs(R, C, seed=R + C)
    dh = torch.randn((R, C), generator=torch.Generator().manual_seed(3)).mul_(0.01).to(torch.bfloat16)
    ab = torch.cat([a, b], 1).cuda()
    kf, ck = guarded(R, 2 * C, torch.uint8, pad_cols=32)
    pf, s_ck = scale_buffer(2 * C // 128, R)
    qf, q = guarded(R, C, torch.uint8)
    sf, s = scale_buffer(C // 128, R)
    out = dict(q_row=q, s_row=s)
    if cols:
        cf, c = guarded(C, R, torch.uint8)
        tf, t = scale_buffer(R // 128, C)
        out.update(q_col=c, s_col=t)
    print(f"ckpt forward R={R} C={C}", flush=True)
    bs.bs_swiglu_quant_1x128_ckpt(ab[:, :C], ab[:, C:], ck, s_ck, **out)
    torch.cuda.synchronize()
    hb = swiglu.swiglu(bits16(a), bits16(b))
    qr, sr = quant.quant_1x128_rowwise(hb)
    assert np.array_equal(u8(q), qr) and np.array_equal(f32bits(s)[:, :R], sr.T.copy().view(np.uint32))
    kr, ks = quant.quant_1x128_rowwise(np.concatenate([bits16(a), bits16(b)], 1))
    assert np.array_equal(u8(ck), kr) and np.array_equal(f32bits(s_ck)[:, :R], ks.T.copy().view(np.uint32))
    check_canaries(kf, R, 2 * C), check_canaries(qf, R, C)
    check_scale_canaries(pf, 2 * C // 128, R), check_scale_canaries(sf, C // 128, R)
    if cols:
        qc, sc = quant.quant_1x128_colwise(hb)
        assert np.array_equal(u8(c), qc) and np.array_equal(f32bits(t)[:, :C], sc.T.copy().view(np.uint32))
        check_canaries(cf, C, R), check_scale_canaries(tf, R // 128, C)

    kept = block.dequant_rows(kr, ks)
    da = swiglu.round_to_bf16(np.concatenate(block.swiglu_grad(kept[:, :C], kept[:, C:], block.f64(bits16(dh))), 1))
    qf, q = guarded(R, 2 * C, torch.uint8)
    sf, s = scale_buffer(2 * C // 128, R)
    out = dict(q_row=q, s_row=s)
    if cols:
        cf, c = guarded(2 * C, R, torch.uint8)
        tf, t = scale_buffer(R // 128, 2 * C)
        out.update(q_col=c, s_col=t)
    print(f"ckpt backward R={R} C={C}", flush=True)
    bs.bs_swiglu_bwd_quant_1x128_ckpt(ck, s_ck, dh.cuda(), **out)
    torch.cuda.synchronize()
    qr, sr = quant.quant_1x128_rowwise(da)
    assert np.array_equal(f32bits(s)[:, :R], sr.T.copy().view(np.uint32)) and np.array_equal(u8(q), qr)
    check_canaries(qf, R, 2 * C), check_scale_canaries(sf, 2 * C // 128, R)
    if cols:
        qc, sc = quant.quant_1x128_colwise(da)
        assert np.array_equal(u8(c), qc) and np.array_equal(f32bits(t)[:, :2 * C], sc.T.copy().view(np.uint32))
        check_canaries(cf, 2 * C, R), check_scale_canaries(tf, R // 128, 2 * C)
        for only in (("q_row", "s_row"), ("q_col", "s_col")):
            for n in only:
                out[n].fill_(0)
            bs.bs_swiglu_bwd_quant_1x128_ckpt(ck, s_ck, dh.cuda(), **{n: out[n] for n in only})
            assert np.array_equal(u8(out[only[0]]), qr if only[0] == "q_row" else qc)


def test_forward_equals_the_form_without_a_checkpoint():
    need_gpu()
    R, C = 512, 384
    a, b = (t.cuda() for t in _inputs(R, C, seed=11))
    mk = lambda: dict(q_row=torch.empty((R, C), dtype=torch.uint8, device="cuda"), s_row=bs.empty_scales(C // 128, R, "cuda"),  # noqa: E731
                      q_col=torch.empty((C, R), dtype=torch.uint8, device="cuda"), s_col=bs.empty_scales(R // 128, C, "cuda"))
    x, y = mk(), mk()
    ck, s_ck = torch.empty((R, 2 * C), dtype=torch.uint8, device="cuda"), bs.empty_scales(2 * C // 128, R, "cuda")
    bs.bs_swiglu_quant_1x128_ckpt(a, b, ck, s_ck, **x)
    bs.bs_swiglu_quant_1x128(a, b, None, **y)
    assert all(torch.equal(x[n], y[n]) for n in x)


def test_many_tiles_equal_few():
    """288 tiles, one workgroup each, against the same rows 48 or 96 tiles at a time, each shared by two."""
    need_gpu()
    R, C = 2304, 2048
    a, b = (t.cuda() for t in _inputs(R, C, seed=21))
    dh = torch.randn((R, C), generator=torch.Generator().manual_seed(4)).mul_(0.01).to(torch.bfloat16).cuda()
    new = lambda r, c: dict(q_row=torch.zeros((r, c), dtype=torch.uint8, device="cuda"), s_row=bs.empty_scales(c // 128, r, "cuda"))  # noqa: E731

    def run(lo, hi, cols):
        n = hi - lo
        ck, s_ck, h, g = torch.zeros((n, 2 * C), dtype=torch.uint8, device="cuda"), bs.empty_scales(2 * C // 128, n, "cuda"), new(n, C), new(n, 2 * C)
        if cols:
            for d, c in ((h, C), (g, 2 * C)):
                d.update(q_col=torch.zeros((c, n), dtype=torch.uint8, device="cuda"), s_col=bs.empty_scales(n // 128, c, "cuda"))
        bs.bs_swiglu_quant_1x128_ckpt(a[lo:hi], b[lo:hi], ck, s_ck, **h)
        bs.bs_swiglu_bwd_quant_1x128_ckpt(ck, s_ck, dh[lo:hi], **g)
        return ck, s_ck, h, g

    print("ckpt many tiles against few", flush=True)
    ck, s_ck, h, g = run(0, R, True)
    for lo in range(0, R, 384):
        part = run(lo, lo + 384, False)
        assert torch.equal(ck[lo:lo + 384], part[0]) and torch.equal(s_ck[:, lo:lo + 384], part[1][:, :384])
        for whole, few in ((h, part[2]), (g, part[3])):
            assert torch.equal(whole["q_row"][lo:lo + 384], few["q_row"])
            assert torch.equal(whole["s_row"][:, lo:lo + 384], few["s_row"][:, :384])
    for lo in range(0, R, 768):
        part = run(lo, lo + 768, True)
        for whole, few in ((h, part[2]), (g, part[3])):
            assert torch.equal(whole["q_col"][:, lo:lo + 768], few["q_col"])
            assert torch.equal(whole["s_col"][lo // 128:lo // 128 + 6, :whole["q_col"].shape[0]],
                               few["s_col"][:, :whole["q_col"].shape[0]])


@pytest.mark.parametrize("C", [128, 33 * 1024])
def test_gate_values_near_the_largest_bf16(C):
    """a from 1e38 to the largest bf16, where the fp32 exponential's exponent overflows, and their negatives: both
    outputs against the float64 formula, with few tiles and (C = 33 * 1024, 264 of them) with many."""
    need_gpu()
    R = 128
    big = np.array([1e38, 2.3e38, 2.4e38, 3.3895e38], dtype=np.float32)
    a = torch.from_numpy(np.tile(np.concatenate([big, -big]), R * C // 8).reshape(R, C)).to(torch.bfloat16)
    b, dh = inputs_like(a, 1e-20, 5), inputs_like(a, 1e-20, 6)
    ck, s_ck = torch.empty((R, 2 * C), dtype=torch.uint8, device="cuda"), bs.empty_scales(2 * C // 128, R, "cuda")
    q, s = torch.empty((R, C), dtype=torch.uint8, device="cuda"), bs.empty_scales(C // 128, R, "cuda")
    print(f"ckpt large gates C={C}", flush=True)
    bs.bs_swiglu_quant_1x128_ckpt(a.cuda(), b.cuda(), ck, s_ck, q_row=q, s_row=s)
    hr, hs = quant.quant_1x128_rowwise(swiglu.swiglu(bits16(a), bits16(b)))
    assert np.array_equal(u8(q), hr) and np.array_equal(f32bits(s)[:, :R], hs.T.copy().view(np.uint32))
    kr, ks = quant.quant_1x128_rowwise(np.concatenate([bits16(a), bits16(b)], 1))
    assert np.array_equal(u8(ck), kr)
    kept = block.dequant_rows(kr, ks)
    with np.errstate(over="ignore"):
        want = swiglu.round_to_bf16(np.concatenate(block.swiglu_grad(kept[:, :C], kept[:, C:], block.f64(bits16(dh))), 1))
    q, s = torch.empty((R, 2 * C), dtype=torch.uint8, device="cuda"), bs.empty_scales(2 * C // 128, R, "cuda")
    bs.bs_swiglu_bwd_quant_1x128_ckpt(ck, s_ck, dh.cuda(), q_row=q, s_row=s)
    qr, sr = quant.quant_1x128_rowwise(want)
    assert np.array_equal(f32bits(s)[:, :R], sr.T.copy().view(np.uint32)) and np.array_equal(u8(q), qr)


def inputs_like(t, sigma, seed):
    return (torch.randn(t.shape, generator=torch.Generator().manual_seed(seed)) * sigma).to(torch.bfloat16)
