"""GPU gated activation with an 8-bit checkpoint, gate value by gate value: h,
da and db against their float64 formulas rounded once to bf16.

The kernels give codes and scales only.  Each row holds one element that is
not 0, on the diagonal of its tile, so that the scale of its block, the 448th
part of that element's magnitude, tells the element to its last bit; b or dh
is scaled so that none falls under the quantizer's floor of 1e-12."""

import numpy as np
import pytest
import torch

import blockwise_scaled_fp8_bs_amd as bs
from gpu_support import bf16_from_bits, need_gpu
from oracle import block, swiglu
from oracle.quant import bf16_bits_to_f32

pytestmark = pytest.mark.gpu

R, C = 65536, 128
DIAGONAL = np.arange(R) % C


def _bf16(v):
    return bf16_bits_to_f32(swiglu.round_to_bf16(v)).astype(np.float64)


def _even_out(v):
    """The power of two that brings |v| near 1, within bf16's range."""
    _, e = np.frexp(np.where(v == 0, 1.0, v))
    return np.exp2(np.clip(-e, -120, 120).astype(float))


def _mantissas(kind, seed):
    if kind != "random":
        return np.full(R, float(kind))
    return _bf16(np.random.default_rng(seed).uniform(1, 2, R) * np.random.default_rng(seed + 1).choice([-1, 1], R))


def _diagonal(v):
    """bf16 matrix [R, C] with v on the diagonals of its tiles."""
    m = np.zeros((R, C), dtype=np.uint16)
    m[np.arange(R), DIAGONAL] = swiglu.round_to_bf16(v)
    return bf16_from_bits(m).cuda()


def _scale_of(bits):
    mag = np.abs(bf16_bits_to_f32(bits))
    return (np.maximum(mag, np.float32(1e-12)) / np.float32(448)).astype(np.float32)


def _check(got, v, slack):
    """got: scales of blocks whose largest element is v (float64, known to slack, relative) rounded to bf16."""
    on = np.abs(v) < 3.3e38
    assert on.mean() > 0.9
    bits = swiglu.round_to_bf16(np.where(on, v, 0.0))
    wrong = on & (got.view(np.uint32) != _scale_of(bits).view(np.uint32))
    if wrong.any():
        x = np.abs(v[wrong])
        _, e = np.frexp(x)
        step = np.ldexp(1.0, np.maximum(e - 8, -133))
        tie = np.abs(x / step - np.floor(x / step) - 0.5) * step < x * slack[wrong]
        near = np.zeros(x.shape, dtype=bool)
        for d in (-1, 1):
            near |= got[wrong] == _scale_of((bits[wrong].astype(np.int32) + d).astype(np.uint16))
        assert (tie & near).all(), f"{(~(tie & near)).sum()} of {wrong.sum()} off, first v {v[wrong][~(tie & near)][:3]}"
    return int(wrong.sum())


def _parts(whole):
    """Row ranges: 512 tiles at once, a workgroup each, or 256 at a time, each shared by two."""
    return [(0, R)] if whole else [(0, R // 2), (R // 2, R)]


@pytest.mark.parametrize("whole", [True, False], ids=["512 tiles", "256 tiles"])
@pytest.mark.parametrize("b_kind", [1, 3, "random"])
def test_forward_of_every_bf16_gate(b_kind, whole):
    need_gpu()
    bits = np.arange(R, dtype=np.uint32).astype(np.uint16)
    bits[(bits & 0x7F80) == 0x7F80] = 0
    a = bf16_bits_to_f32(bits).astype(np.float64)
    silu = swiglu.swiglu_f64(bits, np.full(R, 0x3F80, dtype=np.uint16))
    b = _mantissas(b_kind, 1) * _even_out(silu)
    A, B = _diagonal(a), _diagonal(b)
    q, s = torch.empty((R, C), dtype=torch.uint8, device="cuda"), torch.empty((1, R), device="cuda")
    ck, s_ck = torch.empty((R, 2 * C), dtype=torch.uint8, device="cuda"), torch.empty((2, R), device="cuda")
    for lo, hi in _parts(whole):
        print(f"ckpt forward of every gate, b {b_kind}, rows {lo} to {hi}", flush=True)
        bs.bs_swiglu_quant_1x128_ckpt(A[lo:hi], B[lo:hi], ck[lo:hi], s_ck[:, lo:hi], q_row=q[lo:hi], s_row=s[:, lo:hi])
    _check(s[0].cpu().numpy(), silu * b, np.full(R, 2.0 ** -48))


def _gates():
    """fp32 gates that a checkpoint can hold: every bf16 one of at least 1e-12 / 448, and others where the derivative
    vanishes, where the fp32 path ends (-69) and over the range between."""
    bits = np.arange(0x8000, dtype=np.uint32).astype(np.uint16)
    mag = bf16_bits_to_f32(bits[(bits & 0x7F80) != 0x7F80])
    mag = mag[mag >= np.float32(2.3e-15)]
    root = np.float32(-1.2784645)
    near = root + np.arange(-2048, 2048) * np.spacing(root)
    rng = np.random.default_rng(5)
    some = [mag, -mag, near, rng.uniform(-69.2, -68.8, 1024), -1.2784645 + rng.normal(0, 1e-3, 2048)]
    n = R - sum(len(t) for t in some)
    some.append(rng.uniform(-90, 25, n))
    return np.concatenate(some).astype(np.float32)


@pytest.mark.parametrize("whole", [True, False], ids=["512 tiles", "256 tiles"])
@pytest.mark.parametrize("kind", [1, 3, "random"])
@pytest.mark.parametrize("half", ["da", "db"])
def test_backward_of_gates(half, kind, whole):
    need_gpu()
    a = _gates()
    a64 = a.astype(np.float64)
    b = np.random.default_rng(6).uniform(0.5, 2, R).astype(np.float32) if kind == "random" else np.full(R, 1.5, dtype=np.float32)
    ga, gb = block.swiglu_grad(a64, b.astype(np.float64), 1.0)
    dh = _mantissas(kind, 7) * _even_out(ga if half == "da" else gb)
    ck = np.zeros((R, 2 * C), dtype=np.uint8)
    ck[np.arange(R), DIAGONAL] = np.where(a < 0, 0xB8, 0x38)      # +-1
    ck[np.arange(R), C + DIAGONAL] = 0x38
    CK, S = torch.from_numpy(ck).cuda(), torch.from_numpy(np.stack([np.abs(a), b])).cuda()
    DH = _diagonal(dh)
    q, s = torch.empty((R, 2 * C), dtype=torch.uint8, device="cuda"), torch.empty((2, R), device="cuda")
    for lo, hi in _parts(whole):
        print(f"ckpt backward of gates, {half}, {kind}, rows {lo} to {hi}", flush=True)
        bs.bs_swiglu_bwd_quant_1x128_ckpt(CK[lo:hi], S[:, lo:hi], DH[lo:hi], q_row=q[lo:hi], s_row=s[:, lo:hi])
    # the formula's own rounding in float64, and what its cancellation near the derivative's zero makes of it
    an = a64 * block._sigmoid(-a64)
    slack = 2.0 ** -48 * (1 + np.abs(an) / np.abs(1 + an)) if half == "da" else np.full(R, 2.0 ** -48)
    v = (ga if half == "da" else gb) * dh
    _check(s[0 if half == "da" else 1].cpu().numpy(), v, slack)
