"""MXFP4 quantizer of weights: codes, scale bytes and values bit for bit."""

import numpy as np
import pytest
import torch

import blockwise_scaled_fp8_bs_amd as bs
from gpu_support import bf16_from_bits, bits16, check_canaries, guarded, need_gpu, u8
from oracle import few
from oracle.quant import bf16_bits_to_f32

pytestmark = pytest.mark.gpu


def _check(bits, pad=0, values=True):
    """Quantizes bf16 bit patterns [R, C] with canaries around every output."""
    R, C = bits.shape
    x = torch.full((R, C + pad), 3.0, dtype=torch.bfloat16)
    x[:, :C] = bf16_from_bits(bits)
    x = x.cuda()[:, :C]
    fq, q = guarded(R, C // 2, torch.uint8)
    fs, s = guarded(C // 32, (R + 15) // 16 * 16, torch.uint8)
    fy, y = guarded(R, C, torch.bfloat16) if values else (None, None)
    bs.bs_mx4_quant_1x32(x, q, s, y=y)
    torch.cuda.synchronize()
    codes, byte = few.quant_mx4(bf16_bits_to_f32(bits))
    assert np.array_equal(u8(q), few.pack(codes))
    assert np.array_equal(u8(s)[:, :R], byte.T)
    check_canaries(fq, R, C // 2)
    check_canaries(fs, C // 32, R)
    if values:
        want = few.weights(few.pack(codes), byte, "mxfp4")
        got = y.float().cpu().numpy()
        assert np.array_equal(got, want) and np.array_equal(np.signbit(got), np.signbit(want))
        check_canaries(fy, R, C)


@pytest.mark.parametrize("R,C", [(1, 32), (1, 256), (3, 96), (31, 288), (33, 224), (77, 672), (128, 1024), (300, 544)])
def test_blocks_of_any_count(R, C):
    need_gpu()
    print(f"mx4 {R} x {C}", flush=True)
    rng = np.random.default_rng(R * 1000 + C)
    v = (rng.standard_normal((R, C)) * np.exp2(rng.integers(-12, 12, (R, C)))).astype(np.float32)
    bits = bits16(torch.from_numpy(v).to(torch.bfloat16)).copy()
    bits[0, :32] = 0
    if R > 2:
        bits[1, :32] = rng.integers(0, 0x80, 32)          # subnormals
        bits[2, 5] = 0x7F7F                               # the largest
        bits[2, 7] = 0xFF7F
    _check(bits, pad=8 * (R % 3), values=R % 2 == 1 or C % 64 == 0)


def test_every_value_under_every_scale_near_it():
    """Every finite bf16 magnitude beside block maxima 2^0 .. 2^9 above it (where it is the first, it is the
    maximum itself), with signs: every rounding step and every scale byte that a quantizer makes."""
    need_gpu()
    print("mx4: every bf16 value", flush=True)
    mags = np.arange(0, 0x7F80, dtype=np.uint32)
    blocks = []
    for up in range(10):
        ex = np.minimum((mags >> 7) + up, 0xFE)
        blocks.append(np.where(up == 0, mags, ex << 7 | 0x7F).astype(np.uint16))
    out = np.zeros((len(mags), 10, 32), np.uint16)
    for i, top in enumerate(blocks):
        out[:, i, :30] = mags[:, None]
        out[:, i, 1:30:2] |= 0x8000
        out[:, i, 30] = top
        out[:, i, 31] = np.maximum(mags, 1) - 1
    _check(out.reshape(-1, 320))


def test_values_may_replace_the_weights():
    need_gpu()
    x = torch.randn(70, 640, device="cuda").to(torch.bfloat16)
    y, q, s = torch.empty_like(x), torch.empty((70, 320), dtype=torch.uint8, device="cuda"), bs.empty_mx_scales(20, 70, "cuda")
    bs.bs_mx4_quant_1x32(x, q, s, y=y)
    q2, s2, keep = torch.empty_like(q), torch.zeros_like(s), x.clone()
    bs.bs_mx4_quant_1x32(keep, q2, s2, y=keep)
    assert torch.equal(q, q2) and torch.equal(s[:, :70], s2[:, :70]) and torch.equal(keep, y)


def test_rows_past_32_bit_offsets():
    """2^31 elements and more: the last rows' codes."""
    need_gpu()
    print("mx4: a matrix past 2^31 elements", flush=True)
    R, C = 8200, 1 << 18
    x = torch.zeros((R, C), dtype=torch.bfloat16, device="cuda")
    tail = torch.randn((9, C), device="cuda").to(torch.bfloat16)
    x[-9:] = tail
    q = torch.empty((R, C // 2), dtype=torch.uint8, device="cuda")
    s = bs.empty_mx_scales(C // 32, R, "cuda")
    bs.bs_mx4_quant_1x32(x, q, s)
    q9, s9 = torch.empty((9, C // 2), dtype=torch.uint8, device="cuda"), bs.empty_mx_scales(C // 32, 9, "cuda")
    bs.bs_mx4_quant_1x32(tail, q9, s9)
    assert torch.equal(q[-9:], q9) and torch.equal(s[:, R - 9:R], s9[:, :9])
    assert int(q[:-9].max()) == 0 and int(s[:, :R - 9].max()) == 0
