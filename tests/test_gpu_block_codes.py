"""Codes and scales of values that are not bf16 (norms and weighted rows are
quantized from fp32): fl32(amax / 448), fl32(v / s) and its e4m3 rounding, as
for bf16 values, bit for bit."""

import numpy as np
import pytest
import torch

import blockwise_scaled_fp8_bs_amd as bs
from gpu_support import need_gpu, u8
from oracle import e4m3

pytestmark = pytest.mark.gpu

EPS = np.float32(1e-12)


def _codes(v):
    """(codes, scales) of fp32 blocks [n, 128]."""
    s = (np.maximum(np.abs(v).max(axis=1), EPS) / np.float32(448)).astype(np.float32)
    y = np.clip((v / s[:, None]).astype(np.float32), np.float32(-448), np.float32(448))
    mag, table = np.abs(y).astype(np.float64), np.array([e4m3.decode_code(c) for c in range(0x7F)])
    at = np.clip(np.searchsorted(table, mag), 1, 0x7E)
    low, high = mag - table[at - 1], table[at] - mag
    code = np.where((high < low) | ((high == low) & (at % 2 == 0)), at, at - 1).astype(np.uint8)
    return code | (np.signbit(y).astype(np.uint8) << 7), s


def _through_the_norm(v):
    """The codes that the norm makes of v [n, 128] fp32: rows of ones have a norm of 1 with eps = 0, and h is w_pre."""
    n = v.shape[0]
    q, s = np.empty((n, 128), dtype=np.uint8), np.empty(n, dtype=np.float32)
    one = torch.ones((1, 16384), dtype=torch.bfloat16, device="cuda")
    gq, gs = torch.empty((1, 16384), dtype=torch.uint8, device="cuda"), bs.empty_scales(128, 1, "cuda")
    for lo in range(0, n, 128):
        m = min(128, n - lo)
        w = torch.from_numpy(v[lo:lo + m].reshape(-1).copy()).cuda()
        bs.bs_resid_norm(one[:, :128 * m], w, eps=0.0, q_row=gq[:, :128 * m], s_row=gs[:m])
        q[lo:lo + m], s[lo:lo + m] = u8(gq)[0, :128 * m].reshape(m, 128), gs[:m, 0].cpu().numpy()
    return q, s


def _next_to_a_tie():
    """(v, s) with v / s as near as 24-bit significands come to the middle between an e4m3 tie and the fp32 value next
    to it, the one place where a quotient that is not rounded right could change a code: v 2^j = s m +- 1, m a tie's
    significand with 25 bits and one more."""
    out = []
    for tie in (17, 19, 21, 23, 25, 27, 29, 31, 9, 11, 13, 15, 5, 7, 3, 1):
        tie <<= 25 - tie.bit_length()
        for m in (tie + 1, tie - 1):
            for sign in (1, -1):
                for j in (24, 25):
                    inverse = pow(m, -1, 1 << j)
                    s = (-sign * inverse) % (1 << j)   # s m + sign = 0 mod 2^j
                    while s < 1 << 24:
                        v = (s * m + sign) >> j
                        if s >= 1 << 23 and 1 << 23 <= v < 1 << 24:
                            out.append((v, s))
                        s += 1 << j
    return out


def test_codes_of_fp32_blocks():
    need_gpu()
    rng = np.random.default_rng(3)
    v = rng.standard_normal((4096, 128)) * np.exp2(rng.integers(-60, 60, (4096, 1)))
    v[:64] *= 1e-16          # below the floor of the largest value
    v[64:128] = np.exp2(rng.integers(-126, 127, (64, 128)).astype(float))
    v[128, :] = 0
    v[129, ::2] = -0.0
    v[130, 0] = 3.4028234e38
    v = v.astype(np.float32)
    print("codes of fp32 blocks", flush=True)
    q, s = _through_the_norm(v)
    want_q, want_s = _codes(v)
    assert np.array_equal(s.view(np.uint32), want_s.view(np.uint32))
    assert np.array_equal(q, want_q)


def test_codes_next_to_a_tie():
    """Quotients as hard as they come, with the scale of the pair reached from a largest value."""
    need_gpu()
    blocks = []
    for v, s in _next_to_a_tie():
        # a largest value whose 448th rounds to s
        top = np.float32(s) * np.float32(448)
        for a in (np.nextafter(top, np.float32(0)), top, np.nextafter(top, np.float32(np.inf))):
            if np.float32(a / np.float32(448)) == np.float32(s):
                b = np.zeros(128, dtype=np.float32)
                b[0] = a
                # v over every power of two that keeps it under the largest value
                for i in range(1, 21):
                    x = np.ldexp(np.float32(v), 9 - i)
                    b[i], b[i + 20] = (x, -x) if x <= a else (0, 0)
                blocks.append(b)
                break
    v = np.stack(blocks)
    assert v.shape[0] >= 16
    print(f"codes next to a tie: {v.shape[0]} blocks", flush=True)
    q, s = _through_the_norm(v)
    want_q, want_s = _codes(v)
    assert np.array_equal(s.view(np.uint32), want_s.view(np.uint32))
    assert np.array_equal(q, want_q)


def test_weighted_rows_are_quantized_from_their_fp32_products():
    need_gpu()
    T, D = 512, 256
    g = torch.Generator().manual_seed(4)
    x, w = torch.randn((T, D), generator=g).to(torch.bfloat16), torch.rand((T, 1), generator=g) * 2 - 1
    row_slot = torch.randperm(T, generator=g).to(torch.int32)
    q, s = torch.empty((T, D), dtype=torch.uint8, device="cuda"), bs.empty_scales(D // 128, T, "cuda")
    c, t = torch.empty((D, T), dtype=torch.uint8, device="cuda"), bs.empty_scales(T // 128, D, "cuda")
    print("codes of weighted rows", flush=True)
    bs.bs_moe_gather_quant_1x128(x.cuda(), row_slot.cuda(), 1, w=w.cuda(), q_row=q, s_row=s, q_col=c, s_col=t)
    v = (x.float() * w)[row_slot.long()].numpy()
    for got_q, got_s, m in ((q, s, v), (c, t, v.T.copy())):
        n = m.shape[0]
        want_q, want_s = _codes(m.reshape(-1, 128))
        assert np.array_equal(u8(got_q), want_q.reshape(n, -1))
        assert np.array_equal(got_s.cpu().numpy()[:, :n].T, want_s.reshape(n, -1))
