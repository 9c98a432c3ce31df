"""The product of few rows with quantized weights, against float64."""

import numpy as np
import pytest
import torch

import blockwise_scaled_fp8_bs_amd as bs
from few_support import (KINDS, bf16, codes_of, device_weight, f64, finite_codes, guarded_rows, random_scales, untouched)
from gpu_support import need_gpu
from oracle import few

pytestmark = pytest.mark.gpu

TOKENS = (1, 2, 7, 16, 17, 31, 33, 64, 65, 150)
SHAPES = {"e4m3": ((128, 128), (384, 640), (1152, 2176)),
          "mxfp8": ((1, 32), (50, 96), (200, 160), (1001, 1312)),
          "mxfp4": ((3, 32), (16, 64), (129, 736), (515, 2080))}
CASES = [(kind, T, *SHAPES[kind][(i + j) % len(SHAPES[kind])]) for j, kind in enumerate(KINDS) for i, T in enumerate(TOKENS)]
CASES += [(kind, 1, *shape) for kind in KINDS for shape in SHAPES[kind]]


@pytest.mark.parametrize("kind,T,N,K", CASES)
def test_within_the_sum_s_bound(kind, T, N, K):
    need_gpu()
    print(f"few_mm {kind} T {T} N {N} K {K}", flush=True)
    rng = np.random.default_rng([T, N, K])
    q, s = finite_codes(rng, kind, N, K), random_scales(rng, kind, N, K)
    pad = T % 2
    w, sw = device_weight(q, s, kind, pad)
    x = bf16(rng, (T, K + 8 * pad))[:, :K]
    res = bf16(rng, (T, N + pad))[:, :N] if T % 3 else None
    ref, wv = None, few.weights(q, s, kind)
    for dtype in (torch.bfloat16, torch.float32):
        full, out = guarded_rows(T, N, dtype, extra=4 if T % 4 == 0 else 3)
        got = bs.bs_few_mm(x, w, sw, KINDS[kind], residual=res, out=out)
        assert got is out and untouched(full, T, N)
        ref, bound = few.few_mm(f64(x), wv, None if res is None else f64(res), bf16=dtype == torch.bfloat16)
        assert (np.abs(f64(out) - ref) <= bound).all()
        # the same again, and into an output of the call's own
        assert torch.equal(bs.bs_few_mm(x, w, sw, KINDS[kind], residual=res, out_dtype=dtype), out)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("T,N,K", [(1, 384, 1408), (5, 256, 4224), (16, 128, 256), (40, 640, 896), (64, 256, 1152), (70, 256, 384)])
def test_whole_numbers_are_exact(kind, T, N, K):
    """Small integers under power-of-two scales that differ from block to block: any value read from another
    place, added twice or left out shows."""
    need_gpu()
    print(f"few_mm integers {kind} T {T} N {N} K {K}", flush=True)
    rng = np.random.default_rng([T, N, K, 1])
    v = rng.choice([0, 1, 2, 3, 4, 6], (N, K)) * rng.choice([-1, 1], (N, K))
    q = codes_of(v, kind)
    if kind == "e4m3":
        s = np.exp2(rng.integers(-2, 3, (N // 128, K // 128))).astype(np.float32)
    else:
        s = rng.integers(125, 130, (N, K // 32)).astype(np.uint8)
    x = torch.from_numpy(rng.integers(-8, 9, (T, K)).astype(np.float32)).to(torch.bfloat16).cuda()
    # |sum| <= 8 * 24 * K < 2^20, in quarters: exact in fp32
    w, sw = device_weight(q, s, kind)
    out = bs.bs_few_mm(x, w, sw, KINDS[kind], out_dtype=torch.float32)
    assert np.array_equal(f64(out), f64(x) @ few.weights(q, s, kind).T)


@pytest.mark.parametrize("kind", KINDS)
def test_rows_of_x_do_not_touch_each_other(kind):
    """A row of NaN and one of infinities change their own rows of the output alone."""
    need_gpu()
    rng = np.random.default_rng(5)
    N, K = 256, 640
    q, s = finite_codes(rng, kind, N, K), random_scales(rng, kind, N, K)
    w, sw = device_weight(q, s, kind)
    for T in (3, 16, 20, 64):
        print(f"few_mm {kind} with NaN among {T} rows", flush=True)
        x = bf16(rng, (T, K))
        clean = bs.bs_few_mm(x, w, sw, KINDS[kind])
        x[1] = float("nan")
        x[2, 5] = float("inf")
        out = bs.bs_few_mm(x, w, sw, KINDS[kind])
        assert out[1].isnan().all() and not out[2].isfinite().all()
        rest = [t for t in range(T) if t not in (1, 2)]
        assert torch.equal(out[rest], clean[rest])


def test_nan_codes_scales_and_small_weights():
    need_gpu()
    rng = np.random.default_rng(6)
    x = bf16(rng, (4, 256))
    for kind in KINDS:
        print(f"few_mm {kind} with NaN weights", flush=True)
        q, s = finite_codes(rng, kind, 256, 256), random_scales(rng, kind, 256, 256)
        rows = [9]
        if kind == "mxfp4":
            s[9, 3] = 255                 # E8M0's NaN
        elif kind == "mxfp8":
            q[9, 77] = 0x7F
        else:
            s[1, 0] = np.nan              # a block of 128 rows
            rows = list(range(128, 256))
        w, sw = device_weight(q, s, kind)
        out = bs.bs_few_mm(x, w, sw, KINDS[kind]).isnan().all(0).cpu()
        assert out[rows].all() and not out[[n for n in range(256) if n not in rows]].any()
    # products in fp32's normal range from weights near the bottom of bf16's
    for kind, low in (("mxfp4", 3), ("mxfp8", 12)):
        v = rng.choice([1, 2, 3, 4], (64, 64))
        s = np.full((64, 2), low, np.uint8)
        w, sw = device_weight(codes_of(v, kind), s, kind)
        x = torch.full((2, 64), 2.0 ** 100, device="cuda").to(torch.bfloat16)
        out = bs.bs_few_mm(x, w, sw, KINDS[kind], out_dtype=torch.float32)
        assert np.array_equal(f64(out)[0], v.sum(1) * 2.0 ** (100 + low - 127))


def test_residual_in_place_and_no_rows():
    need_gpu()
    rng = np.random.default_rng(7)
    q, s = finite_codes(rng, "mxfp4", 70, 96), random_scales(rng, "mxfp4", 70, 96)
    w, sw = device_weight(q, s, "mxfp4")
    x, res = bf16(rng, (5, 96)), bf16(rng, (5, 70))
    want = bs.bs_few_mm(x, w, sw, KINDS["mxfp4"], residual=res)
    got = bs.bs_few_mm(x, w, sw, KINDS["mxfp4"], residual=res, out=res)
    assert got is res and torch.equal(got, want)
    assert bs.bs_few_mm(x[:0], w, sw, KINDS["mxfp4"]).shape == (0, 70)


def test_more_rows_than_one_launch_holds_at_a_time():
    need_gpu()
    print("few_mm with 5000 rows", flush=True)
    rng = np.random.default_rng(8)
    q, s = finite_codes(rng, "mxfp8", 48, 160), random_scales(rng, "mxfp8", 48, 160)
    w, sw = device_weight(q, s, "mxfp8")
    x = bf16(rng, (5000, 160))
    out = bs.bs_few_mm(x, w, sw, KINDS["mxfp8"])
    ref, bound = few.few_mm(f64(x), few.weights(q, s, "mxfp8"))
    assert (np.abs(f64(out) - ref) <= bound).all()


def test_weights_past_32_bit_offsets():
    need_gpu()
    print("few_mm: weights past 2^31 bytes", flush=True)
    N, K = 17000, 1 << 17
    q = torch.zeros((N, K), dtype=torch.uint8, device="cuda")
    q[-20:] = 0x38                                           # 1.0
    s = torch.full((K // 32, 17008), 127, dtype=torch.uint8, device="cuda")
    x = torch.ones((2, K), device="cuda").to(torch.bfloat16)
    out = bs.bs_few_mm(x, q, s, bs.BS_WEIGHT_MXFP8, out_dtype=torch.float32)
    assert (out[:, -20:] == K).all() and (out[:, :-20] == 0).all()
