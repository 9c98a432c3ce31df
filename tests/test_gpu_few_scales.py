"""Scales of the few-token calls: what lies around those of the weights is not taken for them."""

import numpy as np
import pytest
import torch

import blockwise_scaled_fp8_bs_amd as bs
from few_support import KINDS, bf16, device_experts, device_weight, f64, finite_codes, random_scales
from gpu_support import need_gpu
from oracle import few

pytestmark = pytest.mark.gpu

NAN = {"e4m3": float("nan"), "mxfp8": 255, "mxfp4": 255}
ENDS = [("e4m3", 128), ("e4m3", 384), ("mxfp8", 32), ("mxfp8", 224), ("mxfp8", 672), ("mxfp4", 32), ("mxfp4", 160), ("mxfp4", 736)]


@pytest.mark.parametrize("kind,K", ENDS)
def test_rows_behind_the_last_of_a_product(kind, K):
    """Contractions whose last unit is a part of one, NaN in the rows of scales that follow."""
    need_gpu()
    rng = np.random.default_rng([K, 9])
    N = 256
    q, s = finite_codes(rng, kind, N, K), random_scales(rng, kind, N, K)
    w, sw = device_weight(q, s, kind)
    full = torch.full((sw.shape[0] + 16, sw.shape[1]), NAN[kind], dtype=sw.dtype, device="cuda")
    full[:sw.shape[0]] = sw
    for T in (1, 5, 16, 40):
        print(f"few_mm {kind} K {K} with NaN behind the scales, T {T}", flush=True)
        x = bf16(rng, (T, K))
        out = bs.bs_few_mm(x, w, full[:sw.shape[0]], KINDS[kind], out_dtype=torch.float32)
        ref, bound = few.few_mm(f64(x), few.weights(q, s, kind), bf16=False)
        assert (np.abs(f64(out) - ref) <= bound).all()


@pytest.mark.parametrize("kind,K", ENDS)
def test_rows_behind_the_last_of_experts(kind, K):
    """The same between experts, in both of their contractions."""
    need_gpu()
    rng = np.random.default_rng([K, 10])
    E = 3
    args, values = [], []
    for N in (2 * K, K):
        qs = [finite_codes(rng, kind, N, K) for _ in range(E)]
        ss = [random_scales(rng, kind, N, K) for _ in range(E)]
        q, s = device_experts(qs, ss, kind)
        full = torch.full((E, s.shape[1] + 16, s.shape[2]), NAN[kind], dtype=s.dtype, device="cuda")
        full[:, :s.shape[1]] = s
        args += [q, full[:, :s.shape[1]]]
        values.append([few.weights(a, b, kind) for a, b in zip(qs, ss)])
    for T in (1, 6, 33):
        print(f"moe_few {kind} widths {K} with NaN behind the scales, T {T}", flush=True)
        x = bf16(rng, (T, K))
        idx = np.stack([rng.permutation(E)[:2] for _ in range(T)]).astype(np.int32)
        w = rng.uniform(0.1, 1, (T, 2)).astype(np.float32)
        out = bs.bs_moe_few(x, torch.from_numpy(idx).cuda(), torch.from_numpy(w).cuda(), *args, KINDS[kind])
        ref, bound = few.moe(f64(x), idx, w.astype(np.float64), *values)
        assert (np.abs(f64(out) - ref) <= bound).all()


@pytest.mark.parametrize("kind", ["mxfp8", "mxfp4"])
def test_every_scale_byte_with_every_code(kind):
    """All codes under all scales, alone in their rows: exact where the weight is a normal number of bf16's range; below
    that it is rounded to bf16's subnormal ones, multiples of 2^-133, and off by 2^-134 at most, half a step; above, it
    is infinite (and would make NaN of a zero of x)."""
    need_gpu()
    codes = 256 if kind == "mxfp8" else 16
    for byte in range(255):
        print(f"few_mm {kind}: every code under scale byte {byte}", flush=True)
        at = byte % 32
        q = np.zeros((codes, 32), np.uint8)
        q[:, at] = np.arange(codes)
        if kind == "mxfp8":
            q[[0x7F, 0xFF]] = 0                               # NaN
        else:
            q = few.pack(q)
        s = np.full((codes, 1), byte, np.uint8)
        weight = few.weights(q, s, kind)[:, at]
        up = 2.0 ** min(max(127 - byte, -100), 100)           # the products are around 1, or normal at least
        x = torch.zeros((1, 32), dtype=torch.bfloat16, device="cuda")
        x[0, at] = up
        w, sw = device_weight(q, s, kind)
        out, want = f64(bs.bs_few_mm(x, w, sw, KINDS[kind], out_dtype=torch.float32))[0], weight * up
        small, infinite = np.abs(weight) < 2.0 ** -126, np.abs(weight) >= 2.0 ** 128
        normal = ~small & ~infinite
        assert np.array_equal(out[normal], want[normal])
        assert (np.abs(out[small] - want[small]) <= 2.0 ** -134 * up).all()
        assert np.isinf(out[infinite]).all() and (np.sign(out[infinite]) == np.sign(weight[infinite])).all()
