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
