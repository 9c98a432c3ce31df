"""Weights of the three formats for the few-token tests (test code only)."""

import numpy as np
import torch

import blockwise_scaled_fp8_bs_amd as bs
from oracle import e4m3, few

KINDS = {"e4m3": bs.BS_WEIGHT_E4M3_128X128, "mxfp8": bs.BS_WEIGHT_MXFP8, "mxfp4": bs.BS_WEIGHT_MXFP4}


def finite_codes(rng, kind, N, K):
    """Random codes without e4m3's NaNs; packed for mxfp4."""
    if kind == "mxfp4":
        return rng.integers(0, 256, (N, K // 2)).astype(np.uint8)
    q = rng.integers(0, 256, (N, K)).astype(np.uint8)
    return np.where((q & 127) == 127, q ^ 1, q)


def codes_of(values, kind):
    """Codes of small numbers that the format holds."""
    values = np.asarray(values, np.float64)
    if kind != "mxfp4":
        return e4m3.encode(values.astype(np.float32))
    return few.pack(few._encode(values))


def random_scales(rng, kind, N, K):
    """Logical scales that keep weights around 2^-6, differing from block to block."""
    if kind == "e4m3":
        return (np.exp2(rng.uniform(-14, -11, (N // 128, K // 128)))).astype(np.float32)
    base = 127 - 14 if kind == "mxfp8" else 127 - 7
    return rng.integers(base - 2, base + 3, (N, K // 32)).astype(np.uint8)


def device_weight(q, s, kind, pad=0, device="cuda"):
    """Codes with a padded row stride and K-major scales with `pad` more columns, garbage in the padding."""
    q = torch.from_numpy(np.ascontiguousarray(q))
    full = torch.full((q.shape[0], q.shape[1] + 16 * pad), 0x7E, dtype=torch.uint8)
    full[:, :q.shape[1]] = q
    st = torch.from_numpy(np.ascontiguousarray(s.T))
    width = (st.shape[1] + 3) // 4 * 4 if kind == "e4m3" else (st.shape[1] + 15) // 16 * 16
    sc = torch.full((st.shape[0], width + 16 * pad), float("nan")) if kind == "e4m3" else \
        torch.full((st.shape[0], width + 16 * pad), 255, dtype=torch.uint8)
    sc[:, :st.shape[1]] = st
    return full.to(device)[:, :q.shape[1]], sc.to(device)


def device_experts(qs, ss, kind, pad=0):
    """The same for a list of experts: [E, N, ...] and [E, K blocks, ...]."""
    both = [device_weight(q, s, kind, pad) for q, s in zip(qs, ss)]
    wide = torch.stack([torch.nn.functional.pad(q, (0, 16 * pad), value=0x7E) for q, _ in both])
    return wide[:, :, :both[0][0].shape[1]], torch.stack([s for _, s in both])


def bf16(rng, shape, sigma=1.0, device="cuda"):
    t = torch.from_numpy(rng.standard_normal(shape).astype(np.float32) * np.float32(sigma)).to(torch.bfloat16)
    return t.to(device)


def f64(t):
    return t.detach().cpu().double().numpy()


def guarded_rows(T, N, dtype, extra=3):
    """An output view inside a tensor of sevens, with an odd row stride."""
    full = torch.full((T + 1, N + extra), 7.0, dtype=dtype, device="cuda")
    return full, full[:T, :N]


def untouched(full, T, N):
    keep = full.clone()
    keep[:T, :N] = 7.0
    return bool((keep == 7.0).all())
