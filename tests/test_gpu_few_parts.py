"""The activations between the experts' kernels in one and two bf16 parts, by the workspace that the call has."""

import numpy as np
import pytest
import torch

import blockwise_scaled_fp8_bs_amd as bs
from blockwise_scaled_fp8_bs_amd import _lib
from few_support import KINDS, bf16, device_experts, f64, finite_codes, random_scales
from gpu_support import need_gpu
from oracle import few

pytestmark = pytest.mark.gpu


def _experts(rng, kind, E, D, H):
    args, values = [], []
    for N, K in ((2 * H, D), (D, H)):
        qs = [finite_codes(rng, kind, N, K) for _ in range(E)]
        ss = [random_scales(rng, kind, N, K) for _ in range(E)]
        args += device_experts(qs, ss, kind)
        values.append([few.weights(q, s, kind) for q, s in zip(qs, ss)])
    return args, values


def _call(kind, x, idx, w, args, nbytes, guard=256):
    """The C entry with a workspace of nbytes and a guard behind it."""
    T, D = x.shape
    q12, s12, qo, so = args
    E, H = q12.shape[0], q12.shape[1] // 2
    k = 1 if idx is None else idx.shape[1]
    out = torch.empty_like(x)
    ws = torch.full((nbytes + guard,), 0xA5, dtype=torch.uint8, device="cuda")
    p = lambda t: None if t is None else t.data_ptr()  # noqa: E731
    status = _lib.load().bs_moe_few(KINDS[kind], T, D, H, E, k, p(x), x.stride(0), p(idx), p(w), p(q12), q12.stride(0), q12.stride(1),
                                    p(s12), s12.stride(0), s12.stride(1), p(qo), qo.stride(0), qo.stride(1), p(so), so.stride(0),
                                    so.stride(1), None, 0, p(out), out.stride(0), p(ws), nbytes, torch.cuda.current_stream().cuda_stream)
    assert status == 0, _lib.load().bs_last_error().decode()
    torch.cuda.synchronize()
    assert (ws[nbytes:] == 0xA5).all()
    return out


# the waves of a workgroup share tiles or stream them, with and without shares of the output
SIZES = [(1, 256, 512, 1, 1), (1, 640, 384, 8, 8), (1, 128, 4096, 8, 8), (2, 384, 4096, 16, 8), (3, 256, 128, 4, 2), (4, 128, 4096, 8, 8),
         (5, 512, 1024, 1, 1), (7, 128, 384, 4, 3), (8, 128, 2048, 16, 8), (8, 2176, 128, 2, 2)]


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("T,D,H,E,k", SIZES)
def test_two_parts_leave_the_rounding_of_the_result(kind, T, D, H, E, k):
    need_gpu()
    print(f"moe_few {kind} T {T} D {D} H {H} E {E} k {k}: parts of h", flush=True)
    if kind != "e4m3":
        D, H = D + 32, H + 32 * (T % 4)
    rng = np.random.default_rng([T, D, H, E, k, 11])
    args, values = _experts(rng, kind, E, D, H)
    x = bf16(rng, (T, D))
    idx = np.stack([rng.permutation(E)[:k] for _ in range(T)]).astype(np.int32)
    w = rng.uniform(0.05, 1, (T, k)).astype(np.float32)
    d_idx, d_w = torch.from_numpy(idx).cuda(), torch.from_numpy(w).cuda()
    lib = _lib.load()
    least, full = lib.bs_moe_few_workspace_bytes(T, D, H, E, k), lib.bs_moe_few_full_workspace_bytes(T, D, H, E, k)
    assert full == least + T * k * H * 2
    ref, bound = few.moe(f64(x), idx, w.astype(np.float64), *values, parts=2)
    fine = _call(kind, x, d_idx, d_w, args, full)
    assert (np.abs(f64(fine) - ref) <= bound).all()
    # the binding's calls, and any more room
    assert torch.equal(bs.bs_moe_few(x, d_idx, d_w, *args, KINDS[kind]), fine)
    assert torch.equal(_call(kind, x, d_idx, d_w, args, full + 4096), fine)
    # less: one part, h's rounding beside the result's
    _, loose = few.moe(f64(x), idx, w.astype(np.float64), *values)
    for nbytes in (least, full - 2):
        coarse = _call(kind, x, d_idx, d_w, args, nbytes)
        assert (np.abs(f64(coarse) - ref) <= loose).all()
    # against float64: the result's rounding alone is off by 2^-9 / sqrt(3) to 2^-8 / sqrt(3) of the norm, by mantissas
    norm = np.sqrt(np.mean(ref ** 2))
    assert np.sqrt(np.mean((f64(fine) - ref) ** 2)) <= 2.0 ** -8 / 3 ** 0.5 * norm
    rounded = torch.from_numpy(ref).to(torch.bfloat16)
    assert np.sqrt(np.mean((f64(fine) - f64(rounded)) ** 2)) <= 0.25 * np.sqrt(np.mean((f64(rounded) - ref) ** 2))


def test_more_tokens_keep_one():
    need_gpu()
    lib = _lib.load()
    for T in (9, 64, 100):
        assert lib.bs_moe_few_full_workspace_bytes(T, 256, 128, 4, 2) == lib.bs_moe_few_workspace_bytes(T, 256, 128, 4, 2)


def test_infinite_activations_have_no_second_part():
    """Infinite and NaN activations, and those that round to infinity, give what one part gives."""
    need_gpu()
    print("moe_few: infinite activations in two parts", flush=True)
    D = H = 32
    v = np.zeros((2 * H, D))
    v[:H, 0], v[H:, 1] = 1.0, 1.0
    one = lambda n: np.full((n, 1), 127, np.uint8)  # noqa: E731
    from few_support import codes_of
    args = (*device_experts([codes_of(v, "mxfp8")], [one(2 * H)], "mxfp8"), *device_experts([codes_of(np.eye(D), "mxfp8")], [one(D)], "mxfp8"))
    gates, ups = [float("inf"), float("nan"), 2.0 ** 100, 300.0, 2.0 ** 64, -50.0, 3.0], [1.0, 1.0, 2.0 ** 100, float("-inf"), 2.0 ** 63.99, 1.0, 5.0]
    x = torch.zeros((len(gates), D))
    x[:, 0], x[:, 1] = torch.tensor(gates), torch.tensor(ups)
    x = x.to(torch.bfloat16).cuda()
    T = len(gates)
    lib = _lib.load()
    two = _call("mxfp8", x, None, None, args, lib.bs_moe_few_full_workspace_bytes(T, D, H, 1, 1))
    part = _call("mxfp8", x, None, None, args, lib.bs_moe_few_workspace_bytes(T, D, H, 1, 1))
    big = ~torch.isfinite(part)
    assert big[:4].any() and torch.equal(torch.isnan(two), torch.isnan(part))
    assert torch.equal(torch.nan_to_num(two[big], nan=7.0), torch.nan_to_num(part[big], nan=7.0))
