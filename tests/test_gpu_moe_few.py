"""The gated experts of few routed tokens, against float64."""

import numpy as np
import pytest
import torch

import blockwise_scaled_fp8_bs_amd as bs
from few_support import KINDS, bf16, codes_of, device_experts, f64, finite_codes, random_scales
from gpu_support import need_gpu
from oracle import few

pytestmark = pytest.mark.gpu


def _experts(rng, kind, E, D, H, pad=0):
    """(device codes and scales of w12, of out_proj; their float64 values)."""
    out = []
    for N, K in ((2 * H, D), (D, H)):
        qs = [finite_codes(rng, kind, N, K) for _ in range(E)]
        ss = [random_scales(rng, kind, N, K) for _ in range(E)]
        out.append((*device_experts(qs, ss, kind, pad), [few.weights(q, s, kind) for q, s in zip(qs, ss)]))
    (q12, s12, v12), (qo, so, vo) = out
    return (q12, s12, qo, so), v12, vo


def _choices(rng, T, E, k):
    idx = np.stack([rng.permutation(E)[:k] for _ in range(T)]).astype(np.int32)
    idx[rng.random((T, k)) < 0.15] = -1
    if T > 2:
        idx[1] = -1
    w = rng.uniform(0.05, 1, (T, k)).astype(np.float32)
    w[idx < 0] = np.nan      # never used
    return idx, w


def _run(kind, x, idx, w, weights, residual=None, **kw):
    put = lambda v: None if v is None else torch.from_numpy(v).cuda()  # noqa: E731
    q12, s12, qo, so = weights
    return bs.bs_moe_few(x, put(idx), put(w), q12, s12, qo, so, KINDS[kind], residual=residual, **kw)


CASES = [(1, 128, 128, 4, 2), (1, 640, 384, 8, 8), (3, 256, 128, 1, 1), (6, 128, 512, 5, 3), (16, 256, 256, 16, 4),
         (17, 384, 128, 8, 2), (32, 128, 256, 2, 1), (40, 256, 128, 3, 2), (64, 128, 128, 64, 8), (67, 128, 128, 6, 2),
         (130, 128, 256, 4, 1),
         # few columns and long contractions: workgroups share them
         (1, 128, 2048, 8, 8), (10, 128, 1024, 16, 6), (24, 384, 1152, 12, 4), (40, 128, 1536, 4, 2), (66, 128, 1024, 2, 2)]


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("T,D,H,E,k", CASES)
def test_within_the_bound(kind, T, D, H, E, k):
    need_gpu()
    if kind != "e4m3" and T % 2:        # widths that are not multiples of a unit
        D, H = D + 32, H + 96
    print(f"moe_few {kind} T {T} D {D} H {H} E {E} k {k}", flush=True)
    rng = np.random.default_rng([T, D, H, E, k])
    weights, v12, vo = _experts(rng, kind, E, D, H, pad=T % 2)
    idx, w = _choices(rng, T, E, k)
    x = bf16(rng, (T, D + 8 * (T % 2)))[:, :D]
    res = bf16(rng, (T, D)) if T % 3 else None
    out = _run(kind, x, idx, w, weights, res)
    ref, bound = few.moe(f64(x), idx, w.astype(np.float64), v12, vo, None if res is None else f64(res))
    assert (np.abs(f64(out) - ref) <= bound).all()
    # a typical error is far below the bound: the roundings to bf16 of h and of the result, both at random
    assert np.sqrt(np.mean((f64(out) - ref) ** 2)) <= 2.0 ** -8 * np.sqrt(np.mean(ref ** 2))
    assert torch.equal(_run(kind, x, idx, w, weights, res), out)


@pytest.mark.parametrize("kind,T,H,E,k", [("e4m3", 40, 128, 3, 2), ("mxfp8", 64, 96, 12, 2), ("mxfp4", 40, 64, 3, 2),
                                          ("mxfp4", 64, 160, 12, 2), ("mxfp4", 64, 32, 200, 32), ("mxfp8", 33, 64, 1, 1)])
def test_wide_outputs_beside_many_tokens(kind, T, H, E, k):
    """4096 columns and more: the waves take two tiles of them at a time."""
    need_gpu()
    D = 4096 + (0 if kind == "e4m3" else 32)
    print(f"moe_few {kind} T {T} D {D} H {H} E {E} k {k}", flush=True)
    rng = np.random.default_rng([T, D, H, E, k])
    weights, v12, vo = _experts(rng, kind, E, D, H)
    idx, w = _choices(rng, T, E, k)
    x, res = bf16(rng, (T, D)), bf16(rng, (T, D))
    out = _run(kind, x, idx, w, weights, res)
    ref, bound = few.moe(f64(x), idx, w.astype(np.float64), v12, vo, f64(res))
    assert (np.abs(f64(out) - ref) <= bound).all()
    assert torch.equal(_run(kind, x, idx, w, weights, res), out)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("T,E,k", [(1, 6, 3), (9, 40, 4), (33, 7, 3), (64, 3, 2), (70, 5, 2)])
def test_whole_numbers_are_exact(kind, T, E, k):
    """Gates of 128 and more, where silu(a) = a in fp32, and small integers for everything else: any token,
    slot, expert, row or column taken for another shows."""
    need_gpu()
    print(f"moe_few integers {kind} T {T} E {E} k {k}", flush=True)
    rng = np.random.default_rng([T, E, k, 2])
    D, H = 256, 384
    one = (lambda N, K: np.ones((N // 128, K // 128), np.float32)) if kind == "e4m3" else (lambda N, K: np.full((N, K // 32), 127, np.uint8))
    x = rng.integers(0, 2, (T, D)).astype(np.float32)
    x[:, 0] = 64.0
    v12, vo = [], []
    for _ in range(E):
        v = np.zeros((2 * H, D))
        v[:H, 0] = rng.choice([2, 4], H)                      # a = 128 or 256
        v[H:, 1:] = rng.choice([0, 0, 0, 1], (H, D - 1)) * rng.choice([-1, 1], (H, D - 1))
        v12.append(v)
        vo.append(rng.choice([0, 0, 1, -1, 2], (D, H)).astype(np.float64))
    weights = (*device_experts([codes_of(v, kind) for v in v12], [one(2 * H, D)] * E, kind),
               *device_experts([codes_of(v, kind) for v in vo], [one(D, H)] * E, kind))
    idx = np.stack([rng.permutation(E)[:k] for _ in range(T)]).astype(np.int32)
    idx[rng.random((T, k)) < 0.2] = E                        # not routed
    w = np.exp2(rng.integers(-2, 2, (T, k))).astype(np.float32)
    res = torch.from_numpy(rng.integers(-100, 100, (T, D)).astype(np.float32)).to(torch.bfloat16).cuda()
    out = _run(kind, torch.from_numpy(x).to(torch.bfloat16).cuda(), idx, w, weights, res)
    want = f64(res).copy()
    for t in range(T):
        for j in range(k):
            if idx[t, j] < E:
                ab = v12[idx[t, j]] @ x[t]
                h = w[t, j] * ab[:H] * ab[H:]
                assert np.abs(ab[H:]).max() < 256            # h in 8 bits, sums below 2^24 quarters
                want[t] += vo[idx[t, j]] @ h
    assert torch.equal(out.cpu(), torch.from_numpy(want).to(torch.bfloat16))


def test_an_expert_named_twice_counts_with_both_weights():
    need_gpu()
    rng = np.random.default_rng(3)
    weights, v12, vo = _experts(rng, "mxfp8", 4, 128, 160)
    for T in (2, 20):
        print(f"moe_few: an expert named twice, T {T}", flush=True)
        x = bf16(rng, (T, 128))
        idx = np.tile(np.array([[2, 0, 2]], np.int32), (T, 1))
        idx[1::3] = (1, 1, 1)
        w = rng.uniform(0.1, 1, (T, 3)).astype(np.float32)
        out = _run("mxfp8", x, idx, w, weights)
        ref, bound = few.moe(f64(x), idx, w.astype(np.float64), v12, vo)
        assert (np.abs(f64(out) - ref) <= bound).all()


def test_nothing_routed_leaves_the_residual():
    need_gpu()
    rng = np.random.default_rng(4)
    for kind in KINDS:
        weights, _, _ = _experts(rng, kind, 4, 128, 128)
        for T in (1, 30):
            print(f"moe_few {kind}: nothing routed, T {T}", flush=True)
            x, res = bf16(rng, (T, 128)), bf16(rng, (T, 128))
            x[0] = float("nan")
            idx, w = np.full((T, 2), -1, np.int32), np.full((T, 2), np.inf, np.float32)
            idx[:, 1] = 4
            assert torch.equal(_run(kind, x, idx, w, weights, res), res)
            assert (_run(kind, x, idx, w, weights) == 0).all()


def test_tokens_do_not_touch_each_other():
    need_gpu()
    rng = np.random.default_rng(5)
    weights, _, _ = _experts(rng, "mxfp4", 3, 256, 128)
    for T in (4, 25, 64):
        print(f"moe_few with NaN among {T} tokens", flush=True)
        x = bf16(rng, (T, 256))
        idx = np.stack([rng.permutation(3)[:2] for _ in range(T)]).astype(np.int32)
        w = rng.uniform(0.1, 1, (T, 2)).astype(np.float32)
        clean = _run("mxfp4", x, idx, w, weights)
        x[2] = float("nan")
        w[3, 0] = np.inf
        out = _run("mxfp4", x, idx, w, weights)
        rest = [t for t in range(T) if t not in (2, 3)]
        assert out[2].isnan().all() and not out[3].isfinite().any() and torch.equal(out[rest], clean[rest])


@pytest.mark.parametrize("T,E,k", [(64, 1024, 32), (64, 1024, 4), (3, 700, 32)])
def test_many_experts(T, E, k):
    """Hundreds of experts in one chunk of tokens: the largest tables."""
    need_gpu()
    print(f"moe_few E {E} k {k} T {T}", flush=True)
    rng = np.random.default_rng([T, E, k])
    D, H = 32, 32
    weights, v12, vo = _experts(rng, "mxfp4", E, D, H)
    idx, w = _choices(rng, T, E, k)
    x = bf16(rng, (T, D))
    out = _run("mxfp4", x, idx, w, weights)
    ref, bound = few.moe(f64(x), idx, w.astype(np.float64), v12, vo)
    assert (np.abs(f64(out) - ref) <= bound).all()


@pytest.mark.parametrize("kind", KINDS)
def test_a_gated_ffn_needs_no_choices(kind):
    need_gpu()
    rng = np.random.default_rng(6)
    weights, v12, vo = _experts(rng, kind, 1, 256, 384)
    for T in (1, 19, 64, 100):
        print(f"moe_few {kind}: gated FFN, T {T}", flush=True)
        x, res = bf16(rng, (T, 256)), bf16(rng, (T, 256))
        idx, one = np.zeros((T, 1), np.int32), np.ones((T, 1), np.float32)
        out = _run(kind, x, None, None, weights, res)
        assert torch.equal(out, _run(kind, x, idx, one, weights, res))
        ref, bound = few.moe(f64(x), idx, one, v12, vo, f64(res))
        assert (np.abs(f64(out) - ref) <= bound).all()
        assert _run(kind, x, None, None, weights, res, out=res) is res and torch.equal(res, out)
    assert _run(kind, x[:0], None, None, weights).shape == (0, 256)


def test_gates_at_the_ends():
    """silu far out on both sides, zero and infinite gates."""
    need_gpu()
    D, H = 32, 32
    v = np.zeros((2 * H, D))
    v[:H, 0], v[H:, 1] = 1.0, 1.0
    weights = (*device_experts([codes_of(v, "mxfp8")], [np.full((2 * H, 1), 127, np.uint8)], "mxfp8"),
               *device_experts([codes_of(np.eye(D), "mxfp8")], [np.full((D, 1), 127, np.uint8)], "mxfp8"))
    gates = [0.0, -0.0, -1e30, -200.0, -88.5, -40.0, 1e-30, 88.5, 200.0, 1e30]
    x = torch.zeros((len(gates), D))
    x[:, 0], x[:, 1] = torch.tensor(gates), 1.0
    x = x.to(torch.bfloat16).cuda()
    out = f64(_run("mxfp8", x, None, None, weights))
    a = f64(x)[:, 0]
    with np.errstate(over="ignore"):
        want = a / (1 + np.exp(-a))
    # fp32's exp(-a) is infinite below -88.7: silu is 0 there, and below 2^-120 everywhere near
    assert (np.abs(out - want[:, None]) <= 2.0 ** -7 * np.abs(want)[:, None] + 2.0 ** -120).all()
