"""Every way in which the few-token kernels are launched, against float64: each
test first asks what its sizes run, so that a changed rule cannot empty it."""

import numpy as np
import pytest
import torch

import blockwise_scaled_fp8_bs_amd as bs
from few_support import (KINDS, bf16, codes_of, device_experts, device_weight, f64, finite_codes, guarded_rows, random_scales,
                         untouched)
from gpu_support import need_gpu
from oracle import few

pytestmark = pytest.mark.gpu

UNIT = {"e4m3": 128, "mxfp8": 128, "mxfp4": 256}     # weights of a row in a unit, at most


# --- products: two tiles of columns a workgroup

def _columns(kind):
    return (8192, 4224, 8320) if kind == "e4m3" else (8192, 4097, 8200, 6161, 8209, 8225)


WIDE = [(kind, T, N, K) for kind in KINDS
        for i, (T, K) in enumerate(((17, 256), (32, 768), (33, 256), (64, 640), (70, 384)))
        for N in (_columns(kind)[i % len(_columns(kind))], _columns(kind)[-1 - i % 2])]


@pytest.mark.parametrize("kind,T,N,K", WIDE)
def test_products_by_two_tiles(kind, T, N, K):
    need_gpu()
    if kind != "e4m3":
        K -= 96 if T % 2 else 32        # the last unit is a part of one
    plan = bs.bs_diag_few_mm_plan(KINDS[kind], T, N, K)
    assert plan["tiles"] == 2 and plan["rows"] == (32 if T <= 32 else 64)
    print(f"few_mm {kind} T {T} N {N} K {K}", flush=True)
    rng = np.random.default_rng([T, N, K, 3])
    q, s = finite_codes(rng, kind, N, K), random_scales(rng, kind, N, K)
    w, sw = device_weight(q, s, kind, T % 2)
    x, res = bf16(rng, (T, K)), bf16(rng, (T, N + 1))[:, :N] if T % 2 else None
    wv = few.weights(q, s, kind)
    for dtype in (torch.bfloat16, torch.float32):
        full, out = guarded_rows(T, N, dtype, extra=4 if T % 4 == 0 else 3)
        bs.bs_few_mm(x, w, sw, KINDS[kind], residual=res, out=out)
        assert untouched(full, T, N)
        ref, bound = few.few_mm(f64(x), wv, None if res is None else f64(res), bf16=dtype == torch.bfloat16)
        assert (np.abs(f64(out) - ref) <= bound).all()
        assert torch.equal(bs.bs_few_mm(x, w, sw, KINDS[kind], residual=res, out_dtype=dtype), out)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("T", [17, 33, 66])
def test_whole_numbers_by_two_tiles(kind, T):
    need_gpu()
    N, K = _columns(kind)[-1], 640
    assert bs.bs_diag_few_mm_plan(KINDS[kind], T, N, K)["tiles"] == 2
    print(f"few_mm integers {kind} T {T} N {N} K {K}", flush=True)
    rng = np.random.default_rng([T, N, 4])
    q = codes_of(rng.choice([0, 1, 2, 3, 4, 6], (N, K)) * rng.choice([-1, 1], (N, K)), kind)
    if kind == "e4m3":
        s = np.exp2(rng.integers(-2, 3, (N // 128, K // 128))).astype(np.float32)
    else:
        s = rng.integers(125, 130, (N, K // 32)).astype(np.uint8)
    x = torch.from_numpy(rng.integers(-8, 9, (T, K)).astype(np.float32)).to(torch.bfloat16).cuda()
    # |sum| <= 8 * 24 * 640 < 2^17, in quarters: exact in fp32
    out = bs.bs_few_mm(x, *device_weight(q, s, kind), KINDS[kind], out_dtype=torch.float32)
    assert np.array_equal(f64(out), f64(x) @ few.weights(q, s, kind).T)


# --- experts

def _experts(rng, kind, E, D, H):
    args, values = [], []
    for N, K in ((2 * H, D), (D, H)):
        qs = [finite_codes(rng, kind, N, K) for _ in range(E)]
        ss = [random_scales(rng, kind, N, K) for _ in range(E)]
        args += device_experts(qs, ss, kind)
        values.append([few.weights(q, s, kind) for q, s in zip(qs, ss)])
    return args, values


def _choices(rng, T, E, k):
    """Choices that use every expert where there are as many of them, a tenth dropped."""
    order = np.concatenate([rng.permutation(E) for _ in range((T * k + E - 1) // E + 1)])
    idx = np.empty((T, k), np.int32)
    at = 0
    for t in range(T):
        mine = []
        while len(mine) < k:
            if order[at % len(order)] not in mine:
                mine.append(order[at % len(order)])
            at += 1
        idx[t] = mine
    idx[rng.random((T, k)) < 0.1] = -1
    w = rng.uniform(0.05, 1, (T, k)).astype(np.float32)
    w[idx < 0] = np.nan     # never used
    return idx, w


def _check(rng, kind, T, D, H, E, k, idx, w):
    args, values = _experts(rng, kind, E, D, H)
    x = bf16(rng, (T, D))
    put = lambda v: torch.from_numpy(v).cuda()  # noqa: E731
    call = lambda **kw: bs.bs_moe_few(x, put(idx), put(w), *args, KINDS[kind], **kw)  # noqa: E731
    ref, bound = few.moe(f64(x), idx, w.astype(np.float64), *values)
    plain = call()
    assert (np.abs(f64(plain) - ref) <= bound).all()
    # on a residual, rows of odd strides
    res = bf16(rng, (T, D + 1))[:, :D]
    full, out = guarded_rows(T, D, torch.bfloat16)
    call(residual=res, out=out)
    assert untouched(full, T, D)
    ref, bound = few.moe(f64(x), idx, w.astype(np.float64), *values, f64(res))
    assert (np.abs(f64(out) - ref) <= bound).all()
    assert torch.equal(call(residual=res.contiguous()), out) and torch.equal(call(), plain)


# (T, D, H, E, k), tokens of an item, tiles of the output of a workgroup
SHARED = [((1, 128, 4096, 8, 8), 16, 1), ((4, 128, 4096, 8, 8), 16, 1), ((8, 128, 2048, 16, 8), 16, 1),
          ((16, 256, 2048, 24, 8), 16, 1), ((24, 128, 2048, 24, 3), 16, 1), ((40, 128, 2048, 8, 4), 32, 1),
          ((66, 128, 2048, 16, 4), 32, 1), ((130, 128, 4096, 4, 2), 32, 1), ((40, 4096, 640, 16, 2), 16, 2)]


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("sizes,tokens,tiles", SHARED)
def test_workgroups_that_share_columns(kind, sizes, tokens, tiles):
    need_gpu()
    T, D, H, E, k = sizes
    if kind != "e4m3":
        H += 32 * (T % 3)
    plan = bs.bs_diag_moe_few_plan(KINDS[kind], T, D, H, E, k)
    assert plan["splits"] > 1 and plan["tokens"] == tokens and plan["out_tiles"] == tiles
    print(f"moe_few {kind} T {T} D {D} H {H} E {E} k {k}, {plan['splits']} shares", flush=True)
    rng = np.random.default_rng([T, D, H, E, k, 5])
    _check(rng, kind, T, D, H, E, k, *_choices(rng, T, E, k))


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("sizes,tokens,tiles", [((128, 2560, 256, 4, 2), 32, 2), ((100, 2816, 128, 16, 3), 16, 2),
                                                ((64, 4096, 256, 4, 2), 32, 1), ((20, 4224, 128, 8, 3), 16, 2)])
def test_tiles_of_the_output(kind, sizes, tokens, tiles):
    """Two at a time where one would need a second round of the CUs, also by the tokens of a second chunk."""
    need_gpu()
    T, D, H, E, k = sizes
    if kind != "e4m3":
        H += 32
    plan = bs.bs_diag_moe_few_plan(KINDS[kind], T, D, H, E, k)
    assert plan["out_tiles"] == tiles and plan["tokens"] == tokens and plan["splits"] == 1
    print(f"moe_few {kind} T {T} D {D} H {H} E {E} k {k}, {tiles} tiles of the output", flush=True)
    rng = np.random.default_rng([T, D, H, E, k, 9])
    _check(rng, kind, T, D, H, E, k, *_choices(rng, T, E, k))


# (T, D, H, E, k), tokens of an item, tiles of h that a wave streams at a time
STREAMED = [((1, 384, 6144, 8, 8), 16, 1), ((2, 384, 4096, 16, 8), 16, 1), ((4, 512, 2048, 24, 8), 16, 1),
            ((5, 384, 4096, 12, 4), 16, 1), ((8, 384, 2048, 24, 4), 16, 1), ((12, 384, 2048, 24, 6), 16, 1),
            ((40, 384, 4096, 16, 3), 16, 2), ((64, 640, 4096, 16, 2), 16, 2), ((40, 384, 4096, 5, 2), 32, 1),
            ((70, 384, 4096, 5, 2), 32, 1)]


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("sizes,tokens,tiles", STREAMED)
def test_waves_that_stream_several_tiles(kind, sizes, tokens, tiles):
    """Several tiles of several units a wave, so that loads run ahead into the next one's."""
    need_gpu()
    T, D, H, E, k = sizes
    if kind != "e4m3":
        D, H = D + 32 * (T % 4), H + 32 * (T % 3)
    plan = bs.bs_diag_moe_few_plan(KINDS[kind], T, D, H, E, k)
    rng = np.random.default_rng([T, D, H, E, k, 6])
    idx, w = _choices(rng, T, E, k)
    chunk = idx[:64]
    items = sum(-(-int((chunk == e).any(1).sum()) // plan["tokens"]) for e in range(E))
    assert plan["up_tiles"] == tiles and plan["tokens"] == tokens and items <= plan["items"]
    assert items * (H // (16 * tiles)) > 1.2 * plan["up_waves"] and D > UNIT[kind]
    print(f"moe_few {kind} T {T} D {D} H {H} E {E} k {k}, {items} items", flush=True)
    _check(rng, kind, T, D, H, E, k, idx, w)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("sizes,tokens", [((3, 256, 128, 4, 2), 16), ((6, 640, 512, 5, 3), 16), ((40, 2048, 256, 4, 2), 32)])
def test_waves_that_share_a_tile(kind, sizes, tokens):
    need_gpu()
    T, D, H, E, k = sizes
    plan = bs.bs_diag_moe_few_plan(KINDS[kind], T, D, H, E, k)
    assert plan["up_tiles"] == 0 and plan["tokens"] == tokens
    print(f"moe_few {kind} T {T} D {D} H {H} E {E} k {k}, shared tiles", flush=True)
    rng = np.random.default_rng([T, D, H, E, k, 7])
    _check(rng, kind, T, D, H, E, k, *_choices(rng, T, E, k))


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("T,H,D,E,k", [(4, 2048, 256, 32, 8), (24, 2048, 256, 24, 4), (64, 4096, 256, 12, 3), (64, 4096, 256, 4, 2)])
def test_whole_numbers_in_streamed_and_shared_tiles(kind, T, H, D, E, k):
    """Gates of 128 and more, where silu(a) = a in fp32, and small integers for everything else: any token, slot,
    expert, row or column taken for another shows.  Both kernels take the paths above."""
    need_gpu()
    plan = bs.bs_diag_moe_few_plan(KINDS[kind], T, D, H, E, k)
    assert plan["up_tiles"] > 0 and plan["splits"] > 1
    print(f"moe_few integers {kind} T {T} D {D} H {H} E {E} k {k}", flush=True)
    rng = np.random.default_rng([T, E, k, 8])
    one = (lambda N, K: np.ones((N // 128, K // 128), np.float32)) if kind == "e4m3" else (lambda N, K: np.full((N, K // 32), 127, np.uint8))
    x = rng.integers(0, 2, (T, D)).astype(np.float32)
    x[:, 0] = 64.0
    v12, vo = [], []
    for _ in range(E):
        v = np.zeros((2 * H, D))
        v[:H, 0] = rng.choice([2, 4], H)                     # a = 128 or 256
        v[H:, 1:] = rng.choice([0, 0, 0, 1], (H, D - 1)) * rng.choice([-1, 1], (H, D - 1))
        v12.append(v)
        o = np.zeros((D, H))                                 # few of them, so that sums stay below 2^24 quarters
        o[np.arange(D)[:, None], rng.integers(0, H, (D, 64))] = rng.choice([1, -1, 2], (D, 64))
        vo.append(o)
    args = (*device_experts([codes_of(v, kind) for v in v12], [one(2 * H, D)] * E, kind),
            *device_experts([codes_of(v, kind) for v in vo], [one(D, H)] * E, kind))
    idx, w = _choices(rng, T, E, k)
    w = np.exp2(rng.integers(-2, 2, (T, k))).astype(np.float32)
    res = torch.from_numpy(rng.integers(-100, 100, (T, D)).astype(np.float32)).to(torch.bfloat16).cuda()
    out = bs.bs_moe_few(torch.from_numpy(x).to(torch.bfloat16).cuda(), torch.from_numpy(idx).cuda(), torch.from_numpy(w).cuda(), *args,
                        KINDS[kind], residual=res)
    want = f64(res).copy()
    most = np.abs(want)
    for t in range(T):
        for j in range(k):
            if idx[t, j] >= 0:
                ab = v12[idx[t, j]] @ x[t]
                h = w[t, j] * ab[:H] * ab[H:]
                assert np.abs(ab[H:]).max() < 256            # h in 8 bits
                want[t] += vo[idx[t, j]] @ h
                most[t] += np.abs(vo[idx[t, j]]) @ np.abs(h)
    assert most.max() < 2 ** 22
    assert torch.equal(out.cpu(), torch.from_numpy(want).to(torch.bfloat16))
