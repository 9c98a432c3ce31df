"""GPU dispatch and combine against the oracle: index arrays and the codes of
unweighted rows bit for bit, sums within their roundings."""

import numpy as np
import pytest
import torch

import blockwise_scaled_fp8_bs_amd as bs
from blockwise_scaled_fp8_bs_amd import inputs
from gpu_support import (bits16, check_canaries, check_scale_canaries, f32bits, guarded, need_gpu, scale_buffer,
                         special_input, u8)
from oracle import block, quant

pytestmark = pytest.mark.gpu


def _experts(T, k, E, seed, skew=1.0, drop=True):
    rng = np.random.default_rng(seed)
    v = rng.standard_normal((T, E)) + skew * rng.standard_normal(E)
    idx = np.argsort(-v, axis=1)[:, :k].astype(np.int32)
    if drop and T > 2:
        idx[::5, 0] = -1
        idx[2] = -1
    return idx


@pytest.mark.parametrize("T,k,E,align", [
    (1, 1, 1, 1), (1, 8, 64, 1), (24, 8, 64, 1), (24, 8, 64, 128), (100, 2, 8, 128), (513, 2, 7, 128), (1000, 3, 129, 16),
    (4096, 2, 8, 128), (4097, 2, 8, 128), (9000, 8, 256, 128), (70001, 2, 8, 128), (66000, 2, 1000, 1),
    (3000, 32, 512, 5),
])
def test_plan(T, k, E, align):
    need_gpu()
    idx = _experts(T, k, E, seed=T + E)
    if T > 3:
        idx[1, 0] = E + 5      # out of range: not routed
        idx[3, 0] = -7
    M = bs.bs_moe_plan_rows(T, k, E, align)
    for extra in (0, 256):
        print(f"plan T={T} k={k} E={E} align={align} M={M + extra}", flush=True)
        p = bs.bs_moe_plan(torch.from_numpy(idx).cuda(), E, align=align, M=M + extra)
        torch.cuda.synchronize()
        want = block.plan(np.where((idx < 0) | (idx >= E), -1, idx), E, align, M + extra)
        for got, ref, name in zip(p, want, p._fields):
            assert np.array_equal(got.cpu().numpy(), ref), name


def test_plan_of_nothing():
    need_gpu()
    p = bs.bs_moe_plan(torch.empty((0, 2), dtype=torch.int32, device="cuda"), 8)
    assert not p.group_end.any() and not p.counts.any() and p.row_slot.numel() == 0
    p = bs.bs_moe_plan(torch.full((40, 2), -1, dtype=torch.int32, device="cuda"), 8)
    assert not p.group_end.any() and (p.row_slot == -1).all() and (p.slot_row == -1).all()


@pytest.mark.parametrize("T,k,E,D,align", [(200, 2, 8, 384, 128), (33, 7, 16, 128, 128), (24, 8, 64, 256, 1),
                                           (1, 3, 8, 256, 1), (90, 1, 4, 640, 128)])
def test_gather_codes_bit_exact(T, k, E, D, align):
    need_gpu()
    x = special_input(T, D, seed=T)
    idx = _experts(T, k, E, seed=3)
    M = bs.bs_moe_plan_rows(T, k, E, align)
    _, _, _, row_slot = block.plan(idx, E, align, M)
    cols = M % 128 == 0
    rows = np.where(row_slot >= 0, row_slot // k, 0)
    v = np.where((row_slot >= 0)[:, None], bits16(x)[rows], 0).astype(np.uint16)
    xf, xg = guarded(T, D, torch.bfloat16)
    xg.copy_(x)
    yf, y = guarded(M, D, torch.bfloat16)
    qf, q = guarded(M, D, torch.uint8)
    sf, s = scale_buffer(D // 128, M)
    out = dict(y=y, q_row=q, s_row=s)
    if cols:
        cf, c = guarded(D, M, torch.uint8)
        tf, t = scale_buffer(M // 128, D)
        out.update(q_col=c, s_col=t)
    print(f"gather T={T} k={k} D={D} M={M} cols={cols}", flush=True)
    bs.bs_moe_gather_quant_1x128(xg, torch.from_numpy(row_slot).cuda(), k, **out)
    torch.cuda.synchronize()
    assert np.array_equal(bits16(y), v)
    qr, sr = quant.quant_1x128_rowwise(v)
    assert np.array_equal(u8(q), qr) and np.array_equal(f32bits(s)[:, :M], sr.T.copy().view(np.uint32))
    check_canaries(yf, M, D), check_canaries(qf, M, D), check_scale_canaries(sf, D // 128, M)
    if cols:
        qc, sc = quant.quant_1x128_colwise(v)
        assert np.array_equal(u8(c), qc) and np.array_equal(f32bits(t)[:, :D], sc.T.copy().view(np.uint32))
        check_canaries(cf, D, M), check_scale_canaries(tf, M // 128, D)
    for only in ({"y": y}, {"q_row": q, "s_row": s}, {n: out[n] for n in ("q_col", "s_col") if cols}):
        if only:
            for o in only.values():
                o.fill_(0 if o.dtype == torch.uint8 else -1)
            bs.bs_moe_gather_quant_1x128(xg, torch.from_numpy(row_slot).cuda(), k, **only)
            ref = {"y": v, "q_row": qr, "q_col": qc if cols else None}
            for n, o in only.items():
                if n in ref:
                    assert np.array_equal(bits16(o) if n == "y" else u8(o), ref[n]), n


def test_gather_ignores_slots_out_of_range():
    need_gpu()
    x = inputs.bf16_normal((4, 128), 1.0, 1).cuda()
    rs = torch.tensor([0, 8, -5, 7, 2 ** 31 - 1, -2 ** 31, 3, 1], dtype=torch.int32, device="cuda")
    y = torch.empty((8, 128), dtype=torch.bfloat16, device="cuda")
    bs.bs_moe_gather_quant_1x128(x, rs, 2, y=y)
    for r, slot in enumerate(rs.tolist()):
        assert torch.equal(y[r], x[slot // 2] if 0 <= slot < 8 else torch.zeros_like(y[r]))


@pytest.mark.parametrize("k", list(range(1, 33)))
def test_gather_divides_every_slot_right(k):
    need_gpu()
    T = 3000
    slots = torch.cat([torch.arange(0, 200), torch.randint(0, T * k, (300,)), torch.arange(T * k - 12, T * k)])
    x = torch.arange(T, dtype=torch.float32)
    x = torch.stack([x // 256, x % 256], 1).repeat(1, 64).to(torch.bfloat16).cuda()   # row index in two exact values
    y = torch.empty((512, 128), dtype=torch.bfloat16, device="cuda")
    bs.bs_moe_gather_quant_1x128(x, slots.to(torch.int32).cuda(), k, y=y)
    got = (y[:, 0].float() * 256 + y[:, 1].float()).long().cpu()
    assert torch.equal(got, slots // k)


def test_gather_weighted_codes():
    need_gpu()
    T, k, E, D = 150, 4, 8, 384
    x = inputs.bf16_normal((T, D), 0.01, 1)
    w = torch.rand((T, k), generator=torch.Generator().manual_seed(2))
    w[7] = 0.0
    idx = _experts(T, k, E, seed=9)
    M = bs.bs_moe_plan_rows(T, k, E, 128)
    _, _, _, row_slot = block.plan(idx, E, 128, M)
    q, s = torch.empty((M, D), dtype=torch.uint8, device="cuda"), bs.empty_scales(D // 128, M, "cuda")
    c, t = torch.empty((D, M), dtype=torch.uint8, device="cuda"), bs.empty_scales(M // 128, D, "cuda")
    y = torch.empty((M, D), dtype=torch.bfloat16, device="cuda")
    print("gather weighted", flush=True)
    bs.bs_moe_gather_quant_1x128(x.cuda(), torch.from_numpy(row_slot).cuda(), k, w=w.cuda(), y=y, q_row=q, s_row=s,
                                 q_col=c, s_col=t)
    torch.cuda.synchronize()
    v = block.gather(block.f64(bits16(x)), row_slot, k, w.numpy())
    # one fp32 product, then as any quantizer
    assert max(block.check_codes(u8(q), s.cpu().numpy()[:, :M].T, v, 2.0 ** -24)) <= 1
    assert max(block.check_codes(u8(c), t.cpu().numpy()[:, :D].T, v.T.copy(), 2.0 ** -24)) <= 1
    got = y.cpu().double().numpy()
    assert (np.abs(got - v) <= np.abs(v) * (2.0 ** -8 + 2.0 ** -23)).all()


@pytest.mark.parametrize("T,k,D", [(1, 8, 4096), (24, 8, 256), (101, 2, 1000), (7, 1, 8), (50, 32, 136), (33, 5, 5120)])
def test_combine_and_dw(T, k, D):
    need_gpu()
    E = max(k, 8)
    idx = _experts(T, k, E, seed=4)
    M = bs.bs_moe_plan_rows(T, k, E, 1) + 3
    _, _, slot_row, _ = block.plan(idx, E, 1, M)
    if T > 2:
        slot_row[1, 0] = M + 4      # outside: adds nothing
    y = inputs.bf16_normal((M, D), 1.0, 5)
    res = inputs.bf16_normal((T, D), 1.0, 6)
    dout = inputs.bf16_normal((T, D), 0.1, 7)
    w = torch.randn((T, k), generator=torch.Generator().manual_seed(8))
    if T > 2:
        w[2] = float("nan")         # a token without rows: its weights are not read
    yf, yg = guarded(M, D, torch.bfloat16)
    yg.copy_(y)
    of, og = guarded(T, D, torch.bfloat16)
    sr = torch.from_numpy(slot_row).cuda()
    Y, RES, DO = (block.f64(bits16(v)) for v in (y, res, dout))
    for ww in (w, None):
        for r in (res, None):
            print(f"combine T={T} k={k} D={D} w={ww is not None} res={r is not None}", flush=True)
            bs.bs_moe_combine(yg, sr, w=None if ww is None else ww.cuda(), residual=None if r is None else r.cuda(),
                              out=og)
            torch.cuda.synchronize()
            want, mag = block.combine(Y, slot_row, None if ww is None else ww.numpy(), None if r is None else RES)
            got = block.f64(bits16(og))
            # k fused multiply-adds in fp32, one rounding to bf16
            assert (np.abs(got - want) <= np.abs(want) * 2.0 ** -8 + mag * (k + 1) * 2.0 ** -24 + 1e-38).all()
            check_canaries(of, T, D)
    inplace = res.clone().cuda()
    bs.bs_moe_combine(yg, sr, w=w.cuda(), residual=inplace, out=inplace)
    ref = bs.bs_moe_combine(yg, sr, w=w.cuda(), residual=res.cuda())
    assert torch.equal(inplace.view(torch.int16), ref.view(torch.int16))
    dw = bs.bs_moe_combine_dw(dout.cuda(), yg, sr).cpu().double().numpy()
    want, mag = block.combine_dw(DO, Y, slot_row)
    # at most ceil(D / 512) * 8 + 6 additions follow one another
    assert (np.abs(dw - want) <= mag * (D // 64 + 16) * 2.0 ** -24 + 1e-38).all()


def test_on_a_side_stream_and_in_a_graph():
    need_gpu()
    T, k, E, D = 300, 2, 8, 256
    x = inputs.bf16_normal((T, D), 1.0, 1).cuda()
    logits = torch.randn((T, E), generator=torch.Generator().manual_seed(1)).cuda()

    def step():
        idx, w = bs.bs_moe_route(logits, k)
        p = bs.bs_moe_plan(idx, E)
        y = torch.empty((p.row_slot.shape[0], D), dtype=torch.bfloat16, device="cuda")
        bs.bs_moe_gather_quant_1x128(x, p.row_slot, k, y=y)
        out = bs.bs_moe_combine(y, p.slot_row, w=w, residual=x)
        dw = bs.bs_moe_combine_dw(x, y, p.slot_row)
        return idx, w, *p, y, out, dw, bs.bs_moe_route_bwd(logits, idx, w, dw)

    ref = [t.clone() for t in step()]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = step()
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, ref))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        outs = step()
    for r in range(3):
        for t in outs:
            t.fill_(3)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        for n, (a, b) in enumerate(zip(outs, ref)):
            assert torch.equal(a, b), (r, n)
    graph.reset()


def test_gather_from_rows_more_than_2_gib_apart():
    """Row strides that put the last rows past 32-bit offsets, against the same rows side by side."""
    need_gpu()
    T, D, k, ld = 300, 256, 2, 2 ** 22 - 64
    big = torch.empty(((T - 1) * ld + D,), dtype=torch.bfloat16, device="cuda")
    x = big.as_strided((T, D), (ld, 1))
    x.copy_(inputs.bf16_normal((T, D), 1.0, 1))
    g = torch.Generator().manual_seed(2)
    idx = torch.randint(0, 4, (T, k), generator=g).to(torch.int32).cuda()
    w = torch.rand((T, k), generator=g).cuda()
    p = bs.bs_moe_plan(idx, 4)
    M = p.row_slot.shape[0]
    got = []
    for src in (x, x.contiguous()):
        for weight in (None, w):
            print(f"gather stride {src.stride(0)} weighted {weight is not None}", flush=True)
            o = dict(y=torch.empty((M, D), dtype=torch.bfloat16, device="cuda"), q_row=torch.empty((M, D), dtype=torch.uint8, device="cuda"),
                     s_row=bs.empty_scales(D // 128, M, "cuda"), q_col=torch.empty((D, M), dtype=torch.uint8, device="cuda"),
                     s_col=bs.empty_scales(M // 128, D, "cuda"))
            bs.bs_moe_gather_quant_1x128(src, p.row_slot, k, w=weight, **o)
            got.append([t[:, :M] if n == "s_row" else t[:, :D] if n == "s_col" else t for n, t in o.items()])
    for a, b in zip(got[:2], got[2:]):
        assert all(torch.equal(s.contiguous().view(torch.uint8), t.contiguous().view(torch.uint8)) for s, t in zip(a, b))
