"""GPU gather at the sizes whose workgroups take several column tiles each, in
strips: against the plain quantizer and against the same rows in parts."""

import pytest
import torch

import blockwise_scaled_fp8_bs_amd as bs
from gpu_support import need_gpu

pytestmark = pytest.mark.gpu


def _outputs(M, D):
    return dict(y=torch.zeros((M, D), dtype=torch.bfloat16, device="cuda"), q_row=torch.zeros((M, D), dtype=torch.uint8, device="cuda"),
                s_row=torch.zeros((D // 128, M), device="cuda"), q_col=torch.zeros((D, M), dtype=torch.uint8, device="cuda"),
                s_col=torch.zeros((M // 128, D), device="cuda"))


def _same(a, b):
    return torch.equal(a.contiguous().view(torch.uint8), b.contiguous().view(torch.uint8))


@pytest.mark.parametrize("T,k,ld", [(210000, 2, 640), (421000, 1, 640), (210000, 2, 5184)],
                         ids=["two slots", "one slot", "rows past 2 GiB"])
def test_gather_in_strips(T, k, ld):
    """Five column tiles: a strip of four and one of a single tile."""
    need_gpu()
    D, E, part = 640, 8, 65536
    g = torch.Generator(device="cuda").manual_seed(T + k)
    x = torch.empty((T, ld), dtype=torch.bfloat16, device="cuda")[:, :D]
    x.copy_(torch.randn((T, D), generator=g, device="cuda"))
    idx = torch.randint(-1, E, (T, k), generator=g, device="cuda", dtype=torch.int32)
    w = torch.rand((T, k), generator=g, device="cuda")
    row_slot = bs.bs_moe_plan(idx, E).row_slot
    M = row_slot.shape[0]
    assert (M // 128) * (D // 128) >= 16384 > (part // 128) * (D // 128)  # in strips as a whole, not in parts
    rows = x[(row_slot // k).clamp_min(0).long()].masked_fill_((row_slot < 0)[:, None], 0)
    plain, whole, some = _outputs(M, D), _outputs(M, D), _outputs(part, D)
    print(f"gather in strips T={T} k={k} ld={ld}", flush=True)
    bs.bs_moe_gather_quant_1x128(x, row_slot, k, **whole)
    del plain["y"]
    bs.bs_quant_1x128(rows, **plain)
    assert _same(whole["y"], rows) and all(_same(whole[n], plain[n]) for n in plain)
    del plain, rows
    for weight in (None, w):
        for names in (("q_row", "s_row", "q_col", "s_col"), ("q_row", "s_row"), ("y", "q_col", "s_col")):
            for t in whole.values():
                t.zero_()
            bs.bs_moe_gather_quant_1x128(x, row_slot, k, w=weight, **{n: whole[n] for n in names})
            for lo in range(0, M, part):
                n = min(part, M - lo)
                few = dict(y=some["y"][:n], q_row=some["q_row"][:n], s_row=some["s_row"], q_col=some["q_col"][:, :n],
                           s_col=some["s_col"][:n // 128])
                bs.bs_moe_gather_quant_1x128(x, row_slot[lo:lo + n].contiguous(), k, w=weight, **{m: few[m] for m in names})
                got = dict(y=whole["y"][lo:lo + n], q_row=whole["q_row"][lo:lo + n], s_row=whole["s_row"][:, lo:lo + n],
                           q_col=whole["q_col"][:, lo:lo + n], s_col=whole["s_col"][lo // 128:(lo + n) // 128])
                few["s_row"] = few["s_row"][:, :n]
                assert all(_same(got[m], few[m]) for m in names), (weight is not None, names, lo)
