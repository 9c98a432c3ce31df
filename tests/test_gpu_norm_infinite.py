"""GPU residual norms of rows that are not finite."""

import numpy as np
import pytest
import torch

import blockwise_scaled_fp8_bs_amd as bs
from blockwise_scaled_fp8_bs_amd import inputs
from gpu_support import need_gpu
from oracle import block

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("D", [64, 4096, 5120, 8192, 16384])
def test_rows_that_are_not_finite(D):
    """1 / sqrt(inf) is 0: in a row with an infinity the finite elements are
    normalized to 0 and the infinity itself to NaN; a NaN takes the whole row."""
    need_gpu()
    R = 6
    x, u = inputs.bf16_normal((R, D), 1.0, 1), inputs.bf16_normal((R, D), 1.0, 2)
    u[1, D - 1] = float("inf")
    u[2, 0], u[2, 3] = float("-inf"), float("inf")
    u[3, 5] = float("nan")
    x[4, 7] = float("-inf")
    w_post, w_pre = torch.full((D,), 1.5), torch.full((D,), 0.5)
    r, h = torch.empty((R, D), dtype=torch.bfloat16, device="cuda"), torch.empty((R, D), dtype=torch.bfloat16, device="cuda")
    rstd_u, rstd_r = torch.empty(R, device="cuda"), torch.empty(R, device="cuda")
    print(f"norm of rows that are not finite D={D}", flush=True)
    bs.bs_resid_norm(x.cuda(), w_pre.cuda(), u=u.cuda(), w_post=w_post.cuda(), eps=1e-6, r=r, h=h, rstd_u=rstd_u,
                     rstd_r=rstd_r)
    eps = float(np.float32(1e-6))
    with np.errstate(invalid="ignore"):
        want_r = block.resid(x.double().numpy(), u.double().numpy(), w_post.double().numpy(), None, 1.0, eps)
        r64 = r.cpu().double().numpy()
        want_h = block.norm(r64, w_pre.double().numpy(), eps)
        want_ru, want_rr = block.rstd(u.double().numpy(), eps), block.rstd(r64, eps)
    for got, want in ((r64, want_r), (h.cpu().double().numpy(), want_h), (rstd_u.cpu().double().numpy(), want_ru),
                      (rstd_r.cpu().double().numpy(), want_rr)):
        assert np.array_equal(np.isnan(got), np.isnan(want))
        on = np.isfinite(want)
        # half a step of bf16 and three roundings of fp32
        assert (np.abs(got[on] - want[on]) <= np.abs(want[on]) * (2.0 ** -8 + 2.0 ** -22)).all()
        assert np.array_equal(got[np.isinf(want)], want[np.isinf(want)])
    assert want_ru[1] == want_ru[2] == 0 and np.isnan(want_r[1]).sum() == 1 and want_rr[4] == 0
    # a row of zeros with no eps: 1 / sqrt(0) is infinite, and 0 times that NaN
    zero = torch.zeros((1, D), dtype=torch.bfloat16, device="cuda")
    bs.bs_resid_norm(zero, w_pre.cuda(), eps=0.0, h=h[:1], rstd_r=rstd_r[:1])
    assert float(rstd_r[0]) == float("inf") and torch.isnan(h[0]).all()
