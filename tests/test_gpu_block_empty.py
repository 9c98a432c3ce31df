"""GPU calls of the MoE block on no rows."""

import pytest
import torch

import blockwise_scaled_fp8_bs_amd as bs
from gpu_support import need_gpu

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("B", [0, 1, 2])
def test_no_rows_with_a_gate(B):
    need_gpu()
    D = 256
    x = torch.empty((B, 0, D) if B else (0, 3, D), dtype=torch.bfloat16, device="cuda", requires_grad=True)
    u = torch.empty_like(x, requires_grad=True)
    w_post, w_pre = (torch.ones(D, device="cuda", requires_grad=True) for _ in range(2))
    gate = torch.ones((B, D), device="cuda", requires_grad=True)
    print(f"norm of no rows, a gate of {B}", flush=True)
    r, h = bs.resid_norm(x, w_pre, u=u, w_post=w_post, gate=gate)
    assert r.shape == h.shape == x.shape
    (r.float().sum() + h.float().sum()).backward()
    for t in (x, u, w_post, w_pre, gate):
        assert t.grad.shape == t.shape and not t.grad.any()


def test_no_rows_into_prepared_outputs():
    """Codes of no rows, into views of buffers that were made for more."""
    need_gpu()
    D = 256
    q, s = torch.empty((128, D), dtype=torch.uint8, device="cuda"), bs.empty_scales(D // 128, 128, "cuda").fill_(5.0)
    x = torch.empty((0, D), dtype=torch.bfloat16, device="cuda")
    w = torch.ones(D, device="cuda")
    print("codes of no rows", flush=True)
    bs.bs_resid_norm(x, w, q_row=q[:0], s_row=s)
    bs.bs_moe_gather_quant_1x128(x, torch.empty(0, dtype=torch.int32, device="cuda"), 2, q_row=q[:0], s_row=s)
    assert (s == 5.0).all()


def test_no_tokens_through_the_autograd_pieces():
    """A sum's gradient of no elements comes with strides of 0."""
    need_gpu()
    D = 256
    x = torch.empty((0, D), dtype=torch.bfloat16, device="cuda", requires_grad=True)
    logits = torch.empty((0, 8), device="cuda", requires_grad=True)
    print("autograd pieces of no tokens", flush=True)
    idx, w = bs.moe_route(logits, 2)
    plan = bs.bs_moe_plan(idx, 8)
    y = bs.moe_combine(bs.moe_dispatch(x, plan), plan, w, x)
    y.sum().backward()
    assert y.shape == x.grad.shape == (0, D) and logits.grad.shape == (0, 8)
