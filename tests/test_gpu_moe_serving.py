"""Which weights and plans the expert layer answers with."""

import pytest
import torch

import blockwise_scaled_fp8_bs_amd as bs
from gpu_support import need_gpu

pytestmark = pytest.mark.gpu


def test_served_layer_answers_with_its_present_weights():
    """After each way to exchange the weights: the output of a layer that was never laid out."""
    need_gpu()
    torch.manual_seed(3)
    m = bs.Float8BlockwiseMoE(128, 128, 4, 2, device="cuda").eval()
    plain = bs.Float8BlockwiseMoE(128, 128, 4, 2, device="cuda").eval()
    x = torch.randn(5, 128, device="cuda").to(torch.bfloat16)
    new = lambda t: torch.nn.Parameter(torch.empty_like(t).uniform_(-0.2, 0.2))  # noqa: E731

    def want(state):
        plain.load_state_dict(state)
        return plain(x)

    print("served layer with exchanged weights", flush=True)
    with torch.no_grad():
        m.prepare_serving()
        old = m(x)
        assert torch.equal(old, want(m.state_dict()))
        other = {n: p.detach().clone().mul_(2) for n, p in m.named_parameters()}
        got = torch.func.functional_call(m, other, (x,))
        assert torch.equal(got, want({**m.state_dict(), **other})) and not torch.equal(got, old)
        assert torch.equal(m(x), old)
        m.w12 = new(m.w12)
        assert torch.equal(m(x), want(m.state_dict())) and not torch.equal(m(x), old)
        m.prepare_serving()
        m.out_proj.data = new(m.out_proj).data
        with pytest.raises(RuntimeError, match="call it again"):
            m(x)


def test_plans_with_groups_that_are_not_padded_to_128_rows():
    """The layer's weight gradients contract whole 128-row blocks of a group."""
    need_gpu()
    T, k, E, D, H = 300, 2, 4, 128, 128
    g = torch.Generator().manual_seed(1)
    x = torch.randn((T, D), generator=g).to(torch.bfloat16).cuda()
    idx = torch.randint(-1, E, (T, k), generator=g).to(torch.int32).cuda()
    w = torch.rand((T, k), generator=g).cuda()
    w12, wo = (torch.randn(s, generator=g).mul_(0.1).to(torch.bfloat16).cuda().requires_grad_(True)
               for s in ((E, 2 * H, D), (E, D, H)))
    for kw in (dict(align=192), dict(align=1, M=bs.bs_moe_plan_rows(T, k, E)), dict(align=64, M=bs.bs_moe_plan_rows(T, k, E))):
        plan = bs.bs_moe_plan(idx, E, **kw)
        assert plan.align == kw["align"]
        with pytest.raises(ValueError, match="the plan is for"):
            bs.float8_blockwise_moe_ffn(x, idx, w, w12, wo, plan=plan)
    # one expert, as many rows as slots, some not routed
    one = bs.bs_moe_plan(idx[:128, :1].contiguous(), 1, align=1)
    with pytest.raises(ValueError, match="the plan is for"):
        bs.float8_blockwise_moe_ffn(x[:128], idx[:128, :1].contiguous(), w[:128, :1].contiguous(), w12[:1].detach(), wo[:1].detach(), plan=one)
    # more padding than needed gives the same outputs and gradients
    got = []
    for plan in (bs.bs_moe_plan(idx, E), bs.bs_moe_plan(idx, E, align=256)):
        print(f"experts with groups of whole {plan.align} rows", flush=True)
        y = bs.float8_blockwise_moe_ffn(x, idx, w, w12, wo, plan=plan)
        got.append([y, *torch.autograd.grad(y, (w12, wo), x)])
    for a, b in zip(*got):
        assert torch.equal(a, b)
