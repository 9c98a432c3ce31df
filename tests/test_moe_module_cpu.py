"""The expert layer as a module: no GPU."""

import pytest
import torch

import blockwise_scaled_fp8_bs_amd as bs


@pytest.mark.parametrize("change", [lambda m: m.to(torch.bfloat16), lambda m: m.bfloat16(), lambda m: m.to("cpu", torch.bfloat16),
                                    lambda m: m.float().bfloat16(), lambda m: torch.nn.Sequential(m).bfloat16()[0]])
def test_a_model_cast_to_bf16_keeps_the_balance_in_fp32(change):
    """The router takes its bias in fp32 only, and steps of 1e-3 would vanish in bf16."""
    m = bs.Float8BlockwiseMoE(128, 128, 4, 2)
    with torch.no_grad():
        m.balance.copy_(torch.tensor([1.001, -0.0003, 2.5, 0.1]))
    want = m.balance.clone()
    m = change(m)
    assert m.balance.dtype == torch.float32 and torch.equal(m.balance, want)
    assert "balance" in m.state_dict() and m.state_dict()["balance"].dtype == torch.float32
    assert all(p.dtype == torch.bfloat16 for p in m.parameters())


def test_the_balance_moves_with_the_module():
    m = bs.Float8BlockwiseMoE(128, 128, 4, 2)
    m.to("meta", torch.bfloat16)
    assert m.balance.device.type == "meta" and m.balance.dtype == torch.float32
