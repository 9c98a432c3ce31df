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
