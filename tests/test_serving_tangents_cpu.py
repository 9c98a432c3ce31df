"""Forward-mode tangents and layers prepared for serving: no GPU, the kernels are stood in for."""

import pytest
import torch
from torch.autograd import forward_ad

import blockwise_scaled_fp8_bs_amd as bs
from blockwise_scaled_fp8_bs_amd import binding, binding_few, moe, serving

LAYERS = {"linear": lambda: bs.Float8BlockwiseLinear(128, 128), "mx": lambda: bs.Float8MXLinear(128, 128),
          "ffn": lambda: bs.Float8BlockwiseGatedFFN(128, 512), "moe": lambda: bs.Float8BlockwiseMoE(128, 128, 4, 2)}


@pytest.fixture
def layer(request, monkeypatch):
    """The layer as prepare_serving() leaves it, on kernels that answer with ones."""
    ones = lambda x, *a, **kw: torch.ones((x.shape[0], 128), dtype=torch.bfloat16)  # noqa: E731
    monkeypatch.setattr(binding_few, "bs_few_mm", ones)
    monkeypatch.setattr(binding_few, "bs_moe_few", ones)
    monkeypatch.setattr(binding, "bs_scaled_mm", ones)
    monkeypatch.setattr(binding, "bs_mx_scaled_mm", ones)
    monkeypatch.setattr(serving, "token_rows", lambda x, features: x.view(-1, features))
    monkeypatch.setattr(moe, "_rows", lambda t, name: t.view(-1, t.shape[-1]))
    monkeypatch.setattr(moe, "moe_route", lambda logits, k, **kw: (torch.zeros((len(logits), k), dtype=torch.int32),
                                                                   torch.ones((len(logits), k))))
    m = LAYERS[request.param]().eval()
    m._lay_out(lambda *weights: (None,) * {"linear": 5, "mx": 5, "ffn": 9, "moe": 9}[request.param] + (64,))
    return m


@pytest.mark.parametrize("layer", LAYERS, indirect=True)
def test_a_tangent_is_refused(layer):
    x = torch.randn(3, 128).to(torch.bfloat16)
    with torch.no_grad(), forward_ad.dual_level():
        assert (layer(x) == 1).all()
        with pytest.raises(RuntimeError, match="tangent"):
            layer(forward_ad.make_dual(x, torch.ones_like(x)))
        assert forward_ad.unpack_dual(layer(x)).tangent is None


@pytest.mark.parametrize("layer", ["moe"], indirect=True)
def test_a_residual_s_tangent_is_refused(layer):
    x = torch.randn(3, 128).to(torch.bfloat16)
    with torch.no_grad(), forward_ad.dual_level():
        assert (layer(x, residual=x) == 1).all()
        with pytest.raises(RuntimeError, match="tangent"):
            layer(x, residual=forward_ad.make_dual(x, torch.ones_like(x)))
