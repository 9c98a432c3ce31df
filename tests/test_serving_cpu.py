"""What a module keeps of the weights that it laid out for serving: no GPU."""

import copy
import pickle

import pytest
import torch

import blockwise_scaled_fp8_bs_amd as bs
from blockwise_scaled_fp8_bs_amd.serving import ServedWeights


class Layer(ServedWeights, torch.nn.Module):
    _served_names = ("a", "b")

    def __init__(self):
        super().__init__()
        self.a, self.b = (torch.nn.Parameter(torch.randn(4, 4)) for _ in range(2))

    def prepare_serving(self):
        return self._lay_out(lambda a, b: (a.clone(), b.clone()))


def _same(layer):
    got = layer._layout()
    return torch.equal(got[0], layer.a) and torch.equal(got[1], layer.b)


def test_the_layout_is_that_of_the_weights():
    m = Layer()
    assert m._layout() is None
    assert _same(m.prepare_serving()) and not m._serving[0].requires_grad
    m.eval()
    assert _same(m)
    m.train()
    assert m._layout() is None


@pytest.mark.parametrize("name", ["a", "b"])
def test_other_weights_have_none(name):
    m = Layer().prepare_serving()
    seen = []
    m.forward = lambda: seen.append(m._layout())
    torch.func.functional_call(m, {name: torch.zeros(4, 4)}, ())
    assert seen == [None] and _same(m)
    setattr(m, name, torch.nn.Parameter(torch.zeros(4, 4)))
    assert m._layout() is None


@pytest.mark.parametrize("change", [lambda m: m.a.mul_(2), lambda m: setattr(m.b, "data", torch.zeros(4, 4))])
def test_weights_that_changed_underneath_raise(change):
    m = Layer().prepare_serving()
    with torch.no_grad():
        change(m)
    with pytest.raises(RuntimeError, match="call it again"):
        m._layout()
    assert _same(m.prepare_serving())


def test_moves_loads_and_copies_drop_it():
    m = Layer().prepare_serving()
    for other in (copy.deepcopy(m), pickle.loads(pickle.dumps(m))):
        assert other._layout() is None and m._layout() is not None
    m.load_state_dict(m.state_dict())
    assert m._layout() is None
    m.prepare_serving().double()
    assert m._layout() is None


def test_inference_weights_are_refused():
    with torch.inference_mode():
        m = Layer()
    with pytest.raises(RuntimeError, match="inference"):
        m.prepare_serving()


@pytest.mark.parametrize("layer", [lambda: bs.Float8BlockwiseLinear(128, 128), lambda: bs.Float8MXLinear(128, 128),
                                   lambda: bs.Float8BlockwiseGatedFFN(128, 512), lambda: bs.Float8BlockwiseMoE(128, 128, 4, 2)])
def test_formats_that_there_are_not(layer):
    m = layer()
    with pytest.raises(ValueError, match="weights must be one of"):
        m.prepare_serving("int8")
    with pytest.raises(ValueError, match="few_tokens"):
        m.prepare_serving(few_tokens=-1)
    assert m._layout() is None
