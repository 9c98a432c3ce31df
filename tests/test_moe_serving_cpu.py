"""Which weights a served expert layer answers with: the library's calls are
replaced by recorders, a layout by a copy of the weights it was made of."""

import copy
import pickle

import pytest
import torch

import blockwise_scaled_fp8_bs_amd as bs
from blockwise_scaled_fp8_bs_amd import moe


@pytest.fixture
def layer(monkeypatch):
    """(module, answer): answer(call) runs call() and returns the weights w12, out_proj that its products took."""
    T, D, E, k = 3, 128, 4, 2
    used = []

    def group_m(ends, q, w, s, zeros=False):
        used.append(w)
        return torch.zeros((T * k, w.shape[1]), dtype=torch.bfloat16)

    def plain(x, idx, w, w12, out_proj, **kw):
        used.extend((w12.detach().clone(), out_proj.detach().clone()))
        return x

    def plan(idx, E, align=128):
        z = torch.zeros(E, dtype=torch.int32)
        return bs.MoEPlan(z, z, idx, torch.zeros(T * k, dtype=torch.int32))

    monkeypatch.setattr(moe, "_rows", lambda t, name: t.view(-1, t.shape[-1]))
    monkeypatch.setattr(moe, "_expert_weights", lambda w: (w.detach().clone(), None, None, None))
    monkeypatch.setattr(moe, "moe_route", lambda logits, k, **kw: (torch.zeros((T, k), dtype=torch.int32), torch.ones((T, k))))
    monkeypatch.setattr(moe, "_group_m", group_m)
    monkeypatch.setattr(moe, "float8_blockwise_moe_ffn", plain)
    monkeypatch.setattr(moe._k, "bs_moe_plan", plan)
    monkeypatch.setattr(moe._k, "bs_moe_gather_quant_1x128", lambda *a, **kw: None)
    monkeypatch.setattr(moe._k, "bs_moe_combine", lambda *a, **kw: torch.zeros((T, D), dtype=torch.bfloat16))
    monkeypatch.setattr(moe._b, "bs_swiglu_quant_1x128", lambda *a, **kw: None)
    m = bs.Float8BlockwiseMoE(D, 128, E, k).eval()
    x = torch.zeros((T, D), dtype=torch.bfloat16)

    def answer(call=None):
        used.clear()
        with torch.no_grad():
            call() if call is not None else m(x)
        assert len(used) == 2
        return used

    return m, x, answer


def _same(got, w12, out_proj):
    return torch.equal(got[0], w12) and torch.equal(got[1], out_proj)


def test_the_layout_is_served_while_the_weights_are_those_it_was_made_of(layer):
    m, x, answer = layer
    m.prepare_serving()
    got = answer()
    assert got[0] is m._serving[0] and _same(got, m.w12, m.out_proj)


def test_weights_that_were_replaced_are_not_answered_with_the_old_layout(layer):
    m, x, answer = layer

    def fresh():
        # as many in-place writes as the layer's own weights have had: their version numbers are equal
        return torch.nn.Parameter(torch.empty_like(m.w12).uniform_(-1, 1))

    for replace in (lambda: setattr(m, "w12", fresh()), lambda: setattr(m, "out_proj", torch.nn.Parameter(torch.empty_like(m.out_proj).uniform_(-1, 1))),
                    lambda: m.load_state_dict({n: v + 1 for n, v in m.state_dict().items()}, assign=True)):
        m.prepare_serving()
        replace()
        assert _same(answer(), m.w12, m.out_proj)


def test_weights_passed_for_one_call_are_the_ones_it_answers_with(layer):
    m, x, answer = layer
    m.prepare_serving()
    other = {n: p.detach().clone().mul_(2) for n, p in m.named_parameters()}
    got = answer(lambda: torch.func.functional_call(m, other, (x,)))
    assert _same(got, other["w12"], other["out_proj"])
    # and afterwards the layout again
    assert answer()[0] is m._serving[0]


@pytest.mark.parametrize("change", ["in place", "memory", "view of other memory"])
def test_weights_that_changed_underneath_raise(layer, change):
    m, x, answer = layer
    m.prepare_serving()
    with torch.no_grad():
        if change == "in place":
            m.out_proj.mul_(2)
        elif change == "memory":
            m.w12.data = m.w12.detach().clone()
        else:
            m.w12.data = torch.zeros((8,) + m.w12.shape[1:], dtype=m.w12.dtype)[4:]
    with pytest.raises(RuntimeError, match="call it again"):
        answer()
    m.prepare_serving()
    assert _same(answer(), m.w12, m.out_proj)


def test_weights_whose_changes_nothing_counts_are_not_laid_out():
    with torch.inference_mode():
        m = bs.Float8BlockwiseMoE(128, 128, 4, 2).eval()
    with pytest.raises(RuntimeError, match="inference"):
        m.prepare_serving()


def test_a_copy_has_no_layout(layer):
    m, x, answer = layer
    m.prepare_serving()
    for other in (copy.deepcopy(m), pickle.loads(pickle.dumps(m))):
        assert m._serving is not None and other._serving is None
        with torch.no_grad():
            other.w12.mul_(3)
        assert _same(answer(lambda: other(x)), other.w12, other.out_proj)
