"""GPU router where fp32 alone would answer wrongly: ties hidden behind ties."""

import numpy as np
import pytest
import torch

import blockwise_scaled_fp8_bs_amd as bs
from gpu_support import need_gpu
from oracle import block

pytestmark = pytest.mark.gpu


def _f64(t):
    return t.double().numpy()


@pytest.mark.parametrize("E,G,tg", [(64, 4, 2), (256, 8, 2), (24, 8, 4), (40, 8, 3)])
def test_route_hidden_tie_after_the_groups_are_chosen(E, G, tg):
    """As test_route_tie_at_the_last_place_next_to_a_better_expert, with groups
    dropped: groups of whole lanes (64, 256) and of other sizes."""
    need_gpu()
    l = torch.full((40, E), -4.0)
    l[:, :3] = torch.tensor([4.0, 3.0, 2.0])
    l[:, 5] = l[:, 9] = 0.0
    l[:, E - 1] = 0.25
    assert len({e // (E // G) for e in (0, 1, 2, 5, 9, E - 1)}) == tg < G
    bias = torch.zeros(E)
    bias[E - 1] = 0.5 - 1.0 / (1.0 + float(np.exp(-0.25)))  # a score of 0.5, plus its rounding
    seen = set()
    for step in range(-2, 3):
        b = bias.clone()
        for _ in range(abs(step)):
            b[E - 1] = torch.nextafter(b[E - 1], torch.tensor(float(np.sign(step))))
        kw = dict(n_group=G, topk_group=tg, group_best=1)
        print(f"route hidden tie in groups E={E} G={G} step={step}", flush=True)
        want_idx, want_w = block.route(_f64(l), 4, bias=_f64(b), kind=block.SIGMOID, **kw)
        idx, w = bs.bs_moe_route(l.cuda(), 4, bias=b.cuda(), score=bs.BS_SCORE_SIGMOID, **kw)
        assert np.array_equal(idx.cpu().numpy(), want_idx)
        # fp32 exponentials, k additions and a quotient
        assert (np.abs(w.cpu().double().numpy() - want_w) <= want_w * 2.0 ** -19).all()
        seen.add(int(want_idx[0, 3]))
    assert seen == {5, E - 1}  # both sides of the tie were met
