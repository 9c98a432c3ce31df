"""What a plan says about its padding, and which plans the expert layer takes: no GPU."""

import copy
import pickle

import pytest
import torch

import blockwise_scaled_fp8_bs_amd as bs
from blockwise_scaled_fp8_bs_amd import moe


def _plan(T, k, E, M, align=None):
    new = lambda *shape: torch.zeros(shape, dtype=torch.int32)  # noqa: E731
    arrays = new(E), new(E), new(T, k), new(M)
    return bs.MoEPlan(*arrays) if align is None else bs.MoEPlan(*arrays, align=align)


def test_a_plan_is_four_arrays_and_knows_its_alignment():
    p = _plan(4, 2, 3, 384, align=128)
    assert len(p) == 4 and all(isinstance(t, torch.Tensor) for t in p)
    assert p._fields == ("group_end", "counts", "slot_row", "row_slot") and p.align == 128
    for q in (copy.copy(p), copy.deepcopy(p), pickle.loads(pickle.dumps(p))):
        assert isinstance(q, bs.MoEPlan) and q.align == 128
    assert _plan(4, 2, 3, 384).align is None


def _rows(*a):
    return bs.bs_moe_plan_rows(*a)


@pytest.mark.parametrize("T,k,E,M,align", [
    (1000, 2, 8, 3456, 192),                            # a multiple of 128 rows in all, groups of a multiple of 64
    (1000, 2, 8, _rows(1000, 2, 8, 128), 1),            # rows enough for padded groups, groups not padded
    (128, 1, 1, 128, 1),                                # one expert: the last slots may not be routed
    (1000, 2, 8, _rows(1000, 2, 8, 128), None),         # made by hand: nobody knows
], ids=str)
def test_plans_whose_groups_may_end_inside_128_rows_are_refused(T, k, E, M, align):
    assert M % 128 == 0 and M >= _rows(T, k, E, 128)
    if align == 192:
        assert M == _rows(T, k, E, align)
    with pytest.raises(ValueError, match="the plan is for .* padded to 128 rows"):
        moe._check_plan(_plan(T, k, E, M, align), (T, k), E)


@pytest.mark.parametrize("align", [128, 256, 384])
def test_plans_of_whole_128_rows_are_taken(align):
    moe._check_plan(_plan(1000, 2, 8, _rows(1000, 2, 8, align), align), (1000, 2), 8)


@pytest.mark.parametrize("T,k,E,M", [(1000, 2, 8, 2816), (999, 2, 8, 2944), (1000, 3, 8, 4096), (1000, 2, 9, 3200)])
def test_plans_of_other_sizes_are_refused(T, k, E, M):
    with pytest.raises(ValueError, match="the plan is for"):
        moe._check_plan(_plan(T, k, E, M, 128), (1000, 2), 8)
