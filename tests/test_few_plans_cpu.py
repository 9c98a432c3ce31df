"""What the few-token calls would launch, and the workspace for it: no GPU."""

import random

import pytest

import blockwise_scaled_fp8_bs_amd as bs
from blockwise_scaled_fp8_bs_amd import _lib

KINDS = (bs.BS_WEIGHT_E4M3_128X128, bs.BS_WEIGHT_MXFP8, bs.BS_WEIGHT_MXFP4)


def _sizes(rng, kind):
    step = 128 if kind == bs.BS_WEIGHT_E4M3_128X128 else 32
    E = min(1024, int(2 ** rng.uniform(0, 10.3)))
    size = lambda top: step * max(1, int(2 ** rng.uniform(0, top)) // step)  # noqa: E731
    return int(2 ** rng.uniform(0, 9)), rng.choice([size(15), size(15), 4096]), size(15), E, rng.randint(1, min(E, 32))


def test_the_workspace_holds_what_a_launch_leaves_in_it():
    rng = random.Random(1)
    shared = set()
    for _ in range(4000):
        kind = rng.choice(KINDS)
        T, D, H, E, k = _sizes(rng, kind)
        plan = bs.bs_diag_moe_few_plan(kind, T, D, H, E, k)
        # h of every slot, and the sums of workgroups that share columns
        need = T * k * H * 2 + (plan["splits"] * T * D * 4 if plan["splits"] > 1 else 0)
        assert _lib.load().bs_moe_few_workspace_bytes(T, D, H, E, k) >= need
        shared.add((plan["tokens"], plan["out_tiles"], plan["splits"] > 1))
        # the items' first rows and experts are kept in 16 bits each
        assert plan["items"] <= 2 ** 15 and min(T, 64) * k < 2 ** 16
    assert {s for s in shared if s[2]} == {(16, 1, True), (16, 2, True), (32, 1, True), (32, 2, True)}


@pytest.mark.parametrize("fn,sizes", [(bs.bs_diag_few_mm_plan, (3, 1, 64, 64)), (bs.bs_diag_few_mm_plan, (1, 0, 64, 64)),
                                      (bs.bs_diag_few_mm_plan, (1, 1, 0, 64)), (bs.bs_diag_few_mm_plan, (1, 1, 64, 0)),
                                      (bs.bs_diag_moe_few_plan, (-1, 1, 64, 64, 4, 2)), (bs.bs_diag_moe_few_plan, (1, 0, 64, 64, 4, 2)),
                                      (bs.bs_diag_moe_few_plan, (1, 1, 64, 64, 4, 5)), (bs.bs_diag_moe_few_plan, (1, 1, 64, 0, 4, 2))])
def test_sizes_without_a_plan(fn, sizes):
    with pytest.raises(bs.BsError):
        fn(*sizes)


def test_sizes_past_a_launch_s_threads():
    """2^32 along an axis: the next size is refused, not left to the launch to fail."""
    lib, P, SHAPE = _lib.load(), 0x10000, 2
    quant = lambda R, C: lib.bs_mx4_quant_1x32(P, R, C, C, P, max(C // 2, 16), P, R + 15 & ~15, None, 0, None)  # noqa: E731
    for R, C in ((2 ** 29 - 255, 32), (2 ** 29 - 255, 256), (2 ** 28 - 127, 288)):
        assert quant(R, C) == SHAPE and "one launch" in lib.bs_last_error().decode()
    for T, N in ((1, 2 ** 27 - 127), (8, 2 ** 27 - 127), (9, 2 ** 28 - 127), (16, 2 ** 28 - 127)):
        N = (N + 127) // 128 * 128
        for n, refused in ((N - 128, False), (N, True)):
            plan = bs.bs_diag_few_mm_plan(bs.BS_WEIGHT_E4M3_128X128, T, n, 128)
            assert (plan["workgroups"] * plan["threads"] >= 2 ** 32) == refused
        call = lib.bs_few_mm(bs.BS_WEIGHT_E4M3_128X128, T, N, 128, P, 128, P, 128, P, N // 128, None, 0, P, N, 0, None)
        assert call == SHAPE and "one launch" in lib.bs_last_error().decode()


@pytest.mark.parametrize("kind", KINDS)
def test_products_take_one_round_of_the_cus_where_they_can(kind):
    """Beside 17 rows and more, a workgroup fills a CU: two tiles of columns where one takes a second round of the 256."""
    for T, one, two in ((17, 4096, 4224), (32, 4096, 5120), (64, 4096, 6144), (64, 1024, 8064), (65, 2048, 2176), (128, 2048, 4096),
                        (256, 1024, 1152)):
        plan = bs.bs_diag_few_mm_plan(kind, T, one, 1024)
        chunks = -(-T // plan["rows"])
        assert plan["tiles"] == 1 and plan["workgroups"] * chunks <= 256
        plan = bs.bs_diag_few_mm_plan(kind, T, two, 1024)
        assert plan["tiles"] == 2 and (plan["workgroups"] * chunks <= 256 or two > 8192 // chunks)


def test_workspace_of_both_parts():
    """Room for a second part of the activations up to 8 tokens; the least is what it was."""
    lib = _lib.load()
    for T, D, H, E, k in ((1, 96, 64, 4, 2), (3, 96, 64, 4, 2), (8, 128, 8192, 16, 8)):
        assert lib.bs_moe_few_full_workspace_bytes(T, D, H, E, k) == lib.bs_moe_few_workspace_bytes(T, D, H, E, k) + T * k * H * 2
    for T, D, H, E, k in ((9, 96, 64, 4, 2), (64, 128, 8192, 16, 8), (0, 96, 64, 4, 2), (3, 96, 64, 4, 33), (-1, 96, 64, 4, 2)):
        assert lib.bs_moe_few_full_workspace_bytes(T, D, H, E, k) == lib.bs_moe_few_workspace_bytes(T, D, H, E, k)
