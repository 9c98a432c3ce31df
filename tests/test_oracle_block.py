"""Pins of the MoE-block oracle: closed forms, brute force and differences of
its own forward for every gradient."""

import numpy as np
import pytest

from oracle import block, e4m3


def _logits(T, E, seed, masked=True):
    l = np.random.default_rng(seed).standard_normal((T, E)) * 1.5
    if masked and T > 2:
        l[1] = -np.inf
        l[2, : E // 2] = -np.inf
    return l


@pytest.mark.parametrize("kind", [block.SOFTMAX, block.SIGMOID])
@pytest.mark.parametrize("renorm", [True, False])
def test_route_gradient_equals_differences(kind, renorm):
    T, E, k = 5, 12, 3
    l = _logits(T, E, 3)
    bias = np.random.default_rng(4).standard_normal(E) * 0.05
    kw = dict(kind=kind, renorm=renorm, scale=1.7)
    idx, w = block.route(l, k, bias=bias, n_group=3, topk_group=2, group_best=2, **kw)
    g = np.random.default_rng(5).standard_normal((T, k))
    d = block.route_bwd(l, idx, g, **kw)
    assert np.all(idx[1] == -1) and not w[1].any() and not d[1].any()
    h = 1e-6
    for t in range(T):
        for e in range(E):
            if np.isneginf(l[t, e]):
                assert d[t, e] == 0
                continue
            ends = []
            for s in (h, -h):
                m = l.copy()
                m[t, e] += s
                i2, w2 = block.route(m, k, bias=bias, n_group=3, topk_group=2, group_best=2, **kw)
                assert np.array_equal(i2, idx)
                ends.append((w2 * g).sum())
            assert abs((ends[0] - ends[1]) / (2 * h) - d[t, e]) < 1e-7


def test_route_groups_masks_and_ties():
    l = np.array([[0.0, 3.0, 2.0, 2.0, 9.0, -np.inf, 2.0, 2.0]])
    # without groups: descending, ties to the lowest index
    assert block.route(l, 4)[0].tolist() == [[4, 1, 2, 3]]
    # groups of two; the best pair sum of sigmoids is (2, 2), the best single the one with 9
    assert block.route(l, 2, n_group=4, topk_group=1, kind=block.SIGMOID, group_best=2)[0].tolist() == [[2, 3]]
    assert block.route(l, 2, n_group=4, topk_group=1, group_best=1)[0].tolist() == [[4, -1]]
    # a bias changes the choice and not the weight
    bias = np.zeros(8)
    bias[0] = 10.0
    idx, w = block.route(l, 1, bias=bias, kind=block.SIGMOID, renorm=False)
    assert idx.tolist() == [[0]] and w.tolist() == [[0.5]]


def test_plan_is_a_stable_sort_with_padding():
    rng = np.random.default_rng(0)
    idx = rng.integers(-1, 6, (37, 3)).astype(np.int32)
    M = (37 * 3 + 5 * 7) // 8 * 8 + 8
    ends, counts, slot_row, row_slot = block.plan(idx, 5, 8, M)
    flat = idx.reshape(-1)
    for e in range(5):
        slots = np.flatnonzero(flat == e)
        lo = ends[e - 1] if e else 0
        assert ends[e] % 8 == 0 and ends[e] - lo >= slots.size and counts[e] == slots.size
        assert row_slot[lo:lo + slots.size].tolist() == slots.tolist()      # stable
        assert np.all(row_slot[lo + slots.size:ends[e]] == -1)
    on = slot_row.reshape(-1) >= 0
    assert np.array_equal(on, (flat >= 0) & (flat < 5))
    assert np.array_equal(row_slot[slot_row.reshape(-1)[on]], np.flatnonzero(on))
    assert np.all(row_slot[ends[-1]:] == -1)


def test_gather_combine_and_their_transposes():
    # <combine(y), d> = <y, gather(d)> and the gradient of w is the row products
    rng = np.random.default_rng(1)
    T, k, E, D = 9, 2, 4, 16
    idx = np.stack([rng.permutation(E)[:k] for _ in range(T)]).astype(np.int32)
    idx[3] = -1
    M = 64
    _, _, slot_row, row_slot = block.plan(idx, E, 8, M)
    y, d, w = rng.standard_normal((M, D)), rng.standard_normal((T, D)), rng.random((T, k))
    out, mag = block.combine(y, slot_row, w)
    assert np.allclose((out * d).sum(), (y * block.gather(d, row_slot, k, w)).sum(), rtol=1e-13)
    dw, _ = block.combine_dw(d, y, slot_row)
    assert np.allclose((dw * w).sum(), (out * d).sum(), rtol=1e-13)
    assert not out[3].any() and np.all(mag >= np.abs(out) - 1e-12)


@pytest.mark.parametrize("post,gated,pre", [(1, 1, 1), (1, 0, 1), (0, 1, 1), (0, 0, 1), (1, 1, 0), (None, 0, 1)])
def test_norm_gradients_equal_differences(post, gated, pre):
    rng = np.random.default_rng(2)
    R, D, B, eps, alpha = 6, 8, 3, 1e-3, 0.6
    x = rng.standard_normal((R, D))
    u = rng.standard_normal((R, D)) if post is not None else None
    wq = rng.standard_normal(D) if post else None
    gate = rng.standard_normal((B, D)) if gated else None
    wp = rng.standard_normal(D) if pre else None
    dh, dr = (rng.standard_normal((R, D)) if pre else None), rng.standard_normal((R, D))

    def loss(x, u, wq, gate, wp):
        r = x if u is None else block.resid(x, u, wq, gate, alpha, eps)
        v = (r * dr).sum()
        return v + (block.norm(r, wp, eps) * dh).sum() if pre else v

    args = {"x": x, "u": u, "wq": wq, "gate": gate, "wp": wp}
    r = x if u is None else block.resid(x, u, wq, gate, alpha, eps)
    got = block.norm_bwd(r, wp, dh, dr, u, wq, gate, alpha, eps)
    for name, key in (("x", "dx"), ("u", "du"), ("wq", "dw_post"), ("gate", "dgate"), ("wp", "dw_pre")):
        if args[name] is None:
            assert key not in got
            continue
        for i in np.ndindex(args[name].shape):
            ends = []
            for s in (1e-6, -1e-6):
                m = {n: None if v is None else v.copy() for n, v in args.items()}
                m[name][i] += s
                ends.append(loss(**m))
            assert abs((ends[0] - ends[1]) / 2e-6 - got[key][i]) < 1e-6, (key, i)


def test_swiglu_gradient_equals_differences():
    rng = np.random.default_rng(7)
    a, b, d = (rng.standard_normal(50) * 3 for _ in range(3))
    f = lambda a, b: a / (1 + np.exp(-a)) * b  # noqa: E731
    da, db = block.swiglu_grad(a, b, d)
    h = 1e-6
    assert np.allclose(da, d * (f(a + h, b) - f(a - h, b)) / (2 * h), atol=1e-7)
    assert np.allclose(db, d * (f(a, b + h) - f(a, b - h)) / (2 * h), atol=1e-7)


def test_half_step_is_the_spacing_of_the_codes():
    v = np.sort(e4m3.decode(np.arange(0x7F, dtype=np.uint8)))
    mid = (v[1:] + v[:-1]) / 2
    assert np.allclose(block.half_step(mid), (v[1:] - v[:-1]) / 2, rtol=0)
    q = np.array([[0x38] * 128], dtype=np.uint8)           # 1.0 everywhere
    s = np.array([[2.0 / 448.0]], dtype=np.float32)
    v = np.full((1, 128), 2.0 / 448.0)
    v[0, 0] = 2.0
    q[0, 0] = 0x7E                                          # 448
    ok = block.check_codes(q, s, v, 0.0)
    assert max(ok) <= 1
    q[0, 5] = 0x39                                          # one step off
    assert block.check_codes(q, s, v, 0.0)[1] > 1
    assert block.check_codes(q, s * np.float32(1 + 1e-5), v, 0.0)[0] > 1
    assert block.dequant_rows(q, s)[0, 0] == np.float64(np.float32(448.0) * s[0, 0])
