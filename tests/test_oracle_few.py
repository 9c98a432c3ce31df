"""Pins of the few-token oracle (CPU): MXFP4 against exact rational arithmetic
and the format's table, weights and products against plain loops."""

from fractions import Fraction

import numpy as np
import pytest

from oracle import e4m3, few


def _bf16(v):
    f = np.asarray(v, np.float32).view(np.uint32)
    return (((f + 0x7FFF + ((f >> 16) & 1)) >> 16) << 16).view(np.float32)


def test_e2m1_table():
    assert [few.decode_e2m1(c) for c in range(8)] == [0, 0.5, 1, 1.5, 2, 3, 4, 6]
    assert [few.decode_e2m1(c) for c in range(8, 16)] == [-0.0, -0.5, -1, -1.5, -2, -3, -4, -6]
    assert tuple(few.decode_e2m1(c) for c in range(8)) == few.E2M1


def test_encoder_is_nearest_even_by_rationals():
    vals = [Fraction(few.decode_e2m1(c)) for c in range(8)]
    grid = np.arange(0, 513) / 64.0    # every midpoint among them
    for v in grid:
        a = min(Fraction(float(v)), Fraction(6))
        dist = [abs(a - w) for w in vals]
        near = [c for c in range(8) if dist[c] == min(dist)]
        want = near[0] if len(near) == 1 else [c for c in near if c % 2 == 0][0]
        assert few.encode_e2m1(v) == want and few.encode_e2m1(-v) == want + 8
    y = np.concatenate([grid, -grid])
    assert np.array_equal(few._encode(y), [few.encode_e2m1(v) for v in y])


def test_quantizer_by_rationals():
    rng = np.random.default_rng(0)
    x = _bf16(rng.standard_normal((6, 96)) * np.exp2(rng.integers(-20, 20, (6, 96))))
    x[0, :32] = 0
    x[1, :32] = _bf16(rng.standard_normal(32) * 2.0 ** -130)
    x[2, 3] = 3.38e38
    x = _bf16(x)
    codes, s = few.quant_mx4(x)
    for r in range(6):
        for b in range(3):
            blk = [Fraction(float(v)) for v in x[r, 32 * b:32 * b + 32]]
            amax = max(abs(v) for v in blk)
            e = -127
            if amax:
                e = 200
                while Fraction(2) ** e > amax:
                    e -= 1
                e = min(max(e - 2, -127), 127)
            assert s[r, b] == e + 127
            for v, f, c in zip(x[r, 32 * b:32 * b + 32], blk, codes[r, 32 * b:32 * b + 32]):
                q = f / Fraction(2) ** e
                a = min(abs(q), Fraction(6))
                d = [abs(a - Fraction(w)) for w in few.E2M1]
                near = [i for i in range(8) if d[i] == min(d)]
                want = near[0] if len(near) == 1 else [i for i in near if i % 2 == 0][0]
                assert c == want + (8 if np.signbit(v) else 0)


def test_pack_and_values():
    rng = np.random.default_rng(1)
    codes = rng.integers(0, 16, (4, 64)).astype(np.uint8)
    q = few.pack(codes)
    assert q[1, 2] == codes[1, 4] + 16 * codes[1, 5] and np.array_equal(few.unpack(q), codes)
    s = rng.integers(110, 140, (4, 2)).astype(np.uint8)
    w = few.weights(q, s, "mxfp4")
    q8 = rng.integers(0, 120, (4, 64)).astype(np.uint8)
    w8 = few.weights(q8, s, "mxfp8")
    for n in range(4):
        for k in range(64):
            two = 2.0 ** (int(s[n, k // 32]) - 127)
            assert w[n, k] == few.decode_e2m1(int(codes[n, k])) * two
            assert w8[n, k] == e4m3.decode_code(int(q8[n, k])) * two
    q = rng.integers(0, 120, (256, 384)).astype(np.uint8)
    s = rng.uniform(0.1, 1, (2, 3)).astype(np.float32)
    w = few.weights(q, s, "e4m3")
    for n, k in ((0, 0), (127, 128), (128, 127), (255, 383)):
        assert w[n, k] == e4m3.decode_code(int(q[n, k])) * float(s[n // 128, k // 128])


@pytest.mark.parametrize("residual", [False, True])
def test_experts_by_loops(residual):
    rng = np.random.default_rng(2)
    T, D, H, E, k = 4, 6, 5, 3, 2
    x, w12, wo = rng.standard_normal((T, D)), rng.standard_normal((E, 2 * H, D)), rng.standard_normal((E, D, H))
    idx = np.array([[0, 2], [-1, 1], [1, 1], [-1, 7]])
    w = rng.uniform(0.1, 1, (T, k))
    w[3] = np.nan    # of choices that are none
    r = rng.standard_normal((T, D)) if residual else None
    out, bound = few.moe(x, idx, w, w12, wo, r)
    for t in range(T):
        for d in range(D):
            want = r[t, d] if residual else 0.0
            for j in range(k):
                e = idx[t, j]
                if not 0 <= e < E:
                    continue
                for h in range(H):
                    a, b = sum(w12[e, h] * x[t]), sum(w12[e, H + h] * x[t])
                    want += w[t, j] * wo[e, d, h] * (a / (1 + np.exp(-a)) * b)
            assert abs(out[t, d] - want) < 1e-12 and 0 <= bound[t, d] < 1
