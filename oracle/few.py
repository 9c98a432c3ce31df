"""Serving few tokens from quantized weights, CPU oracle.

TEST INFRASTRUCTURE ONLY (see the package docstring).

* the MXFP4 quantizer: OCP Microscaling v1.0 with E2M1 elements (1 sign, 2
  exponent, 1 mantissa bit, bias 1: 0, 0.5, 1, 1.5, 2, 3, 4, 6), blocks of 32
  along a row, scale 2^e, e = floor(log2 amax) - 2 clamped to [-127, 127]
  (2: the exponent of 6), elements rounded to the nearest value, ties to the
  even code, saturating;
* weights of the three formats as float64;
* the product of few rows with them, and the gated experts of routed tokens,
  in float64, each with a bound on what a kernel with fp32 sums may be off by.

Bounds.  A rounding to bf16 is off by at most 2^-8 of the value (half a step,
eps / 2).  A sum of n fp32 terms of magnitudes that add up to S is off by at
most n 2^-23 S, in any order and also where an addition rounds by a whole step
(the matrix cores' adders); the terms are products of bf16 numbers, exact in
fp32.  A block's scale (128x128) multiplies the block's sum by one fused
operation more.
"""

import numpy as np

from . import e4m3

E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)
MX_BLOCK = 32
HALF_BF16 = 2.0 ** -8
STEP_F32 = 2.0 ** -23


def decode_e2m1(code):
    """Value of one 4-bit code, from the bit fields."""
    sign, ex, frac = code >> 3, (code >> 1) & 3, code & 1
    v = frac * 0.5 if ex == 0 else (1 + frac * 0.5) * 2.0 ** (ex - 1)
    return -v if sign else v


def encode_e2m1(y):
    """Code of one finite number: the nearest value, ties to the even code."""
    sign = 8 if np.signbit(y) else 0
    a = min(abs(float(y)), 6.0)
    best = min(range(8), key=lambda c: (abs(decode_e2m1(c) - a), c & 1))
    return sign | best


def _encode(y):
    """Vectorized form: counts the midpoints below, a tie counted where the upper code is the even one."""
    a = np.abs(y)
    c = np.zeros(y.shape, np.uint8)
    for lo in range(7):
        mid = (E2M1[lo] + E2M1[lo + 1]) / 2
        c += (a > mid) | ((a == mid) & ((lo + 1) % 2 == 0))
    return c | np.where(np.signbit(y), 8, 0).astype(np.uint8)


def quant_mx4(x):
    """x [R, C] (float array of bf16 values) -> codes [R, C] (unpacked), bytes [R, C/32]."""
    x = np.asarray(x, np.float64)
    R, C = x.shape
    b = x.reshape(R, C // MX_BLOCK, MX_BLOCK)
    amax = np.abs(b).max(2)
    e = np.frexp(amax)[1] - 1 - 2
    e = np.clip(np.where(amax == 0, -127, e), -127, 127)
    return _encode(np.ldexp(b, -e[..., None])).reshape(R, C), (e + 127).astype(np.uint8)


def pack(codes):
    """Codes [R, C] -> bytes [R, C/2], even columns in the low bits."""
    return codes[:, 0::2] | (codes[:, 1::2] << 4)


def unpack(q):
    out = np.empty((q.shape[0], 2 * q.shape[1]), np.uint8)
    out[:, 0::2], out[:, 1::2] = q & 15, q >> 4
    return out


def weights(q, s, kind):
    """float64 [N, K] of codes q and logical scales: "e4m3" s [N/128, K/128],
    "mxfp8" and "mxfp4" (packed codes) bytes [N, K/32]."""
    if kind == "e4m3":
        return e4m3.decode(q) * np.repeat(np.repeat(np.asarray(s, np.float64), 128, 0), 128, 1)
    v = e4m3.decode(q) if kind == "mxfp8" else np.array([decode_e2m1(c) for c in range(16)])[unpack(q)]
    return v * np.repeat(np.exp2(np.asarray(s, np.float64) - 127), MX_BLOCK, 1)


def few_mm(x, w, residual=None, bf16=True):
    """(out, bound): residual + x w^T in float64."""
    ref, mag = x @ w.T, np.abs(x) @ np.abs(w).T
    if residual is not None:
        ref, mag = ref + residual, mag + np.abs(residual)
    bound = (w.shape[1] + 64) * STEP_F32 * mag
    return ref, (bound + HALF_BF16 * (np.abs(ref) + bound) if bf16 else bound)


def moe(x, idx, w, w12, wo, residual=None, parts=1):
    """(out, bound) of residual + sum_j w_j wo_e (silu(a) b), [a | b] = w12_e x:
    x [T, D], idx and w [T, k], w12 [E][2H, D], wo [E][D, H], all float64.

    With da, db the bounds of a and b: |silu'| <= 1.1, so silu(a) b is off by at
    most |silu(a)| db + 1.1 da (|b| + db), times the weight, and 2^-20 of itself
    for the arithmetic of the formula; h is rounded once to bf16, or kept in two
    parts: what the first rounding left out, at most 2^-8 of h, is rounded to bf16
    in turn (off by at most 2^-8 of that, or half a step of bf16's smallest
    numbers, 2^-134), and the sums have twice the terms.
    """
    T, D = x.shape
    out = np.zeros((T, D)) if residual is None else np.array(residual, np.float64)
    mag = np.abs(out)
    err = np.zeros((T, D))
    terms = 1
    for t in range(T):
        for e in sorted(set(int(v) for v in idx[t] if 0 <= v < len(w12))):
            weight = sum(w[t, j] for j in range(idx.shape[1]) if idx[t, j] == e)
            H = wo[e].shape[1]
            ab, dab = few_mm(x[t:t + 1], w12[e], bf16=False)
            a, b, da, db = ab[0, :H], ab[0, H:], dab[0, :H], dab[0, H:]
            with np.errstate(over="ignore"):
                g = a / (1 + np.exp(-a))
            h = weight * g * b
            dh = abs(weight) * (np.abs(g) * db + 1.1 * da * (np.abs(b) + db)) + 2.0 ** -20 * np.abs(h)
            dh = dh + HALF_BF16 ** parts * (np.abs(h) + dh) + (2.0 ** -134 if parts > 1 else 0.0)
            out[t] += wo[e] @ h
            mag[t] += np.abs(wo[e]) @ (np.abs(h) + dh)
            err[t] += np.abs(wo[e]) @ dh
            terms += parts * H
    err = err + (terms + 64) * STEP_F32 * mag
    return out, err + HALF_BF16 * (np.abs(out) + err)
