"""Around the experts' products of an MoE block, CPU oracle.

TEST INFRASTRUCTURE ONLY (see the package docstring).

Plain float64 definitions of the router and its gradient, the sort of the
routed slots by expert, the gather and the weighted combine, the residual
norms and their gradients, and the gated activation's backward from an 8-bit
checkpoint, written from their formulas with loops over tokens where that is
the plainest form.
"""

import numpy as np

from .e4m3 import decode
from .quant import bf16_bits_to_f32

SOFTMAX, SIGMOID = 0, 1


def f64(bits):
    """bf16 bit patterns -> float64."""
    return bf16_bits_to_f32(np.asarray(bits, dtype=np.uint16)).astype(np.float64)


# ---- router ----

def _sigmoid(v):
    e = np.exp(-np.abs(v))
    return np.where(v >= 0, 1.0 / (1.0 + e), e / (1.0 + e))


def scores(logits, kind):
    """Score of every expert; a masked (-inf) one has 0."""
    l = np.asarray(logits, dtype=np.float64)
    if kind == SIGMOID:
        return _sigmoid(l)
    top = l.max(axis=1, keepdims=True)
    e = np.exp(l - np.where(np.isneginf(top), 0.0, top))
    return e / np.where(e.sum(axis=1, keepdims=True) == 0, 1.0, e.sum(axis=1, keepdims=True))


def route(logits, k, bias=None, kind=SOFTMAX, n_group=1, topk_group=1, group_best=1, renorm=True, scale=1.0):
    """(idx [T, k], w [T, k] float64), token by token."""
    l = np.asarray(logits, dtype=np.float64)
    T, E = l.shape
    s = scores(l, kind)
    value = s + np.asarray(bias, dtype=np.float64) if bias is not None else l
    worth = value if bias is not None else s
    idx = np.full((T, k), -1, dtype=np.int32)
    w = np.zeros((T, k))
    size = E // n_group
    for t in range(T):
        live = [e for e in range(E) if not (np.isneginf(l[t, e]) or np.isneginf(value[t, e]))]
        if n_group > 1:
            ranked = []
            for g in range(n_group):
                best = sorted((worth[t, e] for e in live if e // size == g), reverse=True)[:group_best]
                if best:
                    ranked.append((-sum(best), g))
            kept = {g for _, g in sorted(ranked)[:topk_group]}
            live = [e for e in live if e // size in kept]
        order = sorted(live, key=lambda e: (-value[t, e], e))[:k]
        if not order:
            continue
        idx[t, :len(order)] = order
        c = s[t, order]
        if renorm and kind == SOFTMAX:
            c = np.exp(l[t, order] - l[t, order].max())
            c = c / c.sum()
        elif renorm:
            c = c / (c.sum() + 1e-20)
        w[t, :len(order)] = scale * c
    return idx, w


def route_bwd(logits, idx, dw, kind=SOFTMAX, renorm=True, scale=1.0):
    """dlogits [T, E] by the chain rule, from the Jacobian of each token's scores.
    Renormalized softmax weights are the softmax over the chosen logits alone
    (the sum over all experts cancels), so its Jacobian is taken over those:
    the others' gradient is 0, not the rest of a cancellation."""
    l = np.asarray(logits, dtype=np.float64)
    T, E = l.shape
    s = scores(l, kind)
    out = np.zeros((T, E))
    for t in range(T):
        on = idx[t] >= 0
        e, g = idx[t][on], np.asarray(dw, dtype=np.float64)[t][on]
        if e.size == 0:
            continue
        c = s[t, e]
        if renorm and kind == SOFTMAX:
            p = np.exp(l[t, e] - l[t, e].max())
            p = p / p.sum()
            out[t, e] = scale * p * (g - (p * g).sum())
            continue
        if renorm:
            total = c.sum() + 1e-20
            ds = scale * (g / total - (g * c).sum() / total ** 2)
        else:
            ds = scale * g
        if kind == SIGMOID:
            out[t, e] = ds * c * _sigmoid(-l[t, e])
        else:
            full = np.zeros(E)
            full[e] = ds
            out[t] = s[t] * (full - (full * s[t]).sum())
    return out


# ---- dispatch and combine ----

def plan(idx, E, align, M):
    """(group_end, counts, slot_row, row_slot): slots appended to their expert's rows in order."""
    flat = np.asarray(idx).reshape(-1)
    slot_row = np.full(flat.size, -1, dtype=np.int32)
    row_slot = np.full(M, -1, dtype=np.int32)
    ends, counts, at = [], [], 0
    for e in range(E):
        slots = np.flatnonzero(flat == e)
        slot_row[slots] = np.arange(at, at + slots.size)
        row_slot[at:at + slots.size] = slots
        counts.append(slots.size)
        at += -(-slots.size // align) * align
        ends.append(at)
    return (np.array(ends, dtype=np.int32), np.array(counts, dtype=np.int32), slot_row.reshape(np.shape(idx)),
            row_slot)


def gather(x, row_slot, k, w=None):
    """float64 rows of x [T, D] (float64) in expert order, zeros where there is no slot."""
    v = np.zeros((row_slot.size, x.shape[1]))
    for r, slot in enumerate(row_slot):
        if 0 <= slot < x.shape[0] * k:
            v[r] = x[slot // k] * (1.0 if w is None else np.float64(np.asarray(w).reshape(-1)[slot]))
    return v


def combine(y, slot_row, w=None, residual=None):
    """(sum, sum of magnitudes) of residual + w y[slot_row], float64."""
    T, k = slot_row.shape
    out = np.zeros((T, y.shape[1])) if residual is None else residual.copy()
    mag = np.abs(out)
    for t in range(T):
        for j in range(k):
            r = slot_row[t, j]
            if 0 <= r < y.shape[0]:
                term = y[r] * (1.0 if w is None else np.float64(w[t, j]))
                out[t] += term
                mag[t] += np.abs(term)
    return out, mag


def combine_dw(dout, y, slot_row):
    """(dw, sum of magnitudes) of the dot products, float64."""
    T, k = slot_row.shape
    dw, mag = np.zeros((T, k)), np.zeros((T, k))
    for t in range(T):
        for j in range(k):
            r = slot_row[t, j]
            if 0 <= r < y.shape[0]:
                dw[t, j] = dout[t] @ y[r]
                mag[t, j] = np.abs(dout[t]) @ np.abs(y[r])
    return dw, mag


# ---- residual norms ----

def rstd(v, eps):
    return 1.0 / np.sqrt((v * v).mean(axis=1) + eps)


def resid(x, u, w_post, gate, alpha, eps):
    """x + alpha gate N(u) w_post in float64 (before its rounding); gate [B, D] or None, w_post None: no norm."""
    R = x.shape[0]
    g = 1.0 if gate is None else np.repeat(gate, R // gate.shape[0], axis=0)
    n = u if w_post is None else u * rstd(u, eps)[:, None] * w_post
    return x + alpha * g * n


def norm(r, w_pre, eps):
    return r * rstd(r, eps)[:, None] * w_pre


def norm_bwd(r, w_pre, dh, dr, u, w_post, gate, alpha, eps, rstd_u=None, rstd_r=None):
    """dict of float64 gradients; rstd_* replace the recomputed ones."""
    R, D = (dr if r is None else r).shape
    out = {}
    total = np.zeros((R, D)) if dr is None else dr.copy()
    if w_pre is not None:
        s = (rstd(r, eps) if rstd_r is None else rstd_r)[:, None]
        n = r * s
        q = dh * w_pre
        total += s * (q - n * (q * n).mean(axis=1, keepdims=True))
        out["dw_pre"] = (dh * n).sum(axis=0)
    out["dx"] = total
    if u is not None:
        B = 1 if gate is None else gate.shape[0]
        g = np.ones((R, D)) if gate is None else np.repeat(gate, R // B, axis=0)
        dp = alpha * g * total
        if w_post is None:
            out["du"] = dp
            m, wq = u, np.ones(D)
        else:
            s = (rstd(u, eps) if rstd_u is None else rstd_u)[:, None]
            m, wq = u * s, w_post
            dm = dp * w_post
            out["du"] = s * (dm - m * (dm * m).mean(axis=1, keepdims=True))
            out["dw_post"] = (dp * m).sum(axis=0)
        if gate is not None:
            out["dgate"] = (alpha * total * m * wq).reshape(B, R // B, D).sum(axis=1)
    return out


# ---- gated activation from an 8-bit checkpoint ----

def dequant_rows(codes, scales):
    """fl32(code * scale) of 1x128 row codes [R, C] with scales [R, C / 128], as float64."""
    v = decode(codes).astype(np.float32).reshape(codes.shape[0], -1, 128)
    return (v * np.asarray(scales, dtype=np.float32)[:, :, None]).reshape(codes.shape).astype(np.float64)


def swiglu_grad(a, b, dh):
    """(da, db) in float64."""
    s, ns = _sigmoid(a), _sigmoid(-a)
    return dh * b * s * (1.0 + a * ns), dh * (a * s)


# ---- 1x128 quantization of float64 values (not only bf16 ones) ----

def half_step(y):
    """Half the spacing of e4m3 values around |y|."""
    ex = np.floor(np.log2(np.maximum(np.abs(y), 2.0 ** -6)))
    return 0.5 * 2.0 ** (np.minimum(ex, 8.0) - 3.0)


def check_codes(codes, scales, v, value_err):
    """Worst excess of a 1x128 row quantization of v [R, C] (float64), whose
    computed values were off by at most value_err (relative to the block's
    largest): (scale error / its bound, code error / its bound), each <= 1 if
    right.  codes uint8 [R, C], scales float32 [R, C / 128]."""
    R, C = v.shape
    blocks = v.reshape(R, C // 128, 128)
    s = np.maximum(np.abs(blocks).max(axis=2), np.float64(np.float32(1e-12))) / 448.0
    got = np.asarray(scales, dtype=np.float64)
    worst_s = (np.abs(got - s) / (s * (2.0 ** -23 + value_err))).max() if s.size else 0.0
    y = blocks / got[:, :, None]
    err = np.abs(decode(codes).astype(np.float64).reshape(y.shape) - y)
    # the quotient is one fp32 division of a value that is off by value_err of the largest
    bound = half_step(y) + np.abs(y) * 2.0 ** -22 + 448.0 * value_err
    return worst_s, (err / bound).max() if y.size else 0.0
