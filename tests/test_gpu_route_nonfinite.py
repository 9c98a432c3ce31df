"""GPU router: a NaN or +inf logit is chosen first, whatever the choice goes
by, so that it shows in the weights; a masked one is not."""

import numpy as np
import pytest
import torch

import blockwise_scaled_fp8_bs_amd as bs
from gpu_support import need_gpu
from oracle import block

pytestmark = pytest.mark.gpu

INF = float("inf")


def _choice(l, k, bias, kind, G, tg, gb):
    """Indices for one token of float64 logits, by the definition: NaN counts as +inf, and where softmax scores are NaN
    the logits that make them so count as +inf and the others as 0."""
    E = l.size
    far = np.isnan(l) | (l == INF)
    if kind == block.SIGMOID:
        s = np.where(np.isnan(l), INF, block._sigmoid(np.where(far, 0.0, l)))
        s = np.where(l == INF, 1.0, s)
    elif far.any():
        s = np.where(far, INF, 0.0)
    else:
        s = block.scores(l[None], kind)[0]
    masked = np.isneginf(l) | (np.zeros(E, bool) if bias is None else np.isneginf(bias))
    value = np.where(np.isnan(l), INF, l) if bias is None else s + np.where(masked, 0.0, bias)
    worth = s if bias is None else value
    live = [e for e in range(E) if not masked[e]]
    if G > 1:
        n = E // G
        best = {g: sorted((worth[e] for e in live if e // n == g), reverse=True)[:gb] for g in range(G)}
        kept = sorted((g for g in best if best[g]), key=lambda g: (-sum(best[g]), g))[:tg]
        live = [e for e in live if e // n in kept]
    order = sorted(live, key=lambda e: (-value[e], e))[:k]
    return order + [-1] * (k - len(order))


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16], ids=["f32", "bf16"])
@pytest.mark.parametrize("kind", [block.SOFTMAX, block.SIGMOID], ids=["softmax", "sigmoid"])
@pytest.mark.parametrize("E,G,tg,gb", [(64, 1, 1, 1), (64, 8, 2, 1), (64, 8, 2, 2), (256, 8, 4, 2), (40, 8, 3, 2), (24, 3, 1, 1),
                                       (8, 4, 2, 1), (1000, 8, 2, 2)])
def test_logits_that_are_not_finite(E, G, tg, gb, kind, dtype):
    need_gpu()
    T, k = 24, 4
    rng = np.random.default_rng(E + G)
    l = torch.from_numpy(rng.standard_normal((T, E)).astype(np.float32)).to(dtype)
    at = torch.from_numpy(rng.integers(0, E, T))
    rows = torch.arange(T)
    l[rows[:8], at[:8]] = float("nan")
    l[rows[8:16], at[8:16]] = INF
    l[rows[4:16], at[rows[4:16]].add(E // 2) % E] = -INF
    l[2, (at[2] + 1) % E] = INF                     # both in a token
    l[3] = -INF
    l[3, at[3]] = float("nan")                      # nothing else is left
    for biased in (None, "zero", "normal", "masking"):
        bias = None
        if biased:
            bias = torch.from_numpy(rng.standard_normal(E).astype(np.float32) * 0.1 * (biased == "normal"))
        if biased == "masking":
            bias[at[0]] = bias[at[9]] = -INF
        for renorm in (True, False):
            print(f"route not finite E={E} G={G} kind={kind} {dtype} bias={biased} renorm={renorm}", flush=True)
            idx, w = bs.bs_moe_route(l.cuda(), k, bias=None if bias is None else bias.cuda(), score=kind, n_group=G, topk_group=tg,
                                     group_best=gb, renormalize=renorm)
            idx, w = idx.cpu(), w.cpu()
            L = l.double().numpy()
            for t in range(T):
                want = _choice(L[t], k, None if bias is None else bias.double().numpy(), kind, G, tg, gb)
                assert idx[t].tolist() == want, t
                chosen = [e for e in want if e >= 0]
                far = [not np.isfinite(L[t, e]) for e in chosen]
                nan = [np.isnan(L[t, e]) for e in chosen]
                if kind == block.SOFTMAX:
                    bad = [any(far) if renorm else bool((np.isnan(L[t]) | (L[t] == INF)).any())] * len(chosen)
                else:
                    bad = [any(nan)] * len(chosen) if renorm else nan
                assert torch.isnan(w[t, :len(chosen)]).tolist() == [bool(b) for b in bad], t
                assert (w[t, len(chosen):] == 0).all()
