"""The operators around the expert products of an MoE block, as cases to measure.

Five operators, each in a plain form (elementary torch operations) and through the library's entry points:

* ``route``     scores, balance bias, groups, top-k and weights of a router, and the gradient of its logits;
* ``dispatch``  the sort of the routed tokens by expert, and their rows gathered and quantized 1x128;
* ``combine``   the weighted sum of the experts' outputs on the residual, with its two gradients;
* ``norm``      norm of a block's output, gate, scaled residual and the next norm, with the quantizer and gradients;
* ``ckpt``      the gated activation that keeps [a | b] in 8 bits, and the backward pass that reads them.

e4m3 codes are returned as float8 tensors beside their scales.
"""

import math

import torch

own = False

EPS = 1e-12       # floor of a block's amax (quantizer)
NORM_EPS = 1e-6
TINY = 1e-20      # added to the sum of sigmoid scores


def listed():
    route = dict(op="route", score="sigmoid", bias=True, n_group=8, topk_group=4, group_best=2, renorm=True,
                 scale=2.5, dtype="f32")
    return [
        # one token of a serving step: latency alone
        dict(route, name="route_one_token", T=1, E=256, k=8, grad=False),
        # a training step's router over many experts in groups, balanced by a bias
        dict(route, name="route_train_groups", T=16384, E=256, k=8, grad=True),
        # the benchmark's expert count over its whole token batch, bf16 logits, softmax
        dict(op="route", name="route_train_softmax", T=128000, E=8, k=2, score="softmax", bias=False, n_group=1,
             topk_group=1, group_best=1, renorm=True, scale=1.0, dtype="bf16", grad=True),
        # a small serving batch: rows only, groups of any size
        dict(op="dispatch", name="dispatch_decode", T=24, k=8, E=64, D=4096, align=1, cols=False),
        # 128000 routed rows of 5120 over 8 experts, the benchmark's MoE layer: forward and wgrad operands
        dict(op="dispatch", name="dispatch_train", T=64000, k=2, E=8, D=5120, align=128, cols=True),
        dict(op="combine", name="combine_decode", T=24, k=8, E=64, D=4096, align=1, grad=False),
        # its way back: out, dw and the quantized weighted rows of the gradient
        dict(op="combine", name="combine_train", T=64000, k=2, E=8, D=5120, align=128, grad=True),
        # one token between two blocks of a served model
        dict(op="norm", name="norm_decode", B=1, S=1, D=4096, post=True, gate=True, out="bf16", dtype="bf16",
             grad=False),
        # odd sequences with a gate row of their own (conditioned blocks), bf16 output
        dict(op="norm", name="norm_per_sample_gate", B=5, S=231, D=2048, post=True, gate=True, out="bf16",
             dtype="f32", grad=True),
        # the FFN workload's token batch: next block's quantized operands, and the backward pass
        dict(op="norm", name="norm_train", B=1, S=16384, D=5120, post=True, gate=True, out="both", dtype="f32",
             grad=True),
        # a small layer
        dict(op="ckpt", name="ckpt_small", R=1152, C=640),
        # the FFN up-projection of the benchmark
        dict(op="ckpt", name="ckpt_train", R=16384, C=8192),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["route", "dispatch", "combine", "norm", "ckpt"])
    if op == "route":
        score = rng.choice(["softmax", "sigmoid"])
        n_group = rng.choice([1, 1, 4, 8])
        E = n_group * rng.randint(2, 256 // n_group)
        topk_group = rng.randint(1, n_group)
        k = rng.randint(1, min(8, topk_group * (E // n_group)))
        return dict(op=op, T=_log_int(rng, 1, 16384), E=E, k=k, score=score, bias=rng.random() < 0.5, n_group=n_group,
                    topk_group=topk_group, group_best=rng.choice([1, 2]), renorm=rng.random() < 0.7,
                    scale=rng.choice([1.0, 2.5]), dtype=rng.choice(["f32", "bf16"]), grad=rng.random() < 0.6)
    if op in ("dispatch", "combine"):
        E = rng.choice([4, 8, 16, 64, 129])
        k = rng.randint(1, min(8, E))
        D = 128 * rng.randint(1, 56)
        rows = min(128000, 128000 * 5120 // D)
        case = dict(op=op, T=max(1, _log_int(rng, 1, rows) // k), k=k, E=E, D=D, align=rng.choice([1, 128]))
        case["cols" if op == "dispatch" else "grad"] = case["align"] == 128 and rng.random() < 0.8
        return case
    if op == "norm":
        out = rng.choice(["bf16", "rows", "both"])
        D = 128 * rng.randint(1, 64) if out != "bf16" else 8 * rng.randint(4, 1024)
        R = _log_int(rng, 1, min(16384, 16384 * 5120 // D))
        B = rng.randint(1, min(7, R))
        S = R // B
        if out == "both":
            B, S = 1, (B * S + 127) // 128 * 128
        return dict(op=op, B=B, S=S, D=D, post=rng.random() < 0.7, gate=rng.random() < 0.6, out=out,
                    dtype=rng.choice(["f32", "bf16"]), grad=rng.random() < 0.5)
    C = 128 * rng.randint(1, 64)
    return dict(op=op, R=128 * max(1, _log_int(rng, 1, 16384 * 8192 // C // 128)), C=C)


# ----------------------------------------------------------------------------
# inputs
# ----------------------------------------------------------------------------

def _normal(g, shape, sigma=1.0, dtype=torch.bfloat16):
    t = torch.randn(shape, generator=g, device="cuda", dtype=torch.float32)
    return (t * sigma).to(dtype)


def _dtype(case):
    return torch.float32 if case["dtype"] == "f32" else torch.bfloat16


def _experts(case, g):
    """k distinct experts per token, some experts in more demand than others; every 61st token is not routed."""
    T, E = case["T"], case["E"]
    demand = torch.randn(E, generator=g, device="cuda") * 0.5
    order = (torch.randn((T, E), generator=g, device="cuda") + demand).argsort(1, descending=True)
    idx = order[:, :case["k"]].to(torch.int32).contiguous()
    idx[60::61] = -1
    return idx


def _rows(case):
    """Rows that hold every group padded to `align`, whatever the routing."""
    n, a = case["T"] * case["k"], case["align"]
    return (n + min(case["E"], n) * (a - 1)) // a * a


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    st = {"case": dict(case)}
    op = case["op"]
    if op == "route":
        T, E = case["T"], case["E"]
        st["logits"] = _normal(g, (T, E), 1.0, _dtype(case))
        if T > 1:
            st["logits"][60::61] = -math.inf     # padding tokens of the batch: nothing to choose
        st["bias"] = _normal(g, (E,), 0.05, torch.float32) if case["bias"] else None
        if case["grad"]:
            st["dw"] = _normal(g, (T, case["k"]), 1.0, torch.float32)
    elif op == "dispatch":
        st["idx"] = _experts(case, g)
        st["x"] = _normal(g, (case["T"], case["D"]))
    elif op == "combine":
        T, k, D = case["T"], case["k"], case["D"]
        idx = _experts(case, g)
        st["group_end"], _, st["slot_row"], st["row_slot"] = _plan(idx, case["E"], case["align"], _rows(case))
        st["y"] = _normal(g, (_rows(case), D))
        st["w"] = torch.rand((T, k), generator=g, device="cuda") + 0.05
        st["w"] /= st["w"].sum(1, keepdim=True)
        st["residual"] = _normal(g, (T, D))
        if case["grad"]:
            st["dout"] = _normal(g, (T, D), 0.01)
    elif op == "norm":
        R, D, dt = case["B"] * case["S"], case["D"], _dtype(case)
        st["x"] = _normal(g, (R, D), 2.0)
        st["w_pre"] = (1 + _normal(g, (D,), 0.1, torch.float32)).to(dt)
        st["u"] = st["w_post"] = st["gate"] = None
        if case["post"]:
            st["u"] = _normal(g, (R, D), 0.7)
            st["w_post"] = (1 + _normal(g, (D,), 0.1, torch.float32)).to(dt)
            if case["gate"]:
                st["gate"] = _normal(g, (case["B"], D), 0.5, dt)
        st["alpha"] = 0.5
        if case["grad"]:
            st["dh"], st["dr"] = _normal(g, (R, D), 0.01), _normal(g, (R, D), 0.01)
    else:
        R, C = case["R"], case["C"]
        ab = _normal(g, (R, 2 * C))
        st["a"], st["b"] = ab[:, :C], ab[:, C:]     # the halves of one product's output, as the FFN holds them
        st["dh"] = _normal(g, (R, C), 0.01)
    return st


# ----------------------------------------------------------------------------
# plain forms
# ----------------------------------------------------------------------------

def _scale(amax):
    """fl32(max(amax, EPS) / 448); the divisor is a tensor, since a number's reciprocal would be multiplied by."""
    return amax.clamp_min(EPS) / torch.full_like(amax, 448.0)


def _quant(v):
    """1x128 codes and K-major scales of fp32 v [R, C] along rows."""
    R, C = v.shape
    b = v.view(R, C // 128, 128)
    s = _scale(b.abs().amax(2))
    q = (b / s[..., None]).clamp(-448.0, 448.0).to(torch.float8_e4m3fn)
    return q.view(R, C), s.t().contiguous()


def _quant_cols(v):
    """The same along columns, written transposed: codes [C, R], scales [R / 128, C]."""
    R, C = v.shape
    b = v.view(R // 128, 128, C)
    s = _scale(b.abs().amax(1))
    q = (b / s[:, None]).clamp(-448.0, 448.0).to(torch.float8_e4m3fn)
    return q.view(R, C).t().contiguous(), s


def _bf16_once(d):
    """float64 -> bf16 with one rounding (nearest even), as float64: a value that rounding to fp32 put on a tie
    is moved back to its side of it first."""
    f = d.float()
    tie = (f.view(torch.int32) & 0xFFFF) == 0x8000
    rest = d - f.double()
    up = torch.full_like(f, math.inf)
    f = torch.where(tie & (rest > 0), torch.nextafter(f, up), f)
    f = torch.where(tie & (rest < 0), torch.nextafter(f, -up), f)
    return f.to(torch.bfloat16)


def _scores(l, score):
    if score == "sigmoid":
        return 1.0 / (1.0 + torch.exp(-l))
    e = torch.exp(l - l.amax(1, keepdim=True))
    return e / e.sum(1, keepdim=True)


def _route(st):
    """float64: the choice is between values next to one another."""
    case = st["case"]
    k, E, G = case["k"], case["E"], case["n_group"]
    l = st["logits"].double()
    some = l > -math.inf
    s = torch.where(some, _scores(l, case["score"]), 0.0)
    rank = s + st["bias"].double() if st["bias"] is not None else l
    rank = torch.where(some, rank, -math.inf)
    if G > 1:
        best, at = torch.sort(rank.view(-1, G, E // G), dim=2, descending=True, stable=True)
        n = min(case["group_best"], E // G)
        worth = best if st["bias"] is not None else torch.where(best > -math.inf, s.view(-1, G, E // G).gather(2, at),
                                                                -math.inf)
        there = worth[:, :, :n] > -math.inf
        gs = torch.where(there, worth[:, :, :n], 0.0).sum(2)
        gs = torch.where(there.any(2), gs, -math.inf)
        keep = torch.sort(gs, dim=1, descending=True, stable=True).indices[:, :case["topk_group"]]
        kept = torch.zeros_like(gs, dtype=torch.bool).scatter_(1, keep, True)
        rank = torch.where(kept[:, :, None].expand(-1, -1, E // G).reshape(-1, E), rank, -math.inf)
    val, idx = torch.sort(rank, dim=1, descending=True, stable=True)
    val, idx = val[:, :k], idx[:, :k]
    chosen = val > -math.inf
    sj = torch.where(chosen, s.gather(1, idx), 0.0)
    w = sj
    if case["renorm"]:
        total = sj.sum(1, keepdim=True) + (TINY if case["score"] == "sigmoid" else 0.0)
        w = torch.where(chosen, sj / total, 0.0)
    w = w * case["scale"]
    out = {"idx": torch.where(chosen, idx, -1).to(torch.int32), "w": w.float()}
    if case["grad"]:
        g = torch.where(chosen, st["dw"].double(), 0.0)
        c = case["scale"]
        if case["score"] == "softmax" and case["renorm"]:
            d = w * (g - (w * g).sum(1, keepdim=True) / c)
        elif case["score"] == "softmax":
            d = c * sj * g
        else:
            d = g - (w * g).sum(1, keepdim=True) / c if case["renorm"] else g
            d = c * d * sj * (1.0 - sj)
            if case["renorm"]:
                d = d / total
        dl = torch.zeros_like(l).scatter_add_(1, idx, torch.where(chosen, d, 0.0))
        if case["score"] == "softmax" and not case["renorm"]:
            dl = dl - s * (c * sj * g).sum(1, keepdim=True)
        out["dlogits"] = dl.to(st["logits"].dtype)
    return out


def _plan(idx, E, align, M):
    """group_end [E], counts [E], slot_row [T, k], row_slot [M] of a stable sort of the slots by expert."""
    flat = idx.reshape(-1).long()
    n = flat.numel()
    key = torch.where((flat >= 0) & (flat < E), flat, E)
    skey, order = torch.sort(key, stable=True)
    counts = torch.zeros(E + 1, dtype=torch.int64, device=idx.device).scatter_add_(0, key, torch.ones_like(key))
    first = counts.cumsum(0) - counts
    padded = (counts[:E] + align - 1) // align * align
    ends = padded.cumsum(0)
    start = torch.cat([ends - padded, ends.new_zeros(1)])
    row = start[skey] + torch.arange(n, device=idx.device) - first[skey]
    row = torch.where(skey < E, row, -1)
    slot_row = torch.empty(n, dtype=torch.int32, device=idx.device).scatter_(0, order, row.to(torch.int32))
    row_slot = torch.full((M + 1,), -1, dtype=torch.int32, device=idx.device)
    row_slot.scatter_(0, torch.where(row < 0, M, row), order.to(torch.int32))
    return ends.to(torch.int32), counts[:E].to(torch.int32), slot_row.view(idx.shape), row_slot[:M]


def _gather(x, row_slot, k, w=None):
    slot = row_slot.clamp_min(0).long()
    v = x[slot // k].float()
    if w is not None:
        v = v * w.reshape(-1)[slot][:, None]
    return torch.where((row_slot >= 0)[:, None], v, 0.0)


def _codes(v, cols):
    q, s = _quant(v)
    out = {"q_row": q, "s_row": s}
    if cols:
        out["q_col"], out["s_col"] = _quant_cols(v)
    return out


def _dispatch(st):
    case = st["case"]
    ends, counts, slot_row, row_slot = _plan(st["idx"], case["E"], case["align"], _rows(case))
    v = _gather(st["x"], row_slot, case["k"])
    return dict(_codes(v, case["cols"]), group_end=ends, counts=counts, slot_row=slot_row, row_slot=row_slot)


def _combine(st):
    case = st["case"]
    there = (st["slot_row"] >= 0)
    row = st["slot_row"].clamp_min(0).long()
    w = torch.where(there, st["w"], 0.0)
    out = st["residual"].float()
    dw = []
    for j in range(case["k"]):
        y = st["y"][row[:, j]].float()
        out = out + w[:, j, None] * y
        if case["grad"]:
            dw.append((st["dout"].float() * y).sum(1))
    res = {"out": out.to(torch.bfloat16)}
    if case["grad"]:
        res["dw"] = torch.where(there, torch.stack(dw, 1), 0.0)
        res.update(_codes(_gather(st["dout"], st["row_slot"], case["k"], st["w"]), True))
    return res


def _rstd(t):
    return torch.rsqrt((t.double() ** 2).mean(1, keepdim=True) + NORM_EPS)


def _norm(st):
    """r is a float64 value rounded once; the sums over rows are taken in float64."""
    case = st["case"]
    B, S, D = case["B"], case["S"], case["D"]
    x, u, alpha = st["x"], st["u"], st["alpha"]
    wp = st["w_pre"].float()
    out = {}
    r = x
    if u is not None:
        rstd_u = _rstd(u)
        gate = 1.0 if st["gate"] is None else st["gate"].repeat_interleave(S, 0).double()
        r = _bf16_once(x.double() + alpha * gate * (u.double() * rstd_u * st["w_post"].double()))
        out["r"] = r
    rstd_r = _rstd(r)
    n = r.float() * rstd_r.float()
    h = n * wp
    if case["out"] == "bf16":
        out["h"] = h.to(torch.bfloat16)
    else:
        out.update(_codes(h, case["out"] == "both"))
    if case["grad"]:
        dh = st["dh"].float()
        q = dh * wp
        dr = st["dr"].float() + rstd_r.float() * (q - n * (q * n).mean(1, keepdim=True))
        out["dx"] = dr.to(torch.bfloat16)
        out["dw_pre"] = (dh * n).sum(0, dtype=torch.float64).float()
        if u is not None:
            m = u.float() * rstd_u.float()
            wq = st["w_post"].float()
            gate = 1.0 if st["gate"] is None else st["gate"].float().repeat_interleave(S, 0)
            dp = alpha * gate * dr
            out["dw_post"] = (dp * m).sum(0, dtype=torch.float64).float()
            if st["gate"] is not None:
                out["dgate"] = (alpha * dr * m * wq).view(B, S, D).sum(1, dtype=torch.float64).float()
            dm = dp * wq
            out["du"] = (rstd_u.float() * (dm - m * (dm * m).mean(1, keepdim=True))).to(torch.bfloat16)
    return out


def _ckpt(st):
    """h, da and db are float64 values rounded once to bf16, as the gated activation's kernels define them."""
    a, b = st["a"].double(), st["b"].double()
    out = _codes(_bf16_once(a / (1.0 + torch.exp(-a)) * b).float(), True)
    ck, s_ck = _quant(torch.cat([st["a"], st["b"]], 1).float())
    out["ck"], out["s_ck"] = ck, s_ck
    C = st["case"]["C"]
    kept = (ck.float().view(-1, 2 * C // 128, 128) * s_ck.t()[..., None]).view(-1, 2 * C)
    a, b, dh = kept[:, :C].double(), kept[:, C:].double(), st["dh"].double()
    sg = 1.0 / (1.0 + torch.exp(-a))
    da = _bf16_once(dh * b * sg * (1.0 + a / (1.0 + torch.exp(a))))
    db = _bf16_once(dh * (a * sg))
    out.update({"d" + n: v for n, v in _codes(torch.cat([da, db], 1).float(), True).items()})
    return out


# ----------------------------------------------------------------------------
# the library
# ----------------------------------------------------------------------------

def _empty_codes(bs, R, C, cols, dev):
    q = dict(q_row=torch.empty((R, C), dtype=torch.uint8, device=dev), s_row=bs.empty_scales(C // 128, R, dev))
    if cols:
        q.update(q_col=torch.empty((C, R), dtype=torch.uint8, device=dev), s_col=bs.empty_scales(R // 128, C, dev))
    return q


def _as_values(q, R, C):
    out = {n: t.view(torch.float8_e4m3fn) if t.dtype == torch.uint8 else t for n, t in q.items()}
    out["s_row"] = out["s_row"][:, :R]
    if "s_col" in out:
        out["s_col"] = out["s_col"][:, :C]
    return out


def _run_own(st):
    import blockwise_scaled_fp8_bs_amd as bs
    case, op = st["case"], st["case"]["op"]
    if op == "route":
        score = bs.BS_SCORE_SIGMOID if case["score"] == "sigmoid" else bs.BS_SCORE_SOFTMAX
        idx, w = bs.bs_moe_route(st["logits"], case["k"], bias=st["bias"], score=score, n_group=case["n_group"],
                                 topk_group=case["topk_group"], group_best=case["group_best"],
                                 renormalize=case["renorm"], scale=case["scale"])
        out = {"idx": idx, "w": w}
        if case["grad"]:
            out["dlogits"] = bs.bs_moe_route_bwd(st["logits"], idx, w, st["dw"], score=score,
                                                 renormalize=case["renorm"], scale=case["scale"])
        return out
    if op == "dispatch":
        plan = bs.bs_moe_plan(st["idx"], case["E"], align=case["align"])
        M, D = plan.row_slot.shape[0], case["D"]
        q = _empty_codes(bs, M, D, case["cols"], "cuda")
        bs.bs_moe_gather_quant_1x128(st["x"], plan.row_slot, case["k"], **q)
        return dict(_as_values(q, M, D), group_end=plan.group_end, counts=plan.counts, slot_row=plan.slot_row,
                    row_slot=plan.row_slot)
    if op == "combine":
        out = {"out": bs.bs_moe_combine(st["y"], st["slot_row"], w=st["w"], residual=st["residual"])}
        if case["grad"]:
            M, D = st["y"].shape
            out["dw"] = bs.bs_moe_combine_dw(st["dout"], st["y"], st["slot_row"])
            q = _empty_codes(bs, M, D, True, "cuda")
            bs.bs_moe_gather_quant_1x128(st["dout"], st["row_slot"], case["k"], w=st["w"], **q)
            out.update(_as_values(q, M, D))
        return out
    if op == "norm":
        x, u = st["x"], st["u"]
        (R, D), dev = x.shape, x.device
        f32 = torch.float32
        out = {}
        r = torch.empty_like(x) if u is not None else None
        rstd_u = torch.empty(R, dtype=f32, device=dev) if u is not None else None
        rstd_r = torch.empty(R, dtype=f32, device=dev)
        h, q = None, {}
        if case["out"] == "bf16":
            h = torch.empty_like(x)
        else:
            q = _empty_codes(bs, R, D, case["out"] == "both", dev)
        bs.bs_resid_norm(x, st["w_pre"], u=u, w_post=st["w_post"], gate=st["gate"], alpha=st["alpha"], eps=NORM_EPS,
                         r=r, h=h, rstd_u=rstd_u, rstd_r=rstd_r, **q)
        if u is not None:
            out["r"] = r
        out.update({"h": h} if h is not None else _as_values(q, R, D))
        if case["grad"]:
            g = bs.bs_resid_norm_bwd(x if u is None else r, rstd_r, st["w_pre"], st["dh"], dr=st["dr"], u=u,
                                     rstd_u=rstd_u, w_post=st["w_post"], gate=st["gate"], alpha=st["alpha"])
            out["dx"], out["dw_pre"] = g.dx, g.dw_pre
            if u is not None:
                out["du"], out["dw_post"] = g.du, g.dw_post
                if st["gate"] is not None:
                    out["dgate"] = g.dgate
        return out
    R, C = st["dh"].shape
    dev = st["dh"].device
    q = _empty_codes(bs, R, C, True, dev)
    ck, s_ck = torch.empty((R, 2 * C), dtype=torch.uint8, device=dev), bs.empty_scales(2 * C // 128, R, dev)
    bs.bs_swiglu_quant_1x128_ckpt(st["a"], st["b"], ck, s_ck, **q)
    d = _empty_codes(bs, R, 2 * C, True, dev)
    bs.bs_swiglu_bwd_quant_1x128_ckpt(ck, s_ck, st["dh"], **d)
    out = _as_values(q, R, C)
    out["ck"], out["s_ck"] = ck.view(torch.float8_e4m3fn), s_ck[:, :R]
    out.update({"d" + n: v for n, v in _as_values(d, R, 2 * C).items()})
    return out


def run(state):
    if own:
        return _run_own(state)
    return {"route": _route, "dispatch": _dispatch, "combine": _combine, "norm": _norm, "ckpt": _ckpt}[
        state["case"]["op"]](state)


# ----------------------------------------------------------------------------
# what a pass cannot do without
# ----------------------------------------------------------------------------

def _codes_bytes(R, C, cols):
    return (R * C + R * C // 32) * (2 if cols else 1)


def work(case):
    op = case["op"]
    if op == "route":
        T, E, k = case["T"], case["E"], case["k"]
        e = 4 if case["dtype"] == "f32" else 2
        n, f = T * E * e + 8 * T * k + (4 * E if case["bias"] else 0), 8 * T * E
        if case["grad"]:
            n, f = n + 4 * T * k + T * E * e, f + 4 * T * E
        return {"bytes": n, "flops": f}
    if op == "dispatch":
        n, M, D = case["T"] * case["k"], _rows(case), case["D"]
        return {"bytes": 8 * n + 4 * M + 8 * case["E"] + 2 * case["T"] * D + _codes_bytes(M, D, case["cols"]),
                "flops": 4 * M * D}
    if op == "combine":
        T, k, M, D = case["T"], case["k"], _rows(case), case["D"]
        n, f = 2 * T * k * D + 4 * T * D + 8 * T * k, 2 * T * k * D
        if case["grad"]:
            n, f = n + 2 * T * D + 4 * T * k + 4 * M + _codes_bytes(M, D, True), f + 6 * T * k * D
        return {"bytes": n, "flops": f}
    if op == "norm":
        R, D = case["B"] * case["S"], case["D"]
        n = 2 * R * D * (3 if case["post"] else 1)
        n += 2 * R * D if case["out"] == "bf16" else _codes_bytes(R, D, case["out"] == "both")
        f = 8 * R * D
        if case["grad"]:   # dh and dr in, dx out; du out
            n, f = n + 2 * R * D * (4 if case["post"] else 3), f + 20 * R * D
        return {"bytes": n, "flops": f}
    R, C = case["R"], case["C"]
    # in: a, b, dh; out: codes of h, of [a | b] and of [da | db]
    return {"bytes": 6 * R * C + _codes_bytes(R, C, True) + _codes_bytes(R, 2 * C, False) + _codes_bytes(R, 2 * C, True),
            "flops": 30 * R * C}


# ----------------------------------------------------------------------------
# from the definitions, in 64 bits: quotients of codes before their rounding
# ----------------------------------------------------------------------------

def _exact_quot(v, dim):
    """Quotients and scales of 128-blocks of v along dim (1: rows, 0: columns, transposed)."""
    t = v if dim == 1 else v.t()
    n, c = t.shape
    blocks = t.reshape(n, c // 128, 128)
    s = torch.clamp(blocks.abs().max(2).values, min=EPS) / 448.0
    return (blocks / s.unsqueeze(2)).reshape(n, c), s.t()


def _exact_codes(v, cols):
    q, s = _exact_quot(v, 1)
    out = {"q_row": q, "s_row": s}
    if cols:
        out["q_col"], out["s_col"] = _exact_quot(v, 0)
    return out


def _round_bf16(d):
    """Nearest bf16 of float64 values, ties to even: on the integers of a scaled significand."""
    mant, ex = torch.frexp(d)
    ex = torch.clamp(ex, min=-125)             # below: bf16's subnormals, spaced as its smallest normals
    mant = torch.ldexp(d, -ex)
    return torch.ldexp(torch.round(mant * 256.0), ex - 8)


def _exact_route(case, st):
    logits = st["logits"].double().requires_grad_(True)
    T, E = logits.shape
    k, G = case["k"], case["n_group"]
    live = ~torch.isinf(logits.detach())
    if case["score"] == "sigmoid":
        prob = torch.sigmoid(logits)
    else:
        prob = torch.softmax(torch.where(live, logits, -1e300), dim=-1)
    p = prob.detach()
    key = (p + st["bias"].double()[None]) if case["bias"] else logits.detach().clone()
    worth = key if case["bias"] else p
    key = key.masked_fill(~live, -math.inf)
    if G > 1:
        gk, gw = key.reshape(T, G, -1).clone(), worth.reshape(T, G, -1)
        gsum = torch.zeros(T, G, dtype=torch.float64, device=key.device)
        alive = live.reshape(T, G, -1).any(2)
        for _ in range(min(case["group_best"], E // G)):
            top, at = gk.max(2, keepdim=True)
            gsum += torch.where(top > -math.inf, gw.gather(2, at), 0.0).squeeze(2)
            gk.scatter_(2, at, -math.inf)
        gsum = gsum.masked_fill(~alive, -math.inf)
        keep = torch.zeros(T, G, dtype=torch.bool, device=key.device)
        for _ in range(case["topk_group"]):
            best = gsum.max(1, keepdim=True).values
            at = (gsum == best).to(torch.uint8).argmax(1, keepdim=True)
            keep.scatter_(1, at, True)
            gsum = gsum.masked_fill(keep, -math.inf) if case["topk_group"] < G else gsum.scatter(1, at, -math.inf)
        key = key.reshape(T, G, -1).masked_fill(~keep[..., None], -math.inf).reshape(T, E)
    picks = []
    for _ in range(k):
        best = key.max(1, keepdim=True).values
        at = (key == best).to(torch.uint8).argmax(1, keepdim=True)
        picks.append(torch.where(best > -math.inf, at, -1))
        key = key.scatter(1, at, -math.inf)
    idx = torch.cat(picks, 1)
    got = idx >= 0
    sj = torch.where(got, prob.gather(1, idx.clamp(min=0)), 0.0)
    if case["renorm"]:
        den = sj.sum(1, keepdim=True)
        den = den + TINY if case["score"] == "sigmoid" else torch.where(den > 0, den, 1.0)
        w = case["scale"] * sj / den
    else:
        w = case["scale"] * sj
    out = {"idx": idx.to(torch.int32), "w": w.detach()}
    if case["grad"]:
        (dl,) = torch.autograd.grad((w * torch.where(got, st["dw"].double(), 0.0)).sum(), logits)
        out["dlogits"] = torch.where(live, dl, 0.0)
    return out


def _exact_norm(case, st):
    B, S, D = case["B"], case["S"], case["D"]
    leaf = lambda t: None if t is None else t.double().requires_grad_(True)  # noqa: E731
    rms = lambda t: t / torch.sqrt(t.square().mean(-1, keepdim=True) + NORM_EPS)  # noqa: E731
    u, wq, gate, wp = leaf(st["u"]), leaf(st["w_post"]), leaf(st["gate"]), leaf(st["w_pre"])
    out = {}
    x = st["x"].double()
    if u is not None:
        add = st["alpha"] * rms(u) * wq
        if gate is not None:
            add = (add.view(B, S, D) * gate[:, None, :]).reshape(B * S, D)
        r = x + add.detach()
        out["r"] = r
        r = _round_bf16(r)
    else:
        add, r = None, x
    r = r.clone().requires_grad_(True)
    h = rms(r) * wp
    if case["out"] == "bf16":
        out["h"] = h.detach()
    else:
        out.update(_exact_codes(h.detach(), case["out"] == "both"))
    if case["grad"]:
        dr, dwp = torch.autograd.grad(h, [r, wp], st["dh"].double())
        dr = dr + st["dr"].double()
        out["dx"], out["dw_pre"] = dr, dwp
        if u is not None:
            wanted = [t for t in (u, wq, gate) if t is not None]
            grads = torch.autograd.grad(add, wanted, dr)
            out.update(zip(["du", "dw_post", "dgate"], grads))
    return out


def _exact_ckpt(case, st):
    C = case["C"]
    a, b, dh = st["a"].double(), st["b"].double(), st["dh"].double()
    out = _exact_codes(_round_bf16(a * torch.sigmoid(a) * b), True)
    both = torch.cat([a, b], 1)
    out["ck"], out["s_ck"] = _exact_quot(both, 1)
    s32 = out["s_ck"].t().float().double().repeat_interleave(128, 1)      # scales are held in fp32
    kept = ((both / s32).float().to(torch.float8_e4m3fn).double() * s32).float().double()
    a, b = kept[:, :C], kept[:, C:]
    sg = torch.sigmoid(a)
    da = dh * b * (sg + a * sg * torch.sigmoid(-a))
    grads = torch.cat([_round_bf16(da), _round_bf16(dh * a * sg)], 1)
    out.update({"d" + n: v for n, v in _exact_codes(grads, True).items()})
    return out


def exact(case, seed):
    st = prepare(case, seed)
    op = case["op"]
    if op == "route":
        return _exact_route(case, st)
    if op == "norm":
        return _exact_norm(case, st)
    if op == "ckpt":
        return _exact_ckpt(case, st)
    k = case["k"]
    if op == "dispatch":
        flat = st["idx"].reshape(-1).long()
        M, E, a = _rows(case), case["E"], case["align"]
        picked = torch.full((M,), -1, dtype=torch.int64, device=flat.device)
        end, ends, counts = 0, [], []
        for e in range(E):
            slots = (flat == e).nonzero().reshape(-1)
            picked[end:end + slots.numel()] = slots
            counts.append(slots.numel())
            end += (slots.numel() + a - 1) // a * a
            ends.append(end)
        rows = st["x"].double()[(picked.clamp(min=0)) // k] * (picked >= 0).double()[:, None]
        back = torch.full_like(flat, -1)
        back[picked[picked >= 0]] = (picked >= 0).nonzero().reshape(-1)
        ints = lambda v: torch.tensor(v, dtype=torch.int32, device=flat.device)  # noqa: E731
        return dict(_exact_codes(rows, case["cols"]), group_end=ints(ends), counts=ints(counts),
                    slot_row=back.to(torch.int32).view(-1, k), row_slot=picked.to(torch.int32))
    row = st["slot_row"].long()
    w = st["w"].double()
    total = st["residual"].double()
    dws = []
    for j in range(k):
        y = st["y"].double()[row[:, j].clamp(min=0)] * (row[:, j] >= 0).double()[:, None]
        total = total + y * w[:, j, None]
        if case["grad"]:
            dws.append(torch.linalg.vecdot(st["dout"].double(), y))
    out = {"out": total}
    if case["grad"]:
        out["dw"] = torch.stack(dws, 1)
        slot = st["row_slot"].long()
        v = st["dout"].double()[slot.clamp(min=0) // k] * w.reshape(-1)[slot.clamp(min=0), None]
        out.update(_exact_codes(v * (slot >= 0).double()[:, None], True))
    return out
