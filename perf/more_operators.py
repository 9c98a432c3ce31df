"""Serving few tokens from 8- and 4-bit weights, as cases to measure.

Three operators, each in a plain form (elementary torch operations) and through the library's entry points:

* ``quant``  weights to MXFP4: e2m1 codes, two a byte, an E8M0 byte for each 32 along the contraction, and the bf16
             values that they stand for;
* ``mm``     the product of few bf16 rows with weights in blockwise FP8 (128x128), MXFP8 or MXFP4, on a residual;
* ``moe``    the gated experts of few routed tokens and their weighted sum on the residual, weights in the same
             formats; one expert without routing is the gated FFN.

Weights are made and laid out by ``prepare``: a server does so once.
"""

import math

import torch

own = False

EPS = 1e-12                                             # floor of a block's amax (128x128)
E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)         # magnitudes by code


def listed():
    return [
        # a small layer's weights, odd numbers of rows and blocks
        dict(op="quant", name="quant_small", R=77, C=672),
        # the benchmark's expert weights, 8 x 8192 x 5120, laid out for a server
        dict(op="quant", name="quant_experts", R=65536, C=5120),
        # one token through the benchmark's dense layer, on the residual stream
        dict(op="mm", name="mm_one_token_fp8", T=1, N=4096, K=4096, kind="fp8", residual=True, out="bf16"),
        # one token through the FFN up-projection in 4 bits
        dict(op="mm", name="mm_one_token_fp4", T=1, N=8192, K=5120, kind="mxfp4", residual=False, out="bf16"),
        # a small head with fp32 logits: odd columns, a contraction that ends inside a block of tiles
        dict(op="mm", name="mm_odd_fp4", T=3, N=1001, K=4128, kind="mxfp4", residual=False, out="f32"),
        # a few drafted tokens through the FFN down-projection
        dict(op="mm", name="mm_draft_mxfp8", T=7, N=2048, K=7168, kind="mxfp8", residual=True, out="bf16"),
        # a full decoding batch
        dict(op="mm", name="mm_batch_fp4", T=64, N=8192, K=5120, kind="mxfp4", residual=False, out="bf16"),
        # one token through the example's MoE block: latency
        dict(op="moe", name="moe_one_token", T=1, D=2048, H=1024, E=16, k=4, kind="fp8", residual=True),
        # one token, experts of the benchmark's size, in 4 bits
        dict(op="moe", name="moe_one_token_fp4", T=1, D=5120, H=4096, E=8, k=2, kind="mxfp4", residual=True),
        # drafted tokens through the gated FFN of the benchmark: one expert, nothing to route
        dict(op="moe", name="moe_gated_ffn", T=5, D=5120, H=8192, E=1, k=1, kind="mxfp8", residual=True),
        # a decoding batch over many experts
        dict(op="moe", name="moe_decode", T=24, D=4096, H=2048, E=64, k=8, kind="fp8", residual=True),
        # the largest batch, every expert in use
        dict(op="moe", name="moe_batch_fp4", T=64, D=4096, H=2048, E=64, k=8, kind="mxfp4", residual=False),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["quant", "mm", "moe", "moe"])
    if op == "quant":
        C = 32 * _log_int(rng, 1, 512)
        return dict(op=op, R=_log_int(rng, 1, min(65536, 65536 * 5120 // C)), C=C)
    kind = rng.choice(["fp8", "mxfp8", "mxfp4"])
    step = 128 if kind == "fp8" else 32
    T = _log_int(rng, 1, 64)
    if op == "mm":
        K = step * _log_int(rng, 1, 8192 // step)
        N = 128 * rng.randint(1, 64) if kind == "fp8" else _log_int(rng, 16, 8192)
        N = min(N, 8192 * 5120 // K // 128 * 128)
        return dict(op=op, T=T, N=N, K=K, kind=kind, residual=rng.random() < 0.5, out=rng.choice(["bf16", "f32"]))
    E = rng.choice([1, 4, 8, 16, 64, 129])
    k = rng.randint(1, min(8, E))
    D = step * _log_int(rng, 1, 5120 // step)
    most = 64 * 4096 * 2048 // (E * D) // 2
    H = step * _log_int(rng, 1, max(1, min(8192, most) // step))
    return dict(op=op, T=T, D=D, H=H, E=E, k=k, kind=kind, residual=rng.random() < 0.7)


# ----------------------------------------------------------------------------
# the formats, in torch operations
# ----------------------------------------------------------------------------

def _block_exponent(x, emax):
    """x fp32 [R, C] -> e int32 [R, C / 32] = floor(log2 amax) - emax within [-127, 127], -127 for a zero block."""
    amax = x.view(x.shape[0], -1, 32).abs().amax(2)
    e = torch.frexp(amax).exponent - 1 - emax
    return torch.where(amax > 0, e, -127).clamp(-127, 127)


def _mx_scaled(x, e):
    """x / 2^e by blocks, exact (float64)."""
    v = x.view(x.shape[0], -1, 32).double()
    return torch.ldexp(v, -e[:, :, None]).view(x.shape)


def _scale_rows(e):
    """K-major scale bytes [C / 32, R], the row stride a multiple of 16."""
    R, n = e.shape
    s = torch.zeros((n, (R + 15) // 16 * 16), dtype=torch.uint8, device=e.device)
    s[:, :R] = (e + 127).t().to(torch.uint8)
    return s


def _quant_mx4(x):
    """(codes [R, C / 2], exponents [R, C / 32]) of fp32 x: nearest e2m1, ties to the even code, saturating."""
    e = _block_exponent(x, 2)
    v = _mx_scaled(x, e)
    a = v.abs()
    c = (a > 0.25).to(torch.uint8)
    for tie, up in ((0.75, True), (1.25, False), (1.75, True), (2.5, False), (3.5, True), (5.0, False)):
        c += (a >= tie) if up else (a > tie)
    c += 8 * torch.signbit(v)
    return c[:, 0::2] + 16 * c[:, 1::2], e


def _mx4_values(q):
    """e2m1 values fp32 [R, C] of packed codes [R, C / 2]."""
    lut = torch.tensor(E2M1 + tuple(-v for v in E2M1), dtype=torch.float32, device=q.device)
    return lut[torch.stack([q & 15, q >> 4], 2).view(q.shape[0], -1).int()]


def _times_blocks(v, s):
    """fp32 v [R, C] times 2^(byte - 127) of K-major bytes s [C / 32, >= R]."""
    R = v.shape[0]
    two = torch.ldexp(torch.ones((), dtype=torch.float32, device=v.device), s[:, :R].t().int() - 127)
    return (v.view(R, -1, 32) * two[:, :, None]).view(v.shape)


def _weight(W, kind):
    """Codes and scales of weights W fp32 [N, K] as a server lays them out."""
    N, K = W.shape
    if kind == "fp8":
        b = W.view(N // 128, 128, K // 128, 128)
        s = b.abs().amax((1, 3)).clamp_min(EPS) / 448.0
        q = (b / s[:, None, :, None]).clamp(-448.0, 448.0).to(torch.float8_e4m3fn).view(N, K)
        rows = torch.zeros((K // 128, (N // 128 + 3) // 4 * 4), dtype=torch.float32, device=W.device)
        rows[:, :N // 128] = s.t()
        return q.view(torch.uint8), rows
    if kind == "mxfp8":
        e = _block_exponent(W, 8)
        q = _mx_scaled(W, e).clamp(-448.0, 448.0).float().to(torch.float8_e4m3fn)
        return q.view(torch.uint8), _scale_rows(e)
    q, e = _quant_mx4(W)
    return q, _scale_rows(e)


def _plain_weight(q, s, kind):
    """fp32 [N, K] that codes and scales stand for."""
    if kind == "fp8":
        v = q.view(torch.float8_e4m3fn).float()
        N, K = v.shape
        return (v.view(N // 128, 128, K // 128, 128) * s[:, :N // 128].t()[:, None, :, None]).view(N, K)
    return _times_blocks(_mx4_values(q) if kind == "mxfp4" else q.view(torch.float8_e4m3fn).float(), s)


# ----------------------------------------------------------------------------
# inputs
# ----------------------------------------------------------------------------

def _normal(g, shape, sigma=1.0):
    t = torch.randn(shape, generator=g, device="cuda", dtype=torch.float32)
    return (t * sigma).to(torch.bfloat16)


def _experts(g, E, N, K, kind):
    """Expert weights [E, N, K] of deviation 0.02 in the format, one expert after the other."""
    q, s = [], []
    for _ in range(E):
        a, b = _weight(_normal(g, (N, K), 0.02).float(), kind)
        q.append(a)
        s.append(b)
    return torch.stack(q), torch.stack(s)


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    st = {"case": dict(case)}
    if case["op"] == "quant":
        x = _normal(g, (case["R"], case["C"]), 0.02)
        x[5::97, :32] = 0.0          # blocks that were pruned away
        st["x"] = x
        return st
    T = case["T"]
    if case["op"] == "mm":
        st["x"] = _normal(g, (T, case["K"]))
        st["w"], st["s"] = _weight(_normal(g, (case["N"], case["K"]), 0.02).float(), case["kind"])
        st["residual"] = _normal(g, (T, case["N"])) if case["residual"] else None
        return st
    D, H, E, k = case["D"], case["H"], case["E"], case["k"]
    st["x"] = _normal(g, (T, D))
    st["w12"], st["s12"] = _experts(g, E, 2 * H, D, case["kind"])
    st["out_proj"], st["s_out"] = _experts(g, E, D, H, case["kind"])
    st["residual"] = _normal(g, (T, D)) if case["residual"] else None
    st["idx"] = st["w"] = None
    if E > 1:
        demand = torch.randn(E, generator=g, device="cuda") * 0.5
        idx = (torch.randn((T, E), generator=g, device="cuda") + demand).argsort(1, descending=True)[:, :k]
        idx = idx.to(torch.int32).contiguous()
        idx[4::9, k - 1] = -1        # a choice that was dropped
        idx[12::13] = -1             # places of the batch that hold no sequence
        w = torch.rand((T, k), generator=g, device="cuda") + 0.05
        st["idx"], st["w"] = idx, w / w.sum(1, keepdim=True)
    return st


# ----------------------------------------------------------------------------
# plain forms
# ----------------------------------------------------------------------------

def _quant(st):
    q, e = _quant_mx4(st["x"].float())
    s = _scale_rows(e)
    return {"q": q, "s": s[:, :q.shape[0]], "y": _times_blocks(_mx4_values(q), s).to(torch.bfloat16)}


def _mm(st):
    case = st["case"]
    out = st["x"].float() @ _plain_weight(st["w"], st["s"], case["kind"]).t()
    if st["residual"] is not None:
        out = out + st["residual"].float()
    return {"out": out if case["out"] == "f32" else out.to(torch.bfloat16)}


def _moe(st):
    """Every expert on every token; the weights of the tokens that did not choose it are 0."""
    case = st["case"]
    x, H = st["x"].float(), case["H"]
    out = torch.zeros_like(x) if st["residual"] is None else st["residual"].float()
    for e in range(case["E"]):
        ab = x @ _plain_weight(st["w12"][e], st["s12"][e], case["kind"]).t()
        a, b = ab[:, :H], ab[:, H:]
        y = (a / (1.0 + torch.exp(-a)) * b) @ _plain_weight(st["out_proj"][e], st["s_out"][e], case["kind"]).t()
        if st["idx"] is not None:
            y = y * torch.where(st["idx"] == e, st["w"], 0.0).sum(1, keepdim=True)
        out = out + y
    return {"out": out.to(torch.bfloat16)}


# ----------------------------------------------------------------------------
# the library
# ----------------------------------------------------------------------------

def _run_own(st):
    import blockwise_scaled_fp8_bs_amd as bs
    case, op = st["case"], st["case"]["op"]
    if op == "quant":
        x = st["x"]
        R, C = x.shape
        q = torch.empty((R, C // 2), dtype=torch.uint8, device=x.device)
        s = bs.empty_mx_scales(C // 32, R, x.device)
        y = torch.empty_like(x)
        bs.bs_mx4_quant_1x32(x, q, s, y=y)
        return {"q": q, "s": s[:, :R], "y": y}
    kind = {"fp8": bs.BS_WEIGHT_E4M3_128X128, "mxfp8": bs.BS_WEIGHT_MXFP8, "mxfp4": bs.BS_WEIGHT_MXFP4}[case["kind"]]
    if op == "mm":
        dtype = torch.float32 if case["out"] == "f32" else torch.bfloat16
        return {"out": bs.bs_few_mm(st["x"], st["w"], st["s"], kind, residual=st["residual"], out_dtype=dtype)}
    return {"out": bs.bs_moe_few(st["x"], st["idx"], st["w"], st["w12"], st["s12"], st["out_proj"], st["s_out"], kind,
                                 residual=st["residual"])}


def run(state):
    if own:
        return _run_own(state)
    return {"quant": _quant, "mm": _mm, "moe": _moe}[state["case"]["op"]](state)


# ----------------------------------------------------------------------------
# what a pass cannot do without
# ----------------------------------------------------------------------------

def _weight_bytes(N, K, kind):
    if kind == "fp8":
        return N * K + N * K // 4096
    return N * K // (1 if kind == "mxfp8" else 2) + N * K // 32


def work(case):
    if case["op"] == "quant":
        n = case["R"] * case["C"]
        return {"bytes": 2 * n + n // 2 + n // 32 + 2 * n, "flops": 4 * n}
    T, kind = case["T"], case["kind"]
    if case["op"] == "mm":
        N, K = case["N"], case["K"]
        rows = T * N * ((4 if case["out"] == "f32" else 2) + (2 if case["residual"] else 0))
        return {"bytes": _weight_bytes(N, K, kind) + 2 * T * K + rows, "flops": 2 * T * N * K}
    D, H, E, k = case["D"], case["H"], case["E"], case["k"]
    used = E * (1.0 - (1.0 - k / E) ** T)          # experts that some token chose, on average
    n = int(used * (_weight_bytes(2 * H, D, kind) + _weight_bytes(D, H, kind)))
    return {"bytes": n + 2 * T * D * (3 if case["residual"] else 2) + 8 * T * k, "flops": 6 * T * k * D * H}


# ----------------------------------------------------------------------------
# from the definitions, in 64 bits
# ----------------------------------------------------------------------------

def _exact_weight(q, s, kind):
    """float64 [N, K]: every code decoded from its bit fields, times its block's scale."""
    if kind == "mxfp4":
        c = torch.empty((q.shape[0], 2 * q.shape[1]), dtype=torch.int64, device=q.device)
        c[:, 0::2], c[:, 1::2] = (q % 16).long(), (q // 16).long()
        bits, bias = 1, 1
        sign, field = c // 8, c % 8
    else:
        c = q.long()
        bits, bias = 3, 7
        sign, field = c // 128, c % 128
    ex, frac = field >> bits, (field & ((1 << bits) - 1)).double() / (1 << bits)
    v = torch.where(ex > 0, (1.0 + frac) * torch.exp2((ex - bias).double()), frac * 2.0 ** (1 - bias))
    v = torch.where(sign > 0, -v, v)
    N, K = v.shape
    if kind == "fp8":
        return v * s[:, :N // 128].double().t().repeat_interleave(128, 0).repeat_interleave(128, 1)
    return v * torch.exp2(s[:, :N].double() - 127.0).t().repeat_interleave(32, 1)


def exact(case, seed):
    st = prepare(case, seed)
    kind = case.get("kind")
    if case["op"] == "quant":
        x = st["x"].double()
        R, C = x.shape
        amax = x.reshape(R, C // 32, 32).abs().max(2).values
        e = torch.floor(torch.log2(torch.clamp(amax, min=2.0 ** -140))) - 2.0
        e = torch.clamp(e, -127.0, 127.0)
        two = torch.exp2(e).repeat_interleave(32, 1)
        m = (x / two).abs()
        step = torch.where(m < 2.0, 0.5, torch.where(m < 4.0, 1.0, 2.0))   # spacing of the grid around m
        m = torch.clamp(torch.round(m / step) * step, max=6.0)
        neg = torch.signbit(x)
        code = torch.where(m < 2.0, 2.0 * m, torch.where(m < 4.0, m + 2.0, m / 2.0 + 4.0)) + 8.0 * neg
        return {"q": (code[:, 0::2] + 16.0 * code[:, 1::2]).to(torch.uint8), "s": (e + 127.0).t().to(torch.uint8),
                "y": torch.where(neg, -m, m) * two}
    x = st["x"].double()
    if case["op"] == "mm":
        out = torch.mm(x, _exact_weight(st["w"], st["s"], kind).t())
        return {"out": out if st["residual"] is None else st["residual"].double() + out}
    out = torch.zeros_like(x) if st["residual"] is None else st["residual"].double().clone()
    H = case["H"]
    for e in range(case["E"]):
        if st["idx"] is None:
            tok = torch.arange(case["T"], device=x.device)
            weight = torch.ones(case["T"], dtype=torch.float64, device=x.device)
        else:
            tok, j = (st["idx"] == e).nonzero(as_tuple=True)
            weight = st["w"][tok, j].double()
        if tok.numel() == 0:
            continue
        w12 = _exact_weight(st["w12"][e], st["s12"][e], kind)
        gate, up = torch.mm(x[tok], w12[:H].t()), torch.mm(x[tok], w12[H:].t())
        h = torch.sigmoid(gate) * gate * up
        out.index_add_(0, tok, torch.mm(h, _exact_weight(st["out_proj"][e], st["s_out"][e], kind).t()) * weight[:, None])
    return {"out": out}
