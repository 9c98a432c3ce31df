"""Layers prepared for serving: few tokens through the few-token calls, more
through the GEMMs, and the calls as a server strings them together."""

import numpy as np
import pytest
import torch

import blockwise_scaled_fp8_bs_amd as bs
from blockwise_scaled_fp8_bs_amd import serving
from few_support import f64
from gpu_support import need_gpu, u8
from oracle import few

pytestmark = pytest.mark.gpu

FEW = {"fp8": "e4m3", "mxfp8": "mxfp8", "mxfp4": "mxfp4"}


def _x(T, D, seed=0, sigma=1.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn((T, D), generator=g) * sigma).to(torch.bfloat16).cuda()


def _values(w, weights):
    """float64 values of w [N, K] as the format holds them, from the quantizers' codes."""
    N, K = w.shape
    if weights == "fp8":
        q, s = serving.rows_128(w.detach())
        return few.weights(u8(q), s.cpu().numpy()[:, :N // 128].T, "e4m3")
    q, s = (serving.rows_mx8 if weights == "mxfp8" else serving.rows_mx4)(w.detach())[:2]
    return few.weights(u8(q), u8(s)[:, :N].T, weights)


@pytest.mark.parametrize("cls,weights", [(bs.Float8BlockwiseLinear, "fp8"), (bs.Float8BlockwiseLinear, "mxfp4"),
                                         (bs.Float8MXLinear, "mxfp8"), (bs.Float8MXLinear, "mxfp4")])
def test_linear_layers(cls, weights):
    need_gpu()
    torch.manual_seed(0)
    m = cls(640, 384, device="cuda").eval().prepare_serving(weights)
    w = _values(m.weight, weights)
    with torch.no_grad():
        for T in (1, 3, 16, 40, 64, 128):
            print(f"{cls.__name__} {weights} {T} tokens", flush=True)
            x = _x(T, 640, T)
            y = m(x.view(1, T, 640))
            assert y.shape == (1, T, 384)
            ref, bound = few.few_mm(f64(x), w)
            assert (np.abs(f64(y[0]) - ref) <= bound).all()
        # more tokens: the training forward's GEMM on the same codes
        for T in (129, 256, 300):
            print(f"{cls.__name__} {weights} {T} tokens", flush=True)
            x = _x(T, 640, T)
            y = m(x)
            full = torch.zeros((384, 640), dtype=torch.bfloat16, device="cuda")
            full[:T] = x
            plain = cls(640, 384, device="cuda")
            plain.weight.copy_(m.weight if weights != "mxfp4" else serving.rows_mx4(m.weight.detach(), values=True)[2])
            assert torch.equal(y, plain(full)[:T])
        # gradients on: the training forward, which takes whole blocks of tokens
    with pytest.raises(ValueError, match="128"):
        m(_x(3, 640))
    x = _x(128, 640).requires_grad_(True)
    m(x).sum().backward()
    assert x.grad is not None and m.weight.grad is not None


@pytest.mark.parametrize("weights", ["fp8", "mxfp4"])
def test_gated_ffn(weights):
    need_gpu()
    torch.manual_seed(1)
    D, H = 384, 512
    m = bs.Float8BlockwiseGatedFFN(D, H, device="cuda").eval().prepare_serving(weights, few_tokens=40)
    v12 = _values(torch.cat([m.w1, m.w2]), weights)
    vo = _values(m.out_proj, weights)
    with torch.no_grad():
        for T in (1, 7, 40):
            print(f"gated FFN {weights} {T} tokens", flush=True)
            x = _x(T, D, T)
            ref, bound = few.moe(f64(x), np.zeros((T, 1), int), np.ones((T, 1)), [v12], [vo])
            assert (np.abs(f64(m(x)) - ref) <= bound).all()
        for T in (41, 128):
            print(f"gated FFN {weights} {T} tokens", flush=True)
            x = torch.zeros((128, D), dtype=torch.bfloat16, device="cuda")
            x[:T] = _x(T, D, T)
            plain = bs.Float8BlockwiseGatedFFN(D, H, device="cuda")
            for p, q in zip(plain.parameters(), m.parameters()):
                p.copy_(q if weights == "fp8" else serving.rows_mx4(q.detach(), values=True)[2])
            assert torch.equal(m(x[:T]), plain(x)[:T])
        assert m(x[:0]).shape == (0, D)


@pytest.mark.parametrize("weights", ["fp8", "mxfp4"])
def test_expert_layer(weights):
    need_gpu()
    torch.manual_seed(2)
    D, H, E, k = 256, 384, 8, 3
    m = bs.Float8BlockwiseMoE(D, H, E, k, device="cuda").eval()
    v12, vo = ([_values(w, weights) for w in p] for p in (m.w12, m.out_proj))
    with torch.no_grad():
        m.prepare_serving(weights, few_tokens=33)
        for T in (1, 2, 9, 33):
            print(f"experts {weights} {T} tokens", flush=True)
            x, res = _x(T, D, T), _x(T, D, 100 + T)
            y = m(x, residual=res)
            idx, w = bs.moe_route(torch.nn.functional.linear(x, m.router), k, bias=m.balance, **m.how)
            ref, bound = few.moe(f64(x), idx.cpu().numpy(), w.cpu().double().numpy(), v12, vo, f64(res))
            assert (np.abs(f64(y) - ref) <= bound).all() and m.last_counts is None
        # past that, and without few tokens: the grouped GEMMs, bit for bit what they gave
        x = _x(34, D, 9)
        y = m(x)
        assert m.last_counts is not None
        if weights == "mxfp4":
            q = bs.Float8BlockwiseMoE(D, H, E, k, device="cuda").eval()
            q.load_state_dict({**m.state_dict(), "w12": serving.experts_mx4(m.w12.detach())[2],
                               "out_proj": serving.experts_mx4(m.out_proj.detach())[2]})
            m = q
        want = m(x)
        assert torch.equal(y, want)
        assert torch.equal(m.prepare_serving()(x[:2]), want[:2])


def test_layout_of_exchanged_weights():
    """After each way to exchange a weight: never an answer with the old one."""
    need_gpu()
    torch.manual_seed(3)
    x = _x(128, 256)
    for m, name in ((bs.Float8BlockwiseLinear(256, 256, device="cuda"), "weight"),
                    (bs.Float8MXLinear(256, 256, device="cuda"), "weight"),
                    (bs.Float8BlockwiseGatedFFN(256, 512, device="cuda"), "out_proj")):
        print(f"{type(m).__name__} with exchanged weights", flush=True)
        with torch.no_grad():
            m.eval()
            plain = m(x)
            m.prepare_serving(few_tokens=4)
            assert torch.equal(m(x), plain) and m(x[:4]).shape[0] == 4
            p = getattr(m, name)
            other = torch.empty_like(p).uniform_(-0.1, 0.1)
            got = torch.func.functional_call(m, {name: other}, (x,))
            assert not torch.equal(got, plain)
            old = p.detach().clone()
            p.copy_(other)
            with pytest.raises(RuntimeError, match="call it again"):
                m(x)
            assert torch.equal(m.prepare_serving(few_tokens=4)(x), got)
            m.load_state_dict({**m.state_dict(), name: old})
            assert m._serving is None and torch.equal(m(x), plain)
            m.prepare_serving().train()
            assert m._serving is None


class Server:
    """One token step of a small model: norm, experts, norm, head in 4 bits."""

    def __init__(self, T, weights):
        torch.manual_seed(4)
        self.D, self.V = 256, 1000
        self.moe = bs.Float8BlockwiseMoE(self.D, 256, 16, 4, n_group=4, topk_group=2, group_best=2, device="cuda").eval()
        self.moe.prepare_serving(weights, few_tokens=64)
        self.up = bs.Float8BlockwiseLinear(self.D, self.D, device="cuda").eval().prepare_serving(weights)
        self.norm = torch.ones(self.D, device="cuda")
        head = (torch.randn((self.V, self.D), device="cuda") * 0.05).to(torch.bfloat16)
        self.q, self.s, _ = serving.rows_mx4(head)

    @torch.no_grad()
    def __call__(self, x):
        u = self.up(x)
        r, h = bs.resid_norm(x, self.norm, u=u, w_post=self.norm)
        r = self.moe(h, residual=r)
        _, h = bs.resid_norm(r, self.norm)
        return r, bs.bs_few_mm(h, self.q, self.s, bs.BS_WEIGHT_MXFP4, out_dtype=torch.float32)


@pytest.mark.parametrize("weights", ["fp8", "mxfp4"])
@pytest.mark.parametrize("T", [1, 6, 40])
def test_a_step_replays_from_a_graph(T, weights):
    """Two captured steps on the same weights, replayed in turn with eager work between, each against eager."""
    need_gpu()
    print(f"captured step {weights}, {T} tokens", flush=True)
    step = Server(T, weights)
    static = [_x(T, step.D, 10 + i) for i in range(2)]
    step(static[0])
    graphs, outs = [], []
    for x in static:
        g = torch.cuda.CUDAGraph()
        torch.cuda.synchronize()
        with torch.cuda.graph(g):
            outs.append(step(x))
        graphs.append(g)
    for i in range(4):
        for j in (0, 1):
            x = _x(T, step.D, 50 + 2 * i + j)
            want = step(x)
            static[j].copy_(x)
            for o in outs[j]:
                o.fill_(float("nan"))
            torch.cuda.synchronize()
            graphs[j].replay()
            torch.cuda.synchronize()
            assert all(torch.equal(a, b) for a, b in zip(outs[j], want))


def test_steps_on_two_streams_at_once():
    need_gpu()
    print("steps on two streams", flush=True)
    step = Server(24, "fp8")
    xs = [_x(24, step.D, 70 + i) for i in range(8)]
    want = [step(x) for x in xs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = []
    for i, x in enumerate(xs):
        with torch.cuda.stream(streams[i % 2]):
            got.append(step(x))
    torch.cuda.synchronize()
    for a, b in zip(got, want):
        assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


def test_calls_on_a_stream_that_is_not_the_current_one(monkeypatch):
    """Outputs and the workspace come from the pool of the stream passed, where the kernels run."""
    need_gpu()
    print("few-token calls on a side stream", flush=True)
    step = Server(5, "mxfp4")
    x = _x(5, step.D, 3)
    q12, s12, qo, so, kind = step.moe._serving[4:9]
    idx = torch.stack([torch.randperm(16)[:4] for _ in range(5)]).to(torch.int32).cuda()
    w = torch.rand((5, 4)).cuda()

    def calls(stream):
        a = bs.bs_few_mm(x, step.q, step.s, bs.BS_WEIGHT_MXFP4, stream=stream)
        b = bs.bs_moe_few(x, idx, w, q12, s12, qo, so, kind, stream=stream)
        torch.cuda.synchronize()
        return a, b

    want = calls(None)
    side = torch.cuda.Stream()
    seen, real = [], torch.empty

    def empty(*a, **kw):
        seen.append(torch.cuda.current_stream().cuda_stream)
        return real(*a, **kw)

    from blockwise_scaled_fp8_bs_amd import binding_block

    class Recording:
        def __getattr__(self, name):
            return empty if name == "empty" else getattr(torch, name)

    monkeypatch.setattr(binding_block, "torch", Recording())
    torch.cuda.synchronize()
    got = calls(side)
    assert len(seen) == 3 and all(s == side.cuda_stream for s in seen)   # two outputs, one workspace
    assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_binding_refusals():
    need_gpu()
    u8t, bf = torch.uint8, torch.bfloat16
    new = lambda *s, dtype=bf: torch.zeros(s, dtype=dtype, device="cuda")  # noqa: E731
    x, w, s = new(3, 96), new(50, 48, dtype=u8t), new(3, 64, dtype=u8t)
    K4, K8 = bs.BS_WEIGHT_MXFP4, bs.BS_WEIGHT_MXFP8
    for args, kw, match in (((x, w, s, 7), {}, "kind"), ((x, w, s, K8), {}, "w must be"), ((x, w, s.float(), K4), {}, "uint8"),
                            ((x, w, s[:2], K4), {}, "s must be"), ((x, w, s[:, :49], K4), {}, "s must be"),
                            ((x, w.t(), s, K4), {}, "w must"), ((x.t(), w, s, K4), {}, "unit stride"),
                            ((x, w, s, K4), dict(residual=new(3, 49)), "residual"),
                            ((x, w, s, K4), dict(out=new(3, 50, dtype=torch.float16)), "out must be"),
                            ((x, w, s, K4), dict(out_dtype=torch.float16), "out_dtype"),
                            ((x, w, s, K4), dict(out=new(2, 50)), "out"), ((x, w.cpu(), s, K4), {}, "GPU"),
                            ((x, w, s, K4), dict(residual=new(3, 50).cpu()), "GPU")):
        with pytest.raises(ValueError, match=match):
            bs.bs_few_mm(*args, **kw)
    w12, s12, wo, so = new(4, 64, 96, dtype=u8t), new(4, 3, 64, dtype=u8t), new(4, 96, 32, dtype=u8t), new(4, 1, 96, dtype=u8t)
    idx, wt = new(3, 2, dtype=torch.int32), new(3, 2, dtype=torch.float32)
    ok = (x, idx, wt, w12, s12, wo, so, K8)
    bs.bs_moe_few(*ok)
    for i, bad, match in ((1, None, "idx is required"), (1, idx[:2], "idx must be"), (1, idx.long(), "int32"),
                          (2, wt.double(), "float32"), (2, wt[:, :1], "w must"), (3, w12[:, :63], "w12 must be"),
                          (3, w12[0], "w12 must be"), (4, s12[:3], "s12 must be"), (5, wo[:, :95], "out_proj must be"),
                          (6, so[:, :, :95], "s_out must be"), (7, K4, "w12 must be"), (5, wo.cpu(), "GPU"), (1, idx.cpu(), "GPU")):
        args = list(ok)
        args[i] = bad
        with pytest.raises(ValueError, match=match):
            bs.bs_moe_few(*args)
    with pytest.raises(bs.BsError, match="16-byte|multiples of 16"):
        bs.bs_few_mm(x, new(50, 56, dtype=u8t)[:, 8:], s, K4)
    q, sc = new(3, 48, dtype=u8t), new(3, 16, dtype=u8t)
    for args, kw, match in (((x, q[:, :47], sc), {}, "q must"), ((x, q, sc[:2]), {}, "s must"), ((x.float(), q, sc), {}, "bfloat16"),
                            ((x, q, sc), dict(y=new(3, 95)), "y must"), ((x, q.cpu(), sc), {}, "GPU")):
        with pytest.raises(ValueError, match=match):
            bs.bs_mx4_quant_1x32(*args, **kw)
