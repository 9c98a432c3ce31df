"""The MoE block's calls on a stream other than the current one."""

import pytest
import torch

import blockwise_scaled_fp8_bs_amd as bs
from blockwise_scaled_fp8_bs_amd import inputs
from gpu_support import need_gpu

pytestmark = pytest.mark.gpu


def _calls(stream):
    """Every call that allocates, with a plan large enough for a workspace."""
    T, E, k, D = 9000, 16, 4, 256
    g = torch.Generator().manual_seed(1)
    logits, dw = torch.randn((T, E), generator=g).cuda(), torch.randn((T, k), generator=g).cuda()
    x, u, dh = (inputs.bf16_normal((T, D), 1.0, s).cuda() for s in (1, 2, 3))
    w_pre, w_post, gate = torch.randn(D, generator=g).cuda(), torch.randn(D, generator=g).cuda(), torch.randn((1, D), generator=g).cuda()
    r, rstd_u, rstd_r = torch.empty_like(x), torch.empty(T, device="cuda"), torch.empty(T, device="cuda")
    torch.cuda.synchronize()
    idx, w = bs.bs_moe_route(logits, k, stream=stream)
    dl = bs.bs_moe_route_bwd(logits, idx, w, dw, stream=stream)
    plan = bs.bs_moe_plan(idx, E, stream=stream)
    if stream is not None:
        stream.synchronize()  # ys is filled on the current stream
    ys = inputs.bf16_normal((plan.row_slot.shape[0], D), 1.0, 4).cuda()
    torch.cuda.synchronize()
    out = bs.bs_moe_combine(ys, plan.slot_row, w=w, stream=stream)
    d = bs.bs_moe_combine_dw(x, ys, plan.slot_row, stream=stream)
    params = dict(u=u, w_post=w_post, gate=gate)
    bs.bs_resid_norm(x, w_pre, **params, r=r, rstd_u=rstd_u, rstd_r=rstd_r, stream=stream)
    grads = bs.bs_resid_norm_bwd(r, rstd_r, w_pre, dh, rstd_u=rstd_u, **params, stream=stream)
    torch.cuda.synchronize()
    return [idx, w, dl, *plan, out, d, r, rstd_u, rstd_r, *grads]


def test_outputs_and_workspaces_belong_to_the_stream_passed(monkeypatch):
    """What a call allocates, it allocates where its kernel runs: memory of
    another stream's pool could be handed out again while the kernel works."""
    need_gpu()
    print("calls on the current stream", flush=True)
    want = _calls(None)
    side = torch.cuda.Stream()
    seen = []
    real = torch.empty

    def empty(*a, **kw):
        if kw.get("device") is not None and torch.device(kw["device"]).type == "cuda":
            seen.append(torch.cuda.current_stream().cuda_stream)
        return real(*a, **kw)

    from blockwise_scaled_fp8_bs_amd import binding_block

    class Recording:
        def __getattr__(self, name):
            return empty if name == "empty" else getattr(torch, name)

    monkeypatch.setattr(binding_block, "torch", Recording())
    print("calls on a side stream", flush=True)
    got = _calls(side)
    # idx, w; dlogits; the plan; out; dw; dx, du, three parameter gradients and the workspace
    assert len(seen) == 12 and all(s == side.cuda_stream for s in seen)
    for a, b in zip(want, got):
        assert a.dtype == b.dtype and torch.equal(a.view(torch.uint8), b.view(torch.uint8))
