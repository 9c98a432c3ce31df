"""Refusals of the entry points around the experts' products, and of their
Python binding: no GPU, fake pointers, nothing is enqueued."""

import ctypes
import os

import pytest
import torch

import blockwise_scaled_fp8_bs_amd as bs
from blockwise_scaled_fp8_bs_amd import _lib

OK, NULL, SHAPE, LAYOUT, ALIGN, MODE = 0, 1, 2, 3, 4, 5
P, PU = 0x10000, 0x10002


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(_lib.LIB_PATH):
        pytest.fail("libbs.so is not built (python -m blockwise_scaled_fp8_bs_amd.build)")
    return _lib.load()


def call(lib, name, defaults, kw, code, frag):
    args = dict(defaults, **kw)
    assert getattr(lib, name)(*args.values()) == code
    assert frag in lib.bs_last_error().decode()


ROUTE = dict(logits=P, dtype=1, T=16, E=64, ld=64, bias=None, score=1, k=4, n_group=8, topk_group=4, group_best=2,
             renorm=1, scale=1.0, idx=P, w=P, stream=None)


@pytest.mark.parametrize("kw,code,frag", [
    (dict(dtype=7), MODE, "dtype"),
    (dict(score=3), MODE, "score"),
    (dict(T=-1), SHAPE, "T="),
    (dict(E=0), SHAPE, "E=0"),
    (dict(E=1025, ld=1025), SHAPE, "1024"),
    (dict(k=0), SHAPE, "k=0"),
    (dict(k=33), SHAPE, "32"),
    (dict(E=8, k=9, n_group=1, topk_group=1), SHAPE, "min(E, 32)"),
    (dict(scale=0.0), MODE, "scale"),
    (dict(scale=float("nan")), MODE, "scale"),
    (dict(logits=None), NULL, "logits"),
    (dict(ld=63), LAYOUT, "row-major"),
    (dict(logits=PU), ALIGN, "aligned"),
    (dict(idx=PU), ALIGN, "aligned"),
    (dict(n_group=7), SHAPE, "divide"),
    (dict(topk_group=9), SHAPE, "topk_group"),
    (dict(group_best=3), MODE, "group_best"),
    (dict(bias=0x10001), ALIGN, "bias"),
])
def test_route_refusals(lib, kw, code, frag):
    call(lib, "bs_moe_route", ROUTE, kw, code, frag)


ROUTE_BWD = dict(logits=P, dtype=1, T=16, E=64, ld=64, score=1, k=4, renorm=1, scale=1.0, idx=P, w=P, dw=P, d=P, ld_d=64,
                 stream=None)


@pytest.mark.parametrize("kw,code,frag", [
    (dict(dw=None), NULL, "dw"),
    (dict(d=None), NULL, "dlogits"),
    (dict(ld_d=60), LAYOUT, "ld_d"),
    (dict(d=PU), ALIGN, "dlogits"),
    (dict(scale=0.0), MODE, "scale"),
    (dict(E=0), SHAPE, "E=0"),
])
def test_route_bwd_refusals(lib, kw, code, frag):
    call(lib, "bs_moe_route_bwd", ROUTE_BWD, kw, code, frag)


PLAN = dict(idx=P, T=64, k=2, E=8, align=128, M=1152, ends=P, counts=P, slot_row=P, row_slot=P, ws=None, nbytes=0,
            stream=None)


@pytest.mark.parametrize("kw,code,frag", [
    (dict(E=0), SHAPE, "E=0"),
    (dict(E=2000), SHAPE, "1024"),
    (dict(k=0), SHAPE, "k=0"),
    (dict(T=2 ** 31), SHAPE, "2^31"),
    (dict(align=0), SHAPE, "align"),
    (dict(M=1023), SHAPE, "M=1023 must be >= 1024"),
    (dict(ends=None), NULL, "group_end"),
    (dict(idx=None), NULL, "idx"),
    (dict(row_slot=None), NULL, "row_slot"),
    (dict(slot_row=PU), ALIGN, "aligned"),
    (dict(T=5000, M=11024), SHAPE, "workspace"),
    (dict(T=5000, M=11024, nbytes=1 << 20), NULL, "workspace"),
    (dict(T=5000, M=11024, nbytes=1 << 20, ws=0x10004), ALIGN, "workspace"),
])
def test_plan_refusals(lib, kw, code, frag):
    call(lib, "bs_moe_plan", PLAN, kw, code, frag)


def test_plan_rows_and_workspace():
    lib = _lib.load()
    assert lib.bs_moe_plan_rows(24, 8, 64, 1) == 192
    assert lib.bs_moe_plan_rows(64, 2, 8, 128) == (128 + 8 * 127) // 128 * 128
    assert lib.bs_moe_plan_rows(1, 2, 8, 128) == 256           # at most two groups hold rows
    assert lib.bs_moe_plan_rows(0, 2, 8, 128) == 0
    for bad in ((-1, 2, 8, 1), (4, 0, 8, 1), (4, 33, 64, 1), (4, 2, 0, 1), (4, 2, 8, 0)):
        assert lib.bs_moe_plan_rows(*bad) == 0
    assert lib.bs_moe_plan_workspace_bytes(4096, 2, 256) == 0
    assert lib.bs_moe_plan_workspace_bytes(4097, 2, 256) > 0


GATHER = dict(x=P, T=64, D=256, ld_x=256, k=2, row_slot=P, M=256, w=None, y=None, ld_y=0, q_row=P, ld_qr=256, s_row=P,
              ld_sr=256, q_col=P, ld_qc=256, s_col=P, ld_sc=256, stream=None)


@pytest.mark.parametrize("kw,code,frag", [
    (dict(k=0), SHAPE, "k=0"),
    (dict(M=-1), SHAPE, ">= 0"),
    (dict(D=200), SHAPE, "multiple of 128"),
    (dict(x=None), NULL, "x is NULL"),
    (dict(row_slot=None), NULL, "row_slot"),
    (dict(q_row=None, s_row=None, q_col=None, s_col=None), NULL, "no output"),
    (dict(s_row=None), NULL, "both"),
    (dict(ld_x=128), LAYOUT, "ld of x"),
    (dict(x=0x10008), ALIGN, "x must be"),
    (dict(y=P, ld_y=252), LAYOUT, "ld of y"),
    (dict(M=200), SHAPE, "column output"),
    (dict(ld_qc=128), LAYOUT, "transpose"),
    (dict(ld_sr=250), LAYOUT, "K-major"),
    (dict(w=PU), ALIGN, "aligned"),
    (dict(ld_qr=264), ALIGN, "ld_qr"),
])
def test_gather_refusals(lib, kw, code, frag):
    call(lib, "bs_moe_gather_quant_1x128", GATHER, kw, code, frag)


COMBINE = dict(y=P, M=256, D=64, ld_y=64, slot_row=P, w=P, T=8, k=2, res=P, ld_res=64, out=P, ld_out=64, stream=None)


@pytest.mark.parametrize("kw,code,frag", [
    (dict(D=60), SHAPE, "multiple of 8"),
    (dict(k=0), SHAPE, "k=0"),
    (dict(y=None), NULL, "y is NULL"),
    (dict(out=None), NULL, "out"),
    (dict(ld_y=56), LAYOUT, "ld of y"),
    (dict(ld_res=68), ALIGN, "residual"),
    (dict(slot_row=PU), ALIGN, "slot_row"),
])
def test_combine_refusals(lib, kw, code, frag):
    call(lib, "bs_moe_combine", COMBINE, kw, code, frag)


DW = dict(dout=P, T=8, D=64, ld_dout=64, y=P, M=256, ld_y=64, slot_row=P, k=2, dw=P, stream=None)


@pytest.mark.parametrize("kw,code,frag", [
    (dict(D=60), SHAPE, "multiple of 8"),
    (dict(dw=None), NULL, "dw"),
    (dict(dout=None), NULL, "dout"),
    (dict(ld_dout=32), LAYOUT, "dout"),
    (dict(dw=PU), ALIGN, "dw"),
])
def test_combine_dw_refusals(lib, kw, code, frag):
    call(lib, "bs_moe_combine_dw", DW, kw, code, frag)


NORM = dict(x=P, u=P, R=256, D=256, ld_x=256, ld_u=256, w_post=P, gate=P, ld_gate=256, per=128, w_pre=P, dt=1, alpha=1.0,
            eps=1e-6, r=P, ld_r=256, rstd_u=P, rstd_r=P, h=None, ld_h=0, q_row=P, ld_qr=256, s_row=P, ld_sr=256,
            q_col=P, ld_qc=256, s_col=P, ld_sc=256, stream=None)


@pytest.mark.parametrize("kw,code,frag", [
    (dict(dt=9), MODE, "w_dtype"),
    (dict(D=252), SHAPE, "multiple of 8"),
    (dict(D=16512), SHAPE, "16384"),
    (dict(alpha=float("inf")), MODE, "alpha"),
    (dict(eps=-1.0), MODE, "eps"),
    (dict(x=None), NULL, "x is NULL"),
    (dict(r=None), NULL, "r must be set"),
    (dict(u=None), NULL, "need u"),
    (dict(w_post=None), NULL, "rstd_u needs w_post"),
    (dict(w_pre=None), NULL, "need w_pre"),
    (dict(rstd_r=None), NULL, "rstd_r"),
    (dict(per=100), SHAPE, "rows_per_gate"),
    (dict(ld_gate=200), LAYOUT, "ld_gate"),
    (dict(ld_gate=258), ALIGN, "gate rows"),
    (dict(ld_u=200), LAYOUT, "ld of u"),
    (dict(R=128 + 64, per=64), SHAPE, "column output"),
    (dict(D=136), SHAPE, "multiple of 128"),
    (dict(w_pre=0x10008), ALIGN, "w_pre"),
    (dict(u=None, r=None, w_post=None, gate=None, rstd_u=None, rstd_r=None, q_row=None, s_row=None, q_col=None,
          s_col=None), NULL, "no output"),
])
def test_norm_refusals(lib, kw, code, frag):
    call(lib, "bs_resid_norm", NORM, kw, code, frag)


NORM_BWD = dict(r=P, u=P, dh=P, dr=P, R=256, D=256, ld_r=256, ld_u=256, ld_dh=256, ld_dr=256, w_post=P, gate=P,
                ld_gate=256, per=128, w_pre=P, dt=1, alpha=1.0, rstd_u=P, rstd_r=P, dx=P, ld_dx=256, du=P, ld_du=256,
                dw_pre=P, dw_post=P, dgate=P, ws=P, nbytes=1 << 30, stream=None)


@pytest.mark.parametrize("kw,code,frag", [
    (dict(dt=9), MODE, "w_dtype"),
    (dict(D=252), SHAPE, "multiple of 8"),
    (dict(R=0), SHAPE, "R=0"),
    (dict(dx=None), NULL, "dx"),
    (dict(dh=None), NULL, "w_pre"),
    (dict(w_pre=None), NULL, "without w_pre"),
    (dict(u=None), NULL, "need u"),
    (dict(du=None), NULL, "du"),
    (dict(rstd_u=None), NULL, "rstd_u"),
    (dict(gate=None, per=256), NULL, "dgate"),
    (dict(per=100), SHAPE, "rows_per_gate"),
    (dict(nbytes=1000), SHAPE, "workspace"),
    (dict(ws=None), SHAPE, "workspace"),
    (dict(dgate=0x10004), ALIGN, "16-byte"),
    (dict(ld_dh=200), LAYOUT, "dh"),
])
def test_norm_bwd_refusals(lib, kw, code, frag):
    call(lib, "bs_resid_norm_bwd", NORM_BWD, kw, code, frag)


CK = dict(a=P, b=P, R=256, C=256, ld_a=256, ld_b=256, ck=P, ld_ck=512, s_ck=P, ld_sck=256, q_row=P, ld_qr=256, s_row=P,
          ld_sr=256, q_col=P, ld_qc=256, s_col=P, ld_sc=256, stream=None)


@pytest.mark.parametrize("kw,code,frag", [
    (dict(C=200), SHAPE, "multiple of 128"),
    (dict(ck=None), NULL, "ck"),
    (dict(q_row=None, s_row=None, q_col=None, s_col=None), NULL, "no output"),
    (dict(ld_ck=500), LAYOUT, "ld_ck"),
    (dict(ld_ck=520), ALIGN, "ld_ck"),
    (dict(ld_sck=254), LAYOUT, "ld_sck"),
    (dict(ld_b=252), LAYOUT, "ld of b"),
    (dict(R=200), SHAPE, "column output"),
])
def test_ckpt_refusals(lib, kw, code, frag):
    call(lib, "bs_swiglu_quant_1x128_ckpt", CK, kw, code, frag)


CK_BWD = dict(ck=P, R=256, C=256, ld_ck=512, s_ck=P, ld_sck=256, dh=P, ld_dh=256, q_row=P, ld_qr=512, s_row=P, ld_sr=256,
              q_col=P, ld_qc=256, s_col=P, ld_sc=512, stream=None)


@pytest.mark.parametrize("kw,code,frag", [
    (dict(C=200), SHAPE, "multiple of 128"),
    (dict(dh=None), NULL, "dh"),
    (dict(ld_qr=256), LAYOUT, "ld_qr"),
    (dict(ld_sc=256), LAYOUT, "ld_sc"),
    (dict(ld_ck=256), LAYOUT, "ld_ck"),
    (dict(R=200), SHAPE, "column output"),
])
def test_ckpt_bwd_refusals(lib, kw, code, frag):
    call(lib, "bs_swiglu_bwd_quant_1x128_ckpt", CK_BWD, kw, code, frag)


def test_empty_problems_are_ok(lib):
    for name, defaults, kw in (("bs_moe_route", ROUTE, dict(T=0)), ("bs_moe_route_bwd", ROUTE_BWD, dict(T=0)),
                               ("bs_moe_gather_quant_1x128", GATHER, dict(M=0)), ("bs_moe_combine", COMBINE, dict(T=0)),
                               ("bs_moe_combine_dw", DW, dict(T=0)), ("bs_resid_norm", NORM, dict(R=0)),
                               ("bs_resid_norm_bwd", NORM_BWD, dict(R=0, dw_pre=None, dw_post=None, dgate=None)),
                               ("bs_swiglu_quant_1x128_ckpt", CK, dict(R=0)),
                               ("bs_swiglu_bwd_quant_1x128_ckpt", CK_BWD, dict(R=0))):
        assert getattr(lib, name)(*dict(defaults, **kw).values()) == OK, name
        assert lib.bs_last_error() == b""


# ---- the Python binding ----

def test_binding_refuses_cpu_tensors_types_shapes_and_strides():
    l = torch.zeros((4, 8))
    with pytest.raises(ValueError, match="GPU"):
        bs.bs_moe_route(l, 2)
    with pytest.raises(ValueError, match="bfloat16 or float32"):
        bs.bs_moe_route(l.half(), 2)
    with pytest.raises(ValueError, match="int32"):
        bs.bs_moe_plan(torch.zeros((4, 2), dtype=torch.int64), 8)
    with pytest.raises(ValueError, match=r"\[T, k\]"):
        bs.bs_moe_plan(torch.zeros(4, dtype=torch.int32), 8)
    x = torch.zeros((4, 256), dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="bfloat16"):
        bs.bs_moe_gather_quant_1x128(x.float(), torch.zeros(4, dtype=torch.int32), 1)
    with pytest.raises(ValueError, match="GPU"):
        bs.bs_moe_combine(x, torch.zeros((4, 1), dtype=torch.int32))
    with pytest.raises(ValueError, match="GPU"):
        bs.bs_moe_combine_dw(x, x, torch.zeros((4, 1), dtype=torch.int32))
    with pytest.raises(ValueError, match="GPU"):
        bs.bs_resid_norm(x, torch.zeros(256))
    with pytest.raises(ValueError, match="GPU"):
        bs.bs_resid_norm_bwd(x, None, None, None)
    with pytest.raises(ValueError, match="GPU"):
        bs.bs_swiglu_quant_1x128_ckpt(x, x, None, None)
    with pytest.raises(ValueError, match="GPU"):
        bs.bs_swiglu_bwd_quant_1x128_ckpt(None, None, x)


def test_loader_knows_the_float_arguments():
    # a float passed where C takes a float must not arrive as an integer register
    assert ctypes.c_float in _lib.SIGNATURES["bs_moe_route"][1]
    assert _lib.SIGNATURES["bs_resid_norm"][1].count(ctypes.c_float) == 2
    assert _lib.SIGNATURES["bs_resid_norm_bwd"][1].count(ctypes.c_float) == 1


@pytest.mark.parametrize("align", [65537, 2 ** 31 - 1])
def test_plan_refuses_alignments_whose_sums_could_overflow(lib, align):
    call(lib, "bs_moe_plan", PLAN, dict(align=align, M=2 ** 31 - 1), SHAPE, "align")
    assert lib.bs_moe_plan_rows(64, 2, 8, align) == 0
