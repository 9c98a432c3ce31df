"""Refusals of the few-token entry points and of their Python binding: no GPU,
fake pointers, nothing is enqueued."""

import os

import pytest
import torch

import blockwise_scaled_fp8_bs_amd as bs
from blockwise_scaled_fp8_bs_amd import _lib

OK, NULL, SHAPE, LAYOUT, ALIGN, MODE = 0, 1, 2, 3, 4, 5
P, PU, P1 = 0x10000, 0x10002, 0x10001


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(_lib.LIB_PATH):
        pytest.fail("libbs.so is not built (python -m blockwise_scaled_fp8_bs_amd.build)")
    return _lib.load()


def call(lib, name, defaults, kw, code, frag=""):
    assert set(kw) <= set(defaults)
    assert getattr(lib, name)(*dict(defaults, **kw).values()) == code
    assert frag in lib.bs_last_error().decode()


QUANT = dict(x=P, R=64, C=96, ld_x=96, q=P, ld_q=48, s=P, ld_s=64, y=None, ld_y=0, stream=None)


@pytest.mark.parametrize("kw,code,frag", [
    (dict(R=-1), SHAPE, "R=-1"),
    (dict(R=1 << 31), SHAPE, "2^31"),
    (dict(C=80, ld_x=80), SHAPE, "32"),
    (dict(C=-32), SHAPE, "C=-32"),
    (dict(x=None), NULL, "x, q and s"),
    (dict(q=None), NULL, "x, q and s"),
    (dict(s=None), NULL, "x, q and s"),
    (dict(ld_x=88), LAYOUT, "ld_x"),
    (dict(ld_x=1 << 22), LAYOUT, "ld_x"),
    (dict(ld_x=100), ALIGN, "ld_x"),
    (dict(x=PU), ALIGN, "x must"),
    (dict(ld_q=32), LAYOUT, "ld_q"),
    (dict(ld_q=56), ALIGN, "ld_q"),
    (dict(q=PU), ALIGN, "q must"),
    (dict(ld_s=48), LAYOUT, "ld_s"),
    (dict(ld_s=72), LAYOUT, "16"),
    (dict(s=PU), ALIGN, "s must"),
    (dict(y=P, ld_y=88), LAYOUT, "ld_y"),
    (dict(y=PU, ld_y=96), ALIGN, "y must"),
    (dict(R=(1 << 31) - 1, ld_s=1 << 31, C=1 << 16, ld_x=1 << 16, ld_q=1 << 15), SHAPE, "one launch"),
])
def test_quantizer_refusals(lib, kw, code, frag):
    call(lib, "bs_mx4_quant_1x32", QUANT, kw, code, frag)


def test_quantizer_of_nothing(lib):
    for kw in (dict(R=0), dict(C=0), dict(R=0, x=None, q=None, s=None)):
        call(lib, "bs_mx4_quant_1x32", QUANT, kw, OK)


MM = dict(kind=2, T=3, N=50, K=96, x=P, ld_x=96, w=P, ld_w=48, s=P, ld_s=64, res=None, ld_res=0, out=P, ld_out=50, dtype=0,
          stream=None)


@pytest.mark.parametrize("kw,code,frag", [
    (dict(kind=3), MODE, "kind=3"),
    (dict(dtype=2), MODE, "out_dtype"),
    (dict(T=-1), SHAPE, "T=-1"),
    (dict(T=(1 << 21) + 1), SHAPE, "2^21"),
    (dict(N=-1), SHAPE, "N=-1"),
    (dict(K=0), SHAPE, "K=0"),
    (dict(x=None), NULL, "x is NULL"),
    (dict(ld_x=88), LAYOUT, "ld_x"),
    (dict(ld_x=1 << 22), LAYOUT, "2^22"),
    (dict(ld_x=98), ALIGN, "ld_x"),
    (dict(x=PU), ALIGN, "x must"),
    (dict(w=None), NULL, "w and its scales"),
    (dict(s=None), NULL, "w and its scales"),
    (dict(K=80, ld_x=80), SHAPE, "32"),
    (dict(ld_w=32), LAYOUT, "ld of w"),
    (dict(ld_w=1 << 22), LAYOUT, "2^22"),
    (dict(ld_w=56), ALIGN, "multiples of 16"),
    (dict(w=PU), ALIGN, "16-byte"),
    (dict(ld_s=48), LAYOUT, "scales of w"),
    (dict(ld_s=56), ALIGN, "scales of w"),
    (dict(s=P1), ALIGN, "scales of w"),
    (dict(ld_s=1 << 28), LAYOUT, "2^30"),
    (dict(kind=1), LAYOUT, "ld of w"),
    (dict(kind=0, N=64, K=128, ld_x=128, ld_w=128, ld_out=64), SHAPE, "128"),
    (dict(kind=0, N=128, ld_w=96, ld_out=128), SHAPE, "128"),
    (dict(kind=0, N=256, K=128, ld_x=128, ld_w=128, ld_s=1, ld_out=256), LAYOUT, "K-major"),
    (dict(kind=0, N=128, K=128, ld_x=128, ld_w=128, s=PU, ld_out=128), ALIGN, "scales"),
    (dict(out=None), NULL, "out is NULL"),
    (dict(ld_out=49), LAYOUT, "ld_out"),
    (dict(out=P1), ALIGN, "out"),
    (dict(out=PU, dtype=1), ALIGN, "out"),
    (dict(res=P, ld_res=49), LAYOUT, "ld_res"),
    (dict(res=P1, ld_res=50), ALIGN, "residual"),
])
def test_product_refusals(lib, kw, code, frag):
    call(lib, "bs_few_mm", MM, kw, code, frag)


def test_product_of_nothing(lib):
    for kw in (dict(T=0), dict(N=0), dict(T=0, x=None, w=None, s=None, out=None)):
        call(lib, "bs_few_mm", MM, kw, OK)


MOE = dict(kind=1, T=3, D=96, H=64, E=4, k=2, x=P, ld_x=96, idx=P, w=P, w12=P, stride_w12=128 * 96, ld_w12=96, s12=P,
           stride_s12=3 * 128, ld_s12=128, wo=P, stride_wo=96 * 64, ld_wo=64, so=P, stride_so=2 * 96, ld_so=96, res=None,
           ld_res=0, out=P, ld_out=96, ws=P, nbytes=1 << 24, stream=None)


@pytest.mark.parametrize("kw,code,frag", [
    (dict(kind=-1), MODE, "kind"),
    (dict(T=-1), SHAPE, "T=-1"),
    (dict(T=(1 << 21) + 1), SHAPE, "2^21"),
    (dict(E=0), SHAPE, "E=0"),
    (dict(E=1025), SHAPE, "1024"),
    (dict(k=0), SHAPE, "k=0"),
    (dict(k=5), SHAPE, "min(E, 32)"),
    (dict(E=64, k=33), SHAPE, "min(E, 32)"),
    (dict(D=80), SHAPE, "multiples of 32"),
    (dict(H=0), SHAPE, "multiples of 32"),
    (dict(H=1 << 19), SHAPE, "262144"),
    (dict(kind=0), SHAPE, "multiples of 128"),
    (dict(idx=None), NULL, "E = 1"),
    (dict(idx=PU), ALIGN, "idx"),
    (dict(w=PU), ALIGN, "w must"),
    (dict(x=None), NULL, "x is NULL"),
    (dict(ld_x=80), LAYOUT, "ld_x"),
    (dict(w12=None), NULL, "w12"),
    (dict(s12=None), NULL, "w12"),
    (dict(ld_w12=80), LAYOUT, "w12"),
    (dict(stride_w12=8), ALIGN, "w12"),
    (dict(stride_s12=-16), LAYOUT, "w12"),
    (dict(ld_s12=112), LAYOUT, "w12"),
    (dict(ld_s12=136), ALIGN, "w12"),
    (dict(stride_s12=24), ALIGN, "w12"),
    (dict(wo=None), NULL, "out_proj"),
    (dict(wo=PU), ALIGN, "out_proj"),
    (dict(ld_wo=48), LAYOUT, "out_proj"),
    (dict(ld_so=80), LAYOUT, "out_proj"),
    (dict(res=P, ld_res=95), LAYOUT, "ld_res"),
    (dict(out=None), NULL, "out is NULL"),
    (dict(out=P1), ALIGN, "out"),
    (dict(ld_out=95), LAYOUT, "ld_out"),
    (dict(ws=None), SHAPE, "workspace"),
    (dict(nbytes=767), SHAPE, "the workspace has 767 bytes: this needs 768"),
    (dict(ws=PU), ALIGN, "workspace"),
])
def test_experts_refusals(lib, kw, code, frag):
    call(lib, "bs_moe_few", MOE, kw, code, frag)


def test_experts_of_nothing_and_workspace(lib):
    call(lib, "bs_moe_few", MOE, dict(T=0, x=None, out=None, ws=None, nbytes=0), OK)
    size = lib.bs_moe_few_workspace_bytes
    assert size(3, 96, 64, 4, 2) == 768 and size(0, 96, 64, 4, 1) == 0
    # few columns beside a long contraction: workgroups share them, and leave their sums
    assert size(8, 128, 8192, 16, 8) >= 8 * 8 * 8192 * 2 + 2 * 8 * 128 * 4
    for bad in ((-1, 96, 64, 4, 2), (3, 96, 64, 4, 0), (3, 96, 64, 4, 33), (3, 96, -1, 4, 2), (3, 96, 1 << 19, 4, 2),
                (3, 1 << 19, 64, 4, 2), (3, 96, 64, 0, 2), (3, 96, 64, 1025, 2)):
        assert size(*bad) == 0


def test_binding_refuses_what_it_would_have_to_copy():
    """Tensors on the host and of wrong shapes and types: refused before the library is asked."""
    u8, bf16 = torch.uint8, torch.bfloat16
    x = torch.zeros((3, 96), dtype=bf16)
    w, s = torch.zeros((50, 48), dtype=u8), torch.zeros((3, 64), dtype=u8)
    with pytest.raises(ValueError, match="GPU"):
        bs.bs_few_mm(x, w, s, bs.BS_WEIGHT_MXFP4)
    with pytest.raises(ValueError, match="bfloat16"):
        bs.bs_few_mm(x.float(), w, s, bs.BS_WEIGHT_MXFP4)
    with pytest.raises(ValueError, match="GPU"):
        bs.bs_moe_few(x, None, None, w[None], s[None], w[None], s[None], bs.BS_WEIGHT_MXFP4)
    with pytest.raises(ValueError, match="GPU"):
        bs.bs_mx4_quant_1x32(x, w, s)
