"""The C entry points around the experts' products on no rows: codes without
elements may be NULL beside scales that were made for more."""

import pytest

from blockwise_scaled_fp8_bs_amd import _lib
from test_block_cpu import GATHER, NORM, NULL, OK, P, call


@pytest.mark.parametrize("name,defaults,kw", [
    ("bs_moe_gather_quant_1x128", GATHER, dict(M=0, q_row=None)),
    ("bs_moe_gather_quant_1x128", GATHER, dict(M=0, q_row=None, q_col=None)),
    ("bs_moe_gather_quant_1x128", GATHER, dict(M=0, T=0, x=None, row_slot=None, q_row=None, q_col=None, s_col=None)),
    ("bs_resid_norm", NORM, dict(R=0, q_row=None)),
    ("bs_resid_norm", NORM, dict(R=0, per=1, x=None, u=None, r=None, rstd_u=None, q_row=None, q_col=None, s_col=None)),
])
def test_no_rows(name, defaults, kw):
    lib = _lib.load()
    assert getattr(lib, name)(*dict(defaults, **kw).values()) == OK, lib.bs_last_error()


def test_rows_still_need_both():
    call(_lib.load(), "bs_moe_gather_quant_1x128", GATHER, dict(q_col=None), NULL, "q_col and s_col")
    call(_lib.load(), "bs_resid_norm", NORM, dict(s_row=None), NULL, "q_row and s_row")
    assert GATHER["s_row"] == NORM["s_row"] == P
