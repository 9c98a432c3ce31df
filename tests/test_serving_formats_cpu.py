"""What layers prepared for serving keep of each format: no GPU, the quantizers are stood in for."""

import pytest
import torch

import blockwise_scaled_fp8_bs_amd as bs
from blockwise_scaled_fp8_bs_amd import moe, serving

LAYERS = {"linear": lambda: bs.Float8BlockwiseLinear(128, 128), "mx": lambda: bs.Float8MXLinear(128, 128),
          "ffn": lambda: bs.Float8BlockwiseGatedFFN(128, 512), "moe": lambda: bs.Float8BlockwiseMoE(128, 128, 4, 2)}
EIGHT = {"linear": bs.BS_WEIGHT_E4M3_128X128, "mx": bs.BS_WEIGHT_MXFP8, "ffn": bs.BS_WEIGHT_E4M3_128X128,
         "moe": bs.BS_WEIGHT_E4M3_128X128}


@pytest.fixture
def quantizers(monkeypatch):
    """Codes of 4 bits are full of fours, those of 8 bits hold the sum of what they were made of."""
    eight = lambda w: (torch.full((*w.shape[:-1], 1), float(w.float().sum())), torch.ones(1))  # noqa: E731
    monkeypatch.setattr(serving, "rows_128", eight)
    monkeypatch.setattr(serving, "rows_mx8", eight)
    monkeypatch.setattr(moe, "_expert_weights", lambda w: eight(w) + (None,))
    four = lambda w, values=True: (torch.full((*w.shape[:-1], 1), 4.0), torch.ones(1), torch.full_like(w, 0.5))  # noqa: E731
    monkeypatch.setattr(serving, "rows_mx4", four)
    monkeypatch.setattr(serving, "experts_mx4", four)


def _fours(layout):
    return sum(isinstance(t, torch.Tensor) and bool((t == 4.0).all()) for t in layout)


@pytest.mark.parametrize("name", LAYERS)
def test_codes_of_four_bits_are_kept_where_a_pass_reads_them(name, quantizers):
    m = LAYERS[name]()
    weights = 2 if name in ("ffn", "moe") else 1
    layout = m.prepare_serving("mxfp4")._serving
    assert layout[-1] == serving.FEW_TOKENS and layout[-2] == bs.BS_WEIGHT_MXFP4 and _fours(layout) == weights
    # without few tokens: the same values for the GEMMs, and nothing of 4 bits
    none = m.prepare_serving("mxfp4", few_tokens=0)._serving
    assert none[-1] == 0 and none[-2] == EIGHT[name] and _fours(none) == 0 and len(none) == len(layout)
    n = 2 * weights
    assert all(torch.equal(a, b) for a, b in zip(layout[:n], none[:n]))
    # a pass of no tokens takes the codes of 8 bits that are there
    assert all(torch.equal(a.flatten(), b.flatten()) for a, b in zip(none[:n], none[n:2 * n]))


@pytest.mark.parametrize("name", LAYERS)
def test_formats_of_training(name, quantizers):
    layout = LAYERS[name]().prepare_serving()._serving
    assert _fours(layout) == 0 and layout[-2] == EIGHT[name]
    assert layout[-1] == (0 if name == "moe" else serving.FEW_TOKENS)
    assert LAYERS[name]().prepare_serving(few_tokens=7)._serving[-1] == 7


def test_few_tokens_of_wide_layers(quantizers):
    """Less of them by default where the GEMM, in one round, is faster than several of the few-token kernel."""
    for columns, tokens in ((128, 128), (16384, 128), (16512, 64), (32768, 64), (32896, 32), (49152, 32), (65536, 16), (131072, 16)):
        assert serving.few_tokens_of(columns) == tokens
        for cls in (bs.Float8BlockwiseLinear, bs.Float8MXLinear):
            m = cls(128, columns)
            assert m.prepare_serving()._serving[-1] == tokens and m.prepare_serving("mxfp4")._serving[-1] == tokens
            assert m.prepare_serving(few_tokens=100)._serving[-1] == 100
