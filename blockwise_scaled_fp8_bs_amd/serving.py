"""Weights that a module lays out once for serving, and what few tokens take
instead of the GEMMs.

The layers' GEMMs are built for hundreds of rows.  A module that was prepared
for serving answers up to ``few_tokens`` tokens by ``bs_few_mm`` or
``bs_moe_few``: the quantized weights are read once and meet the tokens in
bf16, which are not quantized, so that the result is nearer to the unquantized
layer's than the GEMMs' is.  More tokens take the GEMMs, on the same weights.
"""

import torch
from torch.autograd import forward_ad

from . import binding as _b
from . import binding_few as _f

#: tokens up to which a module prepared for serving takes the few-token calls, narrow dense layers, gated FFNs and
#: experts in 4 bits.  In us, these and the quantizers with the GEMMs: a layer of 8192 x 5120 17 and 63 for 64 tokens, 32
#: and 65 for 128, 62 and 70 for 256, 120 and 71 for 512; a gated FFN of 5120 and 8192 58 and 161, 110 and 165, 184 and
#: 171; 16 experts of 2048 and 1024, top 4, 47 and 92, 67 and 92, 112 and 95.
FEW_TOKENS = 128


def few_tokens_of(columns):
    """The same of a dense layer with that many outputs.

    The few-token kernel takes a round of the CUs for 8192 of them (and 64 tokens), the GEMM for 65536, about four times
    as long; from 32768 on both are bound by the bytes of the weights.  In us, weights from memory: 16384 x 5120 40 and
    82 for 64 tokens, 68 and 87 for 128; 24576 x 5120 58 and 83, 104 and 89; 32768 x 5120 76 and 85, 136 and 91; 65536 x
    5120 91 and 93 for 17 tokens, 105 and 93 for 32, 147 and 95 for 64.
    """
    rounds = -(-columns // 8192) / max(1, -(-columns // 65536))
    return FEW_TOKENS if rounds <= 2 else 64 if rounds <= 4 else 32 if rounds <= 6 else 16


class ServedWeights:
    """Mixin of modules that lay out weights for serving.

    The layout holds for the tensors that it was made of, their memory and
    their versions: other weights (assigned since, or passed for one call by
    ``torch.func.functional_call``) have none, and the same ones written in
    place or given other memory raise.  It goes by autograd's version counter:
    what writes past that (through ``.data``, in a collective, in a kernel of
    one's own) is not seen, and needs prepare_serving() again.  train(), moving
    the module and loading a state drop the layout, and a copy has none.

    A pass captured into a graph reads the memory of the layout that was there,
    whose checks a replay does not repeat: capture it again after
    prepare_serving(), and do not replay it once the layout was dropped, when
    that memory may hold something else.
    """

    _serving = _served = None
    _served_names = ()      # parameters that the layout is made of

    def _lay_out(self, layout):
        """Keeps layout(*weights) as that of the present weights."""
        weights = [getattr(self, n) for n in self._served_names]
        if any(p.is_inference() for p in weights):
            raise RuntimeError("the weights are inference tensors, whose changes nothing counts: make or load the module "
                               "outside torch.inference_mode()")
        with torch.no_grad():
            self._serving = layout(*weights)
        # the tensors, their memory (an alias, so that its address is not handed out again) and their versions
        self._served = [(p, p.detach(), p._version) for p in weights]
        return self

    def _layout(self):
        """The layout if it is that of the present weights, None if there is none of them."""
        if self._serving is None or any(getattr(self, n) is not p for n, (p, _, _) in zip(self._served_names, self._served)):
            return None
        if any(p._version != version or not p.is_set_to(memory) for p, memory, version in self._served):
            raise RuntimeError("the weights changed after prepare_serving(): call it again")
        return self._serving

    def _layout_for(self, *inputs):
        """The layout to answer these inputs with: None also where gradients are on.
        Forward-mode tangents raise, as in training: the kernels would drop them."""
        layout = None if torch.is_grad_enabled() else self._layout()
        if layout is not None and any(t is not None and forward_ad.unpack_dual(t).tangent is not None for t in inputs):
            raise RuntimeError("forward-mode AD is not supported: the input has a tangent, which would be lost")
        return layout

    def _drop_layout(self):
        self._serving = self._served = None

    def __getstate__(self):
        return dict(self.__dict__, _serving=None, _served=None)

    def train(self, mode=True):
        if mode:
            self._drop_layout()
        return super().train(mode)

    def _apply(self, fn, *args, **kw):
        self._drop_layout()
        return super()._apply(fn, *args, **kw)

    def _load_from_state_dict(self, *args, **kw):
        self._drop_layout()
        return super()._load_from_state_dict(*args, **kw)


def check_formats(weights, few_tokens, formats):
    if weights not in formats:
        raise ValueError(f"weights must be one of {list(formats)}, got {weights!r}")
    if few_tokens < 0:
        raise ValueError(f"few_tokens = {few_tokens} must not be negative")


def rows_128(w):
    """128x128 codes [N, K] and scales [K/128, >= N/128] of w [N, K]."""
    N, K = w.shape
    q = torch.empty((N, K), dtype=torch.uint8, device=w.device)
    s = _b.empty_scales(K // 128, N // 128, w.device)
    _b.bs_quant_128x128(w, q, s)
    return q, s


def rows_mx8(w):
    """MXFP8 codes [N, K] and scale bytes [K/32, >= N] of w [N, K]."""
    N, K = w.shape
    q = torch.empty((N, K), dtype=torch.uint8, device=w.device)
    s = _b.empty_mx_scales(K // 32, N, w.device)
    _b.bs_mx_quant_1x32(w, q, s)
    return q, s


def rows_mx4(w, values=False):
    """MXFP4 codes [N, K/2] and scale bytes [K/32, >= N] of w [N, K], and with
    `values` the bf16 weights that they stand for (None without)."""
    N, K = w.shape
    q = torch.empty((N, K // 2), dtype=torch.uint8, device=w.device)
    s = _b.empty_mx_scales(K // 32, N, w.device)
    y = torch.empty_like(w) if values else None
    _f.bs_mx4_quant_1x32(w, q, s, y=y)
    return q, s, y


def experts_mx4(w):
    """rows_mx4 of expert weights w [E, N, K], with values: codes [E, N, K/2],
    scale bytes [E, K/32, N] (N a multiple of 16), bf16 [E, N, K]."""
    E, N, K = w.shape
    q, s, y = rows_mx4(w.view(E * N, K), values=True)
    return q.view(E, N, K // 2), torch.as_strided(s, (E, K // 32, N), (N, s.stride(0), 1)), y.view(E, N, K)


def quantized_rows(x2):
    """1x128 codes and scales of x2 [R, C] along rows alone."""
    R, C = x2.shape
    q = torch.empty((R, C), dtype=torch.uint8, device=x2.device)
    s = _b.empty_scales(C // 128, R, x2.device)
    _b.bs_quant_1x128(x2, q, s)
    return q, s


def token_rows(x, features):
    """x [..., features] (contiguous bf16 on a GPU) as [T, features]."""
    if x.dtype != torch.bfloat16:
        raise ValueError(f"x must be bfloat16, got {x.dtype}")
    if x.shape[-1] != features:
        raise ValueError(f"x has {x.shape[-1]} features, the layer expects {features}")
    if not x.is_contiguous():
        raise ValueError("x must be contiguous (row-major); pass a contiguous tensor instead of relying on a copy")
    if not x.is_cuda:
        raise ValueError("x must be a GPU tensor")
    return x.view(-1, features)


__all__ = ["FEW_TOKENS", "ServedWeights", "check_formats", "experts_mx4", "few_tokens_of", "quantized_rows", "rows_128", "rows_mx4",
           "rows_mx8", "token_rows"]
