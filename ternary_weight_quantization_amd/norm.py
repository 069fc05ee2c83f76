"""Layer norm and root-mean-square norm before the ternary linear layers, over
the C ABI.

``layer_norm`` and ``QATLayerNorm`` normalize the last dimension of a bf16 or
float32 tensor (a residual stream kept in either) and give the bf16
activations that ``QATBitLinear`` and ``TTQLinear`` take. With
``checkpoint=True`` the backward keeps the input in 8 bits (blocks of 128
values share a scale, see ``checkpoint``) instead of the input itself.
``rms_norm`` and ``QATRMSNorm`` add the residual on the way and give bf16
activations or the 8-bit rows (``rows``) that the layers multiply. torch provides memory and the stream; every step runs in libbitnet.so.
"""

import torch

from . import binding as B
from .rows import QuantizedRows, need_activations


def layer_norm(x, weight=None, bias=None, eps=1e-5, out_dtype=torch.bfloat16, checkpoint=False):
    """The layer norm of x [..., K] (bf16 or float32) over its last dimension
    (K <= 32768), times weight [K] plus bias [K] (bf16 or float32, one dtype;
    each may be None), in out_dtype (bf16, what the linear layers take, or
    float32). ``checkpoint=True`` keeps x in 8 bits for the backward. Gradients:
    dX in x's dtype, those of weight and bias in theirs (differentiable once,
    in reverse mode)."""
    need_activations("layer_norm", x)
    return B.ops().layer_norm(x, weight, bias, eps, out_dtype, checkpoint)


class QATLayerNorm(torch.nn.Module):
    """Layer norm with a learned weight (ones) and, with bias=True, a learned
    bias (zeros), whose bf16 output feeds the ternary linear layers."""

    def __init__(self, features, eps=1e-5, bias=True, device="cuda", dtype=torch.bfloat16, checkpoint=False):
        super().__init__()
        self.features = int(features)
        self.eps = eps
        self.checkpoint = checkpoint
        self.weight = torch.nn.Parameter(torch.ones(features, device=device, dtype=dtype))
        self.bias = torch.nn.Parameter(torch.zeros(features, device=device, dtype=dtype)) if bias else None

    def forward(self, x):
        return layer_norm(x, self.weight, self.bias, eps=self.eps, checkpoint=self.checkpoint)

    def extra_repr(self):
        return (f"{self.features}, eps={self.eps}, dtype={self.weight.dtype}, bias={self.bias is not None}"
                + (", checkpoint=True" if self.checkpoint else ""))


def rms_norm(x, weight=None, residual=None, eps=1e-6, out_dtype=torch.bfloat16, quantize=False):
    """The root-mean-square norm over the last dimension (K <= 16384) of h = x, or
    of h = residual + x rounded to the residual's dtype, times weight [K] (bf16 or
    float32, or None). x [..., K]: bf16 or float32, beside a residual of the same
    shape bf16 or the residual's dtype. Returns the norm's output, or with a
    residual (output, h), h being the stream for what follows. The output is a
    tensor in out_dtype (bf16 or float32) or, with ``quantize``, the
    ``QuantizedRows`` that the layers take, made from the norm's float32 values.
    Gradients, straight through the quantization: of x, residual and weight in
    their dtypes (differentiable once, in reverse mode)."""
    need_activations("rms_norm", x)
    y, codes, scales, h = B.ops().rms_norm(x, weight, residual, eps, bool(quantize), out_dtype)
    if quantize:
        y = QuantizedRows(codes, scales, y)
    return y if residual is None else (y, h)


class QATRMSNorm(torch.nn.Module):
    """Root-mean-square norm with a learned weight (ones); with quantize=True its
    output is the 8-bit rows that the linear layers take. ``norm(x)`` gives the
    output, ``norm(x, residual)`` the output and the new stream."""

    def __init__(self, features, eps=1e-6, device="cuda", dtype=torch.bfloat16, quantize=False):
        super().__init__()
        self.features = int(features)
        self.eps = eps
        self.quantize = quantize
        self.weight = torch.nn.Parameter(torch.ones(features, device=device, dtype=dtype))

    def forward(self, x, residual=None):
        return rms_norm(x, self.weight, residual, eps=self.eps, quantize=self.quantize)

    def extra_repr(self):
        return (f"{self.features}, eps={self.eps}, dtype={self.weight.dtype}"
                + (", quantize=True" if self.quantize else ""))
