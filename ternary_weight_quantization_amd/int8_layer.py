"""Linear layers in 8-bit integers over the C ABI: activations with a scale per
token, weights with a scale per output channel. What a model of ternary layers
keeps out of them (its head, say) runs on the same 8-bit rows and the same
integer matrix cores. Training quantizes master weights in every forward, as the
ternary layers do, with straight-through gradients; a frozen layer keeps the
8-bit weights. torch provides memory and the stream; every step runs in
libbitnet.so.
"""

import math

import torch

from . import binding as B
from .rows import layer_input


def int8_linear(x, weight, bias=None):
    """x @ weight.T (+ bias) in bf16, both operands quantized to 8 bits: x [..., K]
    (bf16 activations, or ``QuantizedRows``) with a scale per row, weight [N, K]
    (bf16 or float32 masters) with a scale per row (channel), each the row's
    largest magnitude over 127; bias [N] bf16 or float32 (rounded to bf16), added
    before the output's rounding. K <= 131072. Gradients, straight through both
    quantizations: of x in bf16, of weight and bias in their dtypes
    (differentiable once, in reverse mode). Their products take both quantized
    operands rounded to bf16, those of float32 masters too: gradients are about
    0.0025 of their norm off exact ones, where fp32 products would be 0.0017. With widths rounded up to 64, the forward
    takes (rows + 256) * K <= 2^31 for the rows of x and of weight; where gradients
    are wanted (rows + 256) * 2 * width <= 2^31 has to hold for x, weight and
    the output, and a call past that raises before it computes."""
    return B.ops().int8_linear(*layer_input(x), weight, bias)


def int8_linear_inference(x, w_q, s_w, in_features, bias=None):
    """The same from stored 8-bit weights, e.g. what
    ``QATInt8Linear.export_inference`` returns: w_q int8 [N, Kp] (Kp = in_features
    rounded up to 64, zeros past in_features), s_w float32 [N], a channel's largest
    magnitude. Differentiable in x and bias, within int8_linear's sizes."""
    return B.ops().int8_linear_inference(*layer_input(x), w_q, s_w, int(in_features), bias)


class QATInt8Linear(torch.nn.Module):
    """8-bit linear layer for quantization-aware training: master weights
    [out_features, in_features] in bf16 (or float32), initialised as
    ``QATBitLinear``'s, and with bias=True a zero-initialised bf16 bias.
    ``from_linear``, ``freeze`` / ``unfreeze`` and ``export_inference`` are that
    layer's too."""

    def __init__(self, in_features, out_features, device="cuda", dtype=torch.bfloat16, bias=False):
        super().__init__()
        self.in_features = int(in_features)
        self.out_features = int(out_features)
        w = torch.empty((out_features, in_features), dtype=torch.float32)
        torch.nn.init.kaiming_uniform_(w, a=math.sqrt(5))
        self.weight = torch.nn.Parameter(w.to(device=device, dtype=dtype))
        self.bias = (torch.nn.Parameter(torch.zeros(out_features, device=device, dtype=torch.bfloat16))
                     if bias else None)
        self.register_buffer("_frozen_q", None)
        self.register_buffer("_frozen_s", None)
        self._inference_mode = False

    @classmethod
    def from_linear(cls, linear, dtype=torch.bfloat16):
        m = cls(linear.in_features, linear.out_features, device=linear.weight.device, dtype=dtype,
                bias=linear.bias is not None)
        with torch.no_grad():
            m.weight.copy_(linear.weight.to(dtype))
            if linear.bias is not None:
                m.bias.copy_(linear.bias.to(torch.bfloat16))
        return m

    def forward(self, x):
        if self.frozen:
            return int8_linear_inference(x, self._frozen_q, self._frozen_s, self.in_features, self.bias)
        return int8_linear(x, self.weight, self.bias)

    @torch.no_grad()
    def freeze(self):
        """Quantize the master weights once and run every later forward from
        that; bit for bit the outputs of the training forward at that moment. The
        masters get no gradient while frozen."""
        self._frozen_q, self._frozen_s = B.ops().int8_quantize_weight(self.weight.detach())
        self._inference_mode = True
        return self

    def unfreeze(self):
        """Back to training: every forward quantizes the masters again."""
        self._inference_mode = False
        return self

    @property
    def frozen(self):
        return self._inference_mode and self._frozen_q is not None

    @torch.no_grad()
    def export_inference(self):
        """(w_q int8 [out, Kp], s_w float32 [out]): the frozen state when frozen,
        else that of the current master weights."""
        if self.frozen:
            return self._frozen_q, self._frozen_s
        return B.ops().int8_quantize_weight(self.weight.detach())

    def extra_repr(self):
        r = f"{self.in_features}, {self.out_features}, dtype={self.weight.dtype}, bias={self.bias is not None}"
        return r + (", frozen=True" if self.frozen else "")
