"""The gated pair of ternary projections of a feed-forward block as one
operator, over the C ABI: act(gate(x)) * up(x) for two ternary weights with a
scale each, both products, the activation and the product in one kernel, and its
straight-through backward. It replaces two ``QATBitLinear`` layers and
``gated_activation`` between a norm and the block's down-projection. torch
provides memory and the stream; every step runs in libbitnet.so.
"""

import math

import torch

from . import binding as B
from .checkpoint import ACTIVATIONS
from .layer import ternarize
from .rows import layer_input


def _act(act):
    code = ACTIVATIONS.get(act)
    if code is None:
        raise ValueError(f"act: expected one of {sorted(ACTIVATIONS)}, got {act!r}")
    return code


def gated_bitlinear(x, w_gate, w_up, act="silu"):
    """act(g) * u in bf16, with g and u the ternary layers of x [..., K] (bf16
    activations, or ``QuantizedRows``) with master weights w_gate and w_up [N, K]
    (bf16 or float32, one dtype), each ternarized with its own scale as
    ``QATBitLinear`` does. act: "silu" (g / (1 + e^-g)) or "relu2" (max(g, 0)^2).
    g and u are not rounded between; the backward keeps the output's derivatives
    with respect to them in 24 bits, the 8-bit rows and the 2-bit weights. Gradients: of x in bf16, of the weights in
    theirs (differentiable once, in reverse mode)."""
    code = _act(act)
    return B.ops().gated_bitlinear(*layer_input(x), w_gate, w_up, code)


def gated_bitlinear_inference(x, w_packed, gamma, in_features, act="silu"):
    """The same from a stored ternary state, e.g. what
    ``QATGatedBitLinear.export_inference`` returns: w_packed uint8 [2N, Kp/4], the
    gate's rows first, and gamma float32 [2]. Differentiable in x; the weights
    get no gradient."""
    code = _act(act)
    return B.ops().gated_bitlinear_inference(*layer_input(x), w_packed, gamma, int(in_features), code)


class QATGatedBitLinear(torch.nn.Module):
    """act(gate(x)) * up(x) for quantization-aware training: master weights
    ``gate_weight`` and ``up_weight`` [out_features, in_features], initialised as
    ``QATBitLinear``'s. ``freeze`` / ``unfreeze`` and ``export_inference`` are
    that layer's too."""

    def __init__(self, in_features, out_features, act="silu", device="cuda", dtype=torch.bfloat16):
        super().__init__()
        _act(act)
        self.in_features = int(in_features)
        self.out_features = int(out_features)
        self.act = act
        for name in ("gate_weight", "up_weight"):
            w = torch.empty((out_features, in_features), dtype=torch.float32)
            torch.nn.init.kaiming_uniform_(w, a=math.sqrt(5))
            self.register_parameter(name, torch.nn.Parameter(w.to(device=device, dtype=dtype)))
        self.register_buffer("_frozen_packed", None)
        self.register_buffer("_frozen_gamma", None)
        self._inference_mode = False

    def forward(self, x):
        if self.frozen:
            return gated_bitlinear_inference(x, self._frozen_packed, self._frozen_gamma, self.in_features, self.act)
        return gated_bitlinear(x, self.gate_weight, self.up_weight, self.act)

    @torch.no_grad()
    def freeze(self):
        """Ternarize both master weights once and run every later forward from
        that; bit for bit the outputs of the training forward at that moment. The
        masters get no gradient while frozen."""
        self._frozen_packed, self._frozen_gamma = self._state()
        self._inference_mode = True
        return self

    def unfreeze(self):
        """Back to training: every forward ternarizes the masters again."""
        self._inference_mode = False
        return self

    @property
    def frozen(self):
        return self._inference_mode and self._frozen_packed is not None

    def _state(self):
        (pg, gg), (pu, gu) = ternarize(self.gate_weight.detach()), ternarize(self.up_weight.detach())
        return torch.cat([pg, pu]), torch.cat([gg, gu])

    @torch.no_grad()
    def export_inference(self):
        """(w_packed uint8 [2 out, Kp/4], gamma float32 [2]), the gate's rows first:
        the frozen state when frozen, else that of the current master weights."""
        return (self._frozen_packed, self._frozen_gamma) if self.frozen else self._state()

    def extra_repr(self):
        r = f"{self.in_features}, {self.out_features}, act={self.act}, dtype={self.gate_weight.dtype}"
        return r + (", frozen=True" if self.frozen else "")
