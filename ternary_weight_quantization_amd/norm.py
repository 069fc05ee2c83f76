"""Layer norm before the ternary linear layers, over the C ABI.

``layer_norm`` and ``QATLayerNorm`` normalize the last dimension of a bf16 or
float32 tensor (a residual stream kept in either) and give the bf16
activations that ``QATBitLinear`` and ``TTQLinear`` take. With
``checkpoint=True`` the backward keeps the input in 8 bits (blocks of 128
values share a scale, see ``checkpoint``) instead of the input itself.
torch provides memory and the stream; every step runs in libbitnet.so.
"""

import torch

from . import binding as B


def layer_norm(x, weight=None, bias=None, eps=1e-5, out_dtype=torch.bfloat16, checkpoint=False):
    """The layer norm of x [..., K] (bf16 or float32) over its last dimension
    (K <= 32768), times weight [K] plus bias [K] (bf16 or float32, one dtype;
    each may be None), in out_dtype (bf16, what the linear layers take, or
    float32). ``checkpoint=True`` keeps x in 8 bits for the backward. Gradients:
    dX in x's dtype, those of weight and bias in theirs (differentiable once,
    in reverse mode)."""
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
