"""The linear layer and the softmax cross entropy at the end of a language
model as one operator, over the C ABI: the loss of bf16 hidden states against
a vocabulary of any size, in pieces of the vocabulary, without keeping the
logits, and the gradients of the hidden states and of the weight. torch
provides memory and the stream; every step runs in libbitnet.so.
"""

import math

import torch

from . import binding as B
from .rows import need_activations

REDUCTIONS = {"none": B.BITNET_REDUCE_NONE, "sum": B.BITNET_REDUCE_SUM, "mean": B.BITNET_REDUCE_MEAN}


def linear_cross_entropy(hidden, weight, targets, ignore_index=-100, reduction="mean"):
    """The softmax cross entropy of the logits hidden @ weight.T against
    targets, without forming the logits: hidden [..., D] bf16, weight [V, D]
    bf16 or float32 (rounded to bf16 for the products), int64 targets [...].
    Rows whose target is ignore_index do not count: their loss and gradients
    are 0, whatever they hold. reduction: "mean" over the rows that count (0 if
    there are none), "sum", or "none" (float32 losses of targets' shape). A
    target outside 0 .. V-1 that is not ignore_index gives NaN. Gradients: of
    hidden in bf16, of weight in its dtype (differentiable once, in reverse
    mode). Of a float32 weight each call makes a bf16 copy, which is kept until
    the backward."""
    need_activations("linear_cross_entropy", hidden)
    code = REDUCTIONS.get(reduction)
    if code is None:
        raise ValueError(f"reduction: expected one of {sorted(REDUCTIONS)}, got {reduction!r}")
    return B.ops().linear_cross_entropy(hidden, weight, targets, ignore_index, code)


class LinearCrossEntropy(torch.nn.Module):
    """A language model's head with its loss: weight [vocabulary, features],
    kaiming-uniform(a=sqrt(5)) as the linear layers' masters."""

    def __init__(self, features, vocabulary, device="cuda", dtype=torch.bfloat16, ignore_index=-100, reduction="mean"):
        super().__init__()
        self.ignore_index = int(ignore_index)
        self.reduction = reduction
        w = torch.empty((vocabulary, features), dtype=torch.float32)
        torch.nn.init.kaiming_uniform_(w, a=math.sqrt(5))
        self.weight = torch.nn.Parameter(w.to(device=device, dtype=dtype))

    def forward(self, hidden, targets):
        return linear_cross_entropy(hidden, self.weight, targets, self.ignore_index, self.reduction)

    def extra_repr(self):
        V, D = self.weight.shape
        return f"{D}, {V}, dtype={self.weight.dtype}, ignore_index={self.ignore_index}, reduction={self.reduction}"
