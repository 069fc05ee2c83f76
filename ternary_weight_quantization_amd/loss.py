"""The linear layer and the softmax cross entropy at the end of a language
model as one operator, over the C ABI: the loss of bf16 hidden states against
a vocabulary of any size, in pieces of the vocabulary, without keeping the
logits, and the gradients of the hidden states and of the weight. torch
provides memory and the stream; every step runs in libbitnet.so.
"""

import math

import torch
from torch.autograd.function import once_differentiable

from . import binding as B

REDUCTIONS = {"none": B.BITNET_REDUCE_NONE, "sum": B.BITNET_REDUCE_SUM, "mean": B.BITNET_REDUCE_MEAN}


def _aligned(t):
    """t contiguous, starting at a multiple of 16 bytes."""
    t = t.contiguous()
    return t if t.data_ptr() % 16 == 0 else t.clone()


def _forward(h2, w, t, ignore_index, reduce):
    """(result, lse): the rows' losses [T] or their sum or mean []."""
    T, D = h2.shape
    V, dev = w.shape[0], h2.device
    rows = torch.empty((2, T), dtype=torch.float32, device=dev)  # loss, lse
    total = None if reduce == B.BITNET_REDUCE_NONE else torch.empty((), dtype=torch.float32, device=dev)
    L = B.lib()
    n = L.bitnet_xent_fwd_workspace_bytes(T, V, D)
    ws = torch.empty((n,), dtype=torch.uint8, device=dev)
    at = rows.data_ptr()
    B._launch(L.bitnet_xent_fwd, dev.index, h2.data_ptr(), w.data_ptr(), t.data_ptr(), ignore_index, T, V, D, at,
              at + 4 * T, None if total is None else total.data_ptr(), reduce, ws.data_ptr(), n)
    return (rows[0] if total is None else total), rows


class LinearCrossEntropyFunction(torch.autograd.Function):
    """The loss of h [T, D] bf16 against weight [V, D] (bf16 or float32, which
    is rounded to bf16 for the products). Gradients: dh bf16, dweight in the
    weight's dtype."""

    @staticmethod
    def forward(ctx, h, weight, targets, ignore_index, reduce):
        h2 = _aligned(h)
        w = _aligned(weight.to(torch.bfloat16))
        t = targets.contiguous()
        out, rows = _forward(h2, w, t, ignore_index, reduce)
        ctx.save_for_backward(h2, w, t, rows)
        ctx.meta = (ignore_index, reduce, weight.dtype)
        return out.clone() if reduce == B.BITNET_REDUCE_NONE else out

    @staticmethod
    @once_differentiable
    def backward(ctx, dloss):
        h2, w, t, rows = ctx.saved_tensors
        ignore_index, reduce, wt = ctx.meta
        (T, D), V, dev = h2.shape, w.shape[0], h2.device
        need_h, need_w = ctx.needs_input_grad[:2]
        dh = torch.empty((T, D), dtype=torch.bfloat16, device=dev) if need_h else None
        dw = torch.empty((V, D), dtype=wt, device=dev) if need_w else None
        c = dloss.to(torch.float32).contiguous()
        L = B.lib()
        n = L.bitnet_xent_bwd_workspace_bytes(T, V, D)
        ws = torch.empty((n,), dtype=torch.uint8, device=dev)
        B._launch(L.bitnet_xent_bwd, dev.index, h2.data_ptr(), w.data_ptr(), t.data_ptr(), ignore_index,
                  rows.data_ptr() + 4 * T, c.data_ptr(), reduce, T, V, D, None if dh is None else dh.data_ptr(),
                  None if dw is None else dw.data_ptr(), B.BITNET_F32 if wt == torch.float32 else B.BITNET_BF16,
                  ws.data_ptr(), n)
        return dh, dw, None, None, None


def linear_cross_entropy(hidden, weight, targets, ignore_index=-100, reduction="mean"):
    """The softmax cross entropy of the logits hidden @ weight.T against
    targets, without forming the logits: hidden [..., D] bf16, weight [V, D]
    bf16 or float32, int64 targets [...]. Rows whose target is ignore_index
    do not count: their loss and gradients are 0, whatever they hold.
    reduction: "mean" over the rows that count (0 if there are none), "sum",
    or "none" (float32 losses of targets' shape). A target outside 0 .. V-1
    that is not ignore_index gives NaN."""
    if reduction not in REDUCTIONS:
        raise ValueError(f"reduction: expected one of {sorted(REDUCTIONS)}, got {reduction!r}")
    if hidden.dtype != torch.bfloat16:
        raise TypeError(f"linear_cross_entropy expects bf16 hidden states, got {hidden.dtype}")
    if weight.dtype not in (torch.bfloat16, torch.float32):
        raise TypeError(f"weight: expected bfloat16 or float32, got {weight.dtype}")
    if targets.dtype != torch.int64:
        raise TypeError(f"targets: expected torch.int64, got {targets.dtype}")
    if hidden.dim() < 1 or weight.dim() != 2 or weight.shape[1] != hidden.shape[-1] or 0 in weight.shape:
        raise ValueError(f"weight: expected shape (V, {hidden.shape[-1] if hidden.dim() else 'D'}), got {tuple(weight.shape)}")
    if targets.shape != hidden.shape[:-1]:
        raise ValueError(f"targets: expected shape {tuple(hidden.shape[:-1])}, got {tuple(targets.shape)}")
    if not hidden.is_cuda or weight.device != hidden.device or targets.device != hidden.device:
        raise ValueError("hidden, weight and targets: must be GPU tensors of one device")
    reduce, ignore_index = REDUCTIONS[reduction], int(ignore_index)
    h2, t = hidden.reshape(-1, hidden.shape[-1]), targets.reshape(-1)
    if t.shape[0] == 0:
        # no rows: zeros that still depend on both inputs
        zero = h2.sum(dtype=torch.float32) + weight[:0].sum(dtype=torch.float32)
        return zero + torch.zeros(targets.shape, device=hidden.device) if reduction == "none" else zero
    if torch.is_grad_enabled() and (hidden.requires_grad or weight.requires_grad):
        out = LinearCrossEntropyFunction.apply(h2, weight, t, ignore_index, reduce)
    else:
        out = _forward(_aligned(h2), _aligned(weight.to(torch.bfloat16)), t.contiguous(), ignore_index, reduce)[0]
    return out.reshape(targets.shape) if reduction == "none" else out


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
