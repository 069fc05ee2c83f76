"""Activations kept in 8 bits between the forward and the backward pass, over
the C ABI.

Each 128 consecutive values of a row share a float32 scale, their largest
magnitude s, and every value is kept as the int8 code
round_half_even(127 x / s): 1.03 bytes a value. ``compress`` and
``decompress`` convert whole tensors; ``gated_activation`` is the activation
of a feed-forward block whose backward reads the codes of its inputs. The
layer norm (``norm``) and the trained-ternary linear layer (``ttq_layer``)
keep their inputs the same way with ``checkpoint=True``. ``QATBitLinear``
always does: its backward reads the int8 activations of its forward.
"""

import torch

from . import binding as B

ACTIVATIONS = {"silu": B.BITNET_ACT_SILU, "relu2": B.BITNET_ACT_RELU2}


def compress(x):
    """x [..., K] (bf16 or float32) -> (codes int8 [M, Kc], scales float32
    [M, Kc/128]), M the number of rows, Kc = K rounded up to 128."""
    return B.ops().compress(x)


def decompress(codes, scales, K, dtype=torch.bfloat16):
    """The values [M, K] that (codes, scales) stand for, rounded to dtype
    (bf16 or float32)."""
    return B.ops().decompress(codes, scales, K, dtype)


def gated_activation(gate, up=None, act="silu", checkpoint=True):
    """act(gate) * up for bf16 gate and up of one shape [..., K] (views with
    rows at one stride, such as the halves of one projection's output, are
    read in place), or act(gate) without up. act: "silu" (g / (1 + e^-g)) or
    "relu2" (max(g, 0)^2). ``checkpoint``, the default, keeps gate and up in 8
    bits for the backward: the gradients are then those at the codes' values,
    which are off by up to 1/254 of their block's largest magnitude. With
    ``checkpoint=False`` both are kept as they are. Differentiable once, in
    reverse mode."""
    code = ACTIVATIONS.get(act)
    if code is None:
        raise ValueError(f"act: expected one of {sorted(ACTIVATIONS)}, got {act!r}")
    return B.ops().gated_activation(gate, up, code, checkpoint)
