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
from torch.autograd.function import once_differentiable

from . import binding as B

ACTIVATIONS = {"silu": B.BITNET_ACT_SILU, "relu2": B.BITNET_ACT_RELU2}


def _empty_codes(M, K, device):
    Kc = (K + 127) // 128 * 128
    return (torch.empty((M, Kc), dtype=torch.int8, device=device),
            torch.empty((M, Kc // 128), dtype=torch.float32, device=device))


def _pair_offsets(M, K):
    """Two checkpoints of [M, K] in one buffer: the byte offsets of the first
    one's scales, the second one's codes and scales, and the size."""
    Kc = (K + 127) // 128 * 128
    half = (M * Kc + M * (Kc // 32) + 255) // 256 * 256
    return M * Kc, half, half + M * Kc, 2 * half


@torch.no_grad()
def compress(x):
    """x [..., K] (bf16 or float32) -> (codes int8 [M, Kc], scales float32
    [M, Kc/128]), M the number of rows, Kc = K rounded up to 128."""
    if x.dim() < 1 or x.shape[-1] < 1:
        raise ValueError(f"compress needs a last dimension of at least 1, got {tuple(x.shape)}")
    x2 = x.reshape(-1, x.shape[-1]).contiguous()
    codes, scales = _empty_codes(x2.shape[0], x2.shape[1], x.device)
    if x2.shape[0] > 0:
        B.bitnet_ckpt_pack(x2, codes, scales)
    return codes, scales


@torch.no_grad()
def decompress(codes, scales, K, dtype=torch.bfloat16):
    """The values [M, K] that (codes, scales) stand for, rounded to dtype
    (bf16 or float32)."""
    x = torch.empty((codes.shape[0], int(K)), dtype=dtype, device=codes.device)
    if x.shape[0] > 0:
        B.bitnet_ckpt_unpack(codes, scales, x)
    return x


def _rows(t):
    """t [..., K] as rows [M, K] without a copy where the rows lie at one
    stride (the halves of a [..., 2K] tensor do)."""
    r = t.reshape(-1, t.shape[-1])
    if (r.shape[1] > 1 and r.stride(1) != 1) or (r.shape[0] > 1 and r.stride(0) < r.shape[1]):
        r = r.contiguous()
    return r


class GatedActivationFunction(torch.autograd.Function):
    """y = act(gate) * up (up None: act(gate)), bf16, with the gradients of
    both; checkpoint: gate and up are kept as 8-bit codes."""

    @staticmethod
    def forward(ctx, gate, up, act, checkpoint):
        g = _rows(gate)
        u = None if up is None else _rows(up)
        M, K = g.shape
        y = torch.empty((M, K), dtype=torch.bfloat16, device=gate.device)
        gq = gs = uq = us = kept = None
        if checkpoint:
            s1, q2, s2, size = _pair_offsets(M, K)
            kept = torch.empty((size if u is not None else q2,), dtype=torch.uint8, device=gate.device)
            at = kept.data_ptr()
            gq, gs = at, at + s1
            if u is not None:
                uq, us = at + q2, at + s2
        if M > 0:
            B._launch(B.lib().bitnet_gate_fwd, gate.device.index, act, g.data_ptr(), g.stride(0) if M > 1 else K,
                      None if u is None else u.data_ptr(), K if u is None or M == 1 else u.stride(0), M, K,
                      y.data_ptr(), gq, gs, uq, us)
        if checkpoint:
            ctx.save_for_backward(kept)
        else:
            ctx.save_for_backward(gate, up)
        ctx.meta = (gate.shape, act, checkpoint, up is not None)
        return y.reshape(gate.shape)

    @staticmethod
    @once_differentiable
    def backward(ctx, dy):
        shape, act, checkpoint, gated = ctx.meta
        dY = dy.reshape(-1, shape[-1]).to(torch.bfloat16).contiguous()
        M, K = dY.shape
        dgate = torch.empty_like(dY)
        dup = torch.empty_like(dY) if gated else None
        if M > 0:
            g = u = gq = gs = uq = us = None
            ldg = ldu = K
            if checkpoint:
                kept, = ctx.saved_tensors
                s1, q2, s2, _ = _pair_offsets(M, K)
                at = kept.data_ptr()
                gq, gs = at, at + s1
                if gated:
                    uq, us = at + q2, at + s2
            else:
                gate, up = ctx.saved_tensors
                gr = _rows(gate)
                ur = _rows(up) if gated else None
                g, u = gr.data_ptr(), (ur.data_ptr() if gated else None)
                if M > 1:
                    ldg, ldu = gr.stride(0), (ur.stride(0) if gated else K)
            B._launch(B.lib().bitnet_gate_bwd, dY.device.index, act, dY.data_ptr(), g, ldg, u, ldu, gq, gs, uq, us, M, K,
                      dgate.data_ptr(), K, dup.data_ptr() if gated else None, K)
        return dgate.reshape(shape), (dup.reshape(shape) if gated else None), None, None


def gated_activation(gate, up=None, act="silu", checkpoint=True):
    """act(gate) * up for bf16 gate and up of one shape [..., K] (views with
    rows at one stride, such as the halves of one projection's output, are
    read in place), or act(gate) without up. act: "silu" (g / (1 + e^-g)) or
    "relu2" (max(g, 0)^2). ``checkpoint`` keeps gate and up in 8 bits for the
    backward, else as they are."""
    if act not in ACTIVATIONS:
        raise ValueError(f"act: expected one of {sorted(ACTIVATIONS)}, got {act!r}")
    if gate.dtype != torch.bfloat16 or (up is not None and up.dtype != torch.bfloat16):
        raise TypeError("gated_activation expects bf16 activations")
    if up is not None and up.shape != gate.shape:
        raise ValueError(f"up: expected shape {tuple(gate.shape)}, got {tuple(up.shape)}")
    if gate.dim() < 1 or gate.shape[-1] < 1:
        raise ValueError(f"gated_activation needs a last dimension of at least 1, got {tuple(gate.shape)}")
    if not gate.is_cuda or (up is not None and up.device != gate.device):
        raise ValueError("gate and up: must be GPU tensors of one device")
    needs = torch.is_grad_enabled() and (gate.requires_grad or (up is not None and up.requires_grad))
    if needs:
        return GatedActivationFunction.apply(gate, up, ACTIVATIONS[act], checkpoint)
    g = _rows(gate)
    y = torch.empty(g.shape, dtype=torch.bfloat16, device=gate.device)
    if g.shape[0] > 0:
        B.bitnet_gate_fwd(ACTIVATIONS[act], g, None if up is None else _rows(up), y)
    return y.reshape(gate.shape)
