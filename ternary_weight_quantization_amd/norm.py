"""Layer norm before the ternary linear layers, over the C ABI.

``layer_norm`` and ``QATLayerNorm`` normalize the last dimension of a bf16 or
float32 tensor (a residual stream kept in either) and give the bf16
activations that ``QATBitLinear`` and ``TTQLinear`` take. With
``checkpoint=True`` the backward keeps the input in 8 bits (blocks of 128
values share a scale, see ``checkpoint``) instead of the input itself.
torch provides memory and the stream; every step runs in libbitnet.so.
"""

import torch
from torch.autograd.function import once_differentiable

from . import binding as B
from .checkpoint import _empty_codes


_DTYPES = {torch.bfloat16: B.BITNET_BF16, torch.float32: B.BITNET_F32}


def _ptr(t):
    return None if t is None else t.data_ptr()


def _params(x, weight, bias):
    """(weight, bias) contiguous and their dtype's number, checked against x."""
    K, pd = x.shape[-1], None
    out = []
    for name, t in (("weight", weight), ("bias", bias)):
        if t is not None:
            if t.dtype not in _DTYPES or (pd is not None and _DTYPES[t.dtype] != pd):
                raise TypeError(f"{name}: expected bf16 or float32, one dtype for weight and bias, got {t.dtype}")
            if t.dim() != 1 or t.shape[0] != K:
                raise ValueError(f"{name}: expected shape {(K,)}, got {tuple(t.shape)}")
            if t.device != x.device:
                raise ValueError(f"{name}: on {t.device}, expected {x.device}")
            pd = _DTYPES[t.dtype]
            t = t.contiguous()
        out.append(t)
    return out[0], out[1], (B.BITNET_F32 if pd is None else pd)


class LayerNormFunction(torch.autograd.Function):
    """y = LayerNorm(x) * weight + bias over the last dimension. Gradients:
    dX in x's dtype, dweight and dbias in theirs."""

    @staticmethod
    def forward(ctx, x, weight, bias, eps, out_dtype, checkpoint):
        K = x.shape[-1]
        x2 = x.reshape(-1, K).contiguous()
        w, b, pd = _params(x, weight, bias)
        M, dev = x2.shape[0], x2.device
        y = torch.empty((M, K), dtype=out_dtype, device=dev)
        stats = torch.empty((2, M), dtype=torch.float32, device=dev)  # mu, r
        codes = scales = None
        if checkpoint:
            codes, scales = _empty_codes(M, K, dev)
        if M > 0:
            at = stats.data_ptr()
            B._launch(B.lib().bitnet_layernorm_fwd, dev.index, x2.data_ptr(), _DTYPES[x2.dtype], _ptr(w), _ptr(b), pd, M,
                      K, eps, y.data_ptr(), _DTYPES[out_dtype], at, at + 4 * M, _ptr(codes), _ptr(scales))
        ctx.save_for_backward(None if checkpoint else x2, codes, scales, w, stats)
        ctx.meta = (x.shape, x.dtype, out_dtype, pd)
        return y.reshape(x.shape)

    @staticmethod
    @once_differentiable
    def backward(ctx, dy):
        x2, codes, scales, w, stats = ctx.saved_tensors
        shape, xt, yt, pd = ctx.meta
        K, dev = shape[-1], dy.device
        dY = dy.reshape(-1, K).to(yt).contiguous()
        M = dY.shape[0]
        need_x, need_w, need_b = ctx.needs_input_grad[:3]
        pt = torch.float32 if pd == B.BITNET_F32 else torch.bfloat16
        make = torch.empty if M > 0 else torch.zeros
        dX = make((M, K), dtype=xt, device=dev) if need_x else None
        dw = make((K,), dtype=pt, device=dev) if need_w else None
        db = make((K,), dtype=pt, device=dev) if need_b else None
        if M > 0:
            L, ws, n = B.lib(), None, 0
            if need_w or need_b:
                n = L.bitnet_layernorm_workspace_bytes(M, K)
                ws = torch.empty((n,), dtype=torch.uint8, device=dev)
            at = stats.data_ptr()
            B._launch(L.bitnet_layernorm_bwd, dev.index, dY.data_ptr(), _DTYPES[yt], _ptr(x2), _DTYPES[xt], _ptr(codes),
                      _ptr(scales), _ptr(w), pd, at, at + 4 * M, M, K, _ptr(dX), _ptr(dw), _ptr(db), _ptr(ws), n)
        return (None if dX is None else dX.reshape(shape)), dw, db, None, None, None


def layer_norm(x, weight=None, bias=None, eps=1e-5, out_dtype=torch.bfloat16, checkpoint=False):
    """The layer norm of x [..., K] (bf16 or float32) over its last dimension
    (K <= 32768), times weight [K] plus bias [K] (bf16 or float32, one dtype;
    each may be None), in out_dtype (bf16, what the linear layers take, or
    float32). ``checkpoint=True`` keeps x in 8 bits for the backward."""
    if x.dtype not in _DTYPES:
        raise TypeError(f"layer_norm expects bf16 or float32 activations, got {x.dtype}")
    if out_dtype not in _DTYPES:
        raise TypeError(f"out_dtype: expected bfloat16 or float32, got {out_dtype}")
    if x.dim() < 1 or x.shape[-1] < 1:
        raise ValueError(f"layer_norm needs a last dimension of at least 1, got {tuple(x.shape)}")
    if not x.is_cuda:
        raise ValueError("x: must be a GPU tensor")
    if torch.is_grad_enabled() and (x.requires_grad or (weight is not None and weight.requires_grad)
                                    or (bias is not None and bias.requires_grad)):
        return LayerNormFunction.apply(x, weight, bias, eps, out_dtype, checkpoint)
    x2 = x.reshape(-1, x.shape[-1]).contiguous()
    w, b, pd = _params(x, weight, bias)
    M, K = x2.shape
    y = torch.empty(x.shape, dtype=out_dtype, device=x.device)
    if M > 0:
        B._launch(B.lib().bitnet_layernorm_fwd, x.device.index, x2.data_ptr(), _DTYPES[x2.dtype], _ptr(w), _ptr(b), pd,
                  M, K, eps, y.data_ptr(), _DTYPES[out_dtype], None, None, None, None)
    return y


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
