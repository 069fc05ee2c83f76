"""Refusals of the layer norm, 8-bit checkpoint, gated activation and cross
entropy entry points without a GPU: the C ABI rejects bad arguments with the documented
codes before touching the device, and the Python entry points raise before
they call it."""

import ctypes
import os

import pytest
import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
LIB = os.path.join(ROOT, "ternary_weight_quantization_amd", "libbitnet.so")
OK, ENULL, ESHAPE, EDTYPE, EALIGN, EWS, EHIP = range(7)
P = 1 << 20  # a stand-in device address, aligned; never dereferenced
BF, F32, SIGN1 = 0, 1, 2


@pytest.fixture(scope="module")
def L():
    if not os.path.exists(LIB):
        pytest.fail("libbitnet.so is not built (run `python -m ternary_weight_quantization_amd.build`)")
    from ternary_weight_quantization_amd import binding
    return binding.lib()


def test_layernorm_fwd_refusals(L):
    def f(x=P, xd=BF, w=P, b=P, pd=BF, M=4, K=64, y=P, yd=BF, mean=P, rstd=P, codes=None, scales=None):
        return L.bitnet_layernorm_fwd(x, xd, w, b, pd, M, K, 1e-5, y, yd, mean, rstd, codes, scales, None)

    assert f(x=None) == ENULL and f(y=None) == ENULL and f(codes=P) == ENULL
    assert f(xd=SIGN1) == EDTYPE and f(yd=SIGN1) == EDTYPE and f(pd=7) == EDTYPE
    assert f(M=0) == ESHAPE and f(K=0) == ESHAPE and f(K=32769) == ESHAPE and f(M=(1 << 30) + 1) == ESHAPE
    assert f(x=P + 1) == EALIGN and f(x=P + 2, xd=F32) == EALIGN and f(w=P + 2, pd=F32) == EALIGN
    assert f(y=P + 1) == EALIGN and f(mean=P + 2) == EALIGN and f(codes=P + 8, scales=P) == EALIGN
    assert f(codes=P, scales=P + 2) == EALIGN


def test_layernorm_bwd_refusals(L):
    need = L.bitnet_layernorm_workspace_bytes(4, 64)
    assert need > 0

    def f(dY=P, yd=BF, x=P, xd=BF, codes=None, scales=None, w=P, pd=BF, mean=P, rstd=P, M=4, K=64, dX=P, dw=P, db=P,
          ws=P, n=need):
        return L.bitnet_layernorm_bwd(dY, yd, x, xd, codes, scales, w, pd, mean, rstd, M, K, dX, dw, db, ws, n, None)

    assert f(dY=None) == ENULL and f(mean=None) == ENULL and f(rstd=None) == ENULL and f(x=None) == ENULL
    assert f(x=None, codes=P) == ENULL and f(dX=None, dw=None, db=None) == ENULL
    assert f(yd=SIGN1) == EDTYPE and f(xd=SIGN1) == EDTYPE and f(pd=SIGN1) == EDTYPE
    assert f(K=32769) == ESHAPE and f(M=0) == ESHAPE
    assert f(ws=None) == EWS and f(n=need - 1) == EWS and f(ws=P + 8) == EALIGN
    assert f(dX=P + 1) == EALIGN and f(dw=P + 2, pd=F32) == EALIGN and f(codes=P + 4, scales=P) == EALIGN
    assert L.bitnet_layernorm_workspace_bytes(0, 64) == 0 and L.bitnet_layernorm_workspace_bytes(4, 32769) == 0
    # two rows of partial sums a block, at most one block per 4 rows of up to 2560
    assert need == 2 * 64 * 4
    assert L.bitnet_layernorm_workspace_bytes(9, 64) == 3 * 2 * 64 * 4


def test_checkpoint_refusals(L):
    assert L.bitnet_ckpt_pad(1) == 128 and L.bitnet_ckpt_pad(128) == 128 and L.bitnet_ckpt_pad(129) == 256
    assert L.bitnet_ckpt_pad(0) == 0

    def pack(x=P, d=BF, M=4, K=64, c=P, s=P):
        return L.bitnet_ckpt_pack(x, d, M, K, c, s, None)

    def unpack(x=P, d=BF, M=4, K=64, c=P, s=P):
        return L.bitnet_ckpt_unpack(c, s, M, K, x, d, None)

    for f in (pack, unpack):
        assert f(x=None) == ENULL and f(c=None) == ENULL and f(s=None) == ENULL
        assert f(d=SIGN1) == EDTYPE
        assert f(M=0) == ESHAPE and f(K=0) == ESHAPE and f(K=(1 << 24) + 1) == ESHAPE
        assert f(M=1 << 30, K=2048) == ESHAPE
        assert f(x=P + 1) == EALIGN and f(x=P + 2, d=F32) == EALIGN and f(c=P + 8) == EALIGN and f(s=P + 2) == EALIGN


def test_gate_refusals(L):
    def fwd(act=0, g=P, ldg=64, u=P, ldu=64, M=4, K=64, y=P, gq=None, gs=None, uq=None, us=None):
        return L.bitnet_gate_fwd(act, g, ldg, u, ldu, M, K, y, gq, gs, uq, us, None)

    assert fwd(g=None) == ENULL and fwd(y=None) == ENULL and fwd(gq=P) == ENULL and fwd(gq=P, gs=P) == ENULL
    assert fwd(act=2) == EDTYPE and fwd(act=-1) == EDTYPE
    assert fwd(ldg=63) == ESHAPE and fwd(ldu=63) == ESHAPE and fwd(M=0) == ESHAPE and fwd(ldg=1 << 40) == ESHAPE
    assert fwd(g=P + 1) == EALIGN and fwd(gq=P + 8, gs=P, uq=P, us=P) == EALIGN

    def bwd(act=0, dY=P, g=P, ldg=64, u=P, ldu=64, gq=None, gs=None, uq=None, us=None, M=4, K=64, dg=P, lddg=64, du=P,
            lddu=64):
        return L.bitnet_gate_bwd(act, dY, g, ldg, u, ldu, gq, gs, uq, us, M, K, dg, lddg, du, lddu, None)

    assert bwd(dY=None) == ENULL and bwd(dg=None) == ENULL and bwd(g=None) == ENULL and bwd(u=None) == ENULL
    assert bwd(gq=P) == ENULL and bwd(gq=P, gs=P) == ENULL and bwd(du=None) == ENULL
    assert bwd(act=5) == EDTYPE and bwd(lddg=1) == ESHAPE and bwd(lddu=1) == ESHAPE and bwd(ldg=1) == ESHAPE
    assert bwd(du=P + 1) == EALIGN


def test_ttq_ckpt_refusals(L):
    M, N, K = 128, 256, 320
    need = L.ttq_bwd_ckpt_workspace_bytes(M, N, K)
    assert need >= L.ttq_workspace_bytes(M, N, K) + 2 * M * K
    assert L.ttq_fwd_ckpt_workspace_bytes(M, N, K) == L.ttq_workspace_bytes(M, N, K)
    odd = L.ttq_fwd_ckpt_workspace_bytes(M, N, K + 1)
    assert odd >= 2 * M * (K + 64) and L.ttq_fwd_ckpt_workspace_bytes(M, 0, K) == 0

    def fwd(x=P, wt=P, M=M, N=N, K=K + 1, y=P, c=P, s=P, ws=P, n=odd):
        return L.ttq_fwd_ckpt(x, wt, M, N, K, y, c, s, ws, n, None)

    assert fwd(x=None) == ENULL and fwd(wt=None) == ENULL and fwd(y=None) == ENULL and fwd(s=None) == ENULL
    assert fwd(M=0) == ESHAPE and fwd(ws=None) == EWS and fwd(n=odd - 1) == EWS
    assert fwd(x=P + 8) == EALIGN and fwd(c=P + 8) == EALIGN and fwd(s=P + 2) == EALIGN

    def f(dY=P, c=P, s=P, wt=P, wp=P, M=M, N=N, K=K, dX=P, dW=P, d=BF, g=P, ws=P, n=need):
        return L.ttq_bwd_ckpt(dY, c, s, wt, wp, M, N, K, dX, dW, d, g, ws, n, None)

    assert f(dY=None) == ENULL and f(c=None) == ENULL and f(s=None) == ENULL and f(dX=None, dW=None) == ENULL
    assert f(wt=None) == ENULL and f(wp=None) == ENULL and f(d=SIGN1) == EDTYPE
    assert f(ws=None) == EWS and f(n=need - 1) == EWS and f(M=0) == ESHAPE
    assert f(c=P + 8) == EALIGN and f(dY=P + 8) == EALIGN and f(ws=P + 8) == EALIGN


def test_python_refusals():
    from ternary_weight_quantization_amd import binding as B
    from ternary_weight_quantization_amd.checkpoint import compress, gated_activation
    from ternary_weight_quantization_amd.norm import layer_norm

    x, f = torch.zeros(4, 64, dtype=torch.bfloat16), torch.zeros(4, 64)
    with pytest.raises(TypeError):
        layer_norm(x.half())
    with pytest.raises(TypeError):
        layer_norm(x, out_dtype=torch.float16)
    with pytest.raises(ValueError):
        layer_norm(x)  # not on a GPU
    with pytest.raises(ValueError):
        layer_norm(torch.zeros(4, 0))
    with pytest.raises(TypeError):
        gated_activation(f, f)
    with pytest.raises(ValueError):
        gated_activation(x, x[:, :32])
    with pytest.raises(ValueError):
        gated_activation(x, x, "gelu")
    with pytest.raises(ValueError):
        gated_activation(x, x)
    with pytest.raises(ValueError):
        compress(x)
    with pytest.raises(ValueError):
        compress(torch.zeros(3, 0))
    with pytest.raises(ValueError):
        B._need_codes(torch.zeros(4, 128, dtype=torch.int8), None, 4, 64)
    with pytest.raises(ValueError):
        B._need_rows(x.t().contiguous().t(), 4, 64, "gate")
    with pytest.raises(ValueError):
        B._need_rows(x[:1].expand(4, 64), 4, 64, "gate")


def test_xent_refusals(L):
    T, V, D = 100, 1000, 64
    nf, nb = L.bitnet_xent_fwd_workspace_bytes(T, V, D), L.bitnet_xent_bwd_workspace_bytes(T, V, D)
    assert nf > 0 and nb > 2 * T * V  # G for the one piece
    for f in (L.bitnet_xent_fwd_workspace_bytes, L.bitnet_xent_bwd_workspace_bytes):
        assert f(0, V, D) == 0 and f(T, 0, D) == 0 and f(T, V, 0) == 0 and f(T, V, 65537) == 0
        assert f((1 << 21) + 1, V, 8) == 0 and f(T, (1 << 28) + 1, D) == 0 and f(1 << 20, V, 2048) == 0
    # G never holds the whole vocabulary of a large problem
    assert L.bitnet_xent_bwd_workspace_bytes(4096, 128256, 2560) < 2 * 4096 * 128256 // 4
    assert L.bitnet_xent_fwd_workspace_bytes(16, 32000, 2560) < 1 << 20

    def fwd(h=P, w=P, t=P, T=T, V=V, D=D, loss=P, lse=P, total=P, red=2, ws=P, n=nf):
        return L.bitnet_xent_fwd(h, w, t, -100, T, V, D, loss, lse, total, red, ws, n, None)

    assert fwd(h=None) == ENULL and fwd(w=None) == ENULL and fwd(t=None) == ENULL and fwd(loss=None) == ENULL
    assert fwd(lse=None) == ENULL and fwd(total=None) == ENULL and fwd(red=0) == ENULL
    assert fwd(red=3) == EDTYPE and fwd(T=0) == ESHAPE and fwd(D=70000) == ESHAPE
    assert fwd(ws=None) == EWS and fwd(n=nf - 1) == EWS
    assert fwd(h=P + 8) == EALIGN and fwd(w=P + 2) == EALIGN and fwd(t=P + 4) == EALIGN and fwd(ws=P + 8) == EALIGN

    def bwd(h=P, w=P, t=P, lse=P, dl=P, red=2, T=T, V=V, D=D, dh=P, dw=P, d=BF, ws=P, n=nb):
        return L.bitnet_xent_bwd(h, w, t, -100, lse, dl, red, T, V, D, dh, dw, d, ws, n, None)

    assert bwd(h=None) == ENULL and bwd(lse=None) == ENULL and bwd(dl=None) == ENULL and bwd(dh=None, dw=None) == ENULL
    assert bwd(red=-1) == EDTYPE and bwd(d=SIGN1) == EDTYPE and bwd(V=0) == ESHAPE
    assert bwd(ws=None) == EWS and bwd(n=nb - 1) == EWS
    assert bwd(dh=P + 8) == EALIGN and bwd(dw=P + 4) == EALIGN and bwd(lse=P + 2) == EALIGN


def test_xent_python_refusals():
    from ternary_weight_quantization_amd.loss import linear_cross_entropy

    h, w, t = torch.zeros(4, 8, dtype=torch.bfloat16), torch.zeros(9, 8, dtype=torch.bfloat16), torch.zeros(4).long()
    with pytest.raises(TypeError):
        linear_cross_entropy(h.float(), w, t)
    with pytest.raises(TypeError):
        linear_cross_entropy(h, w.half(), t)
    with pytest.raises(TypeError):
        linear_cross_entropy(h, w, t.int())
    with pytest.raises(ValueError):
        linear_cross_entropy(h, w[:, :4], t)
    with pytest.raises(ValueError):
        linear_cross_entropy(h, w[:0], t)
    with pytest.raises(ValueError):
        linear_cross_entropy(h, w, t[:3])
    with pytest.raises(ValueError):
        linear_cross_entropy(h, w, t, reduction="max")
    with pytest.raises(ValueError):
        linear_cross_entropy(h, w, t)  # not on a GPU


def test_checkpoint_size_limit(L):
    """More values than a launch holds threads for."""
    for M, K in ((1 << 27, 129), ((1 << 27) + 1, 128), (1 << 30, 17)):
        assert L.bitnet_ckpt_pack(P, BF, M, K, P, P, None) == ESHAPE
        assert L.bitnet_ckpt_unpack(P, P, M, K, P, F32, None) == ESHAPE
        assert L.bitnet_gate_fwd(0, P, K, P, K, M, K, P, None, None, None, None, None) == ESHAPE
        assert L.bitnet_gate_bwd(0, P, P, K, P, K, None, None, None, None, M, K, P, K, P, K, None) == ESHAPE


def test_a_ttq_module_pickled_without_the_checkpoint_attribute():
    """One whose state holds no `checkpoint` is one that keeps its input."""
    from ternary_weight_quantization_amd.ttq_layer import TTQLinear

    m = TTQLinear.__new__(TTQLinear)
    torch.nn.Module.__init__(m)
    m.__dict__.update(in_features=64, out_features=32)
    m.weight, m.raw = torch.nn.Parameter(torch.zeros(32, 64)), torch.nn.Parameter(torch.zeros(3))
    assert m.checkpoint is False and repr(m) == "TTQLinear(64, 32, dtype=torch.float32)"
    with pytest.raises(TypeError, match="bf16"):
        m(torch.zeros(2, 64))
