"""Refusals of the RMS norm, 8-bit rows, gated projections and 8-bit linear layer
without a GPU: the C ABI rejects bad arguments with the documented codes before
touching the device, the Python entry points raise before they call it, and
torch's transformations are refused."""

import os

import pytest
import torch
import torch.autograd.forward_ad as fwad

from tests.test_operators_transforms_cpu import without_memory

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
LIB = os.path.join(ROOT, "ternary_weight_quantization_amd", "libbitnet.so")
OK, ENULL, ESHAPE, EDTYPE, EALIGN, EWS, EHIP = range(7)
P = 1 << 20  # a stand-in device address, aligned; never dereferenced
BF, F32, SIGN1 = 0, 1, 2
TBF = torch.bfloat16


@pytest.fixture(scope="module")
def L():
    if not os.path.exists(LIB):
        pytest.fail("libbitnet.so is not built (run `python -m ternary_weight_quantization_amd.build`)")
    from ternary_weight_quantization_amd import binding
    return binding.lib()


def test_rmsnorm_refusals(L):
    def f(x=P, xd=BF, res=P, hd=BF, w=P, pd=BF, M=4, K=64, h=P, y=P, yd=BF, q=None, s=None, r=P):
        return L.bitnet_rmsnorm_fwd(x, xd, res, hd, w, pd, M, K, 1e-6, h, y, yd, q, s, r, None)

    assert f(x=None) == ENULL and f(res=None) == ENULL and f(h=None) == ENULL and f(y=None) == ENULL
    assert f(q=P, s=P) == ENULL and f(y=None, q=P) == ENULL
    assert f(xd=SIGN1) == EDTYPE and f(hd=SIGN1) == EDTYPE and f(pd=SIGN1) == EDTYPE and f(yd=SIGN1) == EDTYPE
    assert f(xd=F32) == EDTYPE and f(res=None, h=None, hd=F32) == EDTYPE
    assert f(M=0) == ESHAPE and f(K=0) == ESHAPE and f(K=16385) == ESHAPE and f(M=(1 << 30) + 1) == ESHAPE
    assert f(x=P + 1) == EALIGN and f(res=P + 2, hd=F32) == EALIGN and f(h=P + 2, hd=F32) == EALIGN
    assert f(w=P + 2, pd=F32) == EALIGN and f(y=P + 1) == EALIGN and f(r=P + 2) == EALIGN
    assert f(y=None, q=P + 8, s=P) == EALIGN and f(y=None, q=P, s=P + 8) == EALIGN

    need = L.bitnet_rmsnorm_workspace_bytes(9, 64)
    assert need == 3 * 64 * 4  # a partial row for each 4 rows
    assert L.bitnet_rmsnorm_workspace_bytes(0, 64) == 0 and L.bitnet_rmsnorm_workspace_bytes(4, 16385) == 0

    def b(dY=P, yd=BF, dH=P, h=P, hd=BF, w=P, pd=BF, r=P, M=9, K=64, dh=P, dx=None, dw=P, ws=P, n=need):
        return L.bitnet_rmsnorm_bwd(dY, yd, dH, h, hd, w, pd, r, M, K, dh, dx, dw, ws, n, None)

    assert b(dY=None) == ENULL and b(h=None) == ENULL and b(r=None) == ENULL and b(dh=None, dw=None) == ENULL
    assert b(yd=SIGN1) == EDTYPE and b(hd=7) == EDTYPE and b(pd=SIGN1) == EDTYPE and b(dx=P) == EDTYPE
    assert b(M=0) == ESHAPE and b(K=16385) == ESHAPE
    assert b(ws=None) == EWS and b(n=need - 1) == EWS and b(ws=P + 8) == EALIGN
    assert b(dY=P + 1) == EALIGN and b(dH=P + 2, hd=F32) == EALIGN and b(dh=P + 1) == EALIGN
    assert b(dx=P + 1, hd=F32) == EALIGN and b(dw=P + 2, pd=F32) == EALIGN


def test_rows_refusals(L):
    def f(x=P, d=BF, M=4, K=64, q=P, s=P):
        return L.bitnet_rows_quant(x, d, M, K, q, s, None)

    for d in (BF, F32):
        assert f(x=None, d=d) == ENULL and f(q=None, d=d) == ENULL and f(s=None, d=d) == ENULL
        assert f(M=0, d=d) == ESHAPE and f(K=0, d=d) == ESHAPE
        assert f(x=P + 1, d=d) == EALIGN and f(q=P + 8, d=d) == EALIGN and f(s=P + 8, d=d) == EALIGN
        assert f(d=d, M=(1 << 23) + 1) == ESHAPE and f(d=d, K=(1 << 24) + 1) == ESHAPE
    assert f(d=SIGN1) == EDTYPE and f(x=P + 2, d=F32) == EALIGN

    def two(x=P, M=4, q=P, s=P, w=P, d=BF, N=3, wq=P, sw=P, K=64):
        return L.bitnet_rows_quant2(x, M, q, s, w, d, N, wq, sw, K, None)

    assert two(x=None) == ENULL and two(q=None) == ENULL and two(s=None) == ENULL
    assert two(w=None) == ENULL and two(wq=None) == ENULL and two(sw=None) == ENULL
    assert two(M=0, N=0) == ESHAPE and two(M=-1) == ESHAPE and two(N=-1) == ESHAPE and two(K=0) == ESHAPE
    assert two(d=SIGN1) == EDTYPE and two(x=P + 1) == EALIGN and two(w=P + 2, d=F32) == EALIGN
    assert two(q=P + 8) == EALIGN and two(sw=P + 8) == EALIGN

    def u(q=P, s=P, M=4, K=64, x=P):
        return L.bitnet_rows_unpack(q, s, M, K, x, None)

    assert u(q=None) == ENULL and u(s=None) == ENULL and u(x=None) == ENULL and u(M=0) == ESHAPE and u(K=0) == ESHAPE
    assert u(M=1 << 30, K=2048) == ESHAPE
    assert u(q=P + 8) == EALIGN and u(s=P + 2) == EALIGN and u(x=P + 1) == EALIGN


def test_gated_refusals(L):
    M, N, K = 300, 200, 130
    nf, nb = L.bitnet_gated_fwd_workspace_bytes(M, N, K), L.bitnet_gated_bwd_workspace_bytes(M, N, K)
    assert nb >= M * 4 * 256 + 192 * 256 + M * 192 * 2
    assert L.bitnet_gated_slopes_bytes(M, N) == M * 6 * 256 and L.bitnet_gated_slopes_bytes(0, N) == 0
    for f in (L.bitnet_gated_fwd_workspace_bytes, L.bitnet_gated_bwd_workspace_bytes):
        assert f(0, N, K) == 0 and f(M, 0, K) == 0 and f(M, N, 0) == 0 and f(1 << 20, 1 << 12, K) == 0
        assert f(M, 1 << 30, K) == 0 and f(1 << 31, N, K) == 0

    def fwd(act=0, q=P, s=P, w=P, g=P, M=M, N=N, K=K, y=P, sl=P, ws=P, n=nf, x=None):
        return L.bitnet_gated_fwd(act, x, q, s, w, g, M, N, K, y, sl, ws, n, None)

    assert fwd(q=None) == ENULL and fwd(s=None) == ENULL and fwd(w=None) == ENULL and fwd(g=None) == ENULL
    assert fwd(y=None) == ENULL and fwd(act=2) == EDTYPE and fwd(M=0) == ESHAPE and fwd(M=1 << 20, N=1 << 12) == ESHAPE
    assert fwd(q=P + 8) == EALIGN and fwd(g=P + 2) == EALIGN and fwd(sl=P + 8) == EALIGN and fwd(y=P + 2) == EALIGN
    if nf:
        assert fwd(ws=None) == EWS and fwd(n=nf - 1) == EWS
    assert fwd(ws=None, n=nf + 1) == EWS
    most = L.bitnet_rows_direct(K)
    assert most >= 1 and L.bitnet_rows_direct(7) == 0 and L.bitnet_rows_direct(1 << 20) == 0
    few = dict(q=None, s=None, n=0)
    assert fwd(x=P, M=most + 1, **few) == ESHAPE and fwd(x=P, M=1, K=1 << 15, **few) == ESHAPE
    assert fwd(x=P + 1, M=1, **few) == EALIGN and fwd(x=P, M=1, y=P + 2, **few) == EALIGN and fwd(x=P, M=0, **few) == ESHAPE

    def bwd(dY=P, sl=P, q=P, s=P, w=P, g=P, M=M, N=N, K=K, dX=P, a=P, b=P, d=BF, ws=P, n=nb):
        return L.bitnet_gated_bwd(dY, sl, q, s, w, g, M, N, K, dX, a, b, d, ws, n, None)

    assert bwd(dY=None) == ENULL and bwd(sl=None) == ENULL and bwd(g=None) == ENULL and bwd(w=None) == ENULL
    assert bwd(dX=None, a=None, b=None) == ENULL and bwd(a=None) == ENULL and bwd(b=None) == ENULL
    assert bwd(q=None) == ENULL and bwd(s=None) == ENULL and bwd(d=SIGN1) == EDTYPE and bwd(N=0) == ESHAPE
    assert bwd(ws=None) == EWS and bwd(n=nb - 1) == EWS and bwd(ws=P + 8) == EALIGN
    assert bwd(dY=P + 1) == EALIGN and bwd(dX=P + 8) == EALIGN and bwd(b=P + 8) == EALIGN and bwd(s=P + 2) == EALIGN


def test_quantize2_refusals(L):
    n = L.bitnet_ternarize_workspace_bytes(200, 130)

    def f(a=P, b=P, d=BF, N=200, K=130, x=P, M=4, p=P, g=P, q=P, s=P, ws=P, n=n):
        return L.bitnet_quantize2(a, b, d, N, K, x, M, p, g, q, s, ws, n, None)

    assert f(a=None) == ENULL and f(b=None) == ENULL and f(p=None) == ENULL and f(g=None) == ENULL
    assert f(q=None) == ENULL and f(s=None) == ENULL and f(d=SIGN1) == EDTYPE
    assert f(N=0) == ESHAPE and f(K=0) == ESHAPE and f(M=0) == ESHAPE and f(N=1 << 31) == ESHAPE
    assert f(a=P + 8) == EALIGN and f(b=P + 8) == EALIGN and f(x=P + 8) == EALIGN and f(p=P + 8) == EALIGN
    assert f(g=P + 2) == EALIGN and f(q=P + 8) == EALIGN and f(s=P + 8) == EALIGN and f(ws=P + 8) == EALIGN
    assert f(ws=None) == EWS and f(n=n - 1) == EWS
    assert f(x=None, M=0, q=None, s=None, ws=None) == EWS  # no rows: M, q and s are not looked at


def test_int8_refusals(L):
    M, N, K = 300, 201, 130
    nf, nb = L.bitnet_int8_fwd_workspace_bytes(M, N, K), L.bitnet_int8_bwd_workspace_bytes(M, N, K)
    assert nb >= (M + N) * 192 * 2 + M * 256 * 2
    for f in (L.bitnet_int8_fwd_workspace_bytes, L.bitnet_int8_bwd_workspace_bytes):
        assert f(0, N, K) == 0 and f(M, 0, K) == 0 and f(M, N, 0) == 0 and f(M, N, 131073) == 0 and f(1 << 24, N, K) == 0

    def fwd(q=P, s=P, w=P, sw=P, b=P, M=M, N=N, K=K, y=P, ws=P, n=nf, x=None):
        return L.bitnet_int8_fwd(x, q, s, w, sw, b, M, N, K, y, ws, n, None)

    assert fwd(q=None) == ENULL and fwd(s=None) == ENULL and fwd(w=None) == ENULL and fwd(sw=None) == ENULL
    assert fwd(y=None) == ENULL and fwd(K=131073) == ESHAPE and fwd(M=0) == ESHAPE and fwd(N=(1 << 24) + 1) == ESHAPE
    assert fwd(q=P + 8) == EALIGN and fwd(sw=P + 4) == EALIGN and fwd(b=P + 2) == EALIGN and fwd(y=P + 2) == EALIGN
    assert fwd(ws=None, n=nf + 1) == EWS
    most = L.bitnet_rows_direct(K)
    assert fwd(x=P, M=most + 1, q=None, s=None) == ESHAPE and fwd(x=P + 1, M=most, q=None, s=None) == EALIGN
    assert fwd(x=P, M=0, q=None, s=None) == ESHAPE and fwd(x=P, M=1, w=None) == ENULL

    def bwd(dY=P, q=P, s=P, w=P, sw=P, M=M, N=N, K=K, dX=P, dW=P, d=BF, db=P, bd=BF, ws=P, n=nb):
        return L.bitnet_int8_bwd(dY, q, s, w, sw, M, N, K, dX, dW, d, db, bd, ws, n, None)

    assert bwd(dY=None) == ENULL and bwd(dX=None, dW=None, db=None) == ENULL and bwd(w=None) == ENULL
    assert bwd(sw=None) == ENULL and bwd(bd=SIGN1) == EDTYPE and bwd(db=P + 1) == EALIGN and bwd(db=P + 2, bd=F32) == EALIGN
    assert bwd(q=None) == ENULL and bwd(s=None) == ENULL and bwd(d=SIGN1) == EDTYPE and bwd(K=131073) == ESHAPE
    assert bwd(ws=None) == EWS and bwd(n=nb - 1) == EWS and bwd(dY=P + 8) == EALIGN and bwd(dW=P + 8) == EALIGN
    assert bwd(s=P + 4) == EALIGN and bwd(ws=P + 8) == EALIGN


def rows_of(M=4, K=64):
    from ternary_weight_quantization_amd.rows import QuantizedRows

    return QuantizedRows(torch.zeros(M, -(-K // 64) * 64, dtype=torch.int8), torch.ones(M), torch.zeros(M, K, dtype=TBF))


def test_python_refusals():
    from ternary_weight_quantization_amd import (QATGatedBitLinear, gated_bitlinear, gated_bitlinear_inference, int8_linear,
                                                 int8_linear_inference, rms_norm)
    from ternary_weight_quantization_amd.layer import bitlinear_inference

    x, f, w = torch.zeros(4, 64, dtype=TBF), torch.zeros(4, 64), torch.zeros(9, 64, dtype=TBF)
    for call in (lambda: rms_norm(x.half()), lambda: rms_norm(x, out_dtype=torch.float16),
                 lambda: gated_bitlinear(f, w, w), lambda: int8_linear(f, w)):
        with pytest.raises(TypeError):
            call()
    for call in (lambda: rms_norm(x), lambda: rms_norm(torch.zeros(3, 0)), lambda: gated_bitlinear(x, w, w, "gelu"),
                 lambda: QATGatedBitLinear(8, 8, act="gelu", device="cpu"), lambda: gated_bitlinear(x, w, w),
                 lambda: gated_bitlinear_inference(x, w.byte(), torch.ones(2), 64), lambda: int8_linear(x, w),
                 lambda: int8_linear_inference(x, w.char(), torch.ones(9), 64), lambda: rows_of().dequantize(),
                 lambda: bitlinear_inference(rows_of(), w.byte(), torch.ones(1), 64), lambda: int8_linear(rows_of(), w)):
        with pytest.raises(ValueError):
            call()


def test_rows_carry_their_shape():
    r = rows_of(4, 60)
    assert r.shape == (4, 60) and not r.requires_grad and "QuantizedRows" in repr(r)
    assert r.detach().codes is r.codes


def calls():
    """(name, function of one float tensor, that tensor)."""
    from ternary_weight_quantization_amd import (gated_bitlinear, gated_bitlinear_inference, int8_linear,
                                                 int8_linear_inference, rms_norm)
    from ternary_weight_quantization_amd import binding as B

    x, w, v = torch.ones(4, 128, dtype=TBF), torch.ones(9, 128, dtype=TBF), torch.ones(128, dtype=TBF)
    q, p = torch.zeros(4, 128, dtype=torch.int8), torch.zeros(6, 32, dtype=torch.uint8)
    s = torch.ones(4)

    def out(r):
        return r[0] if isinstance(r, tuple) else r

    return [
        ("rms_norm", lambda a: rms_norm(a, v), x),
        ("rms_norm", lambda a: rms_norm(x, a), v),
        ("rms_norm", lambda a: out(rms_norm(x, v, a)), x),
        ("dequantize", lambda a: B.ops().rows_values(a, q, s), x),
        ("dequantize", lambda a: B.ops().rows_values(x, q, a), s),
        ("gated_bitlinear", lambda a: gated_bitlinear(a, w, w), x),
        ("gated_bitlinear", lambda a: gated_bitlinear(x, a, w), w),
        ("gated_bitlinear", lambda a: gated_bitlinear(x, w, a), w),
        ("gated_bitlinear", lambda a: gated_bitlinear_inference(a, p, torch.ones(2), 128), x),
        ("int8_linear", lambda a: int8_linear(a, w), x),
        ("int8_linear", lambda a: int8_linear(x, a), w),
        ("int8_linear", lambda a: int8_linear(x, w, a), torch.ones(9)),
        ("int8_linear", lambda a: int8_linear_inference(a, q, s, 128), x),
        ("BitLinear", lambda a: B.ops().rows_bitlinear(a, q, s, w, None), x),
        ("BitLinear", lambda a: B.ops().rows_bitlinear(x, q, s, a, None), w),
        ("BitLinear", lambda a: B.ops().rows_bitlinear_inference(a, q, s, p, torch.ones(1), 128, None), x),
    ]


@pytest.mark.parametrize("grad", [True, False])
@pytest.mark.parametrize("leaf", [True, False])
def test_forward_mode(grad, leaf):
    for name, f, a in calls():
        with torch.set_grad_enabled(grad), fwad.dual_level():
            dual = fwad.make_dual(a.detach().clone().requires_grad_(leaf), torch.ones_like(a))
            with pytest.raises(NotImplementedError, match=f"{name}: no forward-mode derivative"):
                f(dual)


@pytest.mark.parametrize("leaf", [True, False])
def test_traces(leaf):
    from torch.fx.experimental.proxy_tensor import make_fx

    for name, f, a in calls():
        a = a.detach().clone().requires_grad_(leaf)
        for trace in (lambda: torch.jit.trace(f, (a,)), lambda: make_fx(f)(a), lambda: make_fx(f, tracing_mode="fake")(a)):
            with pytest.raises(NotImplementedError, match=f"{name}: cannot be traced"):
                trace()


def test_tensors_without_memory():
    for name, f, a in calls():
        for b in without_memory(a):
            with pytest.raises(NotImplementedError, match=f"{name}: a tensor without memory"):
                f(b)


@pytest.mark.parametrize("transform", ["grad", "vjp", "vmap", "functionalize"])
def test_function_transforms(transform):
    for name, f, a in calls():
        run = {"grad": lambda: torch.func.grad(lambda b: f(b).float().sum())(a), "vjp": lambda: torch.func.vjp(f, a),
               "vmap": lambda: torch.vmap(f)(torch.stack([a, a])), "functionalize": lambda: torch.func.functionalize(f)(a)}
        with pytest.raises(NotImplementedError, match=f"{name}: a tensor without memory"):
            run[transform]()
