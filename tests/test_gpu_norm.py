"""Layer norm on the GPU against its formulas in 64 bits.

Bounds. u = 2^-24 (half an fp32 step), and a rounding to the output type is
off by at most h = finfo(t).eps / 2 relative to the value. A row's sums add
at most 8 chunk sums of depth 4 per thread, 6 steps of a wave and 8 wave
sums, so a sum of n terms is off by at most 28 u times the sum of their
magnitudes, and with the few operations around it (a difference, a division, a
square root, products; two roundings in a code's value) every intermediate is
within D = 40 u of its terms' magnitudes:
  |err mu|      <= D mean|x|
  |err xh|      <= D r (mean|x| + |x|) + D |xh|                     =: ex
  |err y|       <= h |y| + |w| ex + D (|xh w| + |b|)
  |err c1|      <= D mean|g|,   |err c2| <= D mean|g xh| + mean(|g| ex)
  |err dX|      <= h |dX| + r (D (|g| + |c1| + |xh c2|) + err c1 + |xh| err c2 + |c2| ex) + D |dX|
  |err dw|      <= h |dw| + S u sum|dY xh| + sum |dY| ex
  |err db|      <= h |db| + S u sum|dY|
where S counts the additions of a column: a thread's rows (at most M / 256 +
1), 4 rows of a block, and a block's partial of at most 512 in 16 groups (48
more): S = M / 256 + 64.
"""

import numpy as np
import pytest
import torch

from tests.gpu_util import note

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
D = 40 * U


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.fail("no GPU visible")
    from ternary_weight_quantization_amd import binding
    binding.lib()


def half(t):
    return torch.finfo(t).eps / 2


def kept(x):
    """The values of x's 8-bit checkpoint in 64 bits."""
    M, K = x.shape
    v = torch.zeros(M, -(-K // 128) * 128, dtype=torch.float64, device=x.device)
    v[:, :K] = x.double()
    b = v.view(M, -1, 128)
    s = b.abs().amax(-1, keepdim=True)
    q = torch.round(127.0 * b / torch.where(s > 0, s, torch.ones_like(s)))
    return (q * s / 127.0).view(M, -1)[:, :K]


def make(M, K, xt, pt, seed, offset=0.0):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    x = r(M, K) * (1.0 + 4.0 * (torch.arange(K, device="cuda") % 37 == 0)) + offset
    w = b = None
    if pt is not None:
        w, b = (1.0 + 0.3 * r(K)).to(pt), (0.3 * r(K)).to(pt)
    return x.to(xt), w, b, r(M, K)


def check(M, K, xt, pt, yt, ckpt, seed=0, offset=0.0, eps=1e-5):
    from ternary_weight_quantization_amd.norm import layer_norm

    note(f"norm M={M} K={K} x={xt} p={pt} y={yt} ckpt={ckpt}")
    x, w, b, dy = make(M, K, xt, pt, seed, offset)
    dy = dy.to(yt)
    leaves = [t.requires_grad_(True) for t in (x, w, b) if t is not None]
    y = layer_norm(x, w, b, eps=eps, out_dtype=yt, checkpoint=ckpt)
    assert y.dtype == yt and y.shape == x.shape
    grads = torch.autograd.grad(y, leaves, dy)
    with torch.no_grad():
        assert torch.equal(layer_norm(x, w, b, eps=eps, out_dtype=yt), y)
        x64 = x.double()
        mu = x64.mean(1, keepdim=True)
        r = ((x64 - mu).square().mean(1, keepdim=True) + eps).rsqrt()
        wd = torch.ones(K, dtype=torch.float64, device="cuda") if w is None else w.double()
        bd = torch.zeros(K, dtype=torch.float64, device="cuda") if b is None else b.double()
        xh = (x64 - mu) * r
        mx = x64.abs().mean(1, keepdim=True)
        ref = xh * wd + bd
        ex = D * r * (mx + x64.abs()) + D * xh.abs()
        tol = half(yt) * ref.abs() + wd.abs() * ex + D * ((xh * wd).abs() + bd.abs())
        bad = ((y.double() - ref).abs() > tol).sum().item()
        assert bad == 0, ("y", bad, ((y.double() - ref).abs() / tol).max().item())
        if ckpt:
            x64 = kept(x)
            xh = (x64 - mu) * r
            ex = D * r * (mx + x64.abs()) + D * xh.abs()
        d = dy.double()
        gw = d * wd
        c1, c2 = gw.mean(1, keepdim=True), (gw * xh).mean(1, keepdim=True)
        dx = r * (gw - c1 - xh * c2)
        e1 = D * gw.abs().mean(1, keepdim=True)
        e2 = D * (gw * xh).abs().mean(1, keepdim=True) + (gw.abs() * ex).mean(1, keepdim=True)
        tol = (half(xt) + D) * dx.abs() + r * (D * (gw.abs() + c1.abs() + (xh * c2).abs()) + e1 + xh.abs() * e2
                                               + c2.abs() * ex)
        err = (grads[0].double() - dx).abs()
        assert grads[0].dtype == xt and (err <= tol).all(), ("dX", (err / tol).max().item())
        if pt is not None:
            S = M / 256 + 64
            dw, db = (d * xh).sum(0), d.sum(0)
            tol = half(pt) * dw.abs() + S * U * (d * xh).abs().sum(0) + (d.abs() * ex).sum(0)
            err = (grads[1].double() - dw).abs()
            assert grads[1].dtype == pt and (err <= tol).all(), ("dw", (err / tol).max().item())
            tol = half(pt) * db.abs() + S * U * d.abs().sum(0)
            err = (grads[2].double() - db).abs()
            assert grads[2].dtype == pt and (err <= tol).all(), ("db", (err / tol).max().item())
    return y, grads


BF, F32 = torch.bfloat16, torch.float32


# widths around every change of the threads per row and chunks per thread,
# whole and broken blocks of 128, rows shorter than one vector
@pytest.mark.parametrize("K", [1, 2, 7, 8, 9, 15, 127, 128, 129, 511, 512, 640, 1025, 1536, 2047, 2555, 2560, 2561,
                               4096, 4097, 6144, 6145, 6912, 8193, 10240, 10241, 12289, 16383, 20481, 24577, 28673,
                               32768])
def test_widths(K):
    check(5, K, BF, BF, BF, False, seed=K)
    check(3, K, BF, F32, BF, True, seed=K + 1)


@pytest.mark.parametrize("K", [1, 7, 130, 2560, 2563, 6912, 10241, 32767])
@pytest.mark.parametrize("xt,pt,yt,ckpt", [(F32, F32, BF, False), (F32, F32, F32, True), (F32, BF, F32, False),
                                           (BF, None, F32, False), (F32, None, BF, True), (BF, F32, F32, True)])
def test_types(K, xt, pt, yt, ckpt):
    check(6, K, xt, pt, yt, ckpt, seed=K)


@pytest.mark.parametrize("M", [1, 2, 3, 4, 5, 63, 511, 2047, 2048, 2049, 5001])
def test_rows(M):
    check(M, 2560, BF, BF, BF, False, seed=M)
    check(M, 321, F32, F32, BF, True, seed=M)
    check(M, 4224, BF, F32, BF, True, seed=M)


def test_offset_rows():
    """A mean far above the spread: the variance is a sum of centered
    squares."""
    check(64, 2560, F32, F32, F32, False, offset=1000.0)
    check(64, 6912, F32, F32, F32, True, offset=-300.0)


def test_constant_and_zero_rows():
    from ternary_weight_quantization_amd.norm import layer_norm

    x = torch.zeros(4, 300, device="cuda")
    x[1] = 7.0
    x[2, 5] = 1.0
    x[3] = -2.5
    x.requires_grad_(True)
    for ckpt in (False, True):
        y = layer_norm(x, out_dtype=F32, eps=1e-5, checkpoint=ckpt)
        assert torch.equal(y[[0, 1, 3]], torch.zeros(3, 300, device="cuda"))
        dx, = torch.autograd.grad(y, x, torch.ones_like(y))
        assert torch.isfinite(dx).all()


def test_nan_and_infinity_stay_in_their_row():
    from ternary_weight_quantization_amd.norm import layer_norm

    x, w, b, dy = make(9, 2560, BF, F32, 3)
    clean = x.clone()
    x[2, 17] = float("nan")
    x[5, 2559] = float("inf")
    good = [r for r in range(9) if r not in (2, 5)]
    for ckpt in (False, True):
        xs = [t.clone().requires_grad_(True) for t in (x, clean)]
        ys = [layer_norm(t, w, b, checkpoint=ckpt) for t in xs]
        dxs = [torch.autograd.grad(y, t, dy.to(BF))[0] for y, t in zip(ys, xs)]
        assert torch.equal(ys[0][good], ys[1][good]) and torch.equal(dxs[0][good], dxs[1][good])
        assert torch.isnan(ys[0][[2, 5]].float()).all()
        assert torch.isnan(dxs[0][[2, 5]].float()).any(1).all()


def test_views_shapes_and_partial_gradients():
    from ternary_weight_quantization_amd.norm import layer_norm

    x, w, b, dy = make(12, 640, BF, BF, 4)
    dy = dy.to(BF)
    whole = layer_norm(x, w, b)
    wide = torch.randn(12, 1300, device="cuda").to(BF)
    wide[:, 3:643] = x
    assert torch.equal(layer_norm(wide[:, 3:643], w, b), whole)
    assert torch.equal(layer_norm(x.t().contiguous().t(), w, b), whole)
    assert torch.equal(layer_norm(x.view(3, 4, 640), w, b), whole.view(3, 4, 640))
    # parameters that start at an odd element, dY as a transposed view
    flat = torch.zeros(1 + 640, device="cuda", dtype=BF)
    flat[1:] = w
    assert torch.equal(layer_norm(x, flat[1:], b), whole)
    xs, ws, bs = (t.clone().requires_grad_(True) for t in (x, w, b))
    full = torch.autograd.grad(layer_norm(xs, ws, bs), (xs, ws, bs), dy)
    for k, t in enumerate((xs, ws, bs)):
        leaves = [(v if i == k else v.detach()) for i, v in enumerate((xs, ws, bs))]
        got, = torch.autograd.grad(layer_norm(*leaves), t, dy.t().contiguous().t())
        assert torch.equal(got, full[k])
    got, = torch.autograd.grad(layer_norm(x, None, bs), bs, dy)
    assert torch.equal(got, full[2])


def test_no_rows():
    from ternary_weight_quantization_amd.norm import QATLayerNorm

    m = QATLayerNorm(96)
    x = torch.empty(0, 96, device="cuda", dtype=BF, requires_grad=True)
    y = m(x)
    assert y.shape == (0, 96)
    y.sum().backward()
    assert x.grad.shape == (0, 96)
    assert torch.equal(m.weight.grad, torch.zeros_like(m.weight)) and torch.equal(m.bias.grad, torch.zeros_like(m.bias))


def test_same_bits_again_and_on_another_stream():
    from ternary_weight_quantization_amd.norm import layer_norm

    x, w, b, dy = make(3000, 2560, BF, F32, 5)
    dy = dy.to(BF)

    def one():
        leaves = [t.detach().clone().requires_grad_(True) for t in (x, w, b)]
        y = layer_norm(*leaves, checkpoint=True)
        return (y.detach(),) + torch.autograd.grad(y, leaves, dy)

    first = one()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        second = one()
    torch.cuda.current_stream().wait_stream(s)
    torch.cuda.synchronize()
    for p, q in zip(first, second):
        assert torch.equal(p, q)


def test_graph_replays():
    """The C entry points captured once, replayed on new inputs."""
    from ternary_weight_quantization_amd import binding as B

    M, K = 200, 2560
    x, w, b, dy = make(M, K, BF, BF, 6)
    dy = dy.to(BF)
    y, dX = torch.empty_like(x), torch.empty_like(x)
    mean, rstd = torch.empty(2, M, device="cuda")
    dw, db = torch.empty_like(w), torch.empty_like(b)
    ws = torch.empty(B.bitnet_layernorm_workspace_bytes(M, K), dtype=torch.uint8, device="cuda")

    def step():
        B.bitnet_layernorm_fwd(x, w, b, 1e-5, y, mean, rstd)
        B.bitnet_layernorm_bwd(dy, x, w, mean, rstd, dX, dw, db, workspace=ws)

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for seed in (7, 8, 9):
        x2, _, _, dy2 = make(M, K, BF, BF, seed)
        x.copy_(x2)
        dy.copy_(dy2)
        graph.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in (y, dX, dw, db)]
        step()
        torch.cuda.synchronize()
        for p, q in zip(got, (y, dX, dw, db)):
            assert torch.equal(p, q)


def test_gradient_against_differences():
    """d/dt of sum(dY * y(x + t v)) at 0 by central differences, all in
    fp32: the difference's own error is h^2 / 6 times the third derivative
    (of order one after scaling by |v|) plus the outputs' rounding over h."""
    from ternary_weight_quantization_amd.norm import layer_norm

    x, w, b, dy = make(7, 530, F32, F32, 10)
    v = torch.randn(7, 530, device="cuda")
    leaves = [t.requires_grad_(True) for t in (x, w, b)]
    grads = torch.autograd.grad(layer_norm(*leaves, out_dtype=F32), leaves, dy)
    h = 2.0 ** -7
    with torch.no_grad():
        f = lambda t: (layer_norm(x + t * v, w, b, out_dtype=F32).double() * dy.double()).sum()  # noqa: E731
        num = ((f(h) - f(-h)) / (2 * h)).item()
        ana = (grads[0].double() * v.double()).sum().item()
        # outputs off by D each: sum |dY| D (|y| + 2) / h; third derivative: h^2 times the terms' size
        y = layer_norm(x, w, b, out_dtype=F32).double()
        tol = (dy.double().abs() * (y.abs() + 2)).sum().item() * (D / h + h * h)
    assert abs(num - ana) <= tol, (num, ana, tol)


def test_module_before_a_ternary_layer():
    """The norm, the ternary layer and a sum as a loss: gradients reach the
    norm's parameters and equal those of the formulas on the layer's dX."""
    from ternary_weight_quantization_amd.layer import QATBitLinear
    from ternary_weight_quantization_amd.norm import QATLayerNorm

    torch.manual_seed(0)
    norm, lin = QATLayerNorm(256, dtype=F32), QATBitLinear(256, 192)
    x = torch.randn(40, 256, device="cuda", dtype=F32, requires_grad=True)
    y = norm(x)
    dy = torch.randn(40, 192, device="cuda").to(BF)
    out = lin(y)
    dyn, = torch.autograd.grad(out, y, dy, retain_graph=True)
    out.backward(dy)
    x64, d = x.detach().double(), dyn.double()
    xh = (x64 - x64.mean(1, keepdim=True)) / (x64.var(1, unbiased=False, keepdim=True) + 1e-5).sqrt()
    tol = D * 4 * (d.abs() * (1 + xh.abs())).sum(0)
    assert ((norm.weight.grad.double() - (d * xh).sum(0)).abs() <= tol).all()
    assert ((norm.bias.grad.double() - d.sum(0)).abs() <= tol).all()
    assert x.grad is not None and lin.weight.grad is not None
