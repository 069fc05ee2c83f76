"""The RMS norm with residual and 8-bit rows on the GPU against its formulas in
64 bits.

Bounds. u = 2^-24 (half an fp32 step); a rounding to the output type is off by
at most h = finfo(t).eps / 2 relative to the value. A row's sums add at most 4
chunk sums of depth 8 per thread, 6 steps of a wave and 8 wave sums, so with the
few operations around it every intermediate is within D = 64 u of its terms'
magnitudes. With hn = h r, g = dY w, c = mean(g hn):
  |err v|  <= D |v|  (the stream h itself is exactly rounded, so equal)
  |err s|  <= D s,  a code is within 1/2 + 127 * 3 D of 127 v / s
  |err dh| <= half |dh| + r (D (|g| + |hn c|) + |hn| D mean|g hn|) + D |dH|
  |err dw| <= half |dw| + (S u + D) sum|dY hn|
where S counts the additions of a column: a thread's rows (at most M / 256 + 1),
4 rows of a block, and a block's partial of at most 512 in 16 groups (48 more).
"""

import pytest
import torch

from tests.gpu_util import note

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32
U = 2.0 ** -24
D = 64 * U


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.fail("no GPU visible")
    from ternary_weight_quantization_amd import binding
    binding.lib()


def half(t):
    return torch.finfo(t).eps / 2


def randn(*shape, seed, dtype=BF):
    g = torch.Generator().manual_seed(seed)
    return torch.randn(*shape, generator=g).to(device="cuda", dtype=dtype)


def make(M, K, xt, ht, wt, add, seed=0):
    x, r = randn(M, K, seed=seed, dtype=xt if add else ht), None
    if add:
        r = (randn(M, K, seed=seed + 1, dtype=F32) * (1.0 + 5.0 * (torch.arange(K, device="cuda") % 41 == 0))).to(ht)
    w = None if wt is None else (1.0 + 0.3 * randn(K, seed=seed + 2, dtype=F32)).to(wt)
    return x, r, w


def check(M, K, xt=BF, ht=BF, wt=BF, add=True, out=BF, seed=0, eps=1e-6, scale=1.0):
    """out: BF, F32 or "rows"."""
    from ternary_weight_quantization_amd.norm import rms_norm

    note(f"rms M={M} K={K} x={xt} h={ht} w={wt} add={add} out={out}")
    x, r, w = make(M, K, xt, ht, wt, add, seed)
    if scale != 1.0:
        x = x * scale
        r = None if r is None else r * scale
    leaves = [t.requires_grad_(True) for t in (x, r, w) if t is not None]
    kw = dict(residual=r, eps=eps, quantize=True) if out == "rows" else dict(residual=r, eps=eps, out_dtype=out)
    res = rms_norm(x, w, **kw)
    y, h = res if add else (res, None)
    yt = BF if out == "rows" else out
    dy, dh_in = randn(M, K, seed=seed + 3, dtype=yt), randn(M, K, seed=seed + 4, dtype=ht)
    v = y.dequantize() if out == "rows" else y
    assert v.dtype == yt and v.shape == x.shape
    grads = torch.autograd.grad([v, h] if add else [v], leaves, [dy, dh_in] if add else [dy])
    with torch.no_grad():
        again = rms_norm(x, w, **kw)  # without a graph: the same bits
        again = again if add else (again, None)
        if out == "rows":
            assert torch.equal(again[0].codes, y.codes) and torch.equal(again[0].scales, y.scales)
        else:
            assert torch.equal(again[0], y)
        hs = x if not add else (r.float() + x.float()).to(ht)
        if add:
            assert h.dtype == ht and torch.equal(h, hs) and torch.equal(again[1], h)
        h64 = hs.double()
        rr = (h64.square().mean(1, keepdim=True) + eps).rsqrt()
        wd = torch.ones(K, dtype=torch.float64, device="cuda") if w is None else w.double()
        hn = h64 * rr
        ref = hn * wd
        if out == "rows":
            s = ref.abs().amax(1).clamp(min=1e-8)
            assert y.codes.shape == (M, -(-K // 64) * 64) and not y.codes[:, K:].any()
            assert ((y.scales.double() - s).abs() <= D * s).all()
            t = 127.0 * ref / s[:, None]
            far = (y.codes[:, :K].double() - t).abs().max().item()
            assert far <= 0.5 + 127 * 3 * D, far
            assert y.codes.min() >= -127
            # what the rows stand for: one fp32 product, rounded once
            want = (y.codes[:, :K].float() * (y.scales / 127.0)[:, None]).to(BF)
            assert torch.equal(v, want)
        else:
            tol = (half(yt) + D) * ref.abs()
            bad = ((y.double() - ref).abs() > tol + 1e-40).sum().item()
            assert bad == 0, ("y", bad)
        d = dy.double()
        g = d * wd
        c = (g * hn).mean(1, keepdim=True)
        dh = rr * (g - hn * c)
        tol = rr * (D * (g.abs() + (hn * c).abs()) + hn.abs() * D * (g * hn).abs().mean(1, keepdim=True))
        if add:
            dh = dh + dh_in.double()
            tol = tol + D * dh_in.double().abs()
        for i, t in enumerate((x, r) if add else (x,)):
            assert grads[i].dtype == t.dtype
            err = (grads[i].double() - dh).abs()
            assert (err <= tol + half(t.dtype) * dh.abs()).all(), ("dh", i, (err / (tol + half(t.dtype) * dh.abs())).max())
        if w is not None:
            S = M / 256 + 64
            dw = (d * hn).sum(0)
            tol = half(wt) * dw.abs() + (S * U + D) * (d * hn).abs().sum(0)
            assert grads[-1].dtype == wt
            assert ((grads[-1].double() - dw).abs() <= tol).all()


# every threads-per-row and chunk count, odd widths, rows below one chunk
@pytest.mark.parametrize("K", [1, 5, 8, 63, 65, 128, 513, 1000, 1537, 2048, 2555, 2560, 2700, 4096, 5000, 6905, 8192, 9000,
                               12289, 16384])
@pytest.mark.parametrize("out", [BF, "rows"])
def test_widths(K, out):
    check(13, K, out=out, seed=K)


@pytest.mark.parametrize("M", [1, 2, 3, 4, 5, 257, 1025, 2049])
@pytest.mark.parametrize("add", [True, False])
def test_rows(M, add):
    check(M, 320, add=add, out="rows", seed=M)


@pytest.mark.parametrize("xt,ht", [(BF, BF), (BF, F32), (F32, F32)])
@pytest.mark.parametrize("wt", [None, BF, F32])
@pytest.mark.parametrize("out", [BF, F32, "rows"])
@pytest.mark.parametrize("add", [True, False])
def test_types(xt, ht, wt, out, add):
    check(37, 777, xt, ht, wt, add, out, seed=7)
    check(9, 5000, xt, ht, wt, add, out, seed=8)


@pytest.mark.parametrize("scale", [1e-6, 1e-3, 1e4, 1e12])
def test_scales(scale):
    for out in (F32, "rows"):
        check(5, 640, ht=F32, out=out, scale=scale, seed=3)


def test_zero_rows_and_rows_that_are_not_finite():
    """A row of zeros gives codes 0 and the least scale; a row with an infinity
    or a NaN is NaN and leaves the others as they are."""
    from ternary_weight_quantization_amd.norm import rms_norm

    note("rms rows of zeros, NaN, inf")
    x = randn(8, 300, seed=1)
    clean = rms_norm(x, quantize=True)
    x[2] = 0
    x[4, 7] = float("nan")
    x[6, 299] = float("inf")
    for out in (BF, F32):
        y = rms_norm(x, out_dtype=out)
        assert (y[2] == 0).all() and y[4].isnan().all() and not y[[0, 1, 3, 5, 7]].isnan().any()
        assert y[6].isnan().any()
    rows = rms_norm(x, quantize=True)
    assert (rows.codes[2] == 0).all() and rows.scales[2] == torch.tensor(1e-8)
    assert rows.scales[4].isnan() and rows.scales[6].isnan()
    assert not rows.codes[:, 300:].any()
    v = rows.dequantize()
    assert v[4].isnan().all() and v[6].isnan().all() and (v[2] == 0).all()
    keep = [0, 1, 3, 5, 7]
    assert torch.equal(rows.codes[keep], clean.codes[keep]) and torch.equal(rows.scales[keep], clean.scales[keep])


def test_differences():
    """The gradients in float32 against central differences of the output: the
    loss sum(dy y) + sum(dH h) along random directions. With steps e the
    difference quotient is off by e^2 times the third derivative (a few 1e-6
    here) and by the fp32 rounding of y over e: sqrt(M K) u max|dy y| / e."""
    from ternary_weight_quantization_amd.norm import rms_norm

    note("rms differences")
    M, K = 6, 96
    x, r, w = make(M, K, F32, F32, F32, True, seed=21)
    dy, dH = randn(M, K, seed=22, dtype=F32), randn(M, K, seed=23, dtype=F32)
    leaves = [t.requires_grad_(True) for t in (x, r, w)]
    y, h = rms_norm(x, w, r, out_dtype=F32)
    grads = torch.autograd.grad([y, h], leaves, [dy, dH])

    def loss(x, w, r):
        with torch.no_grad():
            y, h = rms_norm(x, w, r, out_dtype=F32)
            return (y.double() * dy.double()).sum() + (h.double() * dH.double()).sum()

    e = 2.0 ** -7
    for i, k in enumerate("xrw"):
        p = randn(*leaves[i].shape, seed=30 + i, dtype=F32)
        a = {"x": x, "w": w, "r": r}
        up = loss(**{**a, k: (a[k] + e * p).detach()})
        dn = loss(**{**a, k: (a[k] - e * p).detach()})
        got, want = (grads[i].double() * p.double()).sum().item(), ((up - dn) / (2 * e)).item()
        size = (grads[i].double() * p.double()).abs().sum().item()
        assert abs(got - want) <= 1e-3 * size, (k, got, want, size)


def test_one_output_used():
    """Only the norm's output, or only the stream, goes into the loss."""
    from ternary_weight_quantization_amd.norm import rms_norm

    note("rms one output used")
    x, r, w = make(7, 200, BF, BF, BF, True, seed=5)
    leaves = [t.requires_grad_(True) for t in (x, r, w)]
    dy = randn(7, 200, seed=6)
    y, h = rms_norm(x, w, r)
    gx, gr, gw = torch.autograd.grad(y, leaves, dy, retain_graph=True)
    zx, zr, zw = torch.autograd.grad([y, h], leaves, [dy, torch.zeros_like(h)], retain_graph=True)
    assert torch.equal(gx, zx) and torch.equal(gr, zr) and torch.equal(gw, zw) and torch.equal(gx, gr)
    hx, hr, hw = torch.autograd.grad(h, leaves, dy)
    assert torch.equal(hx, dy) and torch.equal(hr, dy) and not hw.any()
    # each leaf alone
    for i in range(3):
        y, h = rms_norm(x, w, r, quantize=True)
        g, = torch.autograd.grad([y.dequantize(), h], leaves[i:i + 1], [dy, dy])
        y, h = rms_norm(x, w, r, quantize=True)
        assert torch.equal(g, torch.autograd.grad([y.dequantize(), h], leaves, [dy, dy])[i])


def test_shapes_strides_and_empty_batches():
    from ternary_weight_quantization_amd.norm import QATRMSNorm, rms_norm

    note("rms shapes")
    x = randn(4, 6, 250, seed=1)
    w = randn(250, seed=2)
    y = rms_norm(x, w)
    assert y.shape == x.shape
    t = x.transpose(0, 1)
    assert torch.equal(rms_norm(t, w), y.transpose(0, 1))
    assert torch.equal(rms_norm(x[0, 0], w), y[0, 0])  # one vector
    part = randn(9, 500, seed=3)[:, 3:253]  # rows at a stride, off alignment
    assert torch.equal(rms_norm(part, w), rms_norm(part.contiguous(), w))
    rows = rms_norm(x, w, quantize=True)
    assert rows.shape == x.shape and rows.codes.shape == (24, 256)
    assert torch.equal(rows.dequantize().flatten(0, 1), rms_norm(x.flatten(0, 1), w, quantize=True).dequantize())
    wide = torch.full((260,), float("nan"), device="cuda", dtype=BF)  # a weight that starts off alignment
    wide[1:251] = w
    assert torch.equal(rms_norm(x, wide[1:251]), y)
    m = QATRMSNorm(250, quantize=True)
    e = torch.empty(0, 3, 250, device="cuda", dtype=BF, requires_grad=True)
    rows, h = m(e, torch.empty_like(e))
    assert rows.shape == (0, 3, 250) and h.shape == (0, 3, 250)
    (rows.dequantize().float().sum() + h.float().sum()).backward()
    assert e.grad.shape == e.shape and not m.weight.grad.any()
    assert "quantize=True" in repr(m)


def test_the_binding_and_a_workspace_of_garbage():
    """The C entry points directly: every output, a workspace full of NaN."""
    from ternary_weight_quantization_amd import binding as B

    note("rms binding")
    M, K = 70, 1001
    x, r, w = make(M, K, BF, F32, F32, True, seed=9)
    h, y, rstd = torch.empty_like(r), torch.empty(M, K, device="cuda"), torch.empty(M, device="cuda")
    B.bitnet_rmsnorm_fwd(x, w, 1e-6, res=r, h=h, y=y, rstd=rstd)
    xq, sx = torch.full((M, 1024), 77, dtype=torch.int8, device="cuda"), torch.empty(M, device="cuda")
    h2 = torch.empty_like(h)
    B.bitnet_rmsnorm_fwd(x, w, 1e-6, res=r, h=h2, x_q=xq, s_x=sx)
    assert torch.equal(h, h2) and not xq[:, K:].any()
    dY, dH = randn(M, K, seed=10, dtype=F32), randn(M, K, seed=11, dtype=F32)
    outs = []
    for fill in (float("nan"), 0.0):
        ws = torch.full((B.bitnet_rmsnorm_workspace_bytes(M, K) // 4,), fill, device="cuda")
        dh, dx, dw = torch.empty_like(h), torch.empty_like(x), torch.empty_like(w)
        B.bitnet_rmsnorm_bwd(dY, h, w, rstd, dH=dH, dh=dh, dx=dx, dw=dw, workspace=ws)
        outs.append((dh, dx, dw))
    assert all(torch.equal(a, b) for a, b in zip(*outs))
    assert torch.equal(outs[0][1], outs[0][0].to(BF))
    only = torch.empty_like(x)
    B.bitnet_rmsnorm_bwd(dY, h, w, rstd, dH=dH, dx=only)
    assert torch.equal(only, outs[0][1])
    v = torch.empty(M, K, device="cuda", dtype=BF)
    B.bitnet_rows_unpack(xq, sx, v)
    assert torch.equal(v, (xq[:, :K].float() * (sx / 127.0)[:, None]).to(BF))


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("K", [1, 8, 65, 1000, 4099])
def test_rows_quant(dtype, K):
    """8-bit rows of given activations: exact."""
    from ternary_weight_quantization_amd import binding as B

    note(f"rows_quant {dtype} K={K}")
    x = randn(11, K, seed=K, dtype=dtype)
    x[3] = 0
    if K > 8:
        x[5, :] = 127.0 * 2.0 ** -8
        x[5, 1::2] = 2.5 * 2.0 ** -8  # ties to even
    Kp = -(-K // 64) * 64
    q, s = torch.full((11, Kp), 55, dtype=torch.int8, device="cuda"), torch.empty(11, device="cuda")
    B.bitnet_rows_quant(x, q, s)
    ref_s = x.float().abs().amax(1).clamp(min=1e-8)
    ref = torch.round(127.0 * x.double() / ref_s.double()[:, None])
    assert torch.equal(s, ref_s) and torch.equal(q[:, :K].double(), ref) and not q[:, K:].any()
