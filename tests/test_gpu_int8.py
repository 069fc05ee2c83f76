"""The linear layer in 8-bit integers on the GPU against its formulas in 64 bits.

Bounds. The products are exact integers; u = 2^-24, h = 2^-8 (half a bf16 step).
y carries a conversion to fp32, the scales' quotients and products and the
bias' addition: h |y| + 8 u (|acc sx sw / 127^2| + |b|). x_hat and w_hat are
rounded to bf16 (h) after two fp32 operations, sums of n products add n u of the
sum of their magnitudes:
  |err dX| <= h |dX| + (h + (4 + N) u) sum_n |dY w_hat|
  |err dW| <= h |dW| + (h + (4 + M) u) sum_m |dY x_hat|,  |err db| <= h |db| + M u sum|dY|
and, the roundings being independent, the error's norm is about
sqrt(2) h / sqrt(3) = 0.0032 of the result's, checked as h.
"""

import pytest
import torch

from tests.gpu_util import knobs, note

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32
U = 2.0 ** -24
H = 2.0 ** -8


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.fail("no GPU visible")
    from ternary_weight_quantization_amd import binding
    binding.lib()


def randn(*shape, seed, dtype=BF):
    g = torch.Generator().manual_seed(seed)
    return torch.randn(*shape, generator=g).to(device="cuda", dtype=dtype)


def rows64(x):
    s = x.float().abs().amax(1).clamp(min=1e-8)
    return torch.round(127.0 * x.double() / s.double()[:, None]), s.double()[:, None]


def close(name, got, want, tol, norm=True):
    err = (got.double() - want).abs()
    assert (err <= tol * (1 + 1e-6) + 1e-30).all(), (name, (err / (tol + 1e-30)).max().item())
    if norm and want.numel() > 4096:
        assert (err.norm() / want.norm()).item() <= H, (name, (err.norm() / want.norm()).item())


def check(M, K, N, dtype=BF, bias=BF, seed=0):
    from ternary_weight_quantization_amd.int8_layer import int8_linear

    note(f"int8 M={M} K={K} N={N} {dtype} bias={bias}")
    x = randn(M, K, seed=seed).requires_grad_(True)
    # channels of very different scales
    w = (randn(N, K, seed=seed + 1, dtype=F32) * torch.logspace(-2, 2, N, device="cuda")[:, None]).to(dtype).requires_grad_(True)
    b = None if bias is None else randn(N, seed=seed + 2, dtype=bias).requires_grad_(True)
    y = int8_linear(x, w, b)
    dy = randn(M, N, seed=seed + 3)
    leaves = [t for t in (x, w, b) if t is not None]
    grads = torch.autograd.grad(y, leaves, dy)
    with torch.no_grad():
        (q, s), (wq, sw) = rows64(x), rows64(w)
        xh, wh = q * s / 127.0, wq * sw / 127.0
        p = (q @ wq.t()) * (s * sw.t() / 127.0 ** 2)  # whole numbers: a sum that is 0 is 0
        bd = 0.0 if b is None else b.to(BF).double()
        ref = p + bd
        assert y.dtype == BF and y.shape == (M, N)
        close("y", y, ref, H * ref.abs() + 8 * U * (p.abs() + (0.0 if b is None else bd.abs())), norm=False)
        d = dy.double()
        dx, dw = d @ wh, d.t().contiguous() @ xh
        close("dX", grads[0], dx, H * dx.abs() + (H + (4 + N) * U) * (d.abs() @ wh.abs()))
        close("dW", grads[1], dw, H * dw.abs() + (H + (4 + M) * U) * (d.abs().t().contiguous() @ xh.abs()))
        assert grads[0].dtype == BF and grads[1].dtype == dtype
        if b is not None:
            db = d.sum(0)
            assert grads[2].dtype == bias
            close("db", grads[2], db, H * db.abs() + M * U * d.abs().sum(0), norm=False)
        assert torch.equal(int8_linear(x, w, b), y)
    return x, w, b, y, dy, grads


@pytest.mark.parametrize("M", [1, 2, 31, 32, 33, 63, 64, 65, 130, 257])
def test_tokens(M):
    check(M, 200, 150, seed=M)


@pytest.mark.parametrize("K", [1, 3, 63, 64, 65, 127, 128, 130, 1000, 2100, 4099])
@pytest.mark.parametrize("M", [5, 40, 70])
def test_inner_widths(M, K):
    check(M, K, 72, bias=None, seed=K)


@pytest.mark.parametrize("N", [1, 2, 7, 31, 32, 33, 64, 65, 128, 255, 256, 257, 333])
@pytest.mark.parametrize("M", [5, 70])
def test_outer_widths(M, N):
    check(M, 96, N, seed=N)


@pytest.mark.parametrize("bias", [None, BF, F32])
@pytest.mark.parametrize("dtype", [BF, F32])
def test_types(dtype, bias):
    check(9, 192, 140, dtype, bias, seed=4)
    check(300, 192, 140, dtype, bias, seed=5)


def test_several_tiles():
    check(530, 333, 715, seed=11)


@pytest.mark.parametrize("M,K,N", [(66, 131, 75), (300, 333, 141), (1100, 70, 65)])
def test_float_masters_of_odd_widths(M, K, N):
    check(M, K, N, dtype=F32, seed=M)


@pytest.mark.parametrize("M,K,N", [(70, 130, 75), (300, 192, 140), (530, 333, 715)])
def test_the_large_tiles(M, K, N):
    """Sizes that take smaller tiles, on those of long batches."""
    with knobs(no_skinny=1):
        check(M, K, N, seed=M)


@pytest.mark.parametrize("M,K,N", [(3, 130, 70), (40, 300, 129), (64, 64, 33), (65, 300, 129), (130, 2555, 77),
                                   (192, 130, 4000), (256, 64, 10000), (256, 1000, 13), (257, 130, 70), (333, 1000, 1001),
                                   (129, 700, 18000), (400, 320, 13000), (1000, 65, 4100), (20, 64, 33000),
                                   (40, 130, 17001), (64, 64, 70000)])
def test_few_tokens_have_the_bits_of_the_tiles(M, K, N):
    from ternary_weight_quantization_amd.int8_layer import int8_linear

    x, w, b = randn(M, K, seed=1), randn(N, K, seed=2), randn(N, seed=3)
    few = int8_linear(x, w, b)
    with knobs(no_skinny=1):
        assert torch.equal(int8_linear(x, w, b), few)


def test_split_tiles_have_the_bits_of_whole_ones():
    from ternary_weight_quantization_amd import binding as B

    note("int8 split")
    y = check(300, 700, 400, seed=3)[3]
    for ctas in (-1, 3, 37):
        with knobs(split_ctas=ctas):
            assert torch.equal(check(300, 700, 400, seed=3)[3], y)
    assert B.bitnet_split_timeouts() == 0


def test_the_largest_sums():
    """Codes of +-127 throughout, K = 131072: int32 sums of 2.1e9."""
    from ternary_weight_quantization_amd.int8_layer import int8_linear

    K = 131072
    for M in (2, 70):
        note(f"int8 largest sums M={M}")
        x = torch.ones(M, K, device="cuda", dtype=BF)
        w = torch.ones(9, K, device="cuda", dtype=BF)
        w[1::2] = -1
        y = int8_linear(x, w)
        assert (y[:, ::2] == K).all() and (y[:, 1::2] == -K).all()


@pytest.mark.parametrize("M,N", [(1, 1), (15, 8), (16, 2047), (33, 2048), (70, 2049), (1500, 5000), (40000, 9)])
def test_bias_gradient(M, N):
    """Column sums of dY, odd and even widths, more and fewer rows than groups: at
    most M / 256 + 32 additions in a group, then 16 and 16 of the groups."""
    from ternary_weight_quantization_amd import binding as B

    note(f"int8 bias gradient M={M} N={N}")
    dY, K = randn(M, N, seed=M), 8
    for dt in (BF, F32):
        db = torch.empty(N, dtype=dt, device="cuda")
        B.bitnet_int8_bwd(dY, None, None, None, None, K, db=db)
        want = dY.double().sum(0)
        tol = torch.finfo(dt).eps / 2 * want.abs() + (M / 64 + 96) * U * dY.double().abs().sum(0)
        assert ((db.double() - want).abs() <= tol).all()


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("K", [5, 64, 130, 1000, 1030, 2555, 4104, 16384, 16390])
def test_weight_and_activations_quantized_together(dtype, K):
    """One launch for both, each exactly what the rows alone give."""
    from ternary_weight_quantization_amd import binding as B

    note(f"rows_quant2 {dtype} K={K}")
    Kp = -(-K // 64) * 64
    x, w = randn(7, K, seed=K), randn(9, K, seed=K + 1, dtype=dtype)
    new = lambda n: (torch.full((n, Kp), 7, dtype=torch.int8, device="cuda"), torch.zeros(n, device="cuda"))  # noqa: E731
    (xq, sx), (wq, sw) = new(7), new(9)
    B.bitnet_rows_quant2(x, xq, sx, w, wq, sw)
    for t, q, s in ((x, xq, sx), (w, wq, sw)):
        ref, rs = rows64(t)
        assert torch.equal(q[:, :K].double(), ref) and torch.equal(s.double()[:, None], rs) and not q[:, K:].any()
        q1, s1 = new(len(t))
        B.bitnet_rows_quant(t, q1, s1)
        assert torch.equal(q1, q) and torch.equal(s1, s)


@pytest.mark.parametrize("K", [8, 64, 100, 2048, 2555, 2560, 4096, 4100, 6912, 8192])
@pytest.mark.parametrize("N", [1, 16, 75])
def test_rows_taken_as_they_are(K, N):
    """Few tokens of bf16 rows have the bits of their 8-bit rows, from any element on, a
    NaN kept to its row."""
    from ternary_weight_quantization_amd import binding as B

    note(f"int8 rows as they are K={K} N={N}")
    Kp = -(-K // 64) * 64
    new = lambda n: (torch.empty(n, Kp, dtype=torch.int8, device="cuda"), torch.empty(n, device="cuda"))  # noqa: E731
    wq, sw = new(N)
    B.bitnet_rows_quant(randn(N, K, seed=K), wq, sw)
    b = randn(N, seed=K + 1)
    for M in range(1, B.bitnet_rows_direct(K) + 1):
        for off in (0, 1):
            x = randn(M * K + 1, seed=M)[off:off + M * K].view(M, K)
            x[M - 1, K // 3] = 0 if off else 77.0
            x[0] *= 0.0 if M > 2 else 1.0
            if M == 2:
                x[1, K - 1] = float("nan")
            q, s = new(M)
            B.bitnet_rows_quant(x, q, s)
            y, y2 = torch.empty(M, N, dtype=BF, device="cuda"), torch.zeros(M, N, dtype=BF, device="cuda")
            B.bitnet_int8_fwd(q, s, wq, sw, K, y, bias=b)
            B.bitnet_int8_fwd(None, None, wq, sw, K, y2, bias=b, x=x)
            assert torch.equal(y.view(torch.int16), y2.view(torch.int16))
            assert y2[1].isnan().all() if M == 2 else y2.isfinite().all()


def test_gradients_one_at_a_time():
    from ternary_weight_quantization_amd.int8_layer import int8_linear

    for M in (20, 90):
        x, w, b, y, dy, grads = check(M, 128, 97, seed=8)
        for i, leaf in enumerate((x, w, b)):
            got, = torch.autograd.grad(int8_linear(x, w, b), leaf, dy)
            if i == 2:
                assert torch.equal(got, grads[2])
            else:
                assert ((got.double() - grads[i].double()).norm() / grads[i].double().norm()) <= H


def test_frozen_and_rows():
    from ternary_weight_quantization_amd.int8_layer import QATInt8Linear, int8_linear_inference
    from ternary_weight_quantization_amd.norm import rms_norm

    for M in (1, 6, 100):
        note(f"int8 frozen M={M}")
        m = QATInt8Linear.from_linear(torch.nn.Linear(130, 77).cuda())
        x = randn(M, 130, seed=M).requires_grad_(True)
        y = m(x)
        dy = randn(M, 77, seed=3)
        gx, gb = torch.autograd.grad(y, [x, m.bias], dy)
        wq, sw = m.export_inference()
        assert wq.shape == (77, 192) and torch.equal(int8_linear_inference(x, wq, sw, 130, m.bias), y)
        m.freeze()
        assert m.frozen and "frozen" in repr(m)
        y2 = m(x)
        fx, fb = torch.autograd.grad(y2, [x, m.bias], dy)
        assert torch.equal(y2, y) and torch.equal(fb, gb)
        assert ((fx.double() - gx.double()).norm() / gx.double().norm()) <= H
        with torch.no_grad():
            m.weight.zero_()
        assert torch.equal(m(x), y)
        m2 = QATInt8Linear(130, 77)
        w = torch.nn.Parameter(randn(130, seed=9))
        rows = rms_norm(x, w, quantize=True)
        y3 = m2(rows)
        gx, gw, g2 = torch.autograd.grad(y3, [x, w, m2.weight], dy)
        q, s = rows.codes[:, :130].double(), rows.scales.double()[:, None]
        wq64, sw64 = rows64(m2.weight.detach())
        ref = (q @ wq64.t()) * (s * sw64.t() / 127.0 ** 2)
        mag = (q * s / 127.0).abs() @ (wq64 * sw64 / 127.0).abs().t()
        close("y", y3.detach(), ref, H * ref.abs() + 8 * U * mag, norm=False)
        dw = dy.double().t().contiguous() @ (q * s / 127.0)
        close("dW", g2, dw, H * dw.abs() + (H + (4 + M) * U) * (dy.double().abs().t().contiguous() @ (q * s / 127.0).abs()))
        with torch.no_grad():
            assert torch.equal(m2(rows.detach()), y3)
            m2.freeze()
            assert torch.equal(m2(rows.detach()), y3)


def test_rows_of_zeros_and_nan():
    from ternary_weight_quantization_amd.int8_layer import int8_linear, int8_linear_inference
    from ternary_weight_quantization_amd.norm import rms_norm

    note("int8 zeros and NaN")
    for M in (8, 80):
        x, w, b = randn(M, 100, seed=1), randn(60, 100, seed=2), randn(60, seed=3)
        x[3] = 0
        w[7] = 0
        y = int8_linear(x, w, b)
        assert torch.equal(y[3], b) and (y[:, 7] == b[7]).all()
        ok = int8_linear(rms_norm(x, quantize=True), w, b)
        x[5, 9] = float("nan")
        got = int8_linear(rms_norm(x, quantize=True), w, b)
        keep = [i for i in range(M) if i != 5]
        assert got[5].isnan().all() and torch.equal(got[keep], ok[keep])
        wf = w.float()
        wf[4, 3] = float("inf")  # a float channel that is not finite
        got = int8_linear(x[keep], wf, b)
        assert got[:, 4].isnan().all() and not got[:, :4].isnan().any()


def test_shapes_and_empty_batches():
    from ternary_weight_quantization_amd.int8_layer import QATInt8Linear, int8_linear

    note("int8 shapes")
    w, b = randn(40, 66, seed=1), randn(40, seed=4)
    x = randn(3, 5, 66, seed=2)
    y = int8_linear(x, w, b)
    assert y.shape == (3, 5, 40)
    assert torch.equal(int8_linear(x.transpose(0, 1), w, b), y.transpose(0, 1))
    assert torch.equal(int8_linear(x[1, 1], w, b), y[1, 1])
    assert torch.equal(int8_linear(x, torch.cat([w, w], 1)[:, :66], b), y)
    wide = torch.zeros(50, device="cuda", dtype=BF)
    wide[3:43] = b
    assert torch.equal(int8_linear(x, w, wide[3:43]), y)  # a bias off alignment
    m = QATInt8Linear(66, 40, bias=True)
    e = torch.empty(0, 66, device="cuda", dtype=BF, requires_grad=True)
    m(e).float().sum().backward()
    assert e.grad.shape == e.shape and not m.weight.grad.any() and not m.bias.grad.any()
    m.freeze()
    assert m(e).shape == (0, 40)


def test_a_workspace_of_garbage():
    from ternary_weight_quantization_amd import binding as B

    note("int8 workspace")
    M, K, N = 90, 130, 75
    xq, sx = torch.empty(M, 192, dtype=torch.int8, device="cuda"), torch.empty(M, device="cuda")
    wq, sw = torch.empty(N, 192, dtype=torch.int8, device="cuda"), torch.empty(N, device="cuda")
    B.bitnet_rows_quant(randn(M, K, seed=1), xq, sx)
    B.bitnet_rows_quant(randn(N, K, seed=2, dtype=F32), wq, sw)
    dY = randn(M, N, seed=3)
    outs = []
    for fill in (0xFF, 0x00):
        y = torch.empty(M, N, dtype=BF, device="cuda")
        B.bitnet_int8_fwd(xq, sx, wq, sw, K, y)
        ws = torch.full((B.bitnet_int8_bwd_workspace_bytes(M, N, K),), fill, dtype=torch.uint8, device="cuda")
        dX, dW, db = torch.empty(M, K, dtype=BF, device="cuda"), torch.empty(N, K, device="cuda"), torch.empty(N, device="cuda")
        B.bitnet_int8_bwd(dY, xq, sx, wq, sw, K, dX=dX, dW=dW, db=db, workspace=ws)
        only = torch.empty(N, device="cuda")
        B.bitnet_int8_bwd(dY, None, None, None, None, K, db=only, workspace=ws)
        assert torch.equal(only, db)
        outs.append((y, dX, dW, db))
    assert all(torch.equal(a, b) for a, b in zip(*outs))
