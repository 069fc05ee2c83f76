"""The gated pair of ternary projections on the GPU against its formulas in 64
bits.

Bounds. The products are exact integers; u = 2^-24, h = 2^-8 (half a bf16 step).
g and u carry a conversion and three fp32 products, 4 u each; act(g) in fp32 is
within (16 + 2 |g|) u for silu (the exponent's argument is off by its rounding,
|g| u) and 10 u for relu2, |g| < 88, so y is within h |y| + (24 + 2 |g|) u |y|,
and every slope p = u act'(g), a = act(g) within E = 2^-16 + (24 + 2|g|) u of the
magnitudes of its terms (2^-16: cut off at 24 bits; silu's act' is a sum whose
terms' magnitudes are t and |a| (1 - t)).
D = bf16(dY p gamma c) is off by h |D| + that. Sums of n products in fp32 add
n u of the sum of their magnitudes.
  |err dX| <= h |dX| + sum_n (h + E + 2N u) |Dg qg| + ... (both halves)
  |err dW| <= h |dW| + sum_m (h + E + M u) |D xq|
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


def weights(N, K, seed, dtype=BF, up=3.0):
    """Two weights of different scales."""
    return (randn(N, K, seed=seed, dtype=F32) / K ** 0.5).to(dtype), (up * randn(N, K, seed=seed + 1, dtype=F32) / K ** 0.5).to(dtype)


def rows64(x):
    s = x.float().abs().amax(1).clamp(min=1e-8)
    return torch.round(127.0 * x.double() / s.double()[:, None]), s


def ternary64(w):
    gamma = w.double().abs().mean().float().clamp(min=1e-8)
    return torch.sign(w.double()) * (w.double().abs() > gamma.double() / 2), gamma


class Ref:
    """The formulas in 64 bits with the bounds' terms."""

    def __init__(self, x, wg, wu, act):
        self.q, self.s = rows64(x.detach())
        (self.tg, self.gg), (self.tu, self.gu) = ternary64(wg.detach()), ternary64(wu.detach())
        c = self.c = self.s.double()[:, None] / 127.0
        g, u = (self.q @ self.tg.t()) * c * self.gg.double(), (self.q @ self.tu.t()) * c * self.gu.double()
        if act == "silu":
            t = torch.sigmoid(g)
            self.a, da = g * t, t + g * t * (1 - t)
            mag = t + (g * t * (1 - t)).abs()
        else:
            r = g.clamp(min=0)
            self.a, da = r * r, 2 * r
            mag = da
        self.y, self.p = self.a * u, da * u
        self.rel = (24 + 2 * g.abs().clamp(max=100)) * U
        self.pm = mag * u.abs()

    def grads(self, dy):
        dy = dy.double()
        dg, du = dy * self.p, dy * self.a
        gg, gu = self.gg.double(), self.gu.double()
        x = self.q * self.c
        dx = (dg @ self.tg) * gg + (du @ self.tu) * gu
        dwg, dwu = dg.t().contiguous() @ x, du.t().contiguous() @ x
        E = 2.0 ** -16 + self.rel
        eg, eu = H * dg.abs() + E * dy.abs() * self.pm, (H + E) * du.abs()  # errors of D over its scales
        M, N = dy.shape
        tx = H * dx.abs() + ((eg + 2 * N * U * dg.abs()) @ self.tg.abs()) * gg + ((eu + 2 * N * U * du.abs()) @ self.tu.abs()) * gu
        tg = H * dwg.abs() + (eg + M * U * dg.abs()).t().contiguous() @ x.abs()
        tu = H * dwu.abs() + (eu + M * U * du.abs()).t().contiguous() @ x.abs()
        return (dx, dwg, dwu), (tx, tg, tu)


def close(name, got, want, tol, norm=True):
    err = (got.double() - want).abs()
    assert (err <= tol * (1 + 1e-6) + 1e-30).all(), (name, (err / (tol + 1e-30)).max().item())
    if norm and want.numel() > 4096 and want.norm() > 0:
        assert (err.norm() / want.norm()).item() <= H, (name, (err.norm() / want.norm()).item())


def check(M, K, N, act="silu", dtype=BF, seed=0, shape=None):
    from ternary_weight_quantization_amd.ffn import gated_bitlinear, gated_bitlinear_inference

    note(f"gated M={M} K={K} N={N} {act} {dtype}")
    x = randn(M, K, seed=seed).requires_grad_(True)
    wg, wu = (w.requires_grad_(True) for w in weights(N, K, seed + 1, dtype))
    y = gated_bitlinear(x, wg, wu, act)
    dy = randn(M, N, seed=seed + 5)
    grads = torch.autograd.grad(y, (x, wg, wu), dy)
    ref = Ref(x, wg, wu, act)
    assert y.dtype == BF and y.shape == (M, N)
    close("y", y, ref.y, (H + ref.rel) * ref.y.abs(), norm=False)
    want, tol = ref.grads(dy)
    for name, g, w, t, dt in zip(("dX", "dWg", "dWu"), grads, want, tol, (BF, dtype, dtype)):
        assert g.dtype == dt
        close(name, g, w, t)
    with torch.no_grad():
        assert torch.equal(gated_bitlinear(x, wg, wu, act), y)
    return x, wg, wu, y, dy, grads


@pytest.mark.parametrize("M", [1, 2, 31, 32, 33, 64, 65, 130, 257])
@pytest.mark.parametrize("act", ["silu", "relu2"])
def test_tokens(M, act):
    check(M, 200, 150, act, seed=M)


@pytest.mark.parametrize("K", [1, 3, 63, 64, 65, 127, 130, 1000, 2100])
@pytest.mark.parametrize("M", [5, 70])
def test_inner_widths(M, K):
    check(M, K, 72, seed=K)


@pytest.mark.parametrize("N", [1, 2, 7, 15, 16, 17, 63, 64, 65, 127, 128, 129, 200, 257, 333])
@pytest.mark.parametrize("M", [5, 70])
def test_outer_widths(M, N):
    check(M, 96, N, "relu2", seed=N)


@pytest.mark.parametrize("M", [9, 300])
def test_float_masters(M):
    check(M, 192, 140, dtype=F32, seed=4)


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
                                   (256, 64, 33), (257, 130, 70), (333, 1000, 1001), (129, 700, 9000), (400, 320, 6000),
                                   (1000, 65, 2050), (40, 130, 9001), (64, 64, 33000)])
def test_few_tokens_have_the_bits_of_the_tiles(M, K, N):
    from ternary_weight_quantization_amd.ffn import gated_bitlinear

    x, (wg, wu) = randn(M, K, seed=1), weights(N, K, 2)
    few = gated_bitlinear(x, wg, wu)
    a = x.clone().requires_grad_(True)
    saved = gated_bitlinear(a, wg, wu)
    dx, = torch.autograd.grad(saved, a, torch.ones_like(saved))
    assert torch.equal(saved, few)
    with knobs(no_skinny=1):
        assert torch.equal(gated_bitlinear(x, wg, wu), few)
        y = gated_bitlinear(a, wg, wu)
    if M > 64:  # dX from the slopes that either kernel saved
        dx2, = torch.autograd.grad(y, a, torch.ones_like(y))
        assert torch.equal(dx, dx2)


def test_split_tiles_have_the_bits_of_whole_ones():
    from ternary_weight_quantization_amd import binding as B

    M, K, N = 300, 700, 200
    note("gated split")
    _, wg, wu, y, dy, grads = check(M, K, N, seed=3)
    for ctas in (-1, 3, 37):
        with knobs(split_ctas=ctas):
            _, _, _, y2, _, grads2 = check(M, K, N, seed=3)
        assert torch.equal(y, y2)
    assert B.bitnet_split_timeouts() == 0


def test_gradients_one_at_a_time():
    from ternary_weight_quantization_amd.ffn import gated_bitlinear

    for M in (20, 90):
        x, wg, wu, y, dy, grads = check(M, 128, 96, seed=8)
        for i, leaf in enumerate((x, wg, wu)):
            got, = torch.autograd.grad(gated_bitlinear(x, wg, wu), leaf, dy)
            want, tol = Ref(x, wg, wu, "silu").grads(dy)
            close(i, got, want[i], tol[i])


def test_frozen_and_rows():
    """The stored state and 8-bit rows give the training forward's bits; the
    frozen gradient of x is the formula's."""
    from ternary_weight_quantization_amd.ffn import QATGatedBitLinear, gated_bitlinear, gated_bitlinear_inference
    from ternary_weight_quantization_amd.norm import rms_norm

    for M in (1, 6, 100):
        note(f"gated frozen M={M}")
        m = QATGatedBitLinear(130, 77, act="relu2")
        with torch.no_grad():
            m.up_weight.mul_(2.5)
        x = randn(M, 130, seed=M).requires_grad_(True)
        y = m(x)
        dy = randn(M, 77, seed=3)
        gx, = torch.autograd.grad(y, x, dy)
        packed, gamma = m.export_inference()
        assert torch.equal(gated_bitlinear_inference(x, packed, gamma, 130, "relu2"), y)
        m.freeze()
        assert m.frozen and "frozen" in repr(m)
        y2 = m(x)
        assert torch.equal(y2, y)
        fx, = torch.autograd.grad(y2, x, dy)
        want, tol = Ref(x, m.gate_weight, m.up_weight, "relu2").grads(dy)
        close("frozen dX", fx, want[0], tol[0])
        with torch.no_grad():
            m.gate_weight.zero_()
        assert torch.equal(m(x), y) and not m.unfreeze()(x).any()
        # rows: as the activations that they stand for, quantized
        m2 = QATGatedBitLinear(130, 77)
        w = torch.nn.Parameter(randn(130, seed=9))
        rows = rms_norm(x, w, quantize=True)
        y3 = m2(rows)
        g3 = torch.autograd.grad(y3, [x, w, m2.gate_weight, m2.up_weight], dy, retain_graph=True)
        g4 = torch.autograd.grad(m2(rows), [x, w, m2.gate_weight, m2.up_weight], dy)
        assert all(torch.equal(a, b) for a, b in zip(g3, g4))
        v = rows.detach().dequantize().float()
        ref = Ref.__new__(Ref)
        q, s = rows.codes[:, :130].double(), rows.scales
        assert ((v.double() - q * (s.double() / 127)[:, None]).abs() <= H * v.double().abs() + 1e-30).all()
        with torch.no_grad():
            assert torch.equal(m2(rows.detach()), y3)
            m2.freeze()
            assert torch.equal(m2(rows.detach()), y3)


def test_extremes():
    """Weights of zeros, rows of zeros and NaN, large gates."""
    from ternary_weight_quantization_amd.ffn import gated_bitlinear

    note("gated extremes")
    for M in (8, 80):
        x, (wg, wu) = randn(M, 100, seed=1), weights(60, 100, 2)
        ok = gated_bitlinear(x, wg, wu)
        x[3], x[5, 9] = 0, float("nan")
        for act in ("silu", "relu2"):
            xx, a, b = x.clone().requires_grad_(True), wg.clone().requires_grad_(True), wu.clone().requires_grad_(True)
            y = gated_bitlinear(xx, a, b, act)
            assert (y[3] == 0).all() and y[5].isnan().all()
            keep = [i for i in range(M) if i not in (3, 5)]
            assert y[keep].isfinite().all()
            if act == "silu":
                assert torch.equal(y[keep], ok[keep])
        z = torch.zeros_like(wg).requires_grad_(True)
        x2 = randn(M, 100, seed=4).requires_grad_(True)
        y = gated_bitlinear(x2, z, wu)
        gx, gz = torch.autograd.grad(y, (x2, z), torch.ones_like(y))
        assert not y.any() and not gx.any()
        want, tol = Ref(x2, z, wu, "silu").grads(torch.ones_like(y))
        close("dWg at zero", gz, want[1], tol[1])
        # gates beyond the exponential's range on both sides
        big = (wg.float() * 400).to(BF)
        y = gated_bitlinear(x2, big, wu)
        assert y.isfinite().all()
        ref = Ref(x2, big, wu, "silu")
        tol = (H + ref.rel) * ref.y.abs() + (24 * U * ref.a.abs().clamp(max=1.0) + 2.0 ** -100) * 1e3
        assert ((y.double() - ref.y).abs() <= tol).all()


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("K", [1, 5, 64, 130, 520, 2555, 4104, 8200, 16384, 16390])
def test_both_weights_and_the_rows_together(dtype, K):
    """Two weights ternarized together have the bits that each has alone, whatever
    the workspace held, and the rows' codes are those of the rows alone."""
    from ternary_weight_quantization_amd import binding as B
    from ternary_weight_quantization_amd.layer import ternarize

    note(f"quantize2 {dtype} K={K}")
    Kp, N = -(-K // 64) * 64, 75
    wg, wu = weights(N, K, K, dtype)
    x = randn(37, K, seed=K + 2)
    q1, s1 = (torch.empty(37, Kp, dtype=torch.int8, device="cuda"), torch.empty(37, device="cuda"))
    B.bitnet_rows_quant(x, q1, s1)
    for fill in (0xFF, 0):
        ws = torch.full((B.bitnet_ternarize_workspace_bytes(N, K),), fill, dtype=torch.uint8, device="cuda")
        for rows in (x, None):
            packed = torch.full((2 * N, Kp // 4), 0x55, dtype=torch.uint8, device="cuda")
            gamma = torch.zeros(2, device="cuda")
            q, s = torch.full((37, Kp), 7, dtype=torch.int8, device="cuda"), torch.zeros(37, device="cuda")
            B.bitnet_quantize2(wg, wu, rows, packed, gamma, q, s, ws)
            for i, w in enumerate((wg, wu)):
                p, g = ternarize(w)
                assert torch.equal(packed[i * N:(i + 1) * N], p) and torch.equal(gamma[i:i + 1], g.reshape(1))
            if rows is not None:
                assert torch.equal(q, q1) and torch.equal(s, s1)
            else:
                assert (q == 7).all() and not s.any()


@pytest.mark.parametrize("K", [8, 64, 100, 2048, 2555, 2560, 4096, 4100, 6912, 8192])
@pytest.mark.parametrize("N", [1, 16, 75])
def test_rows_taken_as_they_are(K, N):
    """Few tokens of bf16 rows have the bits of their 8-bit rows, from any element
    on, a NaN kept to its row."""
    from ternary_weight_quantization_amd import binding as B
    from ternary_weight_quantization_amd.layer import ternarize

    note(f"gated rows as they are K={K} N={N}")
    (pg, gg), (pu, gu) = (ternarize(w) for w in weights(N, K, K))
    packed, gamma = torch.cat([pg, pu]), torch.cat([gg, gu])
    Kp = packed.shape[1] * 4
    for M in range(1, B.bitnet_rows_direct(K) + 1):
        for off in (0, 1):
            x = randn(M * K + 1, seed=M)[off:off + M * K].view(M, K)
            x[M - 1, K // 3] = 0 if off else 77.0
            x[0] *= 0.0 if M > 2 else 1.0
            if M == 2:
                x[1, K - 1] = float("nan")
            q, s = torch.empty(M, Kp, dtype=torch.int8, device="cuda"), torch.empty(M, device="cuda")
            B.bitnet_rows_quant(x, q, s)
            for act in (B.BITNET_ACT_SILU, B.BITNET_ACT_RELU2):
                y, y2 = torch.empty(M, N, dtype=BF, device="cuda"), torch.zeros(M, N, dtype=BF, device="cuda")
                sl, sl2 = (torch.zeros(B.bitnet_gated_slopes_bytes(M, N), dtype=torch.uint8, device="cuda") for _ in range(2))
                B.bitnet_gated_fwd(act, q, s, packed, gamma, K, y, sl)
                B.bitnet_gated_fwd(act, None, None, packed, gamma, K, y2, sl2, x=x)
                assert torch.equal(y.view(torch.int16), y2.view(torch.int16)) and torch.equal(sl, sl2)
                assert y2[1].isnan().all() if M == 2 else y2.isfinite().all()


def test_shapes_and_empty_batches():
    from ternary_weight_quantization_amd.ffn import QATGatedBitLinear, gated_bitlinear

    note("gated shapes")
    wg, wu = weights(40, 66, 1)
    x = randn(3, 5, 66, seed=2)
    y = gated_bitlinear(x, wg, wu)
    assert y.shape == (3, 5, 40)
    assert torch.equal(gated_bitlinear(x.transpose(0, 1), wg, wu), y.transpose(0, 1))
    assert torch.equal(gated_bitlinear(x[1, 1], wg, wu), y[1, 1])
    assert torch.equal(gated_bitlinear(x, torch.cat([wg, wu], 1)[:, :66], wu), y)  # rows at a stride
    m = QATGatedBitLinear(66, 40)
    e = torch.empty(0, 66, device="cuda", dtype=BF, requires_grad=True)
    m(e).float().sum().backward()
    assert e.grad.shape == e.shape and not m.gate_weight.grad.any() and not m.up_weight.grad.any()
    m.freeze()
    assert m(e).shape == (0, 40)


def test_a_workspace_of_garbage():
    from ternary_weight_quantization_amd import binding as B

    note("gated workspace")
    M, K, N = 90, 130, 75
    x, (wg, wu) = randn(M, K, seed=1), weights(N, K, 2)
    from ternary_weight_quantization_amd.layer import act_quant, ternarize
    xq, sx = act_quant(x)
    (pg, gg), (pu, gu) = ternarize(wg), ternarize(wu)
    packed, gamma = torch.cat([pg, pu]), torch.cat([gg, gu])
    dY = randn(M, N, seed=3)
    outs = []
    for fill in (0xFF, 0x00):
        y = torch.empty(M, N, dtype=BF, device="cuda")
        slopes = torch.full((B.bitnet_gated_slopes_bytes(M, N),), fill, dtype=torch.uint8, device="cuda")
        B.bitnet_gated_fwd(B.BITNET_ACT_SILU, xq, sx, packed, gamma, K, y, slopes)
        ws = torch.full((B.bitnet_gated_bwd_workspace_bytes(M, N, K),), fill, dtype=torch.uint8, device="cuda")
        dX, dg, du = torch.empty_like(x), torch.empty_like(wg), torch.empty_like(wu)
        B.bitnet_gated_bwd(dY, slopes, xq, sx, packed, gamma, K, dX=dX, dW_gate=dg, dW_up=du, workspace=ws)
        outs.append((y, dX, dg, du))
    assert all(torch.equal(a, b) for a, b in zip(*outs))
