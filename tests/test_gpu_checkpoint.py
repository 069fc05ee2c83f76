"""8-bit checkpoints on the GPU: codes and scales bit for bit against their
definition, and the backward passes that read them against the formulas in 64
bits on the values the codes stand for.

Bounds. u = 2^-24; a rounding to bf16 is off by at most 2^-8 relative to the
value. A code's value q s / 127 takes two fp32 roundings (2 u, then the
output's). The gated activation's fp32 intermediates take fewer than 16
roundings; the exponential's argument g log2(e) is off by 2 u |g|, which the
exponential turns into a relative error, and exp2 and rcp are within 1 ulp
(2 u) each: E = (24 + 3 |g|) u relative to the terms' magnitudes.
"""

import pytest
import torch

from tests.gpu_util import note

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


def ref_codes(x):
    """(codes [M, Kc], scales [M, Kc/128]) of x [M, K] as float64; the
    quotient of fp32 values in 64 bits rounds to the exact quotient's
    integer, ties included."""
    M, K = x.shape
    v = torch.zeros(M, -(-K // 128) * 128, dtype=torch.float64, device=x.device)
    v[:, :K] = x.double()
    b = v.view(M, -1, 128)
    s = b.abs().amax(-1, keepdim=True)
    q = torch.round(127.0 * b / torch.where(s > 0, s, torch.ones_like(s)))
    return q.view(M, -1), s[..., 0]


def values(q, s, K):
    M = q.shape[0]
    return (q.view(M, -1, 128) * s[..., None] / 127.0).view(M, -1)[:, :K]


def randn(*shape, seed=0, dtype=BF):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return torch.randn(*shape, generator=g, device="cuda").to(dtype)


def check_pack(x):
    from ternary_weight_quantization_amd.checkpoint import compress, decompress

    M, K = x.shape
    codes, scales = compress(x)
    q, s = ref_codes(x)
    assert torch.equal(scales.double(), s)
    assert torch.equal(codes.double(), q), (codes.double() - q).abs().max()
    ref = values(q, s, K)
    # two fp32 roundings; the least fp32 and bf16 steps where values are subnormal
    for t, h, least in ((F32, 0.0, 2.0 ** -149), (BF, H, 2.0 ** -133)):
        got = decompress(codes, scales, K, t).double()
        assert ((got - ref).abs() <= (h + 2 * U) * ref.abs() + 127 * 2.0 ** -149 + least).all()


@pytest.mark.parametrize("K", [1, 2, 7, 8, 9, 15, 16, 17, 100, 127, 128, 129, 135, 136, 255, 257, 2555, 2560, 6905,
                               6912])
@pytest.mark.parametrize("M", [1, 3, 34])
@pytest.mark.parametrize("dtype", [BF, F32])
def test_pack_unpack(M, K, dtype):
    note(f"pack M={M} K={K} {dtype}")
    x = randn(M, K, seed=K, dtype=F32)
    x[:, ::5] *= 40.0
    check_pack(x.to(dtype))


@pytest.mark.parametrize("dtype", [BF, F32])
def test_ties_and_borders(dtype):
    """Scale 127 / 2^e: the quotients are the values times a power of two, so
    that half integers are exact ties; and fp32 neighbours of the ties."""
    rows = []
    for e in (0, 3, -20):
        half = torch.arange(-126.5, 127.0, 1.0, device="cuda")  # 254 ties
        row = torch.zeros(2 * 128, device="cuda")
        row[:127], row[127] = half[:127], 127.0
        row[128:255], row[255] = half[127:], -127.0
        rows.append(row * 2.0 ** e)
    x = torch.stack(rows)
    check_pack(x.to(dtype))
    if dtype == F32:
        check_pack(torch.nextafter(x, torch.full_like(x, 1e9)).clamp(-127 * 8.0, 127 * 8.0))
        check_pack(torch.nextafter(x, torch.full_like(x, -1e9)).clamp(-127 * 8.0, 127 * 8.0))


@pytest.mark.parametrize("scale", [1e-45, 3e-42, 1e-39, 1.1e-38, 4e-37, 3.8e-37, 1e-30, 1e-29, 1e30, 2.6e38])
def test_extreme_scales(scale):
    x = torch.linspace(-1, 1, 640, device="cuda").view(2, 320) * scale
    check_pack(x)
    check_pack(x.to(BF))


def test_zero_blocks_nan_and_infinity():
    from ternary_weight_quantization_amd.checkpoint import compress, decompress

    x = randn(3, 400, seed=1, dtype=F32)
    x[0, 128:256] = 0.0
    x[1, 5] = float("nan")
    x[2, 399] = float("-inf")
    codes, scales = compress(x)
    y = decompress(codes, scales, 400, F32)
    assert torch.equal(y[0, 128:256], torch.zeros(128, device="cuda"))
    assert torch.isnan(y[1, :128]).all() and torch.isfinite(y[1, 128:]).all()
    assert torch.isnan(y[2, 384:]).all() and torch.isfinite(y[2, :384]).all()
    assert torch.isfinite(y[0]).all()


def test_views_and_no_rows():
    from ternary_weight_quantization_amd.checkpoint import compress, decompress

    x = randn(10, 300, seed=2)
    want = compress(x)
    for t in (x.t().contiguous().t(), x.view(2, 5, 300), torch.cat([x, x], 1)[:, 300:]):
        got = compress(t)
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    codes, scales = compress(x[:0])
    assert codes.shape == (0, 384) and decompress(codes, scales, 300).shape == (0, 300)


# --- gated activation ------------------------------------------------------------

def act(name, g):
    if name == "silu":
        t = 1 / (1 + torch.exp(-g))
        return g * t, t * (1 + g * (1 - t))
    r = g.clamp(min=0)
    return r * r, 2 * r


def check_gate(gate, up, name, ckpt, dy):
    from ternary_weight_quantization_amd.checkpoint import gated_activation

    gate, up = gate.detach().requires_grad_(True), None if up is None else up.detach().requires_grad_(True)
    leaves = [t for t in (gate, up) if t is not None]
    y = gated_activation(gate, up, name, checkpoint=ckpt)
    grads = torch.autograd.grad(y, leaves, dy)
    with torch.no_grad():
        assert torch.equal(gated_activation(gate, up, name), y)
        K = gate.shape[-1]
        g = gate.double().reshape(-1, K)
        u = torch.ones_like(g) if up is None else up.double().reshape(-1, K)
        d = dy.double().reshape(-1, K)
        E = (24 + 3 * g.abs()) * U
        a, _ = act(name, g)
        ref = a * u
        # 2^-133: the least bf16 step
        assert ((y.double().reshape(-1, K) - ref).abs() <= (H + E) * ref.abs() + 2.0 ** -133).all()
        if ckpt:
            g = values(*ref_codes(gate.reshape(-1, K)), K)
            if up is not None:
                u = values(*ref_codes(up.reshape(-1, K)), K)
        E = (24 + 3 * g.abs()) * U
        a, da = act(name, g)
        dg = d * u * da
        # act' is a sum of two terms: errors relative to t and a (1 - t) (silu), none else
        size = da.abs() if name == "relu2" else (1 / (1 + torch.exp(-g))) * (1 + g.abs())
        got = grads[0].double().reshape(-1, K)
        assert ((got - dg).abs() <= H * dg.abs() + E * (d * u).abs() * size + 2.0 ** -133).all()
        if up is not None:
            du = d * a
            got = grads[1].double().reshape(-1, K)
            assert ((got - du).abs() <= (H + E) * du.abs() + 2.0 ** -133).all()


@pytest.mark.parametrize("K", [1, 7, 8, 13, 128, 129, 300, 2560, 6905])
@pytest.mark.parametrize("name", ["silu", "relu2"])
@pytest.mark.parametrize("ckpt", [True, False])
def test_gated_activation(K, name, ckpt):
    for M in (1, 5, 130):
        note(f"gate M={M} K={K} {name} ckpt={ckpt}")
        check_gate(randn(M, K, seed=1) * 3, randn(M, K, seed=2), name, ckpt, randn(M, K, seed=3))
        check_gate(randn(M, K, seed=4), None, name, ckpt, randn(M, K, seed=5))


@pytest.mark.parametrize("ckpt", [True, False])
def test_gate_halves_and_shapes(ckpt):
    """The halves of one tensor (rows at a stride, the second half at an odd
    element), three dimensions, a dY that is a view, and an expanded input."""
    gu = randn(30, 2 * 333, seed=6)
    check_gate(gu[:, :333], gu[:, 333:], "silu", ckpt, randn(333, 30, seed=7).t())
    gu = randn(3, 10, 2 * 256, seed=8)
    check_gate(gu[..., :256], gu[..., 256:], "relu2", ckpt, randn(3, 10, 256, seed=9))
    check_gate(randn(1, 64, seed=10).expand(20, 64), randn(20, 64, seed=11), "silu", ckpt, randn(20, 64, seed=12))
    check_gate(randn(64, 20, seed=13).t(), randn(20, 64, seed=14), "silu", ckpt, randn(20, 64, seed=15))


def test_gate_gradient_reaches_the_halves():
    from ternary_weight_quantization_amd.checkpoint import gated_activation

    gu = randn(17, 2 * 200, seed=16).requires_grad_(True)
    dy = randn(17, 200, seed=17)
    gated_activation(gu[:, :200], gu[:, 200:], "relu2").backward(dy)
    g, u = (t.detach().clone().requires_grad_(True) for t in (gu[:, :200], gu[:, 200:]))
    want = torch.autograd.grad(gated_activation(g, u, "relu2"), (g, u), dy)
    assert torch.equal(gu.grad, torch.cat(want, 1))


def test_gate_extremes():
    """Large magnitudes, zeros of both signs and NaN: finite where the
    function is, no NaN that the inputs do not have."""
    from ternary_weight_quantization_amd.checkpoint import gated_activation

    g = torch.tensor([[0.0, -0.0, 1e4, -1e4, 300.0, -300.0, 88.0, -88.0, 1e-30, -1e-30, 3e38, -3e38]],
                     device="cuda").to(BF).requires_grad_(True)
    for name in ("silu", "relu2"):
        for ckpt in (True, False):
            y = gated_activation(g, None, name, checkpoint=ckpt)
            dg, = torch.autograd.grad(y, g, torch.ones_like(g))
            assert not torch.isnan(y.float()).any() and not torch.isnan(dg.float()).any()
    n = torch.full((1, 8), float("nan"), device="cuda", dtype=BF)
    assert torch.isnan(gated_activation(n, None, "relu2").float()).all()
    assert torch.isnan(gated_activation(n, None, "silu").float()).all()


def test_gate_no_rows_and_same_bits():
    from ternary_weight_quantization_amd.checkpoint import gated_activation

    e = torch.empty(0, 50, device="cuda", dtype=BF, requires_grad=True)
    gated_activation(e, e * 1, "silu").sum().backward()
    assert e.grad.shape == (0, 50)
    g, u, dy = (randn(500, 2560, seed=s) for s in (18, 19, 20))

    def one():
        p, q = g.clone().requires_grad_(True), u.clone().requires_grad_(True)
        y = gated_activation(p, q)
        return (y.detach(),) + torch.autograd.grad(y, (p, q), dy)

    first = one()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        second = one()
    torch.cuda.current_stream().wait_stream(s)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(first, second))


# --- the trained-ternary layer's weight gradient ----------------------------------

@pytest.mark.parametrize("M,K,N", [(1, 64, 64), (33, 200, 96), (65, 129, 257), (300, 512, 384), (256, 2555, 130)])
@pytest.mark.parametrize("wt", [BF, F32])
def test_ttq_checkpoint(M, K, N, wt):
    """y, dX and the scales' masked sums' inputs are those of the layer
    without a checkpoint; dW = dY^T xh with xh the codes' values rounded to
    bf16 (2^-8 and two fp32 roundings each), products exact, sums of M terms
    in fp32 (M u), one rounding at the end."""
    from ternary_weight_quantization_amd.ttq_layer import ttq_init, ttq_linear

    note(f"ttq checkpoint M={M} K={K} N={N} {wt}")
    x, dy = randn(M, K, seed=21).requires_grad_(True), randn(M, N, seed=22)
    w = (randn(N, K, seed=23, dtype=F32) * 0.05).to(wt).requires_grad_(True)
    p = ttq_init(w.detach()).requires_grad_(True)
    y0 = ttq_linear(x, w, p)
    dx0, dw0, dp0 = torch.autograd.grad(y0, (x, w, p), dy)
    y = ttq_linear(x, w, p, checkpoint=True)
    dx, dw, dp = torch.autograd.grad(y, (x, w, p), dy)
    assert torch.equal(y, y0) and torch.equal(dx, dx0)
    v = values(*ref_codes(x.detach()), K)
    d = dy.double()
    ref = d.t().contiguous() @ v
    size = d.abs().t().contiguous() @ v.abs()
    h = torch.finfo(wt).eps / 2
    err = (dw.double() - ref).abs()
    assert (err <= h * ref.abs() + (H + (M + 4) * U) * size).all(), (err / size).max()
    # the masked sums are those of this dW: sums over N K terms, each off as dW is before its last rounding
    q = torch.zeros_like(ref)
    wd, pd = w.detach().double(), p.detach().double()
    q[wd > pd[0]], q[wd < -pd[0]] = 1, -1
    for got, mask, sign in ((dp[1], q == 1, 1.0), (dp[2], q == -1, -1.0)):
        assert abs(got.double() - sign * ref[mask].sum()) <= (H + (M + 600) * U) * size[mask].sum() + 1e-30
    assert dp[0] == 0


def test_ttq_checkpoint_keeps_codes_only():
    """What the layer saves: the codes and scales, not the bf16 input."""
    from ternary_weight_quantization_amd.ttq_layer import TTQLinear

    m = TTQLinear(512, 256, checkpoint=True)
    x = randn(128, 512, seed=24).requires_grad_(True)
    saved = []
    with torch.autograd.graph.saved_tensors_hooks(lambda t: (saved.append(t), t)[1], lambda t: t):
        y = m(x)
    assert any(t.dtype == torch.int8 and t.shape == (128, 512) for t in saved)
    assert not any(t.dtype == BF and t.shape == (128, 512) for t in saved)
    y.backward(randn(128, 256, seed=25))
    assert m.weight.grad is not None and x.grad is not None


def test_ttq_checkpoint_without_gradients():
    """A forward whose backward cannot run makes no codes: it allocates less by
    at least their size."""
    from ternary_weight_quantization_amd.ttq_layer import TTQLinear

    M, K = 4096, 4096
    m, x = TTQLinear(K, 64, checkpoint=True), randn(M, K, seed=28)

    def peak():
        torch.cuda.synchronize()
        torch.cuda.reset_peak_memory_stats()
        before = torch.cuda.memory_allocated()
        y = m(x)
        return y.detach(), torch.cuda.max_memory_allocated() - before

    with torch.no_grad():
        y0, lean = peak()
    y1, full = peak()
    assert torch.equal(y0, y1) and full - lean >= M * K


def test_checkpointed_block():
    """A feed-forward block as it is trained: norm, two ternary projections,
    gated activation, norm, ternary projection, all with 8-bit checkpoints,
    next to the same block without. Both pairs of gradients are within the
    coding's step of each other: a value is off by at most s / 254 of its
    block's magnitude, here against gradients that differ by less than a tenth
    of their norm."""
    from ternary_weight_quantization_amd.checkpoint import gated_activation
    from ternary_weight_quantization_amd.layer import QATBitLinear
    from ternary_weight_quantization_amd.norm import QATLayerNorm

    torch.manual_seed(0)
    n1, n2 = QATLayerNorm(256), QATLayerNorm(512)
    gate, up, down = QATBitLinear(256, 512), QATBitLinear(256, 512), QATBitLinear(512, 256)
    x0 = randn(100, 256, seed=26)
    dy = randn(100, 256, seed=27)
    got = []
    for ckpt in (False, True):
        n1.checkpoint = n2.checkpoint = ckpt
        for m in (n1, n2, gate, up, down):
            m.zero_grad(set_to_none=True)
        x = x0.clone().requires_grad_(True)
        h = n1(x)
        y = down(n2(gated_activation(gate(h), up(h), "relu2", checkpoint=ckpt)))
        y.backward(dy)
        got.append([y.detach(), x.grad] + [p.grad for m in (n1, n2, gate, up, down) for p in m.parameters()])
    assert torch.equal(got[0][0], got[1][0])
    for a, b in zip(*got):
        a, b = a.double(), b.double()
        assert (a - b).norm() <= 0.1 * a.norm()


@pytest.mark.parametrize("wt", [BF, F32])
@pytest.mark.parametrize("M,K,N", [(512, 1001, 2001), (1024, 2555, 1025), (640, 1285, 1283)])
def test_ttq_checkpoint_odd_widths_in_the_paired_launch(M, K, N, wt):
    """Widths that are padded, at sizes whose two products run in one launch
    (stated by the profiler's kernel names), everything exact: integers, with
    127 in each block so that the codes are the values, scales of 1/2, sums
    below 2^24. dX and a bf16 dW are rounded once; an fp32 dW is equal."""
    from torch.profiler import ProfilerActivity, profile

    from ternary_weight_quantization_amd.ttq_layer import ttq_linear

    note(f"ttq checkpoint, padded pair M={M} K={K} N={N} {wt}")
    g = torch.Generator().manual_seed(M)
    x = torch.randint(-8, 9, (M, K), generator=g).float()
    x[:, ::128] = 127.0
    dy = torch.randint(-2, 3, (M, N), generator=g).float()
    q = torch.randint(-1, 2, (N, K), generator=g).float()
    x, dy = (t.to(device="cuda", dtype=BF) for t in (x, dy))
    q = q.cuda()
    x.requires_grad_(True)
    w, p = q.to(wt).requires_grad_(True), torch.tensor([0.25, 0.5, 0.5], device="cuda", requires_grad=True)
    y = ttq_linear(x, w, p, checkpoint=True)
    first = torch.autograd.grad(y, (x, w, p), dy, retain_graph=True)
    torch.cuda.synchronize()
    with profile(activities=[ProfilerActivity.CPU, ProfilerActivity.CUDA]) as trace:
        dx, dw, dp = torch.autograd.grad(y, (x, w, p), dy)
        torch.cuda.synchronize()
    names = " ".join(e.key for e in trace.key_averages())
    assert "gemm_pair_kernel" in names and "pad_rows_kernel" in names, names
    assert all(torch.equal(a, b) for a, b in zip(first, (dx, dw, dp)))
    xd, dd, qd = x.detach().double(), dy.double(), q.double()
    rdx, rdw = torch.mm(dd, qd) / 2, torch.mm(dd.t().contiguous(), xd)
    assert rdw.abs().max() < 2 ** 24 and rdx.abs().max() < 2 ** 24
    assert torch.equal(y, (torch.mm(xd, qd.t().contiguous()) / 2).to(BF))
    assert torch.equal(dx, rdx.to(BF)) and torch.equal(dw, rdw.to(wt))
    for got, mask, sign in ((dp[1], qd == 1, 1.0), (dp[2], qd == -1, -1.0)):
        ref = sign * rdw[mask].sum()
        assert abs(got.double() - ref) <= U * abs(ref)
    assert dp[0] == 0


@pytest.mark.parametrize("ckpt", [True, False])
def test_silu_of_every_negative_value(ckpt):
    """Down to where silu(g) = g e^g leaves the normal numbers (g = -91.7), e^-g
    passing 2^126 and 2^128 on the way, and 0 or a subnormal below: every
    negative bf16 value, with an up and a dY of powers of two."""
    from ternary_weight_quantization_amd.checkpoint import gated_activation

    bits = torch.arange(0x8000, 0xFF80, dtype=torch.int32).to(torch.int16)
    g = bits.view(BF).cuda()
    g = g[None, :].expand(2, -1).contiguous() if not ckpt else g[:, None].expand(-1, 2).contiguous()
    note(f"silu of every negative value, ckpt={ckpt}")
    up, dy = torch.full_like(g, 4.0), torch.full_like(g, 0.5)
    gs, us = g.clone().requires_grad_(True), up.requires_grad_(True)
    y = gated_activation(gs, us, "silu", checkpoint=ckpt)
    dg, du = torch.autograd.grad(y, (gs, us), dy)
    d = g.double()
    a, da = act("silu", d)
    # the formulas' own rounding in 64 bits is far below; 2^-124: subnormal fp32 terms times 4 may become 0
    E = (24 + 3 * d.abs()) * U
    for got, ref, size in ((y, 4 * a, 4 * a.abs()), (dg, 2 * da, 2 / (1 + torch.exp(-d)) * (1 + d.abs())), (du, a / 2, a.abs() / 2)):
        err = (got.double() - ref).abs()
        assert (err <= H * ref.abs() + E * size + 2.0 ** -124).all(), d[err > H * ref.abs() + E * size + 2.0 ** -124][:9]
