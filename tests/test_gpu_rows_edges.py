"""8-bit rows, the gated pair and the 8-bit layer where their arithmetic and their
sizes end: codes at exact ties, the slopes' rounding, roots of no positive number,
waits that give up, memory full of garbage in every form of the kernels, sizes that
only the forward takes, masters off alignment."""

import pytest
import torch

from tests.gpu_util import knobs, note

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.fail("no GPU visible")
    from ternary_weight_quantization_amd import binding
    binding.lib()


def randn(*shape, seed, dtype=BF):
    g = torch.Generator().manual_seed(seed)
    return torch.randn(*shape, generator=g).to(device="cuda", dtype=dtype)


# --- the norm's codes --------------------------------------------------------

@pytest.mark.parametrize("ht", [BF, F32])
@pytest.mark.parametrize("K", [5, 640, 2555, 5000, 16384])
def test_codes_of_the_norm_at_ties(K, ht):
    """Without a weight, or with one of powers of two, 127 v / s is 127 h w / max|h w|
    whatever r is: values of half the row's largest, and every half integer of a row
    whose largest is 127, are exact ties and go to the even code. bf16 values of up to
    8 bits are elsewhere at least 2^-16 of the quotient away from a tie, far more than
    the quotient's few 2^-24, so every code is the formula's."""
    from ternary_weight_quantization_amd import rms_norm

    note(f"rms codes at ties K={K} {ht}")
    M = 96
    h = randn(M, K, seed=K)
    top = h.float().abs().amax(1, keepdim=True)
    at = torch.arange(0, K, 3, device="cuda")
    h[:32, at] = torch.where(h[:32, at] > 0, top[:32] / 2, -top[:32] / 2).to(BF)
    h[:32, 0] = top[:32, 0].to(BF)  # exact: the largest value itself
    g = torch.Generator().manual_seed(K + 1)
    ties = torch.randint(-254, 255, (32, K), generator=g).cuda() / 2.0 * 2.0 ** torch.arange(-16, 16, device="cuda")[:, None]
    h[32:64] = ties.to(BF)
    h[32:64, 0] = 127.0 * 2.0 ** torch.arange(-16, 16, device="cuda")
    w2 = (2.0 ** torch.randint(-3, 4, (K,), generator=g)).cuda()
    for w in (None, w2.to(BF), w2):
        v = h.double() * (1.0 if w is None else w.double())
        want = torch.round(127.0 * v / v.abs().amax(1, keepdim=True))
        rows = rms_norm(h.to(ht), w, quantize=True)
        assert torch.equal(rows.codes[:, :K].double(), want)
        both, s = rms_norm(torch.zeros_like(h), w, h.to(ht), quantize=True)
        assert torch.equal(both.codes, rows.codes) and torch.equal(both.scales, rows.scales) and torch.equal(s, h.to(ht))


@pytest.mark.parametrize("w", [None, BF])
@pytest.mark.parametrize("K", [3, 300, 5000])
def test_rows_of_the_norm_with_no_root(K, w):
    """eps below 0 or of 0 where the mean square and it have no positive sum: r is NaN
    or infinite, the row NaN as it is in bf16, and the others stay."""
    from ternary_weight_quantization_amd import rms_norm

    note(f"rms without a root K={K}")
    x = randn(9, K, seed=K)
    w = None if w is None else randn(K, seed=1)
    x[2], x[7] = 0, x[7] * 2.0 ** -12
    for eps, bad in ((0.0, [2]), (-1e-4, [2, 7])):
        rows, y = rms_norm(x, w, eps=eps, quantize=True), rms_norm(x, w, eps=eps)
        keep = [i for i in range(9) if i not in bad]
        assert y[bad].isnan().all() and rows.scales[bad].isnan().all() and rows.dequantize()[bad].isnan().all()
        assert y[keep].isfinite().all() and rows.scales[keep].isfinite().all() and not rows.codes[:, K:].any()
        assert torch.equal(rows.scales[keep], rms_norm(x[keep], w, eps=eps, quantize=True).scales)


# --- the pair's slopes -------------------------------------------------------

# Tokens and launch knobs of each form of the forward: few tokens, a middling number on
# the smaller and the larger of its tiles, the tiles of long batches, whole and split.
FORMS = [(1, {}), (5, {}), (40, {}), (90, {}), (700, {}), (90, dict(no_skinny=1)),
         (300, dict(no_skinny=1, split_ctas=3)), (300, dict(no_skinny=1, split_ctas=-1))]


def slopes_of(buf, M, N):
    """p and a [M, N] float32 of the bytes that the forward stores."""
    Nd = -(-N // 64) * 64
    n = 2 * M * 2 * Nd
    hi = buf[:n].view(torch.int16).view(M, 2, Nd)[:, :, :N].int() & 0xFFFF
    lo = buf[n:].view(M, 2, Nd)[:, :, :N].int()
    v = ((hi << 16) | (lo << 8)).view(torch.float32)
    return v[:, 0], v[:, 1]


def pair(M, K, N, seed):
    """8-bit rows and codes as the C entry points take them."""
    from ternary_weight_quantization_amd.layer import act_quant, ternarize

    x, packed = randn(M, K, seed=seed), []
    for i in (1, 2):
        packed.append(ternarize(randn(N, K, seed=seed + i) / K ** 0.5))
    q, s = act_quant(x)
    return x, q, s, torch.cat([p for p, _ in packed]), torch.cat([g for _, g in packed])


@pytest.mark.parametrize("M,kw", FORMS)
def test_slopes_are_rounded_to_24_bits(M, kw):
    """a = g^2 and p = 2 g u have the same fp32 operations here, on the CPU: what is kept
    of them is off by at most half a step of 16 bits, 2^-16 of the value, and not to one
    side. NaN with any payload stays NaN, infinity itself."""
    from ternary_weight_quantization_amd import binding as B

    K, N = 200, 75
    note(f"slopes M={M} {kw}")
    x, q, s, packed, gamma = pair(M, K, N, M)

    def forward(s, gamma):
        y = torch.empty(M, N, dtype=BF, device="cuda")
        sl = torch.zeros(B.bitnet_gated_slopes_bytes(M, N), dtype=torch.uint8, device="cuda")
        B.bitnet_gated_fwd(B.BITNET_ACT_RELU2, q, s, packed, gamma, K, y, sl)
        return y, slopes_of(sl, M, N)

    with knobs(**kw):
        y, (p, a) = forward(s, gamma)
        t = packed.view(2 * N, -1, 1, 4).int() >> (2 * torch.arange(4, device="cuda"))[:, None]  # [word][j // 4][j % 4]
        t = (t & 3).reshape(2 * N, -1)
        acc = (q.double() @ torch.where(t == 3, -1, t).double().t()).float().cpu()
        c = [(s.cpu() * v / torch.full((M,), 127.0))[:, None] for v in gamma.cpu()]
        g, u = (acc[:, :N] * c[0]).clamp(min=0), acc[:, N:] * c[1]
        off = []
        for got, want in ((a, g * g), (p, 2 * g * u)):
            got, want = got.cpu().double(), want.double()
            assert ((got - want).abs() <= 2.0 ** -16 * want.abs()).all()
            off.append(((got - want) / want)[want != 0])
        off = torch.cat(off)
        # the mean of n errors of at most h = 2^-16, evenly spread: h / sqrt(3 n)
        assert off.mean().abs().item() <= 6 * 2.0 ** -16 / (3 * off.numel()) ** 0.5
        bits = torch.tensor([0x7FFFFFFF, 0x7FFFFF80, 0x7F800001, -1, -128, 0x7FC00000], dtype=torch.int32, device="cuda")
        for b in bits:
            nan = s.clone().view(torch.int32)
            nan[M // 2] = b
            y, (p, a) = forward(nan.view(torch.float32), gamma)
            assert y[M // 2].isnan().all() and p[M // 2].isnan().all() and a[M // 2].isnan().all()
            assert y.isnan().sum() == N and a.isnan().sum() == N
            gn = gamma.clone().view(torch.int32)
            gn[1] = b
            y, (p, a) = forward(s, gn.view(torch.float32))
            assert y.isnan().all() and p.isnan().all() and not a.isnan().any()
        big = s.clone()
        big[M // 2] = 3e38
        y, (p, a) = forward(big, gamma)
        pos = g[M // 2] > 0
        assert (a[M // 2][pos] == float("inf")).all() and (a[M // 2][~pos] == 0).all()


@pytest.mark.parametrize("M,kw", FORMS)
def test_rows_of_scale_zero(M, kw):
    """A token masked out by a scale of 0, or one of the least scales, stands for zeros:
    no gradient, and none of its own in the weights'."""
    from ternary_weight_quantization_amd import QATGatedBitLinear, rms_norm

    note(f"rows of scale 0 M={M} {kw}")
    m = QATGatedBitLinear(130, 75)
    x, dy = randn(M, 130, seed=M).requires_grad_(True), randn(M, 75, seed=1)
    off = torch.arange(0, M, 3, device="cuda")
    with knobs(**kw):
        for low in (0.0, 1e-40, 2.0 ** -126):
            rows = rms_norm(x, quantize=True)
            rows.scales[off] = low
            y = m(rows)
            assert not y[off].any()
            dx, dg, du = torch.autograd.grad(y, [rows._carrier, m.gate_weight, m.up_weight], dy)
            assert not dx[off].any() and dx.isfinite().all()
            d0 = dy.clone()
            d0[off] = 0
            wx, wg, wu = torch.autograd.grad(m(rows), [rows._carrier, m.gate_weight, m.up_weight], d0)
            assert torch.equal(dx, wx) and torch.equal(dg, wg) and torch.equal(du, wu)


# --- waits that give up ------------------------------------------------------

@pytest.mark.parametrize("act", ["silu", "relu2"])
def test_a_split_gated_forward_that_gives_up_is_visible(act):
    """A wait for another workgroup's partial tile that gives up (forced with a zero
    spin limit: every kernel ends) leaves its tile of y and of the slopes NaN as a
    whole and is counted; the other tiles are exact."""
    from ternary_weight_quantization_amd import binding as B
    from ternary_weight_quantization_amd.checkpoint import ACTIVATIONS

    M, K, N = 768, 2560, 384
    note(f"gated split gives up {act}")
    x, q, s, packed, gamma = pair(M, K, N, 5)

    def forward():
        y = torch.empty(M, N, dtype=BF, device="cuda")
        sl = torch.zeros(B.bitnet_gated_slopes_bytes(M, N), dtype=torch.uint8, device="cuda")
        B.bitnet_gated_fwd(ACTIVATIONS[act], q, s, packed, gamma, K, y, sl)
        return (y, *slopes_of(sl, M, N))

    B.bitnet_split_timeouts()
    with knobs(split_ctas=64):
        ref = forward()
    assert B.bitnet_split_timeouts() == 0
    with knobs(split_ctas=64, spin_limit=0):
        got = forward()
    count, bad = B.bitnet_split_timeouts(), 0
    for m in range(0, M, 256):
        for n in range(0, N, 128):  # 256 rows of codes are 128 of the gate and 128 of the up projection
            tile = [t[m:m + 256, n:n + 128] for t in got]
            want = [t[m:m + 256, n:n + 128] for t in ref]
            if all(torch.equal(a, b) for a, b in zip(tile, want)):
                continue
            bad += 1
            assert all(a.isnan().all() for a in tile), (m, n)
    note(f"  counted {count}, {bad} tiles")
    assert count == bad
    assert B.bitnet_split_timeouts() == 0
    with knobs(split_ctas=64):
        assert all(torch.equal(a, b) for a, b in zip(forward(), ref))


def test_a_split_gated_backward_that_gives_up_is_visible():
    from ternary_weight_quantization_amd import binding as B

    M, K, N = 768, 768, 384  # D has 2 x 384 columns, dW 2 x 384 rows: 3 x 3 tiles each
    note("gated backward gives up")
    x, q, s, packed, gamma = pair(M, K, N, 6)
    dY = randn(M, N, seed=7)
    y = torch.empty(M, N, dtype=BF, device="cuda")
    sl = torch.zeros(B.bitnet_gated_slopes_bytes(M, N), dtype=torch.uint8, device="cuda")
    B.bitnet_gated_fwd(B.BITNET_ACT_SILU, q, s, packed, gamma, K, y, sl)

    def backward():
        dX, dg, du = (torch.empty(n, K, dtype=BF, device="cuda") for n in (M, N, N))
        B.bitnet_gated_bwd(dY, sl, q, s, packed, gamma, K, dX=dX, dW_gate=dg, dW_up=du)
        return dX, torch.cat([dg, du])

    B.bitnet_split_timeouts()
    with knobs(split_ctas=36):
        ref = backward()
    assert B.bitnet_split_timeouts() == 0
    with knobs(split_ctas=36, spin_limit=0):
        got = backward()
    count, bad = B.bitnet_split_timeouts(), 0
    for a, b in zip(got, ref):
        for j in range(0, M, 256):
            for k in range(0, K, 256):
                t = a[j:j + 256, k:k + 256]
                if t.isnan().any():
                    bad += 1
                    assert t.isnan().all()
                else:
                    assert torch.equal(t, b[j:j + 256, k:k + 256])
    note(f"  counted {count}, {bad} tiles")
    assert count == bad and B.bitnet_split_timeouts() == 0


def test_a_split_8_bit_forward_that_gives_up_is_visible():
    """Its accumulators are INT32_MIN there, which no sum of products is."""
    from ternary_weight_quantization_amd import binding as B

    M, K, N = 768, 2560, 768
    note("int8 split gives up")
    new = lambda n: (torch.empty(n, K, dtype=torch.int8, device="cuda"), torch.empty(n, device="cuda"))  # noqa: E731
    (q, s), (wq, sw) = new(M), new(N)
    B.bitnet_rows_quant2(randn(M, K, seed=1), q, s, randn(N, K, seed=2), wq, sw)

    def forward():
        y = torch.empty(M, N, dtype=BF, device="cuda")
        B.bitnet_int8_fwd(q, s, wq, sw, K, y)
        return y

    B.bitnet_split_timeouts()
    with knobs(split_ctas=64):
        ref = forward()
    assert B.bitnet_split_timeouts() == 0
    with knobs(split_ctas=64, spin_limit=0):
        got = forward()
    count, bad = B.bitnet_split_timeouts(), 0
    c, cw = s / torch.full_like(s, 127.0), sw / torch.full_like(sw, 127.0)
    lost = (-2.0 ** 31 * c[:, None] * cw).to(BF)
    for m in range(0, M, 256):
        for n in range(0, N, 256):
            at = (slice(m, m + 256), slice(n, n + 256))
            if not torch.equal(got[at], ref[at]):
                bad += 1
                assert torch.equal(got[at], lost[at])
    note(f"  counted {count}, {bad} tiles")
    assert count == bad and B.bitnet_split_timeouts() == 0


# --- memory full of garbage --------------------------------------------------

@pytest.mark.parametrize("N", [75, 129])
@pytest.mark.parametrize("M,kw", FORMS)
def test_gated_pair_in_garbage(M, kw, N):
    """Slopes, workspaces and outputs full of NaN or zeros before the calls, every form
    of the forward: the same bits, trained and for dX alone without the rows."""
    from ternary_weight_quantization_amd import binding as B

    K = 130
    note(f"gated in garbage M={M} N={N} {kw}")
    x, q, s, packed, gamma = pair(M, K, N, 1)
    dY = randn(M, N, seed=3)
    outs = []
    with knobs(**kw):
        for fill in (0xFF, 0x00):
            new = lambda n: torch.full((max(n, 16),), fill, dtype=torch.uint8, device="cuda")  # noqa: E731
            out = lambda *n: new(2 * n[0] * n[1]).view(BF)[:n[0] * n[1]].view(n)  # noqa: E731
            y, slopes = out(M, N), new(B.bitnet_gated_slopes_bytes(M, N))
            B.bitnet_gated_fwd(B.BITNET_ACT_SILU, q, s, packed, gamma, K, y, slopes,
                               workspace=new(B.bitnet_gated_fwd_workspace_bytes(M, N, K)))
            need = B.bitnet_gated_bwd_workspace_bytes(M, N, K)
            dX, dg, du, only, w0, w1 = out(M, K), out(N, K), out(N, K), out(M, K), out(N, K), out(N, K)
            B.bitnet_gated_bwd(dY, slopes, q, s, packed, gamma, K, dX=dX, dW_gate=dg, dW_up=du, workspace=new(need))
            B.bitnet_gated_bwd(dY, slopes, None, None, packed, gamma, K, dX=only, workspace=new(need))
            B.bitnet_gated_bwd(dY, slopes, q, s, None, gamma, K, dW_gate=w0, dW_up=w1, workspace=new(need))
            outs.append((y, dX, dg, du, only, w0, w1))
    for a, b in zip(*outs):
        assert a.isfinite().all() and torch.equal(a, b)


@pytest.mark.parametrize("N", [75, 129])
@pytest.mark.parametrize("M,kw", FORMS)
def test_8_bit_layer_in_garbage(M, kw, N):
    from ternary_weight_quantization_amd import binding as B

    K, Kp = 130, 192
    note(f"int8 in garbage M={M} N={N} {kw}")
    dY, outs = randn(M, N, seed=3), []
    with knobs(**kw):
        for fill in (0xFF, 0x00):
            new = lambda n: torch.full((max(n, 16),), fill, dtype=torch.uint8, device="cuda")  # noqa: E731
            out = lambda *n: new(2 * n[0] * n[1]).view(BF)[:n[0] * n[1]].view(n)  # noqa: E731
            rows = lambda n: (new(n * Kp).view(torch.int8).view(n, Kp), new(4 * n).view(F32)[:n])  # noqa: E731
            (q, s), (wq, sw) = rows(M), rows(N)
            B.bitnet_rows_quant(randn(M, K, seed=1), q, s)
            B.bitnet_rows_quant(randn(N, K, seed=2, dtype=F32), wq, sw)
            y, dX, dW, db, only = out(M, N), out(M, K), out(N, K), out(1, N)[0], out(M, K)
            B.bitnet_int8_fwd(q, s, wq, sw, K, y, workspace=new(B.bitnet_int8_fwd_workspace_bytes(M, N, K)))
            need = B.bitnet_int8_bwd_workspace_bytes(M, N, K)
            B.bitnet_int8_bwd(dY, q, s, wq, sw, K, dX=dX, dW=dW, db=db, workspace=new(need))
            B.bitnet_int8_bwd(dY, None, None, wq, sw, K, dX=only, workspace=new(need))
            outs.append((y, dX, dW, db, only))
    for a, b in zip(*outs):
        assert a.isfinite().all() and torch.equal(a, b)


# --- refusals ----------------------------------------------------------------

def test_a_layer_too_large_for_its_backward_is_refused_in_the_forward():
    """(M + 256) 2 Nd past 2^31: the forward alone runs, one whose gradients are wanted
    raises at once."""
    from ternary_weight_quantization_amd import binding as B
    from ternary_weight_quantization_amd import int8_linear, int8_linear_inference

    M, K, N = 33000, 64, 32768
    note("int8 too large for its backward")
    x, w = randn(M, K, seed=1), randn(N, K, seed=2)
    with torch.no_grad():
        y = int8_linear(x, w)
    assert torch.equal(y[-1], int8_linear(x[-1], w))
    with pytest.raises(ValueError, match="backward"):
        int8_linear(x, w.requires_grad_(True))
    assert torch.equal(int8_linear(x[:32000], w).detach(), y[:32000])
    wq, sw = B.ops().int8_quantize_weight(w.detach())
    bias = torch.zeros(N, dtype=BF, device="cuda", requires_grad=True)
    assert torch.equal(int8_linear_inference(x, wq, sw, K), y)
    assert torch.equal(int8_linear_inference(x, wq, sw, K, bias).detach(), y)
    with pytest.raises(ValueError, match="backward"):
        int8_linear_inference(x.requires_grad_(True), wq, sw, K)


@pytest.mark.parametrize("dtype", [BF, F32])
def test_master_weights_off_alignment_freeze(dtype):
    """Masters that are views of a larger buffer, from any element on, train and freeze."""
    from ternary_weight_quantization_amd import QATGatedBitLinear
    from ternary_weight_quantization_amd.layer import ternarize

    note(f"masters off alignment {dtype}")
    N, K = 21, 67
    m = QATGatedBitLinear(K, N, dtype=dtype)
    flat = torch.empty(2 * N * K + 1, dtype=dtype, device="cuda")
    for i, p in enumerate((m.gate_weight, m.up_weight)):
        view = flat[1 + i * N * K:1 + (i + 1) * N * K].view(N, K)
        view.copy_(p.data)
        p.data = view
    x = randn(5, K, seed=1)
    y = m(x)
    m.freeze()
    assert torch.equal(m(x), y)
    packed, gamma = ternarize(m.up_weight.detach().clone())
    assert torch.equal(m.export_inference()[0][N:], packed) and torch.equal(m.export_inference()[1][1:], gamma)
