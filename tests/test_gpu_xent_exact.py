"""Linear layer with softmax cross entropy where the logits are exact: small
integers and powers of two, whose products and sums fp32 holds without a
rounding, so that what is left are the operator's own steps.

u = 2^-24 (half an fp32 step); a rounding to bf16 is off by at most 2^-8 of the
value. With m a row's largest logit and s = sum_v exp(z_v - m) >= 1,
  loss = (m - z_target) + log s
A difference of such logits is exact. Its exponential is off by the rounding of
the argument (2 u |z_v - m|) and 4 u. A target that is the largest makes the
loss log s alone: it is never below 0, and where s is 1 plus one term e, it is
off by the rounding of s (u), the logarithm (2 u near 1) and e's own error: 8 u
in all. p_v = exp(z_v - lse) of the backward is further off by the rounding of
lse = m + log s to fp32, u |lse|.
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


def ints(*shape, low, high, seed):
    g = torch.Generator().manual_seed(seed)
    return torch.randint(low, high + 1, shape, generator=g).to(device="cuda", dtype=F32)


def confident(T, V, scale, gaps, seed):
    """Rows whose target's logit is about 770 scale, far above every other but,
    for gaps > 0, one that is gaps[t] below it; D = 64."""
    D = 64
    h = ints(T, D, low=1, high=2, seed=seed) * torch.where(ints(T, D, low=0, high=1, seed=seed + 1) > 0, 1.0, -1.0)
    h[:, 0] = 1.0
    w = ints(V, D, low=-1, high=1, seed=seed + 2)
    t = torch.randperm(V // 2, generator=torch.Generator().manual_seed(seed + 3))[:T].cuda()
    w[t] = torch.where(h > 0, 1.0, -1.0) * 8.0 * scale
    near = gaps > 0
    w[V // 2 + t[near]] = w[t[near]]
    w[V // 2 + t[near], 0] -= gaps[near]
    assert torch.equal(w.to(BF).float(), w) and torch.equal(h.to(BF).float(), h)
    return h.to(BF), w.to(BF), t


def softmax64(h, w, t):
    z = torch.mm(h.double(), w.double().t().contiguous())
    lse = torch.logsumexp(z, 1)
    return z, lse, z.gather(1, t[:, None])[:, 0]


@pytest.mark.parametrize("tiles", [0, 1])
@pytest.mark.parametrize("T", [9, 40, 130])
@pytest.mark.parametrize("level", [-500.0, -80.0, 0.0, 60.0])
def test_columns_of_minus_infinity(T, level, tiles, set_knobs):
    """Columns whose logits overflow to -inf, whole statistics blocks of 64 and
    128 of them, count as nothing, however low the others are. The loss is off
    by the additions of the sum of 300 exponentials (64 + 25 of them: 89 u), the
    exponentials (2 u times their arguments' size of up to 10, and 4 u) and the
    differences of logits around `level` (4 roundings)."""
    from ternary_weight_quantization_amd.loss import linear_cross_entropy

    note(f"columns of -inf T={T} level={level} tiles={tiles}")
    set_knobs(no_skinny=tiles)
    V, D = 700, 16
    h = torch.ones(T, D, device="cuda", dtype=BF)
    w = ints(V, D, low=-1, high=1, seed=T) / 4 + level / D
    off = torch.zeros(V, dtype=torch.bool, device="cuda")
    off[64:192] = off[256:512] = off[690:] = True
    w[off] = -3e38
    w = w.to(BF)
    keep = (~off).nonzero()[:, 0]
    t = keep[torch.arange(T, device="cuda") * 7 % len(keep)]
    z = torch.mm(h.double(), w.double().t().contiguous())
    lse = torch.logsumexp(z[:, keep], 1)
    want = lse - z.gather(1, t[:, None])[:, 0]
    hs, ws = h.clone().requires_grad_(True), w.clone().requires_grad_(True)
    loss = linear_cross_entropy(hs, ws, t, reduction="none")
    tol = (89 + 24) * U + 8 * U * (abs(level) + 10)
    assert ((loss.double() - want).abs() <= tol).all(), (loss.double() - want).abs().max().item()
    dh, dw = torch.autograd.grad(loss, (hs, ws), torch.ones_like(loss))
    assert not dw[off].any() and torch.isfinite(dh.float()).all()
    G = (z - lse[:, None]).exp()
    G.scatter_add_(1, t[:, None], -torch.ones(T, 1, device="cuda", dtype=torch.float64))
    G = G[:, keep]
    rdh, rdw, wd = torch.mm(G, w[keep].double()), torch.mm(G.t().contiguous(), h.double()), w[keep].double().abs()
    rel = H + 2 * tol + (V + 64) * 2 * U  # of |G| + p, which bounds both parts of the target's element
    size = G.abs() + 2 * (z[:, keep] - lse[:, None]).exp()
    assert ((dh.double() - rdh).abs() <= H * rdh.abs() + rel * torch.mm(size, wd)).all()
    assert ((dw[keep].double() - rdw).abs() <= H * rdw.abs() + rel * torch.mm(size.t().contiguous(), h.double())).all()


@pytest.mark.parametrize("tiles", [0, 1])
def test_nan_among_columns_of_minus_infinity(tiles, set_knobs):
    from ternary_weight_quantization_amd.loss import linear_cross_entropy

    note(f"NaN among columns of -inf, tiles={tiles}")
    set_knobs(no_skinny=tiles)
    h = torch.ones(40, 16, device="cuda", dtype=BF)
    w = ints(700, 16, low=-1, high=1, seed=3)
    w[256:512] = -3e38
    w[300, 2] = float("nan")
    t = torch.arange(40, device="cuda")
    assert torch.isnan(linear_cross_entropy(h, w.to(BF), t, reduction="none")).all()
    # no column left
    w[:] = -3e38
    assert torch.isnan(linear_cross_entropy(h, w.to(BF), t, reduction="none")).all()


@pytest.mark.parametrize("tiles", [0, 1])
@pytest.mark.parametrize("T,V", [(12, 500), (40, 500), (300, 3000)])
@pytest.mark.parametrize("scale", [0.125, 1.0, 2.0])
def test_confident_rows(T, V, scale, tiles, set_knobs):
    """Logits of 100, 770 and 1540: the loss of a row whose target takes all
    is 0, of one with a rival d below it log(1 + e^-d)."""
    from ternary_weight_quantization_amd.loss import linear_cross_entropy

    note(f"confident rows T={T} V={V} scale={scale} tiles={tiles}")
    set_knobs(no_skinny=tiles)
    gaps = (torch.arange(T, device="cuda") % 13).float()  # 0: no rival
    h, w, t = confident(T, V, scale, gaps, seed=T)
    z, lse, zt = softmax64(h, w, t)
    assert (zt == z.amax(1)).all()
    true = torch.log1p(torch.where(gaps > 0, torch.exp(-gaps.double()), 0.0))
    assert (lse - zt - true).abs().max() < 1e-9
    loss = linear_cross_entropy(h, w, t, reduction="none")
    assert (loss >= 0).all(), loss.min().item()
    err = (loss.double() - true).abs()
    assert (err <= 8 * U).all(), (err.max() / U).item()
    assert not loss[gaps == 0].any()


@pytest.mark.parametrize("tiles", [0, 1])
@pytest.mark.parametrize("T,V", [(12, 500), (40, 500), (300, 3000)])
@pytest.mark.parametrize("scale", [0.125, 1.0, 2.0])
def test_gradients_of_confident_rows(T, V, scale, tiles, set_knobs):
    """Logits of 100, 770 and 1540: the gradient of a row whose target takes all
    is 0, those of rows with a rival are off by p u |lse|, the exponentials'
    4 u |z - lse| + 8 u and G's rounding. An exponential, its product with c = 1
    and G's bf16 value below 2^-126, the least normal number, may become 0:
    each loses at most 2^-126, together less than 2^-124."""
    from ternary_weight_quantization_amd.loss import linear_cross_entropy

    note(f"gradients of confident rows T={T} V={V} scale={scale} tiles={tiles}")
    set_knobs(no_skinny=tiles)
    gaps = (torch.arange(T, device="cuda") % 13).float()  # 0: no rival
    h, w, t = confident(T, V, scale, gaps, seed=T)
    z, lse, zt = softmax64(h, w, t)
    assert (zt == z.amax(1)).all()
    hs, ws = h.clone().requires_grad_(True), w.clone().requires_grad_(True)
    loss = linear_cross_entropy(hs, ws, t, reduction="none")
    dh, dw = torch.autograd.grad(loss, (hs, ws), torch.ones_like(loss))
    p = (z - lse[:, None]).exp()
    G = p.clone()
    G.scatter_add_(1, t[:, None], -torch.ones(T, 1, device="cuda", dtype=torch.float64))
    eg = H * G.abs() + p * (U * lse.abs()[:, None] + 4 * U * (z - lse[:, None]).abs() + 8 * U) + 2.0 ** -124
    rdh, rdw = torch.mm(G, w.double()), torch.mm(G.t().contiguous(), h.double())
    edh = H * rdh.abs() + torch.mm(eg, w.double().abs()) + (V + 64) * 2 * U * torch.mm(G.abs(), w.double().abs())
    edw = H * rdw.abs() + torch.mm(eg.t().contiguous(), h.double().abs()) + (T + 64) * 2 * U * torch.mm(
        G.abs().t().contiguous(), h.double().abs())
    assert ((dh.double() - rdh).abs() <= edh + 2.0 ** -126).all(), ((dh.double() - rdh).abs() / edh).max().item()
    assert ((dw.double() - rdw).abs() <= edw + 2.0 ** -126).all()
    # no rival: every other logit is at least 50 below, and V e^-50 times |w| <= 16 is below 1e-15
    assert dh[gaps == 0].abs().max() <= 1e-15


@pytest.mark.parametrize("D", [4096, 4097])
def test_weight_past_two_gigabytes_every_gradient(D):
    """A weight and a dW whose bytes pass 32-bit offsets, in a width that is read
    in place and in one that is padded, every value of dh and dW checked. The
    logits are exact multiples of 1/8, so that the bounds hold G's and the
    outputs' roundings, the exponentials and the sums alone: the loss is off by
    V / 2048 + 120 additions of u and the terms' 2 u |z - m| + 4 u with |z - m| <
    120, p by what the header says, dh and dW by V + 64 and T + 64 additions of
    2 u. The bounds are small beside the values: zeros, or another row's, fail."""
    from ternary_weight_quantization_amd.loss import linear_cross_entropy

    V, T, step = 270001, 70, 30000
    note(f"xent past 2 GiB T={T} V={V} D={D}")
    g = torch.Generator(device="cuda")
    g.manual_seed(D)
    w = torch.empty(V, D, device="cuda", dtype=BF)
    for v in range(0, V, step):
        w[v:v + step] = torch.randint(-2, 3, (min(step, V - v), D), generator=g, device="cuda").to(BF) / 8
    h = torch.randint(-1, 2, (T, D), generator=g, device="cuda").to(BF)
    t = torch.randint(0, V, (T,), generator=g, device="cuda")
    t[0], t[1], t[2] = V - 1, 0, 262144
    hd = h.double()
    chunks = [(v, min(step, V - v)) for v in range(0, V, step)]
    z = torch.cat([torch.mm(hd, w[v:v + n].double().t().contiguous()) for v, n in chunks], 1)
    assert torch.equal(z * 8, (z * 8).round()) and (z.amax(1) - z.amin(1)).max() < 120 and w.numel() * 2 > 2 ** 31
    lse = torch.logsumexp(z, 1)
    want = lse - z.gather(1, t[:, None])[:, 0]
    tol = (V / 2048 + 120 + 2 * 120 + 4) * U + 4 * U * want.abs()
    hs, ws = h.requires_grad_(True), w.requires_grad_(True)
    loss = linear_cross_entropy(hs, ws, t, reduction="none")
    few = linear_cross_entropy(h[:9].detach(), w.detach(), t[:9], reduction="none")
    assert ((loss.double() - want).abs() <= tol).all() and ((few.double() - want[:9]).abs() <= tol[:9]).all()
    dh, dw = torch.autograd.grad(loss, (hs, ws), torch.ones_like(loss))
    with torch.no_grad():
        G = z.sub_(lse[:, None])
        eg = 4 * U * G.abs() + (U * lse.abs()[:, None] + 8 * U) + tol[:, None]
        eg *= G.exp_()
        G.scatter_add_(1, t[:, None], -torch.ones(T, 1, device="cuda", dtype=torch.float64))
        eg += H * G.abs() + 2.0 ** -124
        rdh, edh = torch.zeros(T, D, device="cuda", dtype=torch.float64), torch.zeros(T, D, device="cuda", dtype=torch.float64)
        for v, n in chunks:
            wd, Gv, ev = w[v:v + n].double(), G[:, v:v + n].contiguous(), eg[:, v:v + n].contiguous()
            rdh += torch.mm(Gv, wd)
            edh += torch.mm(ev + (V + 64) * 2 * U * Gv.abs(), wd.abs())
            rdw = torch.mm(Gv.t().contiguous(), hd)
            edw = H * rdw.abs() + torch.mm((ev + (T + 64) * 2 * U * Gv.abs()).t().contiguous(), hd.abs())
            assert ((dw[v:v + n].double() - rdw).abs() <= edw + 2.0 ** -126).all(), v
        edh += H * rdh.abs()
        assert ((dh.double() - rdh).abs() <= edh).all()
        assert (edh <= 0.1 * rdh.abs()).double().mean() > 0.5  # how sharp the bound is, not the kernel
        at = G.gather(1, t[:, None]).abs() * hd.abs()  # |dW| at the targets' rows is about this
        assert (eg.gather(1, t[:, None]) <= 0.01 * at.amax(1, keepdim=True)).all()
