"""Linear layer with softmax cross entropy on the GPU against its formulas in
64 bits.

Bounds. u = 2^-24 (half an fp32 step); a rounding to bf16 is off by at most
2^-8 of the value. A logit is an fp32 sum of D exact products, in any order:
  ez[t]  = (D + 8) 2 u max_v sum_d |h w|      (2 u: either rounding mode)
A sum of exponentials adds at most 64 terms per lane, 1 across lanes, and the
parts of 128 or 32 columns in 64 groups and 20 joins (V / 2048 + 90 terms),
each exponential off by the rounding of its argument (4 u (|z| + |lse|)) and
2 u, so
  el[t]  = ez + (V / 2048 + 120) u + 8 u (max |z| + |lse|)
  |err loss| <= 2 ez + el + 4 u |loss|
  |err G| <= 2^-8 |G| + |c| p (e^(ez + el) - 1 + 16 u (1 + max |z| + |lse|))
  |err dh| <= h |dh| + sum_v |err G| |w| + (V + 64) 2 u sum_v |G w|
  |err dW| <= h |dW| + sum_t |err G| |h| + (T + 64) 2 u sum_t |G h|
and (T + 2) 2^-53 relative for the fp64 sum of the rows' losses. Magnitudes
below 2^-126, the least normal fp32 and bf16 number, may become 0 on the way:
an exponential, its product with c and G's bf16 value each lose at most 2^-126
(times |c| for the first), so |err G| gains 2^-125 (1 + |c|) and an output
2^-126.
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


def make(T, V, D, seed=0, ignored=0, scale=1.5):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    h = torch.randn(T, D, generator=g, device="cuda").to(BF)
    w = (torch.randn(V, D, generator=g, device="cuda") * (scale / D ** 0.5)).to(BF)
    t = torch.randint(0, V, (T,), generator=g, device="cuda")
    t[torch.randperm(T, generator=g, device="cuda")[:ignored]] = -100
    return h, w, t


def reference(h, w, t, c, ignore=-100):
    """(loss rows, their bound, dh, its bound, dW, its bound), bounds without
    the outputs' own rounding."""
    T, V, D = h.shape[0], w.shape[0], w.shape[1]
    h, w = h.detach().double(), w.detach().double()
    keep = t != ignore
    h = torch.where(keep[:, None], h, 0.0)
    z = torch.mm(h, w.t().contiguous())
    S = torch.mm(h.abs(), w.abs().t().contiguous())
    lse = torch.logsumexp(z, 1)
    at = torch.where(keep, t, 0)[:, None]
    zt = z.gather(1, at)[:, 0]
    loss = torch.where(keep, lse - zt, 0.0)
    ez = (D + 8) * 2 * U * S.amax(1)
    top = z.abs().amax(1) + lse.abs()
    el = ez + (V / 2048 + 120) * U + 8 * U * top
    eloss = torch.where(keep, 2 * ez + el + 4 * U * loss.abs(), 0.0)
    c = torch.where(keep, c.double(), 0.0)
    p = (z - lse[:, None]).exp()
    del z, S
    eg = p * (c.abs() * (torch.expm1(ez + el) + 16 * U * (1 + top)))[:, None]
    G = p
    G.scatter_add_(1, at, torch.full_like(at, -1, dtype=torch.float64))
    G *= c[:, None]
    eg += H * G.abs() + 2.0 ** -125 * (1 + c.abs())[:, None]
    dh, dw = torch.mm(G, w), torch.mm(G.t().contiguous(), h)
    ga = G.abs()
    edh = torch.mm(eg, w.abs()) + (V + 64) * 2 * U * torch.mm(ga, w.abs())
    edw = torch.mm(eg.t().contiguous(), h.abs()) + (T + 64) * 2 * U * torch.mm(ga.t().contiguous(), h.abs())
    return loss, eloss, dh, edh, dw, edw


def ok(got, ref, bound, what):
    err = (got.double() - ref).abs()
    bound = bound + 2.0 ** -126
    assert (err <= bound).all(), (what, (err / bound).max().item())


def check(h, w, t, reduction="none", wt=BF):
    from ternary_weight_quantization_amd.loss import linear_cross_entropy

    T, V, D = h.shape[0], w.shape[0], w.shape[1]
    note(f"xent T={T} V={V} D={D} {reduction} {wt} ignored={(t == -100).sum().item()}")
    h = h.detach().requires_grad_(True)
    w = w.detach().to(wt).requires_grad_(True)
    n = max(1, int((t != -100).sum()))
    out = linear_cross_entropy(h, w, t, reduction=reduction)
    with torch.no_grad():
        assert torch.equal(linear_cross_entropy(h, w, t, reduction=reduction), out)
    if reduction == "none":
        up = torch.linspace(-1.0, 2.0, T, device="cuda")
        c = up
    else:
        up = torch.tensor(0.75, device="cuda")
        c = torch.full((T,), 0.75 / (n if reduction == "mean" else 1), device="cuda", dtype=torch.float64)
    dh, dw = torch.autograd.grad(out, (h, w), up)
    loss, eloss, rdh, edh, rdw, edw = reference(h, w, t, c)
    if reduction == "none":
        ok(out, loss, eloss, "loss")
    else:
        d = n if reduction == "mean" else 1
        ok(out, loss.sum() / d, eloss.sum() / d + 2 * U * loss.sum().abs() / d, "loss")
    assert dh.dtype == BF and dw.dtype == wt
    # c rounded to fp32 once or twice
    ok(dh, rdh, (H + 4 * U) * rdh.abs() + edh, "dh")
    ok(dw, rdw, (torch.finfo(wt).eps / 2 + 4 * U) * rdw.abs() + edw, "dW")
    assert not dh[t == -100].any()


@pytest.mark.parametrize("T", [1, 2, 15, 16, 17, 31, 32, 33, 63, 64, 65, 127, 255, 256, 257, 300, 513])
def test_tokens(T):
    check(*make(T, 1000, 192, seed=T))


@pytest.mark.parametrize("V", [1, 2, 31, 32, 33, 63, 64, 65, 127, 128, 129, 255, 256, 257, 383, 385, 511, 513, 3001])
def test_vocabularies(V):
    check(*make(40, V, 128, seed=V))
    check(*make(140, V, 128, seed=V + 1, ignored=20))


@pytest.mark.parametrize("D", [1, 2, 7, 8, 9, 15, 16, 24, 63, 64, 65, 72, 127, 128, 130, 200, 255, 257, 511, 2559, 2560])
def test_widths(D):
    check(*make(20, 700, D, seed=D))
    check(*make(90, 700, D, seed=D + 1), wt=F32)


@pytest.mark.parametrize("reduction", ["mean", "sum", "none"])
@pytest.mark.parametrize("T,ignored", [(10, 3), (200, 1), (200, 199), (300, 150), (600, 520)])
def test_ignored_rows(reduction, T, ignored):
    check(*make(T, 900, 96, seed=ignored, ignored=ignored), reduction=reduction)


@pytest.mark.parametrize("T", [5, 200])
@pytest.mark.parametrize("reduction", ["mean", "sum", "none"])
def test_nothing_counts(T, reduction):
    from ternary_weight_quantization_amd.loss import linear_cross_entropy

    h, w, t = make(T, 300, 64, ignored=T)
    h[0] = float("nan")
    h.requires_grad_(True)
    w.requires_grad_(True)
    out = linear_cross_entropy(h, w, t, reduction=reduction)
    assert not out.any()
    dh, dw = torch.autograd.grad(out, (h, w), torch.ones_like(out))
    assert not dh.any() and not dw.any()


def test_several_pieces():
    """More columns than a piece of G holds, the last piece ragged; dh split
    over a piece's columns."""
    check(*make(2100, 40003, 64, seed=1, ignored=7), reduction="mean")
    check(*make(300, 30001, 320, seed=2))
    check(*make(70, 140001, 1001, seed=3), reduction="sum")


def test_weight_past_two_gigabytes():
    """A weight and a dW whose bytes pass 32-bit offsets, one width that is
    padded and one that is not: losses and dh against a chunked reference, dW
    at the targets' rows, the first and the last."""
    from ternary_weight_quantization_amd.loss import linear_cross_entropy

    V, D, T = 270001, 4096, 70
    g = torch.Generator(device="cuda")
    g.manual_seed(5)
    note(f"xent T={T} V={V} D={D}")
    w = torch.empty(V, D, device="cuda", dtype=BF)
    for v in range(0, V, 30000):
        w[v:v + 30000] = (torch.randn(min(30000, V - v), D, generator=g, device="cuda") * 0.02).to(BF)
    h = torch.randn(T, D, generator=g, device="cuda").to(BF).requires_grad_(True)
    t = torch.randint(0, V, (T,), generator=g, device="cuda")
    t[0], t[1], t[2] = V - 1, 0, 262144
    w.requires_grad_(True)
    loss = linear_cross_entropy(h, w, t, reduction="none")
    few = linear_cross_entropy(h[:9].detach(), w.detach(), t[:9], reduction="none")
    dh, dw = torch.autograd.grad(loss, (h, w), torch.ones_like(loss))
    with torch.no_grad():
        hd = h.double()
        z = torch.cat([torch.mm(hd, w[v:v + 30000].double().t().contiguous()) for v in range(0, V, 30000)], 1)
        lse = torch.logsumexp(z, 1)
        ref = lse - z.gather(1, t[:, None])[:, 0]
        big = (D + 8) * 2 * U * (hd.abs().sum(1) * w.abs().max().double())
        tol = 3 * big + (V / 2048 + 140) * U * (1 + lse.abs() + z.abs().amax(1))
        ok(loss, ref, tol, "loss")
        ok(few, ref[:9], tol[:9], "few")
        G = (z - lse[:, None]).exp()
        G.scatter_add_(1, t[:, None], -torch.ones(T, 1, device="cuda", dtype=torch.float64))
        rel = 2 * H + torch.expm1(2 * tol).max()
        rdh = torch.zeros(T, D, device="cuda", dtype=torch.float64)
        edh = torch.zeros_like(rdh)
        for v in range(0, V, 30000):
            wd = w[v:v + 30000].double()
            rdh += torch.mm(G[:, v:v + 30000].contiguous(), wd)
            edh += torch.mm(G[:, v:v + 30000].abs().contiguous(), wd.abs())
        ok(dh, rdh, H * rdh.abs() + (rel + (V + 64) * 2 * U) * edh, "dh")
        rows = torch.unique(torch.cat([t, torch.tensor([0, V - 1, V // 2, 131072, 131071], device="cuda")]))
        Gr = G[:, rows].t().contiguous()
        rdw = torch.mm(Gr, hd)
        ok(dw[rows], rdw, H * rdw.abs() + (rel + (T + 64) * 2 * U) * torch.mm(Gr.abs(), hd.abs()), "dW")


def test_large_logits():
    """Logits of hundreds: the shift by the maximum, one class that takes
    everything, and a confident correct row whose loss is near 0."""
    h, w, t = make(130, 600, 64, seed=9, scale=400.0)
    z = h.float() @ w.float().t()
    t[:60] = z.argmax(1)[:60]
    check(h, w, t)
    check(h[:30].contiguous(), w, t[:30])


def test_ignored_rows_may_hold_anything():
    from ternary_weight_quantization_amd.loss import linear_cross_entropy

    for T in (30, 200):
        h, w, t = make(T, 500, 128, seed=10, ignored=T // 4)
        bad = h.clone()
        bad[t == -100] = float("nan")
        bad[(t == -100).nonzero()[0]] = float("inf")
        got = []
        for x in (h, bad):
            x, ww = x.clone().requires_grad_(True), w.clone().requires_grad_(True)
            out = linear_cross_entropy(x, ww, t)
            got.append((out.detach(),) + torch.autograd.grad(out, (x, ww)))
        assert all(torch.equal(a, b) for a, b in zip(*got))


@pytest.mark.parametrize("T", [20, 150])
def test_targets_out_of_range_and_nan_rows(T):
    from ternary_weight_quantization_amd.loss import linear_cross_entropy

    h, w, t = make(T, 400, 64, seed=11)
    good = linear_cross_entropy(h, w, t, reduction="none")
    t[3], t[7], t[T - 1] = 400, -1, 1 << 40
    h[5] = float("nan")
    h.requires_grad_(True)
    out = linear_cross_entropy(h, w, t, reduction="none")
    bad = torch.zeros(T, dtype=torch.bool, device="cuda")
    bad[[3, 5, 7, T - 1]] = True
    assert torch.isnan(out[bad]).all() and torch.equal(out[~bad], good[~bad])
    dh, = torch.autograd.grad(out, h, torch.ones_like(out))
    assert torch.isnan(dh[bad].float()).any(1).all() and torch.isfinite(dh[~bad].float()).all()
    # another ignore_index: negative targets are then out of range, the index is not
    t2 = torch.full_like(t, 7)
    assert linear_cross_entropy(h.detach(), w, t2, ignore_index=7).item() == 0.0


def test_shapes_views_and_partial_gradients():
    from ternary_weight_quantization_amd.loss import linear_cross_entropy

    h, w, t = make(120, 300, 128, seed=12, ignored=5)
    want = linear_cross_entropy(h, w, t, reduction="none")
    assert torch.equal(linear_cross_entropy(h.view(2, 60, 128), w, t.view(2, 60), reduction="none"), want.view(2, 60))
    flat = torch.zeros(1 + h.numel(), device="cuda", dtype=BF)
    flat[1:] = h.reshape(-1)
    wide = torch.zeros(300, 200, device="cuda", dtype=BF)
    wide[:, 5:133] = w
    assert torch.equal(linear_cross_entropy(flat[1:].view(120, 128), wide[:, 5:133], t, reduction="none"), want)
    assert torch.equal(linear_cross_entropy(h, w, t.repeat_interleave(2)[::2], reduction="none"), want)
    hs, ws = h.clone().requires_grad_(True), w.clone().requires_grad_(True)
    full = torch.autograd.grad(linear_cross_entropy(hs, ws, t), (hs, ws))
    only_h, = torch.autograd.grad(linear_cross_entropy(hs, w, t), (hs,))
    only_w, = torch.autograd.grad(linear_cross_entropy(h, ws, t), (ws,))
    assert torch.equal(only_h, full[0]) and torch.equal(only_w, full[1])
    empty = linear_cross_entropy(hs[:0], ws, t[:0])
    assert empty.item() == 0.0
    g = torch.autograd.grad(empty, (hs, ws))
    assert not g[0].any() and not g[1].any()
    assert linear_cross_entropy(h[:0], w, t[:0], reduction="none").shape == (0,)


def test_same_bits_again_and_on_another_stream():
    from ternary_weight_quantization_amd.loss import linear_cross_entropy

    h, w, t = make(500, 9000, 320, seed=13, ignored=50)

    def one():
        a, b = h.clone().requires_grad_(True), w.clone().requires_grad_(True)
        out = linear_cross_entropy(a, b, t)
        return (out.detach(),) + torch.autograd.grad(out, (a, b))

    first = one()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        second = one()
    torch.cuda.current_stream().wait_stream(s)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(first, second))


@pytest.mark.parametrize("T", [40, 300])
def test_graph_replays(T):
    """Captured once through the C entry points, replayed with other inputs,
    targets and numbers of ignored rows."""
    from ternary_weight_quantization_amd import binding as B

    V, D = 2000, 256
    h, w, t = make(T, V, D, seed=14)
    loss, lse, total = (torch.empty(n, device="cuda") for n in (T, T, 1))
    up = torch.ones(1, device="cuda")
    dh, dw = torch.empty_like(h), torch.empty_like(w)
    wf = torch.empty(B.bitnet_xent_fwd_workspace_bytes(T, V, D), dtype=torch.uint8, device="cuda")
    wb = torch.empty(B.bitnet_xent_bwd_workspace_bytes(T, V, D), dtype=torch.uint8, device="cuda")

    def step():
        B.bitnet_xent_fwd(h, w, t, -100, loss, lse, total, B.BITNET_REDUCE_MEAN, workspace=wf)
        B.bitnet_xent_bwd(h, w, t, -100, lse, up, dh, dw, B.BITNET_REDUCE_MEAN, workspace=wb)

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for seed, ignored in ((15, 0), (16, 30), (17, T), (18, 3)):
        h2, w2, t2 = make(T, V, D, seed=seed, ignored=ignored)
        h.copy_(h2)
        w.copy_(w2)
        t.copy_(t2)
        wb.fill_(255)  # what the workspace held does not matter
        graph.replay()
        torch.cuda.synchronize()
        got = [v.clone() for v in (loss, lse, total, dh, dw)]
        wf.fill_(127)
        step()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, (loss, lse, total, dh, dw)))


def test_gradient_against_differences():
    """sum_t loss along a direction of h: the difference of fp32 losses, each
    off by its bound, over 2 s, and s^2 / 6 times the third derivative (at
    most the spread of the logits' change cubed)."""
    from ternary_weight_quantization_amd.loss import linear_cross_entropy

    T, V, D = 90, 500, 128
    h, w, t = make(T, V, D, seed=19)
    h = (h.float() * 8).round().div(8).to(BF)  # so that h + s v is exact in bf16
    v = torch.randint(-1, 2, (T, D), device="cuda").to(F32)
    s = 2.0 ** -4
    hs = h.clone().requires_grad_(True)
    dh, = torch.autograd.grad(linear_cross_entropy(hs, w, t, reduction="sum"), hs)
    up, dn = (h.float() + s * v).to(BF), (h.float() - s * v).to(BF)
    exact = (up.float() == h.float() + s * v).all(1) & (dn.float() == h.float() - s * v).all(1)
    assert exact.float().mean() > 0.3
    f = [linear_cross_entropy(x, w, t, reduction="none").double() for x in (up, dn)]
    num = ((f[0] - f[1]) / (2 * s))[exact]
    ana = (dh.double() * v.double()).sum(1)[exact]
    z = v.double() @ w.double().t()
    spread = z.amax(1) - z.amin(1)
    _, eloss, rdh, edh, _, _ = reference(h, w, t, torch.ones(T, device="cuda"))
    tol = (eloss / s + s * s / 6 * spread ** 3 + ((H * rdh.abs() + edh) * v.abs().double()).sum(1))[exact]
    assert ((num - ana).abs() <= tol).all(), ((num - ana).abs() / tol).max()


def test_a_model_with_every_operator():
    """Tokens through norm, ternary feed-forward with a gated activation and
    8-bit checkpoints, final norm and the loss: one backward reaches every
    parameter, twice with the same bits."""
    from ternary_weight_quantization_amd.checkpoint import gated_activation
    from ternary_weight_quantization_amd.layer import QATBitLinear
    from ternary_weight_quantization_amd.loss import LinearCrossEntropy
    from ternary_weight_quantization_amd.norm import QATLayerNorm
    from ternary_weight_quantization_amd.ttq_layer import TTQLinear

    torch.manual_seed(3)
    emb = torch.nn.Embedding(777, 256, device="cuda", dtype=F32)
    n1, n2, n3 = (QATLayerNorm(k, dtype=F32, checkpoint=True) for k in (256, 512, 256))
    gate, up, down = QATBitLinear(256, 512), TTQLinear(256, 512, checkpoint=True), QATBitLinear(512, 256)
    head = LinearCrossEntropy(256, 777)
    modules = (emb, n1, n2, n3, gate, up, down, head)
    x = torch.randint(0, 777, (3, 50), device="cuda")
    y = torch.roll(x, -1, 1)
    y[:, -1] = -100

    def step():
        for m in modules:
            m.zero_grad(set_to_none=True)
        r = emb(x)
        a = n1(r)
        r = r + down(n2(gated_activation(gate(a), up(a), "silu"))).float()
        loss = head(n3(r), y)
        loss.backward()
        return [loss.detach()] + [p.grad.clone() for m in modules for p in m.parameters()]

    first, second = step(), step()
    assert abs(first[0].item() - torch.log(torch.tensor(777.0)).item()) < 1.0
    for g, k in zip(first, second):
        assert torch.isfinite(g).all() and torch.equal(g, k)
    assert all(g.any() for g in first)


def test_not_differentiable_twice():
    from ternary_weight_quantization_amd.checkpoint import gated_activation
    from ternary_weight_quantization_amd.loss import linear_cross_entropy
    from ternary_weight_quantization_amd.norm import layer_norm

    h, w, t = make(12, 40, 64, seed=20)
    h.requires_grad_(True)
    for out in (linear_cross_entropy(h, w, t), layer_norm(h).float().sum(), gated_activation(h).float().sum()):
        with pytest.raises(RuntimeError):
            torch.autograd.grad(out, h, create_graph=True)


@pytest.mark.parametrize("T", [16, 17, 32, 33, 48, 49, 64])
@pytest.mark.parametrize("V", [24575, 24576, 24700])
def test_few_tokens_many_columns(T, V):
    """Around the change of the rows a workgroup takes, each group of 16
    tokens, rows that do not count among them."""
    check(*make(T, V, 72, seed=T + V, ignored=T // 5))


@pytest.mark.parametrize("T", [48, 49, 64])
@pytest.mark.parametrize("V", [57343, 57344])
def test_few_tokens_or_tiles(T, V):
    """Either side of the choice between the kernels."""
    check(*make(T, V, 72, seed=T + V, ignored=T // 5))


@pytest.mark.parametrize("T", [16383, 16384, 40001])
def test_many_rows(T):
    """Several groups of rows per gathering block, runs of ignored rows."""
    h, w, t = make(T, 70, 24, seed=T, ignored=T // 3)
    t[1000:1900] = -100
    check(h, w, t, reduction="mean")
