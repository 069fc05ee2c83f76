"""The operators around the ternary layers as a program uses them: their autograd
functions captured into HIP graphs, where a training step replayed on other
inputs has the bits of the same step run eagerly and a capture that cannot work
is refused; offsets past 2^31; two threads at once."""

import pytest
import torch

from tests.gpu_util import note

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


def captured(step):
    """step() captured after one run of it on a side stream (its result freed
    before the capture)."""
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        step()
    torch.cuda.current_stream().wait_stream(s)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step()
    return graph, out


def replays(step, inputs):
    """Each replay against the eager step on the same inputs, with eager work
    and synchronizations between the replays."""
    graph, out = captured(step)
    for seed in range(4):
        for i, t in enumerate(inputs):
            with torch.no_grad():
                t.copy_(randn(*t.shape, seed=100 * seed + i, dtype=t.dtype))
        graph.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in out]
        want = step()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want)), seed


@pytest.mark.parametrize("checkpoint", [False, True])
def test_layer_norm(checkpoint):
    from ternary_weight_quantization_amd import layer_norm

    note(f"graph of layer norm, checkpoint={checkpoint}")
    x, dy = randn(300, 1000, seed=1, dtype=F32).requires_grad_(True), randn(300, 1000, seed=2)
    w, b = (randn(1000, seed=s).requires_grad_(True) for s in (3, 4))

    def step():
        y = layer_norm(x, w, b, checkpoint=checkpoint)
        return (y.detach(),) + torch.autograd.grad(y, (x, w, b), dy)

    replays(step, (x, w, b, dy))


@pytest.mark.parametrize("checkpoint", [False, True])
@pytest.mark.parametrize("act", ["silu", "relu2"])
def test_gated_activation(checkpoint, act):
    from ternary_weight_quantization_amd import gated_activation

    note(f"graph of {act}, checkpoint={checkpoint}")
    both, dy = randn(77, 2 * 520, seed=5).requires_grad_(True), randn(77, 520, seed=6)

    def step():
        y = gated_activation(both[:, :520], both[:, 520:], act, checkpoint=checkpoint)
        return (y.detach(),) + torch.autograd.grad(y, (both,), dy)

    replays(step, (both, dy))


@pytest.mark.parametrize("M,K,N", [(300, 512, 384), (65, 130, 258)])
def test_ttq_checkpoint(M, K, N):
    from ternary_weight_quantization_amd.ttq_layer import ttq_linear

    note(f"graph of ttq_linear M={M} K={K} N={N}")
    x, w, dy = (randn(*s, seed=7 + i) for i, s in enumerate(((M, K), (N, K), (M, N))))
    x.requires_grad_(True), w.requires_grad_(True)
    p = torch.tensor([0.5, 0.7, 0.6], device="cuda", requires_grad=True)

    def step():
        y = ttq_linear(x, w, p, checkpoint=True)
        return (y.detach(),) + torch.autograd.grad(y, (x, w, p), dy)

    replays(step, (x, w, dy))


@pytest.mark.parametrize("T", [20, 300])
@pytest.mark.parametrize("reduction", ["mean", "none"])
def test_linear_cross_entropy(T, reduction):
    from ternary_weight_quantization_amd import linear_cross_entropy

    note(f"graph of linear_cross_entropy T={T} {reduction}")
    h, w = randn(T, 264, seed=10).requires_grad_(True), randn(1500, 264, seed=11, dtype=F32).requires_grad_(True)
    t = torch.randint(0, 1500, (T,), generator=torch.Generator().manual_seed(12)).cuda()
    t[::5] = -100
    dl = torch.ones((T,) if reduction == "none" else (), device="cuda")

    def step():
        loss = linear_cross_entropy(h, w, t, reduction=reduction)
        return (loss.detach(),) + torch.autograd.grad(loss, (h, w), dl)

    replays(step, (h, w))


def test_a_training_step():
    """Norm, ternary projection, gated activation and loss in one graph, the
    leaves' .grad accumulated by the replay."""
    from ternary_weight_quantization_amd import LinearCrossEntropy, QATLayerNorm, gated_activation
    from ternary_weight_quantization_amd.ttq_layer import TTQLinear

    note("graph of a training step")
    torch.manual_seed(0)
    norm, up, head = QATLayerNorm(256, checkpoint=True), TTQLinear(256, 640, checkpoint=True), LinearCrossEntropy(320, 999)
    params = [p for m in (norm, up, head) for p in m.parameters()]
    x = randn(130, 256, seed=13)
    t = torch.randint(0, 999, (130,), generator=torch.Generator().manual_seed(14)).cuda()

    def step():
        g, u = up(norm(x)).chunk(2, dim=-1)
        loss = head(gated_activation(g, u), t)
        loss.backward()
        return [loss.detach()] + [p.grad for p in params]

    def fresh():
        for p in params:
            p.grad = torch.zeros_like(p)

    fresh()
    graph, out = captured(step)
    for seed in range(3):
        x.copy_(randn(130, 256, seed=20 + seed))
        for g in out[1:]:
            g.zero_()
        graph.replay()
        torch.cuda.synchronize()
        got = [v.clone() for v in out]
        fresh()
        want = step()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_a_capture_next_to_a_live_graph_of_the_default_stream_is_refused():
    """A leaf's gradient accumulator lives as long as any graph that uses it,
    on the stream it was made on, and no capture can take in the default
    stream: the backward says so. On a side stream it works, and after the
    eager results are freed too."""
    from ternary_weight_quantization_amd import gated_activation, layer_norm, linear_cross_entropy
    from ternary_weight_quantization_amd.ttq_layer import ttq_linear

    x, w = randn(40, 128, seed=30).requires_grad_(True), randn(128, seed=31).requires_grad_(True)
    big = randn(256, 128, seed=32).requires_grad_(True)
    p = torch.tensor([0.5, 0.7, 0.6], device="cuda", requires_grad=True)
    t = torch.arange(40, device="cuda")
    for name, f, leaves in (("layer_norm", lambda: layer_norm(x, w), (x, w)),
                            ("gated_activation", lambda: gated_activation(x, x), (x,)),
                            ("ttq_linear", lambda: ttq_linear(x, big, p, checkpoint=True), (x, big, p)),
                            ("linear_cross_entropy", lambda: linear_cross_entropy(x, big, t), (x, big))):
        note(f"refused capture of {name}")

        def step():
            y = f()
            return torch.autograd.grad(y, leaves, torch.ones_like(y))

        eager = f()  # alive, made on the default stream
        graph = torch.cuda.CUDAGraph()
        with pytest.raises(RuntimeError, match="default stream"):
            with torch.cuda.graph(graph):
                step()
        torch.cuda.synchronize()
        want = torch.autograd.grad(eager, leaves, torch.ones_like(eager))
        del eager, graph
        graph, out = captured(step)
        for _ in range(3):
            graph.replay()
            torch.cuda.synchronize()
            assert all(torch.equal(a, b) for a, b in zip(out, want))


def test_a_capture_that_leaves_the_live_leaf_out():
    """A live eager graph of a leaf whose gradient the captured pass does not
    compute is no obstacle."""
    from ternary_weight_quantization_amd import layer_norm

    note("capture of the weight's gradient alone")
    x, dy = randn(40, 128, seed=33).requires_grad_(True), randn(40, 128, seed=34)
    w = randn(128, seed=35).requires_grad_(True)
    eager = layer_norm(x)  # alive, of x alone

    def step():
        return torch.autograd.grad(layer_norm(x, w), (w,), dy)

    graph, out = captured(step)
    for _ in range(3):
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out[0], step()[0])
    assert eager.requires_grad


def test_offsets_past_two_to_the_31():
    """More than 2^31 values: the last rows have the bits of the same rows on
    their own, forward and backward, and the columns' gradients those of the
    rows that are not zero."""
    from ternary_weight_quantization_amd import compress, decompress, gated_activation, layer_norm

    note("2^31 + 20480 values")
    M, K, n = (1 << 19) + 5, 4096, 7
    x = torch.zeros(M, K, device="cuda", dtype=BF)
    tail, dtail = randn(n, K, seed=40), randn(n, K, seed=41)
    x[-n:] = tail
    dy = torch.zeros_like(x)
    dy[-n:] = dtail
    x.requires_grad_(True)
    w = randn(K, seed=42).requires_grad_(True)

    for f in (lambda v: layer_norm(v, w), lambda v: layer_norm(v, w, checkpoint=True),
              lambda v: gated_activation(v, v, "silu") + 0.0 * w, lambda v: gated_activation(v, None, "relu2", False) + 0.0 * w):
        small = tail.clone().requires_grad_(True)
        ys = f(small)
        ds, dws = torch.autograd.grad(ys, (small, w), dtail)
        y = f(x)
        dx, dw = torch.autograd.grad(y, (x, w), dy)
        assert torch.equal(y[-n:], ys) and torch.equal(dx[-n:], ds)
        assert not dx[:-n].any()
        # the sums over 2^19 rows of zeros and n others: the same n terms in fp32, in another order
        assert (dw.double() - dws.double()).abs().max() <= 2.0 ** -7 * dws.double().abs().max()
        del y, dx
    codes, scales = compress(x)
    cs, ss = compress(tail)
    assert torch.equal(codes[-n:], cs) and torch.equal(scales[-n:], ss)
    assert torch.equal(decompress(codes, scales, K)[-n:], decompress(cs, ss, K))


def test_two_threads_at_once():
    """Steps on two streams of two threads, with the bits of the same steps
    one after the other."""
    import threading

    from ternary_weight_quantization_amd import gated_activation, layer_norm, linear_cross_entropy

    note("two threads")

    def step(seed):
        x, w = randn(700, 512, seed=seed).requires_grad_(True), randn(512, seed=seed + 1).requires_grad_(True)
        head = randn(3000, 256, seed=seed + 2).requires_grad_(True)
        t = torch.randint(0, 3000, (700,), generator=torch.Generator().manual_seed(seed)).cuda()
        t[::7] = -100
        torch.cuda.current_stream().synchronize()
        out = []
        for _ in range(10):
            h = layer_norm(x, w, checkpoint=True)
            loss = linear_cross_entropy(gated_activation(h[:, :256], h[:, 256:]), head, t)
            out.append((loss.detach(),) + torch.autograd.grad(loss, (x, w, head)))
        return out

    got = {}

    def work(seed):
        s = torch.cuda.Stream()
        with torch.cuda.stream(s):
            got[seed] = step(seed)
            s.synchronize()

    threads = [threading.Thread(target=work, args=(s,)) for s in (50, 60)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    for seed in (50, 60):
        want = step(seed)
        torch.cuda.synchronize()
        assert len(got[seed]) == 10
        for a, b in zip(got[seed], want):
            assert all(torch.equal(p, q) for p, q in zip(a, b))


def test_a_capture_whose_gradient_reaches_the_default_stream_through_other_nodes_is_refused():
    """Between the operator and the leaf whose eager graph is alive stand a
    view (states of three dimensions), a module's parametrization (the TTQ
    layer's softplus), another of the operators, or nodes that were made on the
    default stream before the capture."""
    from ternary_weight_quantization_amd import gated_activation, layer_norm, linear_cross_entropy
    from ternary_weight_quantization_amd.ttq_layer import TTQLinear

    torch.manual_seed(0)
    h = randn(4, 10, 128, seed=36).requires_grad_(True)
    head, w = randn(256, 128, seed=37), randn(128, seed=38)
    t = torch.arange(40, device="cuda").view(4, 10)
    ttq, x = TTQLinear(128, 256, checkpoint=True), randn(40, 128, seed=39)
    for name, f, leaves in (("states of three dimensions", lambda: linear_cross_entropy(h, head, t), (h,)),
                            ("a parametrization", lambda: ttq(x), (ttq.raw,)),
                            ("a product", lambda: layer_norm(h * 2, w), (h,)),
                            ("halves", lambda: gated_activation(h[..., :64], h[..., 64:]), (h,)),
                            ("norm and loss", lambda: linear_cross_entropy(layer_norm(h.view(40, 128), w), head, t.view(40)),
                             (h,))):
        note(f"refused capture through {name}")

        def step():
            y = f()
            return torch.autograd.grad(y, leaves, torch.ones_like(y))

        eager = f()  # alive, made on the default stream
        graph = torch.cuda.CUDAGraph()
        with pytest.raises(RuntimeError, match="default stream"):
            with torch.cuda.graph(graph):
                step()
        torch.cuda.synchronize()
        want = torch.autograd.grad(eager, leaves, torch.ones_like(eager))
        del eager, graph
        graph, out = captured(step)
        for _ in range(3):
            graph.replay()
            torch.cuda.synchronize()
            assert all(torch.equal(a, b) for a, b in zip(out, want))

    note("refused capture of a node made before it")
    early = h.view(40, 128)
    graph = torch.cuda.CUDAGraph()
    with pytest.raises(RuntimeError, match="default stream"):
        with torch.cuda.graph(graph):
            y = layer_norm(early, w)
            torch.autograd.grad(y, (h,), torch.ones_like(y))
    torch.cuda.synchronize()
