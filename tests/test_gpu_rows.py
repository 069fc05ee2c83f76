"""8-bit rows between the norm and the layers as a program uses them: one norm
for several layers, a block's training step eager and captured into a HIP graph,
streams of their own, two threads at once, offsets past 2^31."""

import threading

import pytest
import torch

from tests.gpu_util import note
from tests.test_gpu_operator_graphs import captured, randn

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.fail("no GPU visible")
    from ternary_weight_quantization_amd import binding
    binding.lib()


class Block(torch.nn.Module):
    """norm -> gated pair -> norm -> down, and an 8-bit layer on the first rows."""

    def __init__(self, K, N, bias=False):
        super().__init__()
        from ternary_weight_quantization_amd import QATBitLinear, QATGatedBitLinear, QATInt8Linear, QATRMSNorm

        torch.manual_seed(K + N)
        self.norm, self.inner = QATRMSNorm(K, quantize=True), QATRMSNorm(N, quantize=True)
        self.up, self.down = QATGatedBitLinear(K, N, act="relu2"), QATBitLinear(N, K, bias=bias)
        self.side = QATInt8Linear(K, K, bias=bias)

    def forward(self, x, res):
        rows, h = self.norm(x, res)
        return self.down(self.inner(self.up(rows))) + self.side(rows), h


def loss_grads(block, x, res, dy, dh):
    y, h = block(x, res)
    leaves = [x, res] + list(block.parameters())
    return [y.detach(), h.detach()] + list(torch.autograd.grad([y, h], leaves, [dy, dh]))


@pytest.mark.parametrize("bias", [False, True])
@pytest.mark.parametrize("M", [3, 64, 100])
def test_ternary_layer_of_rows(M, bias):
    """QATBitLinear of 8-bit rows is the C entry points on their codes, forward
    and backward, trained and frozen; the norm gets its dX."""
    from ternary_weight_quantization_amd import QATBitLinear, rms_norm
    from ternary_weight_quantization_amd import binding as B
    from ternary_weight_quantization_amd.layer import bitlinear_inference, ternarize

    note(f"BitLinear of rows M={M} bias={bias}")
    K, N = 130, 88
    m = QATBitLinear(K, N, bias=bias)
    if bias:
        with torch.no_grad():
            m.bias.copy_(randn(N, seed=8))
    x = randn(M, K, seed=1).requires_grad_(True)
    w = torch.nn.Parameter(randn(K, seed=2))
    rows = rms_norm(x, w, quantize=True)
    y = m(rows)
    dy = randn(M, N, seed=3)
    leaves = [x, w] + list(m.parameters())
    grads = torch.autograd.grad(y, leaves, dy, retain_graph=True)
    packed, gamma = ternarize(m.weight.detach())
    want = torch.empty_like(y)
    B.bitlinear_fwd(rows.codes, rows.scales, packed, gamma, K, want, bias=None if not bias else m.bias.detach())
    assert torch.equal(y, want)
    dX, dW = torch.empty(M, K, dtype=BF, device="cuda"), torch.empty(N, K, dtype=BF, device="cuda")
    B.bitlinear_bwd(dy, rows.codes, rows.scales, packed, gamma, K, dX=dX, dW=dW)
    assert torch.equal(grads[2], dW)
    again = rms_norm(x, w, quantize=True)
    for a, b in zip(grads, torch.autograd.grad(again.dequantize(), [x, w], dX)):
        assert torch.equal(a, b)
    if bias:
        assert ((grads[3].double() - dy.double().sum(0)).abs() <= 2.0 ** -8 * dy.double().sum(0).abs()
                + M * 2.0 ** -24 * dy.double().abs().sum(0)).all()
    with torch.no_grad():
        assert torch.equal(m(rows.detach()), y)
    m.freeze()
    yf = m(rows)
    gf = torch.autograd.grad(yf, [x, w], dy)
    assert torch.equal(yf, y) and torch.equal(bitlinear_inference(rows.detach(), packed, gamma, K, m.bias), y)
    once = rms_norm(x, w, quantize=True)
    assert all(torch.equal(a, b) for a, b in zip(gf, torch.autograd.grad(once.dequantize(), [x, w], dX)))


def test_several_layers_share_rows():
    """Their gradients add up in the rows."""
    from ternary_weight_quantization_amd import QATBitLinear, QATInt8Linear, rms_norm

    note("rows shared")
    x = randn(50, 96, seed=1).requires_grad_(True)
    a, b = QATBitLinear(96, 64), QATInt8Linear(96, 40)
    da, db = randn(50, 64, seed=2), randn(50, 40, seed=3)
    rows = rms_norm(x, quantize=True)
    both, = torch.autograd.grad([a(rows), b(rows)], x, [da, db])
    parts = []
    for m, d in ((a, da), (b, db)):
        rows = rms_norm(x, quantize=True)
        leaf = rows._carrier
        parts.append(torch.autograd.grad(m(rows), leaf, d)[0])
    rows = rms_norm(x, quantize=True)
    want, = torch.autograd.grad(rows.dequantize(), x, parts[0] + parts[1])
    assert torch.equal(both, want)


@pytest.mark.parametrize("M", [5, 200, 300])
def test_a_block_in_a_graph(M):
    """A training step captured and replayed on other inputs has the bits of the
    eager step."""
    note(f"block in a graph M={M}")
    block = Block(160, 224, bias=True)
    x, res = randn(M, 160, seed=1).requires_grad_(True), randn(M, 160, seed=2).requires_grad_(True)
    dy, dh = randn(M, 160, seed=3), randn(M, 160, seed=4)
    graph, out = captured(lambda: loss_grads(block, x, res, dy, dh))
    for seed in range(4):
        with torch.no_grad():
            for i, t in enumerate((x, res, dy, dh, block.up.gate_weight, block.down.weight, block.side.weight)):
                t.copy_(randn(*t.shape, seed=100 * seed + i))
        graph.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in out]
        want = loss_grads(block, x, res, dy, dh)
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want)), seed
        del want


def test_frozen_decoding_in_a_graph():
    note("frozen block in a graph")
    block = Block(160, 224)
    for m in (block.up, block.down, block.side):
        m.freeze()
    x, res = randn(1, 160, seed=1), randn(1, 160, seed=2)

    def step():
        with torch.no_grad():
            return block(x, res)

    graph, out = captured(step)
    for seed in range(4):
        x.copy_(randn(1, 160, seed=10 + seed))
        graph.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in out]
        assert all(torch.equal(a, b) for a, b in zip(got, step())), seed


@pytest.mark.parametrize("layer", ["rms", "gated", "int8", "ternary"])
def test_a_capture_beside_a_live_graph_is_refused(layer):
    """While an eager graph of the same leaves lives, the captured backward
    raises instead of ending the process."""
    from ternary_weight_quantization_amd import QATBitLinear, QATGatedBitLinear, QATInt8Linear, rms_norm

    note(f"refused capture of {layer}")
    x = randn(10, 64, seed=1)
    w = torch.nn.Parameter(randn(64, seed=2))
    m = {"rms": None, "gated": QATGatedBitLinear, "int8": QATInt8Linear, "ternary": QATBitLinear}[layer]
    m = m(64, 32) if m else None

    def forward():
        if m is None:
            return rms_norm(x, w)
        if layer == "ternary":
            return m(rms_norm(x, quantize=True))
        return m(x)

    alive = forward()
    leaves = [w] if m is None else list(m.parameters())
    dy = torch.ones_like(alive)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with pytest.raises(RuntimeError, match="default stream"):
        with torch.cuda.graph(graph):
            torch.autograd.grad(forward(), leaves, dy)
    torch.cuda.synchronize()
    del alive
    out = forward()  # the process goes on
    assert out.isfinite().all()


def test_on_a_stream_of_its_own():
    note("block on a side stream")
    block = Block(96, 160)
    x, res = randn(70, 96, seed=1).requires_grad_(True), randn(70, 96, seed=2).requires_grad_(True)
    dy, dh = randn(70, 96, seed=3), randn(70, 96, seed=4)
    want = loss_grads(block, x, res, dy, dh)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        got = loss_grads(block, x, res, dy, dh)
    s.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_two_threads_at_once():
    note("block in two threads")
    blocks = [Block(96, 160), Block(128, 96)]
    args = []
    for i, b in enumerate(blocks):
        K = b.norm.features
        args.append([randn(40 + 60 * i, K, seed=10 * i + j).requires_grad_(j < 2) for j in range(4)])
    want = [loss_grads(b, *a) for b, a in zip(blocks, args)]
    torch.cuda.synchronize()
    got, errors = [None, None], []

    def work(i):
        try:
            s = torch.cuda.Stream()
            with torch.cuda.stream(s):
                for _ in range(5):
                    got[i] = loss_grads(blocks[i], *args[i])
            s.synchronize()
        except Exception as e:  # noqa: BLE001
            errors.append(e)

    threads = [threading.Thread(target=work, args=(i,)) for i in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not errors, errors
    for i in range(2):
        assert all(torch.equal(a, b) for a, b in zip(got[i], want[i]))


@pytest.mark.parametrize("M", [3, 100])
def test_one_tensor_in_two_places(M):
    """The input as its own residual, one weight as gate and up, a matrix as input and
    weight: the result of two equal tensors, the gradients their sum."""
    from ternary_weight_quantization_amd import gated_bitlinear, int8_linear, rms_norm

    note(f"one tensor in two places M={M}")
    K = 72

    def grads(f, shared, n, seed):
        t = [randn(*shared, seed=seed).requires_grad_(True) for _ in range(n)]
        y = f(*t)
        y = y if isinstance(y, tuple) else (y,)
        d = [randn(*v.shape, seed=seed + 1 + i).to(v.dtype) for i, v in enumerate(y)]
        return list(y), torch.autograd.grad(y, t, d)

    x = randn(M, K, seed=50)
    cases = [(lambda a: rms_norm(a, None, a), lambda a, b: rms_norm(a, None, b), (M, K)),
             (lambda a: gated_bitlinear(x, a, a), lambda a, b: gated_bitlinear(x, a, b), (40, K)),
             (lambda a: int8_linear(a, a), lambda a, b: int8_linear(a, b), (M, K))]
    for i, (one, two, shape) in enumerate(cases):
        y1, (g,) = grads(one, shape, 1, 10 * i)
        y2, (ga, gb) = grads(two, shape, 2, 10 * i)
        assert all(torch.equal(a, b) for a, b in zip(y1, y2))
        assert torch.equal(g, ga + gb)


def test_offsets_past_2_to_the_31():
    """Rows whose elements lie past 2^31 values: the last of a large batch against
    the same rows alone."""
    from ternary_weight_quantization_amd import rms_norm

    M, K = 150_000, 16000
    note("rms past 2^31")
    x = torch.empty(M, K, device="cuda", dtype=BF)
    x[:-64].fill_(1.0)
    x[-64:] = randn(64, K, seed=1)
    w = randn(K, seed=2).requires_grad_(True)
    x.requires_grad_(True)
    rows = rms_norm(x, w, quantize=True)
    small = x.detach()[-64:].clone().requires_grad_(True)
    alone = rms_norm(small, w, quantize=True)
    assert torch.equal(rows.codes[-64:], alone.codes) and torch.equal(rows.scales[-64:], alone.scales)
    v = rows.dequantize()
    assert torch.equal(v[-64:], alone.dequantize())
    dy = torch.zeros(M, K, device="cuda", dtype=BF)
    dy[-64:] = randn(64, K, seed=3)
    gx, = torch.autograd.grad(v, x, dy)
    want, = torch.autograd.grad(alone.dequantize(), small, dy[-64:].clone())
    assert torch.equal(gx[-64:], want) and not gx[:-64].any()


def test_an_example_runs():
    """A step of a feed-forward block with its loss, as documented: gradients
    everywhere, finite."""
    from ternary_weight_quantization_amd import LinearCrossEntropy, QATRMSNorm

    note("block with a loss")
    block, last, head = Block(128, 192), QATRMSNorm(128), LinearCrossEntropy(128, 500)
    h = randn(60, 128, seed=1)
    targets = torch.arange(60, device="cuda")
    y, h = block(torch.zeros_like(h), h)
    out, h = last(y, h)
    head(out, targets).backward()
    for m in (block, last, head):
        for n, p in m.named_parameters():
            assert p.grad is not None and p.grad.isfinite().all() and p.grad.any(), n
