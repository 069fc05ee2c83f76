"""What the operators around the layers refuse of torch's transformations,
without a GPU: a tangent of forward-mode differentiation (with and without
requires_grad, under no_grad), every kind of trace, and tensors that have no
memory, whose data pointers are no addresses. Each refusal comes before the
checks of devices."""

import pytest
import torch
import torch.autograd.forward_ad as fwad

BF = torch.bfloat16


def calls():
    """(name, function of one float tensor, that tensor)."""
    from ternary_weight_quantization_amd.checkpoint import compress, decompress, gated_activation
    from ternary_weight_quantization_amd.loss import linear_cross_entropy
    from ternary_weight_quantization_amd.norm import layer_norm
    from ternary_weight_quantization_amd.ttq_layer import ttq_linear

    x, w, v = torch.ones(4, 128, dtype=BF), torch.ones(9, 128, dtype=BF), torch.ones(128, dtype=BF)
    p, t, q = torch.ones(3), torch.zeros(4).long(), torch.zeros(4, 128, dtype=torch.int8)
    return [
        ("layer_norm", lambda a: layer_norm(a, v), x),
        ("layer_norm", lambda a: layer_norm(x, a), v),
        ("layer_norm", lambda a: layer_norm(x, v, a), v),
        ("layer_norm", lambda a: layer_norm(a, checkpoint=True), x),
        ("gated_activation", lambda a: gated_activation(a, x), x),
        ("gated_activation", lambda a: gated_activation(x, a, checkpoint=False), x),
        ("gated_activation", lambda a: gated_activation(a, act="relu2"), x),
        ("linear_cross_entropy", lambda a: linear_cross_entropy(a, w, t), x),
        ("linear_cross_entropy", lambda a: linear_cross_entropy(x, a, t), w),
        ("ttq_linear", lambda a: ttq_linear(a, w, p, checkpoint=True), x),
        ("ttq_linear", lambda a: ttq_linear(x, a, p, checkpoint=True), w),
        ("ttq_linear", lambda a: ttq_linear(x, w, a, checkpoint=True), p),
        ("compress", lambda a: compress(a)[1], x),
        ("decompress", lambda a: decompress(q, a, 128), torch.ones(4, 1)),
    ]


@pytest.mark.parametrize("grad", [True, False])
@pytest.mark.parametrize("leaf", [True, False])
def test_forward_mode(grad, leaf):
    for name, f, a in calls():
        with torch.set_grad_enabled(grad), fwad.dual_level():
            dual = fwad.make_dual(a.detach().clone().requires_grad_(leaf), torch.ones_like(a))
            with pytest.raises(NotImplementedError, match=f"{name}: no forward-mode derivative"):
                f(dual)


def test_a_tangent_where_forward_mode_is_off():
    """Nothing is differentiated there: the call goes on to its other checks."""
    for _, f, a in calls():
        with fwad.dual_level():
            dual = fwad.make_dual(a, torch.ones_like(a))
            with torch.inference_mode(), pytest.raises(ValueError):
                f(dual)


@pytest.mark.parametrize("leaf", [True, False])
def test_traces(leaf):
    from torch.fx.experimental.proxy_tensor import make_fx

    for name, f, a in calls():
        a = a.detach().clone().requires_grad_(leaf)
        for trace in (lambda: torch.jit.trace(f, (a,)), lambda: make_fx(f)(a), lambda: make_fx(f, tracing_mode="fake")(a)):
            with pytest.raises(NotImplementedError, match=f"{name}: cannot be traced"):
                trace()


def test_modes_that_only_look_on():
    """A dispatch mode that is no trace is no reason to refuse."""
    from torch.utils.flop_counter import FlopCounterMode

    for _, f, a in calls():
        with FlopCounterMode(display=False), pytest.raises(ValueError):
            f(a)


def without_memory(a):
    """Tensors like a that have none: fake ones outside their mode, at an
    offset too, functional ones and those of other devices' metadata."""
    from torch._subclasses import FakeTensorMode

    with FakeTensorMode():
        fake = torch.empty((2 * a.shape[0],) + a.shape[1:], dtype=a.dtype)
        halves = [fake[:a.shape[0]], fake[a.shape[0]:]]
    return halves + [torch._to_functional_tensor(torch.cat([a, a]))[a.shape[0]:], torch.empty_like(a, device="meta")]


def test_tensors_without_memory():
    for name, f, a in calls():
        for b in without_memory(a):
            with pytest.raises(NotImplementedError, match=f"{name}: a tensor without memory"):
                f(b)


@pytest.mark.parametrize("transform", ["grad", "vjp", "vmap", "functionalize"])
def test_function_transforms(transform):
    for name, f, a in calls():
        run = {"grad": lambda: torch.func.grad(lambda b: f(b).float().sum())(a), "vjp": lambda: torch.func.vjp(f, a),
               "vmap": lambda: torch.vmap(f)(torch.stack([a, a])), "functionalize": lambda: torch.func.functionalize(f)(a)}
        with pytest.raises(NotImplementedError, match=f"{name}: a tensor without memory"):
            run[transform]()
