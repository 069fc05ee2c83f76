"""Refusals around 8-bit rows without a GPU, each before the device is touched."""

import os

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
LIB = os.path.join(ROOT, "ternary_weight_quantization_amd", "libbitnet.so")
OK, ENULL, ESHAPE, EDTYPE, EALIGN, EWS, EHIP = range(7)
P = 1 << 20  # a stand-in device address, aligned; never dereferenced
BF, F32 = 0, 1


@pytest.fixture(scope="module")
def L():
    if not os.path.exists(LIB):
        pytest.fail("libbitnet.so is not built (run `python -m ternary_weight_quantization_amd.build`)")
    from ternary_weight_quantization_amd import binding
    return binding.lib()


def test_rows_that_two_weights_share_have_the_limits_of_rows(L):
    def f(x=P, N=200, M=4, K=130, ws=P):
        return L.bitnet_quantize2(P, P, BF, N, K, x, M, P, P, P, P, ws, 1 << 40, None)

    assert f(M=(1 << 23) + 1) == ESHAPE and f(M=1 << 27) == ESHAPE and f(M=1 << 30) == ESHAPE
    assert f(K=(1 << 24) + 1) == ESHAPE
    # at the limits the call goes on to its other checks, and without rows it has none of theirs
    assert f(M=1 << 23, ws=None) == EWS and f(K=1 << 24, ws=None) == EWS
    assert f(x=None, M=1 << 27, ws=None) == EWS and f(x=None, K=(1 << 24) + 1, ws=None) == EWS


def test_both_sides_of_one_launch_have_a_limit_together(L):
    def f(M, N, K=2048, x=P):
        return L.bitnet_rows_quant2(x, M, P, P, P, F32, N, P, P, K, None)

    most = 1 << 23
    assert f(most, most) == ESHAPE and f(most + 1, 1) == ESHAPE and f(0, most + 1) == ESHAPE and f(0, 0) == ESHAPE
    assert f(-1, 4) == ESHAPE and f(4, -1) == ESHAPE and f(4, 4, K=0) == ESHAPE and f(4, 4, K=(1 << 24) + 1) == ESHAPE
    assert f(most, most - 1, x=P + 1) == EALIGN and f(1, most, x=P + 1) == EALIGN  # on to its other checks


def test_what_does_not_take_rows_says_so():
    import torch

    from tests.test_more_operators_cpu import rows_of
    from ternary_weight_quantization_amd import LinearCrossEntropy, TTQLinear, layer_norm, linear_cross_entropy, rms_norm
    from ternary_weight_quantization_amd.layer import BitLinearFunction, FrozenBitLinearFunction
    from ternary_weight_quantization_amd.ttq_layer import ttq_forward_codes, ttq_linear

    r, w, p = rows_of(4, 64), torch.zeros(9, 64, dtype=torch.bfloat16), torch.ones(3)
    t = torch.zeros(4, dtype=torch.int64)
    ttq = TTQLinear.__new__(TTQLinear)  # its scales are made on the GPU
    torch.nn.Module.__init__(ttq)
    ttq.weight, ttq.raw = torch.nn.Parameter(w), torch.nn.Parameter(p)
    for call in (lambda: ttq(r), lambda: ttq_linear(r, w, p), lambda: ttq_linear(r, w, p, checkpoint=True),
                 lambda: ttq_forward_codes(r, w, p), lambda: linear_cross_entropy(r, w, t),
                 lambda: LinearCrossEntropy(64, 9, device="cpu")(r, t), lambda: BitLinearFunction.apply(r, w, None),
                 lambda: FrozenBitLinearFunction.apply(r, w.byte(), p[:1], 64), lambda: layer_norm(r), lambda: rms_norm(r)):
        with pytest.raises(TypeError, match="not QuantizedRows"):
            call()


def test_two_weights_on_their_own_device(L, monkeypatch):
    """The call runs on the weights' device and its current stream, and every tensor has
    to be there (the CPU and "meta" stand for two GPUs)."""
    import torch

    from ternary_weight_quantization_amd import binding as B

    ran = []
    monkeypatch.setattr(B, "_need", lambda *a: None)
    monkeypatch.setattr(B, "_run", lambda fn, like, stream, *args: ran.append((like, stream, len(args))))
    monkeypatch.setattr(B, "_stream", lambda stream: None)
    f32, kinds = torch.float32, [((9, 64), torch.float32)] * 2  # W0, W1, x, codes, gamma, x_q, s_x, workspace
    kinds += [((4, 64), torch.bfloat16), ((18, 16), torch.uint8), ((2,), f32), ((4, 64), torch.int8), ((4,), f32),
              ((64,), torch.uint8)]
    make = lambda i, device: torch.empty(kinds[i][0], dtype=kinds[i][1], device=device)  # noqa: E731
    here = [make(i, "cpu") for i in range(8)]
    B.bitnet_quantize2(*here)
    assert ran[0][0] is here[0] and ran[0][1] is None
    for i in range(1, 8):
        with pytest.raises(ValueError, match="on meta, expected cpu"):
            B.bitnet_quantize2(*[make(j, "meta" if j == i else "cpu") for j in range(8)])
    B.bitnet_quantize2(here[0], here[1], None, here[3], here[4], None, None, here[7])
    assert len(ran) == 2
