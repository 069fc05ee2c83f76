"""The library's entry points for 8-bit checkpoints, the gated activation and
the TTQ layer with codes through their Python wrappers (one per entry point):
the bits of the functions over them, optional arguments, a stream and a
workspace of the caller's."""

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


def codes_like(M, K):
    from ternary_weight_quantization_amd import binding as B

    Kc = B.bitnet_ckpt_pad(K)
    return (torch.full((M, Kc), 77, dtype=torch.int8, device="cuda"), torch.full((M, Kc // 128), -1.0, device="cuda"))


@pytest.mark.parametrize("stream", [False, True])
@pytest.mark.parametrize("M,K,dtype", [(1, 1, BF), (5, 300, F32), (130, 2560, BF)])
def test_pack_unpack(M, K, dtype, stream):
    from ternary_weight_quantization_amd import binding as B
    from ternary_weight_quantization_amd.checkpoint import compress, decompress

    note(f"wrappers of pack and unpack M={M} K={K} {dtype}")
    x = randn(M, K, seed=1, dtype=dtype)
    codes, scales = codes_like(M, K)
    out = torch.empty_like(x)
    torch.cuda.synchronize()
    s = torch.cuda.Stream() if stream else None
    B.bitnet_ckpt_pack(x, codes, scales, stream=s)
    B.bitnet_ckpt_unpack(codes, scales, out, stream=s)
    torch.cuda.synchronize()
    want = compress(x)
    assert torch.equal(codes, want[0]) and torch.equal(scales, want[1])
    assert torch.equal(out, decompress(*want, K, dtype))


@pytest.mark.parametrize("name", ["silu", "relu2"])
@pytest.mark.parametrize("gated", [True, False])
@pytest.mark.parametrize("ckpt", [True, False])
@pytest.mark.parametrize("M,K", [(1, 7), (60, 333)])
def test_gate(name, gated, ckpt, M, K):
    from ternary_weight_quantization_amd import binding as B
    from ternary_weight_quantization_amd.checkpoint import ACTIVATIONS, gated_activation

    note(f"wrappers of the gate {name} gated={gated} ckpt={ckpt} M={M} K={K}")
    both, dy = randn(M, 2 * K + 3, seed=2), randn(M, K, seed=3)
    gate, up = both[:, 1:K + 1], both[:, K + 2:2 * K + 2] if gated else None
    g, u = gate.clone().requires_grad_(True), up.clone().requires_grad_(True) if gated else None
    y0 = gated_activation(g, u, name, checkpoint=ckpt)
    want = torch.autograd.grad(y0, [t for t in (g, u) if t is not None], dy)
    act, y = ACTIVATIONS[name], torch.empty(M, K, device="cuda", dtype=BF)
    gc, uc = (codes_like(M, K) if ckpt else (None, None)), (codes_like(M, K) if ckpt and gated else (None, None))
    B.bitnet_gate_fwd(act, gate, up, y, *gc, *uc)
    assert torch.equal(y, y0)
    # gradients into the halves of one tensor; what lies between them stays
    grads = torch.full((M, 2 * K + 3), 5.0, device="cuda", dtype=BF)
    dg, du = grads[:, 1:K + 1], grads[:, K + 2:2 * K + 2] if gated else None
    if ckpt:
        B.bitnet_gate_bwd(act, dy, dg, du, None, None, *gc, *uc)
    else:
        B.bitnet_gate_bwd(act, dy, dg, du, gate, up)
    assert torch.equal(dg, want[0]) and (not gated or torch.equal(du, want[1]))
    keep = torch.ones(2 * K + 3, dtype=torch.bool, device="cuda")
    keep[1:K + 1] = False
    if gated:
        keep[K + 2:2 * K + 2] = False
    assert (grads[:, keep] == 5.0).all()
    with pytest.raises((ValueError, RuntimeError)):
        B.bitnet_gate_bwd(act, dy, dg, du, None, None)
    with pytest.raises((ValueError, RuntimeError)):
        B.bitnet_gate_bwd(act, dy, dg, None if gated else dg, gate, up)


@pytest.mark.parametrize("own_workspace", [True, False])
@pytest.mark.parametrize("M,K,N", [(1, 64, 64), (65, 129, 258), (300, 512, 384)])
def test_ttq(M, K, N, own_workspace):
    from ternary_weight_quantization_amd import binding as B
    from ternary_weight_quantization_amd.checkpoint import compress
    from ternary_weight_quantization_amd.ttq_layer import ttq_linear, ttq_quantize

    note(f"wrappers of ttq with codes M={M} K={K} N={N}")
    x, w, dy = randn(M, K, seed=4), randn(N, K, seed=5, dtype=F32), randn(M, N, seed=6)
    p = torch.tensor([0.5, 0.7, 0.6], device="cuda")
    leaves = [t.clone().requires_grad_(True) for t in (x, w, p)]
    y0 = ttq_linear(*leaves, checkpoint=True)
    dx0, dw0, dp0 = torch.autograd.grad(y0, leaves, dy)
    packed, wt = ttq_quantize(w, p)
    codes, scales = codes_like(M, K)
    y, dx, dw = (torch.empty(s, device="cuda", dtype=t) for s, t in (((M, N), BF), ((M, K), BF), ((N, K), F32)))
    grads = torch.empty(2, device="cuda")
    wf, wb = (torch.full((max(n, 16),), 255, dtype=torch.uint8, device="cuda") if own_workspace else None
              for n in (B.ttq_fwd_ckpt_workspace_bytes(M, N, K), B.ttq_bwd_ckpt_workspace_bytes(M, N, K)))
    B.ttq_fwd_ckpt(x, wt, y, codes, scales, workspace=wf)
    B.ttq_bwd_ckpt(dy, codes, scales, wt, packed, K, dX=dx, dW=dw, grads=grads, workspace=wb)
    want = compress(x)
    assert torch.equal(codes, want[0]) and torch.equal(scales, want[1])
    assert torch.equal(y, y0) and torch.equal(dx, dx0) and torch.equal(dw, dw0) and torch.equal(grads, dp0[1:])
    # without codes: the same y; dX alone needs none
    y.zero_()
    B.ttq_fwd_ckpt(x, wt, y, workspace=wf)
    dx.zero_()
    B.ttq_bwd_ckpt(dy, None, None, wt, packed, K, dX=dx, workspace=wb)
    assert torch.equal(y, y0)
    assert ((dx.double() - dx0.double()).abs() <= 2.0 ** -7 * (dy.double().abs() @ wt[:, :K].double().abs())).all()
    with pytest.raises(ValueError):
        B.ttq_bwd_ckpt(dy, codes, None, wt, packed, K, dX=dx, dW=dw)
    with pytest.raises(ValueError):
        B.ttq_fwd_ckpt(x, wt, y, codes, None)
