"""8-bit rows, the gated pair and the 8-bit layer where their arithmetic and their
sizes end."""

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
