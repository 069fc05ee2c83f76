"""8-bit rows: what the RMS norm hands to the layers that follow it.

``QuantizedRows`` stands for bf16 activations [..., K] as int8 codes with a
float32 scale a row, the form in which the ternary layers multiply them anyway.
``rms_norm(..., quantize=True)`` makes them; ``QATBitLinear``,
``gated_bitlinear`` and ``int8_linear`` (with their modules) take them in place
of activations and skip their own quantization, so one set of rows serves
several layers. What else takes activations (``TTQLinear``, ``LinearCrossEntropy``,
the norms) refuses them; ``dequantize`` gives it theirs.
"""

from . import binding as B


class QuantizedRows:
    """codes int8 [M, Kp] (Kp = K rounded up to 64, zeros past K), scales
    float32 [M]; row m, column k stands for codes[m, k] * scales[m] / 127.
    ``shape`` is that of the activations, [..., K]. Gradients of the rows'
    values, in bf16, go straight through the quantization to what made them."""

    __slots__ = ("codes", "scales", "_carrier")

    def __init__(self, codes, scales, carrier):
        self.codes, self.scales, self._carrier = codes, scales, carrier

    @property
    def shape(self):
        return self._carrier.shape

    @property
    def device(self):
        return self.codes.device

    @property
    def requires_grad(self):
        return self._carrier.requires_grad

    def detach(self):
        return QuantizedRows(self.codes, self.scales, self._carrier.detach())

    def dequantize(self):
        """The values as a bf16 tensor of ``shape``, differentiable (straight
        through, once, in reverse mode)."""
        return B.ops().rows_values(self._carrier, self.codes, self.scales)

    def __repr__(self):
        return f"QuantizedRows(shape={tuple(self.shape)}, requires_grad={self.requires_grad})"


def need_activations(what, x):
    """Refuses 8-bit rows where only activations are taken."""
    if isinstance(x, QuantizedRows):
        raise TypeError(f"{what} takes activations, not QuantizedRows (their dequantize() gives them)")


def layer_input(x):
    """(tensor, codes, scales) of a layer's input: activations as they are, or
    8-bit rows by their carrier."""
    if isinstance(x, QuantizedRows):
        return x._carrier, x.codes, x.scales
    return x, None, None
