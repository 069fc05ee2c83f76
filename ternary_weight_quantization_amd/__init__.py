"""MI355X-native BitNet b1.58 BitLinear (ternary weights, int8 activations).

The compute path is the HIP library ``libbitnet.so`` built from ``csrc/``
(C ABI declared in ``include/bitnet.h``). ``binding`` wraps its entry points
with the same names; ``layer`` adds the autograd function and the
``QATBitLinear`` module, ``ttq_layer`` the same for the TTQ variant
(``TTQLinear``), ``norm`` the layer norm that stands before them
(``QATLayerNorm``), ``checkpoint`` activations kept in 8 bits with the
gated activation between them, ``loss`` the head of a language model with
its cross entropy (``LinearCrossEntropy``), ``rows`` the 8-bit rows that the RMS
norm (``QATRMSNorm``) hands to the layers, ``ffn`` the gated pair of ternary
projections (``QATGatedBitLinear``) and ``int8_layer`` the layers kept in 8 bits
(``QATInt8Linear``). Submodules load lazily so that importing the package (e.g.
for ``workloads``) neither imports torch nor loads the library.
"""

import importlib

_SUBMODULES = ("binding", "layer", "ttq_layer", "norm", "checkpoint", "loss", "rows", "ffn", "int8_layer",
               "workloads", "build")

__all__ = list(_SUBMODULES)


def __getattr__(name):
    if name in _SUBMODULES:
        return importlib.import_module(f"{__name__}.{name}")
    if name in ("QATBitLinear", "BitLinearFunction"):
        return getattr(importlib.import_module(f"{__name__}.layer"), name)
    if name in ("TTQLinear", "TTQFunction"):
        return getattr(importlib.import_module(f"{__name__}.ttq_layer"), name)
    if name in ("QATLayerNorm", "layer_norm", "QATRMSNorm", "rms_norm"):
        return getattr(importlib.import_module(f"{__name__}.norm"), name)
    if name in ("compress", "decompress", "gated_activation"):
        return getattr(importlib.import_module(f"{__name__}.checkpoint"), name)
    if name in ("LinearCrossEntropy", "linear_cross_entropy"):
        return getattr(importlib.import_module(f"{__name__}.loss"), name)
    if name == "QuantizedRows":
        return getattr(importlib.import_module(f"{__name__}.rows"), name)
    if name in ("QATGatedBitLinear", "gated_bitlinear", "gated_bitlinear_inference"):
        return getattr(importlib.import_module(f"{__name__}.ffn"), name)
    if name in ("QATInt8Linear", "int8_linear", "int8_linear_inference"):
        return getattr(importlib.import_module(f"{__name__}.int8_layer"), name)
    raise AttributeError(name)
