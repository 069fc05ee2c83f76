"""MI355X-native BitNet b1.58 BitLinear (ternary weights, int8 activations).

The compute path is the HIP library ``libbitnet.so`` built from ``csrc/``
(C ABI declared in ``include/bitnet.h``). ``binding`` wraps its entry points
with the same names; ``layer`` adds the autograd function and the
``QATBitLinear`` module, ``ttq_layer`` the same for the TTQ variant
(``TTQLinear``), ``norm`` the layer norm that stands before them
(``QATLayerNorm``), ``checkpoint`` activations kept in 8 bits with the
gated activation between them, and ``loss`` the head of a language model with
its cross entropy (``LinearCrossEntropy``). Submodules load lazily so that importing the package (e.g.
for ``workloads``) neither imports torch nor loads the library.
"""

import importlib

_SUBMODULES = ("binding", "layer", "ttq_layer", "norm", "checkpoint", "loss", "workloads", "build")

__all__ = list(_SUBMODULES)


def __getattr__(name):
    if name in _SUBMODULES:
        return importlib.import_module(f"{__name__}.{name}")
    if name in ("QATBitLinear", "BitLinearFunction"):
        return getattr(importlib.import_module(f"{__name__}.layer"), name)
    if name in ("TTQLinear", "TTQFunction"):
        return getattr(importlib.import_module(f"{__name__}.ttq_layer"), name)
    if name in ("QATLayerNorm", "layer_norm"):
        return getattr(importlib.import_module(f"{__name__}.norm"), name)
    if name in ("compress", "decompress", "gated_activation"):
        return getattr(importlib.import_module(f"{__name__}.checkpoint"), name)
    if name in ("LinearCrossEntropy", "linear_cross_entropy"):
        return getattr(importlib.import_module(f"{__name__}.loss"), name)
    raise AttributeError(name)
