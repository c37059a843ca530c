"""B200-native (sm_100a) DP-GRAPE projection step behind a C ABI (include/grape.h).

``grape`` is the ctypes binding of ``libgrape.so``; the library is built
in-tree with ``python -m random_gradient_projection_b200.build``.  ``lm`` (the two ends of
a language model, for torch tensors) is imported at its first use: the rest does without torch.
"""
from . import grape  # noqa: F401
from .grape import GrapeStep, GrapeError  # noqa: F401


def __getattr__(name):
    if name == "lm":
        import importlib
        return importlib.import_module(".lm", __name__)
    raise AttributeError(f"module {__name__!r} has no attribute {name!r}")
