"""GB300-native persistent MoE decode megakernel.

The compute path lives in libmk.so (CUDA kernels for sm_103a behind the C ABI of
include/mk.h); `binding` is a thin ctypes layer over it (the library is loaded on
first use and its absence is an error) and `sol` holds the speed-of-light byte
arithmetic used to report bandwidth fractions.  `ops` has the operators over several
tokens of a sequence (draft trees, prompt chunks) on the same cache and weights; it takes
torch tensors, and torch is imported with it, not with the package.
"""
import importlib

from . import binding, sol  # noqa: F401

__all__ = ["binding", "ops", "sol"]


def __getattr__(name):
    if name == "ops":
        return importlib.import_module(".ops", __name__)
    raise AttributeError(f"module {__name__!r} has no attribute {name!r}")
