"""One rank's share of tensor-parallel linear layers on one MI355X.

The compute lives in ``libtsl.so``, ``libtsl_block.so`` and ``libtsl_attn.so``
(hand-written HIP kernels for gfx950 behind the C ABIs of ``include/tsl.h``,
``include/tsl_block.h`` and ``include/tsl_attn.h``).  ``binding`` is a thin ctypes layer over them with
the same entry-point names; it raises ImportError when one has not been
built -- there is no fallback.

``synth`` (seeded input generators), ``configs`` (workload sizes) and
``build`` (the compiler driver) do not need the libraries.
"""
import importlib

__all__ = ["binding", "synth", "configs"]


def __getattr__(name):
    if name in ("binding", "synth", "configs", "build"):
        return importlib.import_module("." + name, __name__)
    # entry points re-exported from the binding: loading it loads both libraries
    binding = importlib.import_module(".binding", __name__)
    if hasattr(binding, name):
        return getattr(binding, name)
    raise AttributeError(name)
