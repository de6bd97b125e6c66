"""B200-native Mamba-2 SSD layer: ``forward`` (chunked prefill) and ``step`` (decode),
and the operators around them: ``rms_norm``, ``linear``, ``conv`` and ``conv_step``.

The compute lives in the C-ABI library ``libssd_b200.so`` (hand-written
sm_100a CUDA, declared in ``include/ssd.h``); ``ssd.py`` is a thin ctypes
binding that only marshals arguments, and so is ``layer.py``. Importing this
package does not load the library; the first use of an operator or ``lib``
does, and fails loudly if it is missing. ``inputs`` (seeded synthetic data) needs no GPU.
"""
from __future__ import annotations

import importlib

__all__ = ["forward", "step", "rms_norm", "linear", "conv", "conv_step", "workspace_size", "lib",
           "SSDError", "inputs", "ssd", "layer"]


def __getattr__(name):
    if name in ("inputs", "ssd", "layer"):
        return importlib.import_module(f".{name}", __name__)
    if name in ("forward", "step", "workspace_size", "lib", "SSDError", "poll_status",
                "forward_host", "library_path"):
        mod = importlib.import_module(".ssd", __name__)
        return getattr(mod, name)
    if name in ("rms_norm", "linear", "conv", "conv_step"):
        fn = getattr(importlib.import_module(".layer", __name__), name)
        globals()[name] = fn  # found at once from here on
        return fn
    raise AttributeError(name)
