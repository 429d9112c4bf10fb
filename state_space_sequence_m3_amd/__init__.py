"""MI355X-native Mamba-3 SSM layer core.

The compute lives in ``libm3scan.so`` (hand-written HIP for gfx950, C ABI declared in
``include/m3scan.h`` for the core, ``include/m3block.h`` for the operators around it and ``include/m3attn.h`` for
attention layers between them).  ``state_space_sequence_m3_amd.m3scan``, ``.m3block`` and ``.m3attn`` are the thin ctypes
bindings with the same entry-point names; ``state_space_sequence_m3_amd.inputs`` draws the seeded synthetic workloads.
Importing this package does not load the GPU library; the bindings load it on first use and raise
if it is missing.
"""
from . import inputs  # noqa: F401

__all__ = ["inputs"]
