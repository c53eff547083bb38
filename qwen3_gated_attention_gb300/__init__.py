"""GB300-native (sm_103a) gated full-attention decoder layer: decode and
speculative-verify steps through a C-ABI CUDA library (``libgattn.so``), and for
packed prompts the rows, the attention and the gated delta rule beside it; rows,
attention, received weights and eviction over a cache in pages.

``gattn``   ctypes binding of include/gattn.h (same names, marshalling only)
``device``  torch-owned device buffers around one layer handle; the
            packed-sequence and paged-cache operators on tensors
``synth``   seeded synthetic inputs
``build``   nvcc build of the library and of the module ``_paged``, which reads
            the tensors of the paged-cache calls
"""
from . import synth  # noqa: F401

__all__ = ["synth", "gattn", "device", "build"]
