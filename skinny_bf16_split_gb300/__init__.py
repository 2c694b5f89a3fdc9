"""GB300 (sm_103a) decode projection: y[B,N] = BF16(x[B,K] . W[N,K]^T).

The skinny BF16 linear a decode step applies at tensor-parallel degree 1
(runtime.dep page, DepProjection), as a C-ABI library of hand-written CUDA
kernels with a thin ctypes binding.  Submodules:

  _binding  the C functions under their C names, and ``Projection``
  synth     seeded synthetic inputs shared by tests, benchmark and oracle checks
  build     nvcc build of the library

Around the projections: ``add_rms_norm``, ``quantize_rows``, ``Int8Projection`` and
``gated_delta_rule`` (norm with an 8-bit output, the projection in 8-bit integers and
the gated delta rule of a delta-attention layer), ``norm_rotate``, ``append_kv`` and
``paged_attention`` (heads' norm and rotary position, the paged cache and attention over
it, of a softmax-attention layer; ``rotary_freqs`` makes the rotation's frequencies).

The binding loads the library lazily, on first use, and raises if it is
missing: there is no CPU or library fallback.
"""
from ._binding import *  # noqa: F401,F403
from ._binding import DepError, Int8Projection, Projection, dep_tactic_t, lib, EXPORTS  # noqa: F401
from ._binding import add_rms_norm, gated_delta_rule, quantize_rows  # noqa: F401
from ._binding import append_kv, norm_rotate, paged_attention, rotary_freqs  # noqa: F401
