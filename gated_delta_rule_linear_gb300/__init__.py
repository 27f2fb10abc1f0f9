"""Chunkwise linear-attention forward for NVIDIA GB300 (sm_103a).

The compute lives in libla.so (C ABI, include/la.h): hand-written CUDA
kernels for the chunkwise causal forward pass of the gated delta-rule family
(plain linear attention, elu+1 normalised attention, RetNet decay, GLA gates,
scalar decay, Gated DeltaNet, Kimi Delta Attention, the outer-product gate;
the generalised delta rule), its one-token decode
step, the backward pass (linear, RetNet, scalar decay, GLA, Gated DeltaNet),
and the prologue in front of it (short convolution, L2 normalisation,
gate activations); and the operators of a retention layer around it
(include/la_layer.h): rotary positions, retention over packed sequences
(forward, backward, single tokens) and the block epilogue; and what decoding
with paged caches and beams needs (include/la_serve.h): appending to the cache,
attention over it, beam selection, reordering of states and pages. This package
is only the binding: ctypes marshalling plus a build helper.
"""
from ._binding import (CONSTANTS, GATE_KINDS, LIB_PATH, MODE_IDS, SIGNATURES, LAError, chunk_bwd,
                       chunk_bwd_delta, chunk_fwd, chunk_fwd_gdelta, la_chunk_bwd, la_chunk_bwd_delta, la_chunk_fwd, la_chunk_fwd_gdelta, la_chunk_fwd_noalloc,
                       la_last_error, la_prologue,
                       la_recurrent_step, la_stream_status, la_version, load_library, prologue, recurrent_step)
from ._binding import *  # noqa: F401,F403  (LA_* constants)
from ._layer import (ACT_IDS, LAYER_CONSTANTS, LAYER_SIGNATURES, epilogue, epilogue_bwd, la_epilogue, la_epilogue_bwd,
                     la_packed_bwd, la_packed_fwd, la_packed_step, la_rotary, packed_bwd, packed_fwd, packed_step,
                     rotary)
from ._layer import *  # noqa: F401,F403  (LA_* constants)
from ._serve import (SERVE_SIGNATURES, beam_cache, beam_select, beam_states, cache_append, la_beam_cache,
                     la_beam_select, la_beam_states, la_cache_append, la_paged_attn, paged_attn)

__all__ = ["chunk_fwd", "chunk_bwd", "chunk_bwd_delta", "chunk_fwd_gdelta", "recurrent_step", "prologue",
           "la_chunk_fwd", "la_chunk_bwd", "la_chunk_bwd_delta", "la_chunk_fwd_gdelta", "la_chunk_fwd_noalloc",
           "la_prologue", "la_recurrent_step", "GATE_KINDS",
           "la_stream_status", "la_last_error", "la_version", "load_library", "LAError",
           "packed_fwd", "packed_bwd", "packed_step", "rotary", "epilogue", "epilogue_bwd",
           "la_packed_fwd", "la_packed_bwd", "la_packed_step", "la_rotary", "la_epilogue", "la_epilogue_bwd",
           "cache_append", "paged_attn", "beam_select", "beam_states", "beam_cache",
           "la_cache_append", "la_paged_attn", "la_beam_select", "la_beam_states", "la_beam_cache", "SERVE_SIGNATURES",
           "ACT_IDS", "LAYER_CONSTANTS", "LAYER_SIGNATURES",
           "CONSTANTS", "MODE_IDS", "SIGNATURES", "LIB_PATH"]
