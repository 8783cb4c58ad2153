"""GB300 (sm_103a) CSA/HCA fused Compressor.

The gated-softmax pooling of the cuDNN-frontend "CSA Fused Compressor" page
as hand-written CUDA kernels behind a small C ABI (include/csa_compress.h);
this package holds the kernels (csrc/), their build and a thin Python binding.
Beside it: rotary positions (include/csa_rope.h) and a paged 8-bit cache of
the compressed rows with its attention and page handling (include/csa_cache.h).
"""
from .binding import (SEG_VIOLATIONS, CsaError, csa_check_segments, csa_compress_bwd,
                      csa_compress_bwd_noalloc_ptr, csa_compress_bwd_ptr, csa_compress_fwd,
                      csa_compress_fwd_ptr, load)
from .cache import (CACHE_STATUS, csa_cache_append, csa_cache_attend, csa_cache_compact,
                    csa_cache_copy_pages, csa_cache_fork, csa_cache_free, csa_cache_reserve)
from .nvbuild import build
from .rope import csa_rope, csa_rope_freqs

__all__ = ["CACHE_STATUS", "SEG_VIOLATIONS", "CsaError", "build", "csa_cache_append",
           "csa_cache_attend", "csa_cache_compact", "csa_cache_copy_pages", "csa_cache_fork",
           "csa_cache_free", "csa_cache_reserve", "csa_check_segments", "csa_compress_bwd",
           "csa_compress_bwd_noalloc_ptr", "csa_compress_bwd_ptr", "csa_compress_fwd",
           "csa_compress_fwd_ptr", "csa_rope", "csa_rope_freqs", "load"]
