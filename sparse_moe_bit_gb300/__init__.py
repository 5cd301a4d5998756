"""Sparse 4-bit Mixture-of-Experts block for GB300 (sm_103a).

The compute lives in libmoe.so (CUDA kernels behind the C ABI of
include/moe.h, the Gated DeltaNet prefill scan of include/gdn.h, and rotary
positions, the paged cache and attention over it of include/paged.h, and what
a decode step has between and behind them of include/step.h); this package is
its thin Python binding.
"""
from .moe import (MOE_DEVERR_FP16_RANGE, MOE_DEVERR_GRID_TIMEOUT, MOE_DEVERR_NAN_LOGIT,
                  MOE_DEVERR_RANGE, MOE_DEVERR_WAIT_TIMEOUT, MOE_LAYOUT_DECODE,
                  MOE_LAYOUT_PREFILL, MOE_SCALE_F16, MoE, MoEConfig, MoEError, decode,
                  decode_host, gdn_scan, load_library)
from .paged import (PAGED_DEVERR_LENGTH, PAGED_DEVERR_PAGE, PAGED_DEVERR_WAIT_TIMEOUT,
                    paged_attention, paged_attention_shared, paged_device_error, pages_compact, pages_copy, pages_fork,
                    pages_free, pages_reserve, rope, rope_append, rope_frequencies)
from .step import linear4, rms_norm, sample

__all__ = ["MoE", "MoEConfig", "MoEError", "decode", "decode_host", "gdn_scan", "load_library",
           "MOE_SCALE_F16", "MOE_LAYOUT_PREFILL", "MOE_LAYOUT_DECODE", "MOE_DEVERR_WAIT_TIMEOUT",
           "MOE_DEVERR_NAN_LOGIT", "MOE_DEVERR_GRID_TIMEOUT", "MOE_DEVERR_RANGE",
           "MOE_DEVERR_FP16_RANGE", "PAGED_DEVERR_LENGTH", "PAGED_DEVERR_PAGE",
           "PAGED_DEVERR_WAIT_TIMEOUT", "paged_attention", "paged_attention_shared",
           "paged_device_error", "pages_compact", "pages_copy", "pages_fork",
           "pages_free", "pages_reserve", "rope", "rope_append", "rope_frequencies", "linear4", "rms_norm", "sample"]
