"""B200-native selective scan (Mamba S6): forward, backward and decode step,
with state passing and packed documents, the causal depthwise conv1d that
feeds the scan, the Mamba-2 SSD forward and backward, and the time-major
operators around it: convolution, prompts and single tokens on state caches,
gated norm.

The compute lives in libss.so (hand-written sm_100a CUDA behind the C ABI of
include/ss.h); ``ops`` is its ctypes binding.
"""
from .ops import (SSError, causal_conv1d_fn, causal_conv1d_tm_fn, conv1d_bwd,  # noqa: F401
                  conv1d_fwd, conv1d_step, conv1d_tm_bwd, conv1d_tm_fwd, fwd_path, gated_norm_bwd,
                  gated_norm_fn, gated_norm_fwd, lib, selective_scan_fn, ss_bwd, ss_fwd,
                  ss_state_update, ssd_bwd, ssd_fn, ssd_fwd, ssd_prefill, ssd_step)
