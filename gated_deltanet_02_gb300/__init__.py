"""GB300-native (sm_103a) state-passing linear-attention layer.

Gated linear attention (including the SSD form of Mamba2: a 128 x 64 state,
q / k shared by groups of heads), Gated DeltaNet and normalised kernelised
linear attention: chunked tensor-core prefill with optional prefix-cache
checkpoints, recurrent decode from a slot-indexed state pool, speculative
decode with one state per draft position or a verify-only round plus replay,
slot copies; Mamba's selective scan; the paged key / value cache of a hybrid
stack's softmax layers (write, with the position rotation where wanted, read
back, causal attention over it); the state-space block's short convolution and
scan over packed rows; the residual norm in front of a layer; and the
acceptance of drafted tokens.  All of it sits behind the C ABI
declared in ``include/glinattn.h``; ``glinattn`` is the Python binding and
``inputs`` holds the seeded synthetic input generators.
"""
from .glinattn import (BF16, E4M3, E8M0, F32, GDN, GLA, NLA, GlinattnError, glinattn_accept_drafts,
                       glinattn_add_rms_norm, glinattn_decode, glinattn_kv_append, glinattn_kv_append_rope,
                       glinattn_kv_gather, glinattn_paged_attention, glinattn_prefill, glinattn_replay,
                       glinattn_selective_scan, glinattn_selective_scan_decode, glinattn_selective_scan_packed,
                       glinattn_short_conv, glinattn_spec_decode, glinattn_state_copy, library, state_bytes,
                       status_string, version)

__all__ = ["GLA", "GDN", "NLA", "F32", "BF16", "E4M3", "E8M0", "GlinattnError", "glinattn_prefill", "glinattn_decode",
           "glinattn_spec_decode", "glinattn_replay", "glinattn_state_copy", "glinattn_selective_scan",
           "glinattn_selective_scan_decode", "glinattn_kv_append", "glinattn_kv_gather", "glinattn_paged_attention",
           "glinattn_accept_drafts", "glinattn_kv_append_rope", "glinattn_short_conv", "glinattn_selective_scan_packed",
           "glinattn_add_rms_norm", "library", "version", "status_string", "state_bytes"]
