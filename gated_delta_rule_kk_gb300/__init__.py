"""Gated delta-rule (GDN / KDA) chunked forward and decode for GB300 (sm_103a),
with the short causal convolution in front of such layers and the state space
scan beside them.

The arithmetic lives in the CUDA library built from ``csrc/`` (see
``build_lib.py``); this package holds its ctypes binding and the seeded
synthetic input generators.
"""
from .api import (  # noqa: F401
    gdn_check_device_error, gdn_chunk_fwd, gdn_chunk_segment_count, gdn_chunk_fwd_host, gdn_chunk_fwd_noalloc,
    gdn_chunk_state_bwd, gdn_chunk_state_fwd,
    gdn_chunk_host_workspace_bytes, gdn_decode,
    gdn_noalloc_scratch_bytes, kda_chunk_fwd,
)
from .api_ssm import (  # noqa: F401
    short_conv_bwd, short_conv_decode, short_conv_fwd, ssm_chunk_fwd, ssm_decode,
)
from ._lib import GateKind, GdnError, Status  # noqa: F401
