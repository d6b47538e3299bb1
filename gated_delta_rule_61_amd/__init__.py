"""MI355X (gfx950) gated delta rule: chunked GDN / KDA prefill forward and the
bf16-state decode step, with what stands around them in a recurrent layer (the
short causal convolution, a selective state-space scan and step, an 8-bit cache
of states), as hand-written HIP kernels behind a C ABI (``include/gdn61.h``).
The Python entry points below marshal torch tensors into that ABI; nothing is
computed in Python.
"""

from .binding import (GDNError, causal_conv_fwd, causal_conv_step, chunk_bwd_dh, gdn_chunk_fwd, gdn_decode,
                      kda_chunk_fwd, lib, ssm_chunk_fwd, ssm_step, ssm_workspace_bytes, state_load_q8,
                      state_store_q8, state_to_pool, workspace_bytes)

__all__ = ["GDNError", "causal_conv_fwd", "causal_conv_step", "chunk_bwd_dh", "gdn_chunk_fwd", "gdn_decode",
           "kda_chunk_fwd", "lib", "ssm_chunk_fwd", "ssm_step", "ssm_workspace_bytes", "state_load_q8",
           "state_store_q8", "state_to_pool", "workspace_bytes"]
__version__ = "0.1.0"
