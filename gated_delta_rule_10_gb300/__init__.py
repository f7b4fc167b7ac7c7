"""GB300-native (sm_103a) gated delta rule: chunkwise forward, decode step
and the output epilogue (RMSNorm + SiLU output gate), and the operators a layer
needs around it: linear attention with a decay for each head, the residual RMS
norm and rotary positions; and those of a block: the short causal convolution, the
state space recurrence, the norms after and before the block.

The computation lives in ``libgdr.so`` (hand-written CUDA kernels behind the C
ABI of ``include/gdr.h``); this package only marshals arguments to it.
"""
from ._binding import (BETA_CHANNEL, CHUNK, DECAY_CHANNEL, ERASE_CHANNEL, GDR_BF16, GDR_F32, QMIX,
                       WRITE_CHANNEL, GdrError, Shape, chunk_bwd, chunk_bwd_check, chunk_bwd_workspace_bytes, token_bwd, token_bwd_workspace_bytes, chunk_fwd, chunk_fwd_check, chunk_fwd_workspace_bytes,
                       chunk_fwd_pipelined_workspace_bytes, gate_cumsum, lib, make_shape,
                       pipeline_segments, recurrent_step, rmsnorm_gate, status_string,
                       token_fwd)
from .block import (ConvShape, StateSpaceShape, block_norms, block_norms_bwd, short_conv_bwd,
                    short_conv_bwd_workspace_bytes, short_conv_fwd, short_conv_step,
                    state_space_bwd, state_space_bwd_workspace_bytes, state_space_fwd,
                    state_space_fwd_workspace_bytes, state_space_step)
from .layer import (DecayShape, add_rmsnorm, add_rmsnorm_bwd, add_rmsnorm_fp8, decay_chunk_bwd,
                    decay_chunk_bwd_workspace_bytes, decay_chunk_fwd,
                    decay_chunk_fwd_workspace_bytes, decay_step, rotary, rotary_table)

__all__ = ["BETA_CHANNEL", "CHUNK", "DECAY_CHANNEL", "ERASE_CHANNEL", "WRITE_CHANNEL", "QMIX", "GDR_BF16",
           "GDR_F32", "GdrError", "Shape", "chunk_bwd", "chunk_bwd_check", "chunk_bwd_workspace_bytes", "token_bwd", "token_bwd_workspace_bytes", "chunk_fwd", "chunk_fwd_check", "chunk_fwd_workspace_bytes",
           "chunk_fwd_pipelined_workspace_bytes", "gate_cumsum", "lib", "make_shape",
           "pipeline_segments", "recurrent_step", "rmsnorm_gate", "status_string", "token_fwd",
           "DecayShape", "add_rmsnorm", "add_rmsnorm_bwd", "add_rmsnorm_fp8", "decay_chunk_bwd",
           "decay_chunk_bwd_workspace_bytes", "decay_chunk_fwd", "decay_chunk_fwd_workspace_bytes",
           "decay_step", "rotary", "rotary_table", "ConvShape", "StateSpaceShape", "block_norms",
           "block_norms_bwd", "short_conv_bwd", "short_conv_bwd_workspace_bytes", "short_conv_fwd",
           "short_conv_step", "state_space_bwd", "state_space_bwd_workspace_bytes",
           "state_space_fwd", "state_space_fwd_workspace_bytes", "state_space_step"]
