"""B200-native (sm_100a) token-choice MoE expert layer, forward and backward, with
the layer norm, dropout and shared feed-forward expert of the block around it.

The compute lives in ``libmoe_b200.so`` (hand-written CUDA); ``binding``
exposes its C entry points to Python, ``layer`` strings them into one step,
and ``synth`` draws the seeded synthetic workloads.  Importing this package
does not load the library; the first binding call does, and raises if the
library has not been built.
"""
from .binding import (MOE_BF16, MOE_F32, MOE_ROUND_NEAREST, MOE_ROUND_NONE, MoEError,  # noqa: F401
                      moe_check_status, moe_combine, moe_dropout_bwd, moe_dropout_fwd,
                      moe_expert_ffn_fwd, moe_layer_bwd, moe_layernorm_bwd, moe_layernorm_fwd,
                      moe_permute, moe_route, moe_row_capacity, moe_shared_ffn_bwd,
                      moe_shared_ffn_fwd)

__all__ = ["moe_route", "moe_permute", "moe_expert_ffn_fwd", "moe_combine", "moe_layer_bwd",
           "moe_layernorm_fwd", "moe_layernorm_bwd", "moe_dropout_fwd", "moe_dropout_bwd",
           "moe_shared_ffn_fwd", "moe_shared_ffn_bwd", "moe_check_status", "moe_row_capacity",
           "MoEError"]
