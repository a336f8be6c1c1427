"""GB300-native fused Mixture-of-Experts feed-forward layer.

The layer runs in ``libmoe_gb300.so`` (hand-written CUDA for sm_103a behind the C ABI of
``include/moe.h``). This package is the Python binding (``_lib``, same function names as
the C ABI), ``layer.MoELayer``, which owns the workspace and calls ``moe_forward``, and
``training``, the operators of a training step (``include/moe_train.h`` and ``moe_stack.h``) on
tensors.
"""
from ._lib import (EXPORTED, MOE_BF16, MOE_F32, MOE_GEMM_DECODE_TC,  # noqa: F401
                   MOE_GEMM_INVALID, MOE_GEMM_PAIR_TC, MOE_GEMM_SIMT, MOE_GEMM_SMALL_BATCH,
                   MOE_ROUTE_SIGMOID_GROUPED,
                   MOE_ROUTE_SOFTMAX, MOE_WEIGHTS_FP8_E4M3_B128, MOE_WEIGHTS_NATIVE, MoeError,
                   make_config, moe_abi_version, moe_align, moe_align_noalloc,
                   moe_dequant_fp8_weights,
                   moe_align_workspace_size, moe_apply_expert_map, moe_block_m, moe_combine,
                   moe_combine_local, moe_config_t, moe_device_status, moe_expert_gemm1,
                   moe_expert_gemm1_gathered, moe_expert_gemm1_gathered_workspace_size,
                   moe_expert_gemm1_workspace_size, moe_expert_gemm2,
                   moe_expert_gemm2_workspace_size, moe_forward, moe_gather_rows, moe_gemm_kernel,
                   moe_grouped_swiglu, moe_grouped_swiglu_workspace_size, moe_masked_forward,
                   moe_masked_table, moe_masked_workspace_size, moe_max_padded_rows, moe_route,
                   moe_small_batch, moe_route_logits, moe_selftest_wait_timeout,
                   moe_workspace_layout, moe_workspace_size, status_string)
from ._lib import (MOE_GATE_CHANNEL, MOE_GATE_FULL, MOE_GATE_NONE, MOE_GATE_TOKEN,  # noqa: F401
                   MOE_TRAIN_BLOCK, moe_block_join, moe_block_join_backward, moe_block_norm,
                   moe_block_norm_backward, moe_block_t, moe_block_workspace_size,
                   moe_expert_down, moe_expert_down_backward, moe_expert_up,
                   moe_expert_up_backward, moe_expert_weight_grad, moe_experts_t, moe_permute,
                   moe_permute_backward, moe_route_backward, moe_unpermute,
                   moe_unpermute_backward)
from ._lib import (moe_balance_loss, moe_balance_loss_backward, moe_balance_t,  # noqa: F401
                   moe_balance_workspace_size, moe_drop_t, moe_dropout, moe_dropout_join,
                   moe_dropout_join_backward, moe_embed, moe_embed_backward,
                   moe_embed_workspace_size, moe_layer_norm, moe_layer_norm_backward, moe_layer_t,
                   moe_layer_workspace_size)
