"""MI355X (gfx950) routed MoE MLP of GLM-5.3-Flash: HIP kernels behind a C ABI.

The compute lives in lib/libmoe_mlp.so (built from csrc/ by
`python -m routed_expert_mlp_amd.build`); capi.py is its ctypes binding,
attention.py that of the attention operators over a paged key/value cache, and
projection.py that of what stands around the two: norms, FP8 projections, adapters.
"""
from .attention import (AttnConfig, KVCache, moe_attn_decode, moe_attn_decode_shared, moe_attn_prefill,  # noqa: F401
                        moe_attn_prepare, moe_attn_shared_workspace_bound, moe_attn_shared_workspace_size,
                        moe_attn_workspace_bound, moe_attn_workspace_size, new_cache)
from .capi import (Config, KIND_DENSE, KIND_ROUTED, MoeMlpError, Weights, lib,  # noqa: F401
                   moe_mlp_decode, moe_mlp_prefill, moe_mlp_status_string, moe_mlp_workspace_size,
                   moe_nvfp4_dequant, moe_router_topk, workspace)
from .projection import (Adapters, moe_proj_fp8, moe_proj_lora, moe_proj_lora_workspace_size,  # noqa: F401
                         moe_proj_norm)
