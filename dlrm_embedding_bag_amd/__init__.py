"""MI355X-native DLRMv1 forward hot path.

The compute lives in libdlrm_mi355x.so (hand-written HIP kernels for gfx950
behind the C ABI of include/dlrm_embedding_bag.h).  `abi` is the ctypes
binding with the same entry-point names; `inputs` draws seeded synthetic
inputs.  Importing this package loads nothing; the library is loaded on the
first call and a missing library raises.
"""
from .abi import (  # noqa: F401
    DlrmError, DlrmModel, DlrmPlan, dlrm_emb_interact, dlrm_emb_interact_dots, dlrm_emb_interact_pool, dlrm_forward,
    dlrm_forward_workspace_bytes, dlrm_interact_lower_tri, emb_bag_pool, emb_bag_sum_multi,
    linear_bias_act, linear_bias_act_split, load, mlp_forward)
from .attention_ops import (  # noqa: F401
    KVCache, attention_cached, attention_cached_workspace_bytes, attention_packed,
    attention_packed_grad, attention_packed_grad_workspace_bytes, kv_cache, kv_cache_read,
    kv_cache_write, qk_norm_rope, qk_norm_rope_grad, qk_norm_rope_grad_workspace_bytes)
from .token_ops import (  # noqa: F401
    emb_lookup_grad, emb_lookup_grad_workspace_bytes, emb_lookup_scaled, linear_i8_bias_act,
    rms_norm_residual_i8)
