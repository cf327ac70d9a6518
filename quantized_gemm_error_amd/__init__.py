"""MI355X-native compensated 4-bit linear layer (libspear), the paged key-value cache and attention
between such layers, the norm, microscaled 4-bit products and sampling around them, and their
Python binding."""

from .spear import (  # noqa: F401
    SPEAR_BF16,
    SPEAR_F16,
    SpearError,
    SpearLayer,
    act_to_device,
    layer_to_device,
    load_library,
    new_workspace,
    qweight_rows,
    spear_get_decode_max_m,
    spear_last_error,
    spear_linear,
    spear_linear_decode,
    spear_linear_prefill,
    spear_pack_int4,
    spear_tile_int4,
    spear_select_chunk,
    spear_set_decode_max_m,
    spear_status_string,
    spear_version,
    spear_workspace_bytes,
    spear_workspace_flags,
)
from .attn import (  # noqa: F401
    SpearKVBatch,
    SpearKVCache,
    SpearKVPool,
    new_attn_workspace,
    spear_attn_decode,
    spear_attn_prefill,
    spear_attn_workspace_bytes,
    spear_kv_append,
    spear_kv_compact,
    spear_kv_copy_pages,
    spear_kv_fork,
    spear_kv_free,
    spear_kv_reserve,
)
from .mx import (  # noqa: F401
    SPEAR_F32,
    SPEAR_MXFP4,
    SPEAR_MXFP8,
    SpearMX,
    new_mx_workspace,
    spear_mx_dequantize,
    spear_mx_linear,
    spear_mx_quantize,
    spear_mx_workspace_bytes,
    spear_rms_norm,
)
from .sampling import (  # noqa: F401
    new_sample_workspace,
    spear_sample,
    spear_sample_workspace_bytes,
)
