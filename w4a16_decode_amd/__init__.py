"""w4a16_decode_amd: INT4 group-wise RTN weight quantization and the fused
W4A16 GEMV / skinny GEMM for AMD MI355X (gfx950), plus per-channel INT8
weights with the W8A16 GEMV, the attention side of a decoder layer on a paged
INT4 KV cache, and the turn of a serving loop around it (batch plans, sampling).

Every computation runs in the HIP kernels of ``libq4.so`` behind the C ABI
declared under ``include/``; this package only marshals torch tensors (device
memory, the current HIP stream) into those calls. There is no CPU
fallback: without the built library or a GPU the calls raise.
"""

from .attention import (  # noqa: F401
    PagedKVCache4,
    paged_attention,
    paged_attention_shared,
    paged_attention_shared_workspace_bytes,
    paged_attention_workspace_bytes,
    paged_kv_alloc,
    paged_kv_append,
    paged_kv_dequant,
    qk_norm_rope,
    qk_norm_rope_append,
    rope_table,
)
from .lora import LoraAdapters, gemm_lora, workspace_bytes_lora  # noqa: F401
from .ops import (  # noqa: F401
    ActOrderWeight,
    KVCache4,
    Q4Error,
    QuantizedWeight,
    QuantizedWeight8,
    actorder_perm,
    from_canonical,
    gemm,
    gemm_config,
    gemm_noalloc,
    gemm_perm,
    gemm_shape,
    groups_count,
    kv_cache_alloc,
    kv_dequant,
    kv_quantize_pack,
    packed_bytes,
    q8_from_canonical,
    q8_gemm,
    q8_gemm_config,
    q8_packed_bytes,
    q8_quantize_pack,
    q8_to_canonical,
    q8_workspace_bytes,
    quantize_pack,
    quantize_pack_clip,
    quantize_pack_clip_into,
    quantize_pack_into,
    quantize_pack_perm,
    read_probe,
    rtn_check,
    status_str,
    to_canonical,
    version,
    workspace_bytes,
    workspace_bytes_perm,
)
from .serving import (  # noqa: F401
    BatchPlan,
    PagePool,
    page_pool,
    paged_plan,
    sample,
    sample_workspace_bytes,
)

__all__ = [
    "Q4Error", "QuantizedWeight", "quantize_pack", "quantize_pack_into", "quantize_pack_clip", "quantize_pack_clip_into", "gemm", "gemm_noalloc", "gemm_config", "to_canonical",
    "from_canonical", "packed_bytes", "groups_count", "workspace_bytes", "gemm_shape", "status_str", "version",
    "QuantizedWeight8", "q8_quantize_pack", "q8_gemm", "q8_gemm_config", "q8_to_canonical", "q8_from_canonical",
    "q8_packed_bytes", "q8_workspace_bytes",
    "ActOrderWeight", "actorder_perm", "quantize_pack_perm", "gemm_perm", "workspace_bytes_perm",
    "LoraAdapters", "gemm_lora", "workspace_bytes_lora",
    "KVCache4", "kv_cache_alloc", "kv_quantize_pack", "kv_dequant",
    "PagedKVCache4", "paged_kv_alloc", "paged_kv_append", "paged_kv_dequant", "rope_table", "qk_norm_rope",
    "qk_norm_rope_append", "paged_attention", "paged_attention_workspace_bytes",
    "paged_attention_shared", "paged_attention_shared_workspace_bytes",
    "PagePool", "page_pool", "BatchPlan", "paged_plan", "sample", "sample_workspace_bytes", "read_probe", "rtn_check",
]
