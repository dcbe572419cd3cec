"""MatMulNBits for AMD Instinct MI355X: weight-only block-wise int4 matmul.

The compute path is libmnb.so (HIP kernels for gfx950 behind the C ABI in
include/mnb.h); `block_wise_int4_amd.mnb` is its Python binding.
"""

from .mnb import (  # noqa: F401
    KvCache,
    MNB_F16,
    MNB_F32,
    MnbError,
    PackedWeight,
    Plan,
    cross_attn_workspace,
    lib,
    mnb_abi_version,
    mnb_cross_attn,
    mnb_cross_attn_workspace_bytes,
    mnb_dequant,
    mnb_gemm,
    mnb_gemm_i8,
    mnb_gemm_i8_workspace_bytes,
    mnb_gemm_split_k,
    mnb_gemm_split_k_workspace_bytes,
    mnb_gemm_grouped,
    mnb_gemv,
    mnb_kv_append,
    mnb_kv_tables,
    mnb_pack,
    mnb_packed_bytes,
    mnb_paged_attn,
    mnb_paged_attn_workspace_bytes,
    mnb_plan_grouped,
    mnb_quantize_act_i8,
    mnb_quantize_rtn,
    mnb_status_string,
    mnb_unpack,
    paged_attn_workspace,
)
