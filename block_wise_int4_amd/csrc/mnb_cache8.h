// Internal declarations of the 8-bit key-value cache, the attention over it and
// the rotary positions: kernel arguments and launchers.
#pragma once
#include <hip/hip_runtime.h>
#include <stdint.h>

namespace mnb {

// Rotary positions (mnb_rope). Strides in bytes.
struct RopeArgs {
    const uint8_t *q, *k;
    uint8_t *q_out, *k_out;
    int64_t q_stride, q_out_stride, k_stride, k_out_stride;
    const int32_t *positions;
    const double *freqs;
    int64_t tokens;
    int32_t q_heads, k_heads, head_dim, rot_dim;
    float gain;
};
hipError_t launch_rope(const RopeArgs &a, bool interleaved, int dtype, hipStream_t st);

// The cache's memory: codes by strides in bytes, scales by strides in floats.
struct Cache8 {
    int8_t *k, *v;
    float *k_scale, *v_scale;
    int64_t num_blocks, block_stride, head_stride, token_stride, scale_block, scale_head;
    int32_t heads, page;
};

// Tokens into the cache, and slots back to rows (mnb_kv_append_i8,
// mnb_kv_read_i8). Row strides in bytes.
struct Kv8Args {
    Cache8 cache;
    const uint8_t *k, *v;   // append: read; read: written
    int64_t k_stride, v_stride;
    const int64_t *slots;
    int64_t tokens;
    uint32_t page_magic;    // (set by the launcher)
};
hipError_t launch_kv8_append(const Kv8Args &a, int head_dim, int dtype, hipStream_t st);
hipError_t launch_kv8_read(const Kv8Args &a, int head_dim, int dtype, hipStream_t st);

// Attention over the cache (mnb_paged_attn_i8). q_stride in elements; positions
// past the table's width are never seen.
struct Attn8Args {
    Cache8 cache;
    const void *q;
    void *out;
    const int32_t *table, *lens, *starts;   // starts NULL: one token per request
    int64_t q_stride, tokens;
    int32_t batch, group, max_new, max_len, table_width;
    float scale;
    float per_group;   // (1 / group; set by the launcher)
};
// Float32 partial results the launch needs (0: it splits nothing).
int64_t attn8_workspace_bytes(int64_t batch, int64_t kv_heads, int64_t group, int64_t max_new, int64_t max_len,
                              int head_dim, int dtype);
// False: more workgroups than a launch takes.
bool attn8_fits(int64_t batch, int64_t kv_heads, int64_t group, int64_t max_new, int64_t max_len, int head_dim,
                int dtype);
hipError_t launch_attn8(const Attn8Args &a, int head_dim, int dtype, void *workspace, hipStream_t st);

}  // namespace mnb
