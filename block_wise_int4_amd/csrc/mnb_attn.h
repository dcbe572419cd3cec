// Internal declarations of the attention operators: kernel arguments and the
// launchers of mnb_kv.hip and mnb_attn.hip.
#pragma once
#include <hip/hip_runtime.h>
#include <stdint.h>

namespace mnb {

// Keys a K or V tile shares a block-table entry over: pages hold a whole
// number of these.
constexpr int kPageGranule = 16;
constexpr int64_t kMaxKeyStride = 1LL << 26;

// A step's block tables and slot maps (mnb_kv_tables).
struct KvTablesArgs {
    const int32_t *cached, *added, *free_blocks;
    int64_t n_free, tokens;
    int32_t batch, page, width;
    int32_t *table, *lens, *starts, *taken;
    int64_t *slots;
    uint64_t page_magic;   // (set by the launcher)
};
hipError_t launch_kv_tables(const KvTablesArgs &a, hipStream_t st);

// New keys and values into the cache (mnb_kv_append). Strides in bytes; a
// token's keys (or values) are `heads` rows of row_bytes, one after another.
struct KvAppendArgs {
    const uint8_t *k, *v;
    uint8_t *k_cache, *v_cache;
    const int64_t *slots;
    int64_t tokens, k_stride, v_stride;
    int64_t num_blocks, block_stride, head_stride, token_stride;
    int32_t heads, row_bytes, page;
};
hipError_t launch_kv_append(const KvAppendArgs &a, hipStream_t st);

// Attention of `rows` query rows per (request, key-value head) over keys that
// are paged (table not NULL: the batch strides of K and V step over blocks)
// or one run per request. Row r is query token r / group, query head
// kv_head * group + r % group. Strides in elements; k_row and v_row at most
// kMaxKeyStride (16 rows are addressed from one base with 32-bit offsets).
struct AttnArgs {
    const void *q, *k, *v;
    void *out;
    int64_t q_batch, q_row, q_head;
    int64_t k_batch, k_row, k_head;
    int64_t v_batch, v_row, v_head;
    int64_t o_batch, o_row, o_head;
    const int32_t *lens;    // NULL: every request has max_len keys
    const int32_t *table;   // [batch][table_width], or NULL
    int32_t batch, kv_heads, group, rows;
    int32_t max_len;        // keys beyond this are never valid
    int32_t page, table_width, num_blocks;
    float scale;
};
// Float32 partial results the launch needs (0: it splits nothing).
int64_t attn_workspace_bytes(int64_t batch, int64_t kv_heads, int64_t rows, int64_t max_len, int head_dim,
                             int dtype);
// False: more workgroups than a launch takes.
bool attn_fits(int64_t batch, int64_t kv_heads, int64_t rows, int64_t max_len, int head_dim, int dtype);
// (workspace NULL: one launch, nothing split)
hipError_t launch_attn(const AttnArgs &a, int head_dim, int dtype, void *workspace, hipStream_t st);

// The same sums for float16 calls with many query rows over unpaged keys
// (mnb_cross.hip), which needs no workspace: whether it is the faster one, by
// sizes alone, and whether it can address these strides.
bool cross_many(int64_t batch, int64_t kv_heads, int64_t rows, int64_t max_len, int head_dim, int dtype);
bool cross_fits(const AttnArgs &a, int head_dim);
hipError_t launch_cross(const AttnArgs &a, int head_dim, hipStream_t st);

}  // namespace mnb
