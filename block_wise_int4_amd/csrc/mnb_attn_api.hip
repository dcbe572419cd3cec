// The C ABI of the decoder's attention operators (include/mnb.h): argument
// checks on the host and the hand-over to the launchers. Nothing here
// allocates or synchronizes.
#include <math.h>

#include "../../include/mnb.h"
#include "mnb_attn.h"

using namespace mnb;

namespace {

constexpr int64_t kIntMax = 0x7FFFFFFFLL;

inline bool aligned(const void *p, uintptr_t to) { return (reinterpret_cast<uintptr_t>(p) & (to - 1)) == 0; }

struct Range {
    uintptr_t from, to;
};
inline Range range(const void *p, int64_t bytes) {
    const uintptr_t from = reinterpret_cast<uintptr_t>(p);
    return {from, from + (uintptr_t)bytes};
}

// (an empty range overlaps nothing, wherever it lies)
inline bool overlap(const Range &a, const Range &b) {
    return a.from < b.to && b.from < a.to && a.from < a.to && b.from < b.to;
}

inline int hip_status(hipError_t e) { return e == hipSuccess ? MNB_OK : MNB_ERR_HIP; }

inline int64_t dtype_bytes(int dtype) { return dtype == MNB_F16 ? 2 : 4; }

inline bool known_dtype(int dtype) { return dtype == MNB_F16 || dtype == MNB_F32; }

inline bool page_ok(int64_t page) { return page > 0 && page <= MNB_MAX_PAGE && page % kPageGranule == 0; }

// Strides (elements) that keep every row 16-byte aligned; not negative, and
// small enough that no product with an index in range leaves 64 bits.
int check_strides(int64_t a, int64_t b, int64_t c, int dtype) {
    const int64_t most = 1LL << 40, unit = 16 / dtype_bytes(dtype);
    if (a < 0 || b < 0 || c < 0 || a > most || b > most || c > most) return MNB_ERR_SHAPE;
    if (a % unit || b % unit || c % unit) return MNB_ERR_ALIGN;
    return MNB_OK;
}

int check_cache(const mnb_kv_cache *c) {
    if (!c || !c->k || !c->v) return MNB_ERR_NULL;
    if (!known_dtype(c->dtype)) return MNB_ERR_DTYPE;
    if (c->num_blocks < 1 || c->num_blocks > kIntMax || c->kv_heads < 1 || c->kv_heads > kIntMax ||
        !page_ok(c->page_size) || (c->head_dim != 64 && c->head_dim != 128))
        return MNB_ERR_SHAPE;
    if (int st = check_strides(c->block_stride, c->head_stride, c->token_stride, c->dtype)) return st;
    if (c->token_stride > kMaxKeyStride) return MNB_ERR_SHAPE;
    if (!aligned(c->k, 16) || !aligned(c->v, 16)) return MNB_ERR_ALIGN;
    return c->reserved == 0 ? MNB_OK : MNB_ERR_INVALID;
}

// Head counts and sizes of an attention call; `rows` query rows per
// (request, key-value head).
int check_heads(int64_t B, int64_t Tq, int64_t Tk, int64_t Hq, int64_t Hkv, int64_t head_dim, int dtype) {
    if (!known_dtype(dtype)) return MNB_ERR_DTYPE;
    if (head_dim != 64 && head_dim != 128) return MNB_ERR_SHAPE;
    if (B < 0 || B > MNB_MAX_REQUESTS || Tq < 0 || Tq > MNB_MAX_ROWS || Tk < 0 || Tk > MNB_MAX_KEYS)
        return MNB_ERR_SHAPE;
    if (Hq < 1 || Hkv < 1 || Hq > kIntMax || Hkv > Hq || Hq % Hkv != 0) return MNB_ERR_SHAPE;
    const int64_t rows = Tq * (Hq / Hkv);
    if (rows > kIntMax || B * Hkv > kIntMax) return MNB_ERR_SHAPE;
    return attn_fits(B, Hkv, rows, Tk, (int)head_dim, dtype) ? MNB_OK : MNB_ERR_SHAPE;
}

// The scale the kernels take. Float16 scores are multiplied by scale * log2(e) at
// once, which must not overflow: products of float16 rows are whole multiples of
// 2^-48 and below 2^40, so at 2^80 all scores are finite and different ones 2^32
// apart, and a larger scale has the same softmax.
float kernel_scale(float scale, int dtype) {
    return dtype == MNB_F16 ? copysignf(fminf(fabsf(scale), 0x1p80f), scale) : scale;
}

int check_workspace(int64_t need, const void *workspace, size_t bytes) {
    if (need == 0) return MNB_OK;
    if (!workspace) return MNB_ERR_NULL;
    if (!aligned(workspace, 16)) return MNB_ERR_ALIGN;
    return bytes < (size_t)need ? MNB_ERR_INVALID : MNB_OK;
}

// Workspace of a cross attention call: by sizes alone, whichever kernel its
// strides allow.
int64_t cross_workspace(int64_t B, int64_t Hkv, int64_t rows, int64_t Tk, int head_dim, int dtype) {
    return cross_many(B, Hkv, rows, Tk, head_dim, dtype) ? 0 : attn_workspace_bytes(B, Hkv, rows, Tk, head_dim, dtype);
}

}  // namespace

extern "C" {

int mnb_kv_tables(const int32_t *cached, const int32_t *added, const int32_t *free_blocks, int64_t n_free, int64_t B,
                  int64_t page_size, int64_t max_blocks, int64_t T, int32_t *block_table, int32_t *lens,
                  int32_t *starts, int64_t *slots, int32_t *taken, void *stream) {
    if (B > 0 && (!cached || !added || !block_table || !lens)) return MNB_ERR_NULL;
    if (!starts || !taken || (n_free > 0 && !free_blocks) || (T > 0 && !slots)) return MNB_ERR_NULL;
    if (B < 0 || B > MNB_MAX_REQUESTS || n_free < 0 || n_free > kIntMax || T < 0 || T > MNB_MAX_ROWS)
        return MNB_ERR_SHAPE;
    if (!page_ok(page_size) || max_blocks < 1 || max_blocks > MNB_MAX_KEYS / page_size ||
        (B > 0 && max_blocks > kIntMax / B))
        return MNB_ERR_SHAPE;
    if (!aligned(cached, 4) || !aligned(added, 4) || !aligned(free_blocks, 4) || !aligned(block_table, 4) ||
        !aligned(lens, 4) || !aligned(starts, 4) || !aligned(slots, 8) || !aligned(taken, 4))
        return MNB_ERR_ALIGN;
    // (workgroups read the lengths while others write: lens in the place of
    // cached would race)
    const Range of[] = {range(cached, 4 * B), range(added, 4 * B), range(free_blocks, 4 * n_free),
                        range(block_table, 4 * B * max_blocks), range(lens, 4 * B), range(starts, 4 * (B + 1)),
                        range(slots, 8 * T), range(taken, 4)};
    for (int o = 3; o < 8; ++o)
        for (int i = 0; i < o; ++i)
            if (overlap(of[i], of[o])) return MNB_ERR_INVALID;
    KvTablesArgs a{};
    a.cached = cached;
    a.added = added;
    a.free_blocks = free_blocks;
    a.n_free = n_free;
    a.tokens = T;
    a.batch = (int32_t)B;
    a.page = (int32_t)page_size;
    a.width = (int32_t)max_blocks;
    a.table = block_table;
    a.lens = lens;
    a.starts = starts;
    a.taken = taken;
    a.slots = slots;
    return hip_status(launch_kv_tables(a, static_cast<hipStream_t>(stream)));
}

int mnb_kv_append(const void *k, const void *v, int64_t k_stride, int64_t v_stride, const int64_t *slots, int64_t T,
                  const mnb_kv_cache *cache, void *stream) {
    if (int st = check_cache(cache)) return st;
    if (T < 0 || T > MNB_MAX_ROWS) return MNB_ERR_SHAPE;
    if (int st = check_strides(k_stride, v_stride, 0, cache->dtype)) return st;
    if (T == 0) return MNB_OK;
    if (!k || !v || !slots) return MNB_ERR_NULL;
    if (!aligned(k, 16) || !aligned(v, 16) || !aligned(slots, 8)) return MNB_ERR_ALIGN;
    const int64_t es = dtype_bytes(cache->dtype);
    // (a token's pieces are counted in 32 bits)
    if (cache->kv_heads > kIntMax / (cache->head_dim * es)) return MNB_ERR_SHAPE;
    KvAppendArgs a{};
    a.k = static_cast<const uint8_t *>(k);
    a.v = static_cast<const uint8_t *>(v);
    a.k_cache = static_cast<uint8_t *>(cache->k);
    a.v_cache = static_cast<uint8_t *>(cache->v);
    a.slots = slots;
    a.tokens = T;
    a.k_stride = k_stride * es;
    a.v_stride = v_stride * es;
    a.num_blocks = cache->num_blocks;
    a.block_stride = cache->block_stride * es;
    a.head_stride = cache->head_stride * es;
    a.token_stride = cache->token_stride * es;
    a.heads = (int32_t)cache->kv_heads;
    a.row_bytes = (int32_t)(cache->head_dim * es);
    a.page = (int32_t)cache->page_size;
    return hip_status(launch_kv_append(a, static_cast<hipStream_t>(stream)));
}

size_t mnb_paged_attn_workspace_bytes(int64_t B, int64_t Hq, int64_t Hkv, int64_t head_dim, int64_t max_len,
                                      int dtype) {
    if (check_heads(B, 1, max_len, Hq, Hkv, head_dim, dtype) != MNB_OK || B == 0) return 0;
    return (size_t)attn_workspace_bytes(B, Hkv, Hq / Hkv, max_len, (int)head_dim, dtype);
}

int mnb_paged_attn(const void *q, int64_t q_stride, const mnb_kv_cache *cache, const int32_t *block_table,
                   const int32_t *lens, int64_t B, int64_t Hq, int64_t max_blocks, int64_t max_len, float scale,
                   void *workspace, size_t workspace_bytes, void *out, void *stream) {
    if (int st = check_cache(cache)) return st;
    if (int st = check_heads(B, 1, max_len, Hq, cache->kv_heads, cache->head_dim, cache->dtype)) return st;
    if (max_blocks < 1 || max_blocks > kIntMax / (B > 0 ? B : 1)) return MNB_ERR_SHAPE;
    if (int st = check_strides(q_stride, 0, 0, cache->dtype)) return st;
    if (!isfinite(scale)) return MNB_ERR_INVALID;
    if (B == 0) return MNB_OK;
    if (!q || !block_table || !lens || !out) return MNB_ERR_NULL;
    if (!aligned(q, 16) || !aligned(out, 16) || !aligned(block_table, 4) || !aligned(lens, 4)) return MNB_ERR_ALIGN;
    const int head_dim = (int)cache->head_dim;
    const int64_t group = Hq / cache->kv_heads;
    const int64_t need = attn_workspace_bytes(B, cache->kv_heads, group, max_len, head_dim, cache->dtype);
    if (int st = check_workspace(need, workspace, workspace_bytes)) return st;
    AttnArgs a{};
    a.q = q;
    a.k = cache->k;
    a.v = cache->v;
    a.out = out;
    a.q_batch = q_stride;
    a.q_head = head_dim;
    a.k_batch = a.v_batch = cache->block_stride;
    a.k_row = a.v_row = cache->token_stride;
    a.k_head = a.v_head = cache->head_stride;
    a.o_batch = Hq * head_dim;
    a.o_head = head_dim;
    a.lens = lens;
    a.table = block_table;
    a.batch = (int32_t)B;
    a.kv_heads = (int32_t)cache->kv_heads;
    a.group = a.rows = (int32_t)group;
    a.max_len = (int32_t)max_len;
    a.page = (int32_t)cache->page_size;
    a.table_width = (int32_t)max_blocks;
    a.num_blocks = (int32_t)cache->num_blocks;
    a.scale = kernel_scale(scale, cache->dtype);
    return hip_status(launch_attn(a, head_dim, cache->dtype, workspace, static_cast<hipStream_t>(stream)));
}

size_t mnb_cross_attn_workspace_bytes(int64_t B, int64_t Tq, int64_t Tk, int64_t Hq, int64_t Hkv, int64_t head_dim,
                                      int dtype) {
    if (check_heads(B, Tq, Tk, Hq, Hkv, head_dim, dtype) != MNB_OK || B == 0 || Tq == 0) return 0;
    return (size_t)cross_workspace(B, Hkv, Tq * (Hq / Hkv), Tk, (int)head_dim, dtype);
}

int mnb_cross_attn(const mnb_attn_view *q, const mnb_attn_view *k, const mnb_attn_view *v, const int32_t *lens,
                   int64_t B, int64_t Tq, int64_t Tk, int64_t Hq, int64_t Hkv, int64_t head_dim, float scale,
                   int dtype, void *workspace, size_t workspace_bytes, const mnb_attn_view *out, void *stream) {
    if (!q || !k || !v || !out) return MNB_ERR_NULL;
    if (int st = check_heads(B, Tq, Tk, Hq, Hkv, head_dim, dtype)) return st;
    for (const mnb_attn_view *t : {q, k, v, out})
        if (int st = check_strides(t->batch_stride, t->row_stride, t->head_stride, dtype)) return st;
    if (k->row_stride > kMaxKeyStride || v->row_stride > kMaxKeyStride) return MNB_ERR_SHAPE;
    if (!isfinite(scale)) return MNB_ERR_INVALID;
    if (B == 0 || Tq == 0) return MNB_OK;
    if (!q->data || !out->data || (Tk > 0 && (!k->data || !v->data))) return MNB_ERR_NULL;
    if (!aligned(q->data, 16) || !aligned(k->data, 16) || !aligned(v->data, 16) || !aligned(out->data, 16) ||
        !aligned(lens, 4))
        return MNB_ERR_ALIGN;
    const int64_t rows = Tq * (Hq / Hkv);
    const int64_t need = cross_workspace(B, Hkv, rows, Tk, (int)head_dim, dtype);
    if (int st = check_workspace(need, workspace, workspace_bytes)) return st;
    AttnArgs a{};
    a.q = q->data;
    a.k = k->data;
    a.v = v->data;
    a.out = out->data;
    a.q_batch = q->batch_stride;
    a.q_row = q->row_stride;
    a.q_head = q->head_stride;
    a.k_batch = k->batch_stride;
    a.k_row = k->row_stride;
    a.k_head = k->head_stride;
    a.v_batch = v->batch_stride;
    a.v_row = v->row_stride;
    a.v_head = v->head_stride;
    a.o_batch = out->batch_stride;
    a.o_row = out->row_stride;
    a.o_head = out->head_stride;
    a.lens = lens;
    a.batch = (int32_t)B;
    a.kv_heads = (int32_t)Hkv;
    a.group = (int32_t)(Hq / Hkv);
    a.rows = (int32_t)rows;
    a.max_len = (int32_t)Tk;
    a.scale = kernel_scale(scale, dtype);
    const hipStream_t st = static_cast<hipStream_t>(stream);
    if (cross_many(B, Hkv, rows, Tk, (int)head_dim, dtype) && cross_fits(a, (int)head_dim))
        return hip_status(launch_cross(a, (int)head_dim, st));
    return hip_status(launch_attn(a, (int)head_dim, dtype, need ? workspace : nullptr, st));
}

}  // extern "C"
