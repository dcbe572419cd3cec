// The C ABI of the 8-bit key-value cache, the attention over it and the rotary
// positions (include/mnb.h): argument checks on the host and the hand-over to
// the launchers. Nothing here allocates or synchronizes.
#include <math.h>

#include "../../include/mnb.h"
#include "mnb_cache8.h"
#include "mnb_checks.h"

using namespace mnb;

namespace {

int check_cache8(const mnb_kv_cache_i8 *c) {
    if (!c || !c->k || !c->v || !c->k_scale || !c->v_scale) return MNB_ERR_NULL;
    if (!known_dtype(c->dtype)) return MNB_ERR_DTYPE;
    if (c->num_blocks < 1 || c->num_blocks > kIntMax || c->kv_heads < 1 || c->kv_heads > kIntMax ||
        !page_ok(c->page_size) || (c->head_dim != 64 && c->head_dim != 128))
        return MNB_ERR_SHAPE;
    const int64_t most = 1LL << 40;
    for (int64_t stride : {c->block_stride, c->head_stride, c->token_stride, c->scale_block_stride,
                           c->scale_head_stride})
        if (stride < 0 || stride > most) return MNB_ERR_SHAPE;
    if (c->token_stride > kMaxKeyStride) return MNB_ERR_SHAPE;
    if (c->block_stride % 16 || c->head_stride % 16 || c->token_stride % 16 || c->scale_block_stride % 4 ||
        c->scale_head_stride % 4)
        return MNB_ERR_ALIGN;
    if (!aligned(c->k, 16) || !aligned(c->v, 16) || !aligned(c->k_scale, 16) || !aligned(c->v_scale, 16))
        return MNB_ERR_ALIGN;
    return c->reserved == 0 ? MNB_OK : MNB_ERR_INVALID;
}

Cache8 cache8_of(const mnb_kv_cache_i8 *c) {
    Cache8 to{};
    to.k = c->k;
    to.v = c->v;
    to.k_scale = c->k_scale;
    to.v_scale = c->v_scale;
    to.num_blocks = c->num_blocks;
    to.block_stride = c->block_stride;
    to.head_stride = c->head_stride;
    to.token_stride = c->token_stride;
    to.scale_block = c->scale_block_stride;
    to.scale_head = c->scale_head_stride;
    to.heads = (int32_t)c->kv_heads;
    to.page = (int32_t)c->page_size;
    return to;
}

// T rows of `width` bytes, `stride` bytes apart.
struct Rows {
    const void *at;
    int64_t stride, width;
};

// The last of T rows is within 2^62 bytes of the first, so that addresses and
// ranges are counted in 64 bits.
bool within_reach(int64_t T, int64_t stride, int dtype) {
    return T < 2 || stride == 0 || T - 1 <= (1LL << 62) / (stride * dtype_bytes(dtype));
}

// Rows of one that overlap rows of the other (rows of different strides whose
// ranges meet count as overlapping).
bool rows_overlap(const Rows &a, const Rows &b, int64_t T) {
    if (!overlap(range(a.at, (T - 1) * a.stride + a.width), range(b.at, (T - 1) * b.stride + b.width))) return false;
    if (a.stride != b.stride || T == 1 || a.stride == 0) return true;
    const uintptr_t from = reinterpret_cast<uintptr_t>(a.at), to = reinterpret_cast<uintptr_t>(b.at);
    const int64_t s = a.stride, gap = to >= from ? (int64_t)((to - from) % (uintptr_t)s)
                                                 : (s - (int64_t)((from - to) % (uintptr_t)s)) % s;
    return gap < a.width || s - gap < b.width;   // (row b begins `gap` behind a row a)
}

// An output's rows lie apart from one another.
bool rows_apart(const Rows &a, int64_t T) { return T == 1 || a.stride >= a.width; }

// Keys and values [T][kv_heads][head_dim] beside the cache.
int check_token_rows(const void *k, const void *v, int64_t k_stride, int64_t v_stride, const int64_t *slots,
                     int64_t T, const mnb_kv_cache_i8 *cache) {
    if (int st = check_cache8(cache)) return st;
    if (T < 0 || T > MNB_MAX_ROWS) return MNB_ERR_SHAPE;
    if (int st = check_strides(k_stride, v_stride, 0, cache->dtype)) return st;
    if (!within_reach(T, k_stride, cache->dtype) || !within_reach(T, v_stride, cache->dtype)) return MNB_ERR_SHAPE;
    // (a token's elements are counted in 32 bits)
    if (cache->kv_heads > kIntMax / (cache->head_dim * 16)) return MNB_ERR_SHAPE;
    if (T == 0) return MNB_OK;
    if (!k || !v || !slots) return MNB_ERR_NULL;
    return aligned(k, 16) && aligned(v, 16) && aligned(slots, 8) ? MNB_OK : MNB_ERR_ALIGN;
}

Kv8Args token_args(const void *k, const void *v, int64_t k_stride, int64_t v_stride, const int64_t *slots, int64_t T,
                   const mnb_kv_cache_i8 *cache) {
    const int64_t es = dtype_bytes(cache->dtype);
    Kv8Args a{};
    a.cache = cache8_of(cache);
    a.k = static_cast<const uint8_t *>(k);
    a.v = static_cast<const uint8_t *>(v);
    a.k_stride = k_stride * es;
    a.v_stride = v_stride * es;
    a.slots = slots;
    a.tokens = T;
    return a;
}

// Sizes of an attention call.
int check_sizes(int64_t B, int64_t Hq, int64_t Hkv, int64_t head_dim, int64_t max_len, int64_t max_new, int dtype) {
    if (!known_dtype(dtype)) return MNB_ERR_DTYPE;
    if (head_dim != 64 && head_dim != 128) return MNB_ERR_SHAPE;
    if (B < 0 || B > MNB_MAX_REQUESTS || max_len < 0 || max_len > MNB_MAX_KEYS || max_new < 1 ||
        max_new > MNB_MAX_KEYS)
        return MNB_ERR_SHAPE;
    if (Hq < 1 || Hkv < 1 || Hq > kIntMax || Hkv > Hq || Hq % Hkv != 0) return MNB_ERR_SHAPE;
    if (max_new > kIntMax / (Hq / Hkv) || B * Hkv > kIntMax || Hq > kIntMax / head_dim) return MNB_ERR_SHAPE;
    return attn8_fits(B, Hkv, Hq / Hkv, max_new, max_len, (int)head_dim, dtype) ? MNB_OK : MNB_ERR_SHAPE;
}

}  // namespace

extern "C" {

int mnb_rope(const void *q, int64_t q_stride, void *q_out, int64_t q_out_stride, int64_t q_heads, const void *k,
             int64_t k_stride, void *k_out, int64_t k_out_stride, int64_t k_heads, const int32_t *positions,
             const double *freqs, int64_t T, int64_t head_dim, int64_t rot_dim, int layout, float gain, int dtype,
             void *stream) {
    if (!known_dtype(dtype)) return MNB_ERR_DTYPE;
    const int64_t es = dtype_bytes(dtype), most = kIntMax / 4096;   // (a token's bytes are counted in 32 bits)
    if (T < 0 || T > MNB_MAX_ROWS || q_heads < 0 || q_heads > most || k_heads < 0 || k_heads > most ||
        head_dim < 1 || head_dim > 1024 || head_dim * es % 16 || rot_dim < 2 || rot_dim > head_dim || rot_dim % 2)
        return MNB_ERR_SHAPE;
    if (int st = check_strides(q_heads ? q_stride : 0, q_heads ? q_out_stride : 0, 0, dtype)) return st;
    if (int st = check_strides(k_heads ? k_stride : 0, k_heads ? k_out_stride : 0, 0, dtype)) return st;
    if ((q_heads && (!within_reach(T, q_stride, dtype) || !within_reach(T, q_out_stride, dtype))) ||
        (k_heads && (!within_reach(T, k_stride, dtype) || !within_reach(T, k_out_stride, dtype))))
        return MNB_ERR_SHAPE;
    if ((layout != MNB_ROPE_HALF && layout != MNB_ROPE_INTERLEAVED) || !isfinite(gain)) return MNB_ERR_INVALID;
    if (T == 0 || q_heads + k_heads == 0) return MNB_OK;
    if ((q_heads && (!q || !q_out)) || (k_heads && (!k || !k_out)) || !positions || !freqs) return MNB_ERR_NULL;
    if ((q_heads && (!aligned(q, 16) || !aligned(q_out, 16))) || (k_heads && (!aligned(k, 16) || !aligned(k_out, 16))) ||
        !aligned(positions, 4) || !aligned(freqs, 8))
        return MNB_ERR_ALIGN;
    const int64_t row = head_dim * es;
    const Rows in[2] = {{q, q_stride * es, q_heads * row}, {k, k_stride * es, k_heads * row}};
    const Rows out[2] = {{q_out, q_out_stride * es, q_heads * row}, {k_out, k_out_stride * es, k_heads * row}};
    for (int o = 0; o < 2; ++o) {
        if (out[o].width == 0) continue;
        if (!rows_apart(out[o], T)) return MNB_ERR_INVALID;
        for (int i = 0; i < 2; ++i) {
            if (in[i].width == 0) continue;
            const bool self = i == o && in[i].at == out[o].at && (T == 1 || in[i].stride == out[o].stride);
            if (!self && rows_overlap(in[i], out[o], T)) return MNB_ERR_INVALID;
        }
    }
    if (out[0].width && out[1].width && rows_overlap(out[0], out[1], T)) return MNB_ERR_INVALID;
    RopeArgs a{};
    a.q = static_cast<const uint8_t *>(q);
    a.k = static_cast<const uint8_t *>(k);
    a.q_out = static_cast<uint8_t *>(q_out);
    a.k_out = static_cast<uint8_t *>(k_out);
    a.q_stride = in[0].stride;
    a.k_stride = in[1].stride;
    a.q_out_stride = out[0].stride;
    a.k_out_stride = out[1].stride;
    a.positions = positions;
    a.freqs = freqs;
    a.tokens = T;
    a.q_heads = (int32_t)q_heads;
    a.k_heads = (int32_t)k_heads;
    a.head_dim = (int32_t)head_dim;
    a.rot_dim = (int32_t)rot_dim;
    a.gain = gain;
    return hip_status(launch_rope(a, layout == MNB_ROPE_INTERLEAVED, dtype, static_cast<hipStream_t>(stream)));
}

int mnb_kv_append_i8(const void *k, const void *v, int64_t k_stride, int64_t v_stride, const int64_t *slots,
                     int64_t T, const mnb_kv_cache_i8 *cache, void *stream) {
    if (int st = check_token_rows(k, v, k_stride, v_stride, slots, T, cache)) return st;
    if (T == 0) return MNB_OK;
    return hip_status(launch_kv8_append(token_args(k, v, k_stride, v_stride, slots, T, cache), (int)cache->head_dim,
                                        cache->dtype, static_cast<hipStream_t>(stream)));
}

int mnb_kv_read_i8(const int64_t *slots, int64_t T, const mnb_kv_cache_i8 *cache, void *k, void *v, int64_t k_stride,
                   int64_t v_stride, void *stream) {
    if (int st = check_token_rows(k, v, k_stride, v_stride, slots, T, cache)) return st;
    if (T == 0) return MNB_OK;
    const int64_t es = dtype_bytes(cache->dtype), width = cache->kv_heads * cache->head_dim * es;
    const Rows to[2] = {{k, k_stride * es, width}, {v, v_stride * es, width}};
    if (!rows_apart(to[0], T) || !rows_apart(to[1], T) || rows_overlap(to[0], to[1], T)) return MNB_ERR_INVALID;
    return hip_status(launch_kv8_read(token_args(k, v, k_stride, v_stride, slots, T, cache), (int)cache->head_dim,
                                      cache->dtype, static_cast<hipStream_t>(stream)));
}

size_t mnb_paged_attn_i8_workspace_bytes(int64_t B, int64_t Hq, int64_t Hkv, int64_t head_dim, int64_t max_len,
                                         int64_t max_new, int dtype) {
    if (check_sizes(B, Hq, Hkv, head_dim, max_len, max_new, dtype) != MNB_OK || B == 0) return 0;
    return (size_t)attn8_workspace_bytes(B, Hkv, Hq / Hkv, max_new, max_len, (int)head_dim, dtype);
}

int mnb_paged_attn_i8(const void *q, int64_t q_stride, const mnb_kv_cache_i8 *cache, const int32_t *block_table,
                      const int32_t *lens, const int32_t *starts, int64_t T, int64_t B, int64_t Hq,
                      int64_t max_blocks, int64_t max_len, int64_t max_new, float scale, void *workspace,
                      size_t workspace_bytes, void *out, void *stream) {
    if (int st = check_cache8(cache)) return st;
    if (int st = check_sizes(B, Hq, cache->kv_heads, cache->head_dim, max_len, max_new, cache->dtype)) return st;
    if (T < 0 || T > kIntMax || max_blocks < 1 || max_blocks > kIntMax / (B > 0 ? B : 1)) return MNB_ERR_SHAPE;
    if (!starts && (T != B || max_new != 1)) return MNB_ERR_SHAPE;
    if (int st = check_strides(q_stride, 0, 0, cache->dtype)) return st;
    if (!within_reach(T, q_stride, cache->dtype)) return MNB_ERR_SHAPE;
    if (!isfinite(scale)) return MNB_ERR_INVALID;
    if (B == 0 || T == 0) return MNB_OK;
    if (!q || !block_table || !lens || !out) return MNB_ERR_NULL;
    if (!aligned(q, 16) || !aligned(out, 16) || !aligned(block_table, 4) || !aligned(lens, 4) || !aligned(starts, 4))
        return MNB_ERR_ALIGN;
    const int head_dim = (int)cache->head_dim;
    const int64_t row = Hq * head_dim * dtype_bytes(cache->dtype);
    if (overlap(range(q, (T - 1) * q_stride * dtype_bytes(cache->dtype) + row), range(out, T * row)))
        return MNB_ERR_INVALID;
    const int64_t group = Hq / cache->kv_heads;
    const int64_t need = attn8_workspace_bytes(B, cache->kv_heads, group, max_new, max_len, head_dim, cache->dtype);
    if (int st = check_workspace(need, workspace, workspace_bytes)) return st;
    Attn8Args a{};
    a.cache = cache8_of(cache);
    a.q = q;
    a.out = out;
    a.table = block_table;
    a.lens = lens;
    a.starts = starts;
    a.q_stride = q_stride;
    a.tokens = T;
    a.batch = (int32_t)B;
    a.group = (int32_t)group;
    a.max_new = (int32_t)max_new;
    a.max_len = (int32_t)max_len;
    a.table_width = (int32_t)max_blocks;
    a.scale = kernel_scale(scale, cache->dtype);
    return hip_status(launch_attn8(a, head_dim, cache->dtype, workspace, static_cast<hipStream_t>(stream)));
}

}  // extern "C"
