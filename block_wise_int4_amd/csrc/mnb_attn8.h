// What the two kernels of the attention over the 8-bit cache share: which keys a
// row sees, where its results go, and how a launch over many keys is cut.
#pragma once
#include "mnb_cache8.h"
#include "mnb_device.h"

namespace mnb {

constexpr float kLowest = -3.402823466e38f;   // the maximum before any key
constexpr float kLog2e = 1.4426950408889634f;

typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));

__device__ __forceinline__ float as_float(uint32_t x) { return __builtin_bit_cast(float, x); }
__device__ __forceinline__ uint32_t as_bits(float x) { return __builtin_bit_cast(uint32_t, x); }

// New tokens of request b, and its first row of q.
__device__ __forceinline__ int rows_of(const Attn8Args &a, int64_t b, int64_t &first) {
    first = b;
    if (!a.starts) return 1;
    typedef __attribute__((address_space(4))) const int32_t entry;   // (a scalar load)
    int64_t from = ((entry *)a.starts)[b], to = ((entry *)a.starts)[b + 1];
    from = from < 0 ? 0 : from > a.tokens ? a.tokens : from;
    to = to < from ? from : to > a.tokens ? a.tokens : to;
    first = from;
    return (int)(to - from);
}

// Keys that new token i of n of request b sees.
__device__ __forceinline__ int sees(const Attn8Args &a, int len, int n, int i) {
    const int64_t s = (int64_t)len - n + i + 1;
    return s < 0 ? 0 : s < a.max_len ? (int)s : a.max_len;
}

// Blocks before a part of 16 keys.
__device__ __forceinline__ uint32_t blocks_before(uint32_t part, uint32_t magic) {
    const uint32_t place = __umulhi(part, magic);
    return magic ? place : part;
}

// Token of row r (< 2^24) of a (request, key-value head): r / group, by a reciprocal
// that is off by at most one.
__device__ __forceinline__ int token_of(const Attn8Args &a, int r) {
    int t = (int)((float)r * a.per_group);
    const int rest = r - t * a.group;
    t += rest >= a.group ? 1 : 0;
    return rest < 0 ? t - 1 : t;
}

// Four outputs from dimension d on of row r.
template <typename T, int D>
__device__ __forceinline__ void store_out(const Attn8Args &a, int64_t first, int h, int r, int d, f4 sum, float total) {
    const int token = token_of(a, r);
    T *out = static_cast<T *>(a.out) +
             ((first + token) * ((int64_t)a.cache.heads * a.group) + (int64_t)h * a.group + r - token * a.group) * D + d;
    if (total == 0.0f) sum = f4{0.0f, 0.0f, 0.0f, 0.0f};
    else sum *= 1.0f / total;
    if constexpr (sizeof(T) == 2) {
        const u32x2 w = {as_u32(h2{(_Float16)sum.x, (_Float16)sum.y}), as_u32(h2{(_Float16)sum.z, (_Float16)sum.w})};
        *reinterpret_cast<u32x2 *>(out) = w;
    } else {
        *reinterpret_cast<f4 *>(out) = sum;
    }
}

// How a launch is cut. Pieces of rows of more than one chunk: per (request,
// head, query row, chunk) D sums, and a maximum and the weights' sum.
struct Attn8Split {
    int32_t chunk;        // keys per chunk
    int32_t chunks;       // of max_len
    int32_t rows;         // bound of the rows per (request, head)
    int32_t q_tiles, tile;   // tiles of rows, and rows in each
    uint32_t page_magic;  // ceil(2^32 / (page / 16)), 0 for pages of 16: part * magic >> 32 is
                          // part / (page / 16) for part < 2^26
    float *sums, *stats;
};

// The same sums for up to kFewRows query rows of a (request, key-value head)
// (mnb_attn8_few.hip).
constexpr int kFewRows = 2;
hipError_t launch_attn8_few(const Attn8Args &a, const Attn8Split &sp, int head_dim, int dtype, bool stream,
                            hipStream_t st);

// The same sums for float16 calls with many query rows (mnb_attn8_rows.hip), tiles of
// kRowTile rows.
constexpr int kRowTile = 128;
hipError_t launch_attn8_rows(const Attn8Args &a, const Attn8Split &sp, int head_dim, hipStream_t st);

}  // namespace mnb
