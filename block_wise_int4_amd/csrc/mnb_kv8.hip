// The 8-bit key-value cache: tokens quantized as they are written, and slots
// read back as the numbers they stand for. 26240 float16 tokens of 8 x 128 (164 MB
// either way), appended and read back, three sets of tensors in turn: 44..46 us on the
// device, 3.6 TB/s, and 28, 5.9 TB/s, codes mostly from the last-level cache. Appends
// alone take 41, of the same tokens again and again, which that cache holds, 37: about what
// the vector instructions take (850 a wave for 16 rows of 128, half of them a row's place
// and scale, the rest conversions and exact quotients: 88 thousand cycles a SIMD). 13120
// float32 tokens (135 MB) alone: 33 and, read back, 32. 8 tokens take 3.1 and 2.6, a launch.
#include "mnb_cache8.h"
#include "mnb_device.h"

namespace mnb {

namespace {

typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));

constexpr int kThreads = 256;
constexpr int kPart = 8;    // elements of a row per lane (append)
constexpr int kAhead = 4;   // rows a lane has under way

// Largest scale s with 127 s within float32.
constexpr float kMostScale = 0x1.020406p+121f;

// A slot's place: block, and offset within its page; false outside the cache.
__device__ __forceinline__ bool place_of(const Kv8Args &a, int64_t slot, int64_t &block, int &offset) {
    if (slot < 0) return false;
    // (slots of most caches are below 2^30, where a product gives the quotient: pages are
    // multiples of 16)
    const uint64_t part = (uint64_t)slot >> 4;
    if (part >> 26) block = (int64_t)(part / ((uint32_t)a.cache.page >> 4));
    else block = a.page_magic ? __umulhi((uint32_t)part, a.page_magic) : (uint32_t)part;
    offset = (int)(slot - block * a.cache.page);
    return block < a.cache.num_blocks;
}

// Which row of a workgroup's tokens: token, keys or values, head. r < 2^24, by a
// reciprocal that is off by at most one.
struct Row {
    int64_t token;
    int head;
    bool second, on;
};
__device__ __forceinline__ Row row_of(const Kv8Args &a, int64_t t0, int r, int rows, float per_each) {
    const int each = 2 * a.cache.heads;
    int which = (int)((float)r * per_each);
    const int rest = r - which * each;
    which += rest >= each ? 1 : 0;
    which -= rest < 0 ? 1 : 0;
    int of = r - which * each;
    Row x;
    x.token = t0 + which;
    x.second = of >= a.cache.heads;
    x.head = x.second ? of - a.cache.heads : of;
    x.on = r < rows && x.token < a.tokens;
    return x;
}

// Eight elements of a row.
template <typename T> struct Eight {
    u32x4 w[sizeof(T) == 2 ? 1 : 2];
    __device__ __forceinline__ void load(const uint8_t *from) {
#pragma unroll
        for (int j = 0; j < (sizeof(T) == 2 ? 1 : 2); ++j) w[j] = reinterpret_cast<const u32x4 *>(from)[j];
    }
    __device__ __forceinline__ void as_floats(float *x) const {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if constexpr (sizeof(T) == 2) x[i] = (float)__builtin_bit_cast(h8, w[0])[i];
            else x[i] = __builtin_bit_cast(f4, w[i / 4])[i % 4];
    }
};

template <int N> __device__ __forceinline__ uint32_t turned(uint32_t x) {   // by N of 16 lanes
    return (uint32_t)__builtin_amdgcn_update_dpp((int)x, (int)x, 0x120 + N, 0xF, 0xF, false);
}
__device__ __forceinline__ uint32_t larger(uint32_t x, uint32_t y) { return x > y ? x : y; }

// x / s to the nearest whole number, ties to even, of c within one step of it: the
// remainder (exact: it is a multiple of the smaller operand's last place and below
// 2 s) says where the border lies.
__device__ __forceinline__ float nearest(float c, float x, float s) {
    const float twice = 2.0f * __builtin_fmaf(-c, s, x);
    const bool odd = (int)c & 1;
    if (twice > s || (twice == s && odd)) c += 1.0f;
    else if (twice < -s || (twice == -s && odd)) c -= 1.0f;
    return c;
}

}  // namespace

// A row of D elements is D / 8 lanes; a workgroup takes `per` tokens, keys and values of
// all heads, kAhead rows a lane at a time: a row's load waits for nothing, its slot
// is needed only to store it. A code is x (1 / s) rounded by adding 1.5 * 2^23; only where
// the remainder of one of a lane's eight comes within 2^-12 of half a step can the
// reciprocal's rounding matter, and these are put right exactly.
template <typename T, int D>
__global__ __launch_bounds__(kThreads) void kv8_append_kernel(Kv8Args a, int per, float per_each) {
    constexpr int kLanes = D / kPart, kRows = kThreads / kLanes;
    constexpr float kRound = 12582912.0f;
    const int lane = threadIdx.x % kLanes, rows = per * 2 * a.cache.heads;
    for (int64_t t0 = (int64_t)blockIdx.x * per; t0 < a.tokens; t0 += (int64_t)gridDim.x * per)
        for (int r0 = threadIdx.x / kLanes; r0 < rows; r0 += kRows * kAhead) {
            Row row[kAhead];
            Eight<T> in[kAhead];
            int64_t slot[kAhead];
#pragma unroll
            for (int u = 0; u < kAhead; ++u) {
                row[u] = row_of(a, t0, r0 + u * kRows, rows, per_each);
                slot[u] = -1;
                if (row[u].on) {
                    slot[u] = a.slots[row[u].token];
                    in[u].load((row[u].second ? a.v + row[u].token * a.v_stride : a.k + row[u].token * a.k_stride) +
                               ((int64_t)row[u].head * D + lane * kPart) * (int64_t)sizeof(T));
                }
            }
#pragma unroll
            for (int u = 0; u < kAhead; ++u) {
                int64_t block;
                int offset;
                if (!place_of(a, slot[u], block, offset)) continue;   // (a row's lanes together)
                float x[kPart];
                in[u].as_floats(x);
                // (as whole numbers: infinities and NaN are above every finite one)
                uint32_t top = 0;
#pragma unroll
                for (int i = 0; i < kPart; ++i) top = larger(top, __builtin_bit_cast(uint32_t, x[i]) & 0x7FFFFFFFu);
                if constexpr (kLanes == 16) {
                    top = larger(top, turned<8>(top));
                    top = larger(top, turned<4>(top));
                    top = larger(top, turned<2>(top));
                    top = larger(top, turned<1>(top));
                } else {   // 8 lanes: the other half row's are another row's
#pragma unroll
                    for (int d = 1; d < kLanes; d <<= 1) top = larger(top, (uint32_t)__shfl_xor((int)top, d));
                }
                const bool finite = top < 0x7F800000u;
                const float s = fminf(__builtin_bit_cast(float, top) / 127.0f, kMostScale);
                uint32_t w[2] = {0, 0};
                if (finite && s > 0.0f) {
                    // (the smallest rows 2^64 times as large, which float16 has none of)
                    const float lift = sizeof(T) == 4 && s < 0x1p-60f ? 0x1p64f : 1.0f, step = s * lift;
                    const float by = __builtin_amdgcn_rcpf(step), close = step * (0.5f - 0x1p-12f);
                    float c[kPart], far = 0.0f;
#pragma unroll
                    for (int i = 0; i < kPart; ++i) {
                        if constexpr (sizeof(T) == 4) x[i] *= lift;
                        c[i] = __builtin_fmaf(x[i], by, kRound) - kRound;
                        far = fmaxf(far, __builtin_fabsf(__builtin_fmaf(-c[i], step, x[i])));
                    }
                    if (far >= close)
#pragma unroll
                        for (int i = 0; i < kPart; ++i) c[i] = nearest(c[i], x[i], step);
                    // (a scale below the normal range may be so much too small that 127 is not enough)
#pragma unroll
                    for (int i = 0; i < kPart; i += 4) {
                        uint32_t b[4];
#pragma unroll
                        for (int j = 0; j < 4; ++j) {
                            float code = c[i + j];
                            if constexpr (sizeof(T) == 4) code = fminf(fmaxf(code, -127.0f), 127.0f);
                            b[j] = __builtin_bit_cast(uint32_t, code + kRound);
                        }
                        w[i / 4] = __builtin_amdgcn_perm(__builtin_amdgcn_perm(b[3], b[2], 0x0C0C0400u),
                                                         __builtin_amdgcn_perm(b[1], b[0], 0x0C0C0400u), 0x05040100u);
                    }
                }
                int8_t *to = (row[u].second ? a.cache.v : a.cache.k) + block * a.cache.block_stride +
                             row[u].head * a.cache.head_stride + offset * a.cache.token_stride + lane * kPart;
                *reinterpret_cast<u32x2 *>(to) = u32x2{w[0], w[1]};
                if (lane == 0)
                    (row[u].second ? a.cache.v_scale
                                   : a.cache.k_scale)[block * a.cache.scale_block + row[u].head * a.cache.scale_head +
                                                      offset] = finite ? s : __builtin_nanf("");
            }
        }
}

// Two codes times s, each exact product rounded once to float16, which the mixed multiply-
// add does (a float32 product and its conversion would round twice).
__device__ __forceinline__ uint32_t half_pair(float c0, float c1, float s) {
    uint32_t y;
    asm("v_fma_mixlo_f16 %0, %1, %2, 0" : "=v"(y) : "v"(c0), "v"(s));
    asm("v_fma_mixhi_f16 %0, %1, %2, 0" : "+v"(y) : "v"(c1), "v"(s));
    return y;
}

// 16 bytes of output a lane, kAhead rows at a time.
template <typename T, int D>
__global__ __launch_bounds__(kThreads) void kv8_read_kernel(Kv8Args a, int per, float per_each) {
    constexpr int kOut = 16 / (int)sizeof(T), kLanes = D / kOut, kRows = kThreads / kLanes;
    const int lane = threadIdx.x % kLanes, rows = per * 2 * a.cache.heads;
    for (int64_t t0 = (int64_t)blockIdx.x * per; t0 < a.tokens; t0 += (int64_t)gridDim.x * per)
        for (int r0 = threadIdx.x / kLanes; r0 < rows; r0 += kRows * kAhead) {
            Row row[kAhead];
            int64_t slot[kAhead];
            uint32_t w[kAhead][kOut / 4];
            float s[kAhead];
#pragma unroll
            for (int u = 0; u < kAhead; ++u) {
                row[u] = row_of(a, t0, r0 + u * kRows, rows, per_each);
                slot[u] = row[u].on ? a.slots[row[u].token] : -1;
            }
#pragma unroll
            for (int u = 0; u < kAhead; ++u) {
                int64_t block;
                int offset;
                s[u] = 0.0f;
#pragma unroll
                for (int i = 0; i < kOut / 4; ++i) w[u][i] = 0;
                if (!place_of(a, slot[u], block, offset)) continue;
                const int8_t *from = (row[u].second ? a.cache.v : a.cache.k) + block * a.cache.block_stride +
                                     row[u].head * a.cache.head_stride + offset * a.cache.token_stride + lane * kOut;
                if constexpr (kOut == 8) {
                    const u32x2 both = *reinterpret_cast<const u32x2 *>(from);
                    w[u][0] = both.x;
                    w[u][1] = both.y;
                } else {
                    w[u][0] = *reinterpret_cast<const uint32_t *>(from);
                }
                s[u] = (row[u].second ? a.cache.v_scale
                                      : a.cache.k_scale)[block * a.cache.scale_block +
                                                         row[u].head * a.cache.scale_head + offset];
            }
#pragma unroll
            for (int u = 0; u < kAhead; ++u) {
                if (!row[u].on) continue;
                u32x4 y;
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const uint32_t b = w[u][i * kOut / 16];
                    auto code = [&](int at) { return (float)(int8_t)(b >> at); };
                    if constexpr (sizeof(T) == 2) y[i] = half_pair(code(16 * (i & 1)), code(16 * (i & 1) + 8), s[u]);
                    else y[i] = __builtin_bit_cast(uint32_t, code(8 * i) * s[u]);
                }
                uint8_t *to = const_cast<uint8_t *>(row[u].second ? a.v + row[u].token * a.v_stride
                                                                  : a.k + row[u].token * a.k_stride) +
                              ((int64_t)row[u].head * D + lane * kOut) * (int64_t)sizeof(T);
                *reinterpret_cast<u32x4 *>(to) = y;
            }
        }
}

namespace {

// Tokens per workgroup: rows for its lanes, kAhead times where 1024 workgroups are left
// by that. The same float16 tokens of 8 x 128 again, with and without, us replayed from a
// graph: 4096 appended 9.6 and 10.1, read back 7.5 and 8.6, 26240 35.4..36.6 and 41.4, 27.1
// and 34.4; but 1024 6.3 and 4.7, 4.4 and 4.4.
template <typename T, int D, bool APPEND> hipError_t launch(const Kv8Args &a, hipStream_t st) {
    constexpr int lanes = APPEND ? D / kPart : D * (int)sizeof(T) / 16, rows = kThreads / lanes;
    const int64_t each = 2 * (int64_t)a.cache.heads;
    int64_t per = each < rows ? rows / each : 1;
    const int64_t more = each < rows * kAhead ? rows * kAhead / each : 1;
    if (more > per && a.tokens >= 1024 * more) per = more;
    const int64_t wgs = (a.tokens + per - 1) / per;
    const unsigned grid = (unsigned)(wgs < 65536 ? wgs : 65536);
    const float per_each = 1.0f / (float)each;
    Kv8Args c = a;
    const uint32_t parts = (uint32_t)a.cache.page / 16;
    c.page_magic = parts == 1 ? 0 : (uint32_t)(((1ull << 32) + parts - 1) / parts);
    if constexpr (APPEND) kv8_append_kernel<T, D><<<grid, kThreads, 0, st>>>(c, (int)per, per_each);
    else kv8_read_kernel<T, D><<<grid, kThreads, 0, st>>>(c, (int)per, per_each);
    return hipGetLastError();
}

template <bool APPEND> hipError_t launch_as(const Kv8Args &a, int head_dim, int dtype, hipStream_t st) {
    if (dtype == 1)
        return head_dim == 128 ? launch<_Float16, 128, APPEND>(a, st) : launch<_Float16, 64, APPEND>(a, st);
    return head_dim == 128 ? launch<float, 128, APPEND>(a, st) : launch<float, 64, APPEND>(a, st);
}

}  // namespace

hipError_t launch_kv8_append(const Kv8Args &a, int head_dim, int dtype, hipStream_t st) {
    return launch_as<true>(a, head_dim, dtype, st);
}

hipError_t launch_kv8_read(const Kv8Args &a, int head_dim, int dtype, hipStream_t st) {
    return launch_as<false>(a, head_dim, dtype, st);
}

}  // namespace mnb
