// The 8-bit key-value cache: tokens quantized as they are written, and slots
// read back as the numbers they stand for.
#include "mnb_cache8.h"
#include "mnb_device.h"

namespace mnb {

namespace {

typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));

constexpr int kThreads = 256;
constexpr int kPart = 8;   // elements of a row per lane

// Largest scale s with 127 s within float32.
constexpr float kMostScale = 0x1.020406p+121f;

// A slot's place: block, and offset within its page; false outside the cache.
__device__ __forceinline__ bool place_of(const Cache8 &c, int64_t slot, int64_t &block, int &offset) {
    if (slot < 0) return false;
    // (pages are multiples of 16; slots of most caches fit 32 bits, and 64-bit
    // divisions are slow)
    const uint64_t part = (uint64_t)slot >> 4;
    const uint32_t parts = (uint32_t)c.page >> 4;
    block = part >> 32 ? (int64_t)(part / parts) : (int64_t)((uint32_t)part / parts);
    offset = (int)(slot - block * c.page);
    return block < c.num_blocks;
}

// Eight elements of a row as float32.
template <typename T> __device__ __forceinline__ void load8(const uint8_t *from, float *x) {
    if constexpr (sizeof(T) == 2) {
        const h8 w = *reinterpret_cast<const h8 *>(from);
#pragma unroll
        for (int i = 0; i < 8; ++i) x[i] = (float)w[i];
    } else {
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            const f4 w = reinterpret_cast<const f4 *>(from)[j];
#pragma unroll
            for (int i = 0; i < 4; ++i) x[4 * j + i] = w[i];
        }
    }
}

// x / s to the nearest whole number, ties to even: the float32 quotient is within
// one step of it, and the remainder (exact: it is a multiple of the smaller
// operand's last place and at most s) says where the border lies.
__device__ __forceinline__ int code_of(float x, float s) {
    float c = __builtin_rintf(x / s);
    const float twice = 2.0f * __builtin_fmaf(-c, s, x);
    const bool odd = (int)c & 1;
    if (twice > s || (twice == s && odd)) c += 1.0f;
    else if (twice < -s || (twice == -s && odd)) c -= 1.0f;
    return (int)fminf(fmaxf(c, -127.0f), 127.0f);
}

}  // namespace

// A row of D elements is D / 8 lanes; workgroups take `per` tokens, keys and
// values of all heads.
template <typename T, int D>
__global__ __launch_bounds__(kThreads) void kv8_append_kernel(Kv8Args a, int per) {
    constexpr int kLanes = D / kPart, kRows = kThreads / kLanes;
    const int lane = threadIdx.x % kLanes, heads = a.cache.heads, rows = per * 2 * heads;
    for (int64_t t0 = (int64_t)blockIdx.x * per; t0 < a.tokens; t0 += (int64_t)gridDim.x * per) {
        for (int r = threadIdx.x / kLanes; r < rows; r += kRows) {
            const int which = r / (2 * heads), of = r - which * 2 * heads;
            const int64_t t = t0 + which;
            if (t >= a.tokens) break;
            int64_t block;
            int offset;
            if (!place_of(a.cache, a.slots[t], block, offset)) continue;
            const bool second = of >= heads;
            const int h = second ? of - heads : of;
            const uint8_t *from = (second ? a.v + t * a.v_stride : a.k + t * a.k_stride) +
                                  ((int64_t)h * D + lane * kPart) * (int64_t)sizeof(T);
            float x[kPart];
            load8<T>(from, x);
            // (as whole numbers: infinities and NaN are above every finite one)
            uint32_t top = 0;
#pragma unroll
            for (int i = 0; i < kPart; ++i) {
                const uint32_t bits = __builtin_bit_cast(uint32_t, x[i]) & 0x7FFFFFFFu;
                top = bits > top ? bits : top;
            }
#pragma unroll
            for (int d = 1; d < kLanes; d <<= 1) {
                const uint32_t other = (uint32_t)__shfl_xor((int)top, d);
                top = other > top ? other : top;
            }
            const bool finite = top < 0x7F800000u;
            const float s = fminf(__builtin_bit_cast(float, top) / 127.0f, kMostScale);
            uint32_t w[2] = {0, 0};
            if (finite && s > 0.0f) {
#pragma unroll
                for (int i = 0; i < kPart; ++i) w[i / 4] |= (uint32_t)(code_of(x[i], s) & 0xFF) << (8 * (i % 4));
            }
            int8_t *to = (second ? a.cache.v : a.cache.k) + block * a.cache.block_stride + h * a.cache.head_stride +
                         offset * a.cache.token_stride + lane * kPart;
            *reinterpret_cast<u32x2 *>(to) = u32x2{w[0], w[1]};
            if (lane == 0)
                (second ? a.cache.v_scale : a.cache.k_scale)[block * a.cache.scale_block + h * a.cache.scale_head +
                                                             offset] = finite ? s : __builtin_nanf("");
        }
    }
}

// 16 bytes of output a lane.
template <typename T, int D>
__global__ __launch_bounds__(kThreads) void kv8_read_kernel(Kv8Args a, int per) {
    constexpr int kOut = 16 / (int)sizeof(T), kLanes = D / kOut, kRows = kThreads / kLanes;
    const int lane = threadIdx.x % kLanes, heads = a.cache.heads, rows = per * 2 * heads;
    for (int64_t t0 = (int64_t)blockIdx.x * per; t0 < a.tokens; t0 += (int64_t)gridDim.x * per) {
        for (int r = threadIdx.x / kLanes; r < rows; r += kRows) {
            const int which = r / (2 * heads), of = r - which * 2 * heads;
            const int64_t t = t0 + which;
            if (t >= a.tokens) break;
            const bool second = of >= heads;
            const int h = second ? of - heads : of;
            int64_t block;
            int offset;
            uint32_t w[kOut / 4] = {};
            float s = 0.0f;
            if (place_of(a.cache, a.slots[t], block, offset)) {
                const int8_t *from = (second ? a.cache.v : a.cache.k) + block * a.cache.block_stride +
                                     h * a.cache.head_stride + offset * a.cache.token_stride + lane * kOut;
#pragma unroll
                for (int i = 0; i < kOut / 4; ++i) w[i] = reinterpret_cast<const uint32_t *>(from)[i];
                s = (second ? a.cache.v_scale : a.cache.k_scale)[block * a.cache.scale_block + h * a.cache.scale_head +
                                                                 offset];
            }
            T y[kOut];
#pragma unroll
            for (int i = 0; i < kOut; ++i) {
                const float c = (float)(int8_t)(w[i / 4] >> (8 * (i % 4)));
                if constexpr (sizeof(T) == 4) y[i] = c * s;
                else y[i] = (T)mul_round_odd(c, s);
            }
            uint8_t *to = const_cast<uint8_t *>(second ? a.v + t * a.v_stride : a.k + t * a.k_stride) +
                          ((int64_t)h * D + lane * kOut) * (int64_t)sizeof(T);
            *reinterpret_cast<u32x4 *>(to) = *reinterpret_cast<const u32x4 *>(y);
        }
    }
}

namespace {

// Tokens per workgroup: enough rows for its lanes.
template <typename T, int D, bool APPEND> hipError_t launch(const Kv8Args &a, hipStream_t st) {
    constexpr int lanes = APPEND ? D / kPart : D * (int)sizeof(T) / 16, rows = kThreads / lanes;
    const int64_t each = 2 * (int64_t)a.cache.heads;
    const int per = each < rows ? (int)(rows / each) : 1;
    const int64_t wgs = (a.tokens + per - 1) / per;
    const unsigned grid = (unsigned)(wgs < 65536 ? wgs : 65536);
    if constexpr (APPEND) kv8_append_kernel<T, D><<<grid, kThreads, 0, st>>>(a, per);
    else kv8_read_kernel<T, D><<<grid, kThreads, 0, st>>>(a, per);
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
