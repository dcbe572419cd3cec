// Attention of many query rows over one run of keys per request, float16:
// the same sums as mnb_attn.hip, for calls with enough rows to be bound by
// arithmetic (a text scored against its audio).
//
// A workgroup is four waves on the query rows of one (request, key-value
// head), 32 rows a wave, walking over the keys 32 at a time. Either all four
// have rows of their own (128 a workgroup), or, in smaller calls, two groups of
// two waves share 64 rows, one group on the even 32s of keys and one on the
// odd ones, and their sums are joined in LDS at the end: half the steps and
// twice the workgroups, but each reads all keys for half as many rows. Keys
// and values go from memory to LDS without passing registers (buffer loads to
// LDS, 16 bytes a lane), the next ones on their way while these are used; rows
// past the last valid key read as zeros by the buffer's range.
//   S^T = K Q^T   (32 x 32 x 16 products: a lane holds 16 keys' scores of one
//                 query per 32 keys)
//   O^T = V^T P^T takes P from those registers as they are: the contraction
//                 index is renumbered to the keys a lane holds, and V^T comes
//                 out of LDS through the transposing 8-byte reads.
// LDS rows are as the memory rows; their 16-byte pieces are permuted by a
// function of the row (`swizzle`), so that both kinds of read spread over the
// banks. (The counters still see conflicts in 31% of the LDS cycles of 8 x 448
// rows over 1500 keys; waves wait for LDS in 2% of theirs.)
// Sums that are not finite, or references past 2^20, send a wave over its keys a
// second time, with float32 weights: infinite values, infinite queries, and
// scores too large for the first pass's fused exponents.
// What bounds it: per 64 scores (one a lane) the two products take 16 cycles
// of the matrix unit at D = 64, 32 at D = 128, and the softmax (exponential 8,
// scale and subtract, maximum, sum, conversion) about 25 of the vector unit.
// They only overlap if a wave has both to issue, so the scores of the next 32
// keys are taken while these are turned into weights. Still they add up: 8 x 448
// rows over 811..1500 keys, 12 heads of 64, take 28 us on the device, some 59
// thousand cycles, of which a SIMD's matrix unit is busy 13 and its vector unit
// 23; neither is full.
#include "mnb_attn.h"
#include "mnb_device.h"

namespace mnb {

namespace {

constexpr int kCrossKeys = 32;    // keys per step of a group
constexpr float kRefLowest = -3.402823466e38f;
// The reference lies 2^7 below the running maximum and moves when a score passes
// that maximum by more than 2^8: weights reach 2^15, float16's range, and count
// down to 2^-32 of the maximum's.
constexpr float kLift = 7.0f, kSlack = 8.0f + kLift;

typedef float f2 __attribute__((ext_vector_type(2)));
typedef float f16v __attribute__((ext_vector_type(16)));
typedef _Float16 h4 __attribute__((ext_vector_type(4)));
typedef short s4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef __attribute__((address_space(3))) void lds_void;

__device__ __forceinline__ f16v mma32(h8 a, h8 b, f16v c) {
    return __builtin_amdgcn_mfma_f32_32x32x16_f16(a, b, c, 0, 0, 0);
}

__device__ __forceinline__ f16v mma2(float a, float b, f16v c) {
    return __builtin_amdgcn_mfma_f32_32x32x2f32(a, b, c, 0, 0, 0);
}

// Where 16-byte piece c of LDS row `row` is: c ^ swizzle(row). Sixteen rows
// (of one piece) and eight rows by two adjacent pairs of pieces (the two
// kinds of read) each touch all banks evenly.
template <int D> __device__ __forceinline__ int swizzle(int row) {
    if constexpr (D == 64) return ((row >> 1) & 3) << 1 | ((row >> 3) & 1);
    else return (row & 7) << 1 | ((row >> 3) & 1);
}

// The workgroup meets: this wave's loads into LDS have arrived, and its reads of
// LDS are over, so that the loads requested next, by any wave, may write where
// they read. (The compiler counts neither for loads to LDS.)
__device__ __forceinline__ void meet() {
    asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)\n\ts_barrier" ::: "memory");
}

}  // namespace

// R: waves with rows of their own; 4 / R groups of them.
template <int D, int R> __device__ __forceinline__ void cross_workgroup(const AttnArgs &a) {
    constexpr int kGroups = 4 / R;
    constexpr int kPieces = D / 8;                          // 16-byte pieces of a row
    constexpr int kLoads = kCrossKeys * kPieces / (64 * R);     // pieces per thread and tile
    constexpr int kTile = kCrossKeys * D;                   // elements
    // (an array of its own for each buffer, named in the code: the compiler then
    // knows that reads of one need not wait for loads into another)
    __shared__ __align__(1024) _Float16 s_k0[kGroups][kTile], s_k1[kGroups][kTile], s_v0[kGroups][kTile],
        s_v1[kGroups][kTile];
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane((threadIdx.x >> 6) % R);
    const int group = __builtin_amdgcn_readfirstlane((threadIdx.x >> 6) / R);
    const int col = lane & 31, half = lane >> 5;
    const int h = blockIdx.x;
    const int64_t b = blockIdx.z;
    int n = a.max_len;
    if (a.lens && a.lens[b] < n) n = a.lens[b];
    const int row = blockIdx.y * (32 * R) + wave * 32 + col;
    const bool on = row < a.rows;
    const int token = (int)((uint32_t)(on ? row : 0) / (uint32_t)a.group);
    const int64_t hq = (int64_t)h * a.group + (on ? row : 0) - (int64_t)token * a.group;

    // queries, their sign turned where the scale is negative, so that the
    // largest score is the largest product
    h8 q[D / 16];
    {
        const _Float16 *src = static_cast<const _Float16 *>(a.q) + b * a.q_batch + token * a.q_row + hq * a.q_head;
        const uint32_t flip = a.scale < 0.0f ? 0x80008000u : 0u;
#pragma unroll
        for (int j = 0; j < D / 16; ++j) {
            u32x4 w = *reinterpret_cast<const u32x4 *>(src + 16 * j + 8 * half);
            w ^= flip;
            q[j] = __builtin_bit_cast(h8, w);
        }
    }
    const float mul = __builtin_fabsf(a.scale) * 1.4426950408889634f;

    // this lane's pieces of a tile: LDS slot (t * R + wave) * 64 + lane
    const uint32_t k_row = (uint32_t)a.k_row * 2, v_row = (uint32_t)a.v_row * 2;
    uint32_t k_at[kLoads], v_at[kLoads];
#pragma unroll
    for (int t = 0; t < kLoads; ++t) {
        const int slot = (t * R + wave) * 64 + lane, r = slot / kPieces, c = (slot % kPieces) ^ swizzle<D>(r);
        k_at[t] = (uint32_t)(group * kCrossKeys + r) * k_row + c * 16;
        v_at[t] = (uint32_t)(group * kCrossKeys + r) * v_row + c * 16;
    }
    const _Float16 *k = static_cast<const _Float16 *>(a.k) + b * a.k_batch + h * a.k_head;
    const _Float16 *v = static_cast<const _Float16 *>(a.v) + b * a.v_batch + h * a.v_head;
    const uint32_t rows_in = n > 0 ? n - 1 : 0;
    const __amdgpu_buffer_rsrc_t kr = __builtin_amdgcn_make_buffer_rsrc(
        const_cast<_Float16 *>(k), 0, n > 0 ? (int)(rows_in * k_row + D * 2) : 0, 0x00020000);
    const __amdgpu_buffer_rsrc_t vr = __builtin_amdgcn_make_buffer_rsrc(
        const_cast<_Float16 *>(v), 0, n > 0 ? (int)(rows_in * v_row + D * 2) : 0, 0x00020000);
    // the tile the offsets stand at, and on to the next (past the last tile:
    // zeros, by the buffers' range)
    auto request_k = [&](_Float16 *to) {
#pragma unroll
        for (int t = 0; t < kLoads; ++t) {
            __builtin_amdgcn_raw_ptr_buffer_load_lds(kr, (lds_void *)(to + (t * R + wave) * 512), 16, k_at[t], 0, 0, 0);
            k_at[t] += kGroups * kCrossKeys * k_row;
        }
    };
    auto request_v = [&](_Float16 *to) {
#pragma unroll
        for (int t = 0; t < kLoads; ++t) {
            __builtin_amdgcn_raw_ptr_buffer_load_lds(vr, (lds_void *)(to + (t * R + wave) * 512), 16, v_at[t], 0, 0, 0);
            v_at[t] += kGroups * kCrossKeys * v_row;
        }
    };

    f16v o[D / 32];
#pragma unroll
    for (int i = 0; i < D / 32; ++i)
#pragma unroll
        for (int e = 0; e < 16; ++e) o[i][e] = 0.0f;
    float ref = kRefLowest, l = 0.0f;

    // Scores of 32 keys: element e is key e % 4 + 8 (e / 4) + 4 half.
    auto scores = [&](const _Float16 *sk) {
        f16v s;
#pragma unroll
        for (int e = 0; e < 16; ++e) s[e] = 0.0f;
#pragma unroll
        for (int j = 0; j < D / 16; ++j) {
            const int c = (2 * j + half) ^ swizzle<D>(col);
            s = mma32(*reinterpret_cast<const h8 *>(sk + col * D + c * 8), q[j], s);
        }
        return s;
    };
    // Makes the scores of keys that are not valid (all but the first `left`)
    // -infinity, by one more product: a column that is -infinity in their rows and 0
    // in the others, times ones. (A score that is no number stays so: an infinite
    // query's with a zero row. The pass below that takes such keys again leaves
    // them out by choice.)
    auto mask = [&](f16v s, int left) {
        const u32x4 ones = {half ? 0u : 0x3C00u, 0u, 0u, 0u}, off = {half || col < left ? 0u : 0xFC00u, 0u, 0u, 0u};
        return mma32(__builtin_bit_cast(h8, off), __builtin_bit_cast(h8, ones), s);
    };
    auto largest = [&](const f16v &s) {
        float top = s[0];
#pragma unroll
        for (int e = 1; e < 16; ++e) top = fmaxf(top, s[e]);
        return top * mul;
    };

    // tiles of 32 keys: this group's are group, group + 2, ...
    const int tiles = n > 0 ? (n + kCrossKeys - 1) / kCrossKeys : 0;
    float top = 0.0f;
    // Moves the reference where the largest score passes it by more than the slack.
    auto follow = [&]() {
        if (__any(top > ref + kSlack)) {
            float to = fmaxf(ref, top - kLift);
            to = fmaxf(to, __shfl_xor(to, 32));
            const float keep = __builtin_amdgcn_exp2f(ref - to);
            ref = to;
            l *= keep;
#pragma unroll
            for (int i = 0; i < D / 32; ++i)
#pragma unroll
                for (int e = 0; e < 16; ++e) o[i][e] *= keep;
        }
    };
    // Tile `tile`, whose scores are s: its weights and their product with the
    // values in sv, while the scores of the group's next one (keys in sk) are
    // taken into s_next; the keys after those and the next values are requested.
    auto step = [&](int tile, const f16v &s, f16v &s_next, const _Float16 *sk, _Float16 *sk_free,
                    const _Float16 *sv, _Float16 *sv_free) {
        // the next keys and these values have arrived, and the group is done
        // with the ones before
        meet();
        request_k(sk_free);
        request_v(sv_free);
        if (tile >= tiles) return;   // (the odd group's last step)
        follow();
        s_next = scores(sk);
        // weights, rounded to float16 for the second product; their sum is
        // taken from the rounded values, so that the rounding's mean cancels
        u32x4 p[2];
#pragma unroll
        for (int e = 0; e < 16; e += 2) {
            const f2 x = {__builtin_amdgcn_exp2f(__builtin_fmaf(s[e], mul, -ref)),
                          __builtin_amdgcn_exp2f(__builtin_fmaf(s[e + 1], mul, -ref))};
            const h2 w = __builtin_convertvector(x, h2);
            l = __builtin_amdgcn_fdot2(w, h2{(_Float16)1.0f, (_Float16)1.0f}, l, false);
            p[e / 8][e % 8 / 2] = as_u32(w);
        }
        // p[ks] element j of lane half h is key 16 ks + 8 (j / 4) + 4 h + j % 4
#pragma unroll
        for (int dt = 0; dt < D / 32; ++dt)
#pragma unroll
            for (int ks = 0; ks < 2; ++ks) {
                h8 w;
#pragma unroll
                for (int u = 0; u < 2; ++u) {
                    // 16 lanes read four keys by 16 dimensions: lane L supplies
                    // key L / 4, four dimensions 4 (L % 4) on, and receives
                    // dimension L of the four keys
                    const int r = 16 * ks + 8 * u + 4 * half + (lane & 15) / 4;
                    const int d = 32 * dt + 16 * ((lane >> 4) & 1) + 4 * (lane & 3);
                    const int at = r * D + (((d >> 3) ^ swizzle<D>(r)) << 3) + (d & 7);
                    const h4 x = __builtin_bit_cast(h4, __builtin_amdgcn_ds_read_tr16_b64_v4i16(
                                                            (__attribute__((address_space(3))) s4 *)(sv + at)));
#pragma unroll
                    for (int j = 0; j < 4; ++j) w[4 * u + j] = x[j];
                }
                o[dt] = mma32(w, __builtin_bit_cast(h8, p[ks]), o[dt]);
            }
        const int left = n - (tile + kGroups) * kCrossKeys;
        if (left < kCrossKeys) s_next = mask(s_next, left);
        top = largest(s_next);
    };
    f16v s0, s1;
    if (tiles > 0) {
        request_k(s_k0[group]);
        meet();
        request_k(s_k1[group]);
        request_v(s_v0[group]);
        s0 = scores(s_k0[group]);
        const int left = n - group * kCrossKeys;
        if (left < kCrossKeys) s0 = mask(s0, left);
        top = largest(s0);
    }
    for (int tile = 0; tile < tiles; tile += 2 * kGroups) {
        step(tile + group, s0, s1, s_k1[group], s_k0[group], s_v0[group], s_v1[group]);
        if (tile + kGroups >= tiles) break;
        step(tile + kGroups + group, s1, s0, s_k0[group], s_k1[group], s_v1[group], s_v0[group]);
    }
    // A float16 weight may be zero where the weight is not, and gives NaN with an
    // infinite value. Finite values leave finite sums, so a sum that is not finite
    // says that the wave is to take its keys again, with the weights in float32:
    // this time by itself, straight from memory. So does a reference so large that
    // the rounding of s * mul in it, which the first pass's fused weights do not
    // share, is no small factor (2^-4 at 2^20, 2^8 at 2^32: weights out of range).
    float bad = ref > kRefLowest && __builtin_fabsf(ref) > 0x1p20f ? 1.0f : 0.0f;
#pragma unroll
    for (int i = 0; i < D / 32; ++i)
#pragma unroll
        for (int e = 0; e < 16; ++e) bad = __builtin_fmaf(o[i][e], 0.0f, bad);
    if (__builtin_expect(__any(bad != 0.0f), 0)) {
        ref = kRefLowest;
        l = 0.0f;
#pragma unroll
        for (int i = 0; i < D / 32; ++i)
#pragma unroll
            for (int e = 0; e < 16; ++e) o[i][e] = 0.0f;
        for (int tile = group; tile < tiles; tile += kGroups) {
            const uint32_t first = tile * kCrossKeys;
            f16v s;
#pragma unroll
            for (int e = 0; e < 16; ++e) s[e] = 0.0f;
#pragma unroll
            for (int j = 0; j < D / 16; ++j)
                s = mma32(__builtin_bit_cast(h8, __builtin_amdgcn_raw_buffer_load_b128(
                                                     kr, (first + col) * k_row + (2 * j + half) * 16, 0, 0)),
                          q[j], s);
            const int left = n - (int)first - 4 * half;
#pragma unroll
            for (int e = 0; e < 16; ++e) s[e] = e % 4 + 8 * (e / 4) < left ? s[e] : -__builtin_inff();
            top = largest(s);
            follow();
#pragma unroll
            for (int e = 0; e < 16; ++e) {
                const float w = __builtin_amdgcn_exp2f(s[e] * mul - ref);
                const uint32_t at = (first + e % 4 + 8 * (e / 4) + 4 * half) * v_row + col * 2;
                l += w;
#pragma unroll
                for (int i = 0; i < D / 32; ++i)
                    o[i] = mma2((float)__builtin_bit_cast(
                                    _Float16, __builtin_amdgcn_raw_buffer_load_b16(vr, at + 64 * i, 0, 0)),
                                w, o[i]);
            }
        }
    }
    if constexpr (kGroups == 2) {
        // join the groups: the odd one hands its sums over in the key buffers, each
        // of which holds half of them
        meet();
        constexpr int kHalf = D / 64;
        static_assert(sizeof(s_k0) == kHalf * 2 * 4096, "a key buffer holds half of two waves' sums");
        auto slot = [&](int i, int e) {
            f4 *base = reinterpret_cast<f4 *>(i < kHalf ? &s_k0[0][0] : &s_k1[0][0]);
            return base + ((wave * kHalf + i % kHalf) * 4 + e / 4) * 64 + lane;
        };
        float *s_ml = reinterpret_cast<float *>(&s_v0[0][0]) + (wave * 64 + lane) * 2;
        if (group == 1) {
    #pragma unroll
            for (int i = 0; i < D / 32; ++i)
    #pragma unroll
                for (int e = 0; e < 16; e += 4) *slot(i, e) = f4{o[i][e], o[i][e + 1], o[i][e + 2], o[i][e + 3]};
            s_ml[0] = ref;
            s_ml[1] = l;
        }
        meet();
        if (group == 1) return;
        {
            const float to = fmaxf(ref, s_ml[0]), keep = __builtin_amdgcn_exp2f(ref - to);
            const float f = __builtin_amdgcn_exp2f(s_ml[0] - to);
            l = l * keep + s_ml[1] * f;
    #pragma unroll
            for (int i = 0; i < D / 32; ++i)
    #pragma unroll
                for (int e = 0; e < 16; e += 4) {
                    const f4 x = *slot(i, e);
    #pragma unroll
                    for (int c = 0; c < 4; ++c) o[i][e + c] = o[i][e + c] * keep + x[c] * f;
                }
        }
    }
    l += __shfl_xor(l, 32);
    if (!on) return;
    // (zeros by choice, not by a product: the sums may be 0 * infinity)
    const bool none = l == 0.0f;
    const float by = 1.0f / l;
    auto result = [&](float sum) { return (_Float16)(none ? 0.0f : sum * by); };
    _Float16 *out = static_cast<_Float16 *>(a.out) + b * a.o_batch + token * a.o_row + hq * a.o_head;
#pragma unroll
    for (int dt = 0; dt < D / 32; ++dt)
#pragma unroll
        for (int e = 0; e < 16; e += 4) {
            const u32x2 w = {as_u32(h2{result(o[dt][e]), result(o[dt][e + 1])}),
                             as_u32(h2{result(o[dt][e + 2]), result(o[dt][e + 3])})};
            *reinterpret_cast<u32x2 *>(out + 32 * dt + 2 * e + 4 * half) = w;
        }
}

template <int D, int R> __global__ __launch_bounds__(256, D == 64 ? 3 : 2) void cross_kernel(AttnArgs a) {
    cross_workgroup<D, R>(a);
}

namespace {

template <int D, int R> void launch_rows(const AttnArgs &a, hipStream_t st) {
    const dim3 grid(a.kv_heads, (a.rows + 32 * R - 1) / (32 * R), a.batch);
    cross_kernel<D, R><<<grid, 256, 0, st>>>(a);
}

// Which of the two forms: four waves of rows where workgroups of 128 rows fill
// the chip (at D = 128, which the matrix unit bounds, a quarter of it will do)
// or the keys are few; two groups otherwise. Measured with 512 query rows over
// 1500 keys, us:
//    96 workgroups of 128 rows, D = 64:   24.1 (four) 16.3 (two groups)
//   384                                   35.1        32.3
//   768                                   56.5        63.1
//    96, D = 128                          32.8        24.6
//   192, D = 128                          35.1        36.6
//   192, D = 64, 100 keys                  6.9         7.4
//    96, D = 64, 100 keys                  6.3         5.6
bool four_rows(int64_t wgs, int64_t keys, int head_dim) {
    return wgs >= (head_dim == 128 ? 128 : 512) || (wgs >= 128 && keys <= 256);
}

}  // namespace

// Against mnb_attn.hip's kernel, which reads all keys again for every 16 rows
// but needs no step in common: that one wins while its rows of tiles are few.
// Measured over 1500 keys, 12 heads of 64, us:
//   4 requests of 62 rows (192 row tiles)   10.8 (that one)  15.1 (this one)
//   1 of 340 (264)                          13.8             15.2
//   8 of 62 (384)                           14.8             15.6
//   4 of 200 (624)                          19.7             16.0
//   2 of 448 (672)                          20.6             15.9
//   8 of 448 (2688)                         66.3             30.5
// over 400 keys, 12 of 62 (576) 10.6 and 8.7; with 16 heads of 128 over 8, 4 of
// 62 (256) 14.3 and 22.0, 1 of 448 (448) 20.5 and 22.6, 2 of 448 (896) 36.5 and
// 24.3.
bool cross_many(int64_t batch, int64_t kv_heads, int64_t rows, int64_t max_len, int head_dim, int dtype) {
    const int64_t tiles = (rows + 15) / 16;
    return dtype == 1 && rows > 16 && batch * kv_heads >= (512 + tiles - 1) / tiles;
}

bool cross_fits(const AttnArgs &a, int head_dim) {
    // the buffers' 32-bit ranges; value rows that do not overlap, so that those
    // ranges hide the ones that are not valid; a scale that leaves masked scores
    // infinite; a launch's grid
    if (!(__builtin_fabsf(a.scale) >= 1e-30f)) return false;
    const int64_t most = 0x7FFFFFFFLL, rows = a.max_len + 8 * kCrossKeys;
    const int64_t stride = a.k_row > a.v_row ? a.k_row : a.v_row;
    return a.v_row >= head_dim && rows * stride * 2 + head_dim * 2 <= most && a.kv_heads <= (1 << 22) &&
           ((int64_t)a.rows + 63) / 64 <= 65536;
}

hipError_t launch_cross(const AttnArgs &a, int head_dim, hipStream_t st) {
    const bool full = four_rows((int64_t)a.batch * a.kv_heads * ((a.rows + 127) / 128), a.max_len, head_dim);
    if (head_dim == 128) full ? launch_rows<128, 4>(a, st) : launch_rows<128, 2>(a, st);
    else full ? launch_rows<64, 4>(a, st) : launch_rows<64, 2>(a, st);
    return hipGetLastError();
}

}  // namespace mnb
