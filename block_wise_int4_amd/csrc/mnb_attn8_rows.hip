// Attention of many query rows over the 8-bit cache, float16: the same sums as
// mnb_attn8.hip, for calls with enough rows to be bound by arithmetic (prompts, and
// chunks of them after a cached prefix).
//
// A workgroup is four waves on 128 query rows of one (request, key-value head), 32
// rows a wave, walking over a chunk of the keys 32 at a time. Codes come from memory
// to registers one step ahead, become float16 there (exactly: five instructions
// for four) and go to one of two LDS tiles, whose rows' 16-byte pieces are permuted
// by `swizzle`; the scales beside them. One barrier a step.
//   S^T = CK Q^T  (32 x 32 x 16 products: a lane holds 16 keys' products with one
//                 query), then times scale, key scale and log2(e)
//   O^T = CV^T P^T takes P = w vs from those registers as it is: the contraction
//                 index is renumbered to the keys a lane holds, and CV^T comes out
//                 of LDS through the transposing 8-byte reads.
// Weights are held against a reference 2^7 below the running maximum, which moves
// when a score passes that maximum by more than 2^8; times value scales against the
// largest's power of two so far, they are rounded to float16 (11 bits: as the
// output is). Their sum, the denominator, is float32.
#include "mnb_attn8.h"

namespace mnb {

namespace {

constexpr int kKeys = 32;     // of a step
constexpr float kLift = 7.0f, kSlack = 8.0f + kLift;

typedef float f16v __attribute__((ext_vector_type(16)));
typedef _Float16 h4 __attribute__((ext_vector_type(4)));
typedef short s4 __attribute__((ext_vector_type(4)));

__device__ __forceinline__ f16v mma32(h8 a, h8 b, f16v c) {
    return __builtin_amdgcn_mfma_f32_32x32x16_f16(a, b, c, 0, 0, 0);
}

// Where 16-byte piece c of LDS row `row` is: c ^ swizzle(row). Sixteen rows (of one
// piece) and eight rows by two adjacent pairs of pieces (the two kinds of read) each
// touch all banks evenly.
template <int D> __device__ __forceinline__ int swizzle(int row) {
    if constexpr (D == 64) return ((row >> 1) & 3) << 1 | ((row >> 3) & 1);
    else return (row & 7) << 1 | ((row >> 3) & 1);
}

// Four codes as float16: 128 more than each in the low byte of 1024 + ..., less 1152.
__device__ __forceinline__ void widen(uint32_t w, uint32_t *to) {
    w ^= 0x80808080u;
    const h2 off = {(_Float16)1152.0f, (_Float16)1152.0f};
    to[0] = as_u32(as_h2(__builtin_amdgcn_perm(0x64646464u, w, 0x04010400u)) - off);
    to[1] = as_u32(as_h2(__builtin_amdgcn_perm(0x64646464u, w, 0x04030402u)) - off);
}

__device__ __forceinline__ float halves_max(float x) {
    const u32x2 r = __builtin_bit_cast(u32x2, __builtin_amdgcn_permlane32_swap(as_bits(x), as_bits(x), false, false));
    return fmaxf(as_float(r.x), as_float(r.y));
}

}  // namespace

template <int D> __device__ __forceinline__ void rows_workgroup(const Attn8Args &a, const Attn8Split &sp) {
    constexpr int kPieces = D / 16;             // of a row of codes
    constexpr int kHalf = kKeys * kPieces;      // threads that carry a tile's keys (or values)
    constexpr int kTile = kKeys * D;
    constexpr int kEach = 2 * kHalf / 256;      // pieces per thread, keys and values
    __shared__ __attribute__((aligned(16))) _Float16 s_k[2][kTile], s_v[2][kTile];
    __shared__ __attribute__((aligned(16))) float s_ks[2][kKeys], s_vs[2][kKeys];
    __shared__ uint32_t s_valid[2], s_most[2];
    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int col = lane & 31, half = lane >> 5;
    const int h = blockIdx.x, chunk = blockIdx.z / sp.q_tiles;
    // (the last tiles of rows see most keys: first)
    const int q_tile = sp.q_tiles - 1 - (blockIdx.z - chunk * sp.q_tiles);
    const int64_t b = blockIdx.y;
    const Cache8 &c = a.cache;
    int64_t first;
    const int len = a.lens[b], n_new = rows_of(a, b, first);
    const int row0 = q_tile * kRowTile;
    int rows = (n_new < a.max_new ? n_new : a.max_new) * a.group - row0;
    if (rows <= 0) return;
    if (rows > kRowTile) rows = kRowTile;
    const int n = sees(a, len, n_new, token_of(a, row0 + rows - 1));
    const int begin = chunk * sp.chunk;
    if (begin >= n && chunk > 0) return;
    const int end = n - begin < sp.chunk ? n : begin + sp.chunk;
    // this lane's row
    const int i = wave * 32 + col;
    const bool on = i < rows;
    const int r = row0 + (on ? i : 0), token = token_of(a, r);
    const int mine = sees(a, len, n_new, token);
    // (uniform: keys that all of this wave's rows see)
    const int least = __builtin_amdgcn_readfirstlane(
        sees(a, len, n_new, token_of(a, row0 + (wave * 32 < rows ? wave * 32 : 0))));

    h8 q[D / 16];
    bool finite = true;
    {
        const _Float16 *src = static_cast<const _Float16 *>(a.q) + (first + token) * a.q_stride +
                              ((int64_t)h * a.group + r - token * a.group) * D;
        uint32_t top = 0;
#pragma unroll
        for (int j = 0; j < D / 16; ++j) {
            q[j] = *reinterpret_cast<const h8 *>(src + 16 * j + 8 * half);
            const u32x4 w = __builtin_bit_cast(u32x4, q[j]);
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const uint32_t lo = w[e] & 0x7FFFu, hi = w[e] >> 16 & 0x7FFFu;
                top = lo > top ? lo : top;
                top = hi > top ? hi : top;
            }
        }
        const u32x2 both = __builtin_bit_cast(u32x2, __builtin_amdgcn_permlane32_swap(top, top, false, false));
        finite = both.x < 0x7C00u && both.y < 0x7C00u;
        if (!finite)
#pragma unroll
            for (int j = 0; j < D / 16; ++j) q[j] = h8{};
    }
    const float mul = a.scale * kLog2e;

    // Staging. Thread t carries piece t % kPieces of key t / kPieces (of the keys, then
    // of the values); wave 0's lanes the scales besides: lane l of key l % 32, its
    // key's scale or (from 32 on) its value's.
    const int32_t *table = a.table + b * a.table_width;
    u32x4 codes[kEach];
    float scale = 0.0f;
    bool there = false;
    auto place = [&](int key, int64_t &id, uint32_t &row) {
        const uint32_t part = (uint32_t)key >> 4, before = blocks_before(part, sp.page_magic);
        id = key < end ? table[before] : -1;
        row = (uint32_t)key - before * (uint32_t)c.page;
        return (uint64_t)id < (uint64_t)c.num_blocks;
    };
    auto fetch = [&](int key0) {
#pragma unroll
        for (int e = 0; e < kEach; ++e) {
            const int t = tid + 256 * e, value = t >= kHalf, at = value ? t - kHalf : t;
            int64_t id;
            uint32_t row;
            codes[e] = u32x4{0, 0, 0, 0};
            if (place(key0 + at / kPieces, id, row))
                codes[e] = *reinterpret_cast<const u32x4 *>((value ? c.v : c.k) + id * c.block_stride +
                                                            h * c.head_stride + (int64_t)row * c.token_stride +
                                                            at % kPieces * 16);
        }
        if (wave == 0) {
            int64_t id;
            uint32_t row;
            there = place(key0 + col, id, row);
            scale = 0.0f;
            if (there) scale = (half ? c.v_scale : c.k_scale)[id * c.scale_block + h * c.scale_head + row];
        }
    };
    auto put = [&](int buf) {
#pragma unroll
        for (int e = 0; e < kEach; ++e) {
            const int t = tid + 256 * e, value = t >= kHalf, at = value ? t - kHalf : t;
            const int row = at / kPieces, piece = at % kPieces;
            uint32_t w[8];
#pragma unroll
            for (int k = 0; k < 4; ++k) widen(codes[e][k], w + 2 * k);
            _Float16 *to = (value ? s_v[buf] : s_k[buf]) + row * D;
            *reinterpret_cast<u32x4 *>(to + ((2 * piece) ^ swizzle<D>(row)) * 8) = u32x4{w[0], w[1], w[2], w[3]};
            *reinterpret_cast<u32x4 *>(to + ((2 * piece + 1) ^ swizzle<D>(row)) * 8) = u32x4{w[4], w[5], w[6], w[7]};
        }
        if (wave == 0) {
            if (half) s_vs[buf][col] = scale;
            else s_ks[buf][col] = scale * mul;
            // the largest value scale that is a number
            uint32_t top = half && as_bits(scale) < 0x7F800000u ? as_bits(scale) : 0u;
#pragma unroll
            for (int d = 1; d < 64; d <<= 1) {
                const uint32_t other = (uint32_t)__shfl_xor((int)top, d);
                top = other > top ? other : top;
            }
            const uint64_t valid = __ballot(there);
            if (lane == 0) {
                s_valid[buf] = (uint32_t)valid;
                s_most[buf] = top;
            }
        }
    };

    f16v o[D / 32];
#pragma unroll
    for (int d = 0; d < D / 32; ++d)
#pragma unroll
        for (int e = 0; e < 16; ++e) o[d][e] = 0.0f;
    float ref = kLowest, l = 0.0f;
    int unit = 1;   // biased exponent of the value scales' unit
    const int steps = end > begin ? (end - begin + kKeys - 1) / kKeys : 0;
    if (steps > 0) {
        fetch(begin);
        put(0);
    }
    for (int step = 0; step < steps; ++step) {
        const int buf = step & 1, key0 = begin + step * kKeys;
        __syncthreads();
        if (step + 1 < steps) fetch(key0 + kKeys);
        f16v s;
#pragma unroll
        for (int e = 0; e < 16; ++e) s[e] = 0.0f;
#pragma unroll
        for (int j = 0; j < D / 16; ++j) {
            const int p = (2 * j + half) ^ swizzle<D>(col);
            s = mma32(*reinterpret_cast<const h8 *>(s_k[buf] + col * D + p * 8), q[j], s);
        }
        // element e is key e % 4 + 8 (e / 4) + 4 half
        f4 ks[4], vs[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            ks[j] = *reinterpret_cast<const f4 *>(s_ks[buf] + 8 * j + 4 * half);
            vs[j] = *reinterpret_cast<const f4 *>(s_vs[buf] + 8 * j + 4 * half);
        }
        const uint32_t valid = __builtin_amdgcn_readfirstlane(s_valid[buf]);
        // (from 2^125 on float16 outputs overflow in any case)
        const int scale_bits = __builtin_amdgcn_readfirstlane(s_most[buf]) >> 23, most = scale_bits < 252 ? scale_bits : 252;
#pragma unroll
        for (int e = 0; e < 16; ++e) s[e] *= ks[e / 4][e % 4];
        const bool partial = valid != 0xFFFFFFFFu || key0 + kKeys > least;
        if (partial)   // uniform: the end of a row, or a missing block
#pragma unroll
            for (int e = 0; e < 16; ++e) {
                const int at = e % 4 + 8 * (e / 4) + 4 * half;
                const bool seen = (valid >> at & 1) && key0 + at < mine;
                s[e] = seen ? s[e] : -__builtin_inff();
                vs[e / 4][e % 4] = seen ? vs[e / 4][e % 4] : 0.0f;
            }
        float top = s[0];
#pragma unroll
        for (int e = 1; e < 16; ++e) top = fmaxf(top, s[e]);
        if (__any(top > ref + kSlack)) {
            float to = fmaxf(ref, top - kLift);
            to = halves_max(to);
            const float keep = __builtin_amdgcn_exp2f(ref - to);
            ref = to;
            l *= keep;
#pragma unroll
            for (int d = 0; d < D / 32; ++d)
#pragma unroll
                for (int e = 0; e < 16; ++e) o[d][e] *= keep;
        }
        if (most > unit) {   // uniform: a larger value scale than any before
            const float keep = as_float((uint32_t)(unit - most + 127 > 0 ? unit - most + 127 : 0) << 23);
            unit = most;
#pragma unroll
            for (int d = 0; d < D / 32; ++d)
#pragma unroll
                for (int e = 0; e < 16; ++e) o[d][e] *= keep;
        }
        const float by = as_float((uint32_t)(253 - unit) << 23);   // 2^(126 - unit): value scales below one
        u32x4 p[2];
#pragma unroll
        for (int e = 0; e < 16; e += 2) {
            const float w0 = __builtin_amdgcn_exp2f(s[e] - ref), w1 = __builtin_amdgcn_exp2f(s[e + 1] - ref);
            l += w0;
            l += w1;
            const h2 w = {(_Float16)(w0 * (vs[e / 4][e % 4] * by)), (_Float16)(w1 * (vs[e / 4][e % 4 + 1] * by))};
            p[e / 8][e % 8 / 2] = as_u32(w);
        }
        // p[k] element j of lane half h is key 16 k + 8 (j / 4) + 4 h + j % 4
#pragma unroll
        for (int d = 0; d < D / 32; ++d)
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                h8 w;
#pragma unroll
                for (int u = 0; u < 2; ++u) {
                    // 16 lanes read four keys by 16 dimensions: lane L supplies key
                    // L / 4, four dimensions 4 (L % 4) on, and receives dimension L of
                    // the four keys
                    const int row = 16 * k + 8 * u + 4 * half + (lane & 15) / 4;
                    const int dim = 32 * d + 16 * ((lane >> 4) & 1) + 4 * (lane & 3);
                    const int at = row * D + (((dim >> 3) ^ swizzle<D>(row)) << 3) + (dim & 7);
                    const h4 x = __builtin_bit_cast(h4, __builtin_amdgcn_ds_read_tr16_b64_v4i16(
                                                            (__attribute__((address_space(3))) s4 *)(s_v[buf] + at)));
#pragma unroll
                    for (int j = 0; j < 4; ++j) w[4 * u + j] = x[j];
                }
                o[d] = mma32(w, __builtin_bit_cast(h8, p[k]), o[d]);
            }
        if (step + 1 < steps) put(buf ^ 1);
    }
    const u32x2 ls = __builtin_bit_cast(u32x2, __builtin_amdgcn_permlane32_swap(as_bits(l), as_bits(l), false, false));
    l = as_float(ls.x) + as_float(ls.y);
    if (!on) return;
    if (!finite && l != 0.0f) l = __builtin_nanf("");   // (its products were taken with zeros)
    const float back = as_float((uint32_t)(unit + 1) << 23);   // 2^(unit - 126)
    if (n <= sp.chunk) {
#pragma unroll
        for (int d = 0; d < D / 32; ++d)
#pragma unroll
            for (int e = 0; e < 16; e += 4)
                store_out<_Float16, D>(a, first, h, r, 32 * d + 2 * e + 4 * half,
                                       f4{o[d][e], o[d][e + 1], o[d][e + 2], o[d][e + 3]} * back, l);
    } else {
        const int64_t piece = ((b * c.heads + h) * sp.rows + r) * sp.chunks + chunk;
#pragma unroll
        for (int d = 0; d < D / 32; ++d)
#pragma unroll
            for (int e = 0; e < 16; e += 4)
                *reinterpret_cast<f4 *>(sp.sums + piece * D + 32 * d + 2 * e + 4 * half) =
                    f4{o[d][e], o[d][e + 1], o[d][e + 2], o[d][e + 3]} * back;
        if (half == 0) {
            sp.stats[2 * piece] = ref;
            sp.stats[2 * piece + 1] = l;
        }
    }
}

template <int D> __global__ __launch_bounds__(256, 2) void attn8_rows_kernel(Attn8Args a, Attn8Split sp) {
    rows_workgroup<D>(a, sp);
}

hipError_t launch_attn8_rows(const Attn8Args &a, const Attn8Split &sp, int head_dim, hipStream_t st) {
    const dim3 grid(a.cache.heads, a.batch, (unsigned)(sp.q_tiles * sp.chunks));
    if (head_dim == 128) attn8_rows_kernel<128><<<grid, 256, 0, st>>>(a, sp);
    else attn8_rows_kernel<64><<<grid, 256, 0, st>>>(a, sp);
    return hipGetLastError();
}

}  // namespace mnb
