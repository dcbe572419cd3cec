// Attention of many query rows over the 8-bit cache, float16: the same sums as
// mnb_attn8.hip, for calls with enough rows to be bound by arithmetic (prompts, and
// chunks of them after a cached prefix).
//
// A workgroup is four waves on 128 query rows of one (request, key-value head), 32
// rows a wave, walking over a chunk of the keys 64 at a time. Codes come from memory
// to registers one step ahead, become float16 there (exactly: five instructions
// for four) and go to one of two LDS tiles, whose rows' 16-byte pieces are permuted
// by `swizzle`; the scales beside them. One barrier a step.
//   S^T = CK Q^T  (32 x 32 x 16 products: a lane holds 16 keys' products with one
//                 query), then times scale, key scale and log2(e)
//   O^T = CV^T P^T takes P = w vs from those registers as it is: the contraction
//                 index is renumbered to the keys a lane holds, and CV^T comes out
//                 of LDS through the transposing 8-byte reads.
// Weights are held against a reference, the running maximum or up to 2^8 below it; a
// score less its reference is one multiply-add. That rounds as a float32 score does, but
// equal scores of different steps do not round alike: 2^-10 of a weight at most, below
// kFar. A wave whose scores may be larger (by its queries' largest element and the
// step's key scales) goes on with scores rounded first and the maximum itself taken off
// them, which is exact.
// Weights times value scales are the second product's terms, two float16 numbers each, 22
// bits: one number (11 bits) took 1.9 us of 26.1 off 16 prompts of 62..410 rows and 1.6 of
// 31.0 off 8 x 62 rows after up to 2000 keys, and put outputs off by 2.9e-4 of their size where
// their own rounding is 2.1e-4. A power of two of the row's own, `up`, keeps its largest so
// far at 2^7 .. 2^15, whatever the scales of keys that it does not see or that have no
// weight; it comes with the exponentials, whose arguments it makes up to 2^6 larger (2^-18 of
// a weight). The weights' sum, the denominator, is float32.
//
// 16 prompts of 62..410 rows, 16 heads of 128 over 8, take 27 us: 4.4 GFLOP, 39 MB. Half of
// that is the loop, bound by vector instructions (470 a wave and step, exponentials counted
// as four, against 1536 cycles of matrix products), 13 steps in the fullest CU where the
// mean is 6; a launch and a step take 8. 8 x 62 rows after up to 2000 keys take 25 and
// the join 6: some 200 workgroups of five steps, over 2 us each where a CU has one (5500
// cycles, of which 1536 are matrix and 1900 vector instructions: latency). With 32 keys a step,
// terms of 11 bits, these took 34 and 35 us (24 and 23 with 64). Two teams of four waves on
// alternate steps, joined in LDS, were 1 to 2.5 us slower in calls of few workgroups and 15%
// faster in those that fill every CU once with whole rows.
#include "mnb_attn8.h"

namespace mnb {

namespace {

constexpr int kKeys = 64;     // of a step: four 16-key parts
constexpr float kSlack = 8.0f, kFar = 16384.0f;
constexpr float kMostUp = 60.0f, kMostTerm = 32768.0f, kMostFloat = 3.402823466e38f;
constexpr int kTerm = 7;      // a row's largest term is taken to 2^7 .. 2^8

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

typedef unsigned short us2 __attribute__((ext_vector_type(2)));
__device__ __forceinline__ us2 as_us2(uint32_t x) { return __builtin_bit_cast(us2, x); }

// The largest of a wave's, whose halves have the same.
template <int N> __device__ __forceinline__ float turned(float x) {   // by N of 16 lanes
    const int b = __builtin_bit_cast(int, x);
    return __builtin_bit_cast(float, __builtin_amdgcn_update_dpp(b, b, 0x120 + N, 0xF, 0xF, false));
}
__device__ __forceinline__ float wave_max(float x) {
    const u32x2 r = __builtin_bit_cast(u32x2, __builtin_amdgcn_permlane16_swap(as_bits(x), as_bits(x), false, false));
    x = fmaxf(as_float(r.x), as_float(r.y));
    x = fmaxf(x, turned<8>(x));
    x = fmaxf(x, turned<4>(x));
    x = fmaxf(x, turned<2>(x));
    return fmaxf(x, turned<1>(x));
}

}  // namespace

template <int D> __device__ __forceinline__ void rows_workgroup(const Attn8Args &a, const Attn8Split &sp) {
    constexpr int kPieces = D / 16;             // of a row of codes
    constexpr int kTile = kKeys * D;
    // two tiles of keys and two of values; before and after the loop a quarter for each
    // wave, through which its rows of q come in and its rows of results go out whole
    __shared__ __attribute__((aligned(16))) _Float16 s_tiles[4 * kTile];
    _Float16(*const s_k)[kTile] = reinterpret_cast<_Float16(*)[kTile]>(s_tiles);
    _Float16(*const s_v)[kTile] = s_k + 2;
    __shared__ __attribute__((aligned(16))) float s_ks[2][kKeys], s_vs[2][kKeys];
    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int col = lane & 31, half = lane >> 5;
    const int h = blockIdx.x, chunk = blockIdx.z / sp.q_tiles;
    // (the last tiles of rows see most keys: first)
    const int q_tile = sp.q_tiles - 1 - (blockIdx.z - chunk * sp.q_tiles);
    const int64_t b = blockIdx.y;
    const Cache8 &c = a.cache;
    const int begin = chunk * sp.chunk;
    // (no kernel writes the table, the lengths and the starts while this one reads them:
    // scalar loads)
    typedef __attribute__((address_space(4))) const int32_t entry;
    entry *table = (entry *)(a.table + b * a.table_width);
    int32_t ids[4];      // of the next step's parts
    auto look_up = [&](int key0) {
#pragma unroll
        for (int s = 0; s < 4; ++s) {
            const uint32_t place = blocks_before(((uint32_t)key0 >> 4) + s, sp.page_magic);
            ids[s] = table[place < (uint32_t)a.table_width ? place : a.table_width - 1];
        }
    };
    look_up(begin);
    int64_t first;
    const int len = ((entry *)a.lens)[b], n_new = rows_of(a, b, first);
    const int row0 = q_tile * kRowTile;
    int rows = (n_new < a.max_new ? n_new : a.max_new) * a.group - row0;
    if (rows <= 0) return;
    if (rows > kRowTile) rows = kRowTile;
    const int n = sees(a, len, n_new, token_of(a, row0 + rows - 1));
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
    const float mul = a.scale * kLog2e;

    // Staging. Wave w carries the keys and the values of the step's part w, 16 codes a
    // lane and load, and their scales (lanes 0..15 the keys', 16..31 the values'). So a
    // wave's block is uniform, looked up two steps ahead; its codes are requested one
    // step ahead, through buffers that end with the last key that any row sees.
    constexpr int kLoads = D / 64, kLoadRows = 16 / kLoads;
    const uint32_t stride = (uint32_t)c.token_stride;
    const int row = lane / kPieces, piece = lane % kPieces;   // of a load
    u32x4 codes[2][kLoads];   // of the keys, of the values
    float scale;
    uint64_t valid, valid_next;   // bit k: key k of the step has a block, and some row sees it
    auto fetch = [&](int key0) {
        int ok[4];
        valid_next = 0;
#pragma unroll
        for (int s = 0; s < 4; ++s) {
            const int left = end - key0 - 16 * s;
            ok[s] = __builtin_amdgcn_readfirstlane(
                left < 0 || (uint32_t)ids[s] >= (uint32_t)c.num_blocks ? 0 : left > 16 ? 16 : left);
            valid_next |= (uint64_t)((1u << ok[s]) - 1) << (16 * s);
        }
        const int id = wave == 0 ? ids[0] : wave == 1 ? ids[1] : wave == 2 ? ids[2] : ids[3];
        const int mine_ok = wave == 0 ? ok[0] : wave == 1 ? ok[1] : wave == 2 ? ok[2] : ok[3];
        const uint32_t number = ((uint32_t)key0 >> 4) + wave;
        const uint32_t in_page = (number - blocks_before(number, sp.page_magic) * (uint32_t)(c.page >> 4)) << 4;
        const int64_t from = id * c.block_stride + h * c.head_stride + (int64_t)in_page * stride;
        const uint32_t bytes = mine_ok > 0 ? (uint32_t)(mine_ok - 1) * stride + D : 0u;
#pragma unroll
        for (int v = 0; v < 2; ++v)
#pragma unroll
            for (int i = 0; i < kLoads; ++i)
                codes[v][i] = __builtin_bit_cast(
                    u32x4, __builtin_amdgcn_raw_buffer_load_b128(
                               __builtin_amdgcn_make_buffer_rsrc(const_cast<int8_t *>((v ? c.v : c.k) + from), 0, bytes,
                                                                 0x00020000),
                               (uint32_t)(i * kLoadRows + row) * stride + piece * 16, 0, 0));
        const int64_t at = id * c.scale_block + h * c.scale_head + in_page + (lane & 15);
        scale = 0.0f;
        if ((lane & 15) < mine_ok && lane < 32) scale = (lane < 16 ? c.k_scale : c.v_scale)[at];
    };
    auto put = [&](int buf) {
#pragma unroll
        for (int v = 0; v < 2; ++v)
#pragma unroll
            for (int i = 0; i < kLoads; ++i) {
                const int to_row = 16 * wave + i * kLoadRows + row;
                uint32_t w[8];
#pragma unroll
                for (int k = 0; k < 4; ++k) widen(codes[v][i][k], w + 2 * k);
                _Float16 *to = (v ? s_v[buf] : s_k[buf]) + to_row * D;
                *reinterpret_cast<u32x4 *>(to + ((2 * piece) ^ swizzle<D>(to_row)) * 8) = u32x4{w[0], w[1], w[2], w[3]};
                *reinterpret_cast<u32x4 *>(to + ((2 * piece + 1) ^ swizzle<D>(to_row)) * 8) =
                    u32x4{w[4], w[5], w[6], w[7]};
            }
        if (lane < 32) (lane < 16 ? s_ks : s_vs)[buf][16 * wave + (lane & 15)] = lane < 16 ? scale * mul : scale;
    };

    // Whole rows of a [token][head][D] tensor: lane l of step k carries 16 bytes of the
    // wave's row k * kRowsAtOnce + l / (D / 8); where it is in memory, and in LDS, where a
    // row's 16-byte pieces are permuted by the row. (Loops over k stay loops: the code is
    // run once a launch, out of a cold instruction cache.)
    constexpr int kRowPieces = D / 8, kRowsAtOnce = 64 / kRowPieces, kCarries = 32 / kRowsAtOnce;
    _Float16 *s_mine = s_tiles + wave * kTile;
    auto in_rows = [&](int row, int piece) { return s_mine + row * D + (piece ^ (row & (kRowPieces - 1))) * 8; };
    const int carried = lane / kRowPieces, carried_piece = lane % kRowPieces;
    auto token_head = [&](int row, int64_t &of, int64_t &head) {   // of the wave's row
        const int at = row0 + wave * 32 + row, t = token_of(a, at);
        of = first + t;
        head = (int64_t)h * a.group + at - t * a.group;
    };
    typedef __attribute__((address_space(3))) void lds_void;
    typedef __attribute__((address_space(1))) void global_void;
#pragma unroll 1
    for (int k = 0; k < kCarries; ++k) {
        // (rows behind the last stand for it)
        const int row = k * kRowsAtOnce + carried, last = rows - 1 - wave * 32;
        int64_t of, head;
        token_head(row < last ? row : last, of, head);
        const _Float16 *from = static_cast<const _Float16 *>(a.q) + of * a.q_stride + head * D +
                               (carried_piece ^ (row & (kRowPieces - 1))) * 8;
        __builtin_amdgcn_global_load_lds((global_void *)from, (lds_void *)(s_mine + k * 512), 16, 0, 0);
    }

    h8 q[D / 16];
    bool finite = true;
    f16v o[D / 32];
#pragma unroll
    for (int d = 0; d < D / 32; ++d)
#pragma unroll
        for (int e = 0; e < 16; ++e) o[d][e] = 0.0f;
    // The reference of this lane's row (once a key is seen), the sum of weights
    // exp2(score - ref), of this lane's keys, and the logarithm of its terms' factor.
    float ref = 0.0f, l = 0.0f, up = kMostUp;
    bool started = false, far = false;   // far, of the wave: ref is the running maximum itself
    fetch(begin);
    look_up(begin + kKeys);
    asm volatile("s_waitcnt vmcnt(0)" ::: "memory");   // (the compiler does not count loads to LDS)
    us2 tops = {0, 0};   // largest |q|, as whole numbers: infinities and NaN are above every finite one
#pragma unroll
    for (int j = 0; j < D / 16; ++j) {
        q[j] = *reinterpret_cast<const h8 *>(in_rows(col, 2 * j + half));
        const u32x4 x = __builtin_bit_cast(u32x4, q[j]);
#pragma unroll
        for (int e = 0; e < 4; ++e) tops = __builtin_elementwise_max(tops, as_us2(x[e] & 0x7FFF7FFFu));
    }
    uint32_t top = tops.x > tops.y ? tops.x : tops.y;
    const u32x2 both = __builtin_bit_cast(u32x2, __builtin_amdgcn_permlane32_swap(top, top, false, false));
    top = both.x > both.y ? both.x : both.y;
    finite = top < 0x7C00u;
    if (!finite)
#pragma unroll
        for (int j = 0; j < D / 16; ++j) q[j] = h8{};
    // what no product of codes with one of the wave's queries passes
    const float most_product = 128.0f * D * wave_max((float)as_h2(finite ? top : 0u).x);
    __syncthreads();   // (the tiles' place is free)
    put(0);
    valid = valid_next;
    float minus = -1.0f;
    asm("" : "+s"(minus));   // (known, it makes the multiply-adds below subtractions)
    int buf = 0;
    for (int key0 = begin; key0 < end; key0 += kKeys, buf ^= 1) {
        __syncthreads();
        // (past the last key: no bytes)
        fetch(key0 + kKeys);
        look_up(key0 + 2 * kKeys);
        f16v s[2];
#pragma unroll
        for (int t = 0; t < 2; ++t)
#pragma unroll
            for (int e = 0; e < 16; ++e) s[t][e] = 0.0f;
#pragma unroll
        for (int j = 0; j < D / 16; ++j) {
            const _Float16 *from = s_k[buf] + col * D + ((2 * j + half) ^ swizzle<D>(col)) * 8;
#pragma unroll
            for (int t = 0; t < 2; ++t) s[t] = mma32(*reinterpret_cast<const h8 *>(from + 32 * t * D), q[j], s[t]);
        }
        if (!far && __any(fabsf(s_ks[buf][lane]) * most_product >= kFar)) far = true;
        const float from = far ? 0.0f : up - ref;   // (a product plus zero is rounded alone)
        // element e of half t is key 32 t + e % 4 + 8 (e / 4) + 4 half
        f4 vs[2][4];
#pragma unroll
        for (int t = 0; t < 2; ++t)
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const f4 ks = *reinterpret_cast<const f4 *>(s_ks[buf] + 32 * t + 8 * j + 4 * half);
#pragma unroll
                for (int e = 0; e < 4; ++e) s[t][4 * j + e] = __builtin_fmaf(s[t][4 * j + e], ks[e], from);
                vs[t][j] = *reinterpret_cast<const f4 *>(s_vs[buf] + 32 * t + 8 * j + 4 * half);
            }
        if (valid != ~0ull || key0 + kKeys > least) {   // uniform: the end of a row, or a missing block
#pragma unroll
            for (int t = 0; t < 2; ++t) {
                const int left = mine - key0 - 32 * t;
                uint32_t bits = left >= 32 ? 0xFFFFFFFFu : left <= 0 ? 0u : (1u << left) - 1;
                bits = (bits & (uint32_t)(valid >> (32 * t))) >> (4 * half);
#pragma unroll
                for (int e = 0; e < 16; ++e) {
                    const uint32_t seen = (uint32_t)((int)(bits << (31 - e % 4 - 8 * (e / 4))) >> 31);
                    s[t][e] = as_float((as_bits(s[t][e]) & seen) | (0xFF800000u & ~seen));
                    vs[t][e / 4][e % 4] = as_float(as_bits(vs[t][e / 4][e % 4]) & seen);
                }
            }
        }
        float top = s[0][0];
#pragma unroll
        for (int e = 1; e < 32; ++e) top = fmaxf(top, s[e / 16][e % 16]);
        if (far || __any(top > (started ? up + kSlack : -__builtin_inff()))) {
            top = halves_max(top);
            const bool some = top > -__builtin_inff();
            float by = far ? top - ref : top - up;   // how far the reference moves
            by = started ? fmaxf(by, 0.0f) : some ? by : 0.0f;
            // (sums so far shrink by that; the factor takes up what it can of it)
            const float more = started ? fminf(up + floorf(by), kMostUp) - up : 0.0f;
            const float keep = started ? __builtin_amdgcn_exp2f(-by) : 1.0f;   // (nothing to keep at the start)
            const float keep_sums = started ? __builtin_amdgcn_exp2f(more - by) : 1.0f;
            l *= keep;
#pragma unroll
            for (int d = 0; d < D / 32; ++d)
#pragma unroll
                for (int e = 0; e < 16; ++e) o[d][e] *= keep_sums;
            ref = !far ? ref + by : !some ? ref : started ? fmaxf(ref, top) : top;
            started |= some;
            up += more;
            const float less = far ? ref : by, plus = far ? up : more;
#pragma unroll
            for (int e = 0; e < 32; ++e) s[e / 16][e % 16] = (s[e / 16][e % 16] - less) + plus;
        }
        float sum[2] = {0.0f, 0.0f}, terms[2] = {0.0f, 0.0f};
#pragma unroll
        for (int e = 0; e < 32; ++e) {
            const float w = __builtin_amdgcn_exp2f(s[e / 16][e % 16]);
            sum[e % 2] += w;
            s[e / 16][e % 16] = w * vs[e / 16][e % 16 / 4][e % 4];
            terms[e / 16] = fmaxf(terms[e / 16], s[e / 16][e % 16]);
        }
        float term = fmaxf(terms[0], terms[1]);
        l += __builtin_amdgcn_ldexpf(sum[0] + sum[1], -(int)up);
        if (__any(term > kMostTerm)) {
            // (terms past float32's range, of value scales from 2^59 on, stand for its largest, 2^68 or more of
            // the reference's weight: infinite in float16 but with codes of zero, which infinity makes NaN)
            term = fminf(halves_max(term), kMostFloat);
            const int down = term > kMostTerm ? (int)(as_bits(term) >> 23) - 127 - kTerm : 0;   // 8 .. 120
            const float factor = as_float((uint32_t)(127 - down) << 23);
#pragma unroll
            for (int e = 0; e < 32; ++e) {
                const float x = s[e / 16][e % 16];
                s[e / 16][e % 16] = (x > kMostFloat ? kMostFloat : x) * factor;   // (NaN stays)
            }
#pragma unroll
            for (int d = 0; d < D / 32; ++d)
#pragma unroll
                for (int e = 0; e < 16; ++e) o[d][e] *= factor;
            up -= (float)down;
        }
        // (each term as two float16 numbers: what the first leaves is exact, and the second's;
        // written as multiply-adds, which take and give float16 by themselves)
        u32x4 p[2][2], rest[2][2];
#pragma unroll
        for (int e = 0; e < 32; e += 2) {
            const float x = s[e / 16][e % 16], y = s[e / 16][e % 16 + 1];
            const h2 w = __builtin_bit_cast(h2, __builtin_amdgcn_cvt_pkrtz(x, y));
            const h2 r = {(_Float16)__builtin_fmaf((float)w.x, minus, x), (_Float16)__builtin_fmaf((float)w.y, minus, y)};
            p[e / 16][e % 16 / 8][e % 8 / 2] = as_u32(w);
            rest[e / 16][e % 16 / 8][e % 8 / 2] = as_u32(r);
        }
        // p[t][k] element j of lane half h is key 32 t + 16 k + 8 (j / 4) + 4 h + j % 4
#pragma unroll
        for (int t = 0; t < 2; ++t)
#pragma unroll
            for (int k = 0; k < 2; ++k)
#pragma unroll
                for (int d = 0; d < D / 32; ++d) {
                    h8 w;
#pragma unroll
                    for (int u = 0; u < 2; ++u) {
                        // 16 lanes read four keys by 16 dimensions: lane L supplies key
                        // L / 4, four dimensions 4 (L % 4) on, and receives dimension L of
                        // the four keys
                        const int row = 32 * t + 16 * k + 8 * u + 4 * half + (lane & 15) / 4;
                        const int dim = 32 * d + 16 * ((lane >> 4) & 1) + 4 * (lane & 3);
                        const int at = row * D + (((dim >> 3) ^ swizzle<D>(row)) << 3) + (dim & 7);
                        const h4 x = __builtin_bit_cast(
                            h4, __builtin_amdgcn_ds_read_tr16_b64_v4i16(
                                    (__attribute__((address_space(3))) s4 *)(s_v[buf] + at)));
#pragma unroll
                        for (int j = 0; j < 4; ++j) w[4 * u + j] = x[j];
                    }
                    o[d] = mma32(w, __builtin_bit_cast(h8, p[t][k]), o[d]);
                    o[d] = mma32(w, __builtin_bit_cast(h8, rest[t][k]), o[d]);
                }
        put(buf ^ 1);
        valid = valid_next;
    }
    const u32x2 ls = __builtin_bit_cast(u32x2, __builtin_amdgcn_permlane32_swap(as_bits(l), as_bits(l), false, false));
    l = as_float(ls.x) + as_float(ls.y);
    if (!finite && l != 0.0f) l = __builtin_nanf("");   // (its products were taken with zeros)
    const float back = __builtin_amdgcn_ldexpf(1.0f, -(int)up);
    __syncthreads();   // (the tiles' last reads are over)
    // (the lane counted again, for its places in LDS and memory: kept over the loop these are
    // the registers too many)
    const int lane_now = (int)__builtin_amdgcn_mbcnt_hi(~0u, __builtin_amdgcn_mbcnt_lo(~0u, 0u));
    const int col_now = lane_now & 31, half_now = lane_now >> 5;
    const int carried_now = lane_now / kRowPieces, piece_now = lane_now % kRowPieces;
    if (n <= sp.chunk) {
        const float by = l == 0.0f ? 0.0f : back / l;   // (sums are zeros where no key has weight)
#pragma unroll
        for (int d = 0; d < D / 32; ++d)
#pragma unroll
            for (int e = 0; e < 16; e += 4) {
                const u32x2 w = {as_u32(h2{(_Float16)(o[d][e] * by), (_Float16)(o[d][e + 1] * by)}),
                                 as_u32(h2{(_Float16)(o[d][e + 2] * by), (_Float16)(o[d][e + 3] * by)})};
                *reinterpret_cast<u32x2 *>(in_rows(col_now, 4 * d + e / 4) + 4 * half_now) = w;
            }
        wave_fence();
#pragma unroll 1
        for (int k = 0; k < kCarries; ++k) {
            const int row = k * kRowsAtOnce + carried_now;
            int64_t of, head;
            token_head(row, of, head);
            if (wave * 32 + row < rows)
                *reinterpret_cast<u32x4 *>(static_cast<_Float16 *>(a.out) +
                                           (of * ((int64_t)c.heads * a.group) + head) * D + piece_now * 8) =
                    *reinterpret_cast<const u32x4 *>(in_rows(row, piece_now));
        }
        return;
    }
    // a piece: the sums in two halves of D / 2 dimensions, 4 bytes each
    float *sums = sp.sums + (((b * c.heads + h) * sp.rows + row0 + wave * 32) * sp.chunks + chunk) * D;
#pragma unroll
    for (int d0 = 0; d0 < D / 32; d0 += D / 64) {
#pragma unroll
        for (int d = 0; d < D / 64; ++d)
#pragma unroll
            for (int e = 0; e < 16; e += 4)
                *reinterpret_cast<f4 *>(in_rows(col_now, 8 * d + e / 2 + half_now)) =
                    f4{o[d0 + d][e], o[d0 + d][e + 1], o[d0 + d][e + 2], o[d0 + d][e + 3]} * back;
        wave_fence();
#pragma unroll 1
        for (int k = 0; k < kCarries; ++k) {
            const int row = k * kRowsAtOnce + carried_now;
            if (wave * 32 + row < rows)
                *reinterpret_cast<f4 *>(sums + (int64_t)row * sp.chunks * D + 32 * d0 + piece_now * 4) =
                    *reinterpret_cast<const f4 *>(in_rows(row, piece_now));
        }
        wave_fence();   // (the second half takes the first's place)
    }
    if (wave * 32 + col_now < rows && half_now == 0) {
        const int r = row0 + wave * 32 + col_now;
        float *stats = sp.stats + 2 * (((b * c.heads + h) * sp.rows + r) * sp.chunks + chunk);
        stats[0] = started ? ref : kLowest;
        stats[1] = l;
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
