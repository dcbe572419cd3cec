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

template <int N> struct Number { static constexpr int value = N; };

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
    int32_t ids[2];      // of the next step's parts
    auto look_up = [&](int key0) {
#pragma unroll
        for (int s = 0; s < 2; ++s) {
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

    // Staging. A wave carries 512 codes of one 16-key part a step, 16 a lane: rows of the
    // keys and the same of the values (D = 128), or of one of them (D = 64); its lanes
    // 0..15 besides that part's scales, the keys' or the values'. So a wave's block is
    // uniform, looked up three steps ahead; its codes are requested two steps ahead,
    // through buffers that end with the last key that any row sees.
    constexpr bool kBoth = D == 128;
    const int part = kBoth ? wave >> 1 : wave & 1, value = kBoth ? wave & 1 : wave >> 1;   // (value: of the scales)
    const uint32_t stride = (uint32_t)c.token_stride;
    const int row = kBoth ? wave * 8 + lane / kPieces : (wave & 1) * 16 + lane / kPieces, piece = lane % kPieces;
    const uint32_t at_row = (uint32_t)(row & 15) * stride + piece * 16;
    u32x4 codes[2][kBoth ? 2 : 1];   // of even and odd steps
    float scale[2];
    uint32_t valid[2];   // bit k: key k of the step has a block, and some row sees it
    auto fetch = [&](auto parity, int key0) {
        constexpr int buf = decltype(parity)::value;
        int ok[2];
#pragma unroll
        for (int s = 0; s < 2; ++s) {
            const int left = end - key0 - 16 * s;
            ok[s] = __builtin_amdgcn_readfirstlane(
                left < 0 || (uint64_t)(int64_t)ids[s] >= (uint64_t)c.num_blocks ? 0 : left > 16 ? 16 : left);
        }
        valid[buf] = ((1u << ok[0]) - 1) | ((1u << ok[1]) - 1) << 16;
        const int id = part ? ids[1] : ids[0], mine_ok = part ? ok[1] : ok[0];
        const uint32_t number = ((uint32_t)key0 >> 4) + part;
        const uint32_t in_page = (number - blocks_before(number, sp.page_magic) * (uint32_t)(c.page >> 4)) << 4;
        const int64_t from = id * c.block_stride + h * c.head_stride + (int64_t)in_page * stride;
        const uint32_t bytes = mine_ok > 0 ? (uint32_t)(mine_ok - 1) * stride + D : 0u;
        auto request = [&](const int8_t *base) {
            return __builtin_bit_cast(
                u32x4, __builtin_amdgcn_raw_buffer_load_b128(
                           __builtin_amdgcn_make_buffer_rsrc(const_cast<int8_t *>(base + from), 0, bytes, 0x00020000),
                           at_row, 0, 0));
        };
        if constexpr (kBoth) {
            codes[buf][0] = request(c.k);
            codes[buf][1] = request(c.v);
        } else {
            codes[buf][0] = request(value ? c.v : c.k);
        }
        const float *scales = (value ? c.v_scale : c.k_scale) + id * c.scale_block + h * c.scale_head + in_page;
        scale[buf] = as_float(__builtin_amdgcn_raw_buffer_load_b32(
            __builtin_amdgcn_make_buffer_rsrc(const_cast<float *>(scales), 0, mine_ok * 4u, 0x00020000),
            (lane & 15) * 4, 0, 0));
    };
    const int put_at = row * D, lo = ((2 * piece) ^ swizzle<D>(row)) * 8, hi = ((2 * piece + 1) ^ swizzle<D>(row)) * 8;
    auto put = [&](auto parity) {
        constexpr int buf = decltype(parity)::value;
#pragma unroll
        for (int e = 0; e < (kBoth ? 2 : 1); ++e) {
            uint32_t w[8];
#pragma unroll
            for (int k = 0; k < 4; ++k) widen(codes[buf][e][k], w + 2 * k);
            _Float16 *to = ((kBoth ? e == 1 : value == 1) ? s_v[buf] : s_k[buf]) + put_at;
            *reinterpret_cast<u32x4 *>(to + lo) = u32x4{w[0], w[1], w[2], w[3]};
            *reinterpret_cast<u32x4 *>(to + hi) = u32x4{w[4], w[5], w[6], w[7]};
        }
        if (lane < 16) (value ? s_vs : s_ks)[buf][16 * part + lane] = value ? scale[buf] : scale[buf] * mul;
    };

    // Whole rows of a [token][head][D] tensor: lane l of step k carries 16 bytes of the
    // wave's row k * kRowsAtOnce + l / (D / 8); where it is in memory, and in LDS, where a
    // row's 16-byte pieces are permuted by the row. (Loops over k stay loops: the code is
    // run once a launch, out of a cold instruction cache.)
    constexpr int kRowPieces = D / 8, kRowsAtOnce = 64 / kRowPieces, kCarries = 32 / kRowsAtOnce;
    _Float16 *s_mine = s_tiles + wave * (32 * D);
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
    // exp2(score - ref), of this lane's keys; biased exponent of the value scales' unit.
    float ref = 0.0f, l = 0.0f;
    bool started = false;
    int unit = 1;
    fetch(Number<0>{}, begin);
    look_up(begin + kKeys);
    asm volatile("s_waitcnt vmcnt(0)" ::: "memory");   // (the compiler does not count loads to LDS)
    uint32_t top = 0;
#pragma unroll
    for (int j = 0; j < D / 16; ++j) {
        q[j] = *reinterpret_cast<const h8 *>(in_rows(col, 2 * j + half));
        const u32x4 x = __builtin_bit_cast(u32x4, q[j]);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const uint32_t lo = x[e] & 0x7FFFu, hi = x[e] >> 16 & 0x7FFFu;
            top = lo > top ? lo : top;
            top = hi > top ? hi : top;
        }
    }
    const u32x2 both = __builtin_bit_cast(u32x2, __builtin_amdgcn_permlane32_swap(top, top, false, false));
    finite = both.x < 0x7C00u && both.y < 0x7C00u;
    if (!finite)
#pragma unroll
        for (int j = 0; j < D / 16; ++j) q[j] = h8{};
    fetch(Number<1>{}, begin + kKeys);
    look_up(begin + 2 * kKeys);
    __syncthreads();   // (the tiles' place is free)
    put(Number<0>{});
    auto take = [&](auto parity, int key0) __attribute__((always_inline)) {
        constexpr int buf = decltype(parity)::value;
        __syncthreads();
        const uint32_t seen_keys = valid[buf];
        // (past the last key: no bytes)
        fetch(parity, key0 + 2 * kKeys);
        look_up(key0 + 3 * kKeys);
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
        // the largest value scale that is a number; from 2^125 on float16 outputs overflow
        // in any case
        float scales = 0.0f;
#pragma unroll
        for (int j = 0; j < 4; ++j)
#pragma unroll
            for (int e = 0; e < 4; ++e) scales = fmaxf(scales, vs[j][e]);
        int most = __builtin_amdgcn_readfirstlane((int)as_bits(halves_max(scales))) >> 23;
        most = most < 252 ? most : 252;
        // scores less the reference, plus the unit's power of two: its inverse, 2^(126 -
        // unit), then comes with the weights and leaves value scales below one
        float shift = (float)(126 - unit);
#pragma unroll
        for (int e = 0; e < 16; ++e) s[e] = __builtin_fmaf(s[e], ks[e / 4][e % 4], shift - ref);
        if (seen_keys != 0xFFFFFFFFu || key0 + kKeys > least) {   // uniform: the end of a row, or a missing block
            const int left = mine - key0;
            uint32_t bits = left >= 32 ? 0xFFFFFFFFu : left <= 0 ? 0u : (1u << left) - 1;
            bits = (bits & seen_keys) >> (4 * half);
#pragma unroll
            for (int e = 0; e < 16; ++e) {
                const uint32_t seen = (uint32_t)((int)(bits << (31 - e % 4 - 8 * (e / 4))) >> 31);
                s[e] = as_float((as_bits(s[e]) & seen) | (0xFF800000u & ~seen));
                vs[e / 4][e % 4] = as_float(as_bits(vs[e / 4][e % 4]) & seen);
            }
        }
        float top = s[0];
#pragma unroll
        for (int e = 1; e < 16; ++e) top = fmaxf(top, s[e]);
        if (__any(top > (started ? shift + kSlack : -__builtin_inff())) || most > unit) {
            top = halves_max(top);
            const bool some = top > -__builtin_inff();
            float by = top - shift - kLift;   // how far the reference moves
            by = started ? fmaxf(by, 0.0f) : some ? by : 0.0f;
            const int raised = most > unit ? most : unit, less = unit - raised + 127;
            const float keep = started ? __builtin_amdgcn_exp2f(-by) : 1.0f;   // (nothing to keep at the start)
            const float keep_sums = keep * as_float((uint32_t)(less > 0 ? less : 0) << 23);
            l *= keep;
#pragma unroll
            for (int d = 0; d < D / 32; ++d)
#pragma unroll
                for (int e = 0; e < 16; ++e) o[d][e] *= keep_sums;
            started |= some;
            ref += by;
            by += (float)(raised - unit);
            unit = raised;
            shift = (float)(126 - unit);
#pragma unroll
            for (int e = 0; e < 16; ++e) s[e] -= by;
        }
        u32x4 p[2];
        float sum = 0.0f;
#pragma unroll
        for (int e = 0; e < 16; e += 2) {
            const float w0 = __builtin_amdgcn_exp2f(s[e]), w1 = __builtin_amdgcn_exp2f(s[e + 1]);
            sum += w0;
            sum += w1;
            const h2 w = {(_Float16)(w0 * vs[e / 4][e % 4]), (_Float16)(w1 * vs[e / 4][e % 4 + 1])};
            p[e / 8][e % 8 / 2] = as_u32(w);
        }
        l = __builtin_fmaf(sum, as_float((uint32_t)(unit + 1) << 23), l);   // 2^(unit - 126)
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
        put(Number<buf ^ 1>{});
    };
    for (int key0 = begin; key0 < end; key0 += 2 * kKeys) {
        take(Number<0>{}, key0);
        if (key0 + kKeys < end) take(Number<1>{}, key0 + kKeys);
    }
    const u32x2 ls = __builtin_bit_cast(u32x2, __builtin_amdgcn_permlane32_swap(as_bits(l), as_bits(l), false, false));
    l = as_float(ls.x) + as_float(ls.y);
    if (!finite && l != 0.0f) l = __builtin_nanf("");   // (its products were taken with zeros)
    const float back = as_float((uint32_t)(unit + 1) << 23);   // 2^(unit - 126)
    __syncthreads();   // (the tiles' last reads are over)
    if (n <= sp.chunk) {
        const float by = l == 0.0f ? 0.0f : back / l;   // (sums are zeros where no key has weight)
#pragma unroll
        for (int d = 0; d < D / 32; ++d)
#pragma unroll
            for (int e = 0; e < 16; e += 4) {
                const u32x2 w = {as_u32(h2{(_Float16)(o[d][e] * by), (_Float16)(o[d][e + 1] * by)}),
                                 as_u32(h2{(_Float16)(o[d][e + 2] * by), (_Float16)(o[d][e + 3] * by)})};
                *reinterpret_cast<u32x2 *>(in_rows(col, 4 * d + e / 4) + 4 * half) = w;
            }
#pragma unroll 1
        for (int k = 0; k < kCarries; ++k) {
            const int row = k * kRowsAtOnce + carried;
            int64_t of, head;
            token_head(row, of, head);
            if (wave * 32 + row < rows)
                *reinterpret_cast<u32x4 *>(static_cast<_Float16 *>(a.out) +
                                           (of * ((int64_t)c.heads * a.group) + head) * D + carried_piece * 8) =
                    *reinterpret_cast<const u32x4 *>(in_rows(row, carried_piece));
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
                *reinterpret_cast<f4 *>(in_rows(col, 8 * d + e / 2 + half)) =
                    f4{o[d0 + d][e], o[d0 + d][e + 1], o[d0 + d][e + 2], o[d0 + d][e + 3]} * back;
#pragma unroll 1
        for (int k = 0; k < kCarries; ++k) {
            const int row = k * kRowsAtOnce + carried;
            if (wave * 32 + row < rows)
                *reinterpret_cast<f4 *>(sums + (int64_t)row * sp.chunks * D + 32 * d0 + carried_piece * 4) =
                    *reinterpret_cast<const f4 *>(in_rows(row, carried_piece));
        }
    }
    if (on && half == 0) {
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
