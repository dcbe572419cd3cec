// Tiles of 64 keys of the 8-bit cache as the streaming kernels take them: where they
// are, their codes on the way into LDS, and out of it as matrix operands.
#pragma once
#include "mnb_attn8.h"

namespace mnb {

constexpr int kParts = 4;    // 16-key parts of a tile
constexpr int kKeys = 16 * kParts;

typedef int i32x2 __attribute__((ext_vector_type(2)));
typedef int i32x4 __attribute__((ext_vector_type(4)));
typedef __attribute__((address_space(3))) void lds_void;

__device__ __forceinline__ i32x4 mma64(i32x4 a, i32x4 b, i32x4 c) {
    return __builtin_amdgcn_mfma_i32_16x16x64_i8(a, b, c, 0, 0, 0);
}

// The largest over the four lanes of a column (l % 16).
__device__ __forceinline__ uint32_t column_max(uint32_t x) {
    u32x2 r = __builtin_bit_cast(u32x2, __builtin_amdgcn_permlane32_swap(x, x, false, false));
    x = r.x > r.y ? r.x : r.y;
    r = __builtin_bit_cast(u32x2, __builtin_amdgcn_permlane16_swap(x, x, false, false));
    return r.x > r.y ? r.x : r.y;
}
__device__ __forceinline__ float column_max(float x) {
    // (elements through functions: a bit cast of a vector's element reads the first)
    u32x2 r = __builtin_bit_cast(u32x2, __builtin_amdgcn_permlane32_swap(as_bits(x), as_bits(x), false, false));
    x = fmaxf(as_float(r.x), as_float(r.y));
    r = __builtin_bit_cast(u32x2, __builtin_amdgcn_permlane16_swap(as_bits(x), as_bits(x), false, false));
    return fmaxf(as_float(r.x), as_float(r.y));
}

__device__ __forceinline__ float weight(float x, float m) { return __builtin_amdgcn_exp2f((x - m) * kLog2e); }

// Where 16-byte piece c of LDS row `row` is: c ^ swizzle(row). The first product's
// reads (8 rows, one piece) and the transposing ones (8 of 32 rows, one piece) each
// touch all banks evenly.
template <int D> __device__ __forceinline__ int swizzle(int row) {
    if constexpr (D == 128) return ((row >> 1) & 3) | ((row >> 4) & 1) << 2;
    else return ((row >> 2) & 1) | ((row >> 4) & 1) << 1;
}

// The lower three bytes of four numbers w = n + 0x8080 by their place: signed digits of
// n, the lower two 128 too much, and less again by the sign bit.
__device__ __forceinline__ void digits_of(const uint32_t *w, uint32_t *digit) {
    const uint32_t a01 = __builtin_amdgcn_perm(w[1], w[0], 0x05010400u);   // bytes 0, 0, 1, 1
    const uint32_t a23 = __builtin_amdgcn_perm(w[3], w[2], 0x05010400u);
    const uint32_t b01 = __builtin_amdgcn_perm(w[1], w[0], 0x0C0C0602u);   // bytes 2, 2
    const uint32_t b23 = __builtin_amdgcn_perm(w[3], w[2], 0x06020C0Cu);
    digit[0] = __builtin_amdgcn_perm(a23, a01, 0x05040100u) ^ 0x80808080u;
    digit[1] = __builtin_amdgcn_perm(a23, a01, 0x07060302u) ^ 0x80808080u;
    digit[2] = b01 | b23;
}

// The biased exponent under which a positive number is no more than 1.985 times a power of
// two: three balanced digits hold whole numbers up to 127 (2^16 + 2^8 + 1), 1.992 2^22.
__device__ __forceinline__ int exponent_of(uint32_t bits) {
    return (int)(as_bits(as_float(bits) * (1.0f + 0x1p-7f)) >> 23);
}

// A query row: lane (any column, g = lane / 16) takes 16 dimensions of each 64 from src on,
// which is the row's 16 g.
template <typename T, int D> struct QueryRow {
    static constexpr int kLoads = D / 64, kEach = 16 / (int)sizeof(T);
    u32x4 w[kLoads][sizeof(T)];

    __device__ __forceinline__ void load(const T *src) {
#pragma unroll
        for (int j = 0; j < kLoads; ++j)
#pragma unroll
            for (int p = 0; p < (int)sizeof(T); ++p) w[j][p] = reinterpret_cast<const u32x4 *>(src + 64 * j)[p];
    }
    __device__ __forceinline__ float at(int j, int i) const {
        const u32x4 x = w[j][i / kEach];
        if constexpr (sizeof(T) == 2) return (float)__builtin_bit_cast(h8, x)[i % kEach];
        else return __builtin_bit_cast(f4, x)[i % kEach];
    }
    // In three digits: digit[j][t] is digit t, least significant first, of piece j's numbers
    // n = x 2^(22 - e), 2^e the largest element's power of two (the next one where three
    // digits would not hold the largest): |n| < 2^23. mul 2^exponent: of a
    // sum of products with n, to a score without the key's scale (apart, as it may lie far
    // past float32's range and the score not); NaN (and digits of zeros) for a row that is
    // not finite.
    __device__ __forceinline__ void digits(float scale, i32x4 (*digit)[3], float &mul, int &exponent) const {
        uint32_t top = 0;
#pragma unroll
        for (int j = 0; j < kLoads; ++j)
#pragma unroll
            for (int i = 0; i < 16; ++i) {
                // (as whole numbers: infinities and NaN are above every finite one)
                const uint32_t bits = as_bits(at(j, i)) & 0x7FFFFFFFu;
                top = bits > top ? bits : top;
            }
        top = column_max(top);
        const bool finite = top < 0x7F800000u;
        // (the smallest rows 2^64 times as large)
        const bool small = top < (64u << 23);
        const float lift = small ? 0x1p64f : 1.0f;
        if (small) top = as_bits(as_float(top) * 0x1p64f);
        const int e = top ? exponent_of(top) : 127;
        const float up = as_float((uint32_t)(127 + 22 + 127 - e) << 23);
        mul = finite ? __builtin_amdgcn_frexp_mantf(scale) : __builtin_nanf("");
        exponent = __builtin_amdgcn_frexp_expf(scale) + e - 127 - 22 - (small ? 64 : 0);
#pragma unroll
        for (int j = 0; j < kLoads; ++j)
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                uint32_t n[4], d[3];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const float v = finite ? at(j, 4 * k + i) * lift * up : 0.0f;
                    n[i] = (uint32_t)(int)__builtin_rintf(v) + 0x8080u;
                }
                digits_of(n, d);
#pragma unroll
                for (int t = 0; t < 3; ++t) digit[j][t][k] = (int)d[t];
            }
    }
};

// What a sum of products with a query's numbers is worth as a score: mul 2^exponent times
// the key's scale. (The power of two first: exact unless the whole is below 2^-126, the
// score below 2^-85, or past float32's range.)
__device__ __forceinline__ float score_step(float key_scale, float mul, int exponent) {
    return __builtin_amdgcn_ldexpf(key_scale, exponent) * mul;
}

// Weights times value scales as whole numbers below 2^23: times `up`, 2^22 over the largest's
// power of two, plus 2^23 + 0x8080, whose bytes are the digits; `down` takes their sums back
// (NaN where one was not finite). (Of 22 bits, and queries as well, float32 outputs were off
// by 4.9e-7 of their size, where the float32 formula is by 2.8e-7.)
constexpr float kDigits = 8388608.0f + 32896.0f;
__device__ __forceinline__ void weight_steps(uint32_t most, float &up, float &down) {
    const bool finite = most < 0x7F800000u;
    int e = exponent_of(most);
    e = e < 24 ? 24 : e;
    up = as_float((uint32_t)(127 + 22 + 127 - e) << 23);
    down = finite ? as_float((uint32_t)(e - 22) << 23) : __builtin_nanf("");
}

// A wave's tile. s_keys, s_values: its places in LDS, kKeys rows of D codes, 16-byte
// pieces permuted by `swizzle`.
template <int D, bool STREAM> struct CodeTile {
    static constexpr int kLoads = D / 64;      // of 1 KB per part
    static constexpr int kPieces = D / 16;     // of a row of codes
    static constexpr int kBytes = kKeys * D;
    static constexpr int kCodeLoads = kParts * kLoads;

    const Cache8 &c;
    const int32_t *table;
    const int table_width, lane;
    int end;                 // of the keys that any row sees (set before the first tile is located)
    const uint32_t magic, stride;
    uint8_t *s_keys, *s_values;
    // Lanes 16 s on look after part s: its table entry, then where it is, as bytes to its
    // codes and scales (of keys and of values alike), and how many codes there are: a
    // part past the last key, or without a block, is read through a buffer of no
    // bytes. (Rows of a page past the last key are read, and weigh nothing.) Read from
    // those lanes where a load needs it: worked out in scalar registers it takes 400
    // instructions a tile, and more registers than there are.
    int32_t id;
    uint64_t from, from_scales;
    uint32_t bytes, there;   // (there: a bit for each part)
    uint32_t at[2][kLoads];  // of a load's pieces, in even and odd parts

    __device__ __forceinline__ CodeTile(const Attn8Args &a, const Attn8Split &sp, int64_t b, int lane,
                                        uint8_t *s_keys, uint8_t *s_values)
        : c(a.cache), table(a.table + b * a.table_width), table_width(a.table_width), lane(lane), end(0),
          magic(sp.page_magic), stride((uint32_t)a.cache.token_stride), s_keys(s_keys), s_values(s_values), id(0),
          from(0), from_scales(0), bytes(0), there(0) {
        constexpr int kRows = 64 / kPieces;   // of a load: whole rows, 64 lanes on 1 KB after another
#pragma unroll
        for (int odd = 0; odd < 2; ++odd)
#pragma unroll
            for (int j = 0; j < kLoads; ++j) {
                const int row = j * kRows + lane / kPieces;
                at[odd][j] = (uint32_t)row * stride + ((lane % kPieces) ^ swizzle<D>(16 * odd + row)) * 16;
            }
    }

    // Requests the table entries of the tile at key0 (past the table's end the last one,
    // which is not used).
    __device__ __forceinline__ void look_up(int key0) {
        const uint32_t place = blocks_before(((uint32_t)key0 >> 4) + (lane >> 4), magic);
        id = table[place < (uint32_t)table_width ? place : table_width - 1];
    }

    // Where the tile at key0 is, whose entries have been looked up.
    __device__ __forceinline__ void locate(int key0) {
        const uint32_t part = ((uint32_t)key0 >> 4) + (lane >> 4);
        const uint32_t row = (part - blocks_before(part, magic) * (uint32_t)(c.page >> 4)) << 4;
        const bool ok = (uint32_t)id < (uint32_t)c.num_blocks && key0 + (lane & 48) < end;
        const uint64_t block = ok ? (uint32_t)id : 0u;
        bytes = ok ? 15 * stride + D : 0u;
        from = block * (uint64_t)c.block_stride + (uint64_t)row * stride;
        from_scales = (block * (uint64_t)c.scale_block + row) * 4;
        const uint64_t all = __ballot(ok);
        there = (uint32_t)(all & 1) | (uint32_t)(all >> 16 & 1) << 1 | (uint32_t)(all >> 32 & 1) << 2 |
                (uint32_t)(all >> 48 & 1) << 3;
    }

    static __device__ __forceinline__ uint32_t of_part(uint32_t x, int s) {
        return (uint32_t)__builtin_amdgcn_readlane((int)x, 16 * s);
    }
    __device__ __forceinline__ __amdgpu_buffer_rsrc_t buffer(const void *base, uint64_t at, int s, uint32_t most) const {
        const uint64_t to = (uint64_t)of_part((uint32_t)(at >> 32), s) << 32 | of_part((uint32_t)at, s);
        const uint32_t n = of_part(bytes, s);
        return __builtin_amdgcn_make_buffer_rsrc(const_cast<uint8_t *>(static_cast<const uint8_t *>(base)) + to, 0,
                                                 n < most ? n : most, 0x00020000);
    }
    // Requests codes: kCodeLoads loads.
    __device__ __forceinline__ void load_codes(const int8_t *base, uint8_t *to) const {
#pragma unroll
        for (int s = 0; s < kParts; ++s) {
            const auto rows_in = buffer(base, from, s, ~0u);
#pragma unroll
            for (int j = 0; j < kLoads; ++j)
                __builtin_amdgcn_raw_ptr_buffer_load_lds(rows_in, (lds_void *)(to + (s * kLoads + j) * 1024), 16,
                                                         at[s & 1][j], 0, 0, STREAM ? 2 : 0);
        }
    }

    // Keys: lane (key l % 16, g = l / 16) takes pieces 4 j + g of its row in each part. All
    // but the last BEHIND loads have come back first. (With its waits: the compiler waits
    // for the values' loads as well, which come after.)
    template <int BEHIND> __device__ __forceinline__ void read_keys(i32x4 (*k)[kLoads]) const {
        uint32_t at[2][kLoads];
#pragma unroll
        for (int odd = 0; odd < 2; ++odd)
#pragma unroll
            for (int j = 0; j < kLoads; ++j) {
                const int row = 16 * odd + (lane & 15);
                at[odd][j] = (uint32_t)(size_t)(lds_void *)s_keys + row * D +
                             ((4 * j + (lane >> 4)) ^ swizzle<D>(row)) * 16;
            }
        if constexpr (kLoads == 2)
            asm volatile(
                "s_waitcnt vmcnt(%13)\n\t"
                "ds_read_b128 %0, %8\n\tds_read_b128 %1, %9\n\tds_read_b128 %2, %10\n\tds_read_b128 %3, %11\n\t"
                "ds_read_b128 %4, %8 offset:%12\n\tds_read_b128 %5, %9 offset:%12\n\t"
                "ds_read_b128 %6, %10 offset:%12\n\tds_read_b128 %7, %11 offset:%12\n\t"
                "s_waitcnt lgkmcnt(0)"
                : "=&v"(k[0][0]), "=&v"(k[0][kLoads - 1]), "=&v"(k[1][0]), "=&v"(k[1][kLoads - 1]), "=&v"(k[2][0]),
                  "=&v"(k[2][kLoads - 1]), "=&v"(k[3][0]), "=&v"(k[3][kLoads - 1])
                : "v"(at[0][0]), "v"(at[0][kLoads - 1]), "v"(at[1][0]), "v"(at[1][kLoads - 1]), "n"(32 * D),
                  "n"(BEHIND)
                : "memory");
        else
            asm volatile(
                "s_waitcnt vmcnt(%7)\n\t"
                "ds_read_b128 %0, %4\n\tds_read_b128 %1, %5\n\t"
                "ds_read_b128 %2, %4 offset:%6\n\tds_read_b128 %3, %5 offset:%6\n\t"
                "s_waitcnt lgkmcnt(0)"
                : "=&v"(k[0][0]), "=&v"(k[1][0]), "=&v"(k[2][0]), "=&v"(k[3][0])
                : "v"(at[0][0]), "v"(at[1][0]), "n"(32 * D), "n"(BEHIND)
                : "memory");
    }

    // Values, turned, 16-dimension parts d .. d + 3: 16 lanes read eight keys by 16
    // dimensions. Lane L supplies key L / 2, eight dimensions 8 (L % 2) on, and receives
    // dimension L of the eight keys. RUNS: bytes e of lane (dimension l % 16, g) are keys
    // 16 g + e; otherwise 16 (e / 4) + 4 g + e % 4. (Four parts at a time, and their wait with
    // them: through the builtin the compiler waits for all loads first, the next keys'
    // among them.)
    template <bool RUNS> __device__ __forceinline__ void read_values(i32x2 (*v)[2], int d) const {
        const int col = lane & 15, g = lane >> 4;
        const int row = RUNS ? 16 * g + (col >> 1) : 16 * (col >> 3) + 4 * g + ((col >> 1) & 3);
        const uint32_t base = (uint32_t)(size_t)(lds_void *)s_values + row * D + (col & 1) * 8;
        uint32_t at[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) at[e] = base + ((d + e) ^ swizzle<D>(row)) * 16;
        // (the second eight keys: 8 or 32 rows on, where pieces are permuted alike)
        asm volatile(
            "ds_read_b64_tr_b8 %0, %8\n\tds_read_b64_tr_b8 %1, %8 offset:%12\n\t"
            "ds_read_b64_tr_b8 %2, %9\n\tds_read_b64_tr_b8 %3, %9 offset:%12\n\t"
            "ds_read_b64_tr_b8 %4, %10\n\tds_read_b64_tr_b8 %5, %10 offset:%12\n\t"
            "ds_read_b64_tr_b8 %6, %11\n\tds_read_b64_tr_b8 %7, %11 offset:%12\n\t"
            "s_waitcnt lgkmcnt(0)"
            : "=&v"(v[0][0]), "=&v"(v[0][1]), "=&v"(v[1][0]), "=&v"(v[1][1]), "=&v"(v[2][0]), "=&v"(v[2][1]),
              "=&v"(v[3][0]), "=&v"(v[3][1])
            : "v"(at[0]), "v"(at[1]), "v"(at[2]), "v"(at[3]), "n"((RUNS ? 8 : 32) * D)
            : "memory");
    }
};

// Waits until all but the last BEHIND loads have come back.
template <int BEHIND> __device__ __forceinline__ void wait_loads() {
    asm volatile("s_waitcnt vmcnt(%0)" ::"n"(BEHIND) : "memory");
}

}  // namespace mnb
