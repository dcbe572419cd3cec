// Attention of query rows over the keys of their request (paged, or one run
// per request): o = sum_t w_t V[t] / sum_t w_t, w_t = exp(s_t - m), s_t =
// scale * q . K[t], with a reference m kept near the running maximum.
//
// Work: a row is up to 16 query rows of one (request, key-value head); its
// keys are cut into chunks, and a chunk's tiles of 16 or 32 keys are taken in
// turn by the waves of one workgroup. A wave streams its tiles: keys whole rows
// at a time through a place of its own in LDS, which turns them into the layout
// of the first product, values straight into registers:
//   S^T = K Q^T   A = keys (lane: key l % 16, 16 bytes of its row), B = queries;
//                 the result holds, per lane, four keys 4 (l / 16) + i of one
//                 query l % 16, which is already the B operand's layout of
//   O^T = V^T P^T with the contraction index renumbered: A's rows are
//                 dimensions. A lane loads whole pieces of V rows (l % 16 says
//                 which piece: a row is one coalesced run over 16 lanes), and
//                 piece element e of lane row m is dimension m * (D / 16) + e:
//                 float32 needs no shuffle at all, float16 one byte permute
//                 per pair of keys.
// The next tile's keys are requested as soon as the first product has read
// this one's, its values after the second: something is always in flight,
// three workgroups per CU. Turning the keys in registers instead (four by four
// between lanes, 160 of 339 vector instructions a tile) took 8.9 us for 8 x 452
// keys where this takes 8.1, and 22.7 against 20.2 for 62 float32 query rows
// over 1500 keys.
// The waves' sums are joined in LDS, and the chunks' by a second launch. A wave of
// a float16 call whose sums are not finite (infinite values) takes its tiles once
// more with float32 weights.
//
// Bound: memory where the card is full (32 requests of 500..16384 keys, 1.1 GB:
// 176 us, 6.3 TB/s; a bare read reaches 6.8), and latency below some 30 MB: a
// launch and the chain length - table entry - tile are 6 us by themselves.
#include "mnb_attn.h"
#include "mnb_device.h"

namespace mnb {

namespace {

constexpr int kWaves = 4;   // of a workgroup (8 or 12: no faster where it is alone on its CU, 5% slower where not)
constexpr int kXcds = 8;
constexpr int kQ = 16;                      // query rows per row of tiles
constexpr float kLowest = -3.402823466e38f; // the reference before any key
constexpr float kLog2e = 1.4426950408889634f;

typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef __attribute__((address_space(3))) void lds_void;

template <bool B> struct Flag { static constexpr bool value = B; };

template <int Bytes> struct Piece;
template <> struct Piece<16> { typedef u32x4 type; };
template <> struct Piece<8> { typedef u32x2 type; };

// One tile of keys and values of a float16 or float32 row of D.
template <typename T, int D> struct TileShape {
    static constexpr int kRow = D * (int)sizeof(T);                 // bytes
    static constexpr int kSub = sizeof(T) == 4 && D == 128 ? 1 : 2; // 16-key parts (8 KB of keys, 32 registers of V)
    static constexpr int kKeys = 16 * kSub;
    static constexpr int kTileBytes = kKeys * kRow;                 // of keys in LDS
    static constexpr int kK = kRow / 64;                            // 16-byte pieces of a K row per lane
    static constexpr int kVBytes = kRow / 16 < 16 ? kRow / 16 : 16;
    static constexpr int kV = kRow / 16 / kVBytes;                  // pieces of a V row per lane
    static constexpr int kOut = D / 16;                             // 16-dimension parts of the output
};

// Scores are kept as x = s * mul, weights are exp2 of differences: float16
// folds log2(e) into mul (its scale is at most 2^80, so no score overflows);
// float32 does not, so that scores down to the type's lowest value stay
// finite.
template <typename T> __device__ __forceinline__ float score_mul(float scale) {
    return sizeof(T) == 4 ? scale : scale * kLog2e;
}
template <typename T> __device__ __forceinline__ float weight(float x, float ref) {
    const float d = x - ref;
    return __builtin_amdgcn_exp2f(sizeof(T) == 4 ? d * kLog2e : d);
}

__device__ __forceinline__ f4 mma16(h8 a, h8 b, f4 c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_f16(a, b, c, 0, 0, 0);
}
__device__ __forceinline__ f4 mma4(float a, float b, f4 c) {
    return __builtin_amdgcn_mfma_f32_16x16x4f32(a, b, c, 0, 0, 0);
}

// A load by buffer (bytes past its range read as zeros, from nowhere); STREAM
// leaves no copy in the caches it passes, for caches of keys and values larger
// than those.
template <bool STREAM, typename V> __device__ __forceinline__ V fetch(__amdgpu_buffer_rsrc_t from, uint32_t at) {
    constexpr int how = STREAM ? 2 : 0;
    if constexpr (sizeof(V) == 16)
        return __builtin_bit_cast(V, __builtin_amdgcn_raw_buffer_load_b128(from, at, 0, how));
    else
        return __builtin_bit_cast(V, __builtin_amdgcn_raw_buffer_load_b64(from, at, 0, how));
}

__device__ __forceinline__ int keys_of(const AttnArgs &a, int64_t b) {
    int n = a.max_len;
    if (a.lens && a.lens[b] < n) n = a.lens[b];
    return n;
}

// Blocks before a part of 16 keys.
__device__ __forceinline__ uint32_t blocks_before(uint32_t part, uint32_t magic) {
    const uint32_t place = __umulhi(part, magic);
    return magic ? place : part;
}

// Query token of a query row (a decoding step has one, and no division).
__device__ __forceinline__ int token_of(const AttnArgs &a, int row) {
    return a.rows == a.group ? 0 : (int)((uint32_t)row / (uint32_t)a.group);
}

// Four outputs from dimension d on of a query row.
template <typename T>
__device__ __forceinline__ void store_out(const AttnArgs &a, int64_t b, int h, int row, int d, f4 sum, float total) {
    const int token = token_of(a, row);
    T *out = static_cast<T *>(a.out) + b * a.o_batch + token * a.o_row +
             (int64_t)(h * a.group + row - token * a.group) * a.o_head + d;
    // (zeros by choice, not by a product: the sum may be 0 * infinity)
    if (total == 0.0f) sum = f4{0.0f, 0.0f, 0.0f, 0.0f};
    else sum *= 1.0f / total;
    if constexpr (sizeof(T) == 2) {
        const u32x2 w = {as_u32(h2{(_Float16)sum.x, (_Float16)sum.y}), as_u32(h2{(_Float16)sum.z, (_Float16)sum.w})};
        *reinterpret_cast<u32x2 *>(out) = w;
    } else {
        *reinterpret_cast<f4 *>(out) = sum;
    }
}

}  // namespace

// How a launch is cut. Pieces of rows of more than one chunk: per (request,
// head, query row, chunk) D sums, and a reference and the weights' sum.
struct AttnSplit {
    int32_t chunk;        // keys per chunk
    int32_t chunks;       // of max_len
    int32_t q_tiles, held;   // of `rows`; min(rows, kQ)
    bool together;        // the order of the blocks
    uint32_t page_magic;  // ceil(2^32 / (page / 16)), 0 for pages of 16: part * magic >> 32 is
                          // part / (page / 16) for part < 2^26
    float *sums, *stats;
};

// FEW: one or two waves, rows of as many tiles at most (a kernel of its own: a
// count of waves that is read costs the others 3%).
template <typename T, int D, bool PAGED, bool STREAM, bool FEW>
__device__ __forceinline__ void attn_workgroup(const AttnArgs &a, const AttnSplit &sp) {
    using S = TileShape<T, D>;
    typedef typename Piece<S::kVBytes>::type VP;
    // first the waves' tiles of keys, then their sums [kWaves][held][D + 4]
    extern __shared__ __attribute__((aligned(16))) float s_o[];
    __shared__ float s_m[kWaves][kQ], s_l[kWaves][kQ];
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int col = lane & 15, g = lane >> 4;
    // the head varies fastest, the chunk slowest: blocks go to the XCDs in
    // turn, and the late chunks that only long requests have spread over all
    // of them
    int h = blockIdx.x, chunk = blockIdx.z, q_tile = 0;
    int64_t b = blockIdx.y;
    if (sp.together) {   // rows of tiles of the same keys eight blocks apart: on one XCD
        const uint32_t unit = blockIdx.y * kXcds + blockIdx.x % kXcds;
        if (unit >= (uint32_t)a.batch * (uint32_t)a.kv_heads) return;
        q_tile = blockIdx.x / kXcds;
        b = unit / (uint32_t)a.kv_heads;
        h = unit - (uint32_t)b * a.kv_heads;
    } else if (sp.q_tiles > 1) {
        chunk = blockIdx.z / sp.q_tiles;
        q_tile = blockIdx.z - chunk * sp.q_tiles;
    }
    const int begin = chunk * sp.chunk;
    int key = begin + wave * S::kKeys;
    // (no kernel writes the table while this one reads it: scalar loads)
    typedef __attribute__((address_space(4))) const int32_t table_entry;
    table_entry *table = PAGED ? (table_entry *)(a.table + b * a.table_width) : nullptr;

    // The table entries of the tile at key0 (past the table's end its last
    // entry, which is not used).
    int32_t ids[S::kSub];
    auto look_up = [&](int key0) {
        if constexpr (PAGED) {
#pragma unroll
            for (int s = 0; s < S::kSub; ++s) {
                const uint32_t place = blocks_before(((uint32_t)key0 >> 4) + s, sp.page_magic);
                ids[s] = table[place < (uint32_t)a.table_width ? place : a.table_width - 1];
            }
        }
    };
    look_up(key);
    const int n = keys_of(a, b);
    if (begin >= n && chunk > 0) return;
    const int end = n - begin < sp.chunk ? n : begin + sp.chunk;   // (n may be <= 0: no tile then)
    const int rows = a.rows - q_tile * kQ < kQ ? a.rows - q_tile * kQ : kQ;

    // queries: lane (query col, piece g of each 64-byte run)
    u32x4 q[S::kK];
    {
        const int r = q_tile * kQ + (col < rows ? col : 0), token = token_of(a, r);
        const T *src = static_cast<const T *>(a.q) + b * a.q_batch + token * a.q_row +
                       (int64_t)(h * a.group + r - token * a.group) * a.q_head;
        const uint8_t *p = reinterpret_cast<const uint8_t *>(src) + g * 16;
#pragma unroll
        for (int j = 0; j < S::kK; ++j) q[j] = *reinterpret_cast<const u32x4 *>(p + j * 64);
    }

    // One tile: keys, values, and where the next one is. A part (16 keys) is
    // read through a buffer that ends with its last valid key: what lies behind
    // reads as zeros, and a part without keys reads nothing.
    VP v[S::kSub][4][S::kV];
    int valid[S::kSub];   // leading valid keys of each part
    int64_t from_k[S::kSub], from_v[S::kSub];
    const uint8_t *kp = static_cast<const uint8_t *>(a.k) + h * a.k_head * (int64_t)sizeof(T);
    const uint8_t *vp = static_cast<const uint8_t *>(a.v) + h * a.v_head * (int64_t)sizeof(T);
    const uint32_t k_row = (uint32_t)a.k_row * sizeof(T), v_row = (uint32_t)a.v_row * sizeof(T);
    auto locate = [&](int key0, int *valid) {
#pragma unroll
        for (int s = 0; s < S::kSub; ++s) {
            const int first = key0 + 16 * s;
            int ok = end - first;
            ok = ok < 0 ? 0 : ok > 16 ? 16 : ok;
            int64_t of = b;
            uint32_t row = first;
            if constexpr (PAGED) {
                of = ids[s];
                ok = (uint64_t)of < (uint64_t)a.num_blocks ? ok : 0;
                const uint32_t part = (uint32_t)first >> 4;
                row = (part - blocks_before(part, sp.page_magic) * (uint32_t)(a.page >> 4)) << 4;
            }
            valid[s] = __builtin_amdgcn_readfirstlane(ok);
            from_k[s] = of * a.k_batch * (int64_t)sizeof(T) + (int64_t)((uint64_t)row * k_row);
            from_v[s] = of * a.v_batch * (int64_t)sizeof(T) + (int64_t)((uint64_t)row * v_row);
        }
    };
    auto part_of = [&](const uint8_t *base, int64_t from, int ok, uint32_t row) {
        return __builtin_amdgcn_make_buffer_rsrc(const_cast<uint8_t *>(base + from), 0,
                                                 ok > 0 ? (uint32_t)(ok - 1) * row + S::kRow : 0u, 0x00020000);
    };
    // Keys go through LDS, a tile of the wave's own: a load takes whole rows, 64
    // lanes on 1 KB after another, and a read gives lane (key col, g) piece
    // 4 j + g of its row. Pieces are permuted by the row, so that eight lanes of
    // a read touch all banks. (The counters still see conflicts in 42% of the LDS
    // cycles where rows are 256 bytes, none at 128; waves wait for LDS in less
    // than 1% of theirs. The load unit serves 16 lanes in turn, four
    // neighbours on one run of 64 bytes a cycle: a CU takes in 105 GB/s like this
    // but 37 where every lane loads from another row.)
    constexpr int kPieces = S::kRow / 16, kRows = 64 / kPieces;   // of a row; of a load
    uint8_t *s_k = reinterpret_cast<uint8_t *>(s_o) + wave * S::kTileBytes;
    uint32_t k_at[S::kK], v_at[4];
#pragma unroll
    for (int j = 0; j < S::kK; ++j) {
        const int r = j * kRows + lane / kPieces;
        k_at[j] = (uint32_t)r * k_row + ((lane % kPieces) ^ (r & 7)) * 16;
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) v_at[i] = (4 * g + i) * v_row + col * S::kVBytes;
    auto load_k = [&](const int *valid) {
#pragma unroll
        for (int s = 0; s < S::kSub; ++s) {
            const auto from = part_of(kp, from_k[s], valid[s], k_row);
#pragma unroll
            for (int j = 0; j < S::kK; ++j)
                __builtin_amdgcn_raw_ptr_buffer_load_lds(from, (lds_void *)(s_k + (s * S::kK + j) * 1024), 16, k_at[j],
                                                         0, 0, STREAM ? 2 : 0);
        }
    };
    auto read_k = [&](int s, int j) {
        return *reinterpret_cast<const u32x4 *>(s_k + (16 * s + col) * S::kRow + ((4 * j + g) ^ (col & 7)) * 16);
    };
    auto load_v = [&](const int *valid) {
#pragma unroll
        for (int s = 0; s < S::kSub; ++s) {
            const auto from = part_of(vp, from_v[s], valid[s], v_row);
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int c = 0; c < S::kV; ++c) v[s][i][c] = fetch<STREAM, VP>(from, v_at[i] + c * 256);
        }
    };

    f4 o[S::kOut];
    float ref, l;
    const float mul = score_mul<T>(a.scale);
    // The reference of the weights follows the running maximum: it moves only when
    // a score passes the maximum that set it by more than a factor of 2^8. In
    // float16 it lies 2^7 below that maximum: weights reach 2^15, the type's range,
    // and count down to 2^-32 of the maximum's. (At the maximum itself the end was
    // 2^-25, and the many small weights of a long flat row below one leading key
    // came out as nothing. Float32 sums of 32 keys at a time lose terms below some
    // 2^-29 of themselves in any case.)
    const float lift = sizeof(T) == 4 ? 0.0f : 7.0f, slack = sizeof(T) == 4 ? 5.5f : 8.0f + lift;

    const int step = kWaves * S::kKeys;   // (with fewer waves there is a tile for each, and no next one)
    // Takes this wave's tiles; exact (float16): with the second product in float32.
    auto take = [&](auto exact) __attribute__((always_inline)) {
#pragma unroll
        for (int i = 0; i < S::kOut; ++i) o[i] = f4{0.0f, 0.0f, 0.0f, 0.0f};
        ref = kLowest;
        l = 0.0f;
        if (key < end) {
            locate(key, valid);
            load_k(valid);
            asm volatile("" ::: "memory");   // (in this order: the wait below counts them)
            load_v(valid);
            look_up(key + step);
        }
        for (; key < end; key += step) {
            float x[S::kSub][4];
            // this tile's keys are in LDS: all but the loads after theirs, those of
            // its values, have come back (the compiler does not wait for loads to LDS)
            asm volatile("s_waitcnt vmcnt(%0)" ::"n"(S::kSub * 4 * S::kV) : "memory");
            f4 c[S::kSub];
#pragma unroll
            for (int s = 0; s < S::kSub; ++s) c[s] = f4{0.0f, 0.0f, 0.0f, 0.0f};
            if constexpr (sizeof(T) == 2) {
                // (all reads under way before the first product: left to itself the
                // compiler may wait for each, 7.4 us instead of 6.9 for 452 keys)
                u32x4 kk[S::kK][S::kSub];
#pragma unroll
                for (int j = 0; j < S::kK; ++j)
#pragma unroll
                    for (int s = 0; s < S::kSub; ++s) kk[j][s] = read_k(s, j);
                __builtin_amdgcn_sched_barrier(0);
#pragma unroll
                for (int j = 0; j < S::kK; ++j)
#pragma unroll
                    for (int s = 0; s < S::kSub; ++s)
                        c[s] = mma16(__builtin_bit_cast(h8, kk[j][s]), __builtin_bit_cast(h8, q[j]), c[s]);
            } else {
#pragma unroll
                for (int j = 0; j < S::kK; ++j) {
                    const f4 qq = __builtin_bit_cast(f4, q[j]);
                    f4 kk[S::kSub];
#pragma unroll
                    for (int s = 0; s < S::kSub; ++s) kk[s] = __builtin_bit_cast(f4, read_k(s, j));
#pragma unroll
                    for (int e = 0; e < 4; ++e)
#pragma unroll
                        for (int s = 0; s < S::kSub; ++s) c[s] = mma4(kk[s][e], qq[e], c[s]);
                }
            }
#pragma unroll
            for (int s = 0; s < S::kSub; ++s)
#pragma unroll
                for (int i = 0; i < 4; ++i) x[s][i] = c[s][i] * mul;
            int valid_next[S::kSub];
            locate(key + step, valid_next);
            asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");   // the reads of this tile are over
            load_k(valid_next);
            asm volatile("" ::: "memory");
            look_up(key + 2 * step);
            bool partial = false;
#pragma unroll
            for (int s = 0; s < S::kSub; ++s) partial |= valid[s] < 16;
            if (partial) {   // uniform: the end of a row, or a missing block
#pragma unroll
                for (int s = 0; s < S::kSub; ++s)
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        x[s][i] = 4 * g + i < valid[s] ? x[s][i] : -__builtin_inff();
                // (values past the last valid key are zeros already, unless rows overlap)
                if (v_row < S::kRow)
#pragma unroll
                    for (int s = 0; s < S::kSub; ++s)
#pragma unroll
                        for (int i = 0; i < 4; ++i)
#pragma unroll
                            for (int c = 0; c < S::kV; ++c) v[s][i][c] = 4 * g + i < valid[s] ? v[s][i][c] : VP(0u);
            }
            float top = x[0][0];
#pragma unroll
            for (int s = 0; s < S::kSub; ++s)
#pragma unroll
                for (int i = 0; i < 4; ++i) top = fmaxf(top, x[s][i]);
            if (__any(top > ref + slack)) {
                float to = fmaxf(ref, top - lift);
                to = fmaxf(to, __shfl_xor(to, 16));
                to = fmaxf(to, __shfl_xor(to, 32));
                const float keep = weight<T>(ref, to);
                ref = to;
                l *= keep;
#pragma unroll
                for (int i = 0; i < S::kOut; ++i) o[i] *= keep;
            }
#pragma unroll
            for (int s = 0; s < S::kSub; ++s)
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    x[s][i] = weight<T>(x[s][i], ref);
                    l += x[s][i];
                }
            if constexpr (sizeof(T) == 4) {
#pragma unroll
                for (int s = 0; s < S::kSub; ++s)
#pragma unroll
                    for (int i = 0; i < 4; ++i)
#pragma unroll
                        for (int c = 0; c < S::kV; ++c) {
                            const f4 vv = __builtin_bit_cast(f4, v[s][i][c]);
#pragma unroll
                            for (int e = 0; e < 4; ++e) o[4 * c + e] = mma4(vv[e], x[s][i], o[4 * c + e]);
                        }
            } else if constexpr (decltype(exact)::value) {
#pragma unroll
                for (int s = 0; s < S::kSub; ++s)
#pragma unroll
                    for (int i = 0; i < 4; ++i)
#pragma unroll
                        for (int e = 0; e < S::kOut; ++e) {
                            const h2 pair = as_h2(v[s][i][0][e >> 1]);
                            o[e] = mma4((float)pair[e & 1], x[s][i], o[e]);
                        }
            } else {
                // the weights as a float16 pair hi + lo (22 bits for weights above
                // 2^-10 of the largest, fewer below: hi and lo share the smallest
                // step): the stream leaves the matrix units idle, so the second
                // product is free
                h8 hi, lo;
#pragma unroll
                for (int s = 0; s < 2; ++s)
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const _Float16 w = (_Float16)x[s][i];
                        hi[4 * s + i] = w;
                        lo[4 * s + i] = (_Float16)fmaf(-1.0f, (float)w, x[s][i]);
                    }
#pragma unroll
                for (int e = 0; e < S::kOut; ++e) {
                    u32x4 w;
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const VP &v0 = v[j >> 1][2 * (j & 1)][0], &v1 = v[j >> 1][2 * (j & 1) + 1][0];
                        w[j] = __builtin_amdgcn_perm(v1[e >> 1], v0[e >> 1], e & 1 ? 0x07060302u : 0x05040100u);
                    }
                    o[e] = mma16(__builtin_bit_cast(h8, w), hi, o[e]);
                    o[e] = mma16(__builtin_bit_cast(h8, w), lo, o[e]);
                }
            }
            load_v(valid_next);
#pragma unroll
            for (int s = 0; s < S::kSub; ++s) valid[s] = valid_next[s];
        }
    };
    take(Flag<false>{});
    if constexpr (sizeof(T) == 2) {
        // A float16 weight, or a pair's second part, may be zero or negative where the
        // weight is not, and gives NaN with an infinite value. Finite values leave
        // finite sums (below 2^15 * 2^16 * 2^30 keys), so a sum that is not finite
        // says that the tiles are to be taken again with the weights in float32.
        // Nothing of it is in the first pass's loop.
        float none = 0.0f;
#pragma unroll
        for (int i = 0; i < S::kOut; ++i)
#pragma unroll
            for (int e = 0; e < 4; ++e) none = __builtin_fmaf(o[i][e], 0.0f, none);
        if (__builtin_expect(__any(none != 0.0f), 0)) {
            asm volatile("s_waitcnt vmcnt(0)" ::: "memory");   // (the tile past the end)
            key = begin + wave * S::kKeys;
            look_up(key);
            take(Flag<true>{});
        }
    }

    // (the tile past the end, zeros, has arrived everywhere: its place is free)
    asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
    __syncthreads();

    // join the waves (those that have keys)
    const int tiles = n <= S::kKeys ? 1 : (end - begin + S::kKeys - 1) / S::kKeys;
    const int waves = tiles < kWaves ? tiles : kWaves;
    if (wave < waves) {
        l += __shfl_xor(l, 16);
        l += __shfl_xor(l, 32);
        if (g == 0) {
            s_m[wave][col] = ref;
            s_l[wave][col] = l;
        }
        if (col < rows) {
            // a lane's part e, row m = 4 g + i is dimension m * (D / 16) + e
            // (float16), 64 * (e / 4) + 4 m + e % 4 (float32)
            float *to = s_o + (wave * sp.held + col) * (D + 4);
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int e = 0; e < S::kOut; e += 4) {
                    const int d = sizeof(T) == 2 ? (4 * g + i) * S::kOut + e : 16 * e + 4 * (4 * g + i);
                    *reinterpret_cast<f4 *>(to + d) = f4{o[e][i], o[e + 1][i], o[e + 2][i], o[e + 3][i]};
                }
        }
    }
    __syncthreads();
    const bool whole = n <= sp.chunk;   // this chunk is the row's only one
    for (int e = threadIdx.x; e < rows * (D / 4); e += FEW ? blockDim.x : 64 * kWaves) {
        const int r = e / (D / 4), d = e % (D / 4) * 4;
        float m = s_m[0][r];
        for (int w = 1; w < waves; ++w) m = fmaxf(m, s_m[w][r]);
        f4 sum = {0.0f, 0.0f, 0.0f, 0.0f};
        float total = 0.0f;
        for (int w = 0; w < waves; ++w) {
            const float f = weight<T>(s_m[w][r], m);
            sum += *reinterpret_cast<const f4 *>(s_o + (w * sp.held + r) * (D + 4) + d) * f;
            total += s_l[w][r] * f;
        }
        if (whole) {
            store_out<T>(a, b, h, q_tile * kQ + r, d, sum, total);
        } else {
            const int64_t piece = ((b * a.kv_heads + h) * a.rows + q_tile * kQ + r) * sp.chunks + chunk;
            *reinterpret_cast<f4 *>(sp.sums + piece * D + d) = sum;
            if (d == 0) {
                sp.stats[2 * piece] = m;
                sp.stats[2 * piece + 1] = total;
            }
        }
    }
}

template <typename T, int D, bool PAGED, bool STREAM, bool FEW>
__global__ __launch_bounds__(64 * kWaves, D * (int)sizeof(T) <= 128 ? 4 : 3)
void attn_kernel(AttnArgs a, AttnSplit sp) {
    attn_workgroup<T, D, PAGED, STREAM, FEW>(a, sp);
}

// Joins the chunks of query rows, in a fixed order: a row has 2^shift groups of
// D / 4 lanes, which take every 2^shift-th chunk; then their sums are added.
// Bound: latency (2.4 us alone, 4.5 right behind the first launch), so small and
// without a division. The first launch's last workgroups could join instead, but
// their pieces' way past the XCDs' L2s took as long: 25.4 us against 24.8 for 16
// float32 requests of up to 1503 keys, when that case was cut (it is whole now),
// and 62 against 12 where 32 workgroups join one row.
constexpr int kJoin = 256;
template <typename T, int D>
__global__ __launch_bounds__(kJoin) void attn_join_kernel(AttnArgs a, AttnSplit sp, int shift) {
    constexpr int kLanes = D / 4, kLaneBits = D == 128 ? 5 : 4;
    __shared__ f4 s_sum[kJoin];
    __shared__ float s_m[kJoin], s_l[kJoin];
    const int tid = threadIdx.x, d = tid % kLanes * 4, groups = 1 << shift;
    const int group = (tid >> kLaneBits) & (groups - 1);
    const int row = blockIdx.z * (kJoin >> (kLaneBits + shift)) + (tid >> (kLaneBits + shift));
    const int h = blockIdx.x;
    const int64_t b = blockIdx.y;
    const int n = keys_of(a, b);
    const bool on = row < a.rows;
    const int64_t first = ((b * a.kv_heads + h) * a.rows + (on ? row : 0)) * sp.chunks;
    f4 sum = {0.0f, 0.0f, 0.0f, 0.0f};
    float m = kLowest, l = 0.0f;
    // (the first place of every group is read whatever the length, so that
    // nothing waits for it; absent chunks are left out)
    for (int c = group; c < sp.chunks; c += groups) {
        const float *stats = sp.stats + 2 * (first + c);
        float pm = stats[0], pl = stats[1];
        f4 ps = *reinterpret_cast<const f4 *>(sp.sums + (first + c) * D + d);
        if (c * sp.chunk >= n) break;
        const float to = fmaxf(m, pm), keep = weight<T>(m, to), f = weight<T>(pm, to);
        sum = sum * keep + ps * f;
        l = l * keep + pl * f;
        m = to;
    }
    s_sum[tid] = sum;
    s_m[tid] = m;
    s_l[tid] = l;
    __syncthreads();
    if (group != 0 || !on || n <= sp.chunk) return;
    for (int g = 1; g < groups; ++g) {
        const int from = tid + (g << kLaneBits);
        const float to = fmaxf(m, s_m[from]), keep = weight<T>(m, to), f = weight<T>(s_m[from], to);
        sum = sum * keep + s_sum[from] * f;
        l = l * keep + s_l[from] * f;
        m = to;
    }
    store_out<T>(a, b, h, row, d, sum, l);
}

namespace {

struct Plan {
    int64_t chunk, chunks, q_tiles, held;
    bool together;
};

// How a call is cut into workgroups over `chunk` keys. (Device times below: 16
// query heads of 128 over 8 in float16 unless they say otherwise.)
// A row of up to kWholeBytes of keys and values is one workgroup, and the call
// one launch: a CU alone takes in 384 KB in the time of the second launch (one
// token over 1500 keys, 12 heads of 64: 8.7 us against 7.6 in two launches, but
// 9.7 against 12.3 as a program calls it; 16 x 500 keys 10.4, 12.2 cut in four).
// A longer one takes longer alone (8 x 400..1500: 17.7 against 11.5), until there
// are rows enough to fill the card: from kFullUnits on, three workgroups to four
// CUs, up to kFullBytes are whole. Rows of one length gain from some 120 on, rows
// of all lengths from some 230 (whole and cut, us; eight rows a request):
//            2000 keys each   5..2000 keys   1200 each
//    64        23.1  17.9      21.4  15.2    15.4  12.1
//   128        26.1  26.0      23.0  20.5    17.3  18.3
//   192        31.8  35.5      24.6  23.1    20.6  24.9
//   256        41.1  45.1      27.3  27.1    26.1  29.1
//   512        79.3  85.7      46.1  47.0    49.5  53.7
// (the same in float32 and over heads of 64; 320 equal rows, one and a quarter a
// CU, are the exception: 60.1 and 56.1.)
// Then kMany workgroups (the card holds 768 at a time: requests end at different
// keys, and pieces even that out; 32 x 500..16384 177 us, 182 with 3072) of
// kLeast keys or more (8 x 400..1500 11.5 us, 13.5 with 256; 100 x 100..4000 of
// two heads 44.5, 46.7), and at least kFew of them, one per CU (8 x 400..1500
// 13.6 us with 512, 1 x 8192 13.4 against 12.0).
constexpr int64_t kWholeBytes = 512 << 10, kFullBytes = 1 << 20, kMany = 4096, kLeast = 384, kFew = 256,
                  kFullUnits = 192;
Plan plan(int64_t batch, int64_t kv_heads, int64_t rows, int64_t max_len, int head_dim, int dtype) {
    Plan p;
    p.q_tiles = (rows + kQ - 1) / kQ;
    p.held = rows < kQ ? rows : kQ;
    const int64_t units = batch * kv_heads * p.q_tiles, step = kWaves * 32;
    const int64_t keys = (max_len + step - 1) / step * step;
    int64_t chunk = keys;
    const int64_t whole = (units < kFullUnits ? kWholeBytes : kFullBytes) / (2 * head_dim * (dtype == 1 ? 2 : 4));
    if (max_len > whole) {
        // (in float64: requests x heads x rows x keys may pass 64 bits)
        const double all = (double)units * (double)keys;
        chunk = all / kMany < (double)keys ? (int64_t)(all / kMany) : keys;
        if (chunk < kLeast) chunk = kLeast;
        if (units * ((keys + chunk - 1) / chunk) < kFew) chunk = (int64_t)(all / kFew);
    }
    if (chunk < step) chunk = step;
    chunk = (chunk + step - 1) / step * step;
    p.chunk = chunk < keys ? chunk : keys > step ? keys : step;
    p.chunks = keys > 0 ? (keys + p.chunk - 1) / p.chunk : 1;
    // Rows of tiles of the same keys one after another on one XCD where the keys
    // and values pass half the last-level cache (256 MB), in which the next rows
    // would find them: 62 float32 rows of 64 requests over 1500 keys 207 us
    // against 429, 40 heads of 128 over 2, 300 x 10..2000 keys, 82 against 105;
    // but 20 float16 rows of 16 requests (74 MB) 24.8 against 23.1.
    const double bytes = 2.0 * batch * kv_heads * max_len * head_dim * (dtype == 1 ? 2 : 4);
    p.together = p.q_tiles > 1 && bytes > 128e6 && batch * kv_heads >= 64 && batch * kv_heads <= 65536 * kXcds;
    return p;
}

template <typename T, int D, bool PAGED, bool STREAM>
void launch_rows(const AttnArgs &a, const AttnSplit &sp, const Plan &p, hipStream_t st) {
    const unsigned groups = (unsigned)(((int64_t)a.batch * a.kv_heads + kXcds - 1) / kXcds);
    const dim3 grid = p.together ? dim3((unsigned)(kXcds * p.q_tiles), groups, (unsigned)p.chunks)
                                 : dim3(a.kv_heads, a.batch, (unsigned)(p.q_tiles * p.chunks));
    // Where the card is full (768 workgroups of four waves), one or two waves where
    // there can be no more tiles: 2000 requests of 1..40 keys, 12 heads of 64, 44 us,
    // 65 with four; with fewer workgroups four end sooner (16 rows of 64 requests
    // over 30 keys 5.0 us, 5.7 with one).
    const int tiles = (sp.chunk < a.max_len ? sp.chunk : a.max_len) / TileShape<T, D>::kKeys + 1;
    const bool few = PAGED && tiles <= 2 && (int64_t)grid.x * grid.y * grid.z > 768;
    const int waves = few ? tiles : kWaves;
    const size_t join = (size_t)waves * sp.held * (D + 4) * sizeof(float);
    const size_t keys = (size_t)waves * TileShape<T, D>::kTileBytes, lds = join > keys ? join : keys;
    if (few) attn_kernel<T, D, PAGED, STREAM, PAGED><<<grid, 64 * waves, lds, st>>>(a, sp);
    else attn_kernel<T, D, PAGED, STREAM, false><<<grid, 64 * waves, lds, st>>>(a, sp);
}

template <typename T, int D>
hipError_t launch(const AttnArgs &a, const AttnSplit &sp, const Plan &p, hipStream_t st) {
    // Caches that the L2 (32 MB in all) cannot hold are read past it: requests of
    // 8192 keys each, 1.1 GB, at 6.5 TB/s instead of 5.7 (6.3 for 500..16384 keys),
    // one token of 256 requests over 1500 states (12 heads of 64) 188 us instead of
    // 207; smaller ones may stay there for the next call, and states that the
    // requests share for the next request.
    const double bytes = 2.0 * a.batch * a.kv_heads * a.max_len * D * sizeof(T);
    const bool stream = sp.q_tiles == 1 && bytes > 32e6 && a.k_batch != 0;
    if (a.table && stream) launch_rows<T, D, true, true>(a, sp, p, st);
    else if (a.table) launch_rows<T, D, true, false>(a, sp, p, st);
    else if (stream) launch_rows<T, D, false, true>(a, sp, p, st);
    else launch_rows<T, D, false, false>(a, sp, p, st);
    if (sp.chunks > 1) {
        // a group of lanes per chunk of the row, as far as a workgroup goes
        int shift = 0;
        while ((1 << shift) < sp.chunks && (D / 4) << shift < kJoin) ++shift;
        const int per = kJoin / (D / 4) >> shift;   // rows per workgroup
        const dim3 grid(a.kv_heads, a.batch, (unsigned)((a.rows + per - 1) / per));
        attn_join_kernel<T, D><<<grid, kJoin, 0, st>>>(a, sp, shift);
    }
    return hipGetLastError();
}

}  // namespace

int64_t attn_workspace_bytes(int64_t batch, int64_t kv_heads, int64_t rows, int64_t max_len, int head_dim,
                             int dtype) {
    const Plan p = plan(batch, kv_heads, rows, max_len, head_dim, dtype);
    return p.chunks > 1 ? batch * kv_heads * rows * p.chunks * (head_dim + 2) * 4 : 0;
}

bool attn_fits(int64_t batch, int64_t kv_heads, int64_t rows, int64_t max_len, int head_dim, int dtype) {
    // a launch's grid: threads of x in 32 bits, 65536 workgroups in y and z
    const Plan p = plan(batch, kv_heads, rows, max_len, head_dim, dtype);
    if (batch == 0 || rows == 0) return true;
    if (kv_heads > (1 << 22) - 1 || batch > 65536 || p.q_tiles > 65536 || p.q_tiles * p.chunks > 65536) return false;
    return p.chunks == 1 || rows <= 65536;
}

hipError_t launch_attn(const AttnArgs &a, int head_dim, int dtype, void *workspace, hipStream_t st) {
    Plan p = plan(a.batch, a.kv_heads, a.rows, a.max_len, head_dim, dtype);
    if (!workspace && p.chunks > 1) {
        p.chunk = (a.max_len + 31) / 32 * 32;
        p.chunks = 1;
    }
    AttnSplit sp{};
    sp.chunk = (int32_t)p.chunk;
    sp.chunks = (int32_t)p.chunks;
    sp.q_tiles = (int32_t)p.q_tiles;
    sp.held = (int32_t)p.held;
    sp.together = p.together;
    sp.page_magic = a.table ? (uint32_t)(((1ull << 32) + a.page / 16 - 1) / (a.page / 16)) : 0;
    if (p.chunks > 1) {
        sp.sums = static_cast<float *>(workspace);
        sp.stats = sp.sums + (int64_t)a.batch * a.kv_heads * a.rows * p.chunks * head_dim;
    }
    AttnArgs c = a;
    // (no key past the table's width is valid)
    if (a.table && c.max_len > (int64_t)a.table_width * a.page) c.max_len = a.table_width * a.page;
    if (dtype == 1)
        return head_dim == 128 ? launch<_Float16, 128>(c, sp, p, st) : launch<_Float16, 64>(c, sp, p, st);
    return head_dim == 128 ? launch<float, 128>(c, sp, p, st) : launch<float, 64>(c, sp, p, st);
}

}  // namespace mnb
