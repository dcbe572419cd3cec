// Attention over the 8-bit cache: o = sum_t w_t vs_t cv_t / sum_t w_t, w_t =
// exp(s_t - m), s_t = scale * ks_t * (q . ck_t), codes ck, cv and scales ks, vs,
// m the running maximum.
//
// Both products are whole numbers. A query row is held as its largest element's
// power of two times whole numbers below 2^23, these as three digits of 8 bits;
// a tile's weights w_t vs_t as the power of two of the tile's largest times such
// numbers, in three digits as well. So codes enter the matrix unit as they are
// stored, nothing is rounded between the digits and the 32-bit sums, and float16
// and float32 calls differ in their first loads and last stores alone.
//
// Work: a row of tiles is up to 16 query rows of one (request, key-value head);
// its keys are cut into chunks, and a chunk's tiles of 64 keys are taken in turn
// by the waves of one workgroup, codes through a place of the wave's own in LDS:
//   S^T = CK Q^T  A = codes (lane: key l % 16, 16 bytes of its row), B = a digit of
//                 the queries; per lane four keys 4 (l / 16) + i of one query
//                 l % 16, for each of the tile's four 16-key parts
//   O^T = CV^T P^T  contraction over those 64 keys: a digit of the weights is the
//                 lane's own 16 bytes, packed by byte permutes; A's rows are
//                 dimensions, which come out of LDS through the transposing
//                 8-byte reads.
// The next tile's key codes are requested as soon as this one's are in registers,
// its value codes after the second product's reads.
// The waves' sums are joined in LDS, and the chunks' by a second launch.
//
// Bound by the latency of a tile's steps (two products, their exchange and the softmax
// between) where workgroups are few, by the vector unit and the codes' way through LDS where
// they are many: 16 rows over 32 x 1000 keys of 8 heads of 128 16.4 us, 4.1 TB/s of codes
// and scales, 8 rows over 32 x 8000 111 us, 4.9 TB/s (a stream of reads reaches 6.8). Many
// float32 rows are taken 16 at a time as well, each tile with codes of its own: 16 prompts of
// 410 rows, 16 heads of 128 over 8, 119 us, 8 x 62 rows after up to 2000 keys 36.
#include "mnb_attn8_tiles.h"

#include <algorithm>

namespace mnb {

namespace {

constexpr int kWaves = 4;
constexpr int kQ = 16;       // query rows per row of tiles

}  // namespace

template <typename T, int D, bool STREAM>
__device__ __forceinline__ void attn8_workgroup(const Attn8Args &a, const Attn8Split &sp) {
    using Tile = CodeTile<D, STREAM>;
    constexpr int kLoads = Tile::kLoads, kTile = Tile::kBytes;
    constexpr int kOut = D / 16;        // 16-dimension parts of the output
    constexpr int kBehind = kParts + Tile::kCodeLoads;   // loads of a tile's scales and codes, keys or values
    // the waves' tiles of key and value codes (arrays of their own: the compiler then
    // knows that reads of one need not wait for loads into the other); in the end their
    // sums [kWaves][kQ][D], and maxima and weights' sums [kWaves][kQ]
    __shared__ __attribute__((aligned(16))) uint8_t s_keys[kWaves][kTile], s_values[kWaves][kTile];
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int col = lane & 15, g = lane >> 4;
    const int h = blockIdx.x, chunk = blockIdx.z / sp.q_tiles, q_tile = blockIdx.z - chunk * sp.q_tiles;
    const int64_t b = blockIdx.y;
    const Cache8 &c = a.cache;
    const int begin = chunk * sp.chunk, step = kWaves * kKeys;
    int key = begin + wave * kKeys;
    // (everything that waits for nothing is requested first)
    Tile tile(a, sp, b, lane, s_keys[wave], s_values[wave]);
    tile.look_up(key);
    int64_t first;
    const int n_new = rows_of(a, b, first);
    const int row0 = q_tile * kQ;
    int rows = (n_new < a.max_new ? n_new : a.max_new) * a.group - row0;
    if (rows <= 0) return;
    if (rows > kQ) rows = kQ;
    const int r = row0 + (col < rows ? col : 0), token = token_of(a, r);
    QueryRow<T, D> row;
    row.load(static_cast<const T *>(a.q) + (first + token) * a.q_stride +
             ((int64_t)h * a.group + r - token * a.group) * D + g * 16);
    // (no kernel writes the lengths while this one reads them: a scalar load)
    typedef __attribute__((address_space(4))) const int32_t entry;
    const int len = ((entry *)a.lens)[b];
    // keys that the tile's rows see: the last row most, the first least
    const int n = sees(a, len, n_new, token_of(a, row0 + rows - 1)), least = sees(a, len, n_new, token_of(a, row0));
    if (begin >= n && chunk > 0) return;
    const int end = n - begin < sp.chunk ? n : begin + sp.chunk;
    const int mine = sees(a, len, n_new, token);
    tile.end = end;

    const int8_t *keys = c.k + h * c.head_stride, *values = c.v + h * c.head_stride;
    const float *key_scales = c.k_scale + h * c.scale_head, *value_scales = c.v_scale + h * c.scale_head;
    auto load_scales = [&](const float *base, f4 *to) {
#pragma unroll
        for (int s = 0; s < kParts; ++s)
            to[s] = __builtin_bit_cast(
                f4, __builtin_amdgcn_raw_buffer_load_b128(tile.buffer(base, tile.from_scales, s, 64u), g * 16, 0, 0));
    };

    f4 o[kOut];
#pragma unroll
    for (int i = 0; i < kOut; ++i) o[i] = f4{0.0f, 0.0f, 0.0f, 0.0f};
    float m = kLowest, l = 0.0f;
    f4 ks[kParts], vs[kParts];
    // Requests a tile's keys (and the next one's table entries), its values.
    uint32_t there;
    auto request_keys = [&](int key0) {
        tile.locate(key0);
        load_scales(key_scales, ks);
        tile.load_codes(keys, s_keys[wave]);
        tile.look_up(key0 + step);
        asm volatile("" ::: "memory");   // (in this order: the waits count them)
    };
    auto request_values = [&]() {
        load_scales(value_scales, vs);
        tile.load_codes(values, s_values[wave]);
        there = tile.there;
        asm volatile("" ::: "memory");
    };
    request_keys(key);
    request_values();
    i32x4 q[kLoads][3];   // in digits: lane (query col, pieces 4 j + g)
    float mul;
    int exponent;
    row.digits(a.scale, q, mul, exponent);
    for (; key < end; key += step) {
        float x[kParts][4];
        {
            // (this tile's key codes are in LDS when all but its values' loads have come back)
            i32x4 kk[kParts][kLoads];
            tile.template read_keys<kBehind>(kk);
#pragma unroll
            for (int s = 0; s < kParts; ++s) {
                i32x4 lo = {0, 0, 0, 0}, hi = {0, 0, 0, 0};
#pragma unroll
                for (int j = 0; j < kLoads; ++j) {
                    lo = mma64(kk[s][j], q[j][0], lo);
                    hi = mma64(kk[s][j], q[j][2], hi);
                }
                // (up to 2^21 * 2^8: the two upper digits in one number)
                hi = hi << 8;
#pragma unroll
                for (int j = 0; j < kLoads; ++j) hi = mma64(kk[s][j], q[j][1], hi);
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    x[s][i] = __builtin_fmaf((float)hi[i], 256.0f, (float)lo[i]) * score_step(ks[s][i], mul, exponent);
            }
        }
        // (past the last tile loads of no bytes are requested: with a way around them the
        // compiler counts none, and waits too long for those before)
        request_keys(key + step);
        {
            if (key + kKeys > least || there != (1u << kParts) - 1)   // uniform: the end of a row, or a missing block
#pragma unroll
                for (int s = 0; s < kParts; ++s) {
                    const int left = there >> s & 1 ? mine - key - 16 * s - 4 * g : 0;
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        x[s][i] = i < left ? x[s][i] : -__builtin_inff();
                        vs[s][i] = i < left ? vs[s][i] : 0.0f;
                    }
                }
            float top = x[0][0];
#pragma unroll
            for (int s = 0; s < kParts; ++s)
#pragma unroll
                for (int i = 0; i < 4; ++i) top = fmaxf(top, x[s][i]);
            top = column_max(top);
            if (__any(top > m)) {
                const float to = fmaxf(m, top), keep = weight(m, to);
                m = to;
                l *= keep;
#pragma unroll
                for (int i = 0; i < kOut; ++i) o[i] *= keep;
            }
            // weights times value scales, and the largest of the tile (as whole numbers:
            // they are not negative, and NaN is above all)
            uint32_t most = 0;
#pragma unroll
            for (int s = 0; s < kParts; ++s)
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const float w = weight(x[s][i], m);
                    l += w;
                    x[s][i] = w * vs[s][i];
                    const uint32_t bits = as_bits(x[s][i]) & 0x7FFFFFFFu;
                    most = bits > most ? bits : most;
                }
            most = column_max(most);
            float up, down;
            weight_steps(most, up, down);
            i32x4 p[3];
#pragma unroll
            for (int s = 0; s < kParts; ++s) {
                uint32_t w[4], digit[3];
#pragma unroll
                for (int i = 0; i < 4; ++i) w[i] = as_bits(__builtin_fmaf(x[s][i], up, kDigits));
                digits_of(w, digit);
#pragma unroll
                for (int t = 0; t < 3; ++t) p[t][s] = (int)digit[t];
            }
            // this tile's value codes are in LDS: all but the next keys' loads, and the entry's
            wait_loads<kBehind + 1>();
#pragma unroll
            for (int d = 0; d < kOut; d += 4) {
                i32x2 v[4][2];
                tile.template read_values<false>(v, d);
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    const i32x4 zero = {0, 0, 0, 0}, vv = {v[k][0].x, v[k][0].y, v[k][1].x, v[k][1].y};
                    const i32x4 lo = mma64(vv, p[0], zero), hi = mma64(vv, p[1], mma64(vv, p[2], zero) << 8);
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        o[d + k][i] =
                            __builtin_fmaf(__builtin_fmaf((float)hi[i], 256.0f, (float)lo[i]), down, o[d + k][i]);
                }
            }
        }
        request_values();
    }

    // (the tile past the end, no bytes, has arrived everywhere: its place is free)
    wait_loads<0>();
    __syncthreads();

    // join the waves (those that have keys)
    static_assert(sizeof(s_keys) == kWaves * kQ * D * sizeof(float), "the waves' sums take the key tiles' place");
    float *s_m = reinterpret_cast<float *>(s_values), *s_l = s_m + kWaves * kQ;
    // (four dimensions 4 p of a row; rows turned against one another in the banks)
    auto sums = [&](int wave, int row, int p) {
        return reinterpret_cast<f4 *>(s_keys) + (wave * kQ + row) * (D / 4) + (p ^ (row & 7));
    };
    const int tiles = n <= kKeys ? 1 : (end - begin + kKeys - 1) / kKeys;
    const int waves = tiles < kWaves ? tiles : kWaves;
    if (wave < waves) {
        l += __shfl_xor(l, 16);
        l += __shfl_xor(l, 32);
        if (g == 0) {
            s_m[wave * kQ + col] = m;
            s_l[wave * kQ + col] = l;
        }
#pragma unroll
        for (int d = 0; d < kOut; ++d) *sums(wave, col, 4 * d + g) = o[d];
    }
    __syncthreads();
    const bool whole = n <= sp.chunk;   // this chunk is the rows' only one
    for (int e = threadIdx.x; e < rows * (D / 4); e += 64 * kWaves) {
        const int i = e / (D / 4), p = e % (D / 4);
        float top = s_m[i];
        for (int w = 1; w < waves; ++w) top = fmaxf(top, s_m[w * kQ + i]);
        f4 sum = {0.0f, 0.0f, 0.0f, 0.0f};
        float total = 0.0f;
        for (int w = 0; w < waves; ++w) {
            const float f = weight(s_m[w * kQ + i], top);
            sum += *sums(w, i, p) * f;
            total += s_l[w * kQ + i] * f;
        }
        if (whole) {
            store_out<T, D>(a, first, h, row0 + i, 4 * p, sum, total);
        } else {
            const int64_t piece = ((b * c.heads + h) * sp.rows + row0 + i) * sp.chunks + chunk;
            *reinterpret_cast<f4 *>(sp.sums + piece * D + 4 * p) = sum;
            if (p == 0) {
                sp.stats[2 * piece] = top;
                sp.stats[2 * piece + 1] = total;
            }
        }
    }
}

template <typename T, int D, bool STREAM>
__global__ __launch_bounds__(64 * kWaves, 2) void attn8_kernel(Attn8Args a, Attn8Split sp) {
    attn8_workgroup<T, D, STREAM>(a, sp);
}

// Joins the chunks of query rows, in a fixed order: a row has 2^shift groups of
// D / 4 lanes, which take every 2^shift-th chunk; then their sums are added.
constexpr int kJoin = 256;
constexpr int64_t kJoinLanes = 1 << 18;
template <typename T, int D, bool LOG2>
__global__ __launch_bounds__(kJoin) void attn8_join_kernel(Attn8Args a, Attn8Split sp, int shift) {
    constexpr int kLanes = D / 4, kLaneBits = D == 128 ? 5 : 4;
    auto weight = [](float x, float m) { return __builtin_amdgcn_exp2f(LOG2 ? x - m : (x - m) * kLog2e); };
    __shared__ f4 s_sum[kJoin];
    __shared__ float s_m[kJoin], s_l[kJoin];
    const int tid = threadIdx.x, d = tid % kLanes * 4, groups = 1 << shift;
    const int group = (tid >> kLaneBits) & (groups - 1);
    const int row = blockIdx.z * (kJoin >> (kLaneBits + shift)) + (tid >> (kLaneBits + shift));
    const int h = blockIdx.x;
    const int64_t b = blockIdx.y;
    int64_t first;
    const int len = a.lens[b], n_new = rows_of(a, b, first);
    const int rows = (n_new < a.max_new ? n_new : a.max_new) * a.group;
    const bool on = row < rows;
    // the keys of the row's tile: its last row's
    int last = (int)((uint32_t)row / (uint32_t)sp.tile + 1) * sp.tile - 1;
    last = last < rows ? last : rows - 1;
    const int n = on ? sees(a, len, n_new, token_of(a, last)) : 0;
    const int64_t from_piece = ((b * a.cache.heads + h) * sp.rows + (on ? row : 0)) * sp.chunks;
    f4 sum = {0.0f, 0.0f, 0.0f, 0.0f};
    float m = kLowest, l = 0.0f;
    for (int k = group; k < sp.chunks && k * sp.chunk < n; k += groups) {
        const float *stats = sp.stats + 2 * (from_piece + k);
        const float pm = stats[0], pl = stats[1];
        const f4 ps = *reinterpret_cast<const f4 *>(sp.sums + (from_piece + k) * D + d);
        const float to = fmaxf(m, pm), keep = weight(m, to), f = weight(pm, to);
        sum = sum * keep + ps * f;
        l = l * keep + pl * f;
        m = to;
    }
    s_sum[tid] = sum;
    s_m[tid] = m;
    s_l[tid] = l;
    __syncthreads();
    if (group != 0 || !on || n <= sp.chunk) return;
    for (int k = 1; k < groups; ++k) {
        const int other = tid + (k << kLaneBits);
        const float to = fmaxf(m, s_m[other]), keep = weight(m, to), f = weight(s_m[other], to);
        sum = sum * keep + s_sum[other] * f;
        l = l * keep + s_l[other] * f;
        m = to;
    }
    store_out<T, D>(a, first, h, row, d, sum, l);
}

namespace {

struct Plan {
    int64_t chunk, chunks, rows, q_tiles, tile;
    bool many;
};

// Which kernel, and how a call is cut into workgroups over `chunk` keys. Figures are us
// a call, replayed from a graph; 8 heads of 128 are shared by 16, 8 of 64 by 32.
//
// Few rows: a row whole is one workgroup, and the call one launch. Whole it takes as long
// as its longest row; cut, as long as the CUs' share of all rows, and the join. So it
// stays whole while what the longest row has over a CU's share, for rows of max_len each,
// is no more than the join costs: kJoinBytes of codes for up to kFewRows rows (64
// dimensions, 12 float32 heads: 4 requests of 1500 keys 9.1 us, cut 9.1, of 3000 12.7 and
// 9.9; 8 of 1500 9.4 and 9.9, of 3000 13.7 and 12.1; 16 of 3000 15.5 and 16.5; one of 3000
// and 2 heads 12.2 and 8.8), kTileJoinBytes for tiles of 16, whose workgroups need longer a
// byte (8 heads of 128 shared by 64: 12 requests of 700 keys 12.0 and 11.9, of 1100 16.6 and
// 13.7, 24 of 1100 17.3 and 18.2). 96 and 160 KB for the first are 0.3% and 0.1% slower in
// the mean of 2004 calls of 1..128 requests of up to 520..8000 keys, 32 and 64 KB for the
// second the same and 0.3% of 750; the better side of each call would be 0.8% and 1.1% faster
// (longest rows among short ones, which the call does not know, are the worst: 320 rows of
// tiles of 5..8000 keys 62 whole and 44 cut). Past kFullBytes rows are cut (24 x 16000, 12 x
// 64, 77 cut and 98 whole).
// Longer rows: kMany workgroups (16 x 16000, 8 x 128: 73, with 4096 80; with 1024 the same
// 0.1% over 372 calls, 20% worse at the worst) of kLeast keys or more (512 1% slower over
// those calls, 16 x 3000 22.7 for 18.2; 1024 0.3%), and at least kCus of them (1 x 6000 9.8,
// with 128 11.1; 1 x 16000 with 512 13.1 for 11.8).
//
// Many rows: from kManyRows on, three tiles of this file's kernel, which the other form
// takes as one: 64 requests of 40 rows after 300 keys 26 and 37, of 64 rows 30 and 49; 32
// rows 25 and 28, but 32 of those after 1000 keys 39 and 25. (The border moves with the work:
// calls of few workgroups go on losing by the other form up to some 100 rows, 8 x 500 keys
// 64 rows 17.7 and 12.9. By the tiles of 16 rows, all requests and heads together, times
// max_len head_dim / 128 + 500, above half a million, 5814 calls of 20..410 rows would be
// 2% behind the better form in the mean, by the constant they are 11%.) kManyWgs workgroups
// of kManyKeys keys or more (8 x 8000 keys, 124 rows: 74, with 256 85, with 1024 76), and
// where those are too few kFullWgs of kLeastKeys or more (1 x 2000, 124 rows: 15.6, in
// pieces of 256 18.9; 1 x 410 new 15.7 and 18.7); up to kManyKeys keys are one piece (2 x 200
// new 14.0, in two 14.6).
constexpr int64_t kCus = 256, kJoinBytes = 128 << 10, kTileJoinBytes = 48 << 10, kFullBytes = 1 << 20, kMany = 2048,
                  kLeast = 768, kManyWgs = 512, kManyKeys = 256, kFullWgs = 256, kLeastKeys = 128, kManyRows = 33;

// Whether rows of max_len keys of few query rows stay whole, `units` of them.
bool whole_rows(int64_t rows, int64_t units, int64_t max_len, int head_dim) {
    const int64_t bytes = 2 * max_len * head_dim, join = rows <= kFewRows ? kJoinBytes : kTileJoinBytes;
    return bytes <= kFullBytes && bytes * (kCus - std::min(units, kCus)) <= join * kCus;
}

Plan plan(int64_t batch, int64_t kv_heads, int64_t group, int64_t max_new, int64_t max_len, int head_dim, int dtype) {
    Plan p;
    p.rows = max_new * group;
    p.many = dtype == 1 && p.rows >= kManyRows;
    p.tile = p.many ? kRowTile : kQ;
    p.q_tiles = (p.rows + p.tile - 1) / p.tile;
    const int64_t units = batch * kv_heads * p.q_tiles, step = p.many ? 64 : kWaves * kKeys;
    const int64_t keys = (max_len + step - 1) / step * step;
    int64_t chunk = keys;
    // (in float64: requests x heads x rows x keys may pass 64 bits)
    const double all = (double)units * (double)keys;
    if (p.many) {
        if (all / kManyWgs < (double)keys) chunk = (int64_t)(all / kManyWgs);
        if (chunk < kManyKeys && keys > kManyKeys) chunk = std::max((int64_t)(all / kFullWgs), kLeastKeys);
    } else if (!whole_rows(p.rows, units, max_len, head_dim)) {
        chunk = all / kMany < (double)keys ? (int64_t)(all / kMany) : keys;
        if (chunk < kLeast) chunk = kLeast;
        if (units * ((keys + chunk - 1) / chunk) < kCus) chunk = (int64_t)(all / kCus);
    }
    if (chunk < step) chunk = step;
    chunk = (chunk + step - 1) / step * step;
    p.chunk = chunk < keys ? chunk : keys > step ? keys : step;
    p.chunks = keys > 0 ? (keys + p.chunk - 1) / p.chunk : 1;
    return p;
}

template <typename T, int D> void launch_some(const Attn8Args &a, const Attn8Split &sp, bool stream, hipStream_t st) {
    const dim3 grid(a.cache.heads, a.batch, (unsigned)(sp.q_tiles * sp.chunks));
    if (stream) attn8_kernel<T, D, true><<<grid, 64 * kWaves, 0, st>>>(a, sp);
    else attn8_kernel<T, D, false><<<grid, 64 * kWaves, 0, st>>>(a, sp);
}

template <typename T, int D, bool LOG2> void launch_join(const Attn8Args &a, const Attn8Split &sp, hipStream_t st) {
    const int64_t rows = (a.tokens < a.max_new ? a.tokens : a.max_new) * a.group;
    // a group of lanes per chunk of the row, as far as a workgroup goes and rows do not
    // fill the card by themselves (a call over 1 x 32000 keys 16.3 us, by one group a row
    // 22.6; 8 x 62 rows after up to 2000 keys 30.5, by a group per chunk 32.5)
    const int64_t lanes = (int64_t)a.batch * a.cache.heads * rows * (D / 4);
    int shift = 0;
    while ((1 << shift) < sp.chunks && (D / 4) << shift < kJoin && lanes << shift < kJoinLanes) ++shift;
    const int64_t per = kJoin / (D / 4) >> shift;   // rows per workgroup
    const dim3 grid(a.cache.heads, a.batch, (unsigned)((rows + per - 1) / per));
    attn8_join_kernel<T, D, LOG2><<<grid, kJoin, 0, st>>>(a, sp, shift);
}

template <typename T, int D> hipError_t launch(const Attn8Args &a, const Attn8Split &sp, bool many, hipStream_t st) {
    if constexpr (sizeof(T) == 2) {
        if (many) {
            if (hipError_t e = launch_attn8_rows(a, sp, D, st)) return e;
            if (sp.chunks > 1) launch_join<T, D, true>(a, sp, st);
            return hipGetLastError();
        }
    }
    // Codes that the L2 (32 MB in all) cannot hold are read past it: 32 x 1000 keys, 66 MB,
    // 12.5 us and 14.7 without, 1 GB 132 and 148 (33 MB 8.4 and 8.2).
    const bool stream = sp.q_tiles == 1 && 2.0 * a.batch * a.cache.heads * a.max_len * D > 32e6;
    if (sp.rows <= kFewRows) {
        if (hipError_t e = launch_attn8_few(a, sp, D, sizeof(T) == 2 ? 1 : 0, stream, st)) return e;
    } else {
        launch_some<T, D>(a, sp, stream, st);
    }
    if (sp.chunks > 1) launch_join<T, D, false>(a, sp, st);
    return hipGetLastError();
}

}  // namespace

int64_t attn8_workspace_bytes(int64_t batch, int64_t kv_heads, int64_t group, int64_t max_new, int64_t max_len,
                              int head_dim, int dtype) {
    const Plan p = plan(batch, kv_heads, group, max_new, max_len, head_dim, dtype);
    return p.chunks > 1 ? batch * kv_heads * p.rows * p.chunks * (head_dim + 2) * 4 : 0;
}

bool attn8_fits(int64_t batch, int64_t kv_heads, int64_t group, int64_t max_new, int64_t max_len, int head_dim,
                int dtype) {
    // a launch's grid: threads of x in 32 bits, 65536 workgroups in y and z
    if (batch == 0) return true;
    const Plan p = plan(batch, kv_heads, group, max_new, max_len, head_dim, dtype);
    if (kv_heads > (1 << 22) - 1 || batch > 65536 || p.q_tiles > 65535 || p.q_tiles * p.chunks > 65535) return false;
    return p.chunks == 1 || p.rows <= 65535;
}

hipError_t launch_attn8(const Attn8Args &a, int head_dim, int dtype, void *workspace, hipStream_t st) {
    const Plan p = plan(a.batch, a.cache.heads, a.group, a.max_new, a.max_len, head_dim, dtype);
    Attn8Split sp{};
    sp.chunk = (int32_t)p.chunk;
    sp.chunks = (int32_t)p.chunks;
    sp.rows = (int32_t)p.rows;
    sp.tile = (int32_t)p.tile;
    // (no more tiles of rows than the tokens at hand can fill)
    const int64_t rows = (a.tokens < a.max_new ? a.tokens : a.max_new) * a.group;
    sp.q_tiles = (int32_t)((rows + p.tile - 1) / p.tile);
    const int32_t parts = a.cache.page / 16;
    sp.page_magic = parts == 1 ? 0 : (uint32_t)(((1ull << 32) + parts - 1) / parts);
    if (p.chunks > 1) {
        sp.sums = static_cast<float *>(workspace);
        sp.stats = sp.sums + (int64_t)a.batch * a.cache.heads * p.rows * p.chunks * head_dim;
    }
    Attn8Args c = a;
    c.per_group = 1.0f / (float)a.group;
    // (no key past the table's width is seen)
    if (c.max_len > (int64_t)a.table_width * a.cache.page) c.max_len = a.table_width * a.cache.page;
    if (dtype == 1)
        return head_dim == 128 ? launch<_Float16, 128>(c, sp, p.many, st) : launch<_Float16, 64>(c, sp, p.many, st);
    return head_dim == 128 ? launch<float, 128>(c, sp, p.many, st) : launch<float, 64>(c, sp, p.many, st);
}

}  // namespace mnb
