// Attention of one or two query rows of a (request, key-value head) over the 8-bit
// cache: the single tokens of a decoding step whose heads share keys by no more than
// two. The same whole numbers as in mnb_attn8.hip, but for the digits' place: here
// a row's three digits are three columns of one product, so that a tile takes a third
// of the products, and a score belongs to one lane, so that a tile takes a quarter of
// the vector instructions:
//   S^T = CK Q^T   column 3 r + t is digit t of row r; the products go through LDS, from
//                  where lane k takes the three of key k and row r: its score
//   softmax        a key a lane; maxima over the wave by lane permutes
//   O^T = CV^T P^T the weights' digits go through LDS to become the columns 3 r + t again,
//                  whose sums stay apart until the end.
//
// Long rows are bound by memory: 2 rows, 32 x 500..16384 keys of 8 heads of 128, 571 MB in
// 93..105 us, 5.4..6.1 TB/s (16 x 16 tiles of the other kernel took 116; a stream of reads
// reaches 6.8). One request of 452 keys takes 7.7 us, of one key 6.0: a launch, the chain
// of length, table, codes and scales, two products and the waves' join. Against that form
// (us replayed from a graph): 1 row, 8 x 1500 keys, 10.5 and 12.5; 2 rows 11.1 and 12.4,
// 32 x 16000 169 and 175; over 380 calls each 17% and 12% faster in the mean. (Of three to five
// rows it was 5% to 6% slower: 3 rows, 8 x 2000 keys, 13.7 and 12.8, 5 rows 13.8 and 13.2.)
#include "mnb_attn8_tiles.h"

namespace mnb {

namespace {

constexpr int kMost = 2;                     // rows
constexpr int kColumns = 3 * kMost;
constexpr int kScoreStride = kKeys + 4;      // of a column of products, in words: columns turned in the banks
constexpr int kDigitStride = kKeys + 16;     // of a column of digits, in bytes

// The largest over the wave, in every lane.
template <int N> __device__ __forceinline__ uint32_t turned(uint32_t x) {
    return (uint32_t)__builtin_amdgcn_update_dpp((int)x, (int)x, 0x120 + N, 0xF, 0xF, false);   // by N of 16 lanes
}
__device__ __forceinline__ uint32_t wave_max(uint32_t x) {
    x = column_max(x);
    uint32_t y;
    x = (y = turned<8>(x)) > x ? y : x;
    x = (y = turned<4>(x)) > x ? y : x;
    x = (y = turned<2>(x)) > x ? y : x;
    return (y = turned<1>(x)) > x ? y : x;
}
__device__ __forceinline__ float wave_max(float x) {
    x = column_max(x);
    x = fmaxf(x, as_float(turned<8>(as_bits(x))));
    x = fmaxf(x, as_float(turned<4>(as_bits(x))));
    x = fmaxf(x, as_float(turned<2>(as_bits(x))));
    return fmaxf(x, as_float(turned<1>(as_bits(x))));
}

}  // namespace

template <typename T, int D, bool STREAM, int R, int kWaves>
__device__ __forceinline__ void few_workgroup(const Attn8Args &a, const Attn8Split &sp) {
    using Tile = CodeTile<D, STREAM>;
    constexpr int kLoads = Tile::kLoads, kOut = D / 16;
    constexpr int kBehind = 1 + Tile::kCodeLoads;   // loads of a tile's value scales and codes
    // the waves' tiles of key and value codes, and what passes between lanes (arrays of
    // their own: the compiler then knows that reads of one need not wait for loads
    // into another); in the end their sums [kWaves][kColumns][D], maxima and weights'
    // sums [kWaves][kMost]
    __shared__ __attribute__((aligned(16))) uint8_t s_keys[kWaves][Tile::kBytes], s_values[kWaves][Tile::kBytes];
    __shared__ __attribute__((aligned(16))) int32_t s_pass[kWaves][kColumns * kScoreStride];
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int col = lane & 15, g = lane >> 4;
    const int h = blockIdx.x, chunk = blockIdx.z;
    const int64_t b = blockIdx.y;
    const Cache8 &c = a.cache;
    const int begin = chunk * sp.chunk, step = kWaves * kKeys;
    int key = begin + wave * kKeys;
    // (everything that waits for nothing is requested first)
    Tile tile(a, sp, b, lane, s_keys[wave], s_values[wave]);
    tile.look_up(key);
    int64_t first;
    const int n_new = rows_of(a, b, first);
    const int rows = (n_new < a.max_new ? n_new : a.max_new) * a.group;   // <= R
    if (rows <= 0) return;
    // this lane's column: row (the last one's for the columns behind), and its digit of it
    const int mine = col / 3, digit = col - 3 * mine, r = mine < rows ? mine : rows - 1, token = token_of(a, r);
    QueryRow<T, D> row;
    row.load(static_cast<const T *>(a.q) + (first + token) * a.q_stride +
             ((int64_t)h * a.group + r - token * a.group) * D + g * 16);
    // keys that the last row sees, most of all
    // (no kernel writes the lengths while this one reads them: a scalar load)
    typedef __attribute__((address_space(4))) const int32_t entry;
    const int len = ((entry *)a.lens)[b];
    const int n = sees(a, len, n_new, token_of(a, rows - 1));
    if (begin >= n && chunk > 0) return;
    const int end = n - begin < sp.chunk ? n : begin + sp.chunk;
    tile.end = end;

    const int8_t *keys = c.k + h * c.head_stride, *values = c.v + h * c.head_stride;
    const float *key_scales = c.k_scale + h * c.scale_head, *value_scales = c.v_scale + h * c.scale_head;
    // This lane's key's scale (of block 0 where there is no key: it is not used).
    auto load_scale = [&](const float *base) {
        return reinterpret_cast<const float *>(reinterpret_cast<const uint8_t *>(base) + tile.from_scales)[col];
    };
    int32_t *s_products = s_pass[wave];
    uint8_t *s_digits = reinterpret_cast<uint8_t *>(s_pass[wave]);
    static_assert(kColumns * kDigitStride <= sizeof(s_pass[0]), "the digits take the products' place");

    f4 o[kOut];   // of this lane's column
#pragma unroll
    for (int i = 0; i < kOut; ++i) o[i] = f4{0.0f, 0.0f, 0.0f, 0.0f};
    float m[R], l[R];   // maxima, of the wave; sums, of this lane's keys
#pragma unroll
    for (int i = 0; i < R; ++i) {
        m[i] = kLowest;
        l[i] = 0.0f;
    }
    // Requests a tile's keys (and the next one's table entries), its values.
    float ks, vs;
    uint32_t there;
    auto request_keys = [&](int key0) {
        tile.locate(key0);
        ks = load_scale(key_scales);
        tile.load_codes(keys, s_keys[wave]);
        tile.look_up(key0 + step);
        asm volatile("" ::: "memory");   // (in this order: the waits count them)
    };
    auto request_values = [&]() {
        vs = load_scale(value_scales);
        tile.load_codes(values, s_values[wave]);
        there = tile.there;
        asm volatile("" ::: "memory");
    };
    request_keys(key);
    request_values();
    i32x4 q[kLoads];
    float mul[R];
    int exponent[R];
    int seen[R];   // keys that each row sees
    {
        i32x4 all[kLoads][3];
        float m;
        int e;
        row.digits(a.scale, all, m, e);
#pragma unroll
        for (int j = 0; j < kLoads; ++j)
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const int d0 = all[j][0][k], d1 = all[j][1][k], d2 = all[j][2][k];
                q[j][k] = digit == 0 ? d0 : digit == 1 ? d1 : d2;
            }
#pragma unroll
        for (int i = 0; i < R; ++i) {
            mul[i] = as_float((uint32_t)__builtin_amdgcn_readlane((int)as_bits(m), 3 * i));
            exponent[i] = __builtin_amdgcn_readlane(e, 3 * i);
            seen[i] = i < rows ? sees(a, len, n_new, token_of(a, i)) : 0;
        }
    }
    for (; key < end; key += step) {
        float x[R];
        {
            // (this tile's key codes are in LDS when all but its values' loads have come back)
            i32x4 kk[kParts][kLoads];
            tile.template read_keys<kBehind>(kk);
            i32x4 p[kParts];
#pragma unroll
            for (int s = 0; s < kParts; ++s) {
                p[s] = i32x4{0, 0, 0, 0};
#pragma unroll
                for (int j = 0; j < kLoads; ++j) p[s] = mma64(kk[s][j], q[j], p[s]);
            }
            // (of part s: keys 16 s + 4 g + i of this column)
            if (col < 3 * R)
#pragma unroll
                for (int s = 0; s < kParts; ++s)
                    *reinterpret_cast<i32x4 *>(s_products + col * kScoreStride + 16 * s + 4 * g) = p[s];
            wave_fence();
#pragma unroll
            for (int i = 0; i < R; ++i) {
                const int32_t *p = s_products + 3 * i * kScoreStride + lane;
                const float sum = __builtin_fmaf(
                    __builtin_fmaf((float)p[2 * kScoreStride], 256.0f, (float)p[kScoreStride]), 256.0f, (float)p[0]);
                x[i] = sum * score_step(ks, mul[i], exponent[i]);
            }
            wave_fence();   // (the digits take the products' place)
        }
        // (past the last tile loads of no bytes are requested: with a way around them the
        // compiler counts none, and waits too long for those before)
        request_keys(key + step);
        {
            const int at = there >> g & 1 ? key + lane : 0x7FFFFFFF;
            float up[R], down[R], keep[R];
            uint32_t w[R];
            bool moved = false;
#pragma unroll
            for (int i = 0; i < R; ++i) {
                x[i] = at < seen[i] ? x[i] : -__builtin_inff();
                const float to = fmaxf(m[i], wave_max(x[i]));
                moved |= to > m[i];
                keep[i] = weight(m[i], to);
                m[i] = to;
                const float p = weight(x[i], to);
                l[i] = l[i] * keep[i] + p;
                // (as whole numbers: they are not negative, and NaN is above all)
                x[i] = at < seen[i] ? p * vs : 0.0f;
                weight_steps(wave_max(as_bits(x[i]) & 0x7FFFFFFFu), up[i], down[i]);
                w[i] = as_bits(__builtin_fmaf(x[i], up[i], kDigits)) ^ 0x8080u;
            }
#pragma unroll
            for (int i = 0; i < R; ++i)
#pragma unroll
                for (int t = 0; t < 3; ++t) s_digits[(3 * i + t) * kDigitStride + lane] = (uint8_t)(w[i] >> (8 * t));
            wave_fence();
            // this lane's column: its digits of keys 16 g on; what a step of its sums is
            // worth, and what its sums so far are
            const i32x4 p = *reinterpret_cast<const i32x4 *>(s_digits + (col < kColumns ? col : 0) * kDigitStride + 16 * g);
            wave_fence();   // (the next tile's products take the digits')
            float worth = down[0], kept = keep[0];
#pragma unroll
            for (int i = 1; i < R; ++i) {
                worth = mine == i ? down[i] : worth;
                kept = mine == i ? keep[i] : kept;
            }
            worth *= digit == 0 ? 1.0f : digit == 1 ? 256.0f : 65536.0f;
            if (moved) {   // (uniform)
#pragma unroll
                for (int i = 0; i < kOut; ++i) o[i] *= kept;
            }
            // this tile's value codes are in LDS: all but the next keys' loads, and the entries'
            wait_loads<1 + Tile::kCodeLoads + 1>();
#pragma unroll
            for (int d = 0; d < kOut; d += 4) {
                i32x2 v[4][2];
                tile.template read_values<true>(v, d);
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    const i32x4 zero = {0, 0, 0, 0}, vv = {v[k][0].x, v[k][0].y, v[k][1].x, v[k][1].y};
                    const i32x4 sum = mma64(vv, p, zero);
#pragma unroll
                    for (int i = 0; i < 4; ++i) o[d + k][i] = __builtin_fmaf((float)sum[i], worth, o[d + k][i]);
                }
            }
        }
        request_values();
    }

    // (the tile past the end, no bytes, has arrived everywhere: its place is free)
    wait_loads<0>();
    __syncthreads();

    // join the digits, and the waves (those that have keys)
    static_assert(sizeof(s_keys) >= kWaves * kColumns * D * sizeof(float), "the waves' sums take the key tiles' place");
    float *s_m = reinterpret_cast<float *>(s_values), *s_l = s_m + kWaves * kMost;
    // (four dimensions 4 p of a column; columns turned against one another in the banks)
    auto sums = [&](int wave, int column, int p) {
        return reinterpret_cast<f4 *>(s_keys) + (wave * kColumns + column) * (D / 4) + (p ^ (column & 7));
    };
    const int tiles = n <= kKeys ? 1 : (end - begin + kKeys - 1) / kKeys;
    const int waves = tiles < kWaves ? tiles : kWaves;
    if (wave < waves) {
#pragma unroll
        for (int i = 0; i < R; ++i) {
#pragma unroll
            for (int d = 1; d < 64; d <<= 1) l[i] += __shfl_xor(l[i], d);
            if (lane == 0) {
                s_m[wave * kMost + i] = m[i];
                s_l[wave * kMost + i] = l[i];
            }
        }
        if (col < 3 * R)
#pragma unroll
            for (int d = 0; d < kOut; ++d) *sums(wave, col, 4 * d + g) = o[d];
    }
    __syncthreads();
    const bool whole = n <= sp.chunk;   // this chunk is the rows' only one
    for (int e = threadIdx.x; e < rows * (D / 4); e += 64 * kWaves) {
        const int i = e / (D / 4), p = e % (D / 4);
        float top = s_m[i];
        for (int w = 1; w < waves; ++w) top = fmaxf(top, s_m[w * kMost + i]);
        f4 sum = {0.0f, 0.0f, 0.0f, 0.0f};
        float total = 0.0f;
        for (int w = 0; w < waves; ++w) {
            const float f = weight(s_m[w * kMost + i], top);
            sum += (*sums(w, 3 * i, p) + *sums(w, 3 * i + 1, p) + *sums(w, 3 * i + 2, p)) * f;
            total += s_l[w * kMost + i] * f;
        }
        if (whole) {
            store_out<T, D>(a, first, h, i, 4 * p, sum, total);
        } else {
            const int64_t piece = ((b * c.heads + h) * sp.rows + i) * sp.chunks + chunk;
            *reinterpret_cast<f4 *>(sp.sums + piece * D + 4 * p) = sum;
            if (p == 0) {
                sp.stats[2 * piece] = top;
                sp.stats[2 * piece + 1] = total;
            }
        }
    }
}

template <typename T, int D, bool STREAM, int R, int W>
__global__ __launch_bounds__(64 * W, W == 8 ? 1 : D == 128 ? 2 : 3) void attn8_few_kernel(Attn8Args a, Attn8Split sp) {
    few_workgroup<T, D, STREAM, R, W>(a, sp);
}

namespace {

template <typename T, int D, bool STREAM, int W> void launch_rows(const Attn8Args &a, const Attn8Split &sp, hipStream_t st) {
    const dim3 grid(a.cache.heads, a.batch, (unsigned)sp.chunks);
    if (sp.rows == 1) attn8_few_kernel<T, D, STREAM, 1, W><<<grid, 64 * W, 0, st>>>(a, sp);
    else attn8_few_kernel<T, D, STREAM, kMost, W><<<grid, 64 * W, 0, st>>>(a, sp);
}

template <typename T, int D> void launch(const Attn8Args &a, const Attn8Split &sp, bool stream, hipStream_t st) {
    // Eight waves where a workgroup has its CU alone, and more than two tiles for each of
    // four: 16 x 5..1503 keys, 12 float32 heads of 64, 9.6 us, 11.0 with four (32 x 62..2001,
    // 16 heads of 128 over 8, 17.5 and 17.9; but 1 x 452 8.9 and 8.6).
    const bool eight = (int64_t)a.cache.heads * a.batch * sp.chunks <= 256 && sp.chunk > 512 && a.max_len > 512;
    if (eight) stream ? launch_rows<T, D, true, 8>(a, sp, st) : launch_rows<T, D, false, 8>(a, sp, st);
    else stream ? launch_rows<T, D, true, 4>(a, sp, st) : launch_rows<T, D, false, 4>(a, sp, st);
}

}  // namespace

hipError_t launch_attn8_few(const Attn8Args &a, const Attn8Split &sp, int head_dim, int dtype, bool stream,
                            hipStream_t st) {
    static_assert(kMost == kFewRows, "rows that the plan gives to this kernel");
    if (dtype == 1) head_dim == 128 ? launch<_Float16, 128>(a, sp, stream, st) : launch<_Float16, 64>(a, sp, stream, st);
    else head_dim == 128 ? launch<float, 128>(a, sp, stream, st) : launch<float, 64>(a, sp, stream, st);
    return hipGetLastError();
}

}  // namespace mnb
