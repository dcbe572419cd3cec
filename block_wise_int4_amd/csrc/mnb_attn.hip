// Attention of query rows over the keys of their request (paged, or one run
// per request): o = sum_t w_t V[t] / sum_t w_t, w_t = exp(s_t - m), s_t =
// scale * q . K[t], with a reference m kept near the running maximum.
//
// Work: keys are cut into chunks; one workgroup takes up to 16 query rows of
// one (request, key-value head) over one chunk, its waves every kWaves-th
// tile of 16 or 32 keys. A wave streams its tiles from memory straight into
// the registers that the matrix instructions read (no LDS, no barrier), the
// next tile in flight while one is computed:
//   S^T = K Q^T   A = keys (lane: key l % 16, 16 bytes of its row), B = queries;
//                 the result holds, per lane, four keys 4 (l / 16) + i of one
//                 query l % 16, which is already the B operand's layout of
//   O^T = V^T P^T with the contraction index renumbered: A's rows are
//                 dimensions. A lane loads whole pieces of V rows (l % 16 says
//                 which piece: a row is one coalesced run over 16 lanes), and
//                 piece element e of lane row m is dimension m * (D / 16) + e:
//                 float32 needs no shuffle at all, float16 one byte permute
//                 per pair of keys.
// The waves' sums are joined in LDS, and the chunks' by a second launch.
#include "mnb_attn.h"
#include "mnb_device.h"

namespace mnb {

namespace {

constexpr int kWaves = 4;
constexpr int kQ = 16;                      // query rows per workgroup
constexpr float kLowest = -3.402823466e38f; // the reference before any key
constexpr float kLog2e = 1.4426950408889634f;

typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));

template <int Bytes> struct Piece;
template <> struct Piece<16> { typedef u32x4 type; };
template <> struct Piece<8> { typedef u32x2 type; };

// Registers of one tile of 16 * NS keys of a float16 or float32 row of D.
template <typename T, int D> struct TileShape {
    static constexpr int kRow = D * (int)sizeof(T);                 // bytes
    static constexpr int kSub = sizeof(T) == 4 && D == 128 ? 1 : 2; // 16-key parts (64 registers of K and V at D = 128)
    static constexpr int kKeys = 16 * kSub;
    static constexpr int kK = kRow / 64;                            // 16-byte pieces of a K row per lane
    static constexpr int kVBytes = kRow / 16 < 16 ? kRow / 16 : 16;
    static constexpr int kV = kRow / 16 / kVBytes;                  // pieces of a V row per lane
    static constexpr int kOut = D / 16;                             // 16-dimension parts of the output
};

template <typename T, int D> struct Tile {
    using S = TileShape<T, D>;
    u32x4 k[S::kSub][S::kK];
    typename Piece<S::kVBytes>::type v[S::kSub][4][S::kV];
    int valid[S::kSub];   // leading valid keys of each part
};

// Scores are kept as x = s * mul, weights are exp2 of differences: float16
// folds log2(e) into mul (a finite float16 score is far from overflow);
// float32 does not, so that scores down to the type's lowest value stay
// finite.
template <typename T> __device__ __forceinline__ float score_mul(float scale) {
    return sizeof(T) == 4 ? scale : scale * kLog2e;
}
template <typename T> __device__ __forceinline__ float weight(float x, float ref) {
    const float d = x - ref;
    return __builtin_amdgcn_exp2f(sizeof(T) == 4 ? d * kLog2e : d);
}

__device__ __forceinline__ f4 mma16(h8 a, h8 b, f4 c) { return __builtin_amdgcn_mfma_f32_16x16x32_f16(a, b, c, 0, 0, 0); }
__device__ __forceinline__ f4 mma4(float a, float b, f4 c) { return __builtin_amdgcn_mfma_f32_16x16x4f32(a, b, c, 0, 0, 0); }

__device__ __forceinline__ int64_t keys_of(const AttnArgs &a, int64_t b) {
    int64_t n = a.max_len;
    if (a.lens && a.lens[b] < n) n = a.lens[b];
    if (a.table && n > (int64_t)a.table_width * a.page) n = (int64_t)a.table_width * a.page;
    return n;
}

}  // namespace

// Partial results of a split launch: per (request, head, row, chunk) D sums,
// then per the same the reference and the weights' sum.
struct AttnSplit {
    int32_t chunk;      // keys per chunk (a multiple of kWaves tiles)
    int32_t chunks;     // of max_len
    int32_t q_tiles;    // of `rows`
    uint64_t page_magic;  // ceil(2^32 / (page / 16)): (part * magic) >> 32 = part / (page / 16) for part < 2^26
    float *sums, *stats;
};

template <typename T, int D, bool PAGED>
__global__ __launch_bounds__(64 * kWaves, 2) void attn_kernel(AttnArgs a, AttnSplit sp) {
    using S = TileShape<T, D>;
    __shared__ float s_o[kWaves][kQ][D + 4];
    __shared__ float s_m[kWaves][kQ], s_l[kWaves][kQ];
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int col = lane & 15, g = lane >> 4;
    uint32_t id = blockIdx.x;
    const int chunk = id % sp.chunks;
    id /= sp.chunks;
    const int q_tile = id % sp.q_tiles;
    id /= sp.q_tiles;
    const int h = id % a.kv_heads;
    const int64_t b = id / a.kv_heads;
    const int n = (int)keys_of(a, b);
    const int begin = chunk * sp.chunk;
    if (begin >= n && chunk > 0) return;
    const int end = n - begin < sp.chunk ? n : begin + sp.chunk;   // (n may be <= 0: nothing below runs)
    const int rows = a.rows - q_tile * kQ < kQ ? a.rows - q_tile * kQ : kQ;

    // queries: lane (query col, dimensions of its group g of each 64-byte run)
    u32x4 q[S::kK];
    {
        const int r = q_tile * kQ + (col < rows ? col : 0);
        const T *src = static_cast<const T *>(a.q) + b * a.q_batch + (int64_t)(r / a.group) * a.q_row +
                       (int64_t)(h * a.group + r % a.group) * a.q_head;
        const uint8_t *p = reinterpret_cast<const uint8_t *>(src) + g * 16;
#pragma unroll
        for (int j = 0; j < S::kK; ++j) q[j] = *reinterpret_cast<const u32x4 *>(p + j * 64);
    }
    const uint8_t *kp = static_cast<const uint8_t *>(a.k) + h * a.k_head * (int64_t)sizeof(T);
    const uint8_t *vp = static_cast<const uint8_t *>(a.v) + h * a.v_head * (int64_t)sizeof(T);
    const int64_t k_batch = a.k_batch * (int64_t)sizeof(T), v_batch = a.v_batch * (int64_t)sizeof(T);
    const uint32_t k_row = (uint32_t)a.k_row * sizeof(T), v_row = (uint32_t)a.v_row * sizeof(T);
    const int32_t *table = PAGED ? a.table + b * a.table_width : nullptr;
    const int per_page = PAGED ? a.page >> 4 : 1;

    // Loads a tile's keys and values. Every address stays inside the cache:
    // parts without a valid key read block 0 (or the request's first row),
    // rows past the last valid key read that key's row.
    auto load = [&](Tile<T, D> &t, int key0) {
#pragma unroll
        for (int s = 0; s < S::kSub; ++s) {
            const int first = key0 + 16 * s;
            int valid = end - first;
            valid = valid < 0 ? 0 : valid > 16 ? 16 : valid;
            int64_t kb = 0, vb = 0;
            if constexpr (PAGED) {
                int id = 0, within = 0;
                if (valid > 0) {
                    const uint32_t part = (uint32_t)first >> 4;
                    const uint32_t place = (uint32_t)((part * sp.page_magic) >> 32);
                    within = (int)(part - place * per_page) << 4;
                    id = table[place];
                    if (id < 0 || id >= a.num_blocks) id = within = valid = 0;
                }
                kb = id * k_batch + (int64_t)within * k_row;
                vb = id * v_batch + (int64_t)within * v_row;
            } else {
                const int from = valid > 0 ? first : 0;
                kb = b * k_batch + (int64_t)from * k_row;
                vb = b * v_batch + (int64_t)from * v_row;
            }
            t.valid[s] = valid;
            const int last = valid > 0 ? valid - 1 : 0;
            const uint8_t *ks = kp + kb, *vs = vp + vb;
            const uint32_t ko = (uint32_t)(col < last ? col : last) * k_row + g * 16;
#pragma unroll
            for (int j = 0; j < S::kK; ++j) t.k[s][j] = *reinterpret_cast<const u32x4 *>(ks + ko + j * 64);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int key = 4 * g + i;
                const uint32_t vo = (uint32_t)(key < last ? key : last) * v_row + col * S::kVBytes;
#pragma unroll
                for (int c = 0; c < S::kV; ++c)
                    t.v[s][i][c] = *reinterpret_cast<const typename Piece<S::kVBytes>::type *>(vs + vo + c * 256);
            }
        }
    };

    f4 o[S::kOut];
#pragma unroll
    for (int i = 0; i < S::kOut; ++i) o[i] = f4{0.0f, 0.0f, 0.0f, 0.0f};
    float ref = kLowest, l = 0.0f;
    const float mul = score_mul<T>(a.scale);
    // weights stay below exp2(8): the reference moves only when a score
    // passes it by more than that
    const float slack = sizeof(T) == 4 ? 5.5f : 8.0f;

    auto compute = [&](Tile<T, D> &t) {
        float x[S::kSub][4];
#pragma unroll
        for (int s = 0; s < S::kSub; ++s) {
            f4 c = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
            for (int j = 0; j < S::kK; ++j) {
                if constexpr (sizeof(T) == 2) {
                    c = mma16(__builtin_bit_cast(h8, t.k[s][j]), __builtin_bit_cast(h8, q[j]), c);
                } else {
                    const f4 kk = __builtin_bit_cast(f4, t.k[s][j]), qq = __builtin_bit_cast(f4, q[j]);
                    c = mma4(kk.x, qq.x, c);
                    c = mma4(kk.y, qq.y, c);
                    c = mma4(kk.z, qq.z, c);
                    c = mma4(kk.w, qq.w, c);
                }
            }
#pragma unroll
            for (int i = 0; i < 4; ++i) x[s][i] = c[i] * mul;
            if (t.valid[s] < 16) {   // uniform: the end of a row, or a missing block
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const bool on = 4 * g + i < t.valid[s];
                    x[s][i] = on ? x[s][i] : -__builtin_inff();
#pragma unroll
                    for (int c2 = 0; c2 < S::kV; ++c2)
                        t.v[s][i][c2] = on ? t.v[s][i][c2] : typename Piece<S::kVBytes>::type(0u);
                }
            }
        }
        float top = x[0][0];
#pragma unroll
        for (int s = 0; s < S::kSub; ++s)
#pragma unroll
            for (int i = 0; i < 4; ++i) top = fmaxf(top, x[s][i]);
        if (__any(top > ref + slack)) {
            float to = fmaxf(ref, top);
            to = fmaxf(to, __shfl_xor(to, 16));
            to = fmaxf(to, __shfl_xor(to, 32));
            const float keep = weight<T>(ref, to);
            ref = to;
            l *= keep;
#pragma unroll
            for (int i = 0; i < S::kOut; ++i) o[i] *= keep;
        }
        float p[S::kSub][4];
#pragma unroll
        for (int s = 0; s < S::kSub; ++s)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                p[s][i] = weight<T>(x[s][i], ref);
                l += p[s][i];
            }
        if constexpr (sizeof(T) == 4) {
#pragma unroll
            for (int s = 0; s < S::kSub; ++s)
#pragma unroll
                for (int i = 0; i < 4; ++i)
#pragma unroll
                    for (int c = 0; c < S::kV; ++c) {
                        const f4 vv = __builtin_bit_cast(f4, t.v[s][i][c]);
#pragma unroll
                        for (int e = 0; e < 4; ++e) o[4 * c + e] = mma4(vv[e], p[s][i], o[4 * c + e]);
                    }
        } else {
            // the weights as a float16 pair hi + lo (22 bits): the stream
            // leaves the matrix units idle, so the second product is free
            h8 hi, lo;
#pragma unroll
            for (int s = 0; s < 2; ++s)
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const _Float16 w = (_Float16)p[s][i];
                    hi[4 * s + i] = w;
                    lo[4 * s + i] = (_Float16)(p[s][i] - (float)w);
                }
#pragma unroll
            for (int e = 0; e < S::kOut; ++e) {
                u32x4 w;
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const auto &v0 = t.v[j >> 1][2 * (j & 1)][0], &v1 = t.v[j >> 1][2 * (j & 1) + 1][0];
                    w[j] = __builtin_amdgcn_perm(v1[e >> 1], v0[e >> 1], e & 1 ? 0x07060302u : 0x05040100u);
                }
                o[e] = mma16(__builtin_bit_cast(h8, w), hi, o[e]);
                o[e] = mma16(__builtin_bit_cast(h8, w), lo, o[e]);
            }
        }
    };

    const int step = kWaves * S::kKeys;
    int key = begin + wave * S::kKeys;
    if (key < end) {
        Tile<T, D> t0, t1;
        load(t0, key);
        for (; key < end; key += 2 * step) {
            load(t1, key + step);
            compute(t0);
            if (key + step >= end) break;
            load(t0, key + 2 * step);
            compute(t1);
        }
    }

    // join the waves
    l += __shfl_xor(l, 16);
    l += __shfl_xor(l, 32);
    if (g == 0) {
        s_m[wave][col] = ref;
        s_l[wave][col] = l;
    }
    if (col < rows) {
#pragma unroll
        for (int e = 0; e < S::kOut; ++e)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                // row 4 g + i of part e (float16: element e of a lane's piece;
                // float32: element e % 4 of its piece e / 4)
                const int m = 4 * g + i;
                const int d = sizeof(T) == 2 ? m * S::kOut + e : 64 * (e >> 2) + 4 * m + (e & 3);
                s_o[wave][col][d] = o[e][i];
            }
    }
    __syncthreads();
    const bool whole = n <= sp.chunk;   // this chunk is the row's only one
    const int64_t row0 = ((b * a.kv_heads + h) * a.rows + q_tile * kQ);
    for (int e = threadIdx.x; e < rows * D; e += 64 * kWaves) {
        const int r = e / D, d = e % D;
        float m = s_m[0][r];
#pragma unroll
        for (int w = 1; w < kWaves; ++w) m = fmaxf(m, s_m[w][r]);
        float sum = 0.0f, total = 0.0f;
#pragma unroll
        for (int w = 0; w < kWaves; ++w) {
            const float f = weight<T>(s_m[w][r], m);
            sum += s_o[w][r][d] * f;
            total += s_l[w][r] * f;
        }
        if (whole) {
            const int row = q_tile * kQ + r;
            T *out = static_cast<T *>(a.out) + b * a.o_batch + (int64_t)(row / a.group) * a.o_row +
                     (int64_t)(h * a.group + row % a.group) * a.o_head;
            out[d] = Io<T>::from_f32(total == 0.0f ? 0.0f : sum / total);
        } else {
            const int64_t at = (row0 + r) * sp.chunks + chunk;
            sp.sums[at * D + d] = sum;
            if (d == 0) {
                sp.stats[2 * at] = m;
                sp.stats[2 * at + 1] = total;
            }
        }
    }
}

// Joins the chunks of one query row, in their order.
template <typename T, int D>
__global__ __launch_bounds__(D) void attn_join_kernel(AttnArgs a, AttnSplit sp) {
    uint32_t id = blockIdx.x;
    const int row = id % a.rows;
    const int h = id / a.rows % a.kv_heads;
    const int64_t b = id / a.rows / a.kv_heads;
    const int n = (int)keys_of(a, b);
    if (n <= sp.chunk) return;
    const int chunks = (n + sp.chunk - 1) / sp.chunk;
    const float *stats = sp.stats + 2 * (int64_t)id * sp.chunks;
    const float *sums = sp.sums + (int64_t)id * sp.chunks * D;
    float m = stats[0];
    for (int c = 1; c < chunks; ++c) m = fmaxf(m, stats[2 * c]);
    float sum = 0.0f, total = 0.0f;
    for (int c = 0; c < chunks; ++c) {
        const float f = weight<T>(stats[2 * c], m);
        sum += sums[(int64_t)c * D + threadIdx.x] * f;
        total += stats[2 * c + 1] * f;
    }
    T *out = static_cast<T *>(a.out) + b * a.o_batch + (int64_t)(row / a.group) * a.o_row +
             (int64_t)(h * a.group + row % a.group) * a.o_head;
    out[threadIdx.x] = Io<T>::from_f32(total == 0.0f ? 0.0f : sum / total);
}

namespace {

struct Split {
    int64_t chunk, chunks, q_tiles;
};

// Chunk length: long enough that a chunk's stream (hundreds of KB) outweighs
// its start and its partial result, short enough that the chip has several
// workgroups per place (512 resident) to even out ragged lengths.
Split plan(int64_t batch, int64_t kv_heads, int64_t rows, int64_t max_len) {
    Split s;
    s.q_tiles = (rows + kQ - 1) / kQ;
    const int64_t units = batch * kv_heads * s.q_tiles;
    const int64_t step = kWaves * 32;
    const int64_t keys = (max_len + step - 1) / step * step;
    const int64_t want = 2048;    // workgroups
    int64_t chunk = units > 0 ? keys / (want / units > 0 ? want / units : 1) : keys;
    chunk = (chunk + step - 1) / step * step;
    if (chunk < 2 * step) chunk = 2 * step;
    if (chunk >= keys) chunk = keys > step ? keys : step;
    s.chunk = chunk;
    s.chunks = keys > 0 ? (keys + chunk - 1) / chunk : 1;
    return s;
}

template <typename T, int D>
hipError_t launch(const AttnArgs &a, const AttnSplit &sp, hipStream_t st) {
    const unsigned grid = (unsigned)((int64_t)a.batch * a.kv_heads * sp.q_tiles * sp.chunks);
    if (a.table) attn_kernel<T, D, true><<<grid, 64 * kWaves, 0, st>>>(a, sp);
    else attn_kernel<T, D, false><<<grid, 64 * kWaves, 0, st>>>(a, sp);
    if (sp.chunks > 1)
        attn_join_kernel<T, D><<<(unsigned)((int64_t)a.batch * a.kv_heads * a.rows), D, 0, st>>>(a, sp);
    return hipGetLastError();
}

}  // namespace

int64_t attn_workspace_bytes(int64_t batch, int64_t kv_heads, int64_t rows, int64_t max_len, int head_dim,
                             int dtype) {
    const Split s = plan(batch, kv_heads, rows, max_len);
    return s.chunks > 1 ? batch * kv_heads * rows * s.chunks * (head_dim + 2) * 4 : 0;
}

bool attn_fits(int64_t batch, int64_t kv_heads, int64_t rows, int64_t max_len, int head_dim, int dtype) {
    const int64_t most = (1LL << 24) - 1;   // workgroups: a launch's threads are counted in 32 bits
    const Split s = plan(batch, kv_heads, rows, max_len);
    const int64_t pairs = batch * kv_heads;  // <= 2^31
    if (pairs == 0 || rows == 0) return true;
    if (pairs > most / s.q_tiles || pairs * s.q_tiles > most / s.chunks) return false;
    return s.chunks == 1 || pairs <= most / rows;
}

hipError_t launch_attn(const AttnArgs &a, int head_dim, int dtype, void *workspace, hipStream_t st) {
    const Split s = plan(a.batch, a.kv_heads, a.rows, a.max_len);
    AttnSplit sp{};
    sp.chunk = (int32_t)s.chunk;
    sp.chunks = (int32_t)s.chunks;
    sp.q_tiles = (int32_t)s.q_tiles;
    sp.page_magic = a.table ? ((1ull << 32) + a.page / 16 - 1) / (a.page / 16) : 0;
    sp.sums = static_cast<float *>(workspace);
    sp.stats = sp.sums + (int64_t)a.batch * a.kv_heads * a.rows * s.chunks * head_dim;
    if (dtype == 1) return head_dim == 128 ? launch<_Float16, 128>(a, sp, st) : launch<_Float16, 64>(a, sp, st);
    return head_dim == 128 ? launch<float, 128>(a, sp, st) : launch<float, 64>(a, sp, st);
}

}  // namespace mnb
