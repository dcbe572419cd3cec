// Attention of query rows over the keys of their request (paged, or one run
// per request): o = sum_t exp(s_t - m) V[t] / sum_t exp(s_t - m), s_t = scale
// * q . K[t], m = max s.
//
// One workgroup per query row; its four waves take every fourth key, each
// with a running maximum and sum, and are joined in LDS.
#include "mnb_attn.h"
#include "mnb_device.h"

namespace mnb {

constexpr int kWaves = 4;

template <typename T, int D>
__global__ __launch_bounds__(64 * kWaves) void attn_kernel(AttnArgs a) {
    constexpr int E = D / 64;   // elements of a row per lane
    __shared__ float s_m[kWaves], s_l[kWaves], s_o[kWaves][D];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int64_t id = blockIdx.x;
    const int r = (int)(id % a.rows);
    const int h = (int)(id / a.rows % a.kv_heads);
    const int64_t b = id / a.rows / a.kv_heads;
    const int tq = r / a.group, hq = h * a.group + r % a.group;
    int64_t n = a.max_len;
    if (a.lens) n = a.lens[b] < n ? a.lens[b] : n;
    if (a.table && n > (int64_t)a.table_width * a.page) n = (int64_t)a.table_width * a.page;
    const T *q = static_cast<const T *>(a.q) + b * a.q_batch + tq * a.q_row + hq * a.q_head;
    float x[E], o[E], m = -__builtin_inff(), l = 0.0f;
#pragma unroll
    for (int e = 0; e < E; ++e) {
        x[e] = (float)q[lane + 64 * e];
        o[e] = 0.0f;
    }
    for (int64_t t = wave; t < n; t += kWaves) {
        int64_t kb = b, row = t;
        if (a.table) {
            kb = a.table[b * a.table_width + t / a.page];
            row = t % a.page;
            if (kb < 0 || kb >= a.num_blocks) continue;
        }
        const T *k = static_cast<const T *>(a.k) + kb * a.k_batch + row * a.k_row + h * a.k_head;
        const T *v = static_cast<const T *>(a.v) + kb * a.v_batch + row * a.v_row + h * a.v_head;
        float s = 0.0f;
#pragma unroll
        for (int e = 0; e < E; ++e) s = __builtin_fmaf(x[e], (float)k[lane + 64 * e], s);
#pragma unroll
        for (int d = 32; d; d >>= 1) s += __shfl_xor(s, d);
        s *= a.scale;
        const float top = fmaxf(m, s);
        const float base = top == -__builtin_inff() ? 0.0f : top;
        const float keep = expf(m - base), p = expf(s - base);
        m = top;
        l = l * keep + p;
#pragma unroll
        for (int e = 0; e < E; ++e) o[e] = __builtin_fmaf(p, (float)v[lane + 64 * e], o[e] * keep);
    }
    if (lane == 0) {
        s_m[wave] = m;
        s_l[wave] = l;
    }
#pragma unroll
    for (int e = 0; e < E; ++e) s_o[wave][lane + 64 * e] = o[e];
    __syncthreads();
    float top = s_m[0];
    for (int w = 1; w < kWaves; ++w) top = fmaxf(top, s_m[w]);
    if (top == -__builtin_inff()) top = 0.0f;
    T *out = static_cast<T *>(a.out) + b * a.o_batch + tq * a.o_row + hq * a.o_head;
    for (int d = threadIdx.x; d < D; d += 64 * kWaves) {
        float sum = 0.0f, total = 0.0f;
        for (int w = 0; w < kWaves; ++w) {
            const float f = expf(s_m[w] - top);
            total += s_l[w] * f;
            sum += s_o[w][d] * f;
        }
        out[d] = Io<T>::from_f32(total == 0.0f ? 0.0f : sum / total);
    }
}

int64_t attn_workspace_bytes(int64_t batch, int64_t kv_heads, int64_t rows, int64_t max_len, int head_dim,
                             int dtype) {
    return 0;
}

bool attn_fits(int64_t batch, int64_t kv_heads, int64_t rows, int64_t max_len, int head_dim, int dtype) {
    return batch * kv_heads * rows <= 0x7FFFFFFFLL && (rows == 0 || batch * kv_heads <= 0x7FFFFFFFLL / rows);
}

hipError_t launch_attn(const AttnArgs &a, int head_dim, int dtype, void *workspace, hipStream_t st) {
    const unsigned grid = (unsigned)((int64_t)a.batch * a.kv_heads * a.rows);
    if (dtype == 1) {
        if (head_dim == 128) attn_kernel<_Float16, 128><<<grid, 64 * kWaves, 0, st>>>(a);
        else attn_kernel<_Float16, 64><<<grid, 64 * kWaves, 0, st>>>(a);
    } else {
        if (head_dim == 128) attn_kernel<float, 128><<<grid, 64 * kWaves, 0, st>>>(a);
        else attn_kernel<float, 64><<<grid, 64 * kWaves, 0, st>>>(a);
    }
    return hipGetLastError();
}

}  // namespace mnb
