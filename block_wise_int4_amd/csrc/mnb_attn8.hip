// Attention over the 8-bit cache: o = sum_t w_t vs_t cv_t / sum_t w_t, w_t =
// exp(s_t - m), s_t = scale * ks_t * (q . ck_t), codes ck, cv and scales ks, vs.
//
// First form: a wave takes one query row (token, head) and walks over its keys 64
// at a time, a key a lane for the scores, D / 64 dimensions a lane for the sums.
#include "mnb_cache8.h"
#include "mnb_device.h"

namespace mnb {

namespace {

constexpr float kLowest = -3.402823466e38f;
constexpr float kLog2e = 1.4426950408889634f;

// New tokens of request b, and its first row of q.
__device__ __forceinline__ int rows_of(const Attn8Args &a, int64_t b, int64_t &first) {
    if (!a.starts) {
        first = b;
        return 1;
    }
    int64_t from = a.starts[b], to = a.starts[b + 1];
    from = from < 0 ? 0 : from > a.tokens ? a.tokens : from;
    to = to < from ? from : to > a.tokens ? a.tokens : to;
    first = from;
    return (int)(to - from);
}

}  // namespace

template <typename T, int D> __global__ __launch_bounds__(64) void attn8_kernel(Attn8Args a) {
    __shared__ float s_q[D], s_w[64];
    __shared__ const int8_t *s_v[64];
    const int lane = threadIdx.x, h = blockIdx.x, i = blockIdx.z;
    const int64_t b = blockIdx.y;
    int64_t first;
    const int rows = rows_of(a, b, first);
    if (i >= rows) return;
    int64_t n = (int64_t)a.lens[b] - rows + i + 1;
    n = n < a.max_len ? n : a.max_len;
    const int kv = h / a.group;
    const Cache8 &c = a.cache;
    const T *q = static_cast<const T *>(a.q) + (first + i) * a.q_stride + (int64_t)h * D;
    bool finite = true;
    for (int d = lane; d < D; d += 64) {
        s_q[d] = (float)q[d];
        finite &= __builtin_fabsf(s_q[d]) <= -kLowest;
    }
    const float spoil = __all(finite) ? 0.0f : __builtin_nanf("");
    __syncthreads();
    float o[D / 64] = {}, l = 0.0f, m = kLowest;
    for (int64_t base = 0; base < n; base += 64) {
        const int64_t t = base + lane;
        float x = -__builtin_inff(), vs = 0.0f;
        const int8_t *vp = nullptr;
        if (t < n) {
            const int id = a.table[b * a.table_width + t / c.page];
            const int offset = (int)(t % c.page);
            if (id >= 0 && id < c.num_blocks) {
                const int64_t at = id * c.block_stride + kv * c.head_stride + offset * c.token_stride;
                const int64_t sat = id * c.scale_block + kv * c.scale_head + offset;
                const int8_t *kp = c.k + at;
                vp = c.v + at;
                float sum = 0.0f;
                for (int d = 0; d < D; ++d) sum = __builtin_fmaf(s_q[d], (float)kp[d], sum);
                x = sum * c.k_scale[sat] * a.scale + spoil;
                vs = c.v_scale[sat];
            }
        }
        float top = x;
        for (int d = 1; d < 64; d <<= 1) top = fmaxf(top, __shfl_xor(top, d));
        const float to = fmaxf(m, top), keep = __builtin_amdgcn_exp2f((m - to) * kLog2e);
        m = to;
        const float w = __builtin_amdgcn_exp2f((x - m) * kLog2e);
        float sum = w;
        for (int d = 1; d < 64; d <<= 1) sum += __shfl_xor(sum, d);
        l = l * keep + sum;
        __syncthreads();
        s_w[lane] = vp ? w * vs : 0.0f;
        s_v[lane] = vp;
        __syncthreads();
        for (int e = 0; e < D / 64; ++e) o[e] *= keep;
        for (int j = 0; j < 64; ++j) {
            if (!s_v[j]) continue;
            for (int e = 0; e < D / 64; ++e)
                o[e] = __builtin_fmaf(s_w[j], (float)s_v[j][lane + 64 * e], o[e]);
        }
    }
    T *out = static_cast<T *>(a.out) + ((first + i) * (int64_t)(c.heads * a.group) + h) * D;
    for (int e = 0; e < D / 64; ++e) out[lane + 64 * e] = (T)(l == 0.0f ? 0.0f : o[e] / l);
}

int64_t attn8_workspace_bytes(int64_t, int64_t, int64_t, int64_t, int64_t, int, int) { return 0; }

bool attn8_fits(int64_t batch, int64_t kv_heads, int64_t group, int64_t max_new, int64_t, int, int) {
    return kv_heads * group <= (1 << 22) && batch <= 65536 && max_new <= 65535;
}

hipError_t launch_attn8(const Attn8Args &a, int head_dim, int dtype, void *, hipStream_t st) {
    Attn8Args c = a;
    if (c.max_len > (int64_t)a.table_width * a.cache.page) c.max_len = a.table_width * a.cache.page;
    const int64_t most = a.tokens < a.max_new ? a.tokens : a.max_new;
    const dim3 grid(a.cache.heads * a.group, a.batch, (unsigned)most);
    if (dtype == 1)
        head_dim == 128 ? attn8_kernel<_Float16, 128><<<grid, 64, 0, st>>>(c)
                        : attn8_kernel<_Float16, 64><<<grid, 64, 0, st>>>(c);
    else
        head_dim == 128 ? attn8_kernel<float, 128><<<grid, 64, 0, st>>>(c)
                        : attn8_kernel<float, 64><<<grid, 64, 0, st>>>(c);
    return hipGetLastError();
}

}  // namespace mnb
