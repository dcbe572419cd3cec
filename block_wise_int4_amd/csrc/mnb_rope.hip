// Rotary positions: pairs of a head's dimensions turned by position times
// frequency.
#include "mnb_cache8.h"
#include "mnb_device.h"

namespace mnb {

namespace {

constexpr int kWaves = 4;
constexpr int kMostPairs = 512;

// gain * (cos, sin) of position * freq radians. The fraction of a turn is taken in
// float64: of a float32 angle of 10^5 turns nothing would be left below 2^-7.
__device__ __forceinline__ float2 turn_of(int position, double freq, float gain) {
    const double turns = (double)position * freq * 0.15915494309189535;
    const float part = (float)(turns - __builtin_rint(turns));   // -0.5 .. 0.5
    float s, c;
    sincospif(2.0f * part, &s, &c);
    return float2{gain * c, gain * s};
}

}  // namespace

// A wave takes one token: its lanes work out the pairs' cosines and sines into
// LDS, then turn the heads, a unit a lane and step. VEC: 16-byte pieces (or, in
// the half layout, two of them, one from each half); otherwise a unit is one
// pair or one element behind them.
template <typename T, bool INTERLEAVED, bool VEC>
__global__ __launch_bounds__(64 * kWaves) void rope_kernel(RopeArgs a) {
    constexpr int kPiece = VEC ? 16 / (int)sizeof(T) : 1;
    __shared__ float2 s_turn[kWaves][kMostPairs];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int64_t t = (int64_t)blockIdx.x * kWaves + wave;
    if (t >= a.tokens) return;
    const int pairs = a.rot_dim / 2, position = a.positions[t];
    for (int i = lane; i < pairs; i += 64) s_turn[wave][i] = turn_of(position, a.freqs[i], a.gain);
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();
    // units of a head: those that turn, then those that are copied
    const int turning = INTERLEAVED && VEC ? a.rot_dim / kPiece : pairs / kPiece;
    const int units = turning + (a.head_dim - a.rot_dim) / kPiece;
    const int all = (a.q_heads + a.k_heads) * units;
    for (int e = lane; e < all; e += 64) {
        const int h = e / units, u = e - h * units;
        const bool key = h >= a.q_heads;
        const int at = (key ? h - a.q_heads : h) * a.head_dim;
        const T *from = reinterpret_cast<const T *>(key ? a.k + t * a.k_stride : a.q + t * a.q_stride) + at;
        T *to = reinterpret_cast<T *>(key ? a.k_out + t * a.k_out_stride : a.q_out + t * a.q_out_stride) + at;
        typedef T piece __attribute__((ext_vector_type(kPiece)));
        if (u >= turning) {
            const int d = a.rot_dim + (u - turning) * kPiece;
            *reinterpret_cast<piece *>(to + d) = *reinterpret_cast<const piece *>(from + d);
        } else if constexpr (INTERLEAVED && VEC) {
            piece x = *reinterpret_cast<const piece *>(from + u * kPiece);
#pragma unroll
            for (int i = 0; i < kPiece; i += 2) {
                const float2 cs = s_turn[wave][(u * kPiece + i) / 2];
                const float x0 = (float)x[i], x1 = (float)x[i + 1];
                x[i] = (T)__builtin_fmaf(x0, cs.x, -(x1 * cs.y));
                x[i + 1] = (T)__builtin_fmaf(x0, cs.y, x1 * cs.x);
            }
            *reinterpret_cast<piece *>(to + u * kPiece) = x;
        } else {
            const int d0 = INTERLEAVED ? 2 * u : u * kPiece, d1 = INTERLEAVED ? d0 + 1 : d0 + pairs;
            piece x0 = *reinterpret_cast<const piece *>(from + d0), x1 = *reinterpret_cast<const piece *>(from + d1);
            piece y0, y1;
#pragma unroll
            for (int i = 0; i < kPiece; ++i) {
                const float2 cs = s_turn[wave][u * kPiece + i];
                const float f0 = (float)x0[i], f1 = (float)x1[i];
                y0[i] = (T)__builtin_fmaf(f0, cs.x, -(f1 * cs.y));
                y1[i] = (T)__builtin_fmaf(f0, cs.y, f1 * cs.x);
            }
            *reinterpret_cast<piece *>(to + d0) = y0;
            *reinterpret_cast<piece *>(to + d1) = y1;
        }
    }
}

namespace {

template <typename T, bool INTERLEAVED> hipError_t launch(const RopeArgs &a, hipStream_t st) {
    const unsigned grid = (unsigned)((a.tokens + kWaves - 1) / kWaves);
    constexpr int piece = 16 / (int)sizeof(T);
    // (head_dim is a whole number of pieces)
    if (INTERLEAVED ? a.rot_dim % piece == 0 : a.rot_dim / 2 % piece == 0)
        rope_kernel<T, INTERLEAVED, true><<<grid, 64 * kWaves, 0, st>>>(a);
    else
        rope_kernel<T, INTERLEAVED, false><<<grid, 64 * kWaves, 0, st>>>(a);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_rope(const RopeArgs &a, bool interleaved, int dtype, hipStream_t st) {
    if (dtype == 1) return interleaved ? launch<_Float16, true>(a, st) : launch<_Float16, false>(a, st);
    return interleaved ? launch<float, true>(a, st) : launch<float, false>(a, st);
}

}  // namespace mnb
