// Rotary positions: pairs of a head's dimensions turned by position times
// frequency.
#include "mnb_cache8.h"
#include "mnb_device.h"

namespace mnb {

namespace {

constexpr int kWaves = 4;
constexpr int kMostPairs = 512;
constexpr int kAhead = 4;

// gain * (cos, sin) of position * freq radians. The fraction of a turn is taken in
// float64: of a float32 angle of 10^5 turns nothing would be left below 2^-7. Its first
// 24 bits give the cosine and sine, which are turned on by the rest (up to 2 pi 2^-26
// radians, as much as the rounding of a number near one).
__device__ __forceinline__ float2 turn_of(int position, double freq, float gain) {
    const double turns = (double)position * freq * 0.15915494309189535;
    const double fraction = turns - __builtin_rint(turns);   // -0.5 .. 0.5
    const float part = (float)fraction, rest = 6.2831853f * (float)(fraction - (double)part);
    float s, c;
    sincospif(2.0f * part, &s, &c);
    return float2{gain * __builtin_fmaf(-s, rest, c), gain * __builtin_fmaf(c, rest, s)};
}

// A float32 result rounded to T. (Hidden from the compiler, which would fold some of the
// conversions, and not others, into multiply-adds of another rounding: a head's bits
// would go by its place in the loop.)
template <typename T> __device__ __forceinline__ T rounded(float x) {
    asm("" : "+v"(x));
    return (T)x;
}

}  // namespace

// A wave takes one token: its lanes work out the pairs' cosines and sines into
// LDS, then turn the heads, a unit a lane, kAhead units under way (9999 float32 tokens of
// 24 x 128, interleaved, 246 MB: 50..55 us, 4.5..4.9 TB/s, what a copy reaches; as called 55,
// with one unit 64; 8 float16 tokens 3.6, a launch). VEC: 16-byte pieces
// (or, in the half layout, two of them, one from each half); otherwise a unit is one
// pair, or one element behind them.
template <typename T, bool INTERLEAVED, bool VEC>
__global__ __launch_bounds__(64 * kWaves) void rope_kernel(RopeArgs a, float per_units) {
    constexpr int kPiece = VEC ? 16 / (int)sizeof(T) : 1;
    constexpr bool kTwo = !(INTERLEAVED && VEC);   // a unit is two pieces
    typedef T piece __attribute__((ext_vector_type(kPiece)));
    __shared__ float2 s_turn[kWaves][kMostPairs];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int64_t t = (int64_t)blockIdx.x * kWaves + wave;
    if (t >= a.tokens) return;
    // units of a head: those that turn, then those that are copied
    const int pairs = a.rot_dim / 2, turning = kTwo ? pairs / kPiece : a.rot_dim / kPiece;
    const int units = turning + (a.head_dim - a.rot_dim) / kPiece;
    const int all = (a.q_heads + a.k_heads) * units;
    const int position = a.positions[t];
    bool ready = false;
    for (int e0 = lane; e0 < all + lane; e0 += 64 * kAhead) {   // (the wave's lanes together)
        piece x0[kAhead], x1[kAhead];
        T *to[kAhead];
        int unit[kAhead];
#pragma unroll
        for (int i = 0; i < kAhead; ++i) {
            // (e < 2^24 by a reciprocal that is off by at most one, others by a division)
            const int e = e0 + 64 * i;
            int h = all < (1 << 24) ? (int)((float)e * per_units) : e / units, u = e - h * units;
            if (u >= units) ++h, u -= units;
            if (u < 0) --h, u += units;
            const bool key = h >= a.q_heads;
            const int at = (key ? h - a.q_heads : h) * a.head_dim;
            const int d = u < turning ? (kTwo && INTERLEAVED ? 2 * u : u * kPiece) : a.rot_dim + (u - turning) * kPiece;
            unit[i] = e < all ? u : -1;
            to[i] = reinterpret_cast<T *>(key ? a.k_out + t * a.k_out_stride : a.q_out + t * a.q_out_stride) + at + d;
            if (e < all) {
                const T *from = reinterpret_cast<const T *>(key ? a.k + t * a.k_stride : a.q + t * a.q_stride) + at + d;
                x0[i] = *reinterpret_cast<const piece *>(from);
                if (kTwo && u < turning) x1[i] = *reinterpret_cast<const piece *>(from + (INTERLEAVED ? 1 : pairs));
            }
        }
        if (!ready) {   // (behind the first loads)
            for (int i = lane; i < pairs; i += 64) s_turn[wave][i] = turn_of(position, a.freqs[i], a.gain);
            wave_fence();
            ready = true;
        }
#pragma unroll
        for (int i = 0; i < kAhead; ++i) {
            if (unit[i] < 0) continue;
            if (unit[i] < turning) {
                if constexpr (kTwo) {
                    piece y1;
#pragma unroll
                    for (int j = 0; j < kPiece; ++j) {
                        const float2 cs = s_turn[wave][unit[i] * kPiece + j];
                        const float f0 = (float)x0[i][j], f1 = (float)x1[i][j];
                        x0[i][j] = rounded<T>(__builtin_fmaf(f0, cs.x, -(f1 * cs.y)));
                        y1[j] = rounded<T>(__builtin_fmaf(f0, cs.y, f1 * cs.x));
                    }
                    *reinterpret_cast<piece *>(to[i] + (INTERLEAVED ? 1 : pairs)) = y1;
                } else {
#pragma unroll
                    for (int j = 0; j < kPiece; j += 2) {
                        const float2 cs = s_turn[wave][(unit[i] * kPiece + j) / 2];
                        const float f0 = (float)x0[i][j], f1 = (float)x0[i][j + 1];
                        x0[i][j] = rounded<T>(__builtin_fmaf(f0, cs.x, -(f1 * cs.y)));
                        x0[i][j + 1] = rounded<T>(__builtin_fmaf(f0, cs.y, f1 * cs.x));
                    }
                }
            }
            *reinterpret_cast<piece *>(to[i]) = x0[i];
        }
    }
}

namespace {

// Tokens of a launch, whose threads (64 a token) are counted in 32 bits. (A loop over
// tokens in the kernel takes a register too many: four waves a SIMD for five.)
constexpr int64_t kMostTokens = 1 << 25;

template <typename T, bool INTERLEAVED> hipError_t launch(RopeArgs a, hipStream_t st) {
    constexpr int piece = 16 / (int)sizeof(T);
    const bool vec = INTERLEAVED ? a.rot_dim % piece == 0 : a.rot_dim / 2 % piece == 0;
    const int turning = !vec ? a.rot_dim / 2 : INTERLEAVED ? a.rot_dim / piece : a.rot_dim / 2 / piece;
    const float per_units = 1.0f / (float)(turning + (a.head_dim - a.rot_dim) / (vec ? piece : 1));
    for (int64_t left = a.tokens;;) {
        a.tokens = left < kMostTokens ? left : kMostTokens;
        const unsigned grid = (unsigned)((a.tokens + kWaves - 1) / kWaves);
        // (head_dim is a whole number of pieces)
        if (vec) rope_kernel<T, INTERLEAVED, true><<<grid, 64 * kWaves, 0, st>>>(a, per_units);
        else rope_kernel<T, INTERLEAVED, false><<<grid, 64 * kWaves, 0, st>>>(a, per_units);
        hipError_t e = hipGetLastError();
        if (e != hipSuccess || (left -= a.tokens) == 0) return e;
        if (a.q_heads) a.q += a.tokens * a.q_stride, a.q_out += a.tokens * a.q_out_stride;
        if (a.k_heads) a.k += a.tokens * a.k_stride, a.k_out += a.tokens * a.k_out_stride;
        a.positions += a.tokens;
    }
}

}  // namespace

hipError_t launch_rope(const RopeArgs &a, bool interleaved, int dtype, hipStream_t st) {
    if (dtype == 1) return interleaved ? launch<_Float16, true>(a, st) : launch<_Float16, false>(a, st);
    return interleaved ? launch<float, true>(a, st) : launch<float, false>(a, st);
}

}  // namespace mnb
