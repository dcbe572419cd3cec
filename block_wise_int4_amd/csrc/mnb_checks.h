// Argument checks shared by the C entry points of the attention operators, of
// the 8-bit cache and of the rotary positions. Host only.
#pragma once
#include <hip/hip_runtime.h>
#include <math.h>
#include <stdint.h>

#include "../../include/mnb.h"
#include "mnb_attn.h"

namespace mnb {

constexpr int64_t kIntMax = 0x7FFFFFFFLL;

inline bool aligned(const void *p, uintptr_t to) { return (reinterpret_cast<uintptr_t>(p) & (to - 1)) == 0; }

struct Range {
    uintptr_t from, to;
};
inline Range range(const void *p, int64_t bytes) {
    const uintptr_t from = reinterpret_cast<uintptr_t>(p);
    return {from, from + (uintptr_t)bytes};
}

// (an empty range overlaps nothing, wherever it lies)
inline bool overlap(const Range &a, const Range &b) {
    return a.from < b.to && b.from < a.to && a.from < a.to && b.from < b.to;
}

inline int hip_status(hipError_t e) { return e == hipSuccess ? MNB_OK : MNB_ERR_HIP; }

inline int64_t dtype_bytes(int dtype) { return dtype == MNB_F16 ? 2 : 4; }

inline bool known_dtype(int dtype) { return dtype == MNB_F16 || dtype == MNB_F32; }

inline bool page_ok(int64_t page) { return page > 0 && page <= MNB_MAX_PAGE && page % kPageGranule == 0; }

// Strides (elements) that keep every row 16-byte aligned; not negative, and
// small enough that no product with an index in range leaves 64 bits.
inline int check_strides(int64_t a, int64_t b, int64_t c, int dtype) {
    const int64_t most = 1LL << 40, unit = 16 / dtype_bytes(dtype);
    if (a < 0 || b < 0 || c < 0 || a > most || b > most || c > most) return MNB_ERR_SHAPE;
    if (a % unit || b % unit || c % unit) return MNB_ERR_ALIGN;
    return MNB_OK;
}

// The scale the kernels take. Float16 scores are multiplied by scale * log2(e) at
// once, which must not overflow: products of float16 rows are whole multiples of
// 2^-48 and below 2^40, so at 2^80 all scores are finite and different ones 2^32
// apart, and a larger scale has the same softmax.
inline float kernel_scale(float scale, int dtype) {
    return dtype == MNB_F16 ? copysignf(fminf(fabsf(scale), 0x1p80f), scale) : scale;
}

inline int check_workspace(int64_t need, const void *workspace, size_t bytes) {
    if (need == 0) return MNB_OK;
    if (!workspace) return MNB_ERR_NULL;
    if (!aligned(workspace, 16)) return MNB_ERR_ALIGN;
    return bytes < (size_t)need ? MNB_ERR_INVALID : MNB_OK;
}

}  // namespace mnb
