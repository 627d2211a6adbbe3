// Shared by the convolution, scan and group norm kernels: element conversion,
// activations, 16-byte pieces, and the host's pointer checks.
#pragma once

#include <cuda_bf16.h>

#include "gdn_internal.h"

namespace gdn {

__device__ __forceinline__ float to_f32(float v) { return v; }
__device__ __forceinline__ float to_f32(__nv_bfloat16 v) { return __bfloat162float(v); }
template <typename E> __device__ __forceinline__ E from_f32(float v);
template <> __device__ __forceinline__ float from_f32<float>(float v) { return v; }
template <> __device__ __forceinline__ __nv_bfloat16 from_f32<__nv_bfloat16>(float v) {
    return __float2bfloat16_rn(v);
}

// 1 / (1 + exp(-v)), as e / (1 + e) with e = exp(-|v|) for v < 0: no overflow, and full
// relative accuracy down to the smallest normal result.
__device__ __forceinline__ float sigmoid(float v) {
    const float e = __expf(-fabsf(v));
    return __fdividef(v < 0.f ? e : 1.f, 1.f + e);
}

__device__ __forceinline__ float activate(float v, int act) {
    if (act == GDN_ACT_NONE) return v;
    const float s = sigmoid(v);
    return act == GDN_ACT_SILU ? v * s : s;
}

__device__ __forceinline__ int valid_tokens(const int32_t *lengths, int b, int T) {
    return lengths ? min(max(lengths[b], 0), T) : T;
}

// A byte range, for the overlap checks of the C entries.
struct Span {
    uintptr_t lo = 0, hi = 0;
    Span(const void *p, size_t bytes) {
        if (p) { lo = reinterpret_cast<uintptr_t>(p); hi = lo + bytes; }
    }
    bool meets(const Span &o) const { return lo < o.hi && o.lo < hi; }
};

// Bytes from the first to behind the last element of a strided [B, T, row] tensor.
inline size_t strided_bytes(int B, int T, int64_t row, int64_t sb, int64_t st, size_t e) {
    if (B <= 0 || T <= 0) return 0;
    return (static_cast<size_t>(B - 1) * sb + static_cast<size_t>(T - 1) * st + row) * e;
}

inline bool is_aligned(const void *p, size_t a) {
    return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0;
}

// Whether a strided [B, T, row] tensor's rows are whole, aligned 16-byte pieces.
inline bool pieces16(const void *p, int B, int T, int64_t row, int64_t sb, int64_t st, size_t e) {
    return is_aligned(p, 16) && row * e % 16 == 0 && (B == 1 || sb * e % 16 == 0) &&
           (T == 1 || st * e % 16 == 0);
}

inline size_t elem_bytes(int dtype) { return dtype == GDN_BF16 ? 2 : 4; }

}  // namespace gdn
