// Shared by the convolution, scan and group norm kernels: element conversion,
// activations, 16-byte pieces, and the host's pointer checks.
#pragma once

#include <cstring>
#include <type_traits>

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

// Two fp32 values in one 64-bit register pair: one instruction works on both.
using F2 = uint64_t;
__device__ __forceinline__ F2 pack2(float lo, float hi) {
    F2 r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
    return r;
}
__device__ __forceinline__ void unpack2(F2 v, float &lo, float &hi) {
    asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(v));
}
__device__ __forceinline__ F2 fma2(F2 a, F2 b, F2 c) {
    F2 r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}
__device__ __forceinline__ F2 mul2(F2 a, F2 b) {
    F2 r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ F2 add2(F2 a, F2 b) {
    F2 r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}

// 2^v and 1 / v of the special function unit, results below 2^-126 flushed to 0
// (without the scaling instructions that keep them).
__device__ __forceinline__ float exp2_ftz(float v) {
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(v));
    return r;
}
__device__ __forceinline__ float rcp_ftz(float v) {
    float r;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(v));
    return r;
}

constexpr float kLog2e = 1.44269504088896340736f;

// 1 / (1 + exp(-v)). Far below 0 the exponential is inf and the quotient 0: what is lost
// there is below 2^-126.
__device__ __forceinline__ float sigmoid(float v) { return rcp_ftz(1.f + exp2_ftz(-kLog2e * v)); }

__device__ __forceinline__ float activate(float v, int act) {
    if (act == GDN_ACT_NONE) return v;
    const float s = sigmoid(v);
    return act == GDN_ACT_SILU ? v * s : s;
}

// Of two values: sigmoid, activate.
__device__ __forceinline__ F2 sigmoid2(F2 v) {
    float a, b;
    unpack2(mul2(v, pack2(-kLog2e, -kLog2e)), a, b);
    unpack2(add2(pack2(exp2_ftz(a), exp2_ftz(b)), pack2(1.f, 1.f)), a, b);
    return pack2(rcp_ftz(a), rcp_ftz(b));
}
__device__ __forceinline__ F2 activate2(F2 v, int act) {
    if (act == GDN_ACT_NONE) return v;
    const F2 s = sigmoid2(v);
    return act == GDN_ACT_SILU ? mul2(v, s) : s;
}

__device__ __forceinline__ int valid_tokens(const int32_t *lengths, int b, int T) {
    return lengths ? min(max(lengths[b], 0), T) : T;
}

// V elements moved as one piece (16 bytes, or a single element) and widened to fp32.
template <typename E, int V>
struct Piece {
    static_assert(V == 1 || V * sizeof(E) == 16, "one element or 16 bytes");
    using Raw = typename std::conditional<V == 1, E, uint4>::type;
    Raw raw;
    __device__ __forceinline__ void load(const E *p) { raw = __ldg(reinterpret_cast<const Raw *>(p)); }
    // through the coherent path: for memory that this launch also writes
    __device__ __forceinline__ void load_rw(const E *p) { raw = *reinterpret_cast<const Raw *>(p); }
    __device__ __forceinline__ void store(E *p) const { *reinterpret_cast<Raw *>(p) = raw; }
    __device__ __forceinline__ void zero() { memset(&raw, 0, sizeof(raw)); }
    __device__ __forceinline__ void widen(float (&f)[V]) const {
        if constexpr (V == 1) {
            f[0] = to_f32(raw);
        } else if constexpr (sizeof(E) == 4) {
            f[0] = __uint_as_float(raw.x); f[1] = __uint_as_float(raw.y);
            f[2] = __uint_as_float(raw.z); f[3] = __uint_as_float(raw.w);
        } else {
            // bf16's bits are the high half of the fp32's
            const uint32_t w[4] = {raw.x, raw.y, raw.z, raw.w};
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                f[2 * i] = __uint_as_float(w[i] << 16);
                f[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
            }
        }
    }
    // the same in pairs (a single element in both halves)
    static constexpr int pairs = (V + 1) / 2;
    __device__ __forceinline__ void widen(F2 (&f)[pairs]) const {
        float v[V];
        widen(v);
#pragma unroll
        for (int i = 0; i < pairs; ++i) f[i] = pack2(v[2 * i], v[V == 1 ? 0 : 2 * i + 1]);
    }
    __device__ __forceinline__ void round(const F2 (&f)[pairs]) {
        float v[V + 1];
#pragma unroll
        for (int i = 0; i < pairs; ++i) unpack2(f[i], v[2 * i], v[2 * i + 1]);
        round(reinterpret_cast<const float (&)[V]>(v));
    }
    __device__ __forceinline__ void round(const float (&f)[V]) {
        if constexpr (V == 1) {
            raw = from_f32<E>(f[0]);
        } else if constexpr (sizeof(E) == 4) {
            raw = make_uint4(__float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]),
                             __float_as_uint(f[3]));
        } else {
            uint32_t w[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const __nv_bfloat162 h = __floats2bfloat162_rn(f[2 * i], f[2 * i + 1]);
                w[i] = *reinterpret_cast<const uint32_t *>(&h);
            }
            raw = make_uint4(w[0], w[1], w[2], w[3]);
        }
    }
};

// Widened copies of V consecutive fp32 parameters (16-byte aligned when V is a multiple of 4).
template <int V>
__device__ __forceinline__ void load_f32(const float *p, float (&f)[V]) {
    if constexpr (V % 4 == 0) {
#pragma unroll
        for (int i = 0; i < V / 4; ++i) {
            const float4 q = __ldg(reinterpret_cast<const float4 *>(p) + i);
            f[4 * i] = q.x; f[4 * i + 1] = q.y; f[4 * i + 2] = q.z; f[4 * i + 3] = q.w;
        }
    } else {
#pragma unroll
        for (int i = 0; i < V; ++i) f[i] = __ldg(p + i);
    }
}

// Asynchronous copies of 16 or 4 bytes from global to shared memory, in groups.
__device__ __forceinline__ void copy16_async(void *smem, const void *g) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(
                     static_cast<uint32_t>(__cvta_generic_to_shared(smem))), "l"(g) : "memory");
}
__device__ __forceinline__ void copy4_async(void *smem, const void *g) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(
                     static_cast<uint32_t>(__cvta_generic_to_shared(smem))), "l"(g) : "memory");
}
__device__ __forceinline__ void copy_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N> __device__ __forceinline__ void copy_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
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
