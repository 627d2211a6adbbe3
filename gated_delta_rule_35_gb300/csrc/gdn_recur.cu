// The gated linear recurrence and its backward pass: gdn_recur_fwd and gdn_recur_bwd of
// include/gdn.h. A thread to a channel of a sequence, token by token.
#include "columns.cuh"

namespace gdn {
namespace {

constexpr int kThreads = 128;
constexpr int kEvery = GDN_RECUR_EVERY;

template <typename E>
struct RecurParams {
    const E *dy, *x, *decay, *gate;
    const float *rate, *h0, *dh_final;
    const int32_t *lengths;
    E *y, *dx, *d_decay, *d_gate;
    float *h_final, *states, *d_rate_part, *dh0;
    int64_t x_sb, x_st, a_sb, a_st, g_sb, g_st, dy_sb, dy_st;
    int B, T, D, scaling;
};

__device__ __forceinline__ float max_nan(float a, float b) {
    float r;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
    return r;
}
__device__ __forceinline__ float min_nan(float a, float b) {
    float r;
    asm("min.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
    return r;
}

// s = sigmoid(v) and n = sigmoid(-v) = 1 - s, both to a few roundings of themselves. The
// exponent's bound keeps their quotient in range: what it cuts is below 2^-126.
__device__ __forceinline__ void sigmoids(float v, float &s, float &n) {
    const float e = exp2_ftz(min_nan(-kLog2e * v, 126.f));
    s = rcp_ftz(1.f + e);
    n = e * s;
}

// a = exp(g) and n = 1 - a for g <= 0, both to a few roundings of themselves: with
// g log2 e = k + f, k whole and |f| <= 1/2, a = 2^k + 2^k p and n = (1 - 2^k) - 2^k p, where
// p = 2^f - 1 is a polynomial without a constant term.
__device__ __forceinline__ void decay_factor(float g, float &a, float &n) {
    const float t = max_nan(g * kLog2e, -126.f);
    constexpr float shift = 12582912.f;                // 1.5 2^23: rounds to whole numbers
    const float r = t + shift;
    const float f = t - (r - shift);
    const float scale = __int_as_float((__float_as_int(r) + 127) << 23);
    float p = 1.54035122e-4f;                          // off by 2.1e-8 of itself at most
    p = fmaf(p, f, 1.33907353e-3f);
    p = fmaf(p, f, 9.61823761e-3f);
    p = fmaf(p, f, 5.55035733e-2f);
    p = fmaf(p, f, 2.40226492e-1f);
    p = fmaf(p, f, 6.93147182e-1f);
    p *= f;
    a = fmaf(scale, p, scale);
    n = fmaf(-scale, p, 1.f - scale);
}

struct Factors {
    float s, s_n;     // sigmoid(decay), 1 - it
    float a, a_n;     // the decay factor, 1 - it
    float m, m_log;   // the input's factor, its derivative by log a
    float q, q_n;     // the gate, 1 - it (1 and 0 without one)
};

__device__ __forceinline__ Factors factors(float decay, float gate, bool gated, float rate, bool rated,
                                           int scaling) {
    Factors f;
    sigmoids(decay, f.s, f.s_n);
    if (rated) {
        decay_factor(-rate * f.s, f.a, f.a_n);
    } else {
        f.a = f.s;
        f.a_n = f.s_n;
    }
    f.m = 1.f;
    f.m_log = 0.f;
    if (scaling == GDN_RECUR_COMPLEMENT) {
        f.m = f.a_n;
        f.m_log = -f.a;
    } else if (scaling == GDN_RECUR_ROOT) {
        const float v = fmaf(f.a_n, f.a, f.a_n);       // 1 - a^2
        const float i = v > 0.f ? rsqrtf(v) : 0.f;
        f.m = v * i;
        f.m_log = -f.a * f.a * i;
    }
    f.q = 1.f;
    f.q_n = 0.f;
    if (gated) sigmoids(gate, f.q, f.q_n);
    return f;
}

template <typename E>
__global__ void __launch_bounds__(kThreads) gdn_recur_kernel(const RecurParams<E> p) {
    const int d = blockIdx.x * kThreads + threadIdx.x;
    const int64_t b = blockIdx.y;
    if (d >= p.D) return;
    const int n = valid_tokens(p.lengths, b, p.T);
    const float rate = p.rate ? p.rate[d] : 0.f;
    const int64_t chunks = (static_cast<int64_t>(p.T) + kEvery - 1) / kEvery;
    float h = p.h0 ? p.h0[b * p.D + d] : 0.f;
    for (int t = 0; t < n; ++t) {
        if (p.states && t % kEvery == 0) p.states[(b * chunks + t / kEvery) * p.D + d] = h;
        const Factors f = factors(to_f32(p.decay[b * p.a_sb + t * p.a_st + d]),
                                  p.gate ? to_f32(p.gate[b * p.g_sb + t * p.g_st + d]) : 0.f, p.gate != nullptr,
                                  rate, p.rate != nullptr, p.scaling);
        h = fmaf(f.a, h, f.m * f.q * to_f32(p.x[b * p.x_sb + t * p.x_st + d]));
        p.y[(b * p.T + t) * p.D + d] = from_f32<E>(h);
    }
    if (p.h_final) p.h_final[b * p.D + d] = h;
}

template <typename E>
__global__ void __launch_bounds__(kThreads) gdn_recur_bwd_kernel(const RecurParams<E> p) {
    const int d = blockIdx.x * kThreads + threadIdx.x;
    const int64_t b = blockIdx.y;
    if (d >= p.D) return;
    const int n = valid_tokens(p.lengths, b, p.T);
    const bool rated = p.rate != nullptr, gated = p.gate != nullptr;
    const float rate = rated ? p.rate[d] : 0.f;
    const int64_t chunks = (static_cast<int64_t>(p.T) + kEvery - 1) / kEvery;
    float carry = p.dh_final ? p.dh_final[b * p.D + d] : 0.f, d_rate = 0.f;
    for (int k = (n + kEvery - 1) / kEvery - 1; k >= 0; --k) {
        float before[kEvery];
        float h = p.states[(b * chunks + k) * p.D + d];
        const int tokens = min(kEvery, n - k * kEvery);
        auto at = [&](int i) {
            const int64_t t = static_cast<int64_t>(k) * kEvery + i;
            return factors(to_f32(p.decay[b * p.a_sb + t * p.a_st + d]),
                           gated ? to_f32(p.gate[b * p.g_sb + t * p.g_st + d]) : 0.f, gated, rate, rated,
                           p.scaling);
        };
#pragma unroll
        for (int i = 0; i < kEvery; ++i) {
            if (i >= tokens) break;
            const int64_t t = static_cast<int64_t>(k) * kEvery + i;
            before[i] = h;
            const Factors f = at(i);
            h = fmaf(f.a, h, f.m * f.q * to_f32(p.x[b * p.x_sb + t * p.x_st + d]));
        }
#pragma unroll
        for (int i = kEvery - 1; i >= 0; --i) {
            if (i >= tokens) continue;
            const int64_t t = static_cast<int64_t>(k) * kEvery + i, out = (b * p.T + t) * p.D + d;
            const Factors f = at(i);
            const float x = to_f32(p.x[b * p.x_sb + t * p.x_st + d]);
            const float lam = to_f32(p.dy[b * p.dy_sb + t * p.dy_st + d]) + carry;
            carry = f.a * lam;
            const float dlog = lam * fmaf(f.a, before[i], f.q * x * f.m_log);
            p.dx[out] = from_f32<E>(lam * f.m * f.q);
            if (gated) p.d_gate[out] = from_f32<E>(lam * f.m * x * f.q * f.q_n);
            p.d_decay[out] = from_f32<E>(dlog * (rated ? -rate * f.s * f.s_n : f.a_n));
            d_rate = fmaf(-dlog, f.s, d_rate);
        }
    }
    if (p.dh0) p.dh0[b * p.D + d] = carry;
    if (p.d_rate_part) p.d_rate_part[b * p.D + d] = d_rate;
}

gdn_status check(const gdn_recur_problem *p) {
    if (!p) return GDN_ERR_INVALID_ARG;
    if (p->B <= 0 || p->D <= 0 || p->T < 0 || p->reserved) return GDN_ERR_INVALID_ARG;
    for (int64_t st : {p->x_stride_b, p->x_stride_t, p->decay_stride_b, p->decay_stride_t, p->gate_stride_b,
                       p->gate_stride_t, p->dy_stride_b, p->dy_stride_t})
        if (st < 0) return GDN_ERR_INVALID_ARG;
    if (p->dtype != GDN_F32 && p->dtype != GDN_BF16) return GDN_ERR_INVALID_ARG;
    if (p->scaling < GDN_RECUR_PLAIN || p->scaling > GDN_RECUR_ROOT) return GDN_ERR_INVALID_ARG;
    if (p->B > 65535 || p->D > (1 << 24) || p->T > (1 << 30)) return GDN_ERR_UNSUPPORTED;
    return GDN_OK;
}

size_t bwd_workspace(const gdn_recur_problem *p) {
    return align_up(static_cast<size_t>(p->B) * p->D * 4);
}

template <typename E>
RecurParams<E> params(const gdn_recur_problem *p, const void *x, const void *decay, const void *gate,
                      const float *rate, const int32_t *lengths) {
    RecurParams<E> a = {};
    a.x = static_cast<const E *>(x);
    a.decay = static_cast<const E *>(decay);
    a.gate = static_cast<const E *>(gate);
    a.rate = rate;
    a.lengths = lengths;
    a.x_sb = p->x_stride_b; a.x_st = p->x_stride_t;
    a.a_sb = p->decay_stride_b; a.a_st = p->decay_stride_t;
    a.g_sb = p->gate_stride_b; a.g_st = p->gate_stride_t;
    a.dy_sb = p->dy_stride_b; a.dy_st = p->dy_stride_t;
    a.B = p->B; a.T = p->T; a.D = p->D;
    a.scaling = p->scaling;
    return a;
}

// to <- from, or zeros without it.
cudaError_t copy_or_zero(float *to, const float *from, size_t bytes, cudaStream_t s) {
    if (!to || to == from) return cudaSuccess;
    return from ? cudaMemcpyAsync(to, from, bytes, cudaMemcpyDeviceToDevice, s) : cudaMemsetAsync(to, 0, bytes, s);
}

}  // namespace
}  // namespace gdn

extern "C" {

GDN_API gdn_status gdn_recur_fwd(const gdn_recur_problem *p, const void *x, const void *decay,
                                 const void *gate, const float *rate, const float *h0,
                                 const int32_t *lengths, void *y, float *h_final, float *states,
                                 void *stream) {
    using namespace gdn;
    const gdn_status st = check(p);
    if (st != GDN_OK) return st;
    const bool empty = p->T == 0;
    if (!empty && (!x || !decay || !y)) return GDN_ERR_INVALID_ARG;
    const size_t e = elem_bytes(p->dtype);
    for (const void *ptr : {static_cast<const void *>(rate), static_cast<const void *>(h0),
                            static_cast<const void *>(y), static_cast<const void *>(h_final),
                            static_cast<const void *>(states)})
        if (!is_aligned(ptr, 16)) return GDN_ERR_ALIGNMENT;
    for (const void *ptr : {x, decay, gate})
        if (!is_aligned(ptr, e)) return GDN_ERR_ALIGNMENT;
    if (!is_aligned(lengths, 4)) return GDN_ERR_ALIGNMENT;
    const size_t rows = static_cast<size_t>(p->B) * p->D;
    const size_t chunks = (static_cast<size_t>(p->T) + kEvery - 1) / kEvery;
    const Span in[] = {Span(x, strided_bytes(p->B, p->T, p->D, p->x_stride_b, p->x_stride_t, e)),
                       Span(decay, strided_bytes(p->B, p->T, p->D, p->decay_stride_b, p->decay_stride_t, e)),
                       Span(gate, strided_bytes(p->B, p->T, p->D, p->gate_stride_b, p->gate_stride_t, e)),
                       Span(rate, static_cast<size_t>(p->D) * 4), Span(lengths, static_cast<size_t>(p->B) * 4),
                       Span(h0, rows * 4)};
    const Span sy(y, rows * p->T * e), sh(h_final, rows * 4), ss(states, rows * chunks * 4);
    for (const Span &i : in) {
        const bool in_place = &i == &in[5] && h0 == h_final;
        if (i.meets(sy) || (i.meets(sh) && !in_place) || i.meets(ss)) return GDN_ERR_INVALID_ARG;
    }
    if (sy.meets(sh) || ss.meets(sy) || ss.meets(sh)) return GDN_ERR_INVALID_ARG;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (empty) return copy_or_zero(h_final, h0, rows * 4, s) == cudaSuccess ? GDN_OK : GDN_ERR_CUDA;
    auto go = [&](auto tag) {
        using E = decltype(tag);
        RecurParams<E> a = params<E>(p, x, decay, gate, rate, lengths);
        a.h0 = h0;
        a.y = static_cast<E *>(y);
        a.h_final = h_final;
        a.states = states;
        gdn_recur_kernel<E><<<dim3((p->D + kThreads - 1) / kThreads, p->B), kThreads, 0, s>>>(a);
        return cudaGetLastError();
    };
    const cudaError_t err = p->dtype == GDN_BF16 ? go(__nv_bfloat16()) : go(float());
    return err == cudaSuccess ? GDN_OK : GDN_ERR_CUDA;
}

GDN_API size_t gdn_recur_bwd_workspace_bytes(const gdn_recur_problem *p) {
    return gdn::check(p) == GDN_OK ? gdn::bwd_workspace(p) : SIZE_MAX;
}

GDN_API gdn_status gdn_recur_bwd(const gdn_recur_problem *p, const void *dy, const void *x,
                                 const void *decay, const void *gate, const float *rate,
                                 const float *states, const float *dh_final, const int32_t *lengths,
                                 void *dx, void *d_decay, void *d_gate, float *d_rate, float *dh0,
                                 void *workspace, size_t workspace_bytes, void *stream) {
    using namespace gdn;
    const gdn_status st = check(p);
    if (st != GDN_OK) return st;
    const bool empty = p->T == 0;
    if (!empty && (!dy || !x || !decay || !states || !dx || !d_decay || !gate != !d_gate))
        return GDN_ERR_INVALID_ARG;
    if (d_rate && !rate) return GDN_ERR_INVALID_ARG;
    const size_t e = elem_bytes(p->dtype);
    for (const void *ptr : {static_cast<const void *>(rate), static_cast<const void *>(states),
                            static_cast<const void *>(dh_final), static_cast<const void *>(dx),
                            static_cast<const void *>(d_decay), static_cast<const void *>(d_gate),
                            static_cast<const void *>(d_rate), static_cast<const void *>(dh0),
                            static_cast<const void *>(workspace)})
        if (!is_aligned(ptr, 16)) return GDN_ERR_ALIGNMENT;
    for (const void *ptr : {dy, x, decay, gate})
        if (!is_aligned(ptr, e)) return GDN_ERR_ALIGNMENT;
    if (!is_aligned(lengths, 4)) return GDN_ERR_ALIGNMENT;
    const size_t need = bwd_workspace(p);
    if (!workspace || workspace_bytes < need) return GDN_ERR_WORKSPACE;
    const size_t rows = static_cast<size_t>(p->B) * p->D, all = rows * p->T * e;
    const size_t chunks = (static_cast<size_t>(p->T) + kEvery - 1) / kEvery;
    const Span in[] = {Span(dy, strided_bytes(p->B, p->T, p->D, p->dy_stride_b, p->dy_stride_t, e)),
                       Span(x, strided_bytes(p->B, p->T, p->D, p->x_stride_b, p->x_stride_t, e)),
                       Span(decay, strided_bytes(p->B, p->T, p->D, p->decay_stride_b, p->decay_stride_t, e)),
                       Span(gate, strided_bytes(p->B, p->T, p->D, p->gate_stride_b, p->gate_stride_t, e)),
                       Span(rate, static_cast<size_t>(p->D) * 4), Span(states, rows * chunks * 4),
                       Span(lengths, static_cast<size_t>(p->B) * 4), Span(dh_final, rows * 4)};
    const Span out[] = {Span(dx, all), Span(d_decay, all), Span(d_gate, all),
                        Span(d_rate, static_cast<size_t>(p->D) * 4), Span(workspace, need), Span(dh0, rows * 4)};
    for (const Span &o : out) {
        for (const Span &i : in) {
            const bool in_place = &i == &in[7] && &o == &out[5] && dh0 == dh_final;
            if (o.meets(i) && !in_place) return GDN_ERR_INVALID_ARG;
        }
        for (const Span &o2 : out)
            if (&o != &o2 && o.meets(o2)) return GDN_ERR_INVALID_ARG;
    }
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (empty) {
        cudaError_t err = copy_or_zero(dh0, dh_final, rows * 4, s);
        if (err == cudaSuccess) err = copy_or_zero(d_rate, nullptr, static_cast<size_t>(p->D) * 4, s);
        return err == cudaSuccess ? GDN_OK : GDN_ERR_CUDA;
    }
    auto go = [&](auto tag) {
        using E = decltype(tag);
        RecurParams<E> a = params<E>(p, x, decay, gate, rate, lengths);
        a.dy = static_cast<const E *>(dy);
        a.states = const_cast<float *>(states);
        a.dh_final = dh_final;
        a.dx = static_cast<E *>(dx);
        a.d_decay = static_cast<E *>(d_decay);
        a.d_gate = static_cast<E *>(d_gate);
        a.dh0 = dh0;
        a.d_rate_part = d_rate ? static_cast<float *>(workspace) : nullptr;
        gdn_recur_bwd_kernel<E><<<dim3((p->D + kThreads - 1) / kThreads, p->B), kThreads, 0, s>>>(a);
        const cudaError_t err = cudaGetLastError();
        if (err != cudaSuccess || !d_rate) return err;
        return column_sums(static_cast<const float *>(workspace), p->B, p->D, p->D, d_rate, nullptr, s);
    };
    const cudaError_t err = p->dtype == GDN_BF16 ? go(__nv_bfloat16()) : go(float());
    return err == cudaSuccess ? GDN_OK : GDN_ERR_CUDA;
}

}  // extern "C"
