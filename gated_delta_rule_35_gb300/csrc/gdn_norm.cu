// Group norm of channels-last rows with an activation or a gate: gdn_group_norm of
// include/gdn.h.
//
// One CTA per (sequence, group): a pass for the mean, a pass for the variance about
// it, a pass that normalises.
#include "mixer.cuh"

namespace gdn {
namespace {

constexpr int kThreads = 256;

template <typename E>
struct NormParams {
    const E *x, *gate;
    const float *w, *bias;
    const int32_t *lengths;
    E *y;
    int64_t x_sb, x_st, g_sb, g_st;
    int T, C, G, act;
    float eps;
};

__device__ float block_sum(float v) {
    __shared__ float part[kThreads / 32];
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    __syncthreads();
    if (threadIdx.x % 32 == 0) part[threadIdx.x / 32] = v;
    __syncthreads();
    float s = 0.f;
#pragma unroll
    for (int i = 0; i < kThreads / 32; ++i) s += part[i];
    return s;
}

template <typename E>
__global__ void __launch_bounds__(kThreads) gdn_group_norm_kernel(const NormParams<E> p) {
    const int b = blockIdx.x / p.G, g = blockIdx.x % p.G;
    const int cg = p.C / p.G, n = valid_tokens(p.lengths, b, p.T);
    if (n == 0) return;
    const int64_t count = static_cast<int64_t>(n) * cg;
    const E *x = p.x + b * p.x_sb + g * cg;
    float s = 0.f;
    for (int64_t i = threadIdx.x; i < count; i += kThreads) s += to_f32(x[i / cg * p.x_st + i % cg]);
    const float mean = block_sum(s) / count;
    s = 0.f;
    for (int64_t i = threadIdx.x; i < count; i += kThreads) {
        const float d = to_f32(x[i / cg * p.x_st + i % cg]) - mean;
        s = fmaf(d, d, s);
    }
    const float rstd = rsqrtf(block_sum(s) / count + p.eps);
    for (int64_t i = threadIdx.x; i < count; i += kThreads) {
        const int64_t t = i / cg;
        const int c = g * cg + static_cast<int>(i % cg);
        float v = (to_f32(x[t * p.x_st + i % cg]) - mean) * rstd;
        v = fmaf(v, p.w ? p.w[c] : 1.f, p.bias ? p.bias[c] : 0.f);
        v = p.gate ? v * activate(to_f32(p.gate[b * p.g_sb + t * p.g_st + c]), p.act)
                   : activate(v, p.act);
        p.y[(static_cast<int64_t>(b) * p.T + t) * p.C + c] = from_f32<E>(v);
    }
}

gdn_status check(const gdn_group_norm_problem *p) {
    if (!p) return GDN_ERR_INVALID_ARG;
    if (p->B <= 0 || p->C <= 0 || p->G <= 0 || p->T < 0 || p->C % p->G != 0) return GDN_ERR_INVALID_ARG;
    if (p->x_stride_b < 0 || p->x_stride_t < 0 || p->gate_stride_b < 0 || p->gate_stride_t < 0 ||
        p->reserved || !(p->eps >= 0.f))
        return GDN_ERR_INVALID_ARG;
    if (p->dtype != GDN_F32 && p->dtype != GDN_BF16) return GDN_ERR_INVALID_ARG;
    if (p->act != GDN_ACT_NONE && p->act != GDN_ACT_SILU && p->act != GDN_ACT_SIGMOID)
        return GDN_ERR_INVALID_ARG;
    if (static_cast<int64_t>(p->B) * p->G > 0x7fffffffLL) return GDN_ERR_UNSUPPORTED;
    return GDN_OK;
}

template <typename E>
cudaError_t launch(const gdn_group_norm_problem *pr, const void *x, const float *w,
                   const float *bias, const void *gate, const int32_t *lengths, void *y,
                   cudaStream_t s) {
    NormParams<E> p;
    p.x = static_cast<const E *>(x);
    p.gate = static_cast<const E *>(gate);
    p.w = w;
    p.bias = bias;
    p.lengths = lengths;
    p.y = static_cast<E *>(y);
    p.x_sb = pr->x_stride_b;
    p.x_st = pr->x_stride_t;
    p.g_sb = pr->gate_stride_b;
    p.g_st = pr->gate_stride_t;
    p.T = pr->T;
    p.C = pr->C;
    p.G = pr->G;
    p.act = pr->act;
    p.eps = pr->eps;
    gdn_group_norm_kernel<E><<<pr->B * pr->G, kThreads, 0, s>>>(p);
    return cudaGetLastError();
}

}  // namespace
}  // namespace gdn

extern "C" {

GDN_API gdn_status gdn_group_norm(const gdn_group_norm_problem *p, const void *x,
                                  const float *weight, const float *bias, const void *gate,
                                  const int32_t *lengths, void *y, void *stream) {
    using gdn::Span;
    using gdn::strided_bytes;
    const gdn_status st = gdn::check(p);
    if (st != GDN_OK) return st;
    if (p->T == 0) return GDN_OK;
    if (!x || !y) return GDN_ERR_INVALID_ARG;
    const size_t e = gdn::elem_bytes(p->dtype);
    for (const void *ptr : {static_cast<const void *>(weight), static_cast<const void *>(bias),
                            static_cast<const void *>(y)})
        if (!gdn::is_aligned(ptr, 16)) return GDN_ERR_ALIGNMENT;
    if (!gdn::is_aligned(x, e) || !gdn::is_aligned(gate, e) || !gdn::is_aligned(lengths, 4))
        return GDN_ERR_ALIGNMENT;
    const bool in_place = x == y && (p->T == 1 || p->x_stride_t == p->C) &&
                          (p->B == 1 || p->x_stride_b == static_cast<int64_t>(p->T) * p->C);
    const Span sy(y, static_cast<size_t>(p->B) * p->T * p->C * e);
    const Span sx(x, strided_bytes(p->B, p->T, p->C, p->x_stride_b, p->x_stride_t, e));
    const Span sg(gate, strided_bytes(p->B, p->T, p->C, p->gate_stride_b, p->gate_stride_t, e));
    const size_t row = static_cast<size_t>(p->C) * 4;
    if ((sy.meets(sx) && !in_place) || sy.meets(sg) || sy.meets(Span(weight, row)) ||
        sy.meets(Span(bias, row)) || sy.meets(Span(lengths, static_cast<size_t>(p->B) * 4)))
        return GDN_ERR_INVALID_ARG;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    const cudaError_t err =
        p->dtype == GDN_BF16
            ? gdn::launch<__nv_bfloat16>(p, x, weight, bias, gate, lengths, y, s)
            : gdn::launch<float>(p, x, weight, bias, gate, lengths, y, s);
    return err == cudaSuccess ? GDN_OK : GDN_ERR_CUDA;
}

}  // extern "C"
