// Causal depthwise convolution over tokens with its window state: gdn_conv_fwd of
// include/gdn.h.
//
// A thread owns one channel and a run of tokens and keeps the W - 1 previous
// inputs in registers, so that each input is loaded once per run (plus the W - 1
// before the run).
#include "mixer.cuh"

namespace gdn {
namespace {

constexpr int kRun = 16;        // tokens per thread
constexpr int kThreads = 128;

template <typename E>
struct ConvParams {
    const E *x;
    const float *w, *bias;
    const E *state_in;
    const int32_t *lengths;
    E *y, *state_out;
    int64_t sb, st;
    int T, C, act;
};

// Input at token t of sequence b, channel c; t >= -(W - 1), tokens before 0 come
// from the window state.
template <typename E, int W>
__device__ __forceinline__ E input_at(const ConvParams<E> &p, int b, int t, int c) {
    if (t >= 0) return p.x[b * p.sb + t * p.st + c];
    return p.state_in ? p.state_in[(static_cast<int64_t>(b) * (W - 1) + W - 1 + t) * p.C + c]
                      : from_f32<E>(0.f);
}

template <typename E, int W>
__global__ void __launch_bounds__(kThreads) gdn_conv_kernel(const ConvParams<E> p) {
    const int c = blockIdx.x * kThreads + threadIdx.x;
    const int b = blockIdx.z, t0 = blockIdx.y * kRun;
    if (c >= p.C) return;
    const int n = valid_tokens(p.lengths, b, p.T);
    if (t0 < n) {
        float w[W], win[W];
#pragma unroll
        for (int k = 0; k < W; ++k) w[k] = p.w[static_cast<int64_t>(c) * W + k];
        const float bias = p.bias ? p.bias[c] : 0.f;
#pragma unroll
        for (int k = 0; k < W - 1; ++k) win[k + 1] = to_f32(input_at<E, W>(p, b, t0 - W + 1 + k, c));
        const int t1 = min(t0 + kRun, n);
        for (int t = t0; t < t1; ++t) {
#pragma unroll
            for (int k = 0; k < W - 1; ++k) win[k] = win[k + 1];
            win[W - 1] = to_f32(p.x[b * p.sb + t * p.st + c]);
            float v = bias;
#pragma unroll
            for (int k = 0; k < W; ++k) v = fmaf(w[k], win[k], v);
            p.y[(static_cast<int64_t>(b) * p.T + t) * p.C + c] = from_f32<E>(activate(v, p.act));
        }
    }
    // The thread that read this channel's state_in writes its state_out, after
    // reading all of it: the two may be the same buffer.
    if (t0 == 0 && p.state_out) {
        E last[W - 1];
#pragma unroll
        for (int k = 0; k < W - 1; ++k) last[k] = input_at<E, W>(p, b, n - W + 1 + k, c);
#pragma unroll
        for (int k = 0; k < W - 1; ++k)
            p.state_out[(static_cast<int64_t>(b) * (W - 1) + k) * p.C + c] = last[k];
    }
}

gdn_status check(const gdn_conv_problem *p) {
    if (!p) return GDN_ERR_INVALID_ARG;
    if (p->B <= 0 || p->C <= 0 || p->T < 0 || p->x_stride_b < 0 || p->x_stride_t < 0)
        return GDN_ERR_INVALID_ARG;
    if (p->dtype != GDN_F32 && p->dtype != GDN_BF16) return GDN_ERR_INVALID_ARG;
    if (p->act != GDN_ACT_NONE && p->act != GDN_ACT_SILU && p->act != GDN_ACT_SIGMOID)
        return GDN_ERR_INVALID_ARG;
    if (p->W < 2 || p->W > 4) return GDN_ERR_UNSUPPORTED;
    if (p->B > 65535 || p->T > 65535 * kRun) return GDN_ERR_UNSUPPORTED;
    return GDN_OK;
}

template <typename E, int W>
cudaError_t launch(const gdn_conv_problem *pr, const ConvParams<E> &p, cudaStream_t s) {
    const dim3 grid((pr->C + kThreads - 1) / kThreads, pr->T ? (pr->T + kRun - 1) / kRun : 1, pr->B);
    gdn_conv_kernel<E, W><<<grid, kThreads, 0, s>>>(p);
    return cudaGetLastError();
}

template <typename E>
cudaError_t dispatch(const gdn_conv_problem *pr, const void *x, const float *w, const float *bias,
                     const void *state_in, const int32_t *lengths, void *y, void *state_out,
                     cudaStream_t s) {
    ConvParams<E> p;
    p.x = static_cast<const E *>(x);
    p.w = w;
    p.bias = bias;
    p.state_in = static_cast<const E *>(state_in);
    p.lengths = lengths;
    p.y = static_cast<E *>(y);
    p.state_out = static_cast<E *>(state_out);
    p.sb = pr->x_stride_b;
    p.st = pr->x_stride_t;
    p.T = pr->T;
    p.C = pr->C;
    p.act = pr->act;
    switch (pr->W) {
        case 2: return launch<E, 2>(pr, p, s);
        case 3: return launch<E, 3>(pr, p, s);
        default: return launch<E, 4>(pr, p, s);
    }
}

}  // namespace
}  // namespace gdn

extern "C" {

GDN_API gdn_status gdn_conv_fwd(const gdn_conv_problem *p, const void *x, const float *weight,
                                const float *bias, const void *state_in, const int32_t *lengths,
                                void *y, void *state_out, void *stream) {
    using gdn::Span;
    const gdn_status st = gdn::check(p);
    if (st != GDN_OK) return st;
    const bool empty = p->T == 0;
    if (!empty && (!x || !weight || !y)) return GDN_ERR_INVALID_ARG;
    const size_t e = gdn::elem_bytes(p->dtype);
    for (const void *ptr : {static_cast<const void *>(weight), static_cast<const void *>(bias),
                            state_in, static_cast<const void *>(y),
                            static_cast<const void *>(state_out)})
        if (!gdn::is_aligned(ptr, 16)) return GDN_ERR_ALIGNMENT;
    if (!gdn::is_aligned(x, e) || !gdn::is_aligned(lengths, 4)) return GDN_ERR_ALIGNMENT;
    const size_t row = static_cast<size_t>(p->C) * e;
    const Span sx(x, gdn::strided_bytes(p->B, p->T, p->C, p->x_stride_b, p->x_stride_t, e));
    const Span sw(weight, static_cast<size_t>(p->C) * p->W * 4);
    const Span sbias(bias, static_cast<size_t>(p->C) * 4), sl(lengths, static_cast<size_t>(p->B) * 4);
    const Span sy(y, row * p->T * p->B);
    const Span si(state_in, row * (p->W - 1) * p->B), so(state_out, row * (p->W - 1) * p->B);
    if (sy.meets(sx) || sy.meets(sw) || sy.meets(sbias) || sy.meets(sl) || sy.meets(si) ||
        sy.meets(so) || so.meets(sx) || so.meets(sw) || so.meets(sbias) || so.meets(sl) ||
        (state_in != state_out && so.meets(si)))
        return GDN_ERR_INVALID_ARG;
    if (empty && (!state_out || state_in == state_out)) return GDN_OK;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    const cudaError_t err =
        p->dtype == GDN_BF16
            ? gdn::dispatch<__nv_bfloat16>(p, x, weight, bias, state_in, lengths, y, state_out, s)
            : gdn::dispatch<float>(p, x, weight, bias, state_in, lengths, y, state_out, s);
    return err == cudaSuccess ? GDN_OK : GDN_ERR_CUDA;
}

}  // extern "C"
