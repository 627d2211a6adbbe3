// Backward pass of the short causal convolution: gdn_conv_bwd of include/gdn.h. A thread to
// a channel of a sequence, token by token.
#include "columns.cuh"

namespace gdn {
namespace {

constexpr int kThreads = 128;

template <typename E>
struct ConvBwdParams {
    const E *x, *dy;
    const float *w, *bias;
    const E *state_in, *d_last;
    const int32_t *lengths;
    E *dx, *d_state;
    float *part;      // [runs of all sequences][C W + C]
    int64_t sb, st, dy_sb, dy_st;
    int B, T, C, act;
};

template <typename E, int W>
__global__ void __launch_bounds__(kThreads) gdn_conv_bwd_kernel(const ConvBwdParams<E> p) {
    const int c = blockIdx.x * kThreads + threadIdx.x;
    const int64_t b = blockIdx.y;
    if (c >= p.C) return;
    const int n = valid_tokens(p.lengths, b, p.T);
    float w[W], dw[W], db = 0.f;
    const float bias = p.bias ? p.bias[c] : 0.f;
#pragma unroll
    for (int k = 0; k < W; ++k) {
        w[k] = p.w[static_cast<int64_t>(c) * W + k];
        dw[k] = 0.f;
    }
    // in[k] is input t - W + 1 + k; g[k] the gradient of v at token t - W + 1 + k
    float in[W], g[W];
#pragma unroll
    for (int k = 0; k < W; ++k) {
        in[k] = k > 0 && p.state_in ? to_f32(p.state_in[(b * (W - 1) + k - 1) * p.C + c]) : 0.f;
        g[k] = 0.f;
    }
    // Token t gives the gradient of input t - W + 1; those of the last W - 1 tokens follow.
    E last[W - 1];
    for (int k = 0; k < W - 1; ++k)
        last[k] = p.d_last ? p.d_last[(b * (W - 1) + k) * p.C + c] : from_f32<E>(0.f);
    for (int t = 0; t < n + W - 1; ++t) {
#pragma unroll
        for (int k = 0; k < W - 1; ++k) {
            in[k] = in[k + 1];
            g[k] = g[k + 1];
        }
        g[W - 1] = 0.f;
        if (t < n) {
            in[W - 1] = to_f32(p.x[b * p.sb + t * p.st + c]);
            float v = bias;
#pragma unroll
            for (int k = 0; k < W; ++k) v = fmaf(w[k], in[k], v);
            float d = to_f32(p.dy[b * p.dy_sb + t * p.dy_st + c]);
            if (p.act != GDN_ACT_NONE) {
                const float s = sigmoid(v), s_n = sigmoid(-v);
                d *= p.act == GDN_ACT_SILU ? s * fmaf(v, s_n, 1.f) : s * s_n;
            }
            g[W - 1] = d;
            db += d;
#pragma unroll
            for (int k = 0; k < W; ++k) dw[k] = fmaf(d, in[k], dw[k]);
        }
        // the gradient of input i = t - W + 1: tokens i .. i + W - 1 took it with taps W - 1 .. 0
        const int i = t - W + 1;
        float d = 0.f;
#pragma unroll
        for (int k = 0; k < W; ++k) d = fmaf(w[W - 1 - k], g[k], d);
        const int from_end = i - (n - W + 1);         // place in the window that the call left
        if (from_end >= 0 && from_end < W - 1) d += to_f32(last[from_end]);
        if (i >= 0)
            p.dx[(b * p.T + i) * p.C + c] = from_f32<E>(d);
        else if (p.d_state)
            p.d_state[(b * (W - 1) + W - 1 + i) * p.C + c] = from_f32<E>(d);
    }
    float *part = p.part + b * p.C * (W + 1);
#pragma unroll
    for (int k = 0; k < W; ++k) part[static_cast<int64_t>(c) * W + k] = dw[k];
    part[static_cast<int64_t>(p.C) * W + c] = db;
}

gdn_status check(const gdn_conv_bwd_problem *p) {
    if (!p) return GDN_ERR_INVALID_ARG;
    if (p->B <= 0 || p->C <= 0 || p->T < 0 || p->x_stride_b < 0 || p->x_stride_t < 0 || p->dy_stride_b < 0 ||
        p->dy_stride_t < 0)
        return GDN_ERR_INVALID_ARG;
    if (p->dtype != GDN_F32 && p->dtype != GDN_BF16) return GDN_ERR_INVALID_ARG;
    if (p->act != GDN_ACT_NONE && p->act != GDN_ACT_SILU && p->act != GDN_ACT_SIGMOID)
        return GDN_ERR_INVALID_ARG;
    if (p->W < 2 || p->W > 4) return GDN_ERR_UNSUPPORTED;
    if (p->B > 65535 || p->C > (1 << 30) || p->T > (1 << 30) ||
        static_cast<int64_t>(p->C) * p->T > (1 << 30))
        return GDN_ERR_UNSUPPORTED;
    return GDN_OK;
}

size_t workspace_need(const gdn_conv_bwd_problem *p) {
    return align_up(static_cast<size_t>(p->B) * p->C * (p->W + 1) * 4);
}

template <typename E>
cudaError_t launch(const gdn_conv_bwd_problem *pr, ConvBwdParams<E> &p, float *d_weight, float *d_bias,
                   cudaStream_t s) {
    const dim3 grid((pr->C + kThreads - 1) / kThreads, pr->B);
    switch (pr->W) {
        case 2: gdn_conv_bwd_kernel<E, 2><<<grid, kThreads, 0, s>>>(p); break;
        case 3: gdn_conv_bwd_kernel<E, 3><<<grid, kThreads, 0, s>>>(p); break;
        default: gdn_conv_bwd_kernel<E, 4><<<grid, kThreads, 0, s>>>(p);
    }
    const cudaError_t err = cudaGetLastError();
    if (err != cudaSuccess) return err;
    const int64_t taps = static_cast<int64_t>(pr->C) * pr->W;
    return column_sums(p.part, pr->B, taps + pr->C, taps, d_weight, d_bias, s);
}

}  // namespace
}  // namespace gdn

extern "C" {

GDN_API size_t gdn_conv_bwd_workspace_bytes(const gdn_conv_bwd_problem *p) {
    return gdn::check(p) == GDN_OK ? gdn::workspace_need(p) : SIZE_MAX;
}

GDN_API gdn_status gdn_conv_bwd(const gdn_conv_bwd_problem *p, const void *dy, const void *x,
                                const float *weight, const float *bias, const void *state_in,
                                const void *d_state_out, const int32_t *lengths, void *dx,
                                float *d_weight, float *d_bias, void *d_state_in, void *workspace,
                                size_t workspace_bytes, void *stream) {
    using namespace gdn;
    const gdn_status st = check(p);
    if (st != GDN_OK) return st;
    const bool empty = p->T == 0;
    if (!d_weight || (!empty && (!dy || !x || !weight || !dx))) return GDN_ERR_INVALID_ARG;
    const size_t e = elem_bytes(p->dtype);
    for (const void *ptr : {static_cast<const void *>(weight), static_cast<const void *>(bias), state_in,
                            d_state_out, static_cast<const void *>(dx), static_cast<const void *>(d_weight),
                            static_cast<const void *>(d_bias), static_cast<const void *>(d_state_in),
                            static_cast<const void *>(workspace)})
        if (!is_aligned(ptr, 16)) return GDN_ERR_ALIGNMENT;
    if (!is_aligned(dy, e) || !is_aligned(x, e) || !is_aligned(lengths, 4)) return GDN_ERR_ALIGNMENT;
    const size_t need = workspace_need(p);
    if (!workspace || workspace_bytes < need) return GDN_ERR_WORKSPACE;
    const size_t row = static_cast<size_t>(p->C) * e, channels = static_cast<size_t>(p->C) * 4;
    const size_t window = row * (p->W - 1) * p->B;
    const Span in[] = {Span(dy, strided_bytes(p->B, p->T, p->C, p->dy_stride_b, p->dy_stride_t, e)),
                       Span(x, strided_bytes(p->B, p->T, p->C, p->x_stride_b, p->x_stride_t, e)),
                       Span(weight, channels * p->W), Span(bias, channels), Span(state_in, window),
                       Span(lengths, static_cast<size_t>(p->B) * 4), Span(d_state_out, window)};
    const Span out[] = {Span(dx, row * p->T * p->B), Span(d_weight, channels * p->W), Span(d_bias, channels),
                        Span(workspace, need), Span(d_state_in, window)};
    for (const Span &o : out) {
        for (const Span &i : in) {
            const bool in_place = &i == &in[6] && &o == &out[4] && d_state_in == d_state_out;
            if (o.meets(i) && !in_place) return GDN_ERR_INVALID_ARG;
        }
        for (const Span &o2 : out)
            if (&o != &o2 && o.meets(o2)) return GDN_ERR_INVALID_ARG;
    }
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (empty) {
        cudaError_t err = cudaMemsetAsync(d_weight, 0, channels * p->W, s);
        if (err == cudaSuccess && d_bias) err = cudaMemsetAsync(d_bias, 0, channels, s);
        if (err == cudaSuccess && d_state_in && d_state_in != d_state_out)
            err = d_state_out ? cudaMemcpyAsync(d_state_in, d_state_out, window, cudaMemcpyDeviceToDevice, s)
                              : cudaMemsetAsync(d_state_in, 0, window, s);
        return err == cudaSuccess ? GDN_OK : GDN_ERR_CUDA;
    }
    auto go = [&](auto tag) {
        using E = decltype(tag);
        ConvBwdParams<E> a = {};
        a.x = static_cast<const E *>(x);
        a.dy = static_cast<const E *>(dy);
        a.w = weight;
        a.bias = bias;
        a.state_in = static_cast<const E *>(state_in);
        a.d_last = static_cast<const E *>(d_state_out);
        a.lengths = lengths;
        a.dx = static_cast<E *>(dx);
        a.d_state = static_cast<E *>(d_state_in);
        a.part = static_cast<float *>(workspace);
        a.sb = p->x_stride_b; a.st = p->x_stride_t;
        a.dy_sb = p->dy_stride_b; a.dy_st = p->dy_stride_t;
        a.B = p->B; a.T = p->T; a.C = p->C; a.act = p->act;
        return launch<E>(p, a, d_weight, d_bias, s);
    };
    const cudaError_t err = p->dtype == GDN_BF16 ? go(__nv_bfloat16()) : go(float());
    return err == cudaSuccess ? GDN_OK : GDN_ERR_CUDA;
}

}  // extern "C"
