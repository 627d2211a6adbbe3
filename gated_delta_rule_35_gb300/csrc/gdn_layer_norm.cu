// Layer norm of every token and its backward pass: gdn_layer_norm and gdn_layer_norm_bwd
// of include/gdn.h. A block to a token; the sums over tokens by a thread to a channel.
#include "columns.cuh"

namespace gdn {
namespace {

constexpr int kThreads = 256;
constexpr int kParts = 64;       // rows of partial sums

template <typename E>
struct LayerNormParams {
    const E *x, *dy;
    const float *w, *bias, *stats_in;
    const int32_t *lengths;
    E *y, *dx;
    float *stats, *part;
    int64_t x_sb, x_st, dy_sb, dy_st;
    int64_t rows;
    int T, C;
    bool rms;
    float eps;
};

// Sum over the block, for all of its threads.
__device__ __forceinline__ float block_sum(float v) {
    __shared__ float sums[kThreads / 32];
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    __syncthreads();
    if (threadIdx.x % 32 == 0) sums[threadIdx.x / 32] = v;
    __syncthreads();
    v = 0.f;
#pragma unroll
    for (int i = 0; i < kThreads / 32; ++i) v += sums[i];
    return v;
}

template <typename E>
__global__ void __launch_bounds__(kThreads) gdn_layer_norm_kernel(const LayerNormParams<E> p) {
    for (int64_t row = blockIdx.x; row < p.rows; row += gridDim.x) {
        const int64_t b = row / p.T, t = row % p.T;
        if (t >= valid_tokens(p.lengths, b, p.T)) continue;
        const E *x = p.x + b * p.x_sb + t * p.x_st;
        float mean = 0.f, s = 0.f;
        if (!p.rms) {
            for (int c = threadIdx.x; c < p.C; c += kThreads) s += to_f32(x[c]);
            mean = block_sum(s) / p.C;
        }
        s = 0.f;
        for (int c = threadIdx.x; c < p.C; c += kThreads) {
            const float d = to_f32(x[c]) - mean;
            s = fmaf(d, d, s);
        }
        const float rstd = rsqrtf(block_sum(s) / p.C + p.eps);
        for (int c = threadIdx.x; c < p.C; c += kThreads) {
            const float v = (to_f32(x[c]) - mean) * rstd;
            p.y[row * p.C + c] = from_f32<E>(fmaf(v, p.w ? p.w[c] : 1.f, p.bias ? p.bias[c] : 0.f));
        }
        if (p.stats && threadIdx.x == 0) {
            p.stats[2 * row] = mean;
            p.stats[2 * row + 1] = rstd;
        }
    }
}

template <typename E>
__global__ void __launch_bounds__(kThreads) gdn_layer_norm_dx_kernel(const LayerNormParams<E> p) {
    for (int64_t row = blockIdx.x; row < p.rows; row += gridDim.x) {
        const int64_t b = row / p.T, t = row % p.T;
        if (t >= valid_tokens(p.lengths, b, p.T)) continue;
        const E *x = p.x + b * p.x_sb + t * p.x_st, *dy = p.dy + b * p.dy_sb + t * p.dy_st;
        const float mean = p.stats_in[2 * row], rstd = p.stats_in[2 * row + 1];
        float s = 0.f, sx = 0.f;
        for (int c = threadIdx.x; c < p.C; c += kThreads) {
            const float v = to_f32(dy[c]) * (p.w ? p.w[c] : 1.f);
            s += v;
            sx = fmaf(v, (to_f32(x[c]) - mean) * rstd, sx);
        }
        s = p.rms ? 0.f : block_sum(s) / p.C;
        sx = block_sum(sx) / p.C;
        for (int c = threadIdx.x; c < p.C; c += kThreads) {
            const float v = to_f32(dy[c]) * (p.w ? p.w[c] : 1.f), xhat = (to_f32(x[c]) - mean) * rstd;
            p.dx[row * p.C + c] = from_f32<E>(rstd * (v - s - xhat * sx));
        }
    }
}

template <typename E>
__global__ void __launch_bounds__(kThreads) gdn_layer_norm_dw_kernel(const LayerNormParams<E> p) {
    const int c = blockIdx.x * kThreads + threadIdx.x;
    if (c >= p.C) return;
    float w = 0.f, bias = 0.f;
    for (int64_t row = blockIdx.y; row < p.rows; row += gridDim.y) {
        const int64_t b = row / p.T, t = row % p.T;
        if (t >= valid_tokens(p.lengths, b, p.T)) continue;
        const float dy = to_f32(p.dy[b * p.dy_sb + t * p.dy_st + c]);
        bias += dy;
        w = fmaf(dy, (to_f32(p.x[b * p.x_sb + t * p.x_st + c]) - p.stats_in[2 * row]) * p.stats_in[2 * row + 1], w);
    }
    p.part[blockIdx.y * 2LL * p.C + c] = w;
    p.part[(blockIdx.y * 2LL + 1) * p.C + c] = bias;
}

gdn_status check(const gdn_layer_norm_problem *p) {
    if (!p) return GDN_ERR_INVALID_ARG;
    if (p->B <= 0 || p->C <= 0 || p->T < 0 || (p->flags & ~GDN_LAYER_NORM_RMS)) return GDN_ERR_INVALID_ARG;
    if (p->x_stride_b < 0 || p->x_stride_t < 0 || p->dy_stride_b < 0 || p->dy_stride_t < 0 || !(p->eps >= 0.f))
        return GDN_ERR_INVALID_ARG;
    if (p->dtype != GDN_F32 && p->dtype != GDN_BF16) return GDN_ERR_INVALID_ARG;
    if (p->B > (1 << 30) || p->C > (1 << 30) || p->T > (1 << 30) ||
        static_cast<int64_t>(p->B) * p->T > INT32_MAX)
        return GDN_ERR_UNSUPPORTED;
    return GDN_OK;
}

size_t bwd_workspace(const gdn_layer_norm_problem *p) {
    return align_up(static_cast<size_t>(kParts) * 2 * p->C * 4);
}

template <typename E>
LayerNormParams<E> params(const gdn_layer_norm_problem *p, const void *x, const int32_t *lengths) {
    LayerNormParams<E> a = {};
    a.x = static_cast<const E *>(x);
    a.lengths = lengths;
    a.x_sb = p->x_stride_b; a.x_st = p->x_stride_t;
    a.dy_sb = p->dy_stride_b; a.dy_st = p->dy_stride_t;
    a.rows = static_cast<int64_t>(p->B) * p->T;
    a.T = p->T; a.C = p->C;
    a.rms = (p->flags & GDN_LAYER_NORM_RMS) != 0;
    a.eps = p->eps;
    return a;
}

}  // namespace
}  // namespace gdn

extern "C" {

GDN_API gdn_status gdn_layer_norm(const gdn_layer_norm_problem *p, const void *x,
                                  const float *weight, const float *bias, const int32_t *lengths,
                                  void *y, float *stats, void *stream) {
    using namespace gdn;
    const gdn_status st = check(p);
    if (st != GDN_OK) return st;
    if (p->T == 0) return GDN_OK;
    if (!x || !y) return GDN_ERR_INVALID_ARG;
    const size_t e = elem_bytes(p->dtype);
    for (const void *ptr : {static_cast<const void *>(weight), static_cast<const void *>(bias),
                            static_cast<const void *>(y), static_cast<const void *>(stats)})
        if (!is_aligned(ptr, 16)) return GDN_ERR_ALIGNMENT;
    if (!is_aligned(x, e) || !is_aligned(lengths, 4)) return GDN_ERR_ALIGNMENT;
    const bool in_place = x == y && (p->T == 1 || p->x_stride_t == p->C) &&
                          (p->B == 1 || p->x_stride_b == static_cast<int64_t>(p->T) * p->C);
    const size_t rows = static_cast<size_t>(p->B) * p->T, channels = static_cast<size_t>(p->C) * 4;
    const Span sx(x, strided_bytes(p->B, p->T, p->C, p->x_stride_b, p->x_stride_t, e));
    const Span sy(y, rows * p->C * e), ss(stats, rows * 8);
    for (const Span &i : {Span(weight, channels), Span(bias, channels), Span(lengths, static_cast<size_t>(p->B) * 4)})
        if (i.meets(sy) || i.meets(ss)) return GDN_ERR_INVALID_ARG;
    if ((sx.meets(sy) && !in_place) || sx.meets(ss) || sy.meets(ss)) return GDN_ERR_INVALID_ARG;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    auto go = [&](auto tag) {
        using E = decltype(tag);
        LayerNormParams<E> a = params<E>(p, x, lengths);
        a.w = weight;
        a.bias = bias;
        a.y = static_cast<E *>(y);
        a.stats = stats;
        const unsigned blocks = static_cast<unsigned>(a.rows < 152 * 8 ? a.rows : 152 * 8);
        gdn_layer_norm_kernel<E><<<blocks, kThreads, 0, s>>>(a);
        return cudaGetLastError();
    };
    const cudaError_t err = p->dtype == GDN_BF16 ? go(__nv_bfloat16()) : go(float());
    return err == cudaSuccess ? GDN_OK : GDN_ERR_CUDA;
}

GDN_API size_t gdn_layer_norm_bwd_workspace_bytes(const gdn_layer_norm_problem *p) {
    return gdn::check(p) == GDN_OK ? gdn::bwd_workspace(p) : SIZE_MAX;
}

GDN_API gdn_status gdn_layer_norm_bwd(const gdn_layer_norm_problem *p, const void *dy,
                                      const void *x, const float *stats, const float *weight,
                                      const int32_t *lengths, void *dx, float *d_weight,
                                      float *d_bias, void *workspace, size_t workspace_bytes,
                                      void *stream) {
    using namespace gdn;
    const gdn_status st = check(p);
    if (st != GDN_OK) return st;
    const bool empty = p->T == 0;
    if (!empty && (!dy || !x || !stats || !dx)) return GDN_ERR_INVALID_ARG;
    const size_t e = elem_bytes(p->dtype);
    for (const void *ptr : {static_cast<const void *>(stats), static_cast<const void *>(weight),
                            static_cast<const void *>(dx), static_cast<const void *>(d_weight),
                            static_cast<const void *>(d_bias), static_cast<const void *>(workspace)})
        if (!is_aligned(ptr, 16)) return GDN_ERR_ALIGNMENT;
    if (!is_aligned(dy, e) || !is_aligned(x, e) || !is_aligned(lengths, 4)) return GDN_ERR_ALIGNMENT;
    const size_t need = bwd_workspace(p);
    if (!workspace || workspace_bytes < need) return GDN_ERR_WORKSPACE;
    const size_t rows = static_cast<size_t>(p->B) * p->T, channels = static_cast<size_t>(p->C) * 4;
    const Span in[] = {Span(dy, strided_bytes(p->B, p->T, p->C, p->dy_stride_b, p->dy_stride_t, e)),
                       Span(x, strided_bytes(p->B, p->T, p->C, p->x_stride_b, p->x_stride_t, e)),
                       Span(stats, rows * 8), Span(weight, channels),
                       Span(lengths, static_cast<size_t>(p->B) * 4)};
    const Span out[] = {Span(dx, rows * p->C * e), Span(d_weight, channels), Span(d_bias, channels),
                        Span(workspace, need)};
    for (const Span &o : out) {
        for (const Span &i : in)
            if (o.meets(i)) return GDN_ERR_INVALID_ARG;
        for (const Span &o2 : out)
            if (&o != &o2 && o.meets(o2)) return GDN_ERR_INVALID_ARG;
    }
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (empty) {
        cudaError_t err = d_weight ? cudaMemsetAsync(d_weight, 0, channels, s) : cudaSuccess;
        if (err == cudaSuccess && d_bias) err = cudaMemsetAsync(d_bias, 0, channels, s);
        return err == cudaSuccess ? GDN_OK : GDN_ERR_CUDA;
    }
    auto go = [&](auto tag) {
        using E = decltype(tag);
        LayerNormParams<E> a = params<E>(p, x, lengths);
        a.dy = static_cast<const E *>(dy);
        a.stats_in = stats;
        a.w = weight;
        a.dx = static_cast<E *>(dx);
        a.part = static_cast<float *>(workspace);
        const unsigned blocks = static_cast<unsigned>(a.rows < 152 * 8 ? a.rows : 152 * 8);
        gdn_layer_norm_dx_kernel<E><<<blocks, kThreads, 0, s>>>(a);
        cudaError_t err = cudaGetLastError();
        if (err != cudaSuccess || (!d_weight && !d_bias)) return err;
        const unsigned parts = static_cast<unsigned>(a.rows < kParts ? a.rows : kParts);
        gdn_layer_norm_dw_kernel<E><<<dim3((p->C + kThreads - 1) / kThreads, parts), kThreads, 0, s>>>(a);
        err = cudaGetLastError();
        if (err != cudaSuccess) return err;
        return column_sums(a.part, parts, 2LL * p->C, p->C, d_weight, d_bias, s);
    };
    const cudaError_t err = p->dtype == GDN_BF16 ? go(__nv_bfloat16()) : go(float());
    return err == cudaSuccess ? GDN_OK : GDN_ERR_CUDA;
}

}  // extern "C"
