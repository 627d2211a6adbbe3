// Selective state space scan: gdn_scan_fwd of include/gdn.h.
//
// A thread owns one channel with all of its N states in registers and walks the
// tokens in order.
#include "mixer.cuh"

namespace gdn {
namespace {

constexpr int kThreads = 128;

template <typename E>
struct ScanParams {
    const E *x, *dt, *z, *Bm, *Cm;
    const float *A, *skip, *dt_bias, *h0;
    const int32_t *lengths;
    E *y;
    float *h_final;
    int64_t x_sb, x_st, dt_sb, dt_st, z_sb, z_st, b_sb, b_st, c_sb, c_st;
    int T, D, N, G, softplus;
};

// log(1 + exp(v)) = max(v, 0) + log1p(exp(-|v|)).
__device__ __forceinline__ float softplus(float v) {
    return fmaxf(v, 0.f) + log1pf(expf(-fabsf(v)));
}

template <typename E, int NP>
__global__ void __launch_bounds__(kThreads) gdn_scan_kernel(const ScanParams<E> p) {
    const int d = blockIdx.x * kThreads + threadIdx.x, b = blockIdx.y;
    if (d >= p.D) return;
    const int n = valid_tokens(p.lengths, b, p.T);
    const int g = d / (p.D / p.G);
    const int64_t row = (static_cast<int64_t>(b) * p.D + d) * p.N;
    float h[NP];
#pragma unroll
    for (int i = 0; i < NP; ++i) h[i] = p.h0 && i < p.N ? p.h0[row + i] : 0.f;
    const float bias = p.dt_bias ? p.dt_bias[d] : 0.f, skip = p.skip ? p.skip[d] : 0.f;
    for (int t = 0; t < n; ++t) {
        const float x = to_f32(p.x[b * p.x_sb + t * p.x_st + d]);
        float dt = to_f32(p.dt[b * p.dt_sb + t * p.dt_st + d]) + bias;
        if (p.softplus) dt = softplus(dt);
        const E *bm = p.Bm + b * p.b_sb + t * p.b_st + static_cast<int64_t>(g) * p.N;
        const E *cm = p.Cm + b * p.c_sb + t * p.c_st + static_cast<int64_t>(g) * p.N;
        float y = 0.f;
#pragma unroll
        for (int i = 0; i < NP; ++i) {
            if (i < p.N) {
                const float a = expf(dt * p.A[static_cast<int64_t>(d) * p.N + i]);
                h[i] = fmaf(a, h[i], dt * x * to_f32(bm[i]));
                y = fmaf(to_f32(cm[i]), h[i], y);
            }
        }
        y = fmaf(skip, x, y);
        if (p.z) y *= activate(to_f32(p.z[b * p.z_sb + t * p.z_st + d]), GDN_ACT_SILU);
        p.y[(static_cast<int64_t>(b) * p.T + t) * p.D + d] = from_f32<E>(y);
    }
    if (p.h_final) {
#pragma unroll
        for (int i = 0; i < NP; ++i)
            if (i < p.N) p.h_final[row + i] = h[i];
    }
}

gdn_status check(const gdn_scan_problem *p) {
    if (!p) return GDN_ERR_INVALID_ARG;
    if (p->B <= 0 || p->D <= 0 || p->N <= 0 || p->G <= 0 || p->T < 0 || p->D % p->G != 0)
        return GDN_ERR_INVALID_ARG;
    if (p->dtype != GDN_F32 && p->dtype != GDN_BF16) return GDN_ERR_INVALID_ARG;
    if ((p->flags & ~GDN_SCAN_SOFTPLUS) || p->reserved) return GDN_ERR_INVALID_ARG;
    for (int64_t s : {p->x_stride_b, p->x_stride_t, p->dt_stride_b, p->dt_stride_t, p->z_stride_b,
                      p->z_stride_t, p->b_stride_b, p->b_stride_t, p->c_stride_b, p->c_stride_t})
        if (s < 0) return GDN_ERR_INVALID_ARG;
    if (p->N > 128 || p->B > 65535) return GDN_ERR_UNSUPPORTED;
    return GDN_OK;
}

size_t workspace_need(const gdn_scan_problem *) { return 0; }

template <typename E, int NP>
cudaError_t launch(const gdn_scan_problem *pr, const ScanParams<E> &p, cudaStream_t s) {
    const dim3 grid((pr->D + kThreads - 1) / kThreads, pr->B);
    gdn_scan_kernel<E, NP><<<grid, kThreads, 0, s>>>(p);
    return cudaGetLastError();
}

template <typename E>
cudaError_t dispatch(const gdn_scan_problem *pr, ScanParams<E> &p, cudaStream_t s) {
    p.x_sb = pr->x_stride_b; p.x_st = pr->x_stride_t;
    p.dt_sb = pr->dt_stride_b; p.dt_st = pr->dt_stride_t;
    p.z_sb = pr->z_stride_b; p.z_st = pr->z_stride_t;
    p.b_sb = pr->b_stride_b; p.b_st = pr->b_stride_t;
    p.c_sb = pr->c_stride_b; p.c_st = pr->c_stride_t;
    p.T = pr->T; p.D = pr->D; p.N = pr->N; p.G = pr->G;
    p.softplus = (pr->flags & GDN_SCAN_SOFTPLUS) ? 1 : 0;
    if (pr->N <= 8) return launch<E, 8>(pr, p, s);
    if (pr->N <= 16) return launch<E, 16>(pr, p, s);
    if (pr->N <= 32) return launch<E, 32>(pr, p, s);
    if (pr->N <= 64) return launch<E, 64>(pr, p, s);
    return launch<E, 128>(pr, p, s);
}

}  // namespace
}  // namespace gdn

extern "C" {

GDN_API size_t gdn_scan_workspace_bytes(const gdn_scan_problem *p) {
    return gdn::check(p) == GDN_OK ? gdn::workspace_need(p) : SIZE_MAX;
}

GDN_API gdn_status gdn_scan_fwd(const gdn_scan_problem *p, const void *x, const void *dt,
                                const float *A, const void *Bm, const void *Cm, const float *skip,
                                const void *z, const float *dt_bias, const float *h0,
                                const int32_t *lengths, void *y, float *h_final, void *workspace,
                                size_t workspace_bytes, void *stream) {
    using gdn::Span;
    using gdn::strided_bytes;
    const gdn_status st = gdn::check(p);
    if (st != GDN_OK) return st;
    const bool empty = p->T == 0;
    if (!empty && (!x || !dt || !A || !Bm || !Cm || !y)) return GDN_ERR_INVALID_ARG;
    const size_t e = gdn::elem_bytes(p->dtype);
    for (const void *ptr : {static_cast<const void *>(A), static_cast<const void *>(skip),
                            static_cast<const void *>(dt_bias), static_cast<const void *>(h0),
                            static_cast<const void *>(y), static_cast<const void *>(h_final),
                            static_cast<const void *>(workspace)})
        if (!gdn::is_aligned(ptr, 16)) return GDN_ERR_ALIGNMENT;
    for (const void *ptr : {x, dt, z, Bm, Cm})
        if (!gdn::is_aligned(ptr, e)) return GDN_ERR_ALIGNMENT;
    if (!gdn::is_aligned(lengths, 4)) return GDN_ERR_ALIGNMENT;
    const size_t need = gdn::workspace_need(p);
    if (need && (!workspace || workspace_bytes < need)) return GDN_ERR_WORKSPACE;
    const int64_t GN = static_cast<int64_t>(p->G) * p->N;
    const size_t state = static_cast<size_t>(p->B) * p->D * p->N * 4;
    const Span in[] = {Span(x, strided_bytes(p->B, p->T, p->D, p->x_stride_b, p->x_stride_t, e)),
                       Span(dt, strided_bytes(p->B, p->T, p->D, p->dt_stride_b, p->dt_stride_t, e)),
                       Span(z, strided_bytes(p->B, p->T, p->D, p->z_stride_b, p->z_stride_t, e)),
                       Span(Bm, strided_bytes(p->B, p->T, GN, p->b_stride_b, p->b_stride_t, e)),
                       Span(Cm, strided_bytes(p->B, p->T, GN, p->c_stride_b, p->c_stride_t, e)),
                       Span(A, static_cast<size_t>(p->D) * p->N * 4),
                       Span(skip, static_cast<size_t>(p->D) * 4),
                       Span(dt_bias, static_cast<size_t>(p->D) * 4),
                       Span(lengths, static_cast<size_t>(p->B) * 4),
                       Span(h0, state)};
    const Span sy(y, static_cast<size_t>(p->B) * p->T * p->D * e), sh(h_final, state);
    const Span sw(workspace, need);
    for (const Span &i : in) {
        const bool in_place = &i == &in[9] && h0 == h_final;
        if (i.meets(sy) || (i.meets(sh) && !in_place) || i.meets(sw)) return GDN_ERR_INVALID_ARG;
    }
    if (sy.meets(sh) || sw.meets(sy) || sw.meets(sh)) return GDN_ERR_INVALID_ARG;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    cudaError_t err = cudaSuccess;
    if (empty) {
        if (h_final && h0 && h0 != h_final)
            err = cudaMemcpyAsync(h_final, h0, state, cudaMemcpyDeviceToDevice, s);
        else if (h_final && !h0)
            err = cudaMemsetAsync(h_final, 0, state, s);
        return err == cudaSuccess ? GDN_OK : GDN_ERR_CUDA;
    }
    auto go = [&](auto tag) {
        using E = decltype(tag);
        gdn::ScanParams<E> a;
        a.x = static_cast<const E *>(x);
        a.dt = static_cast<const E *>(dt);
        a.z = static_cast<const E *>(z);
        a.Bm = static_cast<const E *>(Bm);
        a.Cm = static_cast<const E *>(Cm);
        a.A = A; a.skip = skip; a.dt_bias = dt_bias; a.h0 = h0;
        a.lengths = lengths;
        a.y = static_cast<E *>(y);
        a.h_final = h_final;
        return gdn::dispatch<E>(p, a, s);
    };
    err = p->dtype == GDN_BF16 ? go(__nv_bfloat16()) : go(float());
    return err == cudaSuccess ? GDN_OK : GDN_ERR_CUDA;
}

}  // extern "C"
