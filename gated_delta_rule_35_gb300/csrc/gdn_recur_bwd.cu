// Backward pass of the gated linear recurrence: gdn_recur_bwd of include/gdn.h.
//
// With lam the gradient of h, lam_t = dy_t + a_{t+1} lam_{t+1} runs from the last token to the
// first through the same tiles as the forward pass (recur.cuh), of which it needs the decay
// factors alone; lam then stays in registers while the tile's tokens are taken in time's order, h
// anew from the state that the forward pass kept for them:
//   dx = lam m q,  dgate = lam m q (1 - q) x,  dlog = lam (a h_before + q x dm/dlog a)
//   ddecay = -dlog rate s (1 - s) (or dlog (1 - a)),  drate = -sum dlog s
// with dm/dlog a = -a^2 / m for the root, -a for the complement. Bound by memory: four tensors
// read and three written, the states a thirtieth of that.
#include "recur.cuh"

namespace gdn {
namespace {

constexpr int kStages = 2;

template <bool RATED>
__device__ __forceinline__ void decay2(F2 decay, F2 t_scale, F2 &s, F2 &s_n, F2 &a, F2 &a_n) {
    sigmoids2(decay, s, s_n);
    if constexpr (RATED) {
        decay_factor2(mul2(s, t_scale), a, a_n);
    } else {
        a = s;
        a_n = s_n;
    }
}

template <typename E, bool GATED>
constexpr int tile_bytes() { return (GATED ? 4 : 3) * Rows<E>::bytes; }

template <typename E, bool GATED, bool RATED>
__global__ void __launch_bounds__(128, 3) gdn_recur_bwd_kernel(const RecurParams<E> p) {
    __shared__ Exchange ex;
    extern __shared__ uint4 ring[];
    const int lane = threadIdx.x % 32, warp = threadIdx.x / 32, warps = blockDim.x / 32;
    const int ranks = p.ranks, rank = blockIdx.x % ranks, c0 = blockIdx.x / ranks * kRecurChannels;
    const int c = c0 + 2 * lane, D = p.D;
    const int64_t b = blockIdx.y;
    const int n = valid_tokens(p.lengths, b, p.T);
    const int tile = warps * kRecurEvery * ranks;          // of the cluster
    const int tiles = (n + tile - 1) / tile, first = (rank * warps + warp) * kRecurEvery;
    E *mine = reinterpret_cast<E *>(ring) + warp * (kStages * tile_bytes<E, GATED>() / sizeof(E));
    constexpr int rows = Rows<E>::bytes / sizeof(E), tensors = GATED ? 4 : 3;
    auto fill = [&](int i) {                               // i-th from the last
        if (i < tiles) {
            E *to = mine + i % kStages * tensors * rows;
            const int t = (tiles - 1 - i) * tile + first;
            fill_rows(to, p.x + b * p.x_sb, p.x_st, t, n, c0, D, p.fill, 0.f);
            // behind the sequence a is 1
            fill_rows(to + rows, p.decay + b * p.a_sb, p.a_st, t, n, c0, D, p.fill, RATED ? -INFINITY : INFINITY);
            fill_rows(to + 2 * rows, p.dy + b * p.dy_sb, p.dy_st, t, n, c0, D, p.fill, 0.f);
            if constexpr (GATED) fill_rows(to + 3 * rows, p.gate + b * p.g_sb, p.g_st, t, n, c0, D, p.fill, 0.f);
        }
        copy_commit();
    };
#pragma unroll
    for (int i = 0; i < kStages; ++i) fill(i);
    const F2 rate = RATED ? load_pair(p.rate, c, D, p.pairs) : both(0.f), t_scale = mul2(rate, both(-kLog2e));
    const F2 minus_rate = mul2(rate, both(-1.f));
    F2 carry = p.dh_final ? load_pair(p.dh_final + b * D, c, D, p.pairs) : both(0.f), d_rate = both(0.f);
    const int64_t chunks = (static_cast<int64_t>(p.T) + kRecurEvery - 1) / kRecurEvery;
    if (ranks > 1) ptx::cluster_sync();                    // all blocks are there to be written to
    for (int i = 0; i < tiles; ++i) {
        const int t = (tiles - 1 - i) * tile + first, left = n - t;
        F2 h = both(0.f);
        if (left > 0) h = load_pair(p.states + (b * chunks + t / kRecurEvery) * D, c, D, p.pairs);
        copy_wait<kStages - 1>();
        __syncwarp();
        const E *from = mine + i % kStages * tensors * rows + 2 * lane;
        F2 lam[kRecurEvery];                               // first the decay factors
        Through through = {both(1.f), both(0.f)};
#pragma unroll
        for (int j = kRecurEvery - 1; j >= 0; --j) {
            const E *at = from + j * kRecurChannels;
            F2 a_n;
            if constexpr (RATED)
                decay_factor2(mul2(sigmoid2(pair_of(at + rows)), t_scale), lam[j], a_n);
            else
                sigmoids2(pair_of(at + rows), lam[j], a_n);
            through.h = mul2(lam[j], add2(pair_of(at + 2 * rows), through.h));
            through.a = mul2(lam[j], through.a);
        }
        F2 next = exchange<true>(ex, i, ranks, rank, through, carry);
#pragma unroll
        for (int j = kRecurEvery - 1; j >= 0; --j) {
            const F2 a = lam[j];
            lam[j] = add2(pair_of(from + j * kRecurChannels + 2 * rows), next);
            next = mul2(a, lam[j]);
        }
        const int64_t out = (b * p.T + t) * D;
#pragma unroll
        for (int j = 0; j < kRecurEvery; ++j) {
            const E *at = from + j * kRecurChannels;
            F2 s, s_n, a, a_n, inverse, q, q_n;
            decay2<RATED>(pair_of(at + rows), t_scale, s, s_n, a, a_n);
            const F2 m = input_factor2(a, a_n, p.scaling, inverse);
            const F2 x = pair_of(at);
            F2 qx = x, mlam = mul2(m, lam[j]);
            if constexpr (GATED) {
                sigmoids2(pair_of(at + 3 * rows), q, q_n);
                qx = mul2(q, x);
            }
            // dlog = lam a (h + q x (dm/dlog a) / a)
            F2 inner = h;
            if (p.scaling == GDN_RECUR_ROOT)
                inner = fma2(mul2(mul2(a, inverse), both(-1.f)), qx, h);
            else if (p.scaling == GDN_RECUR_COMPLEMENT)
                inner = fma2(qx, both(-1.f), h);
            const F2 dlog = mul2(mul2(lam[j], a), inner);
            h = fma2(a, h, mul2(m, qx));
            d_rate = RATED ? fma2(dlog, s, d_rate) : d_rate;
            if (j < left) {
                const int64_t at_out = out + static_cast<int64_t>(j) * D;
                store_pair(p.dx + at_out, c, D, p.pairs, GATED ? mul2(mlam, q) : mlam);
                if constexpr (GATED) store_pair(p.d_gate + at_out, c, D, p.pairs, mul2(mul2(mlam, qx), q_n));
                store_pair(p.d_decay + at_out, c, D, p.pairs,
                           mul2(dlog, RATED ? mul2(minus_rate, mul2(s, s_n)) : a_n));
            }
        }
        __syncwarp();
        fill(i + kStages);
    }
    copy_wait<0>();
    if (p.dh0 && rank == 0 && warp == 0) store_pair(p.dh0 + b * D, c, D, p.pairs, carry);
    if (RATED && p.d_rate_part) {
        F2 *sums = reinterpret_cast<F2 *>(ring);           // [warp][lane]; the ring is empty
        __syncthreads();
        sums[threadIdx.x] = d_rate;
        __syncthreads();
        if (warp == 0) {
            for (int w = 1; w < warps; ++w) d_rate = add2(d_rate, sums[w * 32 + lane]);
            store_pair(p.d_rate_part + (b * ranks + rank) * D, c, D, p.pairs, mul2(d_rate, both(-1.f)));
        }
    }
}

size_t bwd_workspace(const gdn_recur_problem *p) {
    return align_up(static_cast<size_t>(p->B) * kMaxRanks * p->D * 4);
}

template <typename E, bool GATED, bool RATED>
cudaError_t launch(RecurParams<E> &p, float *d_rate, cudaStream_t s) {
    recur_alignment(p);
    int warps;
    recur_shape(p, sizeof(E) == 2 ? 4 : 2, 3 * 152, warps);
    const cudaError_t err = recur_launch(gdn_recur_bwd_kernel<E, GATED, RATED>, p, warps,
                                         warps * kStages * tile_bytes<E, GATED>(), s);
    if (err != cudaSuccess || !d_rate) return err;
    return column_sums(p.d_rate_part, p.B * p.ranks, p.D, p.D, d_rate, nullptr, s);
}

}  // namespace
}  // namespace gdn

extern "C" {

GDN_API size_t gdn_recur_bwd_workspace_bytes(const gdn_recur_problem *p) {
    return gdn::recur_check(p) == GDN_OK ? gdn::bwd_workspace(p) : SIZE_MAX;
}

GDN_API gdn_status gdn_recur_bwd(const gdn_recur_problem *p, const void *dy, const void *x,
                                 const void *decay, const void *gate, const float *rate,
                                 const float *states, const float *dh_final, const int32_t *lengths,
                                 void *dx, void *d_decay, void *d_gate, float *d_rate, float *dh0,
                                 void *workspace, size_t workspace_bytes, void *stream) {
    using namespace gdn;
    const gdn_status st = recur_check(p);
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
    const size_t chunks = (static_cast<size_t>(p->T) + kRecurEvery - 1) / kRecurEvery;
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
        RecurParams<E> a = recur_params<E>(p, x, decay, gate, rate, lengths);
        a.dy = static_cast<const E *>(dy);
        a.states = const_cast<float *>(states);
        a.dh_final = dh_final;
        a.dx = static_cast<E *>(dx);
        a.d_decay = static_cast<E *>(d_decay);
        a.d_gate = static_cast<E *>(d_gate);
        a.dh0 = dh0;
        a.d_rate_part = d_rate ? static_cast<float *>(workspace) : nullptr;
        if (gate) return rate ? launch<E, true, true>(a, d_rate, s) : launch<E, true, false>(a, d_rate, s);
        return rate ? launch<E, false, true>(a, d_rate, s) : launch<E, false, false>(a, d_rate, s);
    };
    const cudaError_t err = p->dtype == GDN_BF16 ? go(__nv_bfloat16()) : go(float());
    return err == cudaSuccess ? GDN_OK : GDN_ERR_CUDA;
}

}  // extern "C"
