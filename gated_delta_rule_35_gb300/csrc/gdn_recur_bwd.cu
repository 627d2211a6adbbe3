// Backward pass of the gated linear recurrence: gdn_recur_bwd of include/gdn.h.
//
// With lam the gradient of h, lam_t = dy_t + a_{t+1} lam_{t+1} runs from the last token to the
// first through the same tiles as the forward pass (recur.cuh), of which it needs the decay
// factors alone; lam then stays in registers while the tile's tokens are taken in time's order, h
// anew from the state that the forward pass kept for them:
//   dx = lam m q,  dgate = lam m q (1 - q) x,  dlog = lam (a h_before + q x dm/dlog a)
//   ddecay = -dlog rate s (1 - s) (or dlog (1 - a)),  drate = -sum dlog s
// with dm/dlog a = -a^2 / m for the root, -a for the complement. Four tensors read and three
// written, and a quarter byte of states: 14 bytes a value in bf16, against 67 instructions; the
// factors are computed twice, since lam needs those of later tokens and registers hold one array.
//
// B4 T2048 D4096 bf16: 122 us, 3.92 TB/s (59% of a plain copy's 6.68); T32768 D2048 247 us, 3.87 TB/s;
// fp32 B4 T2048 D4096 159 us, 5.9 TB/s; D4097 243 us in bf16, 293 in fp32. Nine to twelve warps of
// 168 registers to an SM issue in 57% of the cycles, 256 blocks on 304 places. 128 registers and 16
// warps with a ring of one tile: 126 us for 132 then, but 281 for 263 on T32768.
#include <utility>

#include "recur.cuh"

namespace gdn {
namespace {

constexpr int kMaxWarps = 6;

template <typename E, int FORM>
__global__ void __launch_bounds__(32 * kMaxWarps, 2) gdn_recur_bwd_kernel(const RecurParams<E> p) {
    constexpr int kStages = kRecurStages<E>;
    __shared__ Exchange<kMaxWarps> ex;
    extern __shared__ uint4 ring[];
    constexpr bool gated = Form<FORM>::gated, rated = Form<FORM>::rated, whole = Form<FORM>::whole;
    constexpr int scaling = Form<FORM>::scaling;
    const bool pairs = whole || p.D % 2 == 0;
    const int lane = threadIdx.x % 32, warp = threadIdx.x / 32, warps = blockDim.x / 32;
    const int ranks = p.ranks, rank = blockIdx.x % ranks, c0 = blockIdx.x / ranks * kRecurChannels;
    const int c = c0 + 2 * lane, D = p.D;
    const bool second = c + 1 < D;
    const int64_t b = blockIdx.y;
    const int n = valid_tokens(p.lengths, b, p.T);
    const int tile = warps * kRecurEvery * ranks;          // of the cluster
    const int tiles = (n + tile - 1) / tile, first = (rank * warps + warp) * kRecurEvery;
    using Tile = Rows<E, whole>;
    const int slot = (gated ? 4 : 3) * Tile::bytes;
    unsigned char *mine = reinterpret_cast<unsigned char *>(ring) + warp * kStages * slot;
    struct Inputs {
        Tile x, decay, dy, gate;
    };
    auto inputs = [&](int i) {                             // i-th from the last
        unsigned char *at = mine + i % kStages * slot;
        const int t = (tiles - 1 - i) * tile + first;
        return Inputs{Tile(at, p.x + b * p.x_sb, p.x_st, t, c0),
                      Tile(at + Tile::bytes, p.decay + b * p.a_sb, p.a_st, t, c0),
                      Tile(at + 2 * Tile::bytes, p.dy + b * p.dy_sb, p.dy_st, t, c0),
                      Tile(at + 3 * Tile::bytes, gated ? p.gate + b * p.g_sb : nullptr, p.g_st, t, c0)};
    };
    auto fill = [&](int i) {
        if (i < tiles) {
            const Inputs in = inputs(i);
            const int left = n - ((tiles - 1 - i) * tile + first), width = min(kRecurChannels, D - c0);
            in.x.fill(left, width, p.x_span, 0.f);
            in.decay.fill(left, width, p.a_span, rated ? -INFINITY : INFINITY);    // behind the sequence a is 1
            in.dy.fill(left, width, p.dy_span, 0.f);
            if (gated) in.gate.fill(left, width, p.g_span, 0.f);
        }
        copy_commit();
    };
#pragma unroll
    for (int i = 0; i < kStages; ++i) fill(i);
    const F2 rate = rated ? load_pair(p.rate, c, D, pairs) : both(0.f), t_scale = mul2(rate, both(-kLog2e));
    const F2 minus_rate = mul2(rate, both(-1.f));
    float rate0, rate1;
    unpack2(rate, rate0, rate1);
    const F2 floors = rated ? pack2(root_floor(rate0), root_floor(rate1)) : both(root_floor(1.f));
    F2 d_rate = both(0.f);
    const int64_t chunks = (static_cast<int64_t>(p.T) + kRecurEvery - 1) / kRecurEvery;
    Scan<true, kMaxWarps> scan(ex, ranks, rank,
                               p.dh_final ? load_pair(p.dh_final + b * D, c, D, pairs) : both(0.f));
    for (int i = 0; i < tiles; ++i) {
        const int t = (tiles - 1 - i) * tile + first, left = c < D ? n - t : 0;
        F2 h = both(0.f);
        if (n > t) h = load_pair(p.states + (b * chunks + t / kRecurEvery) * D, c, D, pairs);
        copy_wait<kStages - 1>();
        __syncwarp();
        const Inputs in = inputs(i);
        F2 lam[kRecurEvery];                               // first the decay factors
        Through through = {both(1.f), both(0.f)};
#pragma unroll
        for (int j = kRecurEvery - 1; j >= 0; --j) {
            lam[j] = sigmoid2(in.decay.pair(j, lane));
            if (rated) lam[j] = decay_factor2(mul2(lam[j], t_scale));
            through.h = mul2(lam[j], add2(in.dy.pair(j, lane), through.h));
            through.a = mul2(lam[j], through.a);
        }
        F2 next = scan.step(i, through);
#pragma unroll
        for (int j = kRecurEvery - 1; j >= 0; --j) {
            const F2 a = lam[j];
            lam[j] = add2(in.dy.pair(j, lane), next);
            next = mul2(a, lam[j]);
        }
        int64_t out = (b * p.T + t) * D + c;
#pragma unroll
        for (int j = 0; j < kRecurEvery; ++j) {
            F2 s, s_n, a, a_n, inverse;
            sigmoids2(in.decay.pair(j, lane), s, s_n);
            if (rated) {
                decay_factor2(mul2(s, t_scale), a, a_n);
            } else {
                a = s;
                a_n = s_n;
            }
            const F2 m = input_factor2(a, a_n, scaling, floors, inverse), x = in.x.pair(j, lane);
            F2 qx = x, dx = mul2(m, lam[j]), d_gate;
            if (gated) {
                F2 q, q_n;
                sigmoids2(in.gate.pair(j, lane), q, q_n);
                qx = mul2(q, x);
                d_gate = mul2(mul2(dx, qx), q_n);
                dx = mul2(dx, q);
            }
            // dlog = lam a (h + q x (dm/dlog a) / a)
            F2 inner = h;
            if (scaling == GDN_RECUR_ROOT)
                inner = fma2(mul2(mul2(a, inverse), qx), both(-1.f), h);
            else if (scaling == GDN_RECUR_COMPLEMENT)
                inner = fma2(qx, both(-1.f), h);
            const F2 dlog = mul2(mul2(lam[j], a), inner);
            h = fma2(a, h, mul2(m, qx));
            const bool there = j < left;
            // s is not quite 0 behind the sequence, and what h ends with need not be finite
            if (rated && there) d_rate = fma2(dlog, s, d_rate);
            store_pair(p.dx + out, dx, there, second, pairs);
            if (gated) store_pair(p.d_gate + out, d_gate, there, second, pairs);
            store_pair(p.d_decay + out, mul2(dlog, rated ? mul2(minus_rate, mul2(s, s_n)) : a_n), there, second,
                       pairs);
            out += D;
        }
        __syncwarp();
        fill(i + kStages);
    }
    copy_wait<0>();
    const F2 carry = scan.last(tiles);
    if (p.dh0 && rank == 0 && warp == 0) store_pair(p.dh0 + b * D + c, carry, c < D, second, pairs);
    if (rated && p.d_rate_part) {
        F2 *sums = reinterpret_cast<F2 *>(ring);           // [warp][lane]; the ring is empty
        sums[threadIdx.x] = d_rate;
        __syncthreads();
        if (warp == 0) {
            for (int w = 1; w < warps; ++w) d_rate = add2(d_rate, sums[w * 32 + lane]);
            store_pair(p.d_rate_part + (b * ranks + rank) * D + c, mul2(d_rate, both(-1.f)), c < D, second, pairs);
        }
    }
}

size_t bwd_workspace(const gdn_recur_problem *p) {
    return p->T ? align_up(static_cast<size_t>(p->B) * kMaxRanks * p->D * 4) : 0;
}

template <typename E, int... FORMS>
cudaError_t launch(RecurParams<E> &p, float *d_rate, cudaStream_t s, std::integer_sequence<int, FORMS...>) {
    using Kernel = void (*)(RecurParams<E>);
    static constexpr Kernel table[] = {gdn_recur_bwd_kernel<E, FORMS>...};
    recur_rows(p);
    const int slot = kRecurStages<E> * (p.gate ? 4 : 3) * recur_row_bytes(p);
    const int warps = recur_shape<E, Exchange<kMaxWarps>>(p, kMaxWarps, slot);
    const cudaError_t err = recur_launch(recur_kernel<E>(table, p), p, warps, warps * slot, s);
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
    if (need && (!workspace || workspace_bytes < need)) return GDN_ERR_WORKSPACE;
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
        return launch<E>(a, d_rate, s, std::make_integer_sequence<int, kForms>());
    };
    const cudaError_t err = p->dtype == GDN_BF16 ? go(__nv_bfloat16()) : go(float());
    return err == cudaSuccess ? GDN_OK : GDN_ERR_CUDA;
}

}  // extern "C"
