// The gated linear recurrence: gdn_recur_fwd of include/gdn.h.
//
// One read of x, decay and gate and one write of y, 8 bytes a value in bf16, against 34 instructions
// a value, five of them special functions. recur.cuh describes the tiles; a few tokens go to a
// kernel of their own, a thread to four channels of a sequence.
//
// B4 T2048 D4096 bf16, states kept: 59 us, 4.66 TB/s (70% of a plain copy's 6.68); 45 us with the
// arithmetic left out and 4 less without the exchange. 256 blocks on 152 SMs load 84% of their
// places, and where there are two the schedulers issue in 70% of the cycles. T32768 D2048, one
// sequence in clusters of 8: 145 us, 3.70 TB/s; 100 without the exchange, whose barrier of the
// cluster takes 1.4 us for every 1024 tokens. fp32 B4 T2048 D4096 93 us, 5.8 TB/s. Rows that are not
// whole pieces (D4097): 123 us in bf16, 164 in fp32. Tiles of 8 tokens to a warp with three times
// the warps took 66 to 76 us for 64, one with a ring of one tile 64.
#include <utility>

#include "recur.cuh"

namespace gdn {
namespace {

constexpr int kMaxWarps = 8;
constexpr int kStepTokens = 8;     // up to here the step kernel
constexpr int kStepThreads = 256;

// A token's decay factor and input of two channels; t_scale: -rate log2 e.
__device__ __forceinline__ void token2(F2 x, F2 decay, F2 gate, F2 t_scale, bool gated, bool rated, int scaling,
                                       F2 &a, F2 &u) {
    F2 n;
    if (rated)
        decay_factor2(mul2(sigmoid2(decay), t_scale), a, n);
    else
        sigmoids2(decay, a, n);
    u = x;
    if (gated) u = mul2(u, sigmoid2(gate));
    if (scaling == GDN_RECUR_ROOT) {
        float v0, v1;
        unpack2(fma2(n, a, n), v0, v1);                // 1 - a^2
        u = mul2(u, pack2(sqrt_ftz(v0), sqrt_ftz(v1)));
    } else if (scaling == GDN_RECUR_COMPLEMENT) {
        u = mul2(u, n);
    }
}

template <typename E, int FORM>
__global__ void __launch_bounds__(32 * kMaxWarps, 2) gdn_recur_kernel(const RecurParams<E> p) {
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
    const int slot = (gated ? 3 : 2) * Tile::bytes;
    unsigned char *mine = reinterpret_cast<unsigned char *>(ring) + warp * kStages * slot;
    struct Inputs {
        Tile x, decay, gate;
    };
    auto inputs = [&](int i) {
        unsigned char *at = mine + i % kStages * slot;
        const int t = i * tile + first;
        return Inputs{Tile(at, p.x + b * p.x_sb, p.x_st, t, c0),
                      Tile(at + Tile::bytes, p.decay + b * p.a_sb, p.a_st, t, c0),
                      Tile(at + 2 * Tile::bytes, gated ? p.gate + b * p.g_sb : nullptr, p.g_st, t, c0)};
    };
    auto fill = [&](int i) {
        if (i < tiles) {
            const Inputs in = inputs(i);
            const int left = n - (i * tile + first), width = min(kRecurChannels, D - c0);
            in.x.fill(left, width, p.x_span, 0.f);
            in.decay.fill(left, width, p.a_span, rated ? -INFINITY : INFINITY);    // behind the sequence a is 1
            if (gated) in.gate.fill(left, width, p.g_span, 0.f);
        }
        copy_commit();
    };
#pragma unroll
    for (int i = 0; i < kStages; ++i) fill(i);
    const F2 t_scale = rated ? mul2(load_pair(p.rate, c, D, pairs), both(-kLog2e)) : both(0.f);
    const int64_t chunks = (static_cast<int64_t>(p.T) + kRecurEvery - 1) / kRecurEvery;
    Scan<false, kMaxWarps> scan(ex, ranks, rank, p.h0 ? load_pair(p.h0 + b * D, c, D, pairs) : both(0.f));
    for (int i = 0; i < tiles; ++i) {
        copy_wait<kStages - 1>();
        __syncwarp();
        const Inputs in = inputs(i);
        F2 a[kRecurEvery], u[kRecurEvery];
        Through through = {both(1.f), both(0.f)};
#pragma unroll
        for (int j = 0; j < kRecurEvery; ++j) {
            token2(in.x.pair(j, lane), in.decay.pair(j, lane), gated ? in.gate.pair(j, lane) : both(0.f), t_scale,
                   gated, rated, scaling, a[j], u[j]);
            through.h = fma2(a[j], through.h, u[j]);
            through.a = mul2(a[j], through.a);
        }
        __syncwarp();
        fill(i + kStages);
        F2 h = scan.step(i, through);
        const int t = i * tile + first, left = c < D ? n - t : 0;
        if (p.states)
            store_pair(p.states + (b * chunks + t / kRecurEvery) * D + c, h, left > 0, second, pairs);
        E *y = p.y + (b * p.T + t) * D + c;
#pragma unroll
        for (int j = 0; j < kRecurEvery; ++j) {
            h = fma2(a[j], h, u[j]);
            store_pair(y, h, j < left, second, pairs);
            y += D;
        }
    }
    copy_wait<0>();
    const F2 state = scan.last(tiles);
    if (p.h_final && rank == 0 && warp == 0) store_pair(p.h_final + b * D + c, state, c < D, second, pairs);
}

// V consecutive values in pairs (a single one in both halves), and back, rounded.
template <int V, typename S>
__device__ __forceinline__ void load_values(const S *at, F2 (&f)[(V + 1) / 2]) {
    if constexpr (V == 1) {
        f[0] = both(to_f32(*at));
    } else if constexpr (sizeof(S) == 4) {
        const float4 q = *reinterpret_cast<const float4 *>(at);
        f[0] = pack2(q.x, q.y);
        f[1] = pack2(q.z, q.w);
    } else {
        const uint2 q = *reinterpret_cast<const uint2 *>(at);
        f[0] = pack2(__uint_as_float(q.x << 16), __uint_as_float(q.x & 0xffff0000u));
        f[1] = pack2(__uint_as_float(q.y << 16), __uint_as_float(q.y & 0xffff0000u));
    }
}
template <int V, typename S>
__device__ __forceinline__ void store_values(S *at, const F2 (&f)[(V + 1) / 2]) {
    float v[V + 1];
#pragma unroll
    for (int k = 0; k < (V + 1) / 2; ++k) unpack2(f[k], v[2 * k], v[2 * k + 1]);
    if constexpr (V == 1) {
        *at = from_f32<S>(v[0]);
    } else if constexpr (sizeof(S) == 4) {
        *reinterpret_cast<float4 *>(at) = make_float4(v[0], v[1], v[2], v[3]);
    } else {
        const __nv_bfloat162 lo = __floats2bfloat162_rn(v[0], v[1]), hi = __floats2bfloat162_rn(v[2], v[3]);
        *reinterpret_cast<uint2 *>(at) = make_uint2(*reinterpret_cast<const uint32_t *>(&lo),
                                                    *reinterpret_cast<const uint32_t *>(&hi));
    }
}

// A few tokens: a thread to V channels of a sequence.
template <typename E, int V, bool GATED, bool RATED>
__global__ void __launch_bounds__(kStepThreads) gdn_recur_step_kernel(const RecurParams<E> p) {
    const int c = (blockIdx.x * kStepThreads + threadIdx.x) * V;
    const int64_t b = blockIdx.y;
    if (c >= p.D) return;
    constexpr int P = (V + 1) / 2;
    const int n = valid_tokens(p.lengths, b, p.T);
    F2 h[P], t_scale[P];
#pragma unroll
    for (int k = 0; k < P; ++k) h[k] = t_scale[k] = both(0.f);
    if (p.h0) load_values<V>(p.h0 + b * p.D + c, h);
    if constexpr (RATED) {
        load_values<V>(p.rate + c, t_scale);
#pragma unroll
        for (int k = 0; k < P; ++k) t_scale[k] = mul2(t_scale[k], both(-kLog2e));
    }
    if (p.states && n > 0) store_values<V>(p.states + b * p.D + c, h);
    const E *x = p.x + b * p.x_sb + c, *decay = p.decay + b * p.a_sb + c;
    const E *gate = GATED ? p.gate + b * p.g_sb + c : nullptr;
    E *y = p.y + b * p.T * p.D + c;
    for (int t = 0; t < n; ++t) {
        F2 xs[P], ds[P], gs[P];
        load_values<V>(x + t * p.x_st, xs);
        load_values<V>(decay + t * p.a_st, ds);
        if constexpr (GATED) load_values<V>(gate + t * p.g_st, gs);
#pragma unroll
        for (int k = 0; k < P; ++k) {
            F2 a, u;
            token2(xs[k], ds[k], GATED ? gs[k] : both(0.f), t_scale[k], GATED, RATED, p.scaling, a, u);
            h[k] = fma2(a, h[k], u);
        }
        store_values<V>(y + static_cast<int64_t>(t) * p.D, h);
    }
    if (p.h_final) store_values<V>(p.h_final + b * p.D + c, h);
}
static_assert(kStepTokens <= kRecurEvery, "the step kernel keeps one state");

template <typename E, bool GATED, bool RATED>
cudaError_t launch_step(const RecurParams<E> &p, cudaStream_t s) {
    constexpr size_t a = 4 * sizeof(E);
    const bool wide = p.D % 4 == 0 && aligned_rows(p.x, p.B, p.T, p.x_sb, p.x_st, sizeof(E), a) &&
                      aligned_rows(p.decay, p.B, p.T, p.a_sb, p.a_st, sizeof(E), a) &&
                      (!GATED || aligned_rows(p.gate, p.B, p.T, p.g_sb, p.g_st, sizeof(E), a));
    const int pieces = wide ? p.D / 4 : p.D;
    const dim3 grid((pieces + kStepThreads - 1) / kStepThreads, p.B);
    if (wide)
        gdn_recur_step_kernel<E, 4, GATED, RATED><<<grid, kStepThreads, 0, s>>>(p);
    else
        gdn_recur_step_kernel<E, 1, GATED, RATED><<<grid, kStepThreads, 0, s>>>(p);
    return cudaGetLastError();
}

template <typename E, int... FORMS>
cudaError_t launch(RecurParams<E> &p, cudaStream_t s, std::integer_sequence<int, FORMS...>) {
    if (p.T <= kStepTokens) {
        if (p.gate) return p.rate ? launch_step<E, true, true>(p, s) : launch_step<E, true, false>(p, s);
        return p.rate ? launch_step<E, false, true>(p, s) : launch_step<E, false, false>(p, s);
    }
    using Kernel = void (*)(RecurParams<E>);
    static constexpr Kernel table[] = {gdn_recur_kernel<E, FORMS>...};
    recur_rows(p);
    const int slot = kRecurStages<E> * (p.gate ? 3 : 2) * recur_row_bytes(p);
    const int warps = recur_shape<E, Exchange<kMaxWarps>>(p, kMaxWarps, slot);
    return recur_launch(recur_kernel<E>(table, p), p, warps, warps * slot, s);
}

}  // namespace
}  // namespace gdn

extern "C" {

GDN_API gdn_status gdn_recur_fwd(const gdn_recur_problem *p, const void *x, const void *decay,
                                 const void *gate, const float *rate, const float *h0,
                                 const int32_t *lengths, void *y, float *h_final, float *states,
                                 void *stream) {
    using namespace gdn;
    const gdn_status st = recur_check(p);
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
    const size_t chunks = (static_cast<size_t>(p->T) + kRecurEvery - 1) / kRecurEvery;
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
        RecurParams<E> a = recur_params<E>(p, x, decay, gate, rate, lengths);
        a.h0 = h0;
        a.y = static_cast<E *>(y);
        a.h_final = h_final;
        a.states = states;
        return launch<E>(a, s, std::make_integer_sequence<int, kForms>());
    };
    const cudaError_t err = p->dtype == GDN_BF16 ? go(__nv_bfloat16()) : go(float());
    return err == cudaSuccess ? GDN_OK : GDN_ERR_CUDA;
}

}  // extern "C"
