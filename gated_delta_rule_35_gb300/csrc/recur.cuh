// Shared by the passes of the gated linear recurrence: the factors of a token, the tiles that
// both passes read through shared memory, and how a state passes from tile to tile.
//
// A block works on 64 channels in tiles of 16 tokens to a warp: a lane has two channels of all
// the warp's tokens, so what a token needs before and after the scan is taken once and two
// channels share an instruction. A warp's rows arrive in its own part of shared memory
// (cp.async, a ring of tiles), nothing to synchronise but the warp. The scan goes
//   within a lane    a tile's factors A = prod a and its end H from a zero state;
//   across warps     each warp passes the block's state through the (A, H) of the warps before it;
//   across blocks    with few channels a cluster of blocks takes consecutive tiles and every
//                    block passes the state through the others' (A, H) first.
// So every input is read once and every output written once, whatever the length.
#pragma once

#include "columns.cuh"

namespace gdn {

constexpr int kRecurEvery = GDN_RECUR_EVERY;   // tokens to a warp's tile: a kept state for each
constexpr int kRecurChannels = 64;             // channels of a block
constexpr int kMaxWarps = 8;
constexpr int kMaxRanks = 8;                   // blocks of a cluster

template <typename E>
struct RecurParams {
    const E *dy, *x, *decay, *gate;
    const float *rate, *h0, *dh_final;
    const int32_t *lengths;
    E *y, *dx, *d_decay, *d_gate;
    float *h_final, *states, *d_rate_part, *dh0;
    int64_t x_sb, x_st, a_sb, a_st, g_sb, g_st, dy_sb, dy_st;
    int B, T, D, scaling;
    // fill: bytes of a copy to shared memory (16, 4 or, element by element, 2);
    // pairs: whether the outputs' channel pairs are aligned
    int fill, pairs, ranks;
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
__device__ __forceinline__ float rsqrt_ftz(float v) {
    float r;
    asm("rsqrt.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(v));
    return r;
}
__device__ __forceinline__ F2 both(float v) { return pack2(v, v); }

// s = sigmoid(v) and n = sigmoid(-v) = 1 - s, both to a few roundings of themselves. The
// exponent's bound keeps their quotient in range: what it cuts is below 2^-126.
__device__ __forceinline__ void sigmoids2(F2 v, F2 &s, F2 &n) {
    float a, b;
    unpack2(mul2(v, both(-kLog2e)), a, b);
    const F2 e = pack2(exp2_ftz(min_nan(a, 126.f)), exp2_ftz(min_nan(b, 126.f)));
    unpack2(add2(e, both(1.f)), a, b);
    s = pack2(rcp_ftz(a), rcp_ftz(b));
    n = mul2(e, s);
}

// a = 2^t and n = 1 - a for t <= 0, both to a few roundings of themselves: with t = k + f, k
// whole and |f| <= 1/2, a = 2^k + 2^k p and n = (1 - 2^k) - 2^k p, where p = 2^f - 1 is a
// polynomial in f without a constant term (off by 2.1e-8 of itself at most), so that n keeps its
// bits where a is next to 1. Below 2^-126 a is 2^-126.
__device__ __forceinline__ void decay_factor2(F2 t, F2 &a, F2 &n) {
    constexpr float shift = 12582912.f;                // 1.5 2^23: rounds to whole numbers
    float t0, t1, r0, r1;
    unpack2(t, t0, t1);
    t = pack2(max_nan(t0, -126.f), max_nan(t1, -126.f));
    const F2 r = add2(t, both(shift));
    const F2 f = add2(t, mul2(add2(r, both(-shift)), both(-1.f)));
    unpack2(r, r0, r1);
    const F2 scale = pack2(__int_as_float((__float_as_int(r0) << 23) + (127 << 23)),
                           __int_as_float((__float_as_int(r1) << 23) + (127 << 23)));
    F2 p = fma2(both(1.54035122e-4f), f, both(1.33907353e-3f));
    p = fma2(p, f, both(9.61823761e-3f));
    p = fma2(p, f, both(5.55035733e-2f));
    p = fma2(p, f, both(2.40226492e-1f));
    p = fma2(p, f, both(6.93147182e-1f));
    p = mul2(p, f);
    a = fma2(scale, p, scale);
    const F2 minus = mul2(scale, both(-1.f));
    n = fma2(minus, p, add2(minus, both(1.f)));
}

// The input's factor m of a and n = 1 - a, and its reciprocal where it is a root; both 0 where 1 -
// a^2 is below the normal range, where the instruction takes it for 0.
__device__ __forceinline__ F2 input_factor2(F2 a, F2 n, int scaling, F2 &inverse) {
    if (scaling == GDN_RECUR_ROOT) {
        const F2 v = fma2(n, a, n);                    // 1 - a^2
        float v0, v1;
        unpack2(v, v0, v1);
        constexpr float tiny = 1.17549435e-38f;
        inverse = pack2(v0 >= tiny ? rsqrt_ftz(v0) : 0.f, v1 >= tiny ? rsqrt_ftz(v1) : 0.f);
        return mul2(v, inverse);
    }
    return scaling == GDN_RECUR_COMPLEMENT ? n : both(1.f);
}

// Two channels of a row in shared or global memory.
__device__ __forceinline__ F2 pair_of(const __nv_bfloat16 *p) {
    const uint32_t w = *reinterpret_cast<const uint32_t *>(p);
    return pack2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
}
__device__ __forceinline__ F2 pair_of(const float *p) { return *reinterpret_cast<const F2 *>(p); }

// Stores channels c and c + 1 (those below D) of a row, rounded.
__device__ __forceinline__ void store_pair(__nv_bfloat16 *row, int c, int D, bool pairs, F2 v) {
    float a, b;
    unpack2(v, a, b);
    if (pairs) {
        if (c < D) *reinterpret_cast<__nv_bfloat162 *>(row + c) = __floats2bfloat162_rn(a, b);
    } else {
        if (c < D) row[c] = __float2bfloat16_rn(a);
        if (c + 1 < D) row[c + 1] = __float2bfloat16_rn(b);
    }
}
__device__ __forceinline__ void store_pair(float *row, int c, int D, bool pairs, F2 v) {
    if (pairs) {
        if (c < D) *reinterpret_cast<F2 *>(row + c) = v;
    } else {
        float a, b;
        unpack2(v, a, b);
        if (c < D) row[c] = a;
        if (c + 1 < D) row[c + 1] = b;
    }
}
__device__ __forceinline__ F2 load_pair(const float *row, int c, int D, bool pairs) {
    if (pairs && c < D) return *reinterpret_cast<const F2 *>(row + c);
    return pack2(c < D ? row[c] : 0.f, c + 1 < D ? row[c + 1] : 0.f);
}

// A warp's tile of one tensor: kRecurEvery rows of kRecurChannels values.
template <typename E>
struct Rows {
    static constexpr int bytes = kRecurEvery * kRecurChannels * sizeof(E);
};

// Copies rows t .. t + 15 (those below n), channels c0 .. c0 + 63 (those below D), of a sequence to
// `to`, asynchronously where the alignment allows. Rows behind the sequence take `other`,
// written for the pair of channels that the lane will read.
template <typename E>
__device__ __forceinline__ void fill_rows(E *to, const E *from, int64_t stride, int t, int n, int c0, int D, int fill,
                                          float other) {
    const int lane = threadIdx.x % 32;
    from += t * stride + c0;
    const int rows = min(kRecurEvery, n - t);
    if (fill == 16) {
        constexpr int V = 16 / sizeof(E), per_row = kRecurChannels / V, step = 32 / per_row;
        const int c = lane % per_row * V;
        int row = lane / per_row;
        from += row * stride + c;
        to += row * kRecurChannels + c;
        if (c0 + c < D) {
#pragma unroll
            for (; row < kRecurEvery; row += step) {
                if (row < rows) copy16_async(to, from);
                from += step * stride;
                to += step * kRecurChannels;
            }
        }
        to -= row * kRecurChannels + c;
    } else if (fill == 4) {
        constexpr int V = 4 / sizeof(E);
        for (int row = 0; row < rows; ++row)
#pragma unroll
            for (int c = lane * V; c < kRecurChannels; c += 32 * V)
                if (c0 + c < D) copy4_async(to + row * kRecurChannels + c, from + row * stride + c);
    } else {
#pragma unroll 4
        for (int row = 0; row < rows; ++row)
            for (int c = lane; c < kRecurChannels; c += 32)
                if (c0 + c < D) to[row * kRecurChannels + c] = from[row * stride + c];
    }
    for (int row = max(rows, 0); row < kRecurEvery; ++row) {
        E *at = to + row * kRecurChannels + 2 * lane;
        at[0] = at[1] = from_f32<E>(other);
    }
}

// (A, H) of two channels.
struct Through {
    F2 a, h;
};

__device__ __forceinline__ void store_cluster(uint32_t addr, const Through &v) {
    asm volatile("st.shared::cluster.v2.b64 [%0], {%1, %2};" ::"r"(addr), "l"(v.a), "l"(v.h) : "memory");
}

// The exchange of a tile: every warp gives its (A, H) and receives the state that its part
// starts from; `state`, the one before all parts, moves on to the one behind them. Parts
// are in time's order, or in the reverse one (REVERSE), by warp and, above that, by rank.
struct Exchange {
    Through warps[2][kMaxWarps][32], ranks[2][kMaxRanks][32];
};

template <bool REVERSE>
__device__ __forceinline__ F2 exchange(Exchange &e, int turn, int ranks, int rank, const Through &mine, F2 &state) {
    const int lane = threadIdx.x % 32, warp = threadIdx.x / 32, warps = blockDim.x / 32;
    Through(&part)[kMaxWarps][32] = e.warps[turn & 1];
    part[warp][lane] = mine;
    __syncthreads();
    F2 from = state;
    if (ranks > 1) {
        Through(&blocks)[kMaxRanks][32] = e.ranks[turn & 1];
        if (warp == 0) {
            Through all = {both(1.f), both(0.f)};
            for (int i = 0; i < warps; ++i) {
                const Through &w = part[REVERSE ? warps - 1 - i : i][lane];
                all.h = fma2(w.a, all.h, w.h);
                all.a = mul2(w.a, all.a);
            }
            const uint32_t addr = ptx::smem_u32(&blocks[rank][lane]);
            for (int r = 0; r < ranks; ++r) store_cluster(ptx::mapa_shared(addr, r), all);
        }
        ptx::cluster_sync();
        for (int i = 0; i < ranks; ++i) {
            const int r = REVERSE ? ranks - 1 - i : i;
            if (r == rank) from = state;
            state = fma2(blocks[r][lane].a, state, blocks[r][lane].h);
        }
    }
    F2 start = from;
    for (int i = 0; i < warps; ++i) {
        const int w = REVERSE ? warps - 1 - i : i;
        if (w == warp) start = from;
        from = fma2(part[w][lane].a, from, part[w][lane].h);
    }
    if (ranks == 1) state = from;
    return start;
}

inline gdn_status recur_check(const gdn_recur_problem *p) {
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


template <typename E>
RecurParams<E> recur_params(const gdn_recur_problem *p, const void *x, const void *decay, const void *gate,
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
inline cudaError_t copy_or_zero(float *to, const float *from, size_t bytes, cudaStream_t s) {
    if (!to || to == from) return cudaSuccess;
    return from ? cudaMemcpyAsync(to, from, bytes, cudaMemcpyDeviceToDevice, s) : cudaMemsetAsync(to, 0, bytes, s);
}


inline bool aligned_rows(const void *p, int B, int T, int64_t sb, int64_t st, size_t e, size_t a) {
    return is_aligned(p, a) && (B == 1 || sb * e % a == 0) && (T == 1 || st * e % a == 0);
}

// Copies of 16 bytes where every input's rows are whole pieces of them, else of 4, else elements.
template <typename E>
void recur_alignment(RecurParams<E> &p) {
    constexpr size_t e = sizeof(E);
    auto all = [&](size_t a) {
        return p.D * e % a == 0 && aligned_rows(p.x, p.B, p.T, p.x_sb, p.x_st, e, a) &&
               aligned_rows(p.decay, p.B, p.T, p.a_sb, p.a_st, e, a) &&
               (!p.gate || aligned_rows(p.gate, p.B, p.T, p.g_sb, p.g_st, e, a)) &&
               (!p.dy || aligned_rows(p.dy, p.B, p.T, p.dy_sb, p.dy_st, e, a));
    };
    p.fill = all(16) ? 16 : all(4) ? 4 : static_cast<int>(e);
    p.pairs = p.D % 2 == 0;
}

// Warps to a block: as many as a sequence's tokens fill, up to `most`. Blocks to a cluster: as
// many as leave the GPU's `places` for blocks filled once, and have tokens.
template <typename E>
void recur_shape(RecurParams<E> &p, int most, int places, int &warps) {
    warps = 1;
    while (warps < most && static_cast<int64_t>(warps) * kRecurEvery < p.T) ++warps;
    const int64_t blocks = static_cast<int64_t>(p.B) * ((p.D + kRecurChannels - 1) / kRecurChannels);
    p.ranks = 1;
    while (p.ranks < kMaxRanks && blocks * p.ranks * 2 <= places &&
           p.T > static_cast<int64_t>(p.ranks) * warps * kRecurEvery)
        p.ranks *= 2;
}

template <typename E>
cudaError_t recur_launch(void (*kernel)(RecurParams<E>), const RecurParams<E> &p, int warps, int bytes,
                         cudaStream_t s) {
    cudaError_t e = cudaFuncSetAttribute(reinterpret_cast<const void *>(kernel),
                                         cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>((p.D + kRecurChannels - 1) / kRecurChannels) * p.ranks, p.B);
    cfg.blockDim = dim3(32 * warps);
    cfg.dynamicSmemBytes = bytes;
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = p.ranks;
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = p.ranks > 1 ? 1 : 0;
    return cudaLaunchKernelEx(&cfg, kernel, p);
}

}  // namespace gdn
