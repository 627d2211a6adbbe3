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
// So every input is read once and every output written once, whatever the length. A thread to a
// channel over all tokens, in their order, took 2198 us for 59 (B4 T2048 D4096 bf16, 16384 channels)
// and 34 ms for 145 us (T32768 D2048); lanes of four channels and 8 tokens would shuffle between
// halves of a warp.
#pragma once

#include <cstddef>

#include "columns.cuh"
#include "rows.cuh"

namespace gdn {

constexpr int kRecurEvery = GDN_RECUR_EVERY;   // tokens to a warp's tile: a kept state for each
constexpr int kRecurChannels = 64;             // channels of a block
constexpr int kMaxRanks = 8;                   // blocks of a cluster

template <typename E>
struct RecurParams {
    const E *dy, *x, *decay, *gate;
    const float *rate, *h0, *dh_final;
    const int32_t *lengths;
    E *y, *dx, *d_decay, *d_gate;
    float *h_final, *states, *d_rate_part, *dh0;
    int64_t x_sb, x_st, a_sb, a_st, g_sb, g_st, dy_sb, dy_st;
    RowSpan x_span, a_span, g_span, dy_span;
    int B, T, D, scaling;
    int whole;     // every input's rows are aligned 16-byte pieces
    int ranks;     // blocks to a cluster
};

__device__ __forceinline__ float rsqrt_ftz(float v) {
    float r;
    asm("rsqrt.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(v));
    return r;
}
__device__ __forceinline__ float sqrt_ftz(float v) {
    float r;
    asm("sqrt.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(v));
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
// polynomial in f without a constant term, so that n keeps its bits where a is next to 1. Of degree
// 6, the one whose largest error relative to 2^f - 1 is least there, found by Lawson's iteration (least
// squares, the weights multiplied by the errors each time) and rounded to fp32: off by 2.2e-8 of itself
// at most. Below 2^-126 a is 2^-126. The scale comes from the rounded k's bits: by the exponential's
// instruction, of which a token takes four already, 65 us for 62 (B4 T2048 D4096 bf16).
__device__ __forceinline__ F2 decay_scale2(F2 t, F2 &p) {
    constexpr float shift = 12582912.f;                // 1.5 2^23: rounds to whole numbers
    float k0, k1;
    unpack2(t, k0, k1);
    t = pack2(max_nan(k0, -126.f), max_nan(k1, -126.f));
    const F2 k = add2(t, both(shift)), f = fma2(add2(k, both(-shift)), both(-1.f), t);
    unpack2(k, k0, k1);
    p = fma2(both(1.54035122e-4f), f, both(1.33907353e-3f));
    p = fma2(p, f, both(9.61823761e-3f));
    p = fma2(p, f, both(5.55035733e-2f));
    p = fma2(p, f, both(2.40226492e-1f));
    p = fma2(p, f, both(6.93147182e-1f));
    p = mul2(p, f);
    return pack2(__int_as_float((__float_as_int(k0) << 23) + (127 << 23)),
                 __int_as_float((__float_as_int(k1) << 23) + (127 << 23)));
}
__device__ __forceinline__ F2 decay_factor2(F2 t) {
    F2 p;
    const F2 scale = decay_scale2(t, p);
    return fma2(scale, p, scale);
}
__device__ __forceinline__ void decay_factor2(F2 t, F2 &a, F2 &n) {
    F2 p;
    const F2 scale = decay_scale2(t, p), w = mul2(scale, p);
    a = add2(scale, w);
    n = fma2(w, both(-1.f), fma2(scale, both(-1.f), both(1.f)));
}

// The form of a problem, which its kernels know when they are compiled: asked in the token loops, it
// took rows that are not whole pieces 140 us for 124 forward and 305 for 243 backward (B4 T2048 D4097
// bf16), and whole ones 85 for 65 and 256 for 129 (D4096).
constexpr int kForms = 24;
template <int FORM>
struct Form {
    static constexpr bool gated = FORM & 1, rated = FORM >> 1 & 1;
    static constexpr int scaling = FORM % 12 >> 2;
    static constexpr bool whole = FORM < 12;           // rows of whole, aligned 16-byte pieces
};
constexpr int recur_form(bool gated, bool rated, int scaling, bool whole) {
    return (whole ? 0 : 12) + scaling * 4 + rated * 2 + gated;
}

// The input's factor m of a and n = 1 - a, and its reciprocal where it is a root; where 1 - a^2 is
// below the normal range m is below 2^-63 and the reciprocal 2^63. `floors` are root_floor's of the channels.
__device__ __forceinline__ F2 input_factor2(F2 a, F2 n, int scaling, F2 floors, F2 &inverse) {
    if (scaling == GDN_RECUR_ROOT) {
        const F2 v = fma2(n, a, n);                    // 1 - a^2
        float v0, v1, f0, f1;
        unpack2(v, v0, v1);
        unpack2(floors, f0, f1);
        inverse = pack2(rsqrt_ftz(fmaxf(v0, f0)), rsqrt_ftz(fmaxf(v1, f1)));
        return mul2(v, inverse);
    }
    return scaling == GDN_RECUR_COMPLEMENT ? n : both(1.f);
}
// The smallest 1 - a^2 whose root a reciprocal is taken of: the normal range's end. In a channel whose rate is
// 0, or below that range, m is 0 for every token and has no gradient: infinity, so that the reciprocal is 0.
__device__ __forceinline__ float root_floor(float rate) {
    constexpr float tiny = 1.17549435e-38f;
    return rate < tiny ? INFINITY : tiny;
}

// Two channels of a row in shared memory.
__device__ __forceinline__ F2 pair_of(const __nv_bfloat16 *p) {
    const uint32_t w = *reinterpret_cast<const uint32_t *>(p);
    return pack2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
}
__device__ __forceinline__ F2 pair_of(const float *p) { return *reinterpret_cast<const F2 *>(p); }

// Channels c and c + 1 of a row of D, those that are there: `pairs` where D is even.
__device__ __forceinline__ F2 load_pair(const float *row, int c, int D, bool pairs) {
    if (pairs) return c < D ? *reinterpret_cast<const F2 *>(row + c) : both(0.f);
    return pack2(c < D ? row[c] : 0.f, c + 1 < D ? row[c + 1] : 0.f);
}
__device__ __forceinline__ void store_pair(float *at, F2 v) { *reinterpret_cast<F2 *>(at) = v; }
__device__ __forceinline__ void store_pair(__nv_bfloat16 *at, F2 v) {
    float a, b;
    unpack2(v, a, b);
    *reinterpret_cast<__nv_bfloat162 *>(at) = __floats2bfloat162_rn(a, b);
}
// `there`: of the pair's first channel, in a row that is to be written.
template <typename S>
__device__ __forceinline__ void store_pair(S *at, F2 v, bool there, bool second, bool pairs) {
    if (pairs) {
        if (there) store_pair(at, v);
    } else {
        float a, b;
        unpack2(v, a, b);
        if (there) at[0] = from_f32<S>(a);
        if (there && second) at[1] = from_f32<S>(b);
    }
}

// A warp's tile of one tensor: kRecurEvery rows of kRecurChannels values. WHOLE rows are copied in
// 16-byte pieces; others value by value in fp32, and in bf16, whose values are less than an
// asynchronous copy moves, as the aligned pieces that they touch.
template <typename E, bool WHOLE>
struct Rows {
    static constexpr bool SHIFTED = !WHOLE && sizeof(E) == 2;
    static constexpr int pitch = kRecurChannels * sizeof(E) + (SHIFTED ? 16 : 0);
    static constexpr int bytes = kRecurEvery * pitch;
    unsigned char *at;
    const E *from;         // channel c0 of the tile's first token
    int64_t stride;

    __device__ __forceinline__ Rows(unsigned char *at, const E *sequence, int64_t stride, int t, int c0)
        : at(at), from(sequence + t * stride + c0), stride(stride) {}

    __device__ __forceinline__ E *row(int j) const {
        unsigned char *r = at + j * pitch;
        if constexpr (SHIFTED)      // by the low bits of the row's address
            r += (static_cast<uint32_t>(reinterpret_cast<uintptr_t>(from)) +
                  static_cast<uint32_t>(stride * static_cast<int>(sizeof(E))) * j) & 15;
        return reinterpret_cast<E *>(r);
    }
    // Channels 2 lane and 2 lane + 1 of token j; what is there in place of channels that the row does
    // not have is of no use.
    __device__ __forceinline__ F2 pair(int j, int lane) const {
        const E *v = row(j) + 2 * lane;
        if constexpr (!SHIFTED) return pair_of(v);
        return pack2(to_f32(v[0]), to_f32(v[1]));
    }
    // Copies the first `rows` rows' values, `width` of the kRecurChannels; the others, behind the
    // sequence, take `other`, written for the pair of channels that the lane will read.
    __device__ __forceinline__ void fill(int rows, int width, const RowSpan &span, float other) const {
        const int lane = threadIdx.x % 32;
        rows = min(rows, kRecurEvery);
        if constexpr (WHOLE) {
            constexpr int V = 16 / sizeof(E), per_row = kRecurChannels / V, step = 32 / per_row;
            const int c = lane % per_row * V, first = lane / per_row;
            if (c < width) {
                const E *f = from + first * stride + c;
                E *to = reinterpret_cast<E *>(at) + first * kRecurChannels + c;
#pragma unroll
                for (int k = 0; k < kRecurEvery / step; ++k) {
                    if (first + k * step < rows) copy16_async(to, f);
                    f += step * stride;
                    to += step * kRecurChannels;
                }
            }
        } else if constexpr (!SHIFTED) {
            const E *f = from + lane;
            E *to = reinterpret_cast<E *>(at) + lane;
            for (int j = 0; j < rows; ++j, f += stride, to += kRecurChannels)
#pragma unroll
                for (int c = 0; c < kRecurChannels; c += 32)
                    if (c + lane < width) copy4_async(to + c, f + c);
        } else {
            const RowCopy<E> copy(span, from, stride, rows, width);          // 9 pieces to a row, two rows at once
            for (int j = lane / 16; j < rows; j += 2) copy(at + j * pitch, from + j * stride, width, lane % 16);
        }
        for (int j = max(rows, 0); j < kRecurEvery; ++j) {
            E *v = row(j) + 2 * lane;
            v[0] = v[1] = from_f32<E>(other);
        }
    }
};

// (A, H) of two channels, which a store to another block takes in one piece of 16 bytes.
struct alignas(16) Through {
    F2 a, h;
};

__device__ __forceinline__ void store_cluster(uint32_t addr, const Through &v) {
    asm volatile("st.shared::cluster.v2.b64 [%0], {%1, %2};" ::"r"(addr), "l"(v.a), "l"(v.h) : "memory");
}

// The exchange of a tile: every warp gives its (A, H) and receives the state that its part
// starts from. Parts are in time's order, or in the reverse one (REVERSE), by warp and, above
// that, by rank. The state before all parts passes on from tile to tile: within a block
// through `state`, which the last warp writes and the others read behind the next
// tile's barrier; in a cluster every thread takes it through all blocks' (A, H).
template <int WARPS>
struct Exchange {
    Through warps[2][WARPS][32], ranks[2][kMaxRanks][32];
    F2 state[2][32];
};
static_assert(sizeof(Through) == 16 && alignof(Exchange<1>) % 16 == 0 && offsetof(Exchange<1>, ranks) % 16 == 0,
              "16-byte stores to another block");

template <bool REVERSE, int WARPS>
struct Scan {
    Exchange<WARPS> &e;
    int warps, ranks, rank, lane, place;               // place: the warp's, in order
    F2 state;                                          // of a cluster: before the next tile

    __device__ __forceinline__ Scan(Exchange<WARPS> &e, int ranks, int rank, F2 state)
        : e(e), warps(blockDim.x / 32), ranks(ranks), rank(REVERSE ? ranks - 1 - rank : rank),
          lane(threadIdx.x % 32), state(state) {
        place = REVERSE ? warps - 1 - static_cast<int>(threadIdx.x / 32) : threadIdx.x / 32;
        if (place == 0) e.state[0][lane] = state;
        if (ranks > 1) ptx::cluster_sync();            // all blocks are there to be written to
    }
    __device__ __forceinline__ F2 step(int turn, const Through &mine) {
        const int now = turn & 1;
        e.warps[now][place][lane] = mine;
        __syncthreads();
        F2 from;
        if (ranks == 1) {
            from = e.state[now][lane];
        } else {
            if (place == 0) {
                Through all = mine;
                for (int w = 1; w < warps; ++w) {
                    const Through &o = e.warps[now][w][lane];
                    all.h = fma2(o.a, all.h, o.h);
                    all.a = mul2(o.a, all.a);
                }
                const uint32_t addr = ptx::smem_u32(&e.ranks[now][rank][lane]);
                for (int r = 0; r < ranks; ++r) store_cluster(ptx::mapa_shared(addr, r), all);
            }
            ptx::cluster_sync();
            from = state;
#pragma unroll
            for (int r = 0; r < kMaxRanks; ++r) {
                if (r >= ranks) break;
                const Through &o = e.ranks[now][r][lane];
                if (r == rank) from = state;
                state = fma2(o.a, state, o.h);
            }
        }
#pragma unroll
        for (int w = 0; w < WARPS - 1; ++w) {
            if (w >= place) break;
            const Through &o = e.warps[now][w][lane];
            from = fma2(o.a, from, o.h);
        }
        if (ranks == 1 && place == warps - 1) e.state[now ^ 1][lane] = fma2(mine.a, from, mine.h);
        return from;
    }
    // The state behind `turns` tiles, for the lanes of any warp of any block.
    __device__ __forceinline__ F2 last(int turns) {
        __syncthreads();
        return ranks == 1 ? e.state[turns & 1][lane] : state;
    }
};

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

template <typename E>
void recur_rows(RecurParams<E> &p) {
    constexpr size_t e = sizeof(E);
    p.whole = p.D * e % 16 == 0 && aligned_rows(p.x, p.B, p.T, p.x_sb, p.x_st, e, 16) &&
              aligned_rows(p.decay, p.B, p.T, p.a_sb, p.a_st, e, 16) &&
              (!p.gate || aligned_rows(p.gate, p.B, p.T, p.g_sb, p.g_st, e, 16)) &&
              (!p.dy || aligned_rows(p.dy, p.B, p.T, p.dy_sb, p.dy_st, e, 16));
    p.x_span = row_span(p.x, p.B, p.T, p.D, p.x_sb, p.x_st, e);
    p.a_span = row_span(p.decay, p.B, p.T, p.D, p.a_sb, p.a_st, e);
    p.g_span = row_span(p.gate, p.B, p.T, p.D, p.g_sb, p.g_st, e);
    p.dy_span = row_span(p.dy, p.B, p.T, p.D, p.dy_sb, p.dy_st, e);
}

// Tiles in a warp's ring. In fp32 one: twice the warps with one tile each (T8192 D2048 70 -> 60 us, its
// gradients 117 -> 100; B4 T2048 D4097 224 -> 177 and 420 -> 322).
template <typename E>
constexpr int kRecurStages = sizeof(E) == 2 ? 2 : 1;

constexpr int kBlockShared = 228 * 1024 / 2 - 1024;    // of one of two blocks to an SM

// Whether a kernel may have that many blocks. They fill the GPU's places for two blocks to an SM once; those
// of a padded batch, whose shorter sequences leave their places early, may go beyond: by a tenth where
// clusters double, by a third in the gradients in bf16, which wait for arithmetic more than for memory. Time with
// more blocks over time without (events around the call, L2 flushed, medians of three runs), lengths spread evenly
// to a mean of 50, 80 and 90% of the longest and all alike:
//                                            forward               backward
//   a tenth, B5 T777 D1024 fp32        0.81 0.97 1.03 0.95   0.82 0.99 0.95 1.15
//   a tenth, B2 T3000 D2560 fp32       0.75 0.94 0.99 1.02   0.76 1.08 1.14 1.07
//   a tenth, B4 T4000 D1280 bf16       0.76 0.90 0.94 0.95   0.81 1.00 0.96 1.00
//   a third, B6 T2048 D2048 bf16       0.91 1.14 1.18 1.07   0.77 0.96 1.02 0.97
//   a third, B6 T2048 D2048 fp32       0.92 1.15 1.21 1.20   0.77 1.03 1.20 1.16
// and where single blocks became clusters, a tenth beyond the places:
//   B2 T4096 D5120 fp32                0.97 1.14 1.16 1.14   0.98 1.22 1.27 1.15
template <typename E>
bool recur_fits(const RecurParams<E> &p, int64_t blocks) {
    const int places = 2 * 152;
    if (!p.lengths) return blocks <= places;
    if (sizeof(E) == 2 && p.dx) return blocks <= places * 4 / 3;
    return blocks <= (p.ranks > 1 ? places * 11 / 10 : places);
}

// Warps to a block: as many as a sequence's tokens fill, up to `most` and to what lets two blocks,
// with `slot` bytes to a warp's ring, share an SM. Blocks to a cluster: as many as fit and have tokens.
template <typename E, typename X>
int recur_shape(RecurParams<E> &p, int most, int slot) {
    const int fit = (kBlockShared - static_cast<int>(sizeof(X))) / slot;
    int warps = 1;
    while (warps < most && warps < fit && static_cast<int64_t>(warps) * kRecurEvery < p.T) ++warps;
    const int64_t blocks = static_cast<int64_t>(p.B) * ((p.D + kRecurChannels - 1) / kRecurChannels);
    p.ranks = 1;
    while (p.ranks < kMaxRanks && recur_fits(p, blocks * p.ranks * 2) &&
           p.T > static_cast<int64_t>(p.ranks) * warps * kRecurEvery)
        p.ranks *= 2;
    return warps;
}

template <typename E>
cudaError_t recur_launch(void (*kernel)(RecurParams<E>), const RecurParams<E> &p, int warps, int bytes,
                         cudaStream_t s) {
    // one bound for all calls: a call of another size on another thread must not lower it
    cudaError_t e = cudaFuncSetAttribute(reinterpret_cast<const void *>(kernel),
                                         cudaFuncAttributeMaxDynamicSharedMemorySize, kBlockShared);
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

// Bytes of a warp's ring slot for one tensor.
template <typename E>
int recur_row_bytes(const RecurParams<E> &p) { return p.whole ? Rows<E, true>::bytes : Rows<E, false>::bytes; }

// The kernel of a problem's form.
template <typename E, typename K>
K recur_kernel(const K (&table)[kForms], const RecurParams<E> &p) {
    return table[recur_form(p.gate, p.rate, p.scaling, p.whole)];
}

}  // namespace gdn
