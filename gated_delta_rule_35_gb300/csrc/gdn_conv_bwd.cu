// Backward pass of the short causal convolution: gdn_conv_bwd of include/gdn.h.
//
// Bound by memory: x and dy read, dx written. A thread owns four channels over a run of tokens,
// token by token: with the window of inputs it takes the value before the activation anew and
// p = dy act', with the window of p the gradient of the input W - 1 tokens before, and adds p x to
// its gradients of the weights, which stay in registers. A run needs the inputs of W - 1 tokens
// before it and p of as many behind it, which its neighbours read too. The runs of a block add
// their gradients of the weights up and leave a row of partial sums. x and dy come through a ring
// in shared memory: of a thread's own where four channels side by side are whole, aligned
// accesses; else a thread's channels lie apart, so that neighbours' accesses do not, and come one by
// one (fp32), or the threads of a run copy the aligned 16-byte pieces that their part of a row touches
// (bf16, whose elements are less than an asynchronous copy moves).
//
// B8 T8192 C8192 W4 SiLU bf16: 555 us, 5.81 TB/s (87% of a plain copy's 6.68; the FMA pipe 57%, issue
// 60%, four blocks of 126 registers to an SM); 11 us of it are the sums over the 64 blocks of runs.
// B4 T4096 C4096 bf16 90 us (two rounds of blocks, the second two thirds full), fp32 136, C4097 195
// and 181. A thread to a channel over all tokens: 5161 us. Three blocks of 256 threads (80 registers)
// would spill: 844 us; eight tokens to a turn 598.
#include "columns.cuh"
#include "rows.cuh"

namespace gdn {
namespace {

constexpr int kThreads = 128;
constexpr int kChannels = 4;    // of a thread
constexpr int kUnroll = 4;      // tokens per turn
constexpr int kStages = 3;      // turns in the ring
constexpr int kMinRun = 8, kMinPieces = 8;
static_assert(kMinRun >= kUnroll && kUnroll >= 3, "W - 1");

template <typename E>
struct ConvBwdParams {
    const E *x, *dy;
    const float *w, *bias;
    const E *state_in, *d_last;
    const int32_t *lengths;
    E *dx, *d_state;
    float *part;      // [block of runs][C W + C]
    int64_t sb, st, dy_sb, dy_st;
    RowSpan x_span, dy_span;
    int B, T, C, act;
    // threads to a row's part (a power of two), parts of a row; tokens to a run, runs of a
    // sequence and of all
    int pieces, groups, run, runs_of_one;
    int64_t runs;
};

__device__ __forceinline__ F2 both(float v) { return pack2(v, v); }

// The four channels of a thread in a row of C: c.. where they are WHOLE, else c, c + apart, ...
template <typename E>
struct Four {
    using Raw = typename std::conditional<sizeof(E) == 4, uint4, uint2>::type;
    static __device__ __forceinline__ void widen(const Raw &raw, F2 (&f)[2]) {
        if constexpr (sizeof(E) == 4) {
            f[0] = pack2(__uint_as_float(raw.x), __uint_as_float(raw.y));
            f[1] = pack2(__uint_as_float(raw.z), __uint_as_float(raw.w));
        } else {
            f[0] = pack2(__uint_as_float(raw.x << 16), __uint_as_float(raw.x & 0xffff0000u));
            f[1] = pack2(__uint_as_float(raw.y << 16), __uint_as_float(raw.y & 0xffff0000u));
        }
    }
    template <bool WHOLE>
    static __device__ __forceinline__ void load(const E *row, int c, int apart, int C, F2 (&f)[2]) {
        if constexpr (WHOLE) {
            widen(*reinterpret_cast<const Raw *>(row + c), f);
        } else {
            float v[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) v[k] = c + k * apart < C ? to_f32(row[c + k * apart]) : 0.f;
            f[0] = pack2(v[0], v[1]);
            f[1] = pack2(v[2], v[3]);
        }
    }
    template <bool WHOLE>
    static __device__ __forceinline__ void store(E *row, int c, int apart, int C, const F2 (&f)[2]) {
        float v[4];
        unpack2(f[0], v[0], v[1]);
        unpack2(f[1], v[2], v[3]);
        if constexpr (!WHOLE) {
#pragma unroll
            for (int k = 0; k < 4; ++k)
                if (c + k * apart < C) row[c + k * apart] = from_f32<E>(v[k]);
        } else if constexpr (sizeof(E) == 4) {
            *reinterpret_cast<float4 *>(row + c) = make_float4(v[0], v[1], v[2], v[3]);
        } else {
            const __nv_bfloat162 lo = __floats2bfloat162_rn(v[0], v[1]), hi = __floats2bfloat162_rn(v[2], v[3]);
            *reinterpret_cast<uint2 *>(row + c) = make_uint2(*reinterpret_cast<const uint32_t *>(&lo),
                                                             *reinterpret_cast<const uint32_t *>(&hi));
        }
    }
};

// dy times the activation's derivative at v.
template <bool SILU>
__device__ __forceinline__ F2 through_act(F2 dy, F2 v, int act) {
    if (SILU) {                 // s (1 + v (1 - s))
        const F2 s = sigmoid2(v);
        return mul2(mul2(dy, s), fma2(v, fma2(s, both(-1.f), both(1.f)), both(1.f)));
    }
    if (act == GDN_ACT_NONE) return dy;
    // s (1 - s) with 1 - s as exp(-v) s, to a few roundings of itself; the exponent's bound keeps
    // the product in range
    float a, b;
    unpack2(mul2(v, both(-kLog2e)), a, b);
    const F2 e = pack2(exp2_ftz(min_nan(a, 126.f)), exp2_ftz(min_nan(b, 126.f)));
    unpack2(add2(e, both(1.f)), a, b);
    const F2 s = pack2(rcp_ftz(a), rcp_ftz(b));
    return mul2(mul2(dy, s), mul2(e, s));
}

// Bytes in the ring for one token of one tensor: the threads' channels, or of each run's part of a
// row the pieces it touches.
template <typename E, bool SHARED>
__host__ __device__ constexpr int token_bytes(int pieces) {
    return kThreads * kChannels * static_cast<int>(sizeof(E)) + (SHARED ? kThreads / pieces * 16 : 0);
}

template <typename E, int W, bool WHOLE, bool SILU>
__global__ void __launch_bounds__(kThreads, 4) gdn_conv_bwd_kernel(const ConvBwdParams<E> p) {
    constexpr int U = kUnroll;
    // the threads of a run fill the ring together; it takes at most a piece of each
    constexpr bool SHARED = !WHOLE && sizeof(E) == 2;
    using Raw = typename Four<E>::Raw;
    extern __shared__ uint4 ring_memory[];
    unsigned char *ring = reinterpret_cast<unsigned char *>(ring_memory);
    const int piece = threadIdx.x & (p.pieces - 1), run = threadIdx.x / p.pieces, runs = kThreads / p.pieces;
    const int group = blockIdx.x % p.groups, c0 = group * p.pieces * kChannels;
    const int apart = WHOLE ? 1 : p.pieces, c = c0 + piece * (WHOLE ? kChannels : 1);
    const int C = p.C, bytes = token_bytes<E, SHARED>(p.pieces);
    const int64_t block = blockIdx.x / p.groups, item = block * runs + run;
    const int64_t b = item < p.runs ? item / p.runs_of_one : 0;
    const int n = item < p.runs ? valid_tokens(p.lengths, b, p.T) : 0;
    // 64 bits: the last run may begin behind 2^31
    const int64_t start = (item - b * p.runs_of_one) * p.run;
    const bool there = item < p.runs && (start < n || start == 0);
    F2 dw[2][W], db[2];
#pragma unroll
    for (int j = 0; j < 2; ++j) {
        db[j] = both(0.f);
#pragma unroll
        for (int k = 0; k < W; ++k) dw[j][k] = both(0.f);
    }
    if (there && (SHARED || c < C)) {            // alike for the threads of a run that fill together
        const int t0 = static_cast<int>(start), end = min(t0 + p.run, n), last = min(end + W - 1, n);
        const uint32_t peers = p.pieces >= 32
                                   ? 0xffffffffu
                                   : ((1u << p.pieces) - 1) << (threadIdx.x % 32 & ~(p.pieces - 1));
        F2 w[2][W], bias[2];
        if constexpr (WHOLE) {
            float f[4 * W], g[4] = {0.f, 0.f, 0.f, 0.f};
            load_f32<4 * W>(p.w + static_cast<int64_t>(c) * W, f);
            if (p.bias) load_f32<4>(p.bias + c, g);
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                bias[j] = pack2(g[2 * j], g[2 * j + 1]);
#pragma unroll
                for (int k = 0; k < W; ++k) w[j][k] = pack2(f[2 * j * W + k], f[(2 * j + 1) * W + k]);
            }
        } else {
            auto at = [&](const float *q, int ch, int stride, int k) {
                return q && ch < C ? q[static_cast<int64_t>(ch) * stride + k] : 0.f;
            };
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                bias[j] = pack2(at(p.bias, c + 2 * j * apart, 1, 0), at(p.bias, c + (2 * j + 1) * apart, 1, 0));
#pragma unroll
                for (int k = 0; k < W; ++k)
                    w[j][k] = pack2(at(p.w, c + 2 * j * apart, W, k), at(p.w, c + (2 * j + 1) * apart, W, k));
            }
        }
        const E *x = p.x + b * p.sb + t0 * p.st, *dy = p.dy + b * p.dy_sb + t0 * p.dy_st;
        // the windows: in[k], g[k] are of token t - W + 1 + k of the turn's first token t
        F2 in[W - 1 + U][2], g[W - 1 + U][2];
#pragma unroll
        for (int k = 0; k < W - 1; ++k) {
            const int t = t0 - W + 1 + k;
            in[k][0] = in[k][1] = g[k][0] = g[k][1] = both(0.f);
            if (t >= 0) {
                if (t < n) Four<E>::template load<WHOLE>(x + (t - t0) * p.st, c, apart, C, in[k]);
            } else if (p.state_in) {
                Four<E>::template load<WHOLE>(p.state_in + (b * (W - 1) + W - 1 + t) * C, c, apart, C, in[k]);
            }
        }
        const E *x_ahead = x, *dy_ahead = dy;
        int ahead = last - t0, slot = 0;
        // of a thread's own, or of its run
        unsigned char *mine = ring + (SHARED ? run * (bytes / runs) : threadIdx.x * (WHOLE ? sizeof(Raw) : sizeof(E)));
        const int width = min(p.pieces * kChannels, C - c0);
        RowCopy<E> x_copy, dy_copy;
        if constexpr (SHARED) {
            x_copy = RowCopy<E>(p.x_span, x + c0, p.st, last - t0, width);
            dy_copy = RowCopy<E>(p.dy_span, dy + c0, p.dy_st, last - t0, width);
        }
        auto fetch = [&](int s) {
#pragma unroll
            for (int u = 0; u < U; ++u)
                if (u < ahead) {
                    unsigned char *to = mine + (s * U + u) * 2 * bytes;
                    const E *from = x_ahead + u * p.st, *dy_from = dy_ahead + u * p.dy_st;
                    if constexpr (WHOLE) {
                        copy_async<sizeof(Raw)>(to, from + c);
                        copy_async<sizeof(Raw)>(to + bytes, dy_from + c);
                    } else if constexpr (SHARED) {
                        x_copy(to, from + c0, width, piece);
                        dy_copy(to + bytes, dy_from + c0, width, piece);
                    } else {
#pragma unroll
                        for (int k = 0; k < kChannels; ++k)
                            if (c + k * apart < C) {
                                copy4_async(to + k * kThreads * 4, from + c + k * apart);
                                copy4_async(to + bytes + k * kThreads * 4, dy_from + c + k * apart);
                            }
                    }
                }
            copy_commit();
            ahead -= U;
            x_ahead += U * p.st;
            dy_ahead += U * p.dy_st;
        };
        auto read = [&](int s, int u, const E *row, int tensor, F2 (&f)[2]) {
            const unsigned char *from = mine + ((s * U + u) * 2 + tensor) * bytes;
            if constexpr (WHOLE) {
                Four<E>::widen(*reinterpret_cast<const Raw *>(from), f);
            } else {
                // what lies in the place of channels that the row does not have is of no use
                const E *v = SHARED ? row_in_copy<E>(from, row + c0) + piece : reinterpret_cast<const E *>(from);
                float h[4];
#pragma unroll
                for (int k = 0; k < 4; ++k) h[k] = to_f32(v[k * (SHARED ? apart : kThreads)]);
                f[0] = pack2(h[0], h[1]);
                f[1] = pack2(h[2], h[3]);
            }
        };
#pragma unroll
        for (int s = 0; s < kStages; ++s) fetch(s);
        // Token u of a turn: its input, p and the sums of the weights' gradients.
        auto take = [&](int u, const E *x_row, const E *dy_row, bool counted) {
            F2 d[2];
            read(slot, u, x_row, 0, in[W - 1 + u]);
            read(slot, u, dy_row, 1, d);
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                F2 v = bias[j];
#pragma unroll
                for (int k = 0; k < W; ++k) v = fma2(w[j][k], in[u + k][j], v);
                d[j] = through_act<SILU>(d[j], v, p.act);
                g[W - 1 + u][j] = d[j];
                if (counted) {
                    db[j] = add2(db[j], d[j]);
#pragma unroll
                    for (int k = 0; k < W; ++k) dw[j][k] = fma2(d[j], in[u + k][j], dw[j][k]);
                }
            }
        };
        // The gradient of the input W - 1 tokens before token u of the turn.
        auto give = [&](int u, F2 (&d)[2]) {
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                d[j] = mul2(w[j][W - 1], g[u][j]);
#pragma unroll
                for (int k = 1; k < W; ++k) d[j] = fma2(w[j][W - 1 - k], g[u + k][j], d[j]);
            }
        };
        const int from = t0 == 0 ? 1 - W : t0;                 // the first input whose gradient is this run's
        E *dx = p.dx + (b * p.T + t0 - W + 1) * C;
        for (int t = t0; t < end + W - 1; t += U) {
            copy_wait<kStages - 1>();
            if constexpr (SHARED) __syncwarp(peers);
            if (t + U <= end && t - W + 1 >= max(from, 0)) {   // every token counted, every input in the run
#pragma unroll
                for (int u = 0; u < U; ++u) {
                    take(u, x + u * p.st, dy + u * p.dy_st, true);
                    F2 d[2];
                    give(u, d);
                    Four<E>::template store<WHOLE>(dx + static_cast<int64_t>(u) * C, c, apart, C, d);
                }
            } else {
#pragma unroll
                for (int u = 0; u < U; ++u) {
                    if (t + u < last) {
                        take(u, x + u * p.st, dy + u * p.dy_st, t + u < end);
                    } else {
                        in[W - 1 + u][0] = in[W - 1 + u][1] = g[W - 1 + u][0] = g[W - 1 + u][1] = both(0.f);
                    }
                    const int i = t + u - W + 1;
                    if (i < from || i >= end) continue;
                    F2 d[2];
                    give(u, d);
                    // the last W - 1 inputs: of the window that the call left
                    if (p.d_last && i > n - W) {
                        F2 f[2];
                        Four<E>::template load<WHOLE>(p.d_last + (b * (W - 1) + i - (n - W + 1)) * C, c, apart, C, f);
                        d[0] = add2(d[0], f[0]);
                        d[1] = add2(d[1], f[1]);
                    }
                    if (i >= 0)
                        Four<E>::template store<WHOLE>(dx + static_cast<int64_t>(u) * C, c, apart, C, d);
                    else if (p.d_state)
                        Four<E>::template store<WHOLE>(p.d_state + (b * (W - 1) + W - 1 + i) * C, c, apart, C, d);
                }
            }
#pragma unroll
            for (int k = 0; k < W - 1; ++k)
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    in[k][j] = in[U + k][j];
                    g[k][j] = g[U + k][j];
                }
            dx += static_cast<int64_t>(U) * C;
            x += U * p.st;
            dy += U * p.dy_st;
            if constexpr (SHARED) __syncwarp(peers);           // all have read what is filled anew
            fetch(slot);
            slot = slot == kStages - 1 ? 0 : slot + 1;
        }
        copy_wait<0>();
    }
    // The block's runs are added up in order: [value][run][piece].
    float *sums = reinterpret_cast<float *>(ring_memory);
    constexpr int M = kChannels * (W + 1);
    __syncthreads();
#pragma unroll
    for (int j = 0; j < 2; ++j) {
        float f[2];
#pragma unroll
        for (int k = 0; k <= W; ++k) {
            unpack2(k < W ? dw[j][k < W ? k : 0] : db[j], f[0], f[1]);
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const int at = k < W ? (2 * j + h) * W + k : kChannels * W + 2 * j + h;
                sums[at * kThreads + threadIdx.x] = f[h];
            }
        }
    }
    __syncthreads();
    float *part = p.part + block * C * (W + 1);
    for (int o = threadIdx.x; o < M * p.pieces; o += kThreads) {
        const int value = o / p.pieces, q = o & (p.pieces - 1);
        const bool tap = value < kChannels * W;
        const int of = tap ? value / W : value - kChannels * W;        // which of the thread's channels
        const int ch = c0 + q * (WHOLE ? kChannels : 1) + of * apart;
        if (ch >= C) continue;
        float s = 0.f;
        for (int r = 0; r < runs; ++r) s += sums[value * kThreads + r * p.pieces + q];
        part[tap ? static_cast<int64_t>(ch) * W + value % W : static_cast<int64_t>(C) * W + ch] = s;
    }
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

// How a problem is cut: 8 to 32 threads to a part of a row; runs of 128 tokens, or 256 where those
// still leave 16 blocks to an SM (B8 T8192 C8192 bf16 583 -> 558 us; B4 T4096 C4096, with 3, 93 ->
// 101), shorter ones where SMs would be without their blocks; of all sequences one after the other.
struct Shape {
    int pieces, groups, run, runs_of_one;
    int64_t runs, blocks;      // runs of all sequences, blocks of them
};
Shape shape(const gdn_conv_bwd_problem *p) {
    const int64_t cv = (p->C + kChannels - 1) / kChannels;
    Shape s;
    s.pieces = kMinPieces;
    while (s.pieces < 32 && s.pieces < cv) s.pieces *= 2;
    s.groups = static_cast<int>((cv + s.pieces - 1) / s.pieces);
    const int per_block = kThreads / s.pieces;
    auto cut = [&](int run) {
        s.run = run;
        s.runs_of_one = (p->T + run - 1) / run;
        s.runs = static_cast<int64_t>(p->B) * s.runs_of_one;
        s.blocks = (s.runs + per_block - 1) / per_block;
        return s.blocks * s.groups;
    };
    for (int run = 256; cut(run) < 152 * (run > 128 ? 16 : 3) && run > kMinRun;) run /= 2;
    return s;
}

size_t workspace_need(const gdn_conv_bwd_problem *p) {
    return align_up(static_cast<size_t>(shape(p).blocks) * p->C * (p->W + 1) * 4);
}

template <typename E, int W, bool WHOLE>
cudaError_t launch(const gdn_conv_bwd_problem *pr, ConvBwdParams<E> &p, float *d_weight, float *d_bias,
                   cudaStream_t s) {
    const Shape cut = shape(pr);
    p.pieces = cut.pieces;
    p.groups = cut.groups;
    p.run = cut.run;
    p.runs_of_one = cut.runs_of_one;
    p.runs = cut.runs;
    if (cut.blocks * cut.groups > INT32_MAX) return cudaErrorInvalidValue;
    constexpr auto shared_bytes = [](int pieces) {
        const int ring = kStages * kUnroll * 2 * token_bytes<E, !WHOLE && sizeof(E) == 2>(pieces);
        const int sums = kChannels * (W + 1) * kThreads * 4;
        return ring > sums ? ring : sums;
    };
    auto kernel = pr->act == GDN_ACT_SILU ? gdn_conv_bwd_kernel<E, W, WHOLE, true>
                                          : gdn_conv_bwd_kernel<E, W, WHOLE, false>;
    // one bound for all calls: a call of another size on another thread must not lower it
    cudaError_t err = cudaFuncSetAttribute(reinterpret_cast<const void *>(kernel),
                                           cudaFuncAttributeMaxDynamicSharedMemorySize, shared_bytes(kMinPieces));
    if (err != cudaSuccess) return err;
    kernel<<<static_cast<unsigned>(cut.blocks * cut.groups), kThreads, shared_bytes(cut.pieces), s>>>(p);
    err = cudaGetLastError();
    if (err != cudaSuccess) return err;
    const int64_t taps = static_cast<int64_t>(pr->C) * W;
    return column_sums(p.part, static_cast<int>(cut.blocks), taps + pr->C, taps, d_weight, d_bias, s);
}

// Whole accesses of four channels where every row is made of them.
template <typename E, int W>
cudaError_t launch_pieces(const gdn_conv_bwd_problem *pr, ConvBwdParams<E> &p, float *d_weight, float *d_bias,
                          cudaStream_t s) {
    constexpr size_t e = sizeof(E), a = kChannels * e;
    auto whole = [&](const void *t, int64_t sb, int64_t st) {
        return is_aligned(t, a) && (pr->B == 1 || sb * e % a == 0) && (pr->T == 1 || st * e % a == 0);
    };
    return pr->C % kChannels == 0 && whole(p.x, p.sb, p.st) && whole(p.dy, p.dy_sb, p.dy_st)
               ? launch<E, W, true>(pr, p, d_weight, d_bias, s)
               : launch<E, W, false>(pr, p, d_weight, d_bias, s);
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
    if (need && (!workspace || workspace_bytes < need)) return GDN_ERR_WORKSPACE;
    const size_t row = static_cast<size_t>(p->C) * e, channels = static_cast<size_t>(p->C) * 4;
    const size_t window = row * (p->W - 1) * p->B;
    const Span in[] = {Span(dy, strided_bytes(p->B, p->T, p->C, p->dy_stride_b, p->dy_stride_t, e)),
                       Span(x, strided_bytes(p->B, p->T, p->C, p->x_stride_b, p->x_stride_t, e)),
                       Span(weight, channels * p->W), Span(bias, channels), Span(state_in, window),
                       Span(lengths, static_cast<size_t>(p->B) * 4), Span(d_state_out, window)};
    const Span out[] = {Span(dx, row * p->T * p->B), Span(d_weight, channels * p->W), Span(d_bias, channels),
                        Span(workspace, need), Span(d_state_in, window)};
    for (const Span &o : out) {
        for (const Span &i : in)
            if (o.meets(i)) return GDN_ERR_INVALID_ARG;
        for (const Span &o2 : out)
            if (&o != &o2 && o.meets(o2)) return GDN_ERR_INVALID_ARG;
    }
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (empty) {
        cudaError_t err = cudaMemsetAsync(d_weight, 0, channels * p->W, s);
        if (err == cudaSuccess && d_bias) err = cudaMemsetAsync(d_bias, 0, channels, s);
        if (err == cudaSuccess && d_state_in)
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
        a.x_span = row_span(x, p->B, p->T, p->C, a.sb, a.st, e);
        a.dy_span = row_span(dy, p->B, p->T, p->C, a.dy_sb, a.dy_st, e);
        a.B = p->B; a.T = p->T; a.C = p->C; a.act = p->act;
        switch (p->W) {
            case 2: return launch_pieces<E, 2>(p, a, d_weight, d_bias, s);
            case 3: return launch_pieces<E, 3>(p, a, d_weight, d_bias, s);
            default: return launch_pieces<E, 4>(p, a, d_weight, d_bias, s);
        }
    };
    const cudaError_t err = p->dtype == GDN_BF16 ? go(__nv_bfloat16()) : go(float());
    return err == cudaSuccess ? GDN_OK : GDN_ERR_CUDA;
}

}  // extern "C"
