// Backward pass of the short causal convolution: gdn_conv_bwd of include/gdn.h.
//
// Bound by memory: x and dy read, dx written. A thread owns V channels (8 or 16 bytes of a row, or one
// channel where rows are not such pieces) over a run of tokens, token by token: with the
// window of inputs it takes the value before the activation anew and p = dy act', with
// the window of p the gradient of the input W - 1 tokens before, and adds p x to its
// gradients of the weights, which stay in registers. x and dy come through a ring of its own in
// shared memory. A run needs the inputs of W - 1 tokens before it and p of as many behind
// it, which its neighbours read too. The runs of a block add their gradients of the weights up and
// leave a row of partial sums.
#include "columns.cuh"

namespace gdn {
namespace {

constexpr int kThreads = 256;
constexpr int kUnroll = 4;      // tokens per turn
constexpr int kStages = 4;      // turns in the ring
constexpr int kMaxRun = 128, kMinRun = 8;
constexpr int kBlocks = 152 * 3;
static_assert(kMinRun >= kUnroll && kUnroll >= 3, "W - 1");

template <typename E>
struct ConvBwdParams {
    const E *x, *dy;
    const float *w, *bias;
    const E *state_in, *d_last;
    const int32_t *lengths;
    E *dx, *d_state;
    float *part;      // [sequence][block of runs][C W + C]
    int64_t sb, st, dy_sb, dy_st;
    int B, T, C, act;
    int pieces, groups, run;    // pieces of a row to a block (a power of two), blocks of pieces, tokens to a run
};

// V values of E as one access (1, 8 or 16 bytes).
template <typename E, int V>
struct Values {
    static constexpr int N = (V + 1) / 2;
    using Raw = typename std::conditional<V == 1, E, typename std::conditional<V * sizeof(E) == 8, uint2, uint4>::type>::type;
    Raw raw;
    __device__ __forceinline__ void load(const E *p) { raw = *reinterpret_cast<const Raw *>(p); }
    __device__ __forceinline__ void widen(F2 (&f)[N]) const {
        if constexpr (V == 1) {
            f[0] = pack2(to_f32(raw), to_f32(raw));
        } else if constexpr (sizeof(E) == 4) {
            f[0] = pack2(__uint_as_float(raw.x), __uint_as_float(raw.y));
            f[1] = pack2(__uint_as_float(raw.z), __uint_as_float(raw.w));
        } else {
            f[0] = pack2(__uint_as_float(raw.x << 16), __uint_as_float(raw.x & 0xffff0000u));
            f[1] = pack2(__uint_as_float(raw.y << 16), __uint_as_float(raw.y & 0xffff0000u));
        }
    }
    static __device__ __forceinline__ void store(E *p, const F2 (&f)[N]) {
        float v[2 * N];
#pragma unroll
        for (int k = 0; k < N; ++k) unpack2(f[k], v[2 * k], v[2 * k + 1]);
        if constexpr (V == 1) {
            *p = from_f32<E>(v[0]);
        } else if constexpr (sizeof(E) == 4) {
            *reinterpret_cast<float4 *>(p) = make_float4(v[0], v[1], v[2], v[3]);
        } else {
            const __nv_bfloat162 lo = __floats2bfloat162_rn(v[0], v[1]), hi = __floats2bfloat162_rn(v[2], v[3]);
            *reinterpret_cast<uint2 *>(p) = make_uint2(*reinterpret_cast<const uint32_t *>(&lo),
                                                       *reinterpret_cast<const uint32_t *>(&hi));
        }
    }
};

__device__ __forceinline__ F2 both(float v) { return pack2(v, v); }

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
    const F2 e = pack2(exp2_ftz(fminf(a, 126.f)), exp2_ftz(fminf(b, 126.f)));
    unpack2(add2(e, both(1.f)), a, b);
    const F2 s = pack2(rcp_ftz(a), rcp_ftz(b));
    return mul2(mul2(dy, s), mul2(e, s));
}

template <typename E, int W, int V, bool SILU>
__global__ void __launch_bounds__(kThreads, 2) gdn_conv_bwd_kernel(const ConvBwdParams<E> p) {
    constexpr int U = kUnroll, N = (V + 1) / 2;
    using Val = Values<E, V>;
    // an asynchronous copy moves 4 bytes at least
    constexpr bool RING = V > 1 || sizeof(E) == 4;
    extern __shared__ uint4 ring_memory[];
    using Raw = typename Val::Raw;
    Raw *mine = reinterpret_cast<Raw *>(ring_memory) + threadIdx.x;
    const int piece = threadIdx.x & (p.pieces - 1), run = threadIdx.x / p.pieces, runs = kThreads / p.pieces;
    const int group = blockIdx.x % p.groups, span = blockIdx.x / p.groups;
    const int c = (group * p.pieces + piece) * V;
    const int64_t b = blockIdx.y;
    const int n = valid_tokens(p.lengths, b, p.T);
    // 64 bits: the last block's runs may lie behind 2^31
    const int64_t start = (static_cast<int64_t>(span) * runs + run) * p.run;
    const bool there = c < p.C && (start < n || start == 0);
    F2 dw[N][W], db[N];
#pragma unroll
    for (int j = 0; j < N; ++j) {
        db[j] = both(0.f);
#pragma unroll
        for (int k = 0; k < W; ++k) dw[j][k] = both(0.f);
    }
    if (there) {
        const int t0 = static_cast<int>(start), end = min(t0 + p.run, n), last = min(end + W - 1, n);
        F2 w[N][W], bias[N];
        {
            float f[V * W], g[V];
            load_f32<V * W>(p.w + static_cast<int64_t>(c) * W, f);
#pragma unroll
            for (int j = 0; j < V; ++j) g[j] = 0.f;
            if (p.bias) load_f32<V>(p.bias + c, g);
#pragma unroll
            for (int j = 0; j < N; ++j) {
                const int o = V == 1 ? 0 : 2 * j + 1;
                bias[j] = pack2(g[2 * j], g[o]);
#pragma unroll
                for (int k = 0; k < W; ++k) w[j][k] = pack2(f[2 * j * W + k], f[o * W + k]);
            }
        }
        // the windows: in[k], g[k] are of token t - W + 1 + k of the turn's first token t
        F2 in[W - 1 + U][N], g[W - 1 + U][N];
#pragma unroll
        for (int k = 0; k < W - 1; ++k) {
            const int t = t0 - W + 1 + k;
            Val v;
            memset(&v.raw, 0, sizeof(v.raw));
            if (t >= 0) {
                if (t < n) v.load(p.x + b * p.sb + t * p.st + c);
            } else if (p.state_in) {
                v.load(p.state_in + (b * (W - 1) + W - 1 + t) * p.C + c);
            }
            v.widen(in[k]);
#pragma unroll
            for (int j = 0; j < N; ++j) g[k][j] = both(0.f);
        }
        const E *x = p.x + b * p.sb + t0 * p.st + c, *dy = p.dy + b * p.dy_sb + t0 * p.dy_st + c;
        int ahead = last - t0, slot = 0;
        auto fetch = [&](int s) {
            if constexpr (RING) {
#pragma unroll
                for (int u = 0; u < U; ++u)
                    if (u < ahead) {
                        copy_async<sizeof(Raw)>(mine + (s * U + u) * 2 * kThreads, x + u * p.st);
                        copy_async<sizeof(Raw)>(mine + ((s * U + u) * 2 + 1) * kThreads, dy + u * p.dy_st);
                    }
                copy_commit();
                ahead -= U;
                x += U * p.st;
                dy += U * p.dy_st;
            }
        };
#pragma unroll
        for (int s = 0; s < kStages; ++s) fetch(s);
        // Token u of a turn: its input, p and the sums of the weights' gradients.
        auto take = [&](int u, const Val &vx, const Val &vdy, bool counted) {
            F2 d[N];
            vx.widen(in[W - 1 + u]);
            vdy.widen(d);
#pragma unroll
            for (int j = 0; j < N; ++j) {
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
        auto give = [&](int u, F2 (&d)[N]) {
#pragma unroll
            for (int j = 0; j < N; ++j) {
                d[j] = mul2(w[j][W - 1], g[u][j]);
#pragma unroll
                for (int k = 1; k < W; ++k) d[j] = fma2(w[j][W - 1 - k], g[u + k][j], d[j]);
            }
        };
        const int from = t0 == 0 ? 1 - W : t0;                 // the first input whose gradient is this run's
        E *dx = p.dx + (b * p.T + t0 - W + 1) * p.C + c;
        for (int t = t0; t < end + W - 1; t += U) {
            if constexpr (RING) copy_wait<kStages - 1>();
            auto read = [&](int u, Val &vx, Val &vdy) {
                if constexpr (RING) {
                    vx.raw = mine[(slot * U + u) * 2 * kThreads];
                    vdy.raw = mine[((slot * U + u) * 2 + 1) * kThreads];
                } else {
                    vx.load(x + u * p.st);
                    vdy.load(dy + u * p.dy_st);
                }
            };
            if (t + U <= end && t - W + 1 >= max(from, 0)) {      // every token counted, every input in the run
#pragma unroll
                for (int u = 0; u < U; ++u) {
                    Val vx, vdy;
                    read(u, vx, vdy);
                    take(u, vx, vdy, true);
                    F2 d[N];
                    give(u, d);
                    Val::store(dx + static_cast<int64_t>(u) * p.C, d);
                }
            } else {
#pragma unroll
                for (int u = 0; u < U; ++u) {
                    if (t + u < last) {
                        Val vx, vdy;
                        read(u, vx, vdy);
                        take(u, vx, vdy, t + u < end);
                    } else {
#pragma unroll
                        for (int j = 0; j < N; ++j) {
                            in[W - 1 + u][j] = both(0.f);
                            g[W - 1 + u][j] = both(0.f);
                        }
                    }
                    const int i = t + u - W + 1;
                    if (i < from || i >= end) continue;
                    F2 d[N];
                    give(u, d);
                    // the last W - 1 inputs: of the window that the call left
                    if (p.d_last && i > n - W) {
                        Val v;
                        F2 f[N];
                        v.load(p.d_last + (b * (W - 1) + i - (n - W + 1)) * p.C + c);
                        v.widen(f);
#pragma unroll
                        for (int j = 0; j < N; ++j) d[j] = add2(d[j], f[j]);
                    }
                    if (i >= 0)
                        Val::store(dx + static_cast<int64_t>(u) * p.C, d);
                    else if (p.d_state)
                        Val::store(p.d_state + (b * (W - 1) + W - 1 + i) * p.C + c, d);
                }
            }
#pragma unroll
            for (int k = 0; k < W - 1; ++k)
#pragma unroll
                for (int j = 0; j < N; ++j) {
                    in[k][j] = in[U + k][j];
                    g[k][j] = g[U + k][j];
                }
            dx += static_cast<int64_t>(U) * p.C;
            if constexpr (RING) {
                fetch(slot);
                slot = slot == kStages - 1 ? 0 : slot + 1;
            } else {
                x += U * p.st;
                dy += U * p.dy_st;
            }
        }
        if constexpr (RING) copy_wait<0>();
    }
    // The block's runs are added up in order: [value][run][piece].
    float *sums = reinterpret_cast<float *>(ring_memory);
    constexpr int M = V * (W + 1);
    __syncthreads();
#pragma unroll
    for (int j = 0; j < N; ++j) {
        float f[2];
#pragma unroll
        for (int k = 0; k <= W; ++k) {
            unpack2(k < W ? dw[j][k < W ? k : 0] : db[j], f[0], f[1]);
#pragma unroll
            for (int h = 0; h < (V == 1 ? 1 : 2); ++h) {
                const int at = k < W ? (2 * j + h) * W + k : V * W + 2 * j + h;
                sums[at * kThreads + threadIdx.x] = f[h];
            }
        }
    }
    __syncthreads();
    float *part = p.part + (b * (gridDim.x / p.groups) + span) * p.C * (W + 1);
    for (int o = threadIdx.x; o < M * p.pieces; o += kThreads) {
        const int value = o / p.pieces, q = o & (p.pieces - 1);
        const int64_t first = static_cast<int64_t>(group * p.pieces + q) * V;
        if (first >= p.C) continue;
        float s = 0.f;
        for (int r = 0; r < runs; ++r) s += sums[value * kThreads + r * p.pieces + q];
        if (value < V * W)
            part[first * W + value] = s;
        else
            part[static_cast<int64_t>(p.C) * W + first + value - V * W] = s;
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

// How a problem is cut with V channels to a thread: up to 32 pieces of a row to a block, runs of
// kMaxRun tokens, shorter ones where those would leave SMs without their blocks.
struct Shape {
    int pieces, groups, run, spans;
};
Shape shape(const gdn_conv_bwd_problem *p, int V) {
    const int64_t cv = (p->C + V - 1) / V;
    Shape s;
    s.pieces = 1;
    while (s.pieces < 32 && s.pieces < cv) s.pieces *= 2;
    s.groups = static_cast<int>((cv + s.pieces - 1) / s.pieces);
    const int runs = kThreads / s.pieces;
    auto spans = [&](int run) { return (static_cast<int64_t>(p->T) + runs * run - 1) / (runs * run); };
    s.run = kMaxRun;
    while (s.run > kMinRun && spans(s.run) * s.groups * p->B < kBlocks) s.run /= 2;
    s.spans = static_cast<int>(spans(s.run));
    return s;
}

constexpr int kPiece = 4;      // channels to a thread

// The larger of both cuts' partial sums: the alignment of the tensors decides between them.
size_t workspace_need(const gdn_conv_bwd_problem *p) {
    const int a = shape(p, kPiece).spans, b = shape(p, 1).spans;
    return align_up(static_cast<size_t>(p->B) * (a > b ? a : b) * p->C * (p->W + 1) * 4);
}

template <typename E, int W, int V>
cudaError_t launch(const gdn_conv_bwd_problem *pr, ConvBwdParams<E> &p, float *d_weight, float *d_bias,
                   cudaStream_t s) {
    const Shape cut = shape(pr, V);
    p.pieces = cut.pieces;
    p.groups = cut.groups;
    p.run = cut.run;
    const int64_t blocks = static_cast<int64_t>(cut.groups) * cut.spans;
    if (blocks > INT32_MAX) return cudaErrorInvalidValue;
    constexpr int ring = V > 1 || sizeof(E) == 4 ? kStages * kUnroll * 2 * kThreads * V * static_cast<int>(sizeof(E)) : 0;
    constexpr int sums = V * (W + 1) * kThreads * 4, bytes = ring > sums ? ring : sums;
    auto kernel = pr->act == GDN_ACT_SILU ? gdn_conv_bwd_kernel<E, W, V, true> : gdn_conv_bwd_kernel<E, W, V, false>;
    cudaError_t err = cudaFuncSetAttribute(reinterpret_cast<const void *>(kernel),
                                           cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
    if (err != cudaSuccess) return err;
    kernel<<<dim3(static_cast<unsigned>(blocks), pr->B), kThreads, bytes, s>>>(p);
    err = cudaGetLastError();
    if (err != cudaSuccess) return err;
    const int64_t taps = static_cast<int64_t>(pr->C) * W;
    return column_sums(p.part, pr->B * cut.spans, taps + pr->C, taps, d_weight, d_bias, s);
}

// Pieces of 8 bytes in bf16 and 16 in fp32 where the rows are whole ones.
template <typename E, int W>
cudaError_t launch_pieces(const gdn_conv_bwd_problem *pr, ConvBwdParams<E> &p, float *d_weight, float *d_bias,
                          cudaStream_t s) {
    constexpr size_t e = sizeof(E), a = kPiece * e;
    auto whole = [&](const void *t, int64_t sb, int64_t st) {
        return is_aligned(t, a) && (pr->B == 1 || sb * e % a == 0) && (pr->T == 1 || st * e % a == 0);
    };
    return pr->C % kPiece == 0 && whole(p.x, p.sb, p.st) && whole(p.dy, p.dy_sb, p.dy_st)
               ? launch<E, W, kPiece>(pr, p, d_weight, d_bias, s)
               : launch<E, W, 1>(pr, p, d_weight, d_bias, s);
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
