// Layer norm of every token and its backward pass: gdn_layer_norm and gdn_layer_norm_bwd of
// include/gdn.h.
//
// Bound by memory: x read and y written; in the backward pass x and dy read and dx written. A row
// is held by `lanes` threads (a power of two) in pieces of V channels (16 bytes, or one channel
// where rows are not whole 16-byte pieces), P to a thread, while its sums are taken:
//   gdn_layer_norm_kernel      a row from registers: the mean, the squares about it, the output;
//   gdn_layer_norm_bwd_kernel  blocks that stay for many rows. A thread keeps its channels, so
//                              the sums over rows that are the gradients of weight and bias
//                              stay in its registers; the next rows are on their way to shared
//                              memory meanwhile. Every block leaves a row of partial sums.
//   the *_wide_* kernels       rows beyond what a block holds: a block to a row that it reads
//                              again for each sum, the sums over rows apart.
#include <utility>

#include "columns.cuh"

namespace gdn {
namespace {

constexpr int kThreads = 256;
constexpr int kMaxLanes = 512;     // threads to a row
constexpr int kWideParts = 64;     // rows of partial sums of the wide kernels
constexpr int kMaxParts = 152 * 3; // blocks of the backward pass

template <typename E>
struct LayerNormParams {
    const E *x, *dy;
    const float *w, *bias, *stats_in;
    const int32_t *lengths;
    E *y, *dx;
    float *stats, *part;
    int64_t x_sb, x_st, dy_sb, dy_st;
    int rows, B, T, C, lanes;
    bool rms;
    float eps;
};

__device__ __forceinline__ F2 both(float v) { return pack2(v, v); }

// Channels c.. of a parameter, 1 without any.
template <int V>
__device__ __forceinline__ void params(const float *p, int c, float other, F2 (&f)[(V + 1) / 2]) {
    float v[V];
    if (p) {
        load_f32<V>(p + c, v);
    } else {
#pragma unroll
        for (int i = 0; i < V; ++i) v[i] = other;
    }
#pragma unroll
    for (int i = 0; i < (V + 1) / 2; ++i) f[i] = pack2(v[2 * i], v[V == 1 ? 0 : 2 * i + 1]);
}

// The halves' sum of a piece's pairs; a single value is in both halves.
template <int V>
__device__ __forceinline__ float halves(F2 v) {
    float a, b;
    unpack2(v, a, b);
    return V == 1 ? a : a + b;
}

// Sums over the `lanes` threads of a row, of N values at once, for all of them. Two calls in a
// row take different `buffer`s.
template <int N, int WARPS>
__device__ __forceinline__ void row_sums(float (&v)[N], int lanes, float (&buffer)[WARPS][N]) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
        if (o >= lanes) continue;                      // alike for all threads
#pragma unroll
        for (int i = 0; i < N; ++i) v[i] += __shfl_xor_sync(0xffffffffu, v[i], o);
    }
    if (lanes <= 32) return;
    const int warp = threadIdx.x / 32, first = warp & ~(lanes / 32 - 1);
    if (threadIdx.x % 32 == 0)
#pragma unroll
        for (int i = 0; i < N; ++i) buffer[warp][i] = v[i];
    __syncthreads();
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] = 0.f;
    for (int w = 0; w < lanes / 32; ++w)
#pragma unroll
        for (int i = 0; i < N; ++i) v[i] += buffer[first + w][i];
}

// A row's sequence and token.
template <typename E>
__device__ __forceinline__ void locate(const LayerNormParams<E> &p, int row, int &b, int &t) {
    b = p.B == 1 ? 0 : row / p.T;
    t = row - b * p.T;
}
template <typename E>
__device__ __forceinline__ bool is_valid(const LayerNormParams<E> &p, int b, int t) {
    return !p.lengths || t < p.lengths[b];
}

template <typename E, int V, int P>
__global__ void __launch_bounds__(kMaxLanes) gdn_layer_norm_kernel(const LayerNormParams<E> p) {
    __shared__ float buffers[2][kMaxLanes / 32][1];
    constexpr int N = (V + 1) / 2;
    const int lanes = p.lanes, lane = threadIdx.x & (lanes - 1);
    const int64_t at = static_cast<int64_t>(blockIdx.x) * (blockDim.x / lanes) + threadIdx.x / lanes;
    bool live = at < p.rows;
    const int row = live ? static_cast<int>(at) : 0;
    int b, t;
    locate(p, row, b, t);
    live = live && is_valid(p, b, t);
    const E *x = p.x + b * p.x_sb + t * p.x_st;
    Piece<E, V> r[P];
#pragma unroll
    for (int q = 0; q < P; ++q) {
        const int c = (q * lanes + lane) * V;
        r[q].zero();
        if (live && c < p.C) r[q].load_rw(x + c);
    }
    const float inv = 1.f / p.C;
    float mean = 0.f, s[1];
    if (!p.rms) {
        F2 sum = both(0.f);
#pragma unroll
        for (int q = 0; q < P; ++q) {
            F2 v[N];
            r[q].widen(v);
#pragma unroll
            for (int k = 0; k < N; ++k) sum = add2(sum, v[k]);
        }
        s[0] = halves<V>(sum);
        row_sums(s, lanes, buffers[0]);
        mean = s[0] * inv;
    }
    const F2 minus = both(-mean);
    F2 sum = both(0.f);
#pragma unroll
    for (int q = 0; q < P; ++q) {
        F2 v[N], sq = both(0.f);
        r[q].widen(v);
#pragma unroll
        for (int k = 0; k < N; ++k) {
            v[k] = add2(v[k], minus);
            sq = fma2(v[k], v[k], sq);
        }
        if ((q * lanes + lane) * V < p.C) sum = add2(sum, sq);
    }
    s[0] = halves<V>(sum);
    row_sums(s, lanes, buffers[1]);
    const float rstd = rsqrtf(fmaf(s[0], inv, p.eps));
    if (!live) return;
    E *y = p.y + static_cast<int64_t>(row) * p.C;
#pragma unroll
    for (int q = 0; q < P; ++q) {
        const int c = (q * lanes + lane) * V;
        if (c >= p.C) break;
        F2 v[N], w[N], bias[N];
        params<V>(p.w, c, 1.f, w);
        params<V>(p.bias, c, 0.f, bias);
        r[q].widen(v);
#pragma unroll
        for (int k = 0; k < N; ++k) v[k] = fma2(mul2(add2(v[k], minus), both(rstd)), w[k], bias[k]);
        r[q].round(v);
        r[q].store(y + c);
    }
    if (p.stats && lane == 0) *reinterpret_cast<float2 *>(p.stats + 2LL * row) = make_float2(mean, rstd);
}

// Rows of a thread in the ring: three, or the one that its block's shared memory holds.
constexpr int row_bytes(int V, int P, int threads) { return threads * 2 * P * (V == 1 ? 4 : 16); }
constexpr int row_stages(int V, int P, int threads) { return 3 * row_bytes(V, P, threads) <= 200 * 1024 ? 3 : 1; }

template <typename E, int V, int P, int THREADS>
__global__ void __launch_bounds__(THREADS, THREADS * P <= 512 ? 3 : 1)
    gdn_layer_norm_bwd_kernel(const LayerNormParams<E> p) {
    constexpr int kStages = row_stages(V, P, THREADS);
    __shared__ float buffers[2][THREADS / 32][2];
    extern __shared__ uint4 ring_memory[];
    constexpr int N = (V + 1) / 2;
    using Slot = typename std::conditional<V == 1, float, uint4>::type;    // a piece, or an element's 4 bytes
    // [stage][x, dy][piece][thread]: a thread fills and reads its own slots
    Slot *mine = reinterpret_cast<Slot *>(ring_memory) + threadIdx.x;
    const int lanes = p.lanes, lane = threadIdx.x & (lanes - 1), per_block = THREADS / lanes;
    const int step = gridDim.x * per_block;
    const int turns = (p.rows + step - 1) / step;      // alike for all threads
    const float inv = 1.f / p.C;
    F2 w[P][N], dw[P][N], db[P][N];
#pragma unroll
    for (int q = 0; q < P; ++q) {
        const int c = (q * lanes + lane) * V;
#pragma unroll
        for (int k = 0; k < N; ++k) w[q][k] = dw[q][k] = db[q][k] = both(0.f);
        if (c < p.C) params<V>(p.w, c, 1.f, w[q]);
    }
    // The row of a turn, -1 where there is none; its stats are asked for a turn ahead.
    const int64_t first = static_cast<int64_t>(blockIdx.x) * per_block + threadIdx.x / lanes;
    auto row_of = [&](int i, int &b, int &t) {
        const int64_t at = first + static_cast<int64_t>(i) * step;
        if (at >= p.rows) return -1;
        const int row = static_cast<int>(at);
        locate(p, row, b, t);
        return is_valid(p, b, t) ? row : -1;
    };
    auto fetch = [&](int i, int stage) {
        int b, t;
        const int row = i < turns ? row_of(i, b, t) : -1;
        Slot *to = mine + stage * 2 * P * THREADS;
        const E *x = p.x + (row < 0 ? 0 : b * p.x_sb + t * p.x_st);
        const E *dy = p.dy + (row < 0 ? 0 : b * p.dy_sb + t * p.dy_st);
#pragma unroll
        for (int q = 0; q < P; ++q) {
            const int c = (q * lanes + lane) * V;
            Slot *tx = to + q * THREADS, *tdy = to + (P + q) * THREADS;
            if (row >= 0 && c < p.C) {
                if constexpr (V > 1) {
                    copy16_async(tx, x + c);
                    copy16_async(tdy, dy + c);
                } else if constexpr (sizeof(E) == 4) {
                    copy4_async(tx, x + c);
                    copy4_async(tdy, dy + c);
                } else {
                    *tx = to_f32(x[c]);
                    *tdy = to_f32(dy[c]);
                }
            } else {
                memset(tx, 0, sizeof(Slot));
                memset(tdy, 0, sizeof(Slot));
            }
        }
        copy_commit();
        return row;
    };
    auto stats_of = [&](int row) {
        return row < 0 ? make_float2(0.f, 0.f) : *reinterpret_cast<const float2 *>(p.stats_in + 2LL * row);
    };
    auto widen = [&](const Slot *at, F2 (&f)[N]) {
        if constexpr (V == 1) {
            f[0] = both(*at);
        } else {
            Piece<E, V> r;
            r.raw = *at;
            r.widen(f);
        }
    };
    int rows[kStages];
#pragma unroll
    for (int i = 0; i < kStages; ++i) rows[i] = fetch(i, i);
    float2 stats = stats_of(rows[0]);
    int stage = 0;
    for (int i = 0; i < turns; ++i) {
        const int row = rows[0];
        float2 next;
        if constexpr (kStages > 1) next = stats_of(rows[1]);
        copy_wait<kStages - 1>();
        const Slot *from = mine + stage * 2 * P * THREADS;
        const F2 minus = both(-stats.x), rstd = both(stats.y);
        F2 s1 = both(0.f), s2 = both(0.f);
#pragma unroll
        for (int q = 0; q < P; ++q) {
            F2 x[N], dy[N];
            widen(from + q * THREADS, x);
            widen(from + (P + q) * THREADS, dy);
#pragma unroll
            for (int k = 0; k < N; ++k) {
                const F2 xhat = mul2(add2(x[k], minus), rstd), v = mul2(dy[k], w[q][k]);
                db[q][k] = add2(db[q][k], dy[k]);
                dw[q][k] = fma2(dy[k], xhat, dw[q][k]);
                s1 = add2(s1, v);
                s2 = fma2(v, xhat, s2);
            }
        }
        float s[2] = {halves<V>(s1), halves<V>(s2)};
        row_sums(s, lanes, buffers[i & 1]);
        const F2 c1 = both(p.rms ? 0.f : -s[0] * inv), c2 = both(-s[1] * inv);
        if (row >= 0) {
            E *dx = p.dx + static_cast<int64_t>(row) * p.C;
#pragma unroll
            for (int q = 0; q < P; ++q) {
                const int c = (q * lanes + lane) * V;
                if (c >= p.C) break;
                F2 x[N], dy[N];
                widen(from + q * THREADS, x);
                widen(from + (P + q) * THREADS, dy);
#pragma unroll
                for (int k = 0; k < N; ++k) {
                    const F2 xhat = mul2(add2(x[k], minus), rstd);
                    x[k] = mul2(rstd, fma2(xhat, c2, add2(mul2(dy[k], w[q][k]), c1)));
                }
                Piece<E, V> r;
                r.round(x);
                r.store(dx + c);
            }
        }
#pragma unroll
        for (int k = 0; k + 1 < kStages; ++k) rows[k] = rows[k + 1];
        rows[kStages - 1] = fetch(i + kStages, stage);
        if constexpr (kStages == 1) next = stats_of(rows[0]);
        stats = next;
        stage = stage == kStages - 1 ? 0 : stage + 1;
    }
    copy_wait<0>();
    if (!p.part) return;
    // Rows that the block held at once are added up through the ring's memory, in order.
    float *sums = reinterpret_cast<float *>(ring_memory);          // [thread][value]
    float *part = p.part + blockIdx.x * 2LL * p.C;
#pragma unroll
    for (int which = 0; which < 2; ++which) {
#pragma unroll
        for (int q = 0; q < P; ++q) {
            const int c = (q * lanes + lane) * V;
            float f[2 * N];
#pragma unroll
            for (int k = 0; k < N; ++k) unpack2(which ? db[q][k] : dw[q][k], f[2 * k], f[2 * k + 1]);
            if (per_block > 1) {
                __syncthreads();
#pragma unroll
                for (int k = 0; k < V; ++k) sums[k * THREADS + threadIdx.x] = f[k];
                __syncthreads();
                if (threadIdx.x >= lanes) continue;
                for (int g = 1; g < per_block; ++g)
#pragma unroll
                    for (int k = 0; k < V; ++k) f[k] += sums[k * THREADS + g * lanes + threadIdx.x];
            }
            if (c < p.C)
#pragma unroll
                for (int k = 0; k < V; ++k) part[which * static_cast<int64_t>(p.C) + c + k] = f[k];
        }
    }
}

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
__global__ void __launch_bounds__(kThreads) gdn_layer_norm_wide_kernel(const LayerNormParams<E> p) {
    for (int64_t row = blockIdx.x; row < p.rows; row += gridDim.x) {
        int b, t;
        locate(p, static_cast<int>(row), b, t);
        if (!is_valid(p, b, t)) continue;
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
__global__ void __launch_bounds__(kThreads) gdn_layer_norm_wide_dx_kernel(const LayerNormParams<E> p) {
    for (int64_t row = blockIdx.x; row < p.rows; row += gridDim.x) {
        int b, t;
        locate(p, static_cast<int>(row), b, t);
        if (!is_valid(p, b, t)) continue;
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
__global__ void __launch_bounds__(kThreads) gdn_layer_norm_wide_dw_kernel(const LayerNormParams<E> p) {
    const int c = blockIdx.x * kThreads + threadIdx.x;
    if (c >= p.C) return;
    float w = 0.f, bias = 0.f;
    for (int64_t row = blockIdx.y; row < p.rows; row += gridDim.y) {
        int b, t;
        locate(p, static_cast<int>(row), b, t);
        if (!is_valid(p, b, t)) continue;
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
    const int64_t rows = static_cast<int64_t>(p->B) * p->T;
    return align_up(static_cast<size_t>(rows < kMaxParts ? rows : kMaxParts) * 2 * p->C * 4);
}
static_assert(kWideParts <= kMaxParts, "workspace");

template <typename E>
LayerNormParams<E> params(const gdn_layer_norm_problem *p, const void *x, const int32_t *lengths) {
    LayerNormParams<E> a = {};
    a.x = static_cast<const E *>(x);
    a.lengths = lengths;
    a.x_sb = p->x_stride_b; a.x_st = p->x_stride_t;
    a.dy_sb = p->dy_stride_b; a.dy_st = p->dy_stride_t;
    a.rows = p->B * p->T;
    a.B = p->B; a.T = p->T; a.C = p->C;
    a.rms = (p->flags & GDN_LAYER_NORM_RMS) != 0;
    a.eps = p->eps;
    return a;
}

// Without lengths, rows at one distance are one sequence: no division to find a row.
template <typename E>
void flatten(LayerNormParams<E> &p) {
    if (p.T == 1) {
        p.x_st = p.x_sb;
        p.dy_st = p.dy_sb;
    }
    if (p.lengths || p.B == 1 || p.x_sb != p.T * p.x_st || (p.dy && p.dy_sb != p.T * p.dy_st)) return;
    p.T = p.rows;
    p.B = 1;
}

// Threads to a row of `pieces`, a power of two, with P pieces to a thread at most.
int lanes_for(int pieces, int P) {
    int lanes = 1;
    while (lanes < kMaxLanes && lanes * P < pieces) lanes *= 2;
    return lanes;
}

template <typename E, int V, int P>
cudaError_t launch_fwd(LayerNormParams<E> &p, cudaStream_t s) {
    const int threads = p.lanes > kThreads ? p.lanes : kThreads, per_block = threads / p.lanes;
    const unsigned blocks = static_cast<unsigned>((static_cast<int64_t>(p.rows) + per_block - 1) / per_block);
    gdn_layer_norm_kernel<E, V, P><<<blocks, threads, 0, s>>>(p);
    return cudaGetLastError();
}

template <typename E, int V>
cudaError_t fwd(LayerNormParams<E> &p, cudaStream_t s) {
    constexpr int most = V == 1 ? 16 : 8;      // pieces to a thread: at most 64 registers as fp32
    const int pieces = p.C / V;
    p.lanes = lanes_for(pieces, most);
    // few rows: more threads to each, so that every SM has work
    while (p.lanes < kMaxLanes && p.lanes < pieces && static_cast<int64_t>(p.rows) * p.lanes < 152 * 4 * kThreads)
        p.lanes *= 2;
    const int per = (pieces + p.lanes - 1) / p.lanes;
    if (per <= 1) return launch_fwd<E, V, 1>(p, s);
    if (per <= 2) return launch_fwd<E, V, 2>(p, s);
    if (per <= 4) return launch_fwd<E, V, 4>(p, s);
    if (per <= 8) return launch_fwd<E, V, 8>(p, s);
    if constexpr (V == 1)
        if (per <= 16) return launch_fwd<E, V, 16>(p, s);
    const unsigned blocks = static_cast<unsigned>(p.rows < 152 * 8 ? p.rows : 152 * 8);
    gdn_layer_norm_wide_kernel<E><<<blocks, kThreads, 0, s>>>(p);
    return cudaGetLastError();
}

template <typename E, int V, int P, int THREADS>
cudaError_t launch_bwd(LayerNormParams<E> &p, int &parts, cudaStream_t s) {
    p.lanes = lanes_for(p.C / V, P);
    const int per_block = THREADS / p.lanes, most = THREADS * P <= 512 ? kMaxParts : 152;
    const int64_t blocks = (static_cast<int64_t>(p.rows) + per_block - 1) / per_block;
    parts = static_cast<int>(blocks < most ? blocks : most);
    constexpr int bytes = row_stages(V, P, THREADS) * row_bytes(V, P, THREADS);
    static_assert(bytes >= THREADS * V * 4, "the ring holds a piece of sums of every thread");
    auto kernel = gdn_layer_norm_bwd_kernel<E, V, P, THREADS>;
    const cudaError_t e = cudaFuncSetAttribute(reinterpret_cast<const void *>(kernel),
                                               cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
    if (e != cudaSuccess) return e;
    kernel<<<parts, THREADS, bytes, s>>>(p);
    return cudaGetLastError();
}

// The pieces that a thread's registers hold, sums over rows among them, and beyond.
template <typename E, int V>
cudaError_t bwd(LayerNormParams<E> &p, int &parts, cudaStream_t s) {
    const int pieces = p.C / V;
    if (pieces <= 256) return launch_bwd<E, V, 1, 256>(p, parts, s);
    if (pieces <= 512) return launch_bwd<E, V, 2, 256>(p, parts, s);
    if constexpr (V == 1) {
        if (pieces <= 1024) return launch_bwd<E, V, 4, 256>(p, parts, s);
        if (pieces <= 2048) return launch_bwd<E, V, 8, 256>(p, parts, s);
        if (pieces <= 8192) return launch_bwd<E, V, 16, 512>(p, parts, s);
    } else {
        if (pieces <= 1024) return launch_bwd<E, V, 2, 512>(p, parts, s);
        if (pieces <= 2048) return launch_bwd<E, V, 4, 512>(p, parts, s);
        if constexpr (V <= 4)
            if (pieces <= 4096) return launch_bwd<E, V, 8, 512>(p, parts, s);
    }
    const unsigned blocks = static_cast<unsigned>(p.rows < 152 * 8 ? p.rows : 152 * 8);
    gdn_layer_norm_wide_dx_kernel<E><<<blocks, kThreads, 0, s>>>(p);
    cudaError_t err = cudaGetLastError();
    if (err != cudaSuccess || !p.part) return err;
    parts = p.rows < kWideParts ? p.rows : kWideParts;
    gdn_layer_norm_wide_dw_kernel<E><<<dim3((p.C + kThreads - 1) / kThreads, parts), kThreads, 0, s>>>(p);
    return cudaGetLastError();
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
        flatten(a);
        constexpr int V = 16 / sizeof(E);
        return pieces16(x, p->B, p->T, p->C, p->x_stride_b, p->x_stride_t, e) ? fwd<E, V>(a, s) : fwd<E, 1>(a, s);
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
    if (need && (!workspace || workspace_bytes < need)) return GDN_ERR_WORKSPACE;
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
        a.part = d_weight || d_bias ? static_cast<float *>(workspace) : nullptr;
        flatten(a);
        constexpr int V = 16 / sizeof(E);
        int parts = 0;
        const cudaError_t err = pieces16(x, p->B, p->T, p->C, p->x_stride_b, p->x_stride_t, e) &&
                                        pieces16(dy, p->B, p->T, p->C, p->dy_stride_b, p->dy_stride_t, e)
                                    ? bwd<E, V>(a, parts, s)
                                    : bwd<E, 1>(a, parts, s);
        if (err != cudaSuccess || !a.part) return err;
        return column_sums(a.part, parts, 2LL * p->C, p->C, d_weight, d_bias, s);
    };
    const cudaError_t err = p->dtype == GDN_BF16 ? go(__nv_bfloat16()) : go(float());
    return err == cudaSuccess ? GDN_OK : GDN_ERR_CUDA;
}

}  // extern "C"
