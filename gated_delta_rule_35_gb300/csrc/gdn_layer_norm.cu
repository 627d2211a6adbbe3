// Layer norm of every token and its backward pass: gdn_layer_norm and gdn_layer_norm_bwd
// of include/gdn.h.
//
// Bound by memory: x read and y written; in the backward pass x and dy read and dx written. Blocks
// stay for many rows. A row is held by `lanes` threads (a power of two up to a warp, or whole
// warps) in pieces of V channels (16 bytes, or one channel where rows are not whole 16-byte
// pieces), P to a thread, which keeps its channels: weight and bias stay in registers, and so do
// the sums over rows that are their gradients, of which every block leaves a row of partial sums.
// The rows of the next turns are on their way to shared memory meanwhile (cp.async, a ring of a
// thread's own). A turn takes R rows, whose sums over threads share their shuffles and barriers:
// the mean, then the squares about it; in the backward pass both sums at once. Rows beyond what a
// block holds go to the *_wide_* kernels, a block to a row that it reads again for each sum.
//
// 65536 x 4096 bf16: 165 us, 6.53 TB/s (98% of a plain copy's 6.68), the gradients 252 us, 6.41 TB/s
// (96%), 6 us of them the sums over the blocks' rows. A block to a row with every value read three
// times took 434 and 2189 us; a part of a warp to a row, weight and bias read for each, 246. fp32
// 32768 x 4096: 177 and 251 us; 65536 x 2560 bf16 137 and 195 (154 and 227 with a power of two of
// threads to a row); rows of 1003: bf16 60 and 85, fp32 64 and 101 (4 single channels to a thread, read one by
// one: 284 and 142 the norm).
#include "columns.cuh"
#include "rows.cuh"

namespace gdn {

// The pairs' operations on single values (beside them: inner scopes would hide the pairs').
__device__ __forceinline__ float fma2(float a, float b, float c) { return fmaf(a, b, c); }
__device__ __forceinline__ float mul2(float a, float b) { return a * b; }
__device__ __forceinline__ float add2(float a, float b) { return a + b; }

namespace {

constexpr int kThreads = 256;
constexpr int kWideParts = 64;     // rows of partial sums of the wide kernels
constexpr int kMaxParts = 152 * 2; // blocks of the backward pass

// Blocks to an SM. Of the backward pass three would spill: 302 us for 257 on 65536 x 4096 bf16; of
// the forward pass three take 177 for 170.
constexpr int blocks_to_sm(int threads) { return threads > 256 ? 1 : 2; }

template <typename E>
struct LayerNormParams {
    const E *x, *dy;
    const float *w, *bias, *stats_in;
    const int32_t *lengths;
    E *y, *dx;
    float *stats, *part;
    int64_t x_sb, x_st, dy_sb, dy_st;
    RowSpan x_span, dy_span;
    int rows, B, T, C, lanes;
    bool rms;
    float eps;
};

// What the arithmetic below takes: pairs of channels, or single ones where V is 1.
template <int V>
struct Lanes {
    static constexpr int N = (V + 1) / 2;
    using T = typename std::conditional<V == 1, float, F2>::type;
    static __device__ __forceinline__ T both(float v) {
        if constexpr (V == 1) return v; else return pack2(v, v);
    }
    static __device__ __forceinline__ float sum(T v) {
        if constexpr (V == 1) {
            return v;
        } else {
            float a, b;
            unpack2(v, a, b);
            return a + b;
        }
    }
    static __device__ __forceinline__ void values(const T (&f)[N], float (&v)[V]) {
        if constexpr (V == 1) {
            v[0] = f[0];
        } else {
#pragma unroll
            for (int k = 0; k < N; ++k) unpack2(f[k], v[2 * k], v[2 * k + 1]);
        }
    }
    // Channels c.. of a parameter, `other` without any.
    static __device__ __forceinline__ void params(const float *p, int c, float other, T (&f)[N]) {
        float v[V];
        if (p) {
            load_f32<V>(p + c, v);
        } else {
#pragma unroll
            for (int i = 0; i < V; ++i) v[i] = other;
        }
#pragma unroll
        for (int i = 0; i < N; ++i) {
            if constexpr (V == 1) f[i] = v[i]; else f[i] = pack2(v[2 * i], v[2 * i + 1]);
        }
    }
};

// Sums of N values over the `lanes` threads of a row, whose first warp is `first_warp` where they are
// whole warps, for all of them. Within a warp the values
// are shared out over the lanes as the sums go on: 6 shuffles for four values, not 20. Calls in a
// row alternate between two `buffer`s.
template <int N, int WARPS>
__device__ __forceinline__ void row_sums(float (&v)[N], int lanes, int first_warp, float (&buffer)[WARPS][N]) {
    static_assert((N == 1 || N == 2 || N == 4) && WARPS * N <= 64, "values");
    constexpr uint32_t all = 0xffffffffu;
    if (lanes < 32) {
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) {
            if (o >= lanes) continue;                  // alike for all threads
#pragma unroll
            for (int i = 0; i < N; ++i) v[i] += __shfl_xor_sync(all, v[i], o);
        }
        return;
    }
    const int lane = threadIdx.x % 32;
    int o = 16;
#pragma unroll
    for (int n = N; n > 1; n /= 2, o /= 2) {           // half of the values to each half of the lanes
        const bool upper = lane & o;
#pragma unroll
        for (int i = 0; i < n / 2; ++i) {
            const float give = upper ? v[i] : v[i + n / 2], keep = upper ? v[i + n / 2] : v[i];
            v[i] = keep + __shfl_xor_sync(all, give, o);
        }
    }
    float s = v[0];
#pragma unroll
    for (int q = 16 / N; q > 0; q /= 2) s += __shfl_xor_sync(all, s, q);
    constexpr int per = 32 / N;                        // lanes that hold a value's sum
    if (lanes == 32) {
#pragma unroll
        for (int i = 0; i < N; ++i) v[i] = __shfl_sync(all, s, i * per);
        return;
    }
    if (lane % per == 0) buffer[threadIdx.x / 32][lane / per] = s;
    __syncthreads();
    // value i of warp w at i + N w: a lane takes every 32nd, the same value of each (16 warps at most);
    // a power of two of them without bounds: 169 us for 179 (65536 x 4096 bf16)
    const float *from = &buffer[first_warp][0];
    const int count = lanes / 32 * N;
    if ((count & (count - 1)) == 0) {
        s = from[lane & (count - 1)];
        if (count > 32) s += from[lane + 32];
        for (int q = N; q < 32 && q < count; q *= 2) s += __shfl_xor_sync(all, s, q);
    } else {
        s = lane < count ? from[lane] : 0.f;
        if (lane + 32 < count) s += from[lane + 32];
#pragma unroll
        for (int q = N; q < 32; q *= 2) s += __shfl_xor_sync(all, s, q);
    }
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] = __shfl_sync(all, s, i);
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

// The rows of a block and their ring, for TENSORS of them (x, then dy): as many rows a turn, up to four
// (two in the backward pass, whose rows have two sums), as leave the ring two turns, three where a
// block has an SM for itself. One, two and four: 220, 182 and 170 us (65536 x 4096 bf16), with a
// third turn 175; blocks of 512 threads 183 with two, 177 with three (32768 x 4096 fp32). A thread fills and reads
// slots of its own; in bf16 rows that are not whole pieces, whose elements are less than an
// asynchronous copy moves, the threads of a row copy the aligned pieces that it touches.
constexpr int kMinLanes = 8;
template <typename E, int V, int P, int THREADS, int TENSORS>
struct RowRing {
    static constexpr bool SHARED = V == 1 && sizeof(E) == 2;
    // a piece, or an element of fp32
    using Slot = typename std::conditional<V == 1, float, uint4>::type;
    using L = Lanes<V>;
    using T = typename L::T;
    static constexpr int N = L::N;
    static constexpr int row_bytes =
        TENSORS * (SHARED ? THREADS * P * 2 + THREADS / kMinLanes * 16 : THREADS * P * static_cast<int>(sizeof(Slot)));
    static constexpr int most = (THREADS > 256 ? 200 : 96) * 1024;
    // what the registers of single channels hold, and bytes enough in flight, count too: rows of 4097 with
    // one, two and four to a turn 398, 328 and 483 us in bf16, 368 and 316 in fp32 (32768 of them)
    static constexpr int wanted = V == 1 && P > 8                                     ? 3 - TENSORS
                                  : TENSORS == 1 && (sizeof(E) == 2 || THREADS == 256) ? 4
                                                                                       : 2;
    static constexpr int R = wanted >= 4 && 8 * row_bytes <= most ? 4 : wanted >= 2 && 4 * row_bytes <= most ? 2 : 1;
    static constexpr int stages = THREADS > 256 && 3 * R * row_bytes <= most ? 3 : 2 * R * row_bytes <= most ? 2 : 1;
    static constexpr int ring = stages * R * row_bytes, sums = THREADS * V * 4;
    static constexpr int bytes = ring > sums ? ring : sums;        // sums: of a piece of every thread

    const LayerNormParams<E> &p;
    unsigned char *memory;
    int lane, lanes, first_warp, step, turns;
    int64_t first;

    __device__ __forceinline__ RowRing(const LayerNormParams<E> &p, uint4 *at)
        : p(p), memory(reinterpret_cast<unsigned char *>(at)), lane(threadIdx.x % p.lanes), lanes(p.lanes) {
        const int per_block = blockDim.x / lanes;
        first_warp = threadIdx.x / lanes * (lanes / 32);
        memory += SHARED ? threadIdx.x / lanes * (lanes * P * 2 + 16) : threadIdx.x * static_cast<int>(sizeof(Slot));
        step = gridDim.x * per_block;
        // alike for all threads
        turns = static_cast<int>((p.rows + static_cast<int64_t>(R) * step - 1) / (static_cast<int64_t>(R) * step));
        first = static_cast<int64_t>(blockIdx.x) * per_block + threadIdx.x / lanes;
    }
    __device__ __forceinline__ int channel(int q) const { return (q * lanes + lane) * V; }
    __device__ __forceinline__ unsigned char *slot(int stage, int r, int n) const {
        return memory + ((stage * R + r) * TENSORS + n) * (row_bytes / TENSORS);
    }
    __device__ __forceinline__ const E *source(int n, int b, int t) const {
        return n == 0 ? p.x + (b * p.x_sb + t * p.x_st) : p.dy + (b * p.dy_sb + t * p.dy_st);
    }
    // Asks for the rows of turn i; those that there are (-1: none).
    __device__ __forceinline__ void fetch(int i, int stage, int (&rows)[R]) const {
        if (i >= turns) {          // 1 x 2048 took 8.9 us for 6.8 with such turns' slots cleared
#pragma unroll
            for (int r = 0; r < R; ++r) rows[r] = -1;
            copy_commit();
            return;
        }
#pragma unroll
        for (int r = 0; r < R; ++r) {
            const int64_t at = first + (static_cast<int64_t>(i) * R + r) * step;
            int b = 0, t = 0;
            rows[r] = -1;
            if (at < p.rows) {
                locate(p, static_cast<int>(at), b, t);
                if (is_valid(p, b, t)) rows[r] = static_cast<int>(at);
            }
#pragma unroll
            for (int n = 0; n < TENSORS; ++n) {
                const E *from = source(n, b, t);
                if constexpr (SHARED) {
                    if (rows[r] < 0) continue;
                    const RowCopy<E> copy(n == 0 ? p.x_span : p.dy_span, from, 0, 1, p.C);
#pragma unroll
                    for (int k = 0; k <= P / 8; ++k) copy(slot(stage, r, n), from, p.C, k * lanes + lane);
                } else {
                    Slot *to = reinterpret_cast<Slot *>(slot(stage, r, n));
#pragma unroll
                    for (int q = 0; q < P; ++q, to += THREADS) {
                        const int c = channel(q);
                        if (rows[r] >= 0 && c < p.C) {
                            if constexpr (V > 1)
                                copy16_async(to, from + c);
                            else
                                copy4_async(to, from + c);
                        } else {
                            memset(to, 0, sizeof(Slot));
                        }
                    }
                }
            }
        }
        copy_commit();
    }
    // Behind the wait for a turn's rows, and before they are filled anew: of rows that threads fill
    // together. Between the two come the sums over threads, with the barrier that many lanes take.
    __device__ __forceinline__ void arrived() const {
        if (!SHARED) return;
        if (lanes > 32) __syncthreads(); else __syncwarp();
    }
    __device__ __forceinline__ void done() const {
        if (SHARED) __syncwarp();
    }
    // Single values are read once, pieces where they are needed.
    struct Row {
        T kept[V == 1 ? P : 1];
    };
    __device__ __forceinline__ void open(int stage, int r, int n, int row, Row &of) const {
        if constexpr (V == 1) {
            const E *v = nullptr;
            if constexpr (SHARED) {
                int b = 0, t = 0;
                if (row >= 0) locate(p, row, b, t);
                v = row_in_copy<E>(slot(stage, r, n), source(n, b, t));
            }
#pragma unroll
            for (int q = 0; q < P; ++q) {
                if constexpr (SHARED)
                    of.kept[q] = row >= 0 && channel(q) < p.C ? to_f32(v[channel(q)]) : 0.f;
                else
                    of.kept[q] = reinterpret_cast<const Slot *>(slot(stage, r, n))[q * THREADS];
            }
        }
    }
    __device__ __forceinline__ void read(const Row &of, int stage, int r, int n, int q, T (&f)[N]) const {
        if constexpr (V == 1) {
            f[0] = of.kept[q];
        } else {
            Piece<E, V> piece;
            piece.raw = reinterpret_cast<const Slot *>(slot(stage, r, n))[q * THREADS];
            piece.widen(f);
        }
    }
    static __device__ __forceinline__ void write(E *at, const T (&f)[N]) {
        if constexpr (V == 1) {
            *at = from_f32<E>(f[0]);
        } else {
            Piece<E, V> piece;
            piece.round(f);
            piece.store(at);
        }
    }
};

template <typename E, int V, int P, int THREADS>
__global__ void __launch_bounds__(THREADS, blocks_to_sm(THREADS))
    gdn_layer_norm_kernel(const LayerNormParams<E> p) {
    using Ring = RowRing<E, V, P, THREADS, 1>;
    using L = typename Ring::L;
    using T = typename Ring::T;
    constexpr int N = Ring::N, R = Ring::R, S = Ring::stages;
    __shared__ float buffers[2][THREADS / 32][R];
    extern __shared__ uint4 ring_memory[];
    Ring ring(p, ring_memory);
    const float inv = 1.f / p.C;
    // 16 channels' weight and bias stay in registers, more are read for every row
    constexpr bool KEEP = P * V <= 16;
    T w[KEEP ? P : 1][N], bias[KEEP ? P : 1][N];
    if constexpr (KEEP) {
#pragma unroll
        for (int q = 0; q < P; ++q) {
            const int c = ring.channel(q) < p.C ? ring.channel(q) : 0;
            L::params(p.w, c, 1.f, w[q]);
            L::params(p.bias, c, 0.f, bias[q]);
        }
    }
    int rows[S][R];
#pragma unroll
    for (int i = 0; i < S; ++i) ring.fetch(i, i, rows[i]);
    int stage = 0;
    for (int i = 0; i < ring.turns; ++i) {
        copy_wait<S - 1>();
        ring.arrived();
        typename Ring::Row xs[R];
#pragma unroll
        for (int r = 0; r < R; ++r) ring.open(stage, r, 0, rows[0][r], xs[r]);
        float mean[R], s[R];
        T sum[R];
#pragma unroll
        for (int r = 0; r < R; ++r) {
            mean[r] = 0.f;
            sum[r] = L::both(0.f);
        }
        if (!p.rms) {
#pragma unroll
            for (int r = 0; r < R; ++r) {
#pragma unroll
                for (int q = 0; q < P; ++q) {
                    T v[N];
                    ring.read(xs[r], stage, r, 0, q, v);
#pragma unroll
                    for (int k = 0; k < N; ++k) sum[r] = add2(sum[r], v[k]);
                }
                s[r] = L::sum(sum[r]);
                sum[r] = L::both(0.f);
            }
            row_sums(s, ring.lanes, ring.first_warp, buffers[0]);
#pragma unroll
            for (int r = 0; r < R; ++r) mean[r] = s[r] * inv;
        }
#pragma unroll
        for (int r = 0; r < R; ++r) {
#pragma unroll
            for (int q = 0; q < P; ++q) {
                T v[N], squares = L::both(0.f);
                ring.read(xs[r], stage, r, 0, q, v);
#pragma unroll
                for (int k = 0; k < N; ++k) {
                    v[k] = add2(v[k], L::both(-mean[r]));
                    squares = fma2(v[k], v[k], squares);
                }
                if (ring.channel(q) < p.C) sum[r] = add2(sum[r], squares);
            }
            s[r] = L::sum(sum[r]);
        }
        // without the first sums the buffers alternate from turn to turn
        row_sums(s, ring.lanes, ring.first_warp, buffers[p.rms ? i & 1 : 1]);
#pragma unroll
        for (int r = 0; r < R; ++r) {
            const int row = rows[0][r];
            if (row < 0) continue;
            const float rstd = rsqrtf(fmaf(s[r], inv, p.eps));
            E *y = p.y + static_cast<int64_t>(row) * p.C;
#pragma unroll
            for (int q = 0; q < P; ++q) {
                const int c = ring.channel(q);
                if (c >= p.C) break;
                T v[N];
                ring.read(xs[r], stage, r, 0, q, v);
                constexpr int one = KEEP ? 1 : 0;
                if constexpr (!KEEP) {
                    L::params(p.w, c, 1.f, w[0]);
                    L::params(p.bias, c, 0.f, bias[0]);
                }
#pragma unroll
                for (int k = 0; k < N; ++k)
                    v[k] = fma2(mul2(add2(v[k], L::both(-mean[r])), L::both(rstd)), w[q * one][k], bias[q * one][k]);
                Ring::write(y + c, v);
            }
            if (p.stats && ring.lane == 0)
                *reinterpret_cast<float2 *>(p.stats + 2LL * row) = make_float2(mean[r], rstd);
        }
#pragma unroll
        for (int k = 0; k + 1 < S; ++k)
#pragma unroll
            for (int r = 0; r < R; ++r) rows[k][r] = rows[k + 1][r];
        ring.done();
        ring.fetch(i + S, stage, rows[S - 1]);
        stage = stage == S - 1 ? 0 : stage + 1;
    }
    copy_wait<0>();
}

template <typename E, int V, int P, int THREADS>
__global__ void __launch_bounds__(THREADS, blocks_to_sm(THREADS))
    gdn_layer_norm_bwd_kernel(const LayerNormParams<E> p) {
    using Ring = RowRing<E, V, P, THREADS, 2>;
    using L = typename Ring::L;
    using T = typename Ring::T;
    constexpr int N = Ring::N, R = Ring::R, S = Ring::stages;
    __shared__ float buffers[2][THREADS / 32][2 * R];
    extern __shared__ uint4 ring_memory[];
    Ring ring(p, ring_memory);
    const float inv = 1.f / p.C;
    T w[P][N], dw[P][N], db[P][N];
#pragma unroll
    for (int q = 0; q < P; ++q) {
        const int c = ring.channel(q);
#pragma unroll
        for (int k = 0; k < N; ++k) dw[q][k] = db[q][k] = L::both(0.f);
        L::params(p.w, c < p.C ? c : 0, 1.f, w[q]);
    }
    int rows[S][R];
    float2 stats[R], next[R];
    auto stats_of = [&](const int (&of)[R], float2 (&to)[R]) {
#pragma unroll
        for (int r = 0; r < R; ++r)
            to[r] = of[r] < 0 ? make_float2(0.f, 0.f) : *reinterpret_cast<const float2 *>(p.stats_in + 2LL * of[r]);
    };
#pragma unroll
    for (int i = 0; i < S; ++i) ring.fetch(i, i, rows[i]);
    stats_of(rows[0], stats);
    int stage = 0;
    for (int i = 0; i < ring.turns; ++i) {
        if constexpr (S > 1) stats_of(rows[1], next);      // asked for a turn ahead
        copy_wait<S - 1>();
        ring.arrived();
        typename Ring::Row xs[R], dys[R];
#pragma unroll
        for (int r = 0; r < R; ++r) {
            ring.open(stage, r, 0, rows[0][r], xs[r]);
            ring.open(stage, r, 1, rows[0][r], dys[r]);
        }
        float s[2 * R];
#pragma unroll
        for (int r = 0; r < R; ++r) {
            const T minus = L::both(-stats[r].x), rstd = L::both(stats[r].y);
            T s1 = L::both(0.f), s2 = L::both(0.f);
#pragma unroll
            for (int q = 0; q < P; ++q) {
                T x[N], dy[N];
                ring.read(xs[r], stage, r, 0, q, x);
                ring.read(dys[r], stage, r, 1, q, dy);
#pragma unroll
                for (int k = 0; k < N; ++k) {
                    const T xhat = mul2(add2(x[k], minus), rstd), v = mul2(dy[k], w[q][k]);
                    db[q][k] = add2(db[q][k], dy[k]);
                    dw[q][k] = fma2(dy[k], xhat, dw[q][k]);
                    s1 = add2(s1, v);
                    s2 = fma2(v, xhat, s2);
                }
            }
            s[2 * r] = L::sum(s1);
            s[2 * r + 1] = L::sum(s2);
        }
        row_sums(s, ring.lanes, ring.first_warp, buffers[i & 1]);
#pragma unroll
        for (int r = 0; r < R; ++r) {
            const int row = rows[0][r];
            if (row < 0) continue;
            const T minus = L::both(-stats[r].x), rstd = L::both(stats[r].y);
            const T c1 = L::both(p.rms ? 0.f : -s[2 * r] * inv), c2 = L::both(-s[2 * r + 1] * inv);
            E *dx = p.dx + static_cast<int64_t>(row) * p.C;
#pragma unroll
            for (int q = 0; q < P; ++q) {
                const int c = ring.channel(q);
                if (c >= p.C) break;
                T x[N], dy[N];
                ring.read(xs[r], stage, r, 0, q, x);
                ring.read(dys[r], stage, r, 1, q, dy);
#pragma unroll
                for (int k = 0; k < N; ++k) {
                    const T xhat = mul2(add2(x[k], minus), rstd);
                    x[k] = mul2(rstd, fma2(xhat, c2, fma2(dy[k], w[q][k], c1)));
                }
                Ring::write(dx + c, x);
            }
        }
#pragma unroll
        for (int k = 0; k + 1 < S; ++k)
#pragma unroll
            for (int r = 0; r < R; ++r) rows[k][r] = rows[k + 1][r];
        ring.done();
        ring.fetch(i + S, stage, rows[S - 1]);
        if constexpr (S == 1) stats_of(rows[0], next);
#pragma unroll
        for (int r = 0; r < R; ++r) stats[r] = next[r];
        stage = stage == S - 1 ? 0 : stage + 1;
    }
    copy_wait<0>();
    if (!p.part) return;
    // Rows that the block held at once are added up through the ring's memory, in order.
    const int lanes = ring.lanes, per_block = blockDim.x / lanes;
    float *sums = reinterpret_cast<float *>(ring_memory);          // [value][thread]
    float *part = p.part + blockIdx.x * 2LL * p.C;
#pragma unroll
    for (int which = 0; which < 2; ++which) {
#pragma unroll
        for (int q = 0; q < P; ++q) {
            const int c = ring.channel(q);
            float f[V];
            if (which) L::values(db[q], f); else L::values(dw[q], f);
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
    a.x_span = row_span(x, p->B, p->T, p->C, a.x_sb, a.x_st, sizeof(E));
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

// Blocks that stay: as many as an SM holds at once, or rows.
template <typename E, int V, int P, int THREADS, int TENSORS>
cudaError_t launch_rows(LayerNormParams<E> &p, int &blocks, cudaStream_t s) {
    using Ring = RowRing<E, V, P, THREADS, TENSORS>;
    const int threads = (p.C / V + P - 1) / P;         // that a row needs
    p.lanes = V == 1 ? kMinLanes : 1;
    while (p.lanes < 32 && p.lanes < threads) p.lanes *= 2;
    if (threads > 32) p.lanes = (threads + 31) / 32 * 32;
    const int per_block = THREADS / p.lanes, sm = blocks_to_sm(THREADS);
    const int64_t all = (static_cast<int64_t>(p.rows) + per_block - 1) / per_block;
    blocks = static_cast<int>(all < 152 * sm ? all : 152 * sm);
    auto kernel = TENSORS == 1 ? gdn_layer_norm_kernel<E, V, P, THREADS> : gdn_layer_norm_bwd_kernel<E, V, P, THREADS>;
    const cudaError_t e = cudaFuncSetAttribute(reinterpret_cast<const void *>(kernel),
                                               cudaFuncAttributeMaxDynamicSharedMemorySize, Ring::bytes);
    if (e != cudaSuccess) return e;
    kernel<<<blocks, per_block * p.lanes, Ring::bytes, s>>>(p);
    return cudaGetLastError();
}

// By the pieces of a row: a block of 256 threads with two pieces (8 or 16 single channels) to a thread,
// then of 512 with what its registers hold. `held`: whether they hold a row.
template <typename E, int V, int TENSORS>
cudaError_t by_pieces(LayerNormParams<E> &p, int &blocks, bool &held, cudaStream_t s) {
    const int pieces = p.C / V;
    held = true;
    if constexpr (V == 1) {
        if (pieces <= 2048) return launch_rows<E, V, 8, 256, TENSORS>(p, blocks, s);
        if (pieces <= 4096) return launch_rows<E, V, 16, 256, TENSORS>(p, blocks, s);
        if (pieces <= 8192) return launch_rows<E, V, 16, 512, TENSORS>(p, blocks, s);
    } else {
        if (pieces <= 512) return launch_rows<E, V, 2, 256, TENSORS>(p, blocks, s);
        if (pieces <= 1024) return launch_rows<E, V, 2, 512, TENSORS>(p, blocks, s);
        if (pieces <= 2048) return launch_rows<E, V, 4, 512, TENSORS>(p, blocks, s);
        if constexpr (V <= 4)
            if (pieces <= 4096) return launch_rows<E, V, 8, 512, TENSORS>(p, blocks, s);
    }
    held = false;
    return cudaSuccess;
}

template <typename E, int V>
cudaError_t fwd(LayerNormParams<E> &p, cudaStream_t s) {
    int blocks;
    bool held;
    const cudaError_t err = by_pieces<E, V, 1>(p, blocks, held, s);
    if (held) return err;
    blocks = p.rows < 152 * 8 ? p.rows : 152 * 8;
    gdn_layer_norm_wide_kernel<E><<<blocks, kThreads, 0, s>>>(p);
    return cudaGetLastError();
}

template <typename E, int V>
cudaError_t bwd(LayerNormParams<E> &p, int &parts, cudaStream_t s) {
    bool held;
    cudaError_t err = by_pieces<E, V, 2>(p, parts, held, s);
    if (held) return err;
    const int blocks = p.rows < 152 * 8 ? p.rows : 152 * 8;
    gdn_layer_norm_wide_dx_kernel<E><<<blocks, kThreads, 0, s>>>(p);
    err = cudaGetLastError();
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
        a.dy_span = row_span(dy, p->B, p->T, p->C, a.dy_sb, a.dy_st, e);
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
