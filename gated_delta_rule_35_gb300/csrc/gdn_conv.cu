// Causal depthwise convolution over tokens with its window state: gdn_conv_fwd of
// include/gdn.h.
//
// Bound by memory: one read of x and one write of y. A thread owns a piece of V
// channels (16 bytes, or one channel where rows are not whole 16-byte pieces) over a
// run of tokens, with its weights and the W - 1 previous inputs in registers, so x is
// read once but for the W - 1 tokens before each run. A turn of the loop takes U
// tokens; the next turns' pieces are on their way to shared memory meanwhile.
//
// B8 T8192 C8192, W = 4, bf16, SiLU: 326 us, 6.58 TB/s (97% of a plain copy's 6.77).
// The ring is what reaches that: with the pieces loaded to registers one turn ahead the
// same arithmetic took 400 us, with eight tokens' loads and no lead 376 us, since the
// weights and the window leave registers for only 16 warps on an SM and their loads
// did not cover the memory's 2.4 us under load. A 64-token run re-reads 3 / 64 of x, from
// L2; 128 tokens measured 328 us, 256 333 us (fewer blocks at the end of the grid).
#include "mixer.cuh"

namespace gdn {
namespace {

constexpr int kThreads = 128;
constexpr int kUnroll = 4;      // tokens per turn
constexpr int kStages = 4;      // turns in the ring, all but one of them in flight
constexpr int kStepTokens = 4;  // up to here the step kernel
constexpr int kMaxRun = 64;     // tokens per thread at most; a call of several runs has kUnroll or more to
                                // each, so that only the first run reads the window state
static_assert(kUnroll >= 3, "W - 1");

template <typename E>
struct ConvParams {
    const E *x;
    const float *w, *bias;
    const E *state_in;
    const int32_t *lengths;
    E *y, *state_out;
    int64_t sb, st;
    int B, T, C, act, run;
};

// Inputs at token t of sequence b, channels c..; t >= -(W - 1), tokens before 0 come
// from the window state.
template <typename E, int W, int V>
__device__ __forceinline__ void input_at(Piece<E, V> &q, const ConvParams<E> &p, int64_t b, int t,
                                         int c) {
    if (t >= 0)
        q.load(p.x + b * p.sb + t * p.st + c);
    else if (p.state_in)
        q.load_rw(p.state_in + (b * (W - 1) + W - 1 + t) * p.C + c);
    else
        q.zero();
}

// SILU: its activation without a branch per value, the others by p.act.
// RING: 16-byte pieces reach the thread through its ring of slots in shared memory.
template <typename E, int W, int V, bool SILU, bool RING = (V > 1)>
__global__ void __launch_bounds__(kThreads) gdn_conv_kernel(const ConvParams<E> p) {
    constexpr int U = kUnroll;
    const int cv = p.C / V;                            // pieces of a row
    const int i = blockIdx.x * kThreads + threadIdx.x;
    const int c = i % cv * V, t0 = i / cv * p.run;     // runs of a piece lie cv threads apart
    const int64_t b = blockIdx.y;
    if (t0 >= p.T) return;
    const int n = valid_tokens(p.lengths, b, p.T);
    if (t0 < n) {
        // in pairs of channels: one instruction works on both
        constexpr int P = (V + 1) / 2;
        F2 w2[P][W], bias2[P];
        float w[V * W], bias[V];
        load_f32<V * W>(p.w + static_cast<int64_t>(c) * W, w);   // [V][W]
        if (p.bias) {
            load_f32<V>(p.bias + c, bias);
        } else {
#pragma unroll
            for (int j = 0; j < V; ++j) bias[j] = 0.f;
        }
        // pair(f, j): channels 2 j and 2 j + 1 of f (its single channel twice where V is 1)
        auto pair = [](const float *f, int j) { return pack2(f[2 * j], f[V == 1 ? 0 : 2 * j + 1]); };
#pragma unroll
        for (int j = 0; j < P; ++j) {
            bias2[j] = pair(bias, j);
#pragma unroll
            for (int k = 0; k < W; ++k)
                w2[j][k] = pack2(w[2 * j * W + k], w[(V == 1 ? 0 : 2 * j + 1) * W + k]);
        }
        F2 in[W - 1 + U][P];     // the window, then this turn's tokens
#pragma unroll
        for (int k = 0; k < W - 1; ++k) {
            Piece<E, V> before;
            float f[V];
            input_at<E, W, V>(before, p, b, t0 - W + 1 + k, c);
            before.widen(f);
#pragma unroll
            for (int j = 0; j < P; ++j) in[k][j] = pair(f, j);
        }
        const E *x = p.x + b * p.sb + t0 * p.st + c;
        E *y = p.y + (b * p.T + t0) * p.C + c;
        int left = min(p.run, n - t0);
        // One token: widen its piece into place u of the turn; its output to y.
        auto take = [&](const Piece<E, V> &q, int u) {
            float f[V];
            q.widen(f);
#pragma unroll
            for (int j = 0; j < P; ++j) in[W - 1 + u][j] = pair(f, j);
        };
        auto give = [&](int u) {
            float out[V + 1];
#pragma unroll
            for (int j = 0; j < P; ++j) {
                F2 v = bias2[j];
#pragma unroll
                for (int k = 0; k < W; ++k) v = fma2(w2[j][k], in[u + k][j], v);
                v = activate2(v, SILU ? GDN_ACT_SILU : p.act);
                unpack2(v, out[2 * j], out[2 * j + 1]);
            }
            Piece<E, V> r;
            r.round(reinterpret_cast<const float (&)[V]>(out));
            r.store(y + static_cast<int64_t>(u) * p.C);
        };
        auto advance = [&] {
#pragma unroll
            for (int k = 0; k < W - 1; ++k)
#pragma unroll
                for (int j = 0; j < P; ++j) in[k][j] = in[U + k][j];
            y += static_cast<int64_t>(U) * p.C;
        };
        if constexpr (RING) {
            // Each thread fills and reads its own slots, so nothing is synchronised.
            extern __shared__ uint4 ring[];
            uint4 *mine = ring + threadIdx.x;
            int ahead = left, slot = 0;
            auto fetch = [&](int s) {
#pragma unroll
                for (int u = 0; u < U; ++u)
                    if (u < ahead) copy16_async(mine + (s * U + u) * kThreads, x + u * p.st);
                copy_commit();
                ahead -= U;
                x += U * p.st;
            };
#pragma unroll
            for (int s = 0; s < kStages - 1; ++s) fetch(s);
            for (; left > 0; left -= U) {
                copy_wait<kStages - 2>();
#pragma unroll
                for (int u = 0; u < U; ++u) {
                    Piece<E, V> q;
                    q.raw = mine[(slot * U + u) * kThreads];
                    take(q, u);
                }
                fetch(slot == 0 ? kStages - 1 : slot - 1);
                slot = slot == kStages - 1 ? 0 : slot + 1;
                if (left >= U) {
#pragma unroll
                    for (int u = 0; u < U; ++u) give(u);
                    advance();
                } else {
#pragma unroll
                    for (int u = 0; u < U; ++u)
                        if (u < left) give(u);
                }
            }
            copy_wait<0>();
        } else {
            for (; left > 0; left -= U) {
                Piece<E, V> q[U];
#pragma unroll
                for (int u = 0; u < U; ++u) {
                    q[u].zero();
                    if (u < left) q[u].load(x + u * p.st);
                }
#pragma unroll
                for (int u = 0; u < U; ++u) take(q[u], u);
#pragma unroll
                for (int u = 0; u < U; ++u)
                    if (u < left) give(u);
                advance();
                x += U * p.st;
            }
        }
    }
    // The thread that read this piece of state_in writes its state_out, after
    // reading all of it: the two may be the same buffer.
    if (t0 == 0 && p.state_out) {
        Piece<E, V> last[W - 1];
#pragma unroll
        for (int k = 0; k < W - 1; ++k) input_at<E, W, V>(last[k], p, b, n - W + 1 + k, c);
#pragma unroll
        for (int k = 0; k < W - 1; ++k) last[k].store(p.state_out + (b * (W - 1) + k) * p.C + c);
    }
}

// A few tokens: a thread takes a piece of NB sequences, whose windows' and tokens' loads
// are in flight together, and reads the weights once for all of them.
constexpr int kStepBatch = 4;

template <typename E, int W, int V, int NB, bool SILU>
__global__ void __launch_bounds__(kThreads) gdn_conv_step_kernel(const ConvParams<E> p) {
    constexpr int P = (V + 1) / 2;
    const int c = (blockIdx.x * kThreads + threadIdx.x) * V;
    const int b0 = blockIdx.y * NB;
    if (c >= p.C) return;
    Piece<E, V> win[NB][W - 1], x[NB];
    int n[NB];
#pragma unroll
    for (int m = 0; m < NB; ++m) {
        const int64_t b = b0 + m;
        n[m] = b < p.B ? valid_tokens(p.lengths, b, p.T) : 0;
#pragma unroll
        for (int k = 0; k < W - 1; ++k) {
            win[m][k].zero();
            if (b < p.B && p.state_in) win[m][k].load_rw(p.state_in + (b * (W - 1) + k) * p.C + c);
        }
        if (n[m] > 0) x[m].load(p.x + b * p.sb + c);
    }
    F2 w2[P][W], bias2[P];
    {
        float w[V * W], bias[V];
        load_f32<V * W>(p.w + static_cast<int64_t>(c) * W, w);
#pragma unroll
        for (int j = 0; j < V; ++j) bias[j] = 0.f;
        if (p.bias) load_f32<V>(p.bias + c, bias);
#pragma unroll
        for (int j = 0; j < P; ++j) {
            const int o = V == 1 ? 0 : 2 * j + 1;
            bias2[j] = pack2(bias[2 * j], bias[o]);
#pragma unroll
            for (int k = 0; k < W; ++k) w2[j][k] = pack2(w[2 * j * W + k], w[o * W + k]);
        }
    }
    for (int t = 0; t < p.T; ++t) {
#pragma unroll
        for (int m = 0; m < NB; ++m) {
            if (t >= n[m]) continue;
            const int64_t b = b0 + m;
            F2 v[P], in[P];
#pragma unroll
            for (int j = 0; j < P; ++j) v[j] = bias2[j];
#pragma unroll
            for (int k = 0; k < W; ++k) {
                if (k < W - 1) win[m][k].widen(in); else x[m].widen(in);
#pragma unroll
                for (int j = 0; j < P; ++j) v[j] = fma2(w2[j][k], in[j], v[j]);
            }
#pragma unroll
            for (int j = 0; j < P; ++j) v[j] = activate2(v[j], SILU ? GDN_ACT_SILU : p.act);
            Piece<E, V> r;
            r.round(v);
            r.store(p.y + (b * p.T + t) * p.C + c);
#pragma unroll
            for (int k = 0; k < W - 2; ++k) win[m][k] = win[m][k + 1];
            win[m][W - 2] = x[m];
            if (t + 1 < n[m]) x[m].load(p.x + b * p.sb + (t + 1) * p.st + c);
        }
    }
    if (!p.state_out) return;
#pragma unroll
    for (int m = 0; m < NB; ++m)
#pragma unroll
        for (int k = 0; k < W - 1; ++k)
            if (b0 + m < p.B) win[m][k].store(p.state_out + (static_cast<int64_t>(b0 + m) * (W - 1) + k) * p.C + c);
}

gdn_status check(const gdn_conv_problem *p) {
    if (!p) return GDN_ERR_INVALID_ARG;
    if (p->B <= 0 || p->C <= 0 || p->T < 0 || p->x_stride_b < 0 || p->x_stride_t < 0)
        return GDN_ERR_INVALID_ARG;
    if (p->dtype != GDN_F32 && p->dtype != GDN_BF16) return GDN_ERR_INVALID_ARG;
    if (p->act != GDN_ACT_NONE && p->act != GDN_ACT_SILU && p->act != GDN_ACT_SIGMOID)
        return GDN_ERR_INVALID_ARG;
    if (p->W < 2 || p->W > 4) return GDN_ERR_UNSUPPORTED;
    // 2^30: indexes of a few blocks past the end stay in 32 bits
    if (p->B > 65535 || p->C > (1 << 30) || p->T > (1 << 30) ||
        static_cast<int64_t>(p->C) * p->T > (1 << 30))
        return GDN_ERR_UNSUPPORTED;
    return GDN_OK;
}

template <typename E, int W, int V>
cudaError_t launch(const gdn_conv_problem *pr, ConvParams<E> &p, cudaStream_t s) {
    const int64_t cv = pr->C / V;
    if (pr->T <= kStepTokens) {
        // kStepBatch sequences to a thread where that still leaves each SM two blocks
        const unsigned blocks = static_cast<unsigned>((cv + kThreads - 1) / kThreads);
        const unsigned batches = (pr->B + kStepBatch - 1) / kStepBatch;
        const bool silu = pr->act == GDN_ACT_SILU;
        if (static_cast<int64_t>(blocks) * batches >= 2 * 152) {
            if (silu)
                gdn_conv_step_kernel<E, W, V, kStepBatch, true><<<dim3(blocks, batches), kThreads, 0, s>>>(p);
            else
                gdn_conv_step_kernel<E, W, V, kStepBatch, false><<<dim3(blocks, batches), kThreads, 0, s>>>(p);
        } else if (silu) {
            gdn_conv_step_kernel<E, W, V, 1, true><<<dim3(blocks, pr->B), kThreads, 0, s>>>(p);
        } else {
            gdn_conv_step_kernel<E, W, V, 1, false><<<dim3(blocks, pr->B), kThreads, 0, s>>>(p);
        }
        return cudaGetLastError();
    }
    // Runs of kMaxRun tokens re-read (W - 1) / kMaxRun of x; shorter ones where those would
    // leave SMs without their four blocks.
    const int64_t T = pr->T;
    p.run = kMaxRun;
    while (p.run > 2 * kUnroll && (T + p.run - 1) / p.run * cv * pr->B < 152LL * 4 * kThreads) p.run /= 2;
    const int64_t threads = (T + p.run - 1) / p.run * cv;
    const dim3 grid(static_cast<unsigned>((threads + kThreads - 1) / kThreads), pr->B);
    constexpr size_t ring = V > 1 ? kStages * kUnroll * kThreads * 16 : 0;
    if (pr->act == GDN_ACT_SILU)
        gdn_conv_kernel<E, W, V, true><<<grid, kThreads, ring, s>>>(p);
    else
        gdn_conv_kernel<E, W, V, false><<<grid, kThreads, ring, s>>>(p);
    return cudaGetLastError();
}

template <typename E, int W>
cudaError_t launch_pieces(const gdn_conv_problem *pr, ConvParams<E> &p, cudaStream_t s) {
    constexpr int V = 16 / sizeof(E);
    return pieces16(p.x, pr->B, pr->T, pr->C, p.sb, p.st, sizeof(E)) ? launch<E, W, V>(pr, p, s)
                                                                     : launch<E, W, 1>(pr, p, s);
}

template <typename E>
cudaError_t dispatch(const gdn_conv_problem *pr, const void *x, const float *w, const float *bias,
                     const void *state_in, const int32_t *lengths, void *y, void *state_out,
                     cudaStream_t s) {
    ConvParams<E> p;
    p.x = static_cast<const E *>(x);
    p.w = w;
    p.bias = bias;
    p.state_in = static_cast<const E *>(state_in);
    p.lengths = lengths;
    p.y = static_cast<E *>(y);
    p.state_out = static_cast<E *>(state_out);
    p.sb = pr->x_stride_b;
    p.st = pr->x_stride_t;
    p.B = pr->B;
    p.T = pr->T;
    p.C = pr->C;
    p.act = pr->act;
    switch (pr->W) {
        case 2: return launch_pieces<E, 2>(pr, p, s);
        case 3: return launch_pieces<E, 3>(pr, p, s);
        default: return launch_pieces<E, 4>(pr, p, s);
    }
}

}  // namespace
}  // namespace gdn

extern "C" {

GDN_API gdn_status gdn_conv_fwd(const gdn_conv_problem *p, const void *x, const float *weight,
                                const float *bias, const void *state_in, const int32_t *lengths,
                                void *y, void *state_out, void *stream) {
    using gdn::Span;
    const gdn_status st = gdn::check(p);
    if (st != GDN_OK) return st;
    const bool empty = p->T == 0;
    if (!empty && (!x || !weight || !y)) return GDN_ERR_INVALID_ARG;
    const size_t e = gdn::elem_bytes(p->dtype);
    for (const void *ptr : {static_cast<const void *>(weight), static_cast<const void *>(bias),
                            state_in, static_cast<const void *>(y),
                            static_cast<const void *>(state_out)})
        if (!gdn::is_aligned(ptr, 16)) return GDN_ERR_ALIGNMENT;
    if (!gdn::is_aligned(x, e) || !gdn::is_aligned(lengths, 4)) return GDN_ERR_ALIGNMENT;
    const size_t row = static_cast<size_t>(p->C) * e;
    const Span sx(x, gdn::strided_bytes(p->B, p->T, p->C, p->x_stride_b, p->x_stride_t, e));
    const Span sw(weight, static_cast<size_t>(p->C) * p->W * 4);
    const Span sbias(bias, static_cast<size_t>(p->C) * 4), sl(lengths, static_cast<size_t>(p->B) * 4);
    const Span sy(y, row * p->T * p->B);
    const Span si(state_in, row * (p->W - 1) * p->B), so(state_out, row * (p->W - 1) * p->B);
    if (sy.meets(sx) || sy.meets(sw) || sy.meets(sbias) || sy.meets(sl) || sy.meets(si) ||
        sy.meets(so) || so.meets(sx) || so.meets(sw) || so.meets(sbias) || so.meets(sl) ||
        (state_in != state_out && so.meets(si)))
        return GDN_ERR_INVALID_ARG;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    cudaError_t err = cudaSuccess;
    if (empty) {             // x, weight and y may be NULL
        const size_t bytes = row * (p->W - 1) * p->B;
        if (state_out && state_in && state_in != state_out)
            err = cudaMemcpyAsync(state_out, state_in, bytes, cudaMemcpyDeviceToDevice, s);
        else if (state_out && !state_in)
            err = cudaMemsetAsync(state_out, 0, bytes, s);
        return err == cudaSuccess ? GDN_OK : GDN_ERR_CUDA;
    }
    err = p->dtype == GDN_BF16
              ? gdn::dispatch<__nv_bfloat16>(p, x, weight, bias, state_in, lengths, y, state_out, s)
              : gdn::dispatch<float>(p, x, weight, bias, state_in, lengths, y, state_out, s);
    return err == cudaSuccess ? GDN_OK : GDN_ERR_CUDA;
}

}  // extern "C"
