// Group norm of channels-last rows with an activation or a gate: gdn_group_norm of
// include/gdn.h.
//
// Bound by memory: one read of x (and of the gate) and one write of y. Three kernels:
//   gdn_norm_rows_kernel   T = 1: a group is cg consecutive values, held in the registers of a
//                          part of a warp between the statistics (the mean first, the
//                          variance about it) and the output;
//   gdn_norm_tokens_kernel any T: a cluster of CTAs shares a sequence's tokens for a slice of
//                          whole groups; what shared memory does not keep is read from
//                          L2 the second time;
//   gdn_norm_wide_kernel   groups of more pieces than a block has threads: a cluster to a group
//                          of a sequence, x read twice.
#include "mixer.cuh"
#include "sm100_ptx.cuh"

namespace gdn {
namespace {

using namespace ptx;

constexpr int kThreads = 256;

template <typename E>
struct NormParams {
    const E *x, *gate;
    const float *w, *bias;
    const int32_t *lengths;
    E *y;
    int64_t x_sb, x_st, g_sb, g_st;
    int B, T, C, G, act;
    float eps;
    // rows kernel: lanes to a group, rows in flight; tokens kernel: groups to a slice,
    // CTAs to a cluster
    int lanes, flight, groups, cluster;
};

__device__ __forceinline__ F2 both(float v) { return pack2(v, v); }
__device__ __forceinline__ float halves(F2 v) {
    float a, b;
    unpack2(v, a, b);
    return a + b;
}

// v (scaled and shifted) through the activation or the gate; one branch for all of a piece.
template <int N>
__device__ __forceinline__ void outputs(F2 (&v)[N], const F2 (&gate)[N], bool gated, int act) {
    if (gated) {
        if (act == GDN_ACT_SILU) {
#pragma unroll
            for (int i = 0; i < N; ++i) v[i] = mul2(v[i], mul2(gate[i], sigmoid2(gate[i])));
        } else if (act == GDN_ACT_SIGMOID) {
#pragma unroll
            for (int i = 0; i < N; ++i) v[i] = mul2(v[i], sigmoid2(gate[i]));
        } else {
#pragma unroll
            for (int i = 0; i < N; ++i) v[i] = mul2(v[i], gate[i]);
        }
    } else if (act == GDN_ACT_SILU) {
#pragma unroll
        for (int i = 0; i < N; ++i) v[i] = mul2(v[i], sigmoid2(v[i]));
    } else if (act == GDN_ACT_SIGMOID) {
#pragma unroll
        for (int i = 0; i < N; ++i) v[i] = sigmoid2(v[i]);
    }
}

// Parameters of channels c.., `other` without any.
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

// ------------------------------------------------------------------ single rows
//
// `lanes` lanes (a power of two) hold a group, P pieces of V channels to a lane, R rows at a
// time, so their sums' shuffles overlap. A thread keeps its channels from row to row: with
// few pieces weight and bias stay in registers.
template <typename E, int V, int P, int R>
__global__ void __launch_bounds__(kThreads) gdn_norm_rows_kernel(NormParams<E> p) {
    const int L = p.lanes, cg = p.C / p.G, slots = p.G * L;
    const int i = blockIdx.x * kThreads + threadIdx.x;
    const int j = i % L;                               // slots and 32 are multiples of L
    const int g = i % slots / L;
    int row = i < slots * p.flight ? i / slots : p.B;
    const float inv = 1.f / cg;
    constexpr bool KEEP = P <= 2;                      // weight and bias in registers
    constexpr int PK = KEEP ? P : 1, N = (V + 1) / 2;
    F2 w[PK][N], bias[PK][N];
    bool in[P];
    int c[P];
#pragma unroll
    for (int q = 0; q < P; ++q) {
        const int at = (q * L + j) * V;
        in[q] = at < cg;
        c[q] = g * cg + (in[q] ? at : 0);
        if constexpr (KEEP) {
            params<V>(p.w, c[q], 1.f, w[q]);
            params<V>(p.bias, c[q], 0.f, bias[q]);
        }
    }
    // sums over the group's lanes, of R rows at once
    auto group_sums = [&](float (&s)[R]) {
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) {
            if (o >= L) continue;                      // alike for all threads
#pragma unroll
            for (int r = 0; r < R; ++r) s[r] += __shfl_xor_sync(0xffffffffu, s[r], o);
        }
    };
    // every thread takes the same number of turns: the shuffles need whole warps
    for (int done = 0; done < p.B; done += R * p.flight, row += R * p.flight) {
        Piece<E, V> x[R][P], gate[R][P];
        bool live[R];
#pragma unroll
        for (int r = 0; r < R; ++r) {
            const int64_t b = row + static_cast<int64_t>(r) * p.flight;
            live[r] = b < p.B && (!p.lengths || p.lengths[b] > 0);
#pragma unroll
            for (int q = 0; q < P; ++q) {
                x[r][q].zero();
                gate[r][q].zero();
                if (live[r] && in[q]) {
                    x[r][q].load_rw(p.x + b * p.x_sb + c[q]);
                    if (p.gate) gate[r][q].load(p.gate + b * p.g_sb + c[q]);
                }
            }
        }
        float mean[R], s[R];
#pragma unroll
        for (int r = 0; r < R; ++r) {
            F2 sum = 0;
#pragma unroll
            for (int q = 0; q < P; ++q) {
                F2 v[N];
                x[r][q].widen(v);
#pragma unroll
                for (int k = 0; k < N; ++k) sum = add2(sum, v[k]);
            }
            mean[r] = V == 1 ? 0.5f * halves(sum) : halves(sum);
        }
        group_sums(mean);
#pragma unroll
        for (int r = 0; r < R; ++r) {
            mean[r] *= inv;
            F2 sum = 0;
#pragma unroll
            for (int q = 0; q < P; ++q) {
                if (P > 1 && !in[q]) continue;
                F2 v[N];
                x[r][q].widen(v);
#pragma unroll
                for (int k = 0; k < N; ++k) {
                    v[k] = add2(v[k], both(-mean[r]));
                    sum = fma2(v[k], v[k], sum);
                }
            }
            s[r] = V == 1 ? 0.5f * halves(sum) : halves(sum);
            if (P == 1 && !in[0]) s[r] = 0.f;
        }
        group_sums(s);
#pragma unroll
        for (int r = 0; r < R; ++r) {
            const F2 rstd = both(rsqrtf(fmaf(s[r], inv, p.eps)));
#pragma unroll
            for (int q = 0; q < P; ++q) {
                if (!live[r] || !in[q]) continue;
                F2 v[N], z[N];
                if constexpr (!KEEP) {
                    params<V>(p.w, c[q], 1.f, w[0]);
                    params<V>(p.bias, c[q], 0.f, bias[0]);
                }
                x[r][q].widen(v);
                gate[r][q].widen(z);
#pragma unroll
                for (int k = 0; k < N; ++k)
                    v[k] = fma2(add2(v[k], both(-mean[r])), mul2(w[KEEP ? q : 0][k], rstd),
                                bias[KEEP ? q : 0][k]);
                outputs(v, z, p.gate != nullptr, p.act);
                x[r][q].round(v);
                x[r][q].store(p.y + (row + static_cast<int64_t>(r) * p.flight) * p.C + c[q]);
            }
        }
    }
}

// ----------------------------------------------------------------- whole sequences
//
// The CTAs of a cluster take equal shares of a sequence's valid tokens, for one slice of
// `groups` groups. A thread keeps one piece of V channels and takes every RP-th
// token. It sums x - k and (x - k)^2, k the channel's mean over its first 4 tokens, over up
// to 32 blocks of 4, and merges these sets by the exact update for two,
//   mean += d nb / n,   M2 += M2b + d^2 na nb / n   with d = mean_b - mean.
// The mean of a set lies at most sqrt(32) of its deviations from k, so at most 33 times the
// variance's rounding is lost, however far the mean is from zero. Channels and threads then
// merge to groups, and the CTAs' groups through distributed shared memory, in rank order.
// Means are added up as differences from one of those that are merged (from a set's k, a
// group's first channel, the first rank), so a mean is rounded at its own size three times
// however many are merged; summed as they were, means of 1e4 to 1e6 deviations were up to 41
// roundings off (20000 tokens of 4 channels). What is scaled by a reciprocal here is such a
// difference or a square, so 1 ulp of rcp_ftz does; divisions took 7.0 us for 6.7 (B3 T1001 C330
// fp32 in a graph).
constexpr int kBlockTokens = 4;
constexpr int kSetBlocks = 32;
// Of a thread's blocks the first kKept stay in shared memory between the statistics and the
// output; the others pass through kRing places there, twice.
constexpr int kKept = 3;
constexpr int kRing = 2;
// Clusters of 16 need the kernels' leave and leave SMs empty: for few and long sequences only (two
// of 16384 tokens and 64 channels 43 -> 23 us; four of 4096 and 1280 would take 49 us for 33).
constexpr int kMaxCluster = 16;

__device__ __forceinline__ float ld_cluster_f32(uint32_t addr) {
    float v;
    asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(addr) : "memory");
    return v;
}

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}

__device__ __forceinline__ void cluster_arrive() {
    asm volatile("barrier.cluster.arrive.release;" ::: "memory");
}
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.acquire;" ::: "memory"); }

// From each CTA's mean and squares of the groups: their mean and 1 / deviation over all K CTAs, a
// lane to a CTA, which has `share` of the n tokens while they last. Ends with an arrival at the
// cluster's barrier: a CTA waits there before it leaves, since others may still read its part.
__device__ __forceinline__ void merge_cluster(float (&part)[2][kThreads], int groups, int K, int n, int share,
                                              int cg, float eps, float *mean, float *rstd) {
    const int lane = threadIdx.x % 32;
    const float share_of_one = rcp_ftz(static_cast<float>(n) * cg);
    const float count = lane < K ? static_cast<float>(min(n, (lane + 1) * share) - min(n, lane * share)) * cg : 0.f;
    auto over_ranks = [&](float v) {       // K is a power of two: lanes 0.. K - 1 have the sum
        for (int o = K / 2; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
        return v;
    };
    __syncthreads();
    if (K > 1) cluster_sync();
    for (int g = threadIdx.x / 32; g < groups; g += kThreads / 32) {
        float m = 0.f, s = 0.f;
        if (lane < K) {
            auto of_rank = [&](float *f) {
                return K > 1 ? ld_cluster_f32(mapa_shared(smem_u32(f), lane)) : *f;
            };
            m = of_rank(&part[0][g]);
            s = of_rank(&part[1][g]);
        }
        const float first = __shfl_sync(0xffffffffu, m, 0);     // rank 0 has tokens
        m -= first;
        const float all = over_ranks(count * m) * share_of_one, d = m - all;
        s = over_ranks(fmaf(count * d, d, s));
        if (lane == 0) {
            mean[g] = first + all;
            rstd[g] = rsqrtf(fmaf(s, share_of_one, eps));
        }
    }
    __syncthreads();
    if (K > 1) cluster_arrive();
}

template <typename E, int V, bool GATED>
__global__ void __launch_bounds__(kThreads, V > 1 ? 2 : 4) gdn_norm_tokens_kernel(NormParams<E> p) {
    __shared__ float means[kThreads * V], squares[kThreads * V];   // [token row][channel of the slice]
    __shared__ float columns[kThreads * V];                        // sums over token rows
    __shared__ float part[2][kThreads];                            // mean, squares of a group
    __shared__ float g_mean[kThreads], g_rstd[kThreads];
    const int cg = p.C / p.G, K = p.cluster, rank = blockIdx.x % K;
    const int g0 = blockIdx.y * p.groups, ng = min(p.groups, p.G - g0);
    const int64_t b = blockIdx.x / K;
    const int n = valid_tokens(p.lengths, b, p.T);
    if (n == 0) return;                                            // the whole cluster
    const int SC = ng * cg, PR = SC / V, RP = kThreads / PR;
    const int row = threadIdx.x / PR, q = threadIdx.x % PR * V, c = g0 * cg + q;
    const int share = (n + K - 1) / K, t_begin = min(n, rank * share), t_end = min(n, t_begin + share);
    const bool mine = row < RP;
    const E *x = p.x + b * p.x_sb + c;

    constexpr int N = (V + 1) / 2;
    constexpr int BT = kBlockTokens;
    using Raw = typename Piece<E, V>::Raw;
    extern __shared__ __align__(16) unsigned char dynamic[];
    Raw *const slots = reinterpret_cast<Raw *>(dynamic) + threadIdx.x;     // this thread's alone
    const int64_t step = RP * p.x_st;
    const E *const first = x + (t_begin + row) * p.x_st;
    const int own = mine ? max(0, (t_end - t_begin - row + RP - 1) / RP) : 0;    // tokens of this thread
    const int blocks = (own + BT - 1) / BT;
    auto place = [](int block) { return (block < kKept ? block : kKept + (block - kKept) % kRing) * BT; };
    // A block's pieces on their way to its place; one group of copies whether or not it exists.
    auto fetch = [&](int block) {
        if (block < blocks) {
            Raw *to = slots + place(block) * kThreads;
            const E *from = first + static_cast<int64_t>(block) * BT * step;
#pragma unroll
            for (int u = 0; u < BT; ++u) {
                if (block * BT + u < own) {
                    if constexpr (sizeof(Raw) == 16)
                        copy16_async(to + u * kThreads, from + u * step);
                    else if constexpr (sizeof(Raw) == 4)
                        copy4_async(to + u * kThreads, from + u * step);
                    else
                        to[u * kThreads] = from[u * step];
                }
            }
        }
        copy_commit();
    };
    auto block_piece = [&](int block, int u) {
        Piece<E, V> q;
        q.raw = slots[(place(block) + u) * kThreads];
        return q;
    };
    for (int i = 0; i < kKept + kRing; ++i) fetch(i);
    if (mine) {
        // the mean of the sets so far, less the current set's k (shift is -k)
        F2 mean[N], m2[N], shift[N];
#pragma unroll
        for (int k = 0; k < N; ++k) mean[k] = m2[k] = shift[k] = 0;
        float count = 0.f;
        for (int set = 0; set < blocks; set += kSetBlocks) {
            F2 s1[N], s2[N];
#pragma unroll
            for (int k = 0; k < N; ++k) s1[k] = s2[k] = 0;
            const int end = min(blocks, set + kSetBlocks);
            for (int i = set; i < end; ++i) {
                if (i < kKept + kRing)
                    copy_wait<kKept + kRing - 1>();
                else
                    copy_wait<kRing - 1>();
                const int here = min(BT, own - i * BT);
                F2 v[BT][N], b1[N], b2[N];
#pragma unroll
                for (int u = 0; u < BT; ++u) {
                    Piece<E, V> q = block_piece(i, u);
                    q.widen(v[u]);
                }
                if (i >= kKept) fetch(i + kRing); else copy_commit();
#pragma unroll
                for (int k = 0; k < N; ++k) {
                    if (i == set) {
                        F2 sum = v[0][k];
#pragma unroll
                        for (int u = 1; u < BT; ++u)
                            if (u < here) sum = add2(sum, v[u][k]);
                        sum = mul2(sum, both(-rcp_ftz(here)));
                        mean[k] = add2(mean[k], fma2(shift[k], both(-1.f), sum));
                        shift[k] = sum;
                    }
                    b1[k] = b2[k] = 0;
                }
#pragma unroll
                for (int u = 0; u < BT; ++u) {
                    if (u >= here) break;
#pragma unroll
                    for (int k = 0; k < N; ++k) {
                        const F2 d = add2(v[u][k], shift[k]);
                        b1[k] = add2(b1[k], d);
                        b2[k] = fma2(d, d, b2[k]);
                    }
                }
#pragma unroll
                for (int k = 0; k < N; ++k) {
                    s1[k] = add2(s1[k], b1[k]);
                    s2[k] = add2(s2[k], b2[k]);
                }
            }
            if (set == 0) {      // no sets before (a branch where k is taken: 12.2 us for 11.3, B3 T2048 C330 bf16)
#pragma unroll
                for (int k = 0; k < N; ++k) mean[k] = 0;
            }
            const float nb = static_cast<float>(min(own - set * BT, kSetBlocks * BT)), na = count;
            count += nb;
            const float f = nb * rcp_ftz(count), by_nb = rcp_ftz(nb);
#pragma unroll
            for (int k = 0; k < N; ++k) {
                const F2 off = mul2(s1[k], both(by_nb));                // the set's mean - its k
                const F2 set2 = fma2(mul2(off, s1[k]), both(-1.f), s2[k]);
                const F2 d = fma2(mean[k], both(-1.f), off);
                mean[k] = fma2(d, both(f), mean[k]);
                m2[k] = add2(m2[k], fma2(mul2(d, d), both(na * f), set2));
            }
        }
        // the second reading begins during the merges
        copy_wait<0>();
        for (int i = kKept; i < kKept + kRing; ++i) fetch(i);
#pragma unroll
        for (int k = 0; k < N; ++k) {
            float a, b;
            float *to = means + row * SC + q + 2 * k, *to2 = squares + row * SC + q + 2 * k;
            unpack2(fma2(shift[k], both(-1.f), mean[k]), a, b);
            to[0] = a;
            if (V > 1) to[1] = b;
            unpack2(m2[k], a, b);
            to2[0] = a;
            if (V > 1) to2[1] = b;
        }
    }
    __syncthreads();
    // Merge the token rows, then the channels, to groups: the weighted means first, then the
    // squares about the group's mean. Threads take the channels, warps the groups; a channel's
    // rows shared out over idle threads cost 23 us for 19 (B3 T2048 C330 bf16).
    const int tokens = t_end - t_begin, more = tokens % RP;
    const float share_of_one = tokens > 0 ? rcp_ftz(static_cast<float>(tokens) * cg) : 0.f;
    const float low = static_cast<float>(tokens / RP), high = low + 1.f;
    // col / cg: with both at most 2048 the product is off by less than 2048 2^-22 / cg, and the
    // quotient no nearer than 1 / (2 cg) to a whole number.
    const float by_cg = rcp_ftz(cg);
    auto group_of = [&](int col) { return static_cast<int>((col + 0.5f) * by_cg); };
    auto over_channels = [&](auto keep) {
        __syncthreads();
        for (int g = threadIdx.x / 32; g < ng; g += kThreads / 32) {
            float sum = 0.f;
#pragma unroll 4
            for (int i = threadIdx.x % 32; i < cg; i += 32) sum += columns[g * cg + i];
            sum = warp_sum(sum);
            if (threadIdx.x % 32 == 0) keep(g, sum);
        }
        __syncthreads();
    };
    for (int col = threadIdx.x; col < SC; col += kThreads) {
        const float first = means[group_of(col) * cg];
        float sum = 0.f;
#pragma unroll 8
        for (int r = 0; r < RP; ++r) sum = fmaf(r < more ? high : low, means[r * SC + col] - first, sum);
        columns[col] = sum;
    }
    over_channels([&](int g, float sum) {
        part[0][g] = fmaf(sum, share_of_one, means[g * cg]);
    });
    for (int col = threadIdx.x; col < SC; col += kThreads) {
        const float m = part[0][group_of(col)];
        float sum = 0.f;
#pragma unroll 8
        for (int r = 0; r < RP; ++r) {
            const float d = means[r * SC + col] - m;
            sum += fmaf((r < more ? high : low) * d, d, squares[r * SC + col]);
        }
        columns[col] = sum;
    }
    over_channels([&](int g, float sum) { part[1][g] = sum; });
    merge_cluster(part, ng, K, n, share, cg, p.eps, g_mean, g_rstd);
    if (mine) {
        F2 w[N], bias[N], mean[N];
        params<V>(p.w, c, 1.f, w);
        params<V>(p.bias, c, 0.f, bias);
#pragma unroll
        for (int k = 0; k < N; ++k) {
            const int ga = (q + 2 * k) / cg, gb = V == 1 ? ga : (q + 2 * k + 1) / cg;
            mean[k] = pack2(-g_mean[ga], -g_mean[gb]);
            w[k] = mul2(w[k], pack2(g_rstd[ga], g_rstd[gb]));
        }
        const int64_t g_step = RP * p.g_st, y_step = static_cast<int64_t>(RP) * p.C;
        const E *gate = GATED ? p.gate + b * p.g_sb + c + (t_begin + row) * p.g_st : nullptr;
        E *y = p.y + (b * p.T + t_begin + row) * p.C + c;
        // kept blocks between those that still arrive
        const int kept = min(blocks, kKept), other = blocks - kept, mixed = 2 * min(kept, other);
        auto order = [&](int i) {
            if (i < mixed) return i & 1 ? i / 2 : kKept + i / 2;
            return other > kept ? kKept + i - kept : i - other;
        };
        Piece<E, V> z[BT];
        auto fetch_gate = [&](int block) {
#pragma unroll
            for (int u = 0; u < BT; ++u)
                if (block * BT + u < own) z[u].load(gate + (static_cast<int64_t>(block) * BT + u) * g_step);
        };
#pragma unroll
        for (int u = 0; u < BT; ++u) z[u].zero();
        if (GATED && blocks > 0) fetch_gate(order(0));
        for (int i = 0; i < blocks; ++i) {
            const int block = order(i);
            if (block >= kKept) copy_wait<kRing - 1>();
            Piece<E, V> r[BT], zn[BT];
#pragma unroll
            for (int u = 0; u < BT; ++u) {
                r[u] = block_piece(block, u);
                zn[u] = z[u];
            }
            if (block >= kKept) fetch(block + kRing);
            if (GATED && i + 1 < blocks) fetch_gate(order(i + 1));
            E *to = y + static_cast<int64_t>(block) * BT * y_step;
#pragma unroll
            for (int u = 0; u < BT; ++u) {
                if (block * BT + u >= own) break;
                F2 v[N], gv[N];
                r[u].widen(v);
                if constexpr (GATED) zn[u].widen(gv);
#pragma unroll
                for (int k = 0; k < N; ++k) v[k] = fma2(add2(v[k], mean[k]), w[k], bias[k]);
                outputs(v, gv, GATED, p.act);
                r[u].round(v);
                r[u].store(to + u * y_step);
            }
        }
        copy_wait<0>();
    }
    if (K > 1) cluster_wait();
}

// The same for a group of more pieces than a block has threads: a cluster to a group, each
// thread taking every kThreads-th piece of a token and merging all its values. 65536 rows of 4096
// channels in bf16 take 369 us (2.9 TB/s): issue 76%, a block's merge for two pieces a thread.
// One sequence of 16384 tokens takes 4116 us, on the 8 SMs of its one cluster.
template <typename E, int V>
__global__ void __launch_bounds__(kThreads) gdn_norm_wide_kernel(NormParams<E> p) {
    __shared__ float part[2][kThreads], counts[kThreads];
    __shared__ float g_mean[1], g_rstd[1];
    const int cg = p.C / p.G, K = p.cluster, rank = blockIdx.x % K, c0 = blockIdx.y * cg;
    const int64_t b = blockIdx.x / K;
    const int n = valid_tokens(p.lengths, b, p.T);
    if (n == 0) return;                                            // the whole cluster
    const int share = (n + K - 1) / K, t_begin = min(n, rank * share), t_end = min(n, t_begin + share);
    const E *x = p.x + b * p.x_sb + c0;
    // Blocks of up to four pieces of a token, loaded together, in sets of 1, 1, 2, 4, .. 64 pieces or
    // a block more. The first set's sums are taken about its first piece's mean (at most sqrt(3) of
    // its deviations from the set's), the others' about the mean of all before them; merged as in
    // the tokens kernel (mean is less the first of these points). A set whose mean lies D from
    // its point adds its own squares and at least D^2 / 2 a value to the total, since it is no
    // larger than what lies before: at most 4 times the variance's rounding is lost. (Sets of 64
    // about their first value: up to 64 V times where that is an outlier, and one load at a time:
    // 65536 rows of 4096 in bf16 420 us for 394, 16384 tokens of 4096 4921 for 4179.)
    float count = 0.f, first = 0.f, mean = 0.f, m2 = 0.f, shift = 0.f, s1 = 0.f, s2 = 0.f;
    int set = 0, most = 1;
    auto merge = [&] {
        const float nb = static_cast<float>(set) * V, na = count;
        if (set == 0) return;
        count += nb;
        if (na == 0.f) first = shift; else most = min(2 * most, 64);
        const float off = s1 / nb, d = shift - first + off - mean, w = nb / count;
        mean = fmaf(d, w, mean);
        m2 += fmaf(d * d, na * w, fmaf(-off, s1, s2));
        set = 0;
    };
    constexpr int U = 4, TURN = kThreads * V;
    for (int64_t t = t_begin; t < t_end; ++t) {
        for (int q = threadIdx.x * V; q < cg; q += U * TURN) {
            Piece<E, V> r[U];
#pragma unroll
            for (int u = 0; u < U; ++u) {
                r[u].zero();
                if (q + u * TURN < cg) r[u].load_rw(x + t * p.x_st + q + u * TURN);
            }
            if (set >= most) merge();
            if (set == 0) {
                shift = first + mean;
                if (count == 0.f) {
                    float f[V];
                    r[0].widen(f);
                    shift = f[0];
#pragma unroll
                    for (int k = 1; k < V; ++k) shift += f[k];
                    shift *= 1.f / V;
                }
                s1 = s2 = 0.f;
            }
#pragma unroll
            for (int u = 0; u < U; ++u) {
                if (q + u * TURN >= cg) break;
                float f[V], p1 = 0.f, p2 = 0.f;      // of the piece
                r[u].widen(f);
#pragma unroll
                for (int k = 0; k < V; ++k) {
                    const float d = f[k] - shift;
                    p1 += d;
                    p2 = fmaf(d, d, p2);
                }
                ++set;
                s1 += p1;
                s2 += p2;
            }
        }
    }
    merge();
    counts[threadIdx.x] = count;
    part[0][threadIdx.x] = first + mean;
    part[1][threadIdx.x] = m2;
    __syncthreads();
    if (threadIdx.x < 32) {
        constexpr int M = kThreads / 32;
        float n_of[M], m_of[M], s_of[M], na = 0.f, m = 0.f, s = 0.f;
        first = part[0][0];                                       // thread 0 has a piece of every token
#pragma unroll
        for (int i = 0; i < M; ++i) {
            n_of[i] = counts[i * 32 + threadIdx.x];
            m_of[i] = part[0][i * 32 + threadIdx.x] - first;
            s_of[i] = part[1][i * 32 + threadIdx.x];
        }
#pragma unroll
        for (int i = 0; i < M; ++i) {
            na += n_of[i];
            m = fmaf(n_of[i], m_of[i], m);
        }
        na = warp_sum(na);
        m = na > 0.f ? warp_sum(m) / na : 0.f;
#pragma unroll
        for (int i = 0; i < M; ++i) {
            const float d = m_of[i] - m;
            s += fmaf(n_of[i] * d, d, s_of[i]);
        }
        m += first;
        s = warp_sum(s);
        __syncwarp();
        if (threadIdx.x == 0) {
            part[0][0] = m;
            part[1][0] = s;
        }
    }
    merge_cluster(part, 1, K, n, share, cg, p.eps, g_mean, g_rstd);
    const E *gate = p.gate ? p.gate + b * p.g_sb + c0 : nullptr;
    E *y = p.y + b * p.T * p.C + c0;
    for (int64_t t = t_begin; t < t_end; ++t) {
        for (int q = threadIdx.x * V; q < cg; q += kThreads * V) {
            constexpr int N = (V + 1) / 2;
            Piece<E, V> r, z;
            F2 v[N], gv[N], w[N], bias[N];
            r.load_rw(x + t * p.x_st + q);
            z.zero();
            if (gate) z.load(gate + t * p.g_st + q);
            params<V>(p.w, c0 + q, 1.f, w);
            params<V>(p.bias, c0 + q, 0.f, bias);
            r.widen(v);
            z.widen(gv);
#pragma unroll
            for (int k = 0; k < N; ++k)
                v[k] = fma2(add2(v[k], both(-g_mean[0])), mul2(w[k], both(g_rstd[0])), bias[k]);
            outputs(v, gv, gate != nullptr, p.act);
            r.round(v);
            r.store(y + t * p.C + q);
        }
    }
    if (K > 1) cluster_wait();
}

gdn_status check(const gdn_group_norm_problem *p) {
    if (!p) return GDN_ERR_INVALID_ARG;
    if (p->B <= 0 || p->C <= 0 || p->G <= 0 || p->T < 0 || p->C % p->G != 0) return GDN_ERR_INVALID_ARG;
    if (p->x_stride_b < 0 || p->x_stride_t < 0 || p->gate_stride_b < 0 || p->gate_stride_t < 0 ||
        p->reserved || !(p->eps >= 0.f))
        return GDN_ERR_INVALID_ARG;
    if (p->dtype != GDN_F32 && p->dtype != GDN_BF16) return GDN_ERR_INVALID_ARG;
    if (p->act != GDN_ACT_NONE && p->act != GDN_ACT_SILU && p->act != GDN_ACT_SIGMOID)
        return GDN_ERR_INVALID_ARG;
    // 2^30: indexes of a block past the end stay in 32 bits
    if (p->B > (1 << 26) || p->G > 65535 || p->C > (1 << 30) || p->T > (1 << 30)) return GDN_ERR_UNSUPPORTED;
    return GDN_OK;
}

template <typename E, int V, int P>
cudaError_t launch_rows(NormParams<E> &p, cudaStream_t s) {
    // two rows at a time: 254 us for 65536 gated rows of 4096 (6.3 TB/s); one 304, four 293
    constexpr int R = P <= 2 ? 2 : 1;
    const int64_t slots = static_cast<int64_t>(p.G) * p.lanes;
    // rows in flight: 8 blocks to an SM, or all rows
    const int64_t most = 152LL * 8 * kThreads / slots;
    const int64_t flight = most < 1 ? 1 : most < p.B ? most : p.B;
    p.flight = static_cast<int>(flight);
    const int64_t blocks = (slots * flight + kThreads - 1) / kThreads;
    gdn_norm_rows_kernel<E, V, P, R><<<static_cast<unsigned>(blocks), kThreads, 0, s>>>(p);
    return cudaGetLastError();
}

template <typename E>
cudaError_t launch_cluster(void (*kernel)(NormParams<E>), int K, int slices, int bytes,
                           NormParams<E> &p, cudaStream_t s) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(K) * p.B, slices);
    p.cluster = K;
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = bytes;
    const void *f = reinterpret_cast<const void *>(kernel);
    cudaError_t e = cudaFuncSetAttribute(f, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
    if (e == cudaSuccess && K > 8) e = cudaFuncSetAttribute(f, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
    if (e != cudaSuccess) return e;
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = K;
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = K > 1 ? 1 : 0;
    e = cudaLaunchKernelEx(&cfg, kernel, p);
    if (e != cudaSuccess && K > 8) {       // no place for 16 (a part of a GPU, say)
        cudaGetLastError();
        return launch_cluster(kernel, 8, slices, bytes, p, s);
    }
    return e;
}

template <typename E, int V>
cudaError_t launch_tokens(NormParams<E> &p, cudaStream_t s) {
    const int cg = p.C / p.G;
    // Slices start at whole pieces.
    int unit = 1;
    while (unit * cg % V != 0) ++unit;
    if (unit <= p.G && unit * static_cast<int64_t>(cg) / V > kThreads) {
        if (cg % V != 0) return launch_tokens<E, 1>(p, s);
        int K = 1;
        while (K < 8 && static_cast<int64_t>(p.B) * p.G * K < 4 * 152 && p.T > 2 * K) K *= 2;
        return launch_cluster(gdn_norm_wide_kernel<E, V>, K, p.G, 0, p, s);
    }
    // Slice and cluster by the turns that a thread takes: its tokens, and about 8 for the
    // merges, for every wave of blocks (2 or 4 to an SM by registers), and the sectors that
    // the ends of a row's slice waste.
    auto slices = [&](int groups) { return (p.G + groups - 1) / groups; };
    constexpr int64_t wave = 152 * (V > 1 ? 2 : 4);
    int groups = unit, K = 1;
    float best = 0.f;
    for (int n = unit; n == unit || (n / 2 < p.G && n * cg / V <= kThreads && n <= kThreads); n *= 2) {
        const int m = n < p.G ? n : p.G, rows = kThreads / (m * cg / V);
        for (int k = 1; k <= kMaxCluster; k *= 2) {
            const int64_t blocks = static_cast<int64_t>(p.B) * slices(m) * k;
            if (k > 8 && blocks > 152) break;      // 16 find places only on an empty GPU
            const int share = (p.T + k - 1) / k;
            const float turns = static_cast<float>((share + rows - 1) / rows + 8) *
                                (1.f + 16.f / (m * cg * sizeof(E)));
            const float cost = turns * ((blocks + wave - 1) / wave);
            if (best == 0.f || cost < best) {
                best = cost;
                groups = m;
                K = k;
            }
        }
    }
    p.groups = groups;
    constexpr int bytes = (kKept + kRing) * kBlockTokens * kThreads * sizeof(typename Piece<E, V>::Raw);
    return launch_cluster(p.gate ? gdn_norm_tokens_kernel<E, V, true> : gdn_norm_tokens_kernel<E, V, false>, K,
                          slices(groups), bytes, p, s);
}

template <typename E, int V>
cudaError_t launch_pieces(NormParams<E> &p, cudaStream_t s) {
    const int cg = p.C / p.G;
    if (V > 1 && p.T == 1 && cg % V != 0) return launch_pieces<E, 1>(p, s);
    if (p.T == 1) {
        const int pieces = cg / V;
        p.lanes = 1;
        while (p.lanes < 32 && p.lanes < pieces) p.lanes *= 2;
        const int per = (pieces + p.lanes - 1) / p.lanes;
        if (per <= 1) return launch_rows<E, V, 1>(p, s);
        if (per <= 2) return launch_rows<E, V, 2>(p, s);
        if (per <= 4) return launch_rows<E, V, 4>(p, s);
        if (per <= 8) return launch_rows<E, V, 8>(p, s);
        if (V <= 4 && per <= 16) return launch_rows<E, V, V <= 4 ? 16 : 8>(p, s);
    }
    return launch_tokens<E, V>(p, s);
}

template <typename E>
cudaError_t launch(const gdn_group_norm_problem *pr, const void *x, const float *w,
                   const float *bias, const void *gate, const int32_t *lengths, void *y,
                   cudaStream_t s) {
    NormParams<E> p;
    p.x = static_cast<const E *>(x);
    p.gate = static_cast<const E *>(gate);
    p.w = w;
    p.bias = bias;
    p.lengths = lengths;
    p.y = static_cast<E *>(y);
    p.x_sb = pr->x_stride_b;
    p.x_st = pr->x_stride_t;
    p.g_sb = pr->gate_stride_b;
    p.g_st = pr->gate_stride_t;
    p.B = pr->B;
    p.T = pr->T;
    p.C = pr->C;
    p.G = pr->G;
    p.act = pr->act;
    p.eps = pr->eps;
    p.lanes = p.flight = p.groups = p.cluster = 1;
    constexpr int V = 16 / sizeof(E);
    const bool pieces = pieces16(x, p.B, p.T, p.C, p.x_sb, p.x_st, sizeof(E)) &&
                        (!gate || pieces16(gate, p.B, p.T, p.C, p.g_sb, p.g_st, sizeof(E)));
    return pieces ? launch_pieces<E, V>(p, s) : launch_pieces<E, 1>(p, s);
}

}  // namespace
}  // namespace gdn

extern "C" {

GDN_API gdn_status gdn_group_norm(const gdn_group_norm_problem *p, const void *x,
                                  const float *weight, const float *bias, const void *gate,
                                  const int32_t *lengths, void *y, void *stream) {
    using gdn::Span;
    using gdn::strided_bytes;
    const gdn_status st = gdn::check(p);
    if (st != GDN_OK) return st;
    if (p->T == 0) return GDN_OK;
    if (!x || !y) return GDN_ERR_INVALID_ARG;
    const size_t e = gdn::elem_bytes(p->dtype);
    for (const void *ptr : {static_cast<const void *>(weight), static_cast<const void *>(bias),
                            static_cast<const void *>(y)})
        if (!gdn::is_aligned(ptr, 16)) return GDN_ERR_ALIGNMENT;
    if (!gdn::is_aligned(x, e) || !gdn::is_aligned(gate, e) || !gdn::is_aligned(lengths, 4))
        return GDN_ERR_ALIGNMENT;
    const bool in_place = x == y && (p->T == 1 || p->x_stride_t == p->C) &&
                          (p->B == 1 || p->x_stride_b == static_cast<int64_t>(p->T) * p->C);
    const Span sy(y, static_cast<size_t>(p->B) * p->T * p->C * e);
    const Span sx(x, strided_bytes(p->B, p->T, p->C, p->x_stride_b, p->x_stride_t, e));
    const Span sg(gate, strided_bytes(p->B, p->T, p->C, p->gate_stride_b, p->gate_stride_t, e));
    const size_t row = static_cast<size_t>(p->C) * 4;
    if ((sy.meets(sx) && !in_place) || sy.meets(sg) || sy.meets(Span(weight, row)) ||
        sy.meets(Span(bias, row)) || sy.meets(Span(lengths, static_cast<size_t>(p->B) * 4)))
        return GDN_ERR_INVALID_ARG;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    const cudaError_t err =
        p->dtype == GDN_BF16
            ? gdn::launch<__nv_bfloat16>(p, x, weight, bias, gate, lengths, y, s)
            : gdn::launch<float>(p, x, weight, bias, gate, lengths, y, s);
    return err == cudaSuccess ? GDN_OK : GDN_ERR_CUDA;
}

}  // extern "C"
