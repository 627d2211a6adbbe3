// Selective state space scan: gdn_scan_fwd of include/gdn.h.
//
// Two kernels by length: gdn_scan_step_kernel for a few tokens (bound by the state's
// traffic) and gdn_scan_kernel for prompts (bound by arithmetic: N exponentials and 5 N
// multiply-adds per token and channel against 4 values moved).
#include <algorithm>

#include "mixer.cuh"
#include "sm100_ptx.cuh"

namespace gdn {
namespace {

constexpr int kThreads = 128;
constexpr int kStepTokens = 8;      // up to here the step kernel

template <typename E>
struct ScanParams {
    const E *x, *dt, *z, *Bm, *Cm;
    const float *A, *skip, *dt_bias, *h0;
    const int32_t *lengths;
    E *y;
    float *h_final;
    int64_t x_sb, x_st, dt_sb, dt_st, z_sb, z_st, b_sb, b_st, c_sb, c_st;
    int B, T, D, N, G, softplus;
    int turns;           // few tokens: sets of sequences to a block
    int rows16;          // B and C rows are whole 16-byte pieces
    int pieces;          // so are those of x, dt, z and y, and each block's part of them
    // Segments of seg tokens each; with more than one, the state at the end of a
    // segment that started from zero (the first one: from h0), h0 itself behind those,
    // and each segment's sum of Delta.
    int segs, seg;
    float *seg_h, *seg_dt;      // [B][segs][D][N], [B][segs][D]
};

// log(1 + exp(v)) = max(v, 0) + log1p(e), e = exp(-|v|) in (0, 1]. log1p(e) = e P(e) with P the
// polynomial of degree 9 through log1p(e) / e at the ten Chebyshev points of [0, 1]: off by at
// most 5.4e-9 of it, 1.5e-8 with its coefficients in fp32, 1.4e-7 with its steps in fp32 too, so
// small Delta keep their relative accuracy. (2 atanh(e / (2 + e)) by its series, with a reciprocal: 2% more
// for the whole scan.)
__device__ __forceinline__ float softplus(float v) {
    const float e = exp2_ftz(-kLog2e * fabsf(v));
    float r = fmaf(-0.0031760570127516985f, e, 0.019542526453733444f);
    r = fmaf(r, e, -0.056373611092567444f);
    r = fmaf(r, e, 0.10543623566627502f);
    r = fmaf(r, e, -0.1526966691017151f);
    r = fmaf(r, e, 0.1966327428817749f);
    r = fmaf(r, e, -0.24951615929603577f);
    r = fmaf(r, e, 0.33329710364341736f);
    r = fmaf(r, e, -0.49999892711639404f);
    r = fmaf(r, e, 1.f);
    return fmaf(e, r, fmaxf(v, 0.f));
}
__device__ __forceinline__ F2 softplus2(F2 v) {
    float a, b;
    unpack2(v, a, b);
    return pack2(softplus(a), softplus(b));
}

// ex2.approx lies 0.5e-8 to 2.7e-8 of its value too low on average for arguments in [-0.5, 0]
// (measured on 2^20 points in each of ten ranges), which a state that hardly decays adds up
// token by token: 1.3e-8 each, 1.9e-6 after 153. With this added to the argument the mean
// lies within 1.3e-8 on both sides of 0, and 2^kLift is 1, so Delta = 0 keeps a state's bits.
constexpr float kLift = 2e-8f;

// Four consecutive elements of an aligned shared row, or zeros.
__device__ __forceinline__ float4 widen4(const float *p, bool in) {
    const float4 q = *reinterpret_cast<const float4 *>(p);
    return in ? q : make_float4(0.f, 0.f, 0.f, 0.f);
}
__device__ __forceinline__ float4 widen4(const __nv_bfloat16 *p, bool in) {
    uint2 q = *reinterpret_cast<const uint2 *>(p);
    if (!in) q = make_uint2(0, 0);
    return make_float4(__uint_as_float(q.x << 16), __uint_as_float(q.x & 0xffff0000u),
                       __uint_as_float(q.y << 16), __uint_as_float(q.y & 0xffff0000u));
}

// ----------------------------------------------------------------- a few tokens
//
// Bound by the states' traffic: each is read and written once. L = NP / 4 lanes share a
// channel, four states to a lane. A thread advances NB sequences at a time, whose states'
// loads are in flight together, and p.turns such sets one after the other: A is read
// once for all of them, and a set's states and tokens arrive while the one before is
// worked on. Of a channel's L lanes, lane m % L takes Delta, the gate and the output of
// sequence m. One token of 256 sequences, 4096 channels, N = 16, bf16: 33 us, 4.3 TB/s (one set
// to a block, 12 blocks to an SM: 40; six, eight and ten blocks of several sets: 35, 33, 48);
// N = 64 in fp32 101 us, 5.5 TB/s (134; 107, 162, -).
constexpr int kBatch = 4;
constexpr int kStepBlocks = 7;      // to an SM, by registers

template <typename E, int NP, int NB>
__global__ void __launch_bounds__(kThreads, NB > 1 ? kStepBlocks : 1) gdn_scan_step_kernel(const ScanParams<E> p) {
    constexpr int L = NP / 4, channels = kThreads / L, OWN = (NB + L - 1) / L;
    constexpr int BC = NB * 2 * NP, BCT = (BC + kThreads - 1) / kThreads;
    __shared__ __align__(16) float bc[2][NB][2][NP];   // a token's B and C rows, of two tokens in turn
    const int per = p.D / p.G, blocks = (per + channels - 1) / channels;
    const int g = blockIdx.x / blocks, c0 = blockIdx.x % blocks * channels;
    const int tid = threadIdx.x, c = tid / L, j = tid % L, n0 = j * 4;
    const bool live = c0 + c < per;
    const int d = g * per + c0 + (live ? c : 0);
    const bool quads = p.N % 4 == 0;   // rows of states are whole 16-byte pieces
    auto quad = [&](const float *row, float (&f)[4]) {
#pragma unroll
        for (int k = 0; k < 4; ++k) f[k] = 0.f;
        if (quads) {
            if (n0 < p.N) {
                const float4 q = *reinterpret_cast<const float4 *>(row + n0);
                f[0] = q.x; f[1] = q.y; f[2] = q.z; f[3] = q.w;
            }
        } else {
#pragma unroll
            for (int k = 0; k < 4; ++k)
                if (n0 + k < p.N) f[k] = row[n0 + k];
        }
    };
    const int64_t state = static_cast<int64_t>(p.D) * p.N, row = static_cast<int64_t>(d) * p.N;
    const int b_first = blockIdx.y * p.turns * NB, b_end = min(p.B, b_first + p.turns * NB);
    float hn[NB][4];
    auto load_states = [&](int b0) {
#pragma unroll
        for (int m = 0; m < NB; ++m) {
#pragma unroll
            for (int k = 0; k < 4; ++k) hn[m][k] = 0.f;
            if (p.h0 && b0 + m < b_end) quad(p.h0 + (b0 + m) * state + row, hn[m]);
        }
    };
    // A token's rows: B and C of all NB sequences over the block, x, dt and z of this lane's.
    E rbc[BCT], rx[OWN], rdt[OWN], rz[OWN];
    auto load_token = [&](int b0, int t) {
#pragma unroll
        for (int i = 0; i < BCT; ++i) {
            const int at = i * kThreads + tid, q = at % NP;
            const int64_t b = b0 + at / (2 * NP);
            rbc[i] = from_f32<E>(0.f);    // behind a sequence's end: B = C = 0, Delta = 0
            if (at < BC && b < b_end && q < p.N && t < valid_tokens(p.lengths, b, p.T)) {
                const int64_t of = static_cast<int64_t>(g) * p.N + q;
                rbc[i] = at / NP % 2 ? p.Cm[b * p.c_sb + t * p.c_st + of] : p.Bm[b * p.b_sb + t * p.b_st + of];
            }
        }
#pragma unroll
        for (int o = 0; o < OWN; ++o) {
            const int64_t b = b0 + o * L + j;
            rx[o] = rdt[o] = rz[o] = from_f32<E>(0.f);
            if (o * L + j < NB && b < b_end && t < valid_tokens(p.lengths, b, p.T)) {
                rx[o] = p.x[b * p.x_sb + t * p.x_st + d];
                rdt[o] = p.dt[b * p.dt_sb + t * p.dt_st + d];
                if (p.z) rz[o] = p.z[b * p.z_sb + t * p.z_st + d];
            }
        }
    };
    load_states(b_first);
    load_token(b_first, 0);
    float A2[4];
    quad(p.A + row, A2);
    const float bias = p.dt_bias ? p.dt_bias[d] : 0.f, skip = p.skip ? p.skip[d] : 0.f;
#pragma unroll
    for (int k = 0; k < 4; ++k) A2[k] *= kLog2e;

    int place = 0;
    for (int b0 = b_first; b0 < b_end; b0 += NB) {
        float h[NB][4];
#pragma unroll
        for (int m = 0; m < NB; ++m)
#pragma unroll
            for (int k = 0; k < 4; ++k) h[m][k] = hn[m][k];
        if (NB > 1) load_states(b0 + NB);
        for (int t = 0; t < p.T; ++t, place ^= 1) {
#pragma unroll
            for (int i = 0; i < BCT; ++i)
                if (BC % kThreads == 0 || i * kThreads + tid < BC)
                    (&bc[place][0][0][0])[i * kThreads + tid] = to_f32(rbc[i]);
            float x[OWN], z[OWN], step[OWN], u[OWN], y[OWN];
            bool mine[OWN];
#pragma unroll
            for (int o = 0; o < OWN; ++o) {
                const int64_t b = b0 + o * L + j;
                mine[o] = o * L + j < NB && b < b_end && t < valid_tokens(p.lengths, b < b_end ? b : 0, p.T);
                x[o] = to_f32(rx[o]);
                z[o] = to_f32(rz[o]);
                step[o] = y[o] = 0.f;
                if (mine[o]) {
                    step[o] = to_f32(rdt[o]) + bias;
                    if (p.softplus) step[o] = softplus(step[o]);
                }
                u[o] = step[o] * x[o];
            }
            const bool same = t + 1 < p.T;
            load_token(same ? b0 : b0 + NB, same ? t + 1 : 0);
            __syncthreads();      // the other place is read by then
#pragma unroll
            for (int m = 0; m < NB; ++m) {
                const int from = (tid & 31 & ~(L - 1)) | m % L;
                const float dt = __shfl_sync(0xffffffffu, step[m / L], from);
                const float du = __shfl_sync(0xffffffffu, u[m / L], from);
                const float4 bq = *reinterpret_cast<const float4 *>(&bc[place][m][0][n0]);
                const float4 cq = *reinterpret_cast<const float4 *>(&bc[place][m][1][n0]);
                const float bv[4] = {bq.x, bq.y, bq.z, bq.w}, cv[4] = {cq.x, cq.y, cq.z, cq.w};
                float sum = 0.f;
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    h[m][k] = fmaf(exp2_ftz(fmaf(dt, A2[k], kLift)), h[m][k], du * bv[k]);
                    sum = fmaf(cv[k], h[m][k], sum);
                }
#pragma unroll
                for (int o = L / 2; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
                if (m % L == j) y[m / L] = sum;
            }
#pragma unroll
            for (int o = 0; o < OWN; ++o) {
                if (!mine[o] || !live) continue;
                if (p.skip) y[o] = fmaf(skip, x[o], y[o]);
                if (p.z) y[o] *= activate(z[o], GDN_ACT_SILU);
                p.y[(static_cast<int64_t>(b0 + o * L + j) * p.T + t) * p.D + d] = from_f32<E>(y[o]);
            }
        }
        if (!p.h_final || !live) continue;
#pragma unroll
        for (int m = 0; m < NB; ++m) {
            if (b0 + m >= b_end) break;
            float *to = p.h_final + (b0 + m) * state + row + n0;
            if (quads) {
                if (n0 < p.N) *reinterpret_cast<float4 *>(to) = make_float4(h[m][0], h[m][1], h[m][2], h[m][3]);
            } else {
#pragma unroll
                for (int k = 0; k < 4; ++k)
                    if (n0 + k < p.N) to[k] = h[m][k];
            }
        }
    }
}

// ---------------------------------------------------------------------- prompts
//
// A block takes 64 channels of one group of one sequence, two lanes to a channel with half of
// its states each (four, then the other lane's four), and walks the tokens in tiles of 32:
//   copy    the next tile's rows on their way to shared memory;
//   widen   Delta and Delta x of every token and channel, B and C as fp32;
//   scan    per token and state: ex2(Delta A), h = a h + (Delta x) B, y += C h, on pairs
//           of states; after four tokens the two lanes exchange their shares of y,
//           each keeping two tokens' sums;
//   finish  D x, the gate, and rows of y in 16-byte pieces.
// Delta's and the gate's special functions are taken once per token and channel, not in both
// lanes. Rows that are not whole 16-byte pieces are copied and stored element by element,
// everything between is alike.
//
// Bound by the scan's instructions: 16 states take about 105 cycles of an SM quarter for 32
// (token, channel) pairs however they are written (packed, scalar or mixed: their
// operands leave the register file no faster). Of 201 us for B4 T2048 D4096 N = 16 in bf16
// the scan takes 131, widening 32, finishing 26, the copies 12. Measured against this,
// in us there and then: a tile's scan between the widening of the next and the
// finishing of the last, in straight code, 230 for 232; warps of their own for these 264;
// four lanes to a channel 262 for 230; blocks of 64 threads 203, of 32 208, of 256 254 (for
// 201; one sequence of 32768 tokens and 2048 channels 622, 649 and 506 for 511).
//
// Two lanes, because shared memory hands a warp B and C 16 bytes a lane in 2 cycles for
// two addresses but in 4 for more: with four lanes to a channel N = 64 took 1237 us (523
// now), with eight N = 128 in fp32 4720 us (1225 now).
constexpr int kTile = 32;
constexpr int kChannels = kThreads / 2;

template <typename E, int NP>
struct Tile {
    static constexpr int V = 16 / sizeof(E);                 // channels of a piece
    static constexpr int pieces = kChannels / V;             // of a row
    static constexpr int row = kChannels * sizeof(E) + 16;   // bytes; 16 more: no bank conflicts
    static constexpr int du_row = 2 * kTile + 4;             // floats of a channel's (Delta, Delta x)
    static constexpr int y_row = kChannels + 16;
    static constexpr int bc = kTile * NP * sizeof(E);
    static constexpr int raw = 3 * kTile * row + 2 * bc;     // x, dt, z, B, C
    static constexpr int du = kChannels * du_row * 4;
    static constexpr int wide = kTile * NP * 4;
    static constexpr int y = kTile * y_row * 4;
    static constexpr int bytes = 2 * raw + du + 2 * wide + y;
};

// GATE: with z. PARTIAL: only the state at the end of a segment that starts from zero.
template <typename E, int NP, bool GATE, bool PARTIAL>
__global__ void __launch_bounds__(kThreads, NP <= 32 ? 3 : NP <= 64 ? 2 : 1) gdn_scan_kernel(ScanParams<E> p) {
    using S = Tile<E, NP>;
    constexpr int SP2 = NP / 4, TT = kTile, V = S::V, PR = S::pieces;     // SP2: pairs of states of a lane
    constexpr int TURNS = TT * PR / kThreads;                // of a thread over a tile's pieces
    static_assert(TT * PR % kThreads == 0, "whole turns");
    extern __shared__ __align__(16) unsigned char smem[];
    // tile k's rows; the tile's (Delta, Delta x), B and C, y
    auto raw_of = [&](int k) { return smem + (k & 1) * S::raw; };
    float *const du = reinterpret_cast<float *>(smem + 2 * S::raw), *const bc = du + S::du / 4;
    float *const yb = bc + 2 * S::wide / 4;

    const int per = p.D / p.G, blocks = (per + kChannels - 1) / kChannels;
    const int g = blockIdx.x / blocks, c0 = blockIdx.x % blocks * kChannels;
    const int nc = min(kChannels, per - c0);       // channels of this block
    const int d0 = g * per + c0;
    const int64_t b = blockIdx.y;
    const int s = blockIdx.z;
    const int n = valid_tokens(p.lengths, b, p.T);
    const int t_begin = s * p.seg, t_end = min(n, t_begin + p.seg);
    if (s > 0 && t_begin >= n) return;
    const int tokens = t_end - t_begin, tiles = (tokens + TT - 1) / TT;

    // The second pass begins once all of the first one's blocks have begun, and waits for
    // their end before it reads what they leave: its first tile is there by then (54 us for 58,
    // B5 T777 D1000 N24 fp32). Its first segments' blocks always wait, so it ends after the
    // first pass.
    if (PARTIAL) ptx::griddep_launch_dependents();

    const int tid = threadIdx.x, c = tid / 2, j = tid % 2;
    const bool live = c < nc;
    const int d = d0 + (live ? c : 0);
    const int64_t state = (b * p.D + d) * p.N;
    auto seg_at = [&](int i) { return ((b * p.segs + i) * p.D + d); };

    F2 A2[SP2], h[SP2];
    auto load_states = [&](const float *row, F2 (&f)[SP2], float scale) {
#pragma unroll
        for (int q = 0; q < SP2; ++q) {
            const int k = (q / 2 * 2 + j) * 4 + q % 2 * 2;
            f[q] = pack2(live && k < p.N ? scale * row[k] : 0.f,
                         live && k + 1 < p.N ? scale * row[k + 1] : 0.f);
        }
    };
    auto store_states = [&](float *row) {
        if (!live) return;
#pragma unroll
        for (int q = 0; q < SP2; ++q) {
            const int k = (q / 2 * 2 + j) * 4 + q % 2 * 2;
            float lo, hi;
            unpack2(h[q], lo, hi);
            if (k < p.N) row[k] = lo;
            if (k + 1 < p.N) row[k + 1] = hi;
        }
    };
    auto decay = [&](F2 step, F2 A2) {
        float lo, hi;
        unpack2(fma2(step, A2, pack2(kLift, kLift)), lo, hi);
        return pack2(exp2_ftz(lo), exp2_ftz(hi));
    };
    load_states(p.A + static_cast<int64_t>(d) * p.N, A2, kLog2e);
#pragma unroll
    for (int q = 0; q < SP2; ++q) h[q] = 0;

    // ------------------------------------------------------------------------- copy
    // Row by row: this thread's piece of every kThreads / PR-th row, of the next tile.
    const int piece = tid % PR * V;
    struct Rows {
        const E *at;
        int64_t turn;        // from row to row of a tile, TURNS of them
    };
    auto rows_of = [&](const E *src, int64_t sb, int64_t st) {
        return Rows{src + b * sb + (t_begin + tid / PR) * st + d0 + piece, kThreads / PR * st};
    };
    Rows rx = rows_of(p.x, p.x_sb, p.x_st), rdt = rows_of(p.dt, p.dt_sb, p.dt_st), rz = rx;
    if (GATE) rz = rows_of(p.z, p.z_sb, p.z_st);
    auto copy_rows = [&](unsigned char *dst, Rows &r, const E *src, int64_t sb, int64_t st, int t0, int rows) {
        if (p.pieces) {
            unsigned char *to = dst + tid / PR * S::row + piece * sizeof(E);
#pragma unroll
            for (int i = 0; i < TURNS; ++i) {
                if (piece < nc && tid / PR + i * (kThreads / PR) < rows)
                    copy16_async(to + i * (kThreads / PR) * S::row, r.at);
                r.at += r.turn;
            }
        } else {
            const int q = tid % kChannels;
            if (q >= nc) return;
#pragma unroll 8
            for (int t = tid / kChannels; t < rows; t += kThreads / kChannels) {
                E *to = reinterpret_cast<E *>(dst + t * S::row) + q;
                const E *from = src + b * sb + (t0 + t) * st + d0 + q;
                if constexpr (sizeof(E) == 4)
                    copy4_async(to, from);
                else
                    *to = *from;
            }
        }
    };
    // B and C the same way, MOST pieces to a row at most.
    constexpr int W = 16 / sizeof(E), MOST = NP / W, STEP = kThreads / MOST, BC = (TT + STEP - 1) / STEP;
    const int at_bc = tid % MOST * W;
    auto bc_rows_of = [&](const E *src, int64_t sb, int64_t st) {
        return Rows{src + b * sb + (t_begin + tid / MOST) * st + static_cast<int64_t>(g) * p.N + at_bc,
                    STEP * st};
    };
    Rows rb = bc_rows_of(p.Bm, p.b_sb, p.b_st), rc = bc_rows_of(p.Cm, p.c_sb, p.c_st);
    auto copy_bc = [&](unsigned char *dst, Rows &r, const E *src, int64_t sb, int64_t st, int t0, int rows) {
        if (p.rows16) {
            E *to = reinterpret_cast<E *>(dst) + tid / MOST * NP + at_bc;
#pragma unroll
            for (int i = 0; i < BC; ++i) {
                if (at_bc < p.N && tid / MOST < STEP && tid / MOST + i * STEP < rows)
                    copy16_async(to + i * STEP * NP, r.at + i * r.turn);
            }
            r.at += TT * st;
        } else {
            const E *from = src + b * sb + t0 * st + static_cast<int64_t>(g) * p.N;
            E *to = reinterpret_cast<E *>(dst);
            // eight loads at a time in flight
            for (int i0 = tid; i0 < rows * NP; i0 += 8 * kThreads) {
                E v[8];
#pragma unroll
                for (int m = 0; m < 8; ++m) {
                    const int i = i0 + m * kThreads, t = i / NP, q = i % NP;
                    if (t < rows && q < p.N) v[m] = from[t * st + q];
                }
#pragma unroll
                for (int m = 0; m < 8; ++m) {
                    const int i = i0 + m * kThreads;
                    if (i / NP < rows && i % NP < p.N) to[i] = v[m];
                }
            }
        }
    };
    auto fetch = [&](int k) {
        const int t0 = t_begin + k * TT, rows = min(TT, t_end - t0);
        unsigned char *raw = raw_of(k);
        if (rows > 0) {
            copy_rows(raw, rx, p.x, p.x_sb, p.x_st, t0, rows);
            copy_rows(raw + TT * S::row, rdt, p.dt, p.dt_sb, p.dt_st, t0, rows);
            copy_bc(raw + 3 * TT * S::row, rb, p.Bm, p.b_sb, p.b_st, t0, rows);
            if (!PARTIAL) {
                if (GATE) copy_rows(raw + 2 * TT * S::row, rz, p.z, p.z_sb, p.z_st, t0, rows);
                copy_bc(raw + 3 * TT * S::row + S::bc, rc, p.Cm, p.c_sb, p.c_st, t0, rows);
            }
        }
        copy_commit();
    };

    // ------------------------------------------------------------------------ widen
    // A thread takes one token of a few pieces; a tile's copies never write B and C behind N,
    // which are 0 from the start. Tokens behind the segment (full: there are none) get Delta = 0
    // and B = C = 0 and change nothing.
    F2 bias[TURNS][V / 2];
#pragma unroll
    for (int i = 0; i < TURNS; ++i) {
        const int q = (i * kThreads + tid) / TT * V;
#pragma unroll
        for (int v = 0; v < V / 2; ++v)
            bias[i][v] = p.dt_bias ? pack2(q + 2 * v < nc ? p.dt_bias[d0 + q + 2 * v] : 0.f,
                                           q + 2 * v + 1 < nc ? p.dt_bias[d0 + q + 2 * v + 1] : 0.f)
                                   : 0;
    }
    auto widen = [&](int k, auto full) {
        const unsigned char *raw = raw_of(k);
        const int rows = tokens - k * TT;
#pragma unroll
        for (int i = 0; i < TURNS; ++i) {
            const int at = i * kThreads + tid, t = at % TT, q = at / TT * V;
            F2 x[V / 2], step[V / 2];
            Piece<E, V> pc;
            pc.load_rw(reinterpret_cast<const E *>(raw + t * S::row) + q);
            pc.widen(x);
            pc.load_rw(reinterpret_cast<const E *>(raw + (TT + t) * S::row) + q);
            pc.widen(step);
            float *to = du + q * S::du_row + 2 * t;
#pragma unroll
            for (int v = 0; v < V / 2; ++v) {
                step[v] = add2(step[v], bias[i][v]);
                const F2 soft = softplus2(step[v]);
                step[v] = p.softplus ? soft : step[v];
                F2 u = mul2(step[v], x[v]);
                if (!full && t >= rows) step[v] = u = 0;
                float s0, s1, u0, u1;
                unpack2(step[v], s0, s1);
                unpack2(u, u0, u1);
                *reinterpret_cast<float2 *>(to + 2 * v * S::du_row) = make_float2(s0, u0);
                *reinterpret_cast<float2 *>(to + (2 * v + 1) * S::du_row) = make_float2(s1, u1);
            }
        }
        constexpr int ROWS = PARTIAL ? TT : 2 * TT;             // B's rows, then C's
#pragma unroll
        for (int i0 = 0; i0 < ROWS * NP; i0 += kThreads * 4) {
            const int i = i0 + tid * 4;
            if (ROWS * NP % (kThreads * 4) != 0 && i >= ROWS * NP) break;
            const E *from = reinterpret_cast<const E *>(raw + 3 * TT * S::row) + i;
            *reinterpret_cast<float4 *>(bc + i) = widen4(from, full || i / NP % TT < rows);
        }
    };

    // ----------------------------------------------------------------------- finish
    F2 skip[V / 2];
#pragma unroll
    for (int v = 0; v < V / 2; ++v)
        skip[v] = p.skip && !PARTIAL ? pack2(piece + 2 * v < nc ? p.skip[d0 + piece + 2 * v] : 0.f,
                                             piece + 2 * v + 1 < nc ? p.skip[d0 + piece + 2 * v + 1] : 0.f)
                                     : 0;
    E *y_at = p.y + (b * p.T + t_begin + tid / PR) * p.D + d0 + piece;     // this thread's first of a tile
    const int64_t y_turn = static_cast<int64_t>(kThreads / PR) * p.D;
    auto finish = [&](int k) {
        const unsigned char *raw = raw_of(k);
        const int t0 = t_begin + k * TT;
#pragma unroll
        for (int i = 0; i < TURNS; ++i) {
            const int t = tid / PR + i * (kThreads / PR);
            F2 v[V / 2], w[V / 2];
            Piece<E, V> pc;
#pragma unroll
            for (int q = 0; q < V / 2; q += 2) {
                const ulonglong2 two =
                    *reinterpret_cast<const ulonglong2 *>(yb + t * S::y_row + piece + 2 * q);
                v[q] = two.x;
                v[q + 1] = two.y;
            }
            if (p.skip) {                 // without: x may be anything
                pc.load_rw(reinterpret_cast<const E *>(raw + t * S::row) + piece);
                pc.widen(w);
#pragma unroll
                for (int q = 0; q < V / 2; ++q) v[q] = fma2(skip[q], w[q], v[q]);
            }
            if constexpr (GATE) {
                pc.load_rw(reinterpret_cast<const E *>(raw + (2 * TT + t) * S::row) + piece);
                pc.widen(w);
#pragma unroll
                for (int q = 0; q < V / 2; ++q) v[q] = mul2(v[q], mul2(w[q], sigmoid2(w[q])));
            }
            pc.round(v);
            E *const to = y_at;
            y_at += y_turn;
            if (t0 + t < t_end && piece < nc) {
                if (p.pieces) {
                    pc.store(to);
                } else {
                    float f[V];
#pragma unroll
                    for (int q = 0; q < V / 2; ++q) unpack2(v[q], f[2 * q], f[2 * q + 1]);
#pragma unroll
                    for (int q = 0; q < V; ++q)
                        if (piece + q < nc) to[q] = from_f32<E>(f[q]);
                }
            }
        }
    };

    // ------------------------------------------------------------------------- scan
    float dt_sum = 0.f;
    auto scan = [&](int t) {
        const float *my = du + c * S::du_row + 2 * t;
        const float *bw = bc + t * NP;
        float yt[4];
        const float4 da = *reinterpret_cast<const float4 *>(my);
        const float4 db = *reinterpret_cast<const float4 *>(my + 4);
        const float step[4] = {da.x, da.z, db.x, db.z}, in[4] = {da.y, da.w, db.y, db.w};
#pragma unroll
        for (int m = 0; m < 4; ++m) {
            const F2 dd = pack2(step[m], step[m]), uu = pack2(in[m], in[m]);
            const ulonglong2 *br = reinterpret_cast<const ulonglong2 *>(bw + m * NP) + j;
            const ulonglong2 *cr = reinterpret_cast<const ulonglong2 *>(bw + (TT + m) * NP) + j;
            F2 acc = 0;
#pragma unroll
            for (int q = 0; q < SP2; q += 2) {
                const ulonglong2 bq = br[q];
                h[q] = fma2(decay(dd, A2[q]), h[q], mul2(uu, bq.x));
                h[q + 1] = fma2(decay(dd, A2[q + 1]), h[q + 1], mul2(uu, bq.y));
                if (!PARTIAL) {
                    const ulonglong2 cq = cr[q];
                    acc = q == 0 ? mul2(cq.x, h[q]) : fma2(cq.x, h[q], acc);
                    acc = fma2(cq.y, h[q + 1], acc);
                }
            }
            float lo, hi;
            unpack2(acc, lo, hi);
            yt[m] = lo + hi;
        }
        if constexpr (PARTIAL) {
            dt_sum += (step[0] + step[1]) + (step[2] + step[3]);
        } else {
            // lane j keeps tokens j and 2 + j
            float *y = yb + t * S::y_row + c;
            const float r0 = __shfl_xor_sync(0xffffffffu, j ? yt[0] : yt[1], 1);
            const float r1 = __shfl_xor_sync(0xffffffffu, j ? yt[2] : yt[3], 1);
            y[j * S::y_row] = (j ? yt[1] : yt[0]) + r0;
            y[(2 + j) * S::y_row] = (j ? yt[3] : yt[2]) + r1;
        }
    };

    if (p.N < NP) {     // B and C behind N, in both raw places
        for (int i = tid; i < 4 * TT * NP; i += kThreads)
            reinterpret_cast<E *>(raw_of(i / (2 * TT * NP)) + 3 * TT * S::row)[i % (2 * TT * NP)] =
                from_f32<E>(0.f);
        __syncthreads();
    }
    fetch(0);
    // the state, while the first tile arrives
    if (p.segs == 1) {
        if (p.h0) load_states(p.h0 + state, h, 1.f);
    } else if (PARTIAL) {
        // h0 starts the first segment; a copy serves the second pass, which may write
        // h_final in h0's place
        if (s == 0) {
            if (p.h0) load_states(p.h0 + state, h, 1.f);
            store_states(p.seg_h + seg_at(p.segs - 1) * p.N);
        }
    } else if (s == 0) {
        ptx::griddep_wait();
        load_states(p.seg_h + seg_at(p.segs - 1) * p.N, h, 1.f);
    } else {
        ptx::griddep_wait();
        for (int i = 0; i < s; ++i) {
            F2 e[SP2];
            load_states(p.seg_h + seg_at(i) * p.N, e, 1.f);
            const float sum = p.seg_dt[seg_at(i)];
            // exp(A sum) in two factors: where Delta A > 0 it may pass the range though its
            // product with a small state does not (nor 0 times it). A normal number times
            // 2^254 is beyond the range anyway.
#pragma unroll
            for (int q = 0; q < SP2; ++q) {
                float lo, hi;
                unpack2(mul2(pack2(sum, sum), A2[q]), lo, hi);
                const F2 f = pack2(exp2_ftz(fminf(lo, 127.f)), exp2_ftz(fminf(hi, 127.f)));
                const F2 rest = pack2(exp2_ftz(fminf(fmaxf(lo - 127.f, 0.f), 127.f)),
                                      exp2_ftz(fminf(fmaxf(hi - 127.f, 0.f), 127.f)));
                h[q] = fma2(mul2(h[q], f), rest, e[q]);
            }
        }
    }
    for (int k = 0; k < tiles; ++k) {
        const int rows = min(TT, tokens - k * TT);
        copy_wait<0>();
        __syncthreads();     // tile k's rows are here; tile k - 1 is finished
        fetch(k + 1);
        if (rows == TT) widen(k, std::true_type()); else widen(k, std::false_type());
        __syncthreads();
        if (NP <= 16 && rows == TT) {
#pragma unroll 4
            for (int t = 0; t < TT; t += 4) scan(t);
        } else {
            for (int t = 0; t < rows; t += 4) scan(t);
        }
        if constexpr (!PARTIAL) {
            __syncthreads();
            finish(k);
        }
    }
    copy_wait<0>();
    if constexpr (PARTIAL) {
        store_states(p.seg_h + seg_at(s) * p.N);
        if (live && j == 0) p.seg_dt[seg_at(s)] = dt_sum;
    } else if (p.h_final && t_end == n) {
        store_states(p.h_final + state);
    }
}

gdn_status check(const gdn_scan_problem *p) {
    if (!p) return GDN_ERR_INVALID_ARG;
    if (p->B <= 0 || p->D <= 0 || p->N <= 0 || p->G <= 0 || p->T < 0 || p->D % p->G != 0)
        return GDN_ERR_INVALID_ARG;
    if (p->dtype != GDN_F32 && p->dtype != GDN_BF16) return GDN_ERR_INVALID_ARG;
    if ((p->flags & ~GDN_SCAN_SOFTPLUS) || p->reserved) return GDN_ERR_INVALID_ARG;
    for (int64_t s : {p->x_stride_b, p->x_stride_t, p->dt_stride_b, p->dt_stride_t, p->z_stride_b,
                      p->z_stride_t, p->b_stride_b, p->b_stride_t, p->c_stride_b, p->c_stride_t})
        if (s < 0) return GDN_ERR_INVALID_ARG;
    // 2^30: token indexes of a tile past the end stay in 32 bits
    if (p->N > 128 || p->B > 65535 || p->D > (1 << 24) || p->T > (1 << 30)) return GDN_ERR_UNSUPPORTED;
    return GDN_OK;
}

int64_t row_blocks(const gdn_scan_problem *p) {
    const int per = p->D / p->G;
    return static_cast<int64_t>(p->G) * ((per + kChannels - 1) / kChannels);
}

// Segments of a prompt: so many that 3 blocks stand on every SM, of 64 tokens at least. The
// first pass over a segment repeats most of the arithmetic, so channels that alone fill
// half of those places are not cut. One sequence of 32768 tokens and 2048 channels (32
// blocks), when chosen: 572 us in 14 segments (511 now), 655 in 9, 590 in 23; 512 tokens
// of it 27 us in 8, 49 in 2. Four of 2048 tokens and 4096 channels (256 blocks): 230 us
// whole (201 now), 296 in 2.
int segments(const gdn_scan_problem *p) {
    const int64_t blocks = p->B * row_blocks(p);
    const int64_t want = 3 * 152 / blocks, most = p->T / 64;
    const int64_t n = want < most ? want : most;
    return n < 2 ? 1 : n > 64 ? 64 : static_cast<int>(n);
}

size_t workspace_need(const gdn_scan_problem *p) {
    const int n = segments(p);
    const size_t rows = static_cast<size_t>(p->B) * n * p->D;
    return n == 1 ? 0 : align_up(rows * p->N * 4) + align_up(rows * 4);
}

// second: behind the first pass on the same stream, which it waits for by itself.
template <typename E>
cudaError_t launch_blocks(void (*kernel)(ScanParams<E>), dim3 grid, int bytes, const ScanParams<E> &p,
                          bool second, cudaStream_t s) {
    const cudaError_t e = cudaFuncSetAttribute(reinterpret_cast<const void *>(kernel),
                                               cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
    if (e != cudaSuccess) return e;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = bytes;
    cfg.stream = s;
    cfg.attrs = attr;
    cfg.numAttrs = second ? 1 : 0;
    return cudaLaunchKernelEx(&cfg, kernel, p);
}

template <typename E, int NP>
cudaError_t launch_prompt(const gdn_scan_problem *pr, ScanParams<E> &p, void *workspace, cudaStream_t s) {
    using S = Tile<E, NP>;
    const int n = segments(pr);
    p.seg = ((pr->T + n - 1) / n + kTile - 1) / kTile * kTile;
    p.segs = (pr->T + p.seg - 1) / p.seg;
    const dim3 grid(static_cast<unsigned>(row_blocks(pr)), pr->B, p.segs);
    if (p.segs > 1) {
        p.seg_h = static_cast<float *>(workspace);
        p.seg_dt = reinterpret_cast<float *>(
            static_cast<char *>(workspace) +
            align_up(static_cast<size_t>(pr->B) * p.segs * pr->D * pr->N * 4));
        const cudaError_t e = launch_blocks(gdn_scan_kernel<E, NP, false, true>,
                                            dim3(grid.x, grid.y, p.segs - 1), S::bytes, p, false, s);
        if (e != cudaSuccess) return e;
    }
    return launch_blocks(p.z ? gdn_scan_kernel<E, NP, true, false> : gdn_scan_kernel<E, NP, false, false>,
                         grid, S::bytes, p, p.segs > 1, s);
}

template <typename E, int NP>
cudaError_t launch_step(const gdn_scan_problem *pr, ScanParams<E> &p, cudaStream_t s) {
    // kBatch sequences to a thread where that still leaves two blocks to an SM
    constexpr int channels = kThreads / (NP / 4);
    const int64_t blocks = pr->G * ((pr->D / pr->G + channels - 1) / channels);
    const int64_t sets = (pr->B + kBatch - 1) / kBatch;
    p.turns = 1;
    if (blocks * sets < 2 * 152) {
        gdn_scan_step_kernel<E, NP, 1><<<dim3(blocks, pr->B), kThreads, 0, s>>>(p);
        return cudaGetLastError();
    }
    // Sets to a block by the turns of all waves, with one more for a block's start.
    constexpr int64_t wave = 152 * kStepBlocks;
    int64_t best = 0;
    for (int w = 1; w <= 4; ++w) {
        const int64_t rows = std::max<int64_t>(1, std::min(sets, w * wave / blocks));
        const int64_t turns = (sets + rows - 1) / rows;
        const int64_t cost = (blocks * ((sets + turns - 1) / turns) + wave - 1) / wave * (turns + 1);
        if (best == 0 || cost < best) {
            best = cost;
            p.turns = static_cast<int>(turns);
        }
    }
    gdn_scan_step_kernel<E, NP, kBatch>
        <<<dim3(blocks, (sets + p.turns - 1) / p.turns), kThreads, 0, s>>>(p);
    return cudaGetLastError();
}

template <typename E>
cudaError_t dispatch(const gdn_scan_problem *pr, ScanParams<E> &p, void *workspace, cudaStream_t s) {
    p.x_sb = pr->x_stride_b; p.x_st = pr->x_stride_t;
    p.dt_sb = pr->dt_stride_b; p.dt_st = pr->dt_stride_t;
    p.z_sb = pr->z_stride_b; p.z_st = pr->z_stride_t;
    p.b_sb = pr->b_stride_b; p.b_st = pr->b_stride_t;
    p.c_sb = pr->c_stride_b; p.c_st = pr->c_stride_t;
    p.B = pr->B; p.T = pr->T; p.D = pr->D; p.N = pr->N; p.G = pr->G;
    p.softplus = (pr->flags & GDN_SCAN_SOFTPLUS) ? 1 : 0;
    p.rows16 = p.pieces = 0;
    p.segs = 1; p.seg = pr->T; p.seg_h = p.seg_dt = nullptr;
    if (pr->T <= kStepTokens) {            // lanes to a channel: a power of two
        if (pr->N <= 8) return launch_step<E, 8>(pr, p, s);
        if (pr->N <= 16) return launch_step<E, 16>(pr, p, s);
        if (pr->N <= 32) return launch_step<E, 32>(pr, p, s);
        if (pr->N <= 64) return launch_step<E, 64>(pr, p, s);
        return launch_step<E, 128>(pr, p, s);
    }
    constexpr size_t e = sizeof(E);
    p.pieces = (pr->D / pr->G) * e % 16 == 0 &&
               pieces16(p.x, pr->B, pr->T, pr->D, p.x_sb, p.x_st, e) &&
               pieces16(p.dt, pr->B, pr->T, pr->D, p.dt_sb, p.dt_st, e) &&
               (!p.z || pieces16(p.z, pr->B, pr->T, pr->D, p.z_sb, p.z_st, e));
    p.rows16 = pieces16(p.Bm, pr->B, pr->T, pr->N, p.b_sb, p.b_st, e) &&
               pieces16(p.Cm, pr->B, pr->T, pr->N, p.c_sb, p.c_st, e);
    // states cost time one by one, so the sizes between powers of two are worth their instances
    if (pr->N <= 8) return launch_prompt<E, 8>(pr, p, workspace, s);
    if (pr->N <= 16) return launch_prompt<E, 16>(pr, p, workspace, s);
    if (pr->N <= 24) return launch_prompt<E, 24>(pr, p, workspace, s);
    if (pr->N <= 32) return launch_prompt<E, 32>(pr, p, workspace, s);
    if (pr->N <= 48) return launch_prompt<E, 48>(pr, p, workspace, s);
    if (pr->N <= 64) return launch_prompt<E, 64>(pr, p, workspace, s);
    if (pr->N <= 96) return launch_prompt<E, 96>(pr, p, workspace, s);
    return launch_prompt<E, 128>(pr, p, workspace, s);
}

}  // namespace
}  // namespace gdn

extern "C" {

GDN_API size_t gdn_scan_workspace_bytes(const gdn_scan_problem *p) {
    return gdn::check(p) == GDN_OK ? gdn::workspace_need(p) : SIZE_MAX;
}

GDN_API gdn_status gdn_scan_fwd(const gdn_scan_problem *p, const void *x, const void *dt,
                                const float *A, const void *Bm, const void *Cm, const float *skip,
                                const void *z, const float *dt_bias, const float *h0,
                                const int32_t *lengths, void *y, float *h_final, void *workspace,
                                size_t workspace_bytes, void *stream) {
    using gdn::Span;
    using gdn::strided_bytes;
    const gdn_status st = gdn::check(p);
    if (st != GDN_OK) return st;
    const bool empty = p->T == 0;
    if (!empty && (!x || !dt || !A || !Bm || !Cm || !y)) return GDN_ERR_INVALID_ARG;
    const size_t e = gdn::elem_bytes(p->dtype);
    for (const void *ptr : {static_cast<const void *>(A), static_cast<const void *>(skip),
                            static_cast<const void *>(dt_bias), static_cast<const void *>(h0),
                            static_cast<const void *>(y), static_cast<const void *>(h_final),
                            static_cast<const void *>(workspace)})
        if (!gdn::is_aligned(ptr, 16)) return GDN_ERR_ALIGNMENT;
    for (const void *ptr : {x, dt, z, Bm, Cm})
        if (!gdn::is_aligned(ptr, e)) return GDN_ERR_ALIGNMENT;
    if (!gdn::is_aligned(lengths, 4)) return GDN_ERR_ALIGNMENT;
    const size_t need = gdn::workspace_need(p);
    if (need && (!workspace || workspace_bytes < need)) return GDN_ERR_WORKSPACE;
    const int64_t GN = static_cast<int64_t>(p->G) * p->N;
    const size_t state = static_cast<size_t>(p->B) * p->D * p->N * 4;
    const Span in[] = {Span(x, strided_bytes(p->B, p->T, p->D, p->x_stride_b, p->x_stride_t, e)),
                       Span(dt, strided_bytes(p->B, p->T, p->D, p->dt_stride_b, p->dt_stride_t, e)),
                       Span(z, strided_bytes(p->B, p->T, p->D, p->z_stride_b, p->z_stride_t, e)),
                       Span(Bm, strided_bytes(p->B, p->T, GN, p->b_stride_b, p->b_stride_t, e)),
                       Span(Cm, strided_bytes(p->B, p->T, GN, p->c_stride_b, p->c_stride_t, e)),
                       Span(A, static_cast<size_t>(p->D) * p->N * 4),
                       Span(skip, static_cast<size_t>(p->D) * 4),
                       Span(dt_bias, static_cast<size_t>(p->D) * 4),
                       Span(lengths, static_cast<size_t>(p->B) * 4),
                       Span(h0, state)};
    const Span sy(y, static_cast<size_t>(p->B) * p->T * p->D * e), sh(h_final, state);
    const Span sw(workspace, need);
    for (const Span &i : in) {
        const bool in_place = &i == &in[9] && h0 == h_final;
        if (i.meets(sy) || (i.meets(sh) && !in_place) || i.meets(sw)) return GDN_ERR_INVALID_ARG;
    }
    if (sy.meets(sh) || sw.meets(sy) || sw.meets(sh)) return GDN_ERR_INVALID_ARG;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    cudaError_t err = cudaSuccess;
    if (empty) {
        if (h_final && h0 && h0 != h_final)
            err = cudaMemcpyAsync(h_final, h0, state, cudaMemcpyDeviceToDevice, s);
        else if (h_final && !h0)
            err = cudaMemsetAsync(h_final, 0, state, s);
        return err == cudaSuccess ? GDN_OK : GDN_ERR_CUDA;
    }
    auto go = [&](auto tag) {
        using E = decltype(tag);
        gdn::ScanParams<E> a;
        a.x = static_cast<const E *>(x);
        a.dt = static_cast<const E *>(dt);
        a.z = static_cast<const E *>(z);
        a.Bm = static_cast<const E *>(Bm);
        a.Cm = static_cast<const E *>(Cm);
        a.A = A; a.skip = skip; a.dt_bias = dt_bias; a.h0 = h0;
        a.lengths = lengths;
        a.y = static_cast<E *>(y);
        a.h_final = h_final;
        return gdn::dispatch<E>(p, a, workspace, s);
    };
    err = p->dtype == GDN_BF16 ? go(__nv_bfloat16()) : go(float());
    return err == cudaSuccess ? GDN_OK : GDN_ERR_CUDA;
}

}  // extern "C"
