// The MoE layer for a few tokens (at most kFewMaxTokens), the form a decoding
// step needs. Page 1 ("Mixture of Experts (MoE) 12段階極小ビジュアル解剖
// シミュレーター"), STEP 1-12; nanoMoE slides 11-40: the same layer as the
// grouped path, token for token.
//
// With a few tokens every expert that is hit serves a handful of rows, so the
// call is bound by the stream of the hit experts' weights (2 d d_ff elements
// each) and, for the smallest layers, by launch latency:
//
//   scores: one workgroup per (16 experts, range of d), partial scores to the
//         workspace (the bf16 layer's fp32 router weights as three exact bf16
//         terms on the matrix cores, the fp32 layer on fp32 MFMAs).
//   plan: one workgroup ranks the tokens (top-k and gates of a token per wave,
//         its partial scores added in range order) and lists the hit experts
//         and their kept rows in (choice, token) order. More than 16 tokens are
//         ranked by a launch of their own, a wave per token.
//   up:   one workgroup per (hit expert, 16 hidden neurons), four waves over K
//         that add through LDS. The grid is sized by min(E, N k), without a
//         host sync; workgroups past the last hit expert end at once.
//   down: one workgroup per (16 output columns, range of the hit experts'
//         K-chunks); its four waves take contiguous parts of the range and
//         keep the gate-weighted sums of all tokens in LDS, one copy per wave,
//         added in wave order. The workgroup of a column block that finishes
//         last adds the ranges' partial sums in range order and writes the
//         output: the combine costs no launch and the result does not depend
//         on which workgroup that is.
//
// Where a bf16 layer's experts have more than a few rows each, their tokens'
// operand loads would outnumber the weights': up and down then run on the tiled
// product (tile.hpp) instead, 64 rows (all an expert can have) by 128 columns a
// workgroup, the down product writing each assignment's fp32 row for a combine
// pass.
//
// A bf16 layer's hidden row is kept as two bf16 terms (hi + lo, 16 significant
// bits): the product that reads it is bound by its weights, so the second MFMA
// is free, and the layer's output then carries only its own final rounding.
//
// Measured: one token of the Mixtral-shaped layer 99 us (two experts, 470 MB;
// up 43 us, down 49, i.e. 5.4 and 4.8 TB/s, scores and plan 10), 61 tokens of the
// 256-expert layer 2150 us (12.8 GB: 6.0 TB/s, what a read-only stream reaches),
// one token of the nanoMoE-sized layer 18 us (19 MB; plan 5, up 6, down 7.5:
// launches and round trips).
#include <algorithm>
#include <type_traits>

#include "activation.hpp"
#include "common.hpp"
#include "ranking.hpp"
#include "skinny.hpp"
#include "tile.hpp"

namespace moe {
namespace {

constexpr int kFewTokens = kFewMaxTokens;
constexpr int kFewAssign = kFewTokens * kMaxTopK;   // assignments of a call
constexpr int kChunk = 256;                         // K elements of one down unit
constexpr int kScoreRange = 512;                    // columns of d per score range
constexpr int kWaves = 4;                           // waves of a workgroup
constexpr int kThreads = kWaves * 64;
constexpr int kPlanWaves = 16;                      // waves of the plan's workgroup

// Dispatch plan of the call (device, in the workspace).
struct FewPlan {
    int nhit;                              // experts with a kept row
    int expert[kMaxExperts];               // their ids, ascending
    int rows[kMaxExperts];                 // kept rows of each
    int row[kMaxExperts][kFewTokens];      // their assignments, slot order
};

// Where the layer's types differ: the hidden row's storage and its terms.
template <typename S>
struct Kind {
    static constexpr bool bf16 = std::is_same<S, SkinnyBf16>::value;
    typedef typename S::type type;
    static constexpr int terms = bf16 ? 2 : 1;   // operand terms of a hidden row
};

// Four adjacent fp32 values at p[0..3] of which n exist.
template <bool ALIGNED>
__device__ __forceinline__ f32x4 load4(const float *p, int n) {
    if (ALIGNED)
        return n > 0 ? *reinterpret_cast<const f32x4 *>(p) : f32x4{0.f, 0.f, 0.f, 0.f};
    f32x4 v;
#pragma unroll
    for (int i = 0; i < 4; ++i)
        v[i] = i < n ? p[i] : 0.f;
    return v;
}

// What rounding z to bf16 leaves, the second term of a hidden value (an
// infinity or a NaN leaves nothing, not the NaN of its difference).
__device__ __forceinline__ float second_term(float z) {
    const float rest = z - bf16_bits_to_f32(f32_to_bf16_bits(z));
    return fabsf(rest) < __builtin_inff() ? rest : 0.f;
}

// ---- scores ------------------------------------------------------------

// Score columns: experts a ranking lane holds (e, e + 64, ...) side by side.
__device__ __host__ __forceinline__ int score_lanes(int E) {
    return E <= 64 ? 1 : E <= 128 ? 2 : 4;
}

// Scores of a lane's expert row w and TT token rows over U K-steps from column
// kb on (none where kb is past d), all loads issued before the MFMAs.
template <typename S, int TT, int U>
__device__ __forceinline__ void score_tile(const float *w, const typename S::type *const (&xt)[TT],
                                           int kb, int d, f32x4 (&acc)[TT]) {
    const int ko = 8 * (int)(__lane_id() >> 4);
#pragma unroll
    for (int i = 0; i < TT; ++i)
        acc[i] = f32x4{0.f, 0.f, 0.f, 0.f};
    if constexpr (Kind<S>::bf16) {
        f32x4 w0[U], w1[U];
        u32x4 b[U][TT];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int k = kb + 32 * u + ko;
            w0[u] = w1[u] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int i = 0; i < TT; ++i)
                b[u][i] = u32x4{0u, 0u, 0u, 0u};
            if (k < d) {   // (d % 8 == 0)
                w0[u] = *reinterpret_cast<const f32x4 *>(w + k);
                w1[u] = *reinterpret_cast<const f32x4 *>(w + k + 4);
#pragma unroll
                for (int i = 0; i < TT; ++i)
                    b[u][i] = *reinterpret_cast<const u32x4 *>(xt[i] + k);
            }
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            u32x4 term[3];
            split8(w0[u], w1[u], term[0], term[1], term[2]);
#pragma unroll
            for (int i = 0; i < TT; ++i)
#pragma unroll
                for (int m = 0; m < 3; ++m)
                    acc[i] = SkinnyBf16::mma(term[m], b[u][i], acc[i]);
        }
    } else {
        const int ke = min(kb + 32 * U, (d + 31) / 32 * 32);
        if (kb < ke)
            skinny_mma<S, TT, 1, 1>(w, xt, 0, kb, ke, d, d, acc);
    }
}

// P[s][t][64 Q]: partial scores of the s-th range of d, expert e at column
// (e mod 64) Q + e / 64. grid: (tiles of 16 experts, ranges); the waves take
// quarters of the range.
template <typename S, int TT>
__global__ __launch_bounds__(kThreads) void few_scores_kernel(
    const typename S::type *__restrict__ x, const float *__restrict__ wg, int N, int d, int E,
    float *__restrict__ P) {
    __shared__ f32x4 part[kWaves][TT][64];
    const int lane = threadIdx.x & 63, wv = threadIdx.x >> 6;
    const int e0 = blockIdx.x * 16;
    const float *w = wg + (int64_t)min(e0 + (lane & 15), E - 1) * d;
    const typename S::type *xt[TT];
#pragma unroll
    for (int i = 0; i < TT; ++i)
        xt[i] = x + (int64_t)min(i * 16 + (lane & 15), N - 1) * d;
    const int kb = blockIdx.y * kScoreRange + wv * (kScoreRange / kWaves);
    f32x4 acc[TT];
    score_tile<S, TT, kScoreRange / kWaves / 32>(w, xt, kb, d, acc);
#pragma unroll
    for (int i = 0; i < TT; ++i)
        part[wv][i][lane] = acc[i];
    __syncthreads();
    const int Q = score_lanes(E);
    for (int q = threadIdx.x; q < TT * 64; q += kThreads) {
        const int i = q >> 6, l = q & 63;
        const int t = i * 16 + (l & 15), e = e0 + 4 * (l >> 4);
        f32x4 v = part[0][i][l];
#pragma unroll
        for (int s = 1; s < kWaves; ++s)
            v += part[s][i][l];
        if (t < N)
#pragma unroll
            for (int c = 0; c < 4; ++c)
                if (e + c < E)
                    P[((int64_t)blockIdx.y * N + t) * (64 * Q) + (e + c) % 64 * Q + (e + c) / 64] =
                        v[c];
    }
}

// One wave ranks token t: partial scores added in range order, noise, top-k
// and softmax of the kept scores into idx[t k ..] and gate[t k ..].
template <int Q>
__device__ __forceinline__ void few_rank(const float *__restrict__ P, int ns,
                                         const float *__restrict__ noise, int N, int E, int k,
                                         int t, int32_t *idx, float *gate) {
    typedef float vec __attribute__((ext_vector_type(Q == 1 ? 2 : Q)));   // (Q == 1: v[0])
    const int lane = __lane_id();
    const float *p = P + ((int64_t)t * 64 + lane) * Q;
    const int64_t step = (int64_t)N * 64 * Q;
    auto load = [&](int r) {
        vec o = {};
        if constexpr (Q == 1)
            o[0] = p[r * step];
        else
            o = *reinterpret_cast<const vec *>(p + r * step);
        return o;
    };
    constexpr int B = 8;   // loads in flight
    vec s = load(0);
    for (int r = 1; r < ns; r += B) {
        vec u[B];
#pragma unroll
        for (int c = 0; c < B; ++c)
            u[c] = load(min(r + c, ns - 1));
#pragma unroll
        for (int c = 0; c < B; ++c)
            if (r + c < ns)
                s += u[c];
    }
    float v[Q];
#pragma unroll
    for (int q = 0; q < Q; ++q) {
        const int e = lane + 64 * q;
        v[q] = -INFINITY;
        if (e < E)   // (columns past E hold no score)
            v[q] = noise ? s[q] + noise[(int64_t)t * E + e] : s[q];
    }
    topk_softmax_wave<Q>(v, E, k, t, true, idx, gate);
}

template <int Q>
__global__ __launch_bounds__(kThreads) void few_rank_kernel(const float *__restrict__ P, int ns,
                                                            const float *__restrict__ noise, int N,
                                                            int E, int k, int32_t *idx,
                                                            float *gate) {
    const int t = blockIdx.x * kWaves + (threadIdx.x >> 6);
    if (t < N)
        few_rank<Q>(P, ns, noise, N, E, k, t, idx, gate);
}

// ---- plan --------------------------------------------------------------

struct FewRoute {
    const float *P, *noise;   // partial scores to rank, or P NULL: ranked already
    int ns;
    int32_t *idx;             // [N, k]
    float *gate;
    int32_t *slot;            // [N, k]
    int32_t *used, *demand, *drops;   // exports, or NULL
    float *gate_sum;
    FewPlan *plan;
    int *done;                // finished ranges per column block of the down product
    int blocks;               // column blocks
};

// Layers whose scores the plan's workgroup computes itself, wave w taking
// K-steps w, w + 16, ...: up to 16 tokens and experts, rows of up to 1024.
constexpr int kPlanScoreWidth = 2 * kPlanWaves * 32;
bool scores_in_plan(int64_t N, int64_t d, int64_t E) {
    return N <= 16 && E <= 16 && d <= kPlanScoreWidth;
}

// One workgroup: scores (SCORE, see above), idx and gates (with SCORE, or when
// P is given), then the plan: the hit
// experts in ascending order, the rows each keeps (the first `cap` of its
// assignments in (choice, token) order) and the exports.
template <typename S, int Q, bool SCORE>
__global__ __launch_bounds__(kPlanWaves * 64) void few_plan_kernel(
    const typename S::type *__restrict__ x, const float *__restrict__ wg, FewRoute r, int N, int d,
    int E, int k, int cap) {
    constexpr int nthr = kPlanWaves * 64;
    static_assert(kFewAssign <= nthr && kMaxExperts <= nthr, "a thread per assignment and expert");
    __shared__ __attribute__((aligned(16))) unsigned char id[kFewAssign];   // see below
    __shared__ int32_t s_idx[kFewAssign];      // [N, k]
    __shared__ float s_gate[kFewAssign];
    __shared__ float by_expert[kFewAssign];    // gates, expert by expert
    __shared__ int count[kMaxExperts], hit_of[kMaxExperts], first[kMaxExperts];
    __shared__ int hits_w[kMaxExperts / 64], count_w[kMaxExperts / 64];
    const int tid = threadIdx.x, lane = tid & 63, wv = tid >> 6, A = N * k;
    if (tid < kMaxExperts)
        count[tid] = 0;
    for (int i = tid; i < r.blocks; i += nthr)
        r.done[i] = 0;
    const bool rank_here = SCORE || r.P;
    if constexpr (SCORE) {
        __shared__ f32x4 part[kPlanWaves][64];
        __shared__ float score[16][64];   // [token][expert]
        const float *w = wg + (int64_t)min(lane & 15, E - 1) * d;
        const typename S::type *xt[1] = {x + (int64_t)min(lane & 15, N - 1) * d};
        f32x4 a, b, c[1];
        score_tile<S, 1, 1>(w, xt, wv * 32, d, c);
        a = c[0];
        score_tile<S, 1, 1>(w, xt, (kPlanWaves + wv) * 32, d, c);
        b = c[0];
        part[wv][lane] = a + b;
        __syncthreads();
        if (wv < 4) {
            // lane: expert 4 wv + q of token l % 16 ... one value per thread
            const int l = (lane >> 2) + 16 * wv, q = lane & 3;
            float v = part[0][l][q];
#pragma unroll
            for (int u = 1; u < kPlanWaves; ++u)
                v += part[u][l][q];
            score[l & 15][4 * (l >> 4) + q] = v;
        }
        __syncthreads();
        if (wv < N)
            few_rank<1>(&score[0][0], 1, r.noise, N, E, k, wv, s_idx, s_gate);
    } else if (r.P) {
        for (int t = wv; t < N; t += kPlanWaves)
            few_rank<Q>(r.P, r.ns, r.noise, N, E, k, t, s_idx, s_gate);
    }
    __syncthreads();
    // thread o: assignment (j, t), o = j N + t, so that threads follow the
    // order in which capacity is given; id[o] is its expert
    const int o = tid, j = o / N, i = (o - j * N) * k + j;
    int e = 0;
    float g = 0.f;
    if (o < A) {
        if (rank_here) {
            e = s_idx[i];
            g = s_gate[i];
            r.idx[i] = e;
            r.gate[i] = g;
        } else {
            e = r.idx[i];
            g = r.gate[i];
        }
        id[o] = (unsigned char)e;
        atomicAdd(&count[e], 1);
    }
    __syncthreads();
    // rank: assignments before o to the same expert, the bytes equal to e in
    // id[0 .. o), four at a time (v has a zero byte for each; the bit trick
    // leaves bit 7 of exactly the zero bytes)
    int rank = 0;
    if (o < A) {
        const unsigned ee = (unsigned)e * 0x01010101u;
        auto equal = [&](unsigned v) {
            v ^= ee;
            return ~(((v & 0x7f7f7f7fu) + 0x7f7f7f7fu) | v | 0x7f7f7f7fu);
        };
        const u32x4 *quad = reinterpret_cast<const u32x4 *>(id);
        for (int c = 0; c < o / 16; ++c) {
            const u32x4 v = quad[c];
            rank += __popc(equal(v[0])) + __popc(equal(v[1])) + __popc(equal(v[2])) +
                    __popc(equal(v[3]));
        }
        const unsigned *word = reinterpret_cast<const unsigned *>(id);
        for (int c = o / 16 * 4; c < o / 4; ++c)
            rank += __popc(equal(word[c]));
        if (o % 4)
            rank += __popc(equal(word[o / 4]) & ((1u << (8 * (o % 4))) - 1u));
    }
    // hit experts in ascending order, and the assignments before each expert
    int n = 0, before = 0;
    uint64_t hits = 0;
    if (tid < kMaxExperts) {
        n = count[tid];
        hits = __ballot(n > 0);
        before = n;
#pragma unroll
        for (int s = 1; s < 64; s <<= 1) {
            const int u = __shfl_up(before, s);
            if (lane >= s)
                before += u;
        }
        if (lane == 63) {
            hits_w[wv] = __popcll(hits);
            count_w[wv] = before;
        }
        before -= n;
    }
    __syncthreads();
    if (tid < kMaxExperts) {
        int a = __popcll(hits & lanemask_lt());
        for (int w = 0; w < wv; ++w) {
            a += hits_w[w];
            before += count_w[w];
        }
        hit_of[tid] = a;
        first[tid] = before;
        if (n > 0) {
            r.plan->expert[a] = tid;
            r.plan->rows[a] = min(n, cap);
        }
        if (tid < E) {
            if (r.used) r.used[tid] = min(n, cap);
            if (r.demand) r.demand[tid] = n;
            if (r.drops) r.drops[tid] = n - min(n, cap);
        }
        if (tid == 0) {
            int c = 0;
            for (int w = 0; w < kMaxExperts / 64; ++w)
                c += hits_w[w];
            r.plan->nhit = c;
        }
    }
    __syncthreads();
    if (o < A) {
        if (rank < cap)
            r.plan->row[hit_of[e]][rank] = i;
        r.slot[i] = rank < cap ? rank : -1;
        by_expert[first[e] + rank] = g;
    }
    if (r.gate_sum) {   // (the same for the whole workgroup)
        __syncthreads();
        if (tid < E) {
            float s = 0.f;   // in (choice, token) order
            for (int c = 0; c < n; ++c)
                s += by_expert[first[tid] + c];
            r.gate_sum[tid] = s;
        }
    }
}

// ---- up ----------------------------------------------------------------

// H (bf16: two terms, [2][N k][d_ff]; fp32: [N k][d_ff]) = act(W_up[e] x +
// b_up[e]) for the rows of the hit experts. grid: (tiles of 16 neurons,
// min(E, N k)); TT token tiles at most.
template <typename S, int TT>
__global__ __launch_bounds__(kThreads, 4) void few_up_kernel(
    const typename S::type *__restrict__ x, const typename S::type *__restrict__ w_up,
    const float *__restrict__ b_up, const FewPlan *__restrict__ plan, int N, int d, int d_ff,
    int k, int act, typename S::type *__restrict__ H) {
    __shared__ f32x4 part[kWaves][TT][64];
    const int a = blockIdx.y, f0 = blockIdx.x * 16;
    if (a >= plan->nhit)
        return;
    const int rows = plan->rows[a], e = plan->expert[a];
    const int *row = plan->row[a];
    const int lane = threadIdx.x & 63, wv = threadIdx.x >> 6;
    const int ntile = (rows + 15) / 16;
    const typename S::type *w = w_up + ((int64_t)e * d_ff + min(f0 + (lane & 15), d_ff - 1)) * d;
    // this wave's K range, in steps of 32
    const int steps = (d + 31) / 32;
    const int kb = (int)((int64_t)wv * steps / kWaves) * 32;
    const int ke = (int)((int64_t)(wv + 1) * steps / kWaves) * 32;
    auto run = [&](auto tiles) {
        constexpr int T = decltype(tiles)::value;
        const typename S::type *xt[T];
        f32x4 c[T];
#pragma unroll
        for (int i = 0; i < T; ++i) {
            const int r = i * 16 + (lane & 15);
            xt[i] = x + (int64_t)(row[r < rows ? r : 0] / k) * d;
            c[i] = f32x4{0.f, 0.f, 0.f, 0.f};
        }
        // operand registers of a batch: U (1 + T) fragments, twice
        constexpr int U = (T == 1 ? 8 : T == 2 ? 4 : 2) / (Kind<S>::bf16 ? 1 : 2);
        skinny_mma<S, T, 1, U>(w, xt, 0, kb, ke, d, d, c);
#pragma unroll
        for (int i = 0; i < T; ++i)
            part[wv][i][lane] = c[i];
    };
    if (TT == 1 || ntile <= 1)
        run(std::integral_constant<int, 1>{});
    else if (TT == 2 || ntile <= 2)
        run(std::integral_constant<int, TT < 2 ? TT : 2>{});
    else
        run(std::integral_constant<int, TT>{});
    __syncthreads();
    // thread -> (row, 4 neurons): tile i's lane l holds neurons 4 (l / 16) + q
    // of row l % 16
    for (int q = threadIdx.x; q < ntile * 64; q += kThreads) {
        const int i = q >> 6, l = q & 63;
        const int r = i * 16 + (l & 15), f = f0 + 4 * (l >> 4);
        if (r >= rows || f >= d_ff)
            continue;
        f32x4 z = part[0][i][l];
#pragma unroll
        for (int s = 1; s < kWaves; ++s)
            z += part[s][i][l];
        if (b_up)
            z += load4<Kind<S>::bf16>(b_up + (int64_t)e * d_ff + f, d_ff - f);
#pragma unroll
        for (int c = 0; c < 4; ++c)
            z[c] = activate(z[c], act);
        typename S::type *dst = H + (int64_t)row[r] * d_ff + f;
        if constexpr (Kind<S>::bf16) {
            float lo[4];
#pragma unroll
            for (int c = 0; c < 4; ++c)
                lo[c] = second_term(z[c]);
            *reinterpret_cast<u32x2 *>(dst) =
                u32x2{pack_bf16x2(z[0], z[1]), pack_bf16x2(z[2], z[3])};
            *reinterpret_cast<u32x2 *>(dst + (int64_t)N * k * d_ff) =
                u32x2{pack_bf16x2(lo[0], lo[1]), pack_bf16x2(lo[2], lo[3])};
        } else {
#pragma unroll
            for (int c = 0; c < 4; ++c)
                if (f + c < d_ff)
                    dst[c] = z[c];
        }
    }
}

// ---- down --------------------------------------------------------------

// out[t] = sum over kept choices of gate (W_down[e] h + b_down[e]). grid:
// (blocks of 16 columns, ranges); part [ranges][N][16 blocks] when there is
// more than one range. The partial sums and the counter are written and read
// past the XCD's own L2 (agent scope), which other XCDs do not see.
template <typename S, int TT>
__global__ __launch_bounds__(kThreads, 4) void few_down_kernel(
    const typename S::type *__restrict__ H, const typename S::type *__restrict__ w_down,
    const float *__restrict__ b_down, const float *__restrict__ gate,
    const FewPlan *__restrict__ plan, int N, int d, int d_ff, int k, int *__restrict__ done,
    float *__restrict__ part, typename S::type *__restrict__ out) {
    constexpr int NT = TT * 16;
    constexpr int NB = Kind<S>::terms;
    constexpr int CB = 16;
    __shared__ float sum[kWaves][NT][CB + 1];
    __shared__ int last;
    const int c0 = blockIdx.x * CB;
    const int lane = threadIdx.x & 63;
    const int wv = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    for (int i = lane; i < NT * (CB + 1); i += 64)
        (&sum[wv][0][0])[i] = 0.f;
    const int chunks = (d_ff + kChunk - 1) / kChunk;
    const int units = plan->nhit * chunks;
    const int parts = (int)gridDim.y * kWaves, me = (int)blockIdx.y * kWaves + wv;
    const int ub = (int)((int64_t)me * units / parts);
    const int ue = (int)((int64_t)(me + 1) * units / parts);
    const int64_t lo = (int64_t)N * k * d_ff;
    for (int u = ub; u < ue;) {
        const int a = u / chunks, uc = u - a * chunks;
        const int un = min(ue - u, chunks - uc);   // chunks of this expert
        const int e = plan->expert[a], rows = plan->rows[a];
        const typename S::type *w =
            w_down + ((int64_t)e * d + min(c0 + (lane & 15), d - 1)) * d_ff;
        const int kb = uc * kChunk, ke = min((uc + un) * kChunk, (d_ff + 31) / 32 * 32);
        u += un;
        const int cc = c0 + 4 * (lane >> 4);
        f32x4 bias = {0.f, 0.f, 0.f, 0.f};
        if (b_down && uc == 0)
            bias = load4<Kind<S>::bf16>(b_down + (int64_t)e * d + cc, d - cc);
        auto run = [&](auto tiles) {
            constexpr int T = decltype(tiles)::value;
            const typename S::type *ht[T];
            f32x4 acc[T];
            int as[T];
#pragma unroll
            for (int i = 0; i < T; ++i) {
                const int r = i * 16 + (lane & 15);
                as[i] = plan->row[a][r < rows ? r : 0];
                ht[i] = H + (int64_t)as[i] * d_ff;
                acc[i] = bias;
            }
            constexpr int U = NB * T <= 2 ? 4 : NB * T <= 4 ? 2 : 1;
            skinny_mma<S, T, NB, U>(w, ht, lo, kb, ke, d_ff, d_ff, acc);
#pragma unroll
            for (int i = 0; i < T; ++i) {
                if (i * 16 + (lane & 15) < rows) {
                    const float g = gate[as[i]];
                    float *s = &sum[wv][as[i] / k][4 * (lane >> 4)];
#pragma unroll
                    for (int q = 0; q < 4; ++q)
                        s[q] = fmaf(g, acc[i][q], s[q]);
                }
            }
        };
        if (NB == 2 && rows <= 8) {
            // both terms of up to 8 rows fill one tile: columns 0-7 the hi
            // terms, columns 8-15 the lo terms of the same rows, added at the
            // end (half the loads and MFMAs of two operand terms)
            const int r = lane & 7;
            const int as = plan->row[a][r < rows ? r : 0];
            const typename S::type *ht[1] = {H + (int64_t)as * d_ff + (lane & 8 ? lo : 0)};
            f32x4 acc[1] = {lane & 8 ? f32x4{0.f, 0.f, 0.f, 0.f} : bias};
            skinny_mma<S, 1, 1, 8>(w, ht, 0, kb, ke, d_ff, d_ff, acc);
            const float g = gate[as];
            float *s = &sum[wv][as / k][4 * (lane >> 4)];
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                const float y = acc[0][q] + __shfl_xor(acc[0][q], 8);
                if ((lane & 15) < rows)
                    s[q] = fmaf(g, y, s[q]);
            }
        } else if (TT == 1 || rows <= 16) {
            run(std::integral_constant<int, 1>{});
        } else if (TT == 2 || rows <= 32) {
            run(std::integral_constant<int, TT < 2 ? TT : 2>{});
        } else {
            run(std::integral_constant<int, TT>{});
        }
    }
    __syncthreads();
    auto wave_sums = [&](int t, int c) {
        float v = sum[0][t][c];
#pragma unroll
        for (int w = 1; w < kWaves; ++w)
            v += sum[w][t][c];
        return v;
    };
    auto store = [&](int t, int c, float lo_v, float hi_v) {
        // columns c and c + 1 of token t
        if constexpr (Kind<S>::bf16) {
            if (c0 + c < d)   // (d % 8 == 0)
                *reinterpret_cast<unsigned *>(out + (int64_t)t * d + c0 + c) =
                    pack_bf16x2(lo_v, hi_v);
        } else {
            if (c0 + c < d)
                out[(int64_t)t * d + c0 + c] = lo_v;
            if (c0 + c + 1 < d)
                out[(int64_t)t * d + c0 + c + 1] = hi_v;
        }
    };
    const int ranges = gridDim.y;
    if (ranges == 1) {
        for (int i = threadIdx.x; i < N * (CB / 2); i += kThreads) {
            const int t = i / (CB / 2), c = 2 * (i % (CB / 2));
            store(t, c, wave_sums(t, c), wave_sums(t, c + 1));
        }
        return;
    }
    const int64_t ld = (int64_t)gridDim.x * CB;   // columns of a partial row
    float *mine = part + (int64_t)blockIdx.y * N * ld + c0;
    for (int i = threadIdx.x; i < N * CB; i += kThreads) {
        const int t = i / CB, c = i % CB;
        __hip_atomic_store(mine + t * ld + c, wave_sums(t, c), __ATOMIC_RELAXED,
                           __HIP_MEMORY_SCOPE_AGENT);
    }
    // Every partial sum of the workgroup has reached memory before it counts
    // (agent-scope stores write through; the wait is for their completion). A
    // release fence instead would write back, and an acquire drop, the whole
    // L2 for every workgroup: 222 against 47 us at the Mixtral-shaped layer.
    asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
    __syncthreads();
    if (threadIdx.x == 0)
        last = __hip_atomic_fetch_add(done + blockIdx.x, 1, __ATOMIC_RELAXED,
                                      __HIP_MEMORY_SCOPE_AGENT) == ranges - 1;
    __syncthreads();
    if (!last)
        return;
    for (int i = threadIdx.x; i < N * (CB / 2); i += kThreads) {
        const int t = i / (CB / 2), c = 2 * (i % (CB / 2));
        const float *p = part + t * ld + c0 + c;
        float v0 = 0.f, v1 = 0.f;
#pragma unroll 8
        for (int s = 0; s < ranges; ++s) {
            v0 += __hip_atomic_load(p + s * N * ld, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
            v1 += __hip_atomic_load(p + s * N * ld + 1, __ATOMIC_RELAXED,
                                    __HIP_MEMORY_SCOPE_AGENT);
        }
        store(t, c, v0, v1);
    }
}

// ---- tiled products ------------------------------------------------------

// One expert's product on the tiled form, 64 rows by kTileCols columns. UP:
// H = act(W x + bias) as above, A the rows of x. Otherwise Y[range][assignment]
// = W h + bias (bias in range 0), fp32: A holds both terms of the rows, 16 hi
// and 16 lo rows per wave, whose products the same lane adds. K: row length of
// W, cols: its rows. grid: (column tiles, min(E, N k), K-ranges). Stages are few
// enough for two workgroups on a CU: one's products cover the other's waits
// (Mixtral-shaped layer, 64 tokens: 398 us with one of 5 and 4 stages, 375 with
// two; the weights alone are 313 us at 6 TB/s).
constexpr int kTileCols = 128;
template <bool UP>
__global__ __launch_bounds__(512) void few_tile_kernel(
    const unsigned short *__restrict__ A, const unsigned short *__restrict__ W,
    const float *__restrict__ bias, const FewPlan *__restrict__ plan, int N, int K, int cols,
    int k, int act, unsigned short *__restrict__ H, float *__restrict__ Y) {
    typedef TileProduct<UP ? 64 : 128, kTileCols, 4, 2, UP ? 3 : 2, false, false> Tile;
    static_assert(kFewTokens <= 64 && Tile::THREADS == 512, "an expert's rows fit the tile");
    __shared__ __attribute__((aligned(1024))) char smem[Tile::LDS];
    __shared__ int row[64];
    const int a = blockIdx.y, n0 = blockIdx.x * kTileCols;
    if (a >= plan->nhit)
        return;
    const int rows = plan->rows[a], e = plan->expert[a];
    const int lane = threadIdx.x & 63;
    const int wv = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    if (threadIdx.x < 64)
        row[threadIdx.x] = plan->row[a][threadIdx.x < rows ? threadIdx.x : 0];
    __syncthreads();
    const int64_t lo = (int64_t)N * k * K;   // of the second term (down)
    const int KT = (K + kStep - 1) / kStep;
    const int kb = (int)((int64_t)blockIdx.z * KT / gridDim.z);
    const int ke = (int)((int64_t)(blockIdx.z + 1) * KT / gridDim.z);
    const unsigned short *We = W + (int64_t)e * cols * K;
    f32x4 acc[Tile::FM][Tile::FN];
#pragma unroll
    for (int i = 0; i < Tile::FM; ++i)
#pragma unroll
        for (int j = 0; j < Tile::FN; ++j)
            acc[i][j] = f32x4{0.f, 0.f, 0.f, 0.f};
    Tile::run(
        smem,
        [&](int r) {
            if constexpr (UP)
                return A + (int64_t)(row[r] / k) * K;
            else
                return A + (int64_t)row[r / 32 * 16 + r % 16] * K + (r & 16 ? lo : 0);
        },
        0, [&](int c) { return We + (int64_t)min(n0 + c, cols - 1) * K; }, 0, K, kb, ke, acc);
    // lane: one row, 16 adjacent columns
    const int r = wv / 2 * 16 + (lane & 15);
    const int n = n0 + wv % 2 * 64 + 16 * (lane >> 4);
    if (r >= rows || n >= cols)
        return;
    float v[16];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        f32x4 t = acc[0][j];
        if constexpr (!UP)
            t += acc[Tile::FM - 1][j];
        if (bias && blockIdx.z == 0 && n + 4 * j < cols)
            t += *reinterpret_cast<const f32x4 *>(bias + (int64_t)e * cols + n + 4 * j);
#pragma unroll
        for (int q = 0; q < 4; ++q)
            v[4 * j + q] = t[q];
    }
    const int64_t o = (int64_t)row[r] * cols + n;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        if (n + 8 * h >= cols)   // (cols % 8 == 0)
            continue;
        float *p = &v[8 * h];
        if constexpr (UP) {
            u32x4 hi, low;
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                float z[2], rest[2];
#pragma unroll
                for (int c = 0; c < 2; ++c) {
                    z[c] = activate(p[2 * q + c], act);
                    rest[c] = second_term(z[c]);
                }
                hi[q] = pack_bf16x2(z[0], z[1]);
                low[q] = pack_bf16x2(rest[0], rest[1]);
            }
            *reinterpret_cast<u32x4 *>(H + o + 8 * h) = hi;
            *reinterpret_cast<u32x4 *>(H + (int64_t)N * k * cols + o + 8 * h) = low;
        } else {
            float *dst = Y + (int64_t)blockIdx.z * N * k * cols + o + 8 * h;
            *reinterpret_cast<f32x4 *>(dst) = f32x4{p[0], p[1], p[2], p[3]};
            *reinterpret_cast<f32x4 *>(dst + 4) = f32x4{p[4], p[5], p[6], p[7]};
        }
    }
}

// out[t] = sum over kept choices, in choice order, of gate * the sum of its
// row's ranges. 8 columns per thread.
__global__ __launch_bounds__(256) void few_combine_kernel(
    const float *__restrict__ Y, int ranges, const float *__restrict__ gate,
    const int32_t *__restrict__ slot, int N, int d, int k, unsigned short *__restrict__ out) {
    const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
    const int per = d / 8;
    if (i >= (int64_t)N * per)
        return;
    const int t = (int)(i / per), c = (int)(i - (int64_t)t * per) * 8;
    const int64_t step = (int64_t)N * k * d;
    f32x4 s0 = {0.f, 0.f, 0.f, 0.f}, s1 = s0;
    for (int j = 0; j < k; ++j) {
        const int as = t * k + j;
        if (slot[as] < 0)
            continue;
        const float *p = Y + (int64_t)as * d + c;
        f32x4 y0 = *reinterpret_cast<const f32x4 *>(p), y1 = *reinterpret_cast<const f32x4 *>(p + 4);
        for (int r = 1; r < ranges; ++r) {
            y0 += *reinterpret_cast<const f32x4 *>(p + r * step);
            y1 += *reinterpret_cast<const f32x4 *>(p + r * step + 4);
        }
        const float g = gate[as];
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            s0[q] = fmaf(g, y0[q], s0[q]);
            s1[q] = fmaf(g, y1[q], s1[q]);
        }
    }
    *reinterpret_cast<u32x4 *>(out + (int64_t)t * d + c) =
        u32x4{pack_bf16x2(s0[0], s0[1]), pack_bf16x2(s0[2], s0[3]), pack_bf16x2(s1[0], s1[1]),
              pack_bf16x2(s1[2], s1[3])};
}

// Whether the experts' products run on the tiled form: bf16 layers of about 8
// rows per expert on average or more (Mixtral-shaped layer: 379 against 421 us at
// 32 tokens and 375 against 579 at 64; below, 385 against 382 at 24).
bool tiled(bool bf16, int64_t N, int64_t E, int k) { return bf16 && N * k > 7 * E; }

// Ranges of the tiled down product's reduction: about two workgroups per CU,
// each of at least 8 K-steps.
int tiled_ranges(int64_t N, int64_t d, int64_t E, int64_t d_ff, int k) {
    const int64_t blocks = (d + kTileCols - 1) / kTileCols * std::min<int64_t>(E, N * k);
    const int64_t r = std::min<int64_t>(512 / blocks, (d_ff + kStep - 1) / kStep / 8);
    return (int)std::min<int64_t>(std::max<int64_t>(r, 1), 8);
}

// Column blocks and ranges of the down product: about 4096 workgroups, each
// wave with at least two chunks when every possible expert is hit.
struct DownGrid {
    int blocks, ranges;
};
DownGrid down_grid(int64_t N, int64_t d, int64_t E, int64_t d_ff, int k) {
    const int64_t hits = std::min<int64_t>(E, N * k);
    DownGrid g;
    g.blocks = (int)((d + 15) / 16);
    const int64_t units = hits * ((d_ff + kChunk - 1) / kChunk);
    const int64_t r = std::min<int64_t>((4096 + g.blocks - 1) / g.blocks, units / (2 * kWaves));
    g.ranges = (int)std::min<int64_t>(std::max<int64_t>(r, 1), 64);
    return g;
}
int score_ranges(int64_t d) { return (int)((d + kScoreRange - 1) / kScoreRange); }

size_t up256(size_t v) { return (v + 255) / 256 * 256; }

}  // namespace

FewLayout few_layout(bool bf16, int64_t N, int64_t d, int64_t E, int64_t d_ff, int k) {
    FewLayout L;
    size_t o = 0;
    const size_t nk = (size_t)(N * k);
    L.idx = o;    o += up256(nk * 4);
    L.gate = o;   o += up256(nk * 4);
    L.slot = o;   o += up256(nk * 4);
    L.plan = o;   o += up256(sizeof(FewPlan));
    L.done = o;   o += up256((size_t)((d + 15) / 16) * 4);
    L.scores = o; o += up256((size_t)score_ranges(d) * N * 64 * score_lanes((int)E) * 4);
    L.H = o;      o += up256(nk * d_ff * 4);   // fp32, or two bf16 terms
    const DownGrid g = down_grid(N, d, E, d_ff, k);
    const size_t joined = (size_t)g.ranges * N * g.blocks * 16 * 4;
    const size_t rows = tiled(bf16, N, E, k)
                            ? (size_t)tiled_ranges(N, d, E, d_ff, k) * nk * d * 4 : 0;
    L.part = o;   o += up256(std::max(joined, rows));
    L.total = o;
    return L;
}

template <typename S, int TT>
static hipError_t few_call(const void *xv, const float *wg, const float *noise, const void *wu,
                           const void *wd, const float *b_up, const float *b_down, int N, int d,
                           int E, int d_ff, int k, int cap, int act, char *ws, FewRoute r,
                           void *out, hipStream_t s) {
    typedef typename S::type T;
    const FewLayout L = few_layout(Kind<S>::bf16, N, d, E, d_ff, k);
    const T *x = static_cast<const T *>(xv);
    float *P = reinterpret_cast<float *>(ws + L.scores);
    T *H = reinterpret_cast<T *>(ws + L.H);
    const int ns = score_ranges(d);
    const DownGrid g = down_grid(N, d, E, d_ff, k);
    const unsigned hits = (unsigned)std::min(E, N * k);
    r.plan = reinterpret_cast<FewPlan *>(ws + L.plan);
    r.done = reinterpret_cast<int *>(ws + L.done);
    r.blocks = g.blocks;
    r.noise = noise;
    r.ns = ns;
    hipError_t err = hipSuccess;
    const bool score = scores_in_plan(N, d, E);
    if (!score) {
        hipLaunchKernelGGL((few_scores_kernel<S, TT>),
                           dim3((unsigned)((E + 15) / 16), (unsigned)ns), dim3(kThreads), 0, s, x,
                           wg, N, d, E, P);
        err = hipGetLastError();
        if (err != hipSuccess)
            return err;
    }
    // The plan's one workgroup ranks a token per wave, so more than its 16 waves'
    // worth are ranked by a launch of their own, spread over the CUs (64 tokens,
    // 64 experts, k = 8: 21 us inside, 4 + 6 us apart).
    const int Q = score_lanes(E);
    const bool inside = N <= kPlanWaves;
    r.P = inside ? P : nullptr;
    auto rank_and_plan = [&](auto lanes) {
        constexpr int QQ = decltype(lanes)::value;
        if (!inside) {
            hipLaunchKernelGGL(few_rank_kernel<QQ>, dim3((unsigned)((N + kWaves - 1) / kWaves)),
                               dim3(kThreads), 0, s, (const float *)P, ns, noise, N, E, k, r.idx,
                               r.gate);
            const hipError_t rc = hipGetLastError();
            if (rc != hipSuccess)
                return rc;
        }
        if (QQ == 1 && TT == 1 && score)
            hipLaunchKernelGGL((few_plan_kernel<S, 1, true>), dim3(1), dim3(kPlanWaves * 64), 0, s,
                               x, wg, r, N, d, E, k, cap);
        else
            hipLaunchKernelGGL((few_plan_kernel<S, QQ, false>), dim3(1), dim3(kPlanWaves * 64), 0,
                               s, x, wg, r, N, d, E, k, cap);
        return hipGetLastError();
    };
    err = Q == 1   ? rank_and_plan(std::integral_constant<int, 1>{})
          : Q == 2 ? rank_and_plan(std::integral_constant<int, 2>{})
                   : rank_and_plan(std::integral_constant<int, 4>{});
    if (err != hipSuccess)
        return err;
    if constexpr (Kind<S>::bf16) {
        if (tiled(true, N, E, k)) {
            const int tr = tiled_ranges(N, d, E, d_ff, k);
            float *Y = reinterpret_cast<float *>(ws + L.part);
            hipLaunchKernelGGL(few_tile_kernel<true>,
                               dim3((unsigned)((d_ff + kTileCols - 1) / kTileCols), hits),
                               dim3(512), 0, s, x, static_cast<const T *>(wu), b_up,
                               (const FewPlan *)r.plan, N, d, d_ff, k, act, H, (float *)nullptr);
            err = hipGetLastError();
            if (err != hipSuccess)
                return err;
            hipLaunchKernelGGL(
                few_tile_kernel<false>,
                dim3((unsigned)((d + kTileCols - 1) / kTileCols), hits, (unsigned)tr), dim3(512), 0,
                s, (const T *)H, static_cast<const T *>(wd), b_down, (const FewPlan *)r.plan, N,
                d_ff, d, k, act, (T *)nullptr, Y);
            err = hipGetLastError();
            if (err != hipSuccess)
                return err;
            hipLaunchKernelGGL(few_combine_kernel,
                               dim3((unsigned)(((int64_t)N * (d / 8) + 255) / 256)), dim3(256), 0,
                               s, (const float *)Y, tr, (const float *)r.gate,
                               (const int32_t *)r.slot, N, d, k, static_cast<T *>(out));
            return hipGetLastError();
        }
    }
    hipLaunchKernelGGL((few_up_kernel<S, TT>), dim3((unsigned)((d_ff + 15) / 16), hits),
                       dim3(kThreads), 0, s, x, static_cast<const T *>(wu), b_up,
                       (const FewPlan *)r.plan, N, d, d_ff, k, act, H);
    err = hipGetLastError();
    if (err != hipSuccess)
        return err;
    hipLaunchKernelGGL((few_down_kernel<S, TT>), dim3((unsigned)g.blocks, (unsigned)g.ranges),
                       dim3(kThreads), 0, s, (const T *)H, static_cast<const T *>(wd), b_down,
                       (const float *)r.gate, (const FewPlan *)r.plan, N, d, d_ff, k, r.done,
                       reinterpret_cast<float *>(ws + L.part), static_cast<T *>(out));
    return hipGetLastError();
}

hipError_t launch_few(bool bf16, bool aligned, const void *x, const float *wg, const float *noise,
                      const void *w_up, const void *w_down, const float *b_up,
                      const float *b_down, int64_t N, int64_t d, int E, int64_t d_ff, int k,
                      int64_t ceff, int act, void *ws, int32_t *idx, float *gate, int32_t *slot,
                      int32_t *used, int32_t *demand, int32_t *drops, float *gate_sum, void *out,
                      hipStream_t s) {
    char *w = static_cast<char *>(ws);
    const FewLayout L = few_layout(bf16, N, d, E, d_ff, k);
    FewRoute r{};
    r.idx = idx ? idx : reinterpret_cast<int32_t *>(w + L.idx);
    r.gate = gate ? gate : reinterpret_cast<float *>(w + L.gate);
    r.slot = slot ? slot : reinterpret_cast<int32_t *>(w + L.slot);
    r.used = used;
    r.demand = demand;
    r.drops = drops;
    r.gate_sum = gate_sum;
    auto go = [&](auto kind, auto tiles) {
        return few_call<decltype(kind), decltype(tiles)::value>(
            x, wg, noise, w_up, w_down, b_up, b_down, (int)N, (int)d, E, (int)d_ff, k, (int)ceff,
            act, w, r, out, s);
    };
    auto with_tiles = [&](auto kind) {
        if (N <= 16)
            return go(kind, std::integral_constant<int, 1>{});
        if (N <= 32)
            return go(kind, std::integral_constant<int, 2>{});
        return go(kind, std::integral_constant<int, 4>{});
    };
    if (bf16)
        return with_tiles(SkinnyBf16{});
    // fp32 rows are read 16 bytes at a time where every row starts aligned
    if (aligned && d % 4 == 0 && d_ff % 4 == 0)
        return with_tiles(SkinnyF32<true>{});
    return with_tiles(SkinnyF32<false>{});
}

}  // namespace moe
