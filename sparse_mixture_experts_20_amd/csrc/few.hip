// The MoE layer for a few tokens (at most kFewMaxTokens), the form a decoding
// step needs. Page 1 ("Mixture of Experts (MoE) 12段階極小ビジュアル解剖
// シミュレーター"), STEP 1-12; nanoMoE slides 11-40: the same layer as the
// grouped path, token for token.
//
// With a few tokens every expert that is hit serves a handful of rows, so the
// call is bound by the stream of the hit experts' weights (2 d d_ff elements
// each) and, for the smallest layers, by launch latency. After the router:
//
//   up:   one workgroup per (hit expert, 16 hidden neurons). Each workgroup
//         derives what it needs of the dispatch plan from the expert ids
//         itself (at most 1024 of them): the set of hit experts, its own
//         expert and that expert's rows in (choice, token) order. No scan
//         launch, and the grid is sized by min(E, N k) without a host sync.
//         Four waves split K and add through LDS.
//   down: one workgroup per 16 output columns walks every hit expert's rows
//         of those columns, its waves taking contiguous ranges of the
//         (expert, K-chunk) sequence, and keeps the gate-weighted sums of all
//         tokens in LDS, one copy per wave, added in wave order: the combine
//         costs no pass of its own and the result does not depend on timing.
//
// The hidden row is kept as two bf16 terms (hi + lo, 16 significant bits):
// the product that reads it is bound by its weights, so the second MFMA is
// free, and the layer's output then carries only its own final rounding.
#include <type_traits>

#include "activation.hpp"
#include "common.hpp"
#include "skinny.hpp"

namespace moe {
namespace {

constexpr int kFewTokens = kFewMaxTokens;
constexpr int kFewAssign = kFewTokens * kMaxTopK;   // assignments of a call
constexpr int kChunk = 256;                         // K elements of one down unit

// Dispatch plan of the call, written by the up product, read by the down
// product (device, in the workspace).
struct FewPlan {
    int nhit;                              // experts with a kept row
    int expert[kMaxExperts];               // their ids, ascending
    int rows[kMaxExperts];                 // kept rows of each
    int row[kMaxExperts][kFewTokens];      // their assignments, slot order
};

// What a workgroup of the up product derives from the ids: the a-th hit expert
// and its kept rows. All threads of the workgroup (a multiple of 64, at least
// 64) call it; ends with a barrier. Returns the number of hit experts.
struct PlanShared {
    unsigned mask[kMaxExperts / 32];
    unsigned char id[kFewAssign];      // expert of assignment (j, t) at j N + t
    int row[kFewTokens];
    int expert, count, kept;
};
__device__ __forceinline__ int few_plan(const int32_t *__restrict__ idx, int N, int k, int cap,
                                        int a, int nthr, PlanShared &p) {
    const int tid = threadIdx.x, A = N * k;
    if (tid < kMaxExperts / 32)
        p.mask[tid] = 0;
    __syncthreads();
    for (int i = tid; i < A; i += nthr) {
        const int e = idx[i], t = i / k, j = i - t * k;
        p.id[j * N + t] = (unsigned char)e;
        atomicOr(&p.mask[e >> 5], 1u << (e & 31));
    }
    __syncthreads();
    int nhit = 0, e = -1;
#pragma unroll
    for (int w = 0; w < kMaxExperts / 32; ++w) {
        unsigned m = p.mask[w];
        const int c = __popc(m);
        if (a >= nhit && a < nhit + c) {
            for (int i = nhit; i < a; ++i)
                m &= m - 1;
            e = w * 32 + __ffs(m) - 1;
        }
        nhit += c;
    }
    if (tid < 64) {
        int base = 0;
        if (e >= 0) {
            for (int c = 0; c < A; c += 64) {
                const int o = c + tid;
                const bool mine = o < A && p.id[o] == e;
                const uint64_t m = __ballot(mine);
                const int r = base + __popcll(m & lanemask_lt());
                if (mine && r < cap) {
                    const int j = o / N, t = o - j * N;
                    p.row[r] = t * k + j;
                }
                base += __popcll(m);
            }
        }
        if (tid == 0) {
            p.expert = e;
            p.count = base;
            p.kept = min(base, cap);
        }
    }
    __syncthreads();
    return nhit;
}

// Exports of the workgroup that owns expert e (its first column tile): the
// plan of the down product, slots, counts and gate sums.
struct FewExports {
    int32_t *slot, *used, *demand, *drops;
    float *gate_sum;
};
__device__ __forceinline__ void few_exports(const PlanShared &p, const float *__restrict__ gate,
                                            int N, int k, int E, int a, int nhit, int nthr,
                                            FewPlan *__restrict__ plan, const FewExports &x) {
    const int tid = threadIdx.x, e = p.expert, A = N * k;
    if (a == 0) {
        if (tid == 0)
            plan->nhit = nhit;
        // experts nobody took
        for (int i = tid; i < E; i += nthr)
            if (!((p.mask[i >> 5] >> (i & 31)) & 1u)) {
                if (x.used) x.used[i] = 0;
                if (x.demand) x.demand[i] = 0;
                if (x.drops) x.drops[i] = 0;
                if (x.gate_sum) x.gate_sum[i] = 0.f;
            }
    }
    if (tid == 0) {
        plan->expert[a] = e;
        plan->rows[a] = p.kept;
        if (x.used) x.used[e] = p.kept;
        if (x.demand) x.demand[e] = p.count;
        if (x.drops) x.drops[e] = p.count - p.kept;
        if (x.gate_sum) {
            float s = 0.f;   // (choice, token) order
            for (int o = 0; o < A; ++o)
                if (p.id[o] == e)
                    s += gate[(o % N) * k + o / N];
            x.gate_sum[e] = s;
        }
    }
    if (tid < p.kept)
        plan->row[a][tid] = p.row[tid];
    if (x.slot && tid < 64) {
        int base = 0;
        for (int c = 0; c < A; c += 64) {
            const int o = c + tid;
            const bool mine = o < A && p.id[o] == e;
            const uint64_t m = __ballot(mine);
            if (mine) {
                const int r = base + __popcll(m & lanemask_lt());
                x.slot[(o % N) * k + o / N] = r < p.kept ? r : -1;
            }
            base += __popcll(m);
        }
    }
}

// H (two bf16 terms, [2][N k][d_ff]) = act(W_up[e] x + b_up[e]) for the rows of
// the hit experts. grid: (column tiles of 16, min(E, N k)); TT token tiles.
constexpr int kUpWaves = 4;
template <int TT>
__global__ __launch_bounds__(kUpWaves * 64) void few_up_kernel(
    const unsigned short *__restrict__ x, const unsigned short *__restrict__ w_up,
    const float *__restrict__ b_up, const int32_t *__restrict__ idx,
    const float *__restrict__ gate, int N, int d, int E, int d_ff, int k, int cap, int act,
    unsigned short *__restrict__ H, FewPlan *__restrict__ plan, FewExports ex) {
    __shared__ PlanShared p;
    __shared__ f32x4 part[kUpWaves][TT][64];
    const int nthr = kUpWaves * 64;
    const int a = blockIdx.y, f0 = blockIdx.x * 16;
    const int nhit = few_plan(idx, N, k, cap, a, nthr, p);
    if (a >= nhit)
        return;
    if (blockIdx.x == 0)
        few_exports(p, gate, N, k, E, a, nhit, nthr, plan, ex);
    const int rows = p.kept, e = p.expert;
    const int lane = threadIdx.x & 63, wv = threadIdx.x >> 6;
    const int ntile = (rows + 15) / 16;
    const unsigned short *w =
        w_up + ((int64_t)e * d_ff + min(f0 + (lane & 15), d_ff - 1)) * d;
    // this wave's K range, in steps of 32
    const int steps = (d + 31) / 32;
    const int kb = (int)((int64_t)wv * steps / kUpWaves) * 32;
    const int ke = (int)((int64_t)(wv + 1) * steps / kUpWaves) * 32;
    f32x4 acc[TT];
#pragma unroll
    for (int i = 0; i < TT; ++i)
        acc[i] = f32x4{0.f, 0.f, 0.f, 0.f};
    auto run = [&](auto tiles) {
        constexpr int T = decltype(tiles)::value;
        const unsigned short *xt[T];
        f32x4 c[T];
#pragma unroll
        for (int i = 0; i < T; ++i) {
            const int r = i * 16 + (lane & 15);
            xt[i] = x + (int64_t)(p.row[r < rows ? r : 0] / k) * d;
            c[i] = f32x4{0.f, 0.f, 0.f, 0.f};
        }
        skinny_mma<T, 1, T == 1 ? 8 : T == 2 ? 4 : 2>(w, xt, 0, kb, ke, d, c);
#pragma unroll
        for (int i = 0; i < T; ++i)
            acc[i] = c[i];
    };
    if (TT == 1 || ntile <= 1)
        run(std::integral_constant<int, 1>{});
    else if (TT == 2 || ntile <= 2)
        run(std::integral_constant<int, TT < 2 ? TT : 2>{});
    else
        run(std::integral_constant<int, TT>{});
#pragma unroll
    for (int i = 0; i < TT; ++i)
        if (i < ntile)
            part[wv][i][lane] = acc[i];
    __syncthreads();
    // thread -> (row, 4 neurons): tile i's lane l holds neurons 4 (l / 16) + q
    // of row l % 16
    for (int q = threadIdx.x; q < ntile * 64; q += nthr) {
        const int i = q >> 6, l = q & 63;
        const int r = i * 16 + (l & 15), f = f0 + 4 * (l >> 4);
        if (r >= rows || f >= d_ff)
            continue;
        f32x4 z = part[0][i][l];
#pragma unroll
        for (int s = 1; s < kUpWaves; ++s)
            z += part[s][i][l];
        if (b_up)
            z += *reinterpret_cast<const f32x4 *>(b_up + (int64_t)e * d_ff + f);
        float h[4], lo[4];
#pragma unroll
        for (int c = 0; c < 4; ++c) {
            h[c] = activate(z[c], act);
            // the rest of an infinity or a NaN would be NaN: it has none
            const float rest = h[c] - bf16_bits_to_f32(f32_to_bf16_bits(h[c]));
            lo[c] = fabsf(rest) < __builtin_inff() ? rest : 0.f;
        }
        unsigned short *dst = H + (int64_t)p.row[r] * d_ff + f;
        *reinterpret_cast<u32x2 *>(dst) = u32x2{pack_bf16x2(h[0], h[1]), pack_bf16x2(h[2], h[3])};
        *reinterpret_cast<u32x2 *>(dst + (int64_t)N * k * d_ff) =
            u32x2{pack_bf16x2(lo[0], lo[1]), pack_bf16x2(lo[2], lo[3])};
    }
}

// out[t] = sum over kept choices of gate (W_down[e] h + b_down[e]), 16 columns
// per workgroup. LDS: one [N][16] copy of the sums per wave.
constexpr int kDownWaves = 16;
template <int TT>
__global__ __launch_bounds__(kDownWaves * 64) void few_down_kernel(
    const unsigned short *__restrict__ H, const unsigned short *__restrict__ w_down,
    const float *__restrict__ b_down, const float *__restrict__ gate,
    const FewPlan *__restrict__ plan, int N, int d, int d_ff, int k,
    unsigned short *__restrict__ out) {
    constexpr int NT = TT * 16;
    __shared__ float sum[kDownWaves][NT][16 + 1];
    const int c0 = blockIdx.x * 16;
    const int lane = threadIdx.x & 63;
    const int wv = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    for (int i = lane; i < NT * 17; i += 64)
        (&sum[wv][0][0])[i] = 0.f;
    const int chunks = (d_ff + kChunk - 1) / kChunk;
    const int units = plan->nhit * chunks;
    const int ub = (int)((int64_t)wv * units / kDownWaves);
    const int ue = (int)((int64_t)(wv + 1) * units / kDownWaves);
    const int64_t lo = (int64_t)N * k * d_ff;
    const int col = min(c0 + (lane & 15), d - 1);
    for (int u = ub; u < ue;) {
        const int a = u / chunks, uc = u - a * chunks;
        const int un = min(ue - u, chunks - uc);   // chunks of this expert
        const int e = plan->expert[a], rows = plan->rows[a];
        const unsigned short *w = w_down + ((int64_t)e * d + col) * d_ff;
        const int kb = uc * kChunk, ke = min((uc + un) * kChunk, (d_ff + 31) / 32 * 32);
        u += un;
        auto run = [&](auto tiles) {
            constexpr int T = decltype(tiles)::value;
            const unsigned short *ht[T];
            f32x4 acc[T];
            int as[T];
            f32x4 bias = {0.f, 0.f, 0.f, 0.f};
            if (b_down && uc == 0 && c0 + 4 * (lane >> 4) < d)
                bias = *reinterpret_cast<const f32x4 *>(b_down + (int64_t)e * d + c0 +
                                                        4 * (lane >> 4));
#pragma unroll
            for (int i = 0; i < T; ++i) {
                const int r = i * 16 + (lane & 15);
                as[i] = plan->row[a][r < rows ? r : 0];
                ht[i] = H + (int64_t)as[i] * d_ff;
                acc[i] = bias;
            }
            skinny_mma<T, 2, T == 1 ? 4 : T == 2 ? 2 : 1>(w, ht, lo, kb, ke, d_ff, acc);
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
        if (TT == 1 || rows <= 16)
            run(std::integral_constant<int, 1>{});
        else if (TT == 2 || rows <= 32)
            run(std::integral_constant<int, TT < 2 ? TT : 2>{});
        else
            run(std::integral_constant<int, TT>{});
    }
    __syncthreads();
    for (int i = threadIdx.x; i < N * 2; i += kDownWaves * 64) {
        const int t = i >> 1, c = (i & 1) * 8;
        if (c0 + c >= d)
            continue;
        float v[8];
#pragma unroll
        for (int q = 0; q < 8; ++q) {
            v[q] = sum[0][t][c + q];
#pragma unroll
            for (int w = 1; w < kDownWaves; ++w)
                v[q] += sum[w][t][c + q];
        }
        *reinterpret_cast<u32x4 *>(out + (int64_t)t * d + c0 + c) =
            u32x4{pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]), pack_bf16x2(v[4], v[5]),
                  pack_bf16x2(v[6], v[7])};
    }
}

// fp32 layers (any widths): a wave takes four weight rows at a time against
// eight token rows, lanes along K, and adds across its lanes at the end.
constexpr int kF32Rows = 4, kF32Toks = 8;
__device__ __forceinline__ float wave_add(float v) {
#pragma unroll
    for (int o = 32; o >= 1; o >>= 1)
        v += __shfl_xor(v, o);
    return v;
}
__device__ __forceinline__ void dots_f32(const float *const (&w)[kF32Rows],
                                         const float *const (&x)[kF32Toks], int K,
                                         float (&acc)[kF32Rows][kF32Toks]) {
#pragma unroll
    for (int i = 0; i < kF32Rows; ++i)
#pragma unroll
        for (int j = 0; j < kF32Toks; ++j)
            acc[i][j] = 0.f;
    for (int c = (int)__lane_id(); c < K; c += 64) {
        float wv[kF32Rows], xv[kF32Toks];
#pragma unroll
        for (int i = 0; i < kF32Rows; ++i)
            wv[i] = w[i][c];
#pragma unroll
        for (int j = 0; j < kF32Toks; ++j)
            xv[j] = x[j][c];
#pragma unroll
        for (int i = 0; i < kF32Rows; ++i)
#pragma unroll
            for (int j = 0; j < kF32Toks; ++j)
                acc[i][j] = fmaf(wv[i], xv[j], acc[i][j]);
    }
#pragma unroll
    for (int i = 0; i < kF32Rows; ++i)
#pragma unroll
        for (int j = 0; j < kF32Toks; ++j)
            acc[i][j] = wave_add(acc[i][j]);
}

__global__ __launch_bounds__(256) void few_up_f32_kernel(
    const float *__restrict__ x, const float *__restrict__ w_up, const float *__restrict__ b_up,
    const int32_t *__restrict__ idx, const float *__restrict__ gate, int N, int d, int E, int d_ff,
    int k, int cap, int act, float *__restrict__ H, FewPlan *__restrict__ plan, FewExports ex) {
    __shared__ PlanShared p;
    const int a = blockIdx.y;
    const int nhit = few_plan(idx, N, k, cap, a, 256, p);
    if (a >= nhit)
        return;
    if (blockIdx.x == 0)
        few_exports(p, gate, N, k, E, a, nhit, 256, plan, ex);
    const int rows = p.kept, e = p.expert;
    const int lane = threadIdx.x & 63;
    const int f0 = (blockIdx.x * 4 + (threadIdx.x >> 6)) * kF32Rows;
    if (f0 >= d_ff)
        return;
    const float *w[kF32Rows];
#pragma unroll
    for (int i = 0; i < kF32Rows; ++i)
        w[i] = w_up + ((int64_t)e * d_ff + min(f0 + i, d_ff - 1)) * d;
    for (int r0 = 0; r0 < rows; r0 += kF32Toks) {
        const float *xr[kF32Toks];
#pragma unroll
        for (int j = 0; j < kF32Toks; ++j)
            xr[j] = x + (int64_t)(p.row[min(r0 + j, rows - 1)] / k) * d;
        float acc[kF32Rows][kF32Toks];
        dots_f32(w, xr, d, acc);
#pragma unroll
        for (int i = 0; i < kF32Rows; ++i)
#pragma unroll
            for (int j = 0; j < kF32Toks; ++j)
                if (lane == i * kF32Toks + j && f0 + i < d_ff && r0 + j < rows) {
                    const float z =
                        b_up ? acc[i][j] + b_up[(int64_t)e * d_ff + f0 + i] : acc[i][j];
                    H[(int64_t)p.row[r0 + j] * d_ff + f0 + i] = activate(z, act);
                }
    }
}

__global__ __launch_bounds__(256) void few_down_f32_kernel(
    const float *__restrict__ H, const float *__restrict__ w_down,
    const float *__restrict__ b_down, const float *__restrict__ gate,
    const FewPlan *__restrict__ plan, int N, int d, int d_ff, int k, float *__restrict__ out) {
    __shared__ float sum[4][kFewTokens][kF32Rows];
    const int lane = threadIdx.x & 63, wv = threadIdx.x >> 6;
    const int c0 = (blockIdx.x * 4 + wv) * kF32Rows;
    if (c0 >= d)
        return;   // (no barrier follows: each wave keeps to its own sums)
    for (int i = lane; i < kFewTokens * kF32Rows; i += 64)
        (&sum[wv][0][0])[i] = 0.f;
    const int nhit = plan->nhit;
    for (int a = 0; a < nhit; ++a) {
        const int e = plan->expert[a], rows = plan->rows[a];
        const float *w[kF32Rows];
#pragma unroll
        for (int i = 0; i < kF32Rows; ++i)
            w[i] = w_down + ((int64_t)e * d + min(c0 + i, d - 1)) * d_ff;
        for (int r0 = 0; r0 < rows; r0 += kF32Toks) {
            const float *hr[kF32Toks];
            int as[kF32Toks];
#pragma unroll
            for (int j = 0; j < kF32Toks; ++j) {
                as[j] = plan->row[a][min(r0 + j, rows - 1)];
                hr[j] = H + (int64_t)as[j] * d_ff;
            }
            float acc[kF32Rows][kF32Toks];
            dots_f32(w, hr, d_ff, acc);
#pragma unroll
            for (int i = 0; i < kF32Rows; ++i)
#pragma unroll
                for (int j = 0; j < kF32Toks; ++j)
                    if (lane == i * kF32Toks + j && c0 + i < d && r0 + j < rows) {
                        const float y = b_down ? acc[i][j] + b_down[(int64_t)e * d + c0 + i]
                                               : acc[i][j];
                        float *s = &sum[wv][as[j] / k][i];
                        *s = fmaf(gate[as[j]], y, *s);
                    }
        }
    }
    __builtin_amdgcn_wave_barrier();
    for (int i = lane; i < N * kF32Rows; i += 64) {
        const int t = i / kF32Rows, c = c0 + i % kF32Rows;
        if (c < d)
            out[(int64_t)t * d + c] = sum[wv][t][i % kF32Rows];
    }
}

}  // namespace

size_t few_plan_bytes() { return sizeof(FewPlan); }

hipError_t launch_few(bool bf16, const void *x, const void *w_up, const void *w_down,
                      const float *b_up, const float *b_down, const int32_t *idx,
                      const float *gate, int64_t N, int64_t d, int E, int64_t d_ff, int k,
                      int64_t ceff, int act, void *H, void *plan, void *out, int32_t *slot,
                      int32_t *used, int32_t *demand, int32_t *drops, float *gate_sum,
                      hipStream_t s) {
    FewPlan *pl = static_cast<FewPlan *>(plan);
    const FewExports ex{slot, used, demand, drops, gate_sum};
    const int n = (int)N, A = n * k;
    const unsigned hits = (unsigned)(E < A ? E : A);
    if (!bf16) {
        hipLaunchKernelGGL(few_up_f32_kernel,
                           dim3((unsigned)((d_ff + 4 * kF32Rows - 1) / (4 * kF32Rows)), hits),
                           dim3(256), 0, s, static_cast<const float *>(x),
                           static_cast<const float *>(w_up), b_up, idx, gate, n, (int)d, E,
                           (int)d_ff, k, (int)ceff, act, static_cast<float *>(H), pl, ex);
        hipError_t err = hipGetLastError();
        if (err != hipSuccess)
            return err;
        hipLaunchKernelGGL(few_down_f32_kernel,
                           dim3((unsigned)((d + 4 * kF32Rows - 1) / (4 * kF32Rows))), dim3(256), 0,
                           s, static_cast<const float *>(H), static_cast<const float *>(w_down),
                           b_down, gate, (const FewPlan *)pl, n, (int)d, (int)d_ff, k,
                           static_cast<float *>(out));
        return hipGetLastError();
    }
    // token tiles an expert can need: min(N, C) rows
    auto go = [&](auto tiles) {
        constexpr int TT = decltype(tiles)::value;
        hipLaunchKernelGGL(few_up_kernel<TT>, dim3((unsigned)((d_ff + 15) / 16), hits),
                           dim3(kUpWaves * 64), 0, s, static_cast<const unsigned short *>(x),
                           static_cast<const unsigned short *>(w_up), b_up, idx, gate, n, (int)d,
                           E, (int)d_ff, k, (int)ceff, act, static_cast<unsigned short *>(H), pl,
                           ex);
        hipError_t err = hipGetLastError();
        if (err != hipSuccess)
            return err;
        hipLaunchKernelGGL(few_down_kernel<TT>, dim3((unsigned)((d + 15) / 16)),
                           dim3(kDownWaves * 64), 0, s, static_cast<const unsigned short *>(H),
                           static_cast<const unsigned short *>(w_down), b_down, gate,
                           (const FewPlan *)pl, n, (int)d, (int)d_ff, k,
                           static_cast<unsigned short *>(out));
        return hipGetLastError();
    };
    if (n <= 16)
        return go(std::integral_constant<int, 1>{});
    if (n <= 32)
        return go(std::integral_constant<int, 2>{});
    return go(std::integral_constant<int, 4>{});
}

}  // namespace moe
