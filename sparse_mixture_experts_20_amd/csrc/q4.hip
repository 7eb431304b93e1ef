// Products of a few rows with weights held in 4 bits: the linear product and
// the routed experts of a decoding step.
//
//   w[m, k] = (q[m, k] - zero[m, k / group]) scale[m, k / group]
//   linear:   out = act(x W^T + b) + r                       1 to 64 rows
//   experts:  out_t = sum_j gate_tj (W_down[e] h + b_down[e]),
//             h = act(W_up[e] x_t + b_up[e]),  e = idx_tj     1 to 64 tokens
//
// q are 4-bit numbers, two to a byte (even k in the low half); scale and zero
// are bf16, one per group of 32, 64 or 128 weights of a row.
//
// Bound by the stream of the weights (half a byte each), so they go from global
// memory straight into MFMA operands: a lane reads 16 bytes, 32 weights of one
// row. Four bits become the bf16 number 128 + q by two bit operations for two
// weights (0x4300 | q: bf16 has a step of 1 there), exactly; the MFMA then
// accumulates sum x (128 + q) of a group, another one the group's sum of x, and
// two fp32 operations per group give scale (sum x (128 + q) - (128 + zero) sum
// x). Every product is exact in the fp32 accumulator; the subtraction cancels
// at most 7 bits or so of its 24. The weights are the MFMA's columns, so a lane
// holds one weight row's results and needs that row's scales alone.
//
// A group must not share an MFMA with another: 32 K-positions, 8 from each
// quarter of the wave. The 16 bytes of a quarter hold 32 consecutive weights, so
// groups of 128 need nothing, and groups of 64 and 32 swap registers between
// halves and quarters of the wave (2 and 4 swaps a load).
#include <algorithm>
#include <type_traits>

#include "activation.hpp"
#include "common.hpp"

namespace moe {
namespace {

constexpr int kQ4Step = 128;   // weights of a row per wave load
constexpr int kMaxAssign = kFewMaxTokens * kMaxTopK;

// 8 packed weights as 128 + q in bf16, in the order 0 4 1 5 2 6 3 7.
__device__ __forceinline__ bf16x8 q4_weights(unsigned d) {
    constexpr unsigned M = 0x000f000fu, C = 0x43004300u;
    return __builtin_bit_cast(
        bf16x8, u32x4{(d & M) | C, ((d >> 4) & M) | C, ((d >> 8) & M) | C, ((d >> 12) & M) | C});
}
// 8 activations in the same order.
__device__ __forceinline__ bf16x8 q4_order(const u32x4 &v) {
    return __builtin_bit_cast(bf16x8, u32x4{__builtin_amdgcn_perm(v[2], v[0], 0x05040100u),
                                            __builtin_amdgcn_perm(v[2], v[0], 0x07060302u),
                                            __builtin_amdgcn_perm(v[3], v[1], 0x05040100u),
                                            __builtin_amdgcn_perm(v[3], v[1], 0x07060302u)});
}

// Groups of 128 / GS weights. The registers of a 16-byte load put in an order
// whose MFMA i holds positions of one group: quarter g's 8 positions of MFMA i
// start at position<GS>(g, i) of the 128.
template <int GS>
__device__ __forceinline__ int q4_position(int g, int i) {
    return GS == 1   ? 32 * g + 8 * i
           : GS == 2 ? 32 * (g & 1) + 16 * (g >> 1) + 8 * (i & 1) + 64 * (i >> 1)
                     : 32 * i + 8 * g;
}
template <int GS>
__device__ __forceinline__ void q4_arrange(u32x4 &d) {
    if constexpr (GS >= 2) {
        auto a = __builtin_amdgcn_permlane32_swap(d[0], d[2], false, false);
        auto b = __builtin_amdgcn_permlane32_swap(d[1], d[3], false, false);
        d = u32x4{a[0], b[0], a[1], b[1]};
    }
    if constexpr (GS == 4) {
        auto a = __builtin_amdgcn_permlane16_swap(d[0], d[1], false, false);
        auto b = __builtin_amdgcn_permlane16_swap(d[2], d[3], false, false);
        d = u32x4{a[0], a[1], b[0], b[1]};
    }
}

// One matrix of 4-bit weights [M, K] (of expert e: offset by e M rows).
struct Q4Matrix {
    const unsigned char *data;
    const unsigned short *scale, *zero;   // zero NULL: 8
};

// Scales of GS adjacent groups.
template <int GS>
struct Q4Groups {
    unsigned short v[GS];
    __device__ __forceinline__ void load(const unsigned short *p, int have) {
        if (GS == 1 || have >= GS) {
            __builtin_memcpy(v, p, sizeof(v));
        } else {
#pragma unroll
            for (int i = 0; i < GS; ++i)
                v[i] = i < have ? p[i] : (unsigned short)0;
        }
    }
};

// tot[rt][i] += products of K columns [kb, ke) (multiples of 128, ke possibly
// past K) of RT row tiles of 16 weight rows with TT tiles of 16 token rows, by
// one wave: lane l ends with weight row l % 16 of tile rt and tokens 4 (l / 16)
// + q of tile i. m[rt]: this lane's weight row; xt[i]: this lane's token row
// (column 0); NB terms per token row, `lo` elements apart, are added. U steps
// are loaded while the previous ones are multiplied.
template <int GS, int RT, int TT, int NB, int U>
__device__ __forceinline__ void q4_product(const Q4Matrix &W, const int64_t (&m)[RT],
                                           const unsigned short *const (&xt)[TT], int64_t lo,
                                           int kb, int ke, int K, f32x4 (&tot)[RT][TT]) {
    constexpr bool AHEAD = TT * NB <= 2;   // token rows are loaded with the weights
    const int g = (int)(__lane_id() >> 4);
    const int KG = K / (kQ4Step / GS);     // groups of a row
    const unsigned char *w[RT];
    const unsigned short *sc[RT], *zp[RT];
#pragma unroll
    for (int r = 0; r < RT; ++r) {
        w[r] = W.data + m[r] * (K / 2) + 16 * g;
        sc[r] = W.scale + m[r] * KG;
        zp[r] = W.zero + (W.zero ? m[r] * KG : 0);
    }
    struct Step {
        u32x4 w[RT];
        Q4Groups<GS> s[RT], z[RT];
        u32x4 x[AHEAD ? TT : 1][AHEAD ? NB : 1][4];
    };
    auto load_x = [&](int i, int n, int k, int j) {
        const int o = k + q4_position<GS>(g, j);
        if (GS == 1 || o < K)
            return *reinterpret_cast<const u32x4 *>(xt[i] + n * lo + o);
        return u32x4{0u, 0u, 0u, 0u};
    };
    auto load = [&](int k, Step &s) {
#pragma unroll
        for (int r = 0; r < RT; ++r) {
            s.w[r] = u32x4{0u, 0u, 0u, 0u};
            if (GS == 1 || k + 32 * g < K)
                s.w[r] = *reinterpret_cast<const u32x4 *>(w[r] + k / 2);
        }
        if constexpr (AHEAD)
#pragma unroll
            for (int i = 0; i < TT; ++i)
#pragma unroll
                for (int n = 0; n < NB; ++n)
#pragma unroll
                    for (int j = 0; j < 4; ++j)
                        s.x[i][n][j] = load_x(i, n, k, j);
        const int at = k / (kQ4Step / GS);
#pragma unroll
        for (int r = 0; r < RT; ++r) {
            s.s[r].load(sc[r] + at, KG - at);
            if (W.zero)
                s.z[r].load(zp[r] + at, KG - at);
        }
    };
    auto multiply = [&](int k, Step &s) {
        const f32x4 nil = {0.f, 0.f, 0.f, 0.f};
        const bf16x8 ones = __builtin_bit_cast(
            bf16x8, u32x4{0x3f803f80u, 0x3f803f80u, 0x3f803f80u, 0x3f803f80u});
        f32x4 acc[RT][TT], sx[TT];
#pragma unroll
        for (int r = 0; r < RT; ++r)
            q4_arrange<GS>(s.w[r]);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            constexpr int P = 4 / GS;   // MFMAs of a group
            if (j % P == 0) {
#pragma unroll
                for (int i = 0; i < TT; ++i) {
                    sx[i] = nil;
#pragma unroll
                    for (int r = 0; r < RT; ++r)
                        acc[r][i] = nil;
                }
            }
            bf16x8 q[RT];
#pragma unroll
            for (int r = 0; r < RT; ++r)
                q[r] = q4_weights(s.w[r][j]);
#pragma unroll
            for (int i = 0; i < TT; ++i)
#pragma unroll
                for (int n = 0; n < NB; ++n) {
                    bf16x8 a;
                    if constexpr (AHEAD)
                        a = q4_order(s.x[i][n][j]);
                    else
                        a = q4_order(load_x(i, n, k, j));
                    sx[i] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, ones, sx[i], 0, 0, 0);
#pragma unroll
                    for (int r = 0; r < RT; ++r)
                        acc[r][i] =
                            __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, q[r], acc[r][i], 0, 0, 0);
                }
            if (j % P == P - 1) {
#pragma unroll
                for (int r = 0; r < RT; ++r) {
                    const float f = bf16_bits_to_f32(s.s[r].v[j / P]);
                    const float c =
                        W.zero ? -128.f - bf16_bits_to_f32(s.z[r].v[j / P]) : -136.f;
#pragma unroll
                    for (int i = 0; i < TT; ++i)
#pragma unroll
                        for (int e = 0; e < 4; ++e)
                            tot[r][i][e] =
                                fmaf(f, fmaf(c, sx[i][e], acc[r][i][e]), tot[r][i][e]);
                }
            }
        }
    };
    Step next[U];
    int k = kb;
    if (k + kQ4Step * U <= ke) {
#pragma unroll
        for (int u = 0; u < U; ++u)
            load(k + kQ4Step * u, next[u]);
        for (k += kQ4Step * U; k + kQ4Step * U <= ke; k += kQ4Step * U) {
            Step cur[U];
#pragma unroll
            for (int u = 0; u < U; ++u)
                cur[u] = next[u];
#pragma unroll
            for (int u = 0; u < U; ++u)
                load(k + kQ4Step * u, next[u]);
#pragma unroll
            for (int u = 0; u < U; ++u)
                multiply(k + kQ4Step * (u - U), cur[u]);
        }
#pragma unroll
        for (int u = 0; u < U; ++u)
            multiply(k + kQ4Step * (u - U), next[u]);
    }
    for (; k < ke; k += kQ4Step) {
        load(k, next[0]);
        multiply(k, next[0]);
    }
}

// The product over a workgroup's K range by all its waves, added through LDS in
// wave order: f(token row, weight row of the RT 16, value) for each result.
// part: waves x RT x TT x 64 f32x4.
template <int GS, int RT, int TT, int NB, typename F>
__device__ __forceinline__ void q4_block(f32x4 *part, const Q4Matrix &W, const int64_t (&m)[RT],
                                         const unsigned short *const (&xt)[TT], int64_t lo, int K,
                                         F f) {
    const int lane = threadIdx.x & 63;
    const int wv = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int waves = blockDim.x >> 6;
    const int steps = (K + kQ4Step - 1) / kQ4Step;
    const int kb = (int)((int64_t)wv * steps / waves) * kQ4Step;
    const int ke = (int)((int64_t)(wv + 1) * steps / waves) * kQ4Step;
    f32x4 tot[RT][TT];
#pragma unroll
    for (int r = 0; r < RT; ++r)
#pragma unroll
        for (int i = 0; i < TT; ++i)
            tot[r][i] = f32x4{0.f, 0.f, 0.f, 0.f};
    constexpr int U = TT * NB <= 1 ? 2 : 1;
    q4_product<GS, RT, TT, NB, U>(W, m, xt, lo, kb, ke, K, tot);
#pragma unroll
    for (int r = 0; r < RT; ++r)
#pragma unroll
        for (int i = 0; i < TT; ++i)
            part[((wv * RT + r) * TT + i) * 64 + lane] = tot[r][i];
    __syncthreads();
    for (int o = threadIdx.x; o < RT * TT * 64; o += blockDim.x) {
        f32x4 v = part[o];
        for (int w = 1; w < waves; ++w)
            v += part[w * RT * TT * 64 + o];
        const int l = o & 63, i = (o >> 6) % TT, r = (o >> 6) / TT;
#pragma unroll
        for (int e = 0; e < 4; ++e)
            f(16 * i + 4 * (l >> 4) + e, 16 * r + (l & 15), v[e]);
    }
}

struct Q4Linear {
    const unsigned short *x;
    Q4Matrix W;
    const float *bias;            // [M] or NULL
    const unsigned short *res;    // [N, M] or NULL
    unsigned short *out;          // [N, M]
    int N, K, act;
    int64_t M;
};

// grid: tiles of 16 RT weight rows.
template <int GS, int RT, int TT>
__global__ __launch_bounds__(512) void q4_linear_kernel(Q4Linear p) {
    extern __shared__ __attribute__((aligned(16))) f32x4 part[];
    const int lane = threadIdx.x & 63;
    const int64_t m0 = (int64_t)blockIdx.x * (16 * RT);
    int64_t m[RT];
    const unsigned short *xt[TT];
#pragma unroll
    for (int r = 0; r < RT; ++r)
        m[r] = min(m0 + 16 * r + (lane & 15), p.M - 1);
#pragma unroll
    for (int i = 0; i < TT; ++i)
        xt[i] = p.x + (int64_t)min(16 * i + (lane & 15), p.N - 1) * p.K;
    q4_block<GS, RT, TT, 1>(part, p.W, m, xt, 0, p.K, [&](int t, int r, float v) {
        const int64_t c = m0 + r;
        if (t >= p.N || c >= p.M)
            return;
        if (p.bias)
            v += p.bias[c];
        v = activate(v, p.act);
        const int64_t o = (int64_t)t * p.M + c;
        if (p.res)
            v += bf16_bits_to_f32(p.res[o]);
        p.out[o] = f32_to_bf16_bits(v);
    });
}

struct Q4Experts {
    const unsigned short *x;      // [N, d]
    const int32_t *idx;           // [N, k]
    const float *gate;            // [N, k]
    Q4Matrix up, down;
    const float *b_up, *b_down;   // [E, d_ff], [E, d] or NULL
    unsigned short *H;            // [2][N k][d_ff]: two bf16 terms
    float *Y;                     // [N k][d]
    int *done;                    // finished workgroups per column block
    unsigned short *out;          // [N, d]
    int N, d, E, d_ff, k, act;
};

// The assignments (t k + j) of assignment a's expert, in ascending order, into
// row[] by the whole workgroup: their number, or 0 when an earlier assignment
// has the same expert (whose workgroup does the work) or a's id is no expert.
__device__ __forceinline__ int q4_rows(const int32_t *__restrict__ idx, int A, int E, int a,
                                       unsigned short *row) {
    const int lane = threadIdx.x & 63;
    const int e = idx[a];
    int n = 0;
    bool first = e >= 0 && e < E;
    for (int c = 0; c < A; c += 64) {
        const uint64_t same = __ballot(c + lane < A && idx[min(c + lane, A - 1)] == e);
        if (c + 64 <= a) {
            first = first && same == 0;
        } else {
            if (c <= a)
                first = first && (same & ((1ull << (a - c)) - 1ull)) == 0;
            if (threadIdx.x < 64 && (same >> lane & 1ull))
                row[n + __popcll(same & lanemask_lt())] = (unsigned short)(c + lane);
            n += __popcll(same);
        }
        if (!first)
            return 0;
    }
    __syncthreads();
    return n;
}

// H = act(W_up[e] x + b_up[e]) of the rows of assignment blockIdx.y's expert.
// grid: (tiles of 16 RT neurons, N k).
template <int GS, int RT, int TT>
__global__ __launch_bounds__(512) void q4_up_kernel(Q4Experts p, int blocks) {
    extern __shared__ __attribute__((aligned(16))) f32x4 part[];
    __shared__ unsigned short row[kMaxAssign];
    const int lane = threadIdx.x & 63, A = p.N * p.k;
    if (blockIdx.y == 0)
        for (int i = blockIdx.x * blockDim.x + threadIdx.x; i < blocks; i += gridDim.x * blockDim.x)
            p.done[i] = 0;
    const int rows = q4_rows(p.idx, A, p.E, blockIdx.y, row);
    if (rows == 0)
        return;
    const int e = p.idx[blockIdx.y], f0 = blockIdx.x * (16 * RT);
    int64_t m[RT];
#pragma unroll
    for (int r = 0; r < RT; ++r)
        m[r] = (int64_t)e * p.d_ff + min(f0 + 16 * r + (lane & 15), p.d_ff - 1);
    for (int t0 = 0; t0 < rows; t0 += 16 * TT) {
        auto run = [&](auto tiles) {
            constexpr int T = decltype(tiles)::value;
            const unsigned short *xt[T];
#pragma unroll
            for (int i = 0; i < T; ++i)
                xt[i] = p.x + (int64_t)(row[min(t0 + 16 * i + (lane & 15), rows - 1)] / p.k) * p.d;
            q4_block<GS, RT, T, 1>(part, p.up, m, xt, 0, p.d, [&](int t, int r, float v) {
                const int f = f0 + r;
                if (t0 + t >= rows || f >= p.d_ff)
                    return;
                if (p.b_up)
                    v += p.b_up[(int64_t)e * p.d_ff + f];
                v = activate(v, p.act);
                // the second term: what rounding to bf16 leaves (nothing of an
                // infinity or a NaN)
                const unsigned short hi = f32_to_bf16_bits(v);
                const float rest = v - bf16_bits_to_f32(hi);
                unsigned short *h = p.H + (int64_t)row[t0 + t] * p.d_ff + f;
                h[0] = hi;
                h[(int64_t)A * p.d_ff] =
                    f32_to_bf16_bits(fabsf(rest) < __builtin_inff() ? rest : 0.f);
            });
        };
        const int left = rows - t0;
        if (TT == 1 || left <= 16)
            run(std::integral_constant<int, 1>{});
        else if (TT == 2 || left <= 32)
            run(std::integral_constant<int, TT < 2 ? TT : 2>{});
        else
            run(std::integral_constant<int, TT>{});
        __syncthreads();
    }
}

// Y = W_down[e] h + b_down[e] of the same rows; the workgroup of a column block
// that finishes last adds each token's choices in order. Y and the counter are
// written and read past the XCD's own L2 (agent scope). grid: (tiles of 16 RT
// columns, N k).
template <int GS, int RT, int TT>
__global__ __launch_bounds__(512) void q4_down_kernel(Q4Experts p) {
    extern __shared__ __attribute__((aligned(16))) f32x4 part[];
    __shared__ unsigned short row[kMaxAssign];
    __shared__ int last;
    const int lane = threadIdx.x & 63, A = p.N * p.k;
    const int rows = q4_rows(p.idx, A, p.E, blockIdx.y, row);
    const int c0 = blockIdx.x * (16 * RT);
    if (rows > 0) {
        const int e = p.idx[blockIdx.y];
        const int64_t lo = (int64_t)A * p.d_ff;
        int64_t m[RT];
#pragma unroll
        for (int r = 0; r < RT; ++r)
            m[r] = (int64_t)e * p.d + min(c0 + 16 * r + (lane & 15), p.d - 1);
        auto store = [&](int t, int r, float v) {
            if (p.b_down)
                v += p.b_down[(int64_t)e * p.d + c0 + r];
            __hip_atomic_store(p.Y + (int64_t)row[t] * p.d + c0 + r, v, __ATOMIC_RELAXED,
                               __HIP_MEMORY_SCOPE_AGENT);
        };
        for (int t0 = 0; t0 < rows; t0 += 16 * TT) {
            const int left = rows - t0;
            auto run = [&](auto tiles) {
                constexpr int T = decltype(tiles)::value;
                const unsigned short *ht[T];
#pragma unroll
                for (int i = 0; i < T; ++i)
                    ht[i] = p.H + (int64_t)row[min(t0 + 16 * i + (lane & 15), rows - 1)] * p.d_ff;
                q4_block<GS, RT, T, 2>(part, p.down, m, ht, lo, p.d_ff,
                                       [&](int t, int r, float v) {
                                           if (t < left && c0 + r < p.d)
                                               store(t0 + t, r, v);
                                       });
            };
            if (left <= 8) {
                // both terms of up to 8 rows fill one tile: its rows 0-7 the
                // first terms, 8-15 the second ones, added at the end
                const unsigned short *ht[1] = {
                    p.H + (int64_t)row[min(t0 + (lane & 7), rows - 1)] * p.d_ff +
                    (lane & 8 ? lo : 0)};
                q4_block<GS, RT, 1, 1>(part, p.down, m, ht, 0, p.d_ff,
                                       [&](int t, int r, float v) {
                                           v += __shfl_xor(v, 32);
                                           if (t < left && c0 + r < p.d)
                                               store(t0 + t, r, v);
                                       });
            } else if (TT == 1 || left <= 16) {
                run(std::integral_constant<int, 1>{});
            } else if (TT == 2 || left <= 32) {
                run(std::integral_constant<int, TT < 2 ? TT : 2>{});
            } else {
                run(std::integral_constant<int, TT>{});
            }
            __syncthreads();
        }
    }
    // Y has reached memory before the workgroup counts (agent-scope stores write
    // through; the wait is for their completion)
    asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
    __syncthreads();
    if (threadIdx.x == 0)
        last = __hip_atomic_fetch_add(p.done + blockIdx.x, 1, __ATOMIC_RELAXED,
                                      __HIP_MEMORY_SCOPE_AGENT) == A - 1;
    __syncthreads();
    if (!last)
        return;
    for (int i = threadIdx.x; i < p.N * 16 * RT; i += blockDim.x) {
        const int t = i / (16 * RT), c = c0 + i % (16 * RT);
        if (c >= p.d)
            continue;
        float s = 0.f;
        for (int j = 0; j < p.k; ++j) {
            const int a = t * p.k + j, e = p.idx[a];
            if (e >= 0 && e < p.E)
                s = fmaf(p.gate[a],
                         __hip_atomic_load(p.Y + (int64_t)a * p.d + c, __ATOMIC_RELAXED,
                                           __HIP_MEMORY_SCOPE_AGENT),
                         s);
        }
        p.out[(int64_t)t * p.d + c] = f32_to_bf16_bits(s);
    }
}

// ---- the format ----------------------------------------------------------

// 8 weights per thread (group / 8 adjacent threads hold a group). Symmetric:
// scale = max |w| / 7 (as stored, bf16), q = 8 + the nearest of w / scale in
// [-8, 7]. With zero: the range is [min(w, 0), max(w, 0)], scale = range / 15,
// zero = the nearest of -min / scale in [0, 15], q = zero + the nearest of
// w / scale, in [0, 15]. A group of zeros has scale 0 and q = zero.
template <bool BF16>
__global__ __launch_bounds__(256) void q4_quantize_kernel(const void *__restrict__ W, int64_t n8,
                                                          int group, unsigned *__restrict__ data,
                                                          unsigned short *__restrict__ scale,
                                                          unsigned short *__restrict__ zero) {
    const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
    const int64_t c = min(i, n8 - 1);
    float w[8];
    if constexpr (BF16) {
        const u32x4 v = reinterpret_cast<const u32x4 *>(W)[c];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            w[2 * j] = __uint_as_float(v[j] << 16);
            w[2 * j + 1] = __uint_as_float(v[j] & 0xffff0000u);
        }
    } else {
        const f32x4 a = reinterpret_cast<const f32x4 *>(W)[2 * c];
        const f32x4 b = reinterpret_cast<const f32x4 *>(W)[2 * c + 1];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            w[j] = a[j];
            w[4 + j] = b[j];
        }
    }
    float hi = 0.f, lo = 0.f;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        hi = fmaxf(hi, w[j]);
        lo = fminf(lo, w[j]);
    }
    for (int o = 1; o < group / 8; o <<= 1) {
        hi = fmaxf(hi, __shfl_xor(hi, o));
        lo = fminf(lo, __shfl_xor(lo, o));
    }
    const unsigned short sb =
        f32_to_bf16_bits(zero ? (hi - lo) * (1.f / 15.f) : fmaxf(hi, -lo) * (1.f / 7.f));
    const float s = bf16_bits_to_f32(sb);
    float z = 8.f;
    if (zero)
        z = s > 0.f ? fminf(fmaxf(rintf(-lo / s), 0.f), 15.f) : 0.f;
    unsigned d = 0;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        const float q = s > 0.f ? fminf(fmaxf(rintf(w[j] / s) + z, 0.f), 15.f) : z;
        d |= ((unsigned)q & 15u) << (4 * j);
    }
    if (i >= n8)
        return;
    data[i] = d;
    if (i % (group / 8) == 0) {
        scale[i / (group / 8)] = sb;
        if (zero)
            zero[i / (group / 8)] = f32_to_bf16_bits(z);
    }
}

template <bool BF16>
__global__ __launch_bounds__(256) void q4_dequantize_kernel(const unsigned *__restrict__ data,
                                                            const unsigned short *__restrict__ scale,
                                                            const unsigned short *__restrict__ zero,
                                                            int64_t n8, int group,
                                                            void *__restrict__ W) {
    const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
    if (i >= n8)
        return;
    const unsigned d = data[i];
    const int64_t at = i / (group / 8);
    const float s = bf16_bits_to_f32(scale[at]);
    const float z = zero ? bf16_bits_to_f32(zero[at]) : 8.f;
    float w[8];
#pragma unroll
    for (int j = 0; j < 8; ++j)
        w[j] = ((float)((d >> (4 * j)) & 15u) - z) * s;
    if constexpr (BF16) {
        reinterpret_cast<u32x4 *>(W)[i] = u32x4{pack_bf16x2(w[0], w[1]), pack_bf16x2(w[2], w[3]),
                                                pack_bf16x2(w[4], w[5]), pack_bf16x2(w[6], w[7])};
    } else {
        reinterpret_cast<f32x4 *>(W)[2 * i] = f32x4{w[0], w[1], w[2], w[3]};
        reinterpret_cast<f32x4 *>(W)[2 * i + 1] = f32x4{w[4], w[5], w[6], w[7]};
    }
}

size_t up256(size_t v) { return (v + 255) / 256 * 256; }

// Calls f(groups of a 128-weight step, row tiles, token tiles).
template <typename F>
hipError_t with_shape(int group, int rt, int tt, F f) {
    auto tiles = [&](auto gs, auto r) {
        if (tt == 1)
            return f(gs, r, std::integral_constant<int, 1>{});
        if (tt == 2)
            return f(gs, r, std::integral_constant<int, 2>{});
        return f(gs, r, std::integral_constant<int, 4>{});
    };
    auto rows = [&](auto gs) {
        return rt == 1 ? tiles(gs, std::integral_constant<int, 1>{})
                       : tiles(gs, std::integral_constant<int, 2>{});
    };
    return group == 128  ? rows(std::integral_constant<int, 1>{})
           : group == 64 ? rows(std::integral_constant<int, 2>{})
                         : rows(std::integral_constant<int, 4>{});
}
int token_tiles(int64_t n) { return n <= 16 ? 1 : n <= 32 ? 2 : 4; }

struct Q4Shape {
    int rt, waves;
};
// Row tiles and waves of a product over `blocks` times M rows.
Q4Shape q4_shape(int64_t M, int64_t K, int64_t blocks) {
    Q4Shape s;
    s.rt = blocks * M >= 16 * 2048 ? 2 : 1;
    const int64_t steps = (K + kQ4Step - 1) / kQ4Step;
    s.waves = steps >= 32 ? 8 : steps >= 8 ? 4 : 2;
    return s;
}
size_t q4_lds(Q4Shape s, int tt) { return (size_t)s.waves * s.rt * tt * 64 * 16; }

}  // namespace

hipError_t launch_linear_q4(const void *x, const void *data, const void *scale, const void *zero,
                            int group, const float *bias, int act, const void *res, int64_t N,
                            int64_t K, int64_t M, void *out, hipStream_t s) {
    Q4Linear p{};
    p.x = static_cast<const unsigned short *>(x);
    p.W = {static_cast<const unsigned char *>(data), static_cast<const unsigned short *>(scale),
           static_cast<const unsigned short *>(zero)};
    p.bias = bias;
    p.res = static_cast<const unsigned short *>(res);
    p.out = static_cast<unsigned short *>(out);
    p.N = (int)N;
    p.K = (int)K;
    p.M = M;
    p.act = act;
    const Q4Shape sh = q4_shape(M, K, 1);
    return with_shape(group, sh.rt, token_tiles(N), [&](auto gs, auto rt, auto tt) {
        constexpr int GS = decltype(gs)::value, RT = decltype(rt)::value, TT = decltype(tt)::value;
        hipLaunchKernelGGL((q4_linear_kernel<GS, RT, TT>),
                           dim3((unsigned)((M + 16 * RT - 1) / (16 * RT))), dim3(sh.waves * 64),
                           q4_lds(sh, TT), s, p);
        return hipGetLastError();
    });
}

Q4ExpertsLayout experts_q4_layout(int64_t N, int64_t d, int64_t d_ff, int k) {
    Q4ExpertsLayout L;
    size_t o = 0;
    L.H = o;    o += up256((size_t)(N * k * d_ff) * 4);
    L.Y = o;    o += up256((size_t)(N * k * d) * 4);
    L.done = o; o += up256((size_t)((d + 15) / 16) * 4);
    L.total = o;
    return L;
}

hipError_t launch_experts_q4(const void *x, const int32_t *idx, const float *gate,
                             const void *const (&up)[3], const void *const (&down)[3], int group,
                             const float *b_up, const float *b_down, int64_t N, int64_t d, int E,
                             int64_t d_ff, int k, int act, void *ws, void *out, hipStream_t s) {
    typedef const unsigned short *u16;
    char *w = static_cast<char *>(ws);
    const Q4ExpertsLayout L = experts_q4_layout(N, d, d_ff, k);
    Q4Experts p{};
    p.x = static_cast<u16>(x);
    p.idx = idx;
    p.gate = gate;
    p.up = {static_cast<const unsigned char *>(up[0]), static_cast<u16>(up[1]),
            static_cast<u16>(up[2])};
    p.down = {static_cast<const unsigned char *>(down[0]), static_cast<u16>(down[1]),
              static_cast<u16>(down[2])};
    p.b_up = b_up;
    p.b_down = b_down;
    p.H = reinterpret_cast<unsigned short *>(w + L.H);
    p.Y = reinterpret_cast<float *>(w + L.Y);
    p.done = reinterpret_cast<int *>(w + L.done);
    p.out = static_cast<unsigned short *>(out);
    p.N = (int)N;
    p.d = (int)d;
    p.E = E;
    p.d_ff = (int)d_ff;
    p.k = k;
    p.act = act;
    const unsigned A = (unsigned)(N * k);
    const int64_t hits = std::min<int64_t>(E, A);
    const Q4Shape us = q4_shape(d_ff, d, hits), ds = q4_shape(d, d_ff, hits);
    const int tt = token_tiles(N);
    const hipError_t err = with_shape(group, us.rt, tt, [&](auto gs, auto rt, auto t) {
        constexpr int GS = decltype(gs)::value, RT = decltype(rt)::value, TT = decltype(t)::value;
        hipLaunchKernelGGL((q4_up_kernel<GS, RT, TT>),
                           dim3((unsigned)((d_ff + 16 * RT - 1) / (16 * RT)), A),
                           dim3(us.waves * 64), q4_lds(us, TT), s, p,
                           (int)((d + 16 * ds.rt - 1) / (16 * ds.rt)));
        return hipGetLastError();
    });
    if (err != hipSuccess)
        return err;
    return with_shape(group, ds.rt, tt, [&](auto gs, auto rt, auto t) {
        constexpr int GS = decltype(gs)::value, RT = decltype(rt)::value, TT = decltype(t)::value;
        hipLaunchKernelGGL((q4_down_kernel<GS, RT, TT>),
                           dim3((unsigned)((d + 16 * RT - 1) / (16 * RT)), A), dim3(ds.waves * 64),
                           q4_lds(ds, TT), s, p);
        return hipGetLastError();
    });
}

hipError_t launch_quantize_q4(bool bf16, const void *W, int64_t n, int group, void *data,
                              void *scale, void *zero, hipStream_t s) {
    const int64_t n8 = n / 8;
    const dim3 grid((unsigned)((n8 + 255) / 256)), block(256);
    if (bf16)
        hipLaunchKernelGGL(q4_quantize_kernel<true>, grid, block, 0, s, W, n8, group,
                           static_cast<unsigned *>(data), static_cast<unsigned short *>(scale),
                           static_cast<unsigned short *>(zero));
    else
        hipLaunchKernelGGL(q4_quantize_kernel<false>, grid, block, 0, s, W, n8, group,
                           static_cast<unsigned *>(data), static_cast<unsigned short *>(scale),
                           static_cast<unsigned short *>(zero));
    return hipGetLastError();
}

hipError_t launch_dequantize_q4(bool bf16, const void *data, const void *scale, const void *zero,
                                int64_t n, int group, void *W, hipStream_t s) {
    const int64_t n8 = n / 8;
    const dim3 grid((unsigned)((n8 + 255) / 256)), block(256);
    if (bf16)
        hipLaunchKernelGGL(q4_dequantize_kernel<true>, grid, block, 0, s,
                           static_cast<const unsigned *>(data),
                           static_cast<const unsigned short *>(scale),
                           static_cast<const unsigned short *>(zero), n8, group, W);
    else
        hipLaunchKernelGGL(q4_dequantize_kernel<false>, grid, block, 0, s,
                           static_cast<const unsigned *>(data),
                           static_cast<const unsigned short *>(scale),
                           static_cast<const unsigned short *>(zero), n8, group, W);
    return hipGetLastError();
}

}  // namespace moe
