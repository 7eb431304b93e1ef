// Routing to experts with scores over all of them, a bias for balance, groups of
// experts and renormalised gates, and its backward.
//
//   s = W_g x + noise                       fp32, as the layer's own router
//   p = softmax(s) over all E, or sigmoid(s)
//   c = p + bias                            the choice alone sees the bias
//   a group (E / G adjacent experts) scores the sum of its best 1 or 2 c; the
//   best groups stay; the k largest c among their experts are chosen (equal
//   values: lower id first)
//   gate_j = scale p_j, or scale p_j / sum of the chosen p
//
// Scores: an fp32 weight is three exact bf16 terms on the matrix cores (fp32
// activations: fp32 MFMAs). With few weights one kernel computes the scores of 16
// tokens and ranks them; otherwise workgroups take 16 experts, up to 64 tokens and
// a range of the columns each; very large products run on the router's own tiles.
// The last two leave partial scores that the ranking adds in range order.
//
// Ranking: one wave a token, lane l holding experts l, l + 64, ...: the scores
// and their sum by DPP moves, groups through LDS, each choice by a 32-bit
// maximum over the wave and a ballot for the lowest id that has it.
//
// Measured (calls in turn on inputs past the last-level cache; kernels from a trace of
// the same): one token, 256 experts of 7168 in 8 groups 15.5 us (two launches, 4.7 and 5.6
// on the GPU: the host takes longer); 8192 tokens 127, in short runs 119 (split of W_g 5,
// the tiled product 101 to 104 for 90 GFLOP of terms, the ranking 21 beside the scores'
// export); 2047 tokens, 8 experts of 4096 14.3.
#include <algorithm>
#include <type_traits>

#include "common.hpp"
#include "ranking.hpp"
#include "route_plan.hpp"
#include "skinny.hpp"
#include "tile.hpp"

namespace moe {
namespace {

// ---- ranking -------------------------------------------------------------

template <int CTRL, int ROWS = 0xf>
__device__ __forceinline__ unsigned dpp_max32(unsigned x) {
    const unsigned o = (unsigned)__builtin_amdgcn_update_dpp((int)x, (int)x, CTRL, ROWS, 0xf, false);
    return o > x ? o : x;
}
__device__ __forceinline__ unsigned wave_max32(unsigned x) {
    x = dpp_max32<0xb1>(x);          // quad_perm [1,0,3,2]
    x = dpp_max32<0x4e>(x);          // quad_perm [2,3,0,1]
    x = dpp_max32<0x124>(x);         // row_ror:4
    x = dpp_max32<0x128>(x);         // row_ror:8
    x = dpp_max32<0x142, 0xa>(x);    // row_bcast:15 into rows 1 and 3
    x = dpp_max32<0x143, 0xc>(x);    // row_bcast:31 into rows 2 and 3
    return (unsigned)__builtin_amdgcn_readlane((int)x, 63);
}
template <int CTRL, int ROWS = 0xf>
__device__ __forceinline__ float dpp_add(float v) {   // (0 where a lane gets nothing)
    return v + __uint_as_float((unsigned)__builtin_amdgcn_update_dpp(
                   0, (int)__float_as_uint(v), CTRL, ROWS, 0xf, false));
}
// The sum over the wave, on every lane (within rows of 16, then across them).
__device__ __forceinline__ float wave_sum(float v) {
    v = dpp_add<0xb1>(v);          // quad_perm [1,0,3,2]
    v = dpp_add<0x4e>(v);          // quad_perm [2,3,0,1]
    v = dpp_add<0x124>(v);         // row_ror:4
    v = dpp_add<0x128>(v);         // row_ror:8
    v = dpp_add<0x142, 0xa>(v);    // row_bcast:15 into rows 1 and 3
    v = dpp_add<0x143, 0xc>(v);    // row_bcast:31 into rows 2 and 3
    return __uint_as_float((unsigned)__builtin_amdgcn_readlane((int)__float_as_uint(v), 63));
}

// The largest of the wave's keys and the lowest expert that has it; its key is
// cleared. Keys are 0 where there is no candidate.
template <int Q>
__device__ __forceinline__ int take_best(unsigned (&key)[Q], unsigned &best) {
    const int lane = __lane_id();
    unsigned m = key[0];
#pragma unroll
    for (int q = 1; q < Q; ++q)
        m = key[q] > m ? key[q] : m;
    best = wave_max32(m);
    int e = 0;
    bool found = false;
#pragma unroll
    for (int q = 0; q < Q; ++q) {
        const uint64_t b = __ballot(key[q] == best);
        if (!found && b) {
            const int l = __builtin_ctzll(b);
            e = 64 * q + l;
            if (lane == l)
                key[q] = 0;
            found = true;
        }
    }
    return e;
}

struct RouteOut {
    int32_t *idx;     // [N, k]
    float *gate;      // [N, k]
    float *scores;    // [N, E] or NULL
};

// The bias of this lane's experts (loaded before the scores are there).
template <int Q>
__device__ __forceinline__ void load_bias(const RouteRule &r, float (&b)[Q]) {
    const int lane = __lane_id();
#pragma unroll
    for (int q = 0; q < Q; ++q)
        b[q] = r.bias ? r.bias[min(lane + 64 * q, r.E - 1)] : 0.f;
}

// One wave ranks token t from its scores s (lane l: experts l + 64 q). tmp: 64 Q
// floats of LDS of this wave's own.
template <int Q>
__device__ __forceinline__ void route_rank(const float (&s)[Q], const float (&bias)[Q],
                                           const RouteRule &r, int64_t t, const RouteOut &o,
                                           float *tmp) {
    const int lane = __lane_id();
    float v[Q], p[Q];
#pragma unroll
    for (int q = 0; q < Q; ++q)
        v[q] = lane + 64 * q < r.E && s[q] == s[q] ? s[q] : -INFINITY;
    if (r.sigmoid) {
#pragma unroll
        for (int q = 0; q < Q; ++q)
            p[q] = 1.f / (1.f + expf(-v[q]));
    } else {
        unsigned m = 0;
#pragma unroll
        for (int q = 0; q < Q; ++q)
            m = max(m, order_of(v[q]));
        const float top = order_value(wave_max32(m));
        float sum = 0.f;
#pragma unroll
        for (int q = 0; q < Q; ++q) {
            // (equal infinities: 1 at the largest, and none where all are -inf)
            p[q] = v[q] == top ? (top > -INFINITY ? 1.f : 0.f) : expf(v[q] - top);
            sum += p[q];
        }
        sum = wave_sum(sum);
#pragma unroll
        for (int q = 0; q < Q; ++q)
            p[q] = sum > 0.f ? p[q] / sum : 0.f;
    }
    unsigned key[Q];
#pragma unroll
    for (int q = 0; q < Q; ++q) {
        const int e = lane + 64 * q;
        key[q] = 0;
        if (e < r.E) {
            if (o.scores)
                o.scores[t * r.E + e] = p[q];
            key[q] = order_of(p[q] + bias[q]);
        }
    }
    if (r.keep < r.groups) {
        // lane: part `lane % sub` of group `lane / sub`
        const int size = r.group_size, sub = 64 >> r.group_bits;
        const int g = lane >> (6 - r.group_bits), part = lane & (sub - 1);
#pragma unroll
        for (int q = 0; q < Q; ++q)
            tmp[lane + 64 * q] = order_value(max(key[q], 0x007fffffu));   // (-inf past E)
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
        float m1 = -INFINITY, m2 = -INFINITY;
        if (g < r.groups)
            for (int i = part; i < size; i += sub) {
                const float c = tmp[g * size + i];
                m2 = fmaxf(m2, fminf(m1, c));
                m1 = fmaxf(m1, c);
            }
        for (int s = 1; s < sub; s <<= 1) {
            const float o1 = __shfl_xor(m1, s), o2 = __shfl_xor(m2, s);
            m2 = fmaxf(fmaxf(m2, o2), fminf(m1, o1));
            m1 = fmaxf(m1, o1);
        }
        // (lane g takes group g's value, so that the ballot finds the lowest group)
        const float score = r.best == 2 && size > 1 ? m1 + m2 : m1;
        const float mine = __shfl(score, min(lane, r.groups - 1) * sub);
        unsigned gk[1] = {lane < r.groups ? order_of(mine) : 0u};
        uint64_t kept = 0;
        for (int i = 0; i < r.keep; ++i) {
            unsigned b;
            kept |= 1ull << take_best<1>(gk, b);
        }
#pragma unroll
        for (int q = 0; q < Q; ++q) {
            const int e = lane + 64 * q;
            // (e / size for e < 256: the factor's error stays below 1 / 256)
            if (e < r.E && !(kept >> ((unsigned)e * r.group_factor >> 16) & 1ull))
                key[q] = 0;
        }
    }
    // choice j on lane j
    int my_e = 0;
    float my_v = -INFINITY, my_p = 0.f, top = -INFINITY;
    for (int j = 0; j < r.k; ++j) {
        unsigned b;
        const int e = take_best<Q>(key, b);
        float ev = v[0], ep = p[0];
#pragma unroll
        for (int q = 1; q < Q; ++q) {
            ev = e / 64 == q ? v[q] : ev;
            ep = e / 64 == q ? p[q] : ep;
        }
        ev = __uint_as_float((unsigned)__builtin_amdgcn_readlane((int)__float_as_uint(ev), e & 63));
        ep = __uint_as_float((unsigned)__builtin_amdgcn_readlane((int)__float_as_uint(ep), e & 63));
        top = fmaxf(top, ev);
        if (lane == j) {
            my_e = e;
            my_v = ev;
            my_p = ep;
        }
    }
    if (r.renorm) {
        // (of a softmax by the chosen scores themselves, which underflow later)
        if (!r.sigmoid)
            my_p = my_v == top ? (top > -INFINITY ? 1.f : 0.f) : expf(my_v - top);
        float den = 0.f;
        for (int j = 0; j < r.k; ++j)   // choice order
            den += __uint_as_float(
                (unsigned)__builtin_amdgcn_readlane((int)__float_as_uint(my_p), j));
        my_p = den > 0.f ? my_p / den : 0.f;
    }
    if (lane < r.k) {
        o.idx[t * r.k + lane] = my_e;
        o.gate[t * r.k + lane] = my_p * r.scale;
    }
}

// ---- scores --------------------------------------------------------------

// Eight fp32 columns of a row from p on, of which n exist: two 16-byte loads at any
// 4-byte address where the whole step exists.
__device__ __forceinline__ f32x8 load_f32(const float *p, int n, bool whole) {
    f32x8 v;
    if (whole) {
        __builtin_memcpy(&v, p, sizeof(v));
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            v[i] = i < n ? p[i] : 0.f;
    }
    return v;
}

// One workgroup: scores of 16 tokens for NT tiles of 16 experts, its NW waves
// taking every NW-th step of 32 columns, added in wave order, then a wave a token
// ranks them. (E <= 64)
template <typename S, int NT, int NW>
__global__ __launch_bounds__(NW * 64) void route_fused_kernel(
    const typename S::type *__restrict__ x, const float *__restrict__ wg,
    const float *__restrict__ noise, int N, int d, RouteRule r, RouteOut o) {
    constexpr bool BF16 = std::is_same<S, SkinnyBf16>::value;
    constexpr int EP = NT * 16;
    __shared__ float red[NW][16][EP + 1];
    __shared__ float tmp[NW][64];
    const int lane = threadIdx.x & 63, wv = threadIdx.x >> 6;
    const int row = lane & 15, ko = 8 * (lane >> 4);
    const int64_t t0 = (int64_t)blockIdx.x * 16;
    const typename S::type *xr = x + min(t0 + row, (int64_t)N - 1) * d;
    float bias[1];
    load_bias(r, bias);
    f32x4 acc[NT];
#pragma unroll
    for (int n = 0; n < NT; ++n)
        acc[n] = f32x4{0.f, 0.f, 0.f, 0.f};
    const int steps = (d + 31) / 32;
    // steps loaded at once (2047x4096x8: 13.5 us with 4, 13.9 with 8)
    constexpr int U = NT == 1 ? 4 : NT == 2 ? 2 : 1;
    for (int c0 = wv; c0 < steps; c0 += NW * U) {
        if constexpr (BF16) {
            u32x4 a[U];
            f32x4 w0[U][NT], w1[U][NT];
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int k = (c0 + u * NW) * 32 + ko, kc = k < d ? k : 0;   // (d % 8 == 0)
                a[u] = *reinterpret_cast<const u32x4 *>(xr + kc);
#pragma unroll
                for (int n = 0; n < NT; ++n) {
                    const float *w = wg + (int64_t)min(n * 16 + row, r.E - 1) * d + kc;
                    w0[u][n] = *reinterpret_cast<const f32x4 *>(w);
                    w1[u][n] = *reinterpret_cast<const f32x4 *>(w + 4);
                }
            }
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const bool ok = (c0 + u * NW) * 32 + ko < d;
                const f32x4 zf = {0.f, 0.f, 0.f, 0.f};
                const u32x4 xa = ok ? a[u] : u32x4{0u, 0u, 0u, 0u};
#pragma unroll
                for (int n = 0; n < NT; ++n) {
                    u32x4 term[3];
                    split8(ok ? w0[u][n] : zf, ok ? w1[u][n] : zf, term[0], term[1], term[2]);
#pragma unroll
                    for (int m = 0; m < 3; ++m)
                        acc[n] = SkinnyBf16::mma(xa, term[m], acc[n]);
                }
            }
        } else {
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int b = (c0 + u * NW) * 32, k = b + ko;
                const bool whole = b + 32 <= d;
                if (b >= d)
                    break;
                const f32x8 xa = load_f32(xr + k, d - k, whole);
                f32x8 w[NT];
#pragma unroll
                for (int n = 0; n < NT; ++n)
                    w[n] = load_f32(wg + (int64_t)min(n * 16 + row, r.E - 1) * d + k, d - k, whole);
#pragma unroll
                for (int n = 0; n < NT; ++n)
                    acc[n] = S::mma(xa, w[n], acc[n]);
            }
        }
    }
    // acc[n][q]: token 4 (lane / 16) + q, expert 16 n + lane % 16
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int q = 0; q < 4; ++q)
            red[wv][4 * (lane >> 4) + q][n * 16 + row] = acc[n][q];
    __syncthreads();
    for (int m = wv; m < 16; m += NW) {
        const int64_t t = t0 + m;
        if (t >= N)
            break;
        float s[1] = {0.f};
        if (lane < r.E) {
            s[0] = red[0][m][lane];
            for (int w = 1; w < NW; ++w)
                s[0] += red[w][m][lane];
            if (noise)
                s[0] += noise[t * r.E + lane];
        }
        route_rank<1>(s, bias, r, t, o, tmp[wv]);
    }
}

// Partial scores P[range][t][ld] of 16 experts and 16 TT tokens over one range of
// d (waves: quarters of it). grid: (token blocks x tiles of 16 experts, ranges).
// Expert e stands at column (e mod 64) Q + e / 64, as the ranking reads it.
template <typename S, int TT>
__global__ __launch_bounds__(256) void route_scores_kernel(
    const typename S::type *__restrict__ x, const float *__restrict__ wg, int N, int d, int E,
    int Q, int ld, float *__restrict__ P) {
    constexpr bool BF16 = std::is_same<S, SkinnyBf16>::value;
    __shared__ f32x4 part[4][TT][64];
    const int lane = threadIdx.x & 63, wv = threadIdx.x >> 6;
    const int row = lane & 15, ko = 8 * (lane >> 4);
    const unsigned et = (E + 15) / 16, tb = blockIdx.x / et;
    const int e0 = (int)(blockIdx.x - tb * et) * 16;
    const int64_t t0 = (int64_t)tb * (16 * TT);
    const float *w = wg + (int64_t)min(e0 + row, E - 1) * d;
    const typename S::type *xt[TT];
    f32x4 acc[TT];
#pragma unroll
    for (int i = 0; i < TT; ++i) {
        xt[i] = x + min(t0 + 16 * i + row, (int64_t)N - 1) * d;
        acc[i] = f32x4{0.f, 0.f, 0.f, 0.f};
    }
    const int steps = (d + 31) / 32, parts = gridDim.y * 4, me = blockIdx.y * 4 + wv;
    const int b = (int)((int64_t)me * steps / parts), e = (int)((int64_t)(me + 1) * steps / parts);
    constexpr int U = 4;
    for (int c = b; c < e; c += U) {
        if constexpr (BF16) {
            f32x4 w0[U], w1[U];
            u32x4 a[U][TT];
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int k = (c + u) * 32 + ko, kc = c + u < e && k < d ? k : 0;
                w0[u] = *reinterpret_cast<const f32x4 *>(w + kc);
                w1[u] = *reinterpret_cast<const f32x4 *>(w + kc + 4);
#pragma unroll
                for (int i = 0; i < TT; ++i)
                    a[u][i] = *reinterpret_cast<const u32x4 *>(xt[i] + kc);
            }
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const bool ok = c + u < e && (c + u) * 32 + ko < d;
                const f32x4 zf = {0.f, 0.f, 0.f, 0.f};
                u32x4 term[3];
                split8(ok ? w0[u] : zf, ok ? w1[u] : zf, term[0], term[1], term[2]);
#pragma unroll
                for (int i = 0; i < TT; ++i) {
                    const u32x4 xa = ok ? a[u][i] : u32x4{0u, 0u, 0u, 0u};
#pragma unroll
                    for (int m = 0; m < 3; ++m)
                        acc[i] = SkinnyBf16::mma(xa, term[m], acc[i]);
                }
            }
        } else {
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int k = (c + u) * 32 + ko;
                const bool whole = (c + u) * 32 + 32 <= d;
                if (c + u >= e)
                    break;
                const f32x8 wf = load_f32(w + k, d - k, whole);
                f32x8 xa[TT];
#pragma unroll
                for (int i = 0; i < TT; ++i)
                    xa[i] = load_f32(xt[i] + k, d - k, whole);
#pragma unroll
                for (int i = 0; i < TT; ++i)
                    acc[i] = S::mma(xa[i], wf, acc[i]);
            }
        }
    }
#pragma unroll
    for (int i = 0; i < TT; ++i)
        part[wv][i][lane] = acc[i];
    __syncthreads();
    for (int q = threadIdx.x; q < TT * 64; q += 256) {
        const int i = q >> 6, l = q & 63, ex = e0 + (l & 15);
        f32x4 v = part[0][i][l];
#pragma unroll
        for (int s = 1; s < 4; ++s)
            v += part[s][i][l];
#pragma unroll
        for (int c = 0; c < 4; ++c) {
            const int64_t t = t0 + 16 * i + 4 * (l >> 4) + c;
            if (t < N && ex < E)
                P[((int64_t)blockIdx.y * N + t) * ld + ex % 64 * Q + ex / 64] = v[c];
        }
    }
}

// Ranking of partial scores, one wave a token: the ranges added in order.
template <int Q>
__global__ __launch_bounds__(256) void route_rank_kernel(const float *__restrict__ P, int ns,
                                                         int ld, const float *__restrict__ noise,
                                                         int N, RouteRule r, RouteOut o) {
    __shared__ float tmp[4][64 * Q];
    typedef float vec __attribute__((ext_vector_type(Q == 1 ? 2 : Q)));   // (Q == 1: v[0])
    const int lane = threadIdx.x & 63, wv = threadIdx.x >> 6;
    const int64_t t = (int64_t)blockIdx.x * 4 + wv;
    if (t >= N)
        return;
    float nz[Q], bias[Q];
    load_bias(r, bias);
#pragma unroll
    for (int q = 0; q < Q; ++q) {
        const int e = lane + 64 * q;
        nz[q] = noise && e < r.E ? noise[t * r.E + e] : 0.f;
    }
    const float *p = P + t * ld + min(lane * Q, ld - Q);
    const int64_t step = (int64_t)N * ld;
    auto load = [&](int s) {
        vec v = {};
        if constexpr (Q == 1)
            v[0] = p[s * step];
        else
            v = *reinterpret_cast<const vec *>(p + s * step);
        return v;
    };
    constexpr int B = 16;   // loads in flight
    vec sum = load(0);
    for (int s = 1; s < ns; s += B) {
        vec u[B];
#pragma unroll
        for (int c = 0; c < B; ++c)
            u[c] = load(min(s + c, ns - 1));
#pragma unroll
        for (int c = 0; c < B; ++c)
            if (s + c < ns)
                sum += u[c];
    }
    float v[Q];
#pragma unroll
    for (int q = 0; q < Q; ++q)
        v[q] = noise ? sum[q] + nz[q] : sum[q];
    route_rank<Q>(v, bias, r, t, o, tmp[wv]);
}

size_t up256(size_t v) { return (v + 255) / 256 * 256; }

}  // namespace

size_t route_workspace_bytes(bool bf16, int64_t N, int64_t d, int E) {
    N = std::min(N, kRouteTokens);
    const RoutePlan p = route_plan(bf16, N, d, E);
    if (p.form == kFused)
        return 0;
    if (p.form == kTiled)
        return router_workspace_bytes(N, d, E);
    return up256((size_t)p.ranges * N * p.ld * 4);
}

// The launches of at most kRouteTokens tokens.
static hipError_t route_part(bool bf16, const RoutePlan &p, const void *xv, const float *wg,
                             const float *noise, int64_t N, int64_t d, const RouteRule &r,
                             int32_t *idx, float *gate, float *scores, void *ws, hipStream_t s) {
    const RouteOut o{idx, gate, scores};
    float *P = static_cast<float *>(ws);
    int ns = p.ranges;
    auto scores_by = [&](auto kind) {
        typedef decltype(kind) S;
        const typename S::type *x = static_cast<const typename S::type *>(xv);
        if (p.form == kFused) {
            const unsigned blocks = (unsigned)((N + 15) / 16);
            auto go = [&](auto nt, auto nw) {
                constexpr int NT = decltype(nt)::value, NW = decltype(nw)::value;
                moeLaunchKernelGGL((route_fused_kernel<S, NT, NW>), dim3(blocks), dim3(NW * 64), 0,
                                   s, x, wg, noise, (int)N, (int)d, r, o);
                return hipGetLastError();
            };
            // A workgroup that has its CU to itself keeps more loads in flight with more
            // waves; more workgroups do that for each other. 4 and 16 waves, us: 4096 tokens
            // of 8 experts of 512 8.0 and 8.7, of 2304 12.9 and 10.8, 32 of 2048 16.4 and
            // 13.7; 8192 of 8 of 768 10.8 and 14.2, of 2048 15.3 and 14.8, 32 of 768 13.5
            // and 15.3; 65536 of 8 of 1024 43 and 102, 32 of 1024 78 and 110. fp32: 8192 of
            // 8 of 768 12.0 and 9.5, 16384 of 16 of 1000 20.2 and 19.5, 65536 84 and 89.
            // With 64 experts 8 waves throughout (4096 of 576 11.8 and 9.2, 65536 79 and 76).
            auto by_blocks = [&](auto nt) {
                return blocks <= (bf16 ? 256u : 1024u) ? go(nt, std::integral_constant<int, 16>{})
                                                       : go(nt, std::integral_constant<int, 4>{});
            };
            return r.E <= 16   ? by_blocks(std::integral_constant<int, 1>{})
                   : r.E <= 32 ? by_blocks(std::integral_constant<int, 2>{})
                               : go(std::integral_constant<int, 4>{},
                                    std::integral_constant<int, 8>{});
        }
        auto go = [&](auto tiles) {
            constexpr int TT = decltype(tiles)::value;
            moeLaunchKernelGGL((route_scores_kernel<S, TT>),
                               dim3((unsigned)((r.E + 15) / 16 * ((N + 16 * TT - 1) / (16 * TT))),
                                    (unsigned)p.ranges),
                               dim3(256), 0, s, x, wg, (int)N, (int)d, r.E, p.Q, p.ld, P);
            return hipGetLastError();
        };
        return p.tt == 1   ? go(std::integral_constant<int, 1>{})
               : p.tt == 2 ? go(std::integral_constant<int, 2>{})
                           : go(std::integral_constant<int, 4>{});
    };
    hipError_t err;
    if (p.form == kTiled)
        err = launch_router_partials(xv, wg, N, d, r.E, ws, P, ns, s);
    else if (bf16)
        err = scores_by(SkinnyBf16{});
    else
        err = scores_by(SkinnyF32<true>{});   // (its products; the loads are load_f32's)
    if (err != hipSuccess || p.form == kFused)
        return err;
    auto rank = [&](auto q) {
        constexpr int Q = decltype(q)::value;
        moeLaunchKernelGGL((route_rank_kernel<Q>), dim3((unsigned)((N + 3) / 4)), dim3(256), 0, s,
                           (const float *)P, ns, p.ld, noise, (int)N, r, o);
        return hipGetLastError();
    };
    return p.Q == 1   ? rank(std::integral_constant<int, 1>{})
           : p.Q == 2 ? rank(std::integral_constant<int, 2>{})
                      : rank(std::integral_constant<int, 4>{});
}

hipError_t launch_route(bool bf16, const void *x, const float *wg, const float *noise, int64_t N,
                        int64_t d, const RouteRule &r, int32_t *idx, float *gate, float *scores,
                        void *ws, hipStream_t s) {
    // one part after the other in the same scratch
    const RoutePlan p = route_plan(bf16, std::min(N, kRouteTokens), d, r.E);
    for (int64_t t = 0; t < N; t += kRouteTokens) {
        const hipError_t err = route_part(
            bf16, p, static_cast<const char *>(x) + t * d * (bf16 ? 2 : 4), wg,
            noise ? noise + t * r.E : nullptr, std::min(N - t, kRouteTokens), d, r, idx + t * r.k,
            gate + t * r.k, scores ? scores + t * r.E : nullptr, ws, s);
        if (err != hipSuccess)
            return err;
    }
    return hipSuccess;
}

}  // namespace moe
