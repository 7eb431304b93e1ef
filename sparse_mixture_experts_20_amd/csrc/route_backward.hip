// Backward of the routing (route.hip): from the gradient of the gates (and, for
// an auxiliary loss, of the scores p) to those of the router's input and weights.
//
//   renormalised gates: S = sum of the chosen p, u_j = p_j / S (the gates over scale),
//                       dp_j = scale / S (dg_j - sum_l u_l dg_l)
//   gates as they are:  dp_j = scale dg_j
//   sigmoid: ds = dp p (1 - p);  softmax: ds = p (dp - sum over all E of dp p)
//   dW_g = ds^T x,  dx = ds W_g + dres
//
// The choice itself (bias, groups, top-k) passes no gradient. With a sigmoid, or
// with renormalised softmax gates (whose normaliser cancels), and no dp of an
// auxiliary loss, ds has k values a token; otherwise E.
//
// dW_g: ds as three exact bf16 terms (as the layer's own backward), the terms of
// all experts beside each other in one [N, 3 E] operand of the tiled product, its
// reduction over the tokens cut into ranges whose partial products a last kernel
// adds, terms and ranges in a fixed order. dx with k values: W_g's columns lie in
// LDS in fp32, 2 or 4 a lane, and a wave adds k rows of them for each token: bound
// by dres and dx. dx with E values: the tiled product of split operands, six
// products of terms (fp32's accuracy, for bf16 dx too: three of them, 2^-16, rounded
// one element of 90 otherwise; 8192 tokens, 256 experts of 7168 then took 283 us, with
// six 377, 2047 tokens, 8 experts of 768 24 either way).
//
// Measured (calls; kernels from a trace of the same, a little longer): 8192 tokens, 256
// experts of 7168, fp32 dx with dres 236 us: ds 9, dW_g 96 to 99 (90 GFLOP of terms, 0.9
// PFLOP/s) and 13 for the sums, dx 119 to 125 (470 MB, 3.9 TB/s); bf16 dx of all scores
// 368, of which its six products 253 (180 GFLOP). 2047 tokens, 8 experts of 768 with an
// auxiliary loss 24.5 in four launches.
#include <algorithm>
#include <type_traits>

#include "common.hpp"
#include "ranking.hpp"
#include "tile.hpp"

namespace moe {
namespace {

__device__ __forceinline__ float sum_of_wave(float v) {
#pragma unroll
    for (int o = 32; o >= 1; o >>= 1)
        v += __shfl_xor(v, o);
    return v;
}
// The three bf16 terms of v.
__device__ __forceinline__ void terms_of(float v, unsigned short (&t)[3]) {
    unsigned h, m, l;
    split3x2(v, 0.f, h, m, l);
    t[0] = (unsigned short)h;
    t[1] = (unsigned short)m;
    t[2] = (unsigned short)l;
}
// Terms of ds and of W_g in each of the products of dx (those below 2^-24 left out).
constexpr int kProducts = 6;
constexpr int kDsTerm[kProducts] = {0, 0, 1, 1, 0, 2};
constexpr int kWgTerm[kProducts] = {0, 1, 0, 1, 2, 0};

struct RouteGrad {
    const int32_t *idx;       // [N, k]
    const float *p;           // [N, E]
    const float *dgate;       // [N, k]
    const float *gates;       // [N, k], or NULL: the shares are formed from p
    const float *dp;          // [N, E] or NULL
    int E, Ep, k;             // Ep: E rounded up to 8
    int sigmoid, renorm;
    float scale;
    float *ds;                // [N, k] (k values a token), or NULL
    unsigned short *ds3;      // [N][3][Ep]
    unsigned short *dsx;      // [N][kProducts][Ep] (E values a token), or NULL
};

// The terms of W_g [E, d] as the products of dx take them: [kProducts Ep][d].
__device__ __forceinline__ void route_split(const float *__restrict__ wg, int E, int Ep, int d,
                                            unsigned short *__restrict__ out,
                                            int64_t i) {   // 8 columns
    const int per = d / 8;
    if (i >= (int64_t)Ep * per)
        return;
    const int e = (int)(i / per), c = (int)(i - (int64_t)e * per) * 8;
    f32x4 a = {0.f, 0.f, 0.f, 0.f}, b = a;
    if (e < E) {
        a = *reinterpret_cast<const f32x4 *>(wg + (int64_t)e * d + c);
        b = *reinterpret_cast<const f32x4 *>(wg + (int64_t)e * d + c + 4);
    }
    u32x4 t[3];
    split8(a, b, t[0], t[1], t[2]);
#pragma unroll
    for (int m = 0; m < kProducts; ++m)
        *reinterpret_cast<u32x4 *>(out + ((int64_t)m * Ep + e) * d + c) = t[kWgTerm[m]];
}

// ds of one token per wave; lane l holds experts l, l + 64, ... and choice l. The
// workgroups past the tokens' (with E values a token) split W_g into wx.
template <int Q>
__global__ __launch_bounds__(256) void route_ds_kernel(RouteGrad r, int N,
                                                       const float *__restrict__ wg, int width,
                                                       unsigned short *__restrict__ wx) {
    const int blocks = (N + 3) / 4;
    if ((int)blockIdx.x >= blocks) {
        route_split(wg, r.E, r.Ep, width, wx,
                    (int64_t)(blockIdx.x - blocks) * 256 + threadIdx.x);
        return;
    }
    const int lane = threadIdx.x & 63;
    const int64_t t = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6);
    if (t >= N)
        return;
    int e = -1;
    float dg = 0.f, pc = 0.f, gate = 0.f;
    if (lane < r.k) {
        e = r.idx[t * r.k + lane];
        if (e < 0 || e >= r.E) {
            e = -1;   // no expert: no gate, no gradient
        } else {
            dg = r.dgate[t * r.k + lane];
            pc = r.p[t * r.E + e];
            gate = r.renorm && r.gates ? r.gates[t * r.k + lane] : 0.f;
        }
    }
    // Gates of a sigmoid, or renormalised, pass their gradient to the chosen scores
    // alone (the sum of dp p over the choices is 0): dc is then of s, else of p.
    const bool direct = r.renorm || r.sigmoid;
    float dc = r.scale * dg;
    if (r.renorm) {
        float S = 0.f, ug = 0.f;
        for (int j = 0; j < r.k; ++j)   // choice order
            S += __uint_as_float(
                (unsigned)__builtin_amdgcn_readlane((int)__float_as_uint(pc), j));
        // (1 / S may be past fp32; the forward's gates do not underflow with p)
        const float share = r.gates ? gate / r.scale : S > 0.f ? pc / S : 0.f;
        for (int j = 0; j < r.k; ++j) {
            const float sj = __uint_as_float(
                (unsigned)__builtin_amdgcn_readlane((int)__float_as_uint(share), j));
            const float gj = __uint_as_float(
                (unsigned)__builtin_amdgcn_readlane((int)__float_as_uint(dg), j));
            ug = fmaf(sj, gj, ug);
        }
        dc = r.scale * share * (dg - ug);
    } else if (r.sigmoid) {
        dc *= pc;
    }
    if (r.sigmoid)
        dc *= 1.f - pc;
    if (e < 0)
        dc = 0.f;
    if (r.ds && lane < r.k)
        r.ds[t * r.k + lane] = dc;
    float p[Q], d[Q];
    float dot = 0.f;
#pragma unroll
    for (int q = 0; q < Q; ++q) {
        const int ex = lane + 64 * q;
        p[q] = r.dsx && ex < r.E ? r.p[t * r.E + ex] : 0.f;
        d[q] = r.dp && ex < r.E ? r.dp[t * r.E + ex] : 0.f;
    }
    auto choices = [&] {
        for (int j = 0; j < r.k; ++j) {
            const int ej = __builtin_amdgcn_readlane(e, j);
            const float v = __uint_as_float(
                (unsigned)__builtin_amdgcn_readlane((int)__float_as_uint(dc), j));
#pragma unroll
            for (int q = 0; q < Q; ++q)
                if (ej == lane + 64 * q)
                    d[q] += v;
        }
    };
    if (!direct)
        choices();
    if (r.dsx) {
        if (r.sigmoid) {
#pragma unroll
            for (int q = 0; q < Q; ++q)
                d[q] *= p[q] * (1.f - p[q]);
        } else {
#pragma unroll
            for (int q = 0; q < Q; ++q)
                dot = fmaf(d[q], p[q], dot);
            dot = sum_of_wave(dot);
#pragma unroll
            for (int q = 0; q < Q; ++q)
                d[q] = p[q] * (d[q] - dot);
        }
    }
    if (direct)
        choices();
#pragma unroll
    for (int q = 0; q < Q; ++q) {
        const int ex = lane + 64 * q;
        if (ex >= r.Ep)
            continue;
        unsigned short term[3];
        terms_of(d[q], term);
        unsigned short *o = r.ds3 + t * 3 * r.Ep + ex;
#pragma unroll
        for (int m = 0; m < 3; ++m)
            o[m * r.Ep] = term[m];
        if (r.dsx) {
            unsigned short *ox = r.dsx + t * kProducts * r.Ep + ex;
#pragma unroll
            for (int m = 0; m < kProducts; ++m)
                ox[m * r.Ep] = term[kDsTerm[m]];
        }
    }
}

// Partial dW_g terms: part[range][3 Ep][d] = ds3^T x over the range's tokens.
// grid: (tiles, ranges).
template <int BM, int BN, int WM, int WN, int S>
__global__ __launch_bounds__(WM *WN * 64) void route_dw_kernel(
    const unsigned short *__restrict__ ds3, const unsigned short *__restrict__ x, int rows, int d,
    int N, float *__restrict__ part) {
    typedef TileProduct<BM, BN, WM, WN, S, true, true> Tile;
    __shared__ __attribute__((aligned(1024))) char smem[Tile::LDS];
    const int tn = (d + BN - 1) / BN;
    const int m0 = (int)(blockIdx.x / tn) * BM, n0 = (int)(blockIdx.x % tn) * BN;
    const int KT = (N + kStep - 1) / kStep;
    const int kb = (int)((int64_t)blockIdx.y * KT / gridDim.y);
    const int ke = (int)((int64_t)(blockIdx.y + 1) * KT / gridDim.y);
    f32x4 acc[Tile::FM][Tile::FN];
#pragma unroll
    for (int i = 0; i < Tile::FM; ++i)
#pragma unroll
        for (int j = 0; j < Tile::FN; ++j)
            acc[i][j] = f32x4{0.f, 0.f, 0.f, 0.f};
    Tile::run(
        smem, [&](int r) { return ds3 + min(m0 + 8 * r, rows - 8); }, rows,
        [&](int r) { return x + min(n0 + 8 * r, d - 8); }, d, N, kb, ke, acc);
    const int lane = threadIdx.x & 63;
    const int wv = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int n = n0 + wv % WN * 64 + 16 * (lane >> 4);
    float *o = part + (int64_t)blockIdx.y * rows * d;
#pragma unroll
    for (int i = 0; i < Tile::FM; ++i) {
        const int m = m0 + (wv / WN * Tile::FM + i) * 16 + (lane & 15);
        if (m < rows)
#pragma unroll
            for (int j = 0; j < Tile::FN; ++j)
                if (n + 4 * j < d)
                    *reinterpret_cast<f32x4 *>(o + (int64_t)m * d + n + 4 * j) = acc[i][j];
    }
}

// dW_g[e] = the ranges' terms of expert e, smallest terms first. 4 columns a thread.
__global__ __launch_bounds__(256) void route_dw_sum_kernel(const float *__restrict__ part, int S,
                                                           int E, int Ep, int d,
                                                           float *__restrict__ dW) {
    const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
    if (i >= (int64_t)E * (d / 4))
        return;
    const int64_t plane = (int64_t)Ep * d;
    const float *p = part + i * 4;
    f32x4 v = {0.f, 0.f, 0.f, 0.f};
    constexpr int B = 8;   // loads in flight
    for (int q = 0; q < 3 * S; q += B) {
        f32x4 u[B];
#pragma unroll
        for (int b = 0; b < B; ++b) {
            const int o = min(q + b, 3 * S - 1);   // term 2 - o / S of range o % S
            u[b] = *reinterpret_cast<const f32x4 *>(p + ((o % S) * 3 + 2 - o / S) * plane);
        }
#pragma unroll
        for (int b = 0; b < B; ++b)
            if (q + b < 3 * S)
                v += u[b];
    }
    *reinterpret_cast<f32x4 *>(dW + i * 4) = v;
}

// Rows of dx: fp32 or bf16, V adjacent values.
template <bool F32, int V>
struct Rows {
    typedef float vec __attribute__((ext_vector_type(V)));
    static __device__ __forceinline__ vec load(const void *p, int64_t o) {
        vec v;
        if constexpr (F32) {
            v = *reinterpret_cast<const vec *>(static_cast<const float *>(p) + o);
        } else {
            unsigned w[V / 2];
            __builtin_memcpy(w, __builtin_assume_aligned(
                                    static_cast<const unsigned short *>(p) + o, 2 * V), 2 * V);
#pragma unroll
            for (int i = 0; i < V / 2; ++i) {
                v[2 * i] = __uint_as_float(w[i] << 16);
                v[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
            }
        }
        return v;
    }
    static __device__ __forceinline__ void store(void *p, int64_t o, const vec &v) {
        if constexpr (F32) {
            *reinterpret_cast<vec *>(static_cast<float *>(p) + o) = v;
        } else {
            unsigned w[V / 2];
#pragma unroll
            for (int i = 0; i < V / 2; ++i)
                w[i] = pack_bf16x2(v[2 * i], v[2 * i + 1]);
            __builtin_memcpy(__builtin_assume_aligned(static_cast<unsigned short *>(p) + o, 2 * V),
                             w, 2 * V);
        }
    }
};

// dx = dres + sum_j ds_j W_g[idx_j], choices in order. grid: (blocks of 64 V
// columns, groups of tokens); W_g's columns of the block in LDS (E x 64 V fp32, and a
// row of zeros for ids that are no expert: a branch around them took 256 us, this 236).
template <bool F32, int V>
__global__ __launch_bounds__(1024) void route_dx_kernel(
    const float *__restrict__ ds, const int32_t *__restrict__ idx, const float *__restrict__ wg,
    const void *__restrict__ dres, int N, int d, int E, int k, void *__restrict__ dx) {
    extern __shared__ __attribute__((aligned(16))) float w[];   // [E + 1][64 V]
    typedef Rows<F32, V> R;
    constexpr int C = 64 * V;
    const int lane = threadIdx.x & 63;
    const int wv = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int c0 = blockIdx.x * C, c = c0 + V * lane;
    const bool ok = c < d;   // (d % 8 == 0)
    for (int i = threadIdx.x; i < (E + 1) * (C / 4); i += 1024) {
        const int e = i / (C / 4), q = i % (C / 4) * 4;
        f32x4 v = {0.f, 0.f, 0.f, 0.f};
        if (e < E && c0 + q < d)
            v = *reinterpret_cast<const f32x4 *>(wg + (int64_t)e * d + c0 + q);
        *reinterpret_cast<f32x4 *>(w + e * C + q) = v;
    }
    __syncthreads();
    // U tokens of a wave in flight; lane 16 u + j holds choice j of token u (its id
    // and ds are broadcast from there: read one by one they were a chain of scalar
    // loads, 217 us for the fine-grained batch)
    constexpr int U = 4;
    static_assert(kMaxTopK <= 16 && U * 16 <= 64, "a lane per choice");
    const int64_t waves = (int64_t)gridDim.y * 16;
    const int hu = lane >> 4, hj = lane & 15;
    struct Choice {
        int e;
        float g;
    };
    auto choices = [&](int64_t t0) {
        const int64_t t = t0 + hu * waves;
        Choice c{E, 0.f};
        if (hj < k && t < N) {
            c.e = idx[t * k + hj];
            c.g = ds[t * k + hj];
        }
        if (c.e < 0 || c.e >= E)
            c = Choice{E, 0.f};   // no expert: nothing, whatever W_g holds
        return c;
    };
    int64_t t0 = (int64_t)blockIdx.y * 16 + wv;
    if (t0 >= N)
        return;
    Choice next = choices(t0);
    for (; t0 < N; t0 += waves * U) {
        const Choice mine = next;
        typename R::vec a[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int64_t t = min(t0 + u * waves, (int64_t)N - 1);
            a[u] = typename R::vec{};
            if (dres)
                a[u] = R::load(dres, t * d + min(c, d - V));
        }
        next = choices(t0 + waves * U);
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int64_t t = t0 + u * waves;
            if (t >= N)
                break;
            typename R::vec s = {};
#pragma unroll 4
            for (int j = 0; j < k; ++j) {
                const int e = __builtin_amdgcn_readlane(mine.e, 16 * u + j);
                const float g = __uint_as_float((unsigned)__builtin_amdgcn_readlane(
                    (int)__float_as_uint(mine.g), 16 * u + j));
                const typename R::vec v =
                    *reinterpret_cast<const typename R::vec *>(w + e * C + V * lane);
#pragma unroll
                for (int i = 0; i < V; ++i)
                    s[i] = fmaf(g, v[i], s[i]);
            }
            if (ok)
                R::store(dx, t * d + c, a[u] + s);
        }
    }
}

// dx = dres + dsx Wx: dsx [N][K], Wx [K][d] bf16.
template <bool F32>
__global__ __launch_bounds__(512) void route_dx_dense_kernel(
    const unsigned short *__restrict__ dsx, const unsigned short *__restrict__ wx,
    const void *__restrict__ dres, int N, int d, int K, void *__restrict__ dx) {
    typedef TileProduct<128, 128, 4, 2, 2, false, true> Tile;
    typedef Rows<F32, 4> R;
    __shared__ __attribute__((aligned(1024))) char smem[Tile::LDS];
    const int tn = (d + 127) / 128;
    const int64_t m0 = (int64_t)(blockIdx.x / tn) * 128;
    const int n0 = (int)(blockIdx.x % tn) * 128;
    f32x4 acc[Tile::FM][Tile::FN];
#pragma unroll
    for (int i = 0; i < Tile::FM; ++i)
#pragma unroll
        for (int j = 0; j < Tile::FN; ++j)
            acc[i][j] = f32x4{0.f, 0.f, 0.f, 0.f};
    Tile::run(
        smem, [&](int r) { return dsx + min(m0 + r, (int64_t)N - 1) * K; }, 0,
        [&](int r) { return wx + min(n0 + 8 * r, d - 8); }, d, K, 0, (K + kStep - 1) / kStep, acc);
    const int lane = threadIdx.x & 63;
    const int wv = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int n = n0 + wv % 2 * 64 + 16 * (lane >> 4);
#pragma unroll
    for (int i = 0; i < Tile::FM; ++i) {
        const int64_t m = m0 + (wv / 2 * Tile::FM + i) * 16 + (lane & 15);
        if (m >= N)
            continue;
#pragma unroll
        for (int j = 0; j < Tile::FN; ++j) {
            const int64_t o = m * d + n + 4 * j;
            if (n + 4 * j >= d)
                continue;
            f32x4 v = acc[i][j];
            if (dres)
                v += R::load(dres, o);
            R::store(dx, o, v);
        }
    }
}

size_t up256(size_t v) { return (v + 255) / 256 * 256; }

// Tiles and token ranges of dW_g, timed in turn (with ds and the sums, us). 256x256
// tiles, a workgroup a CU, for long products whose rows fill them: 256 experts of 7168,
// 4096 tokens 72 (128x128 77), 8192 109 (130), 16384 180 (228), 160 experts 8192 91 (100);
// but 2048 57 (49), 256 experts of 2048, 8192 62 (51), of 4096, 4096 58 (52), 128 of 7168,
// 8192 83 (77). Otherwise 64 or 128 rows by 128 columns; more ranges give more workgroups
// and more partial sums, so one a CU, or two where the tiles are many: for 256, 512 and
// 1024 workgroups 8 experts of 4096, 8192 tokens 25, 27, 35, 16 of 768, 32768 44, 60, 76,
// 32 of 2048, 16384 37, 45, 66, 64 of 7168, 8192 67, 54, 67, 128 of 7168, 8192 132, 77, 93.
struct DwShape {
    int bm, bn;
    int64_t tiles;
    int ranges;
};
DwShape dw_shape(int64_t N, int64_t d, int rows) {
    DwShape s;
    s.bm = rows >= 448 && (double)N * d * rows > 2.1e10 ? 256 : rows > 64 ? 128 : 64;
    s.bn = s.bm == 256 ? 256 : 128;
    s.tiles = (rows + s.bm - 1) / s.bm * ((d + s.bn - 1) / s.bn);
    const int64_t want = s.bm == 128 && s.tiles >= 80 ? 512 : 256, steps = (N + kStep - 1) / kStep;
    s.ranges = (int)std::min<int64_t>(std::max<int64_t>(want / s.tiles, 1),
                                      std::max<int64_t>(steps / 4, 1));
    return s;
}
int padded(int E) { return (E + 7) / 8 * 8; }

}  // namespace

RouteBackwardLayout route_backward_layout(int64_t N, int64_t d, int E, int k, bool dense) {
    RouteBackwardLayout L;
    const int Ep = padded(E), products = dense ? kProducts : 0;
    size_t o = 0;
    L.ds = o;   o += up256((size_t)N * k * 4);
    L.ds3 = o;  o += up256((size_t)N * 3 * Ep * 2);
    L.part = o; o += up256((size_t)dw_shape(N, d, 3 * Ep).ranges * 3 * Ep * d * 4);
    L.dsx = o;  o += up256((size_t)N * products * Ep * 2);
    L.wx = o;   o += up256((size_t)products * Ep * d * 2);
    L.total = o;
    return L;
}

hipError_t launch_route_backward(const void *x, const float *wg, const int32_t *idx,
                                 const float *p, const float *dgate, const float *dp,
                                 const void *dres, int64_t N, int64_t d, int E, int k, int sigmoid,
                                 int renorm, float scale, const float *gates, void *dx, bool dx32,
                                 float *dW, void *ws, hipStream_t s) {
    const bool dense = route_backward_dense(sigmoid, renorm, dp != nullptr);
    const int Ep = padded(E);
    const RouteBackwardLayout L = route_backward_layout(N, d, E, k, dense);
    char *w = static_cast<char *>(ws);
    float *ds = reinterpret_cast<float *>(w + L.ds), *part = reinterpret_cast<float *>(w + L.part);
    unsigned short *ds3 = reinterpret_cast<unsigned short *>(w + L.ds3);
    unsigned short *dsx = reinterpret_cast<unsigned short *>(w + L.dsx);
    unsigned short *wx = reinterpret_cast<unsigned short *>(w + L.wx);
    RouteGrad r{idx, p, dgate, gates, dp, E, Ep, k, sigmoid, renorm, scale, ds, ds3, nullptr};
    if (dense)
        r.dsx = dsx;
    hipError_t err;
    for (int64_t t = 0; t < N; t += kRouteTokens) {
        const int n = (int)std::min(N - t, kRouteTokens);
        const bool split = dense && dx && t == 0;   // the first launch takes W_g as well
        const dim3 tb((unsigned)((n + 3) / 4 + (split ? ((int64_t)Ep * (d / 8) + 255) / 256 : 0)));
        RouteGrad q = r;
        q.idx += t * k;
        q.p += t * E;
        q.dgate += t * k;
        q.gates += gates ? t * k : 0;
        q.dp += dp ? t * E : 0;
        q.ds += t * k;
        q.ds3 += t * 3 * Ep;
        q.dsx += dense ? t * kProducts * Ep : 0;
        if (E <= 64)
            moeLaunchKernelGGL(route_ds_kernel<1>, tb, dim3(256), 0, s, q, n, wg, (int)d, wx);
        else if (E <= 128)
            moeLaunchKernelGGL(route_ds_kernel<2>, tb, dim3(256), 0, s, q, n, wg, (int)d, wx);
        else
            moeLaunchKernelGGL(route_ds_kernel<4>, tb, dim3(256), 0, s, q, n, wg, (int)d, wx);
        if ((err = hipGetLastError()) != hipSuccess)
            return err;
    }
    if (dW) {
        const int rows = 3 * Ep;
        const DwShape sh = dw_shape(N, d, rows);
        const unsigned short *xs = static_cast<const unsigned short *>(x);
        const dim3 grid((unsigned)sh.tiles, (unsigned)sh.ranges);
        if (sh.bm == 256)
            moeLaunchKernelGGL((route_dw_kernel<256, 256, 4, 4, 2>), grid, dim3(1024), 0, s, ds3,
                               xs, rows, (int)d, (int)N, part);
        else if (sh.bm == 128)
            moeLaunchKernelGGL((route_dw_kernel<128, 128, 4, 2, 2>), grid, dim3(512), 0, s, ds3,
                               xs, rows, (int)d, (int)N, part);
        else
            moeLaunchKernelGGL((route_dw_kernel<64, 128, 4, 2, 2>), grid, dim3(512), 0, s, ds3, xs,
                               rows, (int)d, (int)N, part);
        if ((err = hipGetLastError()) != hipSuccess)
            return err;
        moeLaunchKernelGGL(route_dw_sum_kernel, dim3((unsigned)((E * (d / 4) + 255) / 256)),
                           dim3(256), 0, s, (const float *)part, sh.ranges, E, Ep, (int)d, dW);
        if ((err = hipGetLastError()) != hipSuccess)
            return err;
    }
    if (!dx)
        return hipSuccess;
    if (dense) {
        const int K = kProducts * Ep;
        const dim3 grid((unsigned)((N + 127) / 128 * ((d + 127) / 128)));
        if (dx32)
            moeLaunchKernelGGL(route_dx_dense_kernel<true>, grid, dim3(512), 0, s, dsx, wx, dres,
                               (int)N, (int)d, K, dx);
        else
            moeLaunchKernelGGL(route_dx_dense_kernel<false>, grid, dim3(512), 0, s, dsx, wx, dres,
                               (int)N, (int)d, K, dx);
        return hipGetLastError();
    }
    // columns a lane: 4, or 2 where the experts' columns would not fit LDS
    auto go = [&](auto f32, auto v) {
        constexpr int V = decltype(v)::value;
        const int64_t blocks = (d + 64 * V - 1) / (64 * V);
        const size_t lds = (size_t)(E + 1) * 64 * V * 4;
        // (1024 threads each; one and two with 8 experts of 4096, 8192 tokens 53 and 51 us,
        // with 64 56 and 53, 32 of 768, 2048 tokens 8.0 and 8.6)
        const int64_t per_cu = lds <= 80 * 1024 ? 2 : 1;
        const int64_t groups = std::min<int64_t>(std::max<int64_t>(256 * per_cu / blocks, 1),
                                                 (N + 15) / 16);
        moeLaunchKernelGGL((route_dx_kernel<decltype(f32)::value, V>),
                           dim3((unsigned)blocks, (unsigned)groups), dim3(1024), lds, s,
                           (const float *)ds, idx, wg, dres, (int)N, (int)d, E, k, dx);
        return hipGetLastError();
    };
    auto wide = [&](auto f32) {
        return E <= 128 ? go(f32, std::integral_constant<int, 4>{})
                        : go(f32, std::integral_constant<int, 2>{});
    };
    return dx32 ? wide(std::true_type{}) : wide(std::false_type{});
}

}  // namespace moe
