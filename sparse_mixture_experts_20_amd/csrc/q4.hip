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
// weights (0x4300 | q: bf16 has a step of 1 there), exactly. The MFMAs accumulate
// sum x (128 + q) of a group and take 136 times the sum of x off it (symmetric
// weights), or give that sum beside it (zero points), and one or two fp32
// operations per group add scale (sum x (128 + q) - (128 + zero) sum x). Every
// product is exact in the fp32 accumulator; the subtraction cancels at most 7 bits
// or so of its 24. The weights are the MFMA's columns, so a lane holds one weight
// row's results and needs that row's scales alone.
//
// A group must not share an MFMA with another: 32 K-positions, 8 from each
// quarter of the wave. The 16 bytes of a quarter hold 32 consecutive weights, so
// groups of 128 need nothing, and groups of 64 and 32 swap registers between
// halves and quarters of the wave (2 and 4 swaps a load).
//
// Weights alone go through vector memory in the main loop, in a ring of registers:
// loads return in order, so anything younger that is waited for would drain them.
// Activations and scales come from LDS, of all of K or of one range of columns
// while the next one is loaded into registers. Waves of a workgroup split K (few
// weight rows) or share the activations along the rows (many).
//
// Experts: no capacity and no router here, so a workgroup finds its expert's rows
// itself by one ballot over the ids (up to 64 assignments) or reads them from a plan
// (one small launch). A hidden row is kept as two bf16 terms, as the few-token layer
// keeps it: out then carries its own rounding alone.
//
// Measured (calls in turn on inputs past the last-level cache, 256 MB; in brackets on
// three sets, which it keeps where they are small): one row of 7168 by 2048 9.8 us (9.4),
// of which the kernel 7.5; 5 rows of 14336 by 4096 with zero points 19.6 (17.7; 32 MB, 1.7
// TB/s: the activations of all of K are read by each of 256 workgroups); 33 rows of 4096 by
// 14336, groups of 32, 31.2 (29.3; the fp32 scaling of each group of four row tiles, one of
// them nearly empty); one Mixtral-shaped token 35.6 (121 MB, 3.4 TB/s: 15 and 18 for the
// products), 64 of them 231; 61 tokens of 256 experts 705 to 720 (3.3 GB, 4.6 to 4.7 TB/s).
// Conversions: 470 M bf16 weights to 4 bits 332 us (3.6 TB/s), back 233 (5.1).
#include <algorithm>
#include <type_traits>

#include "activation.hpp"
#include "common.hpp"

namespace moe {
namespace {

constexpr int kQ4Load = 128;   // weights of a row per wave load
// By tiles of 16 rows of activations: loads of a wave's step (two take the halves of
// the weight rows' 128-byte lines one after the other) and steps in flight.
constexpr int q4_loads(int tiles) { return tiles == 1 ? 2 : 1; }
constexpr int q4_depth(int tiles) { return tiles <= 4 ? 2 : 1; }
constexpr int q4_step(int tiles) { return kQ4Load * q4_loads(tiles); }
constexpr int kMaxAssign = kFewMaxTokens * kMaxTopK;

// 8 packed weights as 128 + q in bf16, in the order 0 4 1 5 2 6 3 7. (The masks
// come in registers, one scalar and one vector: an instruction takes no two
// literals, and as literals each would cost a second instruction.)
struct Q4Masks {
    unsigned low, one;
    __device__ __forceinline__ Q4Masks() {
        asm("s_mov_b32 %0, 0x000f000f" : "=s"(low));
        asm("v_mov_b32 %0, 0x43004300" : "=v"(one));
    }
    __device__ __forceinline__ bf16x8 weights(unsigned d) const {
        return __builtin_bit_cast(bf16x8,
                                  u32x4{(d & low) | one, ((d >> 4) & low) | one,
                                        ((d >> 8) & low) | one, ((d >> 12) & low) | one});
    }
};

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

// How a workgroup covers its product: wm x wk waves, each RT tiles of 16 weight
// rows, the waves of one row block taking every wk-th step of columns.
struct Q4Waves {
    int wm, wk, lds;   // lds: bytes for the activations and the scales
};
// The activations in LDS, rows of 2^sh chunks of 8 columns: all of K where R rows
// of it fit, else kc columns at a time in two buffers, as many times wk D steps as
// fit (the host sees to it that one does).
struct Q4Tiling {
    int wm, wk, kc, sh;
};
constexpr int kQ4Chunks = 4;   // 16-byte chunks a thread loads at once
__device__ __host__ __forceinline__ int log2_up(int v) {
    int s = 0;
    while ((1 << s) < v)
        ++s;
    return s;
}
// Scales of a row are 2 bytes a group, rows a multiple of 16 bytes (and not of the
// banks) apart.
__device__ __host__ __forceinline__ int q4_scale_stride(int groups) {
    return (groups + 7) / 8 * 8 + 8;
}
// Bytes of kc columns (a multiple of a step): R rows of activations, the scales and
// zero points of WR weight rows.
__device__ __host__ __forceinline__ int64_t q4_bytes(int R, int WR, int64_t kc, int GS, bool zero) {
    return R * (2 * kc + 16) + (int64_t)WR * q4_scale_stride((int)(kc / kQ4Load * GS)) * (zero ? 4 : 2);
}
__device__ __host__ __forceinline__ Q4Tiling q4_tiling(const Q4Waves &w, int R, int WR, int K,
                                                       int tiles, int GS, bool zero) {
    const int step = q4_step(tiles);
    Q4Tiling t;
    t.wm = w.wm;
    t.wk = w.wk;
    t.kc = (K + step - 1) / step * step;
    if (q4_bytes(R, WR, t.kc, GS, zero) > w.lds) {
        // (bytes a column, times 64, and those of no column)
        const int per = 128 * R + WR * GS * (zero ? 2 : 1), none = 16 * R + WR * 32 * (zero ? 2 : 1);
        const int unit = step * w.wk * q4_depth(tiles);
        // no more than the threads load in one go, where that is a unit
        const int most = max(kQ4Chunks * 64 * w.wm * w.wk * 8 / R / unit, 1);
        t.kc = min((int)((int64_t)(w.lds / 2 - none) * 64 / per) / unit, most) * unit;
    }
    t.sh = log2_up(t.kc / 8);
    return t;
}

// Rows of activations in LDS, 8 numbers a chunk in the order of Q4Masks; rows
// are 16 bytes apart modulo the banks.
__device__ __forceinline__ u32x4 q4_order(const u32x4 &v) {
    return u32x4{__builtin_amdgcn_perm(v[2], v[0], 0x05040100u),
                 __builtin_amdgcn_perm(v[2], v[0], 0x07060302u),
                 __builtin_amdgcn_perm(v[3], v[1], 0x05040100u),
                 __builtin_amdgcn_perm(v[3], v[1], 0x07060302u)};
}

// The product of the workgroup's 16 RT WM weight rows from m0 on (rows past
// mlast repeat it) with its token rows: f(token row of the 16 TT, weight row of
// the workgroup, value) for each result. src(r): row r < R of activations;
// at(i, n): the row that this lane takes for tile i and term n of NB (whose
// products are added). TWO: K may take more than one buffer.
template <int GS, bool ZERO, int RT, int TT, int NB, bool TWO, typename SRC, typename AT,
          typename F>
__device__ __forceinline__ void q4_block(char *smem, const Q4Matrix &W, int64_t m0, int64_t mlast,
                                         int K, const Q4Tiling &T, int R, SRC src, AT at, F f) {
    const int lane = threadIdx.x & 63, g = lane >> 4;
    const int wv = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int wm = wv / T.wk, wk = wv % T.wk, threads = blockDim.x;
    constexpr int NL = q4_loads(TT * NB), D = q4_depth(TT * NB), STEP = q4_step(TT * NB);
    const int KG = K / (kQ4Load / GS);   // groups of a row
    const int steps = (K + STEP - 1) / STEP;
    const int mine = (steps - wk + T.wk - 1) / T.wk;   // steps of this wave

    const unsigned char *w[RT];
#pragma unroll
    for (int r = 0; r < RT; ++r)
        w[r] = W.data + min(m0 + (wm * RT + r) * 16 + (lane & 15), mlast) * (K / 2) + 16 * g;
    struct Step {
        u32x4 w[NL][RT];
    };
    // Loads have no branches around them (past the end they repeat the last place,
    // and what they bring is not used), so that a wait can count them.
    auto load = [&](int n, Step &s) {
        const int k = (wk + n * T.wk) * STEP;
#pragma unroll
        for (int r = 0; r < RT; ++r)
#pragma unroll
            for (int h = 0; h < NL; ++h)
                s.w[h][r] = *reinterpret_cast<const u32x4 *>(
                    w[r] + min((k + h * kQ4Load) / 2, K / 2 - 16 - 16 * g));
    };

    // activations: chunk o of the buffer is chunk o % 2^sh of row o / 2^sh; columns
    // past K are zeros (the weights there are not)
    const int rowb = T.kc * 2 + 16;
    const int chunks = R << T.sh, cmask = (1 << T.sh) - 1;
    auto fetch = [&](int o, int k0) {
        return *reinterpret_cast<const u32x4 *>(src(min(o >> T.sh, R - 1)) +
                                                min(k0 + 8 * (o & cmask), K - 8));
    };
    auto put = [&](char *buf, int o, int k0, const u32x4 &v) {
        const int c = o & cmask;
        if (o < chunks && 8 * c < T.kc)
            *reinterpret_cast<u32x4 *>(buf + (o >> T.sh) * rowb + 16 * c) =
                k0 + 8 * c < K ? q4_order(v) : u32x4{0u, 0u, 0u, 0u};
    };
    // scales (and zero points) of the buffer's groups, row by row, 8 at a time where
    // every row's start and length allow: read by the lanes themselves, they took as
    // many requests as the weights (fine-grained batch of 61 tokens: 1030 us, 760
    // without any)
    const int WR = 16 * RT * T.wm, kcg = T.kc / (kQ4Load / GS), ss = q4_scale_stride(kcg);
    const int s_at = R * rowb, z_at = s_at + 2 * WR * ss;
    const bool vec = KG % 8 == 0 && kcg % 8 == 0;
    const unsigned per_row = (unsigned)(vec ? kcg / 8 : kcg), items = WR * per_row;
    struct Item {
        u32x4 s, z;
    };
    auto fetch_scales = [&](unsigned o, int k0) {
        o = min(o, items - 1);
        const int r = (int)(o / per_row), c = (int)(o - r * per_row), g0 = k0 / (kQ4Load / GS);
        const int64_t from = min(m0 + r, mlast) * KG;
        Item v = {};
        if (vec) {
            const int64_t at = from + min(g0 + 8 * c, KG - 8);
            v.s = *reinterpret_cast<const u32x4 *>(W.scale + at);
            if (ZERO)
                v.z = *reinterpret_cast<const u32x4 *>(W.zero + at);
        } else {
            const int64_t at = from + min(g0 + c, KG - 1);
            v.s[0] = W.scale[at];
            if (ZERO)
                v.z[0] = W.zero[at];
        }
        return v;
    };
    auto put_scales = [&](char *buf, unsigned o, int k0, const Item &v) {
        if (o >= items)
            return;
        const int r = (int)(o / per_row), c = (int)(o - r * per_row);
        if (vec) {
            *reinterpret_cast<u32x4 *>(buf + s_at + 2 * (r * ss + 8 * c)) = v.s;
            if (ZERO)
                *reinterpret_cast<u32x4 *>(buf + z_at + 2 * (r * ss + 8 * c)) = v.z;
        } else {
            // (of a step that ends past K, groups past the last one are zeros; whole
            // vectors have none)
            const bool in = k0 / (kQ4Load / GS) + c < KG;
            *reinterpret_cast<unsigned short *>(buf + s_at + 2 * (r * ss + c)) =
                in ? (unsigned short)v.s[0] : 0;
            if (ZERO)
                *reinterpret_cast<unsigned short *>(buf + z_at + 2 * (r * ss + c)) =
                    in ? (unsigned short)v.z[0] : 0;
        }
    };
    // What a thread loads of a buffer at once; the rest, if any, follows in put_all.
    constexpr int XR = kQ4Chunks, SR = 1;
    struct Ahead {
        u32x4 x[XR];
        Item s[SR];
    };
    auto fetch_all = [&](Ahead &v, int k0) {
#pragma unroll
        for (int i = 0; i < SR; ++i)
            v.s[i] = fetch_scales(threadIdx.x + i * threads, k0);
#pragma unroll
        for (int i = 0; i < XR; ++i)
            v.x[i] = fetch(threadIdx.x + i * threads, k0);
    };
    auto put_all = [&](const Ahead &v, char *buf, int k0) {
#pragma unroll
        for (int i = 0; i < SR; ++i)
            put_scales(buf, threadIdx.x + i * threads, k0, v.s[i]);
#pragma unroll
        for (int i = 0; i < XR; ++i)
            put(buf, threadIdx.x + i * threads, k0, v.x[i]);
        for (int o = threadIdx.x + XR * threads; o < chunks; o += 4 * threads) {
            u32x4 t[4];
#pragma unroll
            for (int i = 0; i < 4; ++i)
                t[i] = fetch(o + i * threads, k0);
#pragma unroll
            for (int i = 0; i < 4; ++i)
                put(buf, o + i * threads, k0, t[i]);
        }
        for (unsigned o = threadIdx.x + SR * threads; o < items; o += threads)
            put_scales(buf, o, k0, fetch_scales(o, k0));
    };
    Step ring[D];
    const int end = mine - 1;   // (every wave has a step)
    {
        Ahead v;
        fetch_all(v, 0);
#pragma unroll
        for (int u = 0; u < D; ++u)
            load(min(u, end), ring[u]);
        put_all(v, smem, 0);
    }
    barrier_lds();

    f32x4 tot[RT][TT];
#pragma unroll
    for (int r = 0; r < RT; ++r)
#pragma unroll
        for (int i = 0; i < TT; ++i)
            tot[r][i] = f32x4{0.f, 0.f, 0.f, 0.f};
    int xo[TT][NB];   // this lane's rows in a buffer
#pragma unroll
    for (int i = 0; i < TT; ++i)
#pragma unroll
        for (int n = 0; n < NB; ++n)
            xo[i][n] = at(i, n) * rowb;
    // the factor of the sum of x: 1, or without zero points -(128 + 8) at once
    constexpr unsigned one = ZERO ? 0x3f803f80u : 0xc308c308u;
    const bf16x8 factor = __builtin_bit_cast(bf16x8, u32x4{one, one, one, one});
    const Q4Masks masks;
    auto part_of = [&](const char *buf, int k, u32x4 (&w)[RT]) {   // k: column in the buffer
        const f32x4 nil = {0.f, 0.f, 0.f, 0.f};
        f32x4 acc[RT][TT], sx[TT];
        unsigned short sv[RT][GS], zv[RT][GS];
#pragma unroll
        for (int r = 0; r < RT; ++r) {
            const int at = ((wm * RT + r) * 16 + (lane & 15)) * ss + k / (kQ4Load / GS);
            __builtin_memcpy(sv[r], __builtin_assume_aligned(buf + s_at + 2 * at, 2 * GS), 2 * GS);
            if (ZERO)
                __builtin_memcpy(zv[r], __builtin_assume_aligned(buf + z_at + 2 * at, 2 * GS),
                                 2 * GS);
            q4_arrange<GS>(w[r]);
        }
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
                q[r] = masks.weights(w[r][j]);
            const char *xb = buf + 2 * (k + q4_position<GS>(g, j));
#pragma unroll
            for (int i = 0; i < TT; ++i)
#pragma unroll
                for (int n = 0; n < NB; ++n) {
                    const bf16x8 a = *reinterpret_cast<const bf16x8 *>(xb + xo[i][n]);
                    if (ZERO || RT > 1)
                        sx[i] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, factor, sx[i], 0, 0, 0);
#pragma unroll
                    for (int r = 0; r < RT; ++r) {
                        if (!ZERO && RT == 1)
                            acc[r][i] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(
                                a, factor, acc[r][i], 0, 0, 0);
                        acc[r][i] =
                            __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, q[r], acc[r][i], 0, 0, 0);
                    }
                }
            if (j % P == P - 1) {
#pragma unroll
                for (int r = 0; r < RT; ++r) {
                    const float sr = bf16_bits_to_f32(sv[r][j / P]);
                    const float c = ZERO ? -128.f - bf16_bits_to_f32(zv[r][j / P]) : 1.f;
#pragma unroll
                    for (int i = 0; i < TT; ++i)
#pragma unroll
                        for (int e = 0; e < 4; ++e)
                            tot[r][i][e] = fmaf(sr,
                                                ZERO || RT > 1 ? fmaf(c, sx[i][e], acc[r][i][e])
                                                               : acc[r][i][e],
                                                tot[r][i][e]);
                }
            }
        }
    };
    auto multiply = [&](const char *buf, int k, Step &s) {
#pragma unroll
        for (int h = 0; h < NL; ++h)
            part_of(buf, k + h * kQ4Load, s.w[h]);
    };
    // steps of a wave in a buffer (a multiple of D, or all of them)
    const int per = T.kc / (STEP * T.wk) + (T.kc >= K);
    const int bytes = TWO ? (z_at + (ZERO ? 2 * WR * ss : 0) + 15) / 16 * 16 : 0;
    char *buf = smem;
    for (int n = 0, k0 = 0;; k0 += T.kc) {
        const bool more = TWO && k0 + T.kc < K;
        Ahead v;
        if (more)
            fetch_all(v, k0 + T.kc);
        const int n1 = min(mine, n + per);
        for (; n + D <= n1; n += D) {
#pragma unroll
            for (int u = 0; u < D; ++u) {
                // (in this order: gathered at the loop's end, the loads would all be
                // waited for at its start)
                multiply(buf, (wk + (n + u) * T.wk) * STEP - k0, ring[u]);
                __builtin_amdgcn_sched_barrier(0);
                load(min(n + u + D, end), ring[u]);
                __builtin_amdgcn_sched_barrier(0);
            }
        }
        if (!more) {
#pragma unroll
            for (int u = 0; u < D; ++u)
                if (n + u < n1)
                    multiply(buf, (wk + (n + u) * T.wk) * STEP - k0, ring[u]);
            break;
        }
        buf = smem + (buf == smem ? bytes : 0);
        put_all(v, buf, k0 + T.kc);
        barrier_lds();
    }
    if (T.wk == 1) {
#pragma unroll
        for (int r = 0; r < RT; ++r)
#pragma unroll
            for (int i = 0; i < TT; ++i)
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    f(16 * i + 4 * g + e, (wm * RT + r) * 16 + (lane & 15), tot[r][i][e]);
        return;
    }
    // the waves of a row block add through LDS, in wave order
    barrier_lds();
    f32x4 *part = reinterpret_cast<f32x4 *>(smem);
#pragma unroll
    for (int r = 0; r < RT; ++r)
#pragma unroll
        for (int i = 0; i < TT; ++i)
            part[((wv * RT + r) * TT + i) * 64 + lane] = tot[r][i];
    barrier_lds();
    constexpr int PER = RT * TT * 64;
    for (int o = threadIdx.x; o < T.wm * PER; o += threads) {
        const int in = o % PER, b = o / PER;
        const f32x4 *p = part + (int64_t)b * T.wk * PER + in;
        f32x4 v = p[0];
        for (int q = 1; q < T.wk; ++q)
            v += p[q * PER];
        const int l = in & 63, i = (in >> 6) % TT, r = (in >> 6) / TT;
#pragma unroll
        for (int e = 0; e < 4; ++e)
            f(16 * i + 4 * (l >> 4) + e, (b * RT + r) * 16 + (l & 15), v[e]);
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

// Waves of a SIMD that a form's registers leave room for.
constexpr int q4_waves(int tt, bool two) { return tt == 1 && !two ? 4 : tt < 4 ? 3 : 2; }

// grid: blocks of 16 RT wm weight rows.
template <int GS, bool ZERO, int RT, int TT, bool TWO>
__global__ __launch_bounds__(512, q4_waves(TT, TWO)) void q4_linear_kernel(Q4Linear p,
                                                                           Q4Waves w) {
    extern __shared__ __attribute__((aligned(16))) char smem[];
    const int lane = threadIdx.x & 63;
    const Q4Tiling T = q4_tiling(w, p.N, 16 * RT * w.wm, p.K, TT, GS, ZERO);
    const int64_t m0 = (int64_t)blockIdx.x * (16 * RT * T.wm);
    q4_block<GS, ZERO, RT, TT, 1, TWO>(
        smem, p.W, m0, p.M - 1, p.K, T, p.N, [&](int r) { return p.x + (int64_t)r * p.K; },
        [&](int i, int) { return min(16 * i + (lane & 15), p.N - 1); },
        [&](int t, int r, float v) {
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

struct Q4Plan;
struct Q4Experts {
    const unsigned short *x;      // [N, d]
    const int32_t *idx;           // [N, k]
    const float *gate;            // [N, k]
    Q4Matrix up, down;
    const float *b_up, *b_down;   // [E, d_ff], [E, d] or NULL
    unsigned short *H;            // [2][N k][d_ff]: two bf16 terms
    float *Y;                     // [N k][d]
    int *done;                    // finished workgroups per column block, or NULL: the
                                  // choices are added by a launch of their own
    const Q4Plan *plan;           // NULL with at most 64 assignments
    unsigned short *out;          // [N, d]
    int N, d, E, d_ff, k, act;
    int block;                    // rows of an expert at a time, at most 16 TT
};

// Rows of a call's hit experts, written by q4_plan_kernel where a call has more
// than 64 assignments.
struct Q4Plan {
    struct {
        int expert, rows, first, pad;                  // first: into row[]
    } hit[kMaxExperts];                                // (rows 0 past the last one)
    unsigned short row[kMaxAssign];                    // assignments t k + j
};

// One workgroup, a thread per assignment: hit experts in ascending order, the
// assignments of each in ascending order. Ids outside [0, E) are left out.
__global__ __launch_bounds__(kMaxAssign) void q4_plan_kernel(const int32_t *__restrict__ idx,
                                                             int A, int E, Q4Plan *plan) {
    constexpr int NW = kMaxAssign / 64;
    __shared__ int count[NW][kMaxExperts];   // of a wave; then those of the waves before
    __shared__ int before[kMaxExperts], nhit[kMaxExperts / 64], nrow[kMaxExperts / 64];
    const int tid = threadIdx.x, lane = tid & 63, wv = tid >> 6;
    for (int i = tid; i < NW * kMaxExperts; i += kMaxAssign)
        (&count[0][0])[i] = 0;
    const int e = tid < A ? idx[tid] : -1;
    const bool ok = e >= 0 && e < E;
    uint64_t same = __ballot(ok);   // lanes of the wave with the same expert
#pragma unroll
    for (int b = 0; b < 8; ++b) {
        const uint64_t ones = __ballot((e >> b) & 1);
        same &= (e >> b) & 1 ? ones : ~ones;
    }
    __syncthreads();
    const int rank = __popcll(same & lanemask_lt());
    if (ok && rank == 0)
        count[wv][e] = __popcll(same);
    __syncthreads();
    int n = 0, upto = 0;
    uint64_t hits = 0;
    if (tid < kMaxExperts) {
        for (int w = 0; w < NW; ++w) {
            const int c = count[w][tid];
            count[w][tid] = n;
            n += c;
        }
        hits = __ballot(n > 0);
        upto = n;
#pragma unroll
        for (int s = 1; s < 64; s <<= 1) {
            const int u = __shfl_up(upto, s);
            if (lane >= s)
                upto += u;
        }
        if (lane == 63) {
            nhit[wv] = __popcll(hits);
            nrow[wv] = upto;
        }
    }
    __syncthreads();
    if (tid < kMaxExperts) {
        int a = __popcll(hits & lanemask_lt()), b = upto - n;
        for (int w = 0; w < wv; ++w) {
            a += nhit[w];
            b += nrow[w];
        }
        before[tid] = b;
        if (n > 0) {
            plan->hit[a].expert = tid;
            plan->hit[a].rows = n;
            plan->hit[a].first = b;
        }
        int all = 0;
        for (int w = 0; w < kMaxExperts / 64; ++w)
            all += nhit[w];
        if (tid >= all)
            plan->hit[tid].rows = 0;
    }
    __syncthreads();
    if (ok)
        plan->row[before[e] + count[wv][e] + rank] = (unsigned short)tid;
}

// The rows of this workgroup's expert (blockIdx.y): by the plan, the expert of
// that number; without one (at most 64 assignments) the expert of that
// assignment, unless an earlier one has it too. row: their assignments in
// ascending order (in LDS); returns their number, 0 where there is no work.
__device__ __forceinline__ int q4_rows(const Q4Experts &p, int &e, unsigned short *row) {
    const int lane = threadIdx.x & 63, A = p.N * p.k, a = blockIdx.y;
    int n;
    if (p.plan) {
        const int f = p.plan->hit[a].first;
        n = p.plan->hit[a].rows;
        e = p.plan->hit[a].expert;
        if (n == 0)
            return 0;
        for (int i = threadIdx.x; i < n; i += blockDim.x)
            row[i] = p.plan->row[f + i];
    } else {
        const int mine = lane < A ? p.idx[lane] : -1;
        e = __builtin_amdgcn_readlane(mine, a);
        const uint64_t same = __ballot(mine == e);
        if (e < 0 || e >= p.E || (same & ((1ull << a) - 1ull)) != 0)
            return 0;
        n = __popcll(same);
        if (threadIdx.x < 64 && (same >> lane & 1ull))
            row[__popcll(same & lanemask_lt())] = (unsigned short)lane;
    }
    __syncthreads();
    return n;
}

// H = act(W_up[e] x + b_up[e]) of the rows of assignment blockIdx.y's expert.
// grid: (blocks of 16 RT wm neurons, N k). blocks: those of the down product.
template <int GS, bool ZERO, int RT, int TT, bool TWO>
__global__ __launch_bounds__(512, q4_waves(TT, TWO)) void q4_up_kernel(Q4Experts p, Q4Waves w,
                                                                       int blocks) {
    extern __shared__ __attribute__((aligned(16))) char smem[];
    __shared__ unsigned short row[kMaxAssign];
    const int lane = threadIdx.x & 63, A = p.N * p.k;
    if (p.done && blockIdx.y == 0)
        for (int i = blockIdx.x * blockDim.x + threadIdx.x; i < blocks; i += gridDim.x * blockDim.x)
            p.done[i] = 0;
    int e;
    const int rows = q4_rows(p, e, row);
    if (rows == 0)
        return;
    const int f0 = blockIdx.x * (16 * RT * w.wm);
    const int64_t m0 = (int64_t)e * p.d_ff;
    for (int t0 = 0; t0 < rows; t0 += p.block) {
        const int here = min(rows - t0, p.block);
        auto run = [&](auto tiles) {
            constexpr int T = decltype(tiles)::value;
            q4_block<GS, ZERO, RT, T, 1, TWO>(
                smem, p.up, m0 + f0, m0 + p.d_ff - 1, p.d, q4_tiling(w, here, 16 * RT * w.wm, p.d, T, GS, ZERO), here,
                [&](int r) { return p.x + (int64_t)(row[t0 + r] / p.k) * p.d; },
                [&](int i, int) { return min(16 * i + (lane & 15), here - 1); },
                [&](int t, int r, float v) {
                    const int f = f0 + r;
                    if (t >= here || f >= p.d_ff)
                        return;
                    if (p.b_up)
                        v += p.b_up[m0 + f];
                    v = activate(v, p.act);
                    // the second term: what rounding to bf16 leaves (nothing of
                    // an infinity or a NaN)
                    const unsigned short hi = f32_to_bf16_bits(v);
                    const float rest = v - bf16_bits_to_f32(hi);
                    unsigned short *h = p.H + (int64_t)row[t0 + t] * p.d_ff + f;
                    h[0] = hi;
                    h[(int64_t)A * p.d_ff] =
                        f32_to_bf16_bits(fabsf(rest) < __builtin_inff() ? rest : 0.f);
                });
        };
        if (TT == 1 || here <= 16)
            run(std::integral_constant<int, 1>{});
        else if (TT == 2 || here <= 32)
            run(std::integral_constant<int, TT < 2 ? TT : 2>{});
        else
            run(std::integral_constant<int, TT>{});
        __syncthreads();
    }
}

// Y = W_down[e] h + b_down[e] of the same rows; the workgroup of a column block
// that finishes last adds each token's choices in order. Y and the counter are
// written and read past the XCD's own L2 (agent scope). grid: (blocks of 16 RT
// wm columns, N k).
template <int GS, bool ZERO, int RT, int TT, bool TWO>
__global__ __launch_bounds__(512, q4_waves(TT, TWO)) void q4_down_kernel(Q4Experts p,
                                                                         Q4Waves w) {
    extern __shared__ __attribute__((aligned(16))) char smem[];
    __shared__ unsigned short row[kMaxAssign];
    __shared__ int last;
    const int lane = threadIdx.x & 63, A = p.N * p.k;
    int e;
    const int rows = q4_rows(p, e, row);
    const int cols = 16 * RT * w.wm, c0 = blockIdx.x * cols;
    if (rows > 0) {
        const int64_t m0 = (int64_t)e * p.d, lo = (int64_t)A * p.d_ff;
        for (int t0 = 0; t0 < rows; t0 += p.block) {
            const int here = min(rows - t0, p.block);
            auto store = [&](int t, int r, float v) {
                if (t >= here || c0 + r >= p.d)
                    return;
                if (p.b_down)
                    v += p.b_down[m0 + c0 + r];
                float *y = p.Y + (int64_t)row[t0 + t] * p.d + c0 + r;
                if (p.done)
                    __hip_atomic_store(y, v, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
                else
                    *y = v;
            };
            // rows [0, here) hold the first terms, [here, 2 here) the second ones
            auto src = [&](int r) {
                const bool second = r >= here;
                return p.H + (int64_t)row[t0 + (second ? r - here : r)] * p.d_ff +
                       (second ? lo : 0);
            };
            auto run = [&](auto tiles) {
                constexpr int T = decltype(tiles)::value;
                q4_block<GS, ZERO, RT, T, 2, TWO>(
                    smem, p.down, m0 + c0, m0 + p.d - 1, p.d_ff,
                    q4_tiling(w, 2 * here, cols, p.d_ff, 2 * T, GS, ZERO), 2 * here, src,
                    [&](int i, int n) { return min(16 * i + (lane & 15), here - 1) + n * here; },
                    store);
            };
            if (here <= 8) {
                // both terms fill one tile: its rows 0-7 the first ones, 8-15 the
                // second ones, added at the end
                q4_block<GS, ZERO, RT, 1, 1, TWO>(
                    smem, p.down, m0 + c0, m0 + p.d - 1, p.d_ff,
                    q4_tiling(w, 2 * here, cols, p.d_ff, 1, GS, ZERO), 2 * here, src,
                    [&](int, int) { return min(lane & 7, here - 1) + (lane & 8 ? here : 0); },
                    [&](int t, int r, float v) {
                        v += __shfl_xor(v, 32);
                        if (t < 8)
                            store(t, r, v);
                    });
            } else if (TT == 1 || here <= 16) {
                run(std::integral_constant<int, 1>{});
            } else if (TT == 2 || here <= 32) {
                run(std::integral_constant<int, TT < 2 ? TT : 2>{});
            } else {
                run(std::integral_constant<int, TT>{});
            }
            __syncthreads();
        }
    }
    if (!p.done)
        return;
    // Y has reached memory before the workgroup counts (agent-scope stores write
    // through; the wait is for their completion)
    asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
    __syncthreads();
    if (threadIdx.x == 0)
        last = __hip_atomic_fetch_add(p.done + blockIdx.x, 1, __ATOMIC_RELAXED,
                                      __HIP_MEMORY_SCOPE_AGENT) == (int)gridDim.y - 1;
    __syncthreads();
    if (!last)
        return;
    // (agent-scope loads, as the stores)
    for (int i = threadIdx.x; i < p.N * cols; i += blockDim.x) {
        const int t = i / cols, c = c0 + i % cols;
        if (c >= p.d)
            continue;
        float s = 0.f;
        for (int j = 0; j < p.k; ++j) {
            const int a = t * p.k + j, id = p.idx[a];
            if (id >= 0 && id < p.E)
                s = fmaf(p.gate[a],
                         __hip_atomic_load(p.Y + (int64_t)a * p.d + c, __ATOMIC_RELAXED,
                                           __HIP_MEMORY_SCOPE_AGENT),
                         s);
        }
        p.out[(int64_t)t * p.d + c] = f32_to_bf16_bits(s);
    }
}

// out[t] = sum of its choices' rows, in choice order: 4 columns a thread (d % 4 == 0).
__global__ __launch_bounds__(256) void q4_combine_kernel(Q4Experts p) {
    const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
    const int per = p.d / 4;
    if (i >= (int64_t)p.N * per)
        return;
    const int t = (int)(i / per), c = (int)(i - (int64_t)t * per) * 4;
    f32x4 s = {0.f, 0.f, 0.f, 0.f};
    constexpr int B = 8;   // rows in flight
    for (int j0 = 0; j0 < p.k; j0 += B) {
        f32x4 y[B];
        float g[B];
#pragma unroll
        for (int b = 0; b < B; ++b) {
            const int a = t * p.k + min(j0 + b, p.k - 1), id = p.idx[a];
            y[b] = *reinterpret_cast<const f32x4 *>(p.Y + (int64_t)a * p.d + c);
            g[b] = p.gate[a];
            // (a row without an expert was not written)
            if (j0 + b >= p.k || id < 0 || id >= p.E) {
                g[b] = 0.f;
                y[b] = f32x4{0.f, 0.f, 0.f, 0.f};
            }
        }
#pragma unroll
        for (int b = 0; b < B; ++b)
#pragma unroll
            for (int q = 0; q < 4; ++q)
                s[q] = fmaf(g[b], y[b][q], s[q]);
    }
    unsigned short *o = p.out + (int64_t)t * p.d + c;
#pragma unroll
    for (int q = 0; q < 4; ++q)
        o[q] = f32_to_bf16_bits(s[q]);
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
    const float range = hi - lo;   // (of finite weights past 2^127 it may be past fp32)
    const unsigned short sb = f32_to_bf16_bits(
        !zero                       ? fmaxf(hi, -lo) * (1.f / 7.f)
        : range < __builtin_inff() ? range * (1.f / 15.f)
                                   : hi * (1.f / 15.f) - lo * (1.f / 15.f));
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

// Calls f(groups of a 128-weight step, zero points, row tiles, token tiles, more
// than one buffer).
int token_tiles(int64_t n) { return n <= 16 ? 1 : n <= 32 ? 2 : 4; }

template <typename F>
hipError_t with_shape(int group, bool zero, int rt, int tt, bool two, F f) {
    auto tiles = [&](auto gs, auto z, auto r) {
        if constexpr (decltype(r)::value == 1)   // (one token tile: one weight tile)
            if (tt == 1)
                return two ? f(gs, z, r, std::integral_constant<int, 1>{}, std::true_type{})
                           : f(gs, z, r, std::integral_constant<int, 1>{}, std::false_type{});
        if (tt <= 2)
            return f(gs, z, r, std::integral_constant<int, 2>{}, std::true_type{});
        return f(gs, z, r, std::integral_constant<int, 4>{}, std::true_type{});
    };
    auto rows = [&](auto gs, auto z) {
        if constexpr (!decltype(z)::value)   // (one weight tile with zero points)
            if (rt == 2)
                return tiles(gs, z, std::integral_constant<int, 2>{});
        return tiles(gs, z, std::integral_constant<int, 1>{});
    };
    auto zeros = [&](auto gs) {
        return zero ? rows(gs, std::true_type{}) : rows(gs, std::false_type{});
    };
    return group == 128  ? zeros(std::integral_constant<int, 1>{})
           : group == 64 ? zeros(std::integral_constant<int, 2>{})
                         : zeros(std::integral_constant<int, 4>{});
}

constexpr int kQ4MaxWaves = 8;
constexpr int kQ4Lds = 144 * 1024;

// Waves of a product of `blocks` times M rows of K weights, whose workgroups hold
// up to R rows of activations, of nb terms, in tt tiles.
struct Q4Shape {
    int rt;
    Q4Waves w;
    int threads, smem;
    bool two;   // more than one buffer, for some number of rows
};
Q4Shape q4_shape(int64_t M, int64_t blocks, int tt, int nb, int R, bool zero) {
    Q4Shape s;
    const int64_t strips = blocks * ((M + 15) / 16);   // of 16 weight rows
    // About 4096 waves, 16 on a CU, by cutting the reduction (one Mixtral-shaped
    // token: 31 us with 2 and 8 waves along K in the two products, 35 with 4 and 4).
    int wk = 8;
    while (wk > 1 && strips * wk > 4096)
        wk /= 2;
    if (tt == 1) {
        // Waves along the rows share the activations: two where an expert has more
        // than two rows (16 tokens, 8 experts: 23 us, 26 with one), four where the
        // reduction is not cut.
        s.rt = 1;
        s.w.wm = wk == 1 ? 4 : blocks > 1 && R > 2 ? 2 : 1;
        s.w.wk = s.w.wm == 2 ? std::min(wk, 4) : wk;
        // Where K takes two buffers: few steps of all the waves in one cost barriers, many
        // the workgroups beside it on the CU. 32, 48 and 64 KB, us: not cut, 8 rows of 7168
        // by 70000 87, 70, 83, 61 tokens of 256 experts 794, 717, 740; cut in 2 or 4, 6 rows
        // of 14336 by 12288 37, 35, 53, 2, 6 and 16 Mixtral-shaped tokens 69, 60, 53, 111,
        // 103, 109 and 165, 162, 167; cut in 8, one such token, whose K fits 64, 46, 46, 33.
        s.w.lds = (wk == 8 ? 64 : 48) * 1024;
    } else {
        // Two weight tiles a wave, which halve the reads of the activations (of two terms
        // in the down product), where they leave enough waves. One and two, us: rows of
        // 4096 by 14336, 33 30 and 47, by 65536, 64 124 and 120, 20 of 2048 by 131072 86
        // and 75; experts, up and down product apart, 64 Mixtral-shaped tokens 325 to 295
        // and 295 to 228, 64 of 16 of 7168 by 4096, k 4, 320 to 279 and 279 to 230, 64 of
        // 8 of 2048 by 4096 (2048 and 1024 strips) 65 to 60 and 65 to 70; 32 Mixtral-shaped
        // tokens, k 4, 311 to 306 and 306 to 337. With zero points, whose sums of x take
        // registers, one: 64 rows of 4096 by 131072 231 and 449, 64 Mixtral-shaped tokens
        // 308 and 333.
        s.rt = !zero && strips >= (nb == 2 ? 2048 : 4096) ? 2 : 1;
        s.w.wm = 4;
        s.w.wk = s.rt == 2 ? 2 : std::min(wk, 2);
        s.w.lds = 64 * 1024;
    }
    return s;
}
// Rows of an expert that one pass over its weights takes. With few on average, few:
// all of K then fits LDS (61 tokens of the 256-expert layer, 2 rows on average: 762
// us with passes of 4, 805 with 16, the second passes of some experts included).
int q4_row_block(int64_t N, int64_t mean, int tt) {
    const int64_t most = tt == 1 ? std::max<int64_t>(2 * mean, 4) : 64;
    return (int)std::min<int64_t>(std::min<int64_t>(N, most), 16 * tt);
}
Q4Shape q4_sized(int64_t M, int64_t K, int64_t blocks, int tt, int nb, int R, int group,
                 bool zero) {
    Q4Shape s = q4_shape(M, blocks, tt, nb, R, zero);
    // every wave has a step; two buffers of wk D of them for every form that the kernel
    // takes, unless all of K fits
    const int64_t steps = (K + q4_step(1) - 1) / q4_step(1), Kr = steps * q4_step(1);
    while (s.w.wk > 1 && (s.w.wk > steps || s.w.wm * s.w.wk > kQ4MaxWaves))
        s.w.wk /= 2;
    const int GS = kQ4Load / group, one = 64 * 1024;
    // (cut reductions keep all of K in one buffer where that takes no more than 64 KB: 12
    // rows of 2048 by 12288 9.1 us, 16.9 in two of 48 KB; 3 of 7168 by 12000, groups of 32,
    // 16.0 and 18.7; 32 tokens, 32 experts of 1024 by 1536 39.5 and 42.4; 4 rows of 7168 by
    // 14336 21.7 and 25.8)
    const bool fits = tt == 1 && s.w.wk > 1 && q4_bytes(R, 16 * s.w.wm, Kr, GS, zero) <= one;
    const int most = fits ? one : s.w.lds;
    auto least = [&] {
        const int WR = 16 * s.rt * s.w.wm;
        if (q4_bytes(R, WR, Kr, GS, zero) <= most)
            return (int)q4_bytes(R, WR, Kr, GS, zero);
        int n = 0;
        for (int t = 1; t <= tt * nb; t *= 2)
            n = std::max(n, 2 * ((int)q4_bytes(std::min(R, 16 * t), WR,
                                               q4_step(t) * s.w.wk * q4_depth(t), GS, zero) +
                                 16 * WR * (zero ? 2 : 1)));
        return n;
    };
    while (s.w.wk > 1 && least() > kQ4Lds)
        s.w.wk /= 2;
    s.two = q4_bytes(R, 16 * s.rt * s.w.wm, Kr, GS, zero) > most;
    s.w.lds = s.two ? std::max(most, least()) : least();
    s.threads = s.w.wm * s.w.wk * 64;
    s.smem = std::max(s.w.lds, s.w.wk > 1 ? s.w.wm * s.w.wk * s.rt * tt * 1024 : 0);
    return s;
}

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
    const Q4Shape sh = q4_sized(M, K, 1, token_tiles(N), 1, (int)N, group, zero != nullptr);
    return with_shape(group, zero != nullptr, sh.rt, token_tiles(N), sh.two,
                      [&](auto gs, auto z, auto rt, auto tt, auto two) {
        constexpr int GS = decltype(gs)::value, RT = decltype(rt)::value, TT = decltype(tt)::value;
        const int rows = 16 * RT * sh.w.wm;
        moeLaunchKernelGGL((q4_linear_kernel<GS, decltype(z)::value, RT, TT, decltype(two)::value>), dim3((unsigned)((M + rows - 1) / rows)),
                           dim3(sh.threads), sh.smem, s, p, sh.w);
        return hipGetLastError();
    });
}

Q4ExpertsLayout experts_q4_layout(int64_t N, int64_t d, int64_t d_ff, int k) {
    Q4ExpertsLayout L;
    size_t o = 0;
    L.H = o;    o += up256((size_t)(N * k * d_ff) * 4);
    L.Y = o;    o += up256((size_t)(N * k * d) * 4);
    L.done = o; o += up256((size_t)((d + 15) / 16) * 4);
    L.plan = o; o += up256(sizeof(Q4Plan));
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
    const int64_t A = N * k, hits = std::min<int64_t>(E, A);
    unsigned blocks = (unsigned)A;   // of a column: one for each assignment or hit expert
    if (A > 64) {
        Q4Plan *plan = reinterpret_cast<Q4Plan *>(w + L.plan);
        moeLaunchKernelGGL(q4_plan_kernel, dim3(1), dim3(kMaxAssign), 0, s, idx, (int)A, E, plan);
        const hipError_t err = hipGetLastError();
        if (err != hipSuccess)
            return err;
        p.plan = plan;
        blocks = (unsigned)hits;
    }
    // tiles for the rows an expert has on average, with room for more
    const int64_t mean = (A + hits - 1) / hits;
    const int tt = std::min(token_tiles(N), token_tiles(2 * mean + 4));
    // (an expert has more rows than tokens only where a token names it twice)
    const int R = q4_row_block(N, mean, tt);
    p.block = R;
    const Q4Shape us = q4_sized(d_ff, d, hits, tt, 1, R, group, up[2] != nullptr);
    const Q4Shape ds = q4_sized(d, d_ff, hits, tt, 2, 2 * R, group, down[2] != nullptr);
    const int ur = 16 * us.rt * us.w.wm, dr = 16 * ds.rt * ds.w.wm;
    // The last workgroup of a column block adds the choices where no thread of it has more
    // than one to read (past the L2, one after the other); a launch of its own costs less
    // elsewhere. By the last workgroup and apart, us: one token of 8 experts of 768 by 2048
    // 12.4 and 12.9 (as calls 12.0 and 14.2), 4 15.0 and 15.7, 4 Mixtral-shaped 87.7 and
    // 89.2; one of 256 experts, k 8, of 7168 (2 a thread) 36.4 and 36.0, 16 of 8 of 768 by
    // 2048 (2) 24.4 and 22.8, 8 of 32, k 4, of 512 by 512 (4) 16.5 and 14.5, 64 of 4 of 256
    // by 256 35 and 23, 33 of 128, k 4, of 4096 by 512 92 and 61, 64 of 256, k 16, of 1024
    // by 128 171 and 40.
    const bool apart = N * dr * k > ds.threads;
    if (apart)
        p.done = nullptr;
    const hipError_t err = with_shape(group, up[2] != nullptr, us.rt, tt, us.two,
                                      [&](auto gs, auto z, auto rt, auto t, auto two) {
        constexpr int GS = decltype(gs)::value, RT = decltype(rt)::value, TT = decltype(t)::value;
        moeLaunchKernelGGL((q4_up_kernel<GS, decltype(z)::value, RT, TT, decltype(two)::value>), dim3((unsigned)((d_ff + ur - 1) / ur), blocks),
                           dim3(us.threads), us.smem, s, p, us.w, (int)((d + dr - 1) / dr));
        return hipGetLastError();
    });
    if (err != hipSuccess)
        return err;
    const hipError_t rc = with_shape(group, down[2] != nullptr, ds.rt, tt, ds.two,
                      [&](auto gs, auto z, auto rt, auto t, auto two) {
        constexpr int GS = decltype(gs)::value, RT = decltype(rt)::value, TT = decltype(t)::value;
        moeLaunchKernelGGL((q4_down_kernel<GS, decltype(z)::value, RT, TT, decltype(two)::value>), dim3((unsigned)((d + dr - 1) / dr), blocks),
                           dim3(ds.threads), ds.smem, s, p, ds.w);
        return hipGetLastError();
    });
    if (rc != hipSuccess || !apart)
        return rc;
    moeLaunchKernelGGL(q4_combine_kernel, dim3((unsigned)((N * (d / 4) + 255) / 256)), dim3(256), 0,
                       s, p);
    return hipGetLastError();
}

hipError_t launch_quantize_q4(bool bf16, const void *W, int64_t n, int group, void *data,
                              void *scale, void *zero, hipStream_t s) {
    const int64_t n8 = n / 8;
    const dim3 grid((unsigned)((n8 + 255) / 256)), block(256);
    if (bf16)
        moeLaunchKernelGGL(q4_quantize_kernel<true>, grid, block, 0, s, W, n8, group,
                           static_cast<unsigned *>(data), static_cast<unsigned short *>(scale),
                           static_cast<unsigned short *>(zero));
    else
        moeLaunchKernelGGL(q4_quantize_kernel<false>, grid, block, 0, s, W, n8, group,
                           static_cast<unsigned *>(data), static_cast<unsigned short *>(scale),
                           static_cast<unsigned short *>(zero));
    return hipGetLastError();
}

hipError_t launch_dequantize_q4(bool bf16, const void *data, const void *scale, const void *zero,
                                int64_t n, int group, void *W, hipStream_t s) {
    const int64_t n8 = n / 8;
    const dim3 grid((unsigned)((n8 + 255) / 256)), block(256);
    if (bf16)
        moeLaunchKernelGGL(q4_dequantize_kernel<true>, grid, block, 0, s,
                           static_cast<const unsigned *>(data),
                           static_cast<const unsigned short *>(scale),
                           static_cast<const unsigned short *>(zero), n8, group, W);
    else
        moeLaunchKernelGGL(q4_dequantize_kernel<false>, grid, block, 0, s,
                           static_cast<const unsigned *>(data),
                           static_cast<const unsigned short *>(scale),
                           static_cast<const unsigned short *>(zero), n8, group, W);
    return hipGetLastError();
}

}  // namespace moe
