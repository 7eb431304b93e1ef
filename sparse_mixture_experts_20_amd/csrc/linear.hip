// Linear product with bias, activation and residual in its epilogue, and its
// backward: the dense feed-forward layer or shared expert that stands beside
// the routed experts (nanoMoE slide 32's expert without the routing).
//
//   z = x W^T + b,  out = act(z) + r                     x [N, K], W [M, K]
//   backward: dz = dout act'(z),  dx = dz W,  dW = dz^T x,  db = sum of dz rows
//
// bf16 operands, fp32 accumulation. dz is rounded to bf16 once, as the operand
// of the two matrix products (they run on the bf16 matrix cores; a second term
// would double them): dx and dW carry that rounding, whatever type they are stored
// in (4096x4096x14336 with GELU and bf16 gradients: 0.0024 from the float64
// result in the 2-norm, where the storage alone is 0.0017). db sums the
// fp32 values before that rounding. Without an activation dz is dout itself.
//
// Few rows and a small W: bound by latency, run on the skinny core
// (skinny.hpp): one workgroup per 16 (or 8) output columns, its waves splitting
// K.
//
// Otherwise one kernel for the three products, BM x BN output tiles, K-step
// 64 in an LDS ring of S stages filled by direct global-to-LDS loads (16 bytes a
// lane); waves of (FM 16) x 64 on 16x16x32 MFMAs. An operand whose rows run
// along the reduction (x, W of the forward, dz of dx) is staged row by row; one
// stored the other way (W of dx, both of dW) is staged as it lies and turned
// into fragments by the transposing LDS read. The output's columns are the
// MFMA's rows, and the 64 columns of a wave are dealt to its four fragments so
// that a lane ends with 16 adjacent columns of one row: the epilogue stores
// whole 128-byte lines from registers, with no pass through LDS. When the tiles
// leave CUs idle, the reduction is cut into ranges whose fp32 partials go to
// the workspace and a second kernel adds them in order (no atomics). The two
// products of a small backward share one launch (linear_pair_kernel).
//
// Measured, in TFLOP/s of the products: 8192x2048x7168 with residual 990 (242
// us), 4096x4096x14336 forward 1165 (412 us) and GELU backward 1090 to 1155 with
// its dz pass (832 to 880 us), 2047x3072x768 backward 515 (37 us, both products
// in one launch). 4x7168x2048 9.3 us on the GPU (29 MB of weights).
#include <algorithm>
#include <type_traits>

#include "activation.hpp"
#include "common.hpp"
#include "skinny.hpp"
#include "tile.hpp"

namespace moe {
namespace {

constexpr int kXcdCount = 8;

struct Epilogue {
    unsigned short *out16;          // bf16 output, or NULL
    float *out32;                   // fp32 output, or NULL
    const float *bias;              // [columns] or NULL
    const unsigned short *res;      // bf16 like the output, or NULL
    unsigned short *z16;            // bf16 pre-activations, or NULL
    int act;
    float *sums;                    // [rows] sums of A's rows (pair kernel), or NULL
};

// Epilogue of G adjacent columns (a multiple of 8) of one row at element
// offset o; b: their biases (0 without one).
template <int G>
__device__ __forceinline__ void store_columns(const Epilogue &ep, int64_t o, float (&v)[G],
                                              const float (&b)[G], int valid) {
#pragma unroll
    for (int h = 0; h < G / 8; ++h) {
        if (8 * h >= valid)
            continue;
        float *p = &v[8 * h];
#pragma unroll
        for (int i = 0; i < 8; ++i)
            p[i] += b[8 * h + i];
        if (ep.z16)
            *reinterpret_cast<u32x4 *>(ep.z16 + o + 8 * h) =
                u32x4{pack_bf16x2(p[0], p[1]), pack_bf16x2(p[2], p[3]), pack_bf16x2(p[4], p[5]),
                      pack_bf16x2(p[6], p[7])};
        if (ep.act != kActNone)
#pragma unroll
            for (int i = 0; i < 8; ++i)
                p[i] = activate(p[i], ep.act);
        if (ep.res) {
            const u32x4 r = *reinterpret_cast<const u32x4 *>(ep.res + o + 8 * h);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                p[2 * i] += __uint_as_float(r[i] << 16);
                p[2 * i + 1] += __uint_as_float(r[i] & 0xffff0000u);
            }
        }
        if (ep.out16) {
            *reinterpret_cast<u32x4 *>(ep.out16 + o + 8 * h) =
                u32x4{pack_bf16x2(p[0], p[1]), pack_bf16x2(p[2], p[3]), pack_bf16x2(p[4], p[5]),
                      pack_bf16x2(p[6], p[7])};
        } else {
            *reinterpret_cast<f32x4 *>(ep.out32 + o + 8 * h) = f32x4{p[0], p[1], p[2], p[3]};
            *reinterpret_cast<f32x4 *>(ep.out32 + o + 8 * h + 4) = f32x4{p[4], p[5], p[6], p[7]};
        }
    }
}

// out [rows, cols] = A B over K-steps [kb, ke) of the tile at (m0, n0). AT: A is
// [K][rows] (else [rows][K]); BT: B is [K][cols] (else [cols][K]). With part,
// the fp32 partial products go there instead. SUMS: the first column tile also
// writes ep.sums.
template <typename Tile, bool AT, bool BT, bool SUMS = false>
__device__ __forceinline__ void linear_tile(char *smem, const unsigned short *__restrict__ A,
                                            const unsigned short *__restrict__ B, int rows,
                                            int cols, int K, const Epilogue &ep,
                                            float *__restrict__ part, int m0, int n0, int kb,
                                            int ke) {
    constexpr int FM = Tile::FM, FN = Tile::FN;
    const int lane = threadIdx.x & 63;
    const int wv = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int wm = wv / Tile::WAVES_N, wn = wv % Tile::WAVES_N;

    f32x4 acc[FM][FN];
#pragma unroll
    for (int i = 0; i < FM; ++i)
#pragma unroll
        for (int j = 0; j < FN; ++j)
            acc[i][j] = f32x4{0.f, 0.f, 0.f, 0.f};
    const bool on = SUMS && ep.sums && n0 == 0 && wn == 0;
    f32x4 sum[FM];
#pragma unroll
    for (int i = 0; i < FM; ++i)
        sum[i] = f32x4{0.f, 0.f, 0.f, 0.f};
    Tile::template run<SUMS>(
        smem,
        [&](int r) {
            return AT ? A + min(m0 + 8 * r, rows - 8) : A + (int64_t)min(m0 + r, rows - 1) * K;
        },
        rows,
        [&](int r) {
            return BT ? B + min(n0 + 8 * r, cols - 8) : B + (int64_t)min(n0 + r, cols - 1) * K;
        },
        cols, K, kb, ke, acc, on, sum);
    const int l16 = lane & 15, g = lane >> 4;
    if (on && g == 0) {
#pragma unroll
        for (int i = 0; i < FM; ++i) {
            const int m = m0 + wm * FM * 16 + i * 16 + l16;
            if (m < rows)
                ep.sums[m] = sum[i][0];
        }
    }
    if (SUMS && !ep.out16 && !ep.out32)
        return;
    // lane: row l16 of each 16-row strip, 16 adjacent columns
    const int n = n0 + wn * 64 + 16 * g, valid = min(16, cols - n);
    if (valid <= 0)
        return;
    float bias[16];
#pragma unroll
    for (int c = 0; c < 16; ++c)
        bias[c] = 0.f;
    if (ep.bias && !part) {
#pragma unroll
        for (int h = 0; h < 4; ++h)
            if (4 * h < valid) {
                const f32x4 t = *reinterpret_cast<const f32x4 *>(ep.bias + n + 4 * h);
#pragma unroll
                for (int c = 0; c < 4; ++c)
                    bias[4 * h + c] = t[c];
            }
    }
#pragma unroll
    for (int i = 0; i < FM; ++i) {
        const int m = m0 + wm * FM * 16 + i * 16 + l16;
        if (m >= rows)
            continue;
        const int64_t o = (int64_t)m * cols + n;
        if (part) {
#pragma unroll
            for (int j = 0; j < FN; ++j)
                if (4 * j < valid)
                    *reinterpret_cast<f32x4 *>(part + o + 4 * j) = acc[i][j];
            continue;
        }
        float v[16];
#pragma unroll
        for (int j = 0; j < FN; ++j)
#pragma unroll
            for (int q = 0; q < 4; ++q)
                v[4 * j + q] = acc[i][j][q];
        store_columns<16>(ep, o, v, bias, valid);
    }
}

// Where tile t of tm x tn stands: column blocks of 8 row tiles, rows fastest, so
// that the tiles in flight on an XCD share operand panels in its L2.
struct Place {
    int m, n;   // row and column tile
};
__device__ __forceinline__ Place place_of(int t, int tm, int tn) {
    constexpr int GM = 8;
    const int band = t / (GM * tn), bm = min(GM, tm - band * GM), in = t - band * GM * tn;
    return {band * GM + in % bm, in / bm};
}

// The product by BM x BN tiles. Block b runs on XCD b mod 8; each XCD takes one
// contiguous range of the tiles. grid: (8 x the blocks of an XCD, K-ranges);
// with more than one range, range s writes its fp32 partials to part + s rows
// cols and the epilogue is left to the second kernel.
// whole: of an XCD's tiles, the first that are computed whole; the others by two
// workgroups, the halves of their rows.
template <int BM, int BN, int WM, int WN, int S, bool AT, bool BT>
__global__ __launch_bounds__(WM *WN * 64) void linear_kernel(
    const unsigned short *__restrict__ A, const unsigned short *__restrict__ B, int rows,
    int cols, int K, int whole, Epilogue ep, float *__restrict__ part) {
    constexpr bool HALVES = BM == 256;
    typedef TileProduct<BM, BN, WM, WN, S, AT, BT> Tile;
    typedef TileProduct<HALVES ? BM / 2 : BM, BN, WM, WN, HALVES ? S + 1 : S, AT, BT> Half;
    __shared__ __attribute__((aligned(1024))) char smem[Half::LDS > Tile::LDS ? Half::LDS : Tile::LDS];

    const int tm = (rows + BM - 1) / BM, tn = (cols + BN - 1) / BN, T = tm * tn;
    const int T8 = (T + kXcdCount - 1) / kXcdCount;
    int q = (int)(blockIdx.x / kXcdCount), half = 0;
    const bool split = HALVES && q >= whole;
    if (split) {
        half = (q - whole) & 1;
        q = whole + ((q - whole) >> 1);
    }
    const int L = (int)(blockIdx.x % kXcdCount) * T8 + q;
    if (L >= T)
        return;
    const Place p = place_of(L, tm, tn);
    const int m0 = p.m * BM, n0 = p.n * BN;
    const int KT = (K + kStep - 1) / kStep;
    if constexpr (HALVES) {   // (never in ranges)
        if (!split)
            linear_tile<Tile, AT, BT>(smem, A, B, rows, cols, K, ep, nullptr, m0, n0, 0, KT);
        else if (m0 + half * (BM / 2) < rows)
            linear_tile<Half, AT, BT>(smem, A, B, rows, cols, K, ep, nullptr,
                                      m0 + half * (BM / 2), n0, 0, KT);
    } else {
        const int kb = (int)((int64_t)blockIdx.y * KT / gridDim.y);
        const int ke = (int)((int64_t)(blockIdx.y + 1) * KT / gridDim.y);
        linear_tile<Tile, AT, BT>(smem, A, B, rows, cols, K, ep,
                                  part ? part + (int64_t)blockIdx.y * rows * cols : nullptr, m0,
                                  n0, kb, ke);
    }
}

// Both products of a backward in one launch: dx = dz W and dW = dz^T x, the tiles
// of the longer reduction first. They need nothing of each other, and one's tiles
// fill the CUs that the other leaves idle. ep.sums of dW: db, the sums of dz's
// columns, from the tiles that read them. A gradient that is not wanted has no
// tiles (tn = 0), except that db alone takes dW's first column of tiles, which
// then write nothing else. grid: 8 x the blocks of an XCD.
struct Product {
    const unsigned short *A, *B;
    int rows, cols, K, tn;   // tn: column tiles to compute
    Epilogue ep;
};
__device__ __host__ __forceinline__ int pair_tiles(const Product &p) {   // of an XCD
    return ((p.rows + 127) / 128 * p.tn + kXcdCount - 1) / kXcdCount;
}
__global__ __launch_bounds__(512) void linear_pair_kernel(Product dx, Product dw) {
    typedef TileProduct<128, 128, 4, 2, 4, false, true> TileX;
    typedef TileProduct<128, 128, 4, 2, 4, true, true> TileW;
    __shared__ __attribute__((aligned(1024))) char smem[TileX::LDS];
    const int X8 = pair_tiles(dx), W8 = pair_tiles(dw);
    const bool w_first = dw.K >= dx.K;
    const int q = (int)(blockIdx.x / kXcdCount), xcd = (int)(blockIdx.x % kXcdCount);
    if (w_first ? q < W8 : q >= X8) {
        const int t = xcd * W8 + (w_first ? q : q - X8), tm = (dw.rows + 127) / 128;
        if (t >= tm * dw.tn)
            return;
        const Place p = place_of(t, tm, dw.tn);
        linear_tile<TileW, true, true, true>(smem, dw.A, dw.B, dw.rows, dw.cols, dw.K, dw.ep,
                                             nullptr, p.m * 128, p.n * 128, 0,
                                             (dw.K + kStep - 1) / kStep);
    } else {
        const int t = xcd * X8 + (w_first ? q - W8 : q), tm = (dx.rows + 127) / 128;
        if (t >= tm * dx.tn)
            return;
        const Place p = place_of(t, tm, dx.tn);
        linear_tile<TileX, false, true>(smem, dx.A, dx.B, dx.rows, dx.cols, dx.K, dx.ep, nullptr,
                                        p.m * 128, p.n * 128, 0, (dx.K + kStep - 1) / kStep);
    }
}

// The sum of S partials in order, then the epilogue; 8 columns per thread.
__global__ __launch_bounds__(256) void linear_join_kernel(const float *__restrict__ part, int S,
                                                          int64_t rows, int cols, Epilogue ep) {
    const int64_t i = ((int64_t)blockIdx.x * 256 + threadIdx.x) * 8;
    const int64_t n = rows * cols;
    if (i >= n)
        return;
    f32x4 a = {0.f, 0.f, 0.f, 0.f}, c = a;
    constexpr int B = 4;   // ranges in flight
    for (int s = 0; s < S; s += B) {
        f32x4 u[B][2];
#pragma unroll
        for (int q = 0; q < B; ++q) {
            const float *p = part + min(s + q, S - 1) * n + i;
            u[q][0] = *reinterpret_cast<const f32x4 *>(p);
            u[q][1] = *reinterpret_cast<const f32x4 *>(p + 4);
        }
#pragma unroll
        for (int q = 0; q < B; ++q)
            if (s + q < S) {
                a += u[q][0];
                c += u[q][1];
            }
    }
    float v[8], b[8];
#pragma unroll
    for (int q = 0; q < 4; ++q) {
        v[q] = a[q];
        v[4 + q] = c[q];
    }
    const int col = (int)(i % cols);
#pragma unroll
    for (int q = 0; q < 8; ++q)
        b[q] = ep.bias ? ep.bias[col + q] : 0.f;
    store_columns<8>(ep, i, v, b, 8);
}

// Few rows: 16 output columns per workgroup, kFewWaves waves over K. HALF (at
// most 8 rows): 8 columns per workgroup, so that a narrow product still fills
// the CUs; the MFMA's rows 0-7 and columns 0-7 take the first half of K, rows
// and columns 8-15 the second half of the same weight and token rows, and the
// two diagonal blocks of the result are added.
constexpr int kFewWaves = 8;
template <int TT, bool HALF>
__global__ __launch_bounds__(kFewWaves * 64) void linear_few_kernel(
    const unsigned short *__restrict__ x, const unsigned short *__restrict__ W, int N, int M,
    int K, Epilogue ep) {
    static_assert(!HALF || TT == 1, "one tile of tokens");
    __shared__ f32x4 part[kFewWaves][TT][64];
    constexpr int CB = HALF ? 8 : 16;
    const int lane = threadIdx.x & 63, l16 = lane & 15;
    const int wv = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int c0 = blockIdx.x * CB;
    // columns a wave's lanes walk together, and where this lane's start
    const int steps = HALF ? (K + 63) / 64 : (K + 31) / 32;
    const int shift = HALF && l16 >= 8 ? steps * 32 : 0;
    const unsigned short *w = W + (int64_t)min(c0 + l16 % CB, M - 1) * K + shift;
    const unsigned short *xt[TT];
    f32x4 acc[TT];
#pragma unroll
    for (int i = 0; i < TT; ++i) {
        xt[i] = x + (int64_t)min(i * 16 + l16 % CB, N - 1) * K + shift;
        acc[i] = f32x4{0.f, 0.f, 0.f, 0.f};
    }
    const int kb = (int)((int64_t)wv * steps / kFewWaves) * 32;
    const int ke = (int)((int64_t)(wv + 1) * steps / kFewWaves) * 32;
    skinny_mma<SkinnyBf16, TT, 1, TT == 1 ? 4 : TT == 2 ? 3 : 2>(
        w, xt, 0, kb, ke, K - shift, HALF ? K - steps * 32 : K, acc);
#pragma unroll
    for (int i = 0; i < TT; ++i)
        part[wv][i][lane] = acc[i];
    __syncthreads();
    // thread -> (row, 8 columns): lanes l and l + 16 of a tile hold columns
    // 4 (l / 16) + 0..3 and the next four of row l % 16
    for (int q = threadIdx.x; q < TT * 16 * (CB / 8); q += kFewWaves * 64) {
        const int i = q / (2 * CB), l = (q & 15) + 32 * (q / 16 % (CB / 8));
        const int r = i * 16 + (l & 15), c = c0 + 4 * (l >> 4);
        if (r >= N || c >= M)
            continue;
        f32x4 a = {0.f, 0.f, 0.f, 0.f}, b4 = a;
#pragma unroll
        for (int s = 0; s < kFewWaves; ++s) {
            a += part[s][i][l];
            b4 += part[s][i][l + 16];
            if constexpr (HALF) {   // rows and columns 8 further
                a += part[s][i][l + 40];
                b4 += part[s][i][l + 56];
            }
        }
        float v[8], b[8];
#pragma unroll
        for (int s = 0; s < 4; ++s) {
            v[s] = a[s];
            v[4 + s] = b4[s];
        }
#pragma unroll
        for (int s = 0; s < 8; ++s)
            b[s] = ep.bias ? ep.bias[c + s] : 0.f;
        store_columns<8>(ep, (int64_t)r * M + c, v, b, 8);
    }
}

// dz = dout act'(z) in bf16 (not written without an activation) and, with
// part, the fp32 column sums of this workgroup's rows before the rounding
// (part [gridDim.y][M]). 8 columns per thread: 32 threads across 256
// columns, 8 rows at a time.
__global__ __launch_bounds__(256) void linear_dz_kernel(const unsigned short *__restrict__ dout,
                                                        const unsigned short *__restrict__ z,
                                                        int N, int M, int act, int rows_per_wg,
                                                        unsigned short *__restrict__ dz,
                                                        float *__restrict__ part) {
    __shared__ float red[8][256 + 8];
    const int cx = threadIdx.x & 31, ry = threadIdx.x >> 5;
    const int c = blockIdx.x * 256 + cx * 8;
    const int r0 = blockIdx.y * rows_per_wg, r1 = min(N, r0 + rows_per_wg);
    float s[8] = {};
    if (c < M) {
#pragma unroll 2
        for (int r = r0 + ry; r < r1; r += 8) {
            const int64_t o = (int64_t)r * M + c;
            const u32x4 gr = *reinterpret_cast<const u32x4 *>(dout + o);
            float v[8];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                v[2 * i] = __uint_as_float(gr[i] << 16);
                v[2 * i + 1] = __uint_as_float(gr[i] & 0xffff0000u);
            }
            if (act != kActNone) {
                const u32x4 zr = *reinterpret_cast<const u32x4 *>(z + o);
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const float zl = __uint_as_float(zr[i] << 16);
                    const float zh = __uint_as_float(zr[i] & 0xffff0000u);
                    if (act == kActRelu) {
                        // a choice, so that a masked infinity gives 0; a NaN in z,
                        // which the forward keeps, does not mask
                        v[2 * i] = zl <= 0.f ? 0.f : v[2 * i];
                        v[2 * i + 1] = zh <= 0.f ? 0.f : v[2 * i + 1];
                    } else {
                        v[2 * i] *= act_gelu_grad(zl);
                        v[2 * i + 1] *= act_gelu_grad(zh);
                    }
                }
                *reinterpret_cast<u32x4 *>(dz + o) =
                    u32x4{pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]),
                          pack_bf16x2(v[4], v[5]), pack_bf16x2(v[6], v[7])};
            }
#pragma unroll
            for (int i = 0; i < 8; ++i)
                s[i] += v[i];
        }
    }
    if (!part)
        return;
#pragma unroll
    for (int i = 0; i < 8; ++i)
        red[ry][cx * 8 + i] = s[i];
    __syncthreads();
    const int cc = blockIdx.x * 256 + threadIdx.x;
    if (cc < M) {
        float t = 0.f;
#pragma unroll
        for (int i = 0; i < 8; ++i)
            t += red[i][threadIdx.x];
        part[(int64_t)blockIdx.y * M + cc] = t;
    }
}

// Tile and K-ranges of a product of rows x cols over K.
//  - up to 64 rows: 64x128 tiles (8 waves, five stages), the reduction cut for
//    256 workgroups: a stream of W through LDS with 96 KB in flight per CU;
//  - 256x256 tiles, one workgroup of 16 waves of 64x64 per CU (four per SIMD
//    hide more LDS latency than the 8 waves of 128x64 save in LDS reads, 1061
//    against 1018 TFLOP/s at 4096x4096x14336), when they fill the 256 CUs about
//    once;
//  - 128x128 tiles in up to 256 workgroups: one of 8 waves per CU and a ring of
//    four stages. Alone on its CU a workgroup waits for the latency of its loads,
//    and three K-steps in flight instead of one take a K-step from 0.83 to 0.6 us;
//  - 128x128 tiles in more of them: two of 8 waves per CU, two stages
//    (2048x768x3072 with GELU and z: 22 us, against 28 with the form before; 25
//    with 4 waves of 64x64, which are 2% faster only from K = 4096 on, where the
//    epilogue's share is small).
// On 128x128 tiles the reduction is cut where the model below, in us, gains from
// it: a workgroup's start and end 3 to 5, a K-step from 0.5 with half of the CUs
// busy to 0.66 with all and 1.2 with two workgroups on each, the joining launch
// 4.5 and the partials written and read at 4 TB/s (2048x3072x768: 29 us in 2
// ranges, 32 in one; 512x768x3072: 15 us in one, 21 in 2). Ranges that put two
// workgroups on a CU have to gain a quarter, as the model errs most there
// (2048x14336x1152: 100 us in 3 ranges, 129 in one; 4352x7424x512, where it sees
// 15%: 70 in 3, 64 in one). At most 16 ranges: the joining launch walks them in
// order, so a small gradient over many rows gains from more only where they are
// very many (64x64 weight gradient, 16 against up to 64 ranges: over 16384 rows
// 15.9 and 22.1 us, over 65536 38.0 and 37.2, over 262144 124 and 79; 256x128 over
// 16384 22.7 and 38.1).
enum class Tile { k64, k256, k128x2, k128 };
struct Shape {
    Tile tile;
    int splits;
    double us;   // modelled time, 128x128 tiles only
};
Shape shape_of(int64_t rows, int64_t cols, int64_t K) {
    const int64_t KT = (K + kStep - 1) / kStep;
    if (rows <= 64) {
        const int64_t s = std::min<int64_t>(256 / std::max<int64_t>((cols + 127) / 128, 1), KT / 4);
        return {Tile::k64, (int)std::min<int64_t>(std::max<int64_t>(s, 1), 16), 0};
    }
    if (((rows + 255) / 256) * ((cols + 255) / 256) >= 192)
        return {Tile::k256, 1, 0};
    const int64_t tiles = ((rows + 127) / 128) * ((cols + 127) / 128);
    auto round = [](int64_t n, double steps) {   // n <= 512 workgroups
        const double f = (double)n / 256;
        return n == 0 ? 0 : n <= 256 ? 3 + (0.43 + 0.23 * f) * steps : 5 + (0.11 + 0.55 * f) * steps;
    };
    auto cost = [&](int64_t s) {
        const double steps = (double)((KT + s - 1) / s);
        const double join = 4.5 + (double)(s + 1) * (double)(rows * cols) * 4.0 / 4e6;
        const double us = (double)(s * tiles / 512) * round(512, steps) +
                          round(s * tiles % 512, steps) + (s > 1 ? join : 0.0);
        return s > 1 && s * tiles > 256 ? 1.25 * us : us;
    };
    int64_t best = 1;
    for (int64_t s = 2; s <= 16 && 4 * s <= KT; ++s)
        if (cost(s) < cost(best))
            best = s;
    return {best * tiles > 256 ? Tile::k128x2 : Tile::k128, (int)best, cost(best)};
}
// Whether the two products of a backward run as one launch: both on 128x128
// tiles, and faster so by the same model. Without an activation the pair spares
// the pass for db (2047x3072x768: 39 us, against 51 apart; 8192x1024x1024: 87 us
// paired, 68 apart). Which gradients are wanted does not enter, so that each has
// the same bits whatever the others.
bool paired(int64_t N, int64_t K, int64_t M, bool act) {
    const Shape x = shape_of(N, K, M), w = shape_of(M, K, N);
    auto small = [](const Shape &s) { return s.tile == Tile::k128 || s.tile == Tile::k128x2; };
    if (!small(x) || !small(w))
        return false;
    auto time = [](int64_t k) { return 3 + 0.65 * (double)((k + kStep - 1) / kStep); };
    auto tiles = [](int64_t rows, int64_t cols) {
        return (double)(((rows + 127) / 128) * ((cols + 127) / 128));
    };
    const double tx = time(M), tw = time(N);
    const double pair = std::max(std::max(tx, tw), (tiles(N, K) * tx + tiles(M, K) * tw) / 256 +
                                                       std::min(tx, tw) / 2);
    return pair <= x.us + w.us + (act ? 0 : 8);
}
size_t part_bytes(int64_t rows, int64_t cols, int64_t K) {
    const Shape sh = shape_of(rows, cols, K);
    return sh.splits > 1 ? (size_t)(sh.splits * rows * cols) * sizeof(float) : 0;
}

// Of an XCD's 256x256 tiles, one per CU at a time, those computed whole. A last
// round that fills at most half of the 32 CUs is computed as half tiles instead,
// which fill the others (8192x2048x7168, 3.5 rounds: 254 -> 242 us;
// 4608x4096x4096, 1.1 rounds: 198 -> 165 us).
int64_t whole_tiles(int64_t each) {
    const int64_t last = each % 32;
    return last <= 16 ? each - last : each;
}

template <bool AT, bool BT>
hipError_t launch_product(const void *A, const void *B, int64_t rows, int64_t cols, int64_t K,
                          const Epilogue &ep, float *part, hipStream_t s) {
    const Shape sh = shape_of(rows, cols, K);
    const auto *a = static_cast<const unsigned short *>(A);
    const auto *b = static_cast<const unsigned short *>(B);
    auto go = [&](auto kernel, int bm, int bn, int threads) {
        const int64_t T = ((rows + bm - 1) / bm) * ((cols + bn - 1) / bn);
        const int64_t each = (T + kXcdCount - 1) / kXcdCount;   // tiles of an XCD
        const int64_t whole = bm == 256 ? whole_tiles(each) : each;
        moeLaunchKernelGGL(kernel,
                           dim3((unsigned)(kXcdCount * (whole + 2 * (each - whole))),
                                (unsigned)sh.splits),
                           dim3(threads), 0, s, a, b, (int)rows, (int)cols, (int)K, (int)whole, ep,
                           sh.splits > 1 ? part : (float *)nullptr);
    };
    if (sh.tile == Tile::k64)
        go(linear_kernel<64, 128, 4, 2, AT ? 4 : 5, AT, BT>, 64, 128, 512);
    else if (sh.tile == Tile::k256)
        go(linear_kernel<256, 256, 4, 4, 2, AT, BT>, 256, 256, 1024);
    else if (sh.tile == Tile::k128x2)
        go(linear_kernel<128, 128, 4, 2, 2, AT, BT>, 128, 128, 512);
    else
        go(linear_kernel<128, 128, 4, 2, 4, AT, BT>, 128, 128, 512);
    hipError_t err = hipGetLastError();
    if (err != hipSuccess || sh.splits == 1)
        return err;
    moeLaunchKernelGGL(linear_join_kernel, dim3((unsigned)((rows * cols / 8 + 255) / 256)),
                       dim3(256), 0, s, (const float *)part, sh.splits, rows, (int)cols, ep);
    return hipGetLastError();
}

// Rows of a workgroup of the dz pass: whole groups of the 8 that it takes at a
// time, about 2048 workgroups in all.
int64_t dz_rows(int64_t N, int64_t M) {
    const int64_t want = std::max<int64_t>(1, 2048 / ((M + 255) / 256));
    return ((N + want - 1) / want + 7) / 8 * 8;
}
int dz_groups(int64_t N, int64_t M) { return (int)((N + dz_rows(N, M) - 1) / dz_rows(N, M)); }

size_t up256(size_t v) { return (v + 255) / 256 * 256; }

}  // namespace

// Whether a forward product runs on the skinny kernel: up to 16 rows and 32 MB
// of weights, or up to 64 rows and 4 MB. Beyond, the tiled kernel's stream is
// faster (1x4096x14336: 24 against 34 us; 64x7168x2048: 19 against 35 us), below
// its joining launch costs more (16x1024x1024: 5.1 against 9.6 us; 64x1024x1024:
// 7.9 against 11; 16x4096x512: 10.9 against 12.5; 8x8192x512: 11.3 against 13.9;
// 4x7168x2048: 10.7 against 16). The rule sees K M and not K, which the skinny
// kernel never cuts over workgroups: a narrow product with a long reduction is
// slower on it, with 16 rows from about K = 6000 on (16x8192x512: 17.9 against
// 14.1 us; 16x16384x256: 31.6 against 17.3), with 64 from about 2048 on
// (64x2048x1024: 12.8 against 12.7; 64x4096x512: 21.8 against 14.5; 32x8192x256:
// 25.7 against 14.3).
static bool skinny(int64_t N, int64_t K, int64_t M) {
    return N <= kFewMaxTokens && K * M <= ((int64_t)(N <= 16 ? 16 : 2) << 20);
}

size_t linear_bytes(int64_t N, int64_t K, int64_t M) {
    return skinny(N, K, M) ? 0 : part_bytes(N, M, K);
}

hipError_t launch_linear(const void *x, const void *W, const float *bias, int act,
                         const void *residual, int64_t N, int64_t K, int64_t M, void *out, void *z,
                         void *ws, hipStream_t s) {
    const Epilogue ep{static_cast<unsigned short *>(out), nullptr, bias,
                      static_cast<const unsigned short *>(residual),
                      static_cast<unsigned short *>(z), act, nullptr};
    if (skinny(N, K, M)) {
        auto go = [&](auto tiles, auto half) {
            constexpr int TT = decltype(tiles)::value;
            constexpr bool HALF = decltype(half)::value;
            constexpr int CB = HALF ? 8 : 16;
            moeLaunchKernelGGL((linear_few_kernel<TT, HALF>), dim3((unsigned)((M + CB - 1) / CB)),
                               dim3(kFewWaves * 64), 0, s, static_cast<const unsigned short *>(x),
                               static_cast<const unsigned short *>(W), (int)N, (int)M, (int)K, ep);
            return hipGetLastError();
        };
        const std::false_type whole;
        if (N <= 8 && M < 16 * 256)
            return go(std::integral_constant<int, 1>{}, std::true_type{});
        return N <= 16   ? go(std::integral_constant<int, 1>{}, whole)
               : N <= 32 ? go(std::integral_constant<int, 2>{}, whole)
                         : go(std::integral_constant<int, 4>{}, whole);
    }
    return launch_product<false, false>(x, W, N, M, K, ep, static_cast<float *>(ws), s);
}

LinearBackwardLayout linear_backward_layout(int64_t N, int64_t K, int64_t M, bool act) {
    LinearBackwardLayout L;
    size_t o = 0;
    L.dz = o;   o += act ? up256((size_t)(N * M) * 2) : 0;
    L.sums = o; o += up256((size_t)dz_groups(N, M) * M * sizeof(float));
    L.part = o; o += up256(std::max(part_bytes(N, K, M), part_bytes(M, K, N)));
    L.total = o;
    return L;
}

hipError_t launch_linear_backward(const void *x, const void *W, const void *z, int act,
                                  const void *dout, int64_t N, int64_t K, int64_t M, void *dx,
                                  bool dx32, void *dW, bool dW32, float *db, void *ws,
                                  hipStream_t s) {
    const LinearBackwardLayout L = linear_backward_layout(N, K, M, act != kActNone);
    char *w = static_cast<char *>(ws);
    const void *dz = dout;
    const bool pair = paired(N, K, M, act != kActNone);
    const bool db_in_pair = pair && act == kActNone;
    if (act != kActNone || (db && !db_in_pair)) {
        const int P = dz_groups(N, M);
        const int per = (int)dz_rows(N, M);
        float *sums = reinterpret_cast<float *>(w + L.sums);
        moeLaunchKernelGGL(linear_dz_kernel, dim3((unsigned)((M + 255) / 256), (unsigned)P),
                           dim3(256), 0, s, static_cast<const unsigned short *>(dout),
                           static_cast<const unsigned short *>(z), (int)N, (int)M, act, per,
                           reinterpret_cast<unsigned short *>(w + L.dz), db ? sums : nullptr);
        hipError_t err = hipGetLastError();
        if (err == hipSuccess && db)
            err = launch_column_sums(sums, P, M, M, db, nullptr, s);
        if (err != hipSuccess)
            return err;
        if (act != kActNone)
            dz = w + L.dz;
    }
    float *part = reinterpret_cast<float *>(w + L.part);
    auto plain = [](void *o, bool f32) {
        return Epilogue{f32 ? nullptr : static_cast<unsigned short *>(o),
                        f32 ? static_cast<float *>(o) : nullptr, nullptr, nullptr, nullptr,
                        kActNone, nullptr};
    };
    if (pair) {
        const auto *dz16 = static_cast<const unsigned short *>(dz);
        const int tn = (int)((K + 127) / 128);
        Product px{dz16, static_cast<const unsigned short *>(W), (int)N, (int)K, (int)M,
                   dx ? tn : 0, plain(dx, dx32)};
        Product pw{dz16, static_cast<const unsigned short *>(x), (int)M, (int)K, (int)N,
                   dW ? tn : db_in_pair && db ? 1 : 0, plain(dW, dW32)};
        pw.ep.sums = db_in_pair ? static_cast<float *>(db) : nullptr;
        const int blocks = pair_tiles(px) + pair_tiles(pw);
        if (blocks == 0)
            return hipSuccess;
        moeLaunchKernelGGL(linear_pair_kernel, dim3((unsigned)(kXcdCount * blocks)), dim3(512), 0, s,
                           px, pw);
        return hipGetLastError();
    }
    if (dx) {
        hipError_t err = launch_product<false, true>(dz, W, N, K, M, plain(dx, dx32), part, s);
        if (err != hipSuccess)
            return err;
    }
    if (dW)
        return launch_product<true, true>(dz, x, M, K, N, plain(dW, dW32), part, s);
    return hipSuccess;
}

}  // namespace moe
