// Skinny matrix product on the matrix cores (private; not part of the C ABI):
// 16 weight rows times a few token rows, the core of the few-token layer and
// of the linear product for a few rows.
//
// Such a product is bound by the stream of its weights, so the weights go from
// global memory straight into MFMA operand registers (no LDS): lane l of a
// 16x16x32 bf16 MFMA holds 8 consecutive elements of weight row l % 16 at
// K offset 8 (l / 16), i.e. one 16-byte load, and a wave's load covers 64
// contiguous bytes of 16 rows. The token rows are the other operand, TT tiles
// of 16, read the same way from L2. A batch of U K-steps is loaded while the
// previous one is multiplied, which keeps U KB of weights per wave in flight.
// Columns of the product are independent of each other, so a lane whose token
// does not exist may hold any row's values: its column is never read.
#pragma once

#include "common.hpp"

namespace moe {

// Product of K columns [kbeg, kend) (multiples of 32, kend possibly past K)
// of a weight row and TT token rows into acc (row 4 (l / 16) + q of the weight
// rows, column l % 16 of the tokens). w and xt[i] point at this lane's row
// (column 0); NB operand terms per token row, `lo` elements apart, are added
// (2: a row kept as the sum of two bf16 terms). K % 8 == 0: the last step's
// chunks past K are taken as zeros.
template <int TT, int NB, int U>
__device__ __forceinline__ void skinny_mma(const unsigned short *w,
                                           const unsigned short *const (&xt)[TT], int64_t lo,
                                           int kbeg, int kend, int K, f32x4 (&acc)[TT]) {
    const int ko = 8 * (int)(__lane_id() >> 4);
    const unsigned short *wp = w + ko;
    const int full = min(kend, K / 32 * 32);   // steps that need no mask
    u32x4 a[U], b[U][TT][NB];
    auto load = [&](int k) {
#pragma unroll
        for (int u = 0; u < U; ++u) {
            a[u] = *reinterpret_cast<const u32x4 *>(wp + k + 32 * u);
#pragma unroll
            for (int i = 0; i < TT; ++i)
#pragma unroll
                for (int n = 0; n < NB; ++n)
                    b[u][i][n] =
                        *reinterpret_cast<const u32x4 *>(xt[i] + n * lo + ko + k + 32 * u);
        }
    };
    auto mma = [&](const u32x4 &av, const u32x4 (&bv)[TT][NB]) {
#pragma unroll
        for (int i = 0; i < TT; ++i)
#pragma unroll
            for (int n = 0; n < NB; ++n)
                acc[i] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(
                    __builtin_bit_cast(bf16x8, av), __builtin_bit_cast(bf16x8, bv[i][n]), acc[i],
                    0, 0, 0);
    };
    int k = kbeg;
    if (k + 32 * U <= full) {
        load(k);
        for (k += 32 * U; k + 32 * U <= full; k += 32 * U) {
            u32x4 ac[U], bc[U][TT][NB];
#pragma unroll
            for (int u = 0; u < U; ++u) {
                ac[u] = a[u];
#pragma unroll
                for (int i = 0; i < TT; ++i)
#pragma unroll
                    for (int n = 0; n < NB; ++n)
                        bc[u][i][n] = b[u][i][n];
            }
            load(k);
#pragma unroll
            for (int u = 0; u < U; ++u)
                mma(ac[u], bc[u]);
        }
#pragma unroll
        for (int u = 0; u < U; ++u)
            mma(a[u], b[u]);
    }
    for (; k < kend; k += 32) {
        // single steps, masked where they reach past K
        u32x4 av = {0u, 0u, 0u, 0u}, bv[TT][NB];
#pragma unroll
        for (int i = 0; i < TT; ++i)
#pragma unroll
            for (int n = 0; n < NB; ++n)
                bv[i][n] = u32x4{0u, 0u, 0u, 0u};
        if (k + ko < K) {
            av = *reinterpret_cast<const u32x4 *>(wp + k);
#pragma unroll
            for (int i = 0; i < TT; ++i)
#pragma unroll
                for (int n = 0; n < NB; ++n)
                    bv[i][n] = *reinterpret_cast<const u32x4 *>(xt[i] + n * lo + ko + k);
        }
        mma(av, bv);
    }
}

}  // namespace moe
