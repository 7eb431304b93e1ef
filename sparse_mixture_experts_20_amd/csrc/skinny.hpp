// Skinny matrix product on the matrix cores (private; not part of the C ABI):
// 16 weight rows times a few token rows, the core of the few-token layer and
// of the linear product for a few rows.
//
// Such a product is bound by the stream of its weights, so the weights go from
// global memory straight into MFMA operand registers (no LDS): lane l holds 8
// consecutive elements of weight row l % 16 at K offset 8 (l / 16). bf16: one
// 16-byte load and one 16x16x32 MFMA per K-step of 32; a wave's load covers 64
// contiguous bytes of 16 rows. fp32: two 16-byte loads (single words where the
// rows are not 16-byte aligned) and eight 16x16x4 fp32 MFMAs, the j-th taking
// element j of every lane. The token rows are the other operand, TT tiles of
// 16, read the same way from L2. A batch of U K-steps is loaded while the
// previous one is multiplied. Columns of the product are independent of each
// other, so a lane whose token does not exist may hold any row's values: its
// column is never read.
#pragma once

#include "common.hpp"

namespace moe {

// Eight consecutive elements of a row.
typedef float f32x8 __attribute__((ext_vector_type(8)));
struct SkinnyBf16 {
    typedef unsigned short type;
    typedef u32x4 frag;
    static __device__ __forceinline__ frag load(const type *p) {
        return *reinterpret_cast<const frag *>(p);
    }
    // n: elements of the row left at p (a multiple of 8)
    static __device__ __forceinline__ frag load_tail(const type *p, int n) {
        return n > 0 ? load(p) : frag{0u, 0u, 0u, 0u};
    }
    static __device__ __forceinline__ f32x4 mma(const frag &a, const frag &b, f32x4 c) {
        return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a),
                                                       __builtin_bit_cast(bf16x8, b), c, 0, 0, 0);
    }
};
template <bool ALIGNED>
struct SkinnyF32 {
    typedef float type;
    typedef f32x8 frag;
    static __device__ __forceinline__ frag load(const type *p) {
        if constexpr (ALIGNED) {
            const f32x4 a = *reinterpret_cast<const f32x4 *>(p);
            const f32x4 b = *reinterpret_cast<const f32x4 *>(p + 4);
            return __builtin_shufflevector(a, b, 0, 1, 2, 3, 4, 5, 6, 7);
        } else {
            return frag{p[0], p[1], p[2], p[3], p[4], p[5], p[6], p[7]};
        }
    }
    static __device__ __forceinline__ frag load_tail(const type *p, int n) {
        frag r;
#pragma unroll
        for (int i = 0; i < 8; ++i)
            r[i] = i < n ? p[i] : 0.f;
        return r;
    }
    static __device__ __forceinline__ f32x4 mma(const frag &a, const frag &b, f32x4 c) {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            c = __builtin_amdgcn_mfma_f32_16x16x4f32(a[i], b[i], c, 0, 0, 0);
        return c;
    }
};

// Product of K columns [kbeg, kend) (multiples of 32, kend possibly past K)
// of a weight row and TT token rows per lane into acc (row 4 (l / 16) + q of
// the weight rows, column l % 16 of the tokens). w and xt[i] point at this
// lane's rows (column 0); NB operand terms per token row, `lo` elements apart,
// are added (2: a row kept as the sum of two bf16 terms). K: columns the rows
// have from w and xt[i] on, which may differ between lanes (those past it are
// zeros); all: the smallest K of the wave.
template <typename S, int TT, int NB, int U>
__device__ __forceinline__ void skinny_mma(const typename S::type *w,
                                           const typename S::type *const (&xt)[TT], int64_t lo,
                                           int kbeg, int kend, int K, int all,
                                           f32x4 (&acc)[TT]) {
    typedef typename S::frag frag;
    struct Step {
        frag a, b[TT][NB];
    };
    const int ko = 8 * (int)(__lane_id() >> 4);
    const int full = min(kend, all / 32 * 32);   // steps that need no mask
    // the weights of a batch first: their addresses are known before the token
    // rows', which come from the dispatch plan
    auto load = [&](int k, Step (&s)[U]) {
#pragma unroll
        for (int u = 0; u < U; ++u)
            s[u].a = S::load(w + ko + k + 32 * u);
#pragma unroll
        for (int u = 0; u < U; ++u)
#pragma unroll
            for (int i = 0; i < TT; ++i)
#pragma unroll
                for (int n = 0; n < NB; ++n)
                    s[u].b[i][n] = S::load(xt[i] + n * lo + ko + k + 32 * u);
    };
    auto mma = [&](const Step &s) {
#pragma unroll
        for (int i = 0; i < TT; ++i)
#pragma unroll
            for (int n = 0; n < NB; ++n)
                acc[i] = S::mma(s.a, s.b[i][n], acc[i]);
    };
    Step next[U];
    int k = kbeg;
    if (k + 32 * U <= full) {
        load(k, next);
        for (k += 32 * U; k + 32 * U <= full; k += 32 * U) {
            Step cur[U];
#pragma unroll
            for (int u = 0; u < U; ++u)
                cur[u] = next[u];
            load(k, next);
#pragma unroll
            for (int u = 0; u < U; ++u)
                mma(cur[u]);
        }
#pragma unroll
        for (int u = 0; u < U; ++u)
            mma(next[u]);
    }
    for (; k < kend; k += 32) {
        // single steps, masked where they reach past K
        const int left = K - k - ko;
        Step s;
        s.a = S::load_tail(w + ko + k, left);
#pragma unroll
        for (int i = 0; i < TT; ++i)
#pragma unroll
            for (int n = 0; n < NB; ++n)
                s.b[i][n] = S::load_tail(xt[i] + n * lo + ko + k, left);
        mma(s);
    }
}

}  // namespace moe
