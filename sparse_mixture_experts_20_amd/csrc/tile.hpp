// Tiled matrix product on the matrix cores (private; not part of the C ABI),
// the main loop of the linear product and of the few-token layer's experts with
// more than a few rows: a BM x BN tile of A B over K, K-step 64 in an LDS ring
// of S stages filled by direct global-to-LDS loads (16 bytes a lane), WM x WN
// waves of 16x16x32 bf16 MFMAs. An operand whose rows run along K is staged row
// by row; one stored the other way is staged as it lies and turned into
// fragments by the transposing LDS read. The output's columns are the MFMA's
// rows, and each 64 columns of a wave are dealt to four fragments so that a
// lane ends with 16 adjacent columns of one row: epilogues store whole 128-byte
// lines from registers, with no pass through LDS.
#pragma once

#include "common.hpp"

namespace moe {
namespace {

constexpr int kStep = 64;   // K-step of the tiled product

template <int N>
__device__ __forceinline__ void wait_loads() {   // until at most N are in flight
    asm volatile("s_waitcnt vmcnt(%0)" ::"n"(N) : "memory");
}

// Direct copy of 16 bytes per lane to LDS: lane l's bytes land at base + 16 l.
// In asm so that the compiler does not wait for it before every LDS read; the
// waits are explicit.
__device__ __forceinline__ void copy_to_lds(unsigned base, const void *g) {
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %1, off"
                 ::"s"(base), "v"(g)
                 : "memory", "m0");
}
__device__ __forceinline__ unsigned lds_address(const void *p) {
    return (unsigned)(uintptr_t)((__attribute__((address_space(3))) const void *)p);
}
typedef short s16x4 __attribute__((ext_vector_type(4)));
// Transposing LDS read: within 16 lanes, lane l gets element l % 4 of the 8
// bytes that lane 4 q + l / 4 addresses, as its element q.
__device__ __forceinline__ s16x4 read_transposed(const void *p) {
    return __builtin_amdgcn_ds_read_tr16_b64_v4i16((__attribute__((address_space(3))) s16x4 *)(p));
}

template <int BM, int BN, int WM, int WN, int S, bool AT, bool BT>
struct TileProduct {
    static constexpr int NW = WM * WN, THREADS = NW * 64, WAVES_N = WN;
    static constexpr int FM = BM / WM / 16, FN = 4;
    static constexpr int ABYTES = BM * kStep * 2, BBYTES = BN * kStep * 2;
    static constexpr int STAGE = ABYTES + BBYTES, LDS = S * STAGE;
    static constexpr int IA = ABYTES / (NW * 1024), IB = BBYTES / (NW * 1024);
    static_assert(BN / WN == 64, "a wave holds 64 columns");
    static_assert(IA * NW * 1024 == ABYTES && IB * NW * 1024 == BBYTES, "whole wave copies");
    static_assert(S >= 2 && (S - 2) * (IA + IB) < 64, "a wait counts to 63");

    // acc[i][j] += this wave's part of the tile over K-steps [kb, ke) (of
    // ceil(K / 64)): lane l gets row 16 i + l % 16 of the wave's 16 FM rows
    // and, in acc[i][j][q], column 16 (l / 16) + 4 j + q of its 64 columns.
    // a(r): row r of the tile (with AT: its column 8 r, rows of lda); b likewise
    // for the tile's columns. Rows and columns past the edge may point at any
    // valid place (their products are not read). K % 8 == 0 for an operand that
    // runs along K. smem: LDS bytes, 1024-byte aligned; every thread calls.
    // SUMS: where `on` (per wave), sum[i][q] += the sum along K of A's row
    // 16 i + l % 16 as well, one product with a fragment of ones.
    template <bool SUMS, typename PA, typename PB>
    static __device__ __forceinline__ void run(char *smem, PA a, int lda, PB b, int ldb, int K,
                                               int kb, int ke, f32x4 (&acc)[FM][FN], bool on,
                                               f32x4 (&sum)[FM]) {
        const bf16x8 ones = __builtin_bit_cast(
            bf16x8, u32x4{0x3f803f80u, 0x3f803f80u, 0x3f803f80u, 0x3f803f80u});
        const int lane = threadIdx.x & 63;
        const int wv = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
        const int wm = wv / WN, wn = wv % WN;
        const int KT = (K + kStep - 1) / kStep;

        // Copy sources: per wave copy one 16-byte chunk per lane. Row-major tile:
        // row r of 8 chunks, chunk c kept at position c ^ f(r); tile stored the
        // other way: row k of BM/8 (BN/8) chunks, chunk c at c ^ g(k).
        auto fa = [](int r) { return (r >> 1) & 7; };                       // 16 adjacent rows
        auto fb = [](int r) { return ((r >> 1) & 1) | ((r >> 3) & 6); };    // rows 16 i + 4 j + 0..3
        auto ga = [](int k) {                                          // rows 8 i + 4 j + 0..3
            return BM == 64 ? (k & 2) | ((k >> 1) & 4) : 2 * ((k & 3) | ((k >> 1) & 4));
        };
        auto gb = [](int k) { return (k & 1) | ((k & 2) << 2); };
        // chunk q of a tile: its K offset within the step, and the row (or 8
        // columns) it belongs to
        auto a_off = [&](int q) { return AT ? q / (BM / 8) : 8 * ((q % 8) ^ fa(q / 8)); };
        auto b_off = [&](int q) { return BT ? q / (BN / 8) : 8 * ((q % 8) ^ fb(q / 8)); };
        const int64_t as = AT ? lda : 1, bs = BT ? ldb : 1;   // elements per step of K
        // Each copy's source at K-step 0 and the last step's offset that stays
        // within K: in the last step, chunks past K read the last one of K
        // instead (zeroed below). (A branch for the last step alone was 3% slower.)
        const unsigned short *pa[IA], *pb[IB];
        int la[IA], lb[IB];
#pragma unroll
        for (int i = 0; i < IA; ++i) {
            const int q = (wv * IA + i) * 64 + lane;
            pa[i] = a(AT ? (q % (BM / 8)) ^ ga(a_off(q)) : q / 8) + a_off(q) * as;
            la[i] = (AT ? K - 1 : K - 8) - a_off(q);
        }
#pragma unroll
        for (int i = 0; i < IB; ++i) {
            const int q = (wv * IB + i) * 64 + lane;
            pb[i] = b(BT ? (q % (BN / 8)) ^ gb(b_off(q)) : q / 8) + b_off(q) * bs;
            lb[i] = (BT ? K - 1 : K - 8) - b_off(q);
        }
        const unsigned base = lds_address(smem);
        auto issue = [&](int kt) {
            const unsigned st = base + (unsigned)(kt % S) * STAGE;
#pragma unroll
            for (int i = 0; i < IA; ++i)
                copy_to_lds(st + (unsigned)(wv * IA + i) * 1024,
                            pa[i] + min(kt * kStep, la[i]) * as);
#pragma unroll
            for (int i = 0; i < IB; ++i)
                copy_to_lds(st + ABYTES + (unsigned)(wv * IB + i) * 1024,
                            pb[i] + min(kt * kStep, lb[i]) * bs);
        };
        // chunks of the last step that lie past K, in both operands
        auto zero_tail = [&](int kt) {
            char *st = smem + (kt % S) * STAGE;
            const u32x4 zero = {0u, 0u, 0u, 0u};
            for (int q = threadIdx.x; q < ABYTES / 16; q += NW * 64)
                if (kt * kStep + a_off(q) >= K)
                    *reinterpret_cast<u32x4 *>(st + q * 16) = zero;
            for (int q = threadIdx.x; q < BBYTES / 16; q += NW * 64)
                if (kt * kStep + b_off(q) >= K)
                    *reinterpret_cast<u32x4 *>(st + ABYTES + q * 16) = zero;
        };
        const int l16 = lane & 15, g = lane >> 4;
        auto frag_a = [&](const char *st, int ks, int i) {
            if constexpr (AT) {
                const int col = wm * FM * 16 + i * 16 + 4 * (l16 & 3);
                s16x4 q[2];
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const int k = ks * 32 + 8 * g + 4 * h + (l16 >> 2);
                    q[h] = read_transposed(st + k * BM * 2 + (((col >> 3) ^ ga(k)) << 4) +
                                           (col & 7) * 2);
                }
                return __builtin_bit_cast(bf16x8,
                                          __builtin_shufflevector(q[0], q[1], 0, 1, 2, 3, 4, 5, 6, 7));
            } else {
                const int r = wm * FM * 16 + i * 16 + l16;
                return *reinterpret_cast<const bf16x8 *>(st + r * 128 + (((ks * 4 + g) ^ fa(r)) << 4));
            }
        };
        // fragment j of the wave's 64 columns: its index i is column 16 (i / 4) + 4 j + i % 4
        auto frag_b = [&](const char *st, int ks, int j) {
            st += ABYTES;
            if constexpr (BT) {
                const int col = wn * 64 + 16 * (l16 & 3) + 4 * j;
                s16x4 q[2];
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const int k = ks * 32 + 8 * g + 4 * h + (l16 >> 2);
                    q[h] = read_transposed(st + k * BN * 2 + (((col >> 3) ^ gb(k)) << 4) +
                                           (col & 7) * 2);
                }
                return __builtin_bit_cast(bf16x8,
                                          __builtin_shufflevector(q[0], q[1], 0, 1, 2, 3, 4, 5, 6, 7));
            } else {
                const int r = wn * 64 + 16 * (l16 >> 2) + 4 * j + (l16 & 3);
                return *reinterpret_cast<const bf16x8 *>(st + r * 128 + (((ks * 4 + g) ^ fb(r)) << 4));
            }
        };
#pragma unroll
        for (int s = 0; s < S - 1; ++s)
            if (kb + s < ke)
                issue(kb + s);
        for (int kt = kb; kt < ke; ++kt) {
            // step kt has landed; the later ones issued so far may stay in flight
            // (the last S - 2 steps wait for all that is in flight)
            if (kt + S - 2 < ke)
                wait_loads<(S - 2) * (IA + IB)>();
            else
                wait_loads<0>();
            barrier_lds();
            // (with transposing reads the next copies go out behind the first reads
            // of the step, which the copies' issue would hold up. Both forms timed in
            // turn, behind and before: GELU backward 4096x4096x14336 847 and 918 us,
            // 8192x2048x7168 471 and 532, 16384x768x3072 263 and 255; 2047x3072x768
            // 38.2 and 39.1. Row by row there is no difference: 4096x4096x14336
            // forward 419 and 423 us, 8192x2048x7168 224 and 223)
            if (!BT && kt + S - 1 < ke)
                issue(kt + S - 1);
            if (kt == KT - 1 && K % kStep != 0) {
                zero_tail(kt);
                barrier_lds();
            }
            const char *st = smem + (kt % S) * STAGE;
#pragma unroll
            for (int ks = 0; ks < kStep / 32; ++ks) {
                bf16x8 fB[FN];
#pragma unroll
                for (int j = 0; j < FN; ++j)
                    fB[j] = frag_b(st, ks, j);
                // (the row fragments one by one: with both operands transposed the
                // 16 waves' 128 registers do not hold all of them as well)
#pragma unroll
                for (int i = 0; i < FM; ++i) {
                    const bf16x8 fA = frag_a(st, ks, i);
                    if (BT && ks == 0 && i == 0 && kt + S - 1 < ke)
                        issue(kt + S - 1);
#pragma unroll
                    for (int j = 0; j < FN; ++j)
                        acc[i][j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(fB[j], fA, acc[i][j],
                                                                             0, 0, 0);
                    if (SUMS && on)
                        sum[i] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(ones, fA, sum[i], 0, 0, 0);
                }
            }
        }
    }
    template <typename PA, typename PB>
    static __device__ __forceinline__ void run(char *smem, PA a, int lda, PB b, int ldb, int K,
                                               int kb, int ke, f32x4 (&acc)[FM][FN]) {
        f32x4 none[FM];
        run<false>(smem, a, lda, b, ldb, K, kb, ke, acc, false, none);
    }
};

}  // namespace
}  // namespace moe
