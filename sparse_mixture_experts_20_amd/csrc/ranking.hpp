// What the router and the few-token layer share (private; not part of the C
// ABI): the exact three-term split of fp32 router weights and the top-k with
// softmax of one token's scores by one wave.
#pragma once

#include "common.hpp"

namespace moe {
namespace {

// Exact three-term split of two fp32 weights, w = hi + mid + lo, by
// truncation: hi keeps the upper 16 bits of w (sign, exponent and the top 7
// stored significand bits), mid the upper 16 bits of the residual w - hi
// (exact, at most 16 significant bits), and lo = (w - hi) - mid, which is
// exact and has at most 8 significant bits, so it is a bf16 value too. A
// term's bf16 encoding is its upper 16 bits; the pair is packed with a in the
// low half, b in the high half (bf16 elements 2j and 2j+1 of a vector).
__device__ __forceinline__ void split3x2(float a, float b, unsigned &hi, unsigned &mid,
                                         unsigned &lo) {
    const unsigned ha = __float_as_uint(a) & 0xffff0000u, hb = __float_as_uint(b) & 0xffff0000u;
    const float ra = a - __uint_as_float(ha), rb = b - __uint_as_float(hb);
    const unsigned ma = __float_as_uint(ra) & 0xffff0000u, mb = __float_as_uint(rb) & 0xffff0000u;
    const float la = ra - __uint_as_float(ma), lb = rb - __uint_as_float(mb);
    hi = (ha >> 16) | hb;
    mid = (ma >> 16) | mb;
    lo = (__float_as_uint(la) >> 16) | (__float_as_uint(lb) & 0xffff0000u);
}

// Split of 8 consecutive weights (w0 = elements 0-3, w1 = elements 4-7).
__device__ __forceinline__ void split8(const f32x4 &w0, const f32x4 &w1, u32x4 &hi, u32x4 &mid,
                                       u32x4 &lo) {
    unsigned h[4], m[4], l[4];
    split3x2(w0[0], w0[1], h[0], m[0], l[0]);
    split3x2(w0[2], w0[3], h[1], m[1], l[1]);
    split3x2(w1[0], w1[1], h[2], m[2], l[2]);
    split3x2(w1[2], w1[3], h[3], m[3], l[3]);
    hi = u32x4{h[0], h[1], h[2], h[3]};
    mid = u32x4{m[0], m[1], m[2], m[3]};
    lo = u32x4{l[0], l[1], l[2], l[3]};
}

// Order of scores as unsigned numbers above 0 (NaN ranks as -inf; -0 as +0, which
// compare equal), and back.
__device__ __forceinline__ unsigned order_of(float v) {
    const unsigned b = __float_as_uint(v != v ? -INFINITY : v + 0.f);
    return (b & 0x80000000u) ? ~b : (b | 0x80000000u);
}
__device__ __forceinline__ float order_value(unsigned o) {
    return __uint_as_float((o & 0x80000000u) ? (o & 0x7fffffffu) : ~o);
}
// Ranking key of (score, expert): ordered as the scores, descending, then the
// ids, ascending.
__device__ __forceinline__ uint64_t rank_key(float v, int e) {
    return ((uint64_t)order_of(v) << 32) | (uint64_t)(0xffffffffu - (unsigned)e);
}
__device__ __forceinline__ float key_score(uint64_t key) {
    return order_value((unsigned)(key >> 32));
}
template <int CTRL, int ROWS = 0xf>
__device__ __forceinline__ uint64_t dpp_max(uint64_t x) {
    const int lo = (int)(unsigned)x, hi = (int)(unsigned)(x >> 32);
    const unsigned olo = (unsigned)__builtin_amdgcn_update_dpp(lo, lo, CTRL, ROWS, 0xf, false);
    const unsigned ohi = (unsigned)__builtin_amdgcn_update_dpp(hi, hi, CTRL, ROWS, 0xf, false);
    const uint64_t o = ((uint64_t)ohi << 32) | olo;
    return o > x ? o : x;
}
// The largest key of the wave, on every lane: within quads, rows of 16, then
// across rows; lane 63 ends with the maximum of all 64.
__device__ __forceinline__ uint64_t wave_max_key(uint64_t x) {
    x = dpp_max<0xb1>(x);          // quad_perm [1,0,3,2]
    x = dpp_max<0x4e>(x);          // quad_perm [2,3,0,1]
    x = dpp_max<0x124>(x);         // row_ror:4
    x = dpp_max<0x128>(x);         // row_ror:8
    x = dpp_max<0x142, 0xa>(x);    // row_bcast:15 into rows 1 and 3
    x = dpp_max<0x143, 0xc>(x);    // row_bcast:31 into rows 2 and 3
    const unsigned lo = (unsigned)__builtin_amdgcn_readlane((int)(unsigned)x, 63);
    const unsigned hi = (unsigned)__builtin_amdgcn_readlane((int)(unsigned)(x >> 32), 63);
    return ((uint64_t)hi << 32) | lo;
}

// Top-k of one token's scores held by a whole wave (lane g holds experts g,
// g+64, ...), as the router's ranking by groups of lanes does: every round takes the
// wave's largest ranking key by DPP moves (no LDS shuffles) and the softmax
// sums the kept choices' terms in choice order from uniform reads.
template <int Q>
__device__ __forceinline__ void topk_softmax_wave(const float (&v)[Q], int E, int k, int64_t t,
                                                  bool active, int32_t *__restrict__ idx_out,
                                                  float *__restrict__ gate_out) {
    const int lane = __lane_id();
    uint64_t key[Q];
#pragma unroll
    for (int q = 0; q < Q; ++q) {
        const int e = lane + 64 * q;
        key[q] = e < E ? rank_key(v[q], e) : 0ull;   // 0: no candidate
    }
    float my_v = -INFINITY, v0 = -INFINITY;
    int my_e = 0;
    for (int j = 0; j < k; ++j) {
        uint64_t b = key[0];
#pragma unroll
        for (int q = 1; q < Q; ++q)
            b = key[q] > b ? key[q] : b;
        b = wave_max_key(b);
        const int be = (int)(0xffffffffu - (unsigned)b);
        const float bv = key_score(b);
#pragma unroll
        for (int q = 0; q < Q; ++q)
            if (be == lane + 64 * q)
                key[q] = 0ull;
        if (lane == j) {
            my_v = bv;
            my_e = be;
        }
        if (j == 0)
            v0 = bv;
    }
    const float ex = lane < k ? expf(my_v - v0) : 0.f;
    float den = 0.f;
    for (int j = 0; j < k; ++j)   // choice order
        den += __uint_as_float(
            (unsigned)__builtin_amdgcn_readlane((int)__float_as_uint(ex), j));
    if (active && lane < k) {
        idx_out[t * k + lane] = my_e;
        gate_out[t * k + lane] = ex / den;
    }
}

}  // namespace
}  // namespace moe
