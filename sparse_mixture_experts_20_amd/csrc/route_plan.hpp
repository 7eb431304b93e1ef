// The host's choice between the forms of the routing's score product (private; no
// HIP in here, so that it also builds into a program for the CPU).
#pragma once

#include <algorithm>
#include <cstdint>

namespace moe {

// Which form of the score product (route.hip) a call takes (without tokens the fused one,
// which needs no workspace).
enum RouteForm { kFused, kRanges, kTiled };
struct RoutePlan {
    RouteForm form;
    int Q, ld, tt, ranges;   // experts a lane, row stride of P, token tiles, column ranges
};
inline RoutePlan route_plan(bool bf16, int64_t N, int64_t d, int E) {
    RoutePlan p{};
    p.Q = E <= 64 ? 1 : E <= 128 ? 2 : 4;
    p.ld = E <= 64 ? (E + 15) / 16 * 16 : 64 * p.Q;
    const int64_t weights = (int64_t)(E + 15) / 16 * 16 * d;
    // A fused workgroup reads all of W_g, which saves a launch where that is little: as
    // graphs of calls 64 tokens and 8 experts of width 768 7.9 us (ranges 8.8), of 4096
    // 11.8 (8.7); as calls 2047 of these 13.5 (15.6), 777 of 60 experts of 515 14.5 (16.5).
    if (N == 0 || (E <= 64 && weights <= (N > 1024 ? 65536 : 36864))) {
        p.form = kFused;
        return p;
    }
    // The tiled product (its scratch is laid out for more than 32 experts) costs a
    // launch that splits W_g and the start of its large tiles, and then less per token:
    // measured (us, with the ranking) 26 + 25 for each 2^20 weights + 3.2 for each 10^9
    // products, ranges 8 + 27 (256 experts of 7168: 512 tokens 73 and 34, 2048 tokens 63
    // and 87; of 1024: 2048 tokens 38 and 21).
    if (bf16 && E > 32 && (double)N * weights > 0.75e9 + 1040.0 * p.ld * d) {
        p.form = kTiled;
        return p;
    }
    p.form = kRanges;
    p.tt = N <= 16 ? 1 : N <= 32 ? 2 : 4;
    const int64_t blocks = (E + 15) / 16 * ((N + 16 * p.tt - 1) / (16 * p.tt));
    const int64_t steps = (d + 31) / 32;
    p.ranges = (int)std::min<int64_t>(std::max<int64_t>(512 / blocks, 1), (steps + 15) / 16);
    return p;
}

}  // namespace moe
