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
    // A fused workgroup of 16 tokens reads all of W_g, which saves a launch where that is
    // little. Timed in turn, one kernel and ranges, in graphs of calls (us): 256 tokens, 8
    // experts of 768 7.8 and 8.5, of 2048 7.9 and 8.9, of 3000 10.0 and 8.0, 16 of 2304
    // 11.6 and 9.0, 64 of 800 10.3 and 8.2: to 36864 weights. As calls, whose second
    // launch the host takes 2 us longer for, 1536 tokens, 32 experts of 1536 12.7 and 14.5,
    // 64 of 1024 12.4 and 14.2, 8 of 4104 12.2 and 14.4, of 5120 16.4 and 14.6, of 7168
    // 20.0 and 14.1: to 73728 for a batch. (Past 4096 tokens, in a second round of the
    // CUs, either may be faster: 5000 tokens, 8 of 2304 17.5 and 14.7, 32 of 2048 24.9 and
    // 21.8, 8192 tokens, 8 of 512 9.5 and 10.8, of 2304 17.7 and 19.2, of 4096 23.7 and 23.3.)
    if (N == 0 || (E <= 64 && weights <= (N > 1024 ? 73728 : 36864))) {
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
