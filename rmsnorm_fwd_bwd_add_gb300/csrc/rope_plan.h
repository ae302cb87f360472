// rope_plan.h -- how a rotary call's tokens and heads are dealt out to warps (host
// only; the kernel is in rope_ex.cu).
#pragma once

#include <algorithm>
#include <cstdint>

namespace rmsn {

struct RopePlan {
    int64_t whole;  // tokens of one warp each, ahead of the rest
    int wpt;        // warps a token of the rest
    int cw;         // units of a head a warp takes at a time
    int grid;
};

// Warps a token (k) and units a step (c) for heads of `lanes` units, `in_flight` of them
// loaded ahead.  Each warp computes its units' angles, about half a trip to memory, and
// makes a trip for every few heads.  All warps go through equal rounds of whole tokens;
// what is left, less than a round, is split into as many parts as there are warps for
// (5001 tokens on 2432 warps: 19.7 us with a third round of 137 whole tokens, 17.4 with
// them in 16 parts each).  Up to 12 steps a head are weighed, or the fewest that a long
// head in small units allows (4096 tokens of 8 heads of 1024 off 16-byte boundaries: 75
// us, and 1154 in single units).
inline RopePlan make_rope_plan(int64_t T, int lanes, int heads, int in_flight, int ctas, int cta_warps) {
    const int64_t warps = (int64_t)ctas * cta_warps;
    RopePlan p{T / warps * warps, 1, 1, 0};
    const int64_t rest = T - p.whole;
    int64_t best = INT64_MAX;
    const int least = (lanes + 31) / 32;
    for (int steps = least; steps <= std::max(12, least); ++steps) {
        const int c = (lanes + steps - 1) / steps;  // a head in `steps` equal steps
        auto cost_of = [&](int64_t rounds, int k) {
            const int per_trip = (32 / c) * in_flight * k, trips = (heads + per_trip - 1) / per_trip;
            return rounds * (1 + (1 + 2 * trips) * steps);
        };
        for (int k = 1; k <= 16; k *= 2) {
            const int64_t cost = cost_of(p.whole / warps, 1) + cost_of((rest * k + warps - 1) / warps, k);
            if (cost < best) {
                best = cost;
                p.wpt = k;
                p.cw = c;
            }
        }
        if (c == 1) break;
    }
    const int64_t items = p.whole + rest * p.wpt;
    p.grid = (int)std::min<int64_t>((items + cta_warps - 1) / cta_warps, ctas);
    return p;
}

}  // namespace rmsn
