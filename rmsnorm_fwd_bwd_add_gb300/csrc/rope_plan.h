// rope_plan.h -- how the tokens and heads of the rotary calls, of the 8-bit append and of
// the read are dealt out to warps (host only; the kernels are in rope_ex.cuh and
// kv_cache8.cuh).
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

// How the 8-bit append deals tokens out: those of one warp each, warps a token of the rest
// (a power of two), lanes a head.
struct Append8Plan {
    int64_t whole;
    int wpt, cw, grid;
};

// All warps go through equal rounds of whole tokens; of what is left, less than a round,
// each token is split into as many parts as cost least.  A part costs its positions and
// cosines, and its steps of 32 / cw heads (kv: of k and of v, or of k alone); none is
// without heads.  The costs' ratios are estimates (a step: two 16-byte vectors a unit), the
// choices measured: for 8 to 9800 tokens of 32 + 8 and 8 + 1 heads of 128, 16 + 4 of 64 and 32
// + 8 of 100, and for the rotation of 32 + 8 heads of 128 and 16 + 16 fp32 heads of 80, the
// time was within 2 % of the best of 1, 2, 4, 8 and 16 parts (300 tokens of 32 + 8 heads of
// 128 7.4, 5.2, 4.4, 4.5, 4.4 us, 4.4 so; 1000 8.3, 7.0, 9.0, 12.6, 12.6, and 6.9; 3000 17.9,
// 15.3, 14.6, 16.5, 16.4, and 14.6).
inline Append8Plan make_append8_plan(int64_t T, int cw, int Hq, int Hkv, int kv, int pairs, int units, int ctas, int cta_warps) {
    const int64_t warps = (int64_t)ctas * cta_warps;
    const int hpi = 32 / cw, most = (std::max(Hq, Hkv) + hpi - 1) / hpi;
    Append8Plan p{T / warps * warps, 1, cw, 0};
    const int64_t rest = T - p.whole;
    int64_t best = INT64_MAX;
    for (int k = 1; k <= 16 && k <= most; k *= 2) {
        const int steps = (Hq + hpi * k - 1) / (hpi * k) + kv * ((Hkv + hpi * k - 1) / (hpi * k));
        const int64_t cost = (rest * k + warps - 1) / warps * (200 + 60 * ((pairs + 31) / 32) + 90 * units * steps);
        if (cost < best) {
            best = cost;
            p.wpt = k;
        }
    }
    const int64_t items = p.whole + rest * p.wpt;
    p.grid = (int)std::min<int64_t>((items + cta_warps - 1) / cta_warps, ctas);
    return p;
}

// How a read from the 8-bit cache deals tokens out: lanes a head, warps a token (a power
// of two) or tokens a warp at a time.
struct Read8Plan {
    int cw, wpt, tokens, grid;
};

// As many lanes a head as it has units, or fewer where a token's heads then take a fifth
// fewer steps (8 heads of 45 units: 4 x 3 steps of 15 lanes, 8 x 2 of 32; 16384 such
// tokens 22.7 us, 26.7 so; but 3 heads of 45, 1 x 5 steps of 9 lanes, 3 x 2 of 32: 11.8 and
// 10.1, for the wider stores).
inline Read8Plan make_read8_plan(int64_t T, int units, int Hkv, int sm, int per_sm, int per_sm_tokens, int cta_warps) {
    Read8Plan p{};
    auto steps = [&](int cw) { return (int64_t)((Hkv + 32 / cw - 1) / (32 / cw)) * ((units + cw - 1) / cw); };
    p.cw = std::min(units, 32);
    int64_t most = steps(p.cw) * 4 / 5;
    for (int cw = p.cw - 1; cw >= 1; --cw)
        if (steps(cw) <= most) {
            most = steps(cw) - 1;
            p.cw = cw;
        }
    const int hpi = 32 / p.cw;
    const int64_t warps = (int64_t)sm * per_sm * cta_warps;
    p.wpt = 1;
    while (p.wpt < 64 && 2 * p.wpt * T <= warps && p.wpt * hpi < Hkv) p.wpt *= 2;
    p.tokens = std::max(1, hpi / Hkv);
    const int64_t items = p.tokens > 1 ? (T + p.tokens - 1) / p.tokens : T * p.wpt;
    p.grid = (int)std::min<int64_t>((items + cta_warps - 1) / cta_warps, (int64_t)sm * (p.tokens > 1 ? per_sm_tokens : per_sm));
    return p;
}

}  // namespace rmsn
