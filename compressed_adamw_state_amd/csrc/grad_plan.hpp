// How weight_grad.hip does a product (host only, so that the tests can ask it which
// way a size takes).
#pragma once

#include <cmath>
#include <cstddef>
#include <cstdint>

#include "flashopt_lm.h"

namespace flashopt {

constexpr int kTokens = 32;                      // of a stage

// How a product is done: tiles of 64 x 128 by teams of a block that share out its tokens,
// tiles of 128 x 128, or large ones of 256 x 256 (FP32: 128 x 256); and what of a workspace
// it needs.
struct GradPlan {
    enum Way { kTeams, kSmall, kLarge } way;
    int64_t tn, tk, whole, splits;
    size_t part, bias;                           // bytes
};

// A way's time in us: what every call takes, a stage of a block, a block's beginning
// and end, a second launch, a piece's sums written and read; and how many times a
// block's time a launch takes at `load` blocks a CU: some load + some of its
// whole rounds (of 1 / steps) + a rest.  Fitted to 283 measurements of 16-bit products
// (40 sizes of 64 to 16384 tokens, 128 to 8192 columns, whole and cut into 2 to 16
// pieces) and 602 of FP32 ones (47 sizes), whose times it gives within 4 to 7 % (27 at
// worst); the ways it chose for them took 0.2 % (FP32: 2 %) more than the best ones, 4
// (16) at worst.
struct WayTime {
    double call, stage, ends, join, piece, load, rounds, rest, steps;

    double blocks(int64_t count, int64_t stages) const {
        const double l = (double)count / 256;
        const double r = l <= 1.0 && rest == 0.0
                             ? 1.0 : std::fmax(1.0, load * l + rounds * std::ceil(steps * l) / steps + rest);
        return r * ((double)stages * stage + ends);
    }
};

// m tokens, n x ld outputs (ld: the held input's columns with their padding)
static inline GradPlan grad_plan(int32_t type, int64_t m, int64_t n, int64_t ld, bool bias) {
    static const WayTime times[2][3] = {{{3.69, 0.668, 3.30, 2.00, 0.0098, 0.227, 1.018, 0.0, 1.0},
                                         {3.97, 0.341, 2.14, 2.11, 0.0157, 0.821, 0.0, 0.769, 1.0},
                                         {6.29, 0.681, 3.92, 9.57, 0.0, 1.265, 0.0, 0.342, 1.0}},
                                        {{4.60, 0.776, 1.83, 1.40, 0.0110, 0.255, 0.958, 0.0, 1.0},
                                         {7.60, 0.853, 0.40, 0.22, 0.0222, 0.384, 0.590, 0.0, 1.0},
                                         {10.17, 1.348, 0.0, 0.0, 0.0349, 0.0, 1.123, 0.0, 2.0}}};
    static const int32_t cuts[] = {1, 2, 3, 4, 5, 6, 7, 8, 10, 12, 14, 16, 20, 24, 28, 32};
    const bool fp32 = type == FLASHOPT_FP32;
    const int64_t stages = (m + kTokens - 1) / kTokens;
    GradPlan best = {};
    double least = INFINITY;
    for (int w = 0; w < 3; ++w) {
        const GradPlan::Way way = (GradPlan::Way)w;
        const WayTime& t = times[fp32][w];
        const int64_t teams = way == GradPlan::kTeams ? (fp32 ? 2 : 4) : 1;
        const int64_t high = way == GradPlan::kTeams ? 64 : way == GradPlan::kSmall || fp32 ? 128 : 256;
        const int64_t wide = way == GradPlan::kLarge ? 256 : 128;
        const int64_t tn = (n + high - 1) / high, tk = (ld + wide - 1) / wide, tiles = tn * tk;
        if (way == GradPlan::kTeams && tiles > 4096) continue;           // (2^32 threads and more)
        for (const int64_t cut : cuts) {
            int64_t whole = tiles, splits = cut;
            if (way == GradPlan::kLarge && !fp32) {
                // the tiles behind the last full round of the CUs, if they are half a round at most
                if (cut > 1) break;
                const int64_t rest = tiles % 256;
                splits = rest ? 256 / rest : 1;
                if (stages < 16 * splits) splits = 1;
                if (splits > 1) whole = tiles - rest;
            } else if (cut > 1) {
                if (tiles * cut > 1024 || stages < 2 * cut * teams) break;
                whole = 0;
            }
            const int64_t pieces = (tiles - whole) * splits, parts = splits * teams;
            double time = t.call + (whole ? t.blocks(whole, (stages + teams - 1) / teams) : 0.0);
            if (pieces) time += t.blocks(pieces, (stages + parts - 1) / parts) + t.join + t.piece * (double)pieces;
            if (time >= least) continue;
            least = time;
            best = {way, tn, tk, whole, splits, (size_t)(pieces * high * wide) * sizeof(float),
                    bias ? (size_t)(pieces * high) * sizeof(float) : 0};
        }
    }
    return best;
}

}  // namespace flashopt
