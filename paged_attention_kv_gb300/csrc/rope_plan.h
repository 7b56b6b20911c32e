// How qk_rope_kernel shares a token's heads among warps. Host code only.
#pragma once

#include <climits>

namespace pkv {

// A warp's look-ups (position, cosines and sines, first heads on their way), in
// steps of the heads that it takes.
constexpr int kLookUpSteps = 1;

// Warps that share a token's heads: those for which the rounds of warps, each
// with its look-ups and its steps, come to the least, and the most of these. Few
// tokens get as many as run at once (512 tokens of 10 steps: 7 warps a token 3.7
// us, 10 4.5, 1 6.5), many one each, which looks things up once (6000 tokens: 25
// us, 7 warps 35); between, it goes by how the rounds fill (2240 tokens: 1, 2, 3
// and 4 warps 13.5, 12.4, 11.9, 13.0 us).
inline int rope_parts(long long tokens, int steps, long long warps_at_once) {
    int best = 1;
    long long least = LLONG_MAX;
    for (int p = 1; p <= steps && (p == 1 || tokens * p <= 4 * warps_at_once); ++p) {
        const long long rounds = (tokens * p + warps_at_once - 1) / warps_at_once;
        const long long cost = rounds * ((steps + p - 1) / p + kLookUpSteps);
        if (cost <= least) {
            least = cost;
            best = p;
        }
    }
    return best;
}

}  // namespace pkv
