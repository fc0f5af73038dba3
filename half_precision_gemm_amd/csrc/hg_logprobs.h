// Internal interface of hg_logprobs and hg_logprobs_grad
// (include/hgemm_logprobs.h): what the host passes to the kernels.
#pragma once

#include <stdint.h>

#include <hip/hip_runtime.h>

namespace hg {
namespace probs {

constexpr int kThreads = 256;
constexpr int kGroup = 8;                 // neighbouring logits that one lane loads together
constexpr int kMostParts = 64;            // that rows are cut into to fill the GPU
constexpr int kLongestParts = 65;         // of the longest parts in a row of 2^20 logits, wherever in a group it begins

// A row's parts: `per` groups each, `groups` (1, 2, 4 or 8) for a lane of `waves` (1
// or 4) waves.
struct Parts {
    int32_t waves, groups, parts, per;
};

// What a piece leaves for its row, 16 bytes and `top` keys.
struct Partial {
    float largest, sum, weighted, unused;
};

struct Forward {
    const void *X;
    const int64_t *tokens;
    float *logp, *entropy, *stats, *top_logp;
    int64_t *top_ids;
    Partial *partials;                    // rows×parts, null with one part
    uint64_t *keys;                       // rows×parts×top
    int64_t ldx, M;
    float scale;
    int32_t V, top, type;                 // type as in the public headers
    Parts parts;
};
hipError_t launch_forward(const Forward &f, hipStream_t s);

struct Backward {
    const void *X;
    void *dX;
    const int64_t *tokens;
    const float *stats, *entropy, *dlogp, *dentropy;
    int64_t ldx, ldd, M;
    float scale;
    int32_t V, type;
};
hipError_t launch_backward(const Backward &b, hipStream_t s);

}  // namespace probs
}  // namespace hg
