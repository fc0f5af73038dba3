// Internal interface of hg_adamw (include/hgemm_adamw.h): what the host passes to
// the kernel.
#pragma once

#include <stdint.h>

#include <hip/hip_runtime.h>

namespace hg {
namespace adamw {

constexpr int kThreads = 256;
constexpr int kMost = 48;                 // tensors of a launch: their descriptions travel as its arguments (4 KiB)

// Types as in the public headers, kNone for a master that is not there.
struct Tensor {
    void *param;
    float *master;
    const void *grad;
    void *m;
    uint8_t *ms;
    void *v;
    uint8_t *vs;
    int64_t n;
    int32_t place;                        // in the caller's array
    int8_t param_type, grad_type, state8;
};
struct Batch {
    Tensor t[kMost];
    int32_t first[kMost];                 // the tensors' first pieces
    int32_t count, pieces, each;          // each: elements of a piece / (8·kThreads), 1 or 4
    float beta1, rest1, beta2, rest2, eps, decay, lr;     // rest: 1 - beta
    double log1, log2;                    // of the betas
    const float *factors;
    const int64_t *device_step;
    int64_t step;
    uint64_t seed;
};
static_assert(sizeof(Batch) <= 4096, "");
inline int64_t piece_of(int each) { return (int64_t)each * kThreads * 8; }
hipError_t launch(const Batch &b, hipStream_t s);

}  // namespace adamw
}  // namespace hg
