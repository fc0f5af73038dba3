// Internal interface of hg_adamw (include/hgemm_adamw.h): what the host passes to
// the kernel.
#pragma once

#include <stdint.h>

#include <hip/hip_runtime.h>

namespace hg {
namespace adamw {

constexpr int kThreads = 256;
// A launch's tensors travel as its arguments (4 KiB), each as the words that it
// has: weights, gradient, two moments, a word of numbers, [master], [two arrays of
// scales].  Up to 83 tensors with fp32 moments and weights, 59 with 8-bit moments.
constexpr int kMost = 83, kWords = 415;
constexpr int kFewest = 5;                // words of a tensor
// The word of numbers: elements (37 bits), place in the caller's array (20),
// types as in the public headers (2 each), whether there is a master, 8-bit moments.
constexpr int kPlace = 37, kParam = 57, kGrad = 59, kMaster = 61, kState8 = 62;

// Where a tensor begins: its first piece and word.  (Both of 32 bits: with words in
// an array of 16 the compiler addresses pieces by twice an address that is not a
// multiple of four, whose low bits a scalar load leaves out.)
struct Place {
    int32_t piece, word;
};
struct Batch {
    int32_t count, pieces, used, each;    // each: elements of a piece / (8·kThreads), 1 or 4
    float beta1, rest1, beta2, rest2, eps, decay, lr;     // rest: 1 - beta
    const float *factors;
    const int64_t *device_step;
    int64_t step;
    uint64_t seed;
    double log1, log2;                    // of the betas
    Place place[kMost];
    void *words[kWords];
};
static_assert(sizeof(Batch) <= 4096, "");
inline int64_t piece_of(int each) { return (int64_t)each * kThreads * 8; }
hipError_t launch(const Batch &b, hipStream_t s);

}  // namespace adamw
}  // namespace hg
