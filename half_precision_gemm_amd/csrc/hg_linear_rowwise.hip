// hg_linear_rowwise.hip — the linear layer's forward product for few rows
// (tokens that are generated one at a time, small batches): M <= 64 rows of X
// against an N×K weight (gfx950).
//
// Such a product is the reading of W once: 2·M flops per byte against the 200
// and more that the matrix cores could do, so what counts is bytes in flight
// on every CU from the first cycle on.
//
//  * A workgroup of 8 waves takes 16 (or 32) rows of W; its waves take turns
//    at 128-byte pieces of them (64 k), so the sum is split eight ways inside
//    the workgroup and N/16 workgroups fill the GPU at ordinary widths.
//  * W goes from memory straight to registers in the matrix core's operand
//    layout (lane l: row l mod 16, 8 k from 8·(l div 16) on: one 16-byte load),
//    X likewise from L2; nothing is staged, there is no barrier in the loop,
//    and a wave has DEPTH pieces in flight while it multiplies DEPTH others.
//  * Rows past M or N are read as the last row and their results dropped.
//  * The eight partial sums are added in LDS in a fixed order, eight columns to
//    a thread, and finished there: one launch in all.
//  * Operands need no alignment: global memory takes 16-byte loads at any even
//    address, so a weight with odd rows is not copied first; a last piece of
//    less than 64 k is loaded element by element.
#include "hg_linear.h"

namespace hg {
namespace lin {
namespace {

constexpr int WAVES = 8, THREADS = WAVES * 64, PIECE = 64;

// NB blocks of 16 rows of W, MB blocks of 16 rows of X.
template <int NB, int MB, bool BF16>
__global__ void __launch_bounds__(THREADS, 1) linear_rowwise_kernel(const Product p)
{
    constexpr int DEPTH = NB * 2 + MB * 2 <= 4 ? 4 : NB * 2 + MB * 2 <= 8 ? 2 : 1;
    __shared__ __attribute__((aligned(16))) float part[WAVES][MB * 16][NB * 16];
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int frow = lane & 15, fhi = lane >> 4;
    const int n0 = blockIdx.x * (NB * 16), K = p.K;
    const uint16_t *w[NB], *x[MB];
#pragma unroll
    for (int b = 0; b < NB; ++b)
        w[b] = p.B + (int64_t)min(n0 + 16 * b + frow, p.N - 1) * p.ldb;
#pragma unroll
    for (int b = 0; b < MB; ++b)
        x[b] = p.A + (int64_t)min(16 * b + frow, p.M - 1) * p.lda;

    floatx4 acc[MB][NB];
#pragma unroll
    for (int i = 0; i < MB; ++i)
#pragma unroll
        for (int j = 0; j < NB; ++j)
            acc[i][j] = floatx4{0, 0, 0, 0};
    struct Piece {
        half8 w[NB][2], x[MB][2];
    };
    auto load = [&](int piece, Piece &q) __attribute__((always_inline)) {
        const int k = piece * PIECE + 8 * fhi;
#pragma unroll
        for (int s = 0; s < 2; ++s) {
#pragma unroll
            for (int b = 0; b < NB; ++b)
                q.w[b][s] = __builtin_bit_cast(half8, *reinterpret_cast<const u32x4_any *>(w[b] + k + 32 * s));
#pragma unroll
            for (int b = 0; b < MB; ++b)
                q.x[b][s] = __builtin_bit_cast(half8, *reinterpret_cast<const u32x4_any *>(x[b] + k + 32 * s));
        }
    };
    auto multiply = [&](const Piece &q) __attribute__((always_inline)) {
#pragma unroll
        for (int s = 0; s < 2; ++s)
#pragma unroll
            for (int i = 0; i < MB; ++i)
#pragma unroll
                for (int j = 0; j < NB; ++j)
                    acc[i][j] = mfma_16x16x32<BF16>(q.w[j][s], q.x[i][s], acc[i][j]);
    };
    // This wave's whole pieces: wave, wave + 8, ..; groups of DEPTH, the next
    // group's loads in flight over this one's products.  Each workgroup begins
    // at a turn of its own and wraps around: side by side at the same column of
    // every row, workgroups ask the same memory channels (16×4096×16384 39.1 ->
    // 33.5 us, 1×4096×16448 37.9 -> 29.0).  The order of a sum depends on its
    // column's place alone.
    const int whole = K / PIECE, mine = whole > wave ? (whole - wave + WAVES - 1) / WAVES : 0;
    const int turns = whole / WAVES;                              // that all waves take part in
    int left = mine, turn = turns > 0 ? (int)(blockIdx.x * 5u % (unsigned)turns) : 0, done = 0;
    auto next = [&]() __attribute__((always_inline)) {
        const int at = done < turns ? turn * WAVES + wave : done * WAVES + wave;
        ++done;
        turn = turn + 1 == turns ? 0 : turn + 1;
        return at;
    };
    Piece a[DEPTH], b[DEPTH];
    auto group = [&](Piece (&g)[DEPTH]) __attribute__((always_inline)) {
#pragma unroll
        for (int d = 0; d < DEPTH; ++d)
            load(next(), g[d]);
    };
    auto use = [&](const Piece (&g)[DEPTH]) __attribute__((always_inline)) {
#pragma unroll
        for (int d = 0; d < DEPTH; ++d)
            multiply(g[d]);
        left -= DEPTH;
    };
    if (left >= DEPTH) {
        group(a);
        while (left >= 3 * DEPTH) {
            group(b);
            use(a);
            group(a);
            use(b);
        }
        if (left >= 2 * DEPTH) {
            group(b);
            use(a);
            use(b);
        } else {
            use(a);
        }
    }
    for (; left > 0; --left) {
        Piece q;
        load(next(), q);
        multiply(q);
    }
    // The rest of the sum, by the wave whose turn it is.
    if (K % PIECE != 0 && whole % WAVES == wave) {
        Piece q;
        const int k = whole * PIECE + 8 * fhi;
#pragma unroll
        for (int s = 0; s < 2; ++s) {
#pragma unroll
            for (int j = 0; j < NB; ++j)
                q.w[j][s] = __builtin_bit_cast(half8, load16x8(w[j] + k + 32 * s, K - k - 32 * s));
#pragma unroll
            for (int i = 0; i < MB; ++i)
                q.x[i][s] = __builtin_bit_cast(half8, load16x8(x[i] + k + 32 * s, K - k - 32 * s));
        }
        multiply(q);
    }
    // A lane holds columns 4·(lane div 16) .. +3 of row lane mod 16 of each block.
#pragma unroll
    for (int i = 0; i < MB; ++i)
#pragma unroll
        for (int j = 0; j < NB; ++j)
            *reinterpret_cast<floatx4 *>(&part[wave][16 * i + frow][16 * j + 4 * fhi]) = acc[i][j];
    __syncthreads();
    constexpr int UNITS = NB * 2;                                 // groups of eight columns per row
    if (threadIdx.x >= MB * 16 * UNITS)
        return;                                                   // whole waves (NB = 1: no 8-bit save)
    const int row = threadIdx.x / UNITS, c = threadIdx.x % UNITS * 8;
    float v[8] = {0, 0, 0, 0, 0, 0, 0, 0}, bias[8];
#pragma unroll
    for (int g = 0; g < WAVES; ++g)
#pragma unroll
        for (int e = 0; e < 8; ++e)
            v[e] += part[g][row][c + e];
    load_bias(p.f, n0 + c, bias);
    finish8<BF16>(p.f, row, n0 + c, v, bias);
}

template <int NB, bool BF16>
hipError_t launch(const Product &p, hipStream_t s)
{
    const dim3 grid((unsigned)((p.N + 16 * NB - 1) / (16 * NB)));
    if (p.M <= 16)
        hipLaunchKernelGGL((linear_rowwise_kernel<NB, 1, BF16>), grid, dim3(THREADS), 0, s, p);
    else if (p.M <= 32)
        hipLaunchKernelGGL((linear_rowwise_kernel<NB, 2, BF16>), grid, dim3(THREADS), 0, s, p);
    else
        hipLaunchKernelGGL((linear_rowwise_kernel<NB, 4, BF16>), grid, dim3(THREADS), 0, s, p);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_rowwise(const Product &p, bool bf16, hipStream_t s)
{
    // 32 rows of W per workgroup where that still gives every CU one, and for
    // an 8-bit save, whose blocks of 32 columns stay in one workgroup.
    const bool two = p.f.save == kSave8 || (p.N + 31) / 32 >= cu_count();
    if (two)
        return bf16 ? launch<2, true>(p, s) : launch<2, false>(p, s);
    return bf16 ? launch<1, true>(p, s) : launch<1, false>(p, s);
}

}  // namespace lin
}  // namespace hg
