// hg_linear_rowwise.hip — the linear layer's forward product for few rows
// (tokens that are generated one at a time, small batches): M <= 64 rows of X
// against an N×K weight (gfx950).
//
// Such a product is the reading of W once: 2·M flops per byte against the 200
// and more that the matrix cores could do, so what counts is bytes in flight
// on every CU from the first cycle on, and that they are spread over all of
// the memory's channels.
//
//  * A workgroup of 8 waves takes 16 (or 32) rows of W; its waves take turns
//    at pieces of them, so the sum is split eight ways inside the workgroup and
//    N/16 workgroups fill the GPU at ordinary widths.  The eight partial sums
//    are added in LDS in a fixed order, eight columns to a thread, and finished
//    there: one launch in all.
//  * Each workgroup begins at a place of its own in the sum and wraps around:
//    side by side at the same column of every row, workgroups ask the same
//    memory channels (16×4096×16384 39.1 -> 33.5 us, 1×4096×16448 37.9 ->
//    29.0).  The order of a sum depends on its column's place alone.
//  * Operands that direct loads take go through LDS (linear_stream_kernel),
//    others straight into registers (linear_rowwise_kernel).
#include "hg_linear.h"

extern "C" __device__ void hg_lin_row_load_lds(hg::lin::i32x4 rsrc, hg::lin::lds_u32 *lds, int size, int voffset,
                                               int soffset, int offset,
                                               int aux) __asm("llvm.amdgcn.raw.buffer.load.lds");

namespace hg {
namespace lin {
namespace {

constexpr int WAVES = 8, THREADS = WAVES * 64, PIECE = 64;

// The eight waves' sums, added through LDS and finished.  NB blocks of 16 rows
// of W, MB blocks of 16 rows of X.
template <int NB, int MB, bool BF16>
__device__ __forceinline__ void finish_sums(const Product &p, float (*part)[MB * 16][NB * 16],
                                            const floatx4 (&acc)[MB][NB], int n0, int wave, int lane)
{
    const int frow = lane & 15, fhi = lane >> 4;
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

// NB blocks of 16 rows of W, MB blocks of 16 rows of X, at any address (ODD: odd
// elements too) and of any length.  W goes from memory straight to registers in the matrix core's
// operand layout (lane l: row l mod 16, 8 k from 8·(l div 16) on: one 16-byte
// load, which global memory takes at any even address), X likewise from L2;
// nothing is staged, there is no barrier in the loop, and a wave has DEPTH
// pieces in flight while it multiplies DEPTH others.  Rows past M or N are
// read as the last row and their results dropped; a last piece of less than 64
// k is loaded element by element (requested before the others, or as the row's
// last eight with those before masked: no gain).
template <int NB, int MB, bool ODD>
struct Pieces {
    Raw<ODD> w[NB][2], x[MB][2];
};
template <int NB, int MB, bool ODD, bool BF16>
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
    using Piece = Pieces<NB, MB, ODD>;
    auto load = [&](int piece, Piece &q) __attribute__((always_inline)) {
        const int k = piece * PIECE + 8 * fhi;
#pragma unroll
        for (int s = 0; s < 2; ++s) {
#pragma unroll
            for (int b = 0; b < NB; ++b)
                q.w[b][s].load(w[b] + k + 32 * s);
#pragma unroll
            for (int b = 0; b < MB; ++b)
                q.x[b][s].load(x[b] + k + 32 * s);
        }
    };
    auto multiply = [&](const auto &q) __attribute__((always_inline)) {
#pragma unroll
        for (int s = 0; s < 2; ++s)
#pragma unroll
            for (int i = 0; i < MB; ++i)
#pragma unroll
                for (int j = 0; j < NB; ++j)
                    acc[i][j] = mfma_16x16x32<BF16>(__builtin_bit_cast(half8, q.w[j][s].get(w[j])),
                                                    __builtin_bit_cast(half8, q.x[i][s].get(x[i])), acc[i][j]);
    };
    // This wave's whole pieces: wave, wave + 8, ..; groups of DEPTH, the next
    // group's loads in flight over this one's products.
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
        __builtin_amdgcn_sched_barrier(0);                        // all of them before the products that follow
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
        Pieces<NB, MB, false> q;
        const int k = whole * PIECE + 8 * fhi;
#pragma unroll
        for (int s = 0; s < 2; ++s) {
#pragma unroll
            for (int j = 0; j < NB; ++j)
                q.w[j][s].w = load16x8(w[j] + k + 32 * s, K - k - 32 * s);
#pragma unroll
            for (int i = 0; i < MB; ++i)
                q.x[i][s].w = load16x8(x[i] + k + 32 * s, K - k - 32 * s);
        }
        multiply(q);
    }
    finish_sums<NB, MB, BF16>(p, part, acc, n0, wave, lane);
}

// The same for operands that direct loads take (Product): W and X through a
// ring of LDS slots.  A load instruction fetches 512 bytes of two rows, where
// the kernel above asks for 64 bytes of 16 rows, and lanes past the last row
// fetch nothing.  A stage is 256 k, 32 for each wave.  Rings of at most 80 KiB
// where X is short, so that two workgroups share a CU and one's first loads
// run over the other's end: weights out of HBM, us, kernel above / one
// workgroup per CU / two: 1×16384×4096 29.4 / 27.6 / 24.9, 16×4096×16384 37.2 /
// 29.3 / 28.0, 1×50264×2048 45.0 / 50.5 / 39.7; 1×50264×512 15.6 / - / 20.2,
// so a sum of less than eight stages stays above with NB = 2.
constexpr int SK = 256;                                           // k per stage
template <int NB, int MB>
constexpr int kStreamSlot = 16 * (NB + MB) * SK * 2;
template <int NB, int MB>
constexpr int kStreamSlots = (NB * MB <= 2 ? 80 : 160) * 1024 / kStreamSlot<NB, MB>;

template <int NB, int MB, bool BF16>
__global__ void __launch_bounds__(THREADS, 1) linear_stream_kernel(const Product p)
{
    constexpr int NS = kStreamSlots<NB, MB>, SLOT = kStreamSlot<NB, MB>;
    constexpr int RB = SK * 2, CH = RB / 16, RPI = 64 / CH;       // bytes and chunks per row, rows per load
    constexpr int LW = NB, LX = MB, L = LW + LX;                  // loads per wave and stage
    constexpr int WBYTES = 16 * NB * RB;
    static_assert(SK == WAVES * 32 && LW * WAVES * RPI == 16 * NB && NS >= 3 && (NS - 2) * L <= 63 &&
                      WAVES * MB * NB * 1024 <= NS * SLOT,
                  "");
    __shared__ __attribute__((aligned(1024))) unsigned char smem[NS * SLOT];
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int frow = lane & 15, fhi = lane >> 4;
    const int n0 = blockIdx.x * (NB * 16), K = p.K;
    const uint32_t lds_base = (uint32_t)reinterpret_cast<uintptr_t>(smem);
    const int nk = (K + SK - 1) / SK;
    // The stage of the sum to load next.  The workgroups of one XCD (every
    // eighth) follow each other, because they share an L2 (16×4096×16384 30.6
    // -> 29.1 us against places 5 apart by workgroup; the kernel above 38.5 ->
    // 40.2).
    int at = (int)(((blockIdx.x >> 3) + (blockIdx.x & 7u) * (unsigned)nk / 8) % (unsigned)nk);

    const int wrows = min(p.N - n0, 16 * NB);
    const i32x4 rw = buffer_of(reinterpret_cast<uint64_t>(p.B) + (uint64_t)((int64_t)n0 * p.ldb) * 2,
                               (uint32_t)(wrows - 1) * (uint32_t)p.ldb * 2 + (uint32_t)K * 2);
    const i32x4 rx = buffer_of(reinterpret_cast<uint64_t>(p.A), (uint32_t)(p.M - 1) * (uint32_t)p.lda * 2 + (uint32_t)K * 2);
    uint32_t off[L];
    int ck[L];                                                    // first k of this lane's chunk
#pragma unroll
    for (int i = 0; i < L; ++i) {
        const bool w = i < LW;
        const int r = (wave * (w ? LW : LX) + (w ? i : i - LW)) * RPI + lane / CH;
        ck[i] = ((lane % CH) ^ (r & 15)) * 8;
        off[i] = r < (w ? wrows : p.M) ? (uint32_t)r * (uint32_t)(w ? p.ldb : p.lda) * 2 + ck[i] * 2 : kOutside;
    }
    auto issue = [&](int kt) __attribute__((always_inline)) {
        const uint32_t slot = lds_base + (kt % NS) * SLOT;
        const int k0 = at * SK;
        const bool in = kt < nk;
        at = at + 1 == nk ? 0 : at + 1;
#pragma unroll
        for (int i = 0; i < L; ++i) {
            const bool w = i < LW;
            const uint32_t o = in && ck[i] + k0 < K ? off[i] + (uint32_t)k0 * 2 : kOutside;
            const uint32_t to = slot + (w ? 0 : WBYTES) + (wave * (w ? LW : LX) + (w ? i : i - LW)) * 1024;
            hg_lin_row_load_lds(w ? rw : rx, reinterpret_cast<lds_u32 *>((uintptr_t)to), 16, (int)o, 0, 0, 0);
        }
    };
    floatx4 acc[MB][NB];
#pragma unroll
    for (int i = 0; i < MB; ++i)
#pragma unroll
        for (int j = 0; j < NB; ++j)
            acc[i][j] = floatx4{0, 0, 0, 0};
#pragma unroll
    for (int s = 0; s < NS - 1; ++s)
        issue(s);
    // Stage kt has landed, and every wave has read stage kt-1, whose slot takes
    // the stage NS-1 ahead.
    for (int kt = 0; kt < nk; ++kt) {
        wait_vmcnt<(NS - 2) * L>();
        __builtin_amdgcn_s_barrier();
        __builtin_amdgcn_sched_barrier(0);
        __atomic_signal_fence(__ATOMIC_SEQ_CST);
        const unsigned char *slot = smem + (kt % NS) * SLOT;
        const int c = ((wave * 4 + fhi) ^ frow) * 16;
        half8 w[NB], x[MB];
#pragma unroll
        for (int i = 0; i < MB; ++i)
            x[i] = *reinterpret_cast<const half8 *>(slot + WBYTES + (16 * i + frow) * RB + c);
#pragma unroll
        for (int j = 0; j < NB; ++j)
            w[j] = *reinterpret_cast<const half8 *>(slot + (16 * j + frow) * RB + c);
        issue(kt + NS - 1);
        wait_lgkmcnt<0>();
        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int i = 0; i < MB; ++i)
#pragma unroll
            for (int j = 0; j < NB; ++j)
                acc[i][j] = mfma_16x16x32<BF16>(w[j], x[i], acc[i][j]);
    }
    wait_vmcnt<0>();
    __builtin_amdgcn_s_barrier();
    __builtin_amdgcn_sched_barrier(0);
    __atomic_signal_fence(__ATOMIC_SEQ_CST);
    finish_sums<NB, MB, BF16>(p, reinterpret_cast<float(*)[MB * 16][NB * 16]>(smem), acc, n0, wave, lane);
}

template <int NB, int MB, bool BF16>
hipError_t launch(const Product &p, bool stream, bool odd, hipStream_t s)
{
    return start(stream ? linear_stream_kernel<NB, MB, BF16>
                 : odd  ? linear_rowwise_kernel<NB, MB, true, BF16>
                        : linear_rowwise_kernel<NB, MB, false, BF16>,
                 (p.N + 16 * NB - 1) / (16 * NB), THREADS, s, p);
}

template <int NB, bool BF16>
hipError_t launch(const Product &p, bool stream, bool odd, hipStream_t s)
{
    return p.M <= 16   ? launch<NB, 1, BF16>(p, stream, odd, s)
           : p.M <= 32 ? launch<NB, 2, BF16>(p, stream, odd, s)
                       : launch<NB, 4, BF16>(p, stream, odd, s);
}

}  // namespace

hipError_t launch_rowwise(const Product &p, bool direct, bool odd, bool bf16, hipStream_t s)
{
    const bool two = weight_blocks(p.N, p.f.save == kSave8) == 2;
    const bool stream = direct && (!two || p.K >= 8 * SK);
    if (two)
        return bf16 ? launch<2, true>(p, stream, odd, s) : launch<2, false>(p, stream, odd, s);
    return bf16 ? launch<1, true>(p, stream, odd, s) : launch<1, false>(p, stream, odd, s);
}

}  // namespace lin
}  // namespace hg
