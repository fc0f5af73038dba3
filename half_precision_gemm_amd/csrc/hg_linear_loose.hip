// hg_linear_loose.hip — the linear layer's forward product on 64×64 tiles with
// operands at any address and of any row length (gfx950).
//
// Direct buffer→LDS loads want 16-byte pieces that end with their row, so an
// operand with odd rows is otherwise copied to aligned ones first, by a launch
// of its own.  Here the pieces pass through registers, as 16-byte loads that
// global memory takes at any even address: the saved launch is worth more than
// the slower loop (333×1111×777 12.4 -> 9.2 us, 1000×1000×4001 32.4 -> 28.8).
//
//  * One workgroup of 4 waves (2×2) per tile, 64-wide stages: a thread moves
//    two 16-byte pieces of either operand, eight neighbours 128 bytes of a row.
//    DEPTH stages are in flight in registers, the compiler's own counting waits
//    for the oldest only; two LDS slots, one barrier per stage.
//    (Rows at odd elements loaded as aligned words and shifted, as the forms for
//    few rows do: 333×1111×777 9.3 -> 11.4 us, not here.)
//  * Rows past the last are read as the last row and their results dropped.
//  * The end of the sum that is no whole stage comes first: its loads are in
//    flight together with the first whole stages'.
#include "hg_linear.h"

namespace hg {
namespace lin {
namespace {

constexpr int EDGE = 64, THREADS = 256, DEPTH = 4;

template <bool BF16>
__global__ void __launch_bounds__(THREADS, 2) linear_loose_kernel(const Product p, const Spread w)
{
    using S = Side<EDGE, false>;
    constexpr int WT = EDGE / 2, T = WT / 16, SLOT = 2 * S::BYTES;
    __shared__ __attribute__((aligned(1024))) unsigned char smem[2 * SLOT];
    static_assert(4 * 16 * WT * 4 <= 2 * SLOT, "");
    const Item t = item_at<EDGE>(p, w, blockIdx.x);
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int wm = wave >> 1, wn = wave & 1;
    const int k0 = t.kt0 * kStage, left = p.K - k0;               // of this slice's sum
    const int full = min(t.nk, left / kStage);                    // its whole stages

    // Pieces i: rows tid / 8 + 32·i, chunk tid mod 8.
    const int r0 = threadIdx.x >> 3, c = threadIdx.x & 7;
    const uint16_t *src[2][2];
    uint32_t dst[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const int r = r0 + 32 * i;
        src[0][i] = p.A + (int64_t)min(t.m0 + r, p.M - 1) * p.lda + k0 + 8 * c;
        src[1][i] = p.B + (int64_t)min(t.n0 + r, p.N - 1) * p.ldb + k0 + 8 * c;
        dst[i] = r * S::RB + ((c ^ S::swz(r)) * 16);
    }
    struct Stage {
        u32x4 v[2][2];
    };
    auto load = [&](int kt, Stage &s) __attribute__((always_inline)) {
        const int at = min(kt, full - 1) * kStage;                // past the last: it again, not used
#pragma unroll
        for (int o = 0; o < 2; ++o)
#pragma unroll
            for (int i = 0; i < 2; ++i)
                s.v[o][i] = *reinterpret_cast<const u32x4_any *>(src[o][i] + at);
    };
    auto put = [&](int slot, const Stage &s) __attribute__((always_inline)) {
#pragma unroll
        for (int o = 0; o < 2; ++o)
#pragma unroll
            for (int i = 0; i < 2; ++i)
                *reinterpret_cast<u32x4 *>(smem + slot * SLOT + o * S::BYTES + dst[i]) = s.v[o][i];
    };
    floatx4 acc[T][T];
#pragma unroll
    for (int i = 0; i < T; ++i)
#pragma unroll
        for (int j = 0; j < T; ++j)
            acc[i][j] = floatx4{0, 0, 0, 0};
    auto multiply = [&](int slot) __attribute__((always_inline)) {
        const unsigned char *at = smem + slot * SLOT;
#pragma unroll
        for (int s = 0; s < kStage / 32; ++s) {
            half8 a[T], b[T];
#pragma unroll
            for (int i = 0; i < T; ++i) {
                a[i] = fragment<EDGE, false>(at, lane, wm * WT + 16 * i, s);
                b[i] = fragment<EDGE, false>(at + S::BYTES, lane, wn * WT + 16 * i, s);
            }
#pragma unroll
            for (int i = 0; i < T; ++i)
#pragma unroll
                for (int j = 0; j < T; ++j)
                    acc[i][j] = mfma_16x16x32<BF16>(b[j], a[i], acc[i][j]);
        }
    };
    // Everyone's pieces of a stage are in LDS (and the other slot is read).
    auto meet = [&]() __attribute__((always_inline)) {
        __atomic_signal_fence(__ATOMIC_SEQ_CST);
        wait_lgkmcnt<0>();
        __builtin_amdgcn_s_barrier();
        __builtin_amdgcn_sched_barrier(0);
        __atomic_signal_fence(__ATOMIC_SEQ_CST);
    };
    Stage ring[DEPTH];
    int slot = 0;
    auto begin = [&]() __attribute__((always_inline)) {
        if (full > 0) {
#pragma unroll
            for (int d = 0; d < DEPTH; ++d)
                load(d, ring[d]);
        }
    };
    if (full < t.nk) {
        const int at = full * kStage, n = left - at - 8 * c;
        Stage e;
#pragma unroll
        for (int o = 0; o < 2; ++o)
#pragma unroll
            for (int i = 0; i < 2; ++i)
                e.v[o][i] = load16x8(src[o][i] + at, n);
        begin();
        put(slot, e);
        meet();
        multiply(slot);
        slot = 1;
    } else {
        begin();
    }
    for (int kt = 0; kt < full; kt += DEPTH) {
#pragma unroll
        for (int d = 0; d < DEPTH; ++d) {
            if (kt + d < full) {
                put(slot, ring[d]);
                load(kt + d + DEPTH, ring[d]);
                meet();
                multiply(slot);
                slot ^= 1;
            }
        }
    }
    meet();

    unsigned char *stg = smem + wave * (16 * WT * 4);
    const int row0 = t.m0 + wm * WT;
    Drain<EDGE, WT, BF16> out(p, t, stg, lane, t.n0 + wn * WT);
    out.request(row0);
    settle(out.bias);
#pragma unroll
    for (int i = 0; i < T; ++i) {
        stage_put<WT>(stg, lane, acc[i]);
        __atomic_signal_fence(__ATOMIC_SEQ_CST);
        out.block(row0 + 16 * i, i == T - 1);
        __atomic_signal_fence(__ATOMIC_SEQ_CST);
    }
}

}  // namespace

hipError_t launch_loose(const Product &p, bool bf16, hipStream_t s)
{
    const int64_t tm = ((int64_t)p.M + EDGE - 1) / EDGE, tn = ((int64_t)p.N + EDGE - 1) / EDGE;
    const int64_t total = p.whole + (tm * tn - p.whole) * p.splits;
    if (total <= 0)
        return hipSuccess;
    if (total > kMostBlocks)
        return hipErrorInvalidConfiguration;
    const Spread w{(int)tm, (int)tn, (int)total};
    return start(bf16 ? linear_loose_kernel<true> : linear_loose_kernel<false>, total, THREADS, s, p, w);
}

}  // namespace lin
}  // namespace hg
