// hg_linear_outer.hip — the weight's gradient for few rows (gfx950):
//
//   dW(n, k) = Σ_m dZ(m, n)·X(m, k),  at most 64 terms,
//
// which is the writing of dW: 2·64 flops per element against hundreds that the
// matrix cores could do.  As 64×64 tiles of one stage each, a workgroup spends
// most of its time waiting for its first and only loads.
//
//  * A workgroup of 4 waves (2×2) takes 64 rows of dW and walks along them, 128
//    columns at a time.  Its piece of dZ is read once into registers; X, which
//    every workgroup reads, comes from L2 through three LDS slots, two in flight
//    while the third is multiplied.  Both operands are k-major as they lie
//    (hg_linear.h).  A wave's 32×64 results per turn are what pays for a turn's
//    instructions (32×32: 8192×8192 with 8 rows 47 us, 32×64 39).
//  * The stores of two turns may be in flight as well: the counter of vector
//    memory operations retires in order, so the wait for a slot counts them.
//  * 72 KiB of LDS: two workgroups per CU.
#include "hg_linear.h"

extern "C" __device__ void hg_lin_outer_load_lds(hg::lin::i32x4 rsrc, hg::lin::lds_u32 *lds, int size, int voffset,
                                                 int soffset, int offset,
                                                 int aux) __asm("llvm.amdgcn.raw.buffer.load.lds");

namespace hg {
namespace lin {
namespace {

constexpr int ROWS = 64, COLS = 128, THREADS = 256, NS = 3;

template <bool BF16>
__global__ void __launch_bounds__(THREADS, 2) linear_outer_kernel(const Product p, int tiles_n, int group, int groups)
{
    using SA = Side<ROWS, true>;
    using SB = Side<COLS, true>;
    constexpr int WM = ROWS / 2, WN = COLS / 2, TM = WM / 16, TN = WN / 16, L = SB::L, STEPS = kStage / 32;
    constexpr int STG = 16 * WN * 4, STORES = TM * 2;            // 16×WN blocks take two stores each
    __shared__ __attribute__((aligned(1024))) unsigned char smem[SA::BYTES + NS * SB::BYTES + 4 * STG];
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int wm = wave >> 1, wn = wave & 1;
    const uint32_t lds_base = (uint32_t)reinterpret_cast<uintptr_t>(smem);
    const int m0 = blockIdx.x / groups * ROWS, n0 = blockIdx.x % groups * group * COLS;
    const int count = min(group, tiles_n - n0 / COLS);

    auto load = [](i32x4 r, lds_u32 *dst, int o) __attribute__((always_inline)) {
        hg_lin_outer_load_lds(r, dst, 16, o, 0, 0, 0);
    };
    Panel<ROWS, true, false> pa;
    pa.set(p.A, p.lda, m0, p.M, p.K, 0, wave, lane);
#pragma unroll
    for (int i = 0; i < SA::L; ++i)
        pa.issue(load, 0, true, lds_base, i, wave, lane);
    Panel<COLS, true, false> pb;
    // Strips begin at different places of their runs: side by side they would
    // write to the same memory channels (8×8192×8192 38.6 -> 30.5 us).
    const int rot = (int)((blockIdx.x / groups) * 5u % (unsigned)count);
    auto col = [&](int t) __attribute__((always_inline)) {
        return n0 + (t + rot >= count ? t + rot - count : t + rot) * COLS;
    };
    auto issue = [&](int t) __attribute__((always_inline)) {
        pb.set(p.B, p.ldb, t < count ? col(t) : 0, p.N, p.K, 0, wave, lane);
#pragma unroll
        for (int i = 0; i < L; ++i)
            pb.issue(load, 0, t < count, lds_base + SA::BYTES + t % NS * SB::BYTES, i, wave, lane);
    };
#pragma unroll
    for (int t = 0; t < NS - 1; ++t)
        issue(t);

    unsigned char *stg = smem + SA::BYTES + NS * SB::BYTES + wave * STG;
    const int row0 = m0 + wm * WM;
    const bool inner = m0 + ROWS <= p.M && n0 + count * COLS <= p.N;
    half8 a[STEPS][TM], b[STEPS][TN];
    for (int t = 0; t < count; ++t) {
        // After the loads of turn t come the next one's and, of a strip inside
        // the matrix, the stores of two turns.
        if (inner && t >= NS - 1)
            wait_vmcnt<(NS - 2) * L + (NS - 1) * STORES>();
        else
            wait_vmcnt<(NS - 2) * L>();
        __builtin_amdgcn_s_barrier();
        __builtin_amdgcn_sched_barrier(0);
        __atomic_signal_fence(__ATOMIC_SEQ_CST);
        if (t == 0) {
#pragma unroll
            for (int s = 0; s < STEPS; ++s)
#pragma unroll
                for (int i = 0; i < TM; ++i)
                    a[s][i] = fragment<ROWS, true>(smem, lane, wm * WM + 16 * i, s);
        }
        const unsigned char *slot = smem + SA::BYTES + t % NS * SB::BYTES;
#pragma unroll
        for (int s = 0; s < STEPS; ++s)
#pragma unroll
            for (int j = 0; j < TN; ++j)
                b[s][j] = fragment<COLS, true>(slot, lane, wn * WN + 16 * j, s);
        const Item at{m0, col(t), 0, 1, nullptr};
        Drain<ROWS, WN, BF16, true> out(p, at, stg, lane, at.n0 + wn * WN);
        out.request(row0);
        issue(t + NS - 1);
        wait_lgkmcnt<0>();
        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int i = 0; i < TM; ++i) {
            floatx4 acc[TN];
#pragma unroll
            for (int j = 0; j < TN; ++j) {
                acc[j] = floatx4{0, 0, 0, 0};
#pragma unroll
                for (int s = 0; s < STEPS; ++s)
                    acc[j] = mfma_16x16x32<BF16>(b[s][j], a[s][i], acc[j]);
            }
            stage_put<WN>(stg, lane, acc);
            __atomic_signal_fence(__ATOMIC_SEQ_CST);
            out.block(row0 + 16 * i, i == TM - 1);
            __atomic_signal_fence(__ATOMIC_SEQ_CST);
        }
    }
    // the last slots' zero fills are in before the LDS is given up
    wait_vmcnt<0>();
}

}  // namespace

hipError_t launch_outer(const Product &p, bool bf16, hipStream_t s)
{
    // Runs of tiles so long that the workgroups are in place together (8×8256×
    // 8192, dW alone: 516 workgroups on 512 places 55 us, 387 42; a quarter as
    // long 40, but 8×8192×8192 36.5 against 33.7 and 16×4096×4096 17.3 / 13.3).
    const int64_t tm = ((int64_t)p.M + ROWS - 1) / ROWS, tn = ((int64_t)p.N + COLS - 1) / COLS;
    const int64_t places = 2 * (int64_t)cu_count();
    const int64_t most = tm < places ? places / tm : 1, group = (tn + most - 1) / most;
    const int64_t groups = (tn + group - 1) / group, total = tm * groups;
    if (total <= 0)
        return hipSuccess;
    if (total > kMostBlocks)
        return hipErrorInvalidConfiguration;
    return start(bf16 ? linear_outer_kernel<true> : linear_outer_kernel<false>, total, THREADS, s, p, (int)tn, (int)group,
                 (int)groups);
}

}  // namespace lin
}  // namespace hg
