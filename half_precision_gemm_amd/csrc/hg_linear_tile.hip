// hg_linear_tile.hip — the products of the linear layer and of its gradient
// on 256×256 tiles (gfx950): C(i, j) = Σ_k A(i, k)·B(j, k), each operand
// k-contiguous or k-major (hg_linear.h), for products with at least as many
// tiles as the GPU has compute units.
//
//  * One workgroup = 4 waves (2×2, one per SIMD), 128×128 = 8×8 blocks of
//    v_mfma_f32_16x16x32 each: 256 fp32 accumulators per lane (AGPRs), 64
//    flops per byte read from LDS.
//  * 64-wide stages, 3 slots of A and 2 of B (32 KiB each, all of the LDS),
//    one barrier per stage.  A stage is four quarters of 32 matrix
//    instructions (k-step × half of the A blocks); fragment reads run a
//    quarter (A) or a k-step (B) ahead and loads two stages ahead, one of
//    either every few matrix instructions, at compile-time positions: with one
//    wave per SIMD, bursts would hold back the matrix core.
//  * Persistent: a workgroup walks a strided list of tiles and requests the
//    next tile's first two stages before it finishes the current one, so the
//    epilogue's arithmetic and stores run over those loads.
//  * Epilogue: a wave passes its results 16 rows at a time through 8 KiB of
//    LDS (the A slot that the next tile's first loads leave idle) into lanes
//    that hold eight consecutive columns: whole lines per store, one bias
//    vector per lane and tile, and the block of 32 columns of an 8-bit save in
//    four neighbouring lanes.  The loop over the row blocks is a real loop
//    (only the writes to LDS are unrolled), because the epilogue with its
//    activations is long and would not fit the instruction cache eight times.
#include "hg_linear.h"

extern "C" __device__ void hg_lin_tile_load_lds(hg::lin::i32x4 rsrc, hg::lin::lds_u32 *lds, int size, int voffset,
                                                int soffset, int offset,
                                                int aux) __asm("llvm.amdgcn.raw.buffer.load.lds");

namespace hg {
namespace lin {
namespace {

constexpr int EDGE = 256, THREADS = 256;
constexpr int NSA = 3, NSB = 2;                     // slots of A and B
constexpr int WT = 128, T = WT / 16;                // wave sub-tile, its 16×16 blocks
constexpr int TQ = T / 2, PQ = TQ * T;              // A blocks and matrix instructions per quarter
constexpr int SLOT = EDGE * kStage * 2;
constexpr int LDS_B = NSA * SLOT, LDS_BYTES = (NSA + NSB) * SLOT;
constexpr int L = Side<EDGE, false>::L;             // loads per wave, operand and stage
static_assert(Side<EDGE, true>::L == L && L == 8 && LDS_BYTES <= 160 * 1024 && 4 * 16 * WT * 4 <= SLOT, "");

// What follows matrix instruction k of quarter q: RA + i reads A block i of
// the next quarter, RB + i the quarter's i-th B block of the next k-step, LD +
// i is ring load i (quarters 0 and 1: A of stage kt+2, whose slot the previous
// stage's barrier freed; 2, after the barrier, and 3: B of stage kt+2, whose
// slot this stage's barrier frees).  The barrier is in front of instruction
// BAR of quarter 2: after every read of stage kt, before every read of kt+1.
constexpr int NONE = 0, RA = 1, RB = 8, LD = 16, BAR = 13;
__device__ __forceinline__ constexpr int sched(int q, int k)
{
    if (q == 2) {
        if (k <= 9 && k % 3 == 0)
            return RA + k / 3;
        if (k >= 16 && k % 4 == 0)
            return RB + (k - 16) / 4;
        if (k >= 14 && k <= 26 && k % 4 == 2)
            return LD + (k - 14) / 4;
        return NONE;
    }
    if (k % 4 == 0)
        return k < 16 ? RA + k / 4 : RB + (k - 16) / 4;
    return k % 8 == 2 ? LD + k / 8 : NONE;
}

// One row block of accumulators into a wave's staging area (an LDS address),
// straight from the accumulation registers.  As ordinary stores in a loop over
// the blocks, the compiler copies accumulators to vector registers ahead of
// the loop and spills; unrolled, the epilogue's code is there eight times.
// (The stores' completion is not the compiler's to track: a wave's LDS
// accesses execute in order, so the reads that follow them need no wait; the
// barrier before the next tile does.)
__device__ __forceinline__ void put(const floatx4 (&blk)[T], uint32_t stg, int lane)
{
#pragma unroll
    for (int j = 0; j < T; ++j)
        __asm__ volatile("ds_write_b128 %0, %1"
                         :
                         : "v"(stg + stage_at<WT>(lane & 15, 4 * j + (lane >> 4))), "a"(blk[j])
                         : "memory");
}

template <bool TA, bool TB, bool KCHK, bool BF16>
__global__ void __launch_bounds__(THREADS, 1) linear_tile_kernel(const Product p, const Spread w)
{
    __shared__ __attribute__((aligned(1024))) unsigned char smem[LDS_BYTES];
    int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int wm = wave >> 1, wn = wave & 1;
    const uint32_t lds_base = (uint32_t)reinterpret_cast<uintptr_t>(smem);

    Panel<EDGE, TA, KCHK> pa;
    Panel<EDGE, TB, KCHK> pb;
    auto load = [](i32x4 r, lds_u32 *dst, int o) __attribute__((always_inline)) {
        hg_lin_tile_load_lds(r, dst, 16, o, 0, 0, 0);
    };
    auto issue_a = [&](const Item &t, int kt, int slot, int i) __attribute__((always_inline)) {
        pa.issue(load, kt, kt < t.nk, lds_base + slot * SLOT, i, wave, lane);
    };
    auto issue_b = [&](const Item &t, int kt, int slot, int i) __attribute__((always_inline)) {
        pb.issue(load, kt, kt < t.nk, lds_base + LDS_B + slot * SLOT, i, wave, lane);
    };
    // Stages 0 and 1 of a tile (the K loop issues the rest).
    auto begin = [&](const Item &t) __attribute__((always_inline)) {
        pa.set(p.A, p.lda, t.m0, p.M, p.K, t.kt0, wave, lane);
        pb.set(p.B, p.ldb, t.n0, p.N, p.K, t.kt0, wave, lane);
#pragma unroll
        for (int st = 0; st < 2; ++st) {
#pragma unroll
            for (int i = 0; i < L; ++i)
                issue_a(t, st, st, i);
#pragma unroll
            for (int i = 0; i < L; ++i)
                issue_b(t, st, st, i);
        }
    };
    auto read_a = [&](int slot, int s, int blk) __attribute__((always_inline)) {
        return fragment<EDGE, TA>(smem + slot * SLOT, lane, wm * WT + blk * 16, s);
    };
    auto read_b = [&](int slot, int s, int blk) __attribute__((always_inline)) {
        return fragment<EDGE, TB>(smem + LDS_B + slot * SLOT, lane, wn * WT + blk * 16, s);
    };

    floatx4 acc[T][T];
    half8 fa[2][TQ], fb[2][T];         // A: by quarter parity; B: by k-step
    int id = blockIdx.x;
    Item t = item_at<EDGE>(p, w, id);
    begin(t);
    // An interior epilogue issues at least one store in each of its 32 passes
    // after the next tile's 4·L first loads, and the counter retires in order:
    // with 2·L + 32 operations outstanding stage 0 has landed.
    constexpr int AFTER_FIRST = 2 * L, AFTER_EPILOGUE = 2 * L + 32;
    static_assert(AFTER_EPILOGUE <= 63, "");
    int prev = 0;                      // 0: first tile, 1: after an interior epilogue, 2: after an edge one
    for (;;) {
        // values derived from the lane index are recomputed per tile, not kept
        // in registers across the epilogue
        __asm__ volatile("" : "+v"(lane));
        if (prev == 0)
            wait_vmcnt<AFTER_FIRST>();
        else if (prev == 1)
            wait_vmcnt<AFTER_EPILOGUE>();
        else
            wait_vmcnt<0>();
        // The writes of put() are in as well: a wave whose part of the last tile
        // was outside the matrix read none of them back, and behind the barrier
        // the others load stage 2 into the same slot.
        wait_lgkmcnt<0>();
        __builtin_amdgcn_s_barrier();
        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int f = 0; f < TQ; ++f)
            fa[0][f] = read_a(0, 0, f);
#pragma unroll
        for (int j = 0; j < T; ++j)
            fb[0][j] = read_b(0, 0, j);
        wait_lgkmcnt<0>();
#pragma unroll
        for (int i = 0; i < T; ++i)
#pragma unroll
            for (int j = 0; j < T; ++j)
                acc[i][j] = floatx4{0, 0, 0, 0};
        int as = 0, bs = 0;
        for (int kt = 0; kt < t.nk; ++kt) {
            const int an = as == NSA - 1 ? 0 : as + 1, a2 = an == NSA - 1 ? 0 : an + 1, bn = bs ^ 1;
            static_for<4>([&](auto qc) __attribute__((always_inline)) {
                constexpr int q = decltype(qc)::value;
                constexpr int s = q >> 1, h = q & 1;
                constexpr int tq = (q + 1) & 3, ra_set = tq & 1, ra_step = tq >> 1, rb_step = q < 2 ? 1 : 0;
                const int ra_slot = q == 3 ? an : as, rb_slot = q < 2 ? bs : bn;
                static_for<PQ>([&](auto kc) __attribute__((always_inline)) {
                    constexpr int k = decltype(kc)::value;
                    if constexpr (q == 2 && k == BAR) {
                        // this wave's loads of stage kt+1 have landed (A of
                        // kt+2 may be in flight), its reads of kt are done
                        wait_vmcnt<L>();
                        wait_lgkmcnt<0>();
                        __builtin_amdgcn_s_barrier();
                        __builtin_amdgcn_sched_barrier(0);
                    }
                    // A blocks in snake order: consecutive instructions share
                    // an operand, which draws less power
                    constexpr int j = k / TQ, a = (j & 1) ? TQ - 1 - k % TQ : k % TQ;
                    acc[h * TQ + a][j] = mfma_16x16x32<BF16>(fb[s][j], fa[h][a], acc[h * TQ + a][j]);
                    constexpr int op = sched(q, k);
                    if constexpr (op >= LD) {
                        if constexpr (q < 2)
                            issue_a(t, kt + 2, a2, h * (L / 2) + op - LD);
                        else
                            issue_b(t, kt + 2, bs, h * (L / 2) + op - LD);
                    } else if constexpr (op >= RB) {
                        constexpr int jb = h * (T / 2) + op - RB;
                        fb[rb_step][jb] = read_b(rb_slot, rb_step, jb);
                    } else if constexpr (op >= RA) {
                        fa[ra_set][op - RA] = read_a(ra_slot, ra_step, ra_set * TQ + op - RA);
                    }
                    __builtin_amdgcn_sched_barrier(0);
                });
            });
            as = an;
            bs = bn;
        }
        // the ring's last loads (zero fills) and everyone's reads are done:
        // the slots are free
        wait_vmcnt<0>();
        wait_lgkmcnt<0>();
        __builtin_amdgcn_s_barrier();
        __builtin_amdgcn_sched_barrier(0);

        // the matrix core's last results are in their registers (the stores of
        // put() are not seen by the compiler's check for that)
        __asm__ volatile("s_nop 15\n\ts_nop 15");

        const int row0 = t.m0 + wm * WT;
        const int stg = 2 * SLOT + wave * (16 * WT * 4);
        prev = t.m0 + EDGE <= p.M && t.n0 + EDGE <= p.N ? 1 : 2;
        Drain<EDGE, WT, BF16> out(p, t, smem + stg, lane, t.n0 + wn * WT);
        out.request(row0);
        __builtin_amdgcn_sched_barrier(0);
        id += gridDim.x;
        const bool more = id < w.items;
        if (more) {
            t = item_at<EDGE>(p, w, id);
            begin(t);
        }
        __builtin_amdgcn_sched_barrier(0);
        settle(out.bias);
#pragma clang loop unroll(disable)
        for (int i = 0; i < T; ++i) {
            static_for<T>([&](auto ic) __attribute__((always_inline)) {
                constexpr int b = decltype(ic)::value;
                if (i == b)
                    put(acc[b], lds_base + stg, lane);
            });
            __atomic_signal_fence(__ATOMIC_SEQ_CST);
            out.block(row0 + 16 * i, i == T - 1);
            __atomic_signal_fence(__ATOMIC_SEQ_CST);
        }
        if (!more)
            break;
    }
}

template <bool TA, bool TB, bool BF16>
hipError_t launch(const Product &p, hipStream_t s)
{
    const int tiles_m = (int)(((int64_t)p.M + EDGE - 1) / EDGE), tiles_n = (p.N + EDGE - 1) / EDGE;
    const int64_t total = p.whole + ((int64_t)tiles_m * tiles_n - p.whole) * p.splits;
    if (total <= 0)
        return hipSuccess;
    if (total > 0x7fffffff - 4096)
        return hipErrorInvalidConfiguration;
    const Spread w{tiles_m, tiles_n, (int)total};
    // one workgroup per CU, a multiple of 8 so that a workgroup's tiles stay on its XCD
    int64_t grid = cu_count();
    grid = grid / 8 * 8 > 0 ? grid / 8 * 8 : grid;
    if (grid > total)
        grid = total;
    return start(!(TA && TB) && p.K % kStage != 0 ? linear_tile_kernel<TA, TB, !(TA && TB), BF16>
                                                  : linear_tile_kernel<TA, TB, false, BF16>,
                 grid, THREADS, s, p, w);
}

}  // namespace

hipError_t launch_tile(const Product &p, Layout l, bool bf16, hipStream_t s)
{
    switch (l) {
    case Layout::NN: return bf16 ? launch<false, false, true>(p, s) : launch<false, false, false>(p, s);
    case Layout::NT: return bf16 ? launch<false, true, true>(p, s) : launch<false, true, false>(p, s);
    default: return bf16 ? launch<true, true, true>(p, s) : launch<true, true, false>(p, s);
    }
}

}  // namespace lin
}  // namespace hg
