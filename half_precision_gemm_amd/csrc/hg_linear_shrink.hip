// hg_linear_shrink.hip — the first half of the low-rank adapters' product
// (gfx950): T = s_g·X·A_gᵀ, g the row's adapter, rank values a row, for the
// forward kernels that multiply it by B_g (hg_linear.h, Adapters).
//
// A row costs 2·rank flops per element of X it reads, so this is the reading of
// X and of the adapters in use.
//
//  * Few rows (shrink_rows_kernel): a workgroup per row and four values of T;
//    each row reads its adapter whatever the others' are, from L2 where they
//    share it.
//  * More: 16 rows of X and 16 to 64 of the rank per workgroup on the matrix
//    cores, the sum split over its eight waves; one turn for every adapter among
//    the 16 rows, of which each row keeps its own's.  Where rows are few enough to
//    leave CUs idle, several workgroups share a block's adapters (slots): most of
//    them end at once where prompts lie one after the other, and rows of different
//    adapters side by side are taken in parallel.
//    shrink_stream_kernel takes X and A through a ring in LDS, 512 bytes of a row
//    per load, shrink_tile_kernel straight into registers, at any address.
#include "hg_linear.h"

extern "C" __device__ void hg_lin_shrink_load_lds(hg::lin::i32x4 rsrc, hg::lin::lds_u32 *lds, int size, int voffset,
                                                  int soffset, int offset,
                                                  int aux) __asm("llvm.amdgcn.raw.buffer.load.lds");

namespace hg {
namespace lin {
namespace {

// Stores one row's value k of T.
template <bool BF16>
__device__ __forceinline__ void store_t(const Shrink &q, int64_t row, int k, float v)
{
    if (q.wide) {
        static_cast<float *>(q.T)[row * q.ldt + k] = v;
        return;
    }
    uint16_t *t = static_cast<uint16_t *>(q.T) + row * q.ldt + k;
    const uint16_t high = narrow<BF16>(v);
    const float rest = v - widen<BF16>(high);
    t[0] = high;
    // (of an infinity or NaN there is no rest)
    t[(q.rank + 7) / 8 * 8] = __builtin_fabsf(widen<BF16>(high)) < __builtin_inff() ? narrow<BF16>(rest) : (uint16_t)0;
}
// Zeros behind the rank, thread `t` of `n`.
__device__ __forceinline__ void store_zeros(const Shrink &q, int64_t row, int t, int n)
{
    const int up = (q.rank + 7) / 8 * 8;
    if (q.wide) {
        for (int k = q.rank + t; k < up; k += n)
            static_cast<float *>(q.T)[row * q.ldt + k] = 0.0f;
        return;
    }
    uint16_t *r = static_cast<uint16_t *>(q.T) + row * q.ldt;
    for (int k = q.rank + t; k < q.ldt; k += n)
        if (k < up || k >= up + q.rank)
            r[k] = 0;
}

constexpr int RT = 256, PER = 4;                                  // threads; values of a row per workgroup

template <bool BF16>
__global__ void __launch_bounds__(RT) shrink_rows_kernel(const Shrink q, int parts)
{
    __shared__ float sums[RT / 64][PER];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int64_t row = blockIdx.x / parts;
    const int r0 = blockIdx.x % parts * PER;
    const int64_t g = q.which[row];
    if (g < 0 || g >= q.count)
        return;
    const uint16_t *x = q.X + row * q.ldx, *a = q.A + g * q.stride;
    float v[PER] = {};
    for (int k = threadIdx.x * 8; k < q.K; k += RT * 8) {
        float xs[8], as[8];
        u32x4 w[PER];
#pragma unroll
        for (int i = 0; i < PER; ++i)
            w[i] = load16x8(a + min(r0 + i, q.rank - 1) * q.lda + k, q.K - k);
        load8<BF16>(x + k, q.K - k, xs);
#pragma unroll
        for (int i = 0; i < PER; ++i) {
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                as[e] = widen<BF16>((uint16_t)(w[i][e >> 1] >> (16 * (e & 1))));
                v[i] = __builtin_fmaf(as[e], xs[e], v[i]);
            }
        }
    }
#pragma unroll
    for (int i = 0; i < PER; ++i) {
#pragma unroll
        for (int d = 1; d < 64; d *= 2)
            v[i] += __shfl_xor(v[i], d);
        if (lane == 0)
            sums[wave][i] = v[i];
    }
    __syncthreads();
    if (threadIdx.x < PER && r0 + (int)threadIdx.x < q.rank) {
        float t = 0.0f;
#pragma unroll
        for (int w = 0; w < RT / 64; ++w)
            t += sums[w][threadIdx.x];
        store_t<BF16>(q, row, r0 + threadIdx.x, q.scales ? q.scales[g] * t : t);
    }
    if (r0 == 0)
        store_zeros(q, row, threadIdx.x, RT);
}

constexpr int TW = 8, TT = TW * 64;                               // waves and threads of a block's workgroup

// A workgroup's place: blocks of 16 rows, 16·RB of the rank, one of `slots` among
// the block's workgroups.
struct Place {
    int blocks, slots;
};
// f(adapter) for this workgroup's adapters of a block, in ascending order; `mine`:
// the adapter of the lane's row.
template <class F>
__device__ __forceinline__ void for_adapters(int mine, int slot, int slots, F &&f)
{
    int n = 0;
    for (int g = -1;; ++n) {
        g = least_of_rows(mine > g ? mine : 0x7fffffff);
        if (g == 0x7fffffff)
            return;
        if (n % slots == slot)
            f(g);
    }
}
// The waves' sums of a block's values of T, added in order and stored in the rows
// that have adapter g.
template <int RB, bool BF16>
__device__ __forceinline__ void end_turn(const Shrink &q, float (*part)[16][RB * 16], const floatx4 (&acc)[RB], int row0,
                                         int r0, int g, int wave, int lane)
{
    const int frow = lane & 15, fhi = lane >> 4;
    const Adapters who{q.which, nullptr, nullptr, 0, 0, 0, q.count, q.rank};
    // (a lane holds values 4·fhi .. +3 of 16 of row frow)
#pragma unroll
    for (int j = 0; j < RB; ++j)
        *reinterpret_cast<floatx4 *>(&part[wave][frow][16 * j + 4 * fhi]) = acc[j];
    __syncthreads();
    for (int i = threadIdx.x; i < 16 * RB * 16; i += TT) {
        const int r = i / (RB * 16), k = i % (RB * 16);
        float t = 0.0f;
#pragma unroll
        for (int w = 0; w < TW; ++w)
            t += part[w][r][k];
        if (r0 + k < q.rank && adapter_of(who, row0 + r, q.M) == g)
            store_t<BF16>(q, row0 + r, r0 + k, q.scales ? q.scales[g] * t : t);
    }
    __syncthreads();
}

template <int RB, bool BF16>
__global__ void __launch_bounds__(TT) shrink_tile_kernel(const Shrink q, const Place w)
{
    __shared__ __attribute__((aligned(16))) float part[TW][16][RB * 16];
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int frow = lane & 15, fhi = lane >> 4;
    const int r0 = blockIdx.y * (RB * 16);
    const Adapters who{q.which, nullptr, nullptr, 0, 0, 0, q.count, q.rank};
    for (int block = blockIdx.x; block < w.blocks; block += gridDim.x) {
        const int row0 = block * 16, mine = adapter_of(who, row0 + frow, q.M);
        const uint16_t *x = q.X + min(row0 + frow, q.M - 1) * q.ldx + 8 * fhi;
        for_adapters(mine, blockIdx.z, w.slots, [&](int g) __attribute__((always_inline)) {
            const uint16_t *a[RB];
#pragma unroll
            for (int j = 0; j < RB; ++j)
                a[j] = q.A + g * q.stride + min(r0 + 16 * j + frow, q.rank - 1) * q.lda + 8 * fhi;
            floatx4 acc[RB];
#pragma unroll
            for (int j = 0; j < RB; ++j)
                acc[j] = floatx4{0, 0, 0, 0};
            // 64 of the sum at a time, eight waves in turn; a last piece that is
            // not whole element by element
            constexpr int D = 2;
            const int whole = q.K / 64;
            auto step = [&](int piece, auto load) __attribute__((always_inline)) {
                half8 xs[2], as[2][RB];
#pragma unroll
                for (int s = 0; s < 2; ++s) {
                    const int k = piece * 64 + 32 * s;
                    xs[s] = __builtin_bit_cast(half8, load(x + k, q.K - k - 8 * fhi));
#pragma unroll
                    for (int j = 0; j < RB; ++j)
                        as[s][j] = __builtin_bit_cast(half8, load(a[j] + k, q.K - k - 8 * fhi));
                }
#pragma unroll
                for (int s = 0; s < 2; ++s)
#pragma unroll
                    for (int j = 0; j < RB; ++j)
                        acc[j] = mfma_16x16x32<BF16>(as[s][j], xs[s], acc[j]);
            };
            auto plain = [](const uint16_t *p, int) __attribute__((always_inline)) {
                const u32x4 v = *reinterpret_cast<const u32x4_any *>(p);
                return v;
            };
            int piece = wave;
            for (; piece + (D - 1) * TW < whole; piece += D * TW) {
#pragma unroll
                for (int d = 0; d < D; ++d)
                    step(piece + d * TW, plain);
            }
            for (; piece < whole; piece += TW)
                step(piece, plain);
            if (q.K % 64 != 0 && whole % TW == wave)
                step(whole, [](const uint16_t *p, int n) __attribute__((always_inline)) { return load16x8(p, n); });
            end_turn<RB, BF16>(q, part, acc, row0, r0, g, wave, lane);
        });
        if (blockIdx.y == 0 && blockIdx.z == 0)
            for (int r = wave; r < 16; r += TW)
                if (row0 + r < q.M)
                    store_zeros(q, row0 + r, lane, 64);
    }
}

// The same for operands that direct loads take (rows of whole 16-byte pieces at
// 16-byte addresses), as linear_stream_kernel of hg_linear_rowwise.hip: stages of
// 256 k, 32 for each wave, workgroups beginning at different places of the sum.
constexpr int SK = 256;                                           // k per stage
template <int RB>
constexpr int kShrinkSlot = 16 * (1 + RB) * SK * 2;
// Two workgroups to a CU, or, DEEP, one with all of its LDS: where there are no more
// than CUs, more of each one's stages in flight (87×64×15424, rank 63, with 16 of the
// rank in a workgroup instead of 64: 47 -> 32 us for the whole layer).
template <int RB, bool DEEP>
constexpr int kShrinkSlots = DEEP ? 10 : 80 * 1024 / kShrinkSlot<RB> < 3 ? 3 : 80 * 1024 / kShrinkSlot<RB>;

template <int RB, bool DEEP, bool BF16>
__global__ void __launch_bounds__(TT) shrink_stream_kernel(const Shrink q, const Place w)
{
    constexpr int NS = kShrinkSlots<RB, DEEP>, SLOT = kShrinkSlot<RB>;
    constexpr int ROW = SK * 2, CH = ROW / 16, RPI = 64 / CH, L = 1 + RB;     // bytes and chunks per row, rows per load
    static_assert(SK == TW * 32 && TW * RPI == 16 && NS >= 3 && (NS - 2) * L <= 63 && TW * RB * 1024 <= NS * SLOT, "");
    __shared__ __attribute__((aligned(1024))) unsigned char smem[NS * SLOT];
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int frow = lane & 15, fhi = lane >> 4, K = q.K;
    const int r0 = blockIdx.y * (RB * 16), ranks = min(q.rank - r0, RB * 16);
    const uint32_t lds_base = (uint32_t)reinterpret_cast<uintptr_t>(smem);
    const int nk = (K + SK - 1) / SK;
    const Adapters who{q.which, nullptr, nullptr, 0, 0, 0, q.count, q.rank};
    const int r = wave * RPI + lane / CH, ck = ((lane % CH) ^ (r & 15)) * 8;      // this lane's row of 16 and first k
    for (int block = blockIdx.x; block < w.blocks; block += gridDim.x) {
        const int row0 = block * 16, rows = min(q.M - row0, 16), mine = adapter_of(who, row0 + frow, q.M);
        const i32x4 rx = buffer_of(reinterpret_cast<uint64_t>(q.X) + (uint64_t)(row0 * q.ldx) * 2,
                                   (uint32_t)(rows - 1) * (uint32_t)q.ldx * 2 + (uint32_t)K * 2);
        const uint32_t ox = r < rows ? (uint32_t)r * (uint32_t)q.ldx * 2 + ck * 2 : kOutside;
        for_adapters(mine, blockIdx.z, w.slots, [&](int g) __attribute__((always_inline)) {
            const i32x4 ra = buffer_of(reinterpret_cast<uint64_t>(q.A) + (uint64_t)(g * q.stride + r0 * q.lda) * 2,
                                       (uint32_t)(ranks - 1) * (uint32_t)q.lda * 2 + (uint32_t)K * 2);
            int at = (int)(((block >> 3) + (block & 7) * (unsigned)nk / 8) % (unsigned)nk);
            auto issue = [&](int kt) __attribute__((always_inline)) {
                const uint32_t slot = lds_base + (kt % NS) * SLOT + wave * 1024;
                const int k0 = at * SK;
                const bool in = kt < nk && ck + k0 < K;
                at = at + 1 == nk ? 0 : at + 1;
                hg_lin_shrink_load_lds(rx, reinterpret_cast<lds_u32 *>((uintptr_t)slot), 16,
                                       (int)(in ? ox + (uint32_t)k0 * 2 : kOutside), 0, 0, 0);
#pragma unroll
                for (int j = 0; j < RB; ++j) {
                    const uint32_t o = (uint32_t)(16 * j + r) * (uint32_t)q.lda * 2 + ck * 2 + (uint32_t)k0 * 2;
                    hg_lin_shrink_load_lds(ra, reinterpret_cast<lds_u32 *>((uintptr_t)(slot + (1 + j) * (16 * ROW))), 16,
                                           (int)(in && 16 * j + r < ranks ? o : kOutside), 0, 0, 0);
                }
            };
            floatx4 acc[RB];
#pragma unroll
            for (int j = 0; j < RB; ++j)
                acc[j] = floatx4{0, 0, 0, 0};
#pragma unroll
            for (int s = 0; s < NS - 1; ++s)
                issue(s);
            // Stage kt has landed, and every wave has read stage kt-1, whose slot
            // takes the stage NS-1 ahead.
            for (int kt = 0; kt < nk; ++kt) {
                wait_vmcnt<(NS - 2) * L>();
                __builtin_amdgcn_s_barrier();
                __builtin_amdgcn_sched_barrier(0);
                __atomic_signal_fence(__ATOMIC_SEQ_CST);
                const unsigned char *slot = smem + (kt % NS) * SLOT;
                const int c = ((wave * 4 + fhi) ^ frow) * 16;
                half8 x, a[RB];
                x = *reinterpret_cast<const half8 *>(slot + frow * ROW + c);
#pragma unroll
                for (int j = 0; j < RB; ++j)
                    a[j] = *reinterpret_cast<const half8 *>(slot + (16 * (1 + j) + frow) * ROW + c);
                issue(kt + NS - 1);
                wait_lgkmcnt<0>();
                __builtin_amdgcn_sched_barrier(0);
#pragma unroll
                for (int j = 0; j < RB; ++j)
                    acc[j] = mfma_16x16x32<BF16>(a[j], x, acc[j]);
            }
            // the ring's last loads (zero fills) and everyone's reads are done
            wait_vmcnt<0>();
            __builtin_amdgcn_s_barrier();
            __builtin_amdgcn_sched_barrier(0);
            __atomic_signal_fence(__ATOMIC_SEQ_CST);
            end_turn<RB, BF16>(q, reinterpret_cast<float(*)[16][RB * 16]>(smem), acc, row0, r0, g, wave, lane);
        });
        if (blockIdx.y == 0 && blockIdx.z == 0)
            for (int i = wave; i < rows; i += TW)
                store_zeros(q, row0 + i, lane, 64);
    }
}

template <bool BF16>
hipError_t shrink(const Shrink &q, hipStream_t s)
{
    const int parts = (q.rank + PER - 1) / PER;
    if (q.M <= kFewRows)
        return start(shrink_rows_kernel<BF16>, (int64_t)q.M * parts, RT, s, q, parts);
    const int64_t blocks = ((int64_t)q.M + 15) / 16, grid = blocks < (1 << 17) ? blocks : 1 << 17;
    const int rb = (q.rank + 15) / 16;
    const bool deep = blocks * rb <= cu_count();
    const int per = deep ? 1 : rb > 2 ? 4 : rb, ranks = (rb + per - 1) / per;
    // one or four workgroups per CU, at most one per row of a block
    int64_t slots = (deep ? 1 : 4) * (int64_t)cu_count() / (blocks * ranks);
    slots = slots < 1 ? 1 : slots > 16 ? 16 : slots;
    const Place w{(int)blocks, (int)slots};
    auto go = [&](auto kernel) {
        void *args[] = {const_cast<Shrink *>(&q), const_cast<Place *>(&w)};
        return hipLaunchKernel(reinterpret_cast<const void *>(kernel),
                               dim3((unsigned)grid, (unsigned)ranks, (unsigned)slots), dim3(TT), args, 0, s);
    };
    if (q.direct)
        return deep       ? go(shrink_stream_kernel<1, true, BF16>)
               : per == 1 ? go(shrink_stream_kernel<1, false, BF16>)
               : per == 2 ? go(shrink_stream_kernel<2, false, BF16>)
                          : go(shrink_stream_kernel<4, false, BF16>);
    return per == 1 ? go(shrink_tile_kernel<1, BF16>) : per == 2 ? go(shrink_tile_kernel<2, BF16>) : go(shrink_tile_kernel<4, BF16>);
}

}  // namespace

hipError_t launch_shrink(const Shrink &q, bool bf16, hipStream_t s)
{
    return bf16 ? shrink<true>(q, s) : shrink<false>(q, s);
}

}  // namespace lin
}  // namespace hg
