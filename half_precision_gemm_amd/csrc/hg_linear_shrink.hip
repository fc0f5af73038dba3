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
//  * More: 16 rows of X that share an adapter and 16 or 32 of the rank per
//    workgroup on the matrix cores, the sum split over its eight waves.  The rows
//    are gathered from a block of 256, so an adapter is read once or twice for all of
//    a block's rows that have it: with 16 neighbours and a turn for every adapter
//    among them, rows in no order read the adapters several times as often
//    (8192×4096, 64 adapters of rank 16 in no order: 206 us for 46; one adapter
//    to 128 neighbours on average: 22 for 18).
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
    const int up = (q.rank + 7) / 8 * 8;
    uint16_t *t = static_cast<uint16_t *>(q.T) + row * q.ldt + k;
    const uint16_t high = narrow<BF16>(v);
    // (of an infinity or NaN there is no rest)
    const bool in = __builtin_fabsf(widen<BF16>(high)) < __builtin_inff();
    const float rest = in ? v - widen<BF16>(high) : 0.0f;
    const uint16_t low = narrow<BF16>(rest);
    t[0] = high;
    t[up] = low;
    if (!BF16 && !in)
        q.far[row * up + k] = v;
    if (q.parts > 2)
        t[2 * up] = narrow<BF16>(rest - widen<BF16>(low));
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
        if (k >= q.parts * up || k - (k >= 2 * up ? 2 * up : k >= up ? up : 0) >= q.rank)
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

// A workgroup's place: blocks of kRows rows, 16·RB of the rank, one of `slots` among
// the block's workgroups, each of which takes every slots-th piece.
constexpr int kRows = 256;
struct Place {
    int blocks, slots;
};
// A piece: up to 16 rows of a block with the same adapter, in their order.
// Thread t < kRows knows row t's adapter, how many rows before it have the same one,
// and, of a piece's first row, its number (others: -1); count: the block's pieces.
struct Pieces {
    int g, before, number, count;
};
// Rows with the same adapter are found bit by bit of its number, 64 at a time: a
// ballot says which rows have the bit (comparing with each of the rows took 1 us
// more).
__device__ __forceinline__ Pieces pieces_of(const Shrink &q, int row0, int lane, int wave, int *lds)
{
    constexpr int SETS = kRows / 64;
    static_assert(TW >= SETS, "");
    int *const firsts = lds + 32;                                 // (behind what rows_of writes)
    Pieces m{-1, 0, -1, 0};
    uint64_t marks = 0;
    if (wave < SETS) {
        const Adapters who{q.which, nullptr, nullptr, nullptr, 0, 0, 0, q.count, q.rank, q.parts};
        int v[SETS];
        uint64_t same[SETS];
#pragma unroll
        for (int j = 0; j < SETS; ++j)
            v[j] = adapter_of(who, row0 + 64 * j + lane, q.M);
#pragma unroll
        for (int j = 0; j < SETS; ++j) {
            same[j] = __ballot(v[j] >= 0);
            m.g = j == wave ? v[j] : m.g;
        }
        for (int bit = 0; q.count >> bit > 0; ++bit) {
            const uint64_t mine = (m.g >> bit & 1) != 0 ? 0 : ~(uint64_t)0;
#pragma unroll
            for (int j = 0; j < SETS; ++j)
                same[j] &= __ballot((v[j] >> bit & 1) != 0) ^ mine;
        }
#pragma unroll
        for (int j = 0; j < SETS; ++j)
            m.before += j < wave    ? __builtin_popcountll(same[j])
                        : j == wave ? __builtin_popcountll(same[j] & (((uint64_t)1 << lane) - 1))
                                    : 0;
        const bool first = m.g >= 0 && m.before % 16 == 0;
        marks = __ballot(first);
        m.number = first ? __builtin_popcountll(marks & (((uint64_t)1 << lane) - 1)) : -1;
        if (lane == 0)
            firsts[wave] = __builtin_popcountll(marks);
    }
    __syncthreads();
#pragma unroll
    for (int w = 0; w < SETS; ++w) {
        m.number += w < wave && m.number >= 0 ? firsts[w] : 0;
        m.count += firsts[w];
    }
    m.count = __builtin_amdgcn_readfirstlane(m.count);
    return m;
}
// Piece c's adapter, and in lanes l, l + 16, ... its row l within the block (-1: none).
__device__ __forceinline__ int rows_of(const Pieces &m, int c, int *lds, int &g)
{
    if (threadIdx.x < 16)
        lds[threadIdx.x] = -1;
    if (m.number == c) {
        lds[16] = m.g;
        lds[17] = m.before;
    }
    __syncthreads();
    g = __builtin_amdgcn_readfirstlane(lds[16]);
    const unsigned i = (unsigned)(m.before - lds[17]);
    if (m.g == g && i < 16)
        lds[i] = threadIdx.x;
    __syncthreads();
    const int row = lds[threadIdx.x & 15];
    __syncthreads();
    return row;
}
// The waves' sums of a piece's values of T, added in order and stored.
template <int RB, bool BF16>
__device__ __forceinline__ void end_piece(const Shrink &q, float (*part)[16][RB * 16], const floatx4 (&acc)[RB], int row0,
                                          int row, int r0, int g, int wave, int lane)
{
    const int frow = lane & 15, fhi = lane >> 4;
    // (a lane holds values 4·fhi .. +3 of 16 of row frow)
#pragma unroll
    for (int j = 0; j < RB; ++j)
        *reinterpret_cast<floatx4 *>(&part[wave][frow][16 * j + 4 * fhi]) = acc[j];
    __syncthreads();
    // (whole waves take part or none of them)
    for (int i = threadIdx.x; i < 16 * RB * 16; i += TT) {
        const int r = i / (RB * 16), k = i % (RB * 16), to = __shfl(row, r);
        float t = 0.0f;
#pragma unroll
        for (int w = 0; w < TW; ++w)
            t += part[w][r][k];
        if (r0 + k < q.rank && to >= 0)
            store_t<BF16>(q, row0 + to, r0 + k, q.scales ? q.scales[g] * t : t);
    }
    if (r0 == 0)
        for (int r = wave; r < 16; r += TW) {
            const int to = __builtin_amdgcn_readlane(row, r);
            if (to >= 0)
                store_zeros(q, row0 + to, lane, 64);
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
    int *const lds = reinterpret_cast<int *>(part);
    for (int block = blockIdx.x; block < w.blocks; block += gridDim.x) {
        const int row0 = block * kRows;
        const Pieces m = pieces_of(q, row0, lane, wave, lds);
        for (int c = blockIdx.z; c < m.count; c += w.slots) {
            int g;
            const int row = rows_of(m, c, lds, g);
            const uint16_t *x = q.X + (row0 + max(row, 0)) * q.ldx + 8 * fhi;
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
            end_piece<RB, BF16>(q, part, acc, row0, row, r0, g, wave, lane);
        }
        __syncthreads();                  // (the next block's pieces_of writes what this one's reads)
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
constexpr int kShrinkSlots = (DEEP ? 160 : 80) * 1024 / kShrinkSlot<RB>;

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
    int *const lds = reinterpret_cast<int *>(smem);
    const int r = wave * RPI + lane / CH, ck = ((lane % CH) ^ (r & 15)) * 8;      // this lane's row of 16 and first k
    for (int block = blockIdx.x; block < w.blocks; block += gridDim.x) {
        const int row0 = block * kRows, rows = min(q.M - row0, kRows);
        const i32x4 rx = buffer_of(reinterpret_cast<uint64_t>(q.X) + (uint64_t)(row0 * q.ldx) * 2,
                                   (uint32_t)(rows - 1) * (uint32_t)q.ldx * 2 + (uint32_t)K * 2);
        const Pieces m = pieces_of(q, row0, lane, wave, lds);
        for (int c = blockIdx.z; c < m.count; c += w.slots) {
            int g;
            const int row = rows_of(m, c, lds, g), from = __shfl(row, r);
            const uint32_t ox = from >= 0 ? (uint32_t)from * (uint32_t)q.ldx * 2 + ck * 2 : kOutside;
            const i32x4 ra = buffer_of(reinterpret_cast<uint64_t>(q.A) + (uint64_t)(g * q.stride + r0 * q.lda) * 2,
                                       (uint32_t)(ranks - 1) * (uint32_t)q.lda * 2 + (uint32_t)K * 2);
            int at = (int)(((c >> 3) + (c & 7) * (unsigned)nk / 8) % (unsigned)nk);
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
            end_piece<RB, BF16>(q, reinterpret_cast<float(*)[16][RB * 16]>(smem), acc, row0, row, r0, g, wave, lane);
        }
        __syncthreads();                  // (the next block's pieces_of writes what this one's reads)
    }
}

template <bool BF16>
hipError_t shrink(const Shrink &q, hipStream_t s)
{
    const int parts = (q.rank + PER - 1) / PER;
    if (q.M <= kFewRows)
        return start(shrink_rows_kernel<BF16>, (int64_t)q.M * parts, RT, s, q, parts);
    const int64_t blocks = ((int64_t)q.M + kRows - 1) / kRows, grid = blocks < (1 << 17) ? blocks : 1 << 17;
    // a block's pieces at most: an adapter has one that is not whole
    const int rows = q.M < kRows ? q.M : kRows, most = (rows + 15) / 16 + (q.count < rows ? q.count : rows);
    const int rb = (q.rank + 15) / 16;
    const bool deep = blocks * most * rb <= cu_count();
    // (more of the rank in a workgroup leaves one to a CU: 8192×1024, rank 64, 83 us for 79
    // of the layer)
    const int per = deep || rb == 1 ? 1 : 2, ranks = (rb + per - 1) / per;
    // all pieces at once, or two workgroups per CU (8192 rows of 16 prompts: with four,
    // of which half find nothing, 2 us more)
    int64_t slots = deep ? most : 2 * (int64_t)cu_count() / (blocks * ranks);
    slots = slots < 1 ? 1 : slots > most ? most : slots;
    const Place w{(int)blocks, (int)slots};
    auto go = [&](auto kernel) {
        void *args[] = {const_cast<Shrink *>(&q), const_cast<Place *>(&w)};
        return hipLaunchKernel(reinterpret_cast<const void *>(kernel),
                               dim3((unsigned)grid, (unsigned)ranks, (unsigned)slots), dim3(TT), args, 0, s);
    };
    if (q.direct)
        return deep       ? go(shrink_stream_kernel<1, true, BF16>)
               : per == 1 ? go(shrink_stream_kernel<1, false, BF16>)
                          : go(shrink_stream_kernel<2, false, BF16>);
    return per == 1 ? go(shrink_tile_kernel<1, BF16>) : go(shrink_tile_kernel<2, BF16>);
}

}  // namespace

hipError_t launch_shrink(const Shrink &q, bool bf16, hipStream_t s)
{
    return bf16 ? shrink<true>(q, s) : shrink<false>(q, s);
}

}  // namespace lin
}  // namespace hg
