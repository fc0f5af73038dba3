// hg_linear_shrink.hip — the first half of the low-rank adapters' product
// (gfx950): T = s_g·X·A_gᵀ, g the row's adapter, rank values a row, for the
// forward kernels that multiply it by B_g (hg_linear.h, Adapters).
//
// A row costs 2·rank flops per element of X it reads, so this is the reading of
// X and of the adapters in use.
//
//  * Few rows (shrink_rows_kernel): a workgroup per row and quarter of 16 of the
//    rank, fp32 sums of a wide load's products; each row reads its adapter
//    whatever the others' are, from L2 where they share it.
//  * More (shrink_tile_kernel): 16 rows of X and 16 to 64 of the rank per
//    workgroup on the matrix cores, the sum split over its waves; one turn for
//    every adapter among the 16 rows, of which each row keeps its own's.
#include "hg_linear.h"

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

constexpr int TW = 8, TT = TW * 64;                               // waves and threads of shrink_tile_kernel

// RB blocks of 16 of the rank, from 16·RB·blockIdx.y on; the rows' blocks of 16
// are walked.
template <int RB, bool BF16>
__global__ void __launch_bounds__(TT) shrink_tile_kernel(const Shrink q, int blocks)
{
    __shared__ __attribute__((aligned(16))) float part[TW][16][RB * 16];
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int frow = lane & 15, fhi = lane >> 4;
    const int r0 = blockIdx.y * (RB * 16);
    const Adapters who{q.which, nullptr, nullptr, 0, 0, 0, q.count, q.rank};
    for (int block = blockIdx.x; block < blocks; block += gridDim.x) {
        const int row0 = block * 16, mine = adapter_of(who, row0 + frow, q.M);
        const uint16_t *x = q.X + min(row0 + frow, q.M - 1) * q.ldx + 8 * fhi;
        for (int g = -1;;) {
            g = least_of_wave(mine > g ? mine : 0x7fffffff);
            if (g == 0x7fffffff)
                break;
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
                return *reinterpret_cast<const u32x4_any *>(p);
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
        if (blockIdx.y == 0)
            for (int r = wave; r < 16; r += TW)
                if (row0 + r < q.M)
                    store_zeros(q, row0 + r, lane, 64);
    }
}

template <bool BF16>
hipError_t shrink(const Shrink &q, hipStream_t s)
{
    const int parts = (q.rank + PER - 1) / PER;
    if (q.M <= kFewRows)
        return start(shrink_rows_kernel<BF16>, (int64_t)q.M * parts, RT, s, q, parts);
    const int64_t blocks = ((int64_t)q.M + 15) / 16, grid = blocks < (1 << 20) ? blocks : 1 << 20;
    const int rb = (q.rank + 15) / 16, per = rb > 2 ? 4 : rb;
    auto go = [&](auto kernel) {
        const int n = (int)blocks;
        void *args[] = {const_cast<Shrink *>(&q), const_cast<int *>(&n)};
        return hipLaunchKernel(reinterpret_cast<const void *>(kernel), dim3((unsigned)grid, (unsigned)((rb + per - 1) / per)),
                               dim3(TT), args, 0, s);
    };
    return per == 1 ? go(shrink_tile_kernel<1, BF16>) : per == 2 ? go(shrink_tile_kernel<2, BF16>) : go(shrink_tile_kernel<4, BF16>);
}

}  // namespace

hipError_t launch_shrink(const Shrink &q, bool bf16, hipStream_t s)
{
    return bf16 ? shrink<true>(q, s) : shrink<false>(q, s);
}

}  // namespace lin
}  // namespace hg
