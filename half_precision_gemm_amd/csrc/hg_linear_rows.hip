// hg_linear_rows.hip — the passes of the linear layer that go over a matrix
// once: 8-bit checkpoints written and read, dZ = dY·act'(Z) with its column
// sums, partial sums added up, operands copied to aligned rows.
//
// All of them are bound by memory: a thread takes eight consecutive columns
// (16 bytes of 16-bit elements), so a wave moves whole 128-byte lines, and
// everything between the loads and the stores stays in registers.
#include "hg_linear.h"

namespace hg {
namespace lin {
namespace {

constexpr int THREADS = 256;

// Blocks of a grid-stride launch over `units` threads' work.
unsigned blocks_for(int64_t units)
{
    const int64_t b = (units + THREADS - 1) / THREADS, most = (int64_t)cu_count() * 32;
    return (unsigned)(b < most ? b : most);
}

__global__ void __launch_bounds__(THREADS) pad_kernel(const uint16_t *__restrict__ S, int64_t lds,
                                                      uint16_t *__restrict__ D, int64_t ldd, int64_t rows, int64_t cols)
{
    const int64_t units = ldd / 8, total = rows * units;
    for (int64_t i = (int64_t)blockIdx.x * THREADS + threadIdx.x; i < total; i += (int64_t)gridDim.x * THREADS) {
        const int64_t r = i / units, c = (i - r * units) * 8;
        const uint16_t *s = S + r * lds + c;
        u32x4 w = {0, 0, 0, 0};
#pragma unroll
        for (int e = 0; e < 8; ++e)
            if (c + e < cols)
                w[e >> 1] |= (uint32_t)s[e] << (16 * (e & 1));
        *reinterpret_cast<u32x4 *>(D + r * ldd + c) = w;
    }
}

template <bool WIDE>
__global__ void __launch_bounds__(THREADS) zero_kernel(void *C, int64_t ldc, int64_t rows, int64_t cols)
{
    const int64_t total = rows * cols;
    for (int64_t i = (int64_t)blockIdx.x * THREADS + threadIdx.x; i < total; i += (int64_t)gridDim.x * THREADS) {
        const int64_t r = i / cols, c = i - r * cols;
        if (WIDE)
            static_cast<float *>(C)[r * ldc + c] = 0.0f;
        else
            static_cast<uint16_t *>(C)[r * ldc + c] = 0;
    }
}

// Four neighbouring lanes hold one block of 32 columns; units past the last
// column or row take part in the block's largest value with zeros.
template <bool BF16>
__global__ void __launch_bounds__(THREADS) write8_kernel(const uint16_t *__restrict__ X, int64_t ldx,
                                                         uint8_t *__restrict__ C, int64_t ldc, uint8_t *__restrict__ S,
                                                         int64_t lds, int64_t rows, int64_t cols, int xvec, int cvec)
{
    const int64_t units = (cols + kBlock8 - 1) / kBlock8 * 4, total = rows * units;
    const int64_t end = (total + 3) & ~(int64_t)3;
    for (int64_t i = (int64_t)blockIdx.x * THREADS + threadIdx.x; i < end; i += (int64_t)gridDim.x * THREADS) {
        const int64_t r = i / units, c = (i - r * units) * 8;
        const int n = (int)(cols - c < 8 ? cols - c : 8);       // may be <= 0 in a short last block
        float v[8];
        load8<BF16>(X + r * ldx + c, n, xvec, v);
        float a = 0.0f;
#pragma unroll
        for (int e = 0; e < 8; ++e)
            a = __builtin_fmaxf(a, finite_abs(v[e]));
        const int x = scale_exponent<BF16>(max_of_4(a));
        if (n > 0)
            store_codes(C + r * ldc + c, n, cvec, codes8<BF16>(v, x));
        if (c % kBlock8 == 0)
            S[r * lds + c / kBlock8] = (uint8_t)(x + 127);
    }
}

template <bool BF16>
__global__ void __launch_bounds__(THREADS) read8_kernel(const uint8_t *__restrict__ C, int64_t ldc,
                                                        const uint8_t *__restrict__ S, int64_t lds,
                                                        uint16_t *__restrict__ X, int64_t ldx, int64_t rows,
                                                        int64_t cols, int64_t pad, int xvec, int cvec)
{
    const int64_t units = (pad + 7) / 8, total = rows * units;
    for (int64_t i = (int64_t)blockIdx.x * THREADS + threadIdx.x; i < total; i += (int64_t)gridDim.x * THREADS) {
        const int64_t r = i / units, c = (i - r * units) * 8;
        const int n = (int)(cols - c < 8 ? cols - c : 8);
        float v[8] = {0, 0, 0, 0, 0, 0, 0, 0};
        if (n > 0) {
            const float s = scale_of(S[r * lds + c / kBlock8]);
            values8(load_codes(C + r * ldc + c, n, cvec), s, v);
#pragma unroll
            for (int e = 0; e < 8; ++e)
                v[e] = e < n ? v[e] : 0.0f;
        }
        store8<BF16>(X + r * ldx + c, (int)(pad - c < 8 ? pad - c : 8), xvec, v);
    }
}

// dZ and its column sums.  A workgroup takes 256 columns (32 threads of eight)
// of one strip of rows, eight rows at a time; each thread keeps its columns'
// sums in fp32 registers, the eight rows' threads are added in a fixed order
// through LDS, and the strips by a second launch: no atomics.
constexpr int SC = 32, SR = THREADS / SC;
template <bool BF16, int ACT, int SAVE>
__global__ void __launch_bounds__(THREADS) slope_kernel(const Slope p)
{
    __shared__ float part[SR][SC * 8 + 8];
    const int tc = threadIdx.x % SC, tr = threadIdx.x / SC;
    const int64_t c = (int64_t)blockIdx.x * (SC * 8) + tc * 8;
    const int64_t r0 = (int64_t)blockIdx.y * p.strip, r1 = r0 + p.strip < p.rows ? r0 + p.strip : p.rows;
    const int n = (int)(p.cols - c < 8 ? p.cols - c : 8);
    float sum[8] = {0, 0, 0, 0, 0, 0, 0, 0};
    if (n > 0) {
        const uint16_t *dy = static_cast<const uint16_t *>(p.dY) + c;
#pragma unroll 4
        for (int64_t r = r0 + tr; r < r1; r += SR) {
            float y[8], z[8];
            load8<BF16>(dy + r * p.lddy, n, p.yvec, y);
            if constexpr (ACT != kNone) {
                if constexpr (SAVE == kSave8)
                    values8(load_codes(static_cast<const uint8_t *>(p.Z) + r * p.ldz + c, n, p.zvec),
                            scale_of(p.Zs[r * p.ldzs + c / kBlock8]), z);
                else
                    load8<BF16>(static_cast<const uint16_t *>(p.Z) + r * p.ldz + c, n, p.zvec, z);
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    y[e] = e < n ? slope<ACT>(y[e], z[e]) : 0.0f;
            }
#pragma unroll
            for (int e = 0; e < 8; ++e)
                sum[e] += y[e];
            if (p.D)
                *reinterpret_cast<u32x4 *>(static_cast<uint16_t *>(p.D) + r * p.ldd + c) = pack8<BF16>(y);
        }
    }
    if (!p.Q && !p.db)
        return;
#pragma unroll
    for (int e = 0; e < 8; ++e)
        part[tr][tc * 8 + e] = sum[e];
    __syncthreads();
    const int64_t col = (int64_t)blockIdx.x * (SC * 8) + threadIdx.x;
    if (col >= p.cols)
        return;
    float t = 0.0f;
#pragma unroll
    for (int g = 0; g < SR; ++g)
        t += part[g][threadIdx.x];
    if (p.Q)
        p.Q[blockIdx.y * p.cols + col] = t;
    else
        p.db[col] = p.accumulate ? p.db[col] + t : t;
}

// db = (db +) the strips' sums: 32 columns per workgroup, eight threads to a
// column, each every eighth strip.
__global__ void __launch_bounds__(THREADS) sum_strips_kernel(const float *__restrict__ Q, int64_t strips, int64_t cols,
                                                             float *__restrict__ db, int accumulate)
{
    constexpr int CW = 32, G = THREADS / CW;
    __shared__ float part[G][CW];
    const int tc = threadIdx.x % CW, g = threadIdx.x / CW;
    const int64_t col = (int64_t)blockIdx.x * CW + tc;
    float t = 0.0f;
    if (col < cols) {
#pragma unroll 4
        for (int64_t s = g; s < strips; s += G)
            t += Q[s * cols + col];
    }
    part[g][tc] = t;
    __syncthreads();
    if (g != 0 || col >= cols)
        return;
#pragma unroll
    for (int k = 1; k < G; ++k)
        t += part[k][tc];
    db[col] = accumulate ? db[col] + t : t;
}

// The slices' partial sums added in order, then what a product's epilogue does.
template <bool BF16>
__global__ void __launch_bounds__(THREADS) reduce_kernel(const Product p)
{
    const int64_t units = ((int64_t)p.N + kBlock8 - 1) / kBlock8 * 4, total = (int64_t)p.M * units;
    for (int64_t i = (int64_t)blockIdx.x * THREADS + threadIdx.x; i < total; i += (int64_t)gridDim.x * THREADS) {
        const int row = (int)(i / units), col = (int)(i - row * units) * 8;
        float v[8] = {0, 0, 0, 0, 0, 0, 0, 0}, b[8];
        if (col < p.N) {
            const float *q = p.P + (int64_t)row * p.ldp + col;
            const bool two = col + 4 < p.ldp;
            for (int s = 0; s < p.splits; ++s, q += (int64_t)p.M * p.ldp) {
                const floatx4 lo = *reinterpret_cast<const floatx4 *>(q);
                floatx4 hi = {0, 0, 0, 0};
                if (two)
                    hi = *reinterpret_cast<const floatx4 *>(q + 4);
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    v[e] += lo[e];
                    v[4 + e] += hi[e];
                }
            }
        }
        load_bias(p.f, col, b);
        finish8<BF16>(p.f, row, col, v, b);
    }
}

bool aligned(const void *p, int64_t ld, int64_t bytes, int64_t each)
{
    return reinterpret_cast<uintptr_t>(p) % bytes == 0 && ld * each % bytes == 0;
}

template <bool BF16, int ACT>
void slope_save(const Slope &p, dim3 grid, hipStream_t s)
{
    if (p.save == kSave8)
        hipLaunchKernelGGL((slope_kernel<BF16, ACT, kSave8>), grid, dim3(THREADS), 0, s, p);
    else
        hipLaunchKernelGGL((slope_kernel<BF16, ACT, kSave16>), grid, dim3(THREADS), 0, s, p);
}
template <bool BF16>
void slope_act(const Slope &p, dim3 grid, hipStream_t s)
{
    switch (p.act) {
    case kRelu: slope_save<BF16, kRelu>(p, grid, s); break;
    case kGelu: slope_save<BF16, kGelu>(p, grid, s); break;
    case kGeluTanh: slope_save<BF16, kGeluTanh>(p, grid, s); break;
    case kSilu: slope_save<BF16, kSilu>(p, grid, s); break;
    default: hipLaunchKernelGGL((slope_kernel<BF16, kNone, kSave16>), grid, dim3(THREADS), 0, s, p); break;
    }
}

}  // namespace

hipError_t launch_pad(const void *S, int64_t lds, void *D, int64_t ldd, int64_t rows, int64_t cols, hipStream_t s)
{
    hipLaunchKernelGGL(pad_kernel, dim3(blocks_for(rows * (ldd / 8))), dim3(THREADS), 0, s,
                       static_cast<const uint16_t *>(S), lds, static_cast<uint16_t *>(D), ldd, rows, cols);
    return hipGetLastError();
}

hipError_t launch_zero(void *C, int64_t ldc, int64_t rows, int64_t cols, bool wide, hipStream_t s)
{
    if (wide)
        hipLaunchKernelGGL((zero_kernel<true>), dim3(blocks_for(rows * cols)), dim3(THREADS), 0, s, C, ldc, rows, cols);
    else
        hipLaunchKernelGGL((zero_kernel<false>), dim3(blocks_for(rows * cols)), dim3(THREADS), 0, s, C, ldc, rows, cols);
    return hipGetLastError();
}

hipError_t launch_write8(const void *X, int64_t ldx, uint8_t *C, int64_t ldc, uint8_t *S, int64_t lds, int64_t rows,
                         int64_t cols, bool bf16, hipStream_t s)
{
    const unsigned b = blocks_for(rows * ((cols + kBlock8 - 1) / kBlock8 * 4));
    const int xv = aligned(X, ldx, 16, 2), cv = aligned(C, ldc, 8, 1);
    const uint16_t *x = static_cast<const uint16_t *>(X);
    if (bf16)
        hipLaunchKernelGGL((write8_kernel<true>), dim3(b), dim3(THREADS), 0, s, x, ldx, C, ldc, S, lds, rows, cols, xv, cv);
    else
        hipLaunchKernelGGL((write8_kernel<false>), dim3(b), dim3(THREADS), 0, s, x, ldx, C, ldc, S, lds, rows, cols, xv, cv);
    return hipGetLastError();
}

hipError_t launch_read8(const uint8_t *C, int64_t ldc, const uint8_t *S, int64_t lds, void *X, int64_t ldx, int64_t rows,
                        int64_t cols, int64_t pad, bool bf16, hipStream_t s)
{
    const unsigned b = blocks_for(rows * ((pad + 7) / 8));
    const int xv = aligned(X, ldx, 16, 2), cv = aligned(C, ldc, 8, 1);
    uint16_t *x = static_cast<uint16_t *>(X);
    if (bf16)
        hipLaunchKernelGGL((read8_kernel<true>), dim3(b), dim3(THREADS), 0, s, C, ldc, S, lds, x, ldx, rows, cols, pad, xv, cv);
    else
        hipLaunchKernelGGL((read8_kernel<false>), dim3(b), dim3(THREADS), 0, s, C, ldc, S, lds, x, ldx, rows, cols, pad, xv, cv);
    return hipGetLastError();
}

hipError_t launch_slope(const Slope &p, bool bf16, hipStream_t s)
{
    const int64_t strips = (p.rows + p.strip - 1) / p.strip, tiles = (p.cols + SC * 8 - 1) / (SC * 8);
    if (strips > 65535 || tiles > 0x7fffffff)
        return hipErrorInvalidConfiguration;
    const dim3 grid((unsigned)tiles, (unsigned)strips);
    if (bf16)
        slope_act<true>(p, grid, s);
    else
        slope_act<false>(p, grid, s);
    return hipGetLastError();
}

hipError_t launch_sum_strips(const float *Q, int64_t strips, int64_t cols, float *db, bool accumulate, hipStream_t s)
{
    hipLaunchKernelGGL(sum_strips_kernel, dim3((unsigned)((cols + 31) / 32)), dim3(THREADS), 0, s, Q, strips, cols, db,
                       accumulate ? 1 : 0);
    return hipGetLastError();
}

hipError_t launch_reduce(const Product &p, bool bf16, hipStream_t s)
{
    const unsigned b = blocks_for((int64_t)p.M * (((int64_t)p.N + kBlock8 - 1) / kBlock8 * 4));
    if (bf16)
        hipLaunchKernelGGL((reduce_kernel<true>), dim3(b), dim3(THREADS), 0, s, p);
    else
        hipLaunchKernelGGL((reduce_kernel<false>), dim3(b), dim3(THREADS), 0, s, p);
    return hipGetLastError();
}

}  // namespace lin
}  // namespace hg
