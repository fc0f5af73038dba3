// hg_linear_rows.hip — the passes of the linear layer that go over a matrix
// once: 8-bit checkpoints written and read, what the gradient's products wait
// for (dZ = dY·act'(Z) with its column sums, operands brought into rows that
// the tiles can load), partial sums added up.
//
// All of them are bound by memory: a thread takes eight consecutive columns
// (16 bytes of 16-bit elements), so a wave moves whole 128-byte lines, and
// everything between the loads and the stores stays in registers.
#include "hg_linear.h"

namespace hg {
namespace lin {
namespace {

constexpr int THREADS = 256;

// Blocks of a grid-stride pass over `units` threads' work.
int blocks_for(int64_t units)
{
    const int64_t b = (units + THREADS - 1) / THREADS, most = (int64_t)cu_count() * 32;
    return (int)(b < most ? b : most);
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
// column take part in the block's largest value with zeros.  (total is a
// multiple of four, so the four are in the loop together.)
template <bool BF16>
__global__ void __launch_bounds__(THREADS) write8_kernel(const uint16_t *__restrict__ X, int64_t ldx,
                                                         uint8_t *__restrict__ C, int64_t ldc, uint8_t *__restrict__ S,
                                                         int64_t lds, int64_t rows, int64_t cols)
{
    const int64_t units = (cols + kBlock8 - 1) / kBlock8 * 4, total = rows * units;
    for (int64_t i = (int64_t)blockIdx.x * THREADS + threadIdx.x; i < total; i += (int64_t)gridDim.x * THREADS) {
        const int64_t r = i / units, c = (i - r * units) * 8;
        const int n = (int)(cols - c < 8 ? cols - c : 8);       // may be <= 0 in a short last block
        float v[8];
        load8<BF16>(X + r * ldx + c, n, v);
        u32x2 w;
        const int x = encode8<BF16>(v, n, w);
        if (n > 0)
            store_codes(C + r * ldc + c, n, w);
        if (c % kBlock8 == 0)
            S[r * lds + c / kBlock8] = (uint8_t)(x + 127);
    }
}

// The values of n codes from column c of a row on (the others 0).
__device__ __forceinline__ void restore8(const uint8_t *codes, const uint8_t *scales, int64_t c, int n, float (&v)[8])
{
    values8(load_codes(codes + c, n), scale_of(scales[c / kBlock8]), v);
#pragma unroll
    for (int e = 0; e < 8; ++e)
        v[e] = e < n ? v[e] : 0.0f;
}

template <bool BF16>
__global__ void __launch_bounds__(THREADS) read8_kernel(const uint8_t *__restrict__ C, int64_t ldc,
                                                        const uint8_t *__restrict__ S, int64_t lds,
                                                        uint16_t *__restrict__ X, int64_t ldx, int64_t rows,
                                                        int64_t cols)
{
    const int64_t units = (cols + 7) / 8, total = rows * units;
    for (int64_t i = (int64_t)blockIdx.x * THREADS + threadIdx.x; i < total; i += (int64_t)gridDim.x * THREADS) {
        const int64_t r = i / units, c = (i - r * units) * 8;
        const int n = (int)(cols - c < 8 ? cols - c : 8);
        float v[8];
        restore8(C + r * ldc, S + r * lds, c, n, v);
        store8<BF16>(X + r * ldx + c, n, v);
    }
}

// One matrix into aligned rows with zeros behind its last column, by blocks
// block, block + blocks, ..
template <bool BF16>
__device__ __forceinline__ void copy_rows(const Copy &q, int block, int blocks)
{
    const int64_t units = q.ldd / 8, total = q.rows * units;
    for (int64_t i = (int64_t)block * THREADS + threadIdx.x; i < total; i += (int64_t)blocks * THREADS) {
        const int64_t r = i / units, c = (i - r * units) * 8;
        const int n = (int)(q.cols - c < 8 ? q.cols - c : 8);   // at least 1: ldd is cols rounded up to 8
        u32x4 w;
        if (q.scales) {
            float v[8];
            restore8(static_cast<const uint8_t *>(q.src) + r * q.lds, q.scales + r * q.ldss, c, n, v);
            w = pack8<BF16>(v);
        } else {
            w = load16x8(static_cast<const uint16_t *>(q.src) + r * q.lds + c, n);
        }
        *reinterpret_cast<u32x4 *>(static_cast<uint16_t *>(q.dst) + r * q.ldd + c) = w;
    }
}

// dZ and its column sums.  A workgroup takes 128 columns (16 threads of eight)
// of one strip of rows, 16 rows at a time and four of those in flight; each
// thread keeps its columns' sums in fp32 registers, the 16 rows' threads are
// added in a fixed order through LDS, and the strips by a later launch: no
// atomics.  A product's operand is rounded to 16 bits here; the sums take the
// unrounded values.
constexpr int SC = 16, SR = THREADS / SC, SU = 4;
template <bool BF16, int ACT, int SAVE>
__device__ __forceinline__ void slope_strip(const Slope &p, int tile, int strip)
{
    __shared__ float part[SR][SC * 8 + 8];
    const int tc = threadIdx.x % SC, tr = threadIdx.x / SC;
    const int64_t c = (int64_t)tile * (SC * 8) + tc * 8;
    const int64_t r0 = strip * p.strip, r1 = r0 + p.strip < p.rows ? r0 + p.strip : p.rows;
    const int n = (int)(p.cols - c < 8 ? p.cols - c : 8);
    float sum[8] = {0, 0, 0, 0, 0, 0, 0, 0};
    if (n > 0) {
        for (int64_t r = r0 + tr; r < r1; r += SR * SU) {
            float y[SU][8], z[SU][8];
#pragma unroll
            for (int u = 0; u < SU; ++u) {
                // past the strip: its last row again, dropped below
                const int64_t q = r + u * SR < r1 ? r + u * SR : r1 - 1;
                load8<BF16>(static_cast<const uint16_t *>(p.dY) + q * p.lddy + c, n, y[u]);
                if constexpr (ACT != kNone) {
                    if constexpr (SAVE == kSave8)
                        restore8(static_cast<const uint8_t *>(p.Z) + q * p.ldz, p.Zs + q * p.ldzs, c, n, z[u]);
                    else
                        load8<BF16>(static_cast<const uint16_t *>(p.Z) + q * p.ldz + c, n, z[u]);
                }
            }
#pragma unroll
            for (int u = 0; u < SU; ++u) {
                const int64_t q = r + u * SR;
                if (q >= r1)
                    break;
                if constexpr (ACT != kNone) {
#pragma unroll
                    for (int e = 0; e < 8; ++e)
                        y[u][e] = e < n ? slope<ACT>(y[u][e], z[u][e]) : 0.0f;
                }
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    sum[e] += y[u][e];
                if (p.D)
                    *reinterpret_cast<u32x4 *>(static_cast<uint16_t *>(p.D) + q * p.ldd + c) = pack8<BF16>(y[u]);
            }
        }
    }
    if (!p.Q && !p.db)
        return;
#pragma unroll
    for (int e = 0; e < 8; ++e)
        part[tr][tc * 8 + e] = sum[e];
    __syncthreads();
    const int64_t col = (int64_t)tile * (SC * 8) + threadIdx.x;
    if (threadIdx.x >= SC * 8 || col >= p.cols)
        return;
    float t = 0.0f;
#pragma unroll
    for (int g = 0; g < SR; ++g)
        t += part[g][threadIdx.x];
    if (p.Q)
        p.Q[strip * p.cols + col] = t;
    else
        p.db[col] = p.accumulate ? p.db[col] + t : t;
}

template <bool BF16, int ACT, int SAVE>
__global__ void __launch_bounds__(THREADS) prepare_kernel(const Slope g, const Copy x, const Copy w, int tiles,
                                                          int slopes, int xblocks, int wblocks)
{
    const int b = blockIdx.x;
    if (b < slopes)
        slope_strip<BF16, ACT, SAVE>(g, b % tiles, b / tiles);
    else if (b < slopes + xblocks)
        copy_rows<BF16>(x, b - slopes, xblocks);
    else
        copy_rows<BF16>(w, b - slopes - xblocks, wblocks);
}

// The slices of one product's cut tiles added in order, then what its epilogue
// does (K = 0: no slices, every tile).
template <bool BF16>
__device__ __forceinline__ void reduce_tiles(const Product &p, const Spread &w, int block, int blocks)
{
    const int edge = p.edge, units = edge / 8, area = edge * edge;
    const int64_t total = (int64_t)w.items * edge * units;
    for (int64_t i = (int64_t)block * THREADS + threadIdx.x; i < total; i += (int64_t)blocks * THREADS) {
        const int t = (int)(i / (edge * units)), at = (int)(i - (int64_t)t * edge * units);
        const int r = at / units, c = at % units * 8;
        int tm, tn;
        tile_at(p.whole + t, w, tm, tn);
        const int row = tm * edge + r, col = tn * edge + c;
        if (row >= p.M)
            continue;                                       // (four neighbours together)
        float v[8] = {0, 0, 0, 0, 0, 0, 0, 0}, b[8];
        if (col < p.N) {
            const float *q = p.P + (int64_t)t * p.splits * area + r * edge + c;
#pragma unroll 4
            for (int s = 0; s < p.splits; ++s, q += area) {
                const floatx4 lo = *reinterpret_cast<const floatx4 *>(q), hi = *reinterpret_cast<const floatx4 *>(q + 4);
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
template <bool BF16>
__global__ void __launch_bounds__(THREADS) reduce_kernel(const Product p, const Product q, const Spread wp, const Spread wq,
                                                         int pblocks, int qblocks)
{
    if ((int)blockIdx.x < pblocks)
        reduce_tiles<BF16>(p, wp, blockIdx.x, pblocks);
    else
        reduce_tiles<BF16>(q, wq, blockIdx.x - pblocks, qblocks);
}

template <bool BF16>
hipError_t prepare(const Slope &g, const Copy &x, const Copy &w, hipStream_t s)
{
    const int64_t tiles = g.rows > 0 ? (g.cols + SC * 8 - 1) / (SC * 8) : 0;
    const int64_t slopes = g.rows > 0 ? tiles * ((g.rows + g.strip - 1) / g.strip) : 0;
    const int xb = x.rows > 0 ? blocks_for(x.rows * (x.ldd / 8)) : 0, wb = w.rows > 0 ? blocks_for(w.rows * (w.ldd / 8)) : 0;
    const int64_t total = slopes + xb + wb;
    if (total == 0)
        return hipSuccess;
    if (total > kMostBlocks)
        return hipErrorInvalidConfiguration;
    auto go = [&](auto kernel) {
        return start(kernel, total, THREADS, s, g, x, w, (int)(tiles > 0 ? tiles : 1), (int)slopes, xb, wb);
    };
    const bool e = g.save == kSave8;
    switch (g.act) {
    case kRelu: return go(e ? prepare_kernel<BF16, kRelu, kSave8> : prepare_kernel<BF16, kRelu, kSave16>);
    case kGelu: return go(e ? prepare_kernel<BF16, kGelu, kSave8> : prepare_kernel<BF16, kGelu, kSave16>);
    case kGeluTanh: return go(e ? prepare_kernel<BF16, kGeluTanh, kSave8> : prepare_kernel<BF16, kGeluTanh, kSave16>);
    case kSilu: return go(e ? prepare_kernel<BF16, kSilu, kSave8> : prepare_kernel<BF16, kSilu, kSave16>);
    default: return go(prepare_kernel<BF16, kNone, kSave16>);
    }
}

}  // namespace

hipError_t launch_zero(void *C, int64_t ldc, int64_t rows, int64_t cols, bool wide, hipStream_t s)
{
    return start(wide ? zero_kernel<true> : zero_kernel<false>, blocks_for(rows * cols), THREADS, s, C, ldc, rows, cols);
}

hipError_t launch_write8(const void *X, int64_t ldx, uint8_t *C, int64_t ldc, uint8_t *S, int64_t lds, int64_t rows,
                         int64_t cols, bool bf16, hipStream_t s)
{
    const int blocks = blocks_for(rows * ((cols + kBlock8 - 1) / kBlock8 * 4));
    return start(bf16 ? write8_kernel<true> : write8_kernel<false>, blocks, THREADS, s, static_cast<const uint16_t *>(X),
                 ldx, C, ldc, S, lds, rows, cols);
}

hipError_t launch_read8(const uint8_t *C, int64_t ldc, const uint8_t *S, int64_t lds, void *X, int64_t ldx, int64_t rows,
                        int64_t cols, bool bf16, hipStream_t s)
{
    return start(bf16 ? read8_kernel<true> : read8_kernel<false>, blocks_for(rows * ((cols + 7) / 8)), THREADS, s, C, ldc, S,
                 lds, static_cast<uint16_t *>(X), ldx, rows, cols);
}

hipError_t launch_prepare(const Slope &g, const Copy &x, const Copy &w, bool bf16, hipStream_t s)
{
    return bf16 ? prepare<true>(g, x, w, s) : prepare<false>(g, x, w, s);
}

hipError_t launch_reduce(const Product *p, const Product *q, bool bf16, hipStream_t s)
{
    // items: the cut tiles
    auto cut = [](const Product *x) -> Spread {
        if (!x)
            return {0, 0, 0};
        const int tm = (int)(((int64_t)x->M + x->edge - 1) / x->edge), tn = (x->N + x->edge - 1) / x->edge;
        return {tm, tn, tm * tn - x->whole};
    };
    auto blocks = [](const Product *x, const Spread &w) {
        return w.items > 0 ? blocks_for((int64_t)w.items * x->edge * (x->edge / 8)) : 0;
    };
    const Spread wp = cut(p), wq = cut(q);
    const int pb = blocks(p, wp), qb = blocks(q, wq);
    const Product none{};
    if (pb + qb == 0)
        return hipSuccess;
    return start(bf16 ? reduce_kernel<true> : reduce_kernel<false>, pb + qb, THREADS, s, p ? *p : none, q ? *q : none, wp, wq,
                 pb, qb);
}

}  // namespace lin
}  // namespace hg
