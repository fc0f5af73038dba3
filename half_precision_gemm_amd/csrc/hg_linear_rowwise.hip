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

// Where a workgroup's sums begin: at what the rows' adapters add (hg_linear.h,
// Adapters), or at zero.  The waves share the rank's eighths and the blocks of 16
// rows: a lane takes the columns and rows whose sums it holds, with T in fp32 and
// eight of B in one load for each of them, so that 64 rows of 64 adapters cost what
// those of one do.
template <int NB, int MB, bool BF16>
__device__ __forceinline__ void begin_sums(const Product &p, floatx4 (&acc)[MB][NB], int n0, int wave, int lane)
{
    const Adapters &a = p.ad;
    const int frow = lane & 15, fhi = lane >> 4;
    int mine[MB];
#pragma unroll
    for (int i = 0; i < MB; ++i)
        mine[i] = adapter_of(a, 16 * i + frow, p.M);
    // `split` waves share an eighth, each every split-th block of rows
    const int chunks = (a.rank + 7) / 8, split = chunks >= WAVES ? 1 : chunks > 2 ? 2 : 4;
    for (int k = wave / split * 8; k < a.rank; k += 8 * WAVES / split) {
#pragma unroll
        for (int i = 0; i < MB; ++i) {
            if ((i & (split - 1)) != (wave & (split - 1)) || mine[i] < 0)
                continue;
            const float *T = static_cast<const float *>(a.T) + (16 * i + frow) * a.ldt;
            const uint16_t *B = a.B + mine[i] * a.stride;
            if (k + 8 <= a.rank) {
                const floatx4 lo = *reinterpret_cast<const floatx4 *>(T + k), hi = *reinterpret_cast<const floatx4 *>(T + k + 4);
                const float t[8] = {lo[0], lo[1], lo[2], lo[3], hi[0], hi[1], hi[2], hi[3]};
                add_eight<BF16, NB>(a, B, n0 + 4 * fhi, p.N, k, t, acc[i]);
            } else {
#pragma clang loop unroll(disable)
                for (int r = k; r < a.rank; ++r)
                    add_singly<BF16, NB>(a, B, n0 + 4 * fhi, p.N, r, T[r], acc[i]);
            }
        }
    }
}

// The same for one row and a rank of at most 16 without a launch before: every
// workgroup computes T by itself, from X and A in L2, while W comes.  Thread t
// takes eight k of all 16 rows of A at once, whole lines of each.  The chain from
// `which` to A, T and B is 5 us of waits, so W's first loads are requested before
// it, T's sums are formed behind the first stage, and what they give is added when
// the sum over W is done.  The registers that this takes leave a CU one workgroup,
// and every workgroup reads all of A: taken where there is one for each CU.  In
// graphs, bf16, us, this / the launch before it, rank 8 and 16: 1×512×4096 8.0 / 9.3
// and 8.3 / 9.6, 1×1024×1024 6.1 / 7.1 and 6.3 / 7.1, 1×2048×4096 8.3 / 10.5 and 8.6 /
// 10.4, 1×4096×4096 8.6 / 10.6 and 9.0 / 10.6, 1×4096×14336 25.0 / 26.6 and 25.5 /
// 26.7; with more than one workgroup for a CU 1×4608×4096 14.7 / 12.8 and 15.4 / 13.0,
// 1×8128×4096 18.0 / 16.5 and 18.8 / 16.4.  2×4096×4096 in the matrix core's layout
// takes 17.2 for 12.7.  Larger ranks have the launch before: 1×4096×4096 10.9 at rank
// 32, 11.1 at 64, 1×16384×4096 26.1 at 16, 26.3 at 32, 26.7 at 64.
struct NoSums {
    __device__ __forceinline__ NoSums(const Product &, int, int) {}
};
template <int NB, bool BF16>
struct OwnSums {
    const Product &p;
    int lane, wave, g;
    const uint16_t *A;
    u32x4 xs, as[kOwnRank];
    float v[kOwnRank];

    __device__ __forceinline__ OwnSums(const Product &p_, int wave_, int lane_) : p(p_), lane(lane_), wave(wave_)
    {
        g = adapter_of(p.ad, 0, 1);
#pragma unroll
        for (int r = 0; r < kOwnRank; ++r)
            v[r] = 0.0f;
    }
    __device__ __forceinline__ void request(int k0)
    {
        const uint16_t *A = p.own + max(g, 0) * p.own_stride;
        const int k = k0 + threadIdx.x * 8, at = min(k, p.K - 8);
        xs = *reinterpret_cast<const u32x4 *>(p.A + at);
#pragma unroll
        for (int r = 0; r < kOwnRank; ++r)
            as[r] = *reinterpret_cast<const u32x4_any *>(A + min(r, p.ad.rank - 1) * p.own_ld + at);
    }
    // T's sum of this wave, value r in lanes 4r .. 4r + 3.
    __device__ __forceinline__ float sum()
    {
        for (int k0 = 0;;) {
            // (lanes past K hold the last eight again: left out, as zeros in X would make
            // a NaN of an infinity in A)
            if (k0 + (int)threadIdx.x * 8 < p.K) {
                float x[8];
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    x[e] = widen<BF16>((uint16_t)(xs[e >> 1] >> (16 * (e & 1))));
#pragma unroll
                for (int r = 0; r < kOwnRank; ++r)
#pragma unroll
                    for (int e = 0; e < 8; ++e)
                        v[r] = __builtin_fmaf(widen<BF16>((uint16_t)(as[r][e >> 1] >> (16 * (e & 1)))), x[e], v[r]);
            }
            k0 += THREADS * 8;
            if (k0 >= p.K)
                break;
            request(k0);
        }
        // halves of the values are handed to the other half of the lanes, four times
#pragma unroll
        for (int n = kOwnRank / 2, d = 32; n >= 1; n /= 2, d /= 2) {
            const bool high = (lane & d) != 0;
#pragma unroll
            for (int i = 0; i < n; ++i) {
                const float give = high ? v[i] : v[i + n], keep = high ? v[i + n] : v[i];
                v[i] = keep + __shfl_xor(give, d);
            }
        }
        v[0] += __shfl_xor(v[0], 2);
        return v[0] + __shfl_xor(v[0], 1);
    }
    // Adds the adapter's terms, wave w those of values 8w .. of T, lanes of row 0 to the
    // columns that they hold; scratch: LDS that nothing else uses meanwhile.
    __device__ __forceinline__ void add(float t, floatx4 (&acc)[1][NB], int n0, float *scratch)
    {
        if ((lane & 3) == 0)
            scratch[wave * kOwnRank + lane / 4] = t;
        __syncthreads();
        const int k = 8 * wave;
        if (g < 0 || (lane & 15) != 0 || k >= p.ad.rank)
            return;
        const float s = p.own_scales ? p.own_scales[g] : 1.0f;
        const auto one = [&](int r) __attribute__((always_inline)) {
            float w = 0.0f;
#pragma unroll
            for (int i = 0; i < WAVES; ++i)
                w += scratch[i * kOwnRank + r];
            return s * w;
        };
        const uint16_t *B = p.ad.B + g * p.ad.stride;
        const int col0 = n0 + 4 * (lane >> 4);
        if (k + 8 <= p.ad.rank) {
            float v[8];
#pragma unroll
            for (int h = 0; h < 8; ++h)
                v[h] = one(k + h);
            add_eight<BF16, NB>(p.ad, B, col0, p.N, k, v, acc[0]);
        } else {
#pragma clang loop unroll(disable)
            for (int r = k; r < p.ad.rank; ++r)
                add_singly<BF16, NB>(p.ad, B, col0, p.N, r, one(r), acc[0]);
        }
    }
};

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
template <int NB, int MB, bool ODD, bool BF16, int ADAPT>
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
    if constexpr (ADAPT == 1)
        begin_sums<NB, MB, BF16>(p, acc, n0, wave, lane);
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

template <int NB, int MB, bool BF16, int ADAPT>
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
    auto fill = [&]() __attribute__((always_inline)) {
#pragma unroll
        for (int s = 0; s < NS - 1; ++s)
            issue(s);
    };
    // (The adapters' loads are younger than the first stages': those come while
    // these are on their way.)
    fill();
    if constexpr (ADAPT == 1)
        begin_sums<NB, MB, BF16>(p, acc, n0, wave, lane);
    typename std::conditional<ADAPT == 2, OwnSums<NB, BF16>, NoSums>::type own(p, wave, lane);
    float own_t = 0.0f;
    if constexpr (ADAPT == 2)
        own.request(0);
    // Stage kt has landed, and every wave has read stage kt-1, whose slot takes
    // the stage NS-1 ahead.
    for (int kt = 0; kt < nk; ++kt) {
        // (OwnSums' loads are younger than the first stages': these waits are for
        // them too)
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
        if constexpr (ADAPT == 2) {
            if (kt == 0)
                own_t = own.sum();
        }
    }
    wait_vmcnt<0>();
    __builtin_amdgcn_s_barrier();
    __builtin_amdgcn_sched_barrier(0);
    __atomic_signal_fence(__ATOMIC_SEQ_CST);
    if constexpr (ADAPT == 2)
        own.add(own_t, acc, n0, reinterpret_cast<float *>(smem + WAVES * NB * 1024));
    finish_sums<NB, MB, BF16>(p, reinterpret_cast<float(*)[MB * 16][NB * 16]>(smem), acc, n0, wave, lane);
}

template <int NB, int MB, bool BF16, int ADAPT>
hipError_t launch_one(const Product &p, bool stream, bool odd, hipStream_t s)
{
    if constexpr (ADAPT == 2)
        return stream ? start(linear_stream_kernel<NB, MB, BF16, ADAPT>, (p.N + 16 * NB - 1) / (16 * NB), THREADS, s, p)
                      : hipErrorInvalidConfiguration;
    else
    return start(stream ? linear_stream_kernel<NB, MB, BF16, ADAPT>
                 : odd  ? linear_rowwise_kernel<NB, MB, true, BF16, ADAPT>
                        : linear_rowwise_kernel<NB, MB, false, BF16, ADAPT>,
                 (p.N + 16 * NB - 1) / (16 * NB), THREADS, s, p);
}

template <int NB, int MB, bool BF16>
hipError_t launch(const Product &p, bool stream, bool odd, hipStream_t s)
{
    if (p.own != nullptr) {
        if constexpr (NB == 1 && MB == 1)
            return launch_one<NB, MB, BF16, 2>(p, stream, odd, s);
        return hipErrorInvalidConfiguration;
    }
    return p.ad.B != nullptr ? launch_one<NB, MB, BF16, 1>(p, stream, odd, s)
                             : launch_one<NB, MB, BF16, 0>(p, stream, odd, s);
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
