// hg_linear_ring.hip — the products of the linear layer and of its gradient
// on 64×64 and 128×128 tiles (gfx950):
//
//   C(i, j) = Σ_k A(i, k)·B(j, k),  16-bit operands, fp32 sums,
//
// each operand stored k-contiguous or k-major, so that the forward product
// X·Wᵀ (both k-contiguous), dX = dZ·W (W is k-major: its rows are summed over)
// and dW = dZᵀ·X (both k-major) read the caller's arrays as they are.
//
//  * One workgroup of 4 waves (2×2) per tile; the sum is walked in 64-wide
//    stages through a ring of LDS slots filled by direct buffer→LDS loads, all
//    but one of them in flight: with tiles this small a stage is a few hundred
//    cycles of matrix work, and memory latency is what bounds them.
//  * No operand is transposed in memory, and none moves through registers on
//    its way into LDS (hg_linear.h: the slots' layout, the swizzle, the
//    transposing reads, the edges).
//  * The sum may be cut into slices (p.splits) for products with few tiles and
//    a long sum: each slice stores fp32 partial sums, which a second launch
//    adds in order, so the result does not depend on scheduling.
#include "hg_linear.h"

extern "C" __device__ void hg_lin_ring_load_lds(hg::lin::i32x4 rsrc, hg::lin::lds_u32 *lds, int size, int voffset,
                                                int soffset, int offset,
                                                int aux) __asm("llvm.amdgcn.raw.buffer.load.lds");

namespace hg {
namespace lin {
namespace {

constexpr int BK = kStage, NWAVES = 4, THREADS = 256;

// Ring depth: 64×64 tiles take 80 KiB, so that two workgroups share a CU (one
// multiplies while the other waits for memory or finishes its tile).
template <int EDGE>
constexpr int kSlots = EDGE == 64 ? 5 : 4;
template <int EDGE>
constexpr int kLds = kSlots<EDGE> * 2 * EDGE * kStage * 2;

template <int EDGE, bool TA, bool TB, bool KCHK, bool BF16, bool ADAPT = false>
__device__ __forceinline__ void ring_tile(const Product &p, const Spread &w, int id, unsigned char *smem)
{
    using SA = Side<EDGE, TA>;
    using SB = Side<EDGE, TB>;
    constexpr int SLOT = SA::BYTES + SB::BYTES;
    constexpr int NS = kSlots<EDGE>;
    constexpr int WT = EDGE / 2, T = WT / 16;                                // wave sub-tile, its 16×16 blocks
    constexpr int LA = SA::L, L = SA::L + SB::L;
    static_assert(NS >= 4 && (NS - 2) * L <= 63 && NS * SLOT == kLds<EDGE> && kLds<EDGE> >= NWAVES * 16 * WT * 4, "");

    const Item t = item_at<EDGE>(p, w, id);
    const int m0 = t.m0, n0 = t.n0, kt0 = t.kt0, nk = t.nk, K = p.K;
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int wm = wave >> 1, wn = wave & 1;
    const uint32_t lds_base = (uint32_t)reinterpret_cast<uintptr_t>(smem);

    Panel<EDGE, TA, KCHK> pa;
    Panel<EDGE, TB, KCHK> pb;
    pa.set(p.A, p.lda, m0, p.M, K, kt0, wave, lane);
    pb.set(p.B, p.ldb, n0, p.N, K, kt0, wave, lane);
    auto load = [](i32x4 r, lds_u32 *dst, int o) __attribute__((always_inline)) {
        hg_lin_ring_load_lds(r, dst, 16, o, 0, 0, 0);
    };
    auto issue_one = [&](int kt, int i) __attribute__((always_inline)) {
        const uint32_t slot = lds_base + (kt % NS) * SLOT;
        if (i < LA)
            pa.issue(load, kt, kt < nk, slot, i, wave, lane);
        else
            pb.issue(load, kt, kt < nk, slot + SA::BYTES, i - LA, wave, lane);
    };
    auto issue = [&](int kt) __attribute__((always_inline)) {
#pragma unroll
        for (int i = 0; i < L; ++i)
            issue_one(kt, i);
    };

    floatx4 acc[T][T];
#pragma unroll
    for (int i = 0; i < T; ++i)
#pragma unroll
        for (int j = 0; j < T; ++j)
            acc[i][j] = floatx4{0, 0, 0, 0};
#pragma unroll
    for (int s = 0; s < NS - 1; ++s)
        issue(s);

    constexpr int SPS = BK / 32;
    struct Frags {
        half8 a[SPS][T], b[SPS][T];
    };
    constexpr int NR = SPS * 2 * T;
    auto read_one = [&](int kt, Frags &f, auto rc) __attribute__((always_inline)) {
        constexpr int r = decltype(rc)::value;
        constexpr int s = r / (2 * T), q = r % (2 * T);
        const unsigned char *slot = smem + (kt % NS) * SLOT;
        if constexpr (q < T)
            f.a[s][q] = fragment<EDGE, TA>(slot, lane, wm * WT + q * 16, s);
        else
            f.b[s][q - T] = fragment<EDGE, TB>(slot + SA::BYTES, lane, wn * WT + (q - T) * 16, s);
    };
    auto read_stage = [&](int kt, Frags &f) __attribute__((always_inline)) {
        static_for<NR>([&](auto rc) __attribute__((always_inline)) { read_one(kt, f, rc); });
    };
    // Step kt: this wave's loads of stage kt+1 have landed (later stages may
    // be in flight); after the barrier everyone's have, and every wave has
    // finished reading stage kt-1 (its matrix instructions waited for those
    // reads), whose slot then takes stage kt+NS-1.
    // Fragments are read one stage ahead.  Reads past the last stage see
    // zero-filled slots and are not used.
    constexpr int NM = SPS * T * T;
    Frags f0, f1;
    wait_vmcnt<(NS - 2) * L>();
    __builtin_amdgcn_s_barrier();
    __builtin_amdgcn_sched_barrier(0);
    read_stage(0, f0);
    auto step = [&](int kt, const Frags &cur, Frags &nxt) __attribute__((always_inline)) {
        wait_vmcnt<(NS - 3) * L>();
        __builtin_amdgcn_s_barrier();
        __builtin_amdgcn_sched_barrier(0);
        // the stage's loads and reads spread over its matrix instructions
        static_for<NM>([&](auto mc) __attribute__((always_inline)) {
            constexpr int m = decltype(mc)::value;
            constexpr int s = m / (T * T), j = m / T % T, i = m % T;
            acc[i][j] = mfma_16x16x32<BF16>(cur.b[s][j], cur.a[s][i], acc[i][j]);
            static_for<L>([&](auto lc) __attribute__((always_inline)) {
                constexpr int l = decltype(lc)::value;
                if constexpr (l * NM / L == m)
                    issue_one(kt + NS - 1, l);
            });
            static_for<NR>([&](auto rc) __attribute__((always_inline)) {
                constexpr int r = decltype(rc)::value;
                if constexpr (r * NM / NR == m)
                    read_one(kt + 1, nxt, rc);
            });
            __builtin_amdgcn_sched_barrier(0);
        });
    };
    for (int kt = 0; kt < nk; kt += 2) {
        step(kt, f0, f1);
        if (kt + 1 < nk)
            step(kt + 1, f1, f0);
    }
    // The ring's last loads (zero fills) and everyone's reads are done before
    // the slots are used for the staging of the results.
    wait_vmcnt<0>();
    wait_lgkmcnt<0>();
    __builtin_amdgcn_s_barrier();

    unsigned char *stg = smem + wave * (16 * WT * 4);
    const int row0 = m0 + wm * WT;
    bool far = false;
    if constexpr (ADAPT) {
        static_assert(4 * (16 * WT * 4 + kGatherBytes<T, T>) <= kLds<EDGE>, "");
        if (kt0 == 0)
            far = add_adapters<BF16>(p, row0, n0 + wn * WT, lane, smem + 4 * (16 * WT * 4) + wave * kGatherBytes<T, T>, acc);
    }
    Drain<EDGE, WT, BF16> out(p, t, stg, lane, n0 + wn * WT);
    out.request(row0);
    settle(out.bias);
#pragma unroll
    for (int i = 0; i < T; ++i) {
        stage_put<WT>(stg, lane, acc[i]);
        // a wave's LDS accesses execute in order; the fences keep the compiler
        // from moving them across
        __atomic_signal_fence(__ATOMIC_SEQ_CST);
        if constexpr (ADAPT && !BF16) {
            if (__builtin_expect(far, 0))
                add_far<WT>(p, row0 + 16 * i, n0 + wn * WT, lane, stg);
            __atomic_signal_fence(__ATOMIC_SEQ_CST);
        }
        out.block(row0 + 16 * i, i == T - 1);
        __atomic_signal_fence(__ATOMIC_SEQ_CST);
    }
}

template <int EDGE, bool KCHK, bool BF16, bool ADAPT>
__global__ void __launch_bounds__(THREADS, 1) linear_ring_kernel(const Product p, const Spread w)
{
    __shared__ __attribute__((aligned(1024))) unsigned char smem[kLds<EDGE>];
    ring_tile<EDGE, false, false, KCHK, BF16, ADAPT>(p, w, blockIdx.x, smem);
}

// db = (db +) the strips' sums of 32 columns: eight threads to a column, each
// every eighth strip.
__device__ __forceinline__ void sum_strips(const Strips &b, int block, unsigned char *smem)
{
    constexpr int CW = 32, G = THREADS / CW;
    float(*part)[CW] = reinterpret_cast<float(*)[CW]>(smem);
    const int tc = threadIdx.x % CW, g = threadIdx.x / CW;
    const int64_t col = (int64_t)block * CW + tc;
    float t = 0.0f;
    if (col < b.cols) {
#pragma unroll 4
        for (int64_t s = g; s < b.strips; s += G)
            t += b.Q[s * b.cols + col];
    }
    part[g][tc] = t;
    __syncthreads();
    if (g != 0 || col >= b.cols)
        return;
#pragma unroll
    for (int k = 1; k < G; ++k)
        t += part[k][tc];
    b.db[col] = b.accumulate ? b.db[col] + t : t;
}

// The two products of a gradient and the end of its column sums, which do not
// depend on each other, in one launch: their tiles fill the GPU together, the
// longer ones (y_first: y's) first, so that short ones end the launch.
template <int EDGE, bool KCHK, bool BF16>
__global__ void __launch_bounds__(THREADS, 1)
linear_ring_pair_kernel(const Product x, const Product y, const Strips b, const Spread wx, const Spread wy, int y_first)
{
    __shared__ __attribute__((aligned(1024))) unsigned char smem[kLds<EDGE>];
    const int id = blockIdx.x, at_x = y_first ? id - wy.items : id, at_y = y_first ? id : id - wx.items;
    if (at_x >= 0 && at_x < wx.items)
        ring_tile<EDGE, false, true, KCHK, BF16>(x, wx, at_x, smem);
    else if (at_y >= 0 && at_y < wy.items)
        ring_tile<EDGE, true, true, false, BF16>(y, wy, at_y, smem);
    else
        sum_strips(b, id - wx.items - wy.items, smem);
}

Spread spread(const Product &p, int edge, int64_t &total)
{
    const int64_t tm = ((int64_t)p.M + edge - 1) / edge, tn = ((int64_t)p.N + edge - 1) / edge;
    total = p.whole + (tm * tn - p.whole) * p.splits;
    return {(int)tm, (int)tn, total > kMostBlocks ? 0 : (int)total};
}

template <int EDGE, bool BF16>
hipError_t launch(const Product &p, hipStream_t s)
{
    int64_t total;
    const Spread w = spread(p, EDGE, total);
    if (total <= 0)
        return hipSuccess;
    if (total > kMostBlocks)
        return hipErrorInvalidConfiguration;
    if (p.ad.B != nullptr)
        return start(p.K % BK != 0 ? linear_ring_kernel<EDGE, true, BF16, true> : linear_ring_kernel<EDGE, false, BF16, true>,
                     total, THREADS, s, p, w);
    return start(p.K % BK != 0 ? linear_ring_kernel<EDGE, true, BF16, false> : linear_ring_kernel<EDGE, false, BF16, false>,
                 total, THREADS, s, p, w);
}

template <int EDGE, bool BF16>
hipError_t launch_pair(const Product *x, const Product *y, const Strips &b, hipStream_t s)
{
    const Product none{};
    const Product &px = x ? *x : none, &py = y ? *y : none;
    int64_t tx, ty;
    const Spread wx = spread(px, EDGE, tx), wy = spread(py, EDGE, ty);
    const int64_t total = tx + ty + (b.strips > 0 ? (b.cols + 31) / 32 : 0);
    if (total <= 0)
        return hipSuccess;
    if (total > kMostBlocks)
        return hipErrorInvalidConfiguration;
    const int y_first = py.per > px.per;
    // (both k-major: the buffer's range ends the sum)
    return start(px.K % BK != 0 ? linear_ring_pair_kernel<EDGE, true, BF16> : linear_ring_pair_kernel<EDGE, false, BF16>,
                 total, THREADS, s, px, py, b, wx, wy, y_first);
}

}  // namespace

hipError_t launch_ring(const Product &p, int tile, bool bf16, hipStream_t s)
{
    if (tile >= 128)
        return bf16 ? launch<128, true>(p, s) : launch<128, false>(p, s);
    return bf16 ? launch<64, true>(p, s) : launch<64, false>(p, s);
}

hipError_t launch_ring_pair(const Product *x, const Product *w, const Strips &b, int tile, bool bf16, hipStream_t s)
{
    if (tile >= 128)
        return bf16 ? launch_pair<128, true>(x, w, b, s) : launch_pair<128, false>(x, w, b, s);
    return bf16 ? launch_pair<64, true>(x, w, b, s) : launch_pair<64, false>(x, w, b, s);
}

}  // namespace lin
}  // namespace hg
