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
//  * A k-contiguous operand's slot holds one 128-byte row per tile row, and a
//    matrix-core fragment (8 consecutive k of one row) is one 16-byte read.  A
//    k-major operand's slot holds one row of BM (or BN) elements per k; a
//    fragment is two transposing 8-byte reads (ds_read_b64_tr_b16), each of
//    which hands 16 lanes a 4 (k) × 16 (rows) block with the four k of a row
//    in one lane.  Neither form moves data through registers on its way in,
//    and nothing is transposed in memory.
//  * 16-byte chunks are XOR-swizzled within the slot's rows so that the reads
//    are free of bank conflicts; the loads realise the swizzle by which chunk
//    each lane fetches.
//  * Rows, columns and k past the edges load as zeros by the buffer's range
//    check; a k-contiguous operand whose K is no multiple of 64 is checked
//    chunk by chunk (KCHK), because the bytes behind a row are another row's.
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

constexpr int BK = 64, NWAVES = 4, THREADS = 256;
constexpr uint32_t OOB = 0x80000000u;          // an offset past every range

// One operand's slot of one stage, EDGE tile rows.
template <int EDGE, bool KMAJOR>
struct Side {
    static constexpr int RB = KMAJOR ? EDGE * 2 : BK * 2;         // bytes of an LDS row
    static constexpr int CH = RB / 16;                            // its 16-byte chunks
    static constexpr int RPI = 1024 / RB;                         // LDS rows per load instruction
    static constexpr int L = EDGE / (8 * NWAVES);                 // load instructions per wave
    static constexpr int BYTES = EDGE * BK * 2;
    // What the chunk index of LDS row r is XORed with.  k-contiguous: 16 rows
    // are read at one chunk, two rows to a 256-byte line of banks.  k-major: a
    // half wave reads the rows r, r+1, r+2, r+3 and the same + 8, 32 bytes
    // each: pairs of chunks are moved so that they fall on distinct banks.
    static __device__ __forceinline__ int swz(int r)
    {
        if constexpr (!KMAJOR)
            return (r >> 1) & 7;
        else if constexpr (EDGE >= 128)
            return ((r & 3) | ((r >> 1) & 4)) << 1;
        else
            return (((r >> 1) & 1) | ((r >> 2) & 2)) << 1;
    }
};

// Workgroup id → (slice, tile row, tile column): ids regrouped per XCD
// (consecutive ids run on different XCDs), then bands of 4 tile rows walked
// column by column, so that tiles on one XCD share panels in its L2.
__device__ __forceinline__ void place(int wg, int total, int tiles_m, int tiles_n, int &slice, int &tm, int &tn)
{
    const int per = total >> 3, rem = total & 7, x = wg & 7;
    const int q = x * per + min(x, rem) + (wg >> 3);
    const int tiles = tiles_m * tiles_n;
    slice = q / tiles;
    const int l = q - slice * tiles;
    const int band = l / (4 * tiles_n), first = band * 4;
    const int gsz = min(tiles_m - first, 4);
    const int r = l - band * 4 * tiles_n;
    tm = first + r % gsz;
    tn = r / gsz;
}

template <int EDGE, bool TA, bool TB, bool KCHK, bool BF16>
__global__ void __launch_bounds__(THREADS, 1) linear_ring_kernel(const Product p, int tiles_m, int tiles_n, int total)
{
    using SA = Side<EDGE, TA>;
    using SB = Side<EDGE, TB>;
    constexpr int SLOT = SA::BYTES + SB::BYTES;
    constexpr int NS = (128 * 1024) / SLOT < 8 ? (128 * 1024) / SLOT : 8;     // ring depth
    constexpr int WT = EDGE / 2, T = WT / 16;                                // wave sub-tile, its 16×16 blocks
    constexpr int LA = SA::L, L = SA::L + SB::L;
    static_assert(NS >= 4 && LA >= 1 && (NS - 2) * L <= 63 && NS * SLOT >= NWAVES * 16 * WT * 4, "");
    __shared__ __attribute__((aligned(1024))) unsigned char smem[NS * SLOT];

    int slice, tm, tn;
    place(blockIdx.x, total, tiles_m, tiles_n, slice, tm, tn);
    const int m0 = tm * EDGE, n0 = tn * EDGE, K = p.K;
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int wm = wave >> 1, wn = wave & 1;
    const int kt0 = slice * p.per;                                           // stages of this slice
    const int nk = min((K + BK - 1) / BK - kt0, p.per);
    const uint32_t lds_base = (uint32_t)reinterpret_cast<uintptr_t>(smem);

    // Load i of a wave fills 1 KiB of its operand's slot: LDS rows
    // (wave·L + i)·RPI .., lane l the chunk at position l.
    uint32_t off[L];
    int kchunk[L];
    auto chunk = [&](int i, int ch, int rpi, int l0) { return (l0 + i) * rpi + lane / ch; };
#pragma unroll
    for (int i = 0; i < L; ++i) {
        const bool isb = i >= LA;
        const int ch = isb ? SB::CH : SA::CH, rpi = isb ? SB::RPI : SA::RPI;
        const int row = chunk(isb ? i - LA : i, ch, rpi, wave * (isb ? SB::L : LA));
        const int c = (lane % ch) ^ (isb ? SB::swz(row) : SA::swz(row));
        const int64_t ld = isb ? p.ldb : p.lda;
        const int edge = isb ? p.N - n0 : p.M - m0;
        const bool ok = (isb ? TB : TA) ? c * 8 < edge : row < edge;
        off[i] = ok ? (uint32_t)(row * (int)ld * 2 + c * 16) : OOB;
        kchunk[i] = c * 8;
    }
    auto issue_one = [&](int kt, int i) __attribute__((always_inline)) {
        const bool isb = i >= LA, km = isb ? TB : TA;
        const uint16_t *base = isb ? p.B : p.A;
        const int64_t ld = isb ? p.ldb : p.lda;
        const int first = isb ? n0 : m0, edge = min((isb ? p.N : p.M) - first, EDGE);
        const int k = (kt0 + kt) * BK;
        uint32_t o = off[i];
        uint64_t a;
        uint32_t bytes;
        if (km) {
            // rows k .. k+63 of a k-major operand, at most K of them
            a = reinterpret_cast<uint64_t>(base) + ((uint64_t)k * (uint64_t)ld + (uint64_t)first) * 2;
            bytes = (uint32_t)(((min(K - k, BK) - 1) * (int)ld + ((edge + 7) & ~7)) * 2);
        } else {
            a = reinterpret_cast<uint64_t>(base) + ((uint64_t)first * (uint64_t)ld + (uint64_t)k) * 2;
            bytes = (uint32_t)(((edge - 1) * (int)ld + ((K + 7) & ~7) - k) * 2);
            if constexpr (KCHK)
                o = kchunk[i] < K - k ? o : OOB;
        }
        if (kt >= nk)
            bytes = 0;
        const uint32_t dst = lds_base + (kt % NS) * SLOT + (isb ? SA::BYTES : 0) +
                             (wave * (isb ? SB::L : LA) + (isb ? i - LA : i)) * 1024;
        hg_lin_ring_load_lds(buffer_of(a, bytes), reinterpret_cast<lds_u32 *>((uintptr_t)dst), 16, (int)o, 0, 0, 0);
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

    // Fragment of block `blk` and k-step s: lane l holds row l mod 16 of the
    // block and k = 32s + 8·(l div 16) .. +7, for both operands and both
    // storage forms, so the matrix core pairs matching k.
    const int frow = lane & 15, fhi = lane >> 4;
    auto frag = [&](auto side, const unsigned char *slot, int w, int s, int blk) -> half8 {
        using S = typename decltype(side)::type;
        constexpr bool km = std::is_same<S, Side<EDGE, true>>::value;
        if constexpr (!km) {
            const int row = w * WT + blk * 16 + frow;
            return *reinterpret_cast<const half8 *>(slot + row * S::RB + (((4 * s + fhi) ^ S::swz(row)) * 16));
        } else {
            const int row = 32 * s + 8 * fhi + (frow >> 2);
            const int c = (w * WT + blk * 16) / 8 + ((lane >> 1) & 1);
            const unsigned char *q = slot + row * S::RB + ((c ^ S::swz(row)) * 16) + (lane & 1) * 8;
            return read_tr(q, q + 4 * S::RB);
        }
    };
    struct TagA {
        using type = SA;
    };
    struct TagB {
        using type = SB;
    };
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
            f.a[s][q] = frag(TagA{}, slot, wm, s, q);
        else
            f.b[s][q - T] = frag(TagB{}, slot + SA::BYTES, wn, s, q - T);
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
    const int c0 = n0 + wn * WT;
    float bias[8];
    load_bias(p.f, c0 + 8 * (lane % (WT / 8)), bias);
#pragma unroll
    for (int i = 0; i < T; ++i) {
        stage_put<WT>(stg, lane, acc[i]);
        // a wave's LDS accesses execute in order; the fences keep the compiler
        // from moving them across
        __atomic_signal_fence(__ATOMIC_SEQ_CST);
        drain<WT, BF16>(p, stg, lane, m0 + wm * WT + 16 * i, c0, slice, bias);
        __atomic_signal_fence(__ATOMIC_SEQ_CST);
    }
}

template <int EDGE, bool TA, bool TB, bool BF16>
hipError_t launch(const Product &p, hipStream_t s)
{
    const int tiles_m = (int)(((int64_t)p.M + EDGE - 1) / EDGE), tiles_n = (p.N + EDGE - 1) / EDGE;
    const int64_t total = (int64_t)tiles_m * tiles_n * p.splits;
    if (total <= 0)
        return hipSuccess;
    if (total > 0x7fffffff)
        return hipErrorInvalidConfiguration;
    // both k-major: the buffer's range ends the sum
    if (!(TA && TB) && p.K % BK != 0)
        hipLaunchKernelGGL((linear_ring_kernel<EDGE, TA, TB, !(TA && TB), BF16>), dim3((unsigned)total), dim3(THREADS),
                           0, s, p, tiles_m, tiles_n, (int)total);
    else
        hipLaunchKernelGGL((linear_ring_kernel<EDGE, TA, TB, false, BF16>), dim3((unsigned)total), dim3(THREADS), 0,
                           s, p, tiles_m, tiles_n, (int)total);
    return hipGetLastError();
}

template <int EDGE>
hipError_t launch_layout(const Product &p, Layout l, bool bf16, hipStream_t s)
{
    switch (l) {
    case Layout::NN: return bf16 ? launch<EDGE, false, false, true>(p, s) : launch<EDGE, false, false, false>(p, s);
    case Layout::NT: return bf16 ? launch<EDGE, false, true, true>(p, s) : launch<EDGE, false, true, false>(p, s);
    default: return bf16 ? launch<EDGE, true, true, true>(p, s) : launch<EDGE, true, true, false>(p, s);
    }
}

}  // namespace

hipError_t launch_ring(const Product &p, Layout l, int tile, bool bf16, hipStream_t s)
{
    return tile >= 128 ? launch_layout<128>(p, l, bf16, s) : launch_layout<64>(p, l, bf16, s);
}

}  // namespace lin
}  // namespace hg
