// Internal interface of the linear layer (include/hgemm_linear.h): the
// parameters that the host passes to the kernels, and the device code the
// kernels share.  Not part of the public ABI.
#pragma once

#include <stdint.h>

#include <type_traits>
#include <utility>

#include <hip/hip_runtime.h>

#if defined(__HIPCC__)
// v_mul_legacy_f32 (an LLVM intrinsic): a product in which 0 times anything is 0.
extern "C" __device__ float hg_lin_mul_legacy(float a, float b) __asm("llvm.amdgcn.fmul.legacy");
#endif

namespace hg {

int cu_count();   // compute units of the current device (hg_fast.hip)

namespace lin {

// Activations, numbered as in the public headers.
enum { kNone = 0, kRelu = 1, kGelu = 2, kGeluTanh = 3, kSilu = 4 };
// How a matrix is stored next to the 16-bit and fp32 forms.
enum { kSaveNone = 0, kSave16 = 1, kSave8 = 2 };

constexpr int kBlock8 = 32;       // columns that share a scale in an 8-bit checkpoint

// What is done with a finished fp32 sum of products: bias, save, activation,
// residual, store.  Every pointer but C may be null.
struct Finish {
    void *C;                      // rows×cols row-major, fp32 (out32) or 16 bits
    const void *R;                // residual, same type as C; may be C itself
    const float *bias;            // cols values
    void *Z;                      // pre-activation: 16 bits (kSave16) or codes (kSave8)
    uint8_t *Zs;                  // kSave8: scale bytes, rows × ceil(cols / 32)
    int64_t ldc, ldr, ldz, ldzs;
    int32_t rows, cols;
    int32_t act, save;
    int32_t out32;
};

// One product: C[rows×cols] = Σ_k A(i, k)·B(j, k).  An operand is stored
// either k-contiguous (A[i·lda + k]) or, TA / TB, k-major (A[k·lda + i]).
struct Product {
    const uint16_t *A, *B;        // 16-byte aligned, lda and ldb multiples of 8 (not so through registers)
    int64_t lda, ldb;
    int32_t M, N, K;              // rows, cols, length of the sum
    // The first `whole` tiles (edge×edge, in the order of tile_at) are computed
    // in one piece, the others in `splits` slices of `per` 64-wide stages, each
    // of which stores its fp32 partial sums as a tile of its own: slice s of the
    // t-th such tile at P + (t·splits + s)·edge².
    int32_t edge, whole, splits, per;
    float *P;
    Finish f;
};

constexpr int kFewRows = 64;      // rows that the forms for few rows take
// Blocks of 16 rows of W that a workgroup of those takes: two where that still
// gives every CU one, and for a Z in 8 bits, whose blocks of 32 columns stay in
// one workgroup.
inline int weight_blocks(int64_t N, bool save8) { return save8 || (N + 31) / 32 >= cu_count() ? 2 : 1; }
// HIP refuses a launch of 2^32 threads: the most workgroups of 256.
constexpr int64_t kMostBlocks = 0xffffffffll / 256;

enum class Layout { NN, NT, TT };   // (TA, TB) = (0, 0), (0, 1), (1, 1)

// db = (db +) the strips' sums; strips = 0: nothing to do.
struct Strips {
    const float *Q;
    float *db;
    int64_t strips, cols;
    int32_t accumulate;
};

hipError_t launch_ring(const Product &p, int tile, bool bf16, hipStream_t s);               // 64 or 128; NN
hipError_t launch_loose(const Product &p, bool bf16, hipStream_t s);                        // 64, any A and B; NN
// x (NT) and w (TT), either of them null, and the strips' sums in one launch.
hipError_t launch_ring_pair(const Product *x, const Product *w, const Strips &b, int tile, bool bf16, hipStream_t s);
hipError_t launch_outer(const Product &p, bool bf16, hipStream_t s);                        // K <= kFewRows; TT
hipError_t launch_tile(const Product &p, Layout l, bool bf16, hipStream_t s);               // 256
// M <= kFewRows, NN; direct: A and B as Product says, odd: rows at odd elements.
hipError_t launch_rowwise(const Product &p, bool direct, bool odd, bool bf16, hipStream_t s);
// The slices' partial sums of one or two products (either may be null).
hipError_t launch_reduce(const Product *p, const Product *q, bool bf16, hipStream_t s);

// 8-bit checkpoint of X (rows×cols) and back.
hipError_t launch_write8(const void *X, int64_t ldx, uint8_t *C, int64_t ldc, uint8_t *S, int64_t lds,
                         int64_t rows, int64_t cols, bool bf16, hipStream_t s);
hipError_t launch_read8(const uint8_t *C, int64_t ldc, const uint8_t *S, int64_t lds, void *X, int64_t ldx,
                        int64_t rows, int64_t cols, bool bf16, hipStream_t s);

// A matrix copied to rows of ldd 16-bit elements with zeros behind the last
// column: 16-bit elements as they are, or the values of an 8-bit checkpoint.
struct Copy {
    const void *src;
    const uint8_t *scales;        // null: 16-bit elements
    void *dst;
    int64_t lds, ldss, ldd;
    int64_t rows, cols;           // rows = 0: nothing to copy
};
// dZ = dY·act'(Z) rounded to 16 bits (D: rows×ldd, ldd a multiple of 8, zeros
// behind the last column; null: not stored) and the column sums of the
// unrounded dZ in fp32: one row of partial sums for every strip of `strip`
// rows at Q + s·cols, or, with Q null, the result itself in db.
struct Slope {
    const void *dY;
    const void *Z;                // 16 bits or codes, by `save`
    const uint8_t *Zs;
    void *D;
    float *Q, *db;
    int64_t lddy, ldz, ldzs, ldd;
    int64_t rows, cols, strip;    // rows = 0: nothing to do
    int32_t act, save;
    int32_t accumulate;           // db is added to
};
// What the gradient's products wait for, in one launch.
hipError_t launch_prepare(const Slope &g, const Copy &x, const Copy &w, bool bf16, hipStream_t s);

// rows×cols zeros (fp32 or 16 bits).
hipError_t launch_zero(void *C, int64_t ldc, int64_t rows, int64_t cols, bool wide, hipStream_t s);

#if defined(__HIPCC__)

// A launch whose own status is returned (not what an earlier call left).
template <class... P, class... A>
hipError_t start(void (*kernel)(P...), int64_t blocks, int threads, hipStream_t s, const A &...a)
{
    return [&](P... p) {
        void *args[] = {const_cast<void *>(static_cast<const void *>(&p))...};
        return hipLaunchKernel(reinterpret_cast<const void *>(kernel), dim3((unsigned)blocks), dim3((unsigned)threads),
                               args, 0, s);
    }(a...);
}

typedef _Float16 half8 __attribute__((ext_vector_type(8)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef float floatx4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef int32_t i32x4 __attribute__((ext_vector_type(4)));
typedef short shortx4 __attribute__((ext_vector_type(4)));
// The same at any address that suits the elements: global memory takes wide
// accesses there, so rows of odd length need no slower path.
typedef uint32_t u32x4_any __attribute__((ext_vector_type(4), aligned(2)));
typedef uint32_t u32x2_any __attribute__((ext_vector_type(2), aligned(1)));
typedef float floatx4_any __attribute__((ext_vector_type(4), aligned(4)));
typedef __attribute__((address_space(3))) shortx4 lds_shortx4;
typedef __attribute__((address_space(3))) uint32_t lds_u32;

// f(std::integral_constant<int, 0>{}) ... f(std::integral_constant<int, N-1>{}).
template <class F, int... I>
__device__ __forceinline__ void static_for_impl(F &&f, std::integer_sequence<int, I...>)
{
    (f(std::integral_constant<int, I>{}), ...);
}
template <int N, class F>
__device__ __forceinline__ void static_for(F &&f)
{
    static_for_impl(f, std::make_integer_sequence<int, N>{});
}

template <bool BF16>
__device__ __forceinline__ floatx4 mfma_16x16x32(const half8 &a, const half8 &b, const floatx4 &c)
{
    if constexpr (BF16)
        return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a),
                                                       __builtin_bit_cast(bf16x8, b), c, 0, 0, 0);
    else
        return __builtin_amdgcn_mfma_f32_16x16x32_f16(a, b, c, 0, 0, 0);
}

// s_waitcnt on one counter only.
template <int n>
__device__ __forceinline__ void wait_vmcnt()
{
    __builtin_amdgcn_s_waitcnt((n & 15) | ((n >> 4) << 14) | (7 << 4) | (15 << 8));
}
template <int n>
__device__ __forceinline__ void wait_lgkmcnt()
{
    __builtin_amdgcn_s_waitcnt(15 | (3 << 14) | (7 << 4) | ((n & 15) << 8));
}

// Half a fragment of a k-major operand: 16 lanes read a 4 (k) × 16 (rows)
// block, lane l of them the 8 bytes at p (row k = l div 4, columns 4·(l mod
// 4) ..), and get the four k of row l.  The parameter's __restrict__ is what
// keeps the compiler from waiting for every buffer→LDS load in flight before
// this read, as it does where it knows nothing about the address; the ring's
// own waits and barriers order the two.
__device__ __forceinline__ shortx4 read_tr16(const lds_shortx4 *__restrict__ p)
{
    return __builtin_amdgcn_ds_read_tr16_b64_v4i16(const_cast<lds_shortx4 *>(p));
}
__device__ __forceinline__ half8 read_tr(const unsigned char *lo, const unsigned char *hi)
{
    union {
        shortx4 h[2];
        half8 v;
    } u;
    u.h[0] = read_tr16((const lds_shortx4 *)lo);
    u.h[1] = read_tr16((const lds_shortx4 *)hi);
    return u.v;
}

// Raw buffer resource: base address, no stride, `bytes` in range.
__device__ __forceinline__ i32x4 buffer_of(uint64_t base, uint32_t bytes)
{
    i32x4 r;
    r[0] = __builtin_amdgcn_readfirstlane((int)(uint32_t)base);
    r[1] = __builtin_amdgcn_readfirstlane((int)(uint32_t)(base >> 32));
    r[2] = __builtin_amdgcn_readfirstlane((int)bytes);
    r[3] = 0x00020000;
    return r;
}

// ---- The operands of the tiled product kernels: EDGE rows of A or B in
// 64-wide stages of the sum, through LDS slots filled by direct buffer→LDS
// loads of 1 KiB per wave instruction (four waves).
//
//  * k-contiguous: an LDS row holds one row's 64 k (128 bytes).  A
//    matrix-core fragment (lane l: row l mod 16 of a 16-row block, k =
//    8·(l div 16) .. +7 of a 32-wide step) is one 16-byte read.
//  * k-major: an LDS row holds one k's EDGE elements; a fragment is two
//    transposing 8-byte reads.  Both forms give a lane the same k, so either
//    pairs with either.
//  * The 16-byte chunks of an LDS row are XOR-swizzled so that the reads are
//    free of bank conflicts (64 banks of 4 bytes; measured 0 of both forms);
//    a load realises the swizzle by which chunk each lane fetches.
//  * Rows and columns past the edge get an offset past the buffer's range, and
//    stages past the end of the sum an empty range: both load zeros.  A
//    k-contiguous operand whose K is no multiple of 64 checks every chunk's k
//    (KCHK), because the bytes behind a row are another row's.
constexpr int kStage = 64;                          // k per stage
constexpr uint32_t kOutside = 0x80000000u;          // an offset past every range

template <int EDGE, bool KMAJOR>
struct Side {
    static constexpr int RB = KMAJOR ? EDGE * 2 : kStage * 2;     // bytes of an LDS row
    static constexpr int CH = RB / 16;                            // its 16-byte chunks
    static constexpr int RPI = 1024 / RB;                         // LDS rows per load instruction
    static constexpr int L = EDGE / 32;                           // load instructions per wave
    static constexpr int BYTES = EDGE * kStage * 2;               // of a slot
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

// The fragment of k-step s (32 wide) and the 16 rows from `row0` on.
template <int EDGE, bool KMAJOR>
__device__ __forceinline__ half8 fragment(const unsigned char *slot, int lane, int row0, int s)
{
    using S = Side<EDGE, KMAJOR>;
    const int frow = lane & 15, fhi = lane >> 4;
    if constexpr (!KMAJOR) {
        const unsigned char *q = slot + (row0 + frow) * S::RB;
        return *reinterpret_cast<const half8 *>(q + (((4 * s + fhi) ^ S::swz(frow)) * 16));
    } else {
        const int k = 8 * fhi + (frow >> 2);                      // + 32s and + 4 leave swz() alone
        const int c = row0 / 8 + ((lane >> 1) & 1);
        const unsigned char *q = slot + (32 * s + k) * S::RB + ((c ^ S::swz(k)) * 16) + (lane & 1) * 8;
        return read_tr(q, q + 4 * S::RB);
    }
}

// One tile's rows of an operand, as one lane loads them.
template <int EDGE, bool KMAJOR, bool KCHK>
struct Panel {
    using S = Side<EDGE, KMAJOR>;
    uint64_t base;                  // of the slice's first stage
    uint32_t step, range, row;      // bytes: per stage; in range at the first stage; per row
    int left;                       // k from the slice's first stage to the end of the sum
    uint32_t off[S::L];             // this lane's chunk of each load

    // p, ld: the operand; rows first .. of `edge` in all; the sum has K terms,
    // the slice begins at stage kt0.
    __device__ __forceinline__ void set(const uint16_t *p, int64_t ld, int first, int count, int K, int kt0, int wave,
                                        int lane)
    {
        const int edge = min(count - first, EDGE), k0 = kt0 * kStage;
        const int64_t at = KMAJOR ? (int64_t)k0 * ld + first : (int64_t)first * ld + k0;
        base = reinterpret_cast<uint64_t>(p) + (uint64_t)at * 2;
        row = (uint32_t)ld * 2;
        left = K - k0;
        step = KMAJOR ? kStage * row : kStage * 2;
        range = KMAJOR ? (uint32_t)((edge + 7) & ~7) * 2 : (uint32_t)(edge - 1) * row + (uint32_t)((left + 7) & ~7) * 2;
#pragma unroll
        for (int i = 0; i < S::L; ++i) {
            const int r = (wave * S::L + i) * S::RPI + lane / S::CH;
            const int c = (lane % S::CH) ^ S::swz(r);
            off[i] = (KMAJOR ? c * 8 < edge : r < edge) ? (uint32_t)r * row + c * 16 : kOutside;
        }
    }
    // Load i of the slice's stage kt (an empty range unless `in`) into `slot`
    // (an LDS address).
    template <class LOAD>
    __device__ __forceinline__ void issue(LOAD load, int kt, bool in, uint32_t slot, int i, int wave, int lane) const
    {
        uint32_t o = off[i], bytes;
        if constexpr (KMAJOR) {
            bytes = range + (uint32_t)(min(left - kt * kStage, kStage) - 1) * row;
        } else {
            bytes = range - (uint32_t)kt * (kStage * 2);
            if constexpr (KCHK) {
                const int r = (wave * S::L + i) * S::RPI + lane / S::CH;
                o = ((lane % S::CH) ^ S::swz(r)) * 8 < left - kt * kStage ? o : kOutside;
            }
        }
        const i32x4 r = buffer_of(base + (uint64_t)kt * step, in ? bytes : 0);
        load(r, reinterpret_cast<lds_u32 *>((uintptr_t)(slot + (wave * S::L + i) * 1024)), (int)o);
    }
};

// How a product is spread over work items.
struct Spread {
    int tiles_m, tiles_n, items;
};
// Tiles in order: bands of 4 tile rows walked column by column.
__device__ __forceinline__ void tile_at(int l, const Spread &w, int &tm, int &tn)
{
    const int band = l / (4 * w.tiles_n), first = band * 4;
    const int gsz = min(w.tiles_m - first, 4);
    const int r = l - band * 4 * w.tiles_n;
    tm = first + r % gsz;
    tn = r / gsz;
}
// Consecutive ids run on different XCDs, each with its own L2: the ids of one
// XCD take consecutive places, so that its tiles share panels.
__device__ __forceinline__ int per_xcd(int id, int total)
{
    const int per = total >> 3, rem = total & 7, x = id & 7;
    return x * per + min(x, rem) + (id >> 3);
}
// One work item: the tile at (m0, n0), stages kt0 .. of its sum; a slice's
// partial sums go to `part` (null: the whole sum).
struct Item {
    int m0, n0, kt0, nk;
    float *part;
};
template <int EDGE>
__device__ __forceinline__ Item item_at(const Product &p, const Spread &w, int id)
{
    Item t;
    int l, slice = 0;
    t.part = nullptr;
    if (id < p.whole) {
        l = per_xcd(id, p.whole);
        t.kt0 = 0;
        t.nk = (p.K + kStage - 1) / kStage;
    } else {
        const int rest = w.tiles_m * w.tiles_n - p.whole;
        const int q = per_xcd(id - p.whole, rest * p.splits);
        slice = q / rest;
        l = q - slice * rest;
        t.part = p.P + ((int64_t)l * p.splits + slice) * (EDGE * EDGE);
        l += p.whole;
        t.kt0 = slice * p.per;
        t.nk = min((p.K + kStage - 1) / kStage - t.kt0, p.per);
    }
    int tm, tn;
    tile_at(l, w, tm, tn);
    t.m0 = tm * EDGE;
    t.n0 = tn * EDGE;
    return t;
}

template <bool BF16>
__device__ __forceinline__ float widen(uint16_t h)
{
    if constexpr (BF16)
        return __builtin_bit_cast(float, (uint32_t)h << 16);
    else
        return (float)__builtin_bit_cast(_Float16, h);
}
// Rounded to nearest even.
template <bool BF16>
__device__ __forceinline__ uint16_t narrow(float v)
{
    if constexpr (BF16)
        return __builtin_bit_cast(uint16_t, (__bf16)v);
    else
        return __builtin_bit_cast(uint16_t, (_Float16)v);
}

// Eight 16-bit elements from p on: loaded, and taken later.  ODD: p
// may be at an odd element, where a wide load takes three times as long (4×2112
// ×2727 12.8 us, with 2726 6.9): then the aligned words around them are loaded
// and shifted into place.  (The word at either end holds one more element, which
// is not used, and lies in one page with them.)
template <bool ODD>
struct Raw {
    u32x4 w;
    __device__ __forceinline__ void load(const uint16_t *p) { w = *reinterpret_cast<const u32x4_any *>(p); }
    __device__ __forceinline__ u32x4 get(const uint16_t *) const { return w; }
};
template <>
struct Raw<true> {
    u32x4 w;
    uint32_t next;
    __device__ __forceinline__ void load(const uint16_t *p)
    {
        const uintptr_t a = reinterpret_cast<uintptr_t>(p), odd = a >> 1 & 1;
        const uint32_t *q = reinterpret_cast<const uint32_t *>(a - 2 * odd);
        w = *reinterpret_cast<const u32x4_any *>(q);
        next = q[3 + odd];
    }
    // p: as for load, or that plus an even number of elements.
    __device__ __forceinline__ u32x4 get(const uint16_t *p) const
    {
        const uint32_t shift = ((uint32_t)reinterpret_cast<uintptr_t>(p) & 2) * 8;
        return u32x4{__builtin_amdgcn_alignbit(w[1], w[0], shift), __builtin_amdgcn_alignbit(w[2], w[1], shift),
                     __builtin_amdgcn_alignbit(w[3], w[2], shift), __builtin_amdgcn_alignbit(next, w[3], shift)};
    }
};

// The 16-bit elements p[0 .. n-1] of eight, the others 0 (n may pass 8, or be
// none).  Short of eight, every load takes an index that is there, so that
// none of them is behind a branch and they wait for memory together.
__device__ __forceinline__ u32x4 load16x8(const void *p, int n)
{
    const uint16_t *h = static_cast<const uint16_t *>(p);
    u32x4 w = {0, 0, 0, 0};
    if (n >= 8) {
        w = *reinterpret_cast<const u32x4_any *>(h);
    } else if (n > 0) {
        uint32_t x[8];
#pragma unroll
        for (int e = 0; e < 8; ++e)
            x[e] = h[min(e, n - 1)];
#pragma unroll
        for (int e = 0; e < 8; ++e)
            w[e >> 1] |= (e < n ? x[e] : 0u) << (16 * (e & 1));
    }
    return w;
}
template <bool BF16>
__device__ __forceinline__ void load8(const void *p, int n, float (&v)[8])
{
    const u32x4 w = load16x8(p, n);
#pragma unroll
    for (int e = 0; e < 8; ++e)
        v[e] = widen<BF16>((uint16_t)(w[e >> 1] >> (16 * (e & 1))));
}
template <bool BF16>
__device__ __forceinline__ u32x4 pack8(const float (&v)[8])
{
    u32x4 w;
#pragma unroll
    for (int e = 0; e < 4; ++e)
        w[e] = (uint32_t)narrow<BF16>(v[2 * e]) | (uint32_t)narrow<BF16>(v[2 * e + 1]) << 16;
    return w;
}
template <bool BF16>
__device__ __forceinline__ void store8(void *p, int n, const float (&v)[8])
{
    uint16_t *h = static_cast<uint16_t *>(p);
    if (n >= 8) {
        *reinterpret_cast<u32x4_any *>(h) = pack8<BF16>(v);
    } else {
#pragma unroll
        for (int e = 0; e < 8; ++e)
            if (e < n)
                h[e] = narrow<BF16>(v[e]);
    }
}

// ---- Activations, all in fp32.
//
// silu(z) = z·s(z) with the logistic s; gelu_tanh(z) = z·s(2u), u =
// sqrt(2/pi)·(z + 0.044715 z³), since (1 + tanh u)/2 = s(2u).  gelu(z) =
// z·Phi(z) = max(z, 0) - |z|·(1 - Phi(|z|)), where the logarithm of the tail
// 1 - Phi is so smooth that a polynomial carries it: no reciprocal, and one
// exponential (see log2_tail).  Where a factor of z is exactly 0 the product
// is 0 (its limit) also for z = ±inf, which is what the legacy multiply does
// (0 times anything is 0); NaN passes through.  A 256×256 tile pays for its
// activation outside its matrix work (256 elements per lane at 4 cycles an
// operation, 16 for an exponential or reciprocal; 4096×8192×2048 with this GELU
// 126 us, with a rational form of 23 operations 130): the constants are folded.
// The slopes' s(1 - s) is e·s² with s = 1/(1 + e), exact to a few roundings
// where 1 - s would have lost its digits.
constexpr float kLog2e = 1.4426950408889634f;
// s(x) with x given as -x·log2(e).
__device__ __forceinline__ float logistic2(float x) { return __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(x)); }
__device__ __forceinline__ float times(float z, float w) { return hg_lin_mul_legacy(z, w); }
constexpr double kTanh2 = 1.5957691216057308;                // 2·sqrt(2/pi)
// -2u·log2(e) of gelu_tanh.
__device__ __forceinline__ float tanh_arg(float z, float z2)
{
    constexpr float c = (float)(-kTanh2 * 1.4426950408889634);
    return z * __builtin_fmaf(0.044715f * c, z2, c);
}

// log2(1 - Phi(x)), x >= 0: the polynomial of degree 8 with the least largest
// error of 1 - Phi over 0 <= x <= 5.6 (3.9e-8; 7.3e-8 in fp32; 3.1e-4 of the
// tail at most, 2e-5 up to x = 3), falling to -inf beyond.  With a step of the
// exponential (2^-25) and half a one of 1 - tail, Phi is off by 1.4e-7 at most.
__device__ __forceinline__ float log2_tail(float x)
{
    float q = -1.1976953e-6f;
    q = __builtin_fmaf(q, x, 2.0165076e-5f);
    q = __builtin_fmaf(q, x, -9.8708086e-5f);
    q = __builtin_fmaf(q, x, -3.3506381e-4f);
    q = __builtin_fmaf(q, x, 7.3009217e-3f);
    q = __builtin_fmaf(q, x, -5.2643877e-2f);
    q = __builtin_fmaf(q, x, -0.45916504f);
    q = __builtin_fmaf(q, x, -1.1511098f);
    return __builtin_fmaf(q, x, -0.99999994f);
}
// 1 - Phi(|z|).
__device__ __forceinline__ float normal_tail(float z) { return __builtin_amdgcn_exp2f(log2_tail(__builtin_fabsf(z))); }

template <int ACT>
__device__ __forceinline__ float activate(float z)
{
    if constexpr (ACT == kRelu) {
        return z < 0.0f ? 0.0f : z;
    } else if constexpr (ACT == kGelu) {
        return __builtin_fmaxf(z, 0.0f) - times(__builtin_fabsf(z), normal_tail(z));
    } else if constexpr (ACT == kGeluTanh) {
        return times(z, logistic2(tanh_arg(z, z * z)));
    } else if constexpr (ACT == kSilu) {
        return times(z, logistic2(-kLog2e * z));
    } else {
        return z;
    }
}

// dy·act'(z).
template <int ACT>
__device__ __forceinline__ float slope(float dy, float z)
{
    if constexpr (ACT == kRelu) {
        return z > 0.0f ? dy : (z <= 0.0f ? 0.0f : z);
    } else if constexpr (ACT == kGelu) {
        const float tail = normal_tail(z), cdf = z < 0.0f ? tail : 1.0f - tail;
        return dy * (cdf + times(z, 0.39894228f * __builtin_amdgcn_exp2f(-0.5f * kLog2e * z * z)));
    } else if constexpr (ACT == kGeluTanh) {
        const float z2 = z * z, e = __builtin_amdgcn_exp2f(tanh_arg(z, z2));
        const float s = __builtin_amdgcn_rcpf(1.0f + e);
        return dy * (s + times(z * __builtin_fmaf((float)(3 * 0.044715 * kTanh2), z2, (float)kTanh2), times(e, s * s)));
    } else if constexpr (ACT == kSilu) {
        const float e = __builtin_amdgcn_exp2f(-kLog2e * z);
        const float s = __builtin_amdgcn_rcpf(1.0f + e);
        return dy * (s + times(z, times(e, s * s)));
    } else {
        return dy;
    }
}

// f(std::integral_constant<int, act>{}), act uniform.
template <class F>
__device__ __forceinline__ void with_act(int act, F &&f)
{
    switch (act) {
    case kRelu: f(std::integral_constant<int, kRelu>{}); break;
    case kGelu: f(std::integral_constant<int, kGelu>{}); break;
    case kGeluTanh: f(std::integral_constant<int, kGeluTanh>{}); break;
    case kSilu: f(std::integral_constant<int, kSilu>{}); break;
    default: f(std::integral_constant<int, kNone>{}); break;
    }
}

// ---- 8-bit checkpoints.  A block of 32 columns shares the scale 2^e, e the
// smallest exponent with amax <= 448·2^e over the block's finite elements
// (448 is e4m3's largest value), so no element saturates.  A power of two
// makes x·2^-e exact: the only rounding is the one to e4m3.  e is kept where
// every code stands for a normal value of the element type (bf16: e >= -117)
// or an exact one (fp16: -15 <= e <= 8); at the largest e (8, bf16: 120) codes
// stop at 240, because 256·2^e is past the type's range.
template <bool BF16>
__device__ __forceinline__ int scale_exponent(float amax)
{
    const uint32_t b = __builtin_bit_cast(uint32_t, amax);
    const int e = (int)(b >> 23) - 135 + ((b & 0x7fffffu) > 0x600000u ? 1 : 0);
    return BF16 ? max(e, -117) : min(max(e, -15), 8);
}
// The largest of four neighbouring lanes' values (lanes 4i .. 4i + 3).
__device__ __forceinline__ float max_of_4(float v)
{
    const int a = __builtin_bit_cast(int, v);
    v = __builtin_fmaxf(v, __builtin_bit_cast(float, __builtin_amdgcn_mov_dpp(a, 0xb1, 0xf, 0xf, true)));   // 1 0 3 2
    const int b = __builtin_bit_cast(int, v);
    return __builtin_fmaxf(v, __builtin_bit_cast(float, __builtin_amdgcn_mov_dpp(b, 0x4e, 0xf, 0xf, true)));  // 2 3 0 1
}

__device__ __forceinline__ uint32_t pack_codes(float a, float b, float c, float d)
{
    const int w = __builtin_amdgcn_cvt_pk_fp8_f32(a, b, 0, false);
    return (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(c, d, w, true);
}
// One eighth of a block per lane, four neighbouring lanes to a block: the
// codes of the first n values and the block's exponent (returned).
//
// Ordinarily an element costs a multiplication, half a conversion and half of
// a three-way maximum: the maximum skips NaN, the conversion turns NaN into a
// NaN code, and nothing can pass 448 (see scale_exponent).  Blocks with an
// infinity or at the largest exponent go the long way.
template <bool BF16>
__device__ __forceinline__ int encode8(const float (&v)[8], int n, u32x2 &w)
{
    // the largest magnitude whose exponent is below the largest, 448·2^(emax - 1)
    constexpr float ordinary = BF16 ? 448.0f * 0x1p119f : 448.0f * 0x1p7f;
    float a = 0.0f;
#pragma unroll
    for (int e = 0; e < 8; ++e)
        a = __builtin_fmaxf(a, e < n ? __builtin_fabsf(v[e]) : 0.0f);
    a = max_of_4(a);
    if (__builtin_expect(a <= ordinary, 1)) {
        const int x = scale_exponent<BF16>(a);
        const float inv = __builtin_bit_cast(float, (uint32_t)(127 - x) << 23);
#pragma unroll
        for (int i = 0; i < 2; ++i)
            w[i] = pack_codes(v[4 * i] * inv, v[4 * i + 1] * inv, v[4 * i + 2] * inv, v[4 * i + 3] * inv);
        return x;
    }
    a = 0.0f;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        const float m = __builtin_fabsf(v[e]);
        a = e < n && m < __builtin_inff() ? __builtin_fmaxf(a, m) : a;
    }
    const int x = scale_exponent<BF16>(max_of_4(a));
    const float inv = __builtin_bit_cast(float, (uint32_t)(127 - x) << 23);
    const float lim = x == (BF16 ? 120 : 8) ? 240.0f : 448.0f;
    float s[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const float c = __builtin_fminf(__builtin_fmaxf(v[i] * inv, -lim), lim);
        s[i] = __builtin_fabsf(v[i]) < __builtin_inff() ? c : __builtin_nanf("");
    }
#pragma unroll
    for (int i = 0; i < 2; ++i)
        w[i] = pack_codes(s[4 * i], s[4 * i + 1], s[4 * i + 2], s[4 * i + 3]);
    return x;
}
// 2^(byte - 127); byte 0 stands for 2^-127 and 255 for NaN.
__device__ __forceinline__ float scale_of(uint32_t byte)
{
    const uint32_t b = byte == 0 ? 0x00400000u : byte == 255 ? 0x7fc00000u : byte << 23;
    return __builtin_bit_cast(float, b);
}
__device__ __forceinline__ void values8(u32x2 w, float scale, float (&v)[8])
{
    typedef float floatx2 __attribute__((ext_vector_type(2)));
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const floatx2 lo = __builtin_amdgcn_cvt_pk_f32_fp8((int)w[i], false);
        const floatx2 hi = __builtin_amdgcn_cvt_pk_f32_fp8((int)w[i], true);
        v[4 * i] = lo[0] * scale;
        v[4 * i + 1] = lo[1] * scale;
        v[4 * i + 2] = hi[0] * scale;
        v[4 * i + 3] = hi[1] * scale;
    }
}
__device__ __forceinline__ u32x2 load_codes(const uint8_t *p, int n)
{
    u32x2 w = {0, 0};
    if (n >= 8) {
        w = *reinterpret_cast<const u32x2_any *>(p);
    } else if (n > 0) {
        uint32_t x[8];
#pragma unroll
        for (int e = 0; e < 8; ++e)
            x[e] = p[min(e, n - 1)];
#pragma unroll
        for (int e = 0; e < 8; ++e)
            w[e >> 2] |= (e < n ? x[e] : 0u) << (8 * (e & 3));
    }
    return w;
}
__device__ __forceinline__ void store_codes(uint8_t *p, int n, u32x2 w)
{
    if (n >= 8) {
        *reinterpret_cast<u32x2_any *>(p) = w;
        return;
    }
#pragma unroll
    for (int e = 0; e < 8; ++e)
        if (e < n)
            p[e] = (uint8_t)(w[e >> 2] >> (8 * (e & 3)));
}
// Finishes eight consecutive columns col .. col + 7 (col a multiple of 8) of
// one row, `b` their biases.  Called by whole waves in which lanes 4i .. 4i + 3
// hold the four eighths of one block of 32 columns (an 8-bit save takes their
// largest); lanes past the last row or column store nothing.
template <bool BF16>
__device__ __forceinline__ void finish8(const Finish &f, int row, int col, float (&v)[8], const float (&b)[8])
{
    const bool in = row < f.rows;
    const int n = in ? f.cols - col : 0;          // columns of this lane (may pass 8)
    if (f.bias) {
#pragma unroll
        for (int e = 0; e < 8; ++e)
            v[e] += b[e];
    }
    if (f.save == kSave16) {
        if (n > 0)
            store8<BF16>(static_cast<uint16_t *>(f.Z) + (int64_t)row * f.ldz + col, n, v);
    } else if (f.save == kSave8) {
        u32x2 w;
        const int x = encode8<BF16>(v, n, w);
        if (n > 0) {
            store_codes(static_cast<uint8_t *>(f.Z) + (int64_t)row * f.ldz + col, n, w);
            if (col % kBlock8 == 0)
                f.Zs[(int64_t)row * f.ldzs + col / kBlock8] = (uint8_t)(x + 127);
        }
    }
    if (n <= 0)
        return;
    with_act(f.act, [&](auto a) __attribute__((always_inline)) {
#pragma unroll
        for (int e = 0; e < 8; ++e)
            v[e] = activate<decltype(a)::value>(v[e]);
    });
    if (f.out32) {
        float *c = static_cast<float *>(f.C) + (int64_t)row * f.ldc + col;
        const float *r = static_cast<const float *>(f.R) + (int64_t)row * f.ldr + col;
        if (f.R) {
            if (n >= 8) {
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const floatx4 w = *reinterpret_cast<const floatx4_any *>(r + 4 * h);
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        v[4 * h + e] += w[e];
                }
            } else {
                float w[8];
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    w[e] = r[min(e, n - 1)];
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    v[e] += e < n ? w[e] : 0.0f;
            }
        }
        if (n >= 8) {
            *reinterpret_cast<floatx4_any *>(c) = floatx4{v[0], v[1], v[2], v[3]};
            *reinterpret_cast<floatx4_any *>(c + 4) = floatx4{v[4], v[5], v[6], v[7]};
        } else {
#pragma unroll
            for (int e = 0; e < 8; ++e)
                if (e < n)
                    c[e] = v[e];
        }
    } else {
        if (f.R) {
            float r[8];
            load8<BF16>(static_cast<const uint16_t *>(f.R) + (int64_t)row * f.ldr + col, n, r);
#pragma unroll
            for (int e = 0; e < 8; ++e)
                v[e] += r[e];
        }
        store8<BF16>(static_cast<uint16_t *>(f.C) + (int64_t)row * f.ldc + col, n, v);
    }
}

// The biases of columns col .. col + 7 (past the last: its, not used).
__device__ __forceinline__ void load_bias(const Finish &f, int col, float (&b)[8])
{
    if (f.bias) {
#pragma unroll
        for (int e = 0; e < 8; ++e)
            b[e] = f.bias[min(col + e, f.cols - 1)];
    } else {
#pragma unroll
        for (int e = 0; e < 8; ++e)
            b[e] = 0.0f;
    }
}

// Waits for the biases here: otherwise the compiler waits for them inside the
// epilogue's loop, and with them for every store of the passes before.
__device__ __forceinline__ void settle(float (&b)[8])
{
#pragma unroll
    for (int e = 0; e < 8; ++e)
        __asm__ volatile("" : "+v"(b[e]));
}

// ---- Wave-private staging of a 16×W block of sums (fp32) in LDS, from the
// matrix cores' layout (a lane holds columns 16j + 4·(lane div 16) .. +3 of
// row lane mod 16) to eight consecutive columns per lane.  The 16-byte piece
// index is XORed with the row so that neither side has bank conflicts.
template <int W>
__device__ __forceinline__ int stage_at(int row, int piece)
{
    constexpr int PIECES = W / 4;                            // per row
    const int x = W >= 64 ? row & 15 : (row >> 1) & 7;
    return (row * PIECES + (piece ^ (x & (PIECES - 1)))) * 16;
}
template <int W>
__device__ __forceinline__ void stage_put(unsigned char *s, int lane, const floatx4 (&acc)[W / 16])
{
    const int frow = lane & 15, fhi = lane >> 4;
#pragma unroll
    for (int j = 0; j < W / 16; ++j)
        *reinterpret_cast<floatx4 *>(s + stage_at<W>(frow, 4 * j + fhi)) = acc[j];
}
template <int W>
__device__ __forceinline__ void stage_get(const unsigned char *s, int row, int unit, float (&v)[8])
{
    const floatx4 lo = *reinterpret_cast<const floatx4 *>(s + stage_at<W>(row, 2 * unit));
    const floatx4 hi = *reinterpret_cast<const floatx4 *>(s + stage_at<W>(row, 2 * unit + 1));
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        v[e] = lo[e];
        v[4 + e] = hi[e];
    }
}

// Finishes (or, of a slice of the sum, stores as fp32) staged 16×W blocks of one
// wave, one after the other down the item's tile: columns c0 .., rows `row0` ..
// in steps of 16.
//
// A block inside the matrix takes its passes together: the
// reads from LDS, the activation's chains and the stores of PASSES rows per
// lane overlap, and what depends on the call (save, activation, type) is
// decided once per block, not per row.  The residual of the next block is
// requested before this block's stores, because the counter of vector memory
// operations retires in order: a load issued after them would wait for them.
//
// PAST: what is written passes the caches by.  A large product's results are
// more than they hold, and they hold its operands (256×256 tiles, 4096×8192×
// 2048: gradient 272 -> 263 us; with Z 8192×16384×4096 823 -> 817).
template <int EDGE, int W, bool BF16, bool PAST = EDGE == 256>
struct Drain {
    static constexpr int UNITS = W / 8, ROWS = 64 / UNITS;      // lanes per row, rows per pass
    static constexpr int PASSES = 16 / ROWS;
    const Product &p;
    const unsigned char *stg;
    int lane, c0, m0, n0;
    float *part;
    float bias[8];
    u32x4 ahead[PASSES][2];                                     // residual of the next block

    __device__ __forceinline__ Drain(const Product &p_, const Item &t, const unsigned char *stg_, int lane_, int c0_)
        : p(p_), stg(stg_), lane(lane_), c0(c0_), m0(t.m0), n0(t.n0), part(t.part)
    {
        load_bias(p.f, c0 + 8 * (lane % UNITS), bias);
    }
    template <class V, class U>
    __device__ __forceinline__ void put(void *to, U v) const
    {
        if constexpr (PAST)
            __builtin_nontemporal_store((V)v, static_cast<V *>(to));
        else
            *static_cast<V *>(to) = v;
    }
    // Whether no row of the block is outside the matrix and each lane's columns
    // (an 8-bit save: its four neighbours' too) are all in it or all outside.
    // Smaller tiles' blocks have fewer passes to gain and are either in or not
    // (256×256: 4000×4000×1000 47.9 -> 40.2 us, 1729×5000×4000 91.5 -> 83.3; 64×64:
    // 1000×1000×1000 10.1 -> 10.3).
    __device__ __forceinline__ bool even(int row0) const
    {
        const int unit = part ? 1 : p.f.save == kSave8 ? kBlock8 : 8;
        return row0 + 16 <= p.M && (c0 + W <= p.N || (EDGE == 256 && p.N % unit == 0));
    }
    __device__ __forceinline__ bool mine() const { return EDGE != 256 || c0 + 8 * (lane % UNITS) < p.N; }
    // Requests the residual of the block at row0.
    __device__ __forceinline__ void request(int row0)
    {
        const Finish &f = p.f;
        if (!f.R || part || !even(row0) || !mine())
            return;
        const int64_t at = (int64_t)(row0 + lane / UNITS) * f.ldr + c0 + 8 * (lane % UNITS);
        const char *r = static_cast<const char *>(f.R) + at * (f.out32 ? 4 : 2);
        const int64_t step = ROWS * f.ldr * (f.out32 ? 4 : 2);
#pragma unroll
        for (int t = 0; t < PASSES; ++t, r += step) {
            ahead[t][0] = *reinterpret_cast<const u32x4_any *>(r);
            if (f.out32)
                ahead[t][1] = *reinterpret_cast<const u32x4_any *>(r + 16);
        }
    }
    __device__ __forceinline__ void block(int row0, bool last)
    {
        if (EDGE == 256 && (row0 >= p.M || c0 >= p.N))
            return;
        if (!even(row0))
            edge(row0);
        else if (mine())
            whole(row0, last);
    }
    __device__ __forceinline__ void whole(int row0, bool last)
    {
        const Finish &f = p.f;
        const int unit = lane % UNITS, r0 = lane / UNITS, col = c0 + 8 * unit;
        float v[PASSES][8];
#pragma unroll
        for (int t = 0; t < PASSES; ++t)
            stage_get<W>(stg, r0 + ROWS * t, unit, v[t]);
        const int64_t row = row0 + r0;
        if (part) {
            float *d = part + (row0 + r0 - m0) * EDGE + col - n0;
#pragma unroll
            for (int t = 0; t < PASSES; ++t, d += ROWS * EDGE) {
                *reinterpret_cast<floatx4 *>(d) = floatx4{v[t][0], v[t][1], v[t][2], v[t][3]};
                *reinterpret_cast<floatx4 *>(d + 4) = floatx4{v[t][4], v[t][5], v[t][6], v[t][7]};
            }
            return;
        }
        if (f.bias) {
#pragma unroll
            for (int t = 0; t < PASSES; ++t)
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    v[t][e] += bias[e];
        }
        if (f.save == kSave16) {
            uint16_t *z = static_cast<uint16_t *>(f.Z) + row * f.ldz + col;
#pragma unroll
            for (int t = 0; t < PASSES; ++t, z += ROWS * f.ldz)
                put<u32x4_any>(z, pack8<BF16>(v[t]));
        } else if (f.save == kSave8) {
            uint8_t *z = static_cast<uint8_t *>(f.Z) + row * f.ldz + col, *zs = f.Zs + row * f.ldzs + col / kBlock8;
#pragma unroll
            for (int t = 0; t < PASSES; ++t, z += ROWS * f.ldz, zs += ROWS * f.ldzs) {
                u32x2 w;
                const int x = encode8<BF16>(v[t], 8, w);
                put<u32x2_any>(z, w);
                if (unit % 4 == 0)
                    *zs = (uint8_t)(x + 127);
            }
        }
        with_act(f.act, [&](auto a) __attribute__((always_inline)) {
#pragma unroll
            for (int t = 0; t < PASSES; ++t)
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    v[t][e] = activate<decltype(a)::value>(v[t][e]);
        });
        if (f.R) {
#pragma unroll
            for (int t = 0; t < PASSES; ++t)
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    const uint32_t w32 = ahead[t][e >> 2][e & 3], w16 = ahead[t][0][e >> 1] >> (16 * (e & 1));
                    v[t][e] += f.out32 ? __builtin_bit_cast(float, w32) : widen<BF16>((uint16_t)w16);
                }
            if (!last)
                request(row0 + 16);
        }
        if (f.out32) {
            float *c = static_cast<float *>(f.C) + row * f.ldc + col;
#pragma unroll
            for (int t = 0; t < PASSES; ++t, c += ROWS * f.ldc) {
                put<floatx4_any>(c, floatx4{v[t][0], v[t][1], v[t][2], v[t][3]});
                put<floatx4_any>(c + 4, floatx4{v[t][4], v[t][5], v[t][6], v[t][7]});
            }
        } else {
            uint16_t *c = static_cast<uint16_t *>(f.C) + row * f.ldc + col;
#pragma unroll
            for (int t = 0; t < PASSES; ++t, c += ROWS * f.ldc)
                put<u32x4_any>(c, pack8<BF16>(v[t]));
        }
    }
    __device__ __forceinline__ void edge(int row0)
    {
        const int unit = lane % UNITS, col = c0 + 8 * unit;
#pragma clang loop unroll(disable)
        for (int r = lane / UNITS; r < 16; r += ROWS) {
            float v[8];
            stage_get<W>(stg, r, unit, v);
            const int row = row0 + r;
            if (part) {
                if (row < p.M && col < p.N) {
                    float *d = part + (row - m0) * EDGE + col - n0;
                    *reinterpret_cast<floatx4 *>(d) = floatx4{v[0], v[1], v[2], v[3]};
                    *reinterpret_cast<floatx4 *>(d + 4) = floatx4{v[4], v[5], v[6], v[7]};
                }
            } else {
                finish8<BF16>(p.f, row, col, v, bias);
            }
        }
    }
};

#endif  // __HIPCC__

}  // namespace lin
}  // namespace hg
