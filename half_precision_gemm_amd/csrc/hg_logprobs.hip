// hg_logprobs.hip — log probabilities, entropy and the most probable tokens of
// rows of logits, and their gradient (gfx950).
//
// With x* the largest logit of a row, d_j = scale·(x_j - x*), S = Σ e^d_j:
//
//     log p_j = d_j - log S,   H = -Σ p·log p = log S - (Σ d_j·e^d_j) / S
//     dx_j = scale·(dl·(1[j = token] - p_j) - dh·p_j·(log p_j + H))
//
// Forward: one reading of the logits, for a dozen operations on each; what bounds
// it is HBM where rows are many, and launches and latency where they are few.  A
// row is cut into parts; a workgroup holds its part in registers (up to 64 logits
// a lane), so that the maximum is known before the first exponential (no running
// rescale) and the most probable tokens are looked for without a second reading.
// A second launch joins a row's parts, one wave to a row.  The sums of a part are
// relative to its waves' maxima and are brought to one reference as they are
// joined, always in the same order.
//
// The most probable k of a part: a threshold that at least k of the lanes' maxima
// reach is found by bisection over their bits (counted with ballots), so k
// elements reach it and only lanes counted can hold others that do: at most
// kLanes·64 candidates, ordinarily k and a few.  They are ordered by (logit,
// lower number first), each counting the candidates before it.  Equal maxima are
// told apart by where their group of eight lies, in the same order.
//
// Groups of eight logits lie at multiples of 16 bytes (32 of fp32) in memory
// whatever the row's address is, so every load is a whole one; what a row's first
// and last group hold of its neighbours (or of nothing: in the same 32 bytes as a
// logit, so in its page) counts as -inf.
#include "hg_logprobs.h"

#include "hgemm.h"
#include "hg_linear.h"

namespace hg {
namespace probs {
namespace {

using lin::floatx4;
using lin::start;
using lin::u32x4;

constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.69314718055994531f;
constexpr float kFar = -200.0f;                   // 2^kFar is 0 in fp32, and 0·kFar is 0
constexpr int kSpare = 8, kLanes = 32 + kSpare;   // lanes that may hold candidates
static_assert(HG_BF16 == 2 && HG_F16 == 0 && HG_F32 == 1, "");

template <int TYPE>
constexpr int kSize = TYPE == HG_F32 ? 4 : 2;
// Lowest bit of ordered() in which values of the type differ.
template <int TYPE>
constexpr int kLowBit = TYPE == HG_F32 ? 0 : TYPE == HG_F16 ? 13 : 16;

// fp32 as whole numbers in the same order, zeros of either sign alike.
__device__ __forceinline__ uint32_t ordered(float v)
{
    const uint32_t b = __builtin_bit_cast(uint32_t, v + 0.0f);
    return b ^ ((uint32_t)((int32_t)b >> 31) | 0x80000000u);
}
__device__ __forceinline__ float unordered(uint32_t u)
{
    return __builtin_bit_cast(float, u & 0x80000000u ? u ^ 0x80000000u : ~u);
}
__device__ __forceinline__ float without_nan(float v) { return __builtin_fmaxf(v, -__builtin_inff()); }

// Eight logits as they lie in memory.
template <int TYPE>
struct Group {
    u32x4 w[kSize<TYPE> / 2];
    __device__ __forceinline__ void load(const char *p)
    {
#pragma unroll
        for (int i = 0; i < kSize<TYPE> / 2; ++i)
            w[i] = reinterpret_cast<const u32x4 *>(p)[i];
    }
    __device__ __forceinline__ float at(int e) const
    {
        // (a copy: of a vector's element as it stands the compiler casts the first)
        const uint32_t u = w[TYPE == HG_F32 ? e >> 2 : 0][TYPE == HG_F32 ? e & 3 : e >> 1];
        if constexpr (TYPE == HG_F32)
            return __builtin_bit_cast(float, u);
        else
            return lin::widen<TYPE == HG_BF16>((uint16_t)(u >> (16 * (e & 1))));
    }
    // -inf outside elements 0 .. V-1, the group's first being `first`.
    __device__ __forceinline__ void cut(int first, int V)
    {
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const bool in = (unsigned)(first + e) < (unsigned)V;
            if constexpr (TYPE == HG_F32) {
                w[e >> 2][e & 3] = in ? w[e >> 2][e & 3] : 0xff800000u;
            } else {
                const uint32_t none = TYPE == HG_BF16 ? 0xff80u : 0xfc00u, keep = e & 1 ? 0xffffu : 0xffff0000u;
                w[0][e >> 1] = in ? w[0][e >> 1] : (w[0][e >> 1] & keep) | none << (16 * (e & 1));
            }
        }
    }
};

// Where a row's groups begin, and how many elements of the first are before it.
template <int TYPE>
__device__ __forceinline__ const char *first_group(const void *X, int64_t ld, int64_t row, int &head)
{
    const char *p = static_cast<const char *>(X) + row * ld * kSize<TYPE>;
    head = (int)(reinterpret_cast<uintptr_t>(p) / kSize<TYPE>) & (kGroup - 1);
    return p - head * kSize<TYPE>;
}

__device__ __forceinline__ float max_of_wave(float v)
{
#pragma unroll
    for (int d = 1; d < 64; d *= 2)
        v = __builtin_fmaxf(v, __shfl_xor(v, d));
    return v;
}
__device__ __forceinline__ float sum_of_wave(float v)
{
#pragma unroll
    for (int d = 1; d < 64; d *= 2)
        v += __shfl_xor(v, d);
    return v;
}

// Sums relative to `from` added to ones relative to `to` >= from: sum = Σ 2^d,
// weighted = Σ d·2^d, d = c·(x - reference).
__device__ __forceinline__ void join(float from, float s, float t, float to, float c, float &sum, float &weighted)
{
    const float d = __builtin_fmaxf((from - to) * c, kFar), w = __builtin_amdgcn_exp2f(d);
    sum += s * w;                                 // (NaN stays NaN; of nothing, -inf, s is 0)
    weighted += w * (t + d * s);
}

// A threshold (least, lowest) that at least k and, if the keys are all different,
// at most `most` >= k of the wave's E·64 keys (hi, then lo) reach, by their bits
// from the highest on; hi's from 31 - `low` on.  Keys with hi = 0 are none.
template <int E>
__device__ __forceinline__ void threshold(const uint32_t (&hi)[E], const uint32_t (&lo)[E], int bits, int k, int most,
                                          uint32_t &least, uint32_t &lowest)
{
    auto count = [&](auto reaches) __attribute__((always_inline)) {
        int n = 0;
#pragma unroll
        for (int i = 0; i < E; ++i)
            n += __builtin_popcountll(__builtin_amdgcn_ballot_w64(reaches(i)));
        return n;
    };
    least = lowest = 0;
    int n = E * 64;
    for (uint32_t bit = 1u << (bits - 1); bit != 0 && n > most; bit >>= 1) {
        const uint32_t to = least | bit;
        const int m = count([&](int i) { return hi[i] >= to; });
        if (m >= k) {
            least = to;
            n = m;
        }
    }
    if (n <= most)
        return;
    const int above = count([&](int i) { return hi[i] > least; });
    for (uint32_t bit = 1u << 31; bit != 0 && n > most; bit >>= 1) {
        const uint32_t to = lowest | bit;
        const int m = above + count([&](int i) { return hi[i] == least && lo[i] >= to; });
        if (m >= k) {
            lowest = to;
            n = m;
        }
    }
}

// What a whole row is known by.
struct Row {
    float largest, logsum;
    bool nothing;                                 // all logits -inf
    __device__ __forceinline__ float logp(float x, float scale) const
    {
        return nothing ? -__builtin_inff() : (x - largest) * scale - logsum;
    }
};
template <int TYPE>
__device__ __forceinline__ Row finish(const Forward &f, int64_t row, float largest, float sum, float weighted, bool writes)
{
    Row r;
    r.largest = largest;
    r.nothing = sum == 0.0f;
    r.logsum = logf(sum);
    if (writes) {
        if (f.stats) {
            f.stats[2 * row] = largest;
            f.stats[2 * row + 1] = r.logsum;
        }
        if (f.entropy)
            f.entropy[row] = r.nothing ? 0.0f : r.logsum - weighted * kLn2 / sum;
        if (f.logp) {
            const int64_t t = f.tokens[row];
            float l = 0.0f;
            if (t >= 0 && t < f.V) {
                const char *x = static_cast<const char *>(f.X) + (row * f.ldx + t) * kSize<TYPE>;
                float v;
                if constexpr (TYPE == HG_F32)
                    v = *reinterpret_cast<const float *>(x);
                else
                    v = lin::widen<TYPE == HG_BF16>(*reinterpret_cast<const uint16_t *>(x));
                l = r.logp(v, f.scale);
            }
            f.logp[row] = l;
        }
    }
    return r;
}
// The `place`-th most probable token.  (A NaN was taken for -inf among the keys,
// and makes logsum, so its log probability, NaN.)
__device__ __forceinline__ void put_top(const Forward &f, int64_t row, const Row &r, int place, uint64_t key)
{
    const int64_t at = row * f.top + place;
    if (f.top_ids)
        f.top_ids[at] = (uint32_t)~(uint32_t)key;
    if (f.top_logp)
        f.top_logp[at] = r.logp(unordered((uint32_t)(key >> 32)), f.scale);
}

template <int GR, int TYPE, bool TOP>
__global__ void __launch_bounds__(kThreads) part_kernel(const Forward f)
{
    constexpr int WAVES = kThreads / 64, MOST = kLanes * GR * kGroup;
    __shared__ float wave_sums[WAVES][3];
    __shared__ uint32_t best_hi[TOP ? kThreads : 1], best_lo[TOP ? kThreads : 1];
    __shared__ uint64_t found[TOP ? MOST : 1];
    __shared__ int count;
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int64_t items = f.M * f.parts.parts;
    const float c = f.scale * kLog2e;
    for (int64_t item = blockIdx.x; item < items; item += gridDim.x) {
        const int64_t row = item / f.parts.parts;
        const int part = (int)(item - row * f.parts.parts);
        int head;
        const char *p = first_group<TYPE>(f.X, f.ldx, row, head);
        const int groups = (head + f.V + kGroup - 1) / kGroup;               // of the row
        const int g0 = part * f.parts.per, n = min(groups - g0, f.parts.per);       // this part's
        Group<TYPE> x[GR];
        // Groups past the last are loaded as the last and not looked at; of a whole
        // wave none are.
        auto any = [&](int i) { return i * kThreads + wave * 64 < n; };
#pragma unroll
        for (int i = 0; i < GR; ++i)
            if (any(i))
                x[i].load(p + (int64_t)(g0 + min(i * kThreads + (int)threadIdx.x, n - 1)) * (kGroup * kSize<TYPE>));
        float best = -__builtin_inff();
        int best_at = g0 + threadIdx.x;
#pragma unroll
        for (int i = 0; i < GR; ++i) {
            if (!any(i))
                continue;
            const int at = i * kThreads + threadIdx.x, first = (g0 + at) * kGroup - head;
            if (first < 0 || first + kGroup > f.V || at >= n)
                x[i].cut(at < n ? first : f.V, f.V);
            float m = x[i].at(0);
#pragma unroll
            for (int e = 1; e < 8; ++e)
                m = __builtin_fmaxf(m, x[i].at(e));
            best_at = m > best ? g0 + at : best_at;
            best = __builtin_fmaxf(best, m);
        }
        const float m = max_of_wave(best), zero = m == -__builtin_inff() ? 0.0f : m;
        float sum = 0.0f, weighted = 0.0f;
#pragma unroll
        for (int i = 0; i < GR; ++i) {
            if (!any(i))
                continue;
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const float d = (x[i].at(e) - zero) * c, w = __builtin_amdgcn_exp2f(d);
                sum += w;
                weighted = __builtin_fmaf(__builtin_fmaxf(d, kFar), w, weighted);
            }
        }
        sum = sum_of_wave(sum);
        weighted = sum_of_wave(weighted);
        if (lane == 0) {
            wave_sums[wave][0] = m;
            wave_sums[wave][1] = sum;
            wave_sums[wave][2] = weighted;
        }
        if constexpr (TOP) {
            best_hi[threadIdx.x] = (int)threadIdx.x < n ? ordered(best) >> kLowBit<TYPE> : 0;
            best_lo[threadIdx.x] = ~(uint32_t)best_at;
            if (threadIdx.x == 0)
                count = 0;
        }
        __syncthreads();
        float largest = wave_sums[0][0], s = 0.0f, t = 0.0f;
#pragma unroll
        for (int i = 1; i < WAVES; ++i)
            largest = __builtin_fmaxf(largest, wave_sums[i][0]);
        const float to = largest == -__builtin_inff() ? 0.0f : largest;
#pragma unroll
        for (int i = 0; i < WAVES; ++i)
            join(wave_sums[i][0], wave_sums[i][1], wave_sums[i][2], to, c, s, t);
        const bool whole = f.parts.parts == 1;
        Row r{};
        if (whole)
            r = finish<TYPE>(f, row, largest, s, t, threadIdx.x == 0);
        else if (threadIdx.x == 0)
            f.partials[item] = {largest, s, t, 0.0f};
        if constexpr (TOP) {
            uint32_t hi[WAVES], lo[WAVES], least, lowest;
#pragma unroll
            for (int i = 0; i < WAVES; ++i) {
                hi[i] = best_hi[i * 64 + lane];
                lo[i] = best_lo[i * 64 + lane];
            }
            threshold<WAVES>(hi, lo, 32 - kLowBit<TYPE>, f.top, f.top + kSpare, least, lowest);
            uint64_t *keys = f.keys + item * f.top;
            // the lanes with candidates look for them
            const uint32_t mine = (int)threadIdx.x < n ? ordered(best) >> kLowBit<TYPE> : 0;
            if (mine > least || (mine == least && ~(uint32_t)best_at >= lowest)) {
#pragma unroll
                for (int i = 0; i < GR; ++i) {
                    const int at = i * kThreads + threadIdx.x, first = (g0 + at) * kGroup - head;
                    if (at >= n)
                        continue;
#pragma unroll
                    for (int e = 0; e < 8; ++e) {
                        const uint32_t u = ordered(without_nan(x[i].at(e))), h = u >> kLowBit<TYPE>;
                        const bool in = (unsigned)(first + e) < (unsigned)f.V;
                        if (in && (h > least || (h == least && ~(uint32_t)(g0 + at) >= lowest)))
                            found[atomicAdd(&count, 1)] = (uint64_t)u << 32 | ~(uint32_t)(first + e);
                    }
                }
            }
            __syncthreads();
            const int all = count;
            for (int i = threadIdx.x; i < all; i += kThreads) {
                const uint64_t key = found[i];
                int place = 0;
                for (int j = 0; j < all; ++j)
                    place += found[j] > key;
                if (place < f.top) {
                    if (whole)
                        put_top(f, row, r, place, key);
                    else
                        keys[place] = key;
                }
            }
            if (!whole)                           // fewer elements than `top`
                for (int i = all + threadIdx.x; i < f.top; i += kThreads)
                    keys[i] = 0;
        }
        __syncthreads();
    }
}

// One wave joins a row's parts; E·64 keys at most.
template <int E, int TYPE>
__global__ void __launch_bounds__(kThreads) join_kernel(const Forward f)
{
    __shared__ uint64_t found[kThreads / 64][64];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, parts = f.parts.parts;
    const float c = f.scale * kLog2e;
    for (int64_t row = (int64_t)blockIdx.x * (kThreads / 64) + wave; row < f.M; row += (int64_t)gridDim.x * (kThreads / 64)) {
        const Partial none{-__builtin_inff(), 0.0f, 0.0f, 0.0f};
        const Partial a = lane < parts ? f.partials[row * parts + lane] : none;
        const Partial b = lane + 64 < parts ? f.partials[row * parts + lane + 64] : none;
        const float largest = max_of_wave(__builtin_fmaxf(a.largest, b.largest));
        const float to = largest == -__builtin_inff() ? 0.0f : largest;
        float s = 0.0f, t = 0.0f;
        join(a.largest, a.sum, a.weighted, to, c, s, t);
        join(b.largest, b.sum, b.weighted, to, c, s, t);
        const Row r = finish<TYPE>(f, row, largest, sum_of_wave(s), sum_of_wave(t), lane == 0);
        if (f.top == 0)
            continue;
        const uint64_t *keys = f.keys + row * parts * f.top;
        const int all = parts * f.top;
        uint32_t hi[E], lo[E], least, lowest;
#pragma unroll
        for (int i = 0; i < E; ++i) {
            const uint64_t k = 64 * i + lane < all ? keys[64 * i + lane] : 0;
            hi[i] = (uint32_t)(k >> 32);
            lo[i] = (uint32_t)k;
        }
        // the keys are all different, so that at most 64 are left
        threshold<E>(hi, lo, 32, f.top, 64, least, lowest);
        int n = 0;
#pragma unroll
        for (int i = 0; i < E; ++i) {
            const bool in = hi[i] != 0 && (hi[i] > least || (hi[i] == least && lo[i] >= lowest));
            const uint64_t who = __builtin_amdgcn_ballot_w64(in);
            if (in)
                found[wave][n + __builtin_popcountll(who & ((1ull << lane) - 1))] = (uint64_t)hi[i] << 32 | lo[i];
            n += __builtin_popcountll(who);
        }
        __builtin_amdgcn_wave_barrier();
        __atomic_signal_fence(__ATOMIC_SEQ_CST);
        if (lane < n) {
            const uint64_t key = found[wave][lane];
            int place = 0;
            for (int j = 0; j < n; ++j)
                place += found[wave][j] > key;
            if (place < f.top)
                put_top(f, row, r, place, key);
        }
        __atomic_signal_fence(__ATOMIC_SEQ_CST);
        __builtin_amdgcn_wave_barrier();
    }
}

// The gradient: one reading and one writing.  A group's results go where its
// logits came from, in place too (a lane writes what it alone has read).
constexpr int kEach = 4;                          // groups of a lane
template <int TYPE>
__global__ void __launch_bounds__(kThreads) gradient_kernel(const Backward b, int parts)
{
    const int64_t items = b.M * parts;
    const float c = b.scale * kLog2e;
    for (int64_t item = blockIdx.x; item < items; item += gridDim.x) {
        const int64_t row = item / parts;
        const int part = (int)(item - row * parts);
        int head;
        const char *p = first_group<TYPE>(b.X, b.ldx, row, head);
        char *q = static_cast<char *>(b.dX) + (row * b.ldd - head) * kSize<TYPE>;
        const int groups = (head + b.V + kGroup - 1) / kGroup, g0 = part * (kThreads * kEach) + threadIdx.x;
        Group<TYPE> x[kEach];
#pragma unroll
        for (int i = 0; i < kEach; ++i)
            if (g0 + i * kThreads < groups)
                x[i].load(p + (int64_t)(g0 + i * kThreads) * (kGroup * kSize<TYPE>));
        const float largest = b.stats[2 * row], logsum = b.stats[2 * row + 1];
        const bool nothing = logsum == -__builtin_inff();
        const int64_t token = b.tokens ? b.tokens[row] : -1;
        const float dl = token >= 0 && token < b.V ? b.dlogp[row] : 0.0f;
        const float dh = b.dentropy ? b.dentropy[row] : 0.0f, h = b.dentropy ? b.entropy[row] : 0.0f;
        // p·(k0 + k1·log2 p), scaled
        const float k0 = nothing ? 0.0f : -b.scale * (dl + dh * h), k1 = nothing ? 0.0f : -b.scale * dh * kLn2;
        const float ls2 = nothing ? 0.0f : logsum * kLog2e, zero = nothing ? 0.0f : largest;
        const int at_token = token >= 0 && token < b.V && !nothing ? (int)token : -1;
#pragma unroll
        for (int i = 0; i < kEach; ++i) {
            const int g = g0 + i * kThreads, first = g * kGroup - head;
            if (g >= groups)
                continue;
            float v[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const float l = (x[i].at(e) - zero) * c - ls2, w = __builtin_amdgcn_exp2f(l);
                v[e] = w * __builtin_fmaf(k1, __builtin_fmaxf(l, kFar), k0);
            }
            // dl·(1 - p) of the token: exact also where p is near 1
            if ((unsigned)(at_token - first) < 8u) {
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    if (first + e != at_token)
                        continue;
                    const float l = (x[i].at(e) - zero) * c - ls2, w = __builtin_amdgcn_exp2f(l);
                    v[e] = w * __builtin_fmaf(k1, __builtin_fmaxf(l, kFar), -b.scale * dh * h) -
                           b.scale * dl * expm1f(l * kLn2);
                }
            }
            char *to = q + (int64_t)g * (kGroup * kSize<TYPE>);
            const bool inside = first >= 0 && first + kGroup <= b.V;
            if constexpr (TYPE == HG_F32) {
                if (inside) {
                    *reinterpret_cast<lin::floatx4_any *>(to) = floatx4{v[0], v[1], v[2], v[3]};
                    *reinterpret_cast<lin::floatx4_any *>(to + 16) = floatx4{v[4], v[5], v[6], v[7]};
                    continue;
                }
            } else if (inside) {
                *reinterpret_cast<lin::u32x4_any *>(to) = lin::pack8<TYPE == HG_BF16>(v);
                continue;
            }
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                if ((unsigned)(first + e) >= (unsigned)b.V)
                    continue;
                if constexpr (TYPE == HG_F32)
                    reinterpret_cast<float *>(to)[e] = v[e];
                else
                    reinterpret_cast<uint16_t *>(to)[e] = lin::narrow<TYPE == HG_BF16>(v[e]);
            }
        }
    }
}

int64_t grid_of(int64_t items) { return items < (1 << 22) ? items : 1 << 22; }

template <int GR, int TYPE>
hipError_t parts(const Forward &f, hipStream_t s)
{
    return start(f.top > 0 ? part_kernel<GR, TYPE, true> : part_kernel<GR, TYPE, false>, grid_of(f.M * f.parts.parts),
                 kThreads, s, f);
}
template <int TYPE>
hipError_t forward(const Forward &f, hipStream_t s)
{
    const hipError_t e = f.parts.groups == 1   ? parts<1, TYPE>(f, s)
                         : f.parts.groups == 2 ? parts<2, TYPE>(f, s)
                         : f.parts.groups == 4 ? parts<4, TYPE>(f, s)
                                               : parts<8, TYPE>(f, s);
    if (e != hipSuccess || f.parts.parts == 1)
        return e;
    const int keys = f.parts.parts * f.top;
    if (f.parts.parts > 128 || keys > 33 * 64)
        return hipErrorInvalidConfiguration;
    return start(keys <= 64 ? join_kernel<1, TYPE> : keys <= 256 ? join_kernel<4, TYPE> : join_kernel<33, TYPE>,
                 grid_of((f.M + kThreads / 64 - 1) / (kThreads / 64)), kThreads, s, f);
}
template <int TYPE>
hipError_t backward(const Backward &b, hipStream_t s)
{
    const int groups = (b.V + 2 * kGroup - 2) / kGroup, parts = (groups + kThreads * kEach - 1) / (kThreads * kEach);
    return start(gradient_kernel<TYPE>, grid_of(b.M * parts), kThreads, s, b, parts);
}

}  // namespace

hipError_t launch_forward(const Forward &f, hipStream_t s)
{
    return f.type == HG_F32 ? forward<HG_F32>(f, s) : f.type == HG_F16 ? forward<HG_F16>(f, s) : forward<HG_BF16>(f, s);
}
hipError_t launch_backward(const Backward &b, hipStream_t s)
{
    return b.type == HG_F32 ? backward<HG_F32>(b, s) : b.type == HG_F16 ? backward<HG_F16>(b, s) : backward<HG_BF16>(b, s);
}

}  // namespace probs
}  // namespace hg
