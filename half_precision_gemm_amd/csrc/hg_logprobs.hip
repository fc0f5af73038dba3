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
// The most probable k of a part: the lanes fall into 32 or 64 sets, at least k; the
// k-th largest of the sets' maxima is reached by an element of k sets, so it is a
// threshold that the k largest reach, and few others where large logits are
// anywhere (k = 5 of 32 sets: 5.4 on average, 20 of 64: 24).  Only whole groups of
// eight logits are compared with it where they lie, in registers; the few that reach
// it go to LDS, and their logits that do are ordered there by (logit, lower number
// first), each counting those before it.  Where there is no room for what reaches
// it (few tokens allowed, equal logits), a threshold is found that at least k and at
// most k + kSpare lanes' maxima reach, by bisection over their bits (counted with
// ballots); equal maxima are told apart by where their group lies, in the same
// order.  Then only those lanes can hold candidates, at most kLanes·64.  Measured,
// 8192×50264 bf16, us, without the most probable 152: bisection for all k = 5 304, k
// = 32 356; the least of 8 (32) sets' maxima 222, 304; as it is 215, 245.
//
// Groups of eight logits lie at multiples of 16 bytes (32 of fp32) in memory
// whatever the row's address is, so every load is a whole one; what a row's first
// and last group hold of its neighbours (or of nothing: in the same 32 bytes as a
// logit, so in its page) counts as -inf.
#include "hg_logprobs.h"

#include "hgemm_logprobs.h"
#include "hg_linear.h"

namespace hg {
namespace probs {
namespace {

using lin::floatx4;
using lin::start;
using lin::u32x4;

constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.69314718055994531f;
constexpr float kFar = -200.0f;                   // 2^kFar is 0 in fp32, and 0·kFar is 0
constexpr int kSpare = 8, kLanes = 32 + kSpare;   // lanes that may hold candidates after a bisection
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
    // At `at` bytes of a buffer (an offset past its end: zeros).
    __device__ __forceinline__ void load(__amdgpu_buffer_rsrc_t r, int at)
    {
#pragma unroll
        for (int i = 0; i < kSize<TYPE> / 2; ++i)
            w[i] = __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(r, at + 16 * i, 0, 0));
    }
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
    // The same where e is the lane's own.
    __device__ __forceinline__ float any(int e) const
    {
        typename std::conditional<TYPE == HG_F32, float, uint16_t>::type v;
        __builtin_memcpy(&v, reinterpret_cast<const char *>(w) + e * sizeof v, sizeof v);
        if constexpr (TYPE == HG_F32)
            return v;
        else
            return lin::widen<TYPE == HG_BF16>(v);
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

// f of the lanes' values and the same in all lanes: neighbours, pairs, halves of
// eight and of sixteen by DPP, the rows by swaps.  `steps`: the first so many, for
// groups of 2^steps lanes.
template <int steps, class T, class F>
__device__ __forceinline__ T fold(T v, F f)
{
    auto moved = [&](auto c) __attribute__((always_inline)) {
        const int w = __builtin_amdgcn_mov_dpp(__builtin_bit_cast(int, v), decltype(c)::value, 0xf, 0xf, true);
        v = f(v, __builtin_bit_cast(T, w));
    };
    if constexpr (steps > 0)
        moved(std::integral_constant<int, 0xb1>{});               // quad_perm 1 0 3 2
    if constexpr (steps > 1)
        moved(std::integral_constant<int, 0x4e>{});               // quad_perm 2 3 0 1
    if constexpr (steps > 2)
        moved(std::integral_constant<int, 0x141>{});              // row_half_mirror
    if constexpr (steps > 3)
        moved(std::integral_constant<int, 0x140>{});              // row_mirror
    if constexpr (steps > 4) {
        const uint32_t u = __builtin_bit_cast(uint32_t, v);
        const auto r = __builtin_amdgcn_permlane16_swap(u, u, false, false);
        const uint32_t x = r[0], y = r[1];
        v = f(__builtin_bit_cast(T, x), __builtin_bit_cast(T, y));
    }
    if constexpr (steps > 5) {
        const uint32_t u = __builtin_bit_cast(uint32_t, v);
        const auto r = __builtin_amdgcn_permlane32_swap(u, u, false, false);
        const uint32_t x = r[0], y = r[1];
        v = f(__builtin_bit_cast(T, x), __builtin_bit_cast(T, y));
    }
    return v;
}
__device__ __forceinline__ float max_of_wave(float v)
{
    return fold<6>(v, [](float a, float b) { return __builtin_fmaxf(a, b); });
}
__device__ __forceinline__ float sum_of_wave(float v)
{
    return fold<6>(v, [](float a, float b) { return a + b; });
}
// The k-th largest of `sets` (32 or 64, at least k) numbers in LDS, equal ones counted
// as often as they are there; the same in all lanes.  Every lane counts what is
// larger than one of them (of 32, half a wave counts among either half).
__device__ __forceinline__ uint32_t kth_largest(const uint32_t *numbers, int sets, int k)
{
    const int lane = threadIdx.x & 63;
    const uint32_t mine = numbers[lane & (sets - 1)];
    const uint32_t *from = numbers + (sets == 32 ? lane >> 5 << 4 : 0);
    int larger = 0;
#pragma clang loop unroll(disable)
    for (int i = 0; i < (sets == 32 ? 16 : 64); i += 16) {
        u32x4 w[4];
#pragma unroll
        for (int j = 0; j < 4; ++j)
            w[j] = *reinterpret_cast<const u32x4 *>(from + i + 4 * j);
#pragma unroll
        for (int j = 0; j < 4; ++j)
#pragma unroll
            for (int e = 0; e < 4; ++e)
                larger += w[j][e] > mine;
    }
    if (sets == 32) {
        const auto r = __builtin_amdgcn_permlane32_swap((uint32_t)larger, (uint32_t)larger, false, false);
        larger = (int)(r[0] + r[1]);
    }
    // the least of those that fewer than k are larger than
    const uint32_t v = larger < k ? mine : 0xffffffffu;
    return fold<6>(v, [](uint32_t a, uint32_t b) { return a < b ? a : b; });
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

// How many of n keys are larger.  Several are read together: one by one each costs
// LDS' latency.  (What lies behind the last is read, up to a multiple of 8, and not
// counted.)
__device__ __forceinline__ int larger(const uint64_t *keys, int n, uint64_t key)
{
    int count = 0;
    for (int j = 0; j < n; j += 8) {
        uint64_t k[8];
#pragma unroll
        for (int e = 0; e < 8; ++e)
            k[e] = keys[j + e];
#pragma unroll
        for (int e = 0; e < 8; ++e)
            count += j + e < n && k[e] > key;
    }
    return count;
}

// WAVES: of the workgroup; GR: groups of a lane.
template <int WAVES, int GR, int TYPE, bool TOP>
__global__ void __launch_bounds__(WAVES * 64, GR == 8 ? (TYPE == HG_F32 ? 4 : 5) : 6) part_kernel(const Forward f, int rows_on, int parts_on)
{
    constexpr int THREADS = WAVES * 64, LANES = kLanes < THREADS ? kLanes : THREADS;
    constexpr int kFew = WAVES == 1 ? 96 : 192, MOST = LANES * GR * kGroup;
    __shared__ float wave_sums[WAVES][3];
    __shared__ __attribute__((aligned(16))) uint32_t sets[TOP ? 64 : 4];
    __shared__ uint32_t best_hi[TOP ? THREADS : 1], best_lo[TOP ? THREADS : 1];
    __shared__ Group<TYPE> few[TOP ? kFew : 1];
    __shared__ int few_at[TOP ? kFew : 1];
    __shared__ uint64_t found[TOP ? MOST + 8 : 1];
    __shared__ int count, all;
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const float c = f.scale * kLog2e;
    const int parts = f.parts.parts;
    int part = blockIdx.x % (unsigned)parts;
    for (int64_t row = blockIdx.x / (unsigned)parts; row < f.M; row += rows_on, part += parts_on) {
        if (part >= parts) {
            part -= parts;
            if (++row >= f.M)
                break;
        }
        const int64_t item = row * parts + part;
        int head;
        const char *p = first_group<TYPE>(f.X, f.ldx, row, head);
        const int groups = (head + f.V + kGroup - 1) / kGroup;               // of the row
        const int g0 = part * f.parts.per, n = min(groups - g0, f.parts.per);       // this part's
        Group<TYPE> x[GR];
        const __amdgpu_buffer_rsrc_t buffer = __builtin_amdgcn_make_buffer_rsrc(
            const_cast<char *>(p) + (int64_t)g0 * (kGroup * kSize<TYPE>), 0, max(n, 0) * (kGroup * kSize<TYPE>), 0x00020000);
        // Groups past the part's last are zeros, then -inf; of a whole wave none are
        // looked at.
        auto any = [&](int i) { return i * THREADS + wave * 64 < n; };
#pragma unroll
        for (int i = 0; i < GR; ++i)
            if (any(i))
                x[i].load(buffer, (i * THREADS + threadIdx.x) * (kGroup * kSize<TYPE>));
        // groups 1 .. of the row that are whole, up to this part's last
        const unsigned whole_groups = (unsigned)max(min(g0 + n, groups - 1) - 1, 0);
        float best = -__builtin_inff(), of_group[GR];
#pragma unroll
        for (int i = 0; i < GR; ++i) {
            if (!any(i))
                continue;
            const int at = i * THREADS + threadIdx.x;
            if ((unsigned)(g0 + at - 1) >= whole_groups)
                x[i].cut(at < n ? (g0 + at) * kGroup - head : f.V, f.V);
            float m = x[i].at(0);
#pragma unroll
            for (int e = 1; e < 8; ++e)
                m = __builtin_fmaxf(m, x[i].at(e));
            of_group[i] = m;
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
        const int nsets = f.top > 16 ? 64 : 32;
        if constexpr (TOP) {
            const auto most = [](float a, float b) { return __builtin_fmaxf(a, b); };
            const int each = THREADS / nsets;                                 // lanes of a set: 1, 2, 4 or 8
            float set = best;
            if constexpr (WAVES == 1)
                set = each == 2 ? fold<1>(best, most) : best;
            else
                set = each == 8 ? fold<3>(best, most) : fold<2>(best, most);
            if ((threadIdx.x & (each - 1)) == 0)
                sets[threadIdx.x / each] = ordered(set);
            if (threadIdx.x == 0)
                count = all = 0;
        }
        if (lane == 0) {
            wave_sums[wave][0] = m;
            wave_sums[wave][1] = sum;
            wave_sums[wave][2] = weighted;
        }
        __syncthreads();
        float largest = wave_sums[0][0], s = 0.0f, t = 0.0f;
#pragma unroll
        for (int i = 1; i < WAVES; ++i)
            largest = __builtin_fmaxf(largest, wave_sums[i][0]);
        const bool whole = f.parts.parts == 1;
        Row r{};
        if (whole || wave == 0) {
            const float to = largest == -__builtin_inff() ? 0.0f : largest;
#pragma unroll
            for (int i = 0; i < WAVES; ++i)
                join(wave_sums[i][0], wave_sums[i][1], wave_sums[i][2], to, c, s, t);
            if (whole)
                r = finish<TYPE>(f, row, largest, s, t, threadIdx.x == 0);
            else if (threadIdx.x == 0)
                f.partials[item] = {largest, s, t, 0.0f};
        }
        if constexpr (TOP) {
            const int end = min((g0 + n) * kGroup - head, f.V);               // of this part's logits
            // v's key, and its place among the candidates
            auto put = [&](float v, int at) __attribute__((always_inline)) {
                const int place = atomicAdd(&all, 1);
                if (place < MOST)
                    found[place] = (uint64_t)ordered(without_nan(v)) << 32 | ~(uint32_t)at;
            };
            const float reach = unordered(kth_largest(sets, nsets, f.top));
            // Groups that reach it go to LDS (a lane's to places that one atomic operation
            // has taken), where their logits are looked at by a thread each.  (A NaN
            // never is below anything: it comes along, and goes to the end of the order.)
            int mine = 0;
#pragma unroll
            for (int i = 0; i < GR; ++i)
                if (any(i))
                    mine += !(of_group[i] < reach);
            if (mine > 0) {
                int place = atomicAdd(&count, mine);
#pragma unroll
                for (int i = 0; i < GR; ++i) {
                    if (!any(i) || of_group[i] < reach)
                        continue;
                    if (place < kFew) {
                        few[place] = x[i];
                        few_at[place] = g0 + i * THREADS + threadIdx.x;
                    }
                    ++place;
                }
            }
            __syncthreads();
            const int left = count;
            if (left <= kFew) {
                for (int i = threadIdx.x; i < left * kGroup; i += THREADS) {
                    const int at = few_at[i / kGroup] * kGroup - head + i % kGroup;
                    const float v = few[i / kGroup].any(i % kGroup);
                    if (!(v < reach) && at >= 0 && at < end)
                        put(v, at);
                }
                __syncthreads();
            }
            if (left > kFew || all > MOST) {
                int best_at = g0 + threadIdx.x;                               // the first group with the lane's maximum
                float top = -__builtin_inff();
#pragma unroll
                for (int i = 0; i < GR; ++i) {
                    if (!any(i))
                        continue;
                    best_at = of_group[i] > top ? g0 + i * THREADS + threadIdx.x : best_at;
                    top = __builtin_fmaxf(top, of_group[i]);
                }
                best_hi[threadIdx.x] = (int)threadIdx.x < n ? ordered(best) >> kLowBit<TYPE> : 0;
                best_lo[threadIdx.x] = ~(uint32_t)best_at;
                __syncthreads();                  // (everyone has seen `all`)
                if (threadIdx.x == 0)
                    all = 0;
                uint32_t hi[WAVES], lo[WAVES], least, lowest;
#pragma unroll
                for (int i = 0; i < WAVES; ++i) {
                    hi[i] = best_hi[i * 64 + lane];
                    lo[i] = best_lo[i * 64 + lane];
                }
                threshold<WAVES>(hi, lo, 32 - kLowBit<TYPE>, f.top, min(f.top + kSpare, LANES), least, lowest);
                __syncthreads();
#pragma unroll
                for (int i = 0; i < GR; ++i) {
                    const int at = i * THREADS + threadIdx.x, first = (g0 + at) * kGroup - head;
                    if (!any(i) || at >= n || ordered(without_nan(of_group[i])) >> kLowBit<TYPE> < least)
                        continue;
                    const bool ties = ~(uint32_t)(g0 + at) >= lowest;
#pragma unroll
                    for (int e = 0; e < 8; ++e) {
                        const uint32_t h = ordered(without_nan(x[i].at(e))) >> kLowBit<TYPE>;
                        if ((h > least || (h == least && ties)) && first + e >= 0 && first + e < end)
                            put(x[i].at(e), first + e);
                    }
                }
                __syncthreads();
            }
            uint64_t *keys = f.keys + item * f.top;
            const int candidates = all;
            for (int i = threadIdx.x; i < candidates; i += THREADS) {
                const uint64_t key = found[i];
                const int place = larger(found, candidates, key);
                if (place < f.top) {
                    if (whole)
                        put_top(f, row, r, place, key);
                    else
                        keys[place] = key;
                }
            }
            if (!whole)                           // fewer elements than `top`
                for (int i = candidates + threadIdx.x; i < f.top; i += THREADS)
                    keys[i] = 0;
        }
        __syncthreads();
    }
}

// One wave joins a row's parts, at most two to a lane; E·64 keys at most.
template <int E, int TYPE>
__global__ void __launch_bounds__(kThreads) join_kernel(const Forward f)
{
    __shared__ uint64_t found[kThreads / 64][64 + 8];
    __shared__ __attribute__((aligned(16))) uint32_t sets[kThreads / 64][64];
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
        // What the largest keys of `top` lanes reach; if that is more than 64 keys,
        // what a threshold leaves: they are all different.
        auto reaching = [&](int i) __attribute__((always_inline)) {
            return hi[i] != 0 && (hi[i] > least || (hi[i] == least && lo[i] >= lowest));
        };
        auto count = [&]() __attribute__((always_inline)) {
            int c = 0;
#pragma unroll
            for (int i = 0; i < E; ++i)
                c += __builtin_popcountll(__builtin_amdgcn_ballot_w64(reaching(i)));
            return c;
        };
        least = lowest = 0;
        if constexpr (E > 1) {
            uint32_t most = hi[0];
#pragma unroll
            for (int i = 1; i < E; ++i)
                most = max(most, hi[i]);
            sets[wave][lane] = most;
            __atomic_signal_fence(__ATOMIC_SEQ_CST);
            least = kth_largest(sets[wave], 64, f.top);
            __atomic_signal_fence(__ATOMIC_SEQ_CST);
            if (count() > 64)
                threshold<E>(hi, lo, 32, f.top, 64, least, lowest);
        }
        int n = 0;
#pragma unroll
        for (int i = 0; i < E; ++i) {
            const bool in = reaching(i);
            const uint64_t who = __builtin_amdgcn_ballot_w64(in);
            if (in)
                found[wave][n + __builtin_popcountll(who & ((1ull << lane) - 1))] = (uint64_t)hi[i] << 32 | lo[i];
            n += __builtin_popcountll(who);
        }
        __builtin_amdgcn_wave_barrier();
        __atomic_signal_fence(__ATOMIC_SEQ_CST);
        if (lane < n) {
            const uint64_t key = found[wave][lane];
            const int place = larger(found[wave], n, key);
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

template <int WAVES, int GR, int TYPE>
hipError_t parts(const Forward &f, hipStream_t s)
{
    const int64_t grid = grid_of(f.M * f.parts.parts);
    return start(f.top > 0 ? part_kernel<WAVES, GR, TYPE, true> : part_kernel<WAVES, GR, TYPE, false>, grid, WAVES * 64, s, f,
                 (int)(grid / f.parts.parts), (int)(grid % f.parts.parts));
}
template <int WAVES, int TYPE>
hipError_t parts(const Forward &f, hipStream_t s)
{
    return f.parts.groups == 1   ? parts<WAVES, 1, TYPE>(f, s)
           : f.parts.groups == 2 ? parts<WAVES, 2, TYPE>(f, s)
           : f.parts.groups == 4 ? parts<WAVES, 4, TYPE>(f, s)
                                 : parts<WAVES, 8, TYPE>(f, s);
}
template <int TYPE>
hipError_t forward(const Forward &f, hipStream_t s)
{
    const hipError_t e = f.parts.waves == 1 ? parts<1, TYPE>(f, s) : parts<4, TYPE>(f, s);
    if (e != hipSuccess || f.parts.parts == 1)
        return e;
    const int keys = f.parts.parts * f.top;
    static_assert(kMostParts <= kLongestParts && kLongestParts <= 128 && kLongestParts * HG_LOGPROBS_MAX_TOP <= 33 * 64 &&
                      (HG_LOGPROBS_MAX_VOCABULARY + 2 * kGroup - 2) / kGroup <= kLongestParts * 8 * kThreads,
                  "");
    if (f.parts.parts > kLongestParts)
        return hipErrorInvalidConfiguration;
    return start(keys <= 64    ? join_kernel<1, TYPE>
                 : keys <= 256 ? join_kernel<4, TYPE>
                 : keys <= 512 ? join_kernel<8, TYPE>
                               : join_kernel<33, TYPE>,
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
