// hg_adamw.hip — a step of AdamW over many tensors (gfx950).
//
//     m = β1·m + (1 - β1)·g,  v = β2·v + (1 - β2)·g²
//     w = w - lr·(decay·w + (m / c1) / (sqrt(v / c2) + eps)),  c = 1 - β^t
//
// Every element is read and written once, 10 to 28 bytes of it, for a few dozen
// operations: HBM bounds it, and launches where tensors are small.  So one launch
// takes up to 83 tensors, whose descriptions are its arguments (no table in
// memory that a captured graph would need to keep); a workgroup finds its
// tensor among them and takes 2048 or 8192 elements, eight neighbours to a lane.
//
// 8-bit moments: four neighbouring lanes hold the 32 elements that share a scale.
// Random rounding adds a random number below one step of the code to the scaled
// magnitude's bits and cuts off what is below a code.  A magnitude below 2^-6,
// where codes are 2^-9 apart, gets 2^-6 added first, which gives it an exponent
// whose codes are that far apart, and taken off again.
//
// c is 1 - exp(t·log β) by expm1, log β in fp64 from the host: 1 - 0.999 in
// fp32 would be off by 6e-5 of itself.
#include "hg_adamw.h"

#include "hgemm_adamw.h"
#include "hg_linear.h"

namespace hg {
namespace adamw {
namespace {

using lin::floatx4_any;
using lin::floatx4;
using lin::u32x2;

__device__ __forceinline__ uint32_t mix(uint32_t x)
{
    x ^= x >> 16;
    x *= 0x9E3779B9u;
    x ^= x >> 15;
    x *= 0xB504F333u;
    return x ^ x >> 16;
}

// Elements 0 .. n-1 of eight (n may pass 8), the others 0.
__device__ __forceinline__ void load32(const float *p, int n, float (&v)[8])
{
    if (n >= 8) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const floatx4 w = *reinterpret_cast<const floatx4_any *>(p + 4 * h);
#pragma unroll
            for (int e = 0; e < 4; ++e)
                v[4 * h + e] = w[e];
        }
    } else {
#pragma unroll
        for (int e = 0; e < 8; ++e)
            v[e] = e < n ? p[e] : 0.0f;
    }
}
__device__ __forceinline__ void store32(float *p, int n, const float (&v)[8])
{
    if (n >= 8) {
        *reinterpret_cast<floatx4_any *>(p) = floatx4{v[0], v[1], v[2], v[3]};
        *reinterpret_cast<floatx4_any *>(p + 4) = floatx4{v[4], v[5], v[6], v[7]};
    } else {
#pragma unroll
        for (int e = 0; e < 8; ++e)
            if (e < n)
                p[e] = v[e];
    }
}
// The same of any type; `type` is the workgroup's.
__device__ __forceinline__ void load(const void *p, int type, int64_t at, int n, float (&v)[8])
{
    if (type == HG_F32)
        load32(static_cast<const float *>(p) + at, n, v);
    else if (type == HG_BF16)
        lin::load8<true>(static_cast<const uint16_t *>(p) + at, n, v);
    else
        lin::load8<false>(static_cast<const uint16_t *>(p) + at, n, v);
}
__device__ __forceinline__ void store(void *p, int type, int64_t at, int n, const float (&v)[8])
{
    if (type == HG_F32)
        store32(static_cast<float *>(p) + at, n, v);
    else if (type == HG_BF16)
        lin::store8<true>(static_cast<uint16_t *>(p) + at, n, v);
    else
        lin::store8<false>(static_cast<uint16_t *>(p) + at, n, v);
}

// One eighth of a block per lane, as lin::encode8 for bf16, rounded by 16 random
// bits an element: bits SHIFT .. SHIFT + 15 of r.  KEEP: what is above 0 stays so.
template <int SHIFT, bool KEEP>
__device__ __forceinline__ int encode(const float (&v)[8], const uint32_t (&r)[8], u32x2 &w)
{
    constexpr float ordinary = 448.0f * 0x1p119f;
    float a = 0.0f, lim = 448.0f;
#pragma unroll
    for (int e = 0; e < 8; ++e)
        a = __builtin_fmaxf(a, __builtin_fabsf(v[e]));
    a = lin::max_of_4(a);
    const bool far = !(a <= ordinary);
    if (__builtin_expect(far, 0)) {
        a = 0.0f;
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const float m = __builtin_fabsf(v[e]);
            a = m < __builtin_inff() ? __builtin_fmaxf(a, m) : a;
        }
        a = lin::max_of_4(a);
    }
    const int x = lin::scale_exponent<true>(a);
    if (x == 120)
        lim = 240.0f;
    const float inv = __builtin_bit_cast(float, (uint32_t)(127 - x) << 23);
    float q[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        const float y = __builtin_fabsf(v[e]) * inv;
        const bool low = y < 0x1p-6f;
        const float z = low ? y + 0x1p-6f : y;
        const uint32_t add = (SHIFT ? r[e] >> 12 & 0xffff0u : r[e] << 4 & 0xffff0u) | 8u;
        float c = __builtin_bit_cast(float, (__builtin_bit_cast(uint32_t, z) + add) & 0xfff00000u);
        c = low ? c - 0x1p-6f : c;
        if (KEEP)                         // (y itself may have left fp32)
            c = c == 0.0f && v[e] > 0.0f ? 0x1p-9f : c;
        c = y <= lim ? c : __builtin_fabsf(v[e]) < __builtin_inff() ? lim : __builtin_nanf("");
        q[e] = __builtin_copysignf(c, v[e]);
    }
    w[0] = lin::pack_codes(q[0], q[1], q[2], q[3]);
    w[1] = lin::pack_codes(q[4], q[5], q[6], q[7]);
    return x;
}

// The card's own root, off by one step of fp32 at most, which takes numbers below
// 2^-126 for 0; the reciprocal is the card's too (eps, and any root that is not 0, is
// above that).  With the exact ones 64 fp32 tensors of 65536 and 2260 in turn take
// 14.1 us for 13.5, two of 2^25 229 for 228.
__device__ __forceinline__ float root(float x)
{
    const bool low = x < 0x1p-100f;
    return __builtin_amdgcn_sqrtf(low ? x * 0x1p100f : x) * (low ? 0x1p-50f : 1.0f);
}

// A tensor of a batch.
struct Tensor {
    void *param, *grad, *m, *v;
    float *master;
    uint8_t *ms, *vs;
    int64_t n;
    int place, param_type, grad_type;
    bool state8;
    __device__ __forceinline__ explicit Tensor(void *const *w) : param(w[0]), grad(w[1]), m(w[2]), v(w[3])
    {
        const uint64_t x = reinterpret_cast<uint64_t>(w[4]);
        const int with = (int)(x >> kMaster & 1);
        n = (int64_t)(x & ((uint64_t)1 << kPlace) - 1);
        place = (int)(x >> kPlace) & HG_ADAMW_MAX_TENSORS - 1;
        param_type = (int)(x >> kParam & 3);
        grad_type = (int)(x >> kGrad & 3);
        state8 = x >> kState8 & 1;
        master = with ? static_cast<float *>(w[5]) : nullptr;
        ms = state8 ? static_cast<uint8_t *>(w[5 + with]) : nullptr;
        vs = state8 ? static_cast<uint8_t *>(w[6 + with]) : nullptr;
    }
};

__global__ void __launch_bounds__(kThreads) step_kernel(const Batch b)
{
    int i = 0;
    for (int half = 64; half > 0; half /= 2)
        if (i + half < b.count && b.place[i + half].piece <= (int)blockIdx.x)
            i += half;
    const Tensor d(b.words + b.place[i].word);
    const int64_t base = (int64_t)((int)blockIdx.x - b.place[i].piece) * (b.each * kThreads * 8);
    const void *weight = d.master ? d.master : d.param;
    const int weight_type = d.master ? HG_F32 : d.param_type;
    int64_t t = b.step;
    if (b.device_step)
        t = *b.device_step;
    const float lr = b.factors ? b.lr * b.factors[0] : b.lr, gs = b.factors ? b.factors[1] : 1.0f;
    const float r1 = -1.0f / expm1f((float)((double)t * b.log1)), r2 = -1.0f / expm1f((float)((double)t * b.log2));
    const uint32_t words[6] = {(uint32_t)d.place, (uint32_t)t, (uint32_t)(t >> 32), (uint32_t)b.seed, (uint32_t)(b.seed >> 32),
                               (uint32_t)(base >> 32)};
    uint32_t key = 0;
#pragma unroll
    for (int k = 0; k < 6; ++k)
        key = mix(key + words[k] + 0x9E3779B9u);
#pragma unroll 1
    for (int u = 0; u < b.each; ++u) {
        const int64_t at = base + (u * kThreads + threadIdx.x) * 8, left = d.n - at;
        const int n = left > 8 ? 8 : left < 0 ? 0 : (int)left;
        float g[8], m[8], v[8], w[8];
        load(d.grad, d.grad_type, at, n, g);
        load(weight, weight_type, at, n, w);
        if (d.state8) {
            const u32x2 cm = lin::load_codes(static_cast<const uint8_t *>(d.m) + at, n);
            const u32x2 cv = lin::load_codes(static_cast<const uint8_t *>(d.v) + at, n);
            const int64_t block = at / lin::kBlock8;
            lin::values8(cm, lin::scale_of(n > 0 ? d.ms[block] : 0), m);
            lin::values8(cv, lin::scale_of(n > 0 ? d.vs[block] : 0), v);
        } else {
            load32(static_cast<const float *>(d.m) + at, n, m);
            load32(static_cast<const float *>(d.v) + at, n, v);
        }
        if (t < 1)                        // (known after the loads are on their way)
            return;
        {
            // the moments as the sums are written, each product and sum rounded: what
            // the random rounding starts from does not depend on the compiler
#pragma clang fp contract(off)
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const float s = b.factors ? g[e] * gs : g[e];
                m[e] = b.beta1 * m[e] + b.rest1 * s;
                v[e] = b.beta2 * v[e] + b.rest2 * (s * s);
            }
        }
#pragma unroll
        for (int e = 0; e < 8; ++e)
            w[e] -= lr * (b.decay * w[e] + m[e] * r1 * __builtin_amdgcn_rcpf(root(v[e] * r2) + b.eps));
        if (d.master)
            store32(d.master + at, n, w);
        store(d.param, d.param_type, at, n, w);
        if (d.state8) {
            uint32_t r[8];
#pragma unroll
            for (int e = 0; e < 8; ++e)
                r[e] = mix(((uint32_t)at + e) ^ key);
            u32x2 cm, cv;
            const int xm = encode<0, false>(m, r, cm), xv = encode<16, true>(v, r, cv);
            lin::store_codes(static_cast<uint8_t *>(d.m) + at, n, cm);
            lin::store_codes(static_cast<uint8_t *>(d.v) + at, n, cv);
            if (n > 0 && at % lin::kBlock8 == 0) {
                d.ms[at / lin::kBlock8] = (uint8_t)(xm + 127);
                d.vs[at / lin::kBlock8] = (uint8_t)(xv + 127);
            }
        } else {
            store32(static_cast<float *>(d.m) + at, n, m);
            store32(static_cast<float *>(d.v) + at, n, v);
        }
    }
}

}  // namespace

hipError_t launch(const Batch &b, hipStream_t s)
{
    return lin::start(step_kernel, b.pieces, kThreads, s, b);
}

}  // namespace adamw
}  // namespace hg
