// hg_adamw_api.cpp — host side of the C ABI declared in include/hgemm_adamw.h.
#include "hgemm_adamw.h"

#include <math.h>
#include <stdint.h>

#include <algorithm>
#include <new>
#include <vector>

#include "hg_adamw.h"
#include "hg_linear_host.h"

using namespace hg::host;

namespace {

namespace adamw = hg::adamw;

bool is_float(int type) { return type == HG_F16 || type == HG_BF16 || type == HG_F32; }
bool good(const void *p, int64_t size) { return p != nullptr && (reinterpret_cast<uintptr_t>(p) & (uintptr_t)(size - 1)) == 0; }

// A tensor's arrays that are there: what is written, then the gradient.
struct Arrays {
    Span a[7];
    int count = 0;
    void add(const void *p, int64_t bytes)
    {
        if (p != nullptr && bytes > 0)
            a[count++] = span_of(p, bytes);
    }
};
Arrays arrays_of(const hg_adamw_tensor &t)
{
    const int64_t n = t.n, s = t.state_type == HG_E4M3 ? blocks8(n) : 0, e = esize(t.state_type);
    Arrays x;
    x.add(t.param, n * esize(t.param_type));
    x.add(t.master, n * 4);
    x.add(t.m, n * e);
    x.add(t.v, n * e);
    x.add(t.m_scales, s);
    x.add(t.v_scales, s);
    x.add(t.grad, n * esize(t.grad_type));
    return x;
}
bool valid(const hg_adamw_tensor &t)
{
    if (t.n < 0 || t.n > HG_ADAMW_MAX_ELEMENTS || !is_float(t.param_type) || !is_float(t.grad_type) ||
        (t.state_type != HG_F32 && t.state_type != HG_E4M3) || (t.master != nullptr && t.param_type == HG_F32))
        return false;
    if (t.n == 0)
        return true;
    if (!good(t.param, esize(t.param_type)) || !good(t.grad, esize(t.grad_type)) || !good(t.m, esize(t.state_type)) ||
        !good(t.v, esize(t.state_type)) || (t.master != nullptr && !good(t.master, 4)))
        return false;
    if (t.state_type == HG_E4M3 && (t.m_scales == nullptr || t.v_scales == nullptr))
        return false;
    const Arrays x = arrays_of(t);
    for (int i = 0; i < x.count; ++i)
        for (int j = i + 1; j < x.count; ++j)
            if (meet(x.a[i], x.a[j]))
                return false;
    return true;
}
int check(int64_t count, const hg_adamw_tensor *tensors)
{
    if (count < 0 || count > HG_ADAMW_MAX_TENSORS)
        return -1;
    if (count > 0 && tensors == nullptr)
        return -2;
    for (int64_t i = 0; i < count; ++i)
        if (!valid(tensors[i]))
            return -2;
    return HG_OK;
}
bool part(double x) { return x >= 0.0 && x < 1.0; }
bool amount(double x) { return x >= 0.0 && isfinite((float)x); }

}  // namespace

extern "C" {

int hg_adamw_check(int64_t count, const hg_adamw_tensor *tensors)
{
    if (const int e = check(count, tensors))
        return e;
    struct Edge {
        Span s;
        bool written;
    };
    try {
        std::vector<Edge> all;
        all.reserve((size_t)count * 7);
        for (int64_t i = 0; i < count; ++i) {
            const Arrays x = arrays_of(tensors[i]);
            for (int j = 0; j < x.count; ++j)
                all.push_back({x.a[j], j + 1 < x.count});
        }
        std::sort(all.begin(), all.end(), [](const Edge &a, const Edge &b) { return a.s.lo < b.s.lo; });
        uintptr_t any = 0, written = 0;           // the ends so far
        for (const Edge &e : all) {
            if (e.s.lo < (e.written ? any : written))
                return -2;
            any = std::max(any, e.s.hi);
            if (e.written)
                written = std::max(written, e.s.hi);
        }
    } catch (const std::bad_alloc &) {
        return HG_ERR_HIP_BASE + (int)hipErrorOutOfMemory;
    }
    return HG_OK;
}

int hg_adamw(int64_t count, const hg_adamw_tensor *tensors, int64_t step, const int64_t *device_step, double lr,
             double beta1, double beta2, double eps, double decay, const float *factors, uint64_t seed, void *stream)
{
    if (const int e = check(count, tensors))
        return e;
    if (device_step == nullptr && step < 1)
        return -3;
    if ((reinterpret_cast<uintptr_t>(device_step) & 7) != 0)
        return -4;
    if (!amount(lr))
        return -5;
    if (!part(beta1))
        return -6;
    if (!part(beta2))
        return -7;
    if (!amount(eps) || (eps != 0.0 && (eps < HG_ADAMW_LEAST_EPS || eps > 1.0 / HG_ADAMW_LEAST_EPS)))
        return -8;
    if (!amount(decay))
        return -9;
    if ((reinterpret_cast<uintptr_t>(factors) & 3) != 0)
        return -10;
    const Span st = span_of(device_step, 8), f = span_of(factors, 8);
    for (int64_t i = 0; i < count && (device_step != nullptr || factors != nullptr); ++i) {
        const Arrays x = arrays_of(tensors[i]);
        for (int j = 0; j + 1 < x.count; ++j) {
            if (meet(x.a[j], st))
                return -4;
            if (meet(x.a[j], f))
                return -10;
        }
    }
    adamw::Batch b;
    b.count = b.pieces = b.used = 0;
    b.beta1 = (float)beta1;
    b.rest1 = (float)(1.0 - beta1);
    b.beta2 = (float)beta2;
    b.rest2 = (float)(1.0 - beta2);
    b.eps = (float)eps;
    b.decay = (float)decay;
    b.lr = (float)lr;
    b.log1 = log(beta1);
    b.log2 = log(beta2);
    b.factors = factors;
    b.device_step = device_step;
    b.step = step;
    b.seed = seed;
    // Long pieces, unless they would leave CUs without work.
    int64_t pieces = 0;
    for (int64_t i = 0; i < count; ++i)
        pieces += (tensors[i].n + adamw::piece_of(4) - 1) / adamw::piece_of(4);
    b.each = pieces < 4 * (int64_t)hg::cu_count() ? 1 : 4;
    const hipStream_t s = static_cast<hipStream_t>(stream);
    for (int64_t i = 0; i < count; ++i) {
        const hg_adamw_tensor &t = tensors[i];
        if (t.n == 0)
            continue;
        const int64_t n = (t.n + adamw::piece_of(b.each) - 1) / adamw::piece_of(b.each);
        const bool state8 = t.state_type == HG_E4M3;
        const int words = adamw::kFewest + (t.master != nullptr ? 1 : 0) + (state8 ? 2 : 0);
        if (b.count == adamw::kMost || b.used + words > adamw::kWords || b.pieces + n > hg::lin::kMostBlocks) {
            if (const hipError_t e = adamw::launch(b, s))
                return status_of(e);
            b.count = b.pieces = b.used = 0;
        }
        b.place[b.count++] = {b.pieces, b.used};
        const uint64_t numbers = (uint64_t)t.n | (uint64_t)i << adamw::kPlace | (uint64_t)t.param_type << adamw::kParam |
                                 (uint64_t)t.grad_type << adamw::kGrad |
                                 (uint64_t)(t.master != nullptr) << adamw::kMaster | (uint64_t)state8 << adamw::kState8;
        void **w = b.words + b.used;
        b.used += words;
        *w++ = t.param;
        *w++ = const_cast<void *>(t.grad);
        *w++ = t.m;
        *w++ = t.v;
        *w++ = reinterpret_cast<void *>(numbers);
        if (t.master != nullptr)
            *w++ = t.master;
        if (state8) {
            *w++ = t.m_scales;
            *w++ = t.v_scales;
        }
        b.pieces += (int32_t)n;
    }
    return b.count > 0 ? status_of(adamw::launch(b, s)) : HG_OK;
}

}  // extern "C"
