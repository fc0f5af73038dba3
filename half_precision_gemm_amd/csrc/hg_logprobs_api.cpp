// hg_logprobs_api.cpp — host side of the C ABI declared in
// include/hgemm_logprobs.h.
#include "hgemm_logprobs.h"

#include <stdint.h>

#include <algorithm>

#include "hg_linear_host.h"
#include "hg_logprobs.h"

using namespace hg::host;

namespace {

namespace probs = hg::probs;

bool is_logits(int type) { return type == HG_F16 || type == HG_BF16 || type == HG_F32; }
bool aligned(const void *p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

// Parts that rows are cut into: as long as they come (16384 logits, a load of 16
// bytes or two for each of a lane's eight groups) if that gives every CU two, else
// shorter ones, down to 2048.  Rows of up to 4096 logits go to a wave each.
probs::Parts parts_of(int64_t M, int64_t V)
{
    const int64_t groups = (V + 2 * probs::kGroup - 2) / probs::kGroup;       // wherever in one a row begins
    int64_t per = 8;
    if (groups <= 8 * 64) {
        while (per > 1 && groups <= per / 2 * 64)
            per /= 2;
        return {1, (int32_t)per, 1, (int32_t)groups};
    }
    auto parts = [&](int64_t g) { return (groups + g * probs::kThreads - 1) / (g * probs::kThreads); };
    while (per > 1 && (parts(per / 2) == 1 || (M * parts(per) < 2 * hg::cu_count() && parts(per / 2) <= probs::kMostParts)))
        per /= 2;
    const int64_t n = parts(per);
    return {4, (int32_t)per, (int32_t)n, (int32_t)((groups + n - 1) / n)};
}

int check(int64_t M, int64_t V)
{
    if (M < 0 || M > HG_LINEAR_MAX_ROWS)
        return -1;
    return V < 1 || V > HG_LOGPROBS_MAX_VOCABULARY ? -2 : HG_OK;
}
struct Room {
    void *partials, *keys;
};
Room room_of(Arena &a, int64_t M, const probs::Parts &q, int top)
{
    Room r{nullptr, nullptr};
    if (q.parts > 1) {
        r.partials = a.take(M * q.parts * (int64_t)sizeof(probs::Partial));
        r.keys = a.take(M * q.parts * top * 8);
    }
    return r;
}

}  // namespace

extern "C" {

int64_t hg_logprobs_workspace_size(int64_t M, int64_t V, int top)
{
    if (const int e = check(M, V))
        return e;
    if (top < 0 || top > HG_LOGPROBS_MAX_TOP || top > V)
        return -3;
    Arena a{nullptr};
    room_of(a, M, parts_of(M, V), top);
    return a.used;
}

int hg_logprobs(int64_t M, int64_t V, const hg_matrix *X, float scale, const int64_t *tokens, float *logp, float *entropy,
                float *stats, int top, int64_t *top_ids, float *top_logp, void *work, int64_t work_bytes, void *stream)
{
    if (const int e = check(M, V))
        return e;
    if (X == nullptr || !is_logits(X->type) || !valid(X, M, V))
        return -3;
    if (!(scale > 0.0f && scale <= HG_LOGPROBS_MAX_SCALE))
        return -4;
    if (!aligned(tokens, 8) || (logp != nullptr && tokens == nullptr))
        return -5;
    if (!aligned(logp, 4))
        return -6;
    if (!aligned(entropy, 4))
        return -7;
    if (!aligned(stats, 4))
        return -8;
    if (top < 0 || top > HG_LOGPROBS_MAX_TOP || top > V)
        return -9;
    if (!aligned(top_ids, 8))
        return -10;
    if (!aligned(top_logp, 4))
        return -11;
    if (M == 0)
        return HG_OK;
    if (top == 0)
        top_ids = nullptr, top_logp = nullptr;
    else if (top_ids == nullptr && top_logp == nullptr)
        top = 0;
    const Span x = data_span(X, M, V), t = span_of(tokens, M * 8), l = span_of(logp, M * 4), e = span_of(entropy, M * 4),
               st = span_of(stats, M * 8), ids = span_of(top_ids, M * top * 8), tl = span_of(top_logp, M * top * 4);
    if (any_meet({l}, {x, t}))
        return -6;
    if (any_meet({e}, {x, t, l}))
        return -7;
    if (any_meet({st}, {x, t, l, e}))
        return -8;
    if (any_meet({ids}, {x, t, l, e, st}))
        return -10;
    if (any_meet({tl}, {x, t, l, e, st, ids}))
        return -11;
    const probs::Parts parts = parts_of(M, V);
    Arena count{nullptr}, arena{static_cast<char *>(work)};
    room_of(count, M, parts, top);
    if (bad_work(work, count.used) || any_meet({span_of(work, count.used)}, {x, t, l, e, st, ids, tl}))
        return -12;
    if (work_bytes < count.used)
        return -13;
    const Room r = room_of(arena, M, parts, top);
    probs::Forward f{};
    f.X = X->data;
    f.ldx = X->ld;
    f.type = X->type;
    f.tokens = tokens;
    f.logp = logp;
    f.entropy = entropy;
    f.stats = stats;
    f.top_ids = top_ids;
    f.top_logp = top_logp;
    f.partials = static_cast<probs::Partial *>(r.partials);
    f.keys = static_cast<uint64_t *>(r.keys);
    f.M = M;
    f.V = (int32_t)V;
    f.top = top;
    f.scale = scale;
    f.parts = parts;
    return status_of(probs::launch_forward(f, static_cast<hipStream_t>(stream)));
}

int hg_logprobs_grad(int64_t M, int64_t V, const hg_matrix *X, float scale, const int64_t *tokens, const float *stats,
                     const float *entropy, const float *dlogp, const float *dentropy, const hg_matrix *dX, void *stream)
{
    if (const int e = check(M, V))
        return e;
    if (X == nullptr || !is_logits(X->type) || !valid(X, M, V))
        return -3;
    if (!(scale > 0.0f && scale <= HG_LOGPROBS_MAX_SCALE))
        return -4;
    if (!aligned(tokens, 8) || (dlogp != nullptr && tokens == nullptr))
        return -5;
    if (!aligned(stats, 4) || (M > 0 && stats == nullptr))
        return -6;
    if (!aligned(entropy, 4) || (dentropy != nullptr && entropy == nullptr))
        return -7;
    if (!aligned(dlogp, 4))
        return -8;
    if (!aligned(dentropy, 4))
        return -9;
    if (dX == nullptr || dX->type != X->type || !valid(dX, M, V))
        return -10;
    if (M == 0)
        return HG_OK;
    const Span x = data_span(X, M, V), d = data_span(dX, M, V);
    const bool in_place = X->data == dX->data && X->ld == dX->ld;
    if ((!in_place && meet(d, x)) ||
        any_meet({d}, {span_of(dlogp != nullptr ? tokens : nullptr, M * 8), span_of(stats, M * 8),
                       span_of(dentropy != nullptr ? entropy : nullptr, M * 4), span_of(dlogp, M * 4),
                       span_of(dentropy, M * 4)}))
        return -10;
    probs::Backward b{};
    b.X = X->data;
    b.ldx = X->ld;
    b.dX = dX->data;
    b.ldd = dX->ld;
    b.type = X->type;
    b.tokens = dlogp != nullptr ? tokens : nullptr;
    b.stats = stats;
    b.entropy = dentropy != nullptr ? entropy : nullptr;
    b.dlogp = dlogp;
    b.dentropy = dentropy;
    b.M = M;
    b.V = (int32_t)V;
    b.scale = scale;
    return status_of(probs::launch_backward(b, static_cast<hipStream_t>(stream)));
}

}  // extern "C"
