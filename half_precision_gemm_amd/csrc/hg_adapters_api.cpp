// hg_adapters_api.cpp — host side of the C ABI declared in
// include/hgemm_adapters.h.
#include "hgemm_adapters.h"

#include <stdint.h>

#include <algorithm>

#include "hg_linear.h"
#include "hg_linear_host.h"

using namespace hg::host;

namespace {

namespace lin = hg::lin;

// Numbers of X's type for one of T (lin::Adapters).
int parts_of(int type, bool out32) { return type == HG_BF16 && out32 ? 3 : 2; }
// Numbers that a row of T takes: fp32 ones up to a whole eight where it goes row by
// row (`few`), else `parts` 16-bit ones for each, up to the matrix cores' 32.
int64_t width_of(int64_t rank, bool few, int parts) { return few ? up8(rank) : (parts * up8(rank) + 31) / 32 * 32; }
struct Room {
    void *T, *far;
};
Room room_of(Arena &a, int64_t M, int64_t rank, int type, bool few, int parts)
{
    Room r;
    r.T = a.take(M * width_of(rank, few, parts) * (few ? 4 : 2));
    r.far = type == HG_F16 && !few ? a.take(M * up8(rank) * 4) : nullptr;
    return r;
}

// The largest tiles that may be taken: 256×256 ones add the terms of whole
// eights only.
int most_tile_of(int64_t rank) { return rank % 8 == 0 ? 256 : 128; }

struct Beside {
    const hg_adapters *l;
    const hg_matrix *X, *Y;
    int64_t M, N, K;

    bool any() const { return l->count > 0 && l->rank > 0; }
    static bool strides(const void *p, int64_t ld, int64_t stride, int64_t cols, bool touched)
    {
        return ld >= std::max<int64_t>(1, cols) && ld <= HG_LINEAR_MAX_LD && stride >= 0 &&
               stride <= HG_ADAPTERS_MAX_STRIDE && !(touched && p == nullptr) &&
               (reinterpret_cast<uintptr_t>(p) & 1) == 0;
    }
    int valid() const
    {
        if (l == nullptr || l->count < 0 || l->count > HG_ADAPTERS_MAX_COUNT || l->rank < 0 ||
            l->rank > HG_ADAPTERS_MAX_RANK || l->type != X->type)
            return -11;
        if (!any())
            return HG_OK;
        const bool touched = M > 0 && N > 0 && K > 0;
        if (!strides(l->A, l->lda, l->stride_a, K, touched) || !strides(l->B, l->ldb, l->stride_b, l->rank, touched) ||
            (touched && l->which == nullptr) || (reinterpret_cast<uintptr_t>(l->which) & 7) != 0 ||
            (reinterpret_cast<uintptr_t>(l->scales) & 3) != 0)
            return -11;
        return HG_OK;
    }
    bool meets(const Span &s) const
    {
        if (!any())
            return false;
        const int64_t last = l->count - 1, r = l->rank;
        return any_meet({s}, {span_of(l->which, M * 8), span_of(l->scales, l->count * 4),
                              span_of(l->A, (last * l->stride_a + (r - 1) * l->lda + K) * 2),
                              span_of(l->B, (last * l->stride_b + (N - 1) * l->ldb + r) * 2)});
    }
    bool direct_rows() const
    {
        return direct(X, K) && l->lda % 8 == 0 && l->stride_a % 8 == 0 && l->lda <= 2 * (int64_t)HG_LINEAR_MAX_WIDTH &&
               (reinterpret_cast<uintptr_t>(l->A) & 15) == 0;
    }
    int check(const Span &y, const Span &z, const Span &zs) const
    {
        return meets(y) || meets(z) || meets(zs) ? -11 : HG_OK;
    }
    int most_tile() const { return any() ? most_tile_of(l->rank) : 256; }
    int parts() const { return parts_of(X->type, Y->type == HG_F32); }
    Room room(Arena &a, const LinearPlan &q) const
    {
        return any() ? room_of(a, M, l->rank, X->type, q.cut.tile == 0, parts()) : Room{nullptr, nullptr};
    }
    hipError_t begin(lin::Product &p, Arena &a, const LinearPlan &q, bool bf16, hipStream_t s) const
    {
        if (!any())
            return hipSuccess;
        const Room to = room(a, q);
        const bool few = q.cut.tile == 0;
        // (see OwnSums of hg_linear_rowwise.hip)
        if (few && q.direct && lin::weight_blocks(N, p.f.save == lin::kSave8) == 1 && M == 1 && l->rank <= lin::kOwnRank &&
            (N + 15) / 16 <= hg::cu_count()) {
            p.ad = {l->which, static_cast<const uint16_t *>(l->B), nullptr, nullptr, l->stride_b, l->ldb, 0, (int32_t)l->count, l->rank, 2};
            p.own = static_cast<const uint16_t *>(l->A);
            p.own_scales = l->scales;
            p.own_stride = l->stride_a;
            p.own_ld = l->lda;
            return hipSuccess;
        }
        const int64_t ldt = width_of(l->rank, few, parts());
        float *const far = static_cast<float *>(to.far);
        p.ad = {l->which, static_cast<const uint16_t *>(l->B), to.T, far, l->stride_b, l->ldb, ldt, (int32_t)l->count, l->rank,
                parts()};
        return lin::launch_shrink({static_cast<const uint16_t *>(X->data), static_cast<const uint16_t *>(l->A), l->which,
                                   l->scales, to.T, far, X->ld, l->lda, l->stride_a, ldt, (int32_t)M, (int32_t)K,
                                   (int32_t)l->count, l->rank, parts(), few, direct_rows()},
                                  bf16, s);
    }
};

}  // namespace

extern "C" {

int64_t hg_linear_adapters_workspace_size(int64_t M, int64_t N, int64_t K, int64_t rank, const hg_matrix *X,
                                          const hg_matrix *W)
{
    // (for Y of either type)
    const int most = most_tile_of(rank);
    const int64_t need = linear_room(M, N, K, X, W, most, [&](Arena &a, const LinearPlan &q) {
        room_of(a, M, rank, X->type, q.cut.tile == 0, parts_of(X->type, true));
    });
    if (need < 0 && need > -4)
        return need;
    if (rank < 0 || rank > HG_ADAPTERS_MAX_RANK)
        return -4;
    if (need < 0)
        return need - 1;
    // A call may have no adapters, whatever their rank; the layer's tiles may be larger then.
    return most == 256 ? need : std::max(need, linear_room(M, N, K, X, W));
}

int hg_linear_adapters(int act, int64_t M, int64_t N, int64_t K, const hg_matrix *X, const hg_matrix *W,
                       const float *bias, const hg_matrix *R, const hg_matrix *Y, const hg_matrix *Z,
                       const hg_adapters *adapters, void *work, int64_t work_bytes, void *stream)
{
    return linear_call<-12>(act, M, N, K, X, W, bias, R, Y, Z, Beside{adapters, X, Y, M, N, K}, work, work_bytes, stream);
}

}  // extern "C"
