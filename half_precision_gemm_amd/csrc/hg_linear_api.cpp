// hg_linear_api.cpp — host side of the C ABI declared in
// include/hgemm_linear.h: argument checks, workspace layout, kernel choice.
#include "hgemm_linear.h"

#include <stdint.h>

#include <algorithm>
#include <initializer_list>

#include "hg_linear.h"

namespace {

namespace lin = hg::lin;

constexpr int64_t kBK = 64;                       // k per stage of the product kernels

int status_of(hipError_t e) { return e == hipSuccess ? HG_OK : HG_ERR_HIP_BASE + (int)e; }

bool is16(int type) { return type == HG_F16 || type == HG_BF16; }
int64_t up8(int64_t n) { return (n + 7) / 8 * 8; }
int64_t blocks8(int64_t n) { return (n + HG_E4M3_BLOCK - 1) / HG_E4M3_BLOCK; }
int64_t esize(int type) { return type == HG_F32 ? 4 : type == HG_E4M3 ? 1 : 2; }

// Bytes [lo, hi); empty when lo == hi.
struct Span {
    uintptr_t lo, hi;
};
bool meet(const Span &a, const Span &b) { return a.lo < a.hi && b.lo < b.hi && a.lo < b.hi && b.lo < a.hi; }
Span span_of(const void *p, int64_t bytes)
{
    const uintptr_t lo = reinterpret_cast<uintptr_t>(p);
    return p == nullptr || bytes <= 0 ? Span{0, 0} : Span{lo, lo + (uintptr_t)bytes};
}
Span data_span(const hg_matrix *m, int64_t rows, int64_t cols)
{
    if (m == nullptr || rows <= 0 || cols <= 0)
        return {0, 0};
    return span_of(m->data, ((rows - 1) * m->ld + cols) * esize(m->type));
}
Span scale_span(const hg_matrix *m, int64_t rows, int64_t cols)
{
    if (m == nullptr || m->type != HG_E4M3 || rows <= 0 || cols <= 0)
        return {0, 0};
    return span_of(m->scales, (rows - 1) * m->lds + blocks8(cols));
}
bool any_meet(std::initializer_list<Span> a, std::initializer_list<Span> b)
{
    for (const Span &x : a)
        for (const Span &y : b)
            if (meet(x, y))
                return true;
    return false;
}

// Whether a matrix's ld (and its scales') is in range, its address a multiple
// of the element's size and, if its elements are touched, not null.
bool valid(const hg_matrix *m, int64_t rows, int64_t cols)
{
    if (m->ld < std::max<int64_t>(1, cols) || m->ld > HG_LINEAR_MAX_LD)
        return false;
    const bool touched = rows > 0 && cols > 0;
    if (touched && m->data == nullptr)
        return false;
    if ((reinterpret_cast<uintptr_t>(m->data) & (uintptr_t)(esize(m->type) - 1)) != 0)
        return false;
    if (m->type == HG_E4M3) {
        if (m->lds < blocks8(cols) || m->lds > HG_LINEAR_MAX_LD)
            return false;
        if (touched && m->scales == nullptr)
            return false;
    }
    return true;
}

bool vec_ok(const void *p, int64_t ld, int64_t each, int64_t bytes)
{
    return reinterpret_cast<uintptr_t>(p) % (uintptr_t)bytes == 0 && ld * each % bytes == 0;
}

// Whether the product kernels can load this 16-bit operand as it is: 16-byte
// pieces of rows whose length is a multiple of 8 (a piece never holds
// elements of the next row or behind the last one), 32-bit offsets in a tile.
bool direct(const hg_matrix *m, int64_t cols)
{
    return cols % 8 == 0 && m->ld % 8 == 0 && m->ld <= 2 * (int64_t)HG_LINEAR_MAX_WIDTH &&
           (reinterpret_cast<uintptr_t>(m->data) & 15) == 0;
}

// Bump allocation of 256-byte multiples; with a null base it only counts.
struct Arena {
    char *base;
    int64_t used = 0;
    void *take(int64_t bytes)
    {
        void *p = base != nullptr ? base + used : nullptr;
        used += (bytes + 255) / 256 * 256;
        return p;
    }
};

// How a product is cut: the tile edge (0: the row-wise product) and the
// slices of its sum.
struct Cut {
    int tile;
    int splits, per;
};
Cut cut_of(int64_t M, int64_t N, int64_t K)
{
    auto tiles_of = [&](int64_t edge) { return ((M + edge - 1) / edge) * ((N + edge - 1) / edge); };
    Cut c;
    c.tile = tiles_of(256) >= hg::cu_count() ? 256 : tiles_of(128) >= 128 ? 128 : 64;
    const int64_t tiles = std::max<int64_t>(1, tiles_of(c.tile)), stages = (K + kBK - 1) / kBK;
    int64_t s = 1;
    if (tiles < hg::cu_count())
        s = std::min<int64_t>({hg::cu_count() / tiles, stages / 8, (int64_t)32});
    s = std::max<int64_t>(s, 1);
    c.per = (int)((stages + s - 1) / s);
    c.splits = c.per > 0 ? (int)((stages + c.per - 1) / c.per) : 1;
    return c;
}
int64_t partial_bytes(const Cut &c, int64_t M, int64_t N)
{
    return c.splits > 1 ? (int64_t)c.splits * M * ((N + 3) / 4 * 4) * 4 : 0;
}

hipError_t run_product(lin::Product &p, const Cut &c, lin::Layout layout, bool bf16, void *partials, hipStream_t s)
{
    p.splits = c.splits;
    p.per = c.per;
    p.P = static_cast<float *>(partials);
    p.ldp = ((int64_t)p.N + 3) / 4 * 4;
    p.f.vec = p.f.cvec && (p.f.R == nullptr || p.f.rvec) && (p.f.Z == nullptr || p.f.zvec);
    if (p.K == 0) {                              // an empty sum
        p.splits = 0;
        return lin::launch_reduce(p, bf16, s);
    }
    if (c.tile == 0)
        return lin::launch_rowwise(p, bf16, s);
    const hipError_t e =
        c.tile == 256 ? lin::launch_tile(p, layout, bf16, s) : lin::launch_ring(p, layout, c.tile, bf16, s);
    return e != hipSuccess || p.splits <= 1 ? e : lin::launch_reduce(p, bf16, s);
}

void set_output(lin::Finish &f, const hg_matrix *Y, int64_t rows, int64_t cols)
{
    f.C = Y->data;
    f.ldc = Y->ld;
    f.out32 = Y->type == HG_F32;
    f.cvec = vec_ok(Y->data, Y->ld, esize(Y->type), 16);
    f.rows = (int32_t)rows;
    f.cols = (int32_t)cols;
}

int check_sizes(int64_t M, int64_t N, int64_t K, int first)
{
    if (M < 0 || M > HG_LINEAR_MAX_ROWS)
        return -first;
    if (N < 0 || N > HG_LINEAR_MAX_WIDTH)
        return -(first + 1);
    if (K < 0 || K > HG_LINEAR_MAX_WIDTH)
        return -(first + 2);
    return HG_OK;
}

bool bad_work(const void *work, int64_t need) { return need > 0 && (work == nullptr || ((uintptr_t)work & 15) != 0); }

// Whether the forward product goes row by row (one launch, W read once, X once
// per 16 or 32 rows of W) rather than by 64×64 tiles with the sum in slices (a
// second launch, X read once per 64).  Up to 16 rows it always wins or comes
// within 3 us; up to 32 or 64 while X is short.  Measured, row-wise against
// tiles, bf16, us (N × K): M = 32: 4096×4096 14.7 / 16.5, 1024×1024 5.4 / 9.1,
// 16384×4096 40.6 / 40.3, 4096×16384 52.9 / 39.7; M = 64: 1024×1024 7.3 / 9.1,
// 4096×4096 22.3 / 16.5.  Operands that the tiles would have to copy first
// (N·K·4 bytes more) go row by row up to 64.
bool few_rows(int64_t M, int64_t K, bool direct)
{
    return M <= 16 || (M <= 32 && K <= 4096) || (M <= lin::kFewRows && (K <= 1024 || !direct));
}

struct LinearPlan {
    bool few;                                     // the row-wise product
    bool copy_x, copy_w;
    Cut cut;
};
LinearPlan plan_linear(int64_t M, int64_t N, int64_t K, const hg_matrix *X, const hg_matrix *W)
{
    LinearPlan q;
    q.few = few_rows(M, K, direct(X, K) && direct(W, K));
    q.copy_x = !q.few && !direct(X, K);
    q.copy_w = !q.few && !direct(W, K);
    q.cut = q.few ? Cut{0, 1, 0} : cut_of(M, N, K);
    return q;
}
struct LinearRoom {
    void *x, *w, *p;
};
LinearRoom room_linear(Arena &a, const LinearPlan &q, int64_t M, int64_t N, int64_t K)
{
    LinearRoom r;
    r.x = a.take(q.copy_x ? M * up8(K) * 2 : 0);
    r.w = a.take(q.copy_w ? N * up8(K) * 2 : 0);
    r.p = a.take(partial_bytes(q.cut, M, N));
    return r;
}

// Rows per strip of the column sums: enough strips to fill the GPU, at least
// 64 rows each; up to 128 rows are one strip (no second launch).
int64_t strip_of(int64_t M, int64_t N)
{
    const int64_t tiles = std::max<int64_t>(1, (N + 255) / 256);
    if (M <= 128)
        return std::max<int64_t>(M, 1);
    const int64_t want = std::max<int64_t>(1, 8 * (int64_t)hg::cu_count() / tiles);
    const int64_t rows = std::max<int64_t>((M + want - 1) / want, 64);
    return std::max((rows + 7) / 8 * 8, (M + 65534) / 65535);
}

struct GradRoom {
    void *dz, *x, *w, *q, *p;
    Cut cx, cw;
    bool copy_w, copy_x;
};
GradRoom room_grad(Arena &a, int64_t M, int64_t N, int64_t K, const hg_matrix *W, const hg_matrix *X)
{
    GradRoom r;
    r.cx = cut_of(M, K, N);
    r.cw = cut_of(N, K, M);
    r.copy_w = W != nullptr && !direct(W, K);
    r.copy_x = X != nullptr && (X->type == HG_E4M3 || !direct(X, K));
    const int64_t strips = M > 0 ? (M + strip_of(M, N) - 1) / strip_of(M, N) : 0;
    r.dz = a.take(M * up8(N) * 2);
    r.x = a.take(r.copy_x ? M * up8(K) * 2 : 0);
    r.w = a.take(r.copy_w ? N * up8(K) * 2 : 0);
    r.q = a.take(strips > 1 ? strips * N * 4 : 0);
    r.p = a.take(std::max(W != nullptr ? partial_bytes(r.cx, M, K) : 0, X != nullptr ? partial_bytes(r.cw, N, K) : 0));
    return r;
}

}  // namespace

extern "C" {

int64_t hg_linear_workspace_size(int64_t M, int64_t N, int64_t K, const hg_matrix *X, const hg_matrix *W)
{
    if (const int e = check_sizes(M, N, K, 1))
        return e;
    if (X == nullptr || !is16(X->type) || !valid(X, 0, K))
        return -4;
    if (W == nullptr || W->type != X->type || !valid(W, 0, K))
        return -5;
    if (M == 0 || N == 0 || K == 0)
        return 0;
    Arena a{nullptr};
    room_linear(a, plan_linear(M, N, K, X, W), M, N, K);
    return a.used;
}

int hg_linear(int act, int64_t M, int64_t N, int64_t K, const hg_matrix *X, const hg_matrix *W, const float *bias,
              const hg_matrix *R, const hg_matrix *Y, const hg_matrix *Z, void *work, int64_t work_bytes, void *stream)
{
    if (act < HG_ACT_NONE || act > HG_ACT_SILU)
        return -1;
    if (const int e = check_sizes(M, N, K, 2))
        return e;
    const int64_t read = M > 0 && N > 0;          // whether anything is computed
    if (X == nullptr || !is16(X->type) || !valid(X, read * M, K))
        return -5;
    if (W == nullptr || W->type != X->type || !valid(W, read * N, K))
        return -6;
    if ((reinterpret_cast<uintptr_t>(bias) & 3) != 0)
        return -7;
    if (Y != nullptr && R != nullptr && (R->type != Y->type || !valid(R, M, N)))
        return -8;
    if (Y == nullptr || (Y->type != X->type && Y->type != HG_F32) || !valid(Y, M, N))
        return -9;
    if (Z != nullptr && ((Z->type != X->type && Z->type != HG_E4M3) || !valid(Z, M, N)))
        return -10;
    if (M == 0 || N == 0)
        return HG_OK;
    const Span sx = data_span(X, M, K), sw = data_span(W, N, K), sb = span_of(bias, N * 4);
    const Span sr = data_span(R, M, N), sy = data_span(Y, M, N), sz = data_span(Z, M, N), ss = scale_span(Z, M, N);
    const bool in_place = R != nullptr && R->data == Y->data && R->ld == Y->ld;
    if (any_meet({sy}, {sx, sw, sb, in_place ? Span{0, 0} : sr}))
        return -9;
    if (any_meet({sz, ss}, {sx, sw, sb, sr, sy}) || meet(sz, ss))
        return -10;
    const LinearPlan q = plan_linear(M, N, K, X, W);
    Arena count{nullptr};
    if (K > 0)
        room_linear(count, q, M, N, K);
    if (bad_work(work, count.used) || any_meet({span_of(work, count.used)}, {sx, sw, sb, sr, sy, sz, ss}))
        return -11;
    if (work_bytes < count.used)
        return -12;

    const hipStream_t s = static_cast<hipStream_t>(stream);
    const bool bf16 = X->type == HG_BF16;
    Arena arena{static_cast<char *>(work)};
    const LinearRoom room = room_linear(arena, q, M, N, K);
    lin::Product p{};
    p.A = static_cast<const uint16_t *>(X->data);
    p.B = static_cast<const uint16_t *>(W->data);
    p.lda = X->ld;
    p.ldb = W->ld;
    p.M = (int32_t)M;
    p.N = (int32_t)N;
    p.K = (int32_t)K;
    set_output(p.f, Y, M, N);
    p.f.act = act;
    p.f.bias = bias;
    if (R != nullptr) {
        p.f.R = R->data;
        p.f.ldr = R->ld;
        p.f.rvec = vec_ok(R->data, R->ld, esize(R->type), 16);
    }
    if (Z != nullptr) {
        p.f.Z = Z->data;
        p.f.ldz = Z->ld;
        p.f.save = Z->type == HG_E4M3 ? lin::kSave8 : lin::kSave16;
        p.f.Zs = Z->scales;
        p.f.ldzs = Z->lds;
        p.f.zvec = Z->type == HG_E4M3 ? vec_ok(Z->data, Z->ld, 1, 8) : vec_ok(Z->data, Z->ld, 2, 16);
    }
    if (K > 0 && q.copy_x) {
        if (const hipError_t e = lin::launch_pad(X->data, X->ld, room.x, up8(K), M, K, s))
            return status_of(e);
        p.A = static_cast<const uint16_t *>(room.x);
        p.lda = up8(K);
    }
    if (K > 0 && q.copy_w) {
        if (const hipError_t e = lin::launch_pad(W->data, W->ld, room.w, up8(K), N, K, s))
            return status_of(e);
        p.B = static_cast<const uint16_t *>(room.w);
        p.ldb = up8(K);
    }
    return status_of(run_product(p, q.cut, lin::Layout::NN, bf16, room.p, s));
}

int64_t hg_linear_grad_workspace_size(int64_t M, int64_t N, int64_t K, const hg_matrix *dY, const hg_matrix *W,
                                      const hg_matrix *X)
{
    if (const int e = check_sizes(M, N, K, 1))
        return e;
    if (dY == nullptr || !is16(dY->type) || !valid(dY, 0, N))
        return -4;
    if (W != nullptr && (W->type != dY->type || !valid(W, 0, K)))
        return -5;
    if (X != nullptr && ((X->type != dY->type && X->type != HG_E4M3) || !valid(X, 0, K)))
        return -6;
    Arena a{nullptr};
    room_grad(a, M, N, K, W, X);
    return a.used;
}

int hg_linear_grad(int act, int64_t M, int64_t N, int64_t K, const hg_matrix *dY, const hg_matrix *W,
                   const hg_matrix *X, const hg_matrix *Z, const hg_matrix *dX, const hg_matrix *dW, float *dbias,
                   int accumulate, void *work, int64_t work_bytes, void *stream)
{
    if (act < HG_ACT_NONE || act > HG_ACT_SILU)
        return -1;
    if (const int e = check_sizes(M, N, K, 2))
        return e;
    const bool want_x = dX != nullptr, want_w = dW != nullptr, need_z = act != HG_ACT_NONE;
    if (dY == nullptr || !is16(dY->type) || !valid(dY, M, N))
        return -5;
    if (want_x ? W == nullptr || W->type != dY->type || !valid(W, M > 0 ? N : 0, K)
               : W != nullptr && (W->type != dY->type || !valid(W, 0, K)))
        return -6;
    if (want_w ? X == nullptr || (X->type != dY->type && X->type != HG_E4M3) || !valid(X, N > 0 ? M : 0, K)
               : X != nullptr && ((X->type != dY->type && X->type != HG_E4M3) || !valid(X, 0, K)))
        return -7;
    if (need_z && (Z == nullptr || (Z->type != dY->type && Z->type != HG_E4M3) || !valid(Z, M, N)))
        return -8;
    if (want_x && (dX->type != dY->type || !valid(dX, M, K)))
        return -9;
    if (want_w && ((dW->type != dY->type && dW->type != HG_F32) || !valid(dW, N, K)))
        return -10;
    if ((reinterpret_cast<uintptr_t>(dbias) & 3) != 0)
        return -11;
    if (accumulate != 0 && accumulate != 1)
        return -12;
    const hg_matrix *Wr = want_x ? W : nullptr, *Xr = want_w ? X : nullptr, *Zr = need_z ? Z : nullptr;
    const Span i0 = data_span(dY, M, N), i1 = data_span(Wr, N, K), i2 = data_span(Xr, M, K), i3 = scale_span(Xr, M, K),
               i4 = data_span(Zr, M, N), i5 = scale_span(Zr, M, N);
    const Span ox = data_span(dX, M, K), ow = data_span(dW, N, K), ob = span_of(dbias, N * 4);
    if (any_meet({ox}, {i0, i1, i2, i3, i4, i5}))
        return -9;
    if (any_meet({ow}, {i0, i1, i2, i3, i4, i5, ox}))
        return -10;
    if (any_meet({ob}, {i0, i1, i2, i3, i4, i5, ox, ow}))
        return -11;
    Arena count{nullptr};
    room_grad(count, M, N, K, Wr, Xr);
    const Span wk = span_of(work, count.used);
    if (bad_work(work, count.used) || any_meet({wk}, {i0, i1, i2, i3, i4, i5, ox, ow, ob}))
        return -13;
    if (work_bytes < count.used)
        return -14;

    const hipStream_t s = static_cast<hipStream_t>(stream);
    const bool bf16 = dY->type == HG_BF16;
    if (M == 0 || N == 0) {                       // empty sums
        if (want_x && M > 0 && K > 0)
            if (const hipError_t e = lin::launch_zero(dX->data, dX->ld, M, K, false, s))
                return status_of(e);
        if (N == 0 || accumulate)
            return HG_OK;
        if (want_w && K > 0)
            if (const hipError_t e = lin::launch_zero(dW->data, dW->ld, N, K, dW->type == HG_F32, s))
                return status_of(e);
        return dbias != nullptr ? status_of(lin::launch_zero(dbias, N, 1, N, true, s)) : HG_OK;
    }
    Arena arena{static_cast<char *>(work)};
    const GradRoom room = room_grad(arena, M, N, K, Wr, Xr);

    // dZ and the bias's gradient.  Without an activation dZ is dY, which the
    // products read themselves if it is aligned.
    const bool products = (want_x || want_w) && K > 0;
    const bool own_dz = products && (need_z || !direct(dY, N));
    if (own_dz || dbias != nullptr) {
        lin::Slope g{};
        g.dY = dY->data;
        g.lddy = dY->ld;
        g.yvec = vec_ok(dY->data, dY->ld, 2, 16);
        g.act = act;
        if (need_z) {
            g.Z = Z->data;
            g.ldz = Z->ld;
            g.Zs = Z->scales;
            g.ldzs = Z->lds;
            g.save = Z->type == HG_E4M3 ? lin::kSave8 : lin::kSave16;
            g.zvec = Z->type == HG_E4M3 ? vec_ok(Z->data, Z->ld, 1, 8) : vec_ok(Z->data, Z->ld, 2, 16);
        }
        g.D = own_dz ? room.dz : nullptr;
        g.ldd = up8(N);
        g.rows = M;
        g.cols = N;
        g.strip = strip_of(M, N);
        const int64_t strips = (M + g.strip - 1) / g.strip;
        if (dbias != nullptr) {
            g.Q = strips > 1 ? static_cast<float *>(room.q) : nullptr;
            g.db = dbias;
        }
        g.accumulate = accumulate;
        if (const hipError_t e = lin::launch_slope(g, bf16, s))
            return status_of(e);
        if (dbias != nullptr && strips > 1)
            if (const hipError_t e = lin::launch_sum_strips(g.Q, strips, N, dbias, accumulate != 0, s))
                return status_of(e);
    }
    if (!products)
        return HG_OK;
    const uint16_t *dz = static_cast<const uint16_t *>(own_dz ? room.dz : dY->data);
    const int64_t lddz = own_dz ? up8(N) : dY->ld;

    if (want_x) {                                 // dX (M×K) = dZ (M×N) · W (N×K, summed over its rows)
        lin::Product p{};
        p.A = dz;
        p.lda = lddz;
        p.B = static_cast<const uint16_t *>(W->data);
        p.ldb = W->ld;
        if (room.copy_w) {
            if (const hipError_t e = lin::launch_pad(W->data, W->ld, room.w, up8(K), N, K, s))
                return status_of(e);
            p.B = static_cast<const uint16_t *>(room.w);
            p.ldb = up8(K);
        }
        p.M = (int32_t)M;
        p.N = (int32_t)K;
        p.K = (int32_t)N;
        set_output(p.f, dX, M, K);
        if (const hipError_t e = run_product(p, room.cx, lin::Layout::NT, bf16, room.p, s))
            return status_of(e);
    }
    if (want_w) {                                 // dW (N×K) = dZᵀ · X, both summed over their rows
        lin::Product p{};
        p.A = dz;
        p.lda = lddz;
        p.B = static_cast<const uint16_t *>(X->data);
        p.ldb = X->ld;
        if (room.copy_x) {
            const hipError_t e =
                X->type == HG_E4M3
                    ? lin::launch_read8(static_cast<const uint8_t *>(X->data), X->ld, X->scales, X->lds, room.x, up8(K),
                                        M, K, up8(K), bf16, s)
                    : lin::launch_pad(X->data, X->ld, room.x, up8(K), M, K, s);
            if (e != hipSuccess)
                return status_of(e);
            p.B = static_cast<const uint16_t *>(room.x);
            p.ldb = up8(K);
        }
        p.M = (int32_t)N;
        p.N = (int32_t)K;
        p.K = (int32_t)M;
        set_output(p.f, dW, N, K);
        if (accumulate) {
            p.f.R = dW->data;
            p.f.ldr = dW->ld;
            p.f.rvec = p.f.cvec;
        }
        return status_of(run_product(p, room.cw, lin::Layout::TT, bf16, room.p, s));
    }
    return HG_OK;
}

int hg_checkpoint8_write(int64_t M, int64_t N, const hg_matrix *X, const hg_matrix *C, void *stream)
{
    if (const int e = check_sizes(M, N, 0, 1))
        return e;
    if (X == nullptr || !is16(X->type) || !valid(X, M, N))
        return -3;
    if (C == nullptr || C->type != HG_E4M3 || !valid(C, M, N))
        return -4;
    const Span c = data_span(C, M, N), z = scale_span(C, M, N);
    if (any_meet({c, z}, {data_span(X, M, N)}) || meet(c, z))
        return -4;
    if (M == 0 || N == 0)
        return HG_OK;
    return status_of(lin::launch_write8(X->data, X->ld, static_cast<uint8_t *>(C->data), C->ld, C->scales, C->lds, M, N,
                                        X->type == HG_BF16, static_cast<hipStream_t>(stream)));
}

int hg_checkpoint8_read(int64_t M, int64_t N, const hg_matrix *C, const hg_matrix *X, void *stream)
{
    if (const int e = check_sizes(M, N, 0, 1))
        return e;
    if (C == nullptr || C->type != HG_E4M3 || !valid(C, M, N))
        return -3;
    if (X == nullptr || !is16(X->type) || !valid(X, M, N))
        return -4;
    if (any_meet({data_span(X, M, N)}, {data_span(C, M, N), scale_span(C, M, N)}))
        return -4;
    if (M == 0 || N == 0)
        return HG_OK;
    return status_of(lin::launch_read8(static_cast<const uint8_t *>(C->data), C->ld, C->scales, C->lds, X->data, X->ld,
                                       M, N, N, X->type == HG_BF16, static_cast<hipStream_t>(stream)));
}

}  // extern "C"
