// hg_linear_api.cpp — host side of the C ABI declared in
// include/hgemm_linear.h: argument checks, workspace layout, kernel choice (what
// the forward call needs of these: hg_linear_host.h).
#include "hgemm_linear.h"

#include <stdint.h>

#include <algorithm>
#include <initializer_list>

#include "hg_linear.h"
#include "hg_linear_host.h"

using namespace hg::host;

namespace {

namespace lin = hg::lin;

// Two products in one launch, their sums in sa and sb slices.  128×128 tiles
// take 6.0 + 0.62 there: a k-major operand takes twice the LDS reads (64×64 /
// 128×128, M × N × K: 4000×500×700 33.6 / 39.8 us, 900×900×2500 38.7 / 43.0,
// 777×1000×1304 26.6 / 25.5, 2048×2048×2048 80.9 / 63.8).
double expected_us(int64_t cus, int tile, const Shape &a, int sa, const Shape &b, int sb)
{
    const int64_t na = a.tiles(tile) * sa, nb = b.tiles(tile) * sb, items = na + nb;
    const Rate r = tile == 128 ? Rate{6.0, 0.62, cus} : rate_of(cus, tile, items);
    const double ta = r.fix + r.stage * (double)((a.stages() + sa - 1) / sa);
    const double tb = r.fix + r.stage * (double)((b.stages() + sb - 1) / sb);
    // Equal items go in rounds; unequal ones fill up after each other.
    const double work = (double)na * ta + (double)nb * tb;
    const double run = ta < 1.25 * tb && tb < 1.25 * ta
                           ? (double)((items + r.slots - 1) / r.slots) * work / (double)std::max<int64_t>(items, 1)
                           : work / (double)r.slots + 0.25 * std::min(ta, tb);
    const double reduce = reduce_us(a.tiles(tile), tile, sa) + reduce_us(b.tiles(tile), tile, sb);
    return 2.0 + std::max({run, ta, tb}) + (sa > 1 && sb > 1 ? reduce - 3.0 : reduce);
}
// Whether a weight's gradient (b: its rows, its columns, the rows it is summed
// over) is written along its rows (hg_linear_outer.hip) in a launch of its own:
// few rows, and many more tiles than the GPU takes at once (gradients, tiles of
// 64×64 / along the rows, us: 60×3840×1336, 1260 tiles, 22.9 / 24.2,
// 2×512×16384, 2048, 24.8 / 16.7, 16×4096×4096 32.4 / 27.2, 3×2644×13440 62.3 /
// 44.4, 8×8192×8192 85.8 / 66.9).
bool along_rows(const Shape &b)
{
    return b.K <= lin::kFewRows && b.tiles(64) > 6 * (int64_t)hg::cu_count();
}
// Two products: each on its own if either is best on 256×256 tiles, else
// together on one smaller edge.  (One launch for 256×256 tiles of both kinds
// was slower: side by side they share less in L2, 8192×2048 with 4096 rows
// 225 -> 270 us.)
void best_cuts(const Shape &a, const Shape &b, Cut &ca, Cut &cb)
{
    const int64_t cus = hg::cu_count();
    double ua, ub;
    ca = best_cut(a, &ua);
    if (along_rows(b)) {
        cb = {0, 0, 1, 0};
        return;
    }
    cb = best_cut(b, &ub);
    double least = ca.tile == 256 || cb.tile == 256 ? ua + ub : -1.0;
    for (int tile : {64, 128})
        for (int sa : kSlices) {
            if (!may_slice(cus, a.tiles(tile), a, sa))
                break;
            for (int sb : kSlices) {
                if (!may_slice(cus, b.tiles(tile), b, sb) || !may_launch(tile, a.tiles(tile) * sa + b.tiles(tile) * sb))
                    break;
                const double c = expected_us(cus, tile, a, sa, b, sb);
                if (least < 0.0 || c < least) {
                    least = c;
                    ca = cut_into(tile, a, 0, sa);
                    cb = cut_into(tile, b, 0, sb);
                }
            }
        }
    if (least < 0.0) {                            // too many items for one launch
        ca = cut_into(256, a, 0, 1);
        cb = cut_into(256, b, 0, 1);
    }
}
// Rows per strip of the column sums: enough strips to fill the GPU, at least
// 64 rows each; up to 128 rows are one strip, which ends the sums itself.
int64_t strip_of(int64_t M, int64_t N)
{
    const int64_t tiles = std::max<int64_t>(1, (N + 127) / 128);
    if (M <= 128)
        return std::max<int64_t>(M, 1);
    const int64_t want = std::max<int64_t>(1, 16 * (int64_t)hg::cu_count() / tiles);
    const int64_t rows = std::max<int64_t>((M + want - 1) / want, 64);
    return (rows + 63) / 64 * 64;
}

struct GradRoom {
    void *dz, *x, *w, *q, *px, *pw;
    Cut cx, cw;
    bool copy_w, copy_x;
};
GradRoom room_grad(Arena &a, int64_t M, int64_t N, int64_t K, const hg_matrix *W, const hg_matrix *X)
{
    GradRoom r;
    r.cx = r.cw = {64, 0, 1, 0};
    const Shape x{M, K, N}, w{N, K, M};
    if (W != nullptr && X != nullptr)
        best_cuts(x, w, r.cx, r.cw);
    else if (W != nullptr)
        r.cx = best_cut(x);
    else if (X != nullptr)
        r.cw = along_rows(w) ? Cut{0, 0, 1, 0} : best_cut(w);
    r.copy_w = W != nullptr && !direct(W, K);
    r.copy_x = X != nullptr && (X->type == HG_E4M3 || !direct(X, K));
    const int64_t strips = M > 0 ? (M + strip_of(M, N) - 1) / strip_of(M, N) : 0;
    r.dz = a.take(M * up8(N) * 2);
    r.x = a.take(r.copy_x ? M * up8(K) * 2 : 0);
    r.w = a.take(r.copy_w ? N * up8(K) * 2 : 0);
    r.q = a.take(strips > 1 ? strips * N * 4 : 0);
    r.px = a.take(W != nullptr ? partial_bytes(r.cx, x) : 0);
    r.pw = a.take(X != nullptr ? partial_bytes(r.cw, w) : 0);
    return r;
}

}  // namespace

extern "C" {

int64_t hg_linear_workspace_size(int64_t M, int64_t N, int64_t K, const hg_matrix *X, const hg_matrix *W)
{
    return linear_room(M, N, K, X, W);
}

int hg_linear(int act, int64_t M, int64_t N, int64_t K, const hg_matrix *X, const hg_matrix *W, const float *bias,
              const hg_matrix *R, const hg_matrix *Y, const hg_matrix *Z, void *work, int64_t work_bytes, void *stream)
{
    return linear_call<-11>(act, M, N, K, X, W, bias, R, Y, Z, Nothing{}, work, work_bytes, stream);
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
    // A call for one of the gradients may cut its product differently.
    Arena both{nullptr}, x{nullptr}, w{nullptr};
    room_grad(both, M, N, K, W, X);
    room_grad(x, M, N, K, W, nullptr);
    room_grad(w, M, N, K, nullptr, X);
    return std::max({both.used, x.used, w.used});
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

    // dZ, its column sums, and the operands that the products cannot load as
    // they are.  Without an activation dZ is dY, which the products read
    // themselves if it is aligned.
    const bool products = K > 0;
    const bool own_dz = products && (want_x || want_w) && (need_z || !direct(dY, N));
    lin::Slope g{};
    lin::Strips b{};
    if (own_dz || dbias != nullptr) {
        g.dY = dY->data;
        g.lddy = dY->ld;
        g.act = act;
        if (need_z) {
            g.Z = Z->data;
            g.ldz = Z->ld;
            g.Zs = Z->scales;
            g.ldzs = Z->lds;
            g.save = Z->type == HG_E4M3 ? lin::kSave8 : lin::kSave16;
        }
        g.D = own_dz ? room.dz : nullptr;
        g.ldd = up8(N);
        g.rows = M;
        g.cols = N;
        g.strip = strip_of(M, N);
        g.accumulate = accumulate;
        if (dbias != nullptr) {
            const int64_t strips = (M + g.strip - 1) / g.strip;
            if (strips > 1) {
                g.Q = static_cast<float *>(room.q);
                b = {g.Q, dbias, strips, N, accumulate};
            } else {
                g.db = dbias;
            }
        }
    }
    lin::Copy cx{}, cw{};
    if (products && room.copy_x)
        cx = copy_of(X, M, K, room.x);
    if (products && room.copy_w)
        cw = copy_of(W, N, K, room.w);
    if (const hipError_t e = lin::launch_prepare(g, cx, cw, bf16, s))
        return status_of(e);

    lin::Product px{}, pw{};
    px.A = pw.A = static_cast<const uint16_t *>(own_dz ? room.dz : dY->data);
    px.lda = pw.lda = own_dz ? up8(N) : dY->ld;
    const bool do_x = want_x && products, do_w = want_w && products;
    if (do_x) {                                   // dX (M×K) = dZ (M×N) · W (N×K, summed over its rows)
        px.B = static_cast<const uint16_t *>(room.copy_w ? room.w : W->data);
        px.ldb = room.copy_w ? up8(K) : W->ld;
        px.M = (int32_t)M;
        px.N = (int32_t)K;
        px.K = (int32_t)N;
        set_output(px.f, dX, M, K);
        set_cut(px, room.cx, room.px);
    }
    if (do_w) {                                   // dW (N×K) = dZᵀ · X, both summed over their rows
        pw.B = static_cast<const uint16_t *>(room.copy_x ? room.x : X->data);
        pw.ldb = room.copy_x ? up8(K) : X->ld;
        pw.M = (int32_t)N;
        pw.N = (int32_t)K;
        pw.K = (int32_t)M;
        set_output(pw.f, dW, N, K);
        if (accumulate) {
            pw.f.R = dW->data;
            pw.f.ldr = dW->ld;
        }
        set_cut(pw, room.cw, room.pw);
    }
    const bool big_x = do_x && room.cx.tile == 256, big_w = do_w && room.cw.tile == 256;
    const bool outer = do_w && room.cw.tile == 0, pair_w = do_w && !big_w && !outer;
    const int edge = do_x && !big_x ? room.cx.tile : pair_w ? room.cw.tile : 64;
    const lin::Product *one = do_x && !big_x ? &px : nullptr, *two = pair_w ? &pw : nullptr;
    if (const hipError_t e = lin::launch_ring_pair(one, two, b, edge, bf16, s))
        return status_of(e);
    if (outer)
        if (const hipError_t e = lin::launch_outer(pw, bf16, s))
            return status_of(e);
    if (big_x)
        if (const hipError_t e = lin::launch_tile(px, lin::Layout::NT, bf16, s))
            return status_of(e);
    if (big_w)
        if (const hipError_t e = lin::launch_tile(pw, lin::Layout::TT, bf16, s))
            return status_of(e);
    return status_of(lin::launch_reduce(do_x && px.splits > 1 ? &px : nullptr, do_w && pw.splits > 1 ? &pw : nullptr,
                                        bf16, s));
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
                                       M, N, X->type == HG_BF16, static_cast<hipStream_t>(stream)));
}

}  // extern "C"
