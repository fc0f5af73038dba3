// hg_linear_host.h — the host side that hg_linear and hg_linear_adapters share:
// argument checks, workspace layout, kernel choice, the launches of a forward
// product.  Not part of the public ABI.
#pragma once

#include <stdint.h>

#include <algorithm>
#include <initializer_list>

#include "hgemm_linear.h"

#include "hg_linear.h"

namespace hg {
namespace host {

constexpr int64_t kBK = 64;                       // k per stage of the product kernels

inline int status_of(hipError_t e) { return e == hipSuccess ? HG_OK : HG_ERR_HIP_BASE + (int)e; }

inline bool is16(int type) { return type == HG_F16 || type == HG_BF16; }
inline int64_t up8(int64_t n) { return (n + 7) / 8 * 8; }
inline int64_t blocks8(int64_t n) { return (n + HG_E4M3_BLOCK - 1) / HG_E4M3_BLOCK; }
inline int64_t esize(int type) { return type == HG_F32 ? 4 : type == HG_E4M3 ? 1 : 2; }

// Bytes [lo, hi), empty when lo == hi; of a matrix its first `width` bytes of
// every `pitch`.
struct Span {
    uintptr_t lo, hi;
    uint64_t width, pitch;
};
// Different columns of one array (two matrices of the same pitch) do not meet.
inline bool meet(const Span &a, const Span &b)
{
    if (!(a.lo < a.hi && b.lo < b.hi && a.lo < b.hi && b.lo < a.hi))
        return false;
    if (a.pitch != b.pitch)
        return true;
    const Span &l = a.lo <= b.lo ? a : b, &h = a.lo <= b.lo ? b : a;
    const uint64_t d = (uint64_t)(h.lo - l.lo) % a.pitch;
    return d < l.width || d + h.width > a.pitch;
}
inline Span span_of(const void *p, int64_t bytes)
{
    const uintptr_t lo = reinterpret_cast<uintptr_t>(p);
    if (p == nullptr || bytes <= 0)
        return {0, 0, 0, 1};
    return {lo, lo + (uintptr_t)bytes, (uint64_t)bytes, (uint64_t)bytes};
}
inline Span rows_of(const void *p, int64_t rows, int64_t pitch, int64_t width)
{
    Span s = span_of(p, (rows - 1) * pitch + width);
    s.width = (uint64_t)width;
    s.pitch = (uint64_t)pitch;
    return s;
}
inline Span data_span(const hg_matrix *m, int64_t rows, int64_t cols)
{
    if (m == nullptr || rows <= 0 || cols <= 0)
        return span_of(nullptr, 0);
    return rows_of(m->data, rows, m->ld * esize(m->type), cols * esize(m->type));
}
inline Span scale_span(const hg_matrix *m, int64_t rows, int64_t cols)
{
    if (m == nullptr || m->type != HG_E4M3 || rows <= 0 || cols <= 0)
        return span_of(nullptr, 0);
    return rows_of(m->scales, rows, m->lds, blocks8(cols));
}
inline bool any_meet(std::initializer_list<Span> a, std::initializer_list<Span> b)
{
    for (const Span &x : a)
        for (const Span &y : b)
            if (meet(x, y))
                return true;
    return false;
}

// Whether a matrix's ld (and its scales') is in range, its address a multiple
// of the element's size and, if its elements are touched, not null.
inline bool valid(const hg_matrix *m, int64_t rows, int64_t cols)
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

// Whether the product kernels can load this 16-bit operand as it is: 16-byte
// pieces of rows whose length is a multiple of 8 (a piece never holds
// elements of the next row or behind the last one), 32-bit offsets in a tile.
inline bool direct(const hg_matrix *m, int64_t cols)
{
    return cols % 8 == 0 && m->ld % 8 == 0 && m->ld <= 2 * (int64_t)HG_LINEAR_MAX_WIDTH &&
           (reinterpret_cast<uintptr_t>(m->data) & 15) == 0;
}

// Whether a row of a 16-bit matrix may begin at an address that no 32-bit word
// begins at.
inline bool odd_rows(const hg_matrix *m, int64_t rows)
{
    return (reinterpret_cast<uintptr_t>(m->data) & 3) != 0 || (rows > 1 && m->ld % 2 != 0);
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

// How a product is cut: the tile edge (0: the forms for few rows), the tiles that
// are computed in one piece, and the slices of the others' sums.
struct Cut {
    int tile;
    int64_t whole;
    int splits, per;
};
struct Shape {
    int64_t M, N, K;
    int64_t stages() const { return (K + kBK - 1) / kBK; }
    int64_t tiles(int edge) const { return ((M + edge - 1) / edge) * ((N + edge - 1) / edge); }
};

// What the kernels measured on a 256-CU MI355X (graph replays, bf16, operands in
// the last-level cache), in us.  A work item (a tile, or a slice of its sum)
// takes `fix` + `stage` per 64 of the sum, as many at once as the GPU has room
// for:
//
//    edge   alone on its CUs          GPU full                  items per CU
//     64    1.0 + 0.265 / stage       3.2 + 0.45 / stage        2
//    128    5.0 + 0.55                the same                  1
//    256    7.0 + 1.05                13.0 + 1.4 (power, stores) 1
//
// and slices cost a second launch and their partial sums' way through memory:
// 3 us + bytes at 5 TB/s.  Both sides of the choices this makes, measured (M ×
// N × K, us): 1000×1000×1000 64×64 tiles 9.0, in two slices 15.4, 128×128 15.3;
// 128×1024×8192 one slice 33.9, eight 13.8; 2048×4096×4096 128×128 80.3,
// 256×256 in two slices 72.9; 2000×6000×4000 128×128 125, 256×256 91.8;
// 512×4096×4096 64×64 28.3, 128×128 in two slices 30.7.
struct Rate {
    double fix, stage;
    int64_t slots;
};
inline Rate rate_of(int64_t cus, int tile, int64_t items)
{
    const double fill = std::min(1.0, (double)items / (double)cus);
    if (tile == 64)
        return items > cus ? Rate{3.2, 0.45, 2 * cus} : Rate{1.0, 0.265, cus};
    return tile == 128 ? Rate{5.0, 0.55, cus} : Rate{7.0 + 6.0 * fill, 1.05 + 0.35 * fill, cus};
}
inline double reduce_us(int64_t tiles, int tile, int s)
{
    return s > 1 && tiles > 0 ? 3.0 + (double)tiles * (double)s * (double)tile * (double)tile * 8.0 / 5e6 : 0.0;
}
// One product, its tiles from `whole` on in s slices.
inline double expected_us(int64_t cus, int tile, const Shape &p, int64_t whole, int s)
{
    const int64_t tiles = p.tiles(tile), rest = tiles - whole;
    const Rate r = rate_of(cus, tile, whole + rest * s);
    const double one = r.fix + r.stage * (double)p.stages(), part = r.fix + r.stage * (double)((p.stages() + s - 1) / s);
    return 2.0 + (double)((whole + r.slots - 1) / r.slots) * one + (double)((rest * s + r.slots - 1) / r.slots) * part +
           reduce_us(rest, tile, s);
}
inline Cut cut_into(int tile, const Shape &p, int64_t whole, int s)
{
    Cut c;
    c.tile = tile;
    c.per = (int)((p.stages() + s - 1) / s);
    c.splits = c.per > 0 ? (int)((p.stages() + c.per - 1) / c.per) : 1;
    c.whole = c.splits > 1 ? whole : p.tiles(tile);
    return c;
}
// Numbers of slices that are tried, as long as a slice has at least four stages
// and the cut tiles' items are no more than the GPU holds twice.
constexpr int kSlices[] = {1, 2, 3, 4, 6, 8, 12, 16, 24, 32};
inline bool may_slice(int64_t cus, int64_t tiles, const Shape &p, int s)
{
    return s == 1 || (p.stages() >= 4 * s && tiles * s <= 2 * cus);
}

// Whether so many items, and the blocks that end column sums, fit one launch (the
// 256×256 kernel walks its tiles and has no such limit).
inline bool may_launch(int tile, int64_t items)
{
    return tile == 256 || items + (HG_LINEAR_MAX_WIDTH + 31) / 32 <= lin::kMostBlocks;
}

// A product's tiles are cut all, none, or only those of the last round, which
// would leave most of the GPU idle (1729×10332×14080, 287 tiles of 256×256 on 256
// CUs: none 698 us).  most: the largest edge.
inline Cut best_cut(const Shape &p, double *us = nullptr, int most = 256)
{
    const int64_t cus = hg::cu_count();
    Cut best{64, 0, 1, 0};
    double least = 0.0;
    bool first = true;
    for (int tile : {64, 128, 256}) {
        if (tile > most)
            break;
        const int64_t tiles = p.tiles(tile), slots = tile == 64 ? 2 * cus : cus, full = tiles / slots * slots;
        for (int64_t whole : {(int64_t)0, full}) {
            if (whole > 0 && whole == tiles)
                break;
            for (int s : kSlices) {
                if (!may_slice(cus, tiles - whole, p, s) || !may_launch(tile, whole + (tiles - whole) * s))
                    break;
                const double c = expected_us(cus, tile, p, whole, s);
                if (first || c < least) {
                    least = c;
                    best = cut_into(tile, p, whole, s);
                    first = false;
                }
            }
            if (full == 0)
                break;
        }
    }
    if (us != nullptr)
        *us = least;
    return best;
}
inline int64_t partial_bytes(const Cut &c, const Shape &p)
{
    return c.splits > 1 ? (p.tiles(c.tile) - c.whole) * c.splits * c.tile * c.tile * 4 : 0;
}
inline void set_cut(lin::Product &p, const Cut &c, void *partials)
{
    p.edge = c.tile;
    p.whole = (int32_t)c.whole;
    p.splits = c.splits;
    p.per = c.per;
    p.P = static_cast<float *>(partials);
}

inline void set_output(lin::Finish &f, const hg_matrix *Y, int64_t rows, int64_t cols)
{
    f.C = Y->data;
    f.ldc = Y->ld;
    f.out32 = Y->type == HG_F32;
    f.rows = (int32_t)rows;
    f.cols = (int32_t)cols;
}

inline int check_sizes(int64_t M, int64_t N, int64_t K, int first)
{
    if (M < 0 || M > HG_LINEAR_MAX_ROWS)
        return -first;
    if (N < 0 || N > HG_LINEAR_MAX_WIDTH)
        return -(first + 1);
    if (K < 0 || K > HG_LINEAR_MAX_WIDTH)
        return -(first + 2);
    return HG_OK;
}

inline bool bad_work(const void *work, int64_t need) { return need > 0 && (work == nullptr || ((uintptr_t)work & 15) != 0); }

// Whether the forward product of M <= kFewRows rows goes row by row: one
// launch that reads W once, but X once for every 16 or 32 rows of W (a block).
// What it takes, in us, from measurements with weights out of HBM, bf16: the
// CUs take the blocks in rounds;
//   through LDS, ns per k of a round: (0.85 + 0.42·fill) per 16 rows of W and
//     0.33 per 16 of X, fill the part of the CUs that is busy; 2.5 us to begin
//     with, in every round if X's rings leave no room for a second workgroup
//     (with one, a last round that is not full costs half of one more);
//   through registers, ns per 16 rows of W and k: 1.15, and 0.045 for every row
//     of X (rounded up to 16 from 17 on).
// Tiles are priced with weights out of HBM, as a model's weights are: 3 us more
// than out of the last-level cache, and 4.6 TB/s at best.  Both, measured so,
// us (M × N × K), row-wise / tiles: 1×4096×4096 9.2 / 14, 16×4096×4096 10.1 /
// 14, 16×1024×1024 4.1 / 9, 16×4096×16384 28.0 / 36.9, 32×4096×16384 32.7 /
// 37.6, 64×4096×16384 42.0 / 39.3, 32×16384×4096 30.3 / 33.1, 32×50264×2048
// 60.3 / 50.1, 64×8192×8192 35.1 / 38.1, 64×4096×16390 81 / 48.  Operands that
// the tiles would have to copy first (twice their bytes at 5 TB/s, a launch)
// count that, those that they take as they are (loose) do not.
//
// save8: Z in 8 bits, whose blocks of 32 columns stay in one workgroup: 32 rows of
// W in each at any N, half as many workgroups (row-wise / tiles, us: 16×4096×4096
// 12.6 / 13.3, 64×4096×4096 18.0 / 15.0, 16×2048×8192 19.4 / 13.6, 32×4096×8192
// 25.4 / 23.2, 64×2048×4096 17.5 / 13.2, 16×1024×1024 5.6 / 7.6, 64×4096×1024 9.6 /
// 8.9).
inline bool row_by_row(int64_t M, int64_t N, int64_t K, bool save8, bool copy_x, bool copy_w, double tiles_us, bool loose)
{
    if (M > lin::kFewRows)
        return false;
    const int64_t cus = hg::cu_count(), per = lin::weight_blocks(N, save8), blocks = (N + 16 * per - 1) / (16 * per);
    const double rounds = (double)((blocks + cus - 1) / cus), xb = M <= 16 ? 1.0 : M <= 32 ? 2.0 : 4.0;
    double us;
    if (!copy_x && !copy_w && (per == 1 || K >= 2048)) {
        const double fill = std::min(1.0, (double)blocks / (double)cus);
        const bool shared = (double)per * xb <= 2.0;
        const double turns = shared ? 0.5 * (rounds + std::max(1.0, (double)blocks / (double)cus)) : rounds;
        us = 2.5 * (shared ? 1.0 : rounds) + turns * (double)K * ((double)per * (0.85 + 0.42 * fill) + 0.33 * xb) * 1e-3;
    } else {
        const double rows = M > 16 ? 16.0 * xb : (double)M;
        const int64_t b16 = (N + 15) / 16;
        us = 2.2 + (double)std::max((b16 + cus - 1) / cus, per) * (double)K * (1.15 + 0.045 * rows) * 1e-3;
    }
    tiles_us = std::max(tiles_us + 3.0, 4.0 + (double)N * (double)K * 2.0 / 4.6e6);
    if (loose)
        return us < tiles_us;
    double copies = copy_x || copy_w ? 3.0 : 0.0;
    copies += (copy_x ? (double)M * (double)K * 4.0 / 5e6 : 0.0) + (copy_w ? (double)N * (double)K * 4.0 / 5e6 : 0.0);
    return us < tiles_us + copies;
}

struct LinearPlan {
    bool copy_x, copy_w;
    bool direct, loose, odd;          // both operands direct; taken as they are by 64×64 tiles; rows at odd elements
    Cut cut;
};
inline LinearPlan plan_linear(int64_t M, int64_t N, int64_t K, const hg_matrix *X, const hg_matrix *W, bool save8,
                              int most = 256)
{
    LinearPlan q;
    double us;
    q.copy_x = !direct(X, K);
    q.copy_w = !direct(W, K);
    q.direct = !q.copy_x && !q.copy_w;
    q.odd = odd_rows(X, M) || odd_rows(W, N);
    q.cut = best_cut({M, N, K}, &us, most);
    // 64×64 tiles take operands that would have to be copied as they are: the
    // slower loop costs less than the launch (copied / as they are, us:
    // 333×1111×777 12.4 / 9.2, 100×100×101 6.8 / 5.9, 128×1024×8191 22.0 / 14.1,
    // 1000×1000×4001 32.4 / 28.8, 2000×2000×1001 29.8 / 29.0, 700×3000×1001 26.5
    // / 27.1).
    q.loose = !q.direct && q.cut.tile == 64;
    if (row_by_row(M, N, K, save8, q.copy_x, q.copy_w, q.loose ? 1.15 * us : us, q.loose)) {
        q.copy_x = q.copy_w = q.loose = false;
        q.cut = {0, 0, 1, 0};
    } else if (q.loose) {
        q.copy_x = q.copy_w = false;
    }
    return q;
}
inline lin::Copy copy_of(const hg_matrix *m, int64_t rows, int64_t cols, void *to)
{
    return {m->data, m->type == HG_E4M3 ? m->scales : nullptr, to, m->ld, m->lds, up8(cols), rows, cols};
}

struct LinearRoom {
    void *x, *w, *p;
};
inline LinearRoom room_linear(Arena &a, const LinearPlan &q, int64_t M, int64_t N, int64_t K)
{
    LinearRoom r;
    r.x = a.take(q.copy_x ? M * up8(K) * 2 : 0);
    r.w = a.take(q.copy_w ? N * up8(K) * 2 : 0);
    r.p = a.take(q.cut.tile != 0 ? partial_bytes(q.cut, {M, N, K}) : 0);
    return r;
}

// Workspace of the forward product, whatever Y and Z, and of what goes beside it:
// beside(arena, plan).
template <class Beside>
int64_t linear_room(int64_t M, int64_t N, int64_t K, const hg_matrix *X, const hg_matrix *W, int most, Beside beside)
{
    if (const int e = check_sizes(M, N, K, 1))
        return e;
    if (X == nullptr || !is16(X->type) || !valid(X, 0, K))
        return -4;
    if (W == nullptr || W->type != X->type || !valid(W, 0, K))
        return -5;
    if (M == 0 || N == 0 || K == 0)
        return 0;
    // A call that saves Z in 8 bits may take another kernel.
    int64_t need = 0;
    for (const bool save8 : {false, true}) {
        const LinearPlan q = plan_linear(M, N, K, X, W, save8, most);
        Arena a{nullptr};
        room_linear(a, q, M, N, K);
        beside(a, q);
        need = std::max(need, a.used);
    }
    return need;
}
inline int64_t linear_room(int64_t M, int64_t N, int64_t K, const hg_matrix *X, const hg_matrix *W)
{
    return linear_room(M, N, K, X, W, 256, [](Arena &, const LinearPlan &) {});
}

// The forward product: hg_linear's arguments 1 to 10 as they are numbered there
// and what is added beside it (hg_linear: Nothing).  kWorkArgument: the status
// of a bad workspace.
struct Nothing {
    int valid() const { return HG_OK; }                                     // its own arguments
    int check(const Span &, const Span &, const Span &) const { return HG_OK; }   // against Y, Z and Z's scales
    int most_tile() const { return 256; }
    void room(Arena &, const LinearPlan &) const {}                         // its part of the workspace
    bool meets(const Span &) const { return false; }
    // What is launched first.
    hipError_t begin(lin::Product &, Arena &, const LinearPlan &, bool, hipStream_t) const { return hipSuccess; }
};
template <int kWorkArgument, class Beside>
int linear_call(int act, int64_t M, int64_t N, int64_t K, const hg_matrix *X, const hg_matrix *W, const float *bias,
                const hg_matrix *R, const hg_matrix *Y, const hg_matrix *Z, const Beside &beside, void *work,
                int64_t work_bytes, void *stream)
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
    if (const int e = beside.valid())
        return e;
    if (M == 0 || N == 0)
        return HG_OK;
    const Span sx = data_span(X, M, K), sw = data_span(W, N, K), sb = span_of(bias, N * 4);
    const Span sr = data_span(R, M, N), sy = data_span(Y, M, N), sz = data_span(Z, M, N), ss = scale_span(Z, M, N);
    const bool in_place = R != nullptr && R->data == Y->data && R->ld == Y->ld;
    if (any_meet({sy}, {sx, sw, sb, in_place ? span_of(nullptr, 0) : sr}))
        return -9;
    if (any_meet({sz, ss}, {sx, sw, sb, sr, sy}) || meet(sz, ss))
        return -10;
    if (const int e = beside.check(sy, sz, ss))
        return e;
    const LinearPlan q = plan_linear(M, N, K, X, W, Z != nullptr && Z->type == HG_E4M3, beside.most_tile());
    Arena count{nullptr};
    if (K > 0) {
        room_linear(count, q, M, N, K);
        beside.room(count, q);
    }
    const Span wk = span_of(work, count.used);
    if (bad_work(work, count.used) || any_meet({wk}, {sx, sw, sb, sr, sy, sz, ss}) || beside.meets(wk))
        return kWorkArgument;
    if (work_bytes < count.used)
        return kWorkArgument - 1;

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
    }
    if (Z != nullptr) {
        p.f.Z = Z->data;
        p.f.ldz = Z->ld;
        p.f.save = Z->type == HG_E4M3 ? lin::kSave8 : lin::kSave16;
        p.f.Zs = Z->scales;
        p.f.ldzs = Z->lds;
    }
    if (K == 0) {                                 // an empty sum
        p.edge = 64;
        return status_of(lin::launch_reduce(&p, nullptr, bf16, s));
    }
    set_cut(p, q.cut, room.p);
    if (const hipError_t e = beside.begin(p, arena, q, bf16, s))
        return status_of(e);
    lin::Copy cx{}, cw{};
    if (q.copy_x) {
        cx = copy_of(X, M, K, room.x);
        p.A = static_cast<const uint16_t *>(room.x);
        p.lda = up8(K);
    }
    if (q.copy_w) {
        cw = copy_of(W, N, K, room.w);
        p.B = static_cast<const uint16_t *>(room.w);
        p.ldb = up8(K);
    }
    if (const hipError_t e = lin::launch_prepare(lin::Slope{}, cx, cw, bf16, s))
        return status_of(e);
    const hipError_t e = q.cut.tile == 0     ? lin::launch_rowwise(p, q.direct, q.odd, bf16, s)
                         : q.loose            ? lin::launch_loose(p, bf16, s)
                         : q.cut.tile == 256 ? lin::launch_tile(p, lin::Layout::NN, bf16, s)
                                             : lin::launch_ring(p, q.cut.tile, bf16, s);
    if (e != hipSuccess || p.splits <= 1)
        return status_of(e);
    return status_of(lin::launch_reduce(&p, nullptr, bf16, s));
}

}  // namespace host
}  // namespace hg
