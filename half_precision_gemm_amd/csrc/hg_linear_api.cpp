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

// Bytes [lo, hi), empty when lo == hi; of a matrix its first `width` bytes of
// every `pitch`.
struct Span {
    uintptr_t lo, hi;
    uint64_t width, pitch;
};
// Different columns of one array (two matrices of the same pitch) do not meet.
bool meet(const Span &a, const Span &b)
{
    if (!(a.lo < a.hi && b.lo < b.hi && a.lo < b.hi && b.lo < a.hi))
        return false;
    if (a.pitch != b.pitch)
        return true;
    const Span &l = a.lo <= b.lo ? a : b, &h = a.lo <= b.lo ? b : a;
    const uint64_t d = (uint64_t)(h.lo - l.lo) % a.pitch;
    return d < l.width || d + h.width > a.pitch;
}
Span span_of(const void *p, int64_t bytes)
{
    const uintptr_t lo = reinterpret_cast<uintptr_t>(p);
    if (p == nullptr || bytes <= 0)
        return {0, 0, 0, 1};
    return {lo, lo + (uintptr_t)bytes, (uint64_t)bytes, (uint64_t)bytes};
}
Span rows_of(const void *p, int64_t rows, int64_t pitch, int64_t width)
{
    Span s = span_of(p, (rows - 1) * pitch + width);
    s.width = (uint64_t)width;
    s.pitch = (uint64_t)pitch;
    return s;
}
Span data_span(const hg_matrix *m, int64_t rows, int64_t cols)
{
    if (m == nullptr || rows <= 0 || cols <= 0)
        return span_of(nullptr, 0);
    return rows_of(m->data, rows, m->ld * esize(m->type), cols * esize(m->type));
}
Span scale_span(const hg_matrix *m, int64_t rows, int64_t cols)
{
    if (m == nullptr || m->type != HG_E4M3 || rows <= 0 || cols <= 0)
        return span_of(nullptr, 0);
    return rows_of(m->scales, rows, m->lds, blocks8(cols));
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

// Whether the product kernels can load this 16-bit operand as it is: 16-byte
// pieces of rows whose length is a multiple of 8 (a piece never holds
// elements of the next row or behind the last one), 32-bit offsets in a tile.
bool direct(const hg_matrix *m, int64_t cols)
{
    return cols % 8 == 0 && m->ld % 8 == 0 && m->ld <= 2 * (int64_t)HG_LINEAR_MAX_WIDTH &&
           (reinterpret_cast<uintptr_t>(m->data) & 15) == 0;
}

// Whether a row of a 16-bit matrix may begin at an address that no 32-bit word
// begins at.
bool odd_rows(const hg_matrix *m, int64_t rows)
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
Rate rate_of(int64_t cus, int tile, int64_t items)
{
    const double fill = std::min(1.0, (double)items / (double)cus);
    if (tile == 64)
        return items > cus ? Rate{3.2, 0.45, 2 * cus} : Rate{1.0, 0.265, cus};
    return tile == 128 ? Rate{5.0, 0.55, cus} : Rate{7.0 + 6.0 * fill, 1.05 + 0.35 * fill, cus};
}
double reduce_us(int64_t tiles, int tile, int s)
{
    return s > 1 && tiles > 0 ? 3.0 + (double)tiles * (double)s * (double)tile * (double)tile * 8.0 / 5e6 : 0.0;
}
// One product, its tiles from `whole` on in s slices.
double expected_us(int64_t cus, int tile, const Shape &p, int64_t whole, int s)
{
    const int64_t tiles = p.tiles(tile), rest = tiles - whole;
    const Rate r = rate_of(cus, tile, whole + rest * s);
    const double one = r.fix + r.stage * (double)p.stages(), part = r.fix + r.stage * (double)((p.stages() + s - 1) / s);
    return 2.0 + (double)((whole + r.slots - 1) / r.slots) * one + (double)((rest * s + r.slots - 1) / r.slots) * part +
           reduce_us(rest, tile, s);
}
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
Cut cut_into(int tile, const Shape &p, int64_t whole, int s)
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
bool may_slice(int64_t cus, int64_t tiles, const Shape &p, int s)
{
    return s == 1 || (p.stages() >= 4 * s && tiles * s <= 2 * cus);
}

// Whether so many items, and the blocks that end column sums, fit one launch (the
// 256×256 kernel walks its tiles and has no such limit).
bool may_launch(int tile, int64_t items)
{
    return tile == 256 || items + (HG_LINEAR_MAX_WIDTH + 31) / 32 <= lin::kMostBlocks;
}

// A product's tiles are cut all, none, or only those of the last round, which
// would leave most of the GPU idle (1729×10332×14080, 287 tiles of 256×256 on 256
// CUs: none 698 us).
Cut best_cut(const Shape &p, double *us = nullptr)
{
    const int64_t cus = hg::cu_count();
    Cut best{64, 0, 1, 0};
    double least = 0.0;
    bool first = true;
    for (int tile : {64, 128, 256}) {
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
int64_t partial_bytes(const Cut &c, const Shape &p)
{
    return c.splits > 1 ? (p.tiles(c.tile) - c.whole) * c.splits * c.tile * c.tile * 4 : 0;
}
void set_cut(lin::Product &p, const Cut &c, void *partials)
{
    p.edge = c.tile;
    p.whole = (int32_t)c.whole;
    p.splits = c.splits;
    p.per = c.per;
    p.P = static_cast<float *>(partials);
}

void set_output(lin::Finish &f, const hg_matrix *Y, int64_t rows, int64_t cols)
{
    f.C = Y->data;
    f.ldc = Y->ld;
    f.out32 = Y->type == HG_F32;
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
bool row_by_row(int64_t M, int64_t N, int64_t K, bool save8, bool copy_x, bool copy_w, double tiles_us, bool loose)
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
LinearPlan plan_linear(int64_t M, int64_t N, int64_t K, const hg_matrix *X, const hg_matrix *W, bool save8)
{
    LinearPlan q;
    double us;
    q.copy_x = !direct(X, K);
    q.copy_w = !direct(W, K);
    q.direct = !q.copy_x && !q.copy_w;
    q.odd = odd_rows(X, M) || odd_rows(W, N);
    q.cut = best_cut({M, N, K}, &us);
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
lin::Copy copy_of(const hg_matrix *m, int64_t rows, int64_t cols, void *to)
{
    return {m->data, m->type == HG_E4M3 ? m->scales : nullptr, to, m->ld, m->lds, up8(cols), rows, cols};
}

struct LinearRoom {
    void *x, *w, *p;
};
LinearRoom room_linear(Arena &a, const LinearPlan &q, int64_t M, int64_t N, int64_t K)
{
    LinearRoom r;
    r.x = a.take(q.copy_x ? M * up8(K) * 2 : 0);
    r.w = a.take(q.copy_w ? N * up8(K) * 2 : 0);
    r.p = a.take(q.cut.tile != 0 ? partial_bytes(q.cut, {M, N, K}) : 0);
    return r;
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
    if (const int e = check_sizes(M, N, K, 1))
        return e;
    if (X == nullptr || !is16(X->type) || !valid(X, 0, K))
        return -4;
    if (W == nullptr || W->type != X->type || !valid(W, 0, K))
        return -5;
    if (M == 0 || N == 0 || K == 0)
        return 0;
    // A call that saves Z in 8 bits may take another kernel.
    Arena a{nullptr}, b{nullptr};
    room_linear(a, plan_linear(M, N, K, X, W, false), M, N, K);
    room_linear(b, plan_linear(M, N, K, X, W, true), M, N, K);
    return std::max(a.used, b.used);
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
    if (any_meet({sy}, {sx, sw, sb, in_place ? span_of(nullptr, 0) : sr}))
        return -9;
    if (any_meet({sz, ss}, {sx, sw, sb, sr, sy}) || meet(sz, ss))
        return -10;
    const LinearPlan q = plan_linear(M, N, K, X, W, Z != nullptr && Z->type == HG_E4M3);
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
