// How the host side cuts the product of the linear layer with adapters.
#include "adapters_plan_stub.cpp"

// {tile edge (0: row by row), tiles in one piece, slices of the others, operands that
// are copied first, taken as they are by 64×64 tiles, rows of W of a workgroup row by
// row / 16} for adapters of this rank.
extern "C" void adapters_cut(int64_t M, int64_t N, int64_t K, int64_t rank, const hg_matrix *X, const hg_matrix *W, int save8,
                             int64_t *out)
{
    const LinearPlan q = plan_linear(M, N, K, X, W, save8 != 0, most_tile_of(rank));
    const int64_t cut[] = {q.cut.tile, q.cut.whole, q.cut.splits, q.copy_x + q.copy_w, q.loose, hg::lin::weight_blocks(N, save8 != 0)};
    std::copy(cut, cut + 6, out);
}
