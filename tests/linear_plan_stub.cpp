// The host side of the linear layer's C ABI with launches that are written down
// instead of made: one line per launch, "kernel key=value ..", so that a test
// sees on the CPU which kernels a call takes and how its products are cut.
#include "hg_linear_api.cpp"

#include <string>

namespace {
std::string launches;

int64_t blocks_of(const hg::lin::Product &p, int edge)
{
    const int64_t tm = ((int64_t)p.M + edge - 1) / edge, tn = ((int64_t)p.N + edge - 1) / edge;
    return p.whole + (tm * tn - p.whole) * p.splits;
}
hipError_t note(const char *kernel, int64_t edge, int64_t blocks, int64_t splits)
{
    launches += std::string(kernel) + " edge=" + std::to_string(edge) + " blocks=" + std::to_string(blocks) +
                " splits=" + std::to_string(splits) + "\n";
    return hipSuccess;
}
}  // namespace

// What was launched since the last call.
extern "C" const char *plan_launches()
{
    static std::string last;
    last.swap(launches);
    launches.clear();
    return last.c_str();
}

namespace hg {
int cu_count() { return 256; }
namespace lin {
hipError_t launch_ring(const Product &p, int tile, bool, hipStream_t)
{
    return note("ring", tile, blocks_of(p, tile), p.splits);
}
hipError_t launch_loose(const Product &p, bool, hipStream_t) { return note("loose", 64, blocks_of(p, 64), p.splits); }
hipError_t launch_ring_pair(const Product *x, const Product *w, const Strips &b, int tile, bool, hipStream_t)
{
    const int64_t blocks = (x ? blocks_of(*x, tile) : 0) + (w ? blocks_of(*w, tile) : 0) + (b.strips > 0 ? (b.cols + 31) / 32 : 0);
    if ((x && x->edge != tile) || (w && w->edge != tile))
        return hipErrorInvalidValue;
    return blocks > 0 ? note("pair", tile, blocks, std::max(x ? x->splits : 1, w ? w->splits : 1)) : hipSuccess;
}
hipError_t launch_outer(const Product &, bool, hipStream_t) { return note("outer", 0, 0, 1); }
hipError_t launch_tile(const Product &p, Layout, bool, hipStream_t) { return note("tile", 256, 256, p.splits); }
hipError_t launch_rowwise(const Product &, bool, bool, bool, hipStream_t) { return note("rowwise", 0, 0, 1); }
hipError_t launch_reduce(const Product *p, const Product *q, bool, hipStream_t)
{
    return p || q ? note("reduce", 0, 0, 1) : hipSuccess;
}
hipError_t launch_write8(const void *, int64_t, uint8_t *, int64_t, uint8_t *, int64_t, int64_t, int64_t, bool, hipStream_t)
{
    return note("write8", 0, 0, 1);
}
hipError_t launch_read8(const uint8_t *, int64_t, const uint8_t *, int64_t, void *, int64_t, int64_t, int64_t, bool, hipStream_t)
{
    return note("read8", 0, 0, 1);
}
hipError_t launch_prepare(const Slope &g, const Copy &x, const Copy &w, bool, hipStream_t)
{
    return g.rows > 0 || x.rows > 0 || w.rows > 0 ? note("prepare", 0, 0, 1) : hipSuccess;
}
hipError_t launch_zero(void *, int64_t, int64_t, int64_t, bool, hipStream_t) { return note("zero", 0, 0, 1); }
}  // namespace lin
}  // namespace hg
