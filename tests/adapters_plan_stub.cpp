// The host side of the linear layer with adapters, its launches written down as
// in linear_plan_stub.cpp.
#include "linear_plan_stub.cpp"

#include "hg_adapters_api.cpp"

namespace hg {
namespace lin {
hipError_t launch_shrink(const Shrink &q, bool, hipStream_t)
{
    return note(q.wide ? "shrink_wide" : "shrink", q.ldt, q.M, q.rank);
}
}  // namespace lin
}  // namespace hg
