// The gated delta rule's kernels for bfloat16 x/B/C/beta/y.
#include "delta_launch.hpp"

namespace ssd {
namespace delta {
int run_bf16(const Args& a, bool bwd) { return run<bf16>(a, bwd); }
}  // namespace delta
}  // namespace ssd
