// The gated delta rule's kernels for float32 x/B/C/beta/y.
#include "delta_launch.hpp"

namespace ssd {
namespace delta {
int run_f32(const Args& a, bool bwd) { return run<float>(a, bwd); }
}  // namespace delta
}  // namespace ssd
