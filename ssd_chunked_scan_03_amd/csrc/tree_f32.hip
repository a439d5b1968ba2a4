// The tree of drafted tokens for float32 x/B/C/beta/y.
#include "tree.hpp"

namespace ssd {
namespace pool {
int tree_f32(const Args& a) { return run_tree<float>(a); }
}  // namespace pool
}  // namespace ssd
