// The tree of drafted tokens for bfloat16 x/B/C/beta/y.
#include "tree.hpp"

namespace ssd {
namespace pool {
int tree_bf16(const Args& a) { return run_tree<bf16>(a); }
}  // namespace pool
}  // namespace ssd
