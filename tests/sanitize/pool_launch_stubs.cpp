// Stand-ins for the tree's launch sequences, for the host-code sanitizer build: every call that the check
// program makes is refused before any launch, so reaching one of these is itself a failure.
#include <cstdio>
#include <cstdlib>

namespace ssd {
namespace pool {
struct Args;
[[noreturn]] static void reached(const char* what) {
    std::fprintf(stderr, "launch sequence %s reached: a call was not refused on the host\n", what);
    std::abort();
}
int tree_bf16(const Args&) { reached("tree_bf16"); }
int tree_f32(const Args&) { reached("tree_f32"); }
}  // namespace pool
}  // namespace ssd
