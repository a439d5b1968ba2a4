// Stand-ins for the delta rule's launch sequences, for the host-code sanitizer build: every call
// that the check program makes is refused before any launch, so reaching one of these is
// itself a failure.
#include <cstdio>
#include <cstdlib>

namespace ssd {
namespace delta {
struct Args;
[[noreturn]] static void reached(const char* what) {
    std::fprintf(stderr, "launch sequence %s reached: a call was not refused on the host\n", what);
    std::abort();
}
int run_bf16(const Args&, bool) { reached("run_bf16"); }
int run_f32(const Args&, bool) { reached("run_f32"); }
}  // namespace delta
}  // namespace ssd
