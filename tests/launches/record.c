/* Records the launches that the library's entry points make, on the host: the HIP calls of libssd.so bind to
 * the stand-ins below (this program's symbols come first), so nothing reaches a device and no operand is read.
 *
 *   record libssd.so < calls
 *
 * Each line of `calls` is an entry point's name, its descriptor's bytes in hex, how many bytes of every kernel's
 * first argument to show, and the other arguments as integers.  For each launch it prints "launch", the grid's and the
 * work-group's three sizes and those bytes; for each call "status" and what it returned. */
#include <dlfcn.h>
#include <stdint.h>
#include <stdio.h>
#include <stdlib.h>
#include <string.h>

typedef struct {
    uint32_t x, y, z;
} dim3;
static dim3 grid_, block_;
static size_t lds_;
static void* stream_;
static int show;

int __hipPushCallConfiguration(dim3 grid, dim3 block, size_t lds, void* stream) {
    grid_ = grid; block_ = block; lds_ = lds; stream_ = stream;
    return 0;
}
int __hipPopCallConfiguration(dim3* grid, dim3* block, size_t* lds, void** stream) {
    *grid = grid_; *block = block_; *lds = lds_; *stream = stream_;
    return 0;
}
int hipLaunchKernel(const void* f, dim3 grid, dim3 block, void** args, size_t lds, void* stream) {
    printf("launch %u %u %u %u %u %u ", grid.x, grid.y, grid.z, block.x, block.y, block.z);
    for (int i = 0; i < show; ++i) printf("%02x", ((const unsigned char*)args[0])[i]);
    printf("\n");
    return 0;
}
int hipFuncSetAttribute(const void* f, int what, int value) { return 0; }
int hipGetLastError(void) { return 0; }

int main(int argc, char** argv) {
    void* lib = argc > 1 ? dlopen(argv[1], RTLD_NOW | RTLD_LOCAL) : NULL;
    if (!lib) return fprintf(stderr, "%s\n", argc > 1 ? dlerror() : "no library"), 1;
    static char line[8192];
    while (fgets(line, sizeof(line), stdin)) {
        char* name = strtok(line, " \n");
        char* hex = strtok(NULL, " \n");
        char* bytes = strtok(NULL, " \n");
        if (!name || !hex || !bytes) return fprintf(stderr, "bad line\n"), 1;
        int (*f)(void*, ...) = (int (*)(void*, ...))dlsym(lib, name);
        if (!f) return fprintf(stderr, "%s\n", dlerror()), 1;
        unsigned char p[512] __attribute__((aligned(16)));
        size_t n = strlen(hex) / 2;
        if (n > sizeof(p)) return fprintf(stderr, "descriptor too long\n"), 1;
        for (size_t i = 0; i < n; ++i) {
            unsigned v;
            sscanf(hex + 2 * i, "%2x", &v);
            p[i] = (unsigned char)v;
        }
        show = atoi(bytes);
        uint64_t a[24] = {0};
        char* t;
        for (int i = 0; i < 24 && (t = strtok(NULL, " \n")); ++i) a[i] = strtoull(t, NULL, 0);
        const int st = f(p, a[0], a[1], a[2], a[3], a[4], a[5], a[6], a[7], a[8], a[9], a[10], a[11], a[12], a[13], a[14],
                         a[15], a[16], a[17], a[18], a[19], a[20], a[21], a[22], a[23]);
        printf("status %d\n", st);
    }
    return 0;
}
