/* The host code of the delta rule's and the norm's entry points (argument checks, workspace
 * layouts) built with AddressSanitizer and UndefinedBehaviorSanitizer.  Every call below is
 * refused or is a pure host function, on fake device addresses that nothing dereferences.
 * Exit status 0 on success, 1 when a call returns something other than what is expected. */
#include <stdint.h>
#include <stdio.h>
#include <string.h>

#include "ssd.h"

static int fails = 0;
#define EXPECT(cond)                                            \
    do {                                                        \
        if (!(cond)) {                                          \
            printf("line %d: expected %s\n", __LINE__, #cond); \
            ++fails;                                            \
        }                                                       \
    } while (0)

#define FAKE(k) ((void*)((uintptr_t)1 << 44 | (uintptr_t)(k) << 38))

static ssd_problem prob(int64_t b, int64_t T, int64_t H, int64_t P, int64_t N, int64_t G, int dtype) {
    ssd_problem p;
    memset(&p, 0, sizeof(p));
    p.batch = b; p.seqlen = T; p.nheads = H; p.headdim = P; p.dstate = N; p.ngroups = G; p.chunk = 64; p.dtype = dtype;
    return p;
}

static ssd_norm norm(int64_t b, int64_t T, int64_t GB, int64_t GC, int64_t N, int64_t F, float eps, int dtype) {
    ssd_norm p;
    memset(&p, 0, sizeof(p));
    p.batch = b; p.seqlen = T; p.bheads = GB; p.cheads = GC; p.dstate = N; p.pairs = F;
    p.bstride = GB * N; p.cstride = GC * N; p.eps = eps; p.dtype = dtype;
    return p;
}

static int fwd(const ssd_problem* p, void* x, void* y, size_t ws) {
    return ssd_delta_fwd(p, x, FAKE(1), FAKE(2), FAKE(3), FAKE(4), FAKE(5), NULL, y, FAKE(7), FAKE(8), ws, NULL);
}
static int bwd(const ssd_problem* p, void* dx, size_t ws) {
    return ssd_delta_bwd(p, FAKE(0), FAKE(1), FAKE(2), FAKE(3), FAKE(4), FAKE(5), NULL, FAKE(9), NULL, dx, FAKE(11), FAKE(12),
                         FAKE(13), FAKE(14), FAKE(15), NULL, FAKE(8), ws, NULL);
}

int main(void) {
    const int64_t Ps[] = {16, 32, 64, 128}, Ns[] = {16, 32, 64, 128, 256}, big[] = {1, 2, 65535, 65536, 1 << 20, 1ll << 31, 1ll << 40};
    for (int dt = 0; dt < 2; ++dt)
        for (int ip = 0; ip < 4; ++ip)
            for (int in = 0; in < 5; ++in) {
                ssd_problem p = prob(3, 1000 + 7 * ip, 8, Ps[ip], Ns[in], 2, dt);
                const size_t f = ssd_delta_workspace_bytes(&p), v = ssd_delta_varlen_workspace_bytes(&p),
                             b = ssd_delta_bwd_workspace_bytes(&p);
                EXPECT(f > 0 && v > 0 && b > f);
                EXPECT(fwd(&p, FAKE(0), FAKE(6), f - 1) == SSD_ERR_WORKSPACE);
                EXPECT(fwd(&p, NULL, FAKE(6), f) == SSD_ERR_NULL);
                EXPECT(fwd(&p, FAKE(0), FAKE(0), f) == SSD_ERR_ALIAS);
                EXPECT(fwd(&p, (char*)FAKE(0) + 8, FAKE(6), f) == SSD_ERR_ALIGN);
                EXPECT(bwd(&p, FAKE(10), b - 1) == SSD_ERR_WORKSPACE);
                EXPECT(bwd(&p, FAKE(9), b) == SSD_ERR_ALIAS);
                EXPECT(bwd(&p, NULL, b) == SSD_ERR_NULL);
                EXPECT(ssd_delta_fwd_varlen(&p, NULL, FAKE(0), FAKE(1), FAKE(2), FAKE(3), FAKE(4), FAKE(5), NULL, FAKE(6),
                                            NULL, FAKE(8), v, NULL) == SSD_ERR_NULL);
                EXPECT(ssd_delta_step(&p, FAKE(0), FAKE(1), FAKE(2), FAKE(3), FAKE(4), FAKE(5), FAKE(6), FAKE(6), NULL) ==
                       SSD_ERR_ALIAS);
                ssd_norm n = norm(3, 50, 2, 5, Ns[in], 8, 1e-6f, dt);
                const size_t w = ssd_bc_norm_bwd_workspace_bytes(&n);
                EXPECT(w > 0);
                EXPECT(ssd_bc_norm(&n, FAKE(0), FAKE(1), NULL, NULL, NULL, NULL, FAKE(2), FAKE(3), NULL) == SSD_ERR_NULL);
                EXPECT(ssd_bc_norm(&n, FAKE(0), FAKE(1), NULL, NULL, FAKE(4), NULL, FAKE(0), FAKE(3), NULL) == SSD_ERR_ALIAS);
                EXPECT(ssd_bc_norm_bwd(&n, FAKE(0), FAKE(1), FAKE(5), NULL, FAKE(4), NULL, FAKE(2), FAKE(3), FAKE(6), FAKE(7),
                                       FAKE(8), NULL, FAKE(9), w - 1, NULL) == SSD_ERR_WORKSPACE);
            }
    /* sizes whose products leave 64 bits where nothing bounds them first */
    for (unsigned i = 0; i < sizeof(big) / sizeof(big[0]); ++i)
        for (unsigned j = 0; j < sizeof(big) / sizeof(big[0]); ++j)
            for (unsigned k = 0; k < sizeof(big) / sizeof(big[0]); ++k) {
                ssd_problem p = prob(big[i], big[j], big[k], 128, 256, 1, SSD_BF16);
                (void)ssd_delta_workspace_bytes(&p);
                (void)ssd_delta_varlen_workspace_bytes(&p);
                (void)ssd_delta_bwd_workspace_bytes(&p);
                EXPECT(ssd_delta_step(&p, NULL, FAKE(1), FAKE(2), FAKE(3), FAKE(4), FAKE(5), FAKE(6), FAKE(7), NULL) != SSD_OK);
                ssd_norm n = norm(big[i], big[j], big[k], 1, 256, 128, 1e-6f, SSD_BF16);
                (void)ssd_bc_norm_bwd_workspace_bytes(&n);
                n.bstride = big[k] << 20;
                EXPECT(ssd_bc_norm(&n, NULL, FAKE(1), NULL, NULL, FAKE(4), NULL, FAKE(2), FAKE(3), NULL) != SSD_OK);
            }
    EXPECT(fwd(NULL, FAKE(0), FAKE(6), 1 << 20) == SSD_ERR_NULL && bwd(NULL, FAKE(10), 1 << 20) == SSD_ERR_NULL);
    printf(fails ? "FAILED (%d)\n" : "OK\n", fails);
    return fails ? 1 : 0;
}
