/* The host code of the pool's entry points (argument checks) built with AddressSanitizer and
 * UndefinedBehaviorSanitizer.  Every call below is refused, or has nothing to do, on fake device
 * addresses that nothing dereferences.  Exit status 0 on success, 1 when a call returns something other
 * than what is expected. */
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

#define FAKE(k) ((void*)((uintptr_t)1 << 50 | (uintptr_t)(k) << 44))

static ssd_pool_problem prob(int64_t b, int64_t T, int64_t H, int64_t P, int64_t N, int64_t G, int64_t S, int dtype) {
    ssd_pool_problem p;
    memset(&p, 0, sizeof(p));
    p.batch = b; p.seqlen = T; p.nheads = H; p.headdim = P; p.dstate = N; p.ngroups = G; p.dtype = dtype;
    p.xstride = H * P; p.bstride = p.cstride = G * N; p.slots = S; p.slot_stride = H * P * N;
    return p;
}
static int step(const ssd_pool_problem* p, void* x, void* pool, void* y) {
    return ssd_pool_step(p, x, FAKE(1), FAKE(2), FAKE(3), FAKE(4), FAKE(5), NULL, pool, FAKE(7), FAKE(8), y, NULL);
}
static int tree(const ssd_pool_problem* p, void* x, void* pool, void* y) {
    return ssd_tree_step(p, x, FAKE(1), FAKE(2), FAKE(3), FAKE(4), NULL, FAKE(5), FAKE(10), pool, FAKE(7), y, NULL);
}
static int commit(const ssd_pool_problem* p, void* x, void* pool, void* last) {
    return ssd_tree_commit(p, x, FAKE(1), FAKE(2), FAKE(3), FAKE(5), FAKE(10), last, pool, FAKE(7), FAKE(8), NULL);
}

int main(void) {
    const int64_t Ps[] = {16, 32, 64, 128}, Ns[] = {16, 32, 64, 128, 256};
    const int64_t big[] = {-(1ll << 62), -1, 0, 1, 2, 255, 257, 65535, 1 << 20, 1 << 24, 1ll << 31, 1ll << 40, 1ll << 62, INT64_MAX, INT64_MIN};
    const int nb = sizeof(big) / sizeof(big[0]);
    for (int dt = 0; dt < 2; ++dt)
        for (int ip = 0; ip < 4; ++ip)
            for (int in = 0; in < 5; ++in) {
                ssd_pool_problem p = prob(3, 100, 8, Ps[ip], Ns[in], 2, 5, dt);
                EXPECT(step(&p, NULL, FAKE(6), FAKE(9)) == SSD_ERR_NULL);
                EXPECT(step(&p, FAKE(0), FAKE(6), FAKE(6)) == SSD_ERR_ALIAS);
                EXPECT(step(&p, FAKE(0), FAKE(0), FAKE(9)) == SSD_ERR_ALIAS);
                EXPECT(tree(&p, (char*)FAKE(0) + 8, FAKE(6), FAKE(9)) == SSD_ERR_ALIGN);
                EXPECT(tree(&p, FAKE(0), FAKE(6), FAKE(0)) == SSD_ERR_ALIAS);
                EXPECT(commit(&p, FAKE(0), FAKE(6), FAKE(6)) == SSD_ERR_ALIAS);
                EXPECT(commit(&p, FAKE(0), FAKE(6), NULL) == SSD_ERR_NULL);
            }
    /* sizes far out of range, one field at a time and in pairs: refused (or nothing to do), no overflow.  A
     * call that might be accepted gets a NULL operand, so that it is refused after the size checks */
    for (int f = 0; f < 11; ++f)
        for (int g = 0; g < 11; ++g)
            for (int i = 0; i < nb; ++i)
                for (int j = 0; j < nb; ++j) {
                    ssd_pool_problem p = prob(3, 9, 8, 64, 64, 2, 5, SSD_BF16);
                    int64_t* v = (int64_t*)&p;
                    v[f] = big[i];
                    v[g] = big[j];
                    if (p.slots == 0 && p.seqlen == 0) continue;  /* (needs no operand that is NULL below) */
                    const int e = step(&p, NULL, NULL, NULL);  /* (with no rows a valid problem has nothing to do) */
                    EXPECT(e == SSD_ERR_SHAPE || e == SSD_ERR_UNSUPPORTED || e == (p.batch ? SSD_ERR_NULL : SSD_OK));
                    const int a = tree(&p, NULL, FAKE(6), FAKE(9)), c = commit(&p, FAKE(0), FAKE(6), NULL),
                              s = step(&p, FAKE(0), NULL, FAKE(9));
                    EXPECT(a >= 0 && a < SSD_ERR_HIP && c >= 0 && c < SSD_ERR_HIP && s >= 0);
                    if (p.slots > 0) EXPECT(s == SSD_ERR_NULL || s == SSD_ERR_SHAPE || s == SSD_ERR_UNSUPPORTED || p.batch == 0);
                }
    for (int f = 0; f < 6; ++f)
        for (int g = 0; g < 6; ++g)
            for (int i = 0; i < nb; ++i)
                for (int j = 0; j < nb; ++j) {
                    ssd_pages p = {4, 3, 6, 1024, 6 * 1024, 1024};
                    int64_t* v = (int64_t*)&p;
                    v[f] = big[i];
                    v[g] = big[j];
                    const int a = ssd_pool_fork(&p, FAKE(0), FAKE(1), NULL, FAKE(2), NULL),
                              c = ssd_pool_compact(&p, FAKE(0), FAKE(1), FAKE(2), NULL, NULL);
                    EXPECT(a == SSD_ERR_NULL || a == SSD_ERR_SHAPE || a == SSD_ERR_UNSUPPORTED || p.rows == 0);
                    EXPECT(c == SSD_ERR_NULL || c == SSD_ERR_SHAPE || c == SSD_ERR_UNSUPPORTED);
                }
    EXPECT(ssd_pool_fork(NULL, NULL, NULL, NULL, NULL, NULL) == SSD_ERR_NULL);
    EXPECT(ssd_pool_compact(NULL, NULL, NULL, NULL, NULL, NULL) == SSD_ERR_NULL);
    printf(fails ? "FAILED\n" : "OK\n");
    return fails != 0;
}
