/*
 * Drives the host side of the scan's and the logits' entry points (include/mil_ssm.h) under
 * AddressSanitizer and UndefinedBehaviorSanitizer without a GPU, as abi_driver.c does for the cache's:
 * every size query over small, odd, large and nonsensical sizes, and every argument check that returns
 * before work is enqueued.  Test infrastructure: built and run by tests/test_sanitizers_operators.py.
 */
#include <limits.h>
#include <stdint.h>
#include <stdio.h>

#include "mil_ssm.h"

static int fails = 0;
#define EXPECT(call, want)                                                              \
    do {                                                                               \
        int got_ = (int)(call);                                                        \
        if (got_ != (want)) {                                                          \
            printf("line %d: %s -> %d, expected %d\n", __LINE__, #call, got_, (want)); \
            ++fails;                                                                   \
        }                                                                              \
    } while (0)

static const int32_t kSizes[] = {INT_MIN, -1, 0, 1, 2, 16, 63, 64, 65, 127, 128, 256, 8192, 65536, 1 << 19, 1 << 24, 1 << 28,
                                 INT_MAX};
enum { NSIZES = sizeof kSizes / sizeof *kSizes };

static void scan(void)
{
    void *p = (void *)(uintptr_t)0x7f0000000000ull; /* never read or written */
    float *f = (float *)p;
    static const int32_t w[] = {16, 32, 64, 128, 256, 48, INT_MAX};
    size_t most = 0;
    for (int b = 0; b < NSIZES; ++b)
        for (int t = 0; t < NSIZES; ++t)
            for (int h = 0; h < NSIZES; ++h)
                for (int s = 0; s < 49; ++s)
                    for (int dt = 0; dt < 3; ++dt) {
                        const mil_ssm_dims d = {kSizes[b], kSizes[h], w[s / 7], w[s % 7], 1};
                        const int32_t T = kSizes[t];
                        const size_t states = mil_ssm_scan_states_bytes(&d, T, dt, 0),
                                     only = mil_ssm_scan_states_bytes(&d, T, dt, MIL_SCAN_FORWARD_ONLY),
                                     ws = mil_ssm_scan_workspace_bytes(&d, T, dt);
                        if ((states == 0) != (ws == 0) || only > states) {
                            printf("batch %d T %d H %d P %d N %d type %d: %zu %zu %zu bytes\n", d.batch, T, d.nheads,
                                   d.headdim, d.dstate, dt, states, only, ws);
                            ++fails;
                        }
                        most = states > most ? states : most;
                        if (!states) continue; /* each call fails its last check: no memory for it */
                        EXPECT(mil_ssm_scan_forward(&d, T, dt, NULL, p, p, p, p, f, f, NULL, p, NULL, p, states - 1, 0,
                                                    NULL),
                               MIL_E_WORKSPACE);
                        EXPECT(mil_ssm_scan_backward(&d, T, dt, NULL, p, p, p, p, f, f, p, states, p, NULL, p, p, p, p, f,
                                                     f, NULL, p, ws - 1, NULL),
                               MIL_E_WORKSPACE);
                    }
    EXPECT(most > ((size_t)1 << 32), 1);
    const mil_ssm_dims d = {2, 4, 64, 64, 2};
    mil_ssm_dims bad = d;
    bad.ngroups = 3;
    EXPECT(mil_ssm_scan_states_bytes(&bad, 10, MIL_BF16, 0), 0);
    EXPECT(mil_ssm_scan_states_bytes(&d, 10, MIL_BF16, 2u), 0);
    EXPECT(mil_ssm_scan_states_bytes(NULL, 10, MIL_BF16, 0), 0);
    const size_t n = mil_ssm_scan_states_bytes(&d, 10, MIL_BF16, 0);
    EXPECT(mil_ssm_scan_forward(&d, 10, MIL_BF16, NULL, p, p, p, p, f, f, NULL, p, NULL, (char *)p + 64, n, 0, NULL),
           MIL_E_ALIGN);
    EXPECT(mil_ssm_scan_forward(&d, 10, MIL_BF16, NULL, p, p, p, p, f, f, NULL, NULL, NULL, p, n, 0, NULL), MIL_E_INVALID);
    EXPECT(mil_ssm_scan_forward(&d, 10, MIL_BF16, NULL, p, p, p, p, f, f, NULL, p, NULL, p, n, 4u, NULL), MIL_E_INVALID);
}

static void rows_of_logits(void)
{
    const void *z = (const void *)(uintptr_t)0x7f0000000000ull;
    void *out = (void *)(uintptr_t)0x700000000000ull, *ws = (void *)(uintptr_t)0x7f2000000000ull;
    int32_t *ids = (int32_t *)(uintptr_t)0x7f3000000000ull;
    float *f = (float *)(uintptr_t)0x7f4000000000ull;
    static const int64_t strides[] = {INT64_MIN, -1, 0, 1, 128, 1 << 19, (int64_t)1 << 40, (int64_t)1 << 61, INT64_MAX};
    for (int r = 0; r < NSIZES; ++r)
        for (int v = 0; v < NSIZES; ++v)
            for (int dt = 0; dt < 3; ++dt) {
                const int32_t rows = kSizes[r], V = kSizes[v];
                const size_t dn = mil_ssm_distill_workspace_bytes(rows, V, dt);
                for (int k = -1; k <= MIL_TOPK_MAX + 1; k += 5) {
                    const size_t ln = mil_ssm_logprobs_workspace_bytes(rows, V, dt, k);
                    if (ln && (!dn || k < 0 || k > MIL_TOPK_MAX || k > V)) {
                        printf("rows %d V %d type %d k %d: %zu bytes\n", rows, V, dt, k, ln);
                        ++fails;
                    }
                    for (int s = 0; s < (int)(sizeof strides / sizeof *strides); ++s) {
                        const int64_t st = strides[s];
                        const int a = mil_ssm_token_logprobs(z, rows, V, st, dt, 1.f, NULL, k, NULL, f, k > 0 ? ids : NULL,
                                                             k > 0 ? f : NULL, ws, ln ? ln - 1 : 0, NULL),
                                  b = mil_ssm_distill_forward(z, rows, V, st, dt, 1.f, ids, f, k, 0, f, f, ws,
                                                              dn ? dn - 1 : 0, NULL),
                                  c = mil_ssm_distill_grad(z, rows, V, st, dt, 1.f, ids, f, k, 0, f, f, out, st, ws,
                                                           dn ? dn - 1 : 0, NULL),
                                  e = mil_ssm_distill_backward(z, rows, V, st, dt, 1.f, ids, f, k, 0, NULL, f, out,
                                                               V > 0 ? V : 1, NULL);
                        /* no rows: nothing to do.  Otherwise each lacks something */
                        if (rows != 0 && (a == MIL_OK || b == MIL_OK || c == MIL_OK || e == MIL_OK)) {
                            printf("rows %d V %d stride %lld type %d k %d: %d %d %d %d\n", rows, V, (long long)st, dt, k, a,
                                   b, c, e);
                            ++fails;
                        }
                    }
                }
            }
}

int main(void)
{
    scan();
    rows_of_logits();
    printf(fails ? "FAIL %d\n" : "OK\n", fails);
    return fails ? 1 : 0;
}
