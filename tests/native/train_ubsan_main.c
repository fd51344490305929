/* train_ubsan_main.c -- drives the argument checks of the operators around the linear layers
 * with extreme sizes, strides and options under UndefinedBehaviorSanitizer (test only). */
#include <math.h>
#include <stdio.h>
#include <stdlib.h>
#include <string.h>

#include "nvfp4.h"

extern int stub_calls;

static const int64_t kVals[] = {INT64_MIN, -1, 0, 1, 2, 7, 256, 32768, 32769, (int64_t)1 << 31,
                                (int64_t)1 << 40, (int64_t)1 << 60, (int64_t)1 << 62, INT64_MAX};
#define NV ((int)(sizeof kVals / sizeof kVals[0]))
#define FAKE ((void *)0x10000)

static int tally[8];
static void count(nvfp4_status s) {
    if (s < 0 || s > 6) { printf("status %d\n", (int)s); exit(1); }
    ++tally[s];
}

int main(void) {
    for (int i = 0; i < NV; ++i)
        for (int j = 0; j < NV; ++j)
            for (int k = 0; k < NV; ++k)
                for (int l = 0; l < NV; ++l) {
                    nvfp4_norm_params p = {kVals[i], kVals[j], kVals[k], 0, 0, 1, 0, 1e-6f, 0, 1, 1};
                    nvfp4_norm_forward_args f = {FAKE, kVals[l], FAKE, kVals[l], FAKE, FAKE, kVals[l],
                                                 FAKE, (void *)0x20000, kVals[l], FAKE, kVals[l],
                                                 FAKE, FAKE};
                    count(nvfp4_residual_norm_forward(&p, &f, NULL));
                    nvfp4_norm_backward_args b = {FAKE, kVals[l], FAKE, kVals[l], FAKE, FAKE, kVals[l],
                                                  FAKE, FAKE, FAKE, FAKE, kVals[l], FAKE, kVals[l],
                                                  FAKE, kVals[l], FAKE, kVals[l], FAKE, FAKE, FAKE,
                                                  kVals[l]};
                    count(nvfp4_residual_norm_backward(&p, &b, FAKE,
                                                       nvfp4_residual_norm_workspace_bytes(&p), NULL));
                    nvfp4_scan_args a;
                    memset(&a, 0, sizeof a);
                    a.batch = kVals[i];
                    a.time = kVals[j];
                    a.chan = kVals[k];
                    a.g = a.u = a.y = FAKE;
                    a.g_batch = a.g_time = a.u_batch = a.u_time = a.y_batch = a.y_time = kVals[l];
                    size_t need = nvfp4_gated_scan_workspace_bytes(kVals[i], kVals[j], kVals[k], l & 1);
                    count(nvfp4_gated_scan_forward(&a, FAKE, need, NULL));
                    nvfp4_scan_grads d;
                    memset(&d, 0, sizeof d);
                    d.dy = d.dg = d.du = FAKE;
                    d.dy_batch = d.dy_time = d.dg_batch = d.dg_time = d.du_batch = d.du_time = kVals[l];
                    count(nvfp4_gated_scan_backward(&a, &d, FAKE, need, NULL));
                }
    static char table[1 << 16] __attribute__((aligned(16)));
    for (int i = 0; i < NV; ++i) {
        count(nvfp4_adamw_moments(FAKE, FAKE, FAKE, FAKE, kVals[i], FAKE, FAKE, i & 1, NULL));
        nvfp4_adamw_tensor t[3];
        memset(t, 0, sizeof t);
        for (int j = 0; j < 3; ++j) {
            t[j].param = t[j].exp_avg = t[j].exp_avg_sq = FAKE;
            t[j].exp_avg_scale = t[j].exp_avg_sq_scale = FAKE;
            t[j].n = j == 1 ? kVals[i] : 5;
            t[j].weight_decay = j == 2 && i == 3 ? NAN : 0.1;
        }
        nvfp4_adamw_table_bytes(kVals[i]);
        count(nvfp4_adamw_table(t, kVals[i] > 3 ? 3 : kVals[i], i & 1 ? 8 : 32, table, sizeof table));
        nvfp4_status made = nvfp4_adamw_table(t, 3, 8, table, sizeof table);
        count(made);
        const void *grads[3] = {FAKE, NULL, FAKE};
        for (int j = 0; j < NV; ++j) {
            nvfp4_adamw_params p = {1e-3, 0.9, 0.99, 1e-8, kVals[j], 1, 0, 0, NULL};
            nvfp4_status s = nvfp4_adamw_step(table, FAKE, grads, &p, NULL);
            count(s);
            if (made != NVFP4_OK && s != NVFP4_ERR_UNSUPPORTED) { printf("a failed table was taken\n"); return 1; }
        }
        double odd[] = {NAN, INFINITY, -1.0, 1.0, 1e308};
        for (int j = 0; j < 5; ++j) {
            nvfp4_adamw_params p = {odd[j], odd[(j + 1) % 5], odd[(j + 2) % 5], odd[(j + 3) % 5], 1, 1, 0, 0, NULL};
            count(nvfp4_adamw_step(table, FAKE, grads, &p, NULL));
        }
    }
    printf("train ubsan ok: %d launches, statuses", stub_calls);
    for (int i = 0; i < 7; ++i) printf(" %d", tally[i]);
    printf("\n");
    return stub_calls > 0 && tally[NVFP4_OK] > 0 && tally[NVFP4_ERR_SHAPE] > 0 ? 0 : 1;
}
