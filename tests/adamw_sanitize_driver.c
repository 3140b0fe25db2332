/* Host-only exercise of the checks of muon_adamw_mixed_step, muon_adamw8_step
 * and muon_grad_norm, built with AddressSanitizer and
 * UndefinedBehaviorSanitizer by tests/test_sanitize_adamw_cpu.py.  No call here
 * touches a GPU: every pointer is a fake address. */
#include <stdint.h>
#include <stdio.h>
#include <stdlib.h>
#include <string.h>

#include "muon_step.h"

static int failures = 0;

#define EXPECT(cond)                                                           \
    do {                                                                       \
        if (!(cond)) {                                                         \
            fprintf(stderr, "%s:%d: expectation failed: %s\n", __FILE__, __LINE__, #cond); \
            ++failures;                                                        \
        }                                                                      \
    } while (0)

static void *fake(int64_t i, int k) {
    return (void *)(uintptr_t)((1ull << 40) + (uint64_t)i * (1ull << 30) + (uint64_t)k * (1ull << 26));
}

int main(void) {
    const muon_adamw_hparams hp = {0.02, 0.9, 0.95, 1e-8, 0.1, 1};
    const float *factor = (const float *)(uintptr_t)4096;
    const int64_t counts[] = {0, 1, 2, 3, 64, 65, 1000};
    char msg[256];
    for (size_t c = 0; c < sizeof counts / sizeof counts[0]; ++c) {
        const int64_t n = counts[c];
        muon_adamw_mixed_tensor *m = (muon_adamw_mixed_tensor *)calloc((size_t)n + 1, sizeof *m);
        muon_adamw8_tensor *b = (muon_adamw8_tensor *)calloc((size_t)n + 1, sizeof *b);
        muon_grad *g = (muon_grad *)calloc((size_t)n + 1, sizeof *g);
        for (int64_t i = 0; i < n; ++i) {
            const int64_t at = (c & 1) ? i : n - 1 - i; /* in and against address order */
            const int bf16 = (int)(i % 3 != 0);
            const int64_t numel = i % 5 == 4 ? 0 : 1 + i * 777;
            m[i].param = fake(at, 0);
            m[i].master = bf16 ? (float *)fake(at, 1) : NULL;
            m[i].grad = fake(at, 2);
            m[i].exp_avg = (float *)fake(at, 3);
            m[i].exp_avg_sq = (float *)fake(at, 4);
            m[i].numel = numel;
            m[i].param_dtype = bf16;
            m[i].grad_dtype = (int)(i & 1);
            b[i].param = m[i].param;
            b[i].master = m[i].master;
            b[i].grad = m[i].grad;
            b[i].exp_avg = (uint8_t *)fake(at, 3);
            b[i].exp_avg_sq = (uint8_t *)fake(at, 4);
            b[i].exp_avg_scale = (uint8_t *)fake(at, 5);
            b[i].exp_avg_sq_scale = (uint8_t *)fake(at, 6);
            b[i].numel = numel;
            b[i].param_dtype = bf16;
            b[i].grad_dtype = (int)(i & 1);
            g[i].grad = m[i].grad;
            g[i].numel = numel;
            g[i].dtype = (int)(i & 1);
        }
        EXPECT(muon_check_adamw_mixed_args(m, n, &hp, factor, msg, sizeof msg) == MUON_OK && msg[0] == 0);
        EXPECT(muon_check_adamw8_args(b, n, &hp, factor, msg, sizeof msg) == MUON_OK && msg[0] == 0);
        EXPECT(muon_check_grad_norm_args(g, n, 1.0, (double *)(uintptr_t)4096, (float *)(uintptr_t)8192, msg,
                                         sizeof msg) == MUON_OK);
        if (n >= 3) {
            m[2].exp_avg = m[0].exp_avg_sq;
            EXPECT(muon_check_adamw_mixed_args(m, n, &hp, NULL, msg, sizeof msg) == MUON_ERR_INVALID_ARGUMENT);
            EXPECT(strstr(msg, "overlaps") != NULL);
            b[1].exp_avg_scale = b[0].exp_avg_scale;
            EXPECT(muon_check_adamw8_args(b, n, &hp, NULL, msg, 8) == MUON_ERR_INVALID_ARGUMENT);
            EXPECT(strlen(msg) == 7); /* cut to the buffer */
            EXPECT(muon_check_adamw8_args(b, n, &hp, NULL, NULL, 0) == MUON_ERR_INVALID_ARGUMENT);
            g[1].dtype = 9;
            EXPECT(muon_check_grad_norm_args(g, n, 1.0, (double *)(uintptr_t)4096, (float *)(uintptr_t)8192, NULL,
                                             0) == MUON_ERR_INVALID_ARGUMENT);
        }
        free(m);
        free(b);
        free(g);
    }
    muon_adamw8_tensor big;
    memset(&big, 0, sizeof big);
    big.numel = (int64_t)1 << 38; /* the largest */
    big.param_dtype = big.grad_dtype = MUON_F32;
    big.param = (void *)((uintptr_t)1 << 43);
    big.grad = (void *)((uintptr_t)2 << 43);
    big.exp_avg = (uint8_t *)((uintptr_t)3 << 43);
    big.exp_avg_sq = (uint8_t *)((uintptr_t)4 << 43);
    big.exp_avg_scale = (uint8_t *)((uintptr_t)5 << 43);
    big.exp_avg_sq_scale = (uint8_t *)((uintptr_t)6 << 43);
    EXPECT(muon_check_adamw8_args(&big, 1, &hp, NULL, msg, sizeof msg) == MUON_OK);
    big.numel += 1;
    EXPECT(muon_check_adamw8_args(&big, 1, &hp, NULL, msg, sizeof msg) == MUON_ERR_INVALID_ARGUMENT);
    EXPECT(muon_check_adamw_mixed_args(NULL, 1, &hp, NULL, msg, sizeof msg) == MUON_ERR_INVALID_ARGUMENT);
    EXPECT(muon_check_adamw8_args(NULL, 1, &hp, NULL, msg, sizeof msg) == MUON_ERR_INVALID_ARGUMENT);
    EXPECT(muon_check_grad_norm_args(NULL, 1, 1.0, (double *)(uintptr_t)64, (float *)(uintptr_t)128, msg, sizeof msg) ==
           MUON_ERR_INVALID_ARGUMENT);
    if (failures) return 1;
    printf("sanitized AdamW checks: ok\n");
    return 0;
}
