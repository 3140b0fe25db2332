/* Host-only exercise of the checks of muon_blocks_step, muon_router_balance and
 * muon_router_bias_step, and of the block step's plan of schedules, built with
 * AddressSanitizer and UndefinedBehaviorSanitizer by
 * tests/test_blocks_router_cpu.py.  No call here touches a GPU: every pointer is
 * a fake address. */
#include <math.h>
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
    const int64_t counts[] = {0, 1, 2, 3, 64, 65, 1000};
    char msg[256];
    muon_hparams hp;
    memset(&hp, 0, sizeof hp);
    hp.lr = 0.02;
    hp.momentum = 0.95;
    hp.gamma = 0.2;
    hp.nesterov = 1;
    hp.ns_precision = MUON_NS_BF16;
    muon_ns_coeff schedule[16];
    hp.num_ns_steps = (int32_t)muon_schedule("deepseekv4", schedule, 16);
    hp.schedule = schedule;
    EXPECT(hp.num_ns_steps > 0);
    const muon_balance_hparams bh = {1e-3, (const float *)(uintptr_t)4096, MUON_SCORE_SOFTMAX, 0};
    for (size_t c = 0; c < sizeof counts / sizeof counts[0]; ++c) {
        const int64_t n = counts[c];
        muon_block_matrix *m = (muon_block_matrix *)calloc((size_t)n + 1, sizeof *m);
        muon_router *r = (muon_router *)calloc((size_t)n + 1, sizeof *r);
        muon_router_bias *b = (muon_router_bias *)calloc((size_t)n + 1, sizeof *b);
        for (int64_t i = 0; i < n; ++i) {
            const int64_t at = (c & 1) ? i : n - 1 - i; /* in and against address order */
            m[i].param = fake(at, 0);
            m[i].grad = fake(at, 1);
            m[i].momentum = (float *)fake(at, 2);
            m[i].block_rows = 1 + i % 128;
            m[i].rows = m[i].block_rows * (1 + i % 7);
            m[i].cols = m[i].block_cols = 1 + i % 777;
            m[i].param_pitch = m[i].grad_pitch = m[i].momentum_pitch = m[i].cols + i % 3;
            m[i].param_dtype = m[i].grad_dtype = (int)(i & 1);
            r[i].tokens = i % 5 == 4 ? 0 : i % 40 * 31;
            r[i].experts = 1 + (int)(i % 1024);
            r[i].top_k = 1 + (int)(i % 8);
            r[i].sequences = 1;
            r[i].pitch = r[i].dlogits_pitch = r[i].experts + i % 2;
            r[i].chosen_bits = 64;
            r[i].logits = fake(at, 3);
            r[i].dlogits = fake(at, 4);
            r[i].chosen = fake(at, 5);
            r[i].counts = (int64_t *)fake(at, 6);
            r[i].loss = (float *)fake(at, 7);
            b[i].bias = (float *)fake(at, 8);
            b[i].counts = r[i].counts;
            b[i].experts = r[i].experts;
        }
        EXPECT(muon_check_blocks_args(m, n, &hp, msg, sizeof msg) == MUON_OK && msg[0] == 0);
        EXPECT(muon_check_router_balance_args(r, n, &bh, msg, sizeof msg) == MUON_OK && msg[0] == 0);
        EXPECT(muon_check_router_bias_args(b, n, 1e-3, msg, sizeof msg) == MUON_OK && msg[0] == 0);
        if (n >= 3) {
            m[2].param = m[0].momentum;
            EXPECT(muon_check_blocks_args(m, n, &hp, msg, sizeof msg) == MUON_ERR_INVALID_ARGUMENT);
            EXPECT(strstr(msg, "overlaps") != NULL);
            r[2].loss = r[0].loss;
            EXPECT(muon_check_router_balance_args(r, n, &bh, msg, 8) == MUON_ERR_INVALID_ARGUMENT);
            EXPECT(strlen(msg) == 7); /* cut to the buffer */
            EXPECT(muon_check_router_balance_args(r, n, &bh, NULL, 0) == MUON_ERR_INVALID_ARGUMENT);
            b[1].bias = b[0].bias;
            EXPECT(muon_check_router_bias_args(b, n, 1e-3, NULL, 0) == MUON_ERR_INVALID_ARGUMENT);
        }
        free(m);
        free(r);
        free(b);
    }
    muon_block_matrix one;
    memset(&one, 0, sizeof one);
    one.param = fake(0, 0);
    one.grad = fake(1, 0);
    one.momentum = (float *)fake(2, 0);
    one.rows = one.cols = one.block_rows = one.block_cols = 64;
    one.param_pitch = one.grad_pitch = one.momentum_pitch = 64;
    /* every schedule is planned or refused: from one step of nothing to values that overflow */
    const double values[] = {0.0, 1.0, -1.0, 2.0, 3.4445, -4.775, 1e-300, 1e300, -1e300};
    for (int a = 0; a < 9; ++a)
        for (int bb = 0; bb < 9; ++bb)
            for (int cc = 0; cc < 9; ++cc)
                for (int32_t steps = 1; steps <= 16; steps += 5) {
                    for (int k = 0; k < 16; ++k) {
                        schedule[k].a = values[a];
                        schedule[k].b = values[bb];
                        schedule[k].c = values[cc];
                    }
                    hp.num_ns_steps = steps;
                    const muon_status st = muon_check_blocks_args(&one, 1, &hp, msg, sizeof msg);
                    EXPECT(st == MUON_OK || st == MUON_ERR_UNSUPPORTED);
                    if (fabs(values[a]) > 100 || fabs(values[bb]) > 100 || fabs(values[cc]) > 100)
                        EXPECT(st == MUON_ERR_UNSUPPORTED);
                }
    if (failures) return 1;
    printf("sanitized block and router checks: ok\n");
    return 0;
}
