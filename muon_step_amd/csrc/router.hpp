// MoE routers: balance loss, expert counts and gradients, and the step of the
// selection biases (router.hip): what host and kernels share.
#pragma once

#include "common.hpp"

namespace muon {

struct RouterDesc {
    const void *logits;
    void *dlogits;           // or nullptr
    const void *chosen;
    const int32_t *offsets;  // or nullptr: one sequence of all tokens
    const uint8_t *mask;     // or nullptr
    int64_t *counts;
    float *loss;
    uint32_t *hist;          // [sequence][experts + 1]: choices of each expert, and tokens; zero between calls
    double *sums;            // of the loss, one for each workgroup
    uint32_t pitch, dpitch;
    int32_t tokens, experts, top_k, sequences;
    int32_t chosen64;
    int32_t pad_;
};
// Routers of one launch, by value: 32 of 104 bytes and their first workgroups.
constexpr int kRouters = 32;
struct RouterTable {
    uint32_t first[64];  // workgroups before each router; 0xffffffff past the last
    RouterDesc d[kRouters];
};
struct RouterCall {
    double coef;
    const float *grad_scale;  // or nullptr
    uint32_t *live;           // [router of the launch]: sequences that have tokens; zero between calls
    uint32_t per_block;       // tokens of a workgroup
    int32_t sigmoid, accumulate;
};

constexpr int kRouterThreads = 256;
constexpr int kMaxExperts = 1024;
constexpr int kCountWords = 8192;    // counts that a workgroup has room for
constexpr int kSmallThreads = 1024;
constexpr int kFinishThreads = 1024;
// Counts that one of the last launch's workgroups adds up, unless there would be more
// of these than kFinishSlices.  131072 tokens of 256 experts take 50 us in 37 sequences,
// 80 in 4096, of 64 experts 100 in 131072.
constexpr int kFinishWords = 16384, kFinishSlices = 1024;
__host__ __device__ inline uint32_t finish_sequences(int experts) { return kFinishWords / (experts + 1); }  // 15 at least
// Routers whose logits, and 24 for each token's choices, are at most this many, and
// whose counts fit a workgroup, are one workgroup's work each.  In us, as one launch
// and as three: 2048 tokens of 8 experts 10.2 and 11.4, 4096 16.2 and 11.8; 512 of 64
// 9.1 and 12.9, 1024 12.8 and 12.8; 128 of 256 9.1 and 13.5, 512 19.2 and 13.8.
constexpr int64_t kSmallWork = 81920;
inline bool small_router(int64_t tokens, int64_t experts) { return tokens * (experts + 24) <= kSmallWork; }

// Lanes that share a row of `experts` logits: 8 of them each up to 32 experts, 16
// above (which halves what a row costs beside its elements: 27 x 8192 x 64 41.5 to
// 36.7 us).  24 where that leaves fewer places empty are slower, with fewer bytes on
// their way: 72 experts 31 to 34 us, 384 47 to 56.
inline int router_lanes(int experts) {
    const int each = experts <= 32 ? 8 : 16;
    int lanes = 1;
    while (lanes * each < experts) lanes *= 2;
    return lanes;
}

// Counts the choices of each sequence and expert into hist.
hipError_t launch_router_count(const RouterTable &t, uint32_t blocks, const RouterCall &c, hipStream_t st);
// Gradients, and the workgroups' sums of the loss.  All routers of the table have
// the same type and router_lanes().
hipError_t launch_router_balance(const RouterTable &t, uint32_t blocks, const RouterCall &c, int experts, bool bf16,
                                 hipStream_t st);
// All of it for routers that are one workgroup's work each: hist and sums are not used.
hipError_t launch_router_small(const RouterTable &t, int routers, const RouterCall &c, int experts, bool bf16, hipStream_t st);
// Counts and loss from hist and sums (t.first: launch_router_balance's, and its
// `blocks`); hist is zero behind it.
hipError_t launch_router_finish(const RouterTable &t, int routers, uint32_t blocks, const RouterCall &c, hipStream_t st);
// Zeroes memory that hist will lie in, and `live`.
hipError_t launch_router_clear(uint32_t *p, int64_t words, uint32_t *live, hipStream_t st);

struct RouterBiasDesc {
    float *bias;
    const int64_t *counts;
    int64_t experts;
};
constexpr int kRouterBiases = 128;
struct RouterBiasTable {
    RouterBiasDesc d[kRouterBiases];
};
hipError_t launch_router_bias(const RouterBiasTable &t, int routers, float rate, hipStream_t st);

}  // namespace muon
