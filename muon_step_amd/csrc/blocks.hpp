// Muon steps on blocks with a smaller side of at most 128: the heads of an
// attention projection, the factors of an adapter.
//
// X is s x l with s <= 128, so the iteration X <- (a + b A + c A^2) X, A = X X^T,
// need not touch X's long rows at every step: X_k = P_k X_0 with P_k a product
// of s x s polynomials, and A follows in s x s matrices as well,
//     Q = a + b A + c A^2,   A <- Q A Q,   P <- Q P.
// A's rounding noise sits in the directions of small singular values too, where
// each step multiplies it by a^2 (11.9), so A is taken from X = P N again where
// that has grown too far (the host cuts the schedule into segments; the hybrid
// schedule into 4 + 6 steps).  One step over a block then is
//     momentum:  M, N, the partial sums of N N^T                  (reads G, M; writes M)
//     chain:     A = N N^T / ||N||^2, the first segment's P       (s x s, one workgroup a block)
//     regram:    X = P N, the partial sums of X X^T               (reads G, M)
//     chain:     the second segment's P
//     update:    O = P N, W                                       (reads G, M, W; writes W)
// Blocks with a smaller side of at most 16 take their sums and polynomials in fp64, in
// which the schedule is one segment (blocks_narrow.hip): momentum, chain, update.
// N is formed from M and G wherever it is needed: 6 bytes read an element, where
// a stored X would be 4 written and 4 read.
//
// Products run on the matrix cores with each fp32 operand as a sum of two
// 16-bit parts, hi and lo, and three products hi hi + hi lo + lo hi in fp32
// accumulators: bf16 parts (16 bits of significand), and lo lo too, for the first
// N N^T, whose scale is not known before it, fp16 parts (23 bits) of suitably
// scaled matrices everywhere else.
//
// Index basis of the smaller side.  A wave reads 32 lanes x T tiles of it; where
// memory is contiguous along the smaller side (tall blocks, X = N^T) lane i
// takes elements T i .. T i + T - 1, one for each tile, so basis index 32 t + i
// stands for element T i + t; in wide blocks it stands for itself.
//
// Fragments.  v_mfma_f32_32x32x16 wants of either operand, in lane (i, h), i < 32,
// h < 2, eight k of row (column) i; the accumulator holds in lane (j, h) rows
// 8 (r / 4) + 4 h + r % 4, r < 16, of column j.  The order of k is free as long
// as both operands agree, so chunk q (of two) of a tile takes accumulator
// registers 8 q .. 8 q + 7 as they are: an accumulator is the next product's
// operand without leaving its lane.
#pragma once

#include "common.hpp"

namespace muon {

// One weight of a launch: a grid of blocks, `across` of them beside each other.
struct BlockDesc {
    void *param;
    const void *grad;
    float *mom;
    float *ns_out;  // or nullptr
    uint32_t param_pitch, grad_pitch, mom_pitch, out_pitch;  // elements from row to row
    uint32_t across;
    uint32_t pad_;
};
// Weights of one launch, by value: 64 of 56 bytes, their first blocks, and the
// call's scalars fill the 4 KB of a launch's arguments.
constexpr int kBlockTensors = 64;
struct BlockTable {
    uint32_t first[kBlockTensors];  // blocks before each weight; 0xffffffff past the last
    BlockDesc d[kBlockTensors];
};

constexpr int kBlockSide = 128;      // largest smaller side of a block: four tiles of 32
constexpr int kBlockUnit = 128;      // columns of X that a workgroup takes at once: 32 for each wave
constexpr int kMaxChainSteps = 64;
// Largest smaller side of blocks that are worked on in fp64: one tile of its matrix
// instructions, whose products cost less there than their latency.  Sides of 17 to 32
// would take eight times as many: by their rate 8.5 us of a CU for ten steps, or 340 us for
// 10000 blocks of 32 x 256, whose bytes a copy moves in 320.
constexpr int kNarrowSide = 16;

// What one block needs between the launches (index: block of the launch).
struct BlockScalars {
    float inv_norm;   // 1 / ||N 2^shift||
    int32_t shift;    // N 2^shift has an rms of 1/2 to 1
    float update;     // lr x scale of the block's update
    int32_t poly;     // P's fragments are those of P 2^-poly
};
// The sum of squares' range of one part of a block.
struct BlockPart {
    uint32_t largest;  // bits of max |N|; of a NaN where N holds one
    int32_t shift;     // its Gram is that of N 2^-shift
};
struct BlockWork {
    float *gram;           // [block][part][tile], the lower triangle's tiles as lanes hold them
    double *narrow;        // [block][part]: the same of a side of kNarrowSide
    BlockPart *parts;      // [block][part]
    _Float16 *poly;        // [block]: P's rows as operand fragments, hi then lo
    float *poly_own;       // [block]: P's columns as the chain holds them
    BlockScalars *scalars; // [block]
};

struct BlockCall {
    BlockWork w;
    const float *factor;  // or nullptr
    uint32_t base;                  // the launch's first block in the table
    int32_t s, l;                   // smaller and larger side of a block
    int32_t block_rows, block_cols;
    int32_t parts, part_len;        // a block's l columns in `parts` ranges of part_len
    float mu;
    int32_t nesterov;
    float decay;
};

// The polynomials of one segment of the schedule (between two Gram matrices
// taken from X), and what surrounds them.
struct BlockChain {
    BlockWork w;
    int32_t s, l, parts, steps;
    int32_t first, last;       // segment
    int32_t unit_rms, tall;
    float update;              // lr gamma sqrt(max(n, m)); unit RMS: lr gamma sqrt(n m)
    int32_t poly_least;        // P's fragments are those of P 2^-e, e at least this
    struct Step {
        float a, b, c;
    } step[kMaxChainSteps];
};

// All steps of the schedule, for sides up to kNarrowSide.
struct NarrowChain {
    BlockWork w;
    int32_t s, l, parts, steps;
    int32_t unit_rms, poly_least;  // as in BlockChain
    float update;
    int32_t pad_;
    struct Step {
        double a, b, c;
    } step[kMaxChainSteps];
};

inline int block_tiles(int64_t s) { return static_cast<int>((s + 31) / 32); }

hipError_t launch_blocks_momentum(const BlockTable &t, const BlockCall &c, uint32_t blocks, bool tall, bool grad_bf16,
                                  hipStream_t st);
hipError_t launch_blocks_chain(const BlockChain &c, uint32_t blocks, hipStream_t st);
hipError_t launch_narrow_momentum(const BlockTable &t, const BlockCall &c, uint32_t blocks, bool tall, bool grad_bf16,
                                  hipStream_t st);
hipError_t launch_narrow_chain(const NarrowChain &c, uint32_t blocks, hipStream_t st);
hipError_t launch_blocks_regram(const BlockTable &t, const BlockCall &c, uint32_t blocks, bool tall, bool grad_bf16,
                                hipStream_t st);
hipError_t launch_blocks_update(const BlockTable &t, const BlockCall &c, uint32_t blocks, bool tall, bool grad_bf16,
                                bool param_bf16, hipStream_t st);

}  // namespace muon
