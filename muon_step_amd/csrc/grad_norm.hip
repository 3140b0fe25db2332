// The 2-norm of many gradients together, and the factor that clips it.
//
// Squares and sums are fp64 (the square of an fp32 value is exact there), in an
// order that depends on the sizes alone: a workgroup sums its chunks, its lanes
// are joined in a fixed tree, and one workgroup adds up the workgroups' sums.
#include <algorithm>

#include "kernels.hpp"
#include "tensor_table.hpp"

namespace muon {

namespace {

constexpr int kThreads = 256;
constexpr int kChunk = 8192;  // elements of one chunk: four 16-byte loads of bf16 a lane

// Sum over the workgroup, valid in thread 0.
__device__ __forceinline__ double block_total(double v, double *sh) {
    for (int off = 32; off > 0; off >>= 1) v += __shfl_down(v, off, 64);
    if ((threadIdx.x & 63) == 0) sh[threadIdx.x >> 6] = v;
    __syncthreads();
    double r = 0.0;
    if (threadIdx.x == 0)
        for (int w = 0; w < kThreads / 64; ++w) r += sh[w];
    return r;
}

__device__ __forceinline__ void add_square(float x, double &acc) {
    const double d = x;
    acc = __builtin_fma(d, d, acc);  // the product is exact: one rounding
}

__global__ __launch_bounds__(kThreads) void grad_sumsq_kernel(const NormTable t, uint32_t chunks,
                                                              double *__restrict__ partials) {
    __shared__ double sh[kThreads / 64];
    double acc = 0.0;
    for (uint32_t c = blockIdx.x; c < chunks; c += gridDim.x) {
        const int e = owner_of(t.first, c);
        const NormDesc d = t.d[e];
        const bool bf16 = (t.bf16[e >> 6] >> (e & 63)) & 1;
        const int64_t k0 = static_cast<int64_t>(c - t.first[e]) * kChunk;
        const int n = static_cast<int>(min<int64_t>(kChunk, d.numel - k0));
        const bool vec = (reinterpret_cast<uintptr_t>(d.grad) & 15) == 0;  // a chunk starts at a multiple of 16 bytes
        if (bf16) {
            const uint16_t *p = static_cast<const uint16_t *>(d.grad) + k0;
            const int nv = vec ? n / 8 : 0;
            for (int i = threadIdx.x; i < nv; i += kThreads) {
                const u32x4 w = __builtin_nontemporal_load(as_global(reinterpret_cast<const u32x4 *>(p) + i));
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    add_square(__uint_as_float(w[q] << 16), acc);
                    add_square(__uint_as_float(w[q] & 0xffff0000u), acc);
                }
            }
            for (int i = 8 * nv + threadIdx.x; i < n; i += kThreads) add_square(bf16_bits_to_float(*as_global(p + i)), acc);
        } else {
            const float *p = static_cast<const float *>(d.grad) + k0;
            const int nv = vec ? n / 4 : 0;
            for (int i = threadIdx.x; i < nv; i += kThreads) {
                const floatx4 w = __builtin_nontemporal_load(as_global(reinterpret_cast<const floatx4 *>(p) + i));
#pragma unroll
                for (int q = 0; q < 4; ++q) add_square(w[q], acc);
            }
            for (int i = 4 * nv + threadIdx.x; i < n; i += kThreads) add_square(*as_global(p + i), acc);
        }
    }
    const double s = block_total(acc, sh);
    if (threadIdx.x == 0) partials[blockIdx.x] = s;
}

// Adds the workgroups' sums of one launch to the running total (first: starts
// it), and after the last launch writes the norm and the factor.
__global__ __launch_bounds__(kThreads) void grad_norm_kernel(const double *__restrict__ partials, int count,
                                                             double *__restrict__ total, int first, int last,
                                                             double max_norm, double *__restrict__ norm,
                                                             float *__restrict__ factor) {
    __shared__ double sh[kThreads / 64];
    double acc = 0.0;
    for (int i = threadIdx.x; i < count; i += kThreads) acc += partials[i];
    double s = block_total(acc, sh);
    if (threadIdx.x != 0) return;
    if (!first) s += *total;
    *total = s;
    if (!last) return;
    const double r = sqrt(s);
    *norm = r;
    // an infinite norm has no factor either: 0 would turn its gradients to NaN
    // in some places and to nothing in the others
    const bool finite = r <= 1.7976931348623157e308;
    *factor = !finite ? __builtin_nanf("") : (r > max_norm ? static_cast<float>(max_norm / r) : 1.0f);
}

}  // namespace

int64_t grad_norm_chunks(int64_t numel) { return (numel + kChunk - 1) / kChunk; }

hipError_t launch_grad_norm(const NormTable &t, uint32_t chunks, double *ws, bool first, bool last, double max_norm,
                            double *norm, float *factor, hipStream_t st) {
    double *partials = ws, *total = ws + kNormBlocks;
    const uint32_t blocks = std::min<uint32_t>(chunks, kNormBlocks);
    if (blocks > 0) {
        hipLaunchKernelGGL(grad_sumsq_kernel, dim3(blocks), dim3(kThreads), 0, st, t, chunks, partials);
        const hipError_t err = hipGetLastError();
        if (err != hipSuccess) return err;
    }
    hipLaunchKernelGGL(grad_norm_kernel, dim3(1), dim3(kThreads), 0, st, partials, static_cast<int>(blocks), total,
                       first ? 1 : 0, last ? 1 : 0, max_norm, norm, factor);
    return hipGetLastError();
}

}  // namespace muon
