// The 2-norm of many gradients together, and the factor that clips it.
//
// Squares and sums are fp64 (the square of an fp32 value is exact there), in an
// order that depends on the sizes alone: a workgroup sums its chunks, its lanes
// are joined in a fixed tree, and one workgroup adds up the workgroups' sums.
//
// Bound by HBM: two or four bytes are read for one fp64 FMA.  Measured (us):
// 570e6 bf16 in 196 matrices 168.5, 420e6 fp32 in two 247 (6.8 TB/s); with
// chunks of 16 KB 169.5 and 256, handed out in turn instead of in runs 176 and
// 256; with 2048 workgroups 170 and 247; with plain instead of non-temporal
// loads 10% slower.
#include <algorithm>

#include "kernels.hpp"
#include "tensor_table.hpp"
#include "vector_access.hpp"

namespace muon {

namespace {

constexpr int kThreads = 256;

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

template <bool BF16> __device__ __forceinline__ void add_squares(const uint32_t (&w)[4], double &acc) {
#pragma unroll
    for (int q = 0; q < 4; ++q) {
        if constexpr (BF16) {
            add_square(__uint_as_float(w[q] << 16), acc);
            add_square(__uint_as_float(w[q] & 0xffff0000u), acc);
        } else {
            add_square(__uint_as_float(w[q]), acc);
        }
    }
}

// A whole chunk: every load of the lane first.
template <bool BF16> __device__ __forceinline__ void add_whole(const char *p, double &acc) {
    constexpr int kLoads = kNormChunk / 16 / kThreads;
    uint32_t w[kLoads][4];
#pragma unroll
    for (int i = 0; i < kLoads; ++i) load_words<4, BF16 ? 2 : 4>(p + 16 * (threadIdx.x + i * kThreads), w[i]);
#pragma unroll
    for (int i = 0; i < kLoads; ++i) add_squares<BF16>(w[i], acc);
}

// n elements: in 16-byte loads, and one by one what is left behind them.
template <bool BF16> __device__ __forceinline__ void add_part(const char *p, int n, double &acc) {
    constexpr int kSize = BF16 ? 2 : 4, kPer = 16 / kSize;
    for (int i = threadIdx.x; i < n / kPer; i += kThreads) {
        uint32_t w[4];
        load_words<4, kSize>(p + 16 * i, w);
        add_squares<BF16>(w, acc);
    }
    for (int i = n / kPer * kPer + threadIdx.x; i < n; i += kThreads) {
        if constexpr (BF16)
            add_square(bf16_bits_to_float(*as_global(reinterpret_cast<const uint16_t *>(p) + i)), acc);
        else
            add_square(*as_global(reinterpret_cast<const float *>(p) + i), acc);
    }
}

template <bool BF16>
__device__ __forceinline__ void add_chunk(const char *p, int n, double &acc) {
    if (n == kNormChunk / (BF16 ? 2 : 4))
        add_whole<BF16>(p, acc);
    else
        add_part<BF16>(p, n, acc);
}

// Joins the first `count` workgroups' sums, in their order, with the total of
// those before (first: there are none); after the call's last ones writes the
// norm and the factor.  One workgroup.
struct Finish {
    NormWorkspace *ws;
    int first, last;
    double max_norm;
    double *norm;
    float *factor;
};
__device__ __forceinline__ void finish_sums(const Finish &f, uint32_t count, double *sh) {
    double acc = 0.0;
    for (uint32_t i = threadIdx.x; i < count; i += kThreads) acc += f.ws->sums[i];
    double s = block_total(acc, sh);
    if (threadIdx.x != 0) return;
    if (!f.first) s += f.ws->total;
    f.ws->total = s;
    if (!f.last) return;
    const double r = sqrt(s);
    *f.norm = r;
    // an infinite norm has no factor either: 0 would turn its gradients to NaN
    // in some places and to nothing in the others
    const bool finite = r <= 1.7976931348623157e308;
    *f.factor = !finite ? __builtin_nanf("") : (r > f.max_norm ? static_cast<float>(f.max_norm / r) : 1.0f);
}

__global__ __launch_bounds__(kThreads) void grad_norm_finish_kernel(Finish f, uint32_t count) {
    __shared__ double sh[kThreads / 64];
    finish_sums(f, count, sh);
}

// Sums the squares of one table's gradients; workgroup b's sum goes to place
// at + b.  FUSED (small grids): the workgroup that finishes last also joins the
// sums, which saves a small call its second launch.  Who is last is told by a
// ticket: the counter of a grid of 2^k workgroups is never reset, and every
// 2^k-th ticket is a launch's last.  (Launches that overlap against the rules
// spoil their own sums but leave the counter right for those that follow.)
template <bool FUSED>
__global__ __launch_bounds__(kThreads) void grad_norm_kernel(const NormTable t, uint32_t chunks, uint32_t at,
                                                             Finish f) {
    __shared__ double sh[kThreads / 64];
    __shared__ int is_last;
    double acc = 0.0;
    // Consecutive chunks for each workgroup: it looks a tensor up once for many.
    const Owners<kNormTensors> owners(t.first);
    const uint32_t per = (chunks + gridDim.x - 1) / gridDim.x;
    const uint32_t stop = min((blockIdx.x + 1) * per, chunks);
    for (uint32_t c = blockIdx.x * per; c < stop;) {
        const int e = owners.of(c);
        const uint32_t begin = t.first[e], end = e + 1 < kNormTensors ? min(t.first[e + 1], chunks) : chunks;
        const int tail = t.tail[e] & ~kTailBf16;
        const bool bf16 = (t.tail[e] & kTailBf16) != 0;
        const int full = kNormChunk / (bf16 ? 2 : 4);
        const char *g = static_cast<const char *>(t.grad[e]);
        for (; c < min(end, stop); ++c) {
            const char *p = g + static_cast<int64_t>(c - begin) * kNormChunk;
            const int n = c + 1 == end ? tail : full;
            if (bf16)
                add_chunk<true>(p, n, acc);
            else
                add_chunk<false>(p, n, acc);
        }
    }
    const double s = block_total(acc, sh);
    if (threadIdx.x == 0) {
        f.ws->sums[at + blockIdx.x] = s;
        if (FUSED) {
            const uint32_t mask = gridDim.x - 1;
            const uint32_t ticket = __hip_atomic_fetch_add(&f.ws->tickets[__popc(mask)], 1u, __ATOMIC_ACQ_REL,
                                                           __HIP_MEMORY_SCOPE_AGENT);
            is_last = ((ticket + 1) & mask) == 0;
        }
    }
    if (!FUSED) return;
    __syncthreads();
    if (!is_last) return;
    __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "agent");
    finish_sums(f, at + gridDim.x, sh);
}

}  // namespace

hipError_t launch_grad_norm(const NormTable &t, uint32_t chunks, NormCall &call, bool last, hipStream_t st) {
    Finish f{call.ws, call.first ? 1 : 0, last ? 1 : 0, call.max_norm, call.norm, call.factor};
    const uint32_t at = call.at;
    if (last && chunks <= kNormFused) {
        uint32_t blocks = 1;
        while (blocks < chunks) blocks *= 2;
        hipLaunchKernelGGL(grad_norm_kernel<true>, dim3(blocks), dim3(kThreads), 0, st, t, chunks, at, f);
        return hipGetLastError();
    }
    const uint32_t blocks = std::min<uint32_t>(chunks, kNormBlocks);
    if (blocks > 0) {
        hipLaunchKernelGGL(grad_norm_kernel<false>, dim3(blocks), dim3(kThreads), 0, st, t, chunks, at, f);
        const hipError_t err = hipGetLastError();
        if (err != hipSuccess) return err;
    }
    call.at = at + blocks;
    if (!last && call.at + kNormBlocks <= kNormSums) return hipSuccess;  // room for the next table's sums
    hipLaunchKernelGGL(grad_norm_finish_kernel, dim3(1), dim3(kThreads), 0, st, f, call.at);
    call.first = false;
    call.at = 0;
    return hipGetLastError();
}

}  // namespace muon
