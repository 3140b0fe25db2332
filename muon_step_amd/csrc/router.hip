// The balance loss of MoE routers, the tokens that each expert got, the gradient of the
// logits, and the step of the selection biases.
//
// For a sequence s of n tokens (those that take part) whose choices name expert i
// C_i times, p_t a token's normalised scores (softmax, or sigmoids over their sum):
//     loss_s = coef sum_i f_i P_i,   f_i = E C_i / (K n),   P_i = (1 / n) sum_t p_ti
// and the loss is the mean over the sequences that have tokens, S of them.  With
// c_i = coef E C_i / (S K n^2) it is the sum over tokens of sum_i c_i p_ti, and
//     d loss / d x_ti = p_ti (c_i - sum_j c_j p_tj)      times 1 - sigma(x_ti) for sigmoids.
// Counts depend on the choices alone, so one pass over the logits gives loss and
// gradient: count, balance, finish.  As sum_i p_ti = 1, a constant may be taken off
// c_i: off its mean the differences that make up the gradient do not cancel when
// loads are nearly even, and the mean itself goes into the loss.
#include <type_traits>

#include "router.hpp"
#include "tensor_table.hpp"
#include "vector_access.hpp"

namespace muon {

namespace {

constexpr int kWaves = kRouterThreads / 64;
constexpr int kCountWords = 8192;  // of a workgroup's own counts

// A sequence's tokens; what offsets leave out of the tokens is left out here.
struct Span {
    int begin, end;
};
__device__ __forceinline__ Span span_of(const RouterDesc &d, int s) {
    if (!d.offsets) return Span{0, d.tokens};
    const int lo = as_global(d.offsets)[s], hi = as_global(d.offsets)[s + 1];
    return Span{max(lo, 0), min(hi, d.tokens)};
}
// The last sequence of [lo, hi] that begins at or before the token.
__device__ __forceinline__ int sequence_of(const RouterDesc &d, int token, int lo, int hi) {
    if (!d.offsets) return 0;
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (as_global(d.offsets)[mid] <= token)
            lo = mid;
        else
            hi = mid - 1;
    }
    return lo;
}
__device__ __forceinline__ bool takes_part(const RouterDesc &d, int token, int s) {
    const Span p = span_of(d, s);
    return token >= p.begin && token < p.end && (!d.mask || as_global(d.mask)[token] != 0);
}

// One choice a thread and turn.  Counts of the sequences that the workgroup's
// tokens begin with are gathered in shared memory, as many as fit there.
__global__ __launch_bounds__(kRouterThreads) void router_count_kernel(const RouterTable t, const RouterCall c) {
    __shared__ uint32_t own[kCountWords];
    const Owners<64> owners(t.first);
    const int e = owners.of(blockIdx.x);
    const RouterDesc &d = t.d[e];
    const int begin = (blockIdx.x - t.first[e]) * c.per_block, end = min(begin + static_cast<int>(c.per_block), d.tokens);
    if (begin >= end) return;
    const int stride = d.experts + 1;
    const int s0 = sequence_of(d, begin, 0, d.sequences - 1), s1 = sequence_of(d, end - 1, s0, d.sequences - 1);
    const int window = min(kCountWords / stride, s1 - s0 + 1);
    for (int k = threadIdx.x; k < window * stride; k += kRouterThreads) own[k] = 0;
    __syncthreads();
    const uint32_t top = d.top_k;
    const int64_t first = static_cast<int64_t>(begin) * top;
    const uint32_t choices = (end - begin) * top;
    for (uint32_t k = threadIdx.x; k < choices; k += kRouterThreads) {
        const uint32_t row = k / top;
        const int token = begin + row;
        const int s = sequence_of(d, token, s0, s1);
        if (!takes_part(d, token, s)) continue;
        uint32_t *to = s - s0 < window ? own + (s - s0) * stride : nullptr;
        uint32_t *far = d.hist + static_cast<int64_t>(s) * stride;
        const int64_t x = d.chosen64 ? as_global(static_cast<const int64_t *>(d.chosen))[first + k]
                                     : as_global(static_cast<const int32_t *>(d.chosen))[first + k];
        auto add = [&](int i) {
            if (to)
                atomicAdd(to + i, 1u);
            else
                atomicAdd(far + i, 1u);
        };
        if (x >= 0 && x < d.experts) add(static_cast<int>(x));
        if (k == row * top) add(d.experts);
    }
    __syncthreads();
    for (int k = threadIdx.x; k < window * stride; k += kRouterThreads)
        if (own[k] != 0) atomicAdd(d.hist + static_cast<int64_t>(s0) * stride + k, own[k]);
}

// Sum and maximum over the LANES lanes of a row.
template <int LANES> __device__ __forceinline__ float row_sum(float x) {
#pragma unroll
    for (int off = 1; off < LANES; off *= 2) x += __shfl_xor(x, off, 64);
    return x;
}
template <int LANES> __device__ __forceinline__ float row_max(float x) {
#pragma unroll
    for (int off = 1; off < LANES; off *= 2) x = fmaxf(x, __shfl_xor(x, off, 64));
    return x;
}
__device__ __forceinline__ float exp_of(float x) { return __builtin_amdgcn_exp2f(x * 1.44269504088896341f); }

// The lane's logits of a row, those past the row's end as -inf (their score is zero).
template <int PER, bool BF16> __device__ __forceinline__ void load_row(const void *p, int64_t at, int there, float (&x)[PER]) {
    if (there >= PER) {
        if constexpr (BF16) {
#pragma unroll
            for (int k = 0; k < PER; k += 8) {
                uint32_t w[4];
                load_words<4, 2>(static_cast<const uint16_t *>(p) + at + k, w);
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    x[k + 2 * q] = __uint_as_float(w[q] << 16);
                    x[k + 2 * q + 1] = __uint_as_float(w[q] & 0xffff0000u);
                }
            }
        } else {
#pragma unroll
            for (int k = 0; k < PER; k += 4) {
                uint32_t w[4];
                load_words<4, 4>(static_cast<const float *>(p) + at + k, w);
#pragma unroll
                for (int q = 0; q < 4; ++q) x[k + q] = __uint_as_float(w[q]);
            }
        }
    } else {
#pragma unroll
        for (int k = 0; k < PER; ++k) {
            x[k] = -INFINITY;
            if (k < there) {
                if constexpr (BF16)
                    x[k] = bf16_bits_to_float(as_global(static_cast<const uint16_t *>(p))[at + k]);
                else
                    x[k] = as_global(static_cast<const float *>(p))[at + k];
            }
        }
    }
}
template <int PER, bool BF16> __device__ __forceinline__ void store_row(void *p, int64_t at, int there, const float (&x)[PER]) {
    if (there >= PER) {
        if constexpr (BF16) {
#pragma unroll
            for (int k = 0; k < PER; k += 8) {
                const uint32_t w[4] = {pack_bf16x2(x[k], x[k + 1]), pack_bf16x2(x[k + 2], x[k + 3]),
                                       pack_bf16x2(x[k + 4], x[k + 5]), pack_bf16x2(x[k + 6], x[k + 7])};
                store_words<4, 2>(static_cast<uint16_t *>(p) + at + k, w);
            }
        } else {
#pragma unroll
            for (int k = 0; k < PER; k += 4) {
                const uint32_t w[4] = {__float_as_uint(x[k]), __float_as_uint(x[k + 1]), __float_as_uint(x[k + 2]),
                                       __float_as_uint(x[k + 3])};
                store_words<4, 4>(static_cast<float *>(p) + at + k, w);
            }
        }
    } else {
#pragma unroll
        for (int k = 0; k < PER; ++k)
            if (k < there) {
                if constexpr (BF16)
                    as_global(static_cast<uint16_t *>(p))[at + k] = float_to_bf16_bits(x[k]);
                else
                    as_global(static_cast<float *>(p))[at + k] = x[k];
            }
    }
}

// LANES lanes take a row of up to LANES x PER logits, 64 / LANES rows a wave.
template <int LANES, int PER, bool BF16, bool SIGMOID>
__global__ __launch_bounds__(kRouterThreads) void router_balance_kernel(const RouterTable t, const RouterCall c) {
    __shared__ double sh_sum[kWaves];
    __shared__ int sh_sequences;
    constexpr int kRows = 64 / LANES;
    const Owners<64> owners(t.first);
    const int e = owners.of(blockIdx.x);
    const RouterDesc &d = t.d[e];
    const uint32_t mine = blockIdx.x - t.first[e];
    const int begin = mine * c.per_block, end = min(begin + static_cast<int>(c.per_block), d.tokens);
    const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
    const int row0 = lane / LANES, i0 = lane % LANES * PER;  // the lane's row of a wave's rows, and its first expert
    const int stride = d.experts + 1, there = d.experts - i0;
    const float grad_scale = c.grad_scale ? *as_global(c.grad_scale) : 1.0f;

    // the sequences that have tokens
    if (threadIdx.x == 0) sh_sequences = 0;
    __syncthreads();
    int found = 0;
    for (int s = threadIdx.x; s < d.sequences; s += kRouterThreads)
        found += as_global(d.hist)[static_cast<int64_t>(s) * stride + d.experts] != 0;
    if (found) atomicAdd(&sh_sequences, found);
    __syncthreads();
    const int sequences = sh_sequences;

    double loss = 0.0;
    int s = -1;
    Span span{0, 0};
    float away[PER], mean = 0.0f;
#pragma unroll
    for (int k = 0; k < PER; ++k) away[k] = 0.0f;
    for (int base = begin + wave * kRows; base < end; base += kWaves * kRows) {
        const int token = base + row0;
        if (token < end && (s < 0 || token >= span.end)) {
            // the row's sequence, and how far its experts' factors lie from their mean
            s = sequence_of(d, token, max(s, 0), d.sequences - 1);
            span = span_of(d, s);
            const uint32_t *hist = d.hist + static_cast<int64_t>(s) * stride;
            const double n = as_global(hist)[d.experts];
            double total = 0.0;
            uint32_t got[PER];
#pragma unroll
            for (int k = 0; k < PER; ++k) {
                got[k] = k < there ? as_global(hist)[i0 + k] : 0;
                total += got[k];
            }
#pragma unroll
            for (int off = 1; off < LANES; off *= 2) total += __shfl_xor(total, off, 64);
            const double unit = n > 0 ? c.coef / (static_cast<double>(sequences) * d.top_k * n * n) : 0.0;
            mean = static_cast<float>(unit * total);
#pragma unroll
            for (int k = 0; k < PER; ++k) away[k] = k < there ? static_cast<float>(unit * (static_cast<double>(d.experts) * got[k] - total)) : 0.0f;
        }
        const bool inside = token < end && token >= span.begin && token < span.end;
        const bool taking = inside && (!d.mask || as_global(d.mask)[token] != 0);
        float x[PER];
        load_row<PER, BF16>(d.logits, static_cast<int64_t>(taking ? token : begin) * d.pitch + i0, taking ? there : 0, x);
        // w: a score, not yet normalised; q: its derivative's factor
        float w[PER], q[PER], sum = 0.0f, dot = 0.0f;
        auto shifted = [&]() {  // exp(x - max)
            float most = -3.402823466e38f;
#pragma unroll
            for (int k = 0; k < PER; ++k) most = fmaxf(most, x[k]);
            most = row_max<LANES>(most);
#pragma unroll
            for (int k = 0; k < PER; ++k) w[k] = exp_of(x[k] - most);
        };
        auto add = [&]() {
            sum = 0.0f;
            dot = 0.0f;
#pragma unroll
            for (int k = 0; k < PER; ++k) {
                sum += w[k];
                dot = __builtin_fmaf(away[k], w[k], dot);
            }
            sum = row_sum<LANES>(sum);
            dot = row_sum<LANES>(dot);
        };
        if constexpr (SIGMOID) {
#pragma unroll
            for (int k = 0; k < PER; ++k) {
                const float z = exp_of(-fabsf(x[k])), r = __builtin_amdgcn_rcpf(1.0f + z), zr = z * r;
                w[k] = x[k] >= 0.0f ? r : zr;
                q[k] = x[k] >= 0.0f ? zr : r;
            }
            add();
            // rows whose sigmoids all vanish in fp32: there sigma(x) is exp(x)
            const bool vanish = taking && sum < 1e-30f;
            if (__any(vanish)) {
                float kept[PER], kept_sum = sum, kept_dot = dot;
#pragma unroll
                for (int k = 0; k < PER; ++k) kept[k] = w[k];
                shifted();
                add();
                if (!vanish) {
                    sum = kept_sum;
                    dot = kept_dot;
#pragma unroll
                    for (int k = 0; k < PER; ++k) w[k] = kept[k];
                }
            }
        } else {
            shifted();
            add();
        }
        // a row without any score: no probability, no gradient
        const float inv = sum == 0.0f ? 0.0f : 1.0f / sum;
        dot *= inv;
        if (taking && lane % LANES == 0) loss += static_cast<double>(dot) + (sum == 0.0f ? 0.0f : mean);
        if (inside && d.dlogits) {
            float g[PER];
            const float scale = taking ? inv * grad_scale : 0.0f;
#pragma unroll
            for (int k = 0; k < PER; ++k) {
                g[k] = w[k] * (away[k] - dot) * scale;
                if constexpr (SIGMOID) g[k] *= q[k];
                if (!taking) g[k] = 0.0f;
            }
            store_row<PER, BF16>(d.dlogits, static_cast<int64_t>(token) * d.dpitch + i0, there, g);
        }
    }
#pragma unroll
    for (int off = 32; off > 0; off >>= 1) loss += __shfl_down(loss, off, 64);
    if (lane == 0) sh_sum[wave] = loss;
    __syncthreads();
    if (threadIdx.x == 0) {
        double sum = 0.0;
        for (int k = 0; k < kWaves; ++k) sum += sh_sum[k];
        d.sums[mine] = sum;
    }
}

constexpr int kFinishThreads = 1024;
__global__ __launch_bounds__(kFinishThreads) void router_finish_kernel(const RouterTable t, uint32_t blocks, const RouterCall c) {
    __shared__ double sh_sum[kFinishThreads / 64];
    __shared__ unsigned long long counts[kMaxExperts + 1];
    const int e = blockIdx.x;
    const RouterDesc &d = t.d[e];
    const uint32_t next = e + 1 < kRouters ? min(t.first[e + 1], blocks) : blocks, count = next - t.first[e];
    const uint32_t stride = d.experts + 1;
    for (uint32_t i = threadIdx.x; i < stride; i += kFinishThreads) counts[i] = 0;
    __syncthreads();
    const int64_t words = static_cast<int64_t>(d.sequences) * stride;
    uint32_t i = threadIdx.x % stride;
    const uint32_t turn = kFinishThreads % stride;
    for (int64_t k = threadIdx.x; k < words; k += kFinishThreads) {
        const uint32_t n = as_global(d.hist)[k];
        if (n != 0) {
            atomicAdd(&counts[i], static_cast<unsigned long long>(n));
            as_global(d.hist)[k] = 0;
        }
        i += turn;
        if (i >= stride) i -= stride;
    }
    double sum = 0.0;
    for (uint32_t k = threadIdx.x; k < count; k += kFinishThreads) sum += as_global(d.sums)[k];
#pragma unroll
    for (int off = 32; off > 0; off >>= 1) sum += __shfl_down(sum, off, 64);
    if ((threadIdx.x & 63) == 0) sh_sum[threadIdx.x >> 6] = sum;
    __syncthreads();
    for (uint32_t k = threadIdx.x; k < stride - 1; k += kFinishThreads) {
        const int64_t n = static_cast<int64_t>(counts[k]);
        as_global(d.counts)[k] = c.accumulate ? as_global(d.counts)[k] + n : n;
    }
    if (threadIdx.x == 0) {
        double all = 0.0;
        for (int k = 0; k < kFinishThreads / 64; ++k) all += sh_sum[k];
        *d.loss = static_cast<float>(all);
    }
}

__global__ __launch_bounds__(kRouterThreads) void router_clear_kernel(uint32_t *p, int64_t words) {
    for (int64_t k = static_cast<int64_t>(blockIdx.x) * kRouterThreads + threadIdx.x; k < words;
         k += static_cast<int64_t>(gridDim.x) * kRouterThreads)
        p[k] = 0;
}

// b_i <- b_i - rate sign(C_i - mean C), the comparison in whole numbers.
__global__ __launch_bounds__(kRouterThreads) void router_bias_kernel(const RouterBiasTable t, float rate) {
    __shared__ int64_t sh_sum[kWaves];
    const RouterBiasDesc &d = t.d[blockIdx.x];
    int64_t total = 0;
    for (int64_t i = threadIdx.x; i < d.experts; i += kRouterThreads) total += as_global(d.counts)[i];
#pragma unroll
    for (int off = 32; off > 0; off >>= 1) total += __shfl_xor(total, off, 64);
    if ((threadIdx.x & 63) == 0) sh_sum[threadIdx.x >> 6] = total;
    __syncthreads();
    total = 0;
    for (int k = 0; k < kWaves; ++k) total += sh_sum[k];
    for (int64_t i = threadIdx.x; i < d.experts; i += kRouterThreads) {
        const int64_t excess = d.experts * as_global(d.counts)[i] - total;
        const float step = excess > 0 ? -rate : excess < 0 ? rate : 0.0f;
        as_global(d.bias)[i] += step;
    }
}

template <int LANES, int PER>
hipError_t launch_rows(const RouterTable &t, uint32_t blocks, const RouterCall &c, bool bf16, hipStream_t st) {
    const dim3 grid(blocks), block(kRouterThreads);
    if (c.sigmoid) {
        if (bf16)
            hipLaunchKernelGGL((router_balance_kernel<LANES, PER, true, true>), grid, block, 0, st, t, c);
        else
            hipLaunchKernelGGL((router_balance_kernel<LANES, PER, false, true>), grid, block, 0, st, t, c);
    } else {
        if (bf16)
            hipLaunchKernelGGL((router_balance_kernel<LANES, PER, true, false>), grid, block, 0, st, t, c);
        else
            hipLaunchKernelGGL((router_balance_kernel<LANES, PER, false, false>), grid, block, 0, st, t, c);
    }
    return hipGetLastError();
}

}  // namespace

hipError_t launch_router_count(const RouterTable &t, uint32_t blocks, const RouterCall &c, hipStream_t st) {
    hipLaunchKernelGGL(router_count_kernel, dim3(blocks), dim3(kRouterThreads), 0, st, t, c);
    return hipGetLastError();
}

hipError_t launch_router_balance(const RouterTable &t, uint32_t blocks, const RouterCall &c, int experts, bool bf16,
                                 hipStream_t st) {
    switch (router_lanes(experts)) {
        case 1: return launch_rows<1, 8>(t, blocks, c, bf16, st);
        case 2: return launch_rows<2, 8>(t, blocks, c, bf16, st);
        case 4: return launch_rows<4, 8>(t, blocks, c, bf16, st);
        case 8: return launch_rows<8, 8>(t, blocks, c, bf16, st);
        case 16: return launch_rows<16, 8>(t, blocks, c, bf16, st);
        case 32: return launch_rows<32, 8>(t, blocks, c, bf16, st);
        default: return experts <= 512 ? launch_rows<64, 8>(t, blocks, c, bf16, st) : launch_rows<64, 16>(t, blocks, c, bf16, st);
    }
}

hipError_t launch_router_finish(const RouterTable &t, int routers, uint32_t blocks, const RouterCall &c, hipStream_t st) {
    hipLaunchKernelGGL(router_finish_kernel, dim3(routers), dim3(kFinishThreads), 0, st, t, blocks, c);
    return hipGetLastError();
}

hipError_t launch_router_clear(uint32_t *p, int64_t words, hipStream_t st) {
    const int64_t blocks = (words + kRouterThreads - 1) / kRouterThreads;
    hipLaunchKernelGGL(router_clear_kernel, dim3(static_cast<uint32_t>(blocks < 1024 ? blocks : 1024)), dim3(kRouterThreads), 0,
                       st, p, words);
    return hipGetLastError();
}

hipError_t launch_router_bias(const RouterBiasTable &t, int routers, float rate, hipStream_t st) {
    hipLaunchKernelGGL(router_bias_kernel, dim3(routers), dim3(kRouterThreads), 0, st, t, rate);
    return hipGetLastError();
}

}  // namespace muon
