// The first pass of the block step: momentum, N, and the sums of N N^T (blocks.hpp).
#include "blocks_device.hpp"

namespace muon {

namespace {

// One part of one block: M <- mu M + G and the sum of N N^T over the part's
// columns.  Outside 2^-40 <= max |N| <= 2^40, where squares could leave fp32's
// range, the part is summed a second time as N 2^-shift.
template <int T, bool TALL, bool BF16>
__global__ __launch_bounds__(kThreads) void blocks_momentum_kernel(const BlockTable t, const BlockCall c) {
    __shared__ __attribute__((aligned(16))) float sh[2 * kWaves * 1024];
    __shared__ uint32_t sh_largest[kWaves];
    const uint32_t block = blockIdx.x / c.parts, part = blockIdx.x % c.parts;  // block: of the launch
    const Place at = locate<BF16 ? 2 : 4, 2>(t, c, c.base + block);
    const int wave = threadIdx.x >> 6, i = threadIdx.x & 31, h = threadIdx.x >> 5 & 1;
    const int begin = part * c.part_len, end = min(begin + c.part_len, c.l);
    const float factor = c.factor ? *c.factor : 1.0f;
    const float mu = c.mu;
    const bool nesterov = c.nesterov != 0;
    uint32_t largest = 0;
    Triangle<T> sum;

    auto note = [&](float n) { largest = max(largest, __float_as_uint(n) & 0x7fffffffu); };

    // 32 columns from x0 on, element by element, past-the-end ones as zeros;
    // again: M is up to date, and N is scaled by 2^-shift.
    auto each = [&](int x0, bool again, int shift) {
#pragma unroll
        for (int q = 0; q < 2; ++q) {
            bf16x8 hi[T], lo[T];
#pragma unroll
            for (int k = 0; k < T; ++k) {
                const int p = TALL ? T * i + k : 32 * k + i;
                float n[8];
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    const int x = TALL ? x0 + 16 * q + 8 * h + e : x0 + 16 * h + 8 * q + e;
                    n[e] = 0.0f;
                    if (p < c.s && x < end) {
                        const int64_t row = TALL ? x : p, col = TALL ? p : x;
                        float *m = at.mom + row * at.mom_pitch + col;
                        const float g = load_grad<BF16>(at.grad, row * at.grad_pitch + col) * factor;
                        float v = *as_global(m);
                        if (!again) {
                            v = mu * v + g;
                            *as_global(m) = v;
                        }
                        n[e] = nesterov ? mu * v + g : v;
                    }
                    if (again)
                        n[e] = ldexpf(n[e], -shift);
                    else
                        note(n[e]);
                }
                split_bf(n, hi[k], lo[k]);
            }
            sum.add(hi, lo);
        }
    };
    // 32 columns, all of them inside.
    auto whole = [&](int x0) {
        if constexpr (TALL) {
            const bool mine = T * i < c.s;
            const int p = mine ? T * i : 0;
#pragma unroll
            for (int q = 0; q < 2; ++q) {
                float m[8][T], g[8][T];
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    const int64_t row = x0 + 16 * q + 8 * h + e;
                    load_floats<T>(at.mom + row * at.mom_pitch + p, m[e]);
                    load_grads<BF16, T>(at.grad, row * at.grad_pitch + p, g[e]);
                }
                bf16x8 hi[T], lo[T];
#pragma unroll
                for (int k = 0; k < T; ++k) {
                    float n[8];
#pragma unroll
                    for (int e = 0; e < 8; ++e) {
                        const float gf = g[e][k] * factor;
                        m[e][k] = mu * m[e][k] + gf;
                        n[e] = nesterov ? mu * m[e][k] + gf : m[e][k];
                        n[e] = mine ? n[e] : 0.0f;
                        note(n[e]);
                    }
                    split_bf(n, hi[k], lo[k]);
                }
                if (mine) {
#pragma unroll
                    for (int e = 0; e < 8; ++e)
                        store_floats<T>(at.mom + (x0 + 16 * q + 8 * h + e) * at.mom_pitch + p, m[e]);
                }
                sum.add(hi, lo);
            }
        } else {
            bf16x8 hi[2][T], lo[2][T];
            float m[T][16], g[T][16];
#pragma unroll
            for (int k = 0; k < T; ++k) {
                const int64_t row = min(32 * k + i, c.s - 1);
                load_floats<16>(at.mom + row * at.mom_pitch + x0 + 16 * h, m[k]);
                load_grads<BF16, 16>(at.grad, row * at.grad_pitch + x0 + 16 * h, g[k]);
            }
#pragma unroll
            for (int k = 0; k < T; ++k) {
                const bool mine = 32 * k + i < c.s;
#pragma unroll
                for (int q = 0; q < 2; ++q) {
                    float n[8];
#pragma unroll
                    for (int e = 0; e < 8; ++e) {
                        const float gf = g[k][8 * q + e] * factor;
                        float &v = m[k][8 * q + e];
                        v = mu * v + gf;
                        n[e] = nesterov ? mu * v + gf : v;
                        n[e] = mine ? n[e] : 0.0f;
                        note(n[e]);
                    }
                    split_bf(n, hi[q][k], lo[q][k]);
                }
                if (mine) store_floats<16>(at.mom + (32 * k + i) * at.mom_pitch + x0 + 16 * h, m[k]);
            }
#pragma unroll
            for (int q = 0; q < 2; ++q) sum.add(hi[q], lo[q]);
        }
    };

    sum.clear();
    const bool vec = !TALL || c.s % T == 0;
    for (int x0 = begin + 32 * wave; x0 < end; x0 += kBlockUnit) {
        if (vec && x0 + 32 <= end)
            whole(x0);
        else
            each(x0, false, 0);
    }
#pragma unroll
    for (int off = 32; off > 0; off >>= 1) largest = max(largest, static_cast<uint32_t>(__shfl_xor(static_cast<int>(largest), off, 64)));
    if ((threadIdx.x & 63) == 0) sh_largest[wave] = largest;
    __syncthreads();
    largest = max(max(sh_largest[0], sh_largest[1]), max(sh_largest[2], sh_largest[3]));
    int shift = 0;
    if (largest != 0 && largest < 0x7f800000u) {
        int e;
        (void)frexpf(__uint_as_float(largest), &e);
        if (e < -40 || e > 40) shift = e;
    }
    if (shift != 0) {
        sum.clear();
        for (int x0 = begin + 32 * wave; x0 < end; x0 += kBlockUnit) each(x0, true, shift);
    }
    const int64_t slot = static_cast<int64_t>(block) * c.parts + part;
    sum.reduce(c.w.gram + slot * tri(T) * 1024, sh);
    if (threadIdx.x == 0) c.w.parts[slot] = BlockPart{largest, shift};
}

}  // namespace

hipError_t launch_blocks_momentum(const BlockTable &t, const BlockCall &c, uint32_t blocks, bool tall, bool grad_bf16,
                                  hipStream_t st) {
    return choose(c.s, tall, grad_bf16, [&](auto tiles, auto is_tall, auto bf16, auto) {
        hipLaunchKernelGGL((blocks_momentum_kernel<tiles.value, is_tall.value, bf16.value>), dim3(blocks * c.parts),
                           dim3(kThreads), 0, st, t, c);
        return hipGetLastError();
    });
}

}  // namespace muon
