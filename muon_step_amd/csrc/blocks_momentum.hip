// The first pass of the block step: momentum, N, and the sums of N N^T (blocks.hpp), for
// sides above 16.
//
// Bound by memory (10 bytes an element, and 4 s / 2 products of 16-bit parts for
// each: matrix cores 11%, vector units 15% busy at s = 128).  What counts is that
// neighbouring lanes read and write neighbouring memory, and that the next 32
// columns are on their way while the present ones are worked on.  The operand
// layout has neighbouring lanes in different rows; so a wave of a wide block works
// on M and N as they lie, eight lanes to 128 bytes of a row, and turns N's 16-bit
// parts through its own piece of shared memory.  (Loads and stores in the operand
// layout, 16 bytes a lane 32 or 16 rows apart, kept the address units busy: 3.7 and
// 4.1 TB/s.)  In tall blocks lanes that are neighbours in the operand are so in
// memory, T elements each.  1728 heads of 128 x 2048, bf16 gradients (4.5 GB): 1.03
// ms, 4.4 TB/s, where a copy moves 4.9; 16 heads 14 us.
#include "blocks_device.hpp"

namespace muon {

namespace {

// M and G of 32 columns of X, and what a lane does with them.
//   wide  lane 8 i + h, i < 8, h < 8: of rows 8 b + i, columns 4 h .. 4 h + 3
//   tall  lane (i, h), i < 32, h < 2: of columns 16 q + 8 h + e, e < 8, the T entries from T i on
template <int T, bool TALL, bool BF16> struct Columns {
    static constexpr int kSteps = TALL ? 2 : 4 * T;         // parts of the unit, loaded and used in turn
    static constexpr int kValues = TALL ? 8 * T : 4;
    static constexpr bool kPacked = BF16 && (!TALL || T % 2 == 0);
    static constexpr int kGrads = kPacked ? kValues / 2 : kValues;
    static constexpr int kGSize = BF16 ? 2 : 4;
    typedef char *Bytes;
    float m[kSteps][kValues];
    uint32_t g[kSteps][kGrads];
    const Place &at;
    int s, i, h;
    Bytes mom_row = nullptr, put_row = nullptr;
    const char *grad_row = nullptr;
    int left = 0, put_left = 0;
    uint32_t mom_lane, grad_lane, mom_part, grad_part;

    __device__ __forceinline__ Columns(const Place &place, int side, int lane) : at(place), s(side) {
        const uint32_t mp = static_cast<uint32_t>(at.mom_pitch), gp = static_cast<uint32_t>(at.grad_pitch);
        if constexpr (TALL) {
            i = lane & 31;
            h = lane >> 5;
            const uint32_t p = T * i < s ? T * i : 0;
            mom_lane = mom_part = (8 * h * mp + p) * 4;
            grad_lane = grad_part = (8 * h * gp + p) * kGSize;
        } else {
            i = lane >> 3;
            h = lane & 7;
            const uint32_t part = (s & 7) ? min(i, (s & 7) - 1) : i;  // the last, partial eight rows
            mom_lane = (i * mp + 4 * h) * 4;
            grad_lane = (i * gp + 4 * h) * kGSize;
            mom_part = (part * mp + 4 * h) * 4;
            grad_part = (part * gp + 4 * h) * kGSize;
        }
    }
    // Whether the lane's entries of a step belong to the block (wide: `rows` from the step's first on are there).
    __device__ __forceinline__ bool mine(int rows) const { return TALL ? T * i < s : i < rows; }
    __device__ __forceinline__ void begin(int x0) {
        mom_row = reinterpret_cast<Bytes>(at.mom + (TALL ? x0 * at.mom_pitch : x0));
        grad_row = at.grad + (TALL ? x0 * at.grad_pitch : x0) * kGSize;
        left = s;
    }
    __device__ __forceinline__ void begin_store(int x0) {
        put_row = reinterpret_cast<Bytes>(at.mom + (TALL ? x0 * at.mom_pitch : x0));
        put_left = s;
    }
    __device__ __forceinline__ void load(int step) {
        if constexpr (TALL) {
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const Bytes mr = mom_row + e * at.mom_pitch * 4;
                const char *gr = grad_row + e * at.grad_pitch * kGSize;
                floats(mr, &m[step][e * T]);
                if constexpr (kPacked) {
                    const auto v = load_at<typename WordsAt<T / 2, 2>::type>(gr, grad_lane);
#pragma unroll
                    for (int k = 0; k < T / 2; ++k) g[step][e * T / 2 + k] = v[k];
                } else {
#pragma unroll
                    for (int k = 0; k < T; ++k)
                        g[step][e * T + k] = BF16 ? static_cast<uint32_t>(load_at<uint16_t>(gr, grad_lane + 2 * k))
                                                  : load_at<uint32_t>(gr, grad_lane + 4 * k);
                }
            }
            mom_row += 16 * at.mom_pitch * 4;
            grad_row += 16 * at.grad_pitch * kGSize;
            asm volatile("" : "+s"(mom_row), "+s"(grad_row));
        } else {
            const bool full = left >= 8;
            const auto v = load_at<WordsAt<4, 4>::type>(mom_row, full ? mom_lane : mom_part);
            const auto u = load_at<typename WordsAt<kGrads, kGSize>::type>(grad_row, full ? grad_lane : grad_part);
#pragma unroll
            for (int k = 0; k < 4; ++k) m[step][k] = __uint_as_float(v[k]);
#pragma unroll
            for (int k = 0; k < kGrads; ++k) g[step][k] = u[k];
            left -= 8;
            if (left > 0) {  // steps past the last row read that step again
                mom_row += 8 * at.mom_pitch * 4;
                grad_row += 8 * at.grad_pitch * kGSize;
            } else {
                left += 8;
            }
            asm volatile("" : "+s"(mom_row), "+s"(grad_row), "+s"(left));
        }
    }
    // N of a step's values, zero where there is nothing; M's new ones take the old ones' place.
    __device__ __forceinline__ void input(int step, float factor, float mu, bool nesterov, float (&n)[kValues]) {
#pragma unroll
        for (int k = 0; k < kValues; ++k) {
            float gf;
            if constexpr (!BF16)
                gf = __uint_as_float(g[step][k]);
            else if constexpr (kPacked)
                gf = __uint_as_float(k % 2 ? g[step][k / 2] & 0xffff0000u : g[step][k / 2] << 16);
            else
                gf = __uint_as_float(g[step][k] << 16);
            gf *= factor;
            float &v = m[step][k];
            v = mu * v + gf;
            n[k] = nesterov ? __builtin_fmaf(mu, v, gf) : v;  // for the sums alone: one rounding
        }
        if (TALL ? s < 32 * T : s < 8 * (step + 1)) {
            const bool in = mine(s - 8 * step);
#pragma unroll
            for (int k = 0; k < kValues; ++k) n[k] = in ? n[k] : 0.0f;
        }
    }
    __device__ __forceinline__ void store(int step) {
        if constexpr (TALL) {
            if (mine(0)) {
#pragma unroll
                for (int e = 0; e < 8; ++e) put_floats<T>(put_row + e * at.mom_pitch * 4, mom_lane, &m[step][e * T]);
            }
            put_row += 16 * at.mom_pitch * 4;
        } else {
            if (mine(put_left)) put_floats<4>(put_row, mom_lane, m[step]);
            put_left -= 8;
            put_row += 8 * at.mom_pitch * 4;
        }
        asm volatile("" : "+s"(put_row), "+s"(put_left));
    }

  private:
    __device__ __forceinline__ void floats(Bytes row, float *to) const {
        if constexpr (T == 1) {
            to[0] = load_at<float>(row, mom_lane);
        } else {
            const auto v = load_at<typename WordsAt<T, 4>::type>(row, mom_lane);
#pragma unroll
            for (int k = 0; k < T; ++k) to[k] = __uint_as_float(v[k]);
        }
    }
    template <int N> __device__ __forceinline__ static void put_floats(Bytes row, uint32_t lane, const float *from) {
        if constexpr (N == 1) {
            store_at<float>(row, lane, from[0]);
        } else {
            typename WordsAt<N, 4>::type v;
#pragma unroll
            for (int k = 0; k < N; ++k) v[k] = __float_as_uint(from[k]);
            store_at(row, lane, v);
        }
    }
};

// A wave's 32 columns of N as 16-bit parts, row by row; 16 bytes behind each row
// keep lanes that read rows side by side off one another's banks.
template <int T> struct Turned {
    static constexpr int kPitch = 40;
    __attribute__((aligned(16))) __bf16 hi[32 * T][kPitch], lo[32 * T][kPitch];
};

// One part of one block: M <- mu M + G and the sum of N N^T over the part's
// columns.  Outside 2^-40 <= max |N| <= 2^40, where squares could leave fp32's
// range, the part is summed a second time as N 2^-shift.
template <int T, bool TALL, bool BF16>
__global__ __launch_bounds__(kThreads) void blocks_momentum_kernel(const BlockTable t, const BlockCall c) {
    union Shared {
        float sums[2 * kWaves * 1024];
        Turned<TALL ? 1 : T> turned[kWaves];
    };
    __shared__ __attribute__((aligned(16))) Shared sh;
    __shared__ uint32_t sh_largest[kWaves];
    const uint32_t block = blockIdx.x / c.parts, part = blockIdx.x % c.parts;  // block: of the launch
    const Place at = locate<BF16 ? 2 : 4, 2>(t, c, c.base + block);
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63;
    const int begin = part * c.part_len, end = min(begin + c.part_len, c.l);
    const float factor = c.factor ? *c.factor : 1.0f;
    const float mu = c.mu;
    const bool nesterov = c.nesterov != 0;
    float most = 0.0f;
    Triangle<T> sum;
    Columns<T, TALL, BF16> in(at, c.s, lane);

    auto note = [&](float n) { most = fmaxf(most, fabsf(n)); };  // leaves NaNs out

    auto turn = [&](Turned<T> &to, int b, const float (&n)[4]) {
        bf16x4 hi, lo;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            hi[e] = static_cast<__bf16>(n[e]);
            lo[e] = static_cast<__bf16>(n[e] - static_cast<float>(hi[e]));
        }
        *reinterpret_cast<bf16x4 *>(&to.hi[8 * b + in.i][4 * in.h]) = hi;
        *reinterpret_cast<bf16x4 *>(&to.lo[8 * b + in.i][4 * in.h]) = lo;
    };
    // The wave alone writes and reads its piece, and shared memory serves a wave in order.
    auto add_turned = [&](const Turned<T> &from) {
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
        __builtin_amdgcn_wave_barrier();
#pragma unroll
        for (int q = 0; q < 2; ++q) {
            bf16x8 hi[T], lo[T];
#pragma unroll
            for (int k = 0; k < T; ++k) {
                const int row = 32 * k + (lane & 31), col = 16 * q + 8 * (lane >> 5);
                hi[k] = *reinterpret_cast<const bf16x8 *>(&from.hi[row][col]);
                lo[k] = *reinterpret_cast<const bf16x8 *>(&from.lo[row][col]);
            }
            sum.add(hi, lo);
        }
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
        __builtin_amdgcn_wave_barrier();
    };

    // 32 columns from x0 on, element by element, past-the-end ones as zeros;
    // again: M is up to date, and N is scaled by 2^-shift.
    auto one = [&](int p, int x, bool again, int shift) {
        float n = 0.0f;
        if (p < c.s && x < end) {
            const int64_t row = TALL ? x : p, col = TALL ? p : x;
            float *m = at.mom + row * at.mom_pitch + col;
            const float g = load_grad<BF16>(at.grad, row * at.grad_pitch + col) * factor;
            float v = *as_global(m);
            if (!again) {
                v = mu * v + g;
                *as_global(m) = v;
            }
            n = nesterov ? mu * v + g : v;
        }
        if (again)
            n = ldexpf(n, -shift);
        else
            note(n);
        return n;
    };
    auto each = [&](int x0, bool again, int shift) {
        if constexpr (TALL) {
#pragma unroll
            for (int q = 0; q < 2; ++q) {
                bf16x8 hi[T], lo[T];
#pragma unroll
                for (int k = 0; k < T; ++k) {
                    float n[8];
#pragma unroll
                    for (int e = 0; e < 8; ++e) n[e] = one(T * in.i + k, x0 + 16 * q + 8 * in.h + e, again, shift);
                    split_bf(n, hi[k], lo[k]);
                }
                sum.add(hi, lo);
            }
        } else {
            Turned<T> &turned = sh.turned[wave];
#pragma unroll
            for (int b = 0; b < 4 * T; ++b) {
                float n[4];
#pragma unroll
                for (int e = 0; e < 4; ++e) n[e] = one(8 * b + in.i, x0 + 4 * in.h + e, again, shift);
                turn(turned, b, n);
                __builtin_amdgcn_sched_barrier(0);
            }
            add_turned(turned);
        }
    };

    sum.clear();
    // units that lie inside as a whole; in tall blocks lanes that do, too
    const int whole = (TALL && c.s % T != 0) ? begin : begin + (end - begin) / 32 * 32;
    int x0 = begin + 32 * wave;
    if (x0 < whole) {
        in.begin(x0);
#pragma unroll
        for (int k = 0; k < in.kSteps; ++k) in.load(k);
    }
    for (; x0 < whole; x0 += kBlockUnit) {
        const int next = x0 + kBlockUnit;
        if (next < whole) in.begin(next);
        in.begin_store(x0);
        if constexpr (TALL) {
#pragma unroll
            for (int q = 0; q < 2; ++q) {
                float n[8 * T];
                in.input(q, factor, mu, nesterov, n);
                in.store(q);
                if (next < whole) in.load(q);
                bf16x8 hi[T], lo[T];
#pragma unroll
                for (int k = 0; k < T; ++k) {
                    float x[8];
#pragma unroll
                    for (int e = 0; e < 8; ++e) {
                        x[e] = n[e * T + k];
                        note(x[e]);
                    }
                    split_bf(x, hi[k], lo[k]);
                }
                sum.add(hi, lo);
                __builtin_amdgcn_sched_barrier(0);
            }
        } else {
            Turned<T> &turned = sh.turned[wave];
#pragma unroll
            for (int b = 0; b < in.kSteps; ++b) {
                float n[4];
                in.input(b, factor, mu, nesterov, n);
                in.store(b);
                if (next < whole) in.load(b);
#pragma unroll
                for (int e = 0; e < 4; ++e) note(n[e]);
                turn(turned, b, n);
                if (b % 4 == 3) __builtin_amdgcn_sched_barrier(0);
            }
            add_turned(turned);
        }
    }
    // (the wave's next unit, so that every unit has one owner)
    for (; x0 < end; x0 += kBlockUnit) each(x0, false, 0);
    uint32_t largest = __float_as_uint(most);
#pragma unroll
    for (int off = 32; off > 0; off >>= 1)
        largest = max(largest, static_cast<uint32_t>(__shfl_xor(static_cast<int>(largest), off, 64)));
    if (lane == 0) sh_largest[wave] = largest;
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
        for (x0 = begin + 32 * wave; x0 < end; x0 += kBlockUnit) each(x0, true, shift);
    }
    // sums in range: a NaN on their diagonal was one in N
    bool spoilt = false;
#pragma unroll
    for (int k = 0; k < T; ++k)
#pragma unroll
        for (int r = 0; r < 16; ++r) spoilt |= __builtin_isnan(sum.tile[tri(k) + k][r]);
    spoilt = __syncthreads_or(spoilt) != 0;
    if (spoilt) largest = 0x7fc00000u;
    const int64_t slot = static_cast<int64_t>(block) * c.parts + part;
    sum.reduce(c.w.gram + slot * tri(T) * 1024, sh.sums);
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
