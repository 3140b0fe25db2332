// The passes of the block step that multiply N by P (blocks.hpp).
#include "blocks_device.hpp"

namespace muon {

namespace {

// ------------------------------------------------------------ products with N

// M and G of 32 V columns of X as a wave loads them, and N from them.  A lane
// holds column j (wide blocks: columns V j .. V j + V - 1) and, of the smaller
// side, for chunk (t, q) basis indices 32 t + 16 q + 8 a + 4 h + b, a < 2, b < 4.
// They come in phases: in wide blocks each chunk is one, eight rows that lanes
// read side by side; in tall ones the T chunks of one q, as two runs of 4 T
// elements that lie side by side in the lane's row of memory.  A phase's
// registers are loaded for the next columns as soon as they are used up, so that
// a wave always has most of a unit (24 KB at T = 4) on its way.
//
// Places outside of the block are read as others inside of it: what the products
// make of them meets P's zeros (its rows and columns past the smaller side) or
// belongs to columns that nobody stores or sums.  EVEN: a tall block's runs lie
// inside or outside as a whole (4 T divides its smaller side).
template <int T, int V, bool TALL, bool BF16, bool EVEN> struct Stream {
    static_assert(!TALL || V == 1, "a tall block's lane holds one column");
    static constexpr int kPhases = TALL ? 2 : 2 * T, kChunks = TALL ? T : 1;
    static constexpr int kValues = 8 * kChunks * V;              // of a phase
    static constexpr int kGrads = BF16 && (TALL || V == 2) ? kValues / 2 : kValues;  // words of G
    static constexpr int kGSize = BF16 ? 2 : 4;
    typedef const char *Bytes;
    float m[kPhases][kValues];
    uint32_t g[kPhases][kGrads];
    const Place &at;
    const BlockCall &c;
    float factor;
    int j, h, shift;
    // wide: where the next phase's rows begin, and a lane's bytes behind a row's
    // begin: in a whole group of eight rows, and for each b in the last, partial one
    Bytes mom_row = nullptr, grad_row = nullptr, mom_first = nullptr, grad_first = nullptr;
    int left = 0;  // rows from there to the block's end
    uint32_t mom_lane = 0, grad_lane = 0, mom_part[4] = {}, grad_part[4] = {};

    __device__ __forceinline__ Stream(const Place &place, const BlockCall &call, float f, int lane, int sh)
        : at(place), c(call), factor(f), j(lane & 31), h(lane >> 5), shift(sh) {}

    // Before the phases of columns x0 ..; `end`: the first column that is not there.
    int64_t mom_at = 0, grad_at = 0;  // tall: the lane's row of memory
    bool odd = false;                 // wide, V = 2: the lane's second column is what both loads hold
    __device__ __forceinline__ void begin(int x0, int end) {
        if constexpr (TALL) {
            const int64_t row = min(x0 + j, end - 1);
            mom_at = row * at.mom_pitch;
            grad_at = row * at.grad_pitch;
        } else {
            // a pair that would reach past the end starts one column earlier (a
            // single column: its own, twice)
            const int x = x0 + V * j, last = max(end - V, 0);
            const uint32_t col = min(x, last);
            odd = V == 2 && x == last + 1;
            const uint32_t mp = static_cast<uint32_t>(at.mom_pitch), gp = static_cast<uint32_t>(at.grad_pitch);
            mom_lane = (4 * h * mp + col) * 4;
            grad_lane = (4 * h * gp + col) * kGSize;
#pragma unroll
            for (int b = 0; b < 4; ++b) {
                const uint32_t row = min(4 * h + b, (c.s & 7) - 1);  // unused where s % 8 == 0
                mom_part[b] = (row * mp + col) * 4;
                grad_part[b] = (row * gp + col) * kGSize;
            }
            mom_first = reinterpret_cast<Bytes>(at.mom);
            grad_first = at.grad;
            mom_row = mom_first;
            grad_row = grad_first;
            left = c.s;
        }
    }
    __device__ __forceinline__ void load(int ph) {
        if constexpr (TALL) {
#pragma unroll
            for (int a = 0; a < 2; ++a) {
                const int run = T * (16 * ph + 8 * a + 4 * h);
                if constexpr (EVEN) {
                    const int p = run < c.s ? run : 0;
                    words<4 * T, 4>(at.mom + mom_at + p, reinterpret_cast<uint32_t *>(&m[ph][a * 4 * T]));
                    words<(BF16 ? 2 : 4) * T, kGSize>(at.grad + (grad_at + p) * kGSize, &g[ph][a * (BF16 ? 2 : 4) * T]);
                } else {
                    checked(ph, a, run);
                }
            }
        } else {
#pragma unroll
            for (int a = 0; a < 2; ++a) {
                const bool there = left > 0, full = (there ? left : c.s) >= 8;
                const Bytes mr = there ? mom_row : mom_first, gr = there ? grad_row : grad_first;
#pragma unroll
                for (int b = 0; b < 4; ++b) {
                    const int e = 4 * a + b;
                    const Bytes mp = mr + (full ? b * at.mom_pitch * 4 : 0), gp = gr + (full ? b * at.grad_pitch * kGSize : 0);
                    const uint32_t ml = full ? mom_lane : mom_part[b], gl = full ? grad_lane : grad_part[b];
                    if constexpr (V == 1) {
                        m[ph][e] = global<float>(mp, ml);
                        g[ph][e] = BF16 ? static_cast<uint32_t>(global<uint16_t>(gp, gl)) : global<uint32_t>(gp, gl);
                    } else {
                        const auto v = global<FloatsAt<2>::type>(mp, ml);
                        m[ph][2 * e] = v[0];
                        m[ph][2 * e + 1] = v[1];
                        if constexpr (BF16) {
                            typedef uint32_t word __attribute__((aligned(2)));
                            g[ph][e] = global<word>(gp, gl);
                        } else {
                            const auto u = global<FloatsAt<2>::type>(gp, gl);
                            g[ph][2 * e] = __float_as_uint(u[0]);
                            g[ph][2 * e + 1] = __float_as_uint(u[1]);
                        }
                    }
                }
                mom_row += 8 * at.mom_pitch * 4;
                grad_row += 8 * at.grad_pitch * kGSize;
                // the compiler would form every row's address ahead of the loop, and spill them
                left -= 8;
                asm volatile("" : "+s"(mom_row), "+s"(grad_row), "+s"(left));
            }
        }
    }
    // N 2^shift of chunk `sub` of a phase, column v, as fp16 pairs.
    __device__ __forceinline__ void fragment(int ph, int sub, int v, half8 &hi, half8 &lo) const {
        float x[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const int i = TALL ? ((e >> 2) * 4 + (e & 3)) * T + sub : e * V + v;
            float n = m[ph][i];
            if (c.nesterov) n = c.mu * n + grad_value(ph, i) * factor;
            if (V == 2 && v == 0) {  // the block's last column alone: its lane holds it second
                float other = m[ph][i + V - 1];
                if (c.nesterov) other = c.mu * other + grad_value(ph, i + V - 1) * factor;
                n = odd ? other : n;
            }
            x[e] = __builtin_amdgcn_ldexpf(n, shift);
        }
        split_half(x, hi, lo);
    }

  private:
    __device__ __forceinline__ float grad_value(int ph, int i) const {
        if constexpr (!BF16) return __uint_as_float(g[ph][i]);
        if constexpr (kGrads == kValues) return __uint_as_float(g[ph][i] << 16);
        return __uint_as_float(i % 2 ? g[ph][i / 2] & 0xffff0000u : g[ph][i / 2] << 16);
    }
    template <class W> __device__ __forceinline__ static W global(Bytes row, uint32_t lane) {
        return *(const W __attribute__((address_space(1))) *)((const char __attribute__((address_space(1))) *)row + lane);
    }
    // Tall: a run that the smaller side's end may cut.
    __device__ __forceinline__ void checked(int ph, int a, int p) {
#pragma unroll
        for (int i = 0; i < 4 * T; ++i) {
            const int from = min(p + i, c.s - 1);
            m[ph][a * 4 * T + i] = as_global(at.mom)[mom_at + from];
            if constexpr (BF16) {
                const uint32_t v = as_global(reinterpret_cast<const uint16_t *>(at.grad))[grad_at + from];
                uint32_t &w = g[ph][a * 2 * T + i / 2];
                w = i % 2 ? w | v << 16 : v;
            } else {
                g[ph][a * 4 * T + i] = as_global(reinterpret_cast<const uint32_t *>(at.grad))[grad_at + from];
            }
        }
    }
    template <int N, int A> __device__ __forceinline__ static void words(const void *p, uint32_t *to) {
        constexpr int W = N % 4 == 0 ? 4 : 2;
        typedef uint32_t type __attribute__((ext_vector_type(W), aligned(A)));
#pragma unroll
        for (int i = 0; i < N; i += W) {
            const type v = ((const type __attribute__((address_space(1))) *)p)[i / W];
#pragma unroll
            for (int k = 0; k < W; ++k) to[i + k] = v[k];
        }
    }
};

// P's fragments in shared memory.
template <int T> struct Poly {
    half8 hi[T][2 * T][64], lo[T][2 * T][64];
    __device__ __forceinline__ void load(const _Float16 *src) {
        const half8 *from = reinterpret_cast<const half8 *>(src);
        half8 *to = &hi[0][0][0];
        for (int k = threadIdx.x; k < T * T * 256; k += kThreads) to[k] = from[k];
    }
};

// P times the columns that `in` holds.  NT: as (P N)^T, X's columns as rows of the
// result; otherwise as P N.  next: columns to load behind the ones used, none at or past end.
template <bool NT, int T, int V, bool TALL, bool BF16, bool EVEN>
__device__ __forceinline__ void times_poly(floatx16 (&acc)[V][T], Stream<T, V, TALL, BF16, EVEN> &in, const Poly<T> &poly, int lane,
                                           int next, int end) {
    typedef Stream<T, V, TALL, BF16, EVEN> S;
#pragma unroll
    for (int v = 0; v < V; ++v)
#pragma unroll
        for (int i = 0; i < T; ++i)
#pragma unroll
            for (int r = 0; r < 16; ++r) acc[v][i][r] = 0.0f;
    if (next < end) in.begin(next, end);
#pragma unroll
    for (int ph = 0; ph < S::kPhases; ++ph) {
#pragma unroll
        for (int sub = 0; sub < S::kChunks; ++sub) {
            const int chunk = TALL ? 2 * sub + ph : ph;
            half8 ph_hi[T], ph_lo[T], hi[V], lo[V];
#pragma unroll
            for (int i = 0; i < T; ++i) {
                ph_hi[i] = poly.hi[i][chunk][lane];
                ph_lo[i] = poly.lo[i][chunk][lane];
            }
#pragma unroll
            for (int v = 0; v < V; ++v) in.fragment(ph, sub, v, hi[v], lo[v]);
            if (sub + 1 == S::kChunks && next < end) in.load(ph);
#pragma unroll
            for (int k = 0; k < 3; ++k)
#pragma unroll
                for (int i = 0; i < T; ++i)
#pragma unroll
                    for (int v = 0; v < V; ++v) {
                        const half8 a = k == 2 ? ph_lo[i] : ph_hi[i], b = k == 1 ? lo[v] : hi[v];
                        acc[v][i] = NT ? mfma(b, a, acc[v][i]) : mfma(a, b, acc[v][i]);
                    }
            __builtin_amdgcn_sched_barrier(0);
        }
    }
}

// One part of one block: the sum of X X^T, X = P N / ||N||, over the part's columns.
template <int T, bool TALL, bool BF16, bool EVEN>
__global__ __launch_bounds__(kThreads) void blocks_regram_kernel(const BlockTable t, const BlockCall c) {
    union Shared {
        Poly<T> poly;
        float sums[2 * kWaves * 1024];
    };
    __shared__ __attribute__((aligned(16))) Shared sh;
    const uint32_t block = blockIdx.x / c.parts, part = blockIdx.x % c.parts;  // block: of the launch
    const Place at = locate<BF16 ? 2 : 4, 2>(t, c, c.base + block);
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63;
    const int begin = part * c.part_len, end = min(begin + c.part_len, c.l);
    const BlockScalars k = c.w.scalars[block];
    const float scale = c.poly_scale * k.inv_norm * kScaleX;
    Stream<T, 1, TALL, BF16, EVEN> in(at, c, c.factor ? *c.factor : 1.0f, lane, k.shift);
    int x0 = begin + 32 * wave;
    if (x0 < end) {
        in.begin(x0, end);
#pragma unroll
        for (int ph = 0; ph < in.kPhases; ++ph) in.load(ph);
    }
    sh.poly.load(c.w.poly + static_cast<int64_t>(block) * (T * T * 2048));
    __syncthreads();
    Triangle<T> sum;
    sum.clear();
    const int h = lane >> 5;
    for (; x0 < end; x0 += kBlockUnit) {
        floatx16 acc[1][T];
        times_poly<true>(acc, in, sh.poly, lane, x0 + kBlockUnit, end);
        if (x0 + 32 > end) {  // columns that are not there
#pragma unroll
            for (int i = 0; i < T; ++i)
#pragma unroll
                for (int r = 0; r < 16; ++r) acc[0][i][r] = x0 + acc_row(r, h) < end ? acc[0][i][r] : 0.0f;
        }
#pragma unroll
        for (int q = 0; q < 2; ++q) {
            half8 hi[T], lo[T];
#pragma unroll
            for (int i = 0; i < T; ++i) {
                float x[8];
#pragma unroll
                for (int e = 0; e < 8; ++e) x[e] = acc[0][i][8 * q + e] * scale;
                split_half(x, hi[i], lo[i]);
            }
            sum.add(hi, lo);
            __builtin_amdgcn_sched_barrier(0);
        }
    }
    __syncthreads();
    sum.reduce(c.w.gram + (static_cast<int64_t>(block) * c.parts + part) * tri(T) * 1024, sh.sums);
}

// W <- fl(fl(d W) - fl(s O)) and O to ns_out, of one row of memory: its uniform
// begin and the lane's element behind it; N elements that lie side by side.
struct Row {
    char *param;
    char *out;  // or nullptr
    __device__ __forceinline__ void keep() { asm volatile("" : "+s"(param), "+s"(out)); }
};
template <bool PBF16, int N>
__device__ __forceinline__ void update_run(char *param, char *out, uint32_t param_lane, uint32_t out_lane, const float (&o)[N],
                                           float d, float s) {
    typedef char __attribute__((address_space(1))) *place;
    if constexpr (PBF16) {
        const place p = (place)param + param_lane;
        if constexpr (N == 1 || N == 3) {
            typedef uint16_t __attribute__((address_space(1))) *halves;
#pragma unroll
            for (int k = 0; k < N; ++k)
                ((halves)p)[k] = float_to_bf16_bits(d * bf16_bits_to_float(((halves)p)[k]) - s * o[k]);
        } else {
            typedef typename HalvesAt<N>::type __attribute__((address_space(1))) *halves;
            auto v = *(halves)p;
#pragma unroll
            for (int k = 0; k < N; ++k) v[k] = float_to_bf16_bits(d * bf16_bits_to_float(v[k]) - s * o[k]);
            *(halves)p = v;
        }
    } else {
        float *p = (float *)((place)param + param_lane);
        float w[N];
        load_floats<N>(p, w);
#pragma unroll
        for (int k = 0; k < N; ++k) w[k] = d * w[k] - s * o[k];
        store_floats<N>(p, w);
    }
    if (out) store_floats<N>((float *)((place)out + out_lane), o);
}

// The last pass: O = P N / ||N|| and W of one part of one block.
template <int T, bool TALL, bool BF16, bool PBF16, bool EVEN>
__global__ __launch_bounds__(kThreads) void blocks_update_kernel(const BlockTable t, const BlockCall c) {
    // wide blocks: two columns a lane, so that bf16 gradients and weights move in words
    constexpr int V = TALL ? 1 : 2, kPSize = PBF16 ? 2 : 4;
    __shared__ __attribute__((aligned(16))) Poly<T> poly;
    const uint32_t block = blockIdx.x / c.parts, part = blockIdx.x % c.parts;  // block: of the launch
    const Place at = locate<BF16 ? 2 : 4, kPSize>(t, c, c.base + block);
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63, j = lane & 31, h = lane >> 5;
    const int begin = part * c.part_len, end = min(begin + c.part_len, c.l);
    const BlockScalars k = c.w.scalars[block];
    const float scale = c.poly_scale * k.inv_norm;
    Stream<T, V, TALL, BF16, EVEN> in(at, c, c.factor ? *c.factor : 1.0f, lane, k.shift);
    constexpr int kStride = V * kBlockUnit;
    int x0 = begin + 32 * V * wave;
    if (x0 < end) {
        in.begin(x0, end);
#pragma unroll
        for (int ph = 0; ph < in.kPhases; ++ph) in.load(ph);
    }
    poly.load(c.w.poly + static_cast<int64_t>(block) * (T * T * 2048));
    __syncthreads();
    // the lane's place behind the begin of the first of eight rows (wide: of the
    // smaller side, tall: of the larger)
    const int64_t pp = at.param_pitch * kPSize, op = at.out_pitch * 4;
    const uint32_t across = TALL ? T * j : V * j;
    const uint32_t param_lane = 4 * h * static_cast<uint32_t>(pp) + across * kPSize;
    const uint32_t out_lane = 4 * h * static_cast<uint32_t>(op) + across * 4;
    for (; x0 < end; x0 += kStride) {
        floatx16 acc[V][T];
        times_poly<TALL>(acc, in, poly, lane, x0 + kStride, end);
        // `run` elements side by side of row 8 q + 4 h + b of the tiles
        constexpr int N = TALL ? T : V;
        auto store = [&](const Row &row, int b, const float (&o)[N], bool whole, int there) {
            char *param = row.param + b * pp, *out = row.out ? row.out + b * op : nullptr;
            if (whole) {
                update_run<PBF16, N>(param, out, param_lane, out_lane, o, c.decay, k.update);
            } else {
#pragma unroll
                for (int e = 0; e < N; ++e) {
                    const float one[1] = {o[e]};
                    if (e < there) update_run<PBF16, 1>(param, out, param_lane + e * kPSize, out_lane + e * 4, one, c.decay, k.update);
                }
            }
        };
        if constexpr (TALL) {
            Row row{at.param + x0 * pp, at.out ? reinterpret_cast<char *>(at.out) + x0 * op : nullptr};
            const bool whole = c.s % T == 0;
#pragma unroll
            for (int q = 0; q < 4; ++q) {
#pragma unroll
                for (int b = 0; b < 4; ++b) {
                    if (x0 + 8 * q + 4 * h + b >= end || T * j >= c.s) continue;
                    float o[T];
#pragma unroll
                    for (int i = 0; i < T; ++i) o[i] = acc[0][i][4 * q + b] * scale;
                    store(row, b, o, whole, c.s - T * j);
                }
                row.param += 8 * pp;
                row.out = row.out ? row.out + 8 * op : nullptr;
                row.keep();
            }
        } else {
            Row row{at.param + x0 * kPSize, at.out ? reinterpret_cast<char *>(at.out + x0) : nullptr};
            const bool whole = x0 + 32 * V <= end;
            int left = c.s;  // rows from `row` to the block's end
#pragma unroll
            for (int i = 0; i < T; ++i)
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    if (left <= 0) continue;
#pragma unroll
                    for (int b = 0; b < 4; ++b) {
                        if (4 * h + b >= left) continue;
                        float o[V];
#pragma unroll
                        for (int v = 0; v < V; ++v) o[v] = acc[v][i][4 * q + b] * scale;
                        store(row, b, o, whole, end - x0 - V * j);
                    }
                    row.param += 8 * pp;
                    row.out = row.out ? row.out + 8 * op : nullptr;
                    row.keep();
                    left -= 8;
                    asm volatile("" : "+s"(left));
                }
        }
    }
}

}  // namespace

hipError_t launch_blocks_regram(const BlockTable &t, const BlockCall &c, uint32_t blocks, bool tall, bool grad_bf16,
                                hipStream_t st) {
    return choose(c.s, tall, grad_bf16, [&](auto tiles, auto is_tall, auto bf16, auto even) {
        hipLaunchKernelGGL((blocks_regram_kernel<tiles.value, is_tall.value, bf16.value, even.value>), dim3(blocks * c.parts),
                           dim3(kThreads), 0, st, t, c);
        return hipGetLastError();
    });
}

hipError_t launch_blocks_update(const BlockTable &t, const BlockCall &c, uint32_t blocks, bool tall, bool grad_bf16,
                                bool param_bf16, hipStream_t st) {
    return choose(c.s, tall, grad_bf16, [&](auto tiles, auto is_tall, auto bf16, auto even) {
        if (param_bf16)
            hipLaunchKernelGGL((blocks_update_kernel<tiles.value, is_tall.value, bf16.value, true, even.value>),
                               dim3(blocks * c.parts), dim3(kThreads), 0, st, t, c);
        else
            hipLaunchKernelGGL((blocks_update_kernel<tiles.value, is_tall.value, bf16.value, false, even.value>),
                               dim3(blocks * c.parts), dim3(kThreads), 0, st, t, c);
        return hipGetLastError();
    });
}

}  // namespace muon
