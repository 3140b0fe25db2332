// The passes of the block step that multiply N by P (blocks.hpp).
//
// A wave holds P's rows as fragments in turn from shared memory, and N's columns
// from M and G, formed and split in registers: nothing between is stored.  1728 heads
// of 128 x 2048, bf16: X X^T 0.74 ms, 3.7 TB/s of 6 bytes read an element; update 1.06 ms,
// 4.3 TB/s of 10 (a copy: 4.9).  The update is bound by memory (matrix cores 14%, vector
// units 21% busy).  X X^T is not: its sums and P N leave room for one wave a SIMD, in
// which loads, splits (23%) and products (31%: 3 x 2 s 16-bit operations an element for
// P N, 3 s for X X^T) follow one another.  V = 2 columns a lane halves the accesses; V = 4
// spills.
#include "blocks_device.hpp"

namespace muon {

namespace {

// ------------------------------------------------------------ products with N

// M and G of 32 V columns of X as a wave loads them, and N from them.  A lane
// holds column j (wide blocks: columns V j .. V j + V - 1, in one access) and, of
// the smaller side, for chunk (t, q) basis indices 32 t + 16 q + 8 a + 4 h + b,
// a < 2, b < 4.  They come in phases: in wide blocks each chunk is one, eight rows
// that lanes read side by side; in tall ones the T chunks of one q, as two runs of
// 4 T elements that lie side by side in the lane's row of memory.  The registers
// hold kSlots phases; one is loaded anew, for the phase kSlots further on, as soon
// as it is used up, so that a wave always has loads on their way.
//
// Places outside of the block are read as others inside of it: what the products
// make of them meets P's zeros (its rows and columns past the smaller side) or
// belongs to columns that nobody stores or sums.  V > 1: all columns are inside.
// EVEN: a tall block's runs lie inside or outside as a whole (4 T divides its
// smaller side).
template <int T, int V, bool TALL, bool BF16, bool EVEN> struct Stream {
    static_assert(!TALL || V == 1, "a tall block's lane holds one column");
    static constexpr int kPhases = TALL ? 2 : 2 * T, kChunks = TALL ? T : 1;
    static constexpr int kSlots = V > 1 ? 2 : kPhases;
    static constexpr int kValues = 8 * kChunks * V;              // of a phase
    static constexpr int kGrads = BF16 && (TALL || V > 1) ? kValues / 2 : kValues;  // words of G
    static constexpr int kGSize = BF16 ? 2 : 4;
    static_assert(kPhases % kSlots == 0, "a phase has the same slot in every unit");
    typedef const char *Bytes;
    float m[kSlots][kValues];
    uint32_t g[kSlots][kGrads];
    const Place &at;
    const BlockCall &c;
    int j, h;
    float from_mom, from_grad;  // N 2^shift = from_mom M + from_grad G
    int left_shift = 0;         // what they could not hold of the shift
    // wide: where the next group of eight rows begins, how many rows lie from there
    // to the block's end, and the bytes from there to the lane's row 4 h + b and column
    Bytes mom_row = nullptr, grad_row = nullptr;
    int left = 0;
    uint32_t mom_lane[4] = {}, grad_lane[4] = {};
    int64_t mom_at = 0, grad_at = 0;  // tall: the lane's row of memory

    __device__ __forceinline__ Stream(const Place &place, const BlockCall &call, float factor, int lane, int shift)
        : at(place), c(call), j(lane & 31), h(lane >> 5) {
        // O and X need no more of N than 2^-24: scale and momentum go into one
        // factor each.  Beyond 2^100 (an N near fp32's ends) the rest is applied behind.
        const int held = min(max(shift, -100), 100);
        left_shift = shift - held;
        const float scale = __builtin_amdgcn_ldexpf(1.0f, held);
        from_mom = (c.nesterov ? c.mu : 1.0f) * scale;
        from_grad = c.nesterov ? factor * scale : 0.0f;
        if constexpr (!TALL && V > 1) lanes(V * j, 8);
    }
    // Before the phases of columns x0 ..; `end`: the first column that is not there.
    __device__ __forceinline__ void begin(int x0, int end) {
        if constexpr (TALL) {
            const int64_t row = min(x0 + j, end - 1);
            mom_at = row * at.mom_pitch;
            grad_at = row * at.grad_pitch;
        } else {
            if (V == 1 || c.s % 8 != 0) lanes(V > 1 ? V * j : min(j, end - 1 - x0), min(c.s, 8));
            mom_row = reinterpret_cast<Bytes>(at.mom + x0);
            grad_row = at.grad + static_cast<int64_t>(x0) * kGSize;
            left = c.s;
        }
    }
    // Columns x0 .. and their first kSlots phases.
    __device__ __forceinline__ void start(int x0, int end) {
        begin(x0, end);
#pragma unroll
        for (int ph = 0; ph < kSlots; ++ph) load(ph);
    }
    // Behind the use of phase ph of a unit: what takes its place, `next` being the next unit.
    __device__ __forceinline__ void refill(int ph, int next, int end) {
        if (ph + kSlots < kPhases) {
            load(ph);
        } else if (next < end) {
            if (ph + kSlots == kPhases) begin(next, end);
            load(ph);
        }
    }
    // N 2^shift of chunk `sub` of a phase, column v, as fp16 pairs.
    __device__ __forceinline__ void fragment(int ph, int sub, int v, half8 &hi, half8 &lo) const {
        float x[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const int i = TALL ? ((e >> 2) * 4 + (e & 3)) * T + sub : e * V + v;
            x[e] = __builtin_fmaf(from_mom, m[ph % kSlots][i], from_grad * grad_value(ph % kSlots, i));
        }
        if (left_shift != 0) {
#pragma unroll
            for (int e = 0; e < 8; ++e) x[e] = __builtin_amdgcn_ldexpf(x[e], left_shift);
        }
        split_half<false>(x, hi, lo);
    }

  private:
    // The lane's places in a group of which `rows` rows are there, others read as the last of these.
    __device__ __forceinline__ void lanes(uint32_t col, int rows) {
        const uint32_t mp = static_cast<uint32_t>(at.mom_pitch), gp = static_cast<uint32_t>(at.grad_pitch);
#pragma unroll
        for (int b = 0; b < 4; ++b) {
            const uint32_t row = min(4 * h + b, rows - 1);
            mom_lane[b] = (row * mp + col) * 4;
            grad_lane[b] = (row * gp + col) * kGSize;
        }
    }
    // The next phase of the columns begun, into the slot of `ph`.
    __device__ __forceinline__ void load(int ph) {
        const int k = ph % kSlots;
        if constexpr (TALL) {
#pragma unroll
            for (int a = 0; a < 2; ++a) {
                const int run = T * (16 * ph + 8 * a + 4 * h);
                if constexpr (EVEN) {
                    const int p = run < c.s ? run : 0;
                    words<4 * T, 4>(at.mom + mom_at + p, reinterpret_cast<uint32_t *>(&m[k][a * 4 * T]));
                    words<(BF16 ? 2 : 4) * T, kGSize>(at.grad + (grad_at + p) * kGSize, &g[k][a * (BF16 ? 2 : 4) * T]);
                } else {
                    checked(k, a, run);
                }
            }
        } else {
#pragma unroll
            for (int a = 0; a < 2; ++a) {
                const Bytes mp = mom_row, gp = grad_row;
#pragma unroll
                for (int b = 0; b < 4; ++b) {
                    const int e = 4 * a + b;
                    if constexpr (V == 1) {
                        m[k][e] = load_at<float>(mp, mom_lane[b]);
                        g[k][e] = BF16 ? static_cast<uint32_t>(load_at<uint16_t>(gp, grad_lane[b])) : load_at<uint32_t>(gp, grad_lane[b]);
                    } else {
                        const auto v = load_at<typename WordsAt<V, 4>::type>(mp, mom_lane[b]);
                        const auto u = load_at<typename WordsAt<BF16 ? V / 2 : V, kGSize>::type>(gp, grad_lane[b]);
#pragma unroll
                        for (int i = 0; i < V; ++i) m[k][V * e + i] = __uint_as_float(v[i]);
#pragma unroll
                        for (int i = 0; i < (BF16 ? V / 2 : V); ++i) g[k][(BF16 ? V / 2 : V) * e + i] = u[i];
                    }
                }
                if (left > 8) {  // groups past the last one read that one again
                    mom_row += 8 * at.mom_pitch * 4;
                    grad_row += 8 * at.grad_pitch * kGSize;
                    left -= 8;
                    if (left < 8) lanes(mom_lane[0] / 4 - 4 * h * static_cast<uint32_t>(at.mom_pitch), left);
                }
                // the compiler would form every row's address ahead of the loop, and spill them
                asm volatile("" : "+s"(mom_row), "+s"(grad_row), "+s"(left));
            }
        }
    }
    __device__ __forceinline__ float grad_value(int k, int i) const {
        if constexpr (!BF16) return __uint_as_float(g[k][i]);
        if constexpr (kGrads == kValues) return __uint_as_float(g[k][i] << 16);
        return __uint_as_float(i % 2 ? g[k][i / 2] & 0xffff0000u : g[k][i / 2] << 16);
    }
    // Tall: a run that the smaller side's end may cut.
    __device__ __forceinline__ void checked(int k, int a, int p) {
#pragma unroll
        for (int i = 0; i < 4 * T; ++i) {
            const int from = min(p + i, c.s - 1);
            m[k][a * 4 * T + i] = as_global(at.mom)[mom_at + from];
            if constexpr (BF16) {
                const uint32_t v = as_global(reinterpret_cast<const uint16_t *>(at.grad))[grad_at + from];
                uint32_t &w = g[k][a * 2 * T + i / 2];
                w = i % 2 ? w | v << 16 : v;
            } else {
                g[k][a * 4 * T + i] = as_global(reinterpret_cast<const uint32_t *>(at.grad))[grad_at + from];
            }
        }
    }
    template <int N, int A> __device__ __forceinline__ static void words(const void *p, uint32_t *to) {
        constexpr int W = N % 4 == 0 ? 4 : 2;
#pragma unroll
        for (int i = 0; i < N; i += W) {
            const auto v = ((const typename WordsAt<W, A>::type __attribute__((address_space(1))) *)p)[i / W];
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
            if (sub + 1 == S::kChunks) in.refill(ph, next, end);
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

// Columns x0, x0 + stride, ... below `end` of a wave: the sum of X X^T, X = P N 2^shift
// (the chain scales P so that its entries suit fp16).
template <int T, int V, bool TALL, bool BF16, bool EVEN>
__device__ __forceinline__ void regram_columns(Triangle<T> &sum, Stream<T, V, TALL, BF16, EVEN> &in, const Poly<T> &poly, int lane,
                                               int x0, int stride, int end) {
    for (; x0 < end; x0 += stride) {
        floatx16 acc[V][T];
        times_poly<true>(acc, in, poly, lane, x0 + stride, end);
        if (V == 1 && x0 + 32 > end) {  // columns that are not there
#pragma unroll
            for (int i = 0; i < T; ++i)
#pragma unroll
                for (int r = 0; r < 16; ++r) acc[0][i][r] = x0 + acc_row(r, lane >> 5) < end ? acc[0][i][r] : 0.0f;
        }
#pragma unroll
        for (int v = 0; v < V; ++v)
#pragma unroll
            for (int q = 0; q < 2; ++q) {
                half8 hi[T], lo[T];
#pragma unroll
                for (int i = 0; i < T; ++i) {
                    float x[8];
#pragma unroll
                    for (int e = 0; e < 8; ++e) x[e] = acc[v][i][8 * q + e];
                    split_half<false>(x, hi[i], lo[i]);
                }
                sum.add(hi, lo);
                __builtin_amdgcn_sched_barrier(0);
            }
    }
}

// One part of one block: the sum of X X^T, X = P N / ||N||, over the part's columns.
template <int T, bool TALL, bool BF16, bool EVEN>
__global__ __launch_bounds__(kThreads) void blocks_regram_kernel(const BlockTable t, const BlockCall c) {
    constexpr int V = TALL ? 1 : 2;
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
    const float factor = c.factor ? *c.factor : 1.0f;
    // whole units for all waves, V columns a lane; then what is left, one a lane
    const int whole = V == 1 ? begin : begin + (end - begin) / (V * kBlockUnit) * (V * kBlockUnit);
    Stream<T, V, TALL, BF16, EVEN> in(at, c, factor, lane, k.shift);
    Triangle<T> sum;
    sum.clear();
    const int x0 = begin + 32 * V * wave, x1 = whole + 32 * wave;
    if (V > 1 && x0 < whole) in.start(x0, whole);
    if (V == 1 && x1 < end) in.start(x1, end);
    sh.poly.load(c.w.poly + static_cast<int64_t>(block) * (T * T * 2048));
    __syncthreads();
    if constexpr (V > 1) {
        regram_columns(sum, in, sh.poly, lane, x0, V * kBlockUnit, whole);
        if (x1 < end) {
            Stream<T, 1, TALL, BF16, EVEN> rest(at, c, factor, lane, k.shift);
            rest.start(x1, end);
            regram_columns(sum, rest, sh.poly, lane, x1, kBlockUnit, end);
        }
    } else {
        regram_columns(sum, in, sh.poly, lane, x1, kBlockUnit, end);
    }
    __syncthreads();
    sum.reduce(c.w.gram + (static_cast<int64_t>(block) * c.parts + part) * tri(T) * 1024, sh.sums);
}

// Up to N elements of W side by side, as they lie in memory; `there` of them are.
template <bool PBF16, int N> struct Run {
    static constexpr int kWords = PBF16 ? (N + 1) / 2 : N;
    uint32_t w[kWords];
    typedef char __attribute__((address_space(1))) *Address;

    __device__ __forceinline__ void load(const char *row, uint32_t lane, bool whole, int there) {
        const Address p = (Address) const_cast<char *>(row) + lane;
        if (whole) {
            if constexpr (PBF16 && N % 2 == 0) {
                typedef uint32_t type __attribute__((ext_vector_type(kWords), aligned(2)));
                const type v = *(const type __attribute__((address_space(1))) *)p;
#pragma unroll
                for (int k = 0; k < kWords; ++k) w[k] = v[k];
            } else if constexpr (!PBF16 && N % 2 == 0) {
                typedef uint32_t type __attribute__((ext_vector_type(N), aligned(4)));
                const type v = *(const type __attribute__((address_space(1))) *)p;
#pragma unroll
                for (int k = 0; k < kWords; ++k) w[k] = v[k];
            } else {
                single(p, N);
            }
        } else {
            single(p, there);
        }
    }
    // W <- fl(fl(d W) - fl(s o)), and o to `out` unless it is null.
    __device__ __forceinline__ void update(char *row, uint32_t lane, char *out, uint32_t out_lane, bool whole, int there,
                                           const float (&o)[N], float d, float s) {
        const Address p = (Address)row + lane;
        float x[N];
#pragma unroll
        for (int e = 0; e < N; ++e) {
            const float old = !PBF16 ? __uint_as_float(w[e]) : __uint_as_float(e % 2 ? w[e / 2] & 0xffff0000u : w[e / 2] << 16);
            x[e] = d * old - s * o[e];
        }
        if (whole && N % 2 == 0) {
            if constexpr (PBF16 && N % 2 == 0) {
                typedef uint32_t type __attribute__((ext_vector_type(kWords), aligned(2)));
                type v;
#pragma unroll
                for (int k = 0; k < kWords; ++k) v[k] = pack_bf16x2(x[2 * k], x[2 * k + 1]);
                *(type __attribute__((address_space(1))) *)p = v;
            } else if constexpr (N % 2 == 0) {
                typedef float type __attribute__((ext_vector_type(N), aligned(4)));
                type v;
#pragma unroll
                for (int k = 0; k < N; ++k) v[k] = x[k];
                *(type __attribute__((address_space(1))) *)p = v;
            }
        } else {
#pragma unroll
            for (int e = 0; e < N; ++e) {
                if (!whole && e >= there) continue;
                if constexpr (PBF16)
                    ((uint16_t __attribute__((address_space(1))) *)p)[e] = float_to_bf16_bits(x[e]);
                else
                    ((float __attribute__((address_space(1))) *)p)[e] = x[e];
            }
        }
        if (out) {
            const Address q = (Address)out + out_lane;
#pragma unroll
            for (int e = 0; e < N; ++e)
                if (whole || e < there) ((float __attribute__((address_space(1))) *)q)[e] = o[e];
        }
    }

  private:
    __device__ __forceinline__ void single(Address p, int there) {
#pragma unroll
        for (int e = 0; e < N; ++e) {
            const bool in = e < there;
            if constexpr (PBF16) {
                const uint32_t v = in ? ((const uint16_t __attribute__((address_space(1))) *)p)[e] : 0;
                w[e / 2] = e % 2 ? w[e / 2] | v << 16 : v;
            } else {
                w[e] = in ? ((const uint32_t __attribute__((address_space(1))) *)p)[e] : 0;
            }
        }
    }
};

// What the last pass needs beside a Stream.
struct Update {
    const Place &at;
    const BlockCall &c;
    float scale, update;
};

// Columns x0, x0 + stride, ... below `end` of a wave: O = P N 2^shift scale, and W.
// W is read before the products, so that it is there behind them.
template <int T, int V, bool TALL, bool BF16, bool PBF16, bool EVEN>
__device__ __forceinline__ void update_columns(Stream<T, V, TALL, BF16, EVEN> &in, const Update &u, const Poly<T> &poly, int lane,
                                               int x0, int stride, int end) {
    constexpr int kPSize = PBF16 ? 2 : 4;
    constexpr int N = TALL ? T : V;    // elements side by side
    constexpr int kTiles = TALL ? 1 : T;  // of 32 rows of memory
    const int j = lane & 31, h = lane >> 5;
    const Place &at = u.at;
    // the lane's place behind the begin of the first of eight rows
    const int64_t pp = at.param_pitch * kPSize, op = at.out_pitch * 4;
    const uint32_t across = N * j;
    uint32_t param_lane[4], out_lane[4];
#pragma unroll
    for (int b = 0; b < 4; ++b) {
        param_lane[b] = (4 * h + b) * static_cast<uint32_t>(pp) + across * kPSize;
        out_lane[b] = (4 * h + b) * static_cast<uint32_t>(op) + across * 4;
    }
    for (; x0 < end; x0 += stride) {
        // rows of memory from the first one to the end, and elements of a row from the lane's on
        const int rows = TALL ? end - x0 : u.c.s, there = (TALL ? u.c.s : end - x0) - static_cast<int>(across);
        const bool whole = TALL ? u.c.s % T == 0 : V > 1 || x0 + 32 <= end;
        char *row = at.param + (TALL ? x0 * pp : static_cast<int64_t>(x0) * kPSize);
        const char *ahead = row;
        char *out = at.out ? reinterpret_cast<char *>(at.out) + (TALL ? x0 * op : static_cast<int64_t>(x0) * 4) : nullptr;
        int left = rows, ahead_left = rows;
        Run<PBF16, N> w[kTiles][4][4];
#pragma unroll
        for (int tile = 0; tile < kTiles; ++tile)
#pragma unroll
            for (int q = 0; q < 4; ++q) {
#pragma unroll
                for (int b = 0; b < 4; ++b)
                    if (4 * h + b < ahead_left && there > 0) w[tile][q][b].load(ahead, param_lane[b], whole, there);
                ahead += 8 * pp;
                ahead_left -= 8;
                asm volatile("" : "+s"(ahead), "+s"(ahead_left));
            }
        floatx16 acc[V][T];
        times_poly<TALL>(acc, in, poly, lane, x0 + stride, end);
#pragma unroll
        for (int tile = 0; tile < kTiles; ++tile) {
#pragma unroll
            for (int q = 0; q < 4; ++q) {
#pragma unroll
                for (int b = 0; b < 4; ++b) {
                    float o[N];
#pragma unroll
                    for (int e = 0; e < N; ++e) o[e] = (TALL ? acc[0][e][4 * q + b] : acc[e][tile][4 * q + b]) * u.scale;
                    if (4 * h + b < left && there > 0)
                        w[tile][q][b].update(row, param_lane[b], out, out_lane[b], whole, there, o,
                                                 u.c.decay, u.update);
                }
                row += 8 * pp;
                out = out ? out + 8 * op : nullptr;
                left -= 8;
                asm volatile("" : "+s"(row), "+s"(out), "+s"(left));
            }
            __builtin_amdgcn_sched_barrier(0);
        }
    }
}

// The last pass: O = P N / ||N|| and W of one part of one block.
template <int T, bool TALL, bool BF16, bool PBF16, bool EVEN>
__global__ __launch_bounds__(kThreads) void blocks_update_kernel(const BlockTable t, const BlockCall c) {
    // two columns a lane, 8 and 4 bytes of fp32 and bf16 data, where the part is
    // long enough for whole units of all waves
    constexpr int V = TALL ? 1 : 2;
    __shared__ __attribute__((aligned(16))) Poly<T> poly;
    const uint32_t block = blockIdx.x / c.parts, part = blockIdx.x % c.parts;  // block: of the launch
    const Place at = locate<BF16 ? 2 : 4, PBF16 ? 2 : 4>(t, c, c.base + block);
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63;
    const int begin = part * c.part_len, end = min(begin + c.part_len, c.l);
    const BlockScalars k = c.w.scalars[block];
    const float factor = c.factor ? *c.factor : 1.0f;
    const Update u{at, c, __builtin_amdgcn_ldexpf(k.inv_norm, k.poly), k.update};
    const int whole = V == 1 ? begin : begin + (end - begin) / (V * kBlockUnit) * (V * kBlockUnit);
    Stream<T, V, TALL, BF16, EVEN> in(at, c, factor, lane, k.shift);
    const int x0 = begin + 32 * V * wave, x1 = whole + 32 * wave;
    if (V > 1 && x0 < whole) in.start(x0, whole);
    if (V == 1 && x1 < end) in.start(x1, end);
    poly.load(c.w.poly + static_cast<int64_t>(block) * (T * T * 2048));
    __syncthreads();
    if constexpr (V > 1) {
        update_columns<T, V, TALL, BF16, PBF16, EVEN>(in, u, poly, lane, x0, V * kBlockUnit, whole);
        if (x1 < end) {
            Stream<T, 1, TALL, BF16, EVEN> rest(at, c, factor, lane, k.shift);
            rest.start(x1, end);
            update_columns<T, 1, TALL, BF16, PBF16, EVEN>(rest, u, poly, lane, x1, kBlockUnit, end);
        }
    } else {
        update_columns<T, 1, TALL, BF16, PBF16, EVEN>(in, u, poly, lane, x1, kBlockUnit, end);
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
