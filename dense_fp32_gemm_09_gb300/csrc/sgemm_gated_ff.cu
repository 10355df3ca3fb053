// The gated feed-forward block (sgemm_gated_ff_forward, sgemm_gated_ff_backward).
//
//     g = x Wg^T    u = x Wu^T    h = act(g) u            (M x N, from fp32 sums)
//
// Backward, from the kept g and u (in the type of x, or in 8 bits):
//     du = dh act(g)     dg = dh u act'(g)                 element by element, to the workspace
//     dx = dg Wg + du Wu      dWg = dg^T x      dWu = du^T x
// dg and du are rounded to the type of x, the tensor cores' operand type, so that a gradient
// is off by the rounding of its terms (half an ulp each, at random) beside its own: in norm, bf16,
// 2.3e-3 of 64 bits' where the rounding of the result alone is 1.7e-3.  The numbers of an x that comes in
// 8 bits are code times scale, of more bits than the type has: the products take the rounding and the
// rounding of what is left, as two halves of one contraction (the rounding alone: 2.8e-3).  fp16 has too few
// exponents for dg and du and takes them by powers of two for each row and column (ff_gradient_fp16).
//
// The products: sgemm_ff_pair.cuh, and sgemm_ff_token.cu for up to 16 tokens.  Rows that are not on
// 16 bytes cannot be read by tensor maps and, for these, are copied into the workspace first (3001 x 2047 and
// 1999 x 2047 twice: 10 us beside a product of 34).
//
// Measured (us, kernels alone): forward 8192 x 4096 x 8192 bf16 527 to 550 (2.0 to 2.1 PFLOP/s; the
// measured rate of a library product is 1.9, sustained 1.7), with g and u kept in 8 bits 546; the
// gradient 1223 to 1275, of it 122 for ff_gradient (0.8 of the memory), from an x in 8 bits 1984.
// 500 x 1024 x 4096 12.1 and 25.7, from 8 bits 30.8; 16384 x 256 x 64 backward 16.2.
#include <cuda_runtime.h>

#include <algorithm>

#include "sgemm_ff_plan.h"
#include "sgemm_gated_ff.cuh"
#include "sgemm_launch.cuh"
#include "sgemm_tma_host.h"

namespace sgemm {
namespace {

using namespace ff;

constexpr int kThreads = 256;

// Eight 2-byte numbers at p as they are stored, zeros for those from the n-th on; vec: p is on 16 bytes.
template <typename T>
__device__ __forceinline__ uint4 load8(const T* p, int n, bool vec) {
    if (vec && n >= 8) return fetch_here(reinterpret_cast<const uint4*>(p));
    alignas(16) T t[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) t[i] = i < n ? fetch_here(p + i) : T(0.0f);
    return *reinterpret_cast<const uint4*>(t);
}
template <typename T>
__device__ __forceinline__ void numbers8(const uint4& raw, float (&v)[8]) {
    const T* t = reinterpret_cast<const T*>(&raw);
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = to_float(t[i]);
}
template <typename T>
__device__ __forceinline__ void store8(T* p, int n, bool vec, const float (&v)[8]) {
    if (vec && n >= 8) {
        alignas(16) T t[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) t[i] = from_float<T>(v[i]);
        *reinterpret_cast<uint4*>(p) = *reinterpret_cast<const uint4*>(t);
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (i < n) p[i] = from_float<T>(v[i]);
    }
}

struct Aligned {
    bool dh, kept, h;
};
// What dg, du and h again are made of: dh and what was kept of eight columns of a row from c on, of which n > 0
// are inside (the others are 0).  All loads come before the first number is used.
template <typename T, bool KEPT8>
struct Inputs8 {
    uint4 dh, gate, up;              // KEPT8: eight codes, and the scale's bits
    __device__ __forceinline__ void load(const GatedFfBackward& p, long long row, int c, int n, const Aligned& on) {
        dh = load8(static_cast<const T*>(p.dh) + row * p.lddh + c, n, on.dh);
        if constexpr (KEPT8) {
            const long long k = row * act8_pitch(p.N) + c;
            const auto held = [&](const void* from, const float* scales) {
                const uint2 w = fetch_here(reinterpret_cast<const uint2*>(static_cast<const int8_t*>(from) + k));
                return make_uint4(w.x, w.y, __float_as_uint(fetch_here(scales + k / kAct8Block)), 0);
            };
            gate = held(p.kept.gate, p.kept.gate_scales);
            up = held(p.kept.up, p.kept.up_scales);
        } else {
            gate = load8(static_cast<const T*>(p.kept.gate) + row * p.kept.ld + c, n, on.kept);
            up = load8(static_cast<const T*>(p.kept.up) + row * p.kept.ld + c, n, on.kept);
        }
    }
    __device__ __forceinline__ static void kept(const uint4& raw, float (&v)[8]) {
        if constexpr (KEPT8) {
            const float s = __uint_as_float(raw.z);
            mx4::Two t[4];
            act8::values4(raw.x, s, reinterpret_cast<mx4::Two(&)[2]>(t[0]));
            act8::values4(raw.y, s, reinterpret_cast<mx4::Two(&)[2]>(t[2]));
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const float2 f = mx4::parts(t[j]);
                v[2 * j] = f.x;
                v[2 * j + 1] = f.y;
            }
        } else {
            numbers8<T>(raw, v);
        }
    }
    template <int ACT>
    __device__ __forceinline__ void gradients(float (&dg)[8], float (&du)[8], float (&h)[8]) const {
        float (&g)[8] = dg, (&u)[8] = du, d[8];
        numbers8<T>(dh, d);
        kept(gate, g);
        kept(up, u);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const Act a = Act::of<ACT>(g[j]);
            const float v = a.value();
            h[j] = v * u[j];
            g[j] = d[j] * u[j] * a.slope();
            u[j] = d[j] * v;
        }
    }
};
// bf16: dg, du (rows of `pitch`, a multiple of 64), and h again, from dh and what was kept: eight columns
// a thread.
template <typename T, int ACT, bool KEPT8>
__global__ void __launch_bounds__(kThreads)
    ff_gradient(const GatedFfBackward p, T* dg, T* du, long long pitch, const Aligned on) {
    act8::Walk at(blockIdx.x * static_cast<long long>(kThreads) + threadIdx.x,
                  static_cast<long long>(gridDim.x) * kThreads, (p.N + 7) / 8);
    start_dependent();
    for (; at.row < p.M; at.next()) {
        const long long row = at.row;
        const int c = at.col * 8, n = p.N - c;
        float g[8], u[8], h[8];
        Inputs8<T, KEPT8> in;
        in.load(p, row, c, n, on);
        in.template gradients<ACT>(g, u, h);
        store8(dg + row * pitch + c, 8, true, g);
        store8(du + row * pitch + c, 8, true, u);
        if (p.h) store8(static_cast<T*>(p.h) + row * p.ldh + c, n, on.h, h);
    }
}

// fp16: the same in two passes (scale_up in sgemm_gated_ff.cuh).  The first finds the largest finite
// magnitudes of each row and column; maxima do not depend on the order of the atomics.  The second
// makes dg and du again and stores them twice, by the rows' powers of two for dx and by the columns'
// for the weights' gradients.  (One power for the whole matrix would need no second copy, but one large
// token would take the precision of all others.)  A block has 256 columns, a warp a row of them at a
// time, so that a thread's columns stay and so do their maxima and powers.  Against one unscaled copy in one
// pass the gradient of 500 x 4096 x 1024 (tokens x outputs x inputs) takes 35.4 us and took 26.0, of
// 8192 x 8192 x 4096 1485 and 1373 (96 of it the first pass).
struct Scaled {
    __half *dg_rows, *du_rows, *dg_cols, *du_cols;     // rows of `pitch`
    uint32_t *rows, *of_dg, *of_du;                    // fp32 bits: [M], [N], [N]
    long long pitch;
};
constexpr int kTileCols = 256, kRowsAhead = 2;
__global__ void __launch_bounds__(kThreads) ff_clear(uint32_t* p, long long n) {
    start_dependent();
    for (long long i = blockIdx.x * static_cast<long long>(kThreads) + threadIdx.x; i < n;
         i += static_cast<long long>(gridDim.x) * kThreads)
        p[i] = 0;
}
__device__ __forceinline__ uint32_t finite_magnitude(float v) {
    const uint32_t m = act8::magnitude(v);
    return m < kInfinite ? m : 0u;
}
template <int ACT, bool KEPT8, bool STORE>
__global__ void __launch_bounds__(kThreads)
    ff_gradient_fp16(const GatedFfBackward p, const Scaled q, const Aligned on) {
    constexpr int kWarps = kThreads / 32;
    __shared__ uint32_t part[STORE ? 1 : kWarps][2][STORE ? 1 : kTileCols];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int first = blockIdx.x * kTileCols, c = first + 8 * lane, n = p.N - c;
    start_dependent();
    uint32_t mg[8] = {}, mu[8] = {};                   // STORE: unused
    float fg[8], fu[8];
    if constexpr (STORE)
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            fg[j] = j < n ? scale_up(fetch_here(q.of_dg + c + j)) : 0.0f;
            fu[j] = j < n ? scale_up(fetch_here(q.of_du + c + j)) : 0.0f;
        }
    const long long step = static_cast<long long>(gridDim.y) * kWarps;
    for (long long first_row = blockIdx.y * static_cast<long long>(kWarps) + warp; first_row < p.M;
         first_row += kRowsAhead * step) {
        Inputs8<__half, KEPT8> in[kRowsAhead] = {};
#pragma unroll
        for (int i = 0; i < kRowsAhead; ++i)
            if (n > 0 && first_row + i * step < p.M) in[i].load(p, first_row + i * step, c, n, on);
#pragma unroll
        for (int i = 0; i < kRowsAhead; ++i) {
            const long long row = first_row + i * step;
            if (row >= p.M) break;
            float g[8], u[8], h[8];
            in[i].template gradients<ACT>(g, u, h);
            if constexpr (STORE) {
                if (n <= 0) continue;
                const float by = scale_up(fetch_here(q.rows + row));
                const long long to = row * q.pitch + c;
                float v[8];
                const auto put = [&](__half* at, const float (&x)[8], auto factor) {
#pragma unroll
                    for (int j = 0; j < 8; ++j) v[j] = x[j] * factor(j);
                    store8(at + to, 8, true, v);
                };
                put(q.dg_rows, g, [&](int) { return by; });
                put(q.du_rows, u, [&](int) { return by; });
                put(q.dg_cols, g, [&](int j) { return fg[j]; });
                put(q.du_cols, u, [&](int j) { return fu[j]; });
                if (p.h) store8(static_cast<__half*>(p.h) + row * p.ldh + c, n, on.h, h);
            } else {
                uint32_t most = 0;
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    const uint32_t a = finite_magnitude(g[j]), b = finite_magnitude(u[j]);
                    mg[j] = max(mg[j], a);
                    mu[j] = max(mu[j], b);
                    most = max(most, max(a, b));
                }
                most = __reduce_max_sync(0xFFFFFFFFu, most);
                if (lane == 0 && most) atomicMax(q.rows + row, most);
            }
        }
    }
    if constexpr (!STORE) {
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            part[warp][0][8 * lane + j] = mg[j];
            part[warp][1][8 * lane + j] = mu[j];
        }
        __syncthreads();
        for (int i = threadIdx.x; i < 2 * kTileCols; i += kThreads) {
            const int which = i / kTileCols, col = i % kTileCols;
            uint32_t most = 0;
#pragma unroll
            for (int w = 0; w < kWarps; ++w) most = max(most, part[w][which][col]);
            if (most && first + col < p.N) atomicMax((which ? q.of_du : q.of_dg) + first + col, most);
        }
    }
}

// Matrices of 2-byte numbers into rows of `pitch`, a warp a row; blockIdx.y: which.
struct Copies {
    const uint16_t* from[3];
    uint16_t* to[3];
    long long ld[3], rows[3];
    int cols;
    long long pitch;
};
// One row, eight numbers a lane: the row's 16-byte groups of memory, cut at the place where it begins.
// All of the groups are inside the matrix.  (Numbers past the row's end may be written: the copy's
// rows are padded.)
__device__ __forceinline__ void copy_groups(const uint16_t* x, uint16_t* y, int cols) {
    constexpr int kEach = 4;             // of a lane on their way
    const int lane = threadIdx.x & 31, skip = static_cast<int>(reinterpret_cast<uintptr_t>(x) & 15);
    const uint4* const at = reinterpret_cast<const uint4*>(reinterpret_cast<const uint8_t*>(x) - skip);
    // (Counted in numbers: in bytes, rows of 2^30 columns would pass 2^31.)
    const int groups = (skip / 2 + cols + 7) / 8, out = (cols + 7) / 8;
    const auto get = [&](int i) { return i < groups ? fetch_here(at + i) : make_uint4(0, 0, 0, 0); };
    for (int start = lane; start - lane < out; start += 32 * kEach) {
        uint4 own[kEach], last[kEach];   // (lane 31: the next lane's)
#pragma unroll
        for (int j = 0; j < kEach; ++j) {
            own[j] = get(start + 32 * j);
            if (lane == 31) last[j] = get(start + 32 * j + 1);
        }
#pragma unroll
        for (int j = 0; j < kEach; ++j) {
            uint32_t w[8] = {own[j].x, own[j].y, own[j].z, own[j].w};
#pragma unroll
            for (int i = 0; i < 4; ++i) w[4 + i] = __shfl_down_sync(0xFFFFFFFFu, w[i], 1);
            if (lane == 31) w[4] = last[j].x, w[5] = last[j].y, w[6] = last[j].z, w[7] = last[j].w;
#pragma unroll
            for (int i = 0; i < 6; ++i) w[i] = skip & 8 ? w[i + 2] : w[i];
#pragma unroll
            for (int i = 0; i < 5; ++i) w[i] = skip & 4 ? w[i + 1] : w[i];
#pragma unroll
            for (int i = 0; i < 4; ++i) w[i] = __funnelshift_r(w[i], w[i + 1], 8 * (skip & 2));
            if (start + 32 * j < out)
                reinterpret_cast<uint4*>(y)[start + 32 * j] = make_uint4(w[0], w[1], w[2], w[3]);
        }
    }
}
// Rows near the matrix's ends, whose first or last group is partly outside: two numbers a lane.  Rows
// that start between two words are read in whole words all the same, and a word of the copy is
// made of the second number of the lane before and the first of its own.  (All rows so: 3001 x 2047
// x 1999 forward 46.5 us, now 44.4; 100 x 4001 x 4001 52.4 and 47.3.)
__global__ void __launch_bounds__(kThreads) ff_copy_rows(const Copies q) {
    constexpr int kWords = 8;            // of a lane on their way
    const int which = blockIdx.y, lane = threadIdx.x & 31;
    const long long warps = static_cast<long long>(gridDim.x) * (kThreads / 32);
    start_dependent();
    for (long long row = blockIdx.x * (kThreads / 32LL) + threadIdx.x / 32; row < q.rows[which];
         row += warps) {
        const uint16_t* const x = q.from[which] + row * q.ld[which];
        uint16_t* const y = q.to[which] + row * q.pitch;
        // (Seven numbers of a group may lie before the row, and as many after it.)
        if (row * q.ld[which] >= 8 && (q.rows[which] - 1 - row) * q.ld[which] >= 8) {
            copy_groups(x, y, q.cols);
            continue;
        }
        const int off = reinterpret_cast<uintptr_t>(x) & 2 ? 1 : 0;
        for (int start = 0; start < q.cols; start += 64 * kWords) {
            uint32_t w[kWords];
            uint32_t before[kWords];     // (lane 0, off: the number before its word)
#pragma unroll
            for (int j = 0; j < kWords; ++j) {
                const int c = start + 64 * j + 2 * lane + off;     // of the word read
                w[j] = before[j] = 0;
                if (c + 1 < q.cols) w[j] = fetch_here(reinterpret_cast<const uint32_t*>(x + c));
                else if (c < q.cols) w[j] = fetch_here(x + c);
                if (off && lane == 0 && c <= q.cols) before[j] = fetch_here(x + c - 1);
            }
#pragma unroll
            for (int j = 0; j < kWords; ++j) {
                const int c = start + 64 * j + 2 * lane;           // of the word written
                uint32_t v = w[j];
                if (off) {
                    const uint32_t last = __shfl_up_sync(0xFFFFFFFFu, w[j] >> 16, 1);
                    v = (lane == 0 ? before[j] : last) | w[j] << 16;
                }
                if (c < q.cols) *reinterpret_cast<uint32_t*>(y + c) = v;
            }
        }
    }
}

// The parts of split products, added in their order; four columns a thread, blockIdx.y: which of
// the results.
struct Parts {
    struct One {
        const float* partial;        // [part][rows][ld]
        int split, rows;
        void* to;
        long long ldto;
    } of[3];
    long long ld;
    int cols;
};
template <typename T>
__global__ void __launch_bounds__(kThreads) ff_add_parts(const Parts q) {
    const Parts::One& one = q.of[blockIdx.y];
    act8::Walk at(blockIdx.x * static_cast<long long>(kThreads) + threadIdx.x,
                  static_cast<long long>(gridDim.x) * kThreads, (q.cols + 3) / 4);
    start_dependent();
    for (; at.row < one.rows; at.next()) {
        const int c = at.col * 4;
        float4 s = make_float4(0, 0, 0, 0);
#pragma unroll 4
        for (int k = 0; k < one.split; ++k) {
            const float4 v = *reinterpret_cast<const float4*>(
                one.partial + (static_cast<long long>(k) * one.rows + at.row) * q.ld + c);
            s.x += v.x; s.y += v.y; s.z += v.z; s.w += v.w;
        }
        const float v[4] = {s.x, s.y, s.z, s.w};
        T* const to = static_cast<T*>(one.to) + at.row * one.ldto + c;
#pragma unroll
        for (int j = 0; j < 4; ++j)
            if (c + j < q.cols) to[j] = from_float<T>(v[j]);
    }
}

// ----------------------------------------------------------------------------
// Plans
// ----------------------------------------------------------------------------
long long up64(long long n) { return (n + 63) / 64 * 64; }
long long matrix_bytes(long long rows, long long cols) { return rows * up64(cols) * 2; }
long long largest_bytes(long long M, long long N) { return up64(M + 2 * N) * 4; }     // Scaled's
long long up_to(long long n, int m) { return (n + m - 1) / m; }

constexpr int kTokens = 16;          // up to here sgemm_ff_token.cu
constexpr int kPairsOfGpu = 76;      // 152 SMs
// Clocks of a stage: four MMAs of 128 for 256 columns; narrow tiles wait for shared memory.  (Tiles
// of 64 took 8.8 us where 128 took 7.0, 256x4096x1024, and at best 3 % less, 300x300x4096; of 192, 400
// clocks a stage, never the least.)
int stage_clocks(int bn) { return bn == 160 ? 360 : std::max(2 * bn, 320); }

// Rounds of tiles, each as long as its stages.  The model's choice was the fastest of all, or
// within 2 % of it, on 21 shapes from 17 to 12000 tokens.  Tiles of 224 and 160 columns are for h alone:
// they fill the last round better (2048x2048x2048 22.9 us, by 256 24.2; 64x8192x4096 26.5, 30.7; 400x2500x5000
// 30.7, 33.9), but store no whole 128-byte lines, which shows with three results (2000x2048x512,
// gate and up kept: 256 12.8, 224 14.1).  A checkpoint's blocks of 64 are whole in a warp of 256 only.
FfChoice choose_forward(int M, int N, int K, int keep) {
    if (M <= kTokens && keep != kKeep8) return FfChoice{0, 1};
    FfChoice best{256, 1};
    double least = 0;
    for (int bn : {256, 224, 160, 128}) {
        if (bn != 256 && (keep == kKeep8 || (keep != kKeepNone && bn != 128))) continue;
        const long long rounds = up_to(up_to(M, kTileRows) * up_to(N, bn / 2), kPairsOfGpu);
        const double t = static_cast<double>(rounds) * up_to(K, 64) * stage_clocks(bn) + 6.0 * bn;
        if (least == 0 || t < least) best.bn = bn, least = t;
    }
    return best;
}
double item_clocks(long long stages, int bn) { return static_cast<double>(stages) * stage_clocks(bn) + 12.0 * bn; }
// n items of `one` clocks each and m of `two` on `pairs` pairs (Share in sgemm_ff_pair.cuh): how many of
// the second kind pairs with fewer of the first lead by, and how long all take.
struct Spread {
    int extra;
    double clocks;
};
Spread spread(long long n, long long m, double one, double two, long long pairs) {
    const long long more = n % pairs, few = more ? pairs - more : 0;
    const double whole = static_cast<double>(n / pairs) * one;
    Spread best{0, -1.0};
    const long long least = few ? std::min(static_cast<long long>(one / two), m / few) : 0;
    for (long long e = least; e <= least + 1 && e * few <= m; ++e) {
        const long long rounds = (m - e * few) / pairs, left = (m - e * few) % pairs;
        double t = whole + (e + rounds + (left > 0)) * two;
        if (few) t = std::max(t, whole + one + (rounds + (left > few)) * two);
        if (best.clocks < 0 || t < best.clocks) best = {static_cast<int>(e), t};
        if (!few) break;
    }
    return best;
}
// Gradient: one launch for dx and the weights' gradients, so that few tiles of one leave pairs for
// the other.  Few tiles share a contraction between up to sixteen pairs, eight stages each at
// least and no more than two rounds of them; their sums take another pass over the results.
// Measured (us, tokens x outputs x inputs, two launches and one): 500 x 4096 x 1024 28.7, 25.2;
// 1000 x 1024 x 1024 19.0, 13.9; 2000 x 2048 x 512 29.3, 22.0; 8192 x 8192 x 4096 1330, 1249.  Of all
// tiles and parts the model's choice was the fastest, or within 5 % of it, on 21 of 22 shapes
// (one token, 4096 x 4096: 47.0, where four parts of dx and tiles of 256 take 38.6).
struct Gradients {
    int bn, split_x, split_w;
};
// x_parts: 2 for an x in 8 bits.
Gradients choose_gradients(int M, int N, int K, int x_parts) {
    Gradients best{256, 1, 1};
    double least = 0;
    const long long deep_x = 2 * up_to(N, 64), deep_w = x_parts * up_to(M, 64);
    for (int bn : {256, 128}) {
        const long long x = up_to(M, kTileRows) * up_to(K, bn), w = 2 * up_to(N, kTileRows) * up_to(K, bn);
        const auto parts = [](int split, long long tiles, long long stages) {
            return split == 1 || (split <= 16 && stages / split >= 8 && tiles * split <= 2 * kPairsOfGpu);
        };
        for (int i = 1; parts(i, x, deep_x); ++i) {
            for (int j = 1; parts(j, w, deep_w); ++j) {
                double t = spread(x * i, w * j, item_clocks(up_to(deep_x, i), bn),
                                  item_clocks(up_to(deep_w, j), bn), kPairsOfGpu).clocks;
                const double added = (i > 1 ? 1.0 * i * M : 0) + (j > 1 ? 2.0 * j * N : 0);
                if (added > 0) t += 5000 + 8 * added * K / 2500;
                if (least == 0 || t < least) best = {bn, i, j}, least = t;
            }
        }
    }
    return best;
}

// A matrix of 2-byte numbers, boxes of 64 columns by `box` rows, zeros outside.
bool encode(CUtensorMap* tm, const void* base, long long rows, long long cols, long long ld, int box) {
    auto fn = tensor_map_encoder();
    if (!fn) return false;
    cuuint64_t dims[2] = {static_cast<cuuint64_t>(cols), static_cast<cuuint64_t>(rows)};
    // One row has no stride to speak of.
    cuuint64_t strides[1] = {static_cast<cuuint64_t>(rows > 1 ? ld : up64(cols)) * 2};
    cuuint32_t boxes[2] = {64, static_cast<cuuint32_t>(box)};
    cuuint32_t steps[2] = {1, 1};
    return fn(tm, CU_TENSOR_MAP_DATA_TYPE_UINT16, 2, const_cast<void*>(base), dims, strides, boxes,
              steps, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
              CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}
bool rows_on(int bytes, const void* p, long long rows, long long ld) {
    return reinterpret_cast<uintptr_t>(p) % bytes == 0 && (rows <= 1 || ld * 2 % bytes == 0);
}
bool on16(const void* p, long long rows, long long ld) { return rows_on(16, p, rows, ld); }

// What of a call's operands is copied into the workspace first, and where.
struct Operands {
    const void *x, *w_gate, *w_up;
    long long ldx, ldg, ldu;
    Copies copies{};
    int n = 0;
    uint8_t* at;
    Operands(int M, int N, int K, const void* x_, long long ldx_, const void* g, long long ldg_,
             const void* u, long long ldu_, uint8_t* ws)
        : x(x_), w_gate(g), w_up(u), ldx(ldx_), ldg(ldg_), ldu(ldu_), at(ws) {
        copies.cols = K;
        copies.pitch = up64(K);
        if (x) place(x, ldx, M);
        place(w_gate, ldg, N);
        place(w_up, ldu, N);
    }
    void place(const void*& p, long long& ld, long long rows) {
        if (on16(p, rows, ld)) return;
        copies.from[n] = static_cast<const uint16_t*>(p);
        copies.to[n] = reinterpret_cast<uint16_t*>(at);
        copies.ld[n] = ld;
        copies.rows[n++] = rows;
        p = at;
        ld = copies.pitch;
        at += matrix_bytes(rows, copies.cols);
    }
    cudaError_t copy(int sms, cudaStream_t st, int* launches) const {
        if (n == 0) return cudaSuccess;
        const long long most = std::max({copies.rows[0], copies.rows[1], copies.rows[2]});
        const long long blocks = up_to(most, kThreads / 32);
        ++*launches;
        return launch_dependent(ff_copy_rows,
                                dim3(static_cast<unsigned>(std::min<long long>(blocks, sms * 8LL)), n),
                                kThreads, 0, st, copies);
    }
};

template <typename T>
cudaError_t pair(const PairMaps& maps, const PairPlan& pl, int mode, int bn, int act, cudaStream_t st) {
    return std::is_same<T, __half>::value ? pair_f16(maps, pl, mode, bn, act, st)
                                          : pair_bf16(maps, pl, mode, bn, act, st);
}

template <typename T>
cudaError_t forward(const GatedFfForward& p, int sms, cudaStream_t st, int* launches) {
    const FfChoice c = choose_forward(p.M, p.N, p.K, p.kept.keep);
    if (c.bn == 0) {
        const auto all_on = [&](int bytes) {
            return rows_on(bytes, p.x, p.M, p.ldx) && rows_on(bytes, p.w_gate, p.N, p.ldg) &&
                   rows_on(bytes, p.w_up, p.N, p.ldu);
        };
        ++*launches;
        return launch_token(p, all_on(32) ? 32 : all_on(16) ? 16 : 2, sms, st);
    }
    const Operands in(p.M, p.N, p.K, p.x, p.ldx, p.w_gate, p.ldg, p.w_up, p.ldu, p.ws);
    const cudaError_t e = in.copy(sms, st, launches);
    if (e != cudaSuccess) return e;
    PairMaps maps;
    if (!encode(&maps.a[0], in.x, p.M, p.K, in.ldx, 128) ||
        !encode(&maps.b[0], in.w_gate, p.N, p.K, in.ldg, c.bn / 2) ||
        !encode(&maps.b[1], in.w_up, p.N, p.K, in.ldu, c.bn / 2))
        return cudaErrorInvalidValue;
    PairPlan pl{};
    pl.of[0] = {p.M, p.N, static_cast<int>(up_to(p.M, kTileRows)), static_cast<int>(up_to(p.N, c.bn / 2)),
                static_cast<int>(up_to(p.K, 64)), 0, 1};
    pl.pairs = static_cast<int>(std::min<long long>(sms / 2, pl.of[0].items()));
    pl.to[0] = {p.h, p.ldh, on16(p.h, p.M, p.ldh), nullptr, nullptr};
    pl.kept = p.kept;
    pl.kept_vec = on16(p.kept.gate, p.M, p.kept.ld) && on16(p.kept.up, p.M, p.kept.ld);
    pl.status = status_word_ptr();
    ++*launches;
    return pair<T>(maps, pl, kForward, c.bn, p.activation, st);
}

// dg and du to `q` (bf16: of it dg_rows and du_rows, read both ways).
template <typename T, int ACT>
cudaError_t gradient(const GatedFfBackward& p, const Scaled& q, int sms, cudaStream_t st, int* launches) {
    const Aligned on{on16(p.dh, p.M, p.lddh),
                     on16(p.kept.gate, p.M, p.kept.ld) && on16(p.kept.up, p.M, p.kept.ld),
                     on16(p.h, p.M, p.ldh)};
    const bool in8 = p.kept.keep == kKeep8;
    const auto blocks_of = [&](long long units) {
        return static_cast<unsigned>(std::max(1LL, std::min<long long>(units, sms * 8LL)));
    };
    if constexpr (std::is_same<T, __half>::value) {
        constexpr long long kBlocksAnSm = 3;
        const long long words = p.M + 2LL * p.N, tiles = up_to(p.N, kTileCols);
        cudaError_t e = launch_dependent(ff_clear, dim3(blocks_of(up_to(words, kThreads))), kThreads, 0, st,
                                         q.rows, words);
        if (e != cudaSuccess) return e;
        ++*launches;
        const long long bands = std::min(up_to(p.M, kThreads / 32), sms * kBlocksAnSm / tiles);
        const dim3 grid(static_cast<unsigned>(tiles), static_cast<unsigned>(std::max(1LL, bands)));
        e = launch_dependent(in8 ? ff_gradient_fp16<ACT, true, false> : ff_gradient_fp16<ACT, false, false>, grid,
                             kThreads, 0, st, p, q, on);
        if (e != cudaSuccess) return e;
        ++*launches;
        e = launch_dependent(in8 ? ff_gradient_fp16<ACT, true, true> : ff_gradient_fp16<ACT, false, true>, grid,
                             kThreads, 0, st, p, q, on);
        ++*launches;
        return e;
    } else {
        ++*launches;
        return launch_dependent(in8 ? ff_gradient<T, ACT, true> : ff_gradient<T, ACT, false>,
                                dim3(blocks_of(up_to(p.M * up_to(p.N, 8), kThreads))), kThreads, 0, st, p,
                                reinterpret_cast<T*>(q.dg_rows), reinterpret_cast<T*>(q.du_rows), q.pitch, on);
    }
}

// The second half of products whose tiles were split.
template <typename T>
cudaError_t add_parts(const PairPlan& pl, int sms, cudaStream_t st, int* launches) {
    Parts q{};
    int n = 0, rows = 0;
    for (int i = 0; i < 3; ++i) {
        const Product& of = pl.of[i > 0];
        if (!pl.to[i].partial) continue;
        q.of[n++] = {pl.to[i].partial, of.split, of.rows, pl.to[i].c, pl.to[i].ld};
        rows = std::max(rows, of.rows);
    }
    if (n == 0) return cudaSuccess;
    q.ld = pl.partial_ld;
    q.cols = pl.of[0].cols;
    const long long blocks = up_to(rows * up_to(q.cols, 4), kThreads);
    ++*launches;
    return launch_dependent(ff_add_parts<T>,
                            dim3(static_cast<unsigned>(std::min<long long>(blocks, sms * 8LL)), n),
                            kThreads, 0, st, q);
}

template <typename T>
cudaError_t backward(const GatedFfBackward& p, int sms, cudaStream_t st, int* launches) {
    constexpr bool kScaled = std::is_same<T, __half>::value;
    uint8_t* at = p.ws;
    const auto take = [&](long long bytes) {
        uint8_t* const from = at;
        at += bytes;
        return from;
    };
    const auto matrix = [&] { return reinterpret_cast<__half*>(take(matrix_bytes(p.M, p.N))); };
    Scaled q{};
    q.pitch = up64(p.N);
    q.dg_rows = q.dg_cols = matrix();
    q.du_rows = q.du_cols = matrix();
    if (kScaled) {
        q.dg_cols = matrix();
        q.du_cols = matrix();
        q.rows = reinterpret_cast<uint32_t*>(take(largest_bytes(p.M, p.N)));
        q.of_dg = q.rows + p.M;
        q.of_du = q.of_dg + p.N;
    }
    Operands in(p.M, p.N, p.K, p.x, p.ldx, p.w_gate, p.ldg, p.w_up, p.ldu, at);
    const void* rest = nullptr;
    if (p.x_codes) {       // the operands' type holds them in two
        in.x = in.at;
        in.ldx = up64(p.K);
        in.at += matrix_bytes(p.M, p.K);
        rest = in.at;
        in.at += matrix_bytes(p.M, p.K);
        const cudaError_t e = launch_act8_dequantize(
            Act8Dequantize{p.M, p.K, p.dtype, p.x_codes, p.x_scales, const_cast<void*>(in.x), in.ldx,
                           const_cast<void*>(rest)},
            sms, st);
        if (e != cudaSuccess) return e;
        ++*launches;
    }
    cudaError_t e = in.copy(sms, st, launches);
    if (e != cudaSuccess) return e;
    e = p.activation == kSilu ? gradient<T, kSilu>(p, q, sms, st, launches)
                              : gradient<T, kGeluTanh>(p, q, sms, st, launches);
    if (e != cudaSuccess) return e;

    PairMaps maps;
    PairPlan pl{};
    pl.status = status_word_ptr();
    // dx, from dg and Wg, then du and Wu; dWg and dWu.
    const int x_parts = rest ? 2 : 1;
    const Gradients c = choose_gradients(p.M, p.N, p.K, x_parts);
    if (!encode(&maps.a[0], q.dg_rows, p.M, p.N, q.pitch, 128) ||
        !encode(&maps.a[1], q.du_rows, p.M, p.N, q.pitch, 128) ||
        !encode(&maps.a[2], q.dg_cols, p.M, p.N, q.pitch, 64) ||
        !encode(&maps.a[3], q.du_cols, p.M, p.N, q.pitch, 64) ||
        !encode(&maps.b[0], in.w_gate, p.N, p.K, in.ldg, 64) ||
        !encode(&maps.b[1], in.w_up, p.N, p.K, in.ldu, 64) ||
        !encode(&maps.b[2], in.x, p.M, p.K, in.ldx, 64) ||
        (rest && !encode(&maps.b[3], rest, p.M, p.K, in.ldx, 64)))
        return cudaErrorInvalidValue;
    const int tiles_n = static_cast<int>(up_to(p.K, c.bn));
    pl.of[0] = {p.M, p.K, static_cast<int>(up_to(p.M, kTileRows)), tiles_n,
                static_cast<int>(2 * up_to(p.N, 64)), static_cast<int>(up_to(p.N, 64)), c.split_x};
    pl.of[1] = {p.N, p.K, static_cast<int>(2 * up_to(p.N, kTileRows)), tiles_n,
                static_cast<int>(x_parts * up_to(p.M, 64)), static_cast<int>(up_to(p.M, 64)), c.split_w};
    pl.pairs = static_cast<int>(std::min<long long>(sms / 2, pl.of[0].items() + pl.of[1].items()));
    pl.extra = spread(pl.of[0].items(), pl.of[1].items(), item_clocks(up_to(pl.of[0].stages, c.split_x), c.bn),
                      item_clocks(up_to(pl.of[1].stages, c.split_w), c.bn), pl.pairs).extra;
    pl.to[0] = {p.dx, p.lddx, on16(p.dx, p.M, p.lddx), nullptr, q.rows};
    pl.to[1] = {p.dw_gate, p.lddwg, on16(p.dw_gate, p.N, p.lddwg), nullptr, q.of_dg};
    pl.to[2] = {p.dw_up, p.lddwu, on16(p.dw_up, p.N, p.lddwu), nullptr, q.of_du};
    pl.partial_ld = up64(p.K);
    float* partial = reinterpret_cast<float*>(in.at);
    for (int i = 0; i < 3; ++i) {
        const Product& of = pl.of[i > 0];
        if (of.split == 1) continue;
        pl.to[i].partial = partial;
        partial += of.split * (of.rows * pl.partial_ld);
    }
    e = pair<T>(maps, pl, kBackward, c.bn, p.activation, st);
    if (e != cudaSuccess) return e;
    ++*launches;
    return add_parts<T>(pl, sms, st, launches);
}

// Copies of the operands that are not read in place.
size_t copied_bytes(int M, int N, int K, int packed) {
    return static_cast<size_t>((packed & 1 ? matrix_bytes(M, K) : 0) +
                               (packed & 2 ? matrix_bytes(N, K) : 0) +
                               (packed & 4 ? matrix_bytes(N, K) : 0));
}
int packed_bit(int bit, const void* p, long long rows, long long ld) {
    return on16(p, rows, ld) ? 0 : bit;
}

}  // namespace

FfChoice choose_gated_ff(int product, int M, int N, int K, int keep) {
    if (product == kProductForward) return choose_forward(M, N, K, keep);
    const Gradients c = choose_gradients(M, N, K, 1);
    return FfChoice{c.bn, product == kProductInput ? c.split_x : c.split_w};
}
size_t gated_ff_forward_workspace(int M, int N, int K, int packed) {
    return copied_bytes(M, N, K, packed);
}
size_t gated_ff_backward_workspace(int M, int N, int K, int packed) {
    const long long scaled = packed & kPackedFp16 ? 2 * matrix_bytes(M, N) + largest_bytes(M, N) : 0;
    const auto with = [&](int x_parts) {
        const Gradients c = choose_gradients(M, N, K, x_parts);
        const long long parts =
            (c.split_x > 1 ? 1LL * c.split_x * M : 0) + (c.split_w > 1 ? 2LL * c.split_w * N : 0);
        return static_cast<size_t>(2 * matrix_bytes(M, N) + scaled + (x_parts - 1) * matrix_bytes(M, K)) +
               copied_bytes(M, N, K, packed) + static_cast<size_t>(parts * up64(K)) * sizeof(float);
    };
    // (The same bit stands for an x whose rows are copied and for one in 8 bits.)
    return packed & 1 ? std::max(with(1), with(2)) : with(1);
}
int gated_ff_packed(const GatedFfForward& p) {
    if (choose_forward(p.M, p.N, p.K, p.kept.keep).bn == 0) return 0;
    return packed_bit(1, p.x, p.M, p.ldx) | packed_bit(2, p.w_gate, p.N, p.ldg) |
           packed_bit(4, p.w_up, p.N, p.ldu);
}
int gated_ff_packed(const GatedFfBackward& p) {
    return (p.x_codes ? 1 : packed_bit(1, p.x, p.M, p.ldx)) |
           packed_bit(2, p.w_gate, p.N, p.ldg) | packed_bit(4, p.w_up, p.N, p.ldu) |
           (p.dtype == mx4::kF16 ? kPackedFp16 : 0);
}

cudaError_t launch_gated_ff_forward(const GatedFfForward& p, int sms, cudaStream_t stream,
                                    int* launches) {
    *launches = 0;
    return p.dtype == kBf16 ? forward<__nv_bfloat16>(p, sms, stream, launches)
                            : forward<__half>(p, sms, stream, launches);
}
cudaError_t launch_gated_ff_backward(const GatedFfBackward& p, int sms, cudaStream_t stream,
                                     int* launches) {
    *launches = 0;
    return p.dtype == kBf16 ? backward<__nv_bfloat16>(p, sms, stream, launches)
                            : backward<__half>(p, sms, stream, launches);
}

}  // namespace sgemm
