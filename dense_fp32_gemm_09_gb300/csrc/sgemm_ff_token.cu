// The gated feed-forward block for up to 16 tokens: h = act(x Wg^T) (x Wu^T), bound by reading the
// weights once (4 N K bytes).
//
// A block takes eight outputs and its 16 warps every 16th piece of 64 of the contraction.  The
// products are m16n8k16 MMAs whose rows are 8 rows of Wg and the same 8 of Wu, so that a
// thread's sums are g and u of the same output and tokens.  A sum does not depend on the order of
// its terms, so a thread feeds the MMAs 32 consecutive bytes of a row of W and of x as they
// come: nothing passes through shared memory, and a warp's loads are whole 128-byte lines, 4 KB
// of them in flight, or 2 KB from nine tokens on.  (The 256-row tiles of sgemm_ff_pair.cuh spend 16
// times as many MMAs on one token and fill as many SMs as there are tiles.)  The warps' sums are
// added through shared memory in their order.
//
// Measured (us, kernels alone; of the memory's 6.79 TB/s), bf16: one token 8192 x 4096 22.7 to 23.2
// (0.86), 16384 x 4096 41 (0.96), 2048 x 8192 12.7 (0.78), 4096 x 1024 5.3; 16 tokens 8192 x 4096 24.7
// (0.80), 16384 x 4096 42.4 (0.94).  One token 8192 x 4096 by warps of a block and pieces ahead, blocks
// an SM: 8, 4, 2: 30.0; 8, 3, 3: 26.6; 8, 2, 4: 22.7; 16, 2, 2: 22.7, and best on narrow layers.
#include <cuda_runtime.h>

#include <algorithm>
#include <type_traits>

#include "sgemm_ff_plan.h"
#include "sgemm_gated_ff.cuh"
#include "sgemm_launch.cuh"

namespace sgemm {
namespace ff {
namespace {

constexpr int kWarps = 16, kThreads = 32 * kWarps;
constexpr int kPiece = 64;               // of the contraction, 16 a lane

template <typename T>
__device__ __forceinline__ void mma16(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                      uint32_t a3, uint32_t b0, uint32_t b1) {
    if constexpr (std::is_same<T, __half>::value)
        asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
            "{%8, %9}, {%0, %1, %2, %3};"
            : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
            : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
    else
        asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
            "{%8, %9}, {%0, %1, %2, %3};"
            : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
            : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

struct Piece {
    uint32_t w[8];
};
// 16 numbers of a row at p, of which `n` are inside; zeros for the others.  The row is on 16 bytes,
// with on32 on 32.  ONCE: not into the L1 cache.
template <bool ONCE>
__device__ __forceinline__ Piece load_piece(const uint16_t* p, int n, bool on32) {
    Piece r;
    if (n >= 16) {
        if (on32) {
            if (ONCE)
                asm volatile(
                    "ld.global.L1::no_allocate.v8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                    : "=r"(r.w[0]), "=r"(r.w[1]), "=r"(r.w[2]), "=r"(r.w[3]), "=r"(r.w[4]),
                      "=r"(r.w[5]), "=r"(r.w[6]), "=r"(r.w[7]) : "l"(p));
            else
                asm volatile("ld.global.v8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                             : "=r"(r.w[0]), "=r"(r.w[1]), "=r"(r.w[2]), "=r"(r.w[3]), "=r"(r.w[4]),
                               "=r"(r.w[5]), "=r"(r.w[6]), "=r"(r.w[7]) : "l"(p));
        } else {
            const uint4 lo = fetch_here(reinterpret_cast<const uint4*>(p));
            const uint4 hi = fetch_here(reinterpret_cast<const uint4*>(p) + 1);
            r.w[0] = lo.x; r.w[1] = lo.y; r.w[2] = lo.z; r.w[3] = lo.w;
            r.w[4] = hi.x; r.w[5] = hi.y; r.w[6] = hi.z; r.w[7] = hi.w;
        }
        return r;
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        r.w[i] = 0;
        if (2 * i < n) r.w[i] = fetch_here(p + 2 * i);
        if (2 * i + 1 < n) r.w[i] |= static_cast<uint32_t>(fetch_here(p + 2 * i + 1)) << 16;
    }
    return r;
}

// The first and the end of a matrix in memory.
struct Extent {
    const uint8_t *first, *end;
    __device__ __forceinline__ Extent(const void* p, long long rows, int cols, long long ld)
        : first(static_cast<const uint8_t*>(p)), end(first + 2 * ((rows - 1) * ld + cols)) {}
};
// The same of a row that begins anywhere: the 16-byte groups that hold the numbers, as they are in
// memory, and where the first number begins.  Groups that are partly outside the matrix are left for
// later, so that what is on its way meets no branch.
struct Groups {
    uint4 v[3];
    const uint8_t* at;
    int skip, n;                 // bytes before the first number; numbers inside
    int left;                    // bit j: group j is still to be read
};
__device__ __forceinline__ Groups load_groups(const uint16_t* p, int n, const Extent& m) {
    Groups r;
    r.skip = static_cast<int>(reinterpret_cast<uintptr_t>(p) & 15);
    r.at = reinterpret_cast<const uint8_t*>(p) - r.skip;
    r.n = n;
    r.left = 0;
    const int bytes = n > 0 ? r.skip + 2 * min(n, 16) : 0;   // needed from `at` on
#pragma unroll
    for (int j = 0; j < 3; ++j) {
        const uint8_t* const q = r.at + 16 * j;
        const bool need = 16 * j < bytes, in = q >= m.first && q + 16 <= m.end;
        r.v[j] = fetch_if(q, need && in);
        r.left |= (need && !in) << j;
    }
    return r;
}
__device__ __forceinline__ uint4 load_part(const uint8_t* p, const Extent& m) {
    uint32_t h[8];
#pragma unroll
    for (int i = 0; i < 8; ++i)
        h[i] = p + 2 * i >= m.first && p + 2 * i < m.end ? fetch_here(reinterpret_cast<const uint16_t*>(p + 2 * i)) : 0u;
    return make_uint4(h[0] | h[1] << 16, h[2] | h[3] << 16, h[4] | h[5] << 16, h[6] | h[7] << 16);
}
// The numbers, cut out of the groups; zeros past the row's end.
__device__ __forceinline__ Piece cut(Groups& g, const Extent& m) {
    if (g.left) {
#pragma unroll
        for (int j = 0; j < 3; ++j)
            if (g.left >> j & 1) g.v[j] = load_part(g.at + 16 * j, m);
    }
    uint32_t w[12] = {g.v[0].x, g.v[0].y, g.v[0].z, g.v[0].w, g.v[1].x, g.v[1].y,
                      g.v[1].z, g.v[1].w, g.v[2].x, g.v[2].y, g.v[2].z, g.v[2].w};
#pragma unroll
    for (int i = 0; i < 10; ++i) w[i] = g.skip & 8 ? w[i + 2] : w[i];
#pragma unroll
    for (int i = 0; i < 9; ++i) w[i] = g.skip & 4 ? w[i + 1] : w[i];
    Piece r;
#pragma unroll
    for (int i = 0; i < 8; ++i) r.w[i] = __funnelshift_r(w[i], w[i + 1], 8 * (g.skip & 2));
    if (g.n < 16) {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (2 * i + 1 >= g.n) r.w[i] = 2 * i < g.n ? r.w[i] & 0xFFFFu : 0u;
    }
    return r;
}
__device__ __forceinline__ const Piece& cut(const Piece& p, const Extent&) { return p; }

// Persistent: a block takes the groups blockIdx.x, + gridDim.x, ... of eight outputs.
// NT: groups of eight tokens.  ANY: rows that begin anywhere, with more registers for what is on its
// way.  (Copied first to rows on 16 bytes, as the larger tiles need it, one token 8191 x 4095 took 83.4 us,
// now 44.7, sixteen 88 and 55, one 1000 x 777 7.1 and 3.1.  Rows on 16 bytes take 23 and 25: here a third
// load and 40 instructions to cut 16 numbers out, half the warps.)
template <typename T, int ACT, int NT, bool ANY>
__global__ void __launch_bounds__(kThreads, ANY ? 1 : 2) ff_token_kernel(const GatedFfForward p, const bool on32) {
    __shared__ float sums[2][kWarps][2][8][8 * NT];       // gate, up: [output][token]
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int g = lane >> 2, t = lane & 3;
    const int groups = (p.N + 7) / 8, mine = warp * kPiece + 16 * t;
    const int pieces = (p.K + kWarps * kPiece - 1) / (kWarps * kPiece);     // of every warp
    const uint16_t* const x = static_cast<const uint16_t*>(p.x) + g * p.ldx;
    const uint16_t* const w_gate = static_cast<const uint16_t*>(p.w_gate);
    const uint16_t* const w_up = static_cast<const uint16_t*>(p.w_up);
    // A piece is loaded as soon as the one kAhead before it has been multiplied, across groups.
    // With sixteen tokens that of x too, and one piece is as much as the registers of 32 warps hold
    // (16 tokens, 16384 x 4096: two pieces ahead without x 53 us, one 43.4, with x 42.4).
    constexpr int kAhead = NT == 1 ? 2 : 1;
    constexpr bool kTokensAhead = NT == 2;
    using Loaded = std::conditional_t<ANY, Groups, Piece>;
    Loaded a[kAhead][2], b[kTokensAhead ? kAhead : 1][NT];
    const Extent of_x(p.x, p.M, p.K, p.ldx), of_gate(w_gate, p.N, p.K, p.ldg), of_up(w_up, p.N, p.K, p.ldu);
    auto load_tokens = [&](Loaded (&to)[NT], int k) {
#pragma unroll
        for (int n = 0; n < NT; ++n) {
            const int left = 8 * n + g < p.M ? p.K - k : 0;
            if constexpr (ANY) to[n] = load_groups(x + 8 * n * p.ldx + k, left, of_x);
            else to[n] = load_piece<false>(x + 8 * n * p.ldx + k, left, on32);
        }
    };
    int from = blockIdx.x, next = 0;
    const uint16_t* wg = nullptr;
    const uint16_t* wu = nullptr;
    auto load = [&](int i) {
        if (from >= groups) return;
        Loaded (&to)[2] = a[i];
        if (next == 0) {                 // past the last output: its row again, not stored
            const long long row = min(8LL * from + g, p.N - 1LL);
            wg = w_gate + row * p.ldg;
            wu = w_up + row * p.ldu;
        }
        const int k = mine + next * (kWarps * kPiece);
        if constexpr (ANY) {
            to[0] = load_groups(wg + k, p.K - k, of_gate);
            to[1] = load_groups(wu + k, p.K - k, of_up);
        } else {
            to[0] = load_piece<true>(wg + k, p.K - k, on32);
            to[1] = load_piece<true>(wu + k, p.K - k, on32);
        }
        if constexpr (kTokensAhead) load_tokens(b[i], k);
        if (++next == pieces) {
            next = 0;
            from += gridDim.x;
        }
    };
    start_dependent();
#pragma unroll
    for (int i = 0; i < kAhead; ++i) load(i);
    float acc[NT][4] = {};
    int piece = 0, turn = 0;
    for (int group = blockIdx.x; group < groups;) {
#pragma unroll
        for (int i = 0; i < kAhead; ++i) {
            if (group >= groups) break;
            const int k = mine + piece * (kWarps * kPiece);
            if constexpr (!kTokensAhead) load_tokens(b[0], k);
            {
                const Piece gate = cut(a[i][0], of_gate), up = cut(a[i][1], of_up);
#pragma unroll
                for (int n = 0; n < NT; ++n) {
                    const Piece of = cut(b[kTokensAhead ? i : 0][n], of_x);
#pragma unroll
                    for (int s = 0; s < 4; ++s)
                        mma16<T>(acc[n], gate.w[2 * s], up.w[2 * s], gate.w[2 * s + 1], up.w[2 * s + 1],
                                 of.w[2 * s], of.w[2 * s + 1]);
                }
            }
            load(i);
            if (++piece < pieces) continue;
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    sums[turn][warp][j / 2][g][8 * n + 2 * t + j % 2] = acc[n][j];
                    acc[n][j] = 0.0f;
                }
            __syncthreads();
            // One token's neighbouring outputs to neighbouring threads.
            const int token = threadIdx.x / 8, j = threadIdx.x % 8;
            const long long col = 8LL * group + j;
            if (token < p.M && col < p.N) {
                float gate = 0.0f, up = 0.0f;
#pragma unroll
                for (int w = 0; w < kWarps; ++w) {
                    gate += sums[turn][w][0][j][token];
                    up += sums[turn][w][1][j][token];
                }
                if (p.kept.keep == kKeepFull) {
                    static_cast<T*>(p.kept.gate)[token * p.kept.ld + col] = from_float<T>(gate);
                    static_cast<T*>(p.kept.up)[token * p.kept.ld + col] = from_float<T>(up);
                }
                static_cast<T*>(p.h)[token * p.ldh + col] = from_float<T>(act<ACT>(gate) * up);
            }
            // (Two sets of sums: a thread writes one again after the next group's barrier.)
            turn ^= 1;
            piece = 0;
            group += gridDim.x;
        }
    }
}

template <typename T, int ACT>
cudaError_t launch(const GatedFfForward& p, int on, int sms, cudaStream_t st) {
    const int groups = (p.N + 7) / 8;
    const auto run = [&](auto kernel, int blocks) {
        return launch_dependent(kernel, dim3(std::min(groups, blocks * sms)), kThreads, 0, st, p, on == 32);
    };
    if (on < 16)
        return p.M <= 8 ? run(ff_token_kernel<T, ACT, 1, true>, 1) : run(ff_token_kernel<T, ACT, 2, true>, 1);
    return p.M <= 8 ? run(ff_token_kernel<T, ACT, 1, false>, 2) : run(ff_token_kernel<T, ACT, 2, false>, 2);
}

}  // namespace

cudaError_t launch_token(const GatedFfForward& p, int on, int sms, cudaStream_t st) {
    const bool silu = p.activation == kSilu;
    if (p.dtype == kBf16)
        return silu ? launch<__nv_bfloat16, kSilu>(p, on, sms, st)
                    : launch<__nv_bfloat16, kGeluTanh>(p, on, sms, st);
    return silu ? launch<__half, kSilu>(p, on, sms, st) : launch<__half, kGeluTanh>(p, on, sms, st);
}

}  // namespace ff
}  // namespace sgemm
