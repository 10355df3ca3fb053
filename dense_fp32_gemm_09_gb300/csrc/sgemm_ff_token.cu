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
                    "ld.global.nc.L1::no_allocate.v8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                    : "=r"(r.w[0]), "=r"(r.w[1]), "=r"(r.w[2]), "=r"(r.w[3]), "=r"(r.w[4]),
                      "=r"(r.w[5]), "=r"(r.w[6]), "=r"(r.w[7]) : "l"(p));
            else
                asm volatile("ld.global.nc.v8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                             : "=r"(r.w[0]), "=r"(r.w[1]), "=r"(r.w[2]), "=r"(r.w[3]), "=r"(r.w[4]),
                               "=r"(r.w[5]), "=r"(r.w[6]), "=r"(r.w[7]) : "l"(p));
        } else {
            const uint4 lo = __ldg(reinterpret_cast<const uint4*>(p));
            const uint4 hi = __ldg(reinterpret_cast<const uint4*>(p) + 1);
            r.w[0] = lo.x; r.w[1] = lo.y; r.w[2] = lo.z; r.w[3] = lo.w;
            r.w[4] = hi.x; r.w[5] = hi.y; r.w[6] = hi.z; r.w[7] = hi.w;
        }
        return r;
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        r.w[i] = 0;
        if (2 * i < n) r.w[i] = __ldg(p + 2 * i);
        if (2 * i + 1 < n) r.w[i] |= static_cast<uint32_t>(__ldg(p + 2 * i + 1)) << 16;
    }
    return r;
}

// Persistent: a block takes the groups blockIdx.x, + gridDim.x, ... of eight outputs.
// NT: groups of eight tokens.
template <typename T, int ACT, int NT>
__global__ void __launch_bounds__(kThreads, 2) ff_token_kernel(const GatedFfForward p, const bool on32) {
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
    Piece a[kAhead][2], b[kTokensAhead ? kAhead : 1][NT];
    auto load_tokens = [&](Piece (&to)[NT], int k) {
#pragma unroll
        for (int n = 0; n < NT; ++n)
            to[n] = load_piece<false>(x + 8 * n * p.ldx + k, 8 * n + g < p.M ? p.K - k : 0, on32);
    };
    int from = blockIdx.x, next = 0;
    const uint16_t* wg = nullptr;
    const uint16_t* wu = nullptr;
    auto load = [&](int i) {
        if (from >= groups) return;
        Piece (&to)[2] = a[i];
        if (next == 0) {                 // past the last output: its row again, not stored
            const long long row = min(8LL * from + g, p.N - 1LL);
            wg = w_gate + row * p.ldg;
            wu = w_up + row * p.ldu;
        }
        const int k = mine + next * (kWarps * kPiece);
        to[0] = load_piece<true>(wg + k, p.K - k, on32);
        to[1] = load_piece<true>(wu + k, p.K - k, on32);
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
#pragma unroll
            for (int n = 0; n < NT; ++n) {
                const Piece& of = b[kTokensAhead ? i : 0][n];
#pragma unroll
                for (int s = 0; s < 4; ++s)
                    mma16<T>(acc[n], a[i][0].w[2 * s], a[i][1].w[2 * s], a[i][0].w[2 * s + 1],
                             a[i][1].w[2 * s + 1], of.w[2 * s], of.w[2 * s + 1]);
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
cudaError_t launch(const GatedFfForward& p, bool on32, int sms, cudaStream_t st) {
    const int groups = (p.N + 7) / 8;
    const auto run = [&](auto kernel) {
        return launch_dependent(kernel, dim3(std::min(groups, 2 * sms)), kThreads, 0, st, p, on32);
    };
    return p.M <= 8 ? run(ff_token_kernel<T, ACT, 1>) : run(ff_token_kernel<T, ACT, 2>);
}

}  // namespace

cudaError_t launch_token(const GatedFfForward& p, bool on32, int sms, cudaStream_t st) {
    const bool silu = p.activation == kSilu;
    if (p.dtype == kBf16)
        return silu ? launch<__nv_bfloat16, kSilu>(p, on32, sms, st)
                    : launch<__nv_bfloat16, kGeluTanh>(p, on32, sms, st);
    return silu ? launch<__half, kSilu>(p, on32, sms, st) : launch<__half, kGeluTanh>(p, on32, sms, st);
}

}  // namespace ff
}  // namespace sgemm
