// Products of the gated feed-forward block on the tensor cores: tiles of 256 x BN, each by a
// pair of CTAs (tcgen05, cta_group::2, 2-byte operands, fp32 sums).
//
//     forward     act(x Wg^T) (x Wu^T)    both operands with the contraction along their rows
//     backward    dg Wg + du Wu           the weights' contraction across their rows, and in the same
//                 dg^T x, du^T x          launch, both operands' contraction across their rows
//
// The two CTAs hold 128 of a tile's rows each and half of its BN columns' operand; the MMA reads the
// other half from the other SM.  Forward, one CTA's half are rows of Wg and the other's the same
// rows of Wu, so that a token's g and u of BN / 2 outputs lie in one lane of tensor memory,
// and the gate costs no exchange.
//
// Operands are staged 64 deep, in 128-byte lines with the 128-byte swizzle, as tensor-map copies
// deliver them: [rows][64 of the contraction] or, where the contraction runs across rows, blocks of
// [64 of the contraction][64 columns].  What lies outside a matrix arrives as zeros, so no size
// needs padding.
//
// Persistent: a pair takes its share of the work items, one after the other.
//   warp 0: copies of the CTA's own halves; both CTAs' complete on the first one's barrier;
//   warp 1 of the first CTA: the MMAs of both CTAs, four a stage;
//   warps 2..5 and 6..9: the epilogue, 128 rows x each half of the columns.  Tensor memory holds
//     two sets of sums, so that one item's epilogue runs under the next one's MMAs.  A warp has
//     32 rows, one a lane, and passes up to 64 columns at a time through its own 4 KB of shared
//     memory, to store whole 128-byte lines.
//
// Four MMAs of a stage take 512 clocks, so a tile of 256 x 256 x 2048 takes 8.5 us at 1.93 GHz; measured
// are 10.2 to 12 with its share of the start and the end.  The tensor pipes are active 84 (forward, g
// and u to 8 bits) and 93 % of the time (gradient), 4096 x 2048 x 4096; at full size the card's power
// limit holds the clock lower.  Tiles of 256 x 128 fill more pairs where there are few, and forward tiles
// of 224 and 160 columns the last round better: 3001 x 2047 x 1999 has 192 tiles of 256 for 76 pairs, 2.5
// rounds that take 3, and takes 47.6 us by them, by 216 tiles of 224 44.9 (copies of the operands
// included).
#pragma once

#include <cuda_runtime.h>

#include <algorithm>
#include <type_traits>

#include "sgemm_async.cuh"
#include "sgemm_ff_plan.h"
#include "sgemm_gated_ff.cuh"
#include "sgemm_launch.cuh"
#include "sgemm_mx4_tc.cuh"

namespace sgemm {
namespace ff {

using async::mbar_expect_tx;
using async::mbar_fence_init;
using async::mbar_init;
using async::su32;
using mx4::cluster_arrive;
using mx4::cluster_wait;
using mx4::commit;
using mx4::elect_one;
using mx4::fence_after;
using mx4::fence_before;
using mx4::pipe_peek;
using mx4::pipe_wait;
using mx4::warp_index;

constexpr int kPairThreads = 320, kEpilogueWarps = 8;
constexpr int kRows = kTileRows;
constexpr int kDeep = 64;                      // of a stage
constexpr int kLineBytes = 128;
constexpr int kGroup = 16;                     // tiles of rows a raster group
constexpr int kStaged = 4096;                  // bytes of a warp's staging
template <int BN> constexpr int kHalfA = kRows / 2 * kLineBytes;
template <int BN> constexpr int kHalfB = BN / 2 * kLineBytes;
template <int BN> constexpr int kStage = kHalfA<BN> + kHalfB<BN>;
template <int BN> constexpr int kStages = BN >= 224 ? 6 : BN == 160 ? 7 : 8;
template <int BN> constexpr int kPairSmem = kStages<BN> * kStage<BN> + kEpilogueWarps * kStaged + 1024;
static_assert(kPairSmem<256> <= 226 * 1024 && kPairSmem<224> <= 226 * 1024 &&
                  kPairSmem<160> <= 226 * 1024 && kPairSmem<128> <= 226 * 1024, "shared memory");

// Shared-memory operand in 128-byte lines with the 128-byte swizzle; eight lines (1024 bytes)
// are a pattern.  Contraction along the lines: `lead` is not used.  Across them: eight of
// the contraction a pattern, and `lead` bytes from one block of 64 columns to the next.
__device__ __forceinline__ uint64_t line_desc(uint32_t saddr, uint32_t lead) {
    uint64_t d = 0;
    d |= static_cast<uint64_t>((saddr >> 4) & 0x3FFFu);
    d |= static_cast<uint64_t>((lead >> 4) & 0x3FFFu) << 16;
    d |= static_cast<uint64_t>(1024 >> 4) << 32;
    d |= static_cast<uint64_t>(1) << 46;                      // descriptor version
    d |= static_cast<uint64_t>(2) << 61;                      // 128-byte swizzle
    return d;
}
// Instruction: fp32 sums of bf16 or fp16 products, 256 rows by N columns; whether an operand's
// contraction runs across its lines.
__host__ __device__ constexpr uint32_t ff_idesc(bool bf16, int N, bool across_a, bool across_b) {
    return (1u << 4) | (bf16 ? (1u << 7) | (1u << 10) : 0u) | (across_a ? 1u << 15 : 0u) |
           (across_b ? 1u << 16 : 0u) | (static_cast<uint32_t>(N >> 3) << 17) |
           (static_cast<uint32_t>(kRows >> 4) << 24);
}
__device__ __forceinline__ void ff_mma(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc,
                                       uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d), "l"(a), "l"(b),
        "r"(idesc), "r"(accumulate)
        : "memory");
}
// The box at (x, y) (x along the lines) into this CTA, completing on `bar` of the first CTA.
__device__ __forceinline__ void load_box(uint32_t dst, const CUtensorMap* tm, int x, int y,
                                         uint32_t bar) {
    asm volatile(
        "cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.tile"
        ".mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], [%4];" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(tm)), "r"(x), "r"(y), "r"(bar)
        : "memory");
}
__device__ __forceinline__ uint32_t in_first_cta(uint32_t addr) {
    uint32_t r;
    asm("mapa.shared::cluster.u32 %0, %1, 0;" : "=r"(r) : "r"(addr));
    return r;
}
// Relaxed: it announces reads of tensor memory, which the tcgen05 fence before it orders.
__device__ __forceinline__ void arrive_read(uint32_t addr) {
    asm volatile("mbarrier.arrive.relaxed.cluster.shared::cluster.b64 _, [%0];" ::"r"(addr)
                 : "memory");
}
__device__ __forceinline__ bool all_of_group(int barrier, bool ok) {
    uint32_t r;
    asm volatile(
        "{\n\t.reg .pred p, q;\n\tsetp.ne.u32 p, %2, 0;\n\t"
        "barrier.cta.red.and.pred q, %1, 128, p;\n\tselp.b32 %0, 1, 0, q;\n\t}"
        : "=r"(r) : "r"(barrier), "r"(static_cast<uint32_t>(ok)) : "memory");
    return r != 0;
}

template <int STAGES>
struct Ring {
    int stage = 0;
    uint32_t phase = 0;
    __device__ __forceinline__ void next() {
        if (++stage == STAGES) {
            stage = 0;
            phase ^= 1u;
        }
    }
};

// One work item: a tile, and a range of its stages.
struct Item {
    int result;            // PairPlan::to
    int row, col;          // its first row and column of the result
    int first, last;       // stages
    int part;
};
template <int MODE, int BN>
__device__ __forceinline__ Item item_of(const Product& p, int i, bool weights) {
    Item t{};
    const int tile = i / p.split;
    t.part = i - tile * p.split;
    const int group = tile / (kGroup * p.tiles_n), in = tile - group * kGroup * p.tiles_n;
    const int high = min(kGroup, p.tiles_m - group * kGroup);
    int m = group * kGroup + in % high;
    if (weights) {
        const int half = p.tiles_m / 2;
        t.result = m >= half ? 2 : 1;
        if (m >= half) m -= half;
    }
    t.row = m * kRows;
    t.col = in / high * (MODE == kForward ? BN / 2 : BN);
    t.first = static_cast<int>(static_cast<long long>(p.stages) * t.part / p.split);
    t.last = static_cast<int>(static_cast<long long>(p.stages) * (t.part + 1) / p.split);
    return t;
}
// A pair's items.  Those of the first product go round the pairs; where they do not come out even, the
// `few` pairs with one less take pl.extra each of the second product's next, and what is left of
// it goes round, from these pairs on.
template <int MODE, int BN>
struct Share {
    int pair, pairs, ones, lead, few, slot, count;
    __device__ __forceinline__ Share(const PairPlan& pl) {
        pair = static_cast<int>(blockIdx.x) >> 1;
        pairs = static_cast<int>(gridDim.x) >> 1;
        const int n = pl.of[0].tiles_m * pl.of[0].tiles_n * pl.of[0].split;
        ones = count = (n - pair + pairs - 1) / pairs;
        lead = few = slot = 0;
        if constexpr (MODE == kBackward) {
            const int m = pl.of[1].tiles_m * pl.of[1].tiles_n * pl.of[1].split;
            const int more = n % pairs;                // pairs 0 .. more - 1 have one more
            few = more ? pairs - more : 0;
            lead = few && pair >= more ? pl.extra : 0;
            slot = pair >= more ? pair - more : pair + few;
            count += lead + (m - few * pl.extra - slot + pairs - 1) / pairs;
        }
    }
    __device__ __forceinline__ Item at(const PairPlan& pl, int i) const {
        if (MODE == kForward || i < ones) return item_of<MODE, BN>(pl.of[0], pair + i * pairs, false);
        i -= ones;
        return item_of<MODE, BN>(pl.of[1], i < lead ? slot + i * few
                                                    : few * pl.extra + slot + (i - lead) * pairs, true);
    }
};

// A warp's 32 rows of CHUNKS 16-byte chunks: staged one row a lane, stored in whole lines.
// The chunks of the rows that share a 128-byte line are permuted, so that neither side meets a
// bank twice.
template <int CHUNKS>
__device__ __forceinline__ uint32_t staged_at(int row, int chunk) {
    constexpr int kPerLine = 8 / CHUNKS;
    return row * (16 * CHUNKS) + ((chunk ^ (row / kPerLine & (CHUNKS - 1))) << 4);
}
__device__ __forceinline__ void st_shared(uint32_t addr, uint4 v) {
    asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(v.x), "r"(v.y),
                 "r"(v.z), "r"(v.w) : "memory");
}
__device__ __forceinline__ uint4 ld_shared(uint32_t addr) {
    uint4 v;
    asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(addr) : "memory");
    return v;
}
template <typename T>
__device__ __forceinline__ uint32_t pack2(float a, float b);
template <>
__device__ __forceinline__ uint32_t pack2<__nv_bfloat16>(float a, float b) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<const uint32_t*>(&h);
}
template <>
__device__ __forceinline__ uint32_t pack2<__half>(float a, float b) {
    const __half2 h = __floats2half2_rn(a, b);
    return *reinterpret_cast<const uint32_t*>(&h);
}
__device__ __forceinline__ uint32_t ld_shared_word(uint32_t addr) {
    uint32_t v;
    asm volatile("ld.shared.b32 %0, [%1];" : "=r"(v) : "r"(addr) : "memory");
    return v;
}
// Staged rows of USED chunks to `to`, `ld` bytes apart, of which `rows` rows and `bytes` bytes each are
// inside the result.  vec: rows start on 16 bytes; otherwise a warp stores a row at a time, two
// 2-byte numbers a lane.
template <int CHUNKS, int USED = CHUNKS>
__device__ __forceinline__ void store_staged(uint32_t staged, uint8_t* to, long long ld, int rows,
                                             int bytes, bool vec, int lane) {
    constexpr int kPer = 32 / CHUNKS;              // rows a step
    __syncwarp();
    if (vec && bytes >= 16 * USED) {
        const int chunk = lane % CHUNKS;
#pragma unroll
        for (int r0 = 0; r0 < 32; r0 += kPer) {
            const int r = r0 + lane / CHUNKS;
            if (r >= rows || chunk >= USED) break;
            *reinterpret_cast<uint4*>(to + r * ld + 16 * chunk) =
                ld_shared(staged + staged_at<CHUNKS>(r, chunk));
        }
    } else if (lane < 4 * USED && 4 * lane < bytes) {
        const bool both = 4 * lane + 4 <= bytes;
#pragma unroll 4
        for (int r = 0; r < rows; ++r) {
            const uint32_t v = ld_shared_word(staged + staged_at<CHUNKS>(r, lane >> 2) + (lane & 3) * 4);
            uint8_t* const at = to + r * ld + 4 * lane;
            if (both && (reinterpret_cast<uintptr_t>(at) & 3) == 0) {
                *reinterpret_cast<uint32_t*>(at) = v;
            } else {
                *reinterpret_cast<uint16_t*>(at) = static_cast<uint16_t>(v);
                if (both) reinterpret_cast<uint16_t*>(at)[1] = static_cast<uint16_t>(v >> 16);
            }
        }
    }
    __syncwarp();
}
// COLS numbers a lane as 2-byte rows.
template <typename T, int COLS, int N>
__device__ __forceinline__ void put_rows(uint32_t staged, const float (&v)[N], uint8_t* to,
                                         long long ld, int rows, int cols, bool vec, int lane) {
    constexpr int kChunks = COLS > 32 ? 8 : 4;
#pragma unroll
    for (int i = 0; i < COLS; i += 8)
        st_shared(staged + staged_at<kChunks>(lane, i / 8),
                  make_uint4(pack2<T>(v[i], v[i + 1]), pack2<T>(v[i + 2], v[i + 3]),
                             pack2<T>(v[i + 4], v[i + 5]), pack2<T>(v[i + 6], v[i + 7])));
    store_staged<kChunks, COLS / 8>(staged, to, 2 * ld, rows, 2 * min(cols, COLS), vec, lane);
}
// 64 numbers a lane, one block of an 8-bit checkpoint (columns past the end are zeros).
__device__ __forceinline__ void put_codes(uint32_t staged, const float (&v)[64], int8_t* codes,
                                          float* scales, long long pitch, long long row, int col,
                                          int rows, int lane) {
    uint32_t amax = 0;
#pragma unroll
    for (int i = 0; i < 64; ++i) amax = max(amax, act8::magnitude(v[i]));
    const act8::BlockScale s(amax);
    if (lane < rows) scales[(row + lane) * (pitch / kAct8Block) + col / kAct8Block] = s.scale;
#pragma unroll
    for (int i = 0; i < 64; i += 16)
        st_shared(staged + staged_at<4>(lane, i / 16),
                  make_uint4(s.codes4(v[i], v[i + 1], v[i + 2], v[i + 3]),
                             s.codes4(v[i + 4], v[i + 5], v[i + 6], v[i + 7]),
                             s.codes4(v[i + 8], v[i + 9], v[i + 10], v[i + 11]),
                             s.codes4(v[i + 12], v[i + 13], v[i + 14], v[i + 15])));
    store_staged<4>(staged, reinterpret_cast<uint8_t*>(codes + row * pitch + col), pitch, rows, 64, true,
                    lane);
}
template <int COLS>
__device__ __forceinline__ void tmem_get(uint32_t at, float (&v)[COLS]) {
    if constexpr (COLS == 64) {
        mx4::tmem_ld64(at, v);
    } else {
#pragma unroll
        for (int i = 0; i < COLS; i += 16)
            mx4::tmem_ld16(at + i, reinterpret_cast<float(&)[16]>(v[i]));
    }
}

template <typename T, int MODE, int BN, int ACT>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kPairThreads, 1)
    ff_pair_kernel(const __grid_constant__ PairMaps maps, const PairPlan pl) {
    constexpr int kSums = BN > 128 ? 256 : 128;        // columns of tensor memory from one set to the other
    constexpr int kTmemCols = 2 * kSums;
    constexpr int N_STAGES = kStages<BN>;
    extern __shared__ uint8_t smem_raw[];
    __shared__ __align__(8) uint64_t full_bar[N_STAGES], empty_bar[N_STAGES];
    __shared__ __align__(8) uint64_t done_bar[2], free_bar[2];
    __shared__ uint32_t tmem_base_s;
    __shared__ int abort_s;
    const int warp = warp_index(), lane = threadIdx.x & 31;
    const int rank = static_cast<int>(blockIdx.x) & 1;
    const Share<MODE, BN> share(pl);
    volatile int* abort_flag = &abort_s;
    const uint32_t smem0 = (su32(smem_raw) + 1023u) & ~1023u;

    if (threadIdx.x == 0) {
        for (int s = 0; s < N_STAGES; ++s) {
            mbar_init(su32(&full_bar[s]), 1);
            mbar_init(su32(&empty_bar[s]), 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(su32(&done_bar[i]), 1);
            mbar_init(su32(&free_bar[i]), 2 * kEpilogueWarps);
        }
        abort_s = 0;
        mbar_fence_init();
    }
    if (warp == 0 && lane < (MODE == kForward ? 3 : pl.of[1].half < pl.of[1].stages ? 8 : 7)) {
        const CUtensorMap* tm = MODE == kForward ? (lane < 1 ? &maps.a[0] : &maps.b[lane - 1])
                                                 : (lane < 4 ? &maps.a[lane] : &maps.b[lane - 4]);
        asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(tm)) : "memory");
    }
    if (warp == 1) mx4::tmem_alloc<2>(su32(&tmem_base_s), kTmemCols);
    fence_before();
    __syncthreads();
    cluster_arrive();       // the other CTA's barriers exist
    cluster_wait();
    fence_after();
    const uint32_t tmem = tmem_base_s;
    start_dependent();

    if (warp == 0) {
        if (elect_one()) {
            Ring<N_STAGES> ring;
            int issued = 0;
            bool ok = true;
            for (int i = 0; i < share.count && ok; ++i) {
                const Item t = share.at(pl, i);
                const int row = t.row + rank * (kRows / 2);
                const int col = MODE == kForward ? t.col : t.col + rank * (BN / 2);
                for (int s = t.first; s < t.last; ++s) {
                    if (!pipe_wait(su32(&empty_bar[ring.stage]), ring.phase ^ 1u, abort_flag,
                                   pl.status)) {
                        ok = false;
                        break;
                    }
                    const uint32_t fb = in_first_cta(su32(&full_bar[ring.stage]));
                    const uint32_t a = smem0 + ring.stage * kStage<BN>, b = a + kHalfA<BN>;
                    if (rank == 0) mbar_expect_tx(su32(&full_bar[ring.stage]), 2 * kStage<BN>);
                    if constexpr (MODE == kForward) {
                        load_box(a, &maps.a[0], s * kDeep, row, fb);
                        load_box(b, &maps.b[rank], s * kDeep, col, fb);
                    } else {
                        // dg and Wg, then du and Wu; x, then its rest.
                        const int half = pl.of[t.result > 0].half, second = s >= half;
                        const int k = (s - second * half) * kDeep;
                        const CUtensorMap* bm = &maps.b[2 * (t.result > 0) + second];
                        if (t.result == 0) {
                            load_box(a, &maps.a[second], k, row, fb);
                        } else {
                            const CUtensorMap* am = &maps.a[1 + t.result];
                            load_box(a, am, row, k, fb);
                            load_box(a + kDeep * kLineBytes, am, row + 64, k, fb);
                        }
#pragma unroll
                        for (int c = 0; c < BN / 2; c += 64)
                            load_box(b + c / 64 * (kDeep * kLineBytes), bm, col + c, k, fb);
                    }
                    ++issued;
                    ring.next();
                }
            }
            // Copies in flight land before the pair exits, whichever wait gave up.  They signal
            // the first CTA, so it waits for both; what the second may have asked for beyond
            // that had the time limit of the wait that gave up.
            if (rank == 0) {
                volatile int no_abort = 0;
                for (int i = max(0, issued - N_STAGES); i < issued; ++i)
                    pipe_wait(su32(&full_bar[i % N_STAGES]), (i / N_STAGES) & 1, &no_abort, nullptr);
            }
        }
    } else if (warp == 1) {
        if (rank == 0 && elect_one()) {
            constexpr uint32_t kLead = kDeep * kLineBytes;
            // Sixteen of the contraction: 32 bytes of a line, or 16 lines.
            constexpr uint32_t kAlong = 32 / 16, kAcross = 16 * kLineBytes / 16;
            constexpr uint32_t kStepB = MODE == kForward ? kAlong : kAcross;
            const uint64_t a_along = line_desc(smem0, 0), a_across = line_desc(smem0, kLead);
            const uint64_t b_desc = line_desc(smem0 + kHalfA<BN>, MODE == kForward ? 0 : kLead);
            constexpr bool kIsBf16 = sizeof(T) == 2 && !std::is_same<T, __half>::value;
            Ring<N_STAGES> ring;
            bool ready = false, ok = true;
            for (int n = 0; n < share.count && ok; ++n) {
                const Item t = share.at(pl, n);
                const bool across = t.result > 0;          // the contraction runs across dg's rows
                const uint64_t a_desc = across ? a_across : a_along;
                const uint32_t step_a = across ? kAcross : kAlong;
                const uint32_t idesc = across ? ff_idesc(kIsBf16, BN, true, true)
                                              : ff_idesc(kIsBf16, BN, false, MODE != kForward);
                const uint32_t sums = tmem + (n & 1) * kSums;
                // The item before the last one has left this set of sums (first: at once).
                if (!pipe_wait<true>(su32(&free_bar[n & 1]), ((n >> 1) & 1) ^ 1u, abort_flag,
                                     pl.status))
                    break;
                fence_after();
                for (int s = t.first; s < t.last; ++s) {
                    if (!ready && !pipe_wait<true>(su32(&full_bar[ring.stage]), ring.phase,
                                                   abort_flag, pl.status)) {
                        ok = false;
                        break;
                    }
                    fence_after();
                    // The answer about the next stage arrives under this one's MMAs.
                    Ring<N_STAGES> ahead = ring;
                    ahead.next();
                    ready = pipe_peek(su32(&full_bar[ahead.stage]), ahead.phase);
                    const uint32_t at = ring.stage * (kStage<BN> / 16);
#pragma unroll
                    for (int k = 0; k < kDeep / 16; ++k)
                        ff_mma(sums, a_desc + at + k * step_a, b_desc + at + k * kStepB, idesc,
                               s != t.first || k != 0);
                    commit<2>(su32(&empty_bar[ring.stage]));
                    ring = ahead;
                }
                if (ok) commit<2>(su32(&done_bar[n & 1]));      // else both epilogues give up
            }
        }
    } else {
        const int quarter = warp & 3, half = (warp - 2) >> 2;
        const uint32_t staged = smem0 + N_STAGES * kStage<BN> + (warp - 2) * kStaged;
        for (int n = 0; n < share.count; ++n) {
            // All four warps of this half go on, or none.
            const bool ok = all_of_group(
                1 + half, pipe_wait(su32(&done_bar[n & 1]), (n >> 1) & 1, abort_flag, pl.status) &&
                              !*abort_flag);
            if (!ok) break;
            fence_after();
            const Item t = share.at(pl, n);
            const Result& to = pl.to[MODE == kForward ? 0 : t.result];
            const Product& of = pl.of[MODE == kForward ? 0 : t.result > 0];
            const uint32_t sums = tmem + (static_cast<uint32_t>(32 * quarter) << 16) + (n & 1) * kSums;
            const long long row = t.row + rank * (kRows / 2) + 32 * quarter;
            const int rows = static_cast<int>(max(0LL, min(32LL, of.rows - row)));
            auto done_reading = [&] {
                fence_before();
                __syncwarp();
                if (lane == 0) arrive_read(in_first_cta(su32(&free_bar[n & 1])));
            };
            if constexpr (MODE == kForward) {
                constexpr int kCols = BN / 4;                  // outputs of a half
                constexpr int kRead = kCols > 32 ? 64 : 32;    // (those past a half's are not used)
                const FfKept& kept = pl.kept;
                {
                    float g[kRead], u[kRead];
                    tmem_get<kRead>(sums + half * kCols, g);
                    tmem_get<kRead>(sums + BN / 2 + half * kCols, u);
                    done_reading();
                    const int col = t.col + half * kCols, cols = of.cols - col;
                    if (rows == 0 || cols <= 0) continue;
                    if (kept.keep == kKeepFull) {
                        put_rows<T, kCols>(staged, g, static_cast<uint8_t*>(kept.gate) +
                                                          (row * kept.ld + col) * 2,
                                           kept.ld, rows, cols, pl.kept_vec, lane);
                        put_rows<T, kCols>(staged, u, static_cast<uint8_t*>(kept.up) +
                                                          (row * kept.ld + col) * 2,
                                           kept.ld, rows, cols, pl.kept_vec, lane);
                    }
                    if constexpr (kCols == 64) {
                        if (kept.keep == kKeep8) {
                            const long long pitch = act8_pitch(of.cols);
                            put_codes(staged, g, static_cast<int8_t*>(kept.gate), kept.gate_scales,
                                      pitch, row, col, rows, lane);
                            put_codes(staged, u, static_cast<int8_t*>(kept.up), kept.up_scales,
                                      pitch, row, col, rows, lane);
                        }
                    }
#pragma unroll
                    for (int j = 0; j < kCols; ++j) g[j] = act<ACT>(g[j]) * u[j];
                    put_rows<T, kCols>(staged, g,
                                       static_cast<uint8_t*>(to.c) + (row * to.ld + col) * 2, to.ld,
                                       rows, cols, to.vec, lane);
                }
            } else {
                constexpr bool kScaled = std::is_same<T, __half>::value;
                float by = 1.0f;
                if constexpr (kScaled)
                    if (lane < rows) by = scale_back(fetch_here(to.largest + row + lane));
#pragma unroll 1
                for (int c = half * (BN / 2); c < (half + 1) * (BN / 2); c += 64) {
                    float v[64];
                    tmem_get<64>(sums + c, v);
                    if (c + 64 == (half + 1) * (BN / 2)) done_reading();
                    const int col = t.col + c, cols = of.cols - col;
                    if (rows == 0 || cols <= 0) continue;
                    if constexpr (kScaled)
#pragma unroll
                        for (int j = 0; j < 64; ++j) v[j] *= by;
                    if (to.partial) {
                        // One part's fp32 sums, 32 columns at a time.
                        float* at = to.partial +
                                    (static_cast<long long>(t.part) * of.rows + row) * pl.partial_ld + col;
#pragma unroll
                        for (int half = 0; half < 64; half += 32) {
#pragma unroll
                            for (int j = 0; j < 32; j += 4)
                                st_shared(staged + staged_at<8>(lane, j / 4),
                                          make_uint4(__float_as_uint(v[half + j]),
                                                     __float_as_uint(v[half + j + 1]),
                                                     __float_as_uint(v[half + j + 2]),
                                                     __float_as_uint(v[half + j + 3])));
                            store_staged<8>(staged, reinterpret_cast<uint8_t*>(at + half),
                                            4 * pl.partial_ld, rows, 128, true, lane);
                        }
                        continue;
                    }
                    put_rows<T, 64>(staged, v, static_cast<uint8_t*>(to.c) + (row * to.ld + col) * 2, to.ld,
                                    rows, cols, to.vec, lane);
                }
            }
        }
    }
    __syncwarp();
    fence_before();
    __syncthreads();
    cluster_arrive();       // the other CTA is done with this one's memory and barriers
    cluster_wait();
    if (warp == 1) {
        fence_after();
        mx4::tmem_dealloc<2>(tmem, kTmemCols);
    }
}

template <typename T, int MODE, int BN, int ACT>
cudaError_t launch_pair(const PairMaps& maps, const PairPlan& pl, cudaStream_t stream) {
    auto kernel = ff_pair_kernel<T, MODE, BN, ACT>;
    const cudaError_t e = cudaFuncSetAttribute(
        kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kPairSmem<BN>);
    if (e != cudaSuccess) return e;
    return launch_dependent(kernel, dim3(2 * pl.pairs), kPairThreads, kPairSmem<BN>, stream, maps, pl);
}
template <typename T>
cudaError_t launch_pair_of(const PairMaps& maps, const PairPlan& pl, int mode, int bn, int activation,
                           cudaStream_t st) {
    // Items are counted in 32 bits.
    if (pl.of[0].items() + pl.of[1].items() > 0x7FFFFFFF / kGroup) return cudaErrorInvalidConfiguration;
    const auto forward = [&](auto width) {
        constexpr int BN = decltype(width)::value;
        return activation == kSilu ? launch_pair<T, kForward, BN, kSilu>(maps, pl, st)
                                   : launch_pair<T, kForward, BN, kGeluTanh>(maps, pl, st);
    };
    if (mode == kForward)
        switch (bn) {
            case 256: return forward(std::integral_constant<int, 256>());
            case 224: return forward(std::integral_constant<int, 224>());
            case 160: return forward(std::integral_constant<int, 160>());
            default: return forward(std::integral_constant<int, 128>());
        }
    return bn == 256 ? launch_pair<T, kBackward, 256, kSilu>(maps, pl, st)
                     : launch_pair<T, kBackward, 128, kSilu>(maps, pl, st);
}

}  // namespace ff
}  // namespace sgemm
