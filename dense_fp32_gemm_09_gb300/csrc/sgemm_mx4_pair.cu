// The 4-bit product for large matrices: 256 x 256 tiles, each by a pair of CTAs.
//
// A pair of SMs runs one tcgen05.mma over both: each holds 128 of the tile's 256 rows of
// B (n) and 128 of its 256 rows of A (m), and the instruction reads the other's half of A,
// so that an SM's shared memory delivers 8 KB of codes per 128 x 256 x 64 products where a
// CTA alone would need 12 KB.  (Roles, layout and scales as in sgemm_mx4_matmul.cu.)
//
// Persistent: pair i takes the tiles i, i + pairs, ...
//   warp 0: bulk copies of the CTA's own halves, and of the scales: its own rows of B, all
//     256 rows of A (the scales of the column operand are needed by both SMs).
//   warp 1: in the first CTA the MMAs of both; in the second it passes on that a stage
//     has arrived (a bulk copy can only signal a barrier of its own CTA).
//   warps 2..9: the epilogue, 128 lanes x 2 halves of the columns.  The 256 columns of fp32
//     sums leave no room for a second set beside the scales, so a warp first moves its
//     sums to registers, lets the next tile start, and then stores them under its MMAs.
#include <cuda_runtime.h>

#include <algorithm>

#include "sgemm_mx4_tc.cuh"

namespace sgemm {
namespace {

using namespace mx4;
using async::mbar_arrive;
using async::mbar_expect_tx;
using async::mbar_fence_init;
using async::mbar_init;
using async::su32;

constexpr int kThreads = 320, kEpilogueWarps = 8;
constexpr int kTile = 256;
constexpr int kStages = 5;
constexpr int kGroup = 8;        // tiles of m a raster group
constexpr int kCodes = kSlabChunks * 2048;
template <int FORMAT> constexpr int kSf = kSlabGroups<FORMAT> * 512;
template <int FORMAT> constexpr int kStageBytes = 2 * kCodes + 3 * kSf<FORMAT>;
// Scale columns of a stage: four per group and 128 rows (128 of B, 256 of A).
template <int FORMAT> constexpr int kStageCols = 12 * kSlabGroups<FORMAT>;
constexpr int kTmemCols = 512;
static_assert(kTile + kStages * kStageCols<kNvfp4> <= kTmemCols, "tensor memory");
static_assert(kStages * kStageBytes<kNvfp4> <= 220 * 1024, "shared memory");

struct PairPlan {
    Mx4Matmul p;
    int chunks, slabs, tiles_n, tiles_m;
    int* status;
};

struct Tile {
    long long n0, m0;
};
__device__ __forceinline__ Tile tile_at(const PairPlan& pl, int tile) {
    const int group = tile / (kGroup * pl.tiles_n), in = tile - group * kGroup * pl.tiles_n;
    const int high = min(kGroup, pl.tiles_m - group * kGroup);
    return Tile{in / high * static_cast<long long>(kTile),
                (group * kGroup + in % high) * static_cast<long long>(kTile)};
}
__device__ __forceinline__ uint32_t in_first_cta(uint32_t addr) {
    uint32_t r;
    asm("mapa.shared::cluster.u32 %0, %1, 0;" : "=r"(r) : "r"(addr));
    return r;
}
// Relaxed: what it announces was not written by this thread (bulk copies, which the
// barrier has already seen complete) or is ordered by the tcgen05 fence before it (reads of
// tensor memory).  A release would also wait for the thread's copies in flight: 400
// instead of 183 us for the copies alone at 8192^3.
__device__ __forceinline__ void arrive_cluster(uint32_t addr) {
    asm volatile("mbarrier.arrive.relaxed.cluster.shared::cluster.b64 _, [%0];" ::"r"(addr)
                 : "memory");
}

template <int FORMAT>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kThreads, 1)
    mx4_pair_kernel(const PairPlan pl) {
    extern __shared__ __align__(128) uint8_t smem[];
    __shared__ __align__(8) uint64_t full_bar[kStages], peer_bar[kStages], empty_bar[kStages];
    __shared__ __align__(8) uint64_t done_bar, free_bar;
    __shared__ uint32_t tmem_base_s;
    __shared__ int abort_s;
    const Mx4Matmul& p = pl.p;
    const int warp = warp_index(), lane = threadIdx.x & 31;
    const int rank = static_cast<int>(blockIdx.x) & 1;
    const int pairs = static_cast<int>(gridDim.x) >> 1;
    const int tiles = pl.tiles_n * pl.tiles_m;
    const int start = static_cast<int>(blockIdx.x) >> 1;
    volatile int* abort_flag = &abort_s;

    if (threadIdx.x == 0) {
        for (int s = 0; s < kStages; ++s) {
            mbar_init(su32(&full_bar[s]), 1);
            mbar_init(su32(&peer_bar[s]), 1);
            mbar_init(su32(&empty_bar[s]), 1);
        }
        mbar_init(su32(&done_bar), 1);
        mbar_init(su32(&free_bar), 2 * kEpilogueWarps);
        abort_s = 0;
        mbar_fence_init();
    }
    if (warp == 1) tmem_alloc<2>(su32(&tmem_base_s), kTmemCols);
    fence_before();
    __syncthreads();
    cluster_arrive();       // the other CTA's barriers exist
    cluster_wait();
    fence_after();
    const uint32_t tmem = tmem_base_s;
    const uint32_t smem0 = su32(smem);
    asm volatile("griddepcontrol.wait;" ::: "memory");

    if (warp == 0) {
        if (elect_one()) {
            const int groups = pl.chunks / kChunksPerGroup<FORMAT>;
            const long long row_blocks_m = (static_cast<long long>(p.M) + 127) >> 7;
            const long long row_blocks_n = (static_cast<long long>(p.N) + 127) >> 7;
            int stage = 0, issued = 0;
            uint32_t phase = 0;
            bool ok = true;
            for (int t = start; t < tiles && ok; t += pairs) {
                const Tile at = tile_at(pl, t);
                // Blocks of 128 rows; one past the end reads the last again (its sums
                // are never stored).
                const long long pb = min((at.n0 >> 7) + rank, row_blocks_n - 1);
                const long long q0 = at.m0 >> 7, q1 = min(q0 + 1, row_blocks_m - 1);
                const uint8_t* pc = p.b_codes + pb * pl.chunks * 2048;
                const uint8_t* ps = p.b_scales + pb * groups * 512;
                const uint8_t* qc = p.a_codes + (rank ? q1 : q0) * pl.chunks * 2048;
                const uint8_t* qs0 = p.a_scales + q0 * groups * 512;
                const uint8_t* qs1 = p.a_scales + q1 * groups * 512;
                for (int s = 0; s < pl.slabs; ++s) {
                    if (!pipe_wait(su32(&empty_bar[stage]), phase ^ 1u, abort_flag, pl.status)) {
                        ok = false;
                        break;
                    }
                    const int c0 = s * kSlabChunks, nc = min(kSlabChunks, pl.chunks - c0);
                    const int ng = nc / kChunksPerGroup<FORMAT>;
                    const long long g0 = c0 / kChunksPerGroup<FORMAT>;
                    const uint32_t fb = su32(&full_bar[stage]);
                    const uint32_t base = smem0 + stage * kStageBytes<FORMAT>;
                    mbar_expect_tx(fb, 2 * nc * 2048 + 3 * ng * 512);
                    bulk_load(base, pc + c0 * 2048LL, nc * 2048, fb);
                    bulk_load(base + kCodes, qc + c0 * 2048LL, nc * 2048, fb);
                    const uint32_t sf = base + 2 * kCodes;
                    bulk_load(sf, ps + g0 * 512, ng * 512, fb);
                    bulk_load(sf + kSf<FORMAT>, qs0 + g0 * 512, ng * 512, fb);
                    bulk_load(sf + 2 * kSf<FORMAT>, qs1 + g0 * 512, ng * 512, fb);
                    ++issued;
                    if (++stage == kStages) {
                        stage = 0;
                        phase ^= 1u;
                    }
                }
            }
            if (!ok) {   // giving up: copies in flight land before the CTA exits
                volatile int no_abort = 0;
                for (int i = max(0, issued - kStages); i < issued; ++i)
                    pipe_wait(su32(&full_bar[i % kStages]), (i / kStages) & 1, &no_abort, nullptr);
            }
        }
    } else if (warp == 1) {
        if (elect_one()) {
            const uint64_t p_desc = operand_desc(smem0, 2048);
            const uint64_t q_desc = operand_desc(smem0 + kCodes, 2048);
            const uint64_t scales_desc = operand_desc(smem0 + 2 * kCodes, 128);
            int stage = 0;
            uint32_t phase = 0, turn = 0;
            bool ok = true;
            for (int t = start; t < tiles && ok; t += pairs) {
                // The previous tile's sums have left tensor memory (first: at once).
                if (rank == 0 &&
                    !pipe_wait(su32(&free_bar), turn ^ 1u, abort_flag, pl.status)) break;
                turn ^= 1u;
                fence_after();
                for (int s = 0; s < pl.slabs; ++s) {
                    if (!pipe_wait(su32(&full_bar[stage]), phase, abort_flag, pl.status)) {
                        ok = false;
                        break;
                    }
                    if (rank == 1) {
                        arrive_cluster(in_first_cta(su32(&peer_bar[stage])));
                    } else {
                        if (!pipe_wait(su32(&peer_bar[stage]), phase, abort_flag, pl.status)) {
                            ok = false;
                            break;
                        }
                        fence_after();
                        const int nc = min(kSlabChunks, pl.chunks - s * kSlabChunks);
                        // Descriptors count shared memory in units of 16 bytes.
                        const uint32_t at16 = stage * (kStageBytes<FORMAT> / 16);
                        const uint32_t sfp = tmem + kTile + stage * kStageCols<FORMAT>;
                        const uint32_t sfq = sfp + 4 * kSlabGroups<FORMAT>;
#pragma unroll
                        for (int g = 0; g < kSlabGroups<FORMAT>; ++g) {
                            if (g * kChunksPerGroup<FORMAT> >= nc) break;
                            copy_scales<2>(sfp + 4 * g, scales_desc + at16 + 32 * g);
                            copy_scales<2>(sfq + 8 * g,
                                           scales_desc + at16 + (kSf<FORMAT> + 512 * g) / 16);
                            copy_scales<2>(sfq + 8 * g + 4,
                                           scales_desc + at16 + (2 * kSf<FORMAT> + 512 * g) / 16);
                        }
#pragma unroll
                        for (int j = 0; j < kSlabChunks / 2; ++j) {
                            if (2 * j >= nc) break;
                            const int g = FORMAT == kNvfp4 ? j : j / 2;
                            const uint32_t id = FORMAT == kNvfp4 ? 0u : 2u * (j & 1);
                            mma<FORMAT, 2>(tmem, p_desc + at16 + j * 256, q_desc + at16 + j * 256,
                                           mx4_idesc<FORMAT>(256, kTile) | id << 4 | id << 29,
                                           sfp + 4 * g, sfq + 8 * g, s != 0 || j != 0);
                        }
                        commit<2>(su32(&empty_bar[stage]));
                    }
                    if (++stage == kStages) {
                        stage = 0;
                        phase ^= 1u;
                    }
                }
                if (rank == 0) commit<2>(su32(&done_bar));
            }
        }
    } else {
        const int quarter = warp & 3, half = (warp - 2) >> 2;
        constexpr int kCols = kTile / 2;
        float f = p.alpha;
        if (p.a_ts) f *= __ldg(p.a_ts);
        if (p.b_ts) f *= __ldg(p.b_ts);
        uint32_t turn = 0;
        for (int t = start; t < tiles; t += pairs) {
            const bool ok = __all_sync(
                0xFFFFFFFFu, pipe_wait(su32(&done_bar), turn, abort_flag, pl.status));
            if (!ok) break;
            turn ^= 1u;
            fence_after();
            const Tile at = tile_at(pl, t);
            float v[kCols / 16][16];
#pragma unroll
            for (int j = 0; j < kCols / 16; ++j)
                tmem_ld16(tmem + (static_cast<uint32_t>(32 * quarter) << 16) + half * kCols + 16 * j,
                          v[j]);
            fence_before();
            __syncwarp();
            if (lane == 0) arrive_cluster(in_first_cta(su32(&free_bar)));
            const long long n = at.n0 + 128 * rank + 32 * quarter + lane;
            const long long m0 = at.m0 + half * kCols;
            if (n < p.N) {
#pragma unroll
                for (int j = 0; j < kCols / 16; ++j)
#pragma unroll
                    for (int i = 0; i < 16; ++i)
                        if (m0 + 16 * j + i < p.M) store_c(p, f, v[j][i], m0 + 16 * j + i, n);
            }
        }
    }
    __syncwarp();
    fence_before();
    __syncthreads();
    cluster_arrive();       // the other CTA is done with this one's memory and barriers
    cluster_wait();
    asm volatile("griddepcontrol.launch_dependents;");
    if (warp == 1) {
        fence_after();
        tmem_dealloc<2>(tmem, kTmemCols);
    }
}

template <int FORMAT>
cudaError_t launch_pair(const Mx4Matmul& p, int sms, cudaStream_t stream) {
    PairPlan pl{};
    pl.p = p;
    pl.chunks = chunks_of(p.K);
    pl.slabs = (pl.chunks + kSlabChunks - 1) / kSlabChunks;
    const long long tn = (p.N + kTile - 1) / kTile, tm = (p.M + kTile - 1) / kTile;
    if (tn * tm > 0x7FFFFFFF / kGroup) return cudaErrorInvalidConfiguration;
    pl.tiles_n = static_cast<int>(tn);
    pl.tiles_m = static_cast<int>(tm);
    pl.status = status_word_ptr();
    constexpr int smem = kStages * kStageBytes<FORMAT>;
    auto kernel = mx4_pair_kernel<FORMAT>;
    cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return e;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t c{};
    c.gridDim = dim3(2 * static_cast<unsigned>(std::min<long long>(sms / 2, tn * tm)));
    c.blockDim = dim3(kThreads);
    c.dynamicSmemBytes = smem;
    c.stream = stream;
    c.attrs = at;
    c.numAttrs = 1;
    return cudaLaunchKernelEx(&c, kernel, pl);
}

}  // namespace

cudaError_t launch_mx4_pair(const Mx4Matmul& p, int sms, cudaStream_t stream) {
    return p.format == kNvfp4 ? launch_pair<kNvfp4>(p, sms, stream)
                              : launch_pair<kMxfp4>(p, sms, stream);
}

}  // namespace sgemm
