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
//   warp 1 of the first CTA: copies of scales to tensor memory and the MMAs of both CTAs.
//     Four MMAs take 512 cycles, alone or with their 12 copies of scales, and a wait on a
//     ready barrier about 100, so it waits on one a stage and asks about the next one under
//     the MMAs.
//   warp 10: that barrier, once a stage has arrived in its CTA (a bulk copy can only signal
//     a barrier of its own CTA; tensor-map copies can signal the other's, but bring the
//     same bytes at 0.6 of the rate: 212 against 129 us for the copies of 8192^3 alone).
//   warps 2..9: the epilogue, 128 lanes x 2 halves of the columns.  The 256 columns of fp32
//     sums leave no room for a second set beside the scales, so a warp first moves its
//     sums to registers, lets the next tile start, and stores them, through shared memory
//     and as whole lines, under its MMAs.
//
// Bound at 8192^3 (nvfp4 to bf16, 157 us with the operands in L2, 7.0 PFLOP/s; measured with
// parts left out when the whole took 161): 133 us with neither copies nor stores, 133 with
// both but no MMAs, 139 without copies, 145 without stores.  The tensor cores and the copies
// (38 KB a slab and SM) are about even, and each of the three costs the others some.
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

constexpr int kThreads = 352, kEpilogueWarps = 8;
constexpr int kTile = 256;
constexpr int kStages = 5;
constexpr int kGroup = 16;       // tiles of m a raster group
constexpr int kCodes = kSlabChunks * 2048;
template <int FORMAT> constexpr int kSf = kSlabGroups<FORMAT> * 512;
template <int FORMAT> constexpr int kStageBytes = 2 * kCodes + 3 * kSf<FORMAT>;
// Scale columns of a stage: four per group and 128 rows (128 of B, 256 of A).
template <int FORMAT> constexpr int kStageCols = 12 * kSlabGroups<FORMAT>;
constexpr int kTmemCols = 512;
static_assert(kTile + kStages * kStageCols<kNvfp4> <= kTmemCols, "tensor memory");
constexpr int kStageC = 2 * 32 * 128 * 4;    // staging of C: 32 rows of each half, fp32
static_assert(kStages * kStageBytes<kNvfp4> + kStageC <= 226 * 1024, "shared memory");

struct PairPlan {
    Mx4Matmul p;
    int chunks, slabs, tiles_n, tiles_m;
    int c_vec;             // 1: rows of C are 16-byte aligned
    int* status;
};

// Position in the ring of stages.
struct Ring {
    int stage = 0;
    uint32_t phase = 0;
    __device__ __forceinline__ void next() {
        if (++stage == kStages) {
            stage = 0;
            phase ^= 1u;
        }
    }
};
__device__ __forceinline__ long long slabs_of_pair(const PairPlan& pl, int start, int pairs,
                                                   int tiles) {
    return start < tiles ? ((tiles - 1 - start) / pairs + 1) * static_cast<long long>(pl.slabs) : 0;
}

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

__device__ __forceinline__ bool all_of_half(int barrier, bool ok) {
    uint32_t r;
    asm volatile(
        "{\n\t.reg .pred p, q;\n\tsetp.ne.u32 p, %2, 0;\n\t"
        "barrier.cta.red.and.pred q, %1, 128, p;\n\tselp.b32 %0, 1, 0, q;\n\t}"
        : "=r"(r) : "r"(barrier), "r"(static_cast<uint32_t>(ok)) : "memory");
    return r != 0;
}
__device__ __forceinline__ void sync_half(int barrier) {
    asm volatile("barrier.cta.sync %0, 128;" ::"r"(barrier) : "memory");
}

template <int FORMAT>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kThreads, 1)
    mx4_pair_kernel(const PairPlan pl) {
    extern __shared__ __align__(128) uint8_t smem[];
    __shared__ __align__(8) uint64_t full_bar[kStages], ready_bar[kStages], empty_bar[kStages];
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
            mbar_init(su32(&ready_bar[s]), 2);
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
            Ring ring;
            int issued = 0;
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
                    if (!pipe_wait(su32(&empty_bar[ring.stage]), ring.phase ^ 1u, abort_flag, pl.status)) {
                        ok = false;
                        break;
                    }
                    const int c0 = s * kSlabChunks, nc = min(kSlabChunks, pl.chunks - c0);
                    const int ng = nc / kChunksPerGroup<FORMAT>;
                    const long long g0 = c0 / kChunksPerGroup<FORMAT>;
                    const uint32_t fb = su32(&full_bar[ring.stage]);
                    const uint32_t base = smem0 + ring.stage * kStageBytes<FORMAT>;
                    mbar_expect_tx(fb, 2 * nc * 2048 + 3 * ng * 512);
                    bulk_load(base, pc + c0 * 2048LL, nc * 2048, fb);
                    bulk_load(base + kCodes, qc + c0 * 2048LL, nc * 2048, fb);
                    const uint32_t sf = base + 2 * kCodes;
                    bulk_load(sf, ps + g0 * 512, ng * 512, fb);
                    bulk_load(sf + kSf<FORMAT>, qs0 + g0 * 512, ng * 512, fb);
                    bulk_load(sf + 2 * kSf<FORMAT>, qs1 + g0 * 512, ng * 512, fb);
                    ++issued;
                    ring.next();
                }
            }
            if (!ok) {   // giving up: copies in flight land before the CTA exits
                volatile int no_abort = 0;
                for (int i = max(0, issued - kStages); i < issued; ++i)
                    pipe_wait(su32(&full_bar[i % kStages]), (i / kStages) & 1, &no_abort, nullptr);
            }
        }
    } else if (warp == 1) {
        if (rank == 0 && elect_one()) {
            const uint64_t p_desc = operand_desc(smem0, 2048);
            const uint64_t q_desc = operand_desc(smem0 + kCodes, 2048);
            const uint64_t scales_desc = operand_desc(smem0 + 2 * kCodes, 128);
            // A stage has arrived in both CTAs: its scales to tensor memory.
            auto take = [&](const Ring& r, bool ready) {
                if (!ready &&
                    !pipe_wait(su32(&ready_bar[r.stage]), r.phase, abort_flag, pl.status))
                    return false;
                fence_after();
                const uint64_t at = scales_desc + r.stage * (kStageBytes<FORMAT> / 16);
                const uint32_t sfp = tmem + kTile + r.stage * kStageCols<FORMAT>;
                const uint32_t sfq = sfp + 4 * kSlabGroups<FORMAT>;
#pragma unroll
                for (int g = 0; g < kSlabGroups<FORMAT>; ++g) {
                    copy_scales<2>(sfp + 4 * g, at + 32 * g);
                    copy_scales<2>(sfq + 8 * g, at + (kSf<FORMAT> + 512 * g) / 16);
                    copy_scales<2>(sfq + 8 * g + 4, at + (2 * kSf<FORMAT> + 512 * g) / 16);
                }
                return true;
            };
            auto multiply = [&](const Ring& r, int j, bool add) {
                const uint32_t at = r.stage * (kStageBytes<FORMAT> / 16);
                const uint32_t sfp = tmem + kTile + r.stage * kStageCols<FORMAT>;
                const uint32_t sfq = sfp + 4 * kSlabGroups<FORMAT>;
                // nvfp4: a group of four scales per instruction; mxfp4: two of a group.
                const int g = FORMAT == kNvfp4 ? j : j / 2;
                const uint32_t id = FORMAT == kNvfp4 ? 0u : 2u * (j & 1);
                mma<FORMAT, 2>(tmem, p_desc + at + j * 256, q_desc + at + j * 256,
                               mx4_idesc<FORMAT>(256, kTile) | id << 4 | id << 29,
                               sfp + 4 * g, sfq + 8 * g, add);
            };
            Ring ring;
            uint32_t turn = 0;
            bool ready = false, ok = true;
            for (int t = start; t < tiles && ok; t += pairs) {
                // The previous tile's sums have left tensor memory (first: at once).
                if (!pipe_wait(su32(&free_bar), turn ^ 1u, abort_flag, pl.status)) break;
                turn ^= 1u;
                for (int s = 0; s < pl.slabs; ++s) {
                    if (!take(ring, ready)) {
                        ok = false;
                        break;
                    }
                    // The answer about the next stage arrives under this one's MMAs: the
                    // thread's own time, 512 cycles a slab, is what it has least of.
                    Ring ahead = ring;
                    ahead.next();
                    ready = pipe_peek(su32(&ready_bar[ahead.stage]), ahead.phase);
                    multiply(ring, 0, s != 0);
                    multiply(ring, 1, true);
                    if (kSlabChunks * (s + 1) <= pl.chunks) {
                        multiply(ring, 2, true);
                        multiply(ring, 3, true);
                    }
                    commit<2>(su32(&empty_bar[ring.stage]));
                    ring = ahead;
                }
                commit<2>(su32(&done_bar));
            }
        }
    } else if (warp == 10) {
        if (elect_one()) {
            Ring ring;
            const long long total = slabs_of_pair(pl, start, pairs, tiles);
            for (long long i = 0; i < total; ++i, ring.next()) {
                if (!pipe_wait(su32(&full_bar[ring.stage]), ring.phase, abort_flag, pl.status))
                    break;
                arrive_cluster(in_first_cta(su32(&ready_bar[ring.stage])));
            }
        }
    } else {
        const int quarter = warp & 3, half = (warp - 2) >> 2;
        constexpr int kCols = kTile / 2;
        float f = p.alpha;
        if (p.a_ts) f *= __ldg(p.a_ts);
        if (p.b_ts) f *= __ldg(p.b_ts);
        float* const staged = reinterpret_cast<float*>(smem + kStages * kStageBytes<FORMAT> +
                                                       half * (kStageC / 2));
        uint32_t turn = 0;
        for (int t = start; t < tiles; t += pairs) {
            // All four warps of this half go on, or none.
            const bool ok = all_of_half(
                1 + half, pipe_wait(su32(&done_bar), turn, abort_flag, pl.status));
            if (!ok) break;
            turn ^= 1u;
            fence_after();
            const Tile at = tile_at(pl, t);
            float v[2][64];
            const uint32_t mine =
                tmem + (static_cast<uint32_t>(32 * quarter) << 16) + half * kCols;
            tmem_ld64(mine, v[0]);
            tmem_ld64(mine + 64, v[1]);
            fence_before();
            __syncwarp();
            if (lane == 0) arrive_cluster(in_first_cta(su32(&free_bar)));
            const long long n0 = at.n0 + 128 * rank, m0 = at.m0 + half * kCols;
            const int me = 32 * quarter + lane;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                if (m0 + 32 * j >= p.M || n0 >= p.N) break;
                sync_half(1 + half);     // the previous part has been read
#pragma unroll
                for (int i = 0; i < 32; ++i)
                    staged[i * 128 + me] = f * v[j / 2][j % 2 * 32 + i];
                sync_half(1 + half);
                const long long m = m0 + 32 * j;
                if (p.dtype == kF32) store_rows<float>(p, pl.c_vec, staged, 32, m, n0, me);
                else if (p.dtype == kBf16)
                    store_rows<__nv_bfloat16>(p, pl.c_vec, staged, 32, m, n0, me);
                else store_rows<__half>(p, pl.c_vec, staged, 32, m, n0, me);
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
    constexpr int smem = kStages * kStageBytes<FORMAT> + kStageC;
    pl.c_vec = c_rows_aligned(p);
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
