// The 4-bit product for large matrices: 256 x 256 tiles, each by a pair of CTAs.
//
// A pair of SMs runs one tcgen05.mma over both: each holds 128 of the tile's 256 rows of
// B (n) and 128 of its 256 rows of A (m), and the instruction reads the other's half of A,
// so that an SM's shared memory delivers 8 KB of codes per 128 x 256 x 64 products where a
// CTA alone would need 12 KB.  (Roles, layout and scales as in sgemm_mx4_matmul.cu.)
//
// Persistent: pair i takes the tiles i, i + pairs, ...
//   warp 0: tensor-map copies of the CTA's own halves, and of the scales: its own rows of B,
//     all 256 rows of A (the scales of the column operand are needed by both SMs).  Both CTAs'
//     copies complete on the first one's barrier, which the thread of the MMAs waits on, so
//     nothing has to be passed on between them.  (A plain bulk copy can only signal a barrier
//     of its own CTA.  A thread of the second CTA that passes it on has to release what it
//     saw: at 8192^3 296 us from one warp, 205 from three in turn, 152 this way.)
//   warp 1 of the first CTA: copies of scales to tensor memory and the MMAs of both CTAs.
//     Four MMAs take 512 cycles, alone or with their 12 copies of scales, and a wait on a
//     full barrier about 100, so it waits on one a stage and asks about the next one under
//     the MMAs.
//   warps 2..9: the epilogue, 128 lanes x 2 halves of the columns.  The 256 columns of fp32
//     sums leave no room for a second set beside the scales, so a warp first moves its
//     sums to registers, lets the next tile start, and stores them, through shared memory
//     and as whole lines, under its MMAs.
//
// 8192^3, nvfp4 to bf16, operands in L2: 151 to 157 us, 7.0 to 7.3 PFLOP/s; the MMAs alone, at 128 cycles
// each, would take 116.  2048^3 9.3 us, 4096^3 28, 3001 x 2047 x 1999 14.
#include <cuda_runtime.h>

#include <algorithm>

#include "sgemm_mx4_tc.cuh"
#include "sgemm_tma_host.h"

namespace sgemm {
namespace {

using namespace mx4;
using async::mbar_expect_tx;
using async::mbar_fence_init;
using async::mbar_init;
using async::su32;

constexpr int kThreads = 320, kEpilogueWarps = 8;
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

constexpr int kLine = 128;                   // of a tensor map, bytes

// The stored operands as lines of 128 bytes (with lines of 2048 the copies of 8192^3 alone took
// 212 us).  A parameter of its own: its address is taken, and if it were the plan's, the
// plan would be read again after every store (3001 x 2047 x 1999 19 instead of 14 us).
struct PairMaps {
    CUtensorMap a_codes, a_scales, b_codes, b_scales;
};
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

// Lines [line, line + a box) into this CTA, completing on `bar` of the first CTA.
__device__ __forceinline__ void load_lines(uint32_t dst, const CUtensorMap* tm, int line,
                                           uint32_t bar) {
    asm volatile(
        "cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.tile"
        ".mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], [%4];" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(tm)), "r"(0), "r"(line), "r"(bar)
        : "memory");
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
__device__ __forceinline__ void prefetch_map(const CUtensorMap* tm) {
    asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(tm)) : "memory");
}
// Relaxed: it announces reads of tensor memory, which the tcgen05 fence before it orders.
__device__ __forceinline__ void arrive_read(uint32_t addr) {
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
    mx4_pair_kernel(const __grid_constant__ PairMaps maps, const PairPlan pl) {
    extern __shared__ __align__(128) uint8_t smem[];
    __shared__ __align__(8) uint64_t full_bar[kStages], empty_bar[kStages];
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
            mbar_init(su32(&empty_bar[s]), 1);
        }
        mbar_init(su32(&done_bar), 1);
        mbar_init(su32(&free_bar), 2 * kEpilogueWarps);
        abort_s = 0;
        mbar_fence_init();
    }
    if (warp == 0 && lane < 4)
        prefetch_map(lane == 0 ? &maps.b_codes : lane == 1 ? &maps.a_codes
                     : lane == 2 ? &maps.b_scales : &maps.a_scales);
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
                // are never stored).  Boxes are a whole slab: past a row block's last
                // columns they bring the next one's, or zeros, which nothing multiplies.
                const long long pb = min((at.n0 >> 7) + rank, row_blocks_n - 1);
                const long long q0 = at.m0 >> 7, q1 = min(q0 + 1, row_blocks_m - 1);
                const int pl0 = static_cast<int>(pb * pl.chunks * (2048 / kLine));
                const int ql0 = static_cast<int>((rank ? q1 : q0) * pl.chunks * (2048 / kLine));
                const int ps0 = static_cast<int>(pb * groups * (512 / kLine));
                const int qs0 = static_cast<int>(q0 * groups * (512 / kLine));
                const int qs1 = static_cast<int>(q1 * groups * (512 / kLine));
                for (int s = 0; s < pl.slabs; ++s) {
                    if (!pipe_wait(su32(&empty_bar[ring.stage]), ring.phase ^ 1u, abort_flag, pl.status)) {
                        ok = false;
                        break;
                    }
                    const uint32_t fb = in_first_cta(su32(&full_bar[ring.stage]));
                    const uint32_t base = smem0 + ring.stage * kStageBytes<FORMAT>;
                    if (rank == 0) mbar_expect_tx(su32(&full_bar[ring.stage]), 2 * kStageBytes<FORMAT>);
                    const int cl = s * (kCodes / kLine), sl = s * (kSf<FORMAT> / kLine);
                    load_lines(base, &maps.b_codes, pl0 + cl, fb);
                    load_lines(base + kCodes, &maps.a_codes, ql0 + cl, fb);
                    const uint32_t sf = base + 2 * kCodes;
                    load_lines(sf, &maps.b_scales, ps0 + sl, fb);
                    load_lines(sf + kSf<FORMAT>, &maps.a_scales, qs0 + sl, fb);
                    load_lines(sf + 2 * kSf<FORMAT>, &maps.a_scales, qs1 + sl, fb);
                    ++issued;
                    ring.next();
                }
            }
            // Copies in flight land before the pair exits, whichever wait gave up.  They signal
            // the first CTA, so it waits for both; what the second may have asked for beyond
            // that had the time limit of the wait that gave up.
            if (rank == 0) {
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
                    !pipe_wait<true>(su32(&full_bar[r.stage]), r.phase, abort_flag, pl.status))
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
                if (!pipe_wait<true>(su32(&free_bar), turn ^ 1u, abort_flag, pl.status)) break;
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
                    ready = pipe_peek(su32(&full_bar[ahead.stage]), ahead.phase);
                    multiply(ring, 0, s != 0);
                    multiply(ring, 1, true);
                    if (kSlabChunks * (s + 1) <= pl.chunks) {
                        multiply(ring, 2, true);
                        multiply(ring, 3, true);
                    }
                    commit<2>(su32(&empty_bar[ring.stage]));
                    ring = ahead;
                }
                if (ok) commit<2>(su32(&done_bar));      // else both epilogues give up
            }
        }
    } else {
        const int quarter = warp & 3, half = (warp - 2) >> 2;
        constexpr int kCols = kTile / 2;
        float f = p.alpha;
        if (p.a_ts) f *= fetch(p.a_ts);
        if (p.b_ts) f *= fetch(p.b_ts);
        float* const staged = reinterpret_cast<float*>(smem + kStages * kStageBytes<FORMAT> +
                                                       half * (kStageC / 2));
        uint32_t turn = 0;
        for (int t = start; t < tiles; t += pairs) {
            // All four warps of this half go on, or none.
            const bool ok = all_of_half(
                1 + half, pipe_wait(su32(&done_bar), turn, abort_flag, pl.status) && !*abort_flag);
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
            if (lane == 0) arrive_read(in_first_cta(su32(&free_bar)));
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

// `bytes` bytes (whole lines) in boxes of `box` bytes.
bool encode_lines(CUtensorMap* tm, const void* base, long long bytes, int box) {
    auto fn = tensor_map_encoder();
    if (!fn) return false;
    cuuint64_t dims[2] = {kLine, static_cast<cuuint64_t>(bytes / kLine)};
    cuuint64_t strides[1] = {kLine};
    cuuint32_t boxes[2] = {kLine, static_cast<cuuint32_t>(box / kLine)};
    cuuint32_t steps[2] = {1, 1};
    return fn(tm, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<void*>(base), dims, strides, boxes,
              steps, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_NONE,
              CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) ==
           CUDA_SUCCESS;
}

template <int FORMAT>
cudaError_t launch_pair(const Mx4Matmul& p, int sms, cudaStream_t stream) {
    PairPlan pl{};
    PairMaps maps;
    pl.p = p;
    pl.chunks = chunks_of(p.K);
    pl.slabs = (pl.chunks + kSlabChunks - 1) / kSlabChunks;
    const long long tn = (p.N + kTile - 1) / kTile, tm = (p.M + kTile - 1) / kTile;
    if (tn * tm > 0x7FFFFFFF / kGroup) return cudaErrorInvalidConfiguration;
    pl.tiles_n = static_cast<int>(tn);
    pl.tiles_m = static_cast<int>(tm);
    pl.status = status_word_ptr();
    // At least two row blocks of four chunks each, so no box is larger than its matrix.
    const long long ca = row_blocks(p.M) * pl.chunks * 2048, cb = row_blocks(p.N) * pl.chunks * 2048;
    constexpr int per = 2048 * kChunksPerGroup<FORMAT> / 512;      // code bytes a scale byte
    if (std::max(ca, cb) / kLine > 0x7FFFFFFF) return cudaErrorInvalidValue;
    if (!encode_lines(&maps.a_codes, p.a_codes, ca, kCodes) ||
        !encode_lines(&maps.b_codes, p.b_codes, cb, kCodes) ||
        !encode_lines(&maps.a_scales, p.a_scales, ca / per, kSf<FORMAT>) ||
        !encode_lines(&maps.b_scales, p.b_scales, cb / per, kSf<FORMAT>))
        return cudaErrorInvalidValue;
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
    return cudaLaunchKernelEx(&c, kernel, maps, pl);
}

}  // namespace

cudaError_t launch_mx4_pair(const Mx4Matmul& p, int sms, cudaStream_t stream) {
    return p.format == kNvfp4 ? launch_pair<kNvfp4>(p, sms, stream)
                              : launch_pair<kMxfp4>(p, sms, stream);
}

}  // namespace sgemm
