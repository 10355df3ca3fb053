// Product of two 4-bit matrices: C = f * A . B^T + beta * C with f = alpha * ta * tb
// (sgemm_mx4_matmul), on the tensor cores' block-scaled 4-bit form.
//
// tcgen05.mma kind::mxf4nvf4 multiplies 64 columns of codes at a time, each block of 16
// (nvfp4) or 32 (mxfp4) scaled by the product of its two scales, and adds to fp32 sums
// in tensor memory.  The weight B (N rows) is the instruction's 128-row operand and the
// activations A (M rows) its column operand, so that a lane of tensor memory holds one
// column n of C: the 32 lanes of a warp then store 32 neighbours of one row of C, at any
// alignment, and few rows of A cost a narrow instruction instead of empty lanes.
//
// One CTA computes a 128 (n) x BQ (m) tile, or its share of the tile's K range: the CTAs
// of a cluster take consecutive ranges and sum their parts in distributed shared memory
// in rank order, so the result does not depend on timing.
//   warp 0, one thread: bulk copies of slabs 256 columns deep into a ring.  The stored
//     layout is already the operand layout (no swizzle), so a slab is one copy per
//     operand and one for its scales.
//   warp 1, one thread: tcgen05.cp of the scales to tensor memory, then four MMAs a slab.
//     Each stage has its own scale columns: they are overwritten only after the stage's
//     MMAs have completed, as its shared memory is.
//   all four warps: the epilogue, one lane of tensor memory per thread.
// Every wait is bounded; one that gives up sets the device status word and the CTA
// drains, meets its cluster's barriers and exits.
//
// Few rows of A are bound by the weight's bytes where it is large (nvfp4 to bf16, the kernel
// alone, 1 x 16384 x 16384: 24.4 us, 6.2 TB/s) and by latency where it is small (1 x 4096 x 4096:
// 5.3 us, whose 9.4 MB would take 1.4; one CTA an SM, issue slots 6 % used; 16 x 8192 x 4096 7.1).
// 512 x 4096 x 4096 takes 8.8 us, 16384 x 64 x 4096 (mxfp4 to fp32) 7.8 to 8.9.
#include <cuda_runtime.h>

#include <algorithm>
#include <type_traits>

#include "sgemm_mx4_tc.cuh"

namespace sgemm {
namespace {

using namespace mx4;
using async::mbar_expect_tx;
using async::mbar_fence_init;
using async::mbar_init;
using async::su32;

constexpr int kMaxStages = 8;
constexpr int kGroup = 8;

struct MatmulPlan {
    Mx4Matmul p;
    int chunks, slabs, stages, split, tmem_cols, tiles_n, tiles_m, c_vec;
    int* status;
};

// Shared memory of a stage: codes of both operands, then their scales.
template <int FORMAT, int BQ> constexpr int kStageBytes =
    kSlabChunks * (2048 + BQ * 16) + 2 * kSlabGroups<FORMAT> * 512;
// Tensor-memory columns of a stage's scales: four per 128 rows and group.
template <int FORMAT> constexpr int kStageCols = 8 * kSlabGroups<FORMAT>;

// Shared memory of the cluster's CTA `rank` at this CTA's address `at`.
__device__ __forceinline__ uint32_t cluster_address(uint32_t at, int rank) {
    uint32_t r;
    asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(at), "r"(rank));
    return r;
}
__device__ __forceinline__ float4 cluster_load4(uint32_t at, int rank) {
    float4 v;
    asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
                 : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
                 : "r"(cluster_address(at, rank)) : "memory");
    return v;
}
__device__ __forceinline__ float2 cluster_load2(uint32_t at, int rank) {
    float2 v;
    asm volatile("ld.shared::cluster.v2.f32 {%0, %1}, [%2];"
                 : "=f"(v.x), "=f"(v.y) : "r"(cluster_address(at, rank)) : "memory");
    return v;
}

// grid: tiles x split CTAs; clusters of split.
template <int FORMAT, int BQ>
__global__ void __launch_bounds__(128) mx4_matmul_kernel(const MatmulPlan pl) {
    constexpr int kP = kSlabChunks * 2048, kQ = kSlabChunks * BQ * 16;
    constexpr int kSf = kSlabGroups<FORMAT> * 512;
    extern __shared__ __align__(128) uint8_t smem[];
    __shared__ __align__(8) uint64_t full_bar[kMaxStages], empty_bar[kMaxStages], done_bar;
    __shared__ uint32_t tmem_base_s;
    __shared__ int abort_s, issued_s;
    const Mx4Matmul& p = pl.p;
    const int warp = warp_index();
    const int rank = static_cast<int>(blockIdx.x) % pl.split;
    // Tiles run along m in groups of kGroup, then along n, so that the CTAs at work at
    // one time share few operand rows.
    const int tile = static_cast<int>(blockIdx.x) / pl.split;
    const int group = tile / (kGroup * pl.tiles_n), in = tile - group * kGroup * pl.tiles_n;
    const int high = min(kGroup, pl.tiles_m - group * kGroup);
    const long long n0 = in / high * 128LL;
    const long long m0 = static_cast<long long>(group * kGroup + in % high) * BQ;
    const int first = static_cast<int>(static_cast<long long>(pl.slabs) * rank / pl.split);
    const int last = static_cast<int>(static_cast<long long>(pl.slabs) * (rank + 1) / pl.split);
    volatile int* abort_flag = &abort_s;

    if (threadIdx.x == 0) {
        for (int s = 0; s < pl.stages; ++s) {
            mbar_init(su32(&full_bar[s]), 1);
            mbar_init(su32(&empty_bar[s]), 1);
        }
        mbar_init(su32(&done_bar), 1);
        abort_s = 0;
        mbar_fence_init();
    }
    if (warp == 1) tmem_alloc<1>(su32(&tmem_base_s), pl.tmem_cols);
    fence_before();
    __syncthreads();
    fence_after();
    const uint32_t tmem = tmem_base_s;
    const uint32_t smem0 = su32(smem);
    asm volatile("griddepcontrol.wait;" ::: "memory");

    if (warp == 0) {
        if (elect_one()) {
            const int groups = pl.chunks / kChunksPerGroup<FORMAT>;
            const uint8_t* pc = p.b_codes + (n0 >> 7) * pl.chunks * 2048;
            const uint8_t* ps = p.b_scales + (n0 >> 7) * groups * 512;
            const uint8_t* qc = p.a_codes + (m0 >> 7) * pl.chunks * 2048 + (m0 & 127) * 16;
            const uint8_t* qs = p.a_scales + (m0 >> 7) * groups * 512;
            int stage = 0;
            uint32_t phase = 0;
            int issued = 0;
            for (int s = first; s < last; ++s) {
                if (!pipe_wait(su32(&empty_bar[stage]), phase ^ 1u, abort_flag, pl.status)) break;
                const int c0 = s * kSlabChunks, nc = min(kSlabChunks, pl.chunks - c0);
                const int ng = nc / kChunksPerGroup<FORMAT>, g0 = c0 / kChunksPerGroup<FORMAT>;
                const uint32_t fb = su32(&full_bar[stage]);
                const uint32_t base = smem0 + stage * kStageBytes<FORMAT, BQ>;
                mbar_expect_tx(fb, nc * (2048 + BQ * 16) + 2 * ng * 512);
                bulk_load(base, pc + c0 * 2048LL, nc * 2048, fb);
                bulk_load(base + kP + kQ, ps + g0 * 512LL, ng * 512, fb);
                if (BQ == 128) {
                    bulk_load(base + kP, qc + c0 * 2048LL, nc * 2048, fb);
                } else {
                    for (int c = 0; c < nc; ++c)
                        bulk_load(base + kP + c * BQ * 16, qc + (c0 + c) * 2048LL, BQ * 16, fb);
                }
                bulk_load(base + kP + kQ + kSf, qs + g0 * 512LL, ng * 512, fb);
                ++issued;
                if (++stage == pl.stages) {
                    stage = 0;
                    phase ^= 1u;
                }
            }
            issued_s = issued;
        }
    } else if (warp == 1) {
        if (elect_one()) {
            const uint64_t p_desc = operand_desc(smem0, 2048);
            const uint64_t q_desc = operand_desc(smem0 + kP, BQ * 16);
            const uint64_t scales_desc = operand_desc(smem0 + kP + kQ, 128);
            // A's scales come 128 rows at a time, 32 to a column.
            const uint32_t q_col = static_cast<uint32_t>(m0 & 127) >> 5;
            int stage = 0;
            uint32_t phase = 0;
            for (int s = first; s < last; ++s) {
                if (!pipe_wait(su32(&full_bar[stage]), phase, abort_flag, pl.status)) break;
                fence_after();
                const int nc = min(kSlabChunks, pl.chunks - s * kSlabChunks);
                // Descriptors count shared memory in units of 16 bytes.
                const uint32_t at = stage * (kStageBytes<FORMAT, BQ> / 16);
                const uint32_t sfp = tmem + BQ + stage * kStageCols<FORMAT>;
                const uint32_t sfq = sfp + kStageCols<FORMAT> / 2;
#pragma unroll
                for (int g = 0; g < kSlabGroups<FORMAT>; ++g) {
                    if (g * kChunksPerGroup<FORMAT> >= nc) break;
                    copy_scales<1>(sfp + 4 * g, scales_desc + at + 32 * g);
                    copy_scales<1>(sfq + 4 * g, scales_desc + at + (kSf + 512 * g) / 16);
                }
#pragma unroll
                for (int j = 0; j < kSlabChunks / 2; ++j) {
                    if (2 * j >= nc) break;
                    // nvfp4: a group of four scales per instruction; mxfp4: two of a group.
                    const int g = FORMAT == kNvfp4 ? j : j / 2;
                    const uint32_t id = FORMAT == kNvfp4 ? 0u : 2u * (j & 1);
                    mma<FORMAT, 1>(tmem, p_desc + at + j * 256, q_desc + at + j * 2 * BQ,
                                   mx4_idesc<FORMAT>(128, BQ) | id << 4 | id << 29, sfp + 4 * g,
                                   sfq + 4 * g + q_col, s != first || j != 0);
                }
                commit<1>(su32(&empty_bar[stage]));
                if (++stage == pl.stages) {
                    stage = 0;
                    phase ^= 1u;
                }
            }
            commit<1>(su32(&done_bar));
        }
    }
    __syncwarp();
    // (Sums that a wait gave up on are committed as well, but not stored.)
    const bool ok = __all_sync(0xFFFFFFFFu,
                               pipe_wait(su32(&done_bar), 0, abort_flag, pl.status) && !*abort_flag);
    if (!ok && warp == 0 && elect_one()) {
        // Copies in flight land before the CTA exits, whichever of its waits gave up.
        volatile int no_abort = 0;
        for (int i = max(0, issued_s - pl.stages); i < issued_s; ++i)
            pipe_wait(su32(&full_bar[i % pl.stages]), (i / pl.stages) & 1, &no_abort, nullptr);
    }
    __syncwarp();
    fence_after();
    float f = p.alpha;
    if (p.a_ts) f *= __ldg(p.a_ts);
    if (p.b_ts) f *= __ldg(p.b_ts);
    const long long n = n0 + threadIdx.x;
    const uint32_t mine = tmem + (static_cast<uint32_t>(32 * warp) << 16);
    // Sums go through shared memory: to the cluster, or (where the ring was: every MMA has
    // read its stage) to whole lines of C.
    float* const part = reinterpret_cast<float*>(smem + pl.stages * kStageBytes<FORMAT, BQ>);
    float* const staged = reinterpret_cast<float*>(smem);
#pragma unroll 1
    for (int j = 0; j < BQ && m0 + j < p.M; j += 16) {
        float v[16];
        __syncwarp();
        tmem_ld16(mine + j, v);
        if (pl.split > 1) {
#pragma unroll
            for (int i = 0; i < 16; i += 4)
                *reinterpret_cast<float4*>(part + ((j + i) * 128 + 4 * threadIdx.x)) =
                    make_float4(v[i], v[i + 1], v[i + 2], v[i + 3]);
        } else {
#pragma unroll
            for (int i = 0; i < 16; ++i) staged[(j + i) * 128 + threadIdx.x] = f * v[i];
        }
    }
    // Tensor memory goes back before the cluster is waited for: a CTA that holds some
    // while it waits for one that waits for some would end neither.
    fence_before();
    __syncthreads();
    if (warp == 1) {
        fence_after();
        tmem_dealloc<1>(tmem, pl.tmem_cols);
    }
    if (pl.split == 1) {
        if (ok) {
            if (p.dtype == kF32) store_rows<float>(p, pl.c_vec, staged, BQ, m0, n0, threadIdx.x);
            else if (p.dtype == kBf16)
                store_rows<__nv_bfloat16>(p, pl.c_vec, staged, BQ, m0, n0, threadIdx.x);
            else store_rows<__half>(p, pl.c_vec, staged, BQ, m0, n0, threadIdx.x);
        }
    } else {
        cluster_arrive();
        cluster_wait();
        // Rank r sums columns [r, r + 1) * own of the tile, four (or the two that it has) of
        // a lane at a time: parts lie as [columns / 4][128 lanes][4].
        const int own = BQ / pl.split, left = static_cast<int>(min(p.M - m0, BQ + 0LL));
        const uint32_t red = su32(part) + 16 * threadIdx.x;
        const int end = min((rank + 1) * own, left);
        if (own >= 4) {
            const auto sum = [&](auto split) {
                constexpr int kSplit = decltype(split)::value;
                constexpr int kOwn = BQ / kSplit, kStep = kOwn < 16 ? kOwn : 16;
#pragma unroll 1
                for (int c = rank * kOwn; c < end; c += kStep) {
                    // All parts of 16 columns at once: a load takes the cluster's latency.
                    float4 v[kSplit][kStep / 4];
#pragma unroll
                    for (int r = 0; r < kSplit; ++r)
#pragma unroll
                        for (int i = 0; i < kStep / 4; ++i)
                            v[r][i] = cluster_load4(red + (c + 4 * i) * 512, r);
#pragma unroll
                    for (int i = 0; i < kStep / 4; ++i) {
#pragma unroll
                        for (int r = 1; r < kSplit; ++r) {
                            v[0][i].x += v[r][i].x; v[0][i].y += v[r][i].y;
                            v[0][i].z += v[r][i].z; v[0][i].w += v[r][i].w;
                        }
                        if (!ok || n >= p.N) continue;
                        const int m = c + 4 * i;
                        if (m < end) store_c(p, f, v[0][i].x, m0 + m, n);
                        if (m + 1 < end) store_c(p, f, v[0][i].y, m0 + m + 1, n);
                        if (m + 2 < end) store_c(p, f, v[0][i].z, m0 + m + 2, n);
                        if (m + 3 < end) store_c(p, f, v[0][i].w, m0 + m + 3, n);
                    }
                }
            };
            if (pl.split == 2) sum(std::integral_constant<int, 2>());
            else if (pl.split == 4) sum(std::integral_constant<int, 4>());
            else if constexpr (BQ >= 32) sum(std::integral_constant<int, 8>());
        } else if (rank * own < end) {
            const int c = rank * own;
            float2 acc = make_float2(0, 0);
            for (int r = 0; r < pl.split; ++r) {
                const float2 v = cluster_load2(red + (c & ~3) * 512 + (c & 3) * 4, r);
                acc.x += v.x; acc.y += v.y;
            }
            if (ok && n < p.N) {
                store_c(p, f, acc.x, m0 + c, n);
                if (c + 1 < left) store_c(p, f, acc.y, m0 + c + 1, n);
            }
        }
        cluster_arrive();                  // its parts stay until the others have read them
        cluster_wait();
    }
    asm volatile("griddepcontrol.launch_dependents;");
}

// C = beta * C where there is nothing to multiply (K == 0 or alpha == 0).
__global__ void __launch_bounds__(256) mx4_scale_kernel(const Mx4Matmul p) {
    const long long total = static_cast<long long>(p.M) * p.N;
    for (long long e = blockIdx.x * 256LL + threadIdx.x; e < total; e += gridDim.x * 256LL)
        store_c(p, 0.0f, 0.0f, e / p.N, e % p.N);
}

template <int FORMAT, int BQ>
cudaError_t launch_tile(const Mx4Matmul& p, int split, cudaStream_t stream) {
    MatmulPlan pl{};
    pl.p = p;
    pl.chunks = chunks_of(p.K);
    pl.slabs = (pl.chunks + kSlabChunks - 1) / kSlabChunks;
    const long long tiles_n = (p.N + 127) / 128, tiles_m = (p.M + BQ - 1) / BQ;
    const long long tiles = tiles_n * tiles_m;
    if (tiles > 0x7FFFFFFF / kGroup) return cudaErrorInvalidConfiguration;
    pl.tiles_n = static_cast<int>(tiles_n);
    pl.tiles_m = static_cast<int>(tiles_m);
    pl.split = split;
    pl.c_vec = c_rows_aligned(p);
    constexpr int kMost = 220 * 1024;
    const int red = pl.split > 1 ? BQ * 512 : 0;
    const int per = (pl.slabs + pl.split - 1) / pl.split;
    pl.stages = std::min({per, kMaxStages, (kMost - red) / kStageBytes<FORMAT, BQ>});
    const int cols = BQ + pl.stages * kStageCols<FORMAT>;
    pl.tmem_cols = 32;
    while (pl.tmem_cols < cols) pl.tmem_cols *= 2;
    // No more CTAs to an SM, by their shared memory, than find tensor memory there.
    const int resident = 512 / pl.tmem_cols;
    const int least = 228 * 1024 / (resident + 1);
    const int smem = std::max(std::max(pl.stages * kStageBytes<FORMAT, BQ> + red, BQ * 512),
                              resident == 1 ? 116 * 1024 : least);
    pl.status = status_word_ptr();
    auto kernel = mx4_matmul_kernel<FORMAT, BQ>;
    cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                         kMost);
    if (e != cudaSuccess) return e;
    cudaLaunchAttribute at[2];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    at[1].id = cudaLaunchAttributeClusterDimension;
    at[1].val.clusterDim.x = static_cast<unsigned>(pl.split);
    at[1].val.clusterDim.y = at[1].val.clusterDim.z = 1;
    cudaLaunchConfig_t c{};
    c.gridDim = dim3(static_cast<unsigned>(tiles * pl.split));
    c.blockDim = dim3(128);
    c.dynamicSmemBytes = static_cast<size_t>(smem);
    c.stream = stream;
    c.attrs = at;
    c.numAttrs = 2;
    return cudaLaunchKernelEx(&c, kernel, pl);
}

template <int FORMAT>
cudaError_t launch_format(const Mx4Matmul& p, int sms, cudaStream_t stream) {
    const Mx4Choice c = choose_mx4(p.M, p.N, p.K, sms);
    switch (c.tile) {
        case 16: return launch_tile<FORMAT, 16>(p, c.split, stream);
        case 32: return launch_tile<FORMAT, 32>(p, c.split, stream);
        case 64: return launch_tile<FORMAT, 64>(p, c.split, stream);
        case 128: return launch_tile<FORMAT, 128>(p, c.split, stream);
        default: return launch_mx4_pair(p, sms, stream);
    }
}

}  // namespace

// Few rows of A take the narrowest tile that holds them.  More take 64 columns where such
// tiles fit the SMs at once, else 128, and the pairs' 256 x 256 where those do not either
// (us, the kernel alone, 512 x 4096 x 4096: 64 wide 16.5, 128 8.8, pairs 11.0; 2048^3: 64 wide
// 22.8, 128 13.1, pairs 9.3).  Pairs would waste half of a tile on an operand of up to 128 rows.
//
// A K range is split while the CTAs still fit the SMs at once and each keeps four slabs.
// Two parts of a 64-wide tile, or any of a 128-wide one, cost more to add up than a range
// of less than 8192 saves (64 x 4096 x 4096: 1 part 8.3 us, 2 9.6, 4 7.5;
// 256 x 1024 x 8192: 1 part 13.0, 2 11.9, 4 8.9).
Mx4Choice choose_mx4(int M, int N, int K, int sms) {
    const long long tn = (N + 127LL) / 128;
    const int slabs = (chunks_of(K) + kSlabChunks - 1) / kSlabChunks;
    Mx4Choice c{128, 1};
    if (M <= 16) c.tile = 16;
    else if (M <= 32) c.tile = 32;
    else if (M <= 64 || tn * ((M + 63LL) / 64) <= sms) c.tile = 64;
    else if (tn * ((M + 127LL) / 128) > sms && M > 128 && N > 128) c.tile = 256;
    if (c.tile > 64) return c;
    const long long tiles = tn * ((M + c.tile - 1LL) / c.tile);
    for (int split = 2; split <= 8; split *= 2)
        if ((c.tile < 64 || split > 2 || slabs >= 32) && tiles * split <= sms && slabs >= 4 * split)
            c.split = split;
    return c;
}

cudaError_t launch_mx4_matmul(const Mx4Matmul& p, int sms, cudaStream_t stream) {
    if (p.K == 0) {
        const long long blocks = (static_cast<long long>(p.M) * p.N + 255) / 256;
        mx4_scale_kernel<<<static_cast<unsigned>(std::min<long long>(blocks, 8LL * sms)), 256, 0,
                           stream>>>(p);
        return cudaGetLastError();
    }
    return p.format == kNvfp4 ? launch_format<kNvfp4>(p, sms, stream)
                              : launch_format<kMxfp4>(p, sms, stream);
}

}  // namespace sgemm
