// Tensor-core and bulk-copy wrappers of the 4-bit product's kernels (G: CTAs of one MMA).
#pragma once

#include "sgemm_async.cuh"
#include "sgemm_internal.h"
#include "sgemm_mx4.cuh"

namespace sgemm {
namespace mx4 {

constexpr int kSlabChunks = 8;    // a slab: 256 columns of the operands
template <int FORMAT> constexpr int kChunksPerGroup = FORMAT == kNvfp4 ? 2 : 4;
template <int FORMAT> constexpr int kSlabGroups = kSlabChunks / kChunksPerGroup<FORMAT>;

// As async::mbar_wait, with its time limit, but the thread sleeps in the hardware until
// the phase completes or kSleepNs have passed: polls and reads of the global timer by the
// waiting warps slow down the two threads that feed the tensor cores.
constexpr unsigned kSleepNs = 1000000;
// CLUSTER: other CTAs of the cluster take part in the phase, so the wait acquires at their scope.
template <bool CLUSTER = false>
__device__ __forceinline__ bool pipe_try(uint32_t bar, uint32_t parity) {
    uint32_t ok;
    if constexpr (CLUSTER)
        asm volatile(
            "{\n\t.reg .pred p;\n\t"
            "mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2, %3;\n\t"
            "selp.b32 %0, 1, 0, p;\n\t}"
            : "=r"(ok)
            : "r"(bar), "r"(parity), "r"(kSleepNs)
            : "memory");
    else
        asm volatile(
            "{\n\t.reg .pred p;\n\t"
            "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, %3;\n\t"
            "selp.b32 %0, 1, 0, p;\n\t}"
            : "=r"(ok)
            : "r"(bar), "r"(parity), "r"(kSleepNs)
            : "memory");
    return ok != 0;
}
// Whether the phase has completed, without sleeping (at the cluster's scope).
__device__ __forceinline__ bool pipe_peek(uint32_t bar, uint32_t parity) {
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.test_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2;\n\t"
        "selp.b32 %0, 1, 0, p;\n\t}"
        : "=r"(ok)
        : "r"(bar), "r"(parity)
        : "memory");
    return ok != 0;
}
template <bool CLUSTER = false>
__device__ __forceinline__ bool pipe_wait(uint32_t bar, uint32_t parity, volatile int* abort,
                                          int* status) {
    if (pipe_try<CLUSTER>(bar, parity)) return true;
    const unsigned long long t0 = async::gtimer();
    for (unsigned i = 0; i < async::kMaxSpins; ++i) {
        if (pipe_try<CLUSTER>(bar, parity)) return true;
        if (*abort) return false;
        if (async::gtimer() - t0 > async::kWaitNs) break;
    }
    if (status) atomicExch(status, async::kStatusWaitTimeout);
    *abort = 1;
    return false;
}

// True in one thread of the (whole) warp.  Unlike a test of the lane number it tells the
// compiler that one thread runs what follows, whose tensor-core instructions take their
// operands from uniform registers: without it each is wrapped in a loop over the lanes
// (measured per instruction: 47 against 10 cycles for a copy of scales).
__device__ __forceinline__ bool elect_one() {
    uint32_t r;
    asm volatile(
        "{\n\t.reg .pred q;\n\telect.sync _|q, 0xffffffff;\n\tselp.b32 %0, 1, 0, q;\n\t}"
        : "=r"(r));
    return r != 0;
}
__device__ __forceinline__ int warp_index() {
    return __shfl_sync(0xFFFFFFFFu, static_cast<int>(threadIdx.x >> 5), 0);
}

// Shared-memory operand without swizzle: 8 rows x 16 bytes contiguous, `lead` bytes from
// one 16-byte column to the next, 128 bytes from one group of 8 rows to the next.
__device__ __forceinline__ uint64_t operand_desc(uint32_t saddr, uint32_t lead) {
    uint64_t d = 0;
    d |= static_cast<uint64_t>((saddr >> 4) & 0x3FFFu);
    d |= static_cast<uint64_t>((lead >> 4) & 0x3FFFu) << 16;
    d |= static_cast<uint64_t>(128 >> 4) << 32;
    d |= static_cast<uint64_t>(1) << 46;                      // descriptor version
    return d;
}
// Instruction: e2m1 x e2m1, K = 64, M rows by N columns; the scales' type.
template <int FORMAT>
__host__ __device__ constexpr uint32_t mx4_idesc(int M, int N) {
    return (1u << 7) | (1u << 10) | (static_cast<uint32_t>(N >> 3) << 17) |
           (FORMAT == kMxfp4 ? 1u << 23 : 0u) | (static_cast<uint32_t>(M >> 4) << 24);
}
#define SGEMM_MX4_MMA(GROUP, VEC)                                                          \
    asm volatile(                                                                          \
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %6, 0;\n\t"                                   \
        "tcgen05.mma.cta_group::" GROUP ".kind::mxf4nvf4.block_scale.scale_vec::" VEC " "  \
        "[%0], %1, %2, %3, [%4], [%5], p;\n\t}" ::"r"(d), "l"(a), "l"(b), "r"(idesc),      \
        "r"(sfa), "r"(sfb), "r"(accumulate) : "memory")
template <int FORMAT, int G>
__device__ __forceinline__ void mma(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc,
                                    uint32_t sfa, uint32_t sfb, uint32_t accumulate) {
    if constexpr (FORMAT == kNvfp4 && G == 1) SGEMM_MX4_MMA("1", "4X");
    if constexpr (FORMAT == kNvfp4 && G == 2) SGEMM_MX4_MMA("2", "4X");
    if constexpr (FORMAT == kMxfp4 && G == 1) SGEMM_MX4_MMA("1", "2X");
    if constexpr (FORMAT == kMxfp4 && G == 2) SGEMM_MX4_MMA("2", "2X");
}
#undef SGEMM_MX4_MMA
// 512 bytes of scales (128 rows, four blocks) to four tensor-memory columns of each lane
// quarter; with G == 2 in both CTAs, each from its own shared memory.
template <int G>
__device__ __forceinline__ void copy_scales(uint32_t tmem, uint64_t desc) {
    if constexpr (G == 1)
        asm volatile("tcgen05.cp.cta_group::1.32x128b.warpx4 [%0], %1;" ::"r"(tmem), "l"(desc)
                     : "memory");
    else
        asm volatile("tcgen05.cp.cta_group::2.32x128b.warpx4 [%0], %1;" ::"r"(tmem), "l"(desc)
                     : "memory");
}
// Arrives on `bar` (of both CTAs with G == 2) when the MMAs issued so far have completed.
template <int G>
__device__ __forceinline__ void commit(uint32_t bar) {
    if constexpr (G == 1)
        asm volatile(
            "tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(bar)
            : "memory");
    else
        asm volatile(
            "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster"
            ".multicast::cluster.b64 [%0], %1;" ::"r"(bar), "h"(static_cast<uint16_t>(3))
            : "memory");
}
template <int G>
__device__ __forceinline__ void tmem_alloc(uint32_t result, int cols) {
    if constexpr (G == 1) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                         result), "r"(cols) : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    } else {
        asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                         result), "r"(cols) : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
    }
}
template <int G>
__device__ __forceinline__ void tmem_dealloc(uint32_t tmem, int cols) {
    if constexpr (G == 1)
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(cols)
                     : "memory");
    else
        asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(cols)
                     : "memory");
}
__device__ __forceinline__ void bulk_load(uint32_t dst, const void* src, uint32_t bytes,
                                          uint32_t bar) {
    asm volatile(
        "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::
            "r"(dst), "l"(reinterpret_cast<uint64_t>(src)), "r"(bytes), "r"(bar)
        : "memory");
}
__device__ __forceinline__ void tmem_ld16(uint32_t taddr, float (&v)[16]) {
    uint32_t r[16];
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
        "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
          "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]),
          "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
        : "r"(taddr));
    asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
#pragma unroll
    for (int i = 0; i < 16; ++i) v[i] = __uint_as_float(r[i]);
}
// 64 columns with one wait.
__device__ __forceinline__ void tmem_ld64(uint32_t taddr, float (&v)[64]) {
    uint32_t r[64];
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x64.b32 "
        "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16, "
        "%17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31, "
        "%32, %33, %34, %35, %36, %37, %38, %39, %40, %41, %42, %43, %44, %45, %46, "
        "%47, %48, %49, %50, %51, %52, %53, %54, %55, %56, %57, %58, %59, %60, %61, "
        "%62, %63}, [%64];"
        "\n\ttcgen05.wait::ld.sync.aligned;"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]),
          "=r"(r[6]), "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]),
          "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]), "=r"(r[17]),
          "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]),
          "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]),
          "=r"(r[30]), "=r"(r[31]), "=r"(r[32]), "=r"(r[33]), "=r"(r[34]), "=r"(r[35]),
          "=r"(r[36]), "=r"(r[37]), "=r"(r[38]), "=r"(r[39]), "=r"(r[40]), "=r"(r[41]),
          "=r"(r[42]), "=r"(r[43]), "=r"(r[44]), "=r"(r[45]), "=r"(r[46]), "=r"(r[47]),
          "=r"(r[48]), "=r"(r[49]), "=r"(r[50]), "=r"(r[51]), "=r"(r[52]), "=r"(r[53]),
          "=r"(r[54]), "=r"(r[55]), "=r"(r[56]), "=r"(r[57]), "=r"(r[58]), "=r"(r[59]),
          "=r"(r[60]), "=r"(r[61]), "=r"(r[62]), "=r"(r[63])
        : "r"(taddr) : "memory");
#pragma unroll
    for (int i = 0; i < 64; ++i) v[i] = __uint_as_float(r[i]);
}
__device__ __forceinline__ void fence_before() {
    asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
}
__device__ __forceinline__ void fence_after() {
    asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
}
__device__ __forceinline__ void cluster_arrive() {
    asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
}
__device__ __forceinline__ void cluster_wait() {
    asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}

__device__ __forceinline__ void store_c(const Mx4Matmul& p, float f, float acc, long long m,
                                        long long n) {
    const long long at = m * p.ldc + n;
    if (p.dtype == kF32) {
        float* c = static_cast<float*>(p.C) + at;
        *c = p.beta == 0.0f ? f * acc : fmaf(f, acc, p.beta * *c);
    } else if (p.dtype == kBf16) {
        __nv_bfloat16* c = static_cast<__nv_bfloat16*>(p.C) + at;
        *c = from_float<__nv_bfloat16>(p.beta == 0.0f ? f * acc
                                                      : fmaf(f, acc, p.beta * to_float(*c)));
    } else {
        __half* c = static_cast<__half*>(p.C) + at;
        *c = from_float<__half>(p.beta == 0.0f ? f * acc : fmaf(f, acc, p.beta * to_float(*c)));
    }
}


// Rows [m0, m0 + rows) of C, columns [n0, n0 + 128), from sums in shared memory (fp32, 128 a
// row), by 128 threads `me`: 16 bytes each and whole 128-byte lines where C's rows are
// aligned, else side by side.
template <typename T>
__device__ __forceinline__ void store_rows(const Mx4Matmul& p, bool c_vec, const float* staged,
                                           int rows, long long m0, long long n0, int me) {
    constexpr int kVec = 16 / sizeof(T), kPerRow = 128 / kVec, kRows = 128 / kPerRow;
    const int end = static_cast<int>(min(static_cast<long long>(rows), p.M - m0));
    if (!c_vec || n0 + 128 > p.N) {
        if (n0 + me >= p.N) return;
        T* c = static_cast<T*>(p.C) + m0 * p.ldc + n0 + me;
#pragma unroll 4
        for (int row = 0; row < end; ++row, c += p.ldc) {
            const float v = staged[row * 128 + me];
            *c = from_float<T>(p.beta == 0.0f ? v : fmaf(p.beta, to_float(*c), v));
        }
        return;
    }
    const int col = me % kPerRow * kVec;
#pragma unroll 2
    for (int row = me / kPerRow; row < end; row += kRows) {
        T* c = static_cast<T*>(p.C) + (m0 + row) * p.ldc + n0 + col;
        float v[kVec];
#pragma unroll
        for (int k = 0; k < kVec; k += 4)
            *reinterpret_cast<float4*>(v + k) =
                *reinterpret_cast<const float4*>(staged + row * 128 + col + k);
        alignas(16) T out[kVec];
        if (p.beta != 0.0f) {
            *reinterpret_cast<uint4*>(out) = *reinterpret_cast<const uint4*>(c);
#pragma unroll
            for (int k = 0; k < kVec; ++k) v[k] = fmaf(p.beta, to_float(out[k]), v[k]);
        }
#pragma unroll
        for (int k = 0; k < kVec; ++k) out[k] = from_float<T>(v[k]);
        *reinterpret_cast<uint4*>(c) = *reinterpret_cast<const uint4*>(out);
    }
}
inline bool c_rows_aligned(const Mx4Matmul& p) {
    return reinterpret_cast<uintptr_t>(p.C) % 16 == 0 &&
           (p.M == 1 || p.ldc * (p.dtype == kF32 ? 4 : 2) % 16 == 0);
}

}  // namespace mx4
}  // namespace sgemm
