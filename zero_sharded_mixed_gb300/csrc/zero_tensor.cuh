// The tensor-core side of the products: tcgen05 instructions and their
// descriptors, tensor-map copies, and the cluster's addresses and barriers.
//
// Tiles are staged as sub-tiles of rows of 128 bytes (64 bf16) under the 128-byte
// swizzle: 16-byte chunk c of row r stands at chunk c ^ (r % 8).  An operand whose
// reduced dimension is contiguous ("K-major") is one sub-tile of its tile rows; one
// whose kept dimension is contiguous ("MN-major") is a sub-tile of 64 reduced rows
// for every 64 kept columns, 8 KB apart.
#pragma once

#include <cuda.h>

#include <atomic>

#include "zero_common.cuh"
#include "zero_tma.cuh"

namespace zgb {

constexpr int kSubTileBytes = 64 * 128;      // 64 rows of 128 bytes

// One lane of a converged warp.  The copies and products below are issued under
// this predicate by a warp that runs its loop as a whole: their operands are uniform
// registers, and under `lane == 0` a step of four products took 770 cycles to issue
// where the tensor core needs 512.
__device__ __forceinline__ bool elect_one() {
    uint32_t p;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(p));
    return p != 0;
}
__device__ __forceinline__ int uniform_warp() { return __shfl_sync(0xffffffffu, (int)(threadIdx.x / 32), 0); }

// ---- descriptors ---------------------------------------------------------------
// Shared-memory matrix descriptor: address, leading and stride offsets in units of
// 16 bytes, the fixed version bit 46 and the 128-byte swizzle (2 in bits 61..63).
// K-major: groups of 8 rows are 1024 bytes apart and the leading offset is unused;
// 16 further reduced elements are 32 bytes on.  MN-major: groups of 8 reduced rows
// are 1024 bytes apart, groups of 64 kept elements one sub-tile; 16 further
// reduced elements are 2048 bytes on.
__device__ __forceinline__ uint64_t smem_descriptor(uint32_t addr, bool mn_major) {
    const uint64_t leading = mn_major ? kSubTileBytes >> 4 : 1;
    return (uint64_t)((addr & 0x3ffffu) >> 4) | (leading << 16) | ((uint64_t)(1024 >> 4) << 32) | (1ull << 46) |
           (2ull << 61);
}
__device__ __forceinline__ uint32_t descriptor_step(bool mn_major) { return (mn_major ? 2048u : 32u) >> 4; }

// Instruction descriptor of kind::f16: fp32 accumulator (1 in bit 4), the operands' type
// in bits 7 and 10 (1 bf16, 0 fp16), MN-major flags in bits 15 and 16, N / 8 from bit 17,
// M / 16 from bit 24.
__device__ __forceinline__ uint32_t instruction_descriptor(int m, int n, bool a_mn, bool b_mn, bool bf16 = true) {
    return (1u << 4) | ((uint32_t)bf16 << 7) | ((uint32_t)bf16 << 10) | ((uint32_t)a_mn << 15) | ((uint32_t)b_mn << 16) |
           ((uint32_t)(n >> 3) << 17) | ((uint32_t)(m >> 4) << 24);
}

// ---- tensor memory and products ------------------------------------------------
// kPair: the instruction works on the tensor memories and tiles of a pair of CTAs.
template <bool kPair>
__device__ __forceinline__ void tmem_alloc(uint32_t* slot, uint32_t columns) {
    if constexpr (kPair) {
        asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_addr(slot)), "r"(columns) : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;");
    } else {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_addr(slot)), "r"(columns) : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
    }
}
template <bool kPair>
__device__ __forceinline__ void tmem_free(uint32_t tmem, uint32_t columns) {
    if constexpr (kPair)
        asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(columns));
    else
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(columns));
}

// bf16 or fp16 operands, as the instruction descriptor says.
template <bool kPair>
__device__ __forceinline__ void mma_bf16(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, bool accumulate) {
    if constexpr (kPair)
        asm volatile(
            "{\n\t.reg .pred p;\n\tsetp.ne.u32 p, %4, 0;\n\t"
            "tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d), "l"(a), "l"(b), "r"(idesc),
            "r"((uint32_t)accumulate) : "memory");
    else
        asm volatile(
            "{\n\t.reg .pred p;\n\tsetp.ne.u32 p, %4, 0;\n\t"
            "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d), "l"(a), "l"(b), "r"(idesc),
            "r"((uint32_t)accumulate) : "memory");
}

// The barrier (of both CTAs of a pair, `ctas` of the cluster, at the same offset)
// receives one arrival when the products issued so far are done.
template <bool kPair>
__device__ __forceinline__ void mma_commit(uint64_t* bar, uint32_t ctas = 3) {
    if constexpr (kPair)
        asm volatile(
            "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(
                smem_addr(bar)), "h"((uint16_t)ctas) : "memory");
    else
        asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(smem_addr(bar)) : "memory");
}

__device__ __forceinline__ void tcgen05_fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tcgen05_fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }

// 32 columns of the warp's 32 lanes: v[j] = column j of this thread's row.
__device__ __forceinline__ void tmem_load32(uint32_t taddr, uint32_t* v) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
        "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
        "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
        : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]), "=r"(v[7]), "=r"(v[8]),
          "=r"(v[9]), "=r"(v[10]), "=r"(v[11]), "=r"(v[12]), "=r"(v[13]), "=r"(v[14]), "=r"(v[15]), "=r"(v[16]),
          "=r"(v[17]), "=r"(v[18]), "=r"(v[19]), "=r"(v[20]), "=r"(v[21]), "=r"(v[22]), "=r"(v[23]), "=r"(v[24]),
          "=r"(v[25]), "=r"(v[26]), "=r"(v[27]), "=r"(v[28]), "=r"(v[29]), "=r"(v[30]), "=r"(v[31])
        : "r"(taddr));
    asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
}

// 16 columns of the warp's 32 lanes, in two places at once; and back.
__device__ __forceinline__ void tmem_load16_of_two(uint32_t a, uint32_t b, float (&v)[16], float (&w)[16]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
        "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
        : "=f"(v[0]), "=f"(v[1]), "=f"(v[2]), "=f"(v[3]), "=f"(v[4]), "=f"(v[5]), "=f"(v[6]), "=f"(v[7]), "=f"(v[8]), "=f"(v[9]),
          "=f"(v[10]), "=f"(v[11]), "=f"(v[12]), "=f"(v[13]), "=f"(v[14]), "=f"(v[15])
        : "r"(a));
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
        "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
        : "=f"(w[0]), "=f"(w[1]), "=f"(w[2]), "=f"(w[3]), "=f"(w[4]), "=f"(w[5]), "=f"(w[6]), "=f"(w[7]), "=f"(w[8]), "=f"(w[9]),
          "=f"(w[10]), "=f"(w[11]), "=f"(w[12]), "=f"(w[13]), "=f"(w[14]), "=f"(w[15])
        : "r"(b));
    asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
}
__device__ __forceinline__ void tmem_store16(uint32_t taddr, const float (&v)[16]) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], "
        "{%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16};" ::"r"(taddr),
        "f"(v[0]), "f"(v[1]), "f"(v[2]), "f"(v[3]), "f"(v[4]), "f"(v[5]), "f"(v[6]), "f"(v[7]), "f"(v[8]), "f"(v[9]),
        "f"(v[10]), "f"(v[11]), "f"(v[12]), "f"(v[13]), "f"(v[14]), "f"(v[15])
        : "memory");
}
__device__ __forceinline__ void tmem_stored() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// 16 rows x 32 columns from lane `taddr`: of every group g of 8 columns, thread
// 4 i + j of the warp gets columns 2 j and 2 j + 1 of rows i (v[g][0..1]) and i + 8
// (v[g][2..3]).
__device__ __forceinline__ void tmem_load_fragment(uint32_t taddr, float (&v)[4][4]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.16x256b.x4.b32 "
        "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
        : "=f"(v[0][0]), "=f"(v[0][1]), "=f"(v[0][2]), "=f"(v[0][3]), "=f"(v[1][0]), "=f"(v[1][1]), "=f"(v[1][2]), "=f"(v[1][3]),
          "=f"(v[2][0]), "=f"(v[2][1]), "=f"(v[2][2]), "=f"(v[2][3]), "=f"(v[3][0]), "=f"(v[3][1]), "=f"(v[3][2]), "=f"(v[3][3])
        : "r"(taddr));
    asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
}

// ---- clusters --------------------------------------------------------------------
__device__ __forceinline__ uint32_t cluster_rank() {
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}
__device__ __forceinline__ uint32_t cluster_size() {
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_nctarank;" : "=r"(r));
    return r;
}
__device__ __forceinline__ uint32_t peer_addr(uint32_t addr, uint32_t rank) {
    uint32_t r;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(addr), "r"(rank));
    return r;
}
__device__ __forceinline__ void cluster_sync() {
    asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// The two halves of cluster_sync.
__device__ __forceinline__ void cluster_arrive() { asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory"); }
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory"); }
// After fence_barrier_init: the CTAs' barriers exist, and nothing else is ordered.
__device__ __forceinline__ void cluster_started() {
    asm volatile("barrier.cluster.arrive.relaxed.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// Hands over tensor memory alone (its reads are ordered by the tcgen05 fences), so
// the arrival need not order other memory.
__device__ __forceinline__ void peer_arrive(uint32_t bar_addr) {
    asm volatile("mbarrier.arrive.relaxed.cluster.shared::cluster.b64 _, [%0];" ::"r"(bar_addr) : "memory");
}
__device__ __forceinline__ float4 peer_load(uint32_t addr) {
    float4 v;
    asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];" : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w) : "r"(addr));
    return v;
}
__device__ __forceinline__ float peer_load1(uint32_t addr) {
    float v;
    asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(addr));
    return v;
}
__device__ __forceinline__ double peer_load_double(uint32_t addr) {
    double v;
    asm volatile("ld.shared::cluster.f64 %0, [%1];" : "=d"(v) : "r"(addr));
    return v;
}

// ---- tensor-map copies -------------------------------------------------------------
// A box of the matrix at column x (a multiple of 8 elements: copies start on 16-byte
// boundaries) and row y; what lies outside the matrix is filled with zeros.
__device__ __forceinline__ void tensor_load(uint32_t dst, const CUtensorMap* map, int x, int y, uint32_t bar) {
    asm volatile(
        "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], [%4];" ::"r"(dst),
        "l"(map), "r"(x), "r"(y), "r"(bar) : "memory");
}
// The same into this CTA of a pair, counted on a barrier of either.
__device__ __forceinline__ void tensor_load_pair(uint32_t dst, const CUtensorMap* map, int x, int y, uint32_t bar) {
    asm volatile(
        "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes.cta_group::2 [%0], [%1, {%2, %3}], [%4];" ::"r"(dst),
        "l"(map), "r"(x), "r"(y), "r"(bar) : "memory");
}
// The same from matrix z of a batch.
__device__ __forceinline__ void tensor_load_pair(uint32_t dst, const CUtensorMap* map, int x, int y, int z, uint32_t bar) {
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes.cta_group::2 [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(dst),
        "l"(map), "r"(x), "r"(y), "r"(z), "r"(bar) : "memory");
}
__device__ __forceinline__ void tensor_map_prefetch(const CUtensorMap* map) {
    asm volatile("prefetch.tensormap [%0];" ::"l"(map) : "memory");
}
// Orders this thread's writes to shared memory before later reads by the tensor core.
__device__ __forceinline__ void fence_async_shared() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }
__device__ __forceinline__ void fence_barrier_init() { asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory"); }

// ---- four lanes of a fragment's row ----------------------------------------------------
__device__ __forceinline__ void quad_transpose(uint32_t* w) {   // w[g] of lane j becomes w[j] of lane g
    const int lane = threadIdx.x & 31;
    const bool odd = lane & 1, high = lane & 2;
#pragma unroll
    for (int a = 0; a < 4; a += 2) {
        const uint32_t r = __shfl_xor_sync(0xffffffffu, odd ? w[a] : w[a + 1], 1);
        w[a] = odd ? r : w[a];
        w[a + 1] = odd ? w[a + 1] : r;
    }
#pragma unroll
    for (int a = 0; a < 2; ++a) {
        const uint32_t r = __shfl_xor_sync(0xffffffffu, high ? w[a] : w[a + 2], 2);
        w[a] = high ? r : w[a];
        w[a + 2] = high ? w[a + 2] : r;
    }
}
__device__ __forceinline__ void quad_transpose(uint4& u) {
    uint32_t w[4] = {u.x, u.y, u.z, u.w};
    quad_transpose(w);
    u = make_uint4(w[0], w[1], w[2], w[3]);
}

// ---- waits -------------------------------------------------------------------------
constexpr long long kWaitCycles = 1ll << 31;   // SM cycles (about a second) before a wait gives up

// For a converged warp that goes on as a whole: every lane gets the same answer.  A
// wait that gives up leaves ZERO_ETIMEOUT in *status, device memory.
__device__ __forceinline__ bool warp_wait(uint64_t* bar, uint32_t parity, int* status, long long limit = kWaitCycles) {
    if (__all_sync(0xffffffffu, mbar_try_wait(bar, parity))) return true;
    if (__all_sync(0xffffffffu, mbar_wait_bounded(bar, parity, limit))) return true;
    atomicExch(status, ZERO_ETIMEOUT);
    return false;
}

// ---- launches, host --------------------------------------------------------------------
typedef CUresult (*EncodeTiled)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*, const cuuint64_t*,
                                const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                                CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

inline EncodeTiled encode_tiled() {
    static EncodeTiled fn = [] {
        void* p = nullptr;
        cudaDriverEntryPointQueryResult found;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &found) != cudaSuccess ||
            found != cudaDriverEntryPointSuccess) {
            (void)cudaGetLastError();
            p = nullptr;
        }
        return reinterpret_cast<EncodeTiled>(p);
    }();
    return fn;
}

// The current device, if there is one below `most`.  A failed question leaves no error
// behind: a caller goes on without the answer or reports it by its code.
inline bool device_below(int most, int* dev) {
    const cudaError_t e = cudaGetDevice(dev);
    if (e != cudaSuccess) {
        note_cuda_error(e);
        (void)cudaGetLastError();
    }
    return e == cudaSuccess && *dev >= 0 && *dev < most;
}

// Raises a kernel's shared-memory limit, once per device (again after a failure).
typedef std::atomic<bool> Done[64];
inline int allow_smem(const void* kernel, int bytes, Done& done) {
    int dev = 0;
    if (!device_below(64, &dev)) return ZERO_ECUDA;
    if (done[dev].load(std::memory_order_acquire)) return ZERO_OK;
    const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
    if (e != cudaSuccess) {
        note_cuda_error(e);
        (void)cudaGetLastError();
        return ZERO_ECUDA;
    }
    done[dev].store(true, std::memory_order_release);
    return ZERO_OK;
}

// Pairs of SMs; one where the runtime could not say how many there are.
inline int64_t sm_pairs() {
    const int n = sm_count();
    return n < 2 ? 1 : n / 2;
}

}  // namespace zgb
