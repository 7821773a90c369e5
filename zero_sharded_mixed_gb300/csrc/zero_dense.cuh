// What the dense operators of a unit share: the counter-based random bits of
// dropout, the activations with their slopes, and the elementwise end of a
// product (bias, activation, dropout, residual) on eight neighbouring columns.
#pragma once

#include "zero_common.cuh"

namespace zgb {

// ---- dropout ----------------------------------------------------------------
// Philox4x32-10 (Salmon, Moraes, Dror and Shaw, "Parallel random numbers: as
// easy as 1, 2, 3", 2011): ten rounds of two 32 x 32 -> 64 bit products on a
// 128-bit counter under a 64-bit key.  One block of 128 bits serves the eight
// elements of columns 8 c .. 8 c + 7 of one row, 16 bits each, low halves
// first, so a 128-bit vector of bf16 needs one block and the bits of an element
// depend on its row and column alone, not on strides, tiles or the launch.
// 16 bits quantise p to a multiple of 2^-16; the factor on kept elements is
// formed from the quantised p, so the expectation is exact.  32 bits an element
// would double the integer work, which already stands beside the memory time.
struct DropParams {
    uint32_t cut;               // keep where bits >= cut; 0 = no dropout, 65536 = drop everything
    float scale;                // 65536 / (65536 - cut), 0 where everything is dropped
    uint32_t site, step;
    const uint64_t* step_ptr;   // null, or added to step
    uint32_t key[10][2];        // of each round, formed on the host
};

__device__ __forceinline__ uint32_t drop_step(const DropParams& d) {
    return d.step + (d.step_ptr ? (uint32_t)*d.step_ptr : 0u);
}

__device__ __forceinline__ uint4 philox_block(const DropParams& d, uint32_t step, uint32_t row, uint32_t col_block) {
    uint32_t c0 = col_block, c1 = row, c2 = d.site, c3 = step;
#pragma unroll
    for (int r = 0; r < 10; ++r) {
        const uint64_t p0 = (uint64_t)c0 * 0xD2511F53u;
        const uint64_t p1 = (uint64_t)c2 * 0xCD9E8D57u;
        c0 = (uint32_t)(p1 >> 32) ^ c1 ^ d.key[r][0];
        c1 = (uint32_t)p1;
        c2 = (uint32_t)(p0 >> 32) ^ c3 ^ d.key[r][1];
        c3 = (uint32_t)p0;
    }
    return make_uint4(c0, c1, c2, c3);
}

// v[j] = kept ? v[j] * scale : 0 for the eight elements that block b serves; a
// dropped element is 0 whatever it held.  A high half is compared in its place (the
// bits below it cannot carry it over cut), a low one moved there.
__device__ __forceinline__ void drop8(const DropParams& d, const uint4& b, float* v) {
    const uint32_t w[4] = {b.x, b.y, b.z, b.w}, cut = d.cut << 16;
    if (d.cut > 0xffffu) {   // everything: cut has no place in 16 bits
#pragma unroll
        for (int j = 0; j < 8; ++j) v[j] = 0.0f;
        return;
    }
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        v[2 * j] = (w[j] << 16) >= cut ? v[2 * j] * d.scale : 0.0f;
        v[2 * j + 1] = w[j] >= cut ? v[2 * j + 1] * d.scale : 0.0f;
    }
}
__device__ __forceinline__ void drop8(const DropParams& d, uint32_t step, int64_t row, int64_t col_block, float* v) {
    drop8(d, philox_block(d, step, (uint32_t)row, (uint32_t)col_block), v);
}

// Where lane l of a warp holds the block of row l % 8 and column group l / 8 of an
// 8 x 32 part: the 16 bits of row r in this lane's column.  Every lane calls.
__device__ __forceinline__ uint32_t row_bits(const uint4& block, int r) {
    const int lane = threadIdx.x & 31, from = (lane & 24) | r;
    const uint32_t w0 = __shfl_sync(0xffffffffu, block.x, from), w1 = __shfl_sync(0xffffffffu, block.y, from);
    const uint32_t w2 = __shfl_sync(0xffffffffu, block.z, from), w3 = __shfl_sync(0xffffffffu, block.w, from);
    const uint32_t w = lane & 4 ? (lane & 2 ? w3 : w2) : (lane & 2 ? w1 : w0);
    return lane & 1 ? w >> 16 : w & 0xffffu;
}

// Checks a caller's block and forms the kernels' parameters; null = no dropout.
int drop_params(const zero_dropout_t* d, int64_t rows, int64_t cols, DropParams* out);

// db[c] = db_acc[c] + the sum over rows of dz[r, c] (zero_dropout.cu).
int launch_column_sum(int64_t rows, int64_t cols, const uint16_t* dz, int64_t lddz, const void* db_acc, void* db,
                      bool db_f32, cudaStream_t s);

// ---- activations ------------------------------------------------------------
// Evaluated in fp32.  The tanh form of the GELU is z sigmoid(2u), which like the
// SiLU needs one base-2 exponential (its factor folded into the polynomial) and one
// reciprocal, in their approximate forms: about 2^-22 relative, and in the tails
// |z| 2^-24, since the exponential's argument is rounded to 32 bits.  That is far inside
// the rounding of a bf16 result; of an fp32 one it takes the last two bits,
// and more in the tails.
// The erf form's lower tail is 1 + erf in 32 bits, exact to 2^-24 of z itself.
__device__ __forceinline__ float exp2_f(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ float rcp_f(float x) {
    float y;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
// Past the clamps the second term of a slope is below fp32's resolution; without
// them it would be 0 * infinity.  A NaN stays.
__device__ __forceinline__ float clamp_keep_nan(float z, float c) {
    float y;
    asm("{\n\tmin.NaN.f32 %0, %1, %2;\n\tmax.NaN.f32 %0, %0, %3;\n\t}" : "=&f"(y) : "f"(z), "f"(c), "f"(-c));
    return y;
}
constexpr float kLog2E = 1.44269504088896340736f;
constexpr float kGelu2C = 2.0f * 0.79788456080286535588f;   // 2 sqrt(2 / pi)
constexpr float kGeluA = 0.044715f;

__device__ __forceinline__ float sigmoid_2u(float z) {   // sigmoid(2 sqrt(2 / pi) (z + kGeluA z^3))
    return rcp_f(1.0f + exp2_f(z * (-kGelu2C * kLog2E - kGelu2C * kLog2E * kGeluA * (z * z))));
}

template <int kAct>
__device__ __forceinline__ float act_one(float z) {
    if constexpr (kAct == ZERO_ACT_RELU) return z < 0.0f ? 0.0f : z;   // a NaN stays
    if constexpr (kAct == ZERO_ACT_GELU) return 0.5f * z * (1.0f + erff(z * 0.70710678118654752440f));
    if constexpr (kAct == ZERO_ACT_GELU_TANH) return z * sigmoid_2u(z);
    if constexpr (kAct == ZERO_ACT_SILU) return z * rcp_f(1.0f + exp2_f(-kLog2E * z));
    return z;
}

template <int kAct>
__device__ __forceinline__ float slope_one(float z) {
    if constexpr (kAct == ZERO_ACT_RELU) return z > 0.0f ? 1.0f : 0.0f;
    if constexpr (kAct == ZERO_ACT_GELU) {
        z = clamp_keep_nan(z, 20.0f);
        return 0.5f * (1.0f + erff(z * 0.70710678118654752440f)) + z * 0.39894228040143267794f * exp2_f(-0.5f * kLog2E * z * z);
    }
    if constexpr (kAct == ZERO_ACT_GELU_TANH) {
        z = clamp_keep_nan(z, 20.0f);
        const float s = sigmoid_2u(z);
        return s + (s - s * s) * (z * (kGelu2C + 3.0f * kGelu2C * kGeluA * (z * z)));
    }
    if constexpr (kAct == ZERO_ACT_SILU) {
        z = clamp_keep_nan(z, 104.0f);   // past 89 the exponential is already infinite
        const float s = rcp_f(1.0f + exp2_f(-kLog2E * z));
        return s + (s - s * s) * z;
    }
    return 1.0f;
}

// Over kCount values at once: one branch on the activation, so that the chains of
// the values interleave (a branch a value made the end of a product five times as
// long as the product).
template <int kCount>
__device__ __forceinline__ void act_apply(int act, float* v) {
#define ZGB_EACH(A) _Pragma("unroll") for (int j = 0; j < kCount; ++j) v[j] = act_one<A>(v[j])
    switch (act) {
        case ZERO_ACT_RELU: ZGB_EACH(ZERO_ACT_RELU); break;
        case ZERO_ACT_GELU: ZGB_EACH(ZERO_ACT_GELU); break;
        case ZERO_ACT_GELU_TANH: ZGB_EACH(ZERO_ACT_GELU_TANH); break;
        case ZERO_ACT_SILU: ZGB_EACH(ZERO_ACT_SILU); break;
        default: break;
    }
#undef ZGB_EACH
}
template <int kCount>
__device__ __forceinline__ void slope_apply(int act, const float* z, float* v) {
#define ZGB_EACH(A) _Pragma("unroll") for (int j = 0; j < kCount; ++j) v[j] *= slope_one<A>(z[j])
    switch (act) {
        case ZERO_ACT_RELU: ZGB_EACH(ZERO_ACT_RELU); break;
        case ZERO_ACT_GELU: ZGB_EACH(ZERO_ACT_GELU); break;
        case ZERO_ACT_GELU_TANH: ZGB_EACH(ZERO_ACT_GELU_TANH); break;
        case ZERO_ACT_SILU: ZGB_EACH(ZERO_ACT_SILU); break;
        default: break;
    }
#undef ZGB_EACH
}

// ---- eight neighbouring columns ---------------------------------------------
__device__ __forceinline__ void unpack8(uint4 u, float* v) {
    v[0] = bf16_lo(u.x); v[1] = bf16_hi(u.x);
    v[2] = bf16_lo(u.y); v[3] = bf16_hi(u.y);
    v[4] = bf16_lo(u.z); v[5] = bf16_hi(u.z);
    v[6] = bf16_lo(u.w); v[7] = bf16_hi(u.w);
}
__device__ __forceinline__ uint4 pack8(const float* v) {
    return make_uint4(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]), pack_bf16x2(v[4], v[5]),
                      pack_bf16x2(v[6], v[7]));
}

template <bool kF32>
__device__ __forceinline__ void raw8(const uint4* u, float* v) {   // as loaded: one vector of bf16, two of fp32
    if constexpr (kF32) {
        v[0] = __uint_as_float(u[0].x); v[1] = __uint_as_float(u[0].y); v[2] = __uint_as_float(u[0].z); v[3] = __uint_as_float(u[0].w);
        v[4] = __uint_as_float(u[1].x); v[5] = __uint_as_float(u[1].y); v[6] = __uint_as_float(u[1].z); v[7] = __uint_as_float(u[1].w);
    } else {
        unpack8(u[0], v);
    }
}

// A 128-bit load of a stream.  Kernels of this file's launches (below) start before
// their predecessor's writes have ended, so that nothing they read is read-only for
// their lifetime: coherent loads alone, never the read-only path (ld.global.nc), which
// may give a stale line and which the compiler may move above the wait.
__device__ __forceinline__ uint4 ld_live_u4(const void* p) { return __ldcs(reinterpret_cast<const uint4*>(p)); }

// p: the first of the eight, 16-byte aligned.
__device__ __forceinline__ void store8(void* p, bool f32, const float* v) {
    if (f32) {
        reinterpret_cast<float4*>(p)[0] = make_float4(v[0], v[1], v[2], v[3]);
        reinterpret_cast<float4*>(p)[1] = make_float4(v[4], v[5], v[6], v[7]);
    } else {
        *reinterpret_cast<uint4*>(p) = pack8(v);
    }
}

// Whether rows of `ld` elements of `size` bytes from p keep eight-column groups
// on 16-byte boundaries.
inline bool rows_aligned16(const void* p, int64_t ld, int size) {
    return aligned16(p) && (ld * size) % 16 == 0;
}

inline int dtype_size(int32_t dtype) { return dtype == ZERO_F32 ? 4 : 2; }

// 0, or why a matrix argument is refused: rows of at least `cols` elements, an
// element-aligned pointer (any, where there is no element), and rows * ld * size
// within 63 bits.
inline int check_matrix(const void* p, int64_t rows, int64_t cols, int64_t ld, int32_t dtype) {
    if (ld < cols) return ZERO_EINVAL;
    if (rows == 0 || cols == 0) return ZERO_OK;
    if (!p) return ZERO_EINVAL;
    if (ld > 0 && rows > INT64_MAX / 8 / ld) return ZERO_ERANGE;
    return check_aligned(p, dtype_size(dtype));
}

// ---- launches ----------------------------------------------------------------
// The dense operators follow one another in short kernels, so that each is launched
// while its predecessor still runs (programmatic stream serialization): a kernel
// lets its successor start as soon as all its own CTAs have, and itself waits,
// before its first access to global memory, until its predecessor has ended and its
// writes are visible.  Kernels without these two calls (other libraries', this
// library's update) are unaffected before and after.  Saves about 2 us a launch.
__device__ __forceinline__ void await_predecessor() {
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    asm volatile("griddepcontrol.wait;" ::: "memory");
}

// A launch on grid.x * grid.y CTAs in clusters of `cluster` along x, of a kernel
// that calls await_predecessor.  early: before its predecessor has ended.  Its CTAs
// then take the SMs as they come free, which packs large clusters unevenly: the
// column sums of 8192 x 6400, 400 CTAs in clusters of 8, took 136 us after a product
// so, and 80 launched to a free GPU.
template <class... Params, class... Args>
int launch_dense(void (*kernel)(Params...), dim3 grid, unsigned threads, unsigned cluster, bool early, int smem, cudaStream_t s,
                 Args&&... args) {
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = (size_t)smem;
    cfg.stream = s;
    cudaLaunchAttribute attr[2]{};
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = cluster;
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[1].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = early ? 2 : 1;
    const cudaError_t e = cudaLaunchKernelEx(&cfg, kernel, static_cast<Args&&>(args)...);
    if (e != cudaSuccess) {
        note_cuda_error(e);
        (void)cudaGetLastError();
        return ZERO_ECUDA;
    }
    return ZERO_OK;
}

}  // namespace zgb
