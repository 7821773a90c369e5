// What the kernels of the products share: operands, the end of a product as the
// entry points describe it, and reads of an operand at any alignment.
#pragma once

#include "zero_dense.cuh"

namespace zgb {

// A matrix as it is stored, row-major.  The product C[i, j] = sum over t of
// A(i, t) B(j, t) reads an operand with its reduced dimension t along the columns
// (K-major) or along the rows (MN-major).
struct Operand {
    const uint16_t* p;
    int64_t ld, rows, cols;
    bool mn;
};
struct Product {
    int64_t rows, cols, depth;
    Operand a, b;
};
struct Ending {
    const uint16_t* bias;                       // per column, or null
    const uint16_t* slope; int64_t ld_slope;    // pre of the layer below: times act'(slope), or null
    uint16_t* pre; int64_t ld_pre;              // receives the product with its bias, or null
    const void* add; int64_t ld_add;            // residual or acc, of the output's type, or null
    void* out; int64_t ld_out;
    int32_t act;
    bool out_f32;
    bool vec;                                   // every matrix above keeps 8-column groups on 16-byte boundaries
    bool bare;                                  // nothing but a bias beside the product
    DropParams drop;
};

// Eight elements from any element-aligned place q of an operand, of which the first
// n exist (none for n <= 0; the others come as zeros): the one or two 16-byte blocks
// that hold them are loaded first, without a branch around the loads, so that a
// thread's loads of several places fly together, and shifted into one vector later.
// Blocks are read only where they lie wholly inside the operand's own memory; the few
// places where one does not are read element by element.
struct Blocks8 {
    uint4 x, y;
};
__device__ __forceinline__ uintptr_t operand_begin(const Operand& o) { return reinterpret_cast<uintptr_t>(o.p); }
__device__ __forceinline__ uintptr_t operand_end(const Operand& o) {
    return reinterpret_cast<uintptr_t>(o.p + (o.rows - 1) * o.ld + o.cols);
}
__device__ __forceinline__ Blocks8 load_blocks(uintptr_t begin, uintptr_t end, const uint16_t* q, int n) {
    const uintptr_t at = reinterpret_cast<uintptr_t>(q), lo = at & ~(uintptr_t)15;
    Blocks8 b;
    b.x = b.y = make_uint4(0u, 0u, 0u, 0u);
    if (n > 0 && lo >= begin && lo + 16 <= end) b.x = *reinterpret_cast<const uint4*>(lo);
    if ((int)(at & 15) + 2 * (n < 8 ? n : 8) > 16 && lo + 32 <= end) b.y = *reinterpret_cast<const uint4*>(lo + 16);
    return b;
}
__device__ __forceinline__ uint4 shift_blocks(uintptr_t begin, uintptr_t end, const uint16_t* q, int n, const Blocks8& b) {
    const uintptr_t at = reinterpret_cast<uintptr_t>(q), lo = at & ~(uintptr_t)15;
    const uint32_t shift = (uint32_t)(at & 15);
    uint32_t w[8] = {b.x.x, b.x.y, b.x.z, b.x.w, b.y.x, b.y.y, b.y.z, b.y.w};
#pragma unroll
    for (int i = 0; i < 6; ++i) w[i] = shift & 8 ? w[i + 2] : w[i];
#pragma unroll
    for (int i = 0; i < 5; ++i) w[i] = shift & 4 ? w[i + 1] : w[i];
#pragma unroll
    for (int i = 0; i < 4; ++i) w[i] = __funnelshift_r(w[i], w[i + 1], (shift & 2) * 8);
    if (n < 8) {
        if (n > 0 && (lo < begin || lo + (shift + 2 * n > 16 ? 32 : 16) > end)) {
#pragma unroll
            for (int i = 0; i < 4; ++i) w[i] = (2 * i < n ? q[2 * i] : 0u) | (2 * i + 1 < n ? (uint32_t)q[2 * i + 1] << 16 : 0u);
        } else {
#pragma unroll
            for (int i = 0; i < 4; ++i) w[i] &= n >= 2 * i + 2 ? 0xffffffffu : n == 2 * i + 1 ? 0xffffu : 0u;
        }
    } else if (lo < begin || lo + (shift ? 32 : 16) > end) {
#pragma unroll
        for (int i = 0; i < 4; ++i) w[i] = q[2 * i] | ((uint32_t)q[2 * i + 1] << 16);
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
}

// The end of a forward product for one element (no slope).
template <bool kF32>
__device__ __forceinline__ void end_one(const Ending& e, uint32_t step, int64_t row, int64_t col, float v) {
    if (e.bias) v += bf16_one(e.bias[col]);
    if (e.pre) e.pre[row * e.ld_pre + col] = to_bf16(v);
    if (e.act) act_apply<1>(e.act, &v);
    if (e.drop.cut) {
        const uint4 b = philox_block(e.drop, step, (uint32_t)row, (uint32_t)(col >> 3));
        const uint32_t w = col & 4 ? (col & 2 ? b.w : b.z) : (col & 2 ? b.y : b.x);
        v = (col & 1 ? w >> 16 : w & 0xffffu) >= e.drop.cut ? v * e.drop.scale : 0.0f;
    }
    if constexpr (kF32) {
        if (e.add) v += static_cast<const float*>(e.add)[row * e.ld_add + col];
        static_cast<float*>(e.out)[row * e.ld_out + col] = v;
    } else {
        if (e.add) v += bf16_one(static_cast<const uint16_t*>(e.add)[row * e.ld_add + col]);
        static_cast<uint16_t*>(e.out)[row * e.ld_out + col] = to_bf16(v);
    }
}

// The kernel of a few rows (zero_rows.cu), both operands K-major: forward products alone.
constexpr int kMostRows = 4;
int launch_rows(const Product& p, const Ending& e, cudaStream_t s);

}  // namespace zgb
