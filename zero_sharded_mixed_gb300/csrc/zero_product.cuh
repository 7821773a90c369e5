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
    DropParams drop;
};

// Eight elements (r, c) .. (r, c + 7) of an operand, zeros outside it, from any
// element-aligned place: the two 16-byte blocks that hold them, shifted together.
// Blocks are read only where they lie wholly inside the operand's own memory.
__device__ __forceinline__ uint4 fetch8(const Operand& o, int64_t r, int64_t c) {
    uint4 out = make_uint4(0u, 0u, 0u, 0u);
    if (r >= o.rows || c >= o.cols) return out;
    const uint16_t* q = o.p + r * o.ld + c;
    const int64_t left = o.cols - c;
    const uintptr_t at = reinterpret_cast<uintptr_t>(q), lo = at & ~(uintptr_t)15;
    const uint32_t shift = (uint32_t)(at & 15);
    const uintptr_t first = reinterpret_cast<uintptr_t>(o.p), last = reinterpret_cast<uintptr_t>(o.p + (o.rows - 1) * o.ld + o.cols);
    if (shift == 0 && left >= 8) return *reinterpret_cast<const uint4*>(q);
    if (left >= 8 && lo >= first && lo + 32 <= last) {
        const uint4 x = *reinterpret_cast<const uint4*>(lo), y = *reinterpret_cast<const uint4*>(lo + 16);
        uint32_t w[8] = {x.x, x.y, x.z, x.w, y.x, y.y, y.z, y.w};
        if (shift & 8) {
#pragma unroll
            for (int i = 0; i < 6; ++i) w[i] = w[i + 2];
        }
        if (shift & 4) {
#pragma unroll
            for (int i = 0; i < 5; ++i) w[i] = w[i + 1];
        }
        const uint32_t bits = (shift & 2) * 8;
        out.x = __funnelshift_r(w[0], w[1], bits);
        out.y = __funnelshift_r(w[1], w[2], bits);
        out.z = __funnelshift_r(w[2], w[3], bits);
        out.w = __funnelshift_r(w[3], w[4], bits);
        return out;
    }
    uint32_t w[4] = {0u, 0u, 0u, 0u};
#pragma unroll
    for (int j = 0; j < 8; ++j)
        if (j < left) w[j / 2] |= (uint32_t)q[j] << (16 * (j & 1));
    return make_uint4(w[0], w[1], w[2], w[3]);
}

// The end of a product for one element.
template <bool kF32>
__device__ __forceinline__ void end_one(const Ending& e, uint32_t step, int64_t row, int64_t col, float v) {
    if (e.bias) v += bf16_one(e.bias[col]);
    if (e.pre) e.pre[row * e.ld_pre + col] = to_bf16(v);
    if (e.slope) {
        const float z = bf16_one(e.slope[row * e.ld_slope + col]);
        slope_apply<1>(e.act, &z, &v);
    } else if (e.act) {
        act_apply<1>(e.act, &v);
    }
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

// The kernel of a few rows (zero_rows.cu), both operands K-major.
constexpr int kMostRows = 8;
int launch_rows(const Product& p, const Ending& e, cudaStream_t s);

}  // namespace zgb
