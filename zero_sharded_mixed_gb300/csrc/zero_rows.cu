// A linear of a few rows (one new token, a handful of sequences), sm_103a.
//
// Such a product is a read of its weights: every element of w meets at most four
// elements of x, far below what a tensor core could use, and a tile of 128 rows
// would stay almost empty.  A warp takes two columns and runs along their rows of w
// in 16-byte vectors, 512 bytes a step; x comes from the caches.  fp32 products and
// sums: a lane its own vectors in order, then the lanes of the warp, then (where
// there are few columns) the warps among which the reduced dimension was split, all
// in a fixed order.  Bound by the weights' bytes (4096 x 11008, one row, weights not in
// L2: 16.4 us, 5.5 TB/s; 11008 x 4096: 21, 4.3 TB/s) or, below some 20 MB, by the launch
// and one memory latency: 4800 x 1600 in 6.5 us, 5.0 where the weights are still in L2.  Each pair of columns starting at
// another place of its rows was slower (18 and 25 us).
#include "zero_product.cuh"

namespace zgb {

constexpr int kCols = 2;            // columns of a warp
constexpr int kWarps = kThreads / 32;

template <int kM, bool kF32, bool kAligned>
__global__ void __launch_bounds__(kThreads) rows_kernel(const Product p, const Ending e, int split) {
    __shared__ float part[kWarps][kCols * kM];
    const int warp = threadIdx.x / 32, lane = threadIdx.x & 31;
    const int groups = kWarps / split, group = warp / split;
    const int64_t col0 = ((int64_t)blockIdx.x * groups + group) * kCols;
    const int64_t k = p.depth;
    float acc[kCols][kM] = {};
    await_predecessor();
    if (col0 < p.cols) {
        // a column past the end reads the last one again and is not stored
        const int64_t last = p.cols - 1;
        const int64_t bc[kCols] = {col0, col0 + 1 < last ? col0 + 1 : last};
        const int64_t stride = (int64_t)split * 256;
        const int64_t whole = kAligned ? k & ~(int64_t)7 : 0;
        int64_t c = ((int64_t)(warp % split) * 32 + lane) * 8;
#pragma unroll(kM <= 2 ? 4 : 2)
        for (; c < whole; c += stride) {
            uint4 w[kCols], x[kM];
#pragma unroll
            for (int j = 0; j < kCols; ++j) w[j] = ld_live_u4(p.b.p + bc[j] * p.b.ld + c);
#pragma unroll
            for (int i = 0; i < kM; ++i) x[i] = i < p.rows ? *reinterpret_cast<const uint4*>(p.a.p + i * p.a.ld + c) : make_uint4(0u, 0u, 0u, 0u);
            float wv[kCols][8], xv[8];
#pragma unroll
            for (int j = 0; j < kCols; ++j) unpack8(w[j], wv[j]);
#pragma unroll
            for (int i = 0; i < kM; ++i) {
                unpack8(x[i], xv);
#pragma unroll
                for (int j = 0; j < kCols; ++j)
#pragma unroll
                    for (int t = 0; t < 8; ++t) acc[j][i] += wv[j][t] * xv[t];
            }
        }
        if constexpr (kAligned) {
            if (c == whole)   // one lane has the last few elements
                for (; c < k; ++c)
#pragma unroll
                    for (int i = 0; i < kM; ++i)
                        if (i < p.rows) {
                            const float x = bf16_one(p.a.p[i * p.a.ld + c]);
#pragma unroll
                            for (int j = 0; j < kCols; ++j) acc[j][i] += bf16_one(p.b.p[bc[j] * p.b.ld + c]) * x;
                        }
        } else {
            const uintptr_t a0 = operand_begin(p.a), a1 = operand_end(p.a), b0 = operand_begin(p.b), b1 = operand_end(p.b);
#pragma unroll(kM <= 2 ? 3 : 1)
            for (; c < k; c += stride) {
                const int n = k - c < 8 ? (int)(k - c) : 8;
                Blocks8 wb[kCols], xb[kM];
#pragma unroll
                for (int j = 0; j < kCols; ++j) wb[j] = load_blocks(b0, b1, p.b.p + bc[j] * p.b.ld + c, n);
#pragma unroll
                for (int i = 0; i < kM; ++i) xb[i] = load_blocks(a0, a1, p.a.p + i * p.a.ld + c, i < p.rows ? n : 0);
                float wv[kCols][8], xv[8];
#pragma unroll
                for (int j = 0; j < kCols; ++j) unpack8(shift_blocks(b0, b1, p.b.p + bc[j] * p.b.ld + c, n, wb[j]), wv[j]);
#pragma unroll
                for (int i = 0; i < kM; ++i) {
                    unpack8(shift_blocks(a0, a1, p.a.p + i * p.a.ld + c, i < p.rows ? n : 0, xb[i]), xv);   // zeros past the last row
#pragma unroll
                    for (int j = 0; j < kCols; ++j)
#pragma unroll
                        for (int t = 0; t < 8; ++t) acc[j][i] += wv[j][t] * xv[t];
                }
            }
        }
    }
#pragma unroll
    for (int j = 0; j < kCols; ++j)
#pragma unroll
        for (int i = 0; i < kM; ++i) {
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) acc[j][i] += __shfl_xor_sync(0xffffffffu, acc[j][i], o);
            if (lane == 0) part[warp][i * kCols + j] = acc[j][i];
        }
    __syncthreads();
    const int g = threadIdx.x / (kCols * kM), in = threadIdx.x - g * (kCols * kM);
    if (g < groups) {
        const int64_t row = in / kCols, col = ((int64_t)blockIdx.x * groups + g) * kCols + in % kCols;
        if (row < p.rows && col < p.cols) {
            float v = 0.0f;
            for (int i = 0; i < split; ++i) v += part[g * split + i][in];
            end_one<kF32>(e, e.drop.cut ? drop_step(e.drop) : 0u, row, col, v);
        }
    }
}

template <int kM, bool kF32>
static int launch_rows_of(const Product& p, const Ending& e, cudaStream_t s) {
    const int64_t pairs = (p.cols + kCols - 1) / kCols, wanted = (int64_t)sm_count() * 16;   // warps
    int split = 1;
    while (split < kWarps && pairs * split < wanted && p.depth >= split * 512) split *= 2;
    const int64_t grid = (pairs * split + kWarps - 1) / kWarps;
    if (grid > INT32_MAX) return ZERO_ERANGE;
    const bool aligned = rows_aligned16(p.b.p, p.b.ld, 2) && (p.rows == 1 ? aligned16(p.a.p) : rows_aligned16(p.a.p, p.a.ld, 2));
    return launch_dense(aligned ? rows_kernel<kM, kF32, true> : rows_kernel<kM, kF32, false>, dim3((unsigned)grid), kThreads, 1, true, 0,
                        s, p, e, split);
}

int launch_rows(const Product& p, const Ending& e, cudaStream_t s) {
    static_assert(kMostRows == 4, "the sizes below");
    if (e.out_f32)
        return p.rows == 1 ? launch_rows_of<1, true>(p, e, s) : p.rows == 2 ? launch_rows_of<2, true>(p, e, s) : launch_rows_of<4, true>(p, e, s);
    return p.rows == 1 ? launch_rows_of<1, false>(p, e, s) : p.rows == 2 ? launch_rows_of<2, false>(p, e, s) : launch_rows_of<4, false>(p, e, s);
}

}  // namespace zgb
