// Products of a unit with their elementwise ends, and their gradients, sm_103a:
//   zero_linear              y  = residual + D(act(x w^T + bias))
//   zero_linear_grad_input   dx = residual + D'(dz w) act'(pre)
//   zero_linear_grad_weight  dw = acc + dz^T x,  db = db_acc + sum over rows of dz
#include <atomic>
#include <type_traits>

#include "zero_product.cuh"
#include "zero_tensor.cuh"

namespace zgb {

__device__ int g_linear_status;   // ZERO_OK, or ZERO_ETIMEOUT once a bounded wait gave up

int take_linear_status() {
    int v = 0;
    if (cudaMemcpyFromSymbol(&v, g_linear_status, sizeof v) != cudaSuccess) {
        (void)cudaGetLastError();
        return ZERO_ECUDA;
    }
    if (v != ZERO_OK) {
        const int zero = ZERO_OK;
        if (cudaMemcpyToSymbol(g_linear_status, &zero, sizeof zero) != cudaSuccess) {
            (void)cudaGetLastError();
            return ZERO_ECUDA;
        }
    }
    return v == ZERO_OK ? ZERO_OK : ZERO_ETIMEOUT;
}

// ---- the end of a product --------------------------------------------------------
// Accumulators that pass through shared memory stand there in 32 x 32 chunks of fp32.
// Row r of a chunk is 128 bytes; its 16-byte group g stands at group_place(r, g), so
// that rows written by 32 lanes share no bank, and 8 rows (a unit, a warp's) lie on end.
__device__ __forceinline__ uint32_t group_place(int r, int g) { return (uint32_t)r * 128u + (uint32_t)((g ^ (r & 7)) << 4); }

// The pair kernel's end of 16 rows x 32 whole, aligned columns, a warp together,
// with the accumulators as tensor memory gives them (tmem_load_fragment): lane
// 4 i + j holds two columns of every group of eight.  What moves in 16-byte vectors,
// a lane a group (bf16 results and residuals, a Philox block), is exchanged between
// the four lanes of a row by a 4 x 4 transposition of words.  Shared memory is left
// alone: the products and their copies use its whole bandwidth, and a transposition
// through it took 5900 cycles a tile against the 12800 of a product of depth 1600.
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

// fp32: between the fragment's two columns of groups g and g + 1 (g even) and four
// columns of one of them, group g in even lanes and g + 1 in odd ones, which start
// pair_column() after the first of the 32 columns (plus 8 g).  Its own inverse.
__device__ __forceinline__ void pair_exchange(float (&v)[4][4]) {
    const bool odd = threadIdx.x & 1;
#pragma unroll
    for (int g = 0; g < 4; g += 2)
#pragma unroll
        for (int c = 0; c < 4; ++c) {
            const float r = __shfl_xor_sync(0xffffffffu, odd ? v[g][c] : v[g + 1][c], 1);
            v[g][c] = odd ? r : v[g][c];
            v[g + 1][c] = odd ? v[g + 1][c] : r;
        }
}
__device__ __forceinline__ int pair_column() { return 8 * (threadIdx.x & 1) + 4 * ((threadIdx.x & 3) >> 1); }

// kLate: an fp32 residual is read where it is added, for want of registers.
template <bool kF32, bool kLate>
struct FragmentEnd {
    uint4 slope[2], add[2];             // rows i and i + 8: group j
    float4 add32[kF32 && !kLate ? 2 : 1][2];
    bool in[2];

    __device__ __forceinline__ void load(const Ending& e, int64_t row, int64_t col0, int64_t rows) {
        const int j = threadIdx.x & 3;
        in[0] = row < rows;
        in[1] = row + 8 < rows;
        if (!kF32 && e.add) {
#pragma unroll
            for (int h = 0; h < 2; ++h)
                if (in[h]) add[h] = *reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(e.add) + (row + 8 * h) * e.ld_add + col0 + 8 * j);
        }
        if (kF32 && !kLate && e.add) {
#pragma unroll
            for (int h = 0; h < 2; ++h)
#pragma unroll
                for (int p = 0; p < 2; ++p)
                    if (in[h]) add32[h][p] = *reinterpret_cast<const float4*>(static_cast<const float*>(e.add) + (row + 8 * h) * e.ld_add + col0 + 16 * p + pair_column());
        }
        if (e.slope) {
#pragma unroll
            for (int h = 0; h < 2; ++h)
                if (in[h]) slope[h] = *reinterpret_cast<const uint4*>(e.slope + (row + 8 * h) * e.ld_slope + col0 + 8 * j);
        }
    }

    // bf16 rows i and i + 8 of the fragment, 16 bytes a lane
    __device__ __forceinline__ void store_bf16(uint16_t* q, int64_t ld, const float (&v)[4][4]) const {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            uint32_t w[4];
#pragma unroll
            for (int g = 0; g < 4; ++g) w[g] = pack_bf16x2(v[g][2 * h], v[g][2 * h + 1]);
            quad_transpose(w);
            if (in[h]) *reinterpret_cast<uint4*>(q + 8 * h * ld) = make_uint4(w[0], w[1], w[2], w[3]);
        }
    }

    __device__ __forceinline__ void finish(const Ending& e, uint32_t step, int64_t row, int64_t col0, float (&v)[4][4]) {
        const int j = threadIdx.x & 3;
        if (e.bias) {
#pragma unroll
            for (int g = 0; g < 4; ++g) {
                const uint32_t b = *reinterpret_cast<const uint32_t*>(e.bias + col0 + 8 * g + 2 * j);
                v[g][0] += bf16_lo(b); v[g][1] += bf16_hi(b);
                v[g][2] += bf16_lo(b); v[g][3] += bf16_hi(b);
            }
        }
        if (e.pre) store_bf16(e.pre + row * e.ld_pre + col0 + 8 * j, e.ld_pre, v);
        constexpr int kAtOnce = kF32 ? 1 : 4;   // groups whose chains interleave: the sums leave fp32 few registers
        if (e.slope) {
            quad_transpose(slope[0]);
            quad_transpose(slope[1]);
            const uint32_t w[2][4] = {{slope[0].x, slope[0].y, slope[0].z, slope[0].w}, {slope[1].x, slope[1].y, slope[1].z, slope[1].w}};
#pragma unroll
            for (int g = 0; g < 4; g += kAtOnce) {
                float t[kAtOnce][4];
#pragma unroll
                for (int i = 0; i < kAtOnce; ++i)
#pragma unroll
                    for (int h = 0; h < 2; ++h) t[i][2 * h] = bf16_lo(w[h][g + i]), t[i][2 * h + 1] = bf16_hi(w[h][g + i]);
                slope_apply<4 * kAtOnce>(e.act, t[0], v[g]);
            }
        } else if (e.act) {
#pragma unroll
            for (int g = 0; g < 4; g += kAtOnce) act_apply<4 * kAtOnce>(e.act, v[g]);
        }
        if (e.drop.cut) {
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                uint4 b = philox_block(e.drop, step, (uint32_t)(row + 8 * h), (uint32_t)((col0 >> 3) + j));
                quad_transpose(b);
                const uint32_t w[4] = {b.x, b.y, b.z, b.w};
#pragma unroll
                for (int g = 0; g < 4; ++g) {
                    v[g][2 * h] = (w[g] & 0xffffu) >= e.drop.cut ? v[g][2 * h] * e.drop.scale : 0.0f;
                    v[g][2 * h + 1] = (w[g] >> 16) >= e.drop.cut ? v[g][2 * h + 1] * e.drop.scale : 0.0f;
                }
            }
        }
        if constexpr (kF32) {
            // sixteen bytes a lane: a vector holds four columns of one group
            pair_exchange(v);
            const int64_t at = col0 + pair_column();
            float* q = static_cast<float*>(e.out) + row * e.ld_out + at;
            const float* r = static_cast<const float*>(e.add) + row * e.ld_add + at;
#pragma unroll
            for (int h = 0; h < 2; ++h, q += 8 * e.ld_out, r += 8 * e.ld_add) {
                if (!in[h]) continue;
                if (e.add) {
                    float4 t[2];
#pragma unroll
                    for (int p = 0; p < 2; ++p)
                        if constexpr (kLate)
                            t[p] = *reinterpret_cast<const float4*>(r + 16 * p);
                        else
                            t[p] = add32[h][p];
#pragma unroll
                    for (int p = 0; p < 2; ++p) {
                        v[2 * p][2 * h] += t[p].x;
                        v[2 * p][2 * h + 1] += t[p].y;
                        v[2 * p + 1][2 * h] += t[p].z;
                        v[2 * p + 1][2 * h + 1] += t[p].w;
                    }
                }
#pragma unroll
                for (int p = 0; p < 2; ++p)
                    *reinterpret_cast<float4*>(q + 16 * p) =
                        make_float4(v[2 * p][2 * h], v[2 * p][2 * h + 1], v[2 * p + 1][2 * h], v[2 * p + 1][2 * h + 1]);
            }
        } else {
            if (e.add) {
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    quad_transpose(add[h]);
                    const uint32_t w[4] = {add[h].x, add[h].y, add[h].z, add[h].w};
#pragma unroll
                    for (int g = 0; g < 4; ++g) v[g][2 * h] += bf16_lo(w[g]), v[g][2 * h + 1] += bf16_hi(w[g]);
                }
            }
            store_bf16(static_cast<uint16_t*>(e.out) + row * e.ld_out + col0 + 8 * j, e.ld_out, v);
        }
    }
};

// The split kernel's end of eight whole, aligned columns.  load(): what it reads
// beside its accumulators, before they are there.
template <bool kF32>
struct VectorEnd {
    uint4 add[kF32 ? 2 : 1], slope;   // as loaded
    float bias[8];

    __device__ __forceinline__ void load(const Ending& e, int64_t row, int64_t col) {
        if (e.add) {
            const char* q = static_cast<const char*>(e.add) + (row * e.ld_add + col) * (kF32 ? 4 : 2);
            add[0] = reinterpret_cast<const uint4*>(q)[0];
            if constexpr (kF32) add[1] = reinterpret_cast<const uint4*>(q)[1];
        }
        if (e.slope) slope = *reinterpret_cast<const uint4*>(e.slope + row * e.ld_slope + col);
        if (e.bias) {
            unpack8(*reinterpret_cast<const uint4*>(e.bias + col), bias);
        } else {
#pragma unroll
            for (int j = 0; j < 8; ++j) bias[j] = 0.0f;
        }
    }

    __device__ __forceinline__ void finish(const Ending& e, uint32_t step, int64_t row, int64_t col, float (&v)[8]) {
        float t[8];
        if (e.bias) {
#pragma unroll
            for (int j = 0; j < 8; ++j) v[j] += bias[j];
        }
        if (e.pre) *reinterpret_cast<uint4*>(e.pre + row * e.ld_pre + col) = pack8(v);
        if (e.slope) {
            unpack8(slope, t);
            slope_apply<8>(e.act, t, v);
        } else if (e.act) {
            act_apply<8>(e.act, v);
        }
        if (e.drop.cut) drop8(e.drop, step, row, col >> 3, v);
        if (e.add) {
            raw8<kF32>(add, t);
#pragma unroll
            for (int j = 0; j < 8; ++j) v[j] += t[j];
        }
        store8(static_cast<char*>(e.out) + (row * e.ld_out + col) * (kF32 ? 4 : 2), kF32, v);
    }
};

__device__ __forceinline__ float element(float x) { return x; }
__device__ __forceinline__ float element(uint16_t x) { return bf16_one(x); }

// Rows that are not aligned, or whose columns end inside a group: a lane a column, row
// by row, so that a row's accesses still fall together.  v: this lane's accumulators
// of kRows rows; every lane of the warp calls.
template <bool kF32, int kRows>
__device__ __forceinline__ void end_rows(const Ending& e, uint32_t step, int64_t row0, int64_t col0, int64_t rows, int64_t cols,
                                         float (&v)[kRows]) {
    using T = typename std::conditional<kF32, float, uint16_t>::type;
    const int lane = threadIdx.x & 31;
    const int64_t col = col0 + lane;
    // rows that exist, none where the column does not: one comparison a row
    const int n = col < cols ? (rows - row0 < kRows ? (int)(rows - row0) : kRows) : 0;
    if (e.bias) {
        const float bias = col < cols ? bf16_one(e.bias[col]) : 0.0f;
#pragma unroll
        for (int r = 0; r < kRows; ++r) v[r] += bias;
    }
    if (!e.bare) {   // one branch for the common case of none of these
        float t[kRows];
        if (e.pre) {
            uint16_t* q = e.pre + row0 * e.ld_pre + col;
#pragma unroll
            for (int r = 0; r < kRows; ++r, q += e.ld_pre)
                if (r < n) *q = to_bf16(v[r]);
        }
        if (e.slope) {
            const uint16_t* q = e.slope + row0 * e.ld_slope + col;
#pragma unroll
            for (int r = 0; r < kRows; ++r, q += e.ld_slope) t[r] = r < n ? bf16_one(*q) : 0.0f;
            slope_apply<kRows>(e.act, t, v);
        } else if (e.act) {
            act_apply<kRows>(e.act, v);
        }
        if (e.drop.cut) {
#pragma unroll
            for (int r0 = 0; r0 < kRows; r0 += 8) {   // lane l forms the bits of row l % 8 and column group l / 8
                const uint4 block = philox_block(e.drop, step, (uint32_t)(row0 + r0 + (lane & 7)), (uint32_t)((col0 >> 3) + (lane >> 3)));
#pragma unroll
                for (int r = 0; r < 8; ++r) v[r0 + r] = row_bits(block, r) >= e.drop.cut ? v[r0 + r] * e.drop.scale : 0.0f;
            }
        }
        if (e.add) {
            const T* q = static_cast<const T*>(e.add) + row0 * e.ld_add + col;
#pragma unroll
            for (int r = 0; r < kRows; ++r, q += e.ld_add) t[r] = r < n ? element(*q) : 0.0f;
#pragma unroll
            for (int r = 0; r < kRows; ++r) v[r] += t[r];
        }
    }
    T* q = static_cast<T*>(e.out) + row0 * e.ld_out + col;
#pragma unroll
    for (int r = 0; r < kRows; ++r, q += e.ld_out)
        if (r < n) {
            if constexpr (kF32)
                *q = v[r];
            else
                *q = to_bf16(v[r]);
        }
}

// A unit of 8 rows x 32 columns whose parts stand at the same place `chunk` (and row r0
// of it) of the shared memories of CTAs first, first + stride, ..: added in that order,
// then to the end.  A warp together.
// last: the warp reads no more parts after this unit, and arrives at the cluster's
// barrier before its end and its stores.
template <bool kF32>
__device__ __forceinline__ void end_joined(const Ending& e, uint32_t step, const uint8_t* smem, uint32_t chunk, int r0, int64_t row0, int64_t col0,
                                           int64_t rows, int64_t cols, int parts, int first, int stride, bool last) {
    const int lane = threadIdx.x & 31;
    const uint32_t base = smem_addr(smem);
    if (e.vec && col0 + 32 <= cols) {
        // The unit is 1 KB on end in every part: read as it lies, 16 bytes a lane,
        // group g of row lane / 8 and group g ^ 4 four rows on; then lanes of even
        // g take their neighbour's half of the first row, the others of the second.
        // (Two loads of 32 scattered groups: 8 bytes a cycle from other CTAs.)
        const int g = (lane & 7) ^ ((r0 + (lane >> 3)) & 7);
        const bool odd = g & 1;
        const int64_t row = row0 + (lane >> 3) + (odd ? 4 : 0), col = col0 + (odd ? g ^ 4 : g) / 2 * 8;
        VectorEnd<kF32> end;
        if (row < rows) end.load(e, row, col);
        float4 s = make_float4(0.0f, 0.0f, 0.0f, 0.0f), t = s;
        if (parts == 1) {   // half the latency of a peer's
            const float4* own = reinterpret_cast<const float4*>(smem + chunk + r0 * 128) + lane;
            s = own[0];
            t = own[32];
        }
        constexpr int kFly = kF32 ? 2 : 4;   // parts whose loads fly together; an fp32 end has fewer registers
        for (int i = 0; parts > 1 && i < parts; i += kFly) {
            float4 x[kFly], y[kFly];
#pragma unroll
            for (int j = 0; j < kFly; ++j)
                if (i + j < parts) {
                    const uint32_t at = peer_addr(base + chunk, first + (i + j) * stride) + r0 * 128 + lane * 16;
                    x[j] = peer_load(at);
                    y[j] = peer_load(at + 512);
                }
#pragma unroll
            for (int j = 0; j < kFly; ++j)
                if (i + j < parts) {
                    s.x += x[j].x; s.y += x[j].y; s.z += x[j].z; s.w += x[j].w;
                    t.x += y[j].x; t.y += y[j].y; t.z += y[j].z; t.w += y[j].w;
                }
        }
        const float4 give = odd ? s : t, keep = odd ? t : s;
        const float4 got = make_float4(__shfl_xor_sync(0xffffffffu, give.x, 1), __shfl_xor_sync(0xffffffffu, give.y, 1),
                                       __shfl_xor_sync(0xffffffffu, give.z, 1), __shfl_xor_sync(0xffffffffu, give.w, 1));
        if (last) {
            __syncwarp();
            cluster_arrive();
        }
        const float4 lo = odd ? got : keep, hi = odd ? keep : got;
        float v[8] = {lo.x, lo.y, lo.z, lo.w, hi.x, hi.y, hi.z, hi.w};
        if (row < rows) end.finish(e, step, row, col, v);
    } else {
        float v[8] = {};
        if (parts == 1) {
            const uint8_t* own = smem + chunk + (lane & 3) * 4;
#pragma unroll
            for (int r = 0; r < 8; ++r) v[r] = *reinterpret_cast<const float*>(own + group_place(r0 + r, lane >> 2));
        }
        for (int i = 0; parts > 1 && i < parts; i += 2) {
            float x[2][8];
#pragma unroll
            for (int j = 0; j < 2; ++j)
                if (i + j < parts) {
                    const uint32_t at = peer_addr(base + chunk, first + (i + j) * stride) + (lane & 3) * 4;
#pragma unroll
                    for (int r = 0; r < 8; ++r) x[j][r] = peer_load1(at + group_place(r0 + r, lane >> 2));
                }
#pragma unroll
            for (int j = 0; j < 2; ++j)
                if (i + j < parts)
#pragma unroll
                    for (int r = 0; r < 8; ++r) v[r] += x[j][r];
        }
        if (last) {
            __syncwarp();
            cluster_arrive();
        }
        end_rows<kF32, 8>(e, step, row0, col0, rows, cols, v);
    }
}

// ---- waits -------------------------------------------------------------------------
constexpr long long kWaitCycles = 1ll << 31;   // SM cycles (about a second) before a wait gives up

__device__ __forceinline__ void l2_prefetch(const void* p) { asm volatile("prefetch.global.L2 [%0];" ::"l"(p)); }

// For a converged warp that goes on as a whole: every lane gets the same answer.
__device__ __forceinline__ bool warp_wait(uint64_t* bar, uint32_t parity) {
    if (__all_sync(0xffffffffu, mbar_try_wait(bar, parity))) return true;
    if (__all_sync(0xffffffffu, mbar_wait_bounded(bar, parity, kWaitCycles))) return true;
    atomicExch(&g_linear_status, ZERO_ETIMEOUT);
    return false;
}

// ---- the pair kernel -----------------------------------------------------------------
// Large aligned products: pairs of CTAs, each pair one 256 x bn tile at a time (its
// rows split between the two tensor memories, its B tile between the two shared
// memories), tiles taken in turn from a grouped order.  Warp 0 copies, warp 1 of the
// even CTA issues the products, warps 4..19 end the previous tile out of the other
// half of the tensor memory meanwhile.  Bound by the tensor core: 256 x 256 x 64 take 512
// cycles, in which 64 KB come in, what an SM's share of L2 gives; a CTA alone would need
// half as much again for the same products.  Launched from a graph, by how far
// the power limit lets the clock fall: 8192 x 8192 x 8192 in 567 to 619 us (1.78 to 1.94
// PFLOP/s; cuBLAS 545 to 604), 8192 x 1600 times 6400 x 1600 with the tanh GELU and its
// pre-activation in 102 us (1.65 PFLOP/s), with a bias alone in 90; in a program that
// makes other calls between, 119.
struct PairParams {
    CUtensorMap map_a, map_b;
    int64_t rows, cols, depth;
    int32_t tiles_m, tiles_n, bn, k_blocks;
    int32_t run;   // blocks after which an accumulator is handed over
    int32_t box_a; // rows of A that a K-major copy brings
    bool a_mn, b_mn;
    Ending e;
};

constexpr int kStageBytes = 32768;      // 128 rows of A and 128 of B, 64 reduced elements each
constexpr int kPairStages = 6;
constexpr int kEndWarps = 16;
constexpr int kPairThreads = 128 + 32 * kEndWarps;
constexpr int kChunkBytes = 4096;       // 32 x 32 fp32
constexpr int kUnitBytes = 2048;        // 16 x 32 fp32
constexpr int kPairSmem = 1024 + kPairStages * kStageBytes + kEndWarps * kUnitBytes + 256;
// fp32 results: the tensor core cuts its sums where an fp32 addition would round
// them, and 100 additions in a row were off by 1.6e-6 of the result, five times a
// plain fp32 sum's error.  Their accumulators are therefore read after at most kRun
// blocks and added up in registers (0.75e-6; the split kernel adds them up in tensor
// memory).  A bf16 result's sums run on: about 7e-8 of it a block, where its own
// rounding is 1.7e-3.
constexpr int kRun = 13;                // blocks of 64 reduced elements
constexpr int kUnits = 3;               // 16 x 32 parts that a warp sums so, in 48 registers; a fourth would spill
constexpr int kWidest = 256, kWidestRuns = kUnits * 4 * 16;
constexpr int kRasterRows = 8;          // row tiles that are gone through together

__device__ __forceinline__ void tile_place(const PairParams& p, int t, int* tm, int* tn) {
    const int per_group = kRasterRows * p.tiles_n;
    const int g = t / per_group, in = t - g * per_group, first = g * kRasterRows;
    const int size = p.tiles_m - first < kRasterRows ? p.tiles_m - first : kRasterRows;
    *tn = in / size;
    *tm = first + in - *tn * size;
}
__device__ __forceinline__ int tile_width(const PairParams& p, int tn) {   // columns of the tile, up to a multiple of 32
    const int64_t left = p.cols - (int64_t)tn * p.bn;
    return left >= p.bn ? p.bn : (int)((left + 31) / 32 * 32);
}

// A warp of either CTA is done reading an accumulator: one arrival at the even CTA.
__device__ __forceinline__ void release(uint64_t* bar) {
    tcgen05_fence_before();
    __syncwarp();
    if ((threadIdx.x & 31) == 0) peer_arrive(peer_addr(smem_addr(bar), 0));
}

template <bool kF32>
__device__ __forceinline__ void prefetch_sides(const PairParams& p, int t, uint32_t rank, int q, int h) {
    int tm, tn;
    tile_place(p, t, &tm, &tn);
    const int64_t row = (int64_t)tm * 256 + rank * 128 + q * 32 + (threadIdx.x & 31);
    if (row >= p.rows) return;
    const int n = tile_width(p, tn) / 32;
    for (int c = h; c < n; c += 4) {
        const int64_t col = (int64_t)tn * p.bn + c * 32;
        if (col >= p.cols) break;
        if (p.e.add) l2_prefetch(static_cast<const char*>(p.e.add) + (row * p.e.ld_add + col) * (kF32 ? 4 : 2));
        if (p.e.slope) l2_prefetch(p.e.slope + row * p.e.ld_slope + col);
    }
}

// 16 rows x 32 columns that are not aligned or not whole: through 2 KB of shared
// memory to a lane a column.
template <bool kF32>
__device__ __forceinline__ void end_staged(const Ending& e, uint32_t step, int64_t row0, int64_t col0, int64_t rows, int64_t cols,
                                           const float (&v)[4][4], uint8_t* chunk) {
    const int lane = threadIdx.x & 31, i = lane >> 2, j = lane & 3;
    __syncwarp();   // the last unit's readers are done
#pragma unroll
    for (int g = 0; g < 4; ++g) {
        const int group = 2 * g + (j >> 1), in = (j & 1) * 8;
        *reinterpret_cast<float2*>(chunk + group_place(i, group) + in) = make_float2(v[g][0], v[g][1]);
        *reinterpret_cast<float2*>(chunk + group_place(i + 8, group) + in) = make_float2(v[g][2], v[g][3]);
    }
    __syncwarp();
    float t[16];
#pragma unroll
    for (int r = 0; r < 16; ++r) t[r] = *reinterpret_cast<const float*>(chunk + group_place(r, lane >> 2) + (lane & 3) * 4);
    end_rows<kF32, 16>(e, step, row0, col0, rows, cols, t);
}

// kRuns: fp32 results of more than one run, added up in registers.
template <bool kF32, bool kRuns>
__global__ void __launch_bounds__(kPairThreads, 1) pair_kernel(const __grid_constant__ PairParams p) {
    extern __shared__ uint8_t raw_smem[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(raw_smem) + 1023) & ~(uintptr_t)1023);
    uint8_t* chunks = smem + kPairStages * kStageBytes;
    uint64_t* full = reinterpret_cast<uint64_t*>(chunks + kEndWarps * kUnitBytes);
    uint64_t* empty = full + kPairStages;
    uint64_t* acc_full = empty + kPairStages;
    uint64_t* acc_empty = acc_full + 2;
    uint64_t* drained = acc_empty + 2;
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(drained + 1);

    const int warp = uniform_warp(), lane = threadIdx.x & 31;
    const uint32_t rank = cluster_rank();
    const int pair = blockIdx.x / 2, pairs = gridDim.x / 2;
    const int tiles = p.tiles_m * p.tiles_n;

    if (threadIdx.x == 0) {
        for (int s = 0; s < kPairStages; ++s) {
            mbar_init(full + s, 1);
            mbar_init(empty + s, 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(acc_full + i, 1);
            mbar_init(acc_empty + i, 2 * kEndWarps);
        }
        mbar_init(drained, 1);
        fence_barrier_init();
        tensor_map_prefetch(&p.map_a);
        tensor_map_prefetch(&p.map_b);
    }
    if (warp == 2) tmem_alloc<true>(tmem_slot, 512);
    tcgen05_fence_before();
    __syncthreads();
    cluster_started();
    tcgen05_fence_after();
    await_predecessor();
    const uint32_t tmem = *tmem_slot;

    const int half = p.bn / 2;
    const int b_boxes = p.b_mn ? (half + 63) / 64 : 1;
    const uint32_t stage_bytes = (p.a_mn ? 16384u : (uint32_t)p.box_a * 128u) + (p.b_mn ? (uint32_t)b_boxes * kSubTileBytes : (uint32_t)half * 128u);

    if (warp == 0) {
        int s = 0;
        uint32_t round = 0;
        bool ok = true;
        for (int t = pair; ok && t < tiles; t += pairs) {
            int tm, tn;
            tile_place(p, t, &tm, &tn);
            const int row = tm * 256 + (int)rank * 128;
            const int col = tn * p.bn + (int)rank * (tile_width(p, tn) / 2);
            for (int kb = 0; kb < p.k_blocks; ++kb) {
                if (round > 0 && !(ok = warp_wait(empty + s, (round - 1) & 1))) break;
                const uint32_t a = smem_addr(smem + s * kStageBytes), b = a + 16384;
                const uint32_t bar = peer_addr(smem_addr(full + s), 0);
                const int k = kb * 64;
                if (elect_one()) {
                    if (rank == 0) mbar_arrive_expect_tx(full + s, 2 * stage_bytes);
                    if (p.a_mn) {
                        tensor_load_pair(a, &p.map_a, row, k, bar);
                        tensor_load_pair(a + kSubTileBytes, &p.map_a, row + 64, k, bar);
                    } else {
                        tensor_load_pair(a, &p.map_a, k, row, bar);
                    }
                    if (p.b_mn) {
                        for (int i = 0; i < b_boxes; ++i) tensor_load_pair(b + i * kSubTileBytes, &p.map_b, col + 64 * i, k, bar);
                    } else {
                        tensor_load_pair(b, &p.map_b, k, col, bar);
                    }
                }
                if (++s == kPairStages) s = 0, ++round;
            }
        }
        if (!ok && rank == 0)   // copies in flight land before the CTAs end
            for (int i = 0; i < kPairStages; ++i) {
                const uint32_t done = i < s ? round : round - 1;   // the last round issued on stage i
                if (round > 0 || i < s) (void)mbar_wait_bounded(full + i, done & 1, kWaitCycles / 8);
            }
    } else if (warp == 1 && rank == 0) {
        int s = 0, use = 0;   // use: accumulators handed over so far
        uint32_t round = 0;
        bool ok = true;
        const uint32_t a_step = descriptor_step(p.a_mn), b_step = descriptor_step(p.b_mn);
        for (int t = pair; ok && t < tiles; t += pairs) {
            int tm, tn;
            tile_place(p, t, &tm, &tn);
            const uint32_t idesc = instruction_descriptor(256, tile_width(p, tn), p.a_mn, p.b_mn);
            for (int first = 0; ok && first < p.k_blocks; first += p.run, ++use) {
                const int buf = use & 1, end = first + p.run < p.k_blocks ? first + p.run : p.k_blocks;
                if (use >= 2 && !(ok = warp_wait(acc_empty + buf, (use / 2 - 1) & 1))) break;
                tcgen05_fence_after();
                const uint32_t d = tmem + buf * 256;
                for (int kb = first; kb < end; ++kb) {
                    if (!(ok = warp_wait(full + s, round & 1))) break;
                    tcgen05_fence_after();
                    const uint32_t a = smem_addr(smem + s * kStageBytes);
                    const uint64_t da = smem_descriptor(a, p.a_mn), db = smem_descriptor(a + 16384, p.b_mn);
                    const int64_t left = p.depth - (int64_t)kb * 64;
                    if (elect_one()) {
#pragma unroll
                        for (int i = 0; i < 4; ++i)   // the last step of all may end early
                            if (left > 16 * i) mma_bf16<true>(d, da + i * a_step, db + i * b_step, idesc, kb > first || i > 0);
                        mma_commit<true>(empty + s);
                    }
                    if (++s == kPairStages) s = 0, ++round;
                }
                if (ok && elect_one()) mma_commit<true>(acc_full + buf);
            }
        }
        if (!ok) {   // products in flight end before the tensor memory is freed
            if (elect_one()) mma_commit<true>(drained);
            (void)mbar_wait_bounded(drained, 0, kWaitCycles / 8);
        }
    } else if (warp >= 4) {
        // units of 16 rows x 32 columns: of its 32 rows this warp ends one half, over one
        // half of the columns, side by side so that whole lines are written together
        const int w = warp - 4, q = warp & 3, h = w / 4;
        uint8_t* chunk = chunks + w * kUnitBytes;
        const uint32_t step = p.e.drop.cut ? drop_step(p.e.drop) : 0u;
        int use = 0;   // accumulators read so far
        bool ok = true;
        for (int t = pair; ok && t < tiles; t += pairs) {
            int tm, tn;
            tile_place(p, t, &tm, &tn);
            const int64_t row0 = (int64_t)tm * 256 + rank * 128 + q * 32, col_tile = (int64_t)tn * p.bn;
            const int chunks_n = tile_width(p, tn) / 32, first = (h >> 1) * ((chunks_n + 1) / 2);
            const int units = h >> 1 ? chunks_n - first : (chunks_n + 1) / 2;   // of this warp
            const int64_t row_u = row0 + (h & 1) * 16;
            // what the end reads beside the accumulators, on its way to L2 while the product
            // runs (a tile ahead was slower: the reads then stand in the operands' way)
            if (p.e.add || p.e.slope) prefetch_sides<kF32>(p, t, rank, q, h);
            const uint32_t lanes = tmem + ((uint32_t)(q * 32 + (h & 1) * 16) << 16);
            const auto place = [&](int buf, int u) { return lanes + buf * 256 + (first + u) * 32; };
            if constexpr (kRuns) {
                float acc[kUnits][4][4];
                for (int kb = 0; kb < p.k_blocks; kb += p.run, ++use) {
                    const int buf = use & 1;
                    if (!(ok = warp_wait(acc_full + buf, (use / 2) & 1))) break;
                    tcgen05_fence_after();
#pragma unroll
                    for (int i = 0; i < kUnits; ++i) {
                        if (i >= units) continue;
                        if (kb == 0) {
                            tmem_load_fragment(place(buf, i), acc[i]);
                        } else {
                            float v[4][4];
                            tmem_load_fragment(place(buf, i), v);
#pragma unroll
                            for (int g = 0; g < 16; ++g) acc[i][g / 4][g % 4] += v[g / 4][g % 4];
                        }
                    }
                    release(acc_empty + buf);
                }
                if (!ok) break;
#pragma unroll 1
                for (int u = 0; u < units; ++u) {   // one copy of the code: four outgrow the instruction cache
                    const int64_t col0 = col_tile + (first + u) * 32;
                    FragmentEnd<kF32, true> end;
                    if (p.e.vec && col0 + 32 <= p.cols) {
                        end.load(p.e, row_u + (lane >> 2), col0, p.rows);
                        end.finish(p.e, step, row_u + (lane >> 2), col0, acc[0]);
                    } else {
                        end_staged<kF32>(p.e, step, row_u, col0, p.rows, p.cols, acc[0], chunk);
                    }
#pragma unroll
                    for (int g = 0; g < 16; ++g)
#pragma unroll
                        for (int i = 0; i + 1 < kUnits; ++i) acc[i][g / 4][g % 4] = acc[i + 1][g / 4][g % 4];
                }
            } else {
                const int buf = use & 1;
                if (!(ok = warp_wait(acc_full + buf, (use / 2) & 1))) break;
                tcgen05_fence_after();
#pragma unroll 1
                for (int u = 0; u < units; ++u) {
                    const int64_t col0 = col_tile + (first + u) * 32;
                    const bool vec = p.e.vec && col0 + 32 <= p.cols;
                    FragmentEnd<kF32, false> end;
                    float v[4][4];
                    if (vec) end.load(p.e, row_u + (lane >> 2), col0, p.rows);
                    tmem_load_fragment(place(buf, u), v);
                    if (u + 1 == units) release(acc_empty + buf);   // this warp's last read
                    if (vec)
                        end.finish(p.e, step, row_u + (lane >> 2), col0, v);
                    else
                        end_staged<kF32>(p.e, step, row_u, col0, p.rows, p.cols, v, chunk);
                }
                if (units == 0) release(acc_empty + buf);   // a narrow last tile: no unit for this warp
                ++use;
            }
        }
    }
    tcgen05_fence_before();
    __syncthreads();
    cluster_sync();
    tcgen05_fence_after();
    if (warp == 2) tmem_free<true>(tmem, 512);
}

// ---- the split kernel ------------------------------------------------------------------
// Smaller products, and those whose operands are not aligned: a 128 x bn tile a
// cluster, its reduced dimension split over the cluster's CTAs.  Each CTA leaves its
// part in its shared memory; the parts are added in the order of the CTAs (so the
// result repeats) while the end is applied.  Bound by latency where it is small (64 x 1600
// times 1600 x 1600 in 5.7 us, of which the start, the first copies, the two cluster
// barriers and the join take two thirds) and by L2 or the weights' bytes where it is not
// (128 x 4096 times 11008 x 4096 in 22 us, 4.1 TB/s of weights).
// kSoft: warps 0..7 bring the tiles by 16-byte copies and realign them, in place of
// tensor-map copies, which start on 16-byte boundaries only.
struct SplitParams {
    CUtensorMap map_a, map_b;
    Operand a, b;
    int64_t rows, cols, depth;
    int32_t tiles_m, tiles_n, bn, k_blocks, box_a;
    int32_t run;   // kRuns: blocks after which the accumulator is added to the total
    Ending e;
};

constexpr int kSplitStages = 3;
constexpr int kSplitThreads = 288;
constexpr int kSplitSmem = 1024 + kSplitStages * kStageBytes + 128;
constexpr int kSoftSmem = 1024 + kStageBytes + 2 * (256 * 144) + 128;

// What one of the 8 loading warps brings of an operand's tile: sub-tile rows r with
// r % 8 == warp, 16 of them, 64 elements each from any element-aligned place.  K-major,
// sub-tile row r is tile row r; MN-major, reduced row r % 64 at kept elements
// 64 (r / 64) on.  Rows 8 apart lie 16 ld bytes apart, so a warp's rows all start at the
// same place `shift` of a 16-byte block.  The eight or nine blocks that hold a row come
// by asynchronous copies, a stage ahead, to a raw buffer of 144 bytes a row; from there
// each lane takes the two that hold its 8 elements, and a funnel shift a word puts them
// in place, by branches that the warp takes together.  4095 x 1601 times 4097 x 1601:
// 224 us, against 257 with each lane's two blocks loaded straight to registers (2047 x
// 1599 times 1601 x 1599: 62 and 70; 333 x 500 x 9869: 42 and 50; small ones alike).
// Blocks hold up to 7 elements before and after a row's own, its neighbours'; where one
// would reach past the operand's own memory its elements come one by one.
constexpr int kRawPitch = 144, kRawBytes = 256 * kRawPitch;   // 128 rows of A, 128 of B

__device__ __forceinline__ void copy_block(uint32_t dst, uintptr_t src, bool want) {   // zeros where not wanted
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(want ? 16 : 0) : "memory");
}
__device__ __forceinline__ void copies_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int kLeft>
__device__ __forceinline__ void copies_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(kLeft) : "memory"); }

__device__ __noinline__ void fetch_block(uint32_t dst, uintptr_t at, uintptr_t begin, uintptr_t end) {
    uint32_t w[4] = {0u, 0u, 0u, 0u};
#pragma unroll
    for (int i = 0; i < 8; ++i)
        if (at + 2 * i >= begin && at + 2 * i < end)
            w[i / 2] |= (uint32_t)*reinterpret_cast<const uint16_t*>(at + 2 * i) << (16 * (i & 1));
    asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(dst), "r"(w[0]), "r"(w[1]), "r"(w[2]), "r"(w[3]) : "memory");
}

// A lane's blocks of 16 rows of 9: block i = lane + 32 c, of row i / 9.
struct LaneBlocks {
    uint32_t to[5];   // in a raw buffer
    __device__ __forceinline__ static int row(int c) { return (int)((threadIdx.x & 31) + 32 * c) / 9; }
    __device__ __forceinline__ static int block(int c) { return (int)((threadIdx.x & 31) + 32 * c) - 9 * row(c); }
    __device__ __forceinline__ explicit LaneBlocks(int warp) {
#pragma unroll
        for (int c = 0; c < 5; ++c) to[c] = (uint32_t)((warp + 8 * row(c)) * kRawPitch + 16 * block(c));
    }
};

template <bool kMn>
struct SoftTile {
    uintptr_t from[5];          // this lane's blocks in the next stage
    int64_t step;               // bytes to the stage after
    int extent;                 // kept elements from the tile's first, at most 128
    uint32_t shift;             // bytes
    uint32_t mine;              // which of the lane's blocks hold an element, in a whole stage
    int n;                      // sub-tile rows that are wanted

    __device__ __forceinline__ SoftTile(const Operand& o, int64_t mn0, int64_t k0, int rows, int warp) : n(rows) {
        const uintptr_t q = reinterpret_cast<uintptr_t>(o.p + ((kMn ? k0 : mn0) + warp) * o.ld + (kMn ? mn0 : k0));
        const int64_t left = (kMn ? o.cols : o.rows) - mn0, pitch = 16 * o.ld;   // pitch: to 8 rows on
        shift = (uint32_t)(q & 15);
        extent = left < 128 ? (int)left : 128;
        step = kMn ? 8 * pitch : 128;
        mine = 0;
#pragma unroll
        for (int c = 0; c < 5; ++c) {
            const int t = LaneBlocks::row(c), g = LaneBlocks::block(c);
            from[c] = q - shift + (kMn ? (t & 7) * pitch + (t >> 3) * 128 : t * pitch) + 16 * g;
            if (t < 16 && 8 * t < n && wanted(count(t, 64, warp), g)) mine |= 1u << c;
        }
    }
    // how many of the 64 elements of row t of 16 exist, `left` reduced ones from here
    // on (at least 64: all)
    __device__ __forceinline__ int count(int t, int left, int warp) const {
        if (kMn) return warp + 8 * (t & 7) < left ? extent - (t >> 3) * 64 : 0;
        return warp + 8 * t < extent ? left : 0;
    }
    // whether block g holds any of a row's first `have` elements
    __device__ __forceinline__ bool wanted(int have, int g) const { return have > 0 && 16 * g < 2 * have + (int)shift && (g < 8 || shift); }
    // whether any block of a stage's tile (from mn0, k0) reaches past the operand's memory
    static __device__ __forceinline__ bool at_edge(const Operand& o, int64_t mn0, int64_t k0) {
        const int64_t r0 = kMn ? k0 : mn0, c0 = kMn ? mn0 : k0, r1 = r0 + (kMn ? 63 : 127), c1 = c0 + (kMn ? 127 : 63);
        const uintptr_t first = reinterpret_cast<uintptr_t>(o.p + r0 * o.ld + c0);
        const uintptr_t last = reinterpret_cast<uintptr_t>(o.p + (r1 < o.rows ? r1 : o.rows - 1) * o.ld + (c1 < o.cols ? c1 : o.cols - 1));
        return (first & ~(uintptr_t)15) < operand_begin(o) || (last & ~(uintptr_t)15) + 16 > operand_end(o);
    }
    // whole: the stage has 64 reduced elements and none of its blocks reaches past the
    // memory; the lane's addresses only move on (formed anew for each block:
    // 2900 cycles a stage, so 1100)
    __device__ __forceinline__ void bring(const Operand& o, const LaneBlocks& lb, bool whole, bool edge, int left, uint32_t raw, int warp) {
        if (whole) {
#pragma unroll
            for (int c = 0; c < 5; ++c) {
                if (mine >> c & 1) copy_block(raw + lb.to[c], from[c], true);
                from[c] += step;
            }
            return;
        }
#pragma unroll 1
        for (int c = 0; c < 5; ++c) {
            const int t = LaneBlocks::row(c), g = LaneBlocks::block(c);
            uintptr_t b = from[0];
            uint32_t dst = lb.to[0];
#pragma unroll
            for (int i = 1; i < 5; ++i)
                if (c == i) b = from[i], dst = lb.to[i];
            dst += raw;
            if (t < 16 && 8 * t < n) {
                const int have = count(t, left, warp);
                const bool want = wanted(have, g);
                if (edge && want && (b < operand_begin(o) || b + 16 > operand_end(o)))
                    fetch_block(dst, b, operand_begin(o), operand_end(o));
                else
                    copy_block(dst, b, want);
            }
        }
#pragma unroll
        for (int c = 0; c < 5; ++c) from[c] += step;
    }
    // Past the reduced dimension's end there have to be zeros; what is past the kept one's
    // (neighbours, or what the buffer held) only reaches results that are not stored.
    template <int kWords, bool kWhole>   // kWords: whole words of the shift
    __device__ __forceinline__ void place_shifted(int left, const uint8_t* raw, uint8_t* d, int warp) const {
        const int lane = threadIdx.x & 31, g = lane & 7;
        const uint32_t bits = (shift & 2) * 8;
        const uint8_t* s = raw + (warp + 8 * (lane >> 3)) * kRawPitch + 16 * g;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            if (32 * j >= n) break;
            const uint4 x = *reinterpret_cast<const uint4*>(s + 32 * kRawPitch * j);
            const uint4 y = *reinterpret_cast<const uint4*>(s + 32 * kRawPitch * j + 16);
            const uint32_t w[8] = {x.x, x.y, x.z, x.w, y.x, y.y, y.z, y.w};
            uint4 v = make_uint4(__funnelshift_r(w[kWords], w[kWords + 1], bits), __funnelshift_r(w[kWords + 1], w[kWords + 2], bits),
                                 __funnelshift_r(w[kWords + 2], w[kWords + 3], bits), __funnelshift_r(w[kWords + 3], w[kWords + 4], bits));
            if constexpr (!kWhole) {
                const int have = count(4 * j + (lane >> 3), left, warp) - 8 * g;
                if (have < 8) {
                    v.x &= have >= 2 ? 0xffffffffu : have == 1 ? 0xffffu : 0u;
                    v.y &= have >= 4 ? 0xffffffffu : have == 3 ? 0xffffu : 0u;
                    v.z &= have >= 6 ? 0xffffffffu : have == 5 ? 0xffffu : 0u;
                    v.w &= have == 7 ? 0xffffu : 0u;
                }
            }
            *reinterpret_cast<uint4*>(d + j * 4096) = v;
        }
    }
    template <bool kWhole>
    __device__ __forceinline__ void place(int left, const uint8_t* raw, uint8_t* dst, int warp) const {
        const int lane = threadIdx.x & 31;
        uint8_t* d = dst + (warp + 8 * (lane >> 3)) * 128 + (((lane & 7) ^ warp) << 4);   // row % 8 is the warp
        switch (shift >> 2) {
            case 0: place_shifted<0, kWhole>(left, raw, d, warp); break;
            case 1: place_shifted<1, kWhole>(left, raw, d, warp); break;
            case 2: place_shifted<2, kWhole>(left, raw, d, warp); break;
            default: place_shifted<3, kWhole>(left, raw, d, warp); break;
        }
    }
};

// A run of fp32 sums of 32 lanes x 32 columns has ended: acc, at `from`, joins the
// total at `to`, which the first run fills.
__device__ __forceinline__ void add_run(uint32_t from, uint32_t to, bool fill) {
#pragma unroll 1
    for (int c = 0; c < 32; c += 16) {
        float v[16], w[16];
        tmem_load16_of_two(from + c, to + c, v, w);
#pragma unroll
        for (int j = 0; j < 16; ++j) v[j] = fill ? v[j] : v[j] + w[j];
        tmem_store16(to + c, v);
    }
}

// kSoft: kCopied, or which operands the loading warps find MN-major.
// kRuns: fp32 results of parts longer than kRun blocks.  Their runs are added up in a
// second accumulator of the tensor memory, where no registers are taken from the
// loading warps: by those warps themselves, which have to wait for a block's products
// before they place the next one, or, where the tiles are copied, by warps 4..7, which
// have nothing else to do, while the copies of the next run come in.  Without it and
// with it: 64 x 16384 times 512 x 16384 11.7 and 12.0 us, off by 2.1e-6 and 0.65e-6 of
// the result; a 512 x 512 gradient over 65536 tokens 57.6 and 61.4 us, 9.1e-6 and
// 0.79e-6; 41 x 47 over 50257 tokens, unaligned, 66.4 and 69.8 us, 7.0e-6 and 0.77e-6.
enum { kCopied = 0, kSoftKK = 1, kSoftKMn = 2, kSoftMnMn = 3 };
template <bool kF32, int kSoft, bool kRuns>
__global__ void __launch_bounds__(kSplitThreads, 2) split_kernel(const __grid_constant__ SplitParams p) {
    extern __shared__ uint8_t raw_smem[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(raw_smem) + 1023) & ~(uintptr_t)1023);
    constexpr int kStages = kSoft ? 1 : kSplitStages;   // a stage's products are short beside its loads
    uint64_t* full = reinterpret_cast<uint64_t*>(smem + kStages * kStageBytes + (kSoft ? 2 * kRawBytes : 0));
    uint64_t* empty = full + kStages;
    uint64_t* acc_full = empty + kStages;
    uint64_t* run_full = acc_full + 1;
    uint64_t* run_empty = run_full + 1;
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(run_empty + 1);

    const int warp = uniform_warp(), lane = threadIdx.x & 31;
    const int parts = (int)cluster_size(), rank = (int)cluster_rank();
    const int tile = blockIdx.x / parts;
    const int tn = tile / p.tiles_m, tm = tile - tn * p.tiles_m;
    const int64_t row_tile = (int64_t)tm * 128, col_tile = (int64_t)tn * p.bn;
    const int kb0 = (int)((int64_t)p.k_blocks * rank / parts), kb1 = (int)((int64_t)p.k_blocks * (rank + 1) / parts);

    if (threadIdx.x == 0) {
        for (int s = 0; s < kStages; ++s) {
            mbar_init(full + s, kSoft ? 8 : 1);
            mbar_init(empty + s, 1);
        }
        mbar_init(acc_full, 1);
        if (kRuns && !kSoft) {
            mbar_init(run_full, 1);
            mbar_init(run_empty, 4);
        }
        fence_barrier_init();
        if (!kSoft) {
            tensor_map_prefetch(&p.map_a);
            tensor_map_prefetch(&p.map_b);
        }
    }
    constexpr uint32_t kTmemColumns = kRuns ? 256 : 128;
    if (warp == 8) tmem_alloc<false>(tmem_slot, kTmemColumns);
    tcgen05_fence_before();
    __syncthreads();
    tcgen05_fence_after();
    await_predecessor();
    const uint32_t tmem = *tmem_slot, total = tmem + 128;

    // Tile-map copies start each tile at another place of the reduced dimension: with
    // few rows all CTAs would otherwise ask for the same lines of A at the same time
    // (9 x 1600 times 4800 x 1600: 12.7 us; 16 rows, spread wider, 8).
    const int turn = kSoft || kb1 == kb0 ? 0 : tile % (kb1 - kb0);
    // sub-tile rows of a stage: tile rows (K-major), or 64 for every 64 columns
    const int a_left = p.rows - row_tile < 128 ? (int)(p.rows - row_tile) : 128;
    const int a_rows = p.a.mn ? (a_left + 63) / 64 * 64 : kSoft ? a_left : p.box_a;
    const int b_rows = p.b.mn ? (p.bn + 63) / 64 * 64 : p.bn;
    const int64_t cols_left = p.cols - col_tile;
    const int n_chunks = cols_left >= p.bn ? p.bn / 32 : (int)((cols_left + 31) / 32);
    const int q = warp & 3;   // the lanes of the tensor memory that a warp reads
    const uint32_t lanes = (uint32_t)(q * 32) << 16;
    const bool several = kRuns && kb1 - kb0 > p.run;   // runs
    bool ok = true;

    if (warp < 8) {
        if (kSoft) {
            int s = 0;
            uint32_t round = 0;
            SoftTile<kSoft == kSoftMnMn> ta(p.a, row_tile, (int64_t)kb0 * 64, a_rows, warp);
            SoftTile<kSoft != kSoftKK> tb(p.b, col_tile, (int64_t)kb0 * 64, b_rows, warp);
            uint8_t* raw = smem + kStages * kStageBytes;
            const auto left_at = [&](int kb) {
                const int64_t more = p.depth - (int64_t)kb * 64;
                return more < 64 ? (int)more : 64;
            };
            const LaneBlocks lb(warp);
            const auto bring = [&](int kb) {
                if (kb < kb1) {
                    // only the ends of the reduced dimension meet those of the memory
                    const bool ends = kb == 0 || kb >= p.k_blocks - 2;
                    const bool edge_a = ends && ta.at_edge(p.a, row_tile, (int64_t)kb * 64), edge_b = ends && tb.at_edge(p.b, col_tile, (int64_t)kb * 64);
                    const uint32_t to = smem_addr(raw + ((kb - kb0) & 1) * kRawBytes);
                    const int left = left_at(kb);
                    ta.bring(p.a, lb, left == 64 && !edge_a, edge_a, left, to, warp);
                    tb.bring(p.b, lb, left == 64 && !edge_b, edge_b, left, to + 128 * kRawPitch, warp);
                }
                copies_commit();   // a group a stage, empty past the last
            };
            bring(kb0);
            bring(kb0 + 1);
            int run_end = kb0 + p.run;
            for (int kb = kb0; kb < kb1; ++kb) {
                copies_wait<1>();
                __syncwarp();
                if (round > 0 && !(ok = warp_wait(empty + s, (round - 1) & 1))) break;
                if (kRuns && kb == run_end) {   // the run's products are done, the next one's come after this warp's arrival
                    tcgen05_fence_after();
                    if (q * 32 < a_left)
                        for (int c = warp / 4; c < n_chunks; c += 2) add_run(tmem + lanes + c * 32, total + lanes + c * 32, kb - kb0 == p.run);
                    tmem_stored();
                    tcgen05_fence_before();
                    run_end += p.run;
                }
                uint8_t* stage = smem + s * kStageBytes;
                const uint8_t* from = raw + ((kb - kb0) & 1) * kRawBytes;
                const int left = left_at(kb);
                if (left == 64) {
                    ta.template place<true>(left, from, stage, warp);
                    tb.template place<true>(left, from + 128 * kRawPitch, stage + 16384, warp);
                } else {
                    ta.template place<false>(left, from, stage, warp);
                    tb.template place<false>(left, from + 128 * kRawPitch, stage + 16384, warp);
                }
                fence_async_shared();
                __syncwarp();
                if (lane == 0) mbar_arrive(full + s);
                bring(kb + 2);   // where this stage's blocks were
                if (++s == kStages) s = 0, ++round;
            }
            copies_wait<0>();   // none are left but after a failed wait
        } else if (warp == 0) {
            int s = 0;
            uint32_t round = 0;
            const int a_boxes = p.a.mn ? a_rows / 64 : 1, b_boxes = p.b.mn ? b_rows / 64 : 1;
            for (int i = kb0; i < kb1; ++i) {
                const int kb = i + turn < kb1 ? i + turn : i + turn - (kb1 - kb0);
                if (round > 0 && !(ok = warp_wait(empty + s, (round - 1) & 1))) break;
                const uint32_t a = smem_addr(smem + s * kStageBytes), b = a + 16384, bar = smem_addr(full + s);
                const int k = kb * 64;
                if (elect_one()) {
                    mbar_arrive_expect_tx(full + s, (uint32_t)(a_rows + b_rows) * 128u);
                    if (p.a.mn) {
                        for (int j = 0; j < a_boxes; ++j) tensor_load(a + j * kSubTileBytes, &p.map_a, (int)row_tile + 64 * j, k, bar);
                    } else {
                        tensor_load(a, &p.map_a, k, (int)row_tile, bar);
                    }
                    if (p.b.mn) {
                        for (int j = 0; j < b_boxes; ++j) tensor_load(b + j * kSubTileBytes, &p.map_b, (int)col_tile + 64 * j, k, bar);
                    } else {
                        tensor_load(b, &p.map_b, k, (int)col_tile, bar);
                    }
                }
                if (++s == kStages) s = 0, ++round;
            }
            if (!ok)   // copies in flight land before the CTA ends
                for (int i = 0; i < kStages; ++i) {
                    const uint32_t done = i < s ? round : round - 1;
                    if (round > 0 || i < s) (void)mbar_wait_bounded(full + i, done & 1, kWaitCycles / 8);
                }
        } else if (kRuns && warp >= 4) {
            for (int n = p.run, i = 0; n < kb1 - kb0; n += p.run, ++i) {
                if (!(ok = warp_wait(run_full, i & 1))) break;
                tcgen05_fence_after();
                if (q * 32 < a_left)
                    for (int c = 0; c < n_chunks; ++c) add_run(tmem + lanes + c * 32, total + lanes + c * 32, i == 0);
                tmem_stored();
                tcgen05_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(run_empty);
            }
        }
    } else {
        int s = 0;
        uint32_t round = 0;
        const uint32_t idesc = instruction_descriptor(128, p.bn, p.a.mn, p.b.mn);
        const uint32_t a_step = descriptor_step(p.a.mn), b_step = descriptor_step(p.b.mn);
        int run_end = kb0 + p.run;
        uint32_t ended = 0;   // runs
        for (int n = kb0; n < kb1; ++n) {
            const int kb = n + turn < kb1 ? n + turn : n + turn - (kb1 - kb0);
            const bool next = kRuns && n == run_end;
            if (next) {   // the accumulator is handed over
                run_end += p.run;
                if (!kSoft) {
                    if (elect_one()) mma_commit<false>(run_full);
                    if (!(ok = warp_wait(run_empty, ended++ & 1))) break;
                    tcgen05_fence_after();
                }
            }
            const bool fresh = next || n == kb0;
            if (!(ok = warp_wait(full + s, round & 1))) break;
            tcgen05_fence_after();
            const uint32_t a = smem_addr(smem + s * kStageBytes);
            const uint64_t da = smem_descriptor(a, p.a.mn), db = smem_descriptor(a + 16384, p.b.mn);
            const int64_t left = p.depth - (int64_t)kb * 64;
            if (elect_one()) {
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    if (left > 16 * i) mma_bf16<false>(tmem, da + i * a_step, db + i * b_step, idesc, !fresh || i > 0);
                mma_commit<false>(empty + s);
            }
            if (++s == kStages) s = 0, ++round;
        }
        if (elect_one()) mma_commit<false>(acc_full);   // after a failed wait too: the tensor memory is free once it arrives
    }
    __syncwarp();
    ok = warp_wait(acc_full, 0) && ok;
    if (kRuns && !kSoft) {   // warps 0..3 read what warps 4..7 added up
        tcgen05_fence_before();
        __syncthreads();
    }
    tcgen05_fence_after();

    // this CTA's part to its shared memory, chunk (q, c) of the tile at 4 KB each
    if (warp < 8) {
        if (q * 32 < a_left) {
            for (int c = warp / 4; c < n_chunks; c += 2) {
                uint32_t acc[32];
                tmem_load32(tmem + lanes + c * 32, acc);
                if (several) {
                    uint32_t sum[32];
                    tmem_load32(total + lanes + c * 32, sum);
#pragma unroll
                    for (int j = 0; j < 32; ++j) acc[j] = __float_as_uint(__uint_as_float(sum[j]) + __uint_as_float(acc[j]));
                }
                uint8_t* chunk = smem + (q * 4 + c) * kChunkBytes;
#pragma unroll
                for (int g = 0; g < 8; ++g)
                    *reinterpret_cast<uint4*>(chunk + group_place(lane, g)) =
                        p.k_blocks ? make_uint4(acc[4 * g], acc[4 * g + 1], acc[4 * g + 2], acc[4 * g + 3]) : make_uint4(0u, 0u, 0u, 0u);
            }
        }
    }
    tcgen05_fence_before();
    __syncthreads();
    if (parts > 1) cluster_sync();
    tcgen05_fence_after();
    if (warp == 8) tmem_free<false>(tmem, kTmemColumns);

    const int units = (a_left + 7) / 8 * n_chunks, unit0 = warp * parts + rank;   // few units: over all CTAs
    if (warp < 8 && ok && unit0 < units) {
        const uint32_t step = p.e.drop.cut ? drop_step(p.e.drop) : 0u;
        for (int u = unit0; u < units; u += parts * 8) {
            const int rb = u / n_chunks, c = u - rb * n_chunks;   // rows 8 rb .., chunk column c
            const uint32_t chunk = ((rb / 4) * 4 + c) * kChunkBytes;
            const int r0 = (rb & 3) * 8;
            const int64_t row0 = row_tile + rb * 8, col0 = col_tile + c * 32;
            end_joined<kF32>(p.e, step, smem, chunk, r0, row0, col0, p.rows, p.cols, parts, 0, 1, parts > 1 && u + parts * 8 >= units);
        }
    } else if (parts > 1) {
        cluster_arrive();
    }
    __syncwarp();
    if (parts > 1) cluster_wait();   // the parts are read before their CTAs end
}

// ---- the deep kernel -------------------------------------------------------------------
// Few tiles with a long reduced dimension: the pair kernel's 256 x bn tile on a cluster
// of two or four pairs, each with a share of the reduced dimension and six stages of its
// own, joined like the split kernel's.  An operand's element is brought to half as many
// SMs as by the split kernel's tiles, whose copies meet the limit of L2 (about 53 bytes a
// cycle and SM), and more SMs work than there are whole tiles.  512 x 6400 times 1600 x
// 6400 in 16.1 us (650 TFLOP/s): 50 blocks at 390 cycles, of which the tensor core needs
// half, then some 10000 cycles of start, cluster barriers and join.  Bound by L2 while it
// runs and by the join, at ten bytes a cycle from another SM, where the sum is short.
constexpr int kDeepThreads = 576;   // 16 warps for the end, one for the products, one for the copies
constexpr int kDeepSmem = 1024 + kPairStages * kStageBytes + 256;

template <bool kF32>
__global__ void __launch_bounds__(kDeepThreads, 1) deep_kernel(const __grid_constant__ PairParams p) {
    extern __shared__ uint8_t raw_smem[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(raw_smem) + 1023) & ~(uintptr_t)1023);
    uint64_t* full = reinterpret_cast<uint64_t*>(smem + kPairStages * kStageBytes);
    uint64_t* empty = full + kPairStages;
    uint64_t* acc_full = empty + kPairStages;
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(acc_full + 1);

    const int warp = uniform_warp(), lane = threadIdx.x & 31;
    const int ctas = (int)cluster_size(), rank = (int)cluster_rank();
    const int parts = ctas / 2, part = rank / 2, half = rank & 1, even = rank & ~1;
    const int tile = blockIdx.x / ctas, tn = tile / p.tiles_m, tm = tile - tn * p.tiles_m;
    const int width = tile_width(p, tn);
    const int kb0 = (int)((int64_t)p.k_blocks * part / parts), kb1 = (int)((int64_t)p.k_blocks * (part + 1) / parts);

    if (threadIdx.x == 0) {
        for (int s = 0; s < kPairStages; ++s) {
            mbar_init(full + s, 1);
            mbar_init(empty + s, 1);
        }
        mbar_init(acc_full, 1);
        fence_barrier_init();
        tensor_map_prefetch(&p.map_a);
        tensor_map_prefetch(&p.map_b);
    }
    if (warp == 16) tmem_alloc<true>(tmem_slot, 256);
    tcgen05_fence_before();
    __syncthreads();
    cluster_started();
    tcgen05_fence_after();
    await_predecessor();
    const uint32_t tmem = *tmem_slot;
    bool ok = true;

    if (warp == 17) {
        int s = 0;
        uint32_t round = 0;
        const int own_b = p.bn / 2, b_boxes = p.b_mn ? (own_b + 63) / 64 : 1;
        const uint32_t stage_bytes = (p.a_mn ? 16384u : (uint32_t)p.box_a * 128u) + (p.b_mn ? (uint32_t)b_boxes * kSubTileBytes : (uint32_t)own_b * 128u);
        const int row = tm * 256 + half * 128, col = tn * p.bn + half * (width / 2);
        for (int kb = kb0; kb < kb1; ++kb) {
            if (round > 0 && !(ok = warp_wait(empty + s, (round - 1) & 1))) break;
            const uint32_t a = smem_addr(smem + s * kStageBytes), b = a + 16384;
            const uint32_t bar = peer_addr(smem_addr(full + s), even);
            const int k = kb * 64;
            if (elect_one()) {
                if (half == 0) mbar_arrive_expect_tx(full + s, 2 * stage_bytes);
                if (p.a_mn) {
                    tensor_load_pair(a, &p.map_a, row, k, bar);
                    tensor_load_pair(a + kSubTileBytes, &p.map_a, row + 64, k, bar);
                } else {
                    tensor_load_pair(a, &p.map_a, k, row, bar);
                }
                if (p.b_mn) {
                    for (int i = 0; i < b_boxes; ++i) tensor_load_pair(b + i * kSubTileBytes, &p.map_b, col + 64 * i, k, bar);
                } else {
                    tensor_load_pair(b, &p.map_b, k, col, bar);
                }
            }
            if (++s == kPairStages) s = 0, ++round;
        }
        if (!ok && half == 0)   // copies in flight land before the CTAs end
            for (int i = 0; i < kPairStages; ++i) {
                const uint32_t done = i < s ? round : round - 1;   // the last round issued on stage i
                if (round > 0 || i < s) (void)mbar_wait_bounded(full + i, done & 1, kWaitCycles / 8);
            }
    } else if (warp == 16 && half == 0) {
        int s = 0;
        uint32_t round = 0;
        const uint32_t idesc = instruction_descriptor(256, width, p.a_mn, p.b_mn);
        const uint32_t a_step = descriptor_step(p.a_mn), b_step = descriptor_step(p.b_mn);
        for (int kb = kb0; kb < kb1; ++kb) {
            if (!(ok = warp_wait(full + s, round & 1))) break;
            tcgen05_fence_after();
            const uint32_t a = smem_addr(smem + s * kStageBytes);
            const uint64_t da = smem_descriptor(a, p.a_mn), db = smem_descriptor(a + 16384, p.b_mn);
            const int64_t left = p.depth - (int64_t)kb * 64;
            if (elect_one()) {
#pragma unroll
                for (int i = 0; i < 4; ++i)   // the last step of all may end early
                    if (left > 16 * i) mma_bf16<true>(tmem, da + i * a_step, db + i * b_step, idesc, kb > kb0 || i > 0);
                mma_commit<true>(empty + s, 3u << even);
            }
            if (++s == kPairStages) s = 0, ++round;
        }
        if (elect_one()) mma_commit<true>(acc_full, 3u << even);   // after a failed wait too: the tensor memory is free once it arrives
    }
    __syncwarp();
    ok = warp_wait(acc_full, 0) && ok;
    tcgen05_fence_after();

    // this CTA's 128 rows of its pair's part, chunk (q, c) at 4 KB each, where the stages were
    const int64_t row_half = (int64_t)tm * 256 + half * 128, col_tile = (int64_t)tn * p.bn;
    const int rows_left = p.rows - row_half < 0 ? 0 : p.rows - row_half < 128 ? (int)(p.rows - row_half) : 128;
    const int n_chunks = width / 32;
    if (warp < 16 && ok) {
        const int q = warp & 3;
        if (q * 32 < rows_left) {
            for (int c = warp / 4; c < n_chunks; c += 4) {
                uint32_t acc[32];
                tmem_load32(tmem + c * 32 + ((uint32_t)(q * 32) << 16), acc);
                uint8_t* chunk = smem + (q * 8 + c) * kChunkBytes;
#pragma unroll
                for (int g = 0; g < 8; ++g)
                    *reinterpret_cast<uint4*>(chunk + group_place(lane, g)) = make_uint4(acc[4 * g], acc[4 * g + 1], acc[4 * g + 2], acc[4 * g + 3]);
            }
        }
    }
    tcgen05_fence_before();
    __syncthreads();
    cluster_sync();
    tcgen05_fence_after();
    if (warp == 16) tmem_free<true>(tmem, 256);

    const int units = (rows_left + 7) / 8 * n_chunks, unit0 = warp * parts + part;
    if (warp < 16 && ok && unit0 < units) {
        const uint32_t step = p.e.drop.cut ? drop_step(p.e.drop) : 0u;
        for (int u = unit0; u < units; u += parts * 16) {
            const int rb = u / n_chunks, c = u - rb * n_chunks;
            end_joined<kF32>(p.e, step, smem, ((rb / 4) * 8 + c) * kChunkBytes, (rb & 3) * 8, row_half + rb * 8, col_tile + c * 32, p.rows, p.cols,
                             parts, half, 2, u + parts * 16 >= units);
        }
    } else {
        cluster_arrive();
    }
    __syncwarp();
    cluster_wait();   // the parts are read before their CTAs end
}

// ---- launches -----------------------------------------------------------------------------

typedef CUresult (*EncodeTiled)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*, const cuuint64_t*,
                                const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                                CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

static EncodeTiled encode_tiled() {
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

// Whether tensor-map copies can read the operand: 16-byte aligned rows, and sizes
// and row pitch within the map's fields.
static bool copies_reach(const Operand& o) {
    return o.rows > 0 && o.cols > 0 && aligned16(o.p) && (o.rows == 1 || o.ld % 8 == 0) && o.rows < (1ll << 31) - 512 &&
           o.cols < (1ll << 31) - 512 && o.ld < (1ll << 38);
}
static bool make_map(const Operand& o, int box_rows, CUtensorMap* map) {
    const EncodeTiled encode = encode_tiled();
    if (!encode) return false;
    const cuuint64_t dims[2] = {(cuuint64_t)o.cols, (cuuint64_t)o.rows};
    const cuuint64_t pitch[1] = {(cuuint64_t)((o.ld + 7) / 8 * 16)};   // of a single row any
    const cuuint32_t box[2] = {64, (cuuint32_t)box_rows}, unit[2] = {1, 1};
    return encode(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<uint16_t*>(o.p), dims, pitch, box, unit,
                  CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                  CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// The current device, if there is one below `most`.  A failed question leaves no error
// behind: a caller goes on without the answer or reports it by its code.
static bool device_below(int most, int* dev) {
    const cudaError_t e = cudaGetDevice(dev);
    if (e != cudaSuccess) {
        note_cuda_error(e);
        (void)cudaGetLastError();
    }
    return e == cudaSuccess && *dev >= 0 && *dev < most;
}

// Raises a kernel's shared-memory limit, once per device (again after a failure).
typedef std::atomic<bool> Done[64];
static int allow_smem(const void* kernel, int bytes, Done& done) {
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

// What a launch takes and its estimated cycles, from the measured times of each
// kernel's phases on GB300; the least decides.  (Measured either way, in us, pair and
// split kernel: 333 x 1600 x 1600 8.8 and 8.4; 1024 x 1600 x 1600 9.2 and 13; 64 tokens
// by 4800 x 1600 10.7 and 7.1; its 64 x 1600 gradient 20 and 8.5.)
struct Plan {
    int64_t cycles, tiles_m, tiles_n;
    int bn, parts;
};

// Pairs of SMs; one where the runtime could not say how many there are.
static int64_t sm_pairs() {
    const int n = sm_count();
    return n < 2 ? 1 : n / 2;
}

// Waves of pairs, each a tile's blocks (bound by the tensor core, or for narrow tiles
// by shared memory) and the part of its end that nothing hides.
static Plan plan_pair(const Product& p, bool f32) {
    const int64_t pairs = sm_pairs(), k_blocks = (p.depth + 63) / 64;
    const int widest = f32 && k_blocks > kRun ? kWidestRuns : kWidest;
    Plan best{INT64_MAX, (p.rows + 255) / 256, 0, 0, 1};   // no width fits: not taken
    for (int bn = widest; bn >= 32; bn -= 32) {
        const int64_t tn = (p.cols + bn - 1) / bn;
        if (tn > INT32_MAX / 8 / best.tiles_m) break;
        const int64_t waves = (best.tiles_m * tn + pairs - 1) / pairs;
        const int64_t cycles = 4000 + waves * (1500 + k_blocks * (2 * bn > 256 + bn ? 2 * bn : 256 + bn) + 24 * bn);
        if (cycles < best.cycles) best.cycles = cycles, best.tiles_n = tn, best.bn = bn;
    }
    return best;
}

// Waves of CTAs, two to an SM: each a start, its blocks by the groups of 32 rows they
// bring, its share of the end, and the join.  Loading warps wait longer for a block
// than copies do and lose less to a second CTA beside them.
struct Costs {
    int start, group, end, crowd, join, part;   // crowd: percent more with two CTAs to each SM
};
static Plan plan_split(const Product& p, bool f32, bool soft) {
    const Costs t = soft ? Costs{5000, 300, 2500, 60, 2000, 300} : Costs{2000, 112, 11000, 90, 500, 1460};
    const int64_t sms = sm_count(), k_blocks = (p.depth + 63) / 64, rows = p.rows < 128 ? p.rows : 128;
    Plan best{INT64_MAX, (p.rows + 127) / 128, 0, 0, 1};
    for (int bn = 128; bn >= 32; bn /= 2) {
        const int64_t tn = (p.cols + bn - 1) / bn;
        if (tn > INT32_MAX / 8 / best.tiles_m) break;
        for (int n = 1; n <= 8 && (n == 1 || k_blocks >= 2 * n); n *= 2) {
            // fp32 results: more parts before several runs of the tensor core's sums in one
            if (f32 && n < 8 && k_blocks > (int64_t)n * kRun && k_blocks >= 4 * n) continue;
            const int64_t ctas = best.tiles_m * tn * n, waves = (ctas + 2 * sms - 1) / (2 * sms);
            const int64_t crowd = 100 + (ctas <= sms ? 0 : ctas >= 2 * sms ? t.crowd : t.crowd * (ctas - sms) / sms);
            const int64_t blocks = (k_blocks + n - 1) / n * (4 + bn / 32) * t.group + t.end * rows * bn / (128 * 128) / n;
            const int64_t cycles = waves * (t.start + blocks * crowd / 100 + (n > 1 ? t.join + t.part * rows * bn / (128 * 64) * n : 0));
            if (cycles < best.cycles) best.cycles = cycles, best.tiles_n = tn, best.bn = bn, best.parts = n;
        }
    }
    return best;
}

// Clusters of `pairs` pairs that run at the same time, once per device.
static int deep_clusters(const void* kernel, int pairs, std::atomic<int> (&known)[64]) {
    int dev = 0;
    if (!device_below(64, &dev)) return 0;
    int n = known[dev].load(std::memory_order_relaxed);
    if (n == 0) {
        cudaLaunchConfig_t c{};
        cudaLaunchAttribute a{};
        a.id = cudaLaunchAttributeClusterDimension;
        a.val.clusterDim.x = 2 * pairs;
        a.val.clusterDim.y = a.val.clusterDim.z = 1;
        c.gridDim = dim3((unsigned)(2 * pairs));
        c.blockDim = dim3(kDeepThreads);
        c.dynamicSmemBytes = kDeepSmem;
        c.attrs = &a;
        c.numAttrs = 1;
        const cudaError_t e = cudaOccupancyMaxActiveClusters(&n, kernel, &c);
        if (e != cudaSuccess) {
            note_cuda_error(e);
            (void)cudaGetLastError();
            n = 0;
        }
        if (n > 0) known[dev].store(n, std::memory_order_relaxed);
    }
    return n;
}

// Rows of A that a copy brings: no more than there are.  (Boxes of 128 rows over a
// matrix of 5 to 14 took two to three times as long as over one of 16.)
static int32_t box_rows(int64_t rows) { return rows < 128 ? (int32_t)((rows + 7) / 8 * 8) : 128; }

static int launch_pair(const Product& p, const Ending& e, const Plan& plan, cudaStream_t s) {
    static Done done[3];
    const int blocks = (int)((p.depth + 63) / 64), runs = e.out_f32 ? (blocks + kRun - 1) / kRun : 1;
    void (*kernel)(PairParams) = runs > 1 ? pair_kernel<true, true> : e.out_f32 ? pair_kernel<true, false> : pair_kernel<false, false>;
    if (const int rc = allow_smem((const void*)kernel, kPairSmem, done[runs > 1 ? 2 : e.out_f32])) return rc;
    PairParams q{};
    q.rows = p.rows; q.cols = p.cols; q.depth = p.depth;
    q.tiles_m = (int32_t)plan.tiles_m; q.tiles_n = (int32_t)plan.tiles_n; q.bn = plan.bn;
    q.k_blocks = blocks;
    q.run = (q.k_blocks + runs - 1) / runs;
    q.a_mn = p.a.mn; q.b_mn = p.b.mn;
    q.e = e;
    q.box_a = box_rows(p.rows);
    if (!make_map(p.a, p.a.mn ? 64 : q.box_a, &q.map_a) || !make_map(p.b, p.b.mn ? 64 : q.bn / 2, &q.map_b)) return ZERO_ECUDA;
    const int64_t tiles = plan.tiles_m * plan.tiles_n, pairs = sm_pairs();
    return launch_dense(kernel, dim3((unsigned)(2 * (tiles < pairs ? tiles : pairs))), kPairThreads, 2, true, kPairSmem, s, q);
}

// Waves of clusters of pairs, as many at a time as the SMs' groups hold: a start, the
// share's blocks, and the join at about ten bytes a cycle from other SMs.  Not for up to
// 64 rows, of which the split kernel's copies bring no more than there are.  (Measured
// without and with this kernel, in us: 256 x 11008 times 4096 x 11008 36.9 and 26.7;
// 512 x 6400 times 1600 x 6400 21.9 and 16.1; 1024 x 16384 times 1600 x 16384 55 and 38.6;
// 64 x 11008 times 4096 x 11008 21.4 and 24.3; 384 x 4096 times 4096 x 4096 17.4 and 19.1.)
static Plan plan_deep(const Product& p, bool f32) {
    static Done done[2];
    static std::atomic<int> at_once[2][2][64];
    const void* kernel = f32 ? (const void*)deep_kernel<true> : (const void*)deep_kernel<false>;
    const int64_t k_blocks = (p.depth + 63) / 64;
    Plan best{INT64_MAX, (p.rows + 255) / 256, 0, 0, 0};
    if (p.rows <= 64 || k_blocks < 8 || k_blocks > INT32_MAX || allow_smem(kernel, kDeepSmem, done[f32]) != ZERO_OK) return best;
    for (int n = 2; n <= 4; n *= 2) {
        const int64_t clusters = deep_clusters(kernel, n, at_once[f32][n / 4]), blocks = (k_blocks + n - 1) / n;
        if (clusters <= 0 || (f32 && blocks > kRun)) continue;   // fp32 results: short runs, as in the pair kernel
        for (int bn = 64; bn <= kWidest; bn += 32) {
            const int64_t tn = (p.cols + bn - 1) / bn;
            if (tn > INT32_MAX / 16 / best.tiles_m) continue;
            const int64_t waves = (best.tiles_m * tn + clusters - 1) / clusters;
            const int64_t join = 3000 + 512 * bn * (n - 1) / n / 10;
            const int64_t cycles = 5500 + waves * (2000 + blocks * (2 * bn > 256 + bn ? 2 * bn : 256 + bn) * 11 / 10 + join);
            if (cycles < best.cycles) best.cycles = cycles, best.tiles_n = tn, best.bn = bn, best.parts = n;
        }
    }
    return best;
}

static int launch_deep(const Product& p, const Ending& e, const Plan& plan, cudaStream_t s) {
    PairParams q{};
    q.rows = p.rows; q.cols = p.cols; q.depth = p.depth;
    q.tiles_m = (int32_t)plan.tiles_m; q.tiles_n = (int32_t)plan.tiles_n; q.bn = plan.bn;
    q.k_blocks = (int32_t)((p.depth + 63) / 64);
    q.a_mn = p.a.mn; q.b_mn = p.b.mn;
    q.e = e;
    q.box_a = box_rows(p.rows);
    if (!make_map(p.a, p.a.mn ? 64 : q.box_a, &q.map_a) || !make_map(p.b, p.b.mn ? 64 : q.bn / 2, &q.map_b)) return ZERO_ECUDA;
    return launch_dense(e.out_f32 ? deep_kernel<true> : deep_kernel<false>, dim3((unsigned)(plan.tiles_m * plan.tiles_n * plan.parts * 2)),
                        kDeepThreads, (unsigned)plan.parts * 2, true, kDeepSmem, s, q);
}

static int launch_split(const Product& p, const Ending& e, const Plan& plan, bool soft, cudaStream_t s) {
    static Done done[12];
    static void (*const kernels[3][4])(SplitParams) = {
        {split_kernel<false, kCopied, false>, split_kernel<false, kSoftKK, false>, split_kernel<false, kSoftKMn, false>, split_kernel<false, kSoftMnMn, false>},
        {split_kernel<true, kCopied, false>, split_kernel<true, kSoftKK, false>, split_kernel<true, kSoftKMn, false>, split_kernel<true, kSoftMnMn, false>},
        {split_kernel<true, kCopied, true>, split_kernel<true, kSoftKK, true>, split_kernel<true, kSoftKMn, true>, split_kernel<true, kSoftMnMn, true>}};
    const int64_t k_blocks = (p.depth + 63) / 64;
    if (!plan.tiles_n || k_blocks > INT32_MAX) return ZERO_ERANGE;
    const int64_t longest = (k_blocks + plan.parts - 1) / plan.parts, runs = (longest + kRun - 1) / kRun;   // of a part
    const int kind = !soft ? kCopied : p.a.mn ? kSoftMnMn : p.b.mn ? kSoftKMn : kSoftKK, which = !e.out_f32 ? 0 : runs <= 1 ? 1 : 2;
    void (*kernel)(SplitParams) = kernels[which][kind];
    const int smem = soft ? kSoftSmem : kSplitSmem;
    if (const int rc = allow_smem((const void*)kernel, smem, done[which * 4 + kind])) return rc;
    SplitParams q{};
    q.a = p.a; q.b = p.b;
    q.rows = p.rows; q.cols = p.cols; q.depth = p.depth;
    q.tiles_m = (int32_t)plan.tiles_m; q.tiles_n = (int32_t)plan.tiles_n; q.bn = plan.bn; q.k_blocks = (int32_t)k_blocks;
    q.run = (int32_t)((longest + runs - 1) / runs);
    q.e = e;
    q.box_a = box_rows(p.rows);
    if (!soft && (!make_map(p.a, p.a.mn ? 64 : q.box_a, &q.map_a) || !make_map(p.b, p.b.mn ? 64 : q.bn, &q.map_b))) return ZERO_ECUDA;
    return launch_dense(kernel, dim3((unsigned)(plan.tiles_m * plan.tiles_n * plan.parts)), kSplitThreads, (unsigned)plan.parts, true,
                        smem, s, q);
}

static int launch_product(const Product& p, Ending& e, cudaStream_t s) {
    const int size = e.out_f32 ? 4 : 2;
    e.vec = aligned16(e.bias) && (!e.slope || rows_aligned16(e.slope, e.ld_slope, 2)) && (!e.pre || rows_aligned16(e.pre, e.ld_pre, 2)) &&
            (!e.add || rows_aligned16(e.add, e.ld_add, size)) && rows_aligned16(e.out, e.ld_out, size);
    e.bare = !e.pre && !e.slope && !e.act && !e.drop.cut && !e.add;
    if ((p.rows + 127) / 128 > INT32_MAX / 64) return ZERO_ERANGE;
    const bool reach = copies_reach(p.a) && copies_reach(p.b);
    const Plan split = plan_split(p, e.out_f32, !reach), pair = reach ? plan_pair(p, e.out_f32) : Plan{INT64_MAX, 0, 0, 0, 0};
    const Plan deep = reach ? plan_deep(p, e.out_f32) : Plan{INT64_MAX, 0, 0, 0, 0};
    const int64_t whole = pair.cycles < split.cycles ? pair.cycles : split.cycles, tiled = deep.cycles < whole ? deep.cycles : whole;
    // The kernel of a few rows reads the weights at about 2950 bytes a cycle for one row
    // (weights 4800 x 1600, in L2, 4.9 us, 6.7 by tiles; 4096 x 11008 16.4 and 18.6) and
    // half of it for more.  One row always goes there: the one size found where tiles
    // are faster, 11008 x 4096, 21 and 19, is not told apart by the estimates.
    if (p.rows <= kMostRows && !p.a.mn && !p.b.mn) {
        const int64_t read = p.cols * (p.depth / 8) * 16 / 2950;
        if (p.rows == 1 || 3000 + read * (p.rows == 2 ? 14 : 23) / 10 < tiled) return launch_rows(p, e, s);
    }
    if (deep.cycles < whole) return launch_deep(p, e, deep, s);
    return pair.cycles < split.cycles ? launch_pair(p, e, pair, s) : launch_split(p, e, split, !reach, s);
}

static bool act_ok(int32_t act) { return act >= ZERO_ACT_NONE && act <= ZERO_ACT_SILU; }
static bool dtype_ok(int32_t d) { return d == ZERO_BF16 || d == ZERO_F32; }

}  // namespace zgb

extern "C" int zero_linear(int64_t m, int64_t n, int64_t k, const uint16_t* x, int64_t ldx, const uint16_t* w,
                           int64_t ldw, const uint16_t* bias, int32_t act, const zero_dropout_t* drop,
                           const void* residual, int64_t ldr, uint16_t* pre, int64_t ldp, void* y,
                           int32_t y_dtype, int64_t ldy, void* stream) {
    using namespace zgb;
    if (m < 0 || n < 0 || k < 0 || !act_ok(act) || !dtype_ok(y_dtype)) return ZERO_EINVAL;
    Ending e{};
    if (const int rc = drop_params(drop, m, n, &e.drop)) return rc;
    if (const int rc = check_matrix(x, m, k, ldx, ZERO_BF16)) return rc;
    if (const int rc = check_matrix(w, n, k, ldw, ZERO_BF16)) return rc;
    if (const int rc = check_matrix(y, m, n, ldy, y_dtype)) return rc;
    if (residual)
        if (const int rc = check_matrix(residual, m, n, ldr, y_dtype)) return rc;
    if (pre)
        if (const int rc = check_matrix(pre, m, n, ldp, ZERO_BF16)) return rc;
    if (check_aligned(bias, 2)) return ZERO_EALIGN;
    if (m == 0 || n == 0) return ZERO_OK;
    if ((k && (check_device_ptr(x) || check_device_ptr(w))) || check_device_ptr(y) ||
        (bias && check_device_ptr(bias)) || (residual && check_device_ptr(residual)) ||
        (pre && check_device_ptr(pre)) || (e.drop.step_ptr && check_device_ptr(e.drop.step_ptr)))
        return ZERO_EINVAL;
    e.bias = bias;
    e.pre = pre; e.ld_pre = ldp;
    e.add = residual; e.ld_add = ldr;
    e.out = y; e.ld_out = ldy; e.out_f32 = y_dtype == ZERO_F32;
    e.act = act;
    return launch_product(Product{m, n, k, {x, ldx, m, k, false}, {w, ldw, n, k, false}}, e, static_cast<cudaStream_t>(stream));
}

extern "C" int zero_linear_grad_input(int64_t m, int64_t n, int64_t k, const uint16_t* dz, int64_t lddz,
                                      const uint16_t* w, int64_t ldw, int32_t act, const zero_dropout_t* drop,
                                      const uint16_t* pre, int64_t ldp, const void* residual, int64_t ldr,
                                      void* dx, int32_t dx_dtype, int64_t lddx, void* stream) {
    using namespace zgb;
    if (m < 0 || n < 0 || k < 0 || !act_ok(act) || !dtype_ok(dx_dtype)) return ZERO_EINVAL;
    if ((act != ZERO_ACT_NONE) != (pre != nullptr) && m && k) return ZERO_EINVAL;
    Ending e{};
    if (const int rc = drop_params(drop, m, k, &e.drop)) return rc;
    if (const int rc = check_matrix(dz, m, n, lddz, ZERO_BF16)) return rc;
    if (const int rc = check_matrix(w, n, k, ldw, ZERO_BF16)) return rc;
    if (const int rc = check_matrix(dx, m, k, lddx, dx_dtype)) return rc;
    if (pre)
        if (const int rc = check_matrix(pre, m, k, ldp, ZERO_BF16)) return rc;
    if (residual)
        if (const int rc = check_matrix(residual, m, k, ldr, dx_dtype)) return rc;
    if (m == 0 || k == 0) return ZERO_OK;
    if ((n && (check_device_ptr(dz) || check_device_ptr(w))) || check_device_ptr(dx) ||
        (pre && check_device_ptr(pre)) || (residual && check_device_ptr(residual)) ||
        (e.drop.step_ptr && check_device_ptr(e.drop.step_ptr)))
        return ZERO_EINVAL;
    e.slope = pre; e.ld_slope = ldp;
    e.add = residual; e.ld_add = ldr;
    e.out = dx; e.ld_out = lddx; e.out_f32 = dx_dtype == ZERO_F32;
    e.act = act;
    return launch_product(Product{m, k, n, {dz, lddz, m, n, false}, {w, ldw, n, k, true}}, e, static_cast<cudaStream_t>(stream));
}

extern "C" int zero_linear_grad_weight(int64_t m, int64_t n, int64_t k, const uint16_t* dz, int64_t lddz,
                                       const uint16_t* x, int64_t ldx, const void* acc, int64_t ldacc,
                                       void* dw, int32_t dw_dtype, int64_t lddw, const void* db_acc, void* db,
                                       void* stream) {
    using namespace zgb;
    if (m < 0 || n < 0 || k < 0 || !dtype_ok(dw_dtype) || (!db && db_acc)) return ZERO_EINVAL;
    if (const int rc = check_matrix(dz, m, n, lddz, ZERO_BF16)) return rc;
    if (const int rc = check_matrix(x, m, k, ldx, ZERO_BF16)) return rc;
    if (const int rc = check_matrix(dw, n, k, lddw, dw_dtype)) return rc;
    if (acc)
        if (const int rc = check_matrix(acc, n, k, ldacc, dw_dtype)) return rc;
    if (check_aligned(db, dtype_size(dw_dtype)) || check_aligned(db_acc, dtype_size(dw_dtype))) return ZERO_EALIGN;
    if (n == 0) return ZERO_OK;
    if ((m && check_device_ptr(dz)) || (m && k && check_device_ptr(x)) || (k && check_device_ptr(dw)) ||
        (k && acc && check_device_ptr(acc)) || (db && check_device_ptr(db)) || (db_acc && check_device_ptr(db_acc)))
        return ZERO_EINVAL;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (db) {
        const int rc = launch_column_sum(m, n, dz, lddz, db_acc, db, dw_dtype == ZERO_F32, s);
        if (rc != ZERO_OK) return rc;
    }
    if (k == 0) return ZERO_OK;
    Ending e{};
    e.add = acc; e.ld_add = ldacc;
    e.out = dw; e.ld_out = lddw; e.out_f32 = dw_dtype == ZERO_F32;
    return launch_product(Product{n, k, m, {dz, lddz, m, n, true}, {x, ldx, m, k, true}}, e, s);
}
