// Dropout from a counter-based generator, with a residual, and its gradient
// with the activation's slope and the bias gradient, sm_103a.
//
// Forward:  y  = residual + D(x)
// Backward: dx = D'(dy) * act'(pre),  db[c] = db_acc[c] + sum over rows of dx[r, c]
// D keeps an element where its 16 random bits are at least cut and multiplies it
// with scale, and puts 0 elsewhere; the backward pass forms the same bits again,
// so no mask is stored (zero_dense.cuh has the generator).
#include <cmath>

#include "zero_dense.cuh"
#include "zero_tensor.cuh"

namespace zgb {

int drop_params(const zero_dropout_t* d, int64_t rows, int64_t cols, DropParams* out) {
    *out = DropParams{};
    out->scale = 1.0f;
    if (!d) return ZERO_OK;
    if (!(d->p >= 0.0 && d->p <= 1.0)) return ZERO_EINVAL;
    if (d->reserved != 0) return ZERO_EINVAL;
    if (d->step > 0xffffffffull) return ZERO_ERANGE;
    if (d->step_ptr) {
        if (check_aligned(d->step_ptr, 8)) return ZERO_EALIGN;
    }
    out->cut = (uint32_t)std::nearbyint(d->p * 65536.0);
    if (out->cut == 0) return ZERO_OK;
    // the counter holds 32 bits of the row and 32 of the group of eight columns
    if (rows > (int64_t)1 << 32 || cols > (int64_t)1 << 35) return ZERO_ERANGE;
    out->scale = out->cut < 65536u ? (float)(65536.0 / (65536.0 - out->cut)) : 0.0f;
    for (uint32_t r = 0; r < 10; ++r) {   // the key grows by a constant a round
        out->key[r][0] = (uint32_t)d->seed + r * 0x9E3779B9u;
        out->key[r][1] = (uint32_t)(d->seed >> 32) + r * 0xBB67AE85u;
    }
    out->site = d->site;
    out->step = (uint32_t)d->step;
    out->step_ptr = d->step_ptr;
    return ZERO_OK;
}

struct DropoutParams {
    int64_t rows, cols, col_blocks;
    const void* x; int64_t ldx;            // x or dy
    const void* side; int64_t lds;         // the residual or pre, or null
    void* y; int64_t ldy;                  // null: only the sums are wanted
    const void* db_acc; void* db;
    int32_t act;
    bool x_f32, y_f32, side_f32, db_f32;
    DropParams drop;
};

// The last step of the sums: `total` holds this CTA's of `width` columns from col0;
// each CTA of the cluster adds a share of the columns over all of them.
__device__ __forceinline__ void join_sums(const DropoutParams& p, const float* total, int64_t col0, int width) {
    cluster_sync();
    const int n = (int)cluster_size(), c = (int)cluster_rank() * (width / n) + threadIdx.x;
    if ((int)threadIdx.x < width / n && col0 + c < p.cols) {
        float s = 0.0f;
        for (int i = 0; i < n; ++i) s += peer_load1(peer_addr(smem_addr(total + c), i));
        const int64_t at = col0 + c;
        if (p.db_f32) {
            if (p.db_acc) s += static_cast<const float*>(p.db_acc)[at];
            static_cast<float*>(p.db)[at] = s;
        } else {
            if (p.db_acc) s += bf16_one(static_cast<const uint16_t*>(p.db_acc)[at]);
            static_cast<uint16_t*>(p.db)[at] = to_bf16(s);
        }
    }
    __syncwarp();
    cluster_sync();   // the totals are read before their CTAs end
}

// Whole, aligned rows: a thread keeps its eight columns and goes down the rows,
// four of them (two of fp32) in flight, so that addresses are additions and the
// first products of its random numbers, which see the column and constants alone,
// are formed once.  A warp takes `lanes` neighbouring column groups of 32 / lanes
// rows; warps with neighbouring numbers take neighbouring columns, and one wave of
// CTAs goes through the matrix together.  Bound by memory with the random numbers
// close behind: 8192 x 1600 bf16 with a residual in 16.1 us (4.9 TB/s, caches and
// launch included), 65536 x 1600 in 105 us (6.0 TB/s; 98 us without the random
// numbers).  One vector a thread and many waves: 23 and 169 us; more rows in flight
// cost residency: 25 and 182 us.
template <bool kF32>
constexpr int kBatchOf = kF32 ? 2 : 4;

//
// Sums (kSums): the CTAs of a cluster share the column groups of one warp, and their
// warps the rows.  Each thread sums its rows in order, the CTA its threads, then the
// cluster its CTAs, every time in the same order.
constexpr int kShares = 8;

template <bool kGrad, bool kF32, bool kSums>
__global__ void __launch_bounds__(kThreads, 3) dropout_kernel(const DropoutParams p, int lanes, int col_warps, int64_t row_step) {
    await_predecessor();
    const int lane = threadIdx.x & 31, warp = threadIdx.x / 32;
    const int64_t w = (int64_t)blockIdx.x * (kThreads / 32) + warp;
    const int64_t rg = kSums ? blockIdx.x % kShares * (kThreads / 32) + warp : w / col_warps;
    const int64_t cb = (kSums ? blockIdx.x / kShares : w - rg * col_warps) * lanes + lane % lanes;
    int64_t row = rg * (32 / lanes) + lane / lanes;
    float sum[kSums ? 8 : 1] = {};
    if constexpr (kSums) {
        if (cb >= p.col_blocks) row = p.rows;
    } else {
        if (cb >= p.col_blocks || rg * (32 / lanes) >= row_step) return;   // the last CTA may hold a warp too many
    }
    const uint32_t step = p.drop.cut ? drop_step(p.drop) : 0u;
    constexpr int kBatch = kBatchOf<kF32>, xs = kF32 ? 4 : 2, ss = kGrad ? 2 : xs;
    const int ys = p.y_f32 ? 4 : 2;
    const char* x = static_cast<const char*>(p.x) + (row * p.ldx + cb * 8) * xs;
    const char* side = p.side ? static_cast<const char*>(p.side) + (row * p.lds + cb * 8) * ss : nullptr;
    char* y = static_cast<char*>(p.y) + (row * p.ldy + cb * 8) * ys;
    const int64_t dx = row_step * p.ldx * xs, ds = row_step * p.lds * ss, dy = row_step * p.ldy * ys;
    for (; row < p.rows; row += kBatch * row_step) {
        uint4 xv[kBatch][kF32 ? 2 : 1], sv[kBatch][kF32 && !kGrad ? 2 : 1];
#pragma unroll
        for (int j = 0; j < kBatch; ++j) {
            if (row + j * row_step < p.rows) {
                xv[j][0] = ld_live_u4(x);
                if constexpr (kF32) xv[j][1] = ld_live_u4(x + 16);
                if (side) {
                    sv[j][0] = ld_live_u4(side);
                    if constexpr (kF32 && !kGrad) sv[j][1] = ld_live_u4(side + 16);
                }
            }
            x += dx;
            side += side ? ds : 0;
        }
#pragma unroll
        for (int j = 0; j < kBatch; ++j, y += dy) {
            if (row + j * row_step >= p.rows) break;
            float v[8], t[8];
            raw8<kF32>(xv[j], v);
            if (side) raw8<kF32 && !kGrad>(sv[j], t);
            if (kGrad && side) slope_apply<8>(p.act, t, v);
            if (p.drop.cut) drop8(p.drop, step, row + j * row_step, cb, v);
            if (!kGrad && side) {
#pragma unroll
                for (int k = 0; k < 8; ++k) v[k] += t[k];
            }
            if (!kSums || p.y) store8(y, p.y_f32, v);
            if constexpr (kSums) {
#pragma unroll
                for (int k = 0; k < 8; ++k) sum[k] += v[k];
            }
        }
    }
    if constexpr (kSums) {
        __shared__ float part[kThreads / 32 * 8 * 32];   // [warp][row of the warp][8 lanes columns]
        __shared__ float total[8 * 32];
        const int width = 8 * lanes;
        float* q = part + (warp * (32 / lanes) + lane / lanes) * width + lane % lanes * 8;
#pragma unroll
        for (int k = 0; k < 8; ++k) q[k] = sum[k];
        __syncthreads();
        if ((int)threadIdx.x < width) {
            float s = 0.0f;
            for (int i = 0; i < kThreads / lanes; ++i) s += part[i * width + threadIdx.x];
            total[threadIdx.x] = s;
        }
        __syncthreads();
        join_sums(p, total, (int64_t)(blockIdx.x / kShares) * width, width);
    }
}

template <class T>
__device__ __forceinline__ void load_column_of(const T* q, int64_t ld, int n, float* v) {
#pragma unroll
    for (int r = 0; r < 8; ++r, q += ld) {
        if constexpr (sizeof(T) == 4)
            v[r] = r < n ? *q : 0.0f;
        else
            v[r] = r < n ? bf16_one(*q) : 0.0f;
    }
}
__device__ __forceinline__ void load_column(const void* p, bool f32, int64_t row, int64_t ld, int64_t col, int n, float* v) {
    if (f32)
        load_column_of(static_cast<const float*>(p) + row * ld + col, ld, n, v);
    else
        load_column_of(static_cast<const uint16_t*>(p) + row * ld + col, ld, n, v);
}
__device__ __forceinline__ void store_column(void* p, bool f32, int64_t row, int64_t ld, int64_t col, int n, const float* v) {
    if (f32) {
        float* q = static_cast<float*>(p) + row * ld + col;
#pragma unroll
        for (int r = 0; r < 8; ++r, q += ld)
            if (r < n) *q = v[r];
    } else {
        uint16_t* q = static_cast<uint16_t*>(p) + row * ld + col;
#pragma unroll
        for (int r = 0; r < 8; ++r, q += ld)
            if (r < n) *q = to_bf16(v[r]);
    }
}

// Rows that are not aligned: a CTA takes a strip of 64 columns over a share of the
// rows, a warp 8 rows x 32 columns at a time, a lane a column, so that a row's
// accesses fall together; each lane forms the random bits of one row and column group
// and leaves them in shared memory for the lanes of that group.  Sums as above, the
// shares of a strip being the CTAs of a cluster.
constexpr int kStrip = 64;

template <bool kGrad, bool kSums>
__global__ void __launch_bounds__(kThreads) dropout_strip_kernel(const DropoutParams p, int shares) {
    __shared__ float part[kThreads / 64][kStrip];
    __shared__ float total[kStrip];
    __shared__ uint4 bits[kThreads / 32][8][4];   // a warp's part: row, column group
    await_predecessor();
    const int share = blockIdx.x % shares;
    const int64_t col0 = (int64_t)(blockIdx.x / shares) * kStrip;
    const int64_t row_a = p.rows / shares * share + (p.rows % shares) * share / shares;
    const int64_t row_b = p.rows / shares * (share + 1) + (p.rows % shares) * (share + 1) / shares;
    const uint32_t step = p.drop.cut ? drop_step(p.drop) : 0u;
    const int lane = threadIdx.x & 31, warp = threadIdx.x / 32;
    const int64_t col = col0 + (warp & 1) * 32 + lane;
    float sum = 0.0f;
    for (int64_t row0 = row_a + (warp >> 1) * 8; row0 < row_b; row0 += kThreads / 8) {
        // rows of the part that exist, none where the column does not
        const int n = col < p.cols ? (row_b - row0 < 8 ? (int)(row_b - row0) : 8) : 0;
        float v[8], t[8];
        load_column(p.x, p.x_f32, row0, p.ldx, col, n, v);
        if (p.side) load_column(p.side, p.side_f32, row0, p.lds, col, n, t);
        if (kGrad && p.side) slope_apply<8>(p.act, t, v);
        if (p.drop.cut) {
            __syncwarp();
            bits[warp][lane & 7][lane >> 3] =
                philox_block(p.drop, step, (uint32_t)(row0 + (lane & 7)), (uint32_t)((col0 >> 3) + (warp & 1) * 4 + (lane >> 3)));
            __syncwarp();
#pragma unroll
            for (int r = 0; r < 8; ++r)
                v[r] = reinterpret_cast<const uint16_t*>(bits[warp][r])[lane] >= p.drop.cut ? v[r] * p.drop.scale : 0.0f;
        }
        if (!kGrad && p.side) {
#pragma unroll
            for (int r = 0; r < 8; ++r) v[r] += t[r];
        }
        if (p.y) store_column(p.y, p.y_f32, row0, p.ldy, col, n, v);
        if constexpr (kSums) {
#pragma unroll
            for (int r = 0; r < 8; ++r) sum += r < n ? v[r] : 0.0f;
        }
    }
    if constexpr (kSums) {
        part[warp >> 1][(warp & 1) * 32 + lane] = sum;
        __syncthreads();
        if (threadIdx.x < kStrip) {
            float s = 0.0f;
            for (int i = 0; i < kThreads / 64; ++i) s += part[i][threadIdx.x];
            total[threadIdx.x] = s;
        }
        __syncthreads();
        join_sums(p, total, col0, kStrip);
    }
}

template <bool kGrad>
static int launch_dropout(DropoutParams& p, cudaStream_t s) {
    p.col_blocks = (p.cols + 7) / 8;
    const bool vec = p.cols % 8 == 0 && rows_aligned16(p.x, p.ldx, p.x_f32 ? 4 : 2) &&
                     (!p.side || rows_aligned16(p.side, p.lds, p.side_f32 ? 4 : 2)) &&
                     (!p.y || rows_aligned16(p.y, p.ldy, p.y_f32 ? 4 : 2));
    if (!vec) {
        const int64_t strips = (p.cols + kStrip - 1) / kStrip, most = (p.rows + 31) / 32;
        if (strips > INT32_MAX / kShares) return ZERO_ERANGE;
        if constexpr (kGrad)
            if (p.db)
                return launch_dense(dropout_strip_kernel<true, true>, dim3((unsigned)(strips * kShares)), kThreads, kShares, false, 0, s, p,
                                    (int)kShares);
        // as many shares, of at least 32 rows, as are resident at once: a CTA's start
        // costs as much as 8 rows (8 times as many CTAs: 14.6 us for 12.2)
        int64_t shares = (int64_t)sm_count() * ctas_per_sm((const void*)dropout_strip_kernel<kGrad, false>, kThreads, 0) / strips;
        shares = shares < 1 ? 1 : shares > most ? most : shares;
        if (strips > INT32_MAX / shares) return ZERO_ERANGE;
        return launch_dense(dropout_strip_kernel<kGrad, false>, dim3((unsigned)(strips * shares)), kThreads, 1, true, 0, s, p,
                            (int)shares);
    }
    // lanes of a warp along a row
    int lanes = 32;
    while (lanes / 2 >= p.col_blocks) lanes /= 2;
    if constexpr (kGrad)
        if (p.db) {
            // narrower warps, and so more clusters, as long as three CTAs an SM hold them all
            // and a thread has more than two rows (8192 x 1600: 8 lanes 14.4 us, 4 lanes 11.5;
            // past one wave, 2048 x 4096 with a slope: 16 lanes 16.1, 8 lanes 19.4).  Clusters
            // of 8 may fill an SM group less evenly than that counts.
            void (*kernel)(DropoutParams, int, int, int64_t) = p.x_f32 ? dropout_kernel<true, true, true> : dropout_kernel<true, false, true>;
            const int64_t resident = (int64_t)sm_count() * 3;
            const auto rows_of = [](int lanes) { return (int64_t)kShares * (kThreads / 32) * (32 / lanes); };   // of a cluster's pass
            while (lanes > 4 && (p.col_blocks + lanes / 2 - 1) / (lanes / 2) * kShares <= resident && p.rows > 2 * rows_of(lanes)) lanes /= 2;
            if (lanes < 4) lanes = 4;
            const int64_t col_warps = (p.col_blocks + lanes - 1) / lanes;
            if (col_warps > INT32_MAX / kShares) return ZERO_ERANGE;
            return launch_dense(kernel, dim3((unsigned)(col_warps * kShares)), kThreads, kShares, false, 0, s, p, lanes, (int)col_warps,
                                rows_of(lanes));
        }
    // as many groups of rows as give every thread a batch, up to the warps that are
    // resident at once
    void (*kernel)(DropoutParams, int, int, int64_t) = p.x_f32 ? dropout_kernel<kGrad, true, false> : dropout_kernel<kGrad, false, false>;
    const int kBatch = p.x_f32 ? kBatchOf<true> : kBatchOf<false>;
    const int64_t col_warps = (p.col_blocks + lanes - 1) / lanes, rows_of_warp = 32 / lanes;
    if (col_warps > INT32_MAX) return ZERO_ERANGE;
    const int64_t groups = (p.rows + rows_of_warp * kBatch - 1) / (rows_of_warp * kBatch);
    int64_t row_groups = (int64_t)sm_count() * ctas_per_sm((const void*)kernel, kThreads, 0) * (kThreads / 32) / col_warps;
    row_groups = row_groups < 1 ? 1 : row_groups > groups ? groups : row_groups;
    const int64_t grid = (row_groups * col_warps + kThreads / 32 - 1) / (kThreads / 32);
    if (grid > INT32_MAX) return ZERO_ERANGE;
    return launch_dense(kernel, dim3((unsigned)grid), kThreads, 1, true, 0, s, p, lanes, (int)col_warps, row_groups * rows_of_warp);
}

int launch_column_sum(int64_t rows, int64_t cols, const uint16_t* dz, int64_t lddz, const void* db_acc, void* db,
                      bool db_f32, cudaStream_t s) {
    DropoutParams p{};
    p.rows = rows; p.cols = cols;
    p.x = dz; p.ldx = lddz;
    p.db_acc = db_acc; p.db = db; p.db_f32 = db_f32;
    return launch_dropout<true>(p, s);
}

static bool dtype_ok(int32_t d) { return d == ZERO_BF16 || d == ZERO_F32; }

}  // namespace zgb

extern "C" int zero_dropout(int64_t rows, int64_t cols, const void* x, int64_t ldx, int32_t dtype,
                            const zero_dropout_t* drop, const void* residual, int64_t ldr, void* y,
                            int64_t ldy, void* stream) {
    using namespace zgb;
    if (rows < 0 || cols < 0 || !dtype_ok(dtype)) return ZERO_EINVAL;
    DropoutParams p{};
    if (const int rc = drop_params(drop, rows, cols, &p.drop)) return rc;
    if (const int rc = check_matrix(x, rows, cols, ldx, dtype)) return rc;
    if (const int rc = check_matrix(y, rows, cols, ldy, dtype)) return rc;
    if (residual)
        if (const int rc = check_matrix(residual, rows, cols, ldr, dtype)) return rc;
    if (rows == 0 || cols == 0) return ZERO_OK;
    if (check_device_ptr(x) || check_device_ptr(y) || (residual && check_device_ptr(residual)) ||
        (p.drop.step_ptr && check_device_ptr(p.drop.step_ptr)))
        return ZERO_EINVAL;
      p.rows = rows; p.cols = cols;
    p.x = x; p.ldx = ldx; p.side = residual; p.lds = ldr; p.y = y; p.ldy = ldy;
    p.x_f32 = p.y_f32 = p.side_f32 = dtype == ZERO_F32;
    return launch_dropout<false>(p, static_cast<cudaStream_t>(stream));
}

extern "C" int zero_dropout_grad(int64_t rows, int64_t cols, const void* dy, int64_t lddy, int32_t dy_dtype,
                                 const zero_dropout_t* drop, int32_t act, const uint16_t* pre, int64_t ldp,
                                 void* dx, int32_t dx_dtype, int64_t lddx, const void* db_acc, void* db,
                                 int32_t db_dtype, void* stream) {
    using namespace zgb;
    if (rows < 0 || cols < 0 || !dtype_ok(dy_dtype) || !dtype_ok(dx_dtype)) return ZERO_EINVAL;
    if (act < ZERO_ACT_NONE || act > ZERO_ACT_SILU || ((act != ZERO_ACT_NONE) != (pre != nullptr) && rows && cols)) return ZERO_EINVAL;
    if (db ? !dtype_ok(db_dtype) : db_acc != nullptr) return ZERO_EINVAL;
    DropoutParams p{};
    if (const int rc = drop_params(drop, rows, cols, &p.drop)) return rc;
    if (const int rc = check_matrix(dy, rows, cols, lddy, dy_dtype)) return rc;
    if (const int rc = check_matrix(dx, rows, cols, lddx, dx_dtype)) return rc;
    if (pre)
        if (const int rc = check_matrix(pre, rows, cols, ldp, ZERO_BF16)) return rc;
    if (db && (check_aligned(db, dtype_size(db_dtype)) || check_aligned(db_acc, dtype_size(db_dtype))))
        return ZERO_EALIGN;
    if (cols == 0 || (rows == 0 && !db)) return ZERO_OK;
    if ((rows && (check_device_ptr(dy) || check_device_ptr(dx))) || (pre && check_device_ptr(pre)) ||
        (db && check_device_ptr(db)) || (db_acc && check_device_ptr(db_acc)) ||
        (p.drop.step_ptr && check_device_ptr(p.drop.step_ptr)))
        return ZERO_EINVAL;
    p.rows = rows; p.cols = cols;
    p.x = dy; p.ldx = lddy; p.side = pre; p.lds = ldp; p.y = dx; p.ldy = lddx;
    p.act = act;
    p.x_f32 = dy_dtype == ZERO_F32;
    p.y_f32 = dx_dtype == ZERO_F32;
    p.db_acc = db_acc; p.db = db; p.db_f32 = db_dtype == ZERO_F32;
    return launch_dropout<true>(p, static_cast<cudaStream_t>(stream));
}
