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

namespace zgb {

int drop_params(const zero_dropout_t* d, int64_t rows, int64_t cols, DropParams* out) {
    *out = DropParams{0u, 1.0f, 0u, 0u, 0u, 0u, nullptr};
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
    out->key0 = (uint32_t)d->seed;
    out->key1 = (uint32_t)(d->seed >> 32);
    out->site = d->site;
    out->step = (uint32_t)d->step;
    out->step_ptr = d->step_ptr;
    return ZERO_OK;
}

struct DropoutParams {
    int64_t rows, cols, col_blocks;
    const void* x; int64_t ldx;            // x or dy
    const void* side; int64_t lds;         // the residual or pre, or null
    void* y; int64_t ldy;
    int32_t act;
    bool x_f32, y_f32, x_vec, side_vec, y_vec;
    DropParams drop;
};

// One thread takes eight columns of a row at a time, over the whole matrix in
// steps of the grid.
template <bool kGrad>
__global__ void __launch_bounds__(kThreads) dropout_kernel(const DropoutParams p) {
    const int64_t total = p.rows * p.col_blocks;
    const int64_t stride = (int64_t)gridDim.x * kThreads;
    const uint32_t step = p.drop.cut ? drop_step(p.drop) : 0u;
    const int xs = p.x_f32 ? 4 : 2, ys = p.y_f32 ? 4 : 2;
    for (int64_t i = (int64_t)blockIdx.x * kThreads + threadIdx.x; i < total; i += stride) {
        const int64_t row = i / p.col_blocks, cb = i - row * p.col_blocks, col = cb * 8;
        const int count = p.cols - col < 8 ? (int)(p.cols - col) : 8;
        const bool full = count == 8;
        float v[8];
        load8(static_cast<const char*>(p.x) + (row * p.ldx + col) * xs, p.x_f32, p.x_vec && full, count, v);
        if (kGrad && p.side) {
            float z[8];
            load8(static_cast<const uint16_t*>(p.side) + row * p.lds + col, false, p.side_vec && full, count, z);
#pragma unroll
            for (int j = 0; j < 8; ++j) v[j] *= act_slope(p.act, z[j]);
        }
        if (p.drop.cut) drop8(p.drop, step, row, cb, v);
        if (!kGrad && p.side) {
            float r[8];
            load8(static_cast<const char*>(p.side) + (row * p.lds + col) * xs, p.x_f32, p.side_vec && full, count, r);
#pragma unroll
            for (int j = 0; j < 8; ++j) v[j] += r[j];
        }
        store8(static_cast<char*>(p.y) + (row * p.ldy + col) * ys, p.y_f32, p.y_vec && full, count, v);
    }
}

// db for dropout_kernel<true>: one thread a column, recomputing dx in fp32.
__global__ void __launch_bounds__(kThreads)
dropout_column_sum_kernel(const DropoutParams p, const void* db_acc, void* db, bool db_f32) {
    const int64_t cb = ((int64_t)blockIdx.x * kThreads + threadIdx.x);
    if (cb >= p.col_blocks) return;
    const int64_t col = cb * 8;
    const int count = p.cols - col < 8 ? (int)(p.cols - col) : 8;
    const uint32_t step = p.drop.cut ? drop_step(p.drop) : 0u;
    const int xs = p.x_f32 ? 4 : 2, bs = db_f32 ? 4 : 2;
    float sum[8] = {};
    for (int64_t row = 0; row < p.rows; ++row) {
        float v[8];
        load8(static_cast<const char*>(p.x) + (row * p.ldx + col) * xs, p.x_f32, false, count, v);
        if (p.side) {
            float z[8];
            load8(static_cast<const uint16_t*>(p.side) + row * p.lds + col, false, false, count, z);
#pragma unroll
            for (int j = 0; j < 8; ++j) v[j] *= act_slope(p.act, z[j]);
        }
        if (p.drop.cut) drop8(p.drop, step, row, cb, v);
#pragma unroll
        for (int j = 0; j < 8; ++j) sum[j] += v[j];
    }
    if (db_acc) {
        float a[8];
        load8(static_cast<const char*>(db_acc) + col * bs, db_f32, false, count, a);
#pragma unroll
        for (int j = 0; j < 8; ++j) sum[j] += a[j];
    }
    store8(static_cast<char*>(db) + col * bs, db_f32, false, count, sum);
}

static int launch_sums(const DropoutParams& p, const void* db_acc, void* db, bool db_f32, cudaStream_t s) {
    dropout_column_sum_kernel<<<(unsigned)((p.col_blocks + kThreads - 1) / kThreads), kThreads, 0, s>>>(p, db_acc, db,
                                                                                                        db_f32);
    return launch_status();
}

int launch_column_sum(int64_t rows, int64_t cols, const uint16_t* dz, int64_t lddz, const void* db_acc, void* db,
                      bool db_f32, cudaStream_t s) {
    DropoutParams p{};
    p.rows = rows; p.cols = cols; p.col_blocks = (cols + 7) / 8;
    p.x = dz; p.ldx = lddz;
    p.x_vec = rows_aligned16(dz, lddz, 2);
    return launch_sums(p, db_acc, db, db_f32, s);
}

static bool dtype_ok(int32_t d) { return d == ZERO_BF16 || d == ZERO_F32; }

static int launch_dropout(const DropoutParams& p, bool grad, cudaStream_t s) {
    const void* kernel = grad ? (const void*)dropout_kernel<true> : (const void*)dropout_kernel<false>;
    const int64_t resident = (int64_t)sm_count() * ctas_per_sm(kernel, kThreads, 0);
    const unsigned grid = grid_for(p.rows * p.col_blocks, kThreads, resident * 4);
    if (grad)
        dropout_kernel<true><<<grid, kThreads, 0, s>>>(p);
    else
        dropout_kernel<false><<<grid, kThreads, 0, s>>>(p);
    return launch_status();
}

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
    const int size = dtype_size(dtype);
    p.rows = rows; p.cols = cols; p.col_blocks = (cols + 7) / 8;
    p.x = x; p.ldx = ldx; p.side = residual; p.lds = ldr; p.y = y; p.ldy = ldy;
    p.x_f32 = p.y_f32 = dtype == ZERO_F32;
    p.x_vec = rows_aligned16(x, ldx, size);
    p.side_vec = residual && rows_aligned16(residual, ldr, size);
    p.y_vec = rows_aligned16(y, ldy, size);
    return launch_dropout(p, false, static_cast<cudaStream_t>(stream));
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
    p.rows = rows; p.cols = cols; p.col_blocks = (cols + 7) / 8;
    p.x = dy; p.ldx = lddy; p.side = pre; p.lds = ldp; p.y = dx; p.ldy = lddx;
    p.act = act;
    p.x_f32 = dy_dtype == ZERO_F32;
    p.y_f32 = dx_dtype == ZERO_F32;
    p.x_vec = rows_aligned16(dy, lddy, dtype_size(dy_dtype));
    p.side_vec = pre && rows_aligned16(pre, ldp, 2);
    p.y_vec = rows_aligned16(dx, lddx, dtype_size(dx_dtype));
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (db) {   // first: dx may be written over dy
        if (const int rc = launch_sums(p, db_acc, db, db_dtype == ZERO_F32, s)) return rc;
    }
    return rows ? launch_dropout(p, true, s) : ZERO_OK;
}
