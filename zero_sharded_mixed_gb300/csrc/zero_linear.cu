// Products of a unit with their elementwise ends, and their gradients, sm_103a:
//   zero_linear              y  = residual + D(act(x w^T + bias))
//   zero_linear_grad_input   dx = residual + D'(dz w) act'(pre)
//   zero_linear_grad_weight  dw = acc + dz^T x,  db = db_acc + sum over rows of dz
#include "zero_dense.cuh"

namespace zgb {

// C[rows, cols] = sum over `depth` of A B with a strided element A(i, t) at
// a[i * a_row + t * a_depth], B(j, t) at b[j * b_row + t * b_depth], and the end.
struct Product {
    int64_t rows, cols, depth;
    const uint16_t* a; int64_t a_row, a_depth;
    const uint16_t* b; int64_t b_row, b_depth;
};
struct Ending {
    const uint16_t* bias;                       // per column, or null
    const uint16_t* slope; int64_t ld_slope;    // pre of the layer below: times act'(slope), or null
    uint16_t* pre; int64_t ld_pre;              // receives the product with its bias, or null
    const void* add; int64_t ld_add;            // residual or acc, of the output's type, or null
    void* out; int64_t ld_out;
    int32_t act;
    bool out_f32;
    DropParams drop;
};

constexpr int kTile = 64, kDepth = 16;

__device__ __forceinline__ void end8(const Ending& e, uint32_t step, int64_t row, int64_t col, int count, float* v) {
    const bool f32 = e.out_f32;
    const int size = f32 ? 4 : 2;
    float t[8];
    if (e.bias) {
        load8(e.bias + col, false, false, count, t);
        for (int j = 0; j < 8; ++j) v[j] += t[j];
    }
    if (e.pre) store8(e.pre + row * e.ld_pre + col, false, false, count, v);
    if (e.slope) {
        load8(e.slope + row * e.ld_slope + col, false, false, count, t);
        for (int j = 0; j < 8; ++j) v[j] *= act_slope(e.act, t[j]);
    } else if (e.act) {
        for (int j = 0; j < 8; ++j) v[j] = act_apply(e.act, v[j]);
    }
    if (e.drop.cut) drop8(e.drop, step, row, col >> 3, v);
    if (e.add) {
        load8(static_cast<const char*>(e.add) + (row * e.ld_add + col) * size, f32, false, count, t);
        for (int j = 0; j < 8; ++j) v[j] += t[j];
    }
    store8(static_cast<char*>(e.out) + (row * e.ld_out + col) * size, f32, false, count, v);
}

// The plain kernel: a 64 x 64 tile a CTA, 2 x 8 results a thread, fp32 products.
__global__ void __launch_bounds__(kThreads) product_kernel(const Product p, const Ending e) {
    __shared__ float as[kDepth][kTile + 1], bs[kDepth][kTile + 1];
    const int64_t row0 = (int64_t)blockIdx.y * kTile, col0 = (int64_t)blockIdx.x * kTile;
    const int tr = threadIdx.x / 8 * 2, tc = threadIdx.x % 8 * 8;
    float acc[2][8] = {};
    for (int64_t t0 = 0; t0 < p.depth; t0 += kDepth) {
        for (int i = threadIdx.x; i < kTile * kDepth; i += kThreads) {
            // neighbouring threads along whichever of the two is contiguous
            const int r = p.a_depth == 1 ? i / kDepth : i % kTile, t = p.a_depth == 1 ? i % kDepth : i / kTile;
            as[t][r] = row0 + r < p.rows && t0 + t < p.depth
                           ? bf16_one(p.a[(row0 + r) * p.a_row + (t0 + t) * p.a_depth]) : 0.0f;
            const int c = p.b_depth == 1 ? i / kDepth : i % kTile, u = p.b_depth == 1 ? i % kDepth : i / kTile;
            bs[u][c] = col0 + c < p.cols && t0 + u < p.depth
                           ? bf16_one(p.b[(col0 + c) * p.b_row + (t0 + u) * p.b_depth]) : 0.0f;
        }
        __syncthreads();
        for (int t = 0; t < kDepth; ++t)
            for (int i = 0; i < 2; ++i)
                for (int j = 0; j < 8; ++j) acc[i][j] += as[t][tr + i] * bs[t][tc + j];
        __syncthreads();
    }
    const uint32_t step = e.drop.cut ? drop_step(e.drop) : 0u;
    const int64_t col = col0 + tc;
    if (col >= p.cols) return;
    const int count = p.cols - col < 8 ? (int)(p.cols - col) : 8;
    for (int i = 0; i < 2; ++i)
        if (row0 + tr + i < p.rows) end8(e, step, row0 + tr + i, col, count, acc[i]);
}

static int launch_product(const Product& p, const Ending& e, cudaStream_t s) {
    const int64_t gx = (p.cols + kTile - 1) / kTile, gy = (p.rows + kTile - 1) / kTile;
    if (gx > INT32_MAX || gy > 65535) return ZERO_ERANGE;
    product_kernel<<<dim3((unsigned)gx, (unsigned)gy), kThreads, 0, s>>>(p, e);
    return launch_status();
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
    return launch_product(Product{m, n, k, x, ldx, 1, w, ldw, 1}, e, static_cast<cudaStream_t>(stream));
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
    return launch_product(Product{m, k, n, dz, lddz, 1, w, 1, ldw}, e, static_cast<cudaStream_t>(stream));
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
    return launch_product(Product{n, k, m, dz, 1, lddz, x, 1, ldx}, e, s);
}
