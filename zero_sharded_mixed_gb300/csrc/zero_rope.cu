// Rotary positions: the first `rot` elements of every head, taken in rot / 2
// pairs, turned by position * frequency, and its gradient (the same turn back),
// sm_103a.
//
//   a' = s (a cos t - b sin t),  b' = s (b cos t + a sin t),  t = position * theta_i
// with (a, b) = (x[i], x[i + rot/2]) in the half layout and (x[2i], x[2i + 1]) in
// the interleaved one; elements past rot are copied.
//
// The angle is formed in 2^-64ths of a turn: the plan holds
// round(theta_i / 2 pi * 2^64), and its 64-bit product with the position wraps
// where the turn does, so the reduction to one turn is exact at any position and
// an angle is off by at most position * 2^-65 turns (and theta's own 53 bits)
// plus the fp32 rounding of the reduced angle.  No table of sines is read.
#include <cmath>

#include "zero_dense.cuh"

namespace zgb {

struct RopeParams {
    int64_t tokens, heads, dim;
    const void* x; int64_t xt, xh;
    void* y; int64_t yt, yh;
    const int64_t* positions;
    int64_t pos0;
    bool f32, half, copy_rest;
    float sin_sign;
    zero_rope_plan_t plan;
};

__device__ __forceinline__ float rope_load(const void* p, int64_t i, bool f32) {
    return f32 ? static_cast<const float*>(p)[i] : bf16_one(static_cast<const uint16_t*>(p)[i]);
}
__device__ __forceinline__ void rope_store(void* p, int64_t i, bool f32, float v) {
    if (f32)
        static_cast<float*>(p)[i] = v;
    else
        static_cast<uint16_t*>(p)[i] = to_bf16(v);
}

// One CTA a token: the sines of its pairs once in shared memory, then every head.
__global__ void __launch_bounds__(kThreads) rope_kernel(const __grid_constant__ RopeParams p) {
    __shared__ float2 turn[ZERO_ROPE_MAX / 2];
    const int pairs = p.plan.rot / 2;
    for (int64_t t = blockIdx.x; t < p.tokens; t += gridDim.x) {
        const int64_t pos = p.positions ? p.positions[t] : p.pos0 + t;
        for (int i = threadIdx.x; i < pairs; i += kThreads) {
            const int64_t turns = (int64_t)((uint64_t)pos * p.plan.turn[i]);
            float sn, cs;
            sincospif((float)(int32_t)(turns >> 32) * 4.656612873077392578125e-10f, &sn, &cs);
            turn[i] = make_float2(cs * p.plan.scale, sn * p.plan.scale * p.sin_sign);
        }
        __syncthreads();
        for (int64_t j = threadIdx.x; j < p.heads * pairs; j += kThreads) {
            const int64_t h = j / pairs;
            const int i = (int)(j - h * pairs);
            const int64_t ia = p.half ? i : 2 * i, ib = p.half ? i + pairs : 2 * i + 1;
            const int64_t xb = t * p.xt + h * p.xh, yb = t * p.yt + h * p.yh;
            const float a = rope_load(p.x, xb + ia, p.f32), b = rope_load(p.x, xb + ib, p.f32);
            const float2 cs = turn[i];
            rope_store(p.y, yb + ia, p.f32, a * cs.x - b * cs.y);
            rope_store(p.y, yb + ib, p.f32, b * cs.x + a * cs.y);
        }
        if (p.copy_rest) {
            const int rest = (int)(p.dim - p.plan.rot);
            for (int64_t j = threadIdx.x; j < p.heads * rest; j += kThreads) {
                const int64_t h = j / rest, i = j - h * rest + p.plan.rot;
                rope_store(p.y, t * p.yt + h * p.yh + i, p.f32, rope_load(p.x, t * p.xt + h * p.xh + i, p.f32));
            }
        }
        __syncthreads();
    }
}

}  // namespace zgb

extern "C" int zero_rope_fill(int32_t rot, int32_t layout, double base, int32_t scaling, double factor,
                              double context, zero_rope_plan_t* plan) {
    if (!plan || rot < 2 || rot % 2 || rot > ZERO_ROPE_MAX) return ZERO_EINVAL;
    if (layout != ZERO_ROPE_HALF && layout != ZERO_ROPE_INTERLEAVED) return ZERO_EINVAL;
    if (!std::isfinite(base) || base <= 1.0) return ZERO_EINVAL;
    if (scaling < ZERO_ROPE_NONE || scaling > ZERO_ROPE_YARN) return ZERO_EINVAL;
    if (scaling != ZERO_ROPE_NONE && !(std::isfinite(factor) && factor >= 1.0)) return ZERO_EINVAL;
    if (scaling == ZERO_ROPE_YARN && !(std::isfinite(context) && context > 0.0)) return ZERO_EINVAL;
    const double two_pi = 6.283185307179586476925286766559;
    if (scaling == ZERO_ROPE_NTK && rot > 2) {
        base *= std::pow(factor, (double)rot / (rot - 2));
        if (!std::isfinite(base)) return ZERO_EINVAL;
    }
    zero_rope_plan_t out{};
    out.rot = rot;
    out.layout = layout;
    out.scale = scaling == ZERO_ROPE_YARN ? (float)(0.1 * std::log(factor) + 1.0) : 1.0f;
    for (int i = 0; i < rot / 2; ++i) {
        double theta = std::pow(base, -2.0 * i / rot);
        if (scaling == ZERO_ROPE_LINEAR) theta /= factor;
        if (scaling == ZERO_ROPE_YARN) {
            double keep = (context * theta / two_pi - 1.0) / 31.0;   // 0 below 1 turn of the context, 1 above 32
            keep = keep < 0.0 ? 0.0 : keep > 1.0 ? 1.0 : keep;
            theta *= keep + (1.0 - keep) / factor;
        }
        out.turn[i] = (uint64_t)std::nearbyint(theta / two_pi * 18446744073709551616.0);   // theta <= 1: below 2^62
    }
    *plan = out;
    return ZERO_OK;
}

extern "C" int zero_rope(const zero_rope_plan_t* plan, int64_t tokens, int64_t heads, int64_t dim, const void* x,
                         int64_t x_token, int64_t x_head, void* y, int64_t y_token, int64_t y_head,
                         int32_t dtype, const int64_t* positions, int64_t pos0, int32_t inverse, void* stream) {
    using namespace zgb;
    if (!plan || tokens < 0 || heads < 0 || (dtype != ZERO_BF16 && dtype != ZERO_F32)) return ZERO_EINVAL;
    if (inverse != 0 && inverse != 1) return ZERO_EINVAL;
    if (plan->rot < 2 || plan->rot % 2 || plan->rot > ZERO_ROPE_MAX || dim < plan->rot) return ZERO_EINVAL;
    if (plan->layout != ZERO_ROPE_HALF && plan->layout != ZERO_ROPE_INTERLEAVED) return ZERO_EINVAL;
    if (!std::isfinite(plan->scale)) return ZERO_EINVAL;
    // every byte offset fits 63 bits, and no two heads of the output share an element
    const int64_t most = INT64_MAX / 16;
    const int64_t strides[4] = {x_token, x_head, y_token, y_head};
    for (int i = 0; i < 4; ++i) {
        const int64_t count = i % 2 ? heads : tokens;
        if (strides[i] < 0) return ZERO_EINVAL;
        if (count > 1 && strides[i] > most / count) return ZERO_ERANGE;
    }
    if (dim > most || heads > most / dim) return ZERO_ERANGE;
    if (heads > 1 && y_head < dim) return ZERO_EINVAL;
    // tokens apart by whole heads, or (heads outermost) heads apart by whole tokens
    if (tokens > 1 && y_token < dim) return ZERO_EINVAL;
    if (tokens > 1 && heads > 1 && y_token < (heads - 1) * y_head + dim && y_head < (tokens - 1) * y_token + dim)
        return ZERO_EINVAL;
    const int size = dtype_size(dtype);
    if (tokens == 0 || heads == 0) return ZERO_OK;
    if (!x || !y) return ZERO_EINVAL;
    if (x == y && ((tokens > 1 && x_token != y_token) || (heads > 1 && x_head != y_head))) return ZERO_EINVAL;
    if (check_aligned(x, size) || check_aligned(y, size) || check_aligned(positions, 8)) return ZERO_EALIGN;
    if (check_device_ptr(x) || check_device_ptr(y) || (positions && check_device_ptr(positions))) return ZERO_EINVAL;
    RopeParams p{};
    p.tokens = tokens; p.heads = heads; p.dim = dim;
    p.x = x; p.xt = x_token; p.xh = x_head;
    p.y = y; p.yt = y_token; p.yh = y_head;
    p.positions = positions; p.pos0 = pos0;
    p.f32 = dtype == ZERO_F32;
    p.half = plan->layout == ZERO_ROPE_HALF;
    p.copy_rest = dim > plan->rot && x != y;
    p.sin_sign = inverse ? -1.0f : 1.0f;
    p.plan = *plan;
    const int64_t cap = (int64_t)sm_count() * ctas_per_sm((const void*)rope_kernel, kThreads, 0) * 8;
    rope_kernel<<<(unsigned)(tokens < cap ? tokens : cap), kThreads, 0, static_cast<cudaStream_t>(stream)>>>(p);
    return launch_status();
}
