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
    bool copy_rest;
    float sin_sign;
    int32_t cta_tokens, cta_heads;   // what one CTA takes
    zero_rope_plan_t plan;
};

constexpr int kRopeItems = 2048;   // work items of a CTA, eight a thread

template <bool kF32>
__device__ __forceinline__ float rope_load(const void* p, int64_t i) {
    return kF32 ? static_cast<const float*>(p)[i] : bf16_one(static_cast<const uint16_t*>(p)[i]);
}
template <bool kF32>
__device__ __forceinline__ void rope_store(void* p, int64_t i, float v) {
    if (kF32)
        static_cast<float*>(p)[i] = v;
    else
        static_cast<uint16_t*>(p)[i] = to_bf16(v);
}

template <bool kF32>
struct RopeVector {   // 16 bytes of a head
    static constexpr int kCount = kF32 ? 4 : 8;
    static __device__ __forceinline__ void open(uint4 u, float* v) {
        if constexpr (kF32) {
            v[0] = __uint_as_float(u.x); v[1] = __uint_as_float(u.y); v[2] = __uint_as_float(u.z); v[3] = __uint_as_float(u.w);
        } else {
            unpack8(u, v);
        }
    }
    static __device__ __forceinline__ uint4 close(const float* v) {
        if constexpr (kF32)
            return make_uint4(__float_as_uint(v[0]), __float_as_uint(v[1]), __float_as_uint(v[2]), __float_as_uint(v[3]));
        else
            return pack8(v);
    }
};

// One rounding order for every path, so that a result does not depend on alignment.
__device__ __forceinline__ void turn_pair(float2 c, float& first, float& second) {
    const float f = first, o = second;
    first = __fmaf_rn(f, c.x, -__fmul_rn(o, c.y));
    second = __fmaf_rn(o, c.x, __fmul_rn(f, c.y));
}

// A CTA takes cta_tokens tokens of cta_heads heads: it forms the sines of those
// tokens' pairs once in shared memory (one a thread or so), then turns the heads.
// kVec: two 16-byte vectors an item, which hold kCount whole pairs (a's and b's in
// the half layout, neighbours in the interleaved one); else a pair an item.
template <bool kF32, bool kHalf, bool kVec>
__global__ void __launch_bounds__(kThreads) rope_kernel(const __grid_constant__ RopeParams p) {
    __shared__ float2 turn[kThreads > ZERO_ROPE_MAX / 2 ? kThreads : ZERO_ROPE_MAX / 2];   // [cta_tokens][pairs]
    const int pairs = p.plan.rot / 2;
    const int64_t t0 = (int64_t)blockIdx.x * p.cta_tokens, h0 = (int64_t)blockIdx.y * p.cta_heads;
    const int nt = (int)(p.tokens - t0 < p.cta_tokens ? p.tokens - t0 : p.cta_tokens);
    const int nh = (int)(p.heads - h0 < p.cta_heads ? p.heads - h0 : p.cta_heads);
    for (int j = threadIdx.x; j < nt * pairs; j += kThreads) {
        const int t = j / pairs, i = j - t * pairs;
        const int64_t pos = p.positions ? p.positions[t0 + t] : (int64_t)((uint64_t)p.pos0 + (uint64_t)(t0 + t));
        const uint64_t turns = (uint64_t)pos * p.plan.turn[i];
        float sn, cs;
        sincospif((float)(int32_t)(turns >> 32) * 4.656612873077392578125e-10f, &sn, &cs);   // 2^-31 half turns
        turn[j] = make_float2(cs * p.plan.scale, sn * p.plan.scale * p.sin_sign);
    }
    __syncthreads();
    if constexpr (kVec) {
        using V = RopeVector<kF32>;
        constexpr int kBatch = 4, size = kF32 ? 4 : 2;
        const int per_head = pairs / V::kCount, items = nt * nh * per_head;
        for (int j0 = threadIdx.x; j0 < items; j0 += kBatch * kThreads) {
            uint4 a[kBatch], b[kBatch];
            char* out[kBatch];
            const float2* cs[kBatch];
            const int second = (kHalf ? pairs : V::kCount) * size;
#pragma unroll
            for (int k = 0; k < kBatch; ++k) {
                const int j = j0 + k * kThreads;
                if (j < items) {
                    const int th = j / per_head, i = j - th * per_head, t = th / nh, h = th - t * nh;
                    const int64_t in_head = (int64_t)i * V::kCount * (kHalf ? 1 : 2);
                    const char* q = static_cast<const char*>(p.x) + ((t0 + t) * p.xt + (h0 + h) * p.xh + in_head) * size;
                    a[k] = ld_stream_u4(q);
                    b[k] = ld_stream_u4(q + second);
                    out[k] = static_cast<char*>(p.y) + ((t0 + t) * p.yt + (h0 + h) * p.yh + in_head) * size;
                    cs[k] = turn + t * pairs + i * V::kCount;
                }
            }
#pragma unroll
            for (int k = 0; k < kBatch; ++k) {
                if (j0 + k * kThreads < items) {
                    float u[V::kCount], v[V::kCount];
                    V::open(a[k], u);
                    V::open(b[k], v);
#pragma unroll
                    for (int i = 0; i < V::kCount; ++i) {
                        const float2 c = cs[k][i];
                        // the pair's two elements: one of each vector, or neighbours of one
                        float& first = kHalf ? u[i] : i < V::kCount / 2 ? u[2 * i] : v[2 * i - V::kCount];
                        float& other = kHalf ? v[i] : i < V::kCount / 2 ? u[2 * i + 1] : v[2 * i + 1 - V::kCount];
                        turn_pair(c, first, other);
                    }
                    st_stream_u4(out[k], V::close(u));
                    st_stream_u4(out[k] + second, V::close(v));
                }
            }
        }
        if (p.copy_rest) {
            const int rest = (int)((p.dim - p.plan.rot) / V::kCount);
            for (int64_t j = threadIdx.x; j < (int64_t)nt * nh * rest; j += kThreads) {
                const int64_t th = j / rest, t = th / nh, h = th - t * nh, in_head = p.plan.rot + (j - th * rest) * V::kCount;
                st_stream_u4(static_cast<char*>(p.y) + ((t0 + t) * p.yt + (h0 + h) * p.yh + in_head) * size,
                             ld_stream_u4(static_cast<const char*>(p.x) + ((t0 + t) * p.xt + (h0 + h) * p.xh + in_head) * size));
            }
        }
    } else {
        for (int j = threadIdx.x; j < nt * nh * pairs; j += kThreads) {
            const int th = j / pairs, i = j - th * pairs, t = th / nh, h = th - t * nh;
            const int64_t ia = kHalf ? i : 2 * i, ib = kHalf ? i + pairs : 2 * i + 1;
            const int64_t xb = (t0 + t) * p.xt + (h0 + h) * p.xh, yb = (t0 + t) * p.yt + (h0 + h) * p.yh;
            float a = rope_load<kF32>(p.x, xb + ia), b = rope_load<kF32>(p.x, xb + ib);
            turn_pair(turn[t * pairs + i], a, b);
            rope_store<kF32>(p.y, yb + ia, a);
            rope_store<kF32>(p.y, yb + ib, b);
        }
        if (p.copy_rest) {
            const int64_t rest = p.dim - p.plan.rot;
            for (int64_t j = threadIdx.x; j < nt * nh * rest; j += kThreads) {
                const int64_t th = j / rest, i = j - th * rest + p.plan.rot, t = th / nh, h = th - t * nh;
                rope_store<kF32>(p.y, (t0 + t) * p.yt + (h0 + h) * p.yh + i, rope_load<kF32>(p.x, (t0 + t) * p.xt + (h0 + h) * p.xh + i));
            }
        }
    }
}

template <bool kF32, bool kHalf>
static int launch_rope(RopeParams& p, cudaStream_t s) {
    constexpr int count = RopeVector<kF32>::kCount;
    const int pairs = p.plan.rot / 2;
    const bool vec = pairs % count == 0 && p.dim % count == 0 && aligned16(p.x) && aligned16(p.y) && p.xt % count == 0 &&
                     p.xh % count == 0 && p.yt % count == 0 && p.yh % count == 0;
    const int per_head = vec ? pairs / count : pairs;
    const int64_t tokens = kThreads / pairs > 1 ? kThreads / pairs : 1;
    p.cta_tokens = (int32_t)(tokens < p.tokens ? tokens : p.tokens);
    const int64_t heads = kRopeItems / (p.cta_tokens * per_head);
    p.cta_heads = (int32_t)(heads < 1 ? 1 : heads < p.heads ? heads : p.heads);
    const int64_t gx = (p.tokens + p.cta_tokens - 1) / p.cta_tokens, gy = (p.heads + p.cta_heads - 1) / p.cta_heads;
    if (gx > INT32_MAX || gy > 65535) return ZERO_ERANGE;
    const dim3 grid((unsigned)gx, (unsigned)gy);
    if (vec)
        rope_kernel<kF32, kHalf, true><<<grid, kThreads, 0, s>>>(p);
    else
        rope_kernel<kF32, kHalf, false><<<grid, kThreads, 0, s>>>(p);
    return launch_status();
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
    p.copy_rest = dim > plan->rot && x != y;
    p.sin_sign = inverse ? -1.0f : 1.0f;
    p.plan = *plan;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    const bool half = plan->layout == ZERO_ROPE_HALF;
    if (dtype == ZERO_F32) return half ? launch_rope<true, true>(p, s) : launch_rope<true, false>(p, s);
    return half ? launch_rope<false, true>(p, s) : launch_rope<false, false>(p, s);
}
