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
#include <type_traits>

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
    int32_t per_head;                // work items of a head
    uint32_t by_head, by_heads;      // ceil(2^32 / per_head), ceil(2^32 / cta_heads)
    zero_rope_plan_t plan;
};

constexpr int kRopeItems = 4096;   // work items of a CTA, sixteen a thread

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

// n / d for n * d < 2^32, from m = ceil(2^32 / d); d = 1 has no such m.
__device__ __forceinline__ uint32_t divide(uint32_t n, uint32_t m) { return m ? __umulhi(n, m) : n; }

// A CTA takes cta_tokens tokens of cta_heads heads: it forms the sines of those
// tokens' pairs once in shared memory (one a thread or so), then turns the heads.
// kVec: two 16-byte vectors an item, which hold kCount whole pairs (a's and b's in
// the half layout, neighbours in the interleaved one) or up to two of the vectors
// that are copied; else a pair an item, or up to two copied elements.
// Bound by memory: 8192 tokens x 64 heads of 128 bf16 inside a packed projection in
// 45.9 us (5.9 TB/s), 6001 x 25 x 64 fp32 with half of each head turned in 15.5 us
// (5.0 TB/s).  Sixteen items a thread, two bf16 ones (four fp32) in flight: 49 us with
// four of either.
template <bool kF32, bool kHalf, bool kVec>
__global__ void __launch_bounds__(kThreads) rope_kernel(const __grid_constant__ RopeParams p) {
    __shared__ float2 turn[kThreads > ZERO_ROPE_MAX / 2 ? kThreads : ZERO_ROPE_MAX / 2];   // [cta_tokens][pairs]
    using V = RopeVector<kF32>;
    using T = typename std::conditional<kF32, float, uint16_t>::type;
    constexpr int kBatch = kF32 ? 4 : 2, kCount = kVec ? V::kCount : 1;   // items whose loads fly together
    const int pairs = p.plan.rot / 2, turned = pairs / kCount, rest = (int)((p.dim - p.plan.rot) / kCount);
    const int64_t t0 = (int64_t)blockIdx.x * p.cta_tokens, h0 = (int64_t)blockIdx.y * p.cta_heads;
    const int nt = (int)(p.tokens - t0 < p.cta_tokens ? p.tokens - t0 : p.cta_tokens);
    const int nh = (int)(p.heads - h0 < p.cta_heads ? p.heads - h0 : p.cta_heads);
    await_predecessor();
    for (int j = threadIdx.x; j < nt * pairs; j += kThreads) {
        const int t = j / pairs, i = j - t * pairs;
        const int64_t pos = p.positions ? p.positions[t0 + t] : (int64_t)((uint64_t)p.pos0 + (uint64_t)(t0 + t));
        const uint64_t turns = (uint64_t)pos * p.plan.turn[i];
        float sn, cs;
        sincospif((float)(int32_t)(turns >> 32) * 4.656612873077392578125e-10f, &sn, &cs);   // 2^-31 half turns
        turn[j] = make_float2(cs * p.plan.scale, sn * p.plan.scale * p.sin_sign);
    }
    __syncthreads();
    const int items = nt * p.cta_heads * p.per_head;   // those of heads past the last do nothing
    for (int j0 = threadIdx.x; j0 < items; j0 += kBatch * kThreads) {
        typename std::conditional<kVec, uint4, float>::type a[kBatch], b[kBatch];
        T* out[kBatch];
        const float2* cs[kBatch];
        int second[kBatch];   // elements from an item's first to its second; 0: no second; -1: no item
#pragma unroll
        for (int k = 0; k < kBatch; ++k) {
            const uint32_t j = j0 + k * kThreads, th = divide(j, p.by_head), i = j - th * p.per_head;
            const uint32_t t = divide(th, p.by_heads), h = th - t * p.cta_heads;
            second[k] = -1;
            if ((int)j < items && (int)h < nh) {
                const bool turns = (int)i < turned;
                const int left = rest - 2 * ((int)i - turned);   // copied vectors from this item on
                const int64_t in_head = turns ? (int64_t)i * kCount * (kHalf ? 1 : 2) : p.plan.rot + (int64_t)(i - turned) * 2 * kCount;
                second[k] = turns ? (kHalf ? pairs : kCount) : left > 1 ? kCount : 0;
                const T* q = static_cast<const T*>(p.x) + (t0 + t) * p.xt + (h0 + h) * p.xh + in_head;
                out[k] = static_cast<T*>(p.y) + (t0 + t) * p.yt + (h0 + h) * p.yh + in_head;
                cs[k] = turns ? turn + t * pairs + i * kCount : nullptr;
                if constexpr (kVec) {
                    a[k] = ld_live_u4(q);
                    if (second[k]) b[k] = ld_live_u4(q + second[k]);
                } else {
                    a[k] = rope_load<kF32>(q, 0);
                    if (second[k]) b[k] = rope_load<kF32>(q, second[k]);
                }
            }
        }
#pragma unroll
        for (int k = 0; k < kBatch; ++k) {
            if (second[k] < 0) continue;
            if (cs[k]) {
                if constexpr (kVec) {
                    float u[kCount], v[kCount];
                    V::open(a[k], u);
                    V::open(b[k], v);
#pragma unroll
                    for (int i = 0; i < kCount; ++i) {
                        // the pair's two elements: one of each vector, or neighbours of one
                        float& first = kHalf ? u[i] : i < kCount / 2 ? u[2 * i] : v[2 * i - kCount];
                        float& other = kHalf ? v[i] : i < kCount / 2 ? u[2 * i + 1] : v[2 * i + 1 - kCount];
                        turn_pair(cs[k][i], first, other);
                    }
                    a[k] = V::close(u);
                    b[k] = V::close(v);
                } else {
                    turn_pair(cs[k][0], a[k], b[k]);
                }
            }
            if constexpr (kVec) {
                st_stream_u4(out[k], a[k]);
                if (second[k]) st_stream_u4(out[k] + second[k], b[k]);
            } else {
                rope_store<kF32>(out[k], 0, a[k]);
                if (second[k]) rope_store<kF32>(out[k], second[k], b[k]);
            }
        }
    }
}

static uint32_t reciprocal(int32_t d) { return d == 1 ? 0u : (uint32_t)((((uint64_t)1 << 32) + d - 1) / d); }

template <bool kF32, bool kHalf>
static int launch_rope(RopeParams& p, cudaStream_t s) {
    constexpr int count = RopeVector<kF32>::kCount;
    const int pairs = p.plan.rot / 2;
    const bool vec = pairs % count == 0 && p.dim % count == 0 && aligned16(p.x) && aligned16(p.y) && p.xt % count == 0 &&
                     p.xh % count == 0 && p.yt % count == 0 && p.yh % count == 0;
    const int64_t unit = vec ? count : 1, rest = p.copy_rest ? (p.dim - p.plan.rot) / unit : 0;
    const int64_t per_head = pairs / unit + (rest + 1) / 2;
    if (per_head > kRopeItems * 8) return ZERO_ERANGE;   // a head of more than 2^15 elements
    p.per_head = (int32_t)per_head;
    const int64_t tokens = kThreads / pairs > 1 ? kThreads / pairs : 1;   // a sine a thread
    int64_t share = kRopeItems / per_head;                                // heads of a CTA, over its tokens
    share = share < 1 ? 1 : share;
    p.cta_tokens = (int32_t)(tokens < share ? tokens : share);
    if (p.cta_tokens > p.tokens) p.cta_tokens = (int32_t)p.tokens;
    const int64_t heads = share / p.cta_tokens;
    p.cta_heads = (int32_t)(heads < p.heads ? heads : p.heads);
    p.by_head = reciprocal(p.per_head);
    p.by_heads = reciprocal(p.cta_heads);
    const int64_t gx = (p.tokens + p.cta_tokens - 1) / p.cta_tokens, gy = (p.heads + p.cta_heads - 1) / p.cta_heads;
    if (gx > INT32_MAX || gy > 65535) return ZERO_ERANGE;
    return launch_dense(vec ? rope_kernel<kF32, kHalf, true> : rope_kernel<kF32, kHalf, false>, dim3((unsigned)gx, (unsigned)gy),
                        kThreads, 1, true, 0, s, p);
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
