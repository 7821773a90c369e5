// The two ends of a step by orthogonalised momentum under ZeRO, sm_103a: the mean
// reduce-scatter into the owners' momentum with the bf16 matrices that are gathered
// and orthogonalised, and the update of the owners' master weights from the result
// with the bf16 cast and the gather write.
//
//   g = (sum over ranks) / divisor;  m = mu m + g;  u = g + mu m, or m
//   w = w - (lr wd) w;  w = w - (lr scale) o;  out = bf16(w)
//
// every operation one IEEE fp32 rounding, as in the fused AdamW update, so that a step
// does not depend on where a range begins.  Streams, bound by memory: 10 + 2 n_src and
// 12 bytes an element; 30.7 million of them take 117 us from eight ranks (6.8 TB/s) and
// 56 us (6.5 TB/s), a million 3.2 and 4.4 us, a launch and one latency.  A range may begin anywhere in the flat buffers: where all of its
// streams reach a 16-byte boundary after the same number of elements, those go one by
// one and the rest as vectors of eight.
#include <cmath>

#include "zero_update.cuh"

namespace zgb {

struct MuonScalars {
    float divisor, inv_divisor;   // inv_divisor: 1 / divisor where that is exact, else 0
    float mu, lr, wd, scale;
    const float* sched;           // device: lr, or null
    bool nesterov;
};

struct MomentumParams {
    const void* src[ZERO_MAX_SRC];   // offset to the range, like all below
    float* m;
    uint16_t* u;
    int64_t n, head, vecs;           // elements before the vectors, and the vectors
    int32_t n_src;
    MuonScalars h;
};
struct MuonUpdateParams {
    const uint16_t* o;
    float* w;
    uint16_t* out;
    int64_t n, head, vecs;
    MuonScalars h;
};

__device__ __forceinline__ float momentum_one(const MuonScalars& h, float sum, float& m) {
    const float g = h.inv_divisor != 0.0f ? __fmul_rn(sum, h.inv_divisor) : __fdiv_rn(sum, h.divisor);
    m = __fadd_rn(__fmul_rn(h.mu, m), g);
    return h.nesterov ? __fadd_rn(g, __fmul_rn(h.mu, m)) : m;
}
__device__ __forceinline__ float update_one(float decay, float step, float o, float w) {
    return __fsub_rn(__fsub_rn(w, __fmul_rn(decay, w)), __fmul_rn(step, o));
}

// The elements of a range outside its vectors, one a thread of the grid.
template <class F>
__device__ __forceinline__ void for_ends(int64_t n, int64_t head, int64_t vecs, F f) {
    const int64_t stride = (int64_t)gridDim.x * blockDim.x, ends = n - vecs * 8;
    for (int64_t i = (int64_t)blockIdx.x * blockDim.x + threadIdx.x; i < ends; i += stride) f(i < head ? i : i + vecs * 8);
}

// kSrc: sources, all of whose loads are in flight together; 0: any number, four at a time.
template <bool kBf16, int kSrc>
__global__ void __launch_bounds__(kThreads) momentum_kernel(const __grid_constant__ MomentumParams p) {
    constexpr int kFly = kSrc ? kSrc : 4;
    const int64_t stride = (int64_t)gridDim.x * kThreads;
    for (int64_t i = (int64_t)blockIdx.x * kThreads + threadIdx.x; i < p.vecs; i += stride) {
        const int64_t e = p.head + i * 8;
        float s[8] = {};
        float4 m[2];
        for (int r0 = 0; r0 < (kSrc ? 1 : p.n_src); r0 += kFly) {
            uint4 raw[kFly][kBf16 ? 1 : 2];
#pragma unroll
            for (int r = 0; r < kFly; ++r) {
                if (!kSrc && r0 + r >= p.n_src) break;
                const char* q = static_cast<const char*>(p.src[r0 + r]) + e * (kBf16 ? 2 : 4);
                raw[r][0] = ld_stream_u4(q);
                if constexpr (!kBf16) raw[r][1] = ld_stream_u4(q + 16);
            }
            if (r0 == 0) m[0] = ld_stream_f4(p.m + e), m[1] = ld_stream_f4(p.m + e + 4);
#pragma unroll
            for (int r = 0; r < kFly; ++r) {
                if (!kSrc && r0 + r >= p.n_src) break;
                float t[8];
                if constexpr (kBf16) {
                    t[0] = bf16_lo(raw[r][0].x); t[1] = bf16_hi(raw[r][0].x); t[2] = bf16_lo(raw[r][0].y); t[3] = bf16_hi(raw[r][0].y);
                    t[4] = bf16_lo(raw[r][0].z); t[5] = bf16_hi(raw[r][0].z); t[6] = bf16_lo(raw[r][0].w); t[7] = bf16_hi(raw[r][0].w);
                } else {
#pragma unroll
                    for (int k = 0; k < 2; ++k) {
                        t[4 * k] = __uint_as_float(raw[r][k].x); t[4 * k + 1] = __uint_as_float(raw[r][k].y);
                        t[4 * k + 2] = __uint_as_float(raw[r][k].z); t[4 * k + 3] = __uint_as_float(raw[r][k].w);
                    }
                }
#pragma unroll
                for (int k = 0; k < 8; ++k) s[k] = __fadd_rn(s[k], t[k]);
            }
        }
        float v[8] = {m[0].x, m[0].y, m[0].z, m[0].w, m[1].x, m[1].y, m[1].z, m[1].w}, u[8];
#pragma unroll
        for (int k = 0; k < 8; ++k) u[k] = momentum_one(p.h, s[k], v[k]);
        st_stream_f4(p.m + e, make_float4(v[0], v[1], v[2], v[3]));
        st_stream_f4(p.m + e + 4, make_float4(v[4], v[5], v[6], v[7]));
        *reinterpret_cast<uint4*>(p.u + e) =   // read next: stays in L2
            make_uint4(pack_bf16x2(u[0], u[1]), pack_bf16x2(u[2], u[3]), pack_bf16x2(u[4], u[5]), pack_bf16x2(u[6], u[7]));
    }
    for_ends(p.n, p.head, p.vecs, [&](int64_t e) {
        float s = 0.0f;
        for (int r = 0; r < p.n_src; ++r)
            s = __fadd_rn(s, kBf16 ? bf16_one(static_cast<const uint16_t*>(p.src[r])[e]) : static_cast<const float*>(p.src[r])[e]);
        float m = p.m[e];
        p.u[e] = to_bf16(momentum_one(p.h, s, m));
        p.m[e] = m;
    });
}

__global__ void __launch_bounds__(kThreads) muon_update_kernel(const __grid_constant__ MuonUpdateParams p) {
    const float lr = p.h.sched ? *p.h.sched : p.h.lr;
    const float decay = __fmul_rn(lr, p.h.wd), step = __fmul_rn(lr, p.h.scale);
    const int64_t stride = (int64_t)gridDim.x * kThreads;
    for (int64_t i = (int64_t)blockIdx.x * kThreads + threadIdx.x; i < p.vecs; i += stride) {
        const int64_t e = p.head + i * 8;
        const uint4 o = ld_stream_u4(p.o + e);
        const float4 a = ld_stream_f4(p.w + e), b = ld_stream_f4(p.w + e + 4);
        float w[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
        const float t[8] = {bf16_lo(o.x), bf16_hi(o.x), bf16_lo(o.y), bf16_hi(o.y), bf16_lo(o.z), bf16_hi(o.z), bf16_lo(o.w), bf16_hi(o.w)};
#pragma unroll
        for (int k = 0; k < 8; ++k) w[k] = update_one(decay, step, t[k], w[k]);
        st_stream_f4(p.w + e, make_float4(w[0], w[1], w[2], w[3]));
        st_stream_f4(p.w + e + 4, make_float4(w[4], w[5], w[6], w[7]));
        st_stream_u4(p.out + e, make_uint4(pack_bf16x2(w[0], w[1]), pack_bf16x2(w[2], w[3]), pack_bf16x2(w[4], w[5]), pack_bf16x2(w[6], w[7])));
    }
    for_ends(p.n, p.head, p.vecs, [&](int64_t e) {
        const float w = update_one(decay, step, bf16_one(p.o[e]), p.w[e]);
        p.w[e] = w;
        p.out[e] = to_bf16(w);
    });
}

// Elements until a stream of `size` bytes an element reaches a 16-byte boundary,
// modulo the elements between two.
static int to_boundary(const void* p, int size) { return (int)((16 - reinterpret_cast<uintptr_t>(p) % 16) % 16) / size; }

// Whether h (0..7) elements bring the stream to a boundary.
static bool meets(int h, const void* p, int size) { return h % (16 / size) == to_boundary(p, size); }

static void set_vectors(int64_t n, int h, bool meet, int64_t* head, int64_t* vecs) {
    *head = meet && n >= h ? h : 0;
    *vecs = meet && n >= h ? (n - h) / 8 : 0;
}

static int muon_scalars(const zero_muon_t* hp, float divisor, bool update, MuonScalars* h) {
    if (!hp || hp->reserved != 0) return ZERO_EINVAL;
    if (!(divisor > 0.0f) || !std::isfinite(divisor)) return ZERO_EINVAL;
    if (!(hp->momentum >= 0.0f && hp->momentum < 1.0f) || !std::isfinite(hp->weight_decay) || !std::isfinite(hp->scale)) return ZERO_EINVAL;
    if (hp->nesterov != 0 && hp->nesterov != 1) return ZERO_EINVAL;
    if (!hp->sched && !std::isfinite(hp->lr)) return ZERO_EINVAL;
    if (hp->sched && check_aligned(hp->sched, 4)) return ZERO_EALIGN;
    h->divisor = divisor;
    int e2 = 0;
    const float mant = std::frexp(divisor, &e2);
    h->inv_divisor = (mant == 0.5f && e2 >= -125 && e2 <= 127) ? std::ldexp(1.0f, 1 - e2) : 0.0f;
    h->mu = hp->momentum;
    h->nesterov = hp->nesterov != 0;
    h->lr = hp->lr;
    h->wd = hp->weight_decay;
    h->scale = hp->scale;
    h->sched = update ? hp->sched : nullptr;
    return ZERO_OK;
}

constexpr int kMuonWaves = 16;
static unsigned muon_grid(const void* kernel, int64_t n, int64_t vecs) {
    const int64_t ends = n - vecs * 8, work = vecs > ends ? vecs : ends;
    return grid_for(work, kThreads, (int64_t)sm_count() * ctas_per_sm(kernel, kThreads, 0) * kMuonWaves);
}

}  // namespace zgb

extern "C" int zero_reduce_scatter_momentum(const zero_layout_t* L, const void* const* src, int32_t n_src, int32_t src_dtype,
                                            int64_t src_base, float divisor, int32_t rank_begin, int32_t rank_end, int64_t begin,
                                            int64_t end, float* m, uint16_t* u, int32_t out_mode, const zero_muon_t* hp, void* stream) {
    using namespace zgb;
    MomentumParams p{};
    UpdateTarget t{};
    if (const int rc = prepare_target(L, rank_begin, rank_end, begin, end, m, m, m, u, out_mode, false, &t)) return rc;
    if (const int rc = muon_scalars(hp, divisor, false, &p.h)) return rc;
    if (!src || n_src < 1 || (src_dtype != ZERO_BF16 && src_dtype != ZERO_F32) || src_base > begin || src_base < 0) return ZERO_EINVAL;
    if (n_src > ZERO_MAX_SRC) return ZERO_ERANGE;
    const int size = src_dtype == ZERO_BF16 ? 2 : 4;
    for (int r = 0; r < n_src; ++r)
        if (!src[r]) return ZERO_EINVAL;
    for (int r = 0; r < n_src; ++r)
        if (check_aligned(src[r], size)) return ZERO_EALIGN;
    if (begin == end) return ZERO_OK;
    for (int r = 0; r < n_src; ++r)
        if (check_source_ptr(src[r])) return ZERO_EINVAL;
    if (check_device_ptr(t.w) || check_device_ptr(t.out)) return ZERO_EINVAL;
    p.m = t.w;
    p.u = t.out;
    p.n = t.n;
    p.n_src = n_src;
    const int h = to_boundary(p.u, 2);
    bool meet = meets(h, p.m, 4);
    for (int r = 0; r < n_src; ++r) {
        p.src[r] = static_cast<const char*>(src[r]) + (begin - src_base) * size;
        meet = meet && meets(h, p.src[r], size);
    }
    set_vectors(p.n, h, meet, &p.head, &p.vecs);
    void (*kernel)(MomentumParams) = src_dtype == ZERO_F32 ? (n_src == 1 ? momentum_kernel<false, 1> : momentum_kernel<false, 0>)
                                     : n_src == 1         ? momentum_kernel<true, 1>
                                     : n_src == 2         ? momentum_kernel<true, 2>
                                     : n_src == 4         ? momentum_kernel<true, 4>
                                     : n_src == 8         ? momentum_kernel<true, 8>
                                                          : momentum_kernel<true, 0>;
    kernel<<<muon_grid((const void*)kernel, p.n, p.vecs), kThreads, 0, static_cast<cudaStream_t>(stream)>>>(p);
    return launch_status();
}

extern "C" int zero_muon_update(const zero_layout_t* L, const uint16_t* update, int64_t update_base, int32_t rank_begin,
                                int32_t rank_end, int64_t begin, int64_t end, float* master, uint16_t* out, int32_t out_mode,
                                const zero_muon_t* hp, void* stream) {
    using namespace zgb;
    MuonUpdateParams p{};
    UpdateTarget t{};
    if (const int rc = prepare_target(L, rank_begin, rank_end, begin, end, master, master, master, out, out_mode, false, &t)) return rc;
    if (const int rc = muon_scalars(hp, 1.0f, true, &p.h)) return rc;
    if (!update || update_base > begin || update_base < 0) return ZERO_EINVAL;
    if (check_aligned(update, 2)) return ZERO_EALIGN;
    if (begin == end) return ZERO_OK;
    if (check_device_ptr(update) || (p.h.sched && check_device_ptr(p.h.sched)) || check_device_ptr(t.w) || check_device_ptr(t.out)) return ZERO_EINVAL;
    p.o = update + (begin - update_base);
    p.w = t.w;
    p.out = t.out;
    p.n = t.n;
    const int h = to_boundary(p.out, 2);
    set_vectors(p.n, h, meets(h, p.w, 4) && meets(h, p.o, 2), &p.head, &p.vecs);
    muon_update_kernel<<<muon_grid((const void*)muon_update_kernel, p.n, p.vecs), kThreads, 0, static_cast<cudaStream_t>(stream)>>>(p);
    return launch_status();
}
