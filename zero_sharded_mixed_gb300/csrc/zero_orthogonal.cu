// Orthogonalised matrices by a quintic Newton-Schulz iteration, sm_103a:
//   X = U / (|U| + eps);  S times:  A = X X^T,  B = b A + c A A,  X = a X + B X
// on the shorter side (A = X^T X and X = a X + X B for a matrix taller than wide), for a
// batch of equal matrices.  The singular values of U go to the neighbourhood of 1, its
// singular vectors stay: what the Muon optimizer (Jordan et al., 2024) makes of a momentum.
//
// Numbers.  All products run on the tensor core with fp16 operands and fp32 sums: fp16
// has 11 bits where bf16 has 8, at the same rate, and every range here is known: |X| <= 1
// at first and near 1 later, |A| and |B| below 15.  X is stored times 2^12, A and B times
// 2^10, so that even entries of 2^-26 are not subnormal.  An fp16 X alone would lose what
// lies below 2^-11 of its largest directions, which the iteration raises (3.4 times a
// step): a momentum of low rank with a faint rest came out 2 % off, 16 % in bf16.  So X is
// held as the sum of two fp16 numbers, `hi` and `lo` (22 bits), of which the products take
// `hi`, and what they do to `lo` is put in by B's diagonal, its largest part, which is not
// rounded either:  X' = (a + B_ii) (hi + lo) + fp16(B - diagonal) hi.  Against 64 bits:
// 0.3e-3 to 1e-3 of the result by norm, before the 1.7e-3 of its own rounding to bf16;
// with directions of very different strength up to 7e-3 for a bf16 matrix of 128 rows and
// 1.2e-2 for one of 8, whose rounding to bf16 before the call has moved the result by ten
// times that and more, and up to 2e-3 and 7e-3 for an fp32 one (StepEnd).
#include <cuda_fp16.h>

#include <climits>
#include <cmath>

#include "zero_dense.cuh"
#include "zero_tensor.cuh"

namespace zgb {

__device__ int g_orthogonal_status;   // ZERO_OK, or ZERO_ETIMEOUT once a bounded wait gave up
static std::atomic<bool> g_orthogonal_waits;   // whether there was a call: a status check asks no others

int take_orthogonal_status() {
    if (!g_orthogonal_waits.load()) return ZERO_OK;
    int v = 0;
    if (cudaMemcpyFromSymbol(&v, g_orthogonal_status, sizeof v) != cudaSuccess) {
        (void)cudaGetLastError();
        return ZERO_ECUDA;
    }
    if (v != ZERO_OK) {
        const int zero = ZERO_OK;
        if (cudaMemcpyToSymbol(g_orthogonal_status, &zero, sizeof zero) != cudaSuccess) {
            (void)cudaGetLastError();
            return ZERO_ECUDA;
        }
    }
    return v == ZERO_OK ? ZERO_OK : ZERO_ETIMEOUT;
}

constexpr float kX = 4096.0f, kA = 1024.0f, kLo = 2048.0f;   // powers of two that X, A and B, and lo beside hi, are stored times

__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi) {
    const __half2 h = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&h);
}
__device__ __forceinline__ float2 unpack_f16x2(uint32_t x) { return __half22float2(*reinterpret_cast<const __half2*>(&x)); }
__device__ __forceinline__ float round_f16(float x) { return __half2float(__float2half_rn(x)); }

// ---- the input: its norm, and the two fp16 parts of the scaled matrix ---------------------
// Twice through the input (12 x 4800 x 1600: 37 us for 184 MB read, 57 for those and as many
// written); a small one is held by a cluster and read once.
struct SourceParams {
    const void* x; int64_t ldx, stride;
    int32_t rows, cols, groups;        // groups of eight columns a row
    uint32_t inverse, shift;           // g / groups = g inverse >> shift, for the groups of a matrix (fewer than 2^29)
    int32_t parts;
    bool f32, vec;
    double* norm;                      // [batch][parts]
    float* scale;                      // [batch]: X = scale * hi
    float* even;                       // [batch], set to 1 for the first step; or null
    uint16_t* hi;
    uint16_t* lo;                      // null: hi is exact
    int64_t ld, to;                    // of hi and lo: row and matrix stride
    float eps;
};
constexpr int kSourceThreads = 256;

// Groups of eight that a thread has in flight.
constexpr int kFlying = 4;

struct SourceGroup {
    uint4 u[2];
    int32_t row, col;   // col < 0: none
    __device__ __forceinline__ void load(const SourceParams& p, int64_t from, uint32_t g, uint32_t all) {
        row = (int32_t)((uint64_t)g * p.inverse >> p.shift);
        col = g < all ? (int32_t)(g - (uint32_t)row * (uint32_t)p.groups) * 8 : -1;
        u[0] = u[1] = make_uint4(0u, 0u, 0u, 0u);
        if (col < 0) return;
        const int64_t at = from + row * p.ldx + col;
        if (p.vec) {
            const char* q = static_cast<const char*>(p.x) + at * (p.f32 ? 4 : 2);
            u[0] = ld_live_u4(q);
            if (p.f32) u[1] = ld_live_u4(q + 16);
            return;
        }
        const int n = p.cols - col;
        uint32_t w[8];   // fp32, or bf16 in the upper halves
#pragma unroll
        for (int k = 0; k < 8; ++k)
            w[k] = k >= n ? 0u : p.f32 ? static_cast<const uint32_t*>(p.x)[at + k] : (uint32_t)static_cast<const uint16_t*>(p.x)[at + k] << 16;
        u[0] = make_uint4(w[0], w[1], w[2], w[3]);
        u[1] = make_uint4(w[4], w[5], w[6], w[7]);
    }
    __device__ __forceinline__ void get(const SourceParams& p, float (&v)[8]) const {
        if (p.f32 || !p.vec)
            raw8<true>(u, v);
        else
            raw8<false>(u, v);
    }
    // Squares: in fp32 where none can leave its range, else in fp64.
    __device__ __forceinline__ void square(const SourceParams& p, float& near, double& far) const {
        float v[8], most = 0.0f, s = 0.0f;
        get(p, v);
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            most = fmaxf(most, fabsf(v[k]));
            s += v[k] * v[k];
        }
        if ((most > 1e-12f && most < 1e16f && s == s) || (most == 0.0f && s == 0.0f)) {
            near += s;
        } else {
#pragma unroll
            for (int k = 0; k < 8; ++k) far += (double)v[k] * (double)v[k];
        }
    }
    // hi + lo / 2^11 = x f1 f2.
    __device__ __forceinline__ void part(const SourceParams& p, int64_t to, float f1, float f2) const {
        if (col < 0) return;
        float v[8], r[8];
        get(p, v);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            v[j] = v[j] * f1 * f2;
            r[j] = (v[j] - round_f16(v[j])) * kLo;
        }
        const int64_t at = to + row * p.ld + col;
        *reinterpret_cast<uint4*>(p.hi + at) = make_uint4(pack_f16x2(v[0], v[1]), pack_f16x2(v[2], v[3]), pack_f16x2(v[4], v[5]), pack_f16x2(v[6], v[7]));
        if (p.lo)
            *reinterpret_cast<uint4*>(p.lo + at) = make_uint4(pack_f16x2(r[0], r[1]), pack_f16x2(r[2], r[3]), pack_f16x2(r[4], r[5]), pack_f16x2(r[6], r[7]));
    }
};

// Over a warp; fp64 additions are few an SM, so only where they are needed.
__device__ __forceinline__ double warp_sum(float near, double far) {
    for (int o = 16; o; o /= 2) near += __shfl_xor_sync(0xffffffffu, near, o);
    if (__any_sync(0xffffffffu, far != 0.0)) {   // or NaN
        for (int o = 16; o; o /= 2) far += __shfl_xor_sync(0xffffffffu, far, o);
        return (double)near + far;
    }
    return (double)near;
}

// The sum of squares of every `share`-th group of eight from `first`, over a warp's threads:
// in fp32 where none can leave its range, else in fp64.
__device__ __forceinline__ double squares(const SourceParams& p, int z, uint32_t first, uint32_t share) {
    const int64_t from = (int64_t)z * p.stride;
    float sum = 0.0f;
    double far = 0.0;
    const uint32_t all = (uint32_t)p.rows * (uint32_t)p.groups;
    for (uint32_t g = first; g < all; g += kFlying * share) {   // from the end, so that the beginning is in L2 when it is read again
        SourceGroup x[kFlying];
#pragma unroll
        for (int i = 0; i < kFlying; ++i) x[i].load(p, from, all - 1 - (g + i * share), all);   // wraps past `all` where there is none
#pragma unroll
        for (int i = 0; i < kFlying; ++i) x[i].square(p, sum, far);
    }
    return warp_sum(sum, far);
}

// hi + lo / 2^11 = x 2^(12 - e) with e the norm's exponent, and scale = 2^e / norm: the
// power of two costs a bf16 x no bit, and the first step's products take in the scale.
// One thread forms them, in fp32 beside the exponents (fp64 is slow: its root and quotient
// took 0.4 us more, by all threads of a CTA 8 us).
struct SourceScale {
    float f1, f2, scale;   // f1 f2 = 2^(12 - e), in two parts for want of range
};
__device__ __noinline__ SourceScale source_scale(double sum, float eps) {
    if (!(sum < INFINITY)) return SourceScale{64.0f, 64.0f, NAN};   // of what is not finite, NaN
    // sum = m 4^k with 1 <= m < 4, norm = n 2^e
    const int hi = __double2hiint(sum), k = ((hi >> 20) - 1023) >> 1;
    const int of_eps = eps > 0.0f ? ilogbf(eps) : INT_MIN;
    int e = sum > 0.0 && k > of_eps ? k : of_eps;
    if (e == INT_MIN) return SourceScale{64.0f, 64.0f, 0.0f};   // of zeros, zeros
    float n = eps > 0.0f ? ldexpf(eps, -e) : 0.0f;
    if (sum > 0.0) n += ldexpf(sqrtf((float)__hiloint2double(hi - 2 * k * (1 << 20), __double2loint(sum))), k - e);
    // 1 <= n < 4
    for (; n >= 1.0f; ++e) n *= 0.5f;
    const int f = 12 - e;
    return SourceScale{ldexpf(1.0f, f / 2), ldexpf(1.0f, f - f / 2), 1.0f / n};
}
__device__ __forceinline__ void parts_of(const SourceParams& p, int z, const SourceScale& s, uint32_t first, uint32_t share) {
    const float f1 = s.f1, f2 = s.f2;
    const int64_t from = (int64_t)z * p.stride, to = (int64_t)z * p.to;
    const uint32_t all = (uint32_t)p.rows * (uint32_t)p.groups;
    for (uint32_t g = first; g < all; g += kFlying * share) {
        SourceGroup x[kFlying];
#pragma unroll
        for (int i = 0; i < kFlying; ++i) x[i].load(p, from, g + i * share, all);
#pragma unroll
        for (int i = 0; i < kFlying; ++i) x[i].part(p, to, f1, f2);
    }
}

__global__ void __launch_bounds__(kSourceThreads) orthogonal_norm_kernel(const SourceParams p) {
    await_predecessor();
    __shared__ double part[kSourceThreads / 32];
    const double mine = squares(p, blockIdx.y, blockIdx.x * kSourceThreads + threadIdx.x, gridDim.x * kSourceThreads);
    if (threadIdx.x % 32 == 0) part[threadIdx.x / 32] = mine;
    __syncthreads();
    if (threadIdx.x == 0) {
        double t = 0.0;
        for (int w = 0; w < kSourceThreads / 32; ++w) t += part[w];
        p.norm[(int64_t)blockIdx.y * p.parts + blockIdx.x] = t;
    }
}

__global__ void __launch_bounds__(kSourceThreads) orthogonal_source_kernel(const SourceParams p) {
    await_predecessor();
    __shared__ SourceScale scale;
    if (threadIdx.x < 32) {   // one warp adds the parts, every CTA in the same order
        double t = 0.0;
        for (int i = threadIdx.x; i < p.parts; i += 32) t += p.norm[(int64_t)blockIdx.y * p.parts + i];
        t = warp_sum(0.0f, t);
        if (threadIdx.x == 0) {
            scale = source_scale(t, p.eps);
            if (blockIdx.x == 0) {
                p.scale[blockIdx.y] = scale.scale;
                if (p.even) p.even[blockIdx.y] = 1.0f;
            }
        }
    }
    __syncthreads();
    parts_of(p, blockIdx.y, scale, blockIdx.x * kSourceThreads + threadIdx.x, gridDim.x * kSourceThreads);
}

// Both in one, for a matrix that the threads of a cluster of eight hold: read once, and a
// launch less (4 us).
constexpr int kHeldThreads = 1024, kHeldCtas = 8;
constexpr int64_t kHeldGroups = (int64_t)kFlying * kHeldThreads * kHeldCtas;

__global__ void __launch_bounds__(kHeldThreads, 1) orthogonal_held_kernel(const SourceParams p) {
    __shared__ double part[kHeldThreads / 32], total;
    __shared__ SourceScale scale;
    await_predecessor();
    const int z = blockIdx.x / kHeldCtas, rank = blockIdx.x % kHeldCtas;
    const uint32_t all = (uint32_t)p.rows * (uint32_t)p.groups, share = kHeldCtas * kHeldThreads;
    SourceGroup x[kFlying];
#pragma unroll
    for (int i = 0; i < kFlying; ++i) x[i].load(p, (int64_t)z * p.stride, rank * kHeldThreads + threadIdx.x + i * share, all);
    float near = 0.0f;
    double far = 0.0;
#pragma unroll
    for (int i = 0; i < kFlying; ++i) x[i].square(p, near, far);
    const double mine = warp_sum(near, far);
    if (threadIdx.x % 32 == 0) part[threadIdx.x / 32] = mine;
    __syncthreads();
    if (threadIdx.x < 32) {
        const double t = warp_sum(0.0f, part[threadIdx.x]);
        if (threadIdx.x == 0) total = t;
    }
    cluster_sync();
    if (threadIdx.x == 0) {   // every CTA in the same order
        double t[kHeldCtas];
#pragma unroll
        for (int i = 0; i < kHeldCtas; ++i) t[i] = peer_load_double(peer_addr(smem_addr(&total), i));
#pragma unroll
        for (int o = 1; o < kHeldCtas; o *= 2)
#pragma unroll
            for (int i = 0; i < kHeldCtas; i += 2 * o) t[i] += t[i + o];
        scale = source_scale(t[0], p.eps);
        if (rank == 0) {
            p.scale[z] = scale.scale;
            if (p.even) p.even[z] = 1.0f;
        }
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < kFlying; ++i) x[i].part(p, (int64_t)z * p.to, scale.f1, scale.f2);
    cluster_started();   // the totals are read before their CTAs end
}

// ---- products --------------------------------------------------------------------------------
// Pairs of CTAs on 256 x bn tiles, as for the large dense products: warp 0 copies, warp 1
// of the even CTA issues, warps 4..19 end the last tile meanwhile.  A symmetric result is
// computed for the tiles that reach above its diagonal and written to both sides.
// Large ones run at the tensor core's rate (4096 x 11008: X' in 10 waves of tiles at 32900
// cycles each, 32768 being the products' own) and at the clock that the power limit leaves,
// 1.4 to 1.5 GHz: 2.1 ms for 3.11 TFLOP.  At 12 x 4800 x 1600 X' moves 740 MB besides, 216
// to 238 us a step for 184 of products at that clock.  Small ones are bound by latency:
// 256 x 256 takes 3.4 us a product: some 1 from one kernel's end to the next one's first load,
// 1.0 until that arrives, 0.9 for products and their commit, 0.4 to 0.9 for the end (and
// 0.5 more where the first tile's place and the end's first pass come after the wait for the
// kernel before).
enum Step { kGram, kSquare, kApplyWide, kApplyTall };
constexpr bool applies(Step s) { return s == kApplyWide || s == kApplyTall; }
template <Step kStep> constexpr bool kApplies = applies(kStep);

// What the end of a step reads and writes.
struct StepEnding {
    int32_t rows, cols;                    // of the result
    bool first;                            // X = scale * (hi + lo / 2^11)
    int64_t ld, stride;                    // rows of a matrix, and matrices, of all of c and d
    const uint16_t* c_hi;                  // kSquare: A; else X
    const uint16_t* c_lo;                  // or null
    uint16_t* d_hi;                        // A, B or the next X
    uint16_t* d_lo;
    uint16_t* y; int64_t ldy, y_stride;    // the last X: bf16 in place of d
    bool y_vec;
    float* factors; int64_t factor_stride; // scale (a + B_ii)
    bool turned;                           // kSquare: rows of d in the order of turned_row
    float* partial; int64_t partial_stride;   // kGram of few tiles and a long sum: its parts, as matrices of fp32, or null
    const float* scale;
    float* even; float* even_next;         // kEven: how alike the singular values are, of this iteration and of the next
    float a, b, c;
};
struct StepParams {
    CUtensorMap map_a, map_b;
    int32_t depth;                         // the reduced dimension
    int32_t tiles_n, tiles, full, all;     // column tiles; tiles a matrix of which `full` counts the batch's; and with narrow ones after those
    int32_t lights;                        // narrow tiles for pairs with one full tile less
    int32_t bn, k_blocks;
    int32_t splits, share;                 // kGram: parts of the sum, and their blocks
    bool a_mn, b_mn;
    StepEnding e;
};

constexpr int kStageBytes = 32768;      // 128 rows of A and 128 of B, 64 reduced elements each
constexpr int kStages = 6;
constexpr int kEndWarps = 16;
constexpr int kStepThreads = 128 + 32 * kEndWarps;
constexpr int kUnitBytes = 1024;        // 16 rows x 32 columns: an ending warp has two, for hi and lo
constexpr int kStepSmem = 1024 + kStages * kStageBytes + 256 + kEndWarps * 2 * kUnitBytes;

struct Place {
    int z, tm, tn, part;
};
// The order of the tiles.  X' goes through X once: a wide X column by column, a tall
// one row by row, the rows or columns of B together.  A symmetric result has of row tile
// i the column tiles from its own columns on, so that the narrow last tiles are as many
// as can be, and those of the whole batch come last (Turns); its matrices are taken last
// to first, since what the last step wrote last is still in L2 (and what this one read
// last will be when X is read again), the narrow tiles first to last for the same reason.
template <Step kStep>
__device__ __forceinline__ Place place_of(const StepParams& p, int t) {
    Place w;
    w.part = 0;
    if constexpr (kApplies<kStep>) {
        w.z = t / p.tiles;
        t -= w.z * p.tiles;
        if constexpr (kStep == kApplyTall) {
            w.tm = t / p.tiles_n;
            w.tn = t - w.tm * p.tiles_n;
        } else {
            const int tiles_m = (p.e.rows + 255) / 256;
            w.tn = t / tiles_m;
            w.tm = t - w.tn * tiles_m;
        }
    } else if (t < p.full) {
        const int step = 256 / p.bn;
        int n = p.e.cols / p.bn;   // full tiles of a row of tiles
        w.z = t / p.tiles;
        t -= w.z * p.tiles;
        w.z = p.full / p.tiles - 1 - w.z;
        for (w.tm = 0; t >= n; ++w.tm) {
            t -= n;
            n -= step;
        }
        w.tn = w.tm * step + t;
    } else {
        const int tiles_m = (p.e.rows + 255) / 256;
        t -= p.full;
        w.z = t / tiles_m;
        w.tm = t - w.z * tiles_m;
        w.tn = p.tiles_n - 1;
    }
    if (kStep == kGram && p.splits > 1) {
        const int z = w.z / p.splits;
        w.part = w.z - z * p.splits;
        w.z = z;
    }
    return w;
}
// The blocks of a tile's sum.
template <Step kStep>
__device__ __forceinline__ void blocks_of(const StepParams& p, const Place& w, int* from, int* to) {
    *from = kStep == kGram ? w.part * p.share : 0;
    *to = kStep == kGram && *from + p.share < p.k_blocks ? *from + p.share : p.k_blocks;
}
// A pair's tiles: every so many of the full ones; then of the narrow ones, which take half
// to three quarters of the time, the first `lights` are for those pairs that have had one
// full tile less, and the rest for all in turn, those first.  (In one order for all
// 12 x 4800 x 1600 took the pairs up to five full tiles' time where 4.0 are the mean.)
struct Turns {
    int pair, pairs, own, lights, light, place;
    __device__ __forceinline__ explicit Turns(const StepParams& p) : pair(blockIdx.x / 2), pairs(gridDim.x / 2) {
        const int more = p.full % pairs;   // pairs with one more
        own = p.full / pairs + (pair < more ? 1 : 0);
        light = pairs - more;
        place = pair >= more ? pair - more : pair + light;   // in the order for narrow tiles
        lights = place < light && place < p.lights ? (p.lights - place + light - 1) / light : 0;
    }
    __device__ __forceinline__ int tile(const StepParams& p, int i) const {   // its i-th, or -1
        if (i < own) return pair + i * pairs;
        i -= own;
        if (i < lights) return p.full + place + i * light;
        const int t = p.full + p.lights + place + (i - lights) * pairs;
        return t < p.all ? t : -1;
    }
};
// Where row r of B stands for a tall X: X B then has the columns 8 j .. + 7 of every 32 in
// one lane's eight accumulators, as X is read and written.
__device__ __forceinline__ int turned_row(int r) { return (r & ~31) | (r >> 1 & 3) << 3 | (r >> 3 & 3) << 1 | (r & 1); }
__device__ __forceinline__ int width_of(const StepParams& p, int tn) {   // columns of the tile, up to a multiple of 32
    const int left = p.e.cols - tn * p.bn;
    return left >= p.bn ? p.bn : (left + 31) / 32 * 32;
}

// A unit of 16 rows x 32 columns of 16 bits is ended by a warp.  In registers a lane 4 i + j
// has the pairs of columns 8 g + 2 j, + 1 of rows i + 8 h, as the accumulator gives them
// (v[g][2 h], v[g][2 h + 1]); memory is read and written in 16-byte vectors, columns 8 j
// .. + 7 of those rows.  One becomes the other in the warp's own shared memory, by
// the matrix loads and stores: rows of 64 bytes whose vectors are exchanged so that neither
// side has two accesses to a bank.  X B of a tall X has its columns in the order of memory
// (turned_row) and needs none of this, which shared memory, busy with the operands, made
// the bound of a short product's end.
struct UnitPlace {
    uint32_t base, vec, frag, turned;   // shared addresses: of this lane's vector, of the row it names to a matrix access, of that in the transpose
    __device__ __forceinline__ explicit UnitPlace(uint32_t base) : base(base) {
        const uint32_t lane = threadIdx.x & 31, i = lane >> 2, j = lane & 3, g = lane >> 3, r = lane & 7;
        vec = base + i * 64 + 16 * (j ^ (i >> 1 & 3));
        frag = base + r * 64 + 16 * (g ^ (r >> 1 & 3));
        turned = base + lane * 32 + 16 * (r >> 2);   // rows of 32 bytes: of column `lane`
    }
};
__device__ __forceinline__ void unit_store(uint32_t at, const uint4& v) {
    asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(at), "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w) : "memory");
}
__device__ __forceinline__ uint4 unit_load(uint32_t at) {
    uint4 v;
    asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(at) : "memory");
    return v;
}
__device__ __forceinline__ void matrix_load(uint32_t at, uint32_t (&f)[4]) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];" : "=r"(f[0]), "=r"(f[1]), "=r"(f[2]), "=r"(f[3]) : "r"(at) : "memory");
}
__device__ __forceinline__ void matrix_store(uint32_t at, const uint32_t (&f)[4]) {
    asm volatile("stmatrix.sync.aligned.m8n8.x4.shared.b16 [%0], {%1, %2, %3, %4};" ::"r"(at), "r"(f[0]), "r"(f[1]), "r"(f[2]), "r"(f[3]) : "memory");
}
__device__ __forceinline__ void matrix_store_turned(uint32_t at, const uint32_t (&f)[4]) {
    asm volatile("stmatrix.sync.aligned.m8n8.x4.trans.shared.b16 [%0], {%1, %2, %3, %4};" ::"r"(at), "r"(f[0]), "r"(f[1]), "r"(f[2]), "r"(f[3]) : "memory");
}

// Matrices of the workspace have rows of whole units, so that only rows are checked.
// kEven (an fp32 input): what stands for B in its product with lo.  Where some singular values
// are far below the others, B is near zero on their vectors, but its diagonal, which holds a
// share of the others' part, is not, and moves them by rounding errors of the large ones: 3 %
// for 300 x 500 with one direction above a rest of 1e-4.  Leaving the product out errs along
// the large directions alone, by 2^-12 of their own size, which costs matrices of equal
// directions more (1.3e-3 for 0.8e-3).  So the diagonal stands for B where all rows of A have
// most of themselves on theirs, (A_ii)^2 > (A A)_ii / 2 (3/4 for fewer than eight rows, of
// which one faint direction in three leaves two thirds: 2.3e-2 for 9e-3), and else nothing
// does.  The least of a matrix's rows decides, since a row that one large direction has for
// itself looks well alone.
template <Step kStep, bool kEven>
struct StepEnd {
    static constexpr bool kTall = kStep == kApplyTall;
    uint4 hi[2], lo[2];   // a unit's on their way, this lane's vectors
    float4 f[2];          // kTall: the factors of their columns
    float s, f_row[2];    // of a tile: the scale; kApplyWide: the rows' factors
    bool alike;           // kEven: whether the diagonal stands for B on lo
    __device__ __forceinline__ void tile(const StepEnding& p, int z, int row0) {
        s = p.first ? p.scale[z] : 1.0f;
        if constexpr (kEven && kApplies<kStep>) alike = p.even[z] > ((p.rows < p.cols ? p.rows : p.cols) < 8 ? 0.75f : 0.5f);
        if constexpr (kStep == kApplyWide) {
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const int row = row0 + ((threadIdx.x & 31) >> 2) + 8 * h;
                f_row[h] = row < p.rows ? p.factors[z * p.factor_stride + row] : 0.0f;
            }
        }
    }
    __device__ __forceinline__ void load(const StepEnding& p, int z, int row0, int col0) {
        if constexpr (kStep != kGram) {
            const int i = (threadIdx.x & 31) >> 2, j = threadIdx.x & 3;
            const int64_t at = z * p.stride + (row0 + i) * p.ld + col0 + 8 * j;
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                hi[h] = lo[h] = make_uint4(0u, 0u, 0u, 0u);
                if (row0 + i + 8 * h < p.rows) {
                    hi[h] = *reinterpret_cast<const uint4*>(p.c_hi + at + 8 * h * p.ld);
                    if (kApplies<kStep> && p.c_lo) lo[h] = ld_live_u4(p.c_lo + at + 8 * h * p.ld);   // read once
                }
                if constexpr (kTall) f[h] = *reinterpret_cast<const float4*>(p.factors + z * p.factor_stride + col0 + 8 * j + 4 * h);
            }
        }
    }
    // What has been loaded, to shared memory: the registers are free for the next unit's.
    __device__ __forceinline__ void put(const UnitPlace& u) const {
        if constexpr (kStep == kSquare || kStep == kApplyWide) {
            __syncwarp();
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                unit_store(u.vec + 512 * h, hi[h]);
                if (kStep == kApplyWide) unit_store(u.vec + kUnitBytes + 512 * h, lo[h]);
            }
            __syncwarp();
        }
    }
    // kOnce: nothing else reads it soon.
    template <bool kOnce>
    __device__ __forceinline__ static void write(uint16_t* q, const uint4& v) {
        kOnce ? __stcs(reinterpret_cast<uint4*>(q), v) : (void)(*reinterpret_cast<uint4*>(q) = v);
    }
    // Whether a unit meets the diagonal.
    __device__ __forceinline__ static bool on_diagonal(int row0, int col0) { return row0 < col0 + 32 && col0 < row0 + 16; }
    // The result's pairs, from the accumulators and what was loaded.
    __device__ __forceinline__ void form(const StepEnding& p, const UnitPlace& u, int z, int row0, int col0, const float (&v)[4][4], float2 (&w)[2][4]) const {
        if constexpr (kStep == kGram) {
            const float t = s * s * (kA / (kX * kX));
#pragma unroll
            for (int g = 0; g < 4; ++g)
#pragma unroll
                for (int h = 0; h < 2; ++h) w[h][g] = __fmul2_rn(make_float2(v[g][2 * h], v[g][2 * h + 1]), make_float2(t, t));
        }
        if constexpr (kStep == kSquare) {
            const float2 b = make_float2(p.b, p.b), c = make_float2(p.c / kA, p.c / kA);
            float least = 1.0f;
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                uint32_t x[4];
                matrix_load(u.frag + 512 * h, x);
#pragma unroll
                for (int g = 0; g < 4; ++g)
                    w[h][g] = __ffma2_rn(b, unpack_f16x2(x[g]), __fmul2_rn(make_float2(v[g][2 * h], v[g][2 * h + 1]), c));
                if (kEven && on_diagonal(row0, col0)) {
                    const int row = row0 + ((threadIdx.x & 31) >> 2) + 8 * h;
#pragma unroll
                    for (int g = 0; g < 4; ++g)
#pragma unroll
                        for (int k = 0; k < 2; ++k) {
                            const float2 d = unpack_f16x2(x[g]);
                            const float a = k ? d.y : d.x, aa = v[g][2 * h + k];   // A_ii, (A A)_ii
                            if (row == col0 + 8 * g + 2 * (int)(threadIdx.x & 3) + k && row < p.rows && aa > 0.0f) least = fminf(least, a * a / aa);
                        }
                }
            }
            if (kEven && on_diagonal(row0, col0)) {   // floats from 0 on are in the order of their bits
                const uint32_t bits = __reduce_min_sync(0xffffffffu, __float_as_uint(least));
                if ((threadIdx.x & 31) == 0 && bits < __float_as_uint(1.0f)) atomicMin(reinterpret_cast<uint32_t*>(p.even) + z, bits);
            }
        }
        if constexpr (kApplies<kStep>) {
            const float2 c = make_float2(s * (1.0f / kA), s * (1.0f / kA)), l = make_float2(1.0f / kLo, 1.0f / kLo);
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                uint32_t x[4] = {hi[h].x, hi[h].y, hi[h].z, hi[h].w}, y[4] = {lo[h].x, lo[h].y, lo[h].z, lo[h].w};
                if constexpr (!kTall) {
                    matrix_load(u.frag + 512 * h, x);
                    matrix_load(u.frag + kUnitBytes + 512 * h, y);
                }
#pragma unroll
                for (int g = 0; g < 4; ++g) {
                    const float4 e = f[g / 2];
                    const float2 a = !kTall ? make_float2(f_row[h], f_row[h]) : g & 1 ? make_float2(e.z, e.w) : make_float2(e.x, e.y);
                    const float2 product = __fmul2_rn(c, make_float2(v[g][2 * h], v[g][2 * h + 1]));
                    if constexpr (kEven) {
                        const float2 low = __fmul2_rn(l, alike ? a : make_float2(s * p.a, s * p.a));
                        w[h][g] = __ffma2_rn(a, unpack_f16x2(x[g]), __ffma2_rn(low, unpack_f16x2(y[g]), product));
                    } else {
                        w[h][g] = __ffma2_rn(a, __ffma2_rn(l, unpack_f16x2(y[g]), unpack_f16x2(x[g])), product);
                    }
                }
            }
        }
        if constexpr (kStep == kSquare || kStep == kApplyWide) __syncwarp();   // what was loaded has been read
    }
    // Eight of a row out of the four lanes that have them, both rows.
    __device__ __forceinline__ static void gather(const UnitPlace& u, uint32_t area, const uint32_t (&d)[2][4]) {
        if constexpr (!kTall) {
            matrix_store(u.frag + area, d[0]);
            matrix_store(u.frag + area + 512, d[1]);
        }
    }
    __device__ __forceinline__ static uint4 row_of(const UnitPlace& u, uint32_t area, const uint32_t (&d)[2][4], int h) {
        if constexpr (kTall)
            return make_uint4(d[h][0], d[h][1], d[h][2], d[h][3]);
        else
            return unit_load(u.vec + area + 512 * h);
    }
    __device__ __forceinline__ static void finish(const StepEnding& p, const UnitPlace& u, float s, int z, int part, int row0, int col0, bool mirror, float2 (&w)[2][4]) {
        const int i = (threadIdx.x & 31) >> 2, j = threadIdx.x & 3;
        if (kStep == kGram && p.partial) {
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const int row = row0 + i + 8 * h;
                float* q = p.partial + part * p.partial_stride + z * p.stride + row * p.ld + col0 + 2 * j;
#pragma unroll
                for (int g = 0; g < 4; ++g)
                    if (row < p.rows) *reinterpret_cast<float2*>(q + 8 * g) = w[h][g];
            }
            if (!mirror) return;
#pragma unroll 1
            for (int k = 0; k < 16; ++k) {   // few, beside sums of as many terms
                const int row = row0 + i + 8 * (k >> 3), col = col0 + 8 * (k >> 1 & 3) + 2 * j + (k & 1);
                float t = 0.0f;
#pragma unroll
                for (int n = 0; n < 16; ++n)
                    if (n == k) t = n & 1 ? w[n >> 3][n >> 1 & 3].y : w[n >> 3][n >> 1 & 3].x;
                if (row < p.rows && col < p.cols) p.partial[part * p.partial_stride + z * p.stride + col * p.ld + row] = t;
            }
            return;
        }
        uint32_t d[2][4];
        if (kApplies<kStep> && p.y) {
            const float2 c = make_float2(1.0f / kX, 1.0f / kX);
            uint16_t* q = p.y + z * p.y_stride + row0 * p.ldy + col0;
#pragma unroll
            for (int h = 0; h < 2; ++h)
#pragma unroll
                for (int g = 0; g < 4; ++g) {
                    const float2 t = __fmul2_rn(w[h][g], c);
                    d[h][g] = pack_bf16x2(t.x, t.y);
                }
            if (p.y_vec && col0 + 32 <= p.cols) {
                gather(u, 0, d);
                __syncwarp();
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const uint4 e = row_of(u, 0, d, h);
                    if (row0 + i + 8 * h < p.rows) write<false>(q + (i + 8 * h) * p.ldy + 8 * j, e);
                }
            } else {
#pragma unroll
                for (int g = 0; g < 4; ++g)
#pragma unroll
                    for (int c = 0; c < 4; ++c) {
                        const int row = i + 8 * (c >> 1), col = (kTall ? 8 * j + 2 * g : 8 * g + 2 * j) + (c & 1);
                        if (row0 + row < p.rows && col0 + col < p.cols) q[row * p.ldy + col] = (uint16_t)(d[c >> 1][g] >> 16 * (c & 1));
                    }
            }
            return;
        }
        if (kStep == kSquare && on_diagonal(row0, col0)) {
#pragma unroll
            for (int g = 0; g < 4; ++g)
#pragma unroll
                for (int c = 0; c < 4; ++c) {
                    const int row = row0 + i + 8 * (c >> 1), col = col0 + 8 * g + 2 * j + (c & 1);
                    float& t = c & 1 ? w[c >> 1][g].y : w[c >> 1][g].x;
                    if (row == col && row < p.rows) {
                        p.factors[z * p.factor_stride + row] = s * (p.a + t * (1.0f / kA));
                        t = 0.0f;
                        if (kEven && row == 0) p.even_next[z] = 1.0f;
                    }
                }
        }
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int g = 0; g < 4; ++g) d[h][g] = pack_f16x2(w[h][g].x, w[h][g].y);
        gather(u, 0, d);
        uint32_t r[2][4];
        if constexpr (kApplies<kStep>) {
#pragma unroll
            for (int h = 0; h < 2; ++h)
#pragma unroll
                for (int g = 0; g < 4; ++g) {
                    const float2 t = unpack_f16x2(d[h][g]);
                    const float2 e = __fmul2_rn(__fadd2_rn(w[h][g], make_float2(-t.x, -t.y)), make_float2(kLo, kLo));
                    r[h][g] = pack_f16x2(e.x, e.y);
                }
            gather(u, kUnitBytes, r);
        } else if (mirror) {
            matrix_store_turned(u.turned + kUnitBytes, d[0]);
            matrix_store_turned((u.turned + kUnitBytes) ^ 16, d[1]);
        }
        if constexpr (!kTall) __syncwarp();
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const int row = row0 + i + 8 * h;
            const int64_t at = z * p.stride + (kStep == kSquare && p.turned ? turned_row(row) : row) * p.ld + col0 + 8 * j;
            const uint4 e = row_of(u, 0, d, h);
            if (row < p.rows) write<false>(p.d_hi + at, e);
            if constexpr (kApplies<kStep>) {
                const uint4 l = row_of(u, kUnitBytes, r, h);
                if (row < p.rows) write<true>(p.d_lo + at, l);
            }
        }
        if (!kApplies<kStep> && mirror) {   // a lane has a column, of sixteen rows
            const int col = col0 + (threadIdx.x & 31);
            const uint4 e0 = unit_load(u.turned + kUnitBytes), e1 = unit_load((u.turned + kUnitBytes) ^ 16);
            if (col < p.cols && row0 < p.rows) {
                uint4* q = reinterpret_cast<uint4*>(p.d_hi + z * p.stride + (kStep == kSquare && p.turned ? turned_row(col) : col) * p.ld + row0);
                q[0] = e0;
                q[1] = e1;
            }
        }
        if constexpr (kStep == kGram) __syncwarp();   // read before the next unit's is written
    }
};

// A warp of either CTA is done reading an accumulator: one arrival at the even CTA.
__device__ __forceinline__ void release_accumulator(uint64_t* bar) {
    tcgen05_fence_before();
    __syncwarp();
    if ((threadIdx.x & 31) == 0) peer_arrive(peer_addr(smem_addr(bar), 0));
}

__device__ __forceinline__ bool step_wait(uint64_t* bar, uint32_t parity) { return warp_wait(bar, parity, &g_orthogonal_status); }

template <Step kStep, bool kEven>
__global__ void __launch_bounds__(kStepThreads, 1) orthogonal_step_kernel(const __grid_constant__ StepParams p) {
    extern __shared__ uint8_t raw_smem[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(raw_smem) + 1023) & ~(uintptr_t)1023);
    uint64_t* full = reinterpret_cast<uint64_t*>(smem + kStages * kStageBytes);
    uint64_t* empty = full + kStages;
    uint64_t* acc_full = empty + kStages;
    uint64_t* acc_empty = acc_full + 2;
    uint64_t* drained = acc_empty + 2;
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(drained + 1);

    const int warp = uniform_warp();
    const uint32_t rank = cluster_rank();
    const Turns turns(p);
    const int t_first = turns.tile(p, 0);   // every pair has one; placed before the wait below
    const Place first_place = place_of<kStep>(p, t_first);

    if (threadIdx.x == 0) {
        for (int s = 0; s < kStages; ++s) {
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
    start_successor();
    const uint32_t tmem = *tmem_slot;

    // the copying, the issuing and the ending warps wait for the kernel before, each as late as
    // it can: the limits of their other waits then count this kernel's time alone
    if (warp == 0) {
        int s = 0;
        uint32_t round = 0;
        bool ok = true;
        for (int n = 0, t = t_first; ok && t >= 0; t = turns.tile(p, ++n)) {
            const Place w = n == 0 ? first_place : place_of<kStep>(p, t);
            const int row = w.tm * 256 + (int)rank * 128;
            const int half = width_of(p, w.tn) / 2, col = w.tn * p.bn + (int)rank * half;
            const int b_boxes = p.b_mn ? (half + 63) / 64 : 1;
            const uint32_t stage_bytes = 16384u + (p.b_mn ? (uint32_t)b_boxes * kSubTileBytes : (uint32_t)p.bn * 64u);
            int from, to;
            blocks_of<kStep>(p, w, &from, &to);
            if (n == 0) await_predecessor();
            for (int kb = from; kb < to; ++kb) {
                if (round > 0 && !(ok = step_wait(empty + s, (round - 1) & 1))) break;
                const uint32_t a = smem_addr(smem + s * kStageBytes), b = a + 16384;
                const uint32_t bar = peer_addr(smem_addr(full + s), 0);
                const int k = kb * 64;
                if (elect_one()) {
                    if (rank == 0) mbar_arrive_expect_tx(full + s, 2 * stage_bytes);
                    if (p.a_mn) {
                        tensor_load_pair(a, &p.map_a, row, k, w.z, bar);
                        tensor_load_pair(a + kSubTileBytes, &p.map_a, row + 64, k, w.z, bar);
                    } else {
                        tensor_load_pair(a, &p.map_a, k, row, w.z, bar);
                    }
                    if (p.b_mn) {
                        for (int i = 0; i < b_boxes; ++i) tensor_load_pair(b + i * kSubTileBytes, &p.map_b, col + 64 * i, k, w.z, bar);
                    } else {
                        tensor_load_pair(b, &p.map_b, k, col, w.z, bar);
                    }
                }
                if (++s == kStages) s = 0, ++round;
            }
        }
        if (!ok && rank == 0)   // copies in flight land before the CTAs end
            for (int i = 0; i < kStages; ++i) {
                const uint32_t done = i < s ? round : round - 1;   // the last round issued on stage i
                if (round > 0 || i < s) (void)mbar_wait_bounded(full + i, done & 1, kWaitCycles / 8);
            }
    } else if (warp == 1 && rank == 0) {
        int s = 0, use = 0;
        uint32_t round = 0;
        bool ok = true;
        const uint32_t a_step = descriptor_step(p.a_mn), b_step = descriptor_step(p.b_mn);
        for (int t = t_first; ok && t >= 0; t = turns.tile(p, ++use)) {
            const Place w = use == 0 ? first_place : place_of<kStep>(p, t);
            const uint32_t idesc = instruction_descriptor(256, width_of(p, w.tn), p.a_mn, p.b_mn, false);
            const int buf = use & 1;
            if (use >= 2 && !(ok = step_wait(acc_empty + buf, (use / 2 - 1) & 1))) break;
            tcgen05_fence_after();
            const uint32_t d = tmem + buf * 256;
            int from, to;
            blocks_of<kStep>(p, w, &from, &to);
            if (use == 0) await_predecessor();
            for (int kb = from; kb < to; ++kb) {
                if (!(ok = step_wait(full + s, round & 1))) break;
                tcgen05_fence_after();
                const uint32_t a = smem_addr(smem + s * kStageBytes);
                const uint64_t da = smem_descriptor(a, p.a_mn), db = smem_descriptor(a + 16384, p.b_mn);
                const int left = p.depth - kb * 64;
                if (elect_one()) {
#pragma unroll
                    for (int i = 0; i < 4; ++i)   // the last step of all may end early
                        if (left > 16 * i) mma_bf16<true>(d, da + i * a_step, db + i * b_step, idesc, kb > from || i > 0);
                    mma_commit<true>(empty + s);
                }
                if (++s == kStages) s = 0, ++round;
            }
            if (ok && elect_one()) mma_commit<true>(acc_full + buf);
        }
        if (!ok) {   // products in flight end before the tensor memory is freed
            if (elect_one()) mma_commit<true>(drained);
            (void)mbar_wait_bounded(drained, 0, kWaitCycles / 8);
        }
    } else if (warp >= 4) {
        // of its 32 rows this warp ends one half, over one half of the columns, side by
        // side so that whole lines are written together
        const int q = warp & 3, h = (warp - 4) / 4, row_in = (int)rank * 128 + q * 32 + (h & 1) * 16;
        const uint32_t lanes = tmem + ((uint32_t)(q * 32 + (h & 1) * 16) << 16);
        const UnitPlace at(smem_addr(smem + kStages * kStageBytes + 256 + (warp - 4) * 2 * kUnitBytes));
        const auto share = [&](const Place& w, int* first) {   // this warp's units of a tile, and the first
            const int all = width_of(p, w.tn) / 32;
            *first = (h >> 1) * ((all + 1) / 2);
            return h >> 1 ? all - *first : (all + 1) / 2;
        };
        StepEnd<kStep, kEven> end{};
        const auto begin = [&](const Place& w) {   // what a tile's end reads first on its way
            int first;
            if (share(w, &first) > 0 && w.tm * 256 + row_in < p.e.rows) {
                end.tile(p.e, w.z, w.tm * 256 + row_in);
                end.load(p.e, w.z, w.tm * 256 + row_in, w.tn * p.bn + first * 32);
            }
        };
        int t = t_first;
        float v[4][4] = {};
        float2 r[2][4];
        if (t >= 0) {
            // before the first tile the end goes once through rows that do not exist, so that
            // its instructions are there when the product is (0.4 us of a launch); it reads
            // and writes no global memory
            const Place w = first_place;
            end.put(at);
            end.form(p.e, at, w.z, p.e.rows, w.tn * p.bn, v, r);
            end.finish(p.e, at, 0.0f, w.z, w.part, p.e.rows, w.tn * p.bn, w.tn * p.bn >= (w.tm + 1) * 256, r);
            await_predecessor();
            begin(w);
        }
        for (int use = 0; t >= 0; ++use) {
            const Place w = place_of<kStep>(p, t);
            int first;
            const int units = share(w, &first), row0 = w.tm * 256 + row_in, buf = use & 1, col_first = w.tn * p.bn + first * 32;
            const bool mirror = w.tn * p.bn >= (w.tm + 1) * 256, mine = row0 < p.e.rows && units > 0;
            t = turns.tile(p, use + 1);
            if (!step_wait(acc_full + buf, (use / 2) & 1)) break;
            tcgen05_fence_after();
            if (mine) {
#pragma unroll 1
                for (int u = 0; u < units; ++u) {
                    end.put(at);
                    if (!end.kTall && u + 1 < units) end.load(p.e, w.z, row0, col_first + u * 32 + 32);
                    tmem_load_fragment(lanes + buf * 256 + (first + u) * 32, v);
                    if (u + 1 == units) release_accumulator(acc_empty + buf);   // this warp's last read
                    end.form(p.e, at, w.z, row0, col_first + u * 32, v, r);
                    if (end.kTall && u + 1 < units) end.load(p.e, w.z, row0, col_first + u * 32 + 32);
                    end.finish(p.e, at, end.s, w.z, w.part, row0, col_first + u * 32, mirror, r);
                }
            } else {
                release_accumulator(acc_empty + buf);
            }
            if (t >= 0) begin(place_of<kStep>(p, t));
        }
    }
    // the CTAs part when both are done with the tensor memories and each other's barriers;
    // their stores are ordered by the kernel's end alone (waiting for them here as well
    // took 0.7 us a launch)
    tcgen05_fence_before();
    __syncthreads();
    cluster_started();
    tcgen05_fence_after();
    if (warp == 2) tmem_free<true>(tmem, 512);
}

// The parts of a split Gram product added in order (they carry their factor already), eight
// columns a thread.
struct JoinParams {
    const float* partial; int64_t partial_stride, square;
    int32_t splits, side, lds;
    uint16_t* d;
};
// kRuns: in runs of 64, for the digits of long sums (the count took 0.6 us where there are few).
template <bool kRuns>
__global__ void __launch_bounds__(256) orthogonal_join_kernel(const JoinParams p) {
    await_predecessor();
    const int groups = p.lds / 8, g = blockIdx.x * 256 + threadIdx.x, row = g / groups, col = (g - row * groups) * 8;
    if (row >= p.side) return;
    const float* q = p.partial + blockIdx.y * p.square;
    float v[8] = {}, all[8] = {};
    q += (int64_t)row * p.lds + col;
#pragma unroll 8
    for (int i = 0; i < p.splits; ++i, q += p.partial_stride) {
        const float4 a = *reinterpret_cast<const float4*>(q), b = *reinterpret_cast<const float4*>(q + 4);
        v[0] += a.x; v[1] += a.y; v[2] += a.z; v[3] += a.w;
        v[4] += b.x; v[5] += b.y; v[6] += b.z; v[7] += b.w;
        if (kRuns && i % 64 == 63)
#pragma unroll
            for (int k = 0; k < 8; ++k) all[k] += v[k], v[k] = 0.0f;
    }
    if (kRuns)
#pragma unroll
        for (int k = 0; k < 8; ++k) v[k] += all[k];
    *reinterpret_cast<uint4*>(p.d + blockIdx.y * p.square + (int64_t)row * p.lds + col) =
        make_uint4(pack_f16x2(v[0], v[1]), pack_f16x2(v[2], v[3]), pack_f16x2(v[4], v[5]), pack_f16x2(v[6], v[7]));
}

// ---- launches ------------------------------------------------------------------------------
// A batch of equal matrices of the workspace: rows `ld` apart, 16-byte aligned.
struct Matrices {
    const uint16_t* p;
    int64_t rows, cols, ld, stride, batch;
};
static bool make_map3(const Matrices& m, int box_rows, CUtensorMap* map) {
    const EncodeTiled encode = encode_tiled();
    if (!encode) return false;
    const cuuint64_t dims[3] = {(cuuint64_t)m.cols, (cuuint64_t)m.rows, (cuuint64_t)m.batch};
    const cuuint64_t pitch[2] = {(cuuint64_t)m.ld * 2, (cuuint64_t)m.stride * 2};
    const cuuint32_t box[3] = {64, (cuuint32_t)box_rows, 1}, unit[3] = {1, 1, 1};
    return encode(map, CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 3, const_cast<uint16_t*>(m.p), dims, pitch, box, unit,
                  CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                  CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// The tile width with the least estimated time: a tile's blocks (bound by the tensor core,
// or for narrow tiles by shared memory) and the part of its end that nothing hides, as
// often as the busiest pair has them.  A symmetric result takes widths that divide 256.
// 256 x 256 takes 57 us in tiles of 32 columns and some 97 in tiles of 256; 2048 x 8192 461 as
// planned, 500 with 128 for all, 561 with 256, 1469 with 32.
struct StepPlan {
    int64_t tiles, full, all, lights, cycles;
    int bn, tiles_n;
};
static StepPlan plan_step(Step step, int64_t rows, int64_t cols, int64_t depth, int64_t batch, int64_t most) {
    const int64_t k_blocks = (depth + 63) / 64, tm = (rows + 255) / 256;
    const auto time_of = [&](int64_t width) { return 1500 + k_blocks * (2 * width > 256 + width ? 2 * width : 256 + width) + 24 * width; };
    StepPlan best{};
    int64_t least = INT64_MAX;
    for (int bn = 256; bn >= 32; bn = applies(step) ? bn - 32 : bn / 2) {
        const int64_t tn = (cols + bn - 1) / bn;
        int64_t tiles = tm * tn, narrow = 0;
        if (!applies(step)) {
            tiles = 0;
            for (int64_t n = cols / bn; n > 0; n -= 256 / bn) tiles += n;
            narrow = cols % bn ? tm : 0;
        }
        if (tiles + narrow > INT32_MAX / 4 / batch) continue;
        StepPlan q{tiles, tiles * batch, (tiles + narrow) * batch, 0, 0, bn, (int)tn};
        const int64_t pairs = q.all < most ? q.all : most, more = q.full % pairs, light = pairs - more;
        const int64_t whole = time_of(bn), part = time_of((cols % bn + 31) / 32 * 32), fit = (whole + part / 2) / part;
        q.lights = q.all - q.full < (fit > 1 ? fit : 1) * light ? q.all - q.full : (fit > 1 ? fit : 1) * light;
        int64_t cycles = q.full / pairs * whole + (q.lights + light - 1) / light * part;
        if (more && cycles < (q.full / pairs + 1) * whole) cycles = (q.full / pairs + 1) * whole;
        cycles += (q.all - q.full - q.lights + pairs - 1) / pairs * part;
        if (cycles < least) least = q.cycles = cycles, best = q;
    }
    return best;
}

// Parts of a Gram product's sum.  First, where few tiles would leave most pairs idle over a long
// axis: what saves a tenth at least, the join included, which takes 5 us of a product.
// (64 x 11008 takes 92 us, 203 in one part.)  Only for sides of one row of tiles, whose parts
// are whole.  Reckoned for the device that this is made for, so that the workspace does not
// depend on the current one.
// Second, as many as keep a part's sum to kLongestRun blocks at any size: the tensor core's sums
// are cut, not rounded, and lose 7e-8 of themselves for every block, so that a row of 2^28 came
// out 12 % off in 16 parts.
constexpr int kMostSplits = 16;
constexpr int64_t kLongestRun = 1024;
static int gram_splits(int64_t side, int64_t longer, int64_t batch, int64_t square) {
    const int64_t blocks = (longer + 63) / 64, fewest = (blocks + kLongestRun - 1) / kLongestRun;
    int64_t best = 1;
    if (side <= 256) {
        const int64_t one = plan_step(kGram, side, side, longer, batch, 76).cycles;
        int64_t least = one - one / 10;
        for (int n = 2; n <= kMostSplits && n <= blocks / 4; ++n) {
            const int64_t share = (blocks + n - 1) / n;
            if ((n - 1) * share >= blocks || n * batch * square > ((int64_t)1 << 24) || n * batch > 65535) continue;
            const int64_t cycles = plan_step(kGram, side, side, share * 64, batch * n, 76).cycles + 9000 + 300 * n;
            if (cycles < least) least = cycles, best = n;
        }
    }
    if (best < fewest) {   // none of them empty
        const int64_t share = (blocks + fewest - 1) / fewest;
        best = (blocks + share - 1) / share;
    }
    return (int)best;
}

// A step's launch but for its end, which changes from iteration to iteration: formed
// before the first launch, so that a call that cannot be made has launched nothing.
template <Step kStep, bool kEven = false>
static int prepare_step(StepParams& q, int64_t rows, int64_t cols, int64_t depth, const Matrices& a, bool a_mn, const Matrices& b, bool b_mn, int splits = 1) {
    static Done done;
    if (const int rc = allow_smem((const void*)orthogonal_step_kernel<kStep, kEven>, kStepSmem, done)) return rc;
    const int64_t blocks = (depth + 63) / 64, share = (blocks + splits - 1) / splits;
    const StepPlan plan = plan_step(kStep, rows, cols, share * 64 < depth ? share * 64 : depth, a.batch * splits, sm_pairs());
    if (!plan.bn) return ZERO_ERANGE;
    q.depth = (int32_t)depth;
    q.bn = plan.bn;
    q.tiles_n = plan.tiles_n;
    q.tiles = (int32_t)plan.tiles;
    q.full = (int32_t)plan.full;
    q.all = (int32_t)plan.all;
    q.lights = (int32_t)plan.lights;
    q.k_blocks = (int32_t)blocks;
    q.splits = splits;
    q.share = (int32_t)share;
    q.a_mn = a_mn; q.b_mn = b_mn;
    return make_map3(a, a_mn ? 64 : 128, &q.map_a) && make_map3(b, b_mn ? 64 : q.bn / 2, &q.map_b) ? ZERO_OK : ZERO_ECUDA;
}
template <Step kStep, bool kEven = false>
static int launch_step(const StepParams& q, cudaStream_t s) {
    const int64_t pairs = sm_pairs();
    return launch_dense(orthogonal_step_kernel<kStep, kEven>, dim3((unsigned)(2 * (q.all < pairs ? q.all : pairs))), kStepThreads, 2, true, kStepSmem,
                        s, q);
}

// Where everything stands in the workspace.
struct OrthogonalSpace {
    int64_t ldx, lds, square, parts;               // rows of X; rows of A and B, and their elements
    int64_t hi[2], lo[2], a, b, factors, norm, scale, even, partial, bytes;
    int splits;                                    // of the Gram products' sums
};
constexpr int64_t kLongest = (int64_t)1 << 30;

static int orthogonal_space(int64_t batch, int64_t rows, int64_t cols, OrthogonalSpace* w) {
    const int64_t side = rows < cols ? rows : cols, longer = rows < cols ? cols : rows;
    // a side's square and a matrix's groups of eight are counted in 31 bits, a batch's bytes in 62
    if (longer > kLongest || side > 32768 || rows * ((cols + 7) / 8) > INT32_MAX / 4) return ZERO_ERANGE;
    w->ldx = (cols + 63) / 64 * 64;
    w->lds = (side + 63) / 64 * 64;
    w->square = (side + 31) / 32 * 32 * w->lds;   // turned_row moves rows within groups of 32
    const int64_t x = rows * w->ldx * 2, a = w->square * 2;
    const int64_t groups = rows * ((cols + 7) / 8), most = batch > 32 ? 32 : 608 / batch;   // four CTAs an SM, of the batch
    w->parts = (groups + 2 * kFlying * kSourceThreads - 1) / (2 * kFlying * kSourceThreads);
    if (w->parts > most) w->parts = most;
    if (batch > ((int64_t)1 << 60) / (4 * x + 2 * a + 16 * w->lds + 16 * w->parts + 4096)) return ZERO_ERANGE;
    int64_t at = 0;
    const auto take = [&](int64_t bytes) {
        const int64_t here = at;
        at += (bytes + 255) / 256 * 256;
        return here;
    };
    for (int i = 0; i < 2; ++i) w->hi[i] = take(batch * x), w->lo[i] = take(batch * x);
    w->a = take(batch * a);
    w->b = take(batch * a);
    w->factors = take(batch * w->lds * (int64_t)sizeof(float));
    w->norm = take(batch * w->parts * 8);
    w->scale = take(batch * 4);
    w->even = take(2 * batch * 4);
    w->splits = gram_splits(side, longer, batch, w->square);
    w->partial = take(w->splits > 1 ? w->splits * batch * w->square * 4 : 0);
    w->bytes = at;
    return ZERO_OK;
}

}  // namespace zgb

extern "C" int zero_orthogonalize_workspace(int64_t batch, int64_t rows, int64_t cols, int64_t* bytes) {
    using namespace zgb;
    if (batch < 0 || rows < 0 || cols < 0 || !bytes) return ZERO_EINVAL;
    *bytes = 0;
    if (batch == 0 || rows == 0 || cols == 0) return ZERO_OK;
    OrthogonalSpace w{};
    if (const int rc = orthogonal_space(batch, rows, cols, &w)) return rc;
    *bytes = w.bytes;
    return ZERO_OK;
}

extern "C" int zero_orthogonalize(int64_t batch, int64_t rows, int64_t cols, const void* x, int64_t x_stride, int64_t ldx,
                                  int32_t x_dtype, uint16_t* y, int64_t y_stride, int64_t ldy, int32_t steps,
                                  const float* coefficients, float eps, void* workspace, int64_t workspace_bytes, void* stream) {
    using namespace zgb;
    if (batch < 0 || rows < 0 || cols < 0 || (x_dtype != ZERO_BF16 && x_dtype != ZERO_F32)) return ZERO_EINVAL;
    if (steps < 1 || steps > 100 || !coefficients || !(eps >= 0.0f) || !std::isfinite(eps)) return ZERO_EINVAL;
    for (int i = 0; i < 3; ++i)
        if (!std::isfinite(coefficients[i])) return ZERO_EINVAL;
    if (batch == 0 || rows == 0 || cols == 0) return ZERO_OK;
    if (const int rc = check_matrix(x, rows, cols, ldx, x_dtype)) return rc;
    if (const int rc = check_matrix(y, rows, cols, ldy, ZERO_BF16)) return rc;
    if (batch > 1) {
        const int64_t most = INT64_MAX / 8 / batch, extent = (rows - 1) * ldy + cols;
        if (x_stride < 0 || y_stride < 0) return ZERO_EINVAL;
        if (x_stride > most || y_stride > most) return ZERO_ERANGE;
        // results lie one behind the other, or side by side in the rows of a wider matrix
        if (y_stride < extent && (y_stride < cols || (batch - 1) * y_stride + cols > ldy)) return ZERO_EINVAL;
    }
    if (batch > 65535) return ZERO_ERANGE;
    OrthogonalSpace w{};
    if (const int rc = orthogonal_space(batch, rows, cols, &w)) return rc;
    if (!workspace) return ZERO_EINVAL;
    if (reinterpret_cast<uintptr_t>(workspace) % 128) return ZERO_EALIGN;
    if (workspace_bytes < w.bytes) return ZERO_ERANGE;
    if (check_device_ptr(x) || check_device_ptr(y) || check_device_ptr(workspace)) return ZERO_EINVAL;

    cudaStream_t s = static_cast<cudaStream_t>(stream);
    char* base = static_cast<char*>(workspace);
    const auto at = [&](int64_t offset) { return reinterpret_cast<uint16_t*>(base + offset); };
    const bool f32 = x_dtype == ZERO_F32, tall = rows > cols;
    const int64_t side = tall ? cols : rows;

    SourceParams src{};
    src.x = x; src.ldx = ldx; src.stride = batch > 1 ? x_stride : 0;
    src.rows = (int32_t)rows; src.cols = (int32_t)cols; src.groups = (int32_t)((cols + 7) / 8);
    src.parts = (int32_t)w.parts;
    int bits = 0;   // 2^bits >= groups: an error below groups / 2^(29 + bits) a group is none after 2^29 of them
    while (((int64_t)1 << bits) < src.groups) ++bits;
    src.shift = 29 + bits;
    src.inverse = (uint32_t)((((uint64_t)1 << src.shift) + src.groups - 1) / src.groups);
    src.f32 = f32;
    src.vec = cols % 8 == 0 && rows_aligned16(x, ldx, f32 ? 4 : 2) && (batch == 1 || x_stride * (f32 ? 4 : 2) % 16 == 0);
    src.norm = reinterpret_cast<double*>(base + w.norm);
    src.scale = reinterpret_cast<float*>(base + w.scale);
    float* const even = f32 ? reinterpret_cast<float*>(base + w.even) : nullptr;   // [2][batch], of odd and even iterations
    src.even = even;
    src.hi = at(w.hi[0]);
    src.lo = f32 ? at(w.lo[0]) : nullptr;
    src.ld = w.ldx; src.to = rows * w.ldx;
    src.eps = eps;
    const Matrices gram{at(w.a), side, side, w.lds, w.square, batch};
    const Matrices poly{at(w.b), tall ? (side + 31) / 32 * 32 : side, side, w.lds, w.square, batch};
    const Matrices first{at(w.hi[0]), rows, cols, w.ldx, src.to, batch}, second{at(w.hi[1]), rows, cols, w.ldx, src.to, batch};
    StepEnding e{};
    e.factors = reinterpret_cast<float*>(base + w.factors); e.factor_stride = w.lds;
    e.turned = tall;
    e.scale = src.scale;
    e.a = coefficients[0]; e.b = coefficients[1]; e.c = coefficients[2];
    const int64_t longer = tall ? rows : cols;
    // the end of a step of iteration i
    const auto ending = [&](Step step, int i) {
        StepEnding d = e;
        d.first = i == 0;
        if (even) {
            d.even = even + (i & 1) * batch;
            d.even_next = even + (~i & 1) * batch;
        }
        if (applies(step)) {
            d.rows = (int32_t)rows; d.cols = (int32_t)cols;
            d.ld = w.ldx; d.stride = rows * w.ldx;
            d.c_hi = at(w.hi[i & 1]);
            d.c_lo = i == 0 && !f32 ? nullptr : at(w.lo[i & 1]);
            d.d_hi = at(w.hi[~i & 1]);
            d.d_lo = at(w.lo[~i & 1]);
        } else {
            d.rows = d.cols = (int32_t)side;
            d.ld = w.lds; d.stride = w.square;
            d.c_hi = at(w.a);
            d.d_hi = at(step == kGram ? w.a : w.b);
            if (step == kGram && w.splits > 1) {
                d.partial = reinterpret_cast<float*>(base + w.partial);
                d.partial_stride = batch * w.square;
            }
        }
        return d;
    };
    // X stands in two places in turn
    StepParams gram_step[2]{}, square_step{}, apply_step[2]{};
    if (const int rc = (f32 ? prepare_step<kSquare, true> : prepare_step<kSquare, false>)(square_step, side, side, side, gram, false, gram, false, 1)) return rc;
    for (int i = 0; i < 2; ++i) {
        const Matrices& now = i ? second : first;
        if (const int rc = prepare_step<kGram>(gram_step[i], side, side, longer, now, tall, now, tall, w.splits)) return rc;
        // wide: B X, X read along its rows; tall: X B, B being its own transpose
        if (const int rc = tall ? (f32 ? prepare_step<kApplyTall, true> : prepare_step<kApplyTall, false>)(apply_step[i], rows, cols, side, now, false, poly, false, 1)
                                : (f32 ? prepare_step<kApplyWide, true> : prepare_step<kApplyWide, false>)(apply_step[i], rows, cols, side, poly, false, now, true, 1))
            return rc;
    }

    g_orthogonal_waits.store(true);
    if (rows * (int64_t)src.groups <= kHeldGroups) {
        if (const int rc = launch_dense(orthogonal_held_kernel, dim3((unsigned)(kHeldCtas * batch)), kHeldThreads, kHeldCtas, true, 0, s, src)) return rc;
    } else {
        const dim3 grid((unsigned)w.parts, (unsigned)batch);
        if (const int rc = launch_dense(orthogonal_norm_kernel, grid, kSourceThreads, 1, true, 0, s, src)) return rc;
        if (const int rc = launch_dense(orthogonal_source_kernel, grid, kSourceThreads, 1, true, 0, s, src)) return rc;
    }
    for (int i = 0; i < steps; ++i) {
        StepParams &g = gram_step[i & 1], &a = apply_step[i & 1];
        g.e = ending(kGram, i);
        if (const int rc = launch_step<kGram>(g, s)) return rc;
        if (w.splits > 1) {
            JoinParams j{};
            j.partial = g.e.partial; j.partial_stride = g.e.partial_stride; j.square = w.square;
            j.splits = w.splits; j.side = (int32_t)side; j.lds = (int32_t)w.lds;
            j.d = at(w.a);
            if (const int rc = launch_dense(w.splits > 64 ? orthogonal_join_kernel<true> : orthogonal_join_kernel<false>, dim3((unsigned)((side * w.lds / 8 + 255) / 256), (unsigned)batch), 256, 1, true, 0, s, j)) return rc;
        }
        square_step.e = ending(kSquare, i);
        if (const int rc = (f32 ? launch_step<kSquare, true> : launch_step<kSquare, false>)(square_step, s)) return rc;
        a.e = ending(tall ? kApplyTall : kApplyWide, i);
        if (i + 1 == steps) {
            a.e.y = y; a.e.ldy = ldy; a.e.y_stride = batch > 1 ? y_stride : 0;
            a.e.y_vec = rows_aligned16(y, ldy, 2) && (batch == 1 || y_stride % 8 == 0);
        }
        if (const int rc = tall ? (f32 ? launch_step<kApplyTall, true> : launch_step<kApplyTall, false>)(a, s)
                                : (f32 ? launch_step<kApplyWide, true> : launch_step<kApplyWide, false>)(a, s))
            return rc;
    }
    return ZERO_OK;
}
