// Layer norm with the residual's addition, and its gradient with the reduction of
// the gain's and the shift's gradients over all rows, sm_103a.
//
// Forward:  h = x + residual, rounded to its type and kept;  y = (h - mean) rstd gamma + beta
// Backward: g = dy gamma, xhat = (x - mean) rstd,
//           dx = residual + rstd (g - mean(g) - xhat mean(g xhat)),
//           dgamma = acc + sum over rows of dy xhat,  dbeta = acc + sum over rows of dy
//
// A row belongs to a team: some lanes of a warp (up to 512 columns) or a CTA (up to
// 16384), whose threads hold the same columns of every row they see, so that gamma,
// beta and the sums of the weights' gradients stay in registers.  The statistics come
// from the values that a thread holds: the mean first, then the deviations from it with
// their sum, which corrects both, so that neither a large mean nor the order of the
// sum costs digits.  Everything is fp32.
#include <cmath>

#include "zero_dense.cuh"

namespace zgb {

struct NormParams {
    int64_t rows;
    int32_t cols, lanes, take;             // lanes of a warp's team; rows that a team takes at a time
    int64_t ldx, ldr, lds, ldy;
    const void* x;
    const void* residual;                  // forward: joins x; backward: joins dx; or null
    void* sum;
    void* y;                               // or dx
    const void* dy; int64_t lddy;
    const uint16_t* gamma;
    const uint16_t* beta;
    float* mean;
    float* rstd;
    float* part;                           // [2][parts][cols]: the teams' sums of dy xhat and dy, or null
    float eps;
    bool y_f32, weights_vec;
};

// ---- a thread's eight columns (a piece), of which it has kPer ----------------------
// kVec: rows on 16-byte boundaries of whole pieces, columns 8 (t + team j) .. + 7.
// Otherwise column t + team (8 j + k), so that the team's accesses fall together.
struct Team {
    int t, size;
};
template <bool kVec>
__device__ __forceinline__ int column(const Team& m, int j, int k) {
    return kVec ? 8 * (m.t + m.size * j) + k : m.t + m.size * (8 * j + k);
}
__device__ __forceinline__ float one(const float* p) { return __ldcs(p); }
__device__ __forceinline__ float one(const uint16_t* p) { return bf16_one(__ldcs(p)); }

template <bool kF32, bool kVec>
struct Piece {
    uint4 u[kVec ? (kF32 ? 2 : 1) : 2];    // not kVec: eight fp32 values
    __device__ __forceinline__ void load(const void* row, const Team& m, int j, int cols) {
        using T = typename std::conditional<kF32, float, uint16_t>::type;
        const T* q = static_cast<const T*>(row);
        if constexpr (kVec) {
            const int c = column<true>(m, j, 0);
            u[0] = make_uint4(0u, 0u, 0u, 0u);
            if constexpr (kF32) u[1] = u[0];
            if (c < cols) {
                u[0] = ld_live_u4(q + c);
                if constexpr (kF32) u[1] = ld_live_u4(q + c + 4);
            }
        } else {
            float v[8];
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                const int c = column<false>(m, j, k);
                v[k] = c < cols ? one(q + c) : 0.0f;
            }
            u[0] = make_uint4(__float_as_uint(v[0]), __float_as_uint(v[1]), __float_as_uint(v[2]), __float_as_uint(v[3]));
            u[1] = make_uint4(__float_as_uint(v[4]), __float_as_uint(v[5]), __float_as_uint(v[6]), __float_as_uint(v[7]));
        }
    }
    __device__ __forceinline__ void get(float (&v)[8]) const { raw8<!kVec || kF32>(u, v); }
};

template <bool kVec>
__device__ __forceinline__ void store_piece(void* row, bool f32, const Team& m, int j, int cols, const float (&v)[8]) {
    if constexpr (kVec) {
        const int c = column<true>(m, j, 0);
        if (c < cols) store8(static_cast<char*>(row) + (int64_t)c * (f32 ? 4 : 2), f32, v);
    } else {
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            const int c = column<false>(m, j, k);
            if (c >= cols) continue;
            if (f32)
                static_cast<float*>(row)[c] = v[k];
            else
                static_cast<uint16_t*>(row)[c] = to_bf16(v[k]);
        }
    }
}

// A piece of gamma or beta as bf16 pairs; `fill` (a pair) where the vector is absent.
template <bool kVec>
__device__ __forceinline__ uint4 weight_piece(const uint16_t* w, bool vec, const Team& m, int j, int cols, uint32_t fill) {
    if (!w) return make_uint4(fill, fill, fill, fill);
    if (kVec && vec) return column<true>(m, j, 0) < cols ? *reinterpret_cast<const uint4*>(w + column<true>(m, j, 0)) : make_uint4(0u, 0u, 0u, 0u);
    uint32_t p[8];
#pragma unroll
    for (int k = 0; k < 8; ++k) p[k] = column<kVec>(m, j, k) < cols ? w[column<kVec>(m, j, k)] : 0u;
    return make_uint4(p[0] | p[1] << 16, p[2] | p[3] << 16, p[4] | p[5] << 16, p[6] | p[7] << 16);
}
constexpr uint32_t kOnes = 0x3f803f80u;

// ---- sums over a team ---------------------------------------------------------------
// kCount values of every thread of a warp, a power of two: halves are exchanged while
// there are several, so that 8 values take 9 shuffles; lane l ends with value
// l / (32 / kCount).
template <int kCount>
__device__ __forceinline__ float warp_sums(float (&v)[kCount]) {
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int n = kCount / 2, o = 16; o; n /= 2, o /= 2) {
        if (n) {
#pragma unroll
            for (int i = 0; i < n; ++i) {
                const float give = lane & o ? v[i] : v[i + n], keep = lane & o ? v[i + n] : v[i];
                v[i] = keep + __shfl_xor_sync(0xffffffffu, give, o);
            }
        } else {
            v[0] += __shfl_xor_sync(0xffffffffu, v[0], o);
        }
    }
    return v[0];
}

constexpr int kMostWarps = 16, kMostValues = 8;
struct TeamSums {   // shared memory of a CTA that is one team
    float part[2][kMostWarps][kMostValues];
};

// Sums v over the team in a fixed order; every thread gets them.  kCta: one barrier,
// two buffers in turn (a buffer is written again two sums later, after a barrier that
// follows its last read).
template <bool kCta, int kCount>
__device__ __forceinline__ void team_sums(float (&v)[kCount], TeamSums& s, int& turn, int lanes) {
    if constexpr (kCta) {
        const float mine = warp_sums<kCount>(v);
        const int lane = threadIdx.x & 31, warp = threadIdx.x / 32, warps = blockDim.x / 32;
        if (lane % (32 / kCount) == 0) s.part[turn][warp][lane / (32 / kCount)] = mine;
        __syncthreads();
#pragma unroll
        for (int i = 0; i < kCount; ++i) v[i] = 0.0f;
        for (int w = 0; w < warps; ++w)
#pragma unroll
            for (int i = 0; i < kCount; ++i) v[i] += s.part[turn][w][i];
        turn ^= 1;
    } else {
        for (int o = lanes / 2; o; o /= 2)
#pragma unroll
            for (int i = 0; i < kCount; ++i) v[i] += __shfl_xor_sync(0xffffffffu, v[i], o);
    }
}

// Rows that a team has in hand at a time.
template <bool kCta, int kPer>
constexpr int kRowsOf = kCta ? 4 / kPer : 2;

template <bool kCta>
__device__ __forceinline__ Team team_of(const NormParams& p, int64_t* index, int64_t* teams) {
    if (kCta) {
        *index = blockIdx.x;
        *teams = gridDim.x;
        return Team{(int)threadIdx.x, (int)blockDim.x};
    }
    const int per = blockDim.x / p.lanes;
    *index = (int64_t)blockIdx.x * per + threadIdx.x / p.lanes;
    *teams = (int64_t)gridDim.x * per;
    return Team{(int)threadIdx.x % p.lanes, p.lanes};
}

// ---- forward ------------------------------------------------------------------------
template <bool kF32, bool kVec, int kPer, bool kCta>
__global__ void __launch_bounds__(kCta ? 512 : 256) norm_kernel(const NormParams p) {
    __shared__ TeamSums sums;
    constexpr int kRows = kRowsOf<kCta, kPer>, kSize = kF32 ? 4 : 2;
    await_predecessor();
    int64_t index, teams;
    const Team m = team_of<kCta>(p, &index, &teams);
    uint4 gamma[kPer], beta[kPer];
#pragma unroll
    for (int j = 0; j < kPer; ++j) {
        gamma[j] = weight_piece<kVec>(p.gamma, p.weights_vec, m, j, p.cols, kOnes);
        beta[j] = weight_piece<kVec>(p.beta, p.weights_vec, m, j, p.cols, 0u);
    }
    const float share = 1.0f / (float)p.cols;
    int turn = 0;
    // teams of one warp shuffle together: all go on until the last has no row
    const int64_t first = kCta ? index : index - threadIdx.x % 32 / p.lanes;
    for (int64_t at = first * p.take; at < p.rows; at += teams * p.take) {
        const int64_t row0 = at + (index - first) * p.take;
        Piece<kF32, kVec> x[kRows][kPer], r[kRows][kPer];
        const auto has = [&](int i) { return i < p.take && row0 + i < p.rows; };
#pragma unroll
        for (int i = 0; i < kRows; ++i)
#pragma unroll
            for (int j = 0; j < kPer; ++j) {
                const int cols = has(i) ? p.cols : 0;
                x[i][j].load(static_cast<const char*>(p.x) + (row0 + i) * p.ldx * kSize, m, j, cols);
                if (p.residual) r[i][j].load(static_cast<const char*>(p.residual) + (row0 + i) * p.ldr * kSize, m, j, cols);
            }
        float h[kRows][kPer][8], mean[kRows];
#pragma unroll
        for (int i = 0; i < kRows; ++i) {
            mean[i] = 0.0f;
#pragma unroll
            for (int j = 0; j < kPer; ++j) {
                x[i][j].get(h[i][j]);
                if (p.residual) {
                    float t[8];
                    r[i][j].get(t);
#pragma unroll
                    for (int k = 0; k < 8; ++k) {
                        h[i][j][k] += t[k];
                        if (!kF32) h[i][j][k] = bf16_one(to_bf16(h[i][j][k]));   // as kept, and as the gradient will read it
                    }
                    if (has(i)) store_piece<kVec>(static_cast<char*>(p.sum) + (row0 + i) * p.lds * kSize, kF32, m, j, p.cols, h[i][j]);
                }
#pragma unroll
                for (int k = 0; k < 8; ++k) mean[i] += h[i][j][k];
            }
        }
        team_sums<kCta, kRows>(mean, sums, turn, p.lanes);
        float v[2 * kRows];
#pragma unroll
        for (int i = 0; i < kRows; ++i) {
            mean[i] *= share;
            float d1 = 0.0f, d2 = 0.0f;
#pragma unroll
            for (int j = 0; j < kPer; ++j)
#pragma unroll
                for (int k = 0; k < 8; ++k) {
                    const float d = column<kVec>(m, j, k) < p.cols ? h[i][j][k] - mean[i] : 0.0f;
                    h[i][j][k] = d;
                    d1 += d;
                    d2 += d * d;
                }
            v[2 * i] = d1;
            v[2 * i + 1] = d2;
        }
        team_sums<kCta, 2 * kRows>(v, sums, turn, p.lanes);
#pragma unroll
        for (int i = 0; i < kRows; ++i) {
            const float off = v[2 * i] * share;
            const float rstd = 1.0f / sqrtf(v[2 * i + 1] * share - off * off + p.eps);
            if (!has(i)) continue;
            if (m.t == 0) {
                if (p.mean) p.mean[row0 + i] = mean[i] + off;
                if (p.rstd) p.rstd[row0 + i] = rstd;
            }
#pragma unroll
            for (int j = 0; j < kPer; ++j) {
                float a[8], b[8];
                unpack8(gamma[j], a);
                unpack8(beta[j], b);
#pragma unroll
                for (int k = 0; k < 8; ++k) a[k] = (h[i][j][k] - off) * rstd * a[k] + b[k];
                store_piece<kVec>(static_cast<char*>(p.y) + (row0 + i) * p.ldy * (p.y_f32 ? 4 : 2), p.y_f32, m, j, p.cols, a);
            }
        }
    }
}

// ---- backward -----------------------------------------------------------------------
// Sums of dy xhat and dy by column: in registers, or (kPer 4, which has too few) in
// shared memory, each thread its own places.
template <int kPer>
struct WeightSums {
    static constexpr bool kShared = kPer > 2;
    float g[kShared ? 1 : kPer][8], b[kShared ? 1 : kPer][8];
    float4* at;
    __device__ __forceinline__ void clear(float4* mine) {
        at = mine;
        if constexpr (kShared) {
#pragma unroll
            for (int i = 0; i < 4 * kPer; ++i) at[i * blockDim.x] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        } else {
#pragma unroll
            for (int j = 0; j < kPer; ++j)
#pragma unroll
                for (int k = 0; k < 8; ++k) g[j][k] = b[j][k] = 0.0f;
        }
    }
    __device__ __forceinline__ void add(int j, const float (&dg)[8], const float (&db)[8]) {
        if constexpr (kShared) {
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                const float* s = q < 2 ? dg + 4 * q : db + 4 * (q - 2);
                float4 t = at[(4 * j + q) * blockDim.x];
                t.x += s[0]; t.y += s[1]; t.z += s[2]; t.w += s[3];
                at[(4 * j + q) * blockDim.x] = t;
            }
        } else {
#pragma unroll
            for (int k = 0; k < 8; ++k) g[j][k] += dg[k], b[j][k] += db[k];
        }
    }
    __device__ __forceinline__ void get(int j, float (&dg)[8], float (&db)[8]) const {
        if constexpr (kShared) {
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                const float4 t = at[(4 * j + q) * blockDim.x];
                float* s = q < 2 ? dg + 4 * q : db + 4 * (q - 2);
                s[0] = t.x; s[1] = t.y; s[2] = t.z; s[3] = t.w;
            }
        } else {
#pragma unroll
            for (int k = 0; k < 8; ++k) dg[k] = g[j][k], db[k] = b[j][k];
        }
    }
};

template <bool kF32, bool kDyF32, bool kVec, int kPer, bool kCta>
__global__ void __launch_bounds__(kCta ? 512 : 256) norm_grad_kernel(const NormParams p) {
    extern __shared__ float4 shared_sums[];
    __shared__ TeamSums sums;
    constexpr int kRows = kRowsOf<kCta, kPer>, kSize = kF32 ? 4 : 2, kDySize = kDyF32 ? 4 : 2;
    await_predecessor();
    int64_t index, teams;
    const Team m = team_of<kCta>(p, &index, &teams);
    uint4 gamma[kPer];
#pragma unroll
    for (int j = 0; j < kPer; ++j) gamma[j] = weight_piece<kVec>(p.gamma, p.weights_vec, m, j, p.cols, kOnes);
    WeightSums<kPer> acc;
    acc.clear(shared_sums + threadIdx.x);
    const float share = 1.0f / (float)p.cols;
    int turn = 0;
    const int64_t first = kCta ? index : index - threadIdx.x % 32 / p.lanes;
    for (int64_t at = first * p.take; at < p.rows; at += teams * p.take) {
        const int64_t row0 = at + (index - first) * p.take;
        Piece<kF32, kVec> x[kRows][kPer];
        Piece<kDyF32, kVec> dy[kRows][kPer];
        float mean[kRows], rstd[kRows];
        const auto has = [&](int i) { return i < p.take && row0 + i < p.rows; };
#pragma unroll
        for (int i = 0; i < kRows; ++i) {
            mean[i] = has(i) ? p.mean[row0 + i] : 0.0f;
            rstd[i] = has(i) ? p.rstd[row0 + i] : 0.0f;
#pragma unroll
            for (int j = 0; j < kPer; ++j) {
                const int cols = has(i) ? p.cols : 0;
                x[i][j].load(static_cast<const char*>(p.x) + (row0 + i) * p.ldx * kSize, m, j, cols);
                dy[i][j].load(static_cast<const char*>(p.dy) + (row0 + i) * p.lddy * kDySize, m, j, cols);
            }
        }
        float v[2 * kRows];
#pragma unroll
        for (int i = 0; i < kRows; ++i) {
            float s1 = 0.0f, s2 = 0.0f;
#pragma unroll
            for (int j = 0; j < kPer; ++j) {
                float a[8], d[8], w[8];
                x[i][j].get(a);
                dy[i][j].get(d);
                unpack8(gamma[j], w);
#pragma unroll
                for (int k = 0; k < 8; ++k) {   // an absent column has dy = 0 and a finite xhat
                    const float g = d[k] * w[k];
                    s1 += g;
                    s2 += g * ((a[k] - mean[i]) * rstd[i]);
                }
            }
            v[2 * i] = s1;
            v[2 * i + 1] = s2;
        }
        team_sums<kCta, 2 * kRows>(v, sums, turn, p.lanes);
#pragma unroll
        for (int i = 0; i < kRows; ++i) {
            if (!has(i)) continue;
            const float m1 = v[2 * i] * share, m2 = v[2 * i + 1] * share;
#pragma unroll
            for (int j = 0; j < kPer; ++j) {
                float a[8], d[8], w[8];
                x[i][j].get(a);
                dy[i][j].get(d);
                unpack8(gamma[j], w);
                float out[8], dg[8];
#pragma unroll
                for (int k = 0; k < 8; ++k) {
                    const float xhat = (a[k] - mean[i]) * rstd[i];
                    out[k] = rstd[i] * (d[k] * w[k] - m1 - xhat * m2);
                    dg[k] = d[k] * xhat;
                }
                if (p.part) acc.add(j, dg, d);
                if (p.residual) {
                    Piece<kF32, kVec> r;
                    r.load(static_cast<const char*>(p.residual) + (row0 + i) * p.ldr * kSize, m, j, p.cols);
                    r.get(a);
#pragma unroll
                    for (int k = 0; k < 8; ++k) out[k] += a[k];
                }
                store_piece<kVec>(static_cast<char*>(p.y) + (row0 + i) * p.ldy * kSize, kF32, m, j, p.cols, out);
            }
        }
    }
    if (!p.part) return;
    float* part = p.part + (int64_t)blockIdx.x * p.cols;
    const int64_t half = (int64_t)gridDim.x * p.cols;
    if constexpr (kCta) {
#pragma unroll
        for (int j = 0; j < kPer; ++j) {
            float dg[8], db[8];
            acc.get(j, dg, db);
            if constexpr (kVec) {
                if (column<true>(m, j, 0) < p.cols) {
                    store8(part + column<true>(m, j, 0), true, dg);
                    store8(part + half + column<true>(m, j, 0), true, db);
                }
            } else {
#pragma unroll
                for (int k = 0; k < 8; ++k)
                    if (column<false>(m, j, k) < p.cols) {
                        part[column<false>(m, j, k)] = dg[k];
                        part[half + column<false>(m, j, k)] = db[k];
                    }
            }
        }
    } else {
        // the CTA's teams in order; a team of l lanes has 8 kPer l columns, so that
        // the teams' sums fill 8 kPer floats a thread
        float* all = reinterpret_cast<float*>(shared_sums);
        const int width = 8 * kPer * p.lanes, n = blockDim.x / p.lanes;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            __syncthreads();
#pragma unroll
            for (int j = 0; j < kPer; ++j) {
                float dg[8], db[8];
                acc.get(j, dg, db);
#pragma unroll
                for (int k = 0; k < 8; ++k) all[(int)threadIdx.x / p.lanes * width + column<kVec>(m, j, k)] = h ? db[k] : dg[k];
            }
            __syncthreads();
            for (int c = threadIdx.x; c < p.cols; c += blockDim.x) {
                float s = 0.0f;
                for (int i = 0; i < n; ++i) s += all[i * width + c];
                part[h * half + c] = s;
            }
        }
    }
}

// ---- rows of more than 16384 columns ---------------------------------------------------
// A CTA a row, in three passes (two backward) over it, the later ones out of L2.
constexpr int kWideThreads = 512;

template <bool kF32>
__device__ __forceinline__ float value(const void* p, int64_t i) {
    if constexpr (kF32)
        return static_cast<const float*>(p)[i];
    else
        return bf16_one(static_cast<const uint16_t*>(p)[i]);
}
__device__ __forceinline__ void put(void* p, bool f32, int64_t i, float v) {
    if (f32)
        static_cast<float*>(p)[i] = v;
    else
        static_cast<uint16_t*>(p)[i] = to_bf16(v);
}

template <bool kF32>
__global__ void __launch_bounds__(kWideThreads) norm_wide_kernel(const NormParams p) {
    __shared__ TeamSums sums;
    await_predecessor();
    const float share = 1.0f / (float)p.cols;
    int turn = 0;
    for (int64_t row = blockIdx.x; row < p.rows; row += gridDim.x) {
        float m[1] = {0.0f};
        for (int c = threadIdx.x; c < p.cols; c += kWideThreads) {
            float h = value<kF32>(p.x, row * p.ldx + c);
            if (p.residual) {
                h += value<kF32>(p.residual, row * p.ldr + c);
                put(p.sum, kF32, row * p.lds + c, h);
                if (!kF32) h = bf16_one(to_bf16(h));
            }
            m[0] += h;
        }
        team_sums<true, 1>(m, sums, turn, 0);
        const float mean = m[0] * share;
        const void* from = p.residual ? p.sum : p.x;   // a thread's own writes
        const int64_t ld = p.residual ? p.lds : p.ldx;
        float v[2] = {0.0f, 0.0f};
        for (int c = threadIdx.x; c < p.cols; c += kWideThreads) {
            const float d = value<kF32>(from, row * ld + c) - mean;
            v[0] += d;
            v[1] += d * d;
        }
        team_sums<true, 2>(v, sums, turn, 0);
        const float off = v[0] * share, rstd = 1.0f / sqrtf(v[1] * share - off * off + p.eps);
        if (threadIdx.x == 0) {
            if (p.mean) p.mean[row] = mean + off;
            if (p.rstd) p.rstd[row] = rstd;
        }
        for (int c = threadIdx.x; c < p.cols; c += kWideThreads) {
            float y = (value<kF32>(from, row * ld + c) - mean - off) * rstd;
            y = y * (p.gamma ? bf16_one(p.gamma[c]) : 1.0f) + (p.beta ? bf16_one(p.beta[c]) : 0.0f);
            put(p.y, p.y_f32, row * p.ldy + c, y);
        }
    }
}

template <bool kF32, bool kDyF32>
__global__ void __launch_bounds__(kWideThreads) norm_grad_wide_kernel(const NormParams p) {
    __shared__ TeamSums sums;
    await_predecessor();
    const float share = 1.0f / (float)p.cols;
    int turn = 0;
    for (int64_t row = blockIdx.x; row < p.rows; row += gridDim.x) {
        const float mean = p.mean[row], rstd = p.rstd[row];
        float v[2] = {0.0f, 0.0f};
        for (int c = threadIdx.x; c < p.cols; c += kWideThreads) {
            const float g = value<kDyF32>(p.dy, row * p.lddy + c) * (p.gamma ? bf16_one(p.gamma[c]) : 1.0f);
            v[0] += g;
            v[1] += g * ((value<kF32>(p.x, row * p.ldx + c) - mean) * rstd);
        }
        team_sums<true, 2>(v, sums, turn, 0);
        const float m1 = v[0] * share, m2 = v[1] * share;
        for (int c = threadIdx.x; c < p.cols; c += kWideThreads) {
            const float g = value<kDyF32>(p.dy, row * p.lddy + c) * (p.gamma ? bf16_one(p.gamma[c]) : 1.0f);
            const float xhat = (value<kF32>(p.x, row * p.ldx + c) - mean) * rstd;
            float d = rstd * (g - m1 - xhat * m2);
            if (p.residual) d += value<kF32>(p.residual, row * p.ldr + c);
            put(p.y, kF32, row * p.ldy + c, d);
        }
    }
}

// Their weights' gradients: a thread a column, CTA (x, y) the rows of share y.
template <bool kF32, bool kDyF32>
__global__ void __launch_bounds__(256) norm_columns_kernel(const NormParams p) {
    await_predecessor();
    const int c = blockIdx.x * 256 + threadIdx.x;
    if (c >= p.cols) return;
    float dg = 0.0f, db = 0.0f;
    for (int64_t row = blockIdx.y; row < p.rows; row += gridDim.y) {
        const float d = value<kDyF32>(p.dy, row * p.lddy + c);
        dg += d * ((value<kF32>(p.x, row * p.ldx + c) - p.mean[row]) * p.rstd[row]);
        db += d;
    }
    p.part[(int64_t)blockIdx.y * p.cols + c] = dg;
    p.part[((int64_t)gridDim.y + blockIdx.y) * p.cols + c] = db;
}

// ---- the weights' gradients out of the parts ---------------------------------------------
// 32 columns a CTA, 16 warps that each add a share of the parts in order, then the 16.
constexpr int kFinishWarps = 16;
struct FinishParams {
    const float* part;
    int32_t parts, cols;
    const void* acc[2];
    void* out[2];
    bool f32;
};
__global__ void __launch_bounds__(32 * kFinishWarps) norm_finish_kernel(const FinishParams p) {
    __shared__ float s[kFinishWarps][32];
    await_predecessor();
    const int lane = threadIdx.x & 31, warp = threadIdx.x / 32, which = blockIdx.y;
    const int c = blockIdx.x * 32 + lane;
    float v = 0.0f;
    if (p.out[which]) {
        const float* q = p.part + (int64_t)which * p.parts * p.cols + c;
        if (c < p.cols)
#pragma unroll 8
            for (int i = warp; i < p.parts; i += kFinishWarps) v += q[(int64_t)i * p.cols];
        s[warp][lane] = v;
    }
    __syncthreads();
    if (warp || c >= p.cols || !p.out[which]) return;
    for (int w = 1; w < kFinishWarps; ++w) v += s[w][lane];
    if (p.f32) {
        if (p.acc[which]) v += static_cast<const float*>(p.acc[which])[c];
        static_cast<float*>(p.out[which])[c] = v;
    } else {
        if (p.acc[which]) v += bf16_one(static_cast<const uint16_t*>(p.acc[which])[c]);
        static_cast<uint16_t*>(p.out[which])[c] = to_bf16(v);
    }
}

// ---- launches ---------------------------------------------------------------------------
constexpr int kWidestNorm = 16384;

// How a matrix is shared out: lanes of a warp (32 at most) or a CTA of `threads` to a
// row, pieces a thread, rows at a time, CTAs.
struct NormShape {
    bool cta;
    int lanes, per, threads, take;
    int64_t grid;
};
static NormShape norm_shape(int64_t rows, int64_t cols) {
    NormShape s{};
    const int64_t groups = (cols + 7) / 8, sms = sm_count();
    s.cta = groups > 64;
    if (s.cta) {
        s.per = groups <= 512 ? 1 : groups <= 1024 ? 2 : 4;
        s.threads = (int)((groups + s.per * 32 - 1) / (s.per * 32) * 32);
        s.lanes = 32;
    } else {
        s.per = groups <= 32 ? 1 : 2;
        s.threads = 256;
        s.lanes = 1;
        while (s.lanes * s.per < groups) s.lanes *= 2;
    }
    // CTAs that are resident together, and no more rows at a time than give each a pass
    const int64_t resident = sms * (s.cta ? (s.threads <= 128 ? 4 : s.threads <= 256 ? 2 : 1) : 2);
    const int most = s.cta ? 4 / s.per : 2, teams = s.cta ? 1 : s.threads / s.lanes;
    int64_t take = (rows + resident * teams - 1) / (resident * teams);
    s.take = (int)(take < 1 ? 1 : take > most ? most : take);
    s.grid = (rows + (int64_t)s.take * teams - 1) / ((int64_t)s.take * teams);
    if (s.grid > resident) s.grid = resident;
    return s;
}
// Parts that the weights' gradients are summed in.
static int64_t norm_parts(int64_t rows, int64_t cols) {
    if (rows == 0 || cols == 0) return 0;
    if (cols > kWidestNorm) return rows < 64 ? rows : 64;
    return norm_shape(rows, cols).grid;
}

template <bool kF32, bool kVec>
static int launch_norm(const NormParams& p, const NormShape& s, cudaStream_t stream) {
    void (*kernel)(NormParams) = !s.cta ? (s.per == 1 ? norm_kernel<kF32, kVec, 1, false> : norm_kernel<kF32, kVec, 2, false>)
                                 : s.per == 1 ? norm_kernel<kF32, kVec, 1, true>
                                 : s.per == 2 ? norm_kernel<kF32, kVec, 2, true>
                                              : norm_kernel<kF32, kVec, 4, true>;
    return launch_dense(kernel, dim3((unsigned)s.grid), s.threads, 1, true, 0, stream, p);
}
template <bool kF32, bool kDyF32, bool kVec>
static int launch_norm_grad(const NormParams& p, const NormShape& s, cudaStream_t stream) {
    void (*kernel)(NormParams) = !s.cta ? (s.per == 1 ? norm_grad_kernel<kF32, kDyF32, kVec, 1, false> : norm_grad_kernel<kF32, kDyF32, kVec, 2, false>)
                                 : s.per == 1 ? norm_grad_kernel<kF32, kDyF32, kVec, 1, true>
                                 : s.per == 2 ? norm_grad_kernel<kF32, kDyF32, kVec, 2, true>
                                              : norm_grad_kernel<kF32, kDyF32, kVec, 4, true>;
    const int smem = s.cta ? (s.per > 2 ? s.per * 64 * s.threads : 0) : s.per * 32 * s.threads;
    if (smem > 48 * 1024) {
        const cudaError_t e = cudaFuncSetAttribute((const void*)kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
        if (e != cudaSuccess) {
            note_cuda_error(e);
            (void)cudaGetLastError();
            return ZERO_ECUDA;
        }
    }
    return launch_dense(kernel, dim3((unsigned)s.grid), s.threads, 1, true, smem, stream, p);
}

static bool dtype_ok(int32_t d) { return d == ZERO_BF16 || d == ZERO_F32; }

}  // namespace zgb

extern "C" int zero_layer_norm(int64_t rows, int64_t cols, const void* x, int64_t ldx, int32_t dtype, const void* residual,
                               int64_t ldr, void* sum, int64_t lds, const uint16_t* gamma, const uint16_t* beta, float eps,
                               void* y, int32_t y_dtype, int64_t ldy, float* mean, float* rstd, void* stream) {
    using namespace zgb;
    if (rows < 0 || cols < 0 || !dtype_ok(dtype) || !(y_dtype == ZERO_BF16 || y_dtype == dtype)) return ZERO_EINVAL;
    if (!(eps >= 0.0f) || !std::isfinite(eps) || (residual != nullptr) != (sum != nullptr)) return ZERO_EINVAL;
    if (cols > INT32_MAX / 2) return ZERO_ERANGE;
    if (const int rc = check_matrix(x, rows, cols, ldx, dtype)) return rc;
    if (const int rc = check_matrix(y, rows, cols, ldy, y_dtype)) return rc;
    if (residual) {
        if (const int rc = check_matrix(residual, rows, cols, ldr, dtype)) return rc;
        if (const int rc = check_matrix(sum, rows, cols, lds, dtype)) return rc;
    }
    if (check_aligned(gamma, 2) || check_aligned(beta, 2) || check_aligned(mean, 4) || check_aligned(rstd, 4)) return ZERO_EALIGN;
    if (rows == 0 || cols == 0) return ZERO_OK;
    if (check_device_ptr(x) || check_device_ptr(y) || (residual && (check_device_ptr(residual) || check_device_ptr(sum))) ||
        (gamma && check_device_ptr(gamma)) || (beta && check_device_ptr(beta)) || (mean && check_device_ptr(mean)) ||
        (rstd && check_device_ptr(rstd)))
        return ZERO_EINVAL;
    const int size = dtype_size(dtype);
    NormParams p{};
    p.rows = rows; p.cols = (int32_t)cols;
    p.x = x; p.ldx = ldx; p.residual = residual; p.ldr = ldr; p.sum = sum; p.lds = lds; p.y = y; p.ldy = ldy;
    p.gamma = gamma; p.beta = beta; p.mean = mean; p.rstd = rstd;
    p.eps = eps;
    p.y_f32 = y_dtype == ZERO_F32;
    p.weights_vec = aligned16(gamma) && aligned16(beta);
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (cols > kWidestNorm) {
        const int64_t most = 4 * (int64_t)sm_count();
        return launch_dense(dtype == ZERO_F32 ? norm_wide_kernel<true> : norm_wide_kernel<false>, dim3((unsigned)(rows < most ? rows : most)),
                            kWideThreads, 1, true, 0, s, p);
    }
    const bool vec = cols % 8 == 0 && rows_aligned16(x, ldx, size) && rows_aligned16(y, ldy, dtype_size(y_dtype)) &&
                     (!residual || (rows_aligned16(residual, ldr, size) && rows_aligned16(sum, lds, size)));
    const NormShape shape = norm_shape(rows, cols);
    p.lanes = shape.lanes; p.take = shape.take;
    if (dtype == ZERO_F32) return vec ? launch_norm<true, true>(p, shape, s) : launch_norm<true, false>(p, shape, s);
    return vec ? launch_norm<false, true>(p, shape, s) : launch_norm<false, false>(p, shape, s);
}

extern "C" int zero_layer_norm_grad_workspace(int64_t rows, int64_t cols, int64_t* bytes) {
    using namespace zgb;
    if (rows < 0 || cols < 0 || !bytes) return ZERO_EINVAL;
    if (cols > INT32_MAX / 2) return ZERO_ERANGE;
    *bytes = norm_parts(rows, cols) * cols * 2 * (int64_t)sizeof(float);
    return ZERO_OK;
}

extern "C" int zero_layer_norm_grad(int64_t rows, int64_t cols, const void* dy, int64_t lddy, int32_t dy_dtype, const void* x,
                                    int64_t ldx, const float* mean, const float* rstd, const uint16_t* gamma,
                                    const void* residual, int64_t ldr, void* dx, int32_t dtype, int64_t lddx,
                                    const void* dgamma_acc, void* dgamma, const void* dbeta_acc, void* dbeta,
                                    int32_t weight_dtype, void* workspace, int64_t workspace_bytes, void* stream) {
    using namespace zgb;
    if (rows < 0 || cols < 0 || !dtype_ok(dtype) || !(dy_dtype == ZERO_BF16 || dy_dtype == dtype)) return ZERO_EINVAL;
    const bool weights = dgamma || dbeta;
    if ((weights && !dtype_ok(weight_dtype)) || (!dgamma && dgamma_acc) || (!dbeta && dbeta_acc)) return ZERO_EINVAL;
    if (cols > INT32_MAX / 2) return ZERO_ERANGE;
    if (const int rc = check_matrix(dy, rows, cols, lddy, dy_dtype)) return rc;
    if (const int rc = check_matrix(x, rows, cols, ldx, dtype)) return rc;
    if (const int rc = check_matrix(dx, rows, cols, lddx, dtype)) return rc;
    if (residual)
        if (const int rc = check_matrix(residual, rows, cols, ldr, dtype)) return rc;
    if (rows && cols && (!mean || !rstd)) return ZERO_EINVAL;
    if (check_aligned(mean, 4) || check_aligned(rstd, 4) || check_aligned(gamma, 2)) return ZERO_EALIGN;
    if (weights) {
        const int size = dtype_size(weight_dtype);
        if (check_aligned(dgamma, size) || check_aligned(dgamma_acc, size) || check_aligned(dbeta, size) || check_aligned(dbeta_acc, size))
            return ZERO_EALIGN;
    }
    if (cols == 0 || (rows == 0 && !weights)) return ZERO_OK;
    const int64_t parts = weights ? norm_parts(rows, cols) : 0;
    if (parts) {
        if (!workspace) return ZERO_EINVAL;
        if (!aligned16(workspace)) return ZERO_EALIGN;
        if (workspace_bytes < parts * cols * 2 * (int64_t)sizeof(float)) return ZERO_ERANGE;
    }
    if ((rows && (check_device_ptr(dy) || check_device_ptr(x) || check_device_ptr(dx) || check_device_ptr(mean) || check_device_ptr(rstd) ||
                  (residual && check_device_ptr(residual)) || (gamma && check_device_ptr(gamma)))) ||
        (dgamma && check_device_ptr(dgamma)) || (dgamma_acc && check_device_ptr(dgamma_acc)) || (dbeta && check_device_ptr(dbeta)) ||
        (dbeta_acc && check_device_ptr(dbeta_acc)) || (parts && check_device_ptr(workspace)))
        return ZERO_EINVAL;
    const int size = dtype_size(dtype);
    NormParams p{};
    p.rows = rows; p.cols = (int32_t)cols;
    p.x = x; p.ldx = ldx; p.dy = dy; p.lddy = lddy; p.residual = residual; p.ldr = ldr; p.y = dx; p.ldy = lddx;
    p.gamma = gamma;
    p.mean = const_cast<float*>(mean); p.rstd = const_cast<float*>(rstd);
    p.part = parts ? static_cast<float*>(workspace) : nullptr;
    p.weights_vec = aligned16(gamma);
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    const bool f32 = dtype == ZERO_F32, dy_f32 = dy_dtype == ZERO_F32;
    int rc = ZERO_OK;
    if (rows == 0) {
        // the sums are empty
    } else if (cols > kWidestNorm) {
        const int64_t most = 4 * (int64_t)sm_count();
        rc = launch_dense(!f32 ? norm_grad_wide_kernel<false, false> : dy_f32 ? norm_grad_wide_kernel<true, true> : norm_grad_wide_kernel<true, false>,
                          dim3((unsigned)(rows < most ? rows : most)), kWideThreads, 1, true, 0, s, p);
        if (rc == ZERO_OK && parts)
            rc = launch_dense(!f32 ? norm_columns_kernel<false, false> : dy_f32 ? norm_columns_kernel<true, true> : norm_columns_kernel<true, false>,
                              dim3((unsigned)((cols + 255) / 256), (unsigned)parts), 256, 1, true, 0, s, p);
    } else {
        const bool vec = cols % 8 == 0 && rows_aligned16(x, ldx, size) && rows_aligned16(dy, lddy, dtype_size(dy_dtype)) &&
                         rows_aligned16(dx, lddx, size) && (!residual || rows_aligned16(residual, ldr, size));
        const NormShape shape = norm_shape(rows, cols);
        p.lanes = shape.lanes; p.take = shape.take;
        if (!f32)
            rc = vec ? launch_norm_grad<false, false, true>(p, shape, s) : launch_norm_grad<false, false, false>(p, shape, s);
        else if (dy_f32)
            rc = vec ? launch_norm_grad<true, true, true>(p, shape, s) : launch_norm_grad<true, true, false>(p, shape, s);
        else
            rc = vec ? launch_norm_grad<true, false, true>(p, shape, s) : launch_norm_grad<true, false, false>(p, shape, s);
    }
    if (rc != ZERO_OK || !weights) return rc;
    FinishParams q{};
    q.part = p.part; q.parts = (int32_t)parts; q.cols = (int32_t)cols;
    q.acc[0] = dgamma_acc; q.acc[1] = dbeta_acc;
    q.out[0] = dgamma; q.out[1] = dbeta;
    q.f32 = weight_dtype == ZERO_F32;
    return launch_dense(norm_finish_kernel, dim3((unsigned)((cols + 31) / 32), 2), 32 * kFinishWarps, 1, true, 0, s, q);
}
