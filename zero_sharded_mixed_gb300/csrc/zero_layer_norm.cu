// Layer norm with the residual's addition, and its gradient with the reduction of
// the gain's and the shift's gradients over all rows, sm_103a.
//
// Forward:  h = x + residual, rounded to its type and kept;  y = (h - mean) rstd gamma + beta
// Backward: g = dy gamma, xhat = (x - mean) rstd,
//           dx = residual + rstd (g - mean(g) - xhat mean(g xhat)),
//           dgamma = acc + sum over rows of dy xhat,  dbeta = acc + sum over rows of dy
//
// A row belongs to a team: some lanes of a warp, a warp, or up to 16 warps of a CTA
// (16384 columns), whose threads hold the same columns, up to 32, of every row they see,
// so that gamma, beta and the sums of the weights' gradients stay in registers.  Rows to
// come are copied to shared memory ahead of their turn.  Everything is fp32.
#include <atomic>
#include <cmath>
#include <type_traits>

#include "zero_tensor.cuh"
#include "zero_dense.cuh"

namespace zgb {

__device__ int g_norm_status;   // ZERO_OK, or ZERO_ETIMEOUT once a bounded wait gave up
static std::atomic<bool> g_norm_waits;   // whether a kernel with such waits was launched: a status check asks no others

int take_norm_status() {
    if (!g_norm_waits.load()) return ZERO_OK;
    int v = 0;
    if (cudaMemcpyFromSymbol(&v, g_norm_status, sizeof v) != cudaSuccess) {
        (void)cudaGetLastError();
        return ZERO_ECUDA;
    }
    if (v != ZERO_OK) {
        const int zero = ZERO_OK;
        if (cudaMemcpyToSymbol(g_norm_status, &zero, sizeof zero) != cudaSuccess) {
            (void)cudaGetLastError();
            return ZERO_ECUDA;
        }
    }
    return v == ZERO_OK ? ZERO_OK : ZERO_ETIMEOUT;
}

struct NormParams {
    int64_t rows;
    int32_t cols, lanes, warps;            // lanes of a team within a warp, or warps of a team
    int32_t ahead;                         // rows of a team that are on their way while one is worked on
    uint32_t slot, part_bytes, at[3];      // bytes: of a row's slot; of a thread (kVec) or a team in it; where its streams begin there
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
    float* part;                           // [2][parts][cols]: the CTAs' sums of dy xhat and dy, or null
    float eps;
    bool y_f32, weights_vec;
};

// ---- a thread's eight columns (a piece), of which it has up to kPer -----------------------
// Rows on 16-byte boundaries of whole pieces: bf16 columns 8 (t + team j) .. + 7, fp32 two
// quads, 4 (t + team 2 j) .. + 3 and 4 (t + team (2 j + 1)) .. + 3, so that either way a
// team's accesses of 16 bytes lie side by side (eight fp32 columns to a thread would fetch
// each sector of 32 bytes twice: 8192 x 1600 fp32 took 44 and 50 us, for 31 and 37).
// Otherwise (kLoose) column t + team (8 j + k), for the same reason.
enum Lay { kLoose, kEights, kQuads };
__host__ __device__ constexpr Lay lay_of(bool vec, bool f32) { return !vec ? kLoose : f32 ? kQuads : kEights; }
struct Team {
    int t, size, have;   // this thread, the threads, the pieces, quads or elements that this one has
};
template <Lay kLay>
__device__ __forceinline__ int column(const Team& m, int j, int k) {
    return kLay == kEights ? 8 * (m.t + m.size * j) + k : kLay == kQuads ? 4 * (m.t + m.size * (2 * j + k / 4)) + k % 4 : m.t + m.size * (8 * j + k);
}
template <Lay kLay>
__device__ __forceinline__ bool exists(const Team& m, int j, int k) {   // k 0: any of the piece
    return (kLay == kEights ? j : kLay == kQuads ? 2 * j + k / 4 : 8 * j + k) < m.have;
}

// Pairs of fp32 operations in one instruction: the kernels are bound by how many they issue
// (one at a time, 8192 x 1600 took 44 instructions an element and 27 us forward).
__device__ __forceinline__ float2 add2(float2 a, float2 b) { return __fadd2_rn(a, b); }
__device__ __forceinline__ float2 mul2(float2 a, float2 b) { return __fmul2_rn(a, b); }
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) { return __ffma2_rn(a, b, c); }
__device__ __forceinline__ float2 both(float a) { return make_float2(a, a); }

// Eight neighbours of a piece as they are stored: fp32 words or bf16 pairs.
template <bool kF32>
struct Words {
    uint32_t w[kF32 ? 8 : 4];
    __device__ __forceinline__ float2 pair(int k) const {
        if constexpr (kF32)
            return make_float2(__uint_as_float(w[2 * k]), __uint_as_float(w[2 * k + 1]));
        else
            return make_float2(bf16_lo(w[k]), bf16_hi(w[k]));
    }
    // Added, one rounding to the type.
    __device__ __forceinline__ void add(const Words& o) {
#pragma unroll
        for (int k = 0; k < (kF32 ? 8 : 4); ++k) {
            if constexpr (kF32)
                w[k] = __float_as_uint(__uint_as_float(w[k]) + __uint_as_float(o.w[k]));
            else
                asm("add.rn.bf16x2 %0, %0, %1;" : "+r"(w[k]) : "r"(o.w[k]));
        }
    }
};

constexpr int kMostWarps = 16;   // of a CTA, and of a team
constexpr int kMostAhead = 3;    // rows on their way

// A matrix's rows on their way through shared memory: asynchronous copies, some rows
// ahead of their turn, keep the memory busy behind the sums over the team.  A stream goes
// down a team's rows, `hop` elements from one to the next.
// kVec: every thread copies its own pieces to places of its own, so that nothing but its
// own copies have to be waited for; kAt counts the places, of 16 bytes, before this
// stream's.  The threads' places of one number lie side by side, kPitch from one number to
// the next: a warp's copies fill whole lines (a thread's places side by side, with an odd
// pitch for the banks' sake, took a third longer), and at offsets known to the compiler.
// Otherwise the team copies the row's 16-byte blocks as they lie, which hold up to 15
// bytes of the neighbours' on either side, from byte `at` of its slot, and reads elements
// from there; where a block would reach past the matrix's own memory its elements come
// one by one.
template <bool kF32, Lay kLay, int kPer, int kPitch, int kAt>
struct Stream {
    static constexpr int kSize = kF32 ? 4 : 2, kPlaces = kF32 ? 2 : 1;
    static constexpr bool kVec = kLay != kLoose;
    static_assert(!kF32 || kLay != kEights);
    using T = typename std::conditional<kF32, float, uint16_t>::type;
    const T* to_send;   // the next row to send: kVec this thread's first piece of it
    int64_t hop;
    uint32_t at, shift, turn;   // not kVec: where the row to read begins in its first block, and how that moves on
    uintptr_t begin, end;

    __device__ __forceinline__ Stream(const void* q, int64_t ld, uint32_t at, int64_t row, int64_t stride, int64_t rows, int cols, const Team& m)
        : hop(stride * ld), at(at) {
        const T* p = static_cast<const T*>(q);
        to_send = p + row * ld + column<kLay>(Team{kVec ? m.t : 0, 0, 0}, 0, 0);
        if constexpr (!kVec) {
            shift = (uint32_t)(reinterpret_cast<uintptr_t>(to_send) & 15);
            turn = (uint32_t)(hop * kSize) & 15;
            begin = reinterpret_cast<uintptr_t>(p);
            end = reinterpret_cast<uintptr_t>(p + (rows - 1) * ld + cols);
        }
    }
    // slot: kVec a shared address, this thread's; else the team's
    __device__ __forceinline__ void send(uint32_t slot, const Team& m, int cols) {
        if constexpr (kVec) {
#pragma unroll
            for (int j = 0; j < kPer; ++j) {
                if (!exists<kLay>(m, j, 0)) break;
                if constexpr (kLay == kEights) {
                    copy_block(slot + kPitch * (kAt + j), reinterpret_cast<uintptr_t>(to_send + 8 * m.size * j), true);
                } else {
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        if (!exists<kLay>(m, j, 4 * i)) break;
                        const uintptr_t from = reinterpret_cast<uintptr_t>(to_send + 4 * m.size * (2 * j + i));
                        if constexpr (kF32)
                            copy_block(slot + kPitch * (kAt + 2 * j + i), from, true);
                        else
                            copy_half_block(slot + kPitch * (kAt + j) + 8 * i, from);
                    }
                }
            }
        } else {
            const uintptr_t from = reinterpret_cast<uintptr_t>(to_send), first = from & ~(uintptr_t)15, last = from + cols * kSize;
            for (uintptr_t b = first + 16 * m.t; b < last; b += 16 * m.size) {
                const uint32_t to = slot + at + (uint32_t)(b - first);
                if (b >= begin && b + 16 <= end) {
                    copy_block(to, b, true);
                } else {
                    for (uintptr_t e = b; e < b + 16; e += kSize) {
                        if (e < from || e >= last) continue;
                        if constexpr (kF32)
                            asm volatile("st.shared.b32 [%0], %1;" ::"r"(to + (uint32_t)(e - b)), "r"(*reinterpret_cast<const uint32_t*>(e)) : "memory");
                        else
                            asm volatile("st.shared.b16 [%0], %1;" ::"r"(to + (uint32_t)(e - b)), "h"(*reinterpret_cast<const uint16_t*>(e)) : "memory");
                    }
                }
            }
        }
        to_send += hop;
    }
    // One thread: the row's blocks as they lie, in one copy, but those that reach past the
    // matrix's own memory, whose elements come one by one; the copy's bytes, then the copy.
    uintptr_t start, stop;
    __device__ __forceinline__ uint32_t send_edges(uint32_t slot, int cols) {
        const uintptr_t from = reinterpret_cast<uintptr_t>(to_send), first = from & ~(uintptr_t)15, last = from + cols * kSize;
        start = first >= begin ? first : first + 16;
        stop = (last + 15) & ~(uintptr_t)15;
        if (stop > end) stop -= 16;
        const auto put = [&](uintptr_t e) {
            const uint32_t to = slot + at + (uint32_t)(e - first);
            if constexpr (kF32)
                asm volatile("st.shared.b32 [%0], %1;" ::"r"(to), "r"(*reinterpret_cast<const uint32_t*>(e)) : "memory");
            else
                asm volatile("st.shared.b16 [%0], %1;" ::"r"(to), "h"(*reinterpret_cast<const uint16_t*>(e)) : "memory");
        };
        for (uintptr_t e = from; e < start; e += kSize) put(e);
        for (uintptr_t e = stop; e < last; e += kSize) put(e);
        return (uint32_t)(stop - start);
    }
    __device__ __forceinline__ void send_whole(uint8_t* slot, uint64_t* bar) {
        const uintptr_t first = reinterpret_cast<uintptr_t>(to_send) & ~(uintptr_t)15;
        bulk_g2s(slot + at + (start - first), reinterpret_cast<const void*>(start), (uint32_t)(stop - start), bar);
        to_send += hop;
    }
    __device__ __forceinline__ void next_row() {   // to read
        if (!kVec) shift = (shift + turn) & 15;
    }
    __device__ __forceinline__ Words<kF32> get(const uint8_t* slot, const Team& m, int j) const {
        Words<kF32> v;
        if constexpr (kVec) {
#pragma unroll
            for (int i = 0; i < kPlaces; ++i) {
                uint4 u = make_uint4(0u, 0u, 0u, 0u);
                if (kLay == kEights || i == 0 || exists<kLay>(m, j, 4)) u = *reinterpret_cast<const uint4*>(slot + kPitch * (kAt + j * kPlaces + i));
                if (kLay == kQuads && !kF32 && !exists<kLay>(m, j, 4)) u.z = u.w = 0u;
                v.w[4 * i] = u.x; v.w[4 * i + 1] = u.y; v.w[4 * i + 2] = u.z; v.w[4 * i + 3] = u.w;
            }
        } else {
            const T* q = reinterpret_cast<const T*>(slot + at + shift) + column<kLoose>(m, j, 0);
            uint32_t e[8];
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                if constexpr (kF32)
                    e[k] = exists<kLoose>(m, j, k) ? __float_as_uint(q[m.size * k]) : 0u;
                else
                    e[k] = exists<kLoose>(m, j, k) ? q[m.size * k] : 0u;
            }
#pragma unroll
            for (int k = 0; k < (kF32 ? 8 : 4); ++k) v.w[k] = kF32 ? e[k] : e[(2 * k) % 8] | e[(2 * k + 1) % 8] << 16;
        }
        return v;
    }
};

// A piece to a row, q: its first column that this thread has.
template <Lay kLay, bool kF32>
__device__ __forceinline__ void store_words(void* q, const Team& m, int j, const Words<kF32>& v) {
    if constexpr (kLay == kEights) {
        *reinterpret_cast<uint4*>(static_cast<char*>(q) + m.size * j * 16) = make_uint4(v.w[0], v.w[1], v.w[2], v.w[3]);
    } else if constexpr (kLay == kQuads) {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            if (!exists<kLay>(m, j, 4 * i)) break;
            char* to = static_cast<char*>(q) + m.size * (2 * j + i) * (kF32 ? 16 : 8);
            if constexpr (kF32)
                *reinterpret_cast<uint4*>(to) = make_uint4(v.w[4 * i], v.w[4 * i + 1], v.w[4 * i + 2], v.w[4 * i + 3]);
            else
                *reinterpret_cast<uint2*>(to) = make_uint2(v.w[2 * i], v.w[2 * i + 1]);
        }
    } else {
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            if (!exists<kLay>(m, j, k)) break;
            if constexpr (kF32)
                static_cast<uint32_t*>(q)[m.size * (8 * j + k)] = v.w[k];
            else
                static_cast<uint16_t*>(q)[m.size * (8 * j + k)] = (uint16_t)(k & 1 ? v.w[k / 2] >> 16 : v.w[k / 2]);
        }
    }
}
template <Lay kLay>
__device__ __forceinline__ void store_pairs(void* q, bool f32, const Team& m, int j, const float2 (&v)[4]) {
    if (kLay != kEights && f32) {
        Words<true> w;
#pragma unroll
        for (int k = 0; k < 4; ++k) w.w[2 * k] = __float_as_uint(v[k].x), w.w[2 * k + 1] = __float_as_uint(v[k].y);
        if constexpr (kLay != kEights) store_words<kLay, true>(q, m, j, w);
    } else {
        Words<false> w;
#pragma unroll
        for (int k = 0; k < 4; ++k) w.w[k] = pack_bf16x2(v[k].x, v[k].y);
        store_words<kLay, false>(q, m, j, w);
    }
}
// This thread's place in a row of an output, and the bytes from one row of the team to the next.
template <Lay kLay>
__device__ __forceinline__ char* output(void* q, int64_t ld, int size, int64_t row, const Team& m) {
    return static_cast<char*>(q) + (row * ld + column<kLay>(m, 0, 0)) * size;
}

// A piece of gamma or beta as bf16 pairs; `fill` (a pair) where the vector is absent.
template <Lay kLay>
__device__ __forceinline__ Words<false> weight_piece(const uint16_t* w, bool vec, const Team& m, int j, uint32_t fill) {
    Words<false> v;
    if (!w) {
#pragma unroll
        for (int k = 0; k < 4; ++k) v.w[k] = fill;
    } else if (kLay == kEights && vec) {
        const uint4 u = exists<kLay>(m, j, 0) ? *reinterpret_cast<const uint4*>(w + column<kLay>(m, j, 0)) : make_uint4(0u, 0u, 0u, 0u);
        v.w[0] = u.x; v.w[1] = u.y; v.w[2] = u.z; v.w[3] = u.w;
    } else if (kLay == kQuads && vec) {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const uint2 u = exists<kLay>(m, j, 4 * i) ? *reinterpret_cast<const uint2*>(w + column<kLay>(m, j, 4 * i)) : make_uint2(0u, 0u);
            v.w[2 * i] = u.x; v.w[2 * i + 1] = u.y;
        }
    } else {
        uint32_t e[8];
#pragma unroll
        for (int k = 0; k < 8; ++k) e[k] = exists<kLay>(m, j, k) ? w[column<kLay>(m, j, k)] : 0u;
#pragma unroll
        for (int k = 0; k < 4; ++k) v.w[k] = e[2 * k] | e[2 * k + 1] << 16;
    }
    return v;
}
constexpr uint32_t kOnes = 0x3f803f80u;

// ---- teams ----------------------------------------------------------------------------
// kMany: several warps; else `lanes` lanes (a power of two) of one.
template <Lay kLay, bool kMany>
__device__ __forceinline__ Team team_of(const NormParams& p, int* which, int* teams) {
    const int size = kMany ? 32 * p.warps : p.lanes;
    *which = threadIdx.x / size;
    *teams = blockDim.x / size;
    const int t = threadIdx.x - *which * size, all = kLay == kEights ? p.cols / 8 : kLay == kQuads ? p.cols / 4 : p.cols;
    return Team{t, size, all > t ? (all - t + size - 1) / size : 0};
}
__device__ __forceinline__ void team_barrier(int which, int threads) {
    asm volatile("bar.sync %0, %1;" ::"r"(which + 1), "r"(threads) : "memory");
}
// Over `lanes` neighbouring lanes (32: a literal for teams of warps); every lane gets it.
template <int kCount>
__device__ __forceinline__ void lane_sums(float (&v)[kCount], int lanes) {
#pragma unroll
    for (int o = 16; o; o /= 2) {
        if (o >= lanes) continue;
#pragma unroll
        for (int i = 0; i < kCount; ++i) v[i] += __shfl_xor_sync(0xffffffffu, v[i], o);
    }
}

template <bool kMany>
__device__ __forceinline__ void team_meet(int which, const Team& m) {
    if (kMany)
        team_barrier(which, m.size);
    else
        __syncwarp();
}
__device__ __forceinline__ void await_copies(int left) {
    if (left == 0)
        copies_wait<0>();
    else if (left == 1)
        copies_wait<1>();
    else if (left == 2)
        copies_wait<2>();
    else
        copies_wait<3>();
}

// The ring of slots: row after row of a team, `ahead` of them on their way.  send(slot)
// copies the next row, if there is one.  next() is called once a row, by all threads, and
// gives the slot that holds it.
template <bool kVec, bool kMany>
struct Ring {
    uint8_t* base;   // of the first slot: kVec this thread's places, else the team's part
    uint32_t size;
    int ahead, which, i = 0;
    template <class Send>
    __device__ __forceinline__ Ring(uint8_t* base, uint32_t size, int ahead, int which, Send send)
        : base(base), size(size), ahead(ahead), which(which) {
        for (int a = 0; a < ahead; ++a) {
            send(smem_addr(base) + a * size);
            copies_commit();
        }
    }
    template <class Send>
    __device__ __forceinline__ const uint8_t* next(const Team& m, Send send) {
        const uint8_t* here = base + i * size;
        const uint32_t free = smem_addr(base) + (i ? i - 1 : ahead) * size;   // the last row's
        i = i == ahead ? 0 : i + 1;
        if (kVec) {
            send(free);
            copies_commit();
            await_copies(ahead);
        } else if (ahead) {
            await_copies(ahead - 1);
            team_meet<kMany>(which, m);   // the whole row is there, and the last one read
            send(free);
            copies_commit();
        } else {
            team_meet<kMany>(which, m);
            send(smem_addr(here));
            copies_commit();
            await_copies(0);
            team_meet<kMany>(which, m);
        }
        return here;
    }
};

// ---- forward ------------------------------------------------------------------------
// The mean first over the warp's own columns, then the deviations from that number, whose
// sum corrects it and whose squares give the variance; warps are joined by their counts,
// means and squares, the means as differences from the first warp's, so that a mean far
// from the deviations costs no digits: all that is kept of it is one fp32 number `base`
// and the small distance from there.
// Bound by memory where there is a residual (8192 x 1600 bf16 18.3 us, 5.7 TB/s; fp32 31 us,
// 5.9 TB/s; the first row comes after 3 us), by latency without one (bf16 15 us for half of
// the bytes: 12 warps an SM issue in 44 % of the slots) and element by element (8192 x 1601
// 35 us); one row 2.5 us, a launch and two latencies.
struct WarpStats {
    float n, base, off, squares;   // columns, a number near their mean, the mean's distance from it, squared deviations
};

template <bool kF32, bool kVec, int kPer, int kThreads, bool kMany>
__global__ void __launch_bounds__(kThreads, 1) norm_kernel(const NormParams p) {
    extern __shared__ uint4 slots[];
    __shared__ WarpStats stats[2][kMostWarps];
    constexpr int kSize = kF32 ? 4 : 2;
    constexpr Lay kLay = lay_of(kVec, kF32);
    int which, teams, turn = 0;
    const Team m = team_of<kLay, kMany>(p, &which, &teams);
    // a team is no larger than it has to be: the first half of the pieces is there (2048 x 4097
    // bf16 27 us forward; 31 where that is asked for each)
    __builtin_assume(m.have >= kPer / 2 * (kLay == kEights ? 1 : kLay == kQuads ? 2 : 8));
    const int64_t stride = (int64_t)gridDim.x * teams;
    // teams of one warp shuffle together: all go on until the first of them has no row
    const int back = kMany ? 0 : threadIdx.x % 32 / p.lanes;
    int64_t row = (int64_t)blockIdx.x * teams + which;
    constexpr int kPlaces = kPer * (kF32 ? 2 : 1);
    Stream<kF32, kLay, kPer, 16 * kThreads, 0> xs(p.x, p.ldx, p.at[0], row, stride, p.rows, p.cols, m);
    Stream<kF32, kLay, kPer, 16 * kThreads, kPlaces> rs(p.residual, p.ldr, p.at[1], row, stride, p.rows, p.cols, m);
    int64_t sent = row;
    const auto send = [&](uint32_t slot) {
        if (sent < p.rows) {
            xs.send(slot, m, p.cols);
            if (p.residual) rs.send(slot, m, p.cols);
        }
        sent += stride;
    };
    char* sum = output<kLay>(p.sum, p.lds, kSize, row, m);
    char* y = output<kLay>(p.y, p.ldy, p.y_f32 ? 4 : 2, row, m);
    const int64_t sum_hop = stride * p.lds * kSize, y_hop = stride * p.ldy * (p.y_f32 ? 4 : 2);
    await_predecessor();
    Ring<kVec, kMany> ring(reinterpret_cast<uint8_t*>(slots) + (kVec ? threadIdx.x * p.part_bytes : which * p.part_bytes), p.slot, p.ahead, which, send);
    Words<false> gamma[kPer], beta[kPer];
    float n = 0.0f;   // this warp's columns, or the team's
#pragma unroll
    for (int j = 0; j < kPer; ++j) {
        gamma[j] = weight_piece<kLay>(p.gamma, p.weights_vec, m, j, kOnes);
        beta[j] = weight_piece<kLay>(p.beta, p.weights_vec, m, j, 0u);
#pragma unroll
        for (int k = 0; k < 8; ++k) n += exists<kLay>(m, j, k) ? 1.0f : 0.0f;
    }
    {
        float t[1] = {n};
        lane_sums<1>(t, kMany ? 32 : p.lanes);
        n = t[0];
    }
    const float share = n > 0.0f ? 1.0f / n : 0.0f;
    for (; row - back < p.rows; row += stride, sum += sum_hop, y += y_hop, xs.next_row(), rs.next_row()) {
        const bool has = kMany || row < p.rows;
        const uint8_t* slot = ring.next(m, send);
        float2 h[kPer][4], s2 = both(0.0f);
#pragma unroll
        for (int j = 0; j < kPer; ++j) {
            if (!has || !exists<kLay>(m, j, 0)) break;
            Words<kF32> x = xs.get(slot, m, j);
            if (p.residual) {
                x.add(rs.get(slot, m, j));   // as kept, and as the gradient will read it
                store_words<kLay, kF32>(sum, m, j, x);
            }
#pragma unroll
            for (int k = 0; k < 4; ++k) {   // an absent column is 0
                h[j][k] = x.pair(k);
                s2 = add2(s2, h[j][k]);
            }
        }
        float s[1] = {s2.x + s2.y};
        lane_sums<1>(s, kMany ? 32 : p.lanes);
        const float base = s[0] * share;
        float2 d1 = both(0.0f), d2 = both(0.0f);
#pragma unroll
        for (int j = 0; j < kPer; ++j) {   // from here on h is the distance from base
            if (!has || !exists<kLay>(m, j, 0)) break;
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                h[j][k] = add2(h[j][k], both(-base));
                if (kLay == kQuads && k >= 2 && !exists<kLay>(m, j, 4)) h[j][k] = both(0.0f);
                if (!kVec) h[j][k] = make_float2(exists<kLay>(m, j, 2 * k) ? h[j][k].x : 0.0f, exists<kLay>(m, j, 2 * k + 1) ? h[j][k].y : 0.0f);
                d1 = add2(d1, h[j][k]);
                d2 = fma2(h[j][k], h[j][k], d2);
            }
        }
        float d[2] = {d1.x + d1.y, d2.x + d2.y};
        lane_sums<2>(d, kMany ? 32 : p.lanes);
        float middle = base, off = d[0] * share, squares = d[1] - d[0] * off;   // the mean is middle + off
        if constexpr (kMany) {
            if ((threadIdx.x & 31) == 0) stats[turn][threadIdx.x / 32] = WarpStats{n, base, off, squares};
            team_barrier(which, m.size);
            const WarpStats* w = stats[turn] + which * p.warps;
            turn ^= 1;   // written again after the next row's barrier
            middle = w[0].base;
            off = squares = 0.0f;
#pragma unroll 4
            for (int i = 0; i < p.warps; ++i) off += w[i].n * (w[i].base - middle + w[i].off);
            off *= 1.0f / (float)p.cols;
#pragma unroll 4
            for (int i = 0; i < p.warps; ++i) {
                const float t = w[i].base - middle + w[i].off - off;
                squares += w[i].squares + w[i].n * t * t;
            }
        }
        if (squares < 0.0f) squares = 0.0f;   // rounding, where all columns are alike; not of NaN
        const float rstd = 1.0f / sqrtf(squares * (1.0f / (float)p.cols) + p.eps);
        if (!has) continue;
        if (m.t == 0) {
            if (p.mean) p.mean[row] = middle + off;
            if (p.rstd) p.rstd[row] = rstd;
        }
        const float2 move = both(base - middle - off), scale = both(rstd);
#pragma unroll
        for (int j = 0; j < kPer; ++j) {
            if (!exists<kLay>(m, j, 0)) break;
#pragma unroll
            for (int k = 0; k < 4; ++k) h[j][k] = fma2(mul2(add2(h[j][k], move), scale), gamma[j].pair(k), beta[j].pair(k));
            store_pairs<kLay>(y, p.y_f32, m, j, h[j]);
        }
    }
}

// ---- backward -----------------------------------------------------------------------
// Each thread sums dy xhat and dy of its columns down its team's rows, the CTA its teams,
// a second kernel the CTAs, every time in the same order.
// 8192 x 1600 bf16 with a residual takes 24 us for 105 MB: 3.7 until the first rows are
// there, 14 at the memory's full rate, 1.5 for the CTAs' sums and 4 for the second kernel.
// Rows of few CTAs' worth are bound by one row's way through a CTA, 2 us of sums, barrier
// and second pass (1021 x 6401 fp32 23 us for 66 MB, 1021 x 6400 18).
// The ring for teams of warps and rows off the grid: each row comes in one bulk copy a
// stream, by a thread of the team each; next() waits for those alone, and refill() is called
// once a row after a barrier of the team that follows next(), when the row before has been
// read.  (With copies by all threads and a barrier more, 2048 x 4097 bf16 took 44 us for
// 36, 1021 x 6401 fp32 27 for 24.8.  Forward, where fewer streams come, it was no gain.)
// A wait that gives up is the team's matter, since one warp's may end just before the copy
// comes and another's after: the warp goes on to that barrier as if the row were there, and
// behind it all of them see its mark and leave.  (A warp that left by itself would leave the
// others at the barrier for good.)  Marks of two rows in turn, as the sums.
struct BulkRing {
    uint8_t* base;
    uint64_t* full;   // of the slots
    int* gave_up;     // [2], the team's; 0 at first
    uint32_t size;
    int ahead, which, i = 0, last = 0;
    uint32_t phase = 0;
    template <class Send>
    __device__ __forceinline__ BulkRing(uint8_t* base, uint32_t size, int ahead, int which, uint64_t* full, int* gave_up, Send send)
        : base(base), full(full), gave_up(gave_up), size(size), ahead(ahead), which(which) {
        for (int a = 0; a < ahead; ++a) send(base + a * size, full + a);
    }
    template <class Send>
    __device__ __forceinline__ const uint8_t* next(const Team& m, int turn, Send send, long long limit = kWaitCycles) {
        if (ahead == 0) {
            team_barrier(which, m.size);   // the last row has been read
            send(base, full);
        }
        if (!warp_wait(full + i, phase, &g_norm_status, limit)) gave_up[turn] = 1;
        const uint8_t* here = base + i * size;
        last = i ? i - 1 : ahead;
        if (i == ahead) i = 0, phase ^= 1;
        else ++i;
        return here;
    }
    // Behind the barrier: whether the team leaves.  Copies in flight land before the CTA ends.
    __device__ __forceinline__ bool leaves(int turn, long long limit = kWaitCycles) {
        if (!gave_up[turn]) return false;
        const int now = i ? i - 1 : ahead;   // the slot that was waited for; none is on its way to `last`
        (void)mbar_wait_bounded(full + now, i ? phase : phase ^ 1, limit / 8);
        for (int k = 0; k <= ahead; ++k)
            if (k != now && k != last) (void)mbar_wait_bounded(full + k, k < i ? phase ^ 1 : phase, limit / 8);
        return true;
    }
    template <class Send>
    __device__ __forceinline__ void refill(Send send) {
        if (ahead) send(base + last * size, full + last);
    }
};
// A stream's part of a send, by one thread.
template <class S>
__device__ __forceinline__ void send_row(uint8_t* slot, uint64_t* bar, int cols, S& s) {
    fence_async_shared();   // the slot's readers are done
    mbar_arrive_expect_tx(bar, s.send_edges(smem_addr(slot), cols));
    s.send_whole(slot, bar);
}
struct BulkRings {   // of a CTA's teams
    uint64_t full[kMostWarps / 2][kMostAhead + 1];
    int gave_up[kMostWarps / 2][2];
    __device__ __forceinline__ void start(int streams) {
        if (threadIdx.x == 0) {
            for (int t = 0; t < kMostWarps / 2; ++t) {
                for (int i = 0; i <= kMostAhead; ++i) mbar_init(&full[t][i], streams);
                gave_up[t][0] = gave_up[t][1] = 0;
            }
            fence_barrier_init();
        }
        __syncthreads();
    }
};

template <bool kF32, bool kDyF32, bool kVec, int kPer, int kThreads, bool kMany>
__global__ void __launch_bounds__(kThreads, 1) norm_grad_kernel(const NormParams p) {
    extern __shared__ uint4 slots[];
    __shared__ float2 stats[2][kMostWarps];
    constexpr int kSize = kF32 ? 4 : 2;
    constexpr bool kBulk = kMany && !kVec;
    __shared__ BulkRings rings;
    if constexpr (kBulk) rings.start(p.residual ? 3 : 2);
    constexpr Lay kLay = lay_of(kVec, kF32);
    int which, teams, turn = 0;
    const Team m = team_of<kLay, kMany>(p, &which, &teams);
    __builtin_assume(m.have >= kPer / 2 * (kLay == kEights ? 1 : kLay == kQuads ? 2 : 8));
    const int64_t stride = (int64_t)gridDim.x * teams;
    const int back = kMany ? 0 : threadIdx.x % 32 / p.lanes;
    int64_t row = (int64_t)blockIdx.x * teams + which;
    constexpr int kXPlaces = kPer * (kF32 ? 2 : 1), kDyPlaces = kPer * (kDyF32 ? 2 : 1);
    Stream<kF32, kLay, kPer, 16 * kThreads, 0> xs(p.x, p.ldx, p.at[0], row, stride, p.rows, p.cols, m);
    Stream<kDyF32, kLay, kPer, 16 * kThreads, kXPlaces> ds(p.dy, p.lddy, p.at[1], row, stride, p.rows, p.cols, m);
    Stream<kF32, kLay, kPer, 16 * kThreads, kXPlaces + kDyPlaces> rs(p.residual, p.ldr, p.at[2], row, stride, p.rows, p.cols, m);
    int64_t sent = row;
    const auto send = [&](auto slot, auto... bar) {
        if (sent < p.rows) {
            if constexpr (kBulk) {
                if (m.t == 0) send_row(slot, bar..., p.cols, xs);
                if (m.t == 32) send_row(slot, bar..., p.cols, ds);
                if (m.t == (p.warps > 2 ? 64 : 0) && p.residual) send_row(slot, bar..., p.cols, rs);
            } else {
                xs.send(slot, m, p.cols);
                ds.send(slot, m, p.cols);
                if (p.residual) rs.send(slot, m, p.cols);
            }
        }
        sent += stride;
    };
    char* dx = output<kLay>(p.y, p.ldy, kSize, row, m);
    const int64_t dx_hop = stride * p.ldy * kSize;
    await_predecessor();
    auto ring = [&] {
        uint8_t* base = reinterpret_cast<uint8_t*>(slots) + (kVec ? threadIdx.x * p.part_bytes : which * p.part_bytes);
        if constexpr (kBulk)
            return BulkRing(base, p.slot, p.ahead, which, rings.full[which], rings.gave_up[which], send);
        else
            return Ring<kVec, kMany>(base, p.slot, p.ahead, which, send);
    }();
    Words<false> gamma[kPer];
    float2 sum_g[kPer][4], sum_b[kPer][4];
#pragma unroll
    for (int j = 0; j < kPer; ++j) {
        gamma[j] = weight_piece<kLay>(p.gamma, p.weights_vec, m, j, kOnes);
#pragma unroll
        for (int k = 0; k < 4; ++k) sum_g[j][k] = sum_b[j][k] = both(0.0f);
    }
    const float share = 1.0f / (float)p.cols;
    float mean_ahead = row < p.rows ? p.mean[row] : 0.0f, rstd_ahead = row < p.rows ? p.rstd[row] : 0.0f;
    for (; row - back < p.rows; row += stride, dx += dx_hop, xs.next_row(), ds.next_row(), rs.next_row()) {
        const bool has = kMany || row < p.rows;
        const float mean = mean_ahead, rstd = rstd_ahead;
        if (row + stride < p.rows) mean_ahead = p.mean[row + stride], rstd_ahead = p.rstd[row + stride];
        const uint8_t* slot;
        if constexpr (kBulk)
            slot = ring.next(m, turn, send);
        else
            slot = ring.next(m, send);
        const float2 move = both(-mean), scale = both(rstd);
        float2 v1 = both(0.0f), v2 = both(0.0f);
#pragma unroll
        for (int j = 0; j < kPer; ++j) {
            if (!has || !exists<kLay>(m, j, 0)) break;
            const Words<kF32> x = xs.get(slot, m, j);
            const Words<kDyF32> dy = ds.get(slot, m, j);
#pragma unroll
            for (int k = 0; k < 4; ++k) {   // an absent column has dy = 0
                const float2 g = mul2(dy.pair(k), gamma[j].pair(k));
                v1 = add2(v1, g);
                v2 = fma2(g, mul2(add2(x.pair(k), move), scale), v2);
            }
        }
        float v[2] = {v1.x + v1.y, v2.x + v2.y};
        lane_sums<2>(v, kMany ? 32 : p.lanes);
        if constexpr (kMany) {
            if ((threadIdx.x & 31) == 0) stats[turn][threadIdx.x / 32] = make_float2(v[0], v[1]);
            team_barrier(which, m.size);
            if constexpr (kBulk) {
                if (ring.leaves(turn)) break;
                ring.refill(send);
            }
            const float2* w = stats[turn] + which * p.warps;
            turn ^= 1;   // written again after the next row's barrier
            v[0] = v[1] = 0.0f;
#pragma unroll 4
            for (int i = 0; i < p.warps; ++i) v[0] += w[i].x, v[1] += w[i].y;
        }
        if (!has) continue;
        const float2 m1 = both(-v[0] * share), m2 = both(-v[1] * share);
#pragma unroll
        for (int j = 0; j < kPer; ++j) {
            if (!exists<kLay>(m, j, 0)) break;
            const Words<kF32> x = xs.get(slot, m, j);
            const Words<kDyF32> dy = ds.get(slot, m, j);
            float2 out[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const float2 d = dy.pair(k), xhat = mul2(add2(x.pair(k), move), scale);
                out[k] = mul2(fma2(xhat, m2, fma2(d, gamma[j].pair(k), m1)), scale);
                sum_g[j][k] = fma2(d, xhat, sum_g[j][k]);
                sum_b[j][k] = add2(sum_b[j][k], d);
            }
            if (p.residual) {
                const Words<kF32> r = rs.get(slot, m, j);
#pragma unroll
                for (int k = 0; k < 4; ++k) out[k] = add2(out[k], r.pair(k));
            }
            store_pairs<kLay>(dx, kF32, m, j, out);
        }
    }
    if (!p.part) return;
    float* part = p.part + (int64_t)blockIdx.x * p.cols;
    const int64_t half = (int64_t)gridDim.x * p.cols;
    // pair i of this thread's columns, from column c
    const auto column_of = [&](int i) { return column<kLay>(m, i / 4, 2 * (i % 4)); };
    const auto put = [&](int h, int i, float2 v) {
        const int c = column_of(i);
        if constexpr (kVec) {
            if (c < p.cols) *reinterpret_cast<float2*>(part + h * half + c) = v;
        } else {
            if (c < p.cols) part[h * half + c] = v.x;
            if (c + m.size < p.cols) part[h * half + c + m.size] = v.y;
        }
    };
    if (teams == 1) {
#pragma unroll
        for (int i = 0; i < 4 * kPer; ++i) {
            put(0, i, sum_g[i / 4][i % 4]);
            put(1, i, sum_b[i / 4][i % 4]);
        }
        return;
    }
    // several teams: their sums to shared memory, each team's pairs side by side, and added
    // in order, a team a share of the pairs
    float2* all = reinterpret_cast<float2*>(slots);
    const int width = 4 * kPer * m.size;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        __syncthreads();   // the rows, or the first half, have been read
#pragma unroll
        for (int i = 0; i < 4 * kPer; ++i) all[which * width + m.t + m.size * i] = h ? sum_b[i / 4][i % 4] : sum_g[i / 4][i % 4];
        __syncthreads();
#pragma unroll 4
        for (int i = which; i < 4 * kPer; i += teams) {
            float2 s = both(0.0f);
#pragma unroll 4
            for (int t = 0; t < teams; ++t) s = add2(s, all[t * width + m.t + m.size * i]);
            put(h, i, s);
        }
    }
}

// The ring's failure path by itself: a team of two warps waits for a copy that nothing sends.
// One gives up at `limit` cycles; a third warp arrives in the copy's place half as long after
// that, before the other gives up.  Both have to leave.
__global__ void __launch_bounds__(96) norm_wait_selftest_kernel(long long limit) {
    __shared__ BulkRings rings;
    __shared__ uint4 slot;
    rings.start(1);
    const long long begin = clock64();
    const Team m{(int)threadIdx.x, 64, 0};
    if (threadIdx.x < 64) {
        const long long mine = threadIdx.x < 32 ? limit : 2 * limit;
        const auto send = [](auto...) {};
        BulkRing ring(reinterpret_cast<uint8_t*>(&slot), sizeof slot, 1, 0, rings.full[0], rings.gave_up[0], send);
        for (int turn = 0;; turn ^= 1) {
            (void)ring.next(m, turn, send, mine);
            team_barrier(0, m.size);
            if (ring.leaves(turn, mine)) break;
        }
    } else if (threadIdx.x == 64) {
        while (clock64() - begin < limit + limit / 2) __nanosleep(1000);
        mbar_arrive(&rings.full[0][0]);
    }
}
int launch_norm_wait_selftest(int64_t limit, cudaStream_t s) {
    g_norm_waits.store(true);
    norm_wait_selftest_kernel<<<1, 96, 0, s>>>(limit);
    return launch_status();
}

// ---- rows of more than 16384 columns ---------------------------------------------------
// A CTA a row, in three passes (two backward) over it, the later ones out of L2, element by
// element (700 x 20000 bf16 with a residual 77 us, gradient with the weights' 96, for 17 us of
// bytes).
constexpr int kWideThreads = 512;

// Sums over the CTA in a fixed order, to every thread: one barrier, two buffers in turn.
struct CtaSums {
    float part[2][kWideThreads / 32][2];
};
template <int kCount>
__device__ __forceinline__ void cta_sums(float (&v)[kCount], CtaSums& s, int& turn) {
    lane_sums<kCount>(v, 32);
    if ((threadIdx.x & 31) == 0)
#pragma unroll
        for (int i = 0; i < kCount; ++i) s.part[turn][threadIdx.x / 32][i] = v[i];
    __syncthreads();
#pragma unroll
    for (int i = 0; i < kCount; ++i) {
        v[i] = 0.0f;
        for (int w = 0; w < kWideThreads / 32; ++w) v[i] += s.part[turn][w][i];
    }
    turn ^= 1;
}

// A thread's sums over a row.  Where those are of more than 256 terms (kLong) they are added up
// in runs of as many: one after the other, equal terms are rounded the same way each time (the
// mean of 30 million came out 6e-4 off).  For shorter rows the count took 3 % more.
constexpr int kRun = 256;
template <int kCount, bool kLong>
struct RowSums {
    float run[kCount] = {}, all[kLong ? kCount : 1] = {};
    int left = kRun;
    __device__ __forceinline__ void count() {
        if (kLong && --left == 0) {
            left = kRun;
#pragma unroll
            for (int i = 0; i < (kLong ? kCount : 0); ++i) all[i] += run[i], run[i] = 0.0f;
        }
    }
    __device__ __forceinline__ void get(float (&v)[kCount]) const {
#pragma unroll
        for (int i = 0; i < kCount; ++i) v[i] = kLong ? all[i % (kLong ? kCount : 1)] + run[i] : run[i];
    }
};

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

template <bool kF32, bool kLong>
__global__ void __launch_bounds__(kWideThreads) norm_wide_kernel(const NormParams p) {
    __shared__ CtaSums sums;
    await_predecessor();
    const float share = 1.0f / (float)p.cols;
    int turn = 0;
    for (int64_t row = blockIdx.x; row < p.rows; row += gridDim.x) {
        RowSums<1, kLong> sum;
        for (int c = threadIdx.x; c < p.cols; c += kWideThreads) {
            float h = value<kF32>(p.x, row * p.ldx + c);
            if (p.residual) {
                h += value<kF32>(p.residual, row * p.ldr + c);
                put(p.sum, kF32, row * p.lds + c, h);
                if (!kF32) h = bf16_one(to_bf16(h));
            }
            sum.run[0] += h;
            sum.count();
        }
        float m[1];
        sum.get(m);
        cta_sums<1>(m, sums, turn);
        const float mean = m[0] * share;
        const void* from = p.residual ? p.sum : p.x;   // a thread's own writes
        const int64_t ld = p.residual ? p.lds : p.ldx;
        RowSums<2, kLong> far;
        for (int c = threadIdx.x; c < p.cols; c += kWideThreads) {
            const float d = value<kF32>(from, row * ld + c) - mean;
            far.run[0] += d;
            far.run[1] += d * d;
            far.count();
        }
        float v[2];
        far.get(v);
        cta_sums<2>(v, sums, turn);
        const float off = v[0] * share, square = v[1] * share - off * off;
        const float rstd = 1.0f / sqrtf((square < 0.0f ? 0.0f : square) + p.eps);   // as above
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

template <bool kF32, bool kDyF32, bool kLong>
__global__ void __launch_bounds__(kWideThreads) norm_grad_wide_kernel(const NormParams p) {
    __shared__ CtaSums sums;
    await_predecessor();
    const float share = 1.0f / (float)p.cols;
    int turn = 0;
    for (int64_t row = blockIdx.x; row < p.rows; row += gridDim.x) {
        const float mean = p.mean[row], rstd = p.rstd[row];
        RowSums<2, kLong> sums_g;
        for (int c = threadIdx.x; c < p.cols; c += kWideThreads) {
            const float g = value<kDyF32>(p.dy, row * p.lddy + c) * (p.gamma ? bf16_one(p.gamma[c]) : 1.0f);
            sums_g.run[0] += g;
            sums_g.run[1] += g * ((value<kF32>(p.x, row * p.ldx + c) - mean) * rstd);
            sums_g.count();
        }
        float v[2];
        sums_g.get(v);
        cta_sums<2>(v, sums, turn);
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
// 3 us for the parts of 152 CTAs, two memory latencies and a barrier.
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
    const int lane = threadIdx.x & 31, warp = threadIdx.x / 32;
    const int c = blockIdx.x * 32 + lane;
    void* out = blockIdx.y ? p.out[1] : p.out[0];
    const void* acc = blockIdx.y ? p.acc[1] : p.acc[0];
    if (!out) return;
    float v = 0.0f;
    if (c < p.cols) {
        const float* q = p.part + (int64_t)blockIdx.y * p.parts * p.cols + c;
        for (int i0 = warp; i0 < p.parts; i0 += kFinishWarps * 10) {   // 10 loads in flight: the parts of 152 CTAs at once
            float t[10];
#pragma unroll
            for (int k = 0; k < 10; ++k) {
                const int i = i0 + kFinishWarps * k;
                t[k] = i < p.parts ? q[(int64_t)i * p.cols] : 0.0f;
            }
#pragma unroll
            for (int k = 0; k < 10; ++k) v += t[k];
        }
    }
    s[warp][lane] = v;
    __syncthreads();
    if (warp || c >= p.cols) return;
    for (int w = 1; w < kFinishWarps; ++w) v += s[w][lane];
    if (p.f32) {
        if (acc) v += static_cast<const float*>(acc)[c];
        static_cast<float*>(out)[c] = v;
    } else {
        if (acc) v += bf16_one(static_cast<const uint16_t*>(acc)[c]);
        static_cast<uint16_t*>(out)[c] = to_bf16(v);
    }
}

// ---- launches ---------------------------------------------------------------------------
constexpr int kWidestNorm = 16384;

// How a matrix is shared out: lanes of a warp or warps to a row, pieces a thread, threads
// of a CTA (one an SM), CTAs: no more teams to a CTA than give every SM some.
struct NormShape {
    bool many;
    int lanes, warps, per, threads, most;   // most: threads that the kernel is made for
    int64_t teams, grid;   // teams of a CTA
};
static NormShape norm_shape(int64_t rows, int64_t cols, bool vec, bool grad) {
    NormShape s{};
    const int64_t groups = (cols + 7) / 8, sms = sm_count();
    // a gradient element by element takes more registers: fewer pieces a thread (2048 x 4097
    // bf16 35 us with two where four took 39, 8192 x 1601 41 and 49; forward 27 with four, 32
    // with two, but 8192 x 1601 35 and 34)
    s.per = groups <= 32 ? 1 : groups <= 64 || (!vec && grad && groups <= 1024) ? 2 : 4;
    s.many = groups > 32 * s.per;
    s.warps = s.many ? (int)((groups + 32 * s.per - 1) / (32 * s.per)) : 1;
    s.lanes = 1;
    while (!s.many && s.lanes < 32 && s.lanes * s.per < groups) s.lanes *= 2;
    // 12 warps with registers to spare (8192 x 1600 bf16 19 and 25 us where 16 warps took 24
    // and 32); 16, of 128 registers a thread, for the widest rows and element by element
    s.most = s.many && (s.warps > 12 || s.per == 2 || (!vec && !grad)) ? 512 : 384;
    const int64_t in_warp = s.many ? 1 : 32 / s.lanes, most = s.many ? s.most / 32 / s.warps : s.most / 32 * in_warp;
    int64_t teams = (rows + sms - 1) / sms;
    teams = (teams + in_warp - 1) / in_warp * in_warp;   // whole warps
    s.teams = teams > most ? most : teams;
    s.threads = (int)(s.many ? s.teams * s.warps * 32 : s.teams / in_warp * 32);
    s.grid = (rows + s.teams - 1) / s.teams;
    if (s.grid > sms) s.grid = sms;
    return s;
}
// The most parts that the weights' gradients are summed in.
static int64_t norm_parts(int64_t rows, int64_t cols) {
    if (rows == 0 || cols == 0) return 0;
    const int64_t most = cols > kWidestNorm ? 64 : sm_count();
    return rows < most ? rows : most;
}

// Lays out the slots for a row of up to three streams (sizes of an element, 0 where
// absent) and as many rows ahead, at most three, as shared memory holds; its bytes.
constexpr int kNormSharedMemory = 226 * 1024;
static int lay_slots(NormParams& p, const NormShape& s, bool vec, const int (&sizes)[3]) {
    uint32_t at = 0, places = 0;
    for (int i = 0; i < 3; ++i) {
        p.at[i] = at;
        places += s.per * sizes[i] / 2;
        if (sizes[i]) at += (uint32_t)((p.cols * sizes[i] + 15) / 16 * 16 + 16);
    }
    p.part_bytes = vec ? 16 : at;
    p.slot = vec ? places * 16 * s.most : at * (uint32_t)s.teams;
    const int64_t own = (p.rows + s.grid * s.teams - 1) / (s.grid * s.teams);   // rows of a team
    p.ahead = (int32_t)(kNormSharedMemory / p.slot) - 1;
    if (p.ahead > kMostAhead) p.ahead = kMostAhead;
    if (p.ahead >= own) p.ahead = (int32_t)own - 1;
    return (int)p.slot * (p.ahead + 1);
}

template <bool kF32, bool kVec, int kPer, int kThreads, bool kMany>
static int launch_norm(NormParams& p, const NormShape& s, cudaStream_t stream) {
    static Done done;
    void (*const kernel)(NormParams) = norm_kernel<kF32, kVec, kPer, kThreads, kMany>;
    const int size = kF32 ? 4 : 2, smem = lay_slots(p, s, kVec, {size, p.residual ? size : 0, 0});
    if (smem > 46 * 1024)
        if (const int rc = allow_smem((const void*)kernel, kNormSharedMemory, done)) return rc;
    return launch_dense(kernel, dim3((unsigned)s.grid), s.threads, 1, true, smem, stream, p);
}
template <bool kF32, bool kDyF32, bool kVec, int kPer, int kThreads, bool kMany>
static int launch_norm_grad(NormParams& p, const NormShape& s, cudaStream_t stream) {
    static Done done;
    if (kMany && !kVec) g_norm_waits.store(true);
    void (*const kernel)(NormParams) = norm_grad_kernel<kF32, kDyF32, kVec, kPer, kThreads, kMany>;
    const int size = kF32 ? 4 : 2, sums = p.part ? kPer * 32 * s.threads : 0;   // the teams' sums, after the last row
    int smem = lay_slots(p, s, kVec, {size, kDyF32 ? 4 : 2, p.residual ? size : 0});
    if (smem < sums) smem = sums;
    if (smem > 46 * 1024)
        if (const int rc = allow_smem((const void*)kernel, kNormSharedMemory, done)) return rc;
    return launch_dense(kernel, dim3((unsigned)s.grid), s.threads, 1, true, smem, stream, p);
}
template <bool kF32, bool kVec>
static int launch_norm(NormParams& p, const NormShape& s, cudaStream_t stream) {
    if constexpr (kVec)
        if (s.many && s.most == 384) return launch_norm<kF32, kVec, 4, 384, true>(p, s, stream);
    if (s.many) return launch_norm<kF32, kVec, 4, 512, true>(p, s, stream);
    return s.per == 1 ? launch_norm<kF32, kVec, 1, 384, false>(p, s, stream)
           : s.per == 2 ? launch_norm<kF32, kVec, 2, 384, false>(p, s, stream) : launch_norm<kF32, kVec, 4, 384, false>(p, s, stream);
}
template <bool kF32, bool kDyF32, bool kVec>
static int launch_norm_grad(NormParams& p, const NormShape& s, cudaStream_t stream) {
    if constexpr (!kVec) {
        if (s.many && s.per == 2) return launch_norm_grad<kF32, kDyF32, kVec, 2, 512, true>(p, s, stream);
    } else {
        if (!s.many && s.per == 4) return launch_norm_grad<kF32, kDyF32, kVec, 4, 384, false>(p, s, stream);
    }
    if (s.many) return s.most > 384 ? launch_norm_grad<kF32, kDyF32, kVec, 4, 512, true>(p, s, stream) : launch_norm_grad<kF32, kDyF32, kVec, 4, 384, true>(p, s, stream);
    return s.per == 1 ? launch_norm_grad<kF32, kDyF32, kVec, 1, 384, false>(p, s, stream) : launch_norm_grad<kF32, kDyF32, kVec, 2, 384, false>(p, s, stream);
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
        const bool f32 = dtype == ZERO_F32, runs = cols > kRun * kWideThreads;
        return launch_dense(f32 ? (runs ? norm_wide_kernel<true, true> : norm_wide_kernel<true, false>)
                                : (runs ? norm_wide_kernel<false, true> : norm_wide_kernel<false, false>), dim3((unsigned)(rows < most ? rows : most)),
                            kWideThreads, 1, true, 0, s, p);
    }
    const bool vec = cols % 8 == 0 && rows_aligned16(x, ldx, size) && rows_aligned16(y, ldy, dtype_size(y_dtype)) &&
                     (!residual || (rows_aligned16(residual, ldr, size) && rows_aligned16(sum, lds, size)));
    const NormShape shape = norm_shape(rows, cols, vec, false);
    p.lanes = shape.lanes; p.warps = shape.warps;
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
    int64_t parts = weights ? norm_parts(rows, cols) : 0;
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
        if (parts)   // first: dx may be dy or x
            rc = launch_dense(!f32 ? norm_columns_kernel<false, false> : dy_f32 ? norm_columns_kernel<true, true> : norm_columns_kernel<true, false>,
                              dim3((unsigned)((cols + 255) / 256), (unsigned)parts), 256, 1, true, 0, s, p);
        if (rc == ZERO_OK)
            rc = launch_dense(cols > kRun * kWideThreads
                                  ? (!f32 ? norm_grad_wide_kernel<false, false, true> : dy_f32 ? norm_grad_wide_kernel<true, true, true> : norm_grad_wide_kernel<true, false, true>)
                                  : (!f32 ? norm_grad_wide_kernel<false, false, false> : dy_f32 ? norm_grad_wide_kernel<true, true, false> : norm_grad_wide_kernel<true, false, false>),
                              dim3((unsigned)(rows < most ? rows : most)), kWideThreads, 1, true, 0, s, p);
    } else {
        const bool vec = cols % 8 == 0 && rows_aligned16(x, ldx, size) && rows_aligned16(dy, lddy, dtype_size(dy_dtype)) &&
                         rows_aligned16(dx, lddx, size) && (!residual || rows_aligned16(residual, ldr, size));
        const NormShape shape = norm_shape(rows, cols, vec, true);
        p.lanes = shape.lanes; p.warps = shape.warps;
        if (parts) parts = shape.grid;
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
