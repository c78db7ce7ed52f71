// rms_norm.cu -- root-mean-square norm of a row, with the residual's addition
// in front of it and an output in bf16, fp32 or e4m3 with scales, and its
// gradient ("rms_norm", RL-Kernel issue #101, maintainer comment, P0 operator
// list; chain index 2 of PR #264; its weight's gradient belongs to the
// parameter gradients of issue #244, Workstream 3 #153: fixed order, no
// atomicAdd).
//
//   r = x,  or x + residual rounded to residual's type (written to residual_out)
//   y = r * rstd * weight,  rstd = 1 / sqrt(mean(r^2) + eps)
//
//   g = dout * weight,  n = r * rstd
//   dx = rstd * (g - n * mean(g * n)) + dr,   dweight (+)= sum over rows of dout * n
//
// Both are bound by memory: 8 and 15 flop an element, against 7 to 16 bytes.
// A team of threads (part of a warp up to 128 columns, a warp up to 1024, up to
// 16 warps beyond) has a row in registers, up to 32 columns a thread: fewer
// threads a row mean fewer that sum, scale and wait for one another (256 threads
// with 16 columns each, 65536 x 4096 with residual to e4m3: 290 us; 128 with 32:
// 265, 105 % of the copy rate).  The forward has a block for a row and nothing
// that lives longer: rings of rows in shared memory, filled by bulk copies ahead
// of persistent blocks, took 392 us with their waits, and plain loads of the
// next row 300.
//
// The backward needs nothing but r: the sums of r^2 and of g * r come out of
// one reduction.  dweight: a team adds its rows in registers, in order; blocks
// leave partial sums that a last kernel adds in order.  Teams therefore stay, and
// ask for their next row ahead, into the second cache (65536 x 4096, all bf16:
// 347 us without, 316 with, the copy rate).
//
// A thread owns eight consecutive columns at a time.  Rows off 16-byte boundaries
// (any row of an odd H, say) are read in the aligned 16 bytes around each eight and
// shifted on the way; results for such rows go through shared memory and leave in
// aligned 16 bytes as well.
//
// Which thread owns which column, and with it the order of every sum, depends
// on H alone.  Which rows a team of the backward takes depends on the number of
// canonical rows alone.  A sum of squares that leaves fp32 is formed again from
// r * 2^-80.
#include <algorithm>

#include "elements.cuh"
#include "rk_device.cuh"
#include "rk_internal.h"

namespace rk {
namespace {

constexpr float kShrink = 0x1p-80f;  // for rows whose sum of squares leaves fp32

struct Matrix {
    char *p;
    int64_t step;  // bytes from row to row
    int32_t type;  // rk_dtype
    __device__ __forceinline__ char *row(int64_t t) const { return p + t * step; }
};

// ---- teams ----

// The lanes of a warp that belong to the thread's team.
template <int TEAM>
__device__ __forceinline__ unsigned team_lanes() {
    if constexpr (TEAM >= 32)
        return 0xffffffffu;
    else
        return ((1u << TEAM) - 1u) << (threadIdx.x & 31 & ~(TEAM - 1));
}
template <int TEAM>
__device__ __forceinline__ void team_sync() {
    if constexpr (TEAM > 32)
        __syncthreads();
    else
        __syncwarp(team_lanes<TEAM>());
}

// ---- a thread's columns of a row ----

// N words that begin `shift` bytes into w.
template <int N>
__device__ __forceinline__ void shift_words(uint32_t (&w)[N + 4], unsigned shift) {
    if (shift & 8u) {
#pragma unroll
        for (int i = 0; i < N + 2; ++i) w[i] = w[i + 2];
    }
    if (shift & 4u) {
#pragma unroll
        for (int i = 0; i < N + 1; ++i) w[i] = w[i + 1];
    }
    if (shift & 3u) {
#pragma unroll
        for (int i = 0; i < N; ++i) w[i] = __funnelshift_r(w[i], w[i + 1], 8 * (shift & 3u));
    }
}
template <int N>
__device__ __forceinline__ void read_words(const void *p, uint32_t (&w)[4 * N]) {
#pragma unroll
    for (int i = 0; i < N; ++i) {
        const uint4 q = static_cast<const uint4 *>(p)[i];
        w[4 * i] = q.x; w[4 * i + 1] = q.y; w[4 * i + 2] = q.z; w[4 * i + 3] = q.w;
    }
}

// Thread `lane` of the team owns columns 8 (lane + TEAM k) .. + 7; values past H are 0.
template <int TEAM>
struct Columns {
    static __device__ __forceinline__ int at(int lane, int k) { return 8 * (lane + TEAM * k); }

    // The 16 bytes of vector k of a bf16 row on a 16-byte boundary, H a multiple of 8.
    static __device__ __forceinline__ uint4 words(const void *row, int k, int H, int lane) {
        const int c = at(lane, k);
        return c < H ? *reinterpret_cast<const uint4 *>(static_cast<const uint16_t *>(row) + c)
                     : make_uint4(0, 0, 0, 0);
    }

    // Vectors k0 .. k0 + N - 1, wherever the row starts; all loads are on their way before the first
    // is waited for.
    template <int N, typename T>
    static __device__ __forceinline__ void load_as(const T *row, int k0, int H, int lane, float (&x)[N][8]) {
        constexpr int kWords = 8 * sizeof(T) / 4;
        const unsigned shift = (unsigned)(reinterpret_cast<uintptr_t>(row) & 15);
        if (shift == 0 && H % 8 == 0) {
#pragma unroll
            for (int i = 0; i < N; ++i) {
                const int c = at(lane, k0 + i);
#pragma unroll
                for (int e = 0; e < 8; ++e) x[i][e] = 0.f;
                if (c < H) get8(row + c, x[i]);
            }
            return;
        }
        // the aligned 16 bytes that a column of the row lies in, and no others
        const char *from = reinterpret_cast<const char *>(row) - shift, *end = reinterpret_cast<const char *>(row + H);
        uint32_t w[N][kWords + 4];
#pragma unroll
        for (int i = 0; i < N; ++i) {
            const char *p = from + sizeof(T) * at(lane, k0 + i);
#pragma unroll
            for (int j = 0; j < kWords / 4 + 1; ++j) {
                const uint4 q = p + 16 * j < end ? *reinterpret_cast<const uint4 *>(p + 16 * j) : make_uint4(0, 0, 0, 0);
                w[i][4 * j] = q.x; w[i][4 * j + 1] = q.y; w[i][4 * j + 2] = q.z; w[i][4 * j + 3] = q.w;
            }
        }
#pragma unroll
        for (int i = 0; i < N; ++i) {
            shift_words<kWords>(w[i], shift);
            const int left = H - at(lane, k0 + i);
            if constexpr (sizeof(T) == 4) {
#pragma unroll
                for (int e = 0; e < 8; ++e) x[i][e] = __uint_as_float(w[i][e]);
            } else {
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    x[i][2 * e] = bf16_lo(w[i][e]);
                    x[i][2 * e + 1] = bf16_hi(w[i][e]);
                }
            }
            if (left < 8) {
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    if (e >= left) x[i][e] = 0.f;
            }
        }
    }
    template <int N>
    static __device__ __forceinline__ void load(const void *row, int type, int k0, int H, int lane, float (&x)[N][8]) {
        if (type == RK_FP32)
            load_as<N>(static_cast<const float *>(row), k0, H, lane, x);
        else
            load_as<N>(static_cast<const uint16_t *>(row), k0, H, lane, x);
    }

    // Vector k of a row that starts and ends on 16 bytes (e4m3: 8), in global memory or in the stage.
    static __device__ __forceinline__ void store(char *row, int type, int k, int H, int lane, const float (&x)[8]) {
        const int c = at(lane, k);
        if (c >= H) return;
        if (type == RK_FP32)
            put8(reinterpret_cast<float *>(row) + c, x);
        else if (type == RK_BF16)
            put8(reinterpret_cast<uint16_t *>(row) + c, x);
        else
            *reinterpret_cast<uint2 *>(row + c) = pack_e4m3x8(x);
    }

    // A row's `bytes` bytes from the stage (16-byte aligned, 16 bytes and more behind them) to
    // wherever the row starts; element size 1, 2 or 4.
    static __device__ __forceinline__ void flush(const char *stage, char *row, int bytes, int size, int lane) {
        if (size == 4) {
#pragma unroll 4
            for (int b = 4 * lane; b < bytes; b += 4 * TEAM)
                *reinterpret_cast<uint32_t *>(row + b) = *reinterpret_cast<const uint32_t *>(stage + b);
            return;
        }
        const int before = (int)(reinterpret_cast<uintptr_t>(row) & 15);
        for (int p = 16 * lane - before; p < bytes; p += 16 * TEAM) {
            if (p >= 0 && p + 16 <= bytes) {
                uint32_t w[8];
                read_words<2>(stage + (p & ~15), w);
                shift_words<4>(w, (unsigned)p & 15u);
                *reinterpret_cast<uint4 *>(row + p) = make_uint4(w[0], w[1], w[2], w[3]);
                continue;
            }
            for (int b = max(p, 0); b < min(p + 16, bytes); b += size) {
                if (size == 2)
                    *reinterpret_cast<uint16_t *>(row + b) = *reinterpret_cast<const uint16_t *>(stage + b);
                else
                    row[b] = stage[b];
            }
        }
    }
};

__host__ __device__ constexpr int size_of(int type) { return type == RK_E4M3 ? 1 : type == RK_BF16 ? 2 : 4; }
// Bytes of a team's stage.
__host__ __device__ constexpr int stage_bytes(int H) { return (H + 7) / 8 * 32 + 32; }

// Vector k of a bf16 or fp32 row on a 16-byte boundary, H a multiple of 8, as it was read: loads of
// several rows are on their way before one is looked at, whatever their types.
struct Raw {
    uint4 a, b;  // b: the second half of eight fp32
};
template <int TEAM>
__device__ __forceinline__ Raw raw_vector(const char *row, bool wide, bool wanted, int k, int H, int lane) {
    const int c = Columns<TEAM>::at(lane, k);
    const uint4 *p = reinterpret_cast<const uint4 *>(row + (wide ? 4 : 2) * c);
    wanted = wanted && c < H;
    Raw r;
    r.a = wanted ? p[0] : make_uint4(0, 0, 0, 0);
    r.b = wanted && wide ? p[1] : make_uint4(0, 0, 0, 0);
    return r;
}

__device__ __forceinline__ void unpack(uint4 p, float (&x)[8]) {
    const uint32_t q[4] = {p.x, p.y, p.z, p.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        x[2 * i] = bf16_lo(q[i]);
        x[2 * i + 1] = bf16_hi(q[i]);
    }
}

__device__ __forceinline__ void unpack(const Raw &r, bool wide, float (&x)[8]) {
    float narrow[8];
    unpack(r.a, narrow);
    const uint32_t v[8] = {r.a.x, r.a.y, r.a.z, r.a.w, r.b.x, r.b.y, r.b.z, r.b.w};
#pragma unroll
    for (int e = 0; e < 8; ++e) x[e] = wide ? __uint_as_float(v[e]) : narrow[e];
}

// ---- sums and maxima over a team ----

// Sums over the team, in an order that depends on TEAM alone.  A buffer may serve again when
// another one has served in between.
template <int TEAM>
__device__ __forceinline__ float2 team_sums(float a, float b, float2 (&buffer)[32]) {
#pragma unroll
    for (int off = (TEAM < 32 ? TEAM : 32) / 2; off > 0; off >>= 1)
        add2(a, b, __shfl_xor_sync(team_lanes<TEAM>(), a, off), __shfl_xor_sync(team_lanes<TEAM>(), b, off));
    if constexpr (TEAM > 32) {
        if ((threadIdx.x & 31) == 0) buffer[threadIdx.x >> 5] = make_float2(a, b);
        __syncthreads();
        const float2 s = buffer[0];
        a = s.x;
        b = s.y;
#pragma unroll
        for (int w = 1; w < TEAM / 32; ++w) {
            const float2 t = buffer[w];
            add2(a, b, t.x, t.y);
        }
    }
    return make_float2(a, b);
}
template <int TEAM>
__device__ __forceinline__ float team_sum(float a, float2 (&buffer)[32]) {
#pragma unroll
    for (int off = (TEAM < 32 ? TEAM : 32) / 2; off > 0; off >>= 1)
        a = __fadd_rn(a, __shfl_xor_sync(team_lanes<TEAM>(), a, off));
    if constexpr (TEAM > 32) {
        if ((threadIdx.x & 31) == 0) buffer[threadIdx.x >> 5].x = a;
        __syncthreads();
        a = buffer[0].x;
#pragma unroll
        for (int w = 1; w < TEAM / 32; ++w) a = __fadd_rn(a, buffer[w].x);
    }
    return a;
}
template <int TEAM>
__device__ __forceinline__ unsigned team_max(unsigned m, unsigned (&buffer)[32]) {
    m = __reduce_max_sync(team_lanes<TEAM>(), m);
    if constexpr (TEAM > 32) {
        const int lane = threadIdx.x & 31;
        if (lane == 0) buffer[threadIdx.x >> 5] = m;
        __syncthreads();
        m = __reduce_max_sync(0xffffffffu, buffer[lane % (TEAM / 32)]);
    }
    return m;
}

// 1 / sqrt(sum / H + eps) of a sum of squares of k r, for k r (rstd of r is k times that).
__device__ __forceinline__ float root(float sum, float per_column, float eps, float k) {
    return __frsqrt_rn(__fadd_rn(__fmul_rn(sum, per_column), __fmul_rn(__fmul_rn(eps, k), k)));
}

// ---- forward ----

struct NormArgs {
    Matrix x, residual;  // residual.p may be NULL
    const void *weight;
    int32_t weight_type;
    float eps, per_column;  // 1 / H
    const int64_t *targets;
    const int32_t *cu;
    int32_t num_seqs;
    int64_t T;
    int32_t H;
    Matrix out, residual_out;
    float *scales;
    int32_t group;  // columns that share a scale: 128, or 0 for all
    int32_t stage_out, stage_residual;  // rows leave through shared memory
};

__device__ __forceinline__ void row_range(const int32_t *cu, int num_seqs, int64_t T, int64_t *lo, int64_t *hi) {
    *lo = 0;
    *hi = T;
    if (cu) {
        *lo = max((int64_t)0, (int64_t)cu[0]);
        *hi = min(T, (int64_t)cu[num_seqs]);
    }
}

// The scale of the largest magnitude `top` (as bits) and what to multiply with.  A scale is
// 2^-120 at least, so that its reciprocal is finite; 0 if there is nothing to scale.
__device__ __forceinline__ float scale_of(unsigned top, float *inverse) {
    const float s = fmaxf(__fmul_rn(__uint_as_float(top), 1.f / 448.f), 0x1p-120f);
    *inverse = top ? __fdividef(1.f, s) : 0.f;
    return top ? s : 0.f;
}

// How rows are read.
//   kWords    activations in bf16 on 16-byte boundaries: kept as their words
//   kAligned  bf16 or fp32 on 16-byte boundaries: kept as floats
//   kFloats   anything else, shifted on the way
// The weight is on a 16-byte boundary in the first two.  65536 x 4096 bf16 with residual to e4m3
// takes 265 us as words and 481 with all that kFloats is ready for; an fp32 stream (fp32 x and
// residual to fp32) 605 us as kAligned, 105 % of the copy rate.
enum Read { kWords, kAligned, kFloats };

// Vector k of the weight.
template <int TEAM, int READ>
__device__ __forceinline__ void weight_vector(const void *w, int type, int k, int H, int lane, float (&x)[8]) {
    if constexpr (READ == kFloats) {
        float y[1][8];
        Columns<TEAM>::load(w, type, k, H, lane, y);
#pragma unroll
        for (int e = 0; e < 8; ++e) x[e] = y[0][e];
    } else {
        unpack(raw_vector<TEAM>(static_cast<const char *>(w), type == RK_FP32, true, k, H, lane), type == RK_FP32, x);
    }
}

// A thread's part of a row.
template <int NV, int READ>
struct Part {
    float v[NV][8];
    __device__ __forceinline__ void get(int k, float (&x)[8]) const {
#pragma unroll
        for (int e = 0; e < 8; ++e) x[e] = v[k][e];
    }
};
template <int NV>
struct Part<NV, kWords> {
    uint4 p[NV];
    __device__ __forceinline__ void get(int k, float (&x)[8]) const { unpack(p[k], x); }
};

template <int TEAM, int NV, int READ, int ROWS, int BLOCK, int PER_SM>
__global__ void __launch_bounds__(BLOCK, PER_SM) rms_norm_forward(const __grid_constant__ NormArgs a) {
    using C = Columns<TEAM>;
    __shared__ float2 sums[2][32];
    __shared__ unsigned maxima[32];
    extern __shared__ __align__(16) char stages[];  // where rows leave through them
    constexpr int kPair = NV > 1 ? 2 : 1;  // vectors read at once where they are shifted
    const int lane = threadIdx.x % TEAM, H = a.H;
    char *stage = stages + (size_t)(threadIdx.x / TEAM) * stage_bytes(H);
    wait_prior_grid();
    const int64_t t0 = ((int64_t)blockIdx.x * (BLOCK / TEAM) + threadIdx.x / TEAM) * ROWS;
    int64_t lo, hi;
    row_range(a.cu, a.num_seqs, a.T, &lo, &hi);

    // r, as it is kept
    Part<NV, READ> part[ROWS];
    bool live[ROWS];
#pragma unroll
    for (int i = 0; i < ROWS; ++i) {
        const int64_t t = t0 + i;
        live[i] = t >= lo && t < hi && (!a.targets || a.targets[t] >= 0);
        const char *x = a.x.row(t), *z = a.residual.row(t);
        if constexpr (READ == kWords) {
#pragma unroll
            for (int k = 0; k < NV; ++k)
                part[i].p[k] = live[i] ? C::words(x, k, H, lane) : make_uint4(0, 0, 0, 0);
            if (a.residual.p) {
                uint4 q[NV];
#pragma unroll
                for (int k = 0; k < NV; ++k) q[k] = live[i] ? C::words(z, k, H, lane) : make_uint4(0, 0, 0, 0);
                // A sum of two bf16 rounded once is what rounding it to fp32 before would leave: 24
                // bits are more than twice 8 and two.
#pragma unroll
                for (int k = 0; k < NV; ++k) {
                    uint4 &p = part[i].p[k];
                    p = make_uint4(add_bf16x2(p.x, q[k].x), add_bf16x2(p.y, q[k].y), add_bf16x2(p.z, q[k].z),
                                   add_bf16x2(p.w, q[k].w));
                }
            }
        } else if constexpr (READ == kAligned) {
            const bool x_wide = a.x.type == RK_FP32, z_wide = a.residual.type == RK_FP32;
            Raw p[NV], q[NV];
#pragma unroll
            for (int k = 0; k < NV; ++k) p[k] = raw_vector<TEAM>(x, x_wide, live[i], k, H, lane);
#pragma unroll
            for (int k = 0; k < NV; ++k) q[k] = raw_vector<TEAM>(z, z_wide, live[i] && a.residual.p, k, H, lane);
#pragma unroll
            for (int k = 0; k < NV; ++k) {
                unpack(p[k], x_wide, part[i].v[k]);
                if (!a.residual.p) continue;
                float y[8];
                unpack(q[k], z_wide, y);
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    float &v = part[i].v[k][e];
                    v = __fadd_rn(v, y[e]);
                    if (a.residual_out.type == RK_BF16) v = bf16_lo(pack_bf16x2(v, 0.f));
                }
            }
        } else {
#pragma unroll
            for (int k = 0; k < NV; ++k)
#pragma unroll
                for (int e = 0; e < 8; ++e) part[i].v[k][e] = 0.f;
            if (live[i]) {
#pragma unroll
                for (int k = 0; k < NV; k += kPair) {
                    float q[kPair][8];
                    C::load(x, a.x.type, k, H, lane, q);
#pragma unroll
                    for (int j = 0; j < 8 * kPair; ++j) part[i].v[k + j / 8][j % 8] = q[j / 8][j % 8];
                }
            }
            if (a.residual.p && live[i]) {
#pragma unroll
                for (int k = 0; k < NV; k += kPair) {
                    float q[kPair][8];
                    C::load(z, a.residual.type, k, H, lane, q);
#pragma unroll
                    for (int j = 0; j < 8 * kPair; ++j) {
                        float &v = part[i].v[k + j / 8][j % 8];
                        v = __fadd_rn(v, q[j / 8][j % 8]);
                        // what is kept is what the norm, and a backward that reads it, sees
                        if (a.residual_out.type == RK_BF16) v = bf16_lo(pack_bf16x2(v, 0.f));
                    }
                }
            }
        }
    }
#pragma unroll
    for (int i = 0; i < ROWS; ++i) {
        const int64_t t = t0 + i;
        if (t >= a.T) return;  // the whole team
        if (a.residual.p) {
            char *to = READ != kWords && a.stage_residual ? stage : a.residual_out.row(t);
#pragma unroll
            for (int k = 0; k < NV; ++k) {
                if constexpr (READ == kWords) {
                    const int c = C::at(lane, k);
                    if (c < H) *reinterpret_cast<uint4 *>(to + 2 * c) = part[i].p[k];
                } else {
                    C::store(to, a.residual_out.type, k, H, lane, part[i].v[k]);
                }
            }
            if (READ != kWords && a.stage_residual) {
                const int size = size_of(a.residual_out.type);
                team_sync<TEAM>();
                C::flush(stage, a.residual_out.row(t), H * size, size, lane);
                team_sync<TEAM>();
            }
        }
        float rstd = 0.f;
        if (live[i]) {
            float even = 0.f, odd = 0.f;
#pragma unroll
            for (int k = 0; k < NV; ++k) {
                float x[8];
                part[i].get(k, x);
#pragma unroll
                for (int e = 0; e < 8; e += 2) fma2(even, odd, x[e], x[e + 1], x[e], x[e + 1]);
            }
            float sum = team_sum<TEAM>(__fadd_rn(even, odd), sums[0]);
            rstd = root(sum, a.per_column, a.eps, 1.f);
            if (!(sum < INFINITY)) {
                sum = 0.f;
#pragma unroll
                for (int k = 0; k < NV; ++k) {
                    float x[8];
                    part[i].get(k, x);
#pragma unroll
                    for (int e = 0; e < 8; ++e) sum = __fmaf_rn(x[e] * kShrink, x[e] * kShrink, sum);
                }
                rstd = kShrink * root(team_sum<TEAM>(sum, sums[1]), a.per_column, a.eps, kShrink);
            }
        }

        // y, 0 in a row that is not active
        const auto result = [&](int k, float (&y)[8]) {
            float w[8];
            weight_vector<TEAM, READ>(a.weight, a.weight_type, k, H, lane, w);
            part[i].get(k, y);
#pragma unroll
            for (int e = 0; e < 8; e += 2) {
                mul2(y[e], y[e + 1], rstd, rstd);
                mul2(y[e], y[e + 1], w[e], w[e + 1]);
            }
            // (not a branch: the weight's loads would wait for one another)
#pragma unroll
            for (int e = 0; e < 8; ++e) y[e] = live[i] ? y[e] : 0.f;
        };
        const bool e4m3 = a.out.type == RK_E4M3;
        float *scales = a.scales + t * (a.group ? (H + 127) / 128 : 1);
        float inverse = 1.f;
        if (e4m3 && a.group == 0) {
            float top = 0.f;  // fmaxf passes over NaN
#pragma unroll
            for (int k = 0; k < NV; ++k) {
                float y[8];
                result(k, y);
#pragma unroll
                for (int e = 0; e < 8; ++e) top = fmaxf(top, fabsf(y[e]));
            }
            const float s = scale_of(team_max<TEAM>(__float_as_uint(top), maxima), &inverse);
            if (lane == 0) scales[0] = s;
        }
        char *to = a.stage_out ? stage : a.out.row(t);
#pragma unroll
        for (int k = 0; k < NV; ++k) {
            float y[8];
            result(k, y);
            if (e4m3) {
                if (a.group != 0) {  // 128 columns: 16 lanes (H > 128, so that a team has them)
                    float top = 0.f;
#pragma unroll
                    for (int e = 0; e < 8; ++e) top = fmaxf(top, fabsf(y[e]));
                    const unsigned lanes = TEAM < 32 ? team_lanes<TEAM>() : 0xffffu << (threadIdx.x & 16);
                    const float s = scale_of(__reduce_max_sync(lanes, __float_as_uint(top)), &inverse);
                    const int c = C::at(lane, k);
                    if ((lane & 15) == 0 && c < H) scales[c / 128] = s;
                }
#pragma unroll
                for (int e = 0; e < 8; e += 2) mul2(y[e], y[e + 1], inverse, inverse);
            }
            C::store(to, a.out.type, k, H, lane, y);
        }
        if (a.stage_out) {
            const int size = size_of(a.out.type);
            team_sync<TEAM>();
            C::flush(stage, a.out.row(t), H * size, size, lane);
            if (ROWS > 1) team_sync<TEAM>();
        }
    }
}

// ---- backward ----

__device__ __forceinline__ float one(const void *p, int type, int c) {
    return type == RK_FP32 ? get1(static_cast<const float *>(p) + c) : get1(static_cast<const uint16_t *>(p) + c);
}

struct NormBwdArgs {
    Matrix r, dout, dr;  // dr.p may be NULL
    const void *weight;
    int32_t weight_type;
    float eps, per_column;  // 1 / H
    const int32_t *cu;
    int32_t num_seqs;
    int64_t T;
    int32_t H;
    const int32_t *rows;    // the canonical rows, or NULL: those of the cu_seqlens range
    const int64_t *n_rows;  // how many
    const uint8_t *listed;  // which rows are among them
    Matrix dx;
    int32_t stage_dx;  // its rows leave through shared memory
    float *partial;    // [blocks, pitch_of(H)], or NULL: no dweight
};

__host__ __device__ constexpr int64_t pitch_of(int64_t H) { return (H + 7) / 8 * 8; }

// What the backward keeps of a row between its sums and its results: with kWords (r, dout and dr in
// bf16) and kMixed (the same with dout in fp32) its words; otherwise nothing, it is read again,
// from the caches.  65536 x 4096: kWords 316 us, kMixed 398 (both the copy rate); without kMixed its
// case took 610.  All in fp32, kAligned 884 us, 72 % of the copy rate.
constexpr int kMixed = 3;

template <int TEAM, int NV, int READ, int BLOCK, int PER_SM>
__global__ void __launch_bounds__(BLOCK, PER_SM) rms_norm_backward(const __grid_constant__ NormBwdArgs a) {
    using C = Columns<TEAM>;
    constexpr int kTeams = BLOCK / TEAM;
    __shared__ float2 sums[2][32];
    // the teams' stages, and in the end their sums of dweight
    extern __shared__ __align__(16) char stages[];
    const int lane = threadIdx.x % TEAM, H = a.H;
    char *stage = stages + (size_t)(threadIdx.x / TEAM) * stage_bytes(H);
    wait_prior_grid();

    int64_t lo, hi;
    row_range(a.cu, a.num_seqs, a.T, &lo, &hi);
    const int64_t n = a.rows ? *a.n_rows : max((int64_t)0, hi - lo);
    const int64_t teams = (int64_t)gridDim.x * kTeams;
    const int64_t team = (int64_t)blockIdx.x * kTeams + threadIdx.x / TEAM;
    float acc[NV][8];
#pragma unroll
    for (int k = 0; k < NV; ++k)
#pragma unroll
        for (int e = 0; e < 8; ++e) acc[k][e] = 0.f;

    int parity = 0;
    // fewer than 2^31 rows
    const int last = (int)n, step = (int)teams, first = (int)lo;
    const auto row_at = [&](int64_t i) { return i >= last ? 0 : a.rows ? a.rows[i] : first + (int)i; };
    int next = row_at(team);
    for (int64_t i = team; i < last; i += step) {
        const int t = next;
        next = row_at(i + step);
        const auto r = [&] { return a.r.row(t); };
        const auto d = [&] { return a.dout.row(t); };
        const auto z = [&] { return a.dr.row(t); };
        if (lane < 3 && i + step < last) {
            // the team's next row, on its way into the second cache
            const Matrix &m = lane == 0 ? a.r : lane == 1 ? a.dout : a.dr;
            if (m.p) {
                const uintptr_t from = reinterpret_cast<uintptr_t>(m.row(next)), to = from + H * size_of(m.type);
                const uintptr_t first16 = from & ~uintptr_t(15);
                asm volatile("cp.async.bulk.prefetch.L2.global [%0], %1;" ::"l"(first16),
                             "r"((uint32_t)((to + 15 & ~uintptr_t(15)) - first16))
                             : "memory");
            }
        }
        uint4 rw[NV], dw[NV * (READ == kMixed ? 2 : 1)], zw[NV];
        if constexpr (READ == kWords || READ == kMixed) {
#pragma unroll
            for (int k = 0; k < NV; ++k) {
                const int c = C::at(lane, k);
                rw[k] = C::words(r(), k, H, lane);
                if constexpr (READ == kWords) {
                    dw[k] = C::words(d(), k, H, lane);
                } else {
                    const uint4 *from = reinterpret_cast<const uint4 *>(d() + 4 * c);
                    dw[2 * k] = c < H ? from[0] : make_uint4(0, 0, 0, 0);
                    dw[2 * k + 1] = c < H ? from[1] : make_uint4(0, 0, 0, 0);
                }
                zw[k] = a.dr.p ? C::words(z(), k, H, lane) : make_uint4(0, 0, 0, 0);
            }
        }
        constexpr int kPair = NV > 1 ? 2 : 1;
        // vectors k .. k + kPair - 1 of r, dout and the weight
        const auto values = [&](int k, float (&x)[kPair][8], float (&g)[kPair][8], float (&w)[kPair][8]) {
            if constexpr (READ == kFloats) {
                C::load(r(), a.r.type, k, H, lane, x);
                C::load(d(), a.dout.type, k, H, lane, g);
                C::load(a.weight, a.weight_type, k, H, lane, w);
            } else if constexpr (READ == kAligned) {
                const bool r_wide = a.r.type == RK_FP32, d_wide = a.dout.type == RK_FP32;
                Raw p[kPair], q[kPair];
#pragma unroll
                for (int i = 0; i < kPair; ++i) {
                    p[i] = raw_vector<TEAM>(r(), r_wide, true, k + i, H, lane);
                    q[i] = raw_vector<TEAM>(d(), d_wide, true, k + i, H, lane);
                }
#pragma unroll
                for (int i = 0; i < kPair; ++i) {
                    weight_vector<TEAM, READ>(a.weight, a.weight_type, k + i, H, lane, w[i]);
                    unpack(p[i], r_wide, x[i]);
                    unpack(q[i], d_wide, g[i]);
                }
            } else {
#pragma unroll
                for (int i = 0; i < kPair; ++i) {
                    weight_vector<TEAM, READ>(a.weight, a.weight_type, k + i, H, lane, w[i]);
                    unpack(rw[k + i], x[i]);
                    if constexpr (READ == kWords) {
                        unpack(dw[k + i], g[i]);
                    } else {
                        const uint4 p = dw[2 * (k + i)], q = dw[2 * (k + i) + 1];
                        const uint32_t v[8] = {p.x, p.y, p.z, p.w, q.x, q.y, q.z, q.w};
#pragma unroll
                        for (int e = 0; e < 8; ++e) g[i][e] = __uint_as_float(v[e]);
                    }
                }
            }
        };

        // sums of z^2 and g z, z = k r
        float k1 = 1.f;
        float2 s;
        {
            float even1 = 0.f, odd1 = 0.f, even2 = 0.f, odd2 = 0.f;
#pragma unroll
            for (int k = 0; k < NV; k += kPair) {
                float x[kPair][8], g[kPair][8], w[kPair][8];
                values(k, x, g, w);
#pragma unroll
                for (int i = 0; i < kPair; ++i)
#pragma unroll
                    for (int e = 0; e < 8; e += 2) {
                        mul2(g[i][e], g[i][e + 1], w[i][e], w[i][e + 1]);
                        fma2(even1, odd1, x[i][e], x[i][e + 1], x[i][e], x[i][e + 1]);
                        fma2(even2, odd2, g[i][e], g[i][e + 1], x[i][e], x[i][e + 1]);
                    }
            }
            add2(even1, even2, odd1, odd2);
            s = team_sums<TEAM>(even1, even2, sums[parity]);
            parity ^= 1;
        }
        if (!(s.x < INFINITY)) {
            float squares = 0.f, products = 0.f;
#pragma unroll 1
            for (int k = 0; k < NV; ++k) {
#pragma unroll 1
                for (int e = 0; e < 8; ++e) {
                    const int c = C::at(lane, k) + e;
                    if (c >= H) continue;
                    const float x = kShrink * one(r(), a.r.type, c);
                    squares = __fmaf_rn(x, x, squares);
                    products = __fmaf_rn(__fmul_rn(one(d(), a.dout.type, c), one(a.weight, a.weight_type, c)), x, products);
                }
            }
            s = team_sums<TEAM>(squares, products, sums[parity]);
            parity ^= 1;
            k1 = kShrink;
        }
        // rstd = k q,  n = r rstd,  mean(g n) = q mean(g z)
        const float q = root(s.x, a.per_column, a.eps, k1), rstd = q * k1;
        const float c = -__fmul_rn(q, __fmul_rn(s.y, a.per_column));
#pragma unroll
        for (int k = 0; k < NV; k += kPair) {
            float x[kPair][8], g[kPair][8], w[kPair][8], y[kPair][8];
            const bool z_wide = a.dr.type == RK_FP32;
            Raw zr[kPair];
            if constexpr (READ == kAligned) {
#pragma unroll
                for (int i = 0; i < kPair; ++i) zr[i] = raw_vector<TEAM>(z(), z_wide, a.dr.p, k + i, H, lane);
            }
            values(k, x, g, w);
            if constexpr (READ == kAligned) {
#pragma unroll
                for (int i = 0; i < kPair; ++i) unpack(zr[i], z_wide, y[i]);
            } else if constexpr (READ == kFloats) {
                if (a.dr.p) {
                    C::load(z(), a.dr.type, k, H, lane, y);
                } else {
#pragma unroll
                    for (int j = 0; j < 8 * kPair; ++j) y[j / 8][j % 8] = 0.f;
                }
            } else {
#pragma unroll
                for (int i = 0; i < kPair; ++i) unpack(zw[k + i], y[i]);
            }
#pragma unroll
            for (int i = 0; i < kPair; ++i) {
#pragma unroll
                for (int e = 0; e < 8; e += 2) {
                    mul2(x[i][e], x[i][e + 1], rstd, rstd);
                    fma2(acc[k + i][e], acc[k + i][e + 1], g[i][e], g[i][e + 1], x[i][e], x[i][e + 1]);
                    mul2(g[i][e], g[i][e + 1], w[i][e], w[i][e + 1]);
                    fma2(g[i][e], g[i][e + 1], x[i][e], x[i][e + 1], c, c);
                    fma2(y[i][e], y[i][e + 1], rstd, rstd, g[i][e], g[i][e + 1]);
                }
                C::store(a.stage_dx ? stage : a.dx.row(t), a.dx.type, k + i, H, lane, y[i]);
            }
        }
        if (a.stage_dx) {
            const int size = size_of(a.dx.type);
            team_sync<TEAM>();
            C::flush(stage, a.dx.row(t), H * size, size, lane);
            team_sync<TEAM>();
        }
    }

    // 0 in the rows that are not among the canonical ones
    if (a.cu || a.listed) {
        const float zero[8] = {};
        for (int64_t u = team; u < a.T; u += teams) {
            if (a.listed ? a.listed[u] : u >= lo && u < hi) continue;
            char *row = a.dx.row(u);
            if (!a.stage_dx) {
#pragma unroll
                for (int k = 0; k < NV; ++k) C::store(row, a.dx.type, k, H, lane, zero);
            } else {
                for (int c = lane; c < H; c += TEAM) {
                    if (a.dx.type == RK_FP32)
                        reinterpret_cast<float *>(row)[c] = 0.f;
                    else
                        reinterpret_cast<uint16_t *>(row)[c] = 0;
                }
            }
        }
    }
    // a block without rows has nothing to leave, and rms_norm_join does not look for it
    if (!a.partial || (int64_t)blockIdx.x * kTeams >= n) return;
    float *partial = a.partial + (int64_t)blockIdx.x * pitch_of(H);
    if constexpr (kTeams == 1) {
#pragma unroll
        for (int k = 0; k < NV; ++k) C::store(reinterpret_cast<char *>(partial), RK_FP32, k, H, lane, acc[k]);
    } else {
        // the block's teams one after the other
        float *joined = reinterpret_cast<float *>(stages);
        __syncthreads();
        for (int j = 0; j < kTeams; ++j) {
            if ((int)(threadIdx.x / TEAM) == j) {
#pragma unroll
                for (int k = 0; k < NV; ++k) {
                    const int c = C::at(lane, k);
#pragma unroll
                    for (int e = 0; e < 8; ++e)
                        if (c < H) joined[c + e] = j == 0 ? acc[k][e] : __fadd_rn(joined[c + e], acc[k][e]);
                }
            }
            __syncthreads();
        }
        for (int c = threadIdx.x; c < H; c += BLOCK) partial[c] = joined[c];
    }
}

// dweight[c] (+)= the partial sums of the blocks that had rows: lane y takes blocks y, y + 32, ...
// in order, then the lanes' sums are added in order.
constexpr int kJoinLanes = 32;
__global__ void __launch_bounds__(32 * kJoinLanes)
    rms_norm_join(const float *partial, int blocks, int rows_of_block, const int64_t *n_rows, const int32_t *cu,
                  int num_seqs, int64_t T, int H, float *dweight, int accumulate) {
    __shared__ float sums[kJoinLanes][33];
    wait_prior_grid();
    int64_t lo, hi;
    row_range(cu, num_seqs, T, &lo, &hi);
    const int64_t n = n_rows ? *n_rows : max((int64_t)0, hi - lo);
    const int busy = (int)min((int64_t)blocks, (n + rows_of_block - 1) / rows_of_block);
    const int x = threadIdx.x & 31, y = threadIdx.x >> 5, c = blockIdx.x * 32 + x;
    float s = 0.f;
    if (c < H) {
#pragma unroll 4
        for (int b = y; b < busy; b += kJoinLanes) s = __fadd_rn(s, partial[b * pitch_of(H) + c]);
    }
    sums[y][x] = s;
    __syncthreads();
    if (y == 0 && c < H) {
        for (int i = 1; i < kJoinLanes; ++i) s = __fadd_rn(s, sums[i][x]);
        dweight[c] = accumulate ? __fadd_rn(dweight[c], s) : s;
    }
}

// ---- the canonical rows: the active ones among the candidates, order kept ----

constexpr int kListThreads = 1024;
constexpr int kListItems = 8;  // consecutive candidates of a thread
constexpr int kListTile = kListThreads * kListItems;

struct Candidates {
    const int64_t *order;  // or NULL: rows 0, 1, ...
    int64_t n, T;
    const int64_t *targets;  // or NULL: all active
    const int32_t *cu;
    int32_t num_seqs;
};

// Rows of a thread's candidates (-1: none), and how many there are.
__device__ __forceinline__ int candidate_rows(const Candidates &c, int64_t lo, int64_t hi, int (&row)[kListItems]) {
    const int64_t first = (int64_t)blockIdx.x * kListTile + (int64_t)threadIdx.x * kListItems;
    int count = 0;
#pragma unroll
    for (int i = 0; i < kListItems; ++i) {
        row[i] = -1;
        if (first + i >= c.n) continue;
        const int64_t r = c.order ? c.order[first + i] : first + i;
        if (r < lo || r >= hi || (c.targets && c.targets[r] < 0)) continue;
        row[i] = (int)r;
        ++count;
    }
    return count;
}

__device__ __forceinline__ int block_sum(int v, int *scratch) {
    v = __reduce_add_sync(0xffffffffu, v);
    if ((threadIdx.x & 31) == 0) scratch[threadIdx.x >> 5] = v;
    __syncthreads();
    v = __reduce_add_sync(0xffffffffu, scratch[threadIdx.x & 31]);
    __syncthreads();
    return v;
}

__global__ void __launch_bounds__(kListThreads) norm_rows_count(Candidates c, int32_t *counts) {
    __shared__ int scratch[32];
    wait_prior_grid();
    int64_t lo, hi;
    row_range(c.cu, c.num_seqs, c.T, &lo, &hi);
    int row[kListItems];
    const int total = block_sum(candidate_rows(c, lo, hi, row), scratch);
    if (threadIdx.x == 0) counts[blockIdx.x] = total;
}

__global__ void __launch_bounds__(kListThreads)
    norm_rows_write(Candidates c, const int32_t *counts, int32_t *rows, uint8_t *listed, int64_t *n_rows) {  // counts NULL: one block
    __shared__ int scratch[32], warps[32];
    wait_prior_grid();
    int64_t lo, hi;
    row_range(c.cu, c.num_seqs, c.T, &lo, &hi);
    if (!counts) {  // nobody has cleared `listed` either
        for (int64_t t = threadIdx.x; t < c.T; t += kListThreads) listed[t] = 0;
        __syncthreads();
    }
    int before = 0;  // rows of the blocks before this one (fewer than 2^31)
    for (int b = threadIdx.x; counts && b < (int)blockIdx.x; b += kListThreads) before += counts[b];
    before = block_sum(before, scratch);
    int row[kListItems];
    const int mine = candidate_rows(c, lo, hi, row);
    int upto = mine;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, upto, off);
        if (lane >= off) upto += y;
    }
    if (lane == 31) warps[warp] = upto;
    __syncthreads();
    for (int i = 0; i < warp; ++i) upto += warps[i];
    int at = before + upto - mine;
#pragma unroll
    for (int i = 0; i < kListItems; ++i) {
        if (row[i] < 0) continue;
        rows[at++] = row[i];
        listed[row[i]] = 1;
    }
    if (blockIdx.x == gridDim.x - 1 && threadIdx.x == kListThreads - 1) *n_rows = before + upto;
}

// ---- launches ----

size_t round256(size_t b) { return (b + 255) / 256 * 256; }

Matrix matrix(const RulesMatrix *m) {
    if (!m) return Matrix{};
    return Matrix{static_cast<char *>(const_cast<void *>(m->p)), m->ld * size_of(m->type), (int32_t)m->type};
}

// With every row on a boundary of its vectors of 8 and made of whole ones (or missing).
bool plain(const Matrix &m, int64_t H) {
    const int vector = m.type == RK_E4M3 ? 8 : 16;
    return !m.p || (aligned(m.p, vector) && m.step % vector == 0 && H % 8 == 0);
}
bool plain(const Matrix &m, int type, int64_t H) { return !m.p || (m.type == type && plain(m, H)); }

// Widest row, team, vectors of 8 a thread, the forward's rows a team and block and its blocks per
// SM, the backward's block and blocks per SM.  Narrow rows: teams of 8 lanes for 2M rows of 64
// columns take 173 us (residual, e4m3) where warps took 496, of 16 lanes for 1M of 128 167 and 252.
// The backward's blocks per SM are what leaves its sums in registers: at 4096 columns 3, 4 and 5
// blocks of 128 threads took 103, 96 and 104 us for 16384 rows, before rows were asked for ahead.
#define RK_NORM_SHAPES(SHAPE)                \
    SHAPE(64, 8, 1, 4, 128, 8, 256, 3)       \
    SHAPE(128, 16, 1, 4, 128, 8, 256, 3)     \
    SHAPE(256, 32, 1, 4, 128, 8, 256, 3)     \
    SHAPE(512, 32, 2, 2, 128, 8, 256, 2)     \
    SHAPE(1024, 32, 4, 1, 128, 6, 128, 4)    \
    SHAPE(2048, 64, 4, 1, 64, 12, 64, 8)     \
    SHAPE(4096, 128, 4, 1, 128, 7, 128, 4)   \
    SHAPE(8192, 256, 4, 1, 256, 3, 256, 2)   \
    SHAPE(16384, 512, 4, 1, 512, 2, 512, 1)

constexpr int kSmCount = 152;  // what the backward's partial sums are laid out for, on any device
constexpr size_t kMostShared = 200 * 1024;  // beside the static part; a stage of the widest row is a third of it

template <int TEAM, int NV, int READ, int ROWS, int BLOCK, int PER_SM>
cudaError_t forward_launch(const NormArgs &a, const DeviceInfo &di, cudaStream_t st) {
    auto *kernel = rms_norm_forward<TEAM, NV, READ, ROWS, BLOCK, PER_SM>;
    constexpr int64_t kRows = (int64_t)BLOCK / TEAM * ROWS;
    const size_t shared = a.stage_out || a.stage_residual ? (size_t)(BLOCK / TEAM) * stage_bytes(a.H) : 0;
    if (shared > 48 * 1024 - 1024) {
        static std::atomic<uint64_t> allowed{0};
        const cudaError_t e = allow_shared(reinterpret_cast<const void *>(kernel), kMostShared, di, allowed);
        if (e != cudaSuccess) return e;
    }
    return launch_dependent_smem(kernel, (a.T + kRows - 1) / kRows, BLOCK, shared, st, a);
}

template <int TEAM, int NV, int READ, int BLOCK, int PER_SM>
cudaError_t backward_launch(const NormBwdArgs &a, const DeviceInfo &di, cudaStream_t st) {
    auto *kernel = rms_norm_backward<TEAM, NV, READ, BLOCK, PER_SM>;
    size_t shared = a.stage_dx ? (size_t)(BLOCK / TEAM) * stage_bytes(a.H) : 0;
    if (BLOCK > TEAM) shared = std::max(shared, (size_t)pitch_of(a.H) * 4);
    if (shared > 48 * 1024 - 1024) {
        static std::atomic<uint64_t> allowed{0};
        const cudaError_t e = allow_shared(reinterpret_cast<const void *>(kernel), kMostShared, di, allowed);
        if (e != cudaSuccess) return e;
    }
    return launch_dependent_smem(kernel, (int64_t)kSmCount * PER_SM, BLOCK, shared, st, a);
}

int backward_blocks(int64_t H) {
#define SHAPE(MAX, TEAM, NV, ROWS, FBLOCK, FPER, BBLOCK, BPER) \
    if (H <= MAX) return kSmCount * BPER;
    RK_NORM_SHAPES(SHAPE)
#undef SHAPE
    return 0;
}
int rows_of_block(int64_t H) {
#define SHAPE(MAX, TEAM, NV, ROWS, FBLOCK, FPER, BBLOCK, BPER) \
    if (H <= MAX) return BBLOCK / TEAM;
    RK_NORM_SHAPES(SHAPE)
#undef SHAPE
    return 1;
}

struct BwdBuffers {
    float *partial;
    int32_t *rows, *counts;
    int64_t *n_rows;
    uint8_t *listed;
    size_t bytes;
};

BwdBuffers carve(void *base, int64_t T, int64_t n, int64_t H) {
    BwdBuffers b{};
    char *p = static_cast<char *>(base);
    auto take = [&](size_t bytes) {
        char *q = p + b.bytes;
        b.bytes += round256(bytes);
        return static_cast<void *>(q);
    };
    b.partial = static_cast<float *>(take((size_t)backward_blocks(H) * (size_t)pitch_of(H) * 4));
    b.rows = static_cast<int32_t *>(take((size_t)n * 4));
    b.counts = static_cast<int32_t *>(take((size_t)(n / kListTile + 1) * 4));
    b.n_rows = static_cast<int64_t *>(take(8));
    b.listed = static_cast<uint8_t *>(take((size_t)T));
    return b;
}

}  // namespace

cudaError_t launch_rms_norm(const RulesMatrix &x, const RulesMatrix *residual, const void *weight,
                            rk_dtype weight_type, float eps, const int64_t *targets, const int32_t *cu,
                            int num_seqs, int64_t T, int64_t H, const RulesMatrix *residual_out,
                            const RulesMatrix &out, float *scales, int group, const DeviceInfo &di,
                            cudaStream_t st) {
    NormArgs a{matrix(&x), matrix(residual), weight, (int32_t)weight_type, eps, 1.f / (float)H, targets, cu, num_seqs,
               T, (int32_t)H, matrix(&out), matrix(residual_out), scales, H <= 128 ? 0 : group, 0, 0};
    a.stage_out = !plain(a.out, H);
    a.stage_residual = !plain(a.residual_out, H);
    const bool on16 = plain(a.x, H) && plain(a.residual, H) && aligned(weight, 16);
    const bool words = on16 && plain(a.x, RK_BF16, H) && plain(a.residual, RK_BF16, H) && plain(a.residual_out, RK_BF16, H);
#define SHAPE(MAX, TEAM, NV, ROWS, FBLOCK, FPER, BBLOCK, BPER)                                       \
    if (H <= MAX)                                                                                    \
        return words  ? forward_launch<TEAM, NV, kWords, ROWS, FBLOCK, FPER>(a, di, st)              \
               : on16 ? forward_launch<TEAM, NV, kAligned, ROWS, FBLOCK, (FPER * 2 + 2) / 3>(a, di, st) \
                      : forward_launch<TEAM, NV, kFloats, ROWS, FBLOCK, FPER>(a, di, st);
    RK_NORM_SHAPES(SHAPE)
#undef SHAPE
    return cudaErrorInvalidValue;
}

size_t rms_norm_bwd_workspace_bytes(int64_t T, int64_t n, int64_t H) { return carve(nullptr, T, n, H).bytes; }

cudaError_t launch_rms_norm_bwd(const RulesMatrix &dout, const RulesMatrix &r, const void *weight,
                                rk_dtype weight_type, float eps, const RulesMatrix *dr,
                                const int64_t *targets, const int32_t *cu, int num_seqs, int64_t T,
                                int64_t H, const int64_t *order, int64_t n, const RulesMatrix &dx,
                                float *dweight, bool accumulate, void *workspace, const DeviceInfo &di,
                                cudaStream_t st) {
    const BwdBuffers b = carve(workspace, T, n, H);
    NormBwdArgs a{matrix(&r), matrix(&dout), matrix(dr), weight, (int32_t)weight_type, eps, 1.f / (float)H, cu, num_seqs,
                  T, (int32_t)H, nullptr, nullptr, nullptr, matrix(&dx), 0, dweight ? b.partial : nullptr};
    a.stage_dx = !plain(a.dx, H);
    if (targets || order) {
        const Candidates c{order, n, T, targets, cu, num_seqs};
        const int64_t tiles = std::max<int64_t>(1, (n + kListTile - 1) / kListTile);
        // one block does it all: a launch and a fill less (8192 rows of 1024: 26 us, 8200: 30)
        const bool one = tiles == 1 && T <= kListTile;
        cudaError_t e = one ? cudaSuccess : cudaMemsetAsync(b.listed, 0, (size_t)T, st);
        if (e == cudaSuccess && !one) e = launch_dependent(norm_rows_count, tiles, kListThreads, st, c, b.counts);
        if (e == cudaSuccess)
            e = launch_dependent(norm_rows_write, tiles, kListThreads, st, c, one ? (const int32_t *)nullptr : b.counts,
                                 b.rows, b.listed, b.n_rows);
        if (e != cudaSuccess) return e;
        a.rows = b.rows;
        a.n_rows = b.n_rows;
        a.listed = b.listed;
    }
    const bool on16 = plain(a.r, H) && plain(a.dout, H) && plain(a.dr, H) && aligned(weight, 16);
    const bool words = a.r.type == RK_BF16 && (!dr || a.dr.type == RK_BF16);
    const int read = !on16 ? kFloats : !words ? kAligned : a.dout.type == RK_BF16 ? kWords : kMixed;
    const auto run = [&] {
#define SHAPE(MAX, TEAM, NV, ROWS, FBLOCK, FPER, BBLOCK, BPER)                                       \
    if (H <= MAX)                                                                                    \
        return read == kWords     ? backward_launch<TEAM, NV, kWords, BBLOCK, BPER>(a, di, st)       \
               : read == kMixed   ? backward_launch<TEAM, NV, kMixed, BBLOCK, BPER>(a, di, st)       \
               : read == kAligned ? backward_launch<TEAM, NV, kAligned, BBLOCK, BPER>(a, di, st)     \
                                  : backward_launch<TEAM, NV, kFloats, BBLOCK, BPER>(a, di, st);
        RK_NORM_SHAPES(SHAPE)
#undef SHAPE
        return cudaErrorInvalidValue;
    };
    const cudaError_t e = run();
    if (e != cudaSuccess || !dweight) return e;
    return launch_dependent(rms_norm_join, (H + 31) / 32, 32 * kJoinLanes, st, (const float *)a.partial,
                            backward_blocks(H), rows_of_block(H), a.n_rows, cu, num_seqs, T, (int)H, dweight,
                            (int)accumulate);
}

}  // namespace rk
