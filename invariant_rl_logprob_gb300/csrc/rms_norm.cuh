// rms_norm.cuh -- rows of the root-mean-square norm and of its gradient: how a
// team of threads holds, reads, sums and writes them (rms_norm.cu,
// rms_norm_bwd.cu).
//
// A team (part of a warp up to 128 columns, a warp up to 1024 or, in the gradient, 512, up to
// 16 warps beyond) has a row in registers, up to 32 columns a thread: fewer threads a row
// mean fewer that sum, scale and wait for one another (256 threads with 16 columns
// each, 65536 x 4096 with residual to e4m3: 290 us; 128 with 32: 264, 105 % of the
// copy rate).  A thread owns eight consecutive columns at a time.  Rows off 16-byte
// boundaries (any row of an odd H, say) are read in the aligned 16 bytes around each
// eight and shifted on the way; results for such rows go through shared memory and
// leave in aligned 16 bytes as well.
//
// Which thread owns which column, and with it the order of every sum, depends on H
// and, in the gradient, on the types and on whether there is a residual's gradient.
// A sum of squares that leaves fp32 is formed again from r * 2^-80, and the gradient's
// sum of g r from n, of the size of 1, in place of r.
#pragma once

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

// The rows that cu_seqlens covers.
__device__ __forceinline__ void row_range(const int32_t *cu, int num_seqs, int64_t T, int64_t *lo, int64_t *hi) {
    *lo = 0;
    *hi = T;
    if (cu) {
        *lo = max((int64_t)0, (int64_t)cu[0]);
        *hi = min(T, (int64_t)cu[num_seqs]);
    }
}

// How rows are read.
//   kWords    activations in bf16 on 16-byte boundaries: kept as their words
//   kAligned  bf16 or fp32 on 16-byte boundaries: kept as floats
//   kFloats   anything else, shifted on the way
// The weight is on a 16-byte boundary in the first two.  65536 x 4096 bf16 with residual to e4m3
// takes 264 us as words and 481 with all that kFloats is ready for; an fp32 stream (fp32 x and
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

// ---- launches ----

inline Matrix matrix(const RulesMatrix *m) {
    if (!m) return Matrix{};
    return Matrix{static_cast<char *>(const_cast<void *>(m->p)), m->ld * size_of(m->type), (int32_t)m->type};
}

// With every row on a boundary of its vectors of 8 and made of whole ones (or missing).
inline bool plain(const Matrix &m, int64_t H) {
    const int vector = m.type == RK_E4M3 ? 8 : 16;
    return !m.p || (aligned(m.p, vector) && m.step % vector == 0 && H % 8 == 0);
}
inline bool plain(const Matrix &m, int type, int64_t H) { return !m.p || (m.type == type && plain(m, H)); }

constexpr size_t kMostShared = 200 * 1024;  // beside the static part; a stage of the widest row is a third of it

}  // namespace
}  // namespace rk
