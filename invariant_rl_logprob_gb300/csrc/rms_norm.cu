// rms_norm.cu -- root-mean-square norm of a row, with the residual's addition
// in front of it and an output in bf16, fp32 or e4m3 with scales ("rms_norm",
// RL-Kernel issue #101, maintainer comment, P0 operator list; chain index 2 of
// PR #264).
//
//   r = x,  or x + residual rounded to residual's type (written to residual_out)
//   y = r * rstd * weight,  rstd = 1 / sqrt(mean(r^2) + eps)
//
// Bound by memory: 8 flop an element (in 8 bits 14), against 4 to 16 bytes.  A block has a row, or a
// few narrow ones, in registers (rms_norm.cuh) and nothing lives longer: rings of
// rows in shared memory, filled by bulk copies ahead of persistent blocks, took
// 392 us with their waits where this takes 265, and plain loads of the next row 300.
#include "rms_norm.cuh"

namespace rk {
namespace {

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

// The scale of the largest magnitude `top` (as bits): 2^-120 at least, so that its reciprocal is
// finite; 0 if there is nothing to scale.
__device__ __forceinline__ float scale_of(unsigned top) {
    return top ? fmaxf(__fmul_rn(__uint_as_float(top), 1.f / 448.f), 0x1p-120f) : 0.f;
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
        Divisor divisor(0.f);
        if (e4m3 && a.group == 0) {
            float top = 0.f;  // fmaxf passes over NaN
#pragma unroll
            for (int k = 0; k < NV; ++k) {
                float y[8];
                result(k, y);
#pragma unroll
                for (int e = 0; e < 8; ++e) top = fmaxf(top, fabsf(y[e]));
            }
            const float scale = scale_of(team_max<TEAM>(__float_as_uint(top), maxima));
            if (lane == 0) scales[0] = scale;
            divisor = Divisor(scale);
        }
        char *to = a.stage_out ? stage : a.out.row(t);
        if (!e4m3) {
#pragma unroll
            for (int k = 0; k < NV; ++k) {
                float y[8];
                result(k, y);
                C::store(to, a.out.type, k, H, lane, y);
            }
        } else {
#pragma unroll
            for (int k = 0; k < NV; ++k) {
                float y[8];
                result(k, y);
                if (a.group != 0) {  // 128 columns: 16 lanes (H > 128, so that a team has them)
                    float top = 0.f;
#pragma unroll
                    for (int e = 0; e < 8; ++e) top = fmaxf(top, fabsf(y[e]));
                    const unsigned lanes = TEAM < 32 ? team_lanes<TEAM>() : 0xffffu << (threadIdx.x & 16);
                    const float scale = scale_of(__reduce_max_sync(lanes, __float_as_uint(top)));
                    const int c = C::at(lane, k);
                    if ((lane & 15) == 0 && c < H) scales[c / 128] = scale;
                    divisor = Divisor(scale);
                }
                divisor.divide(y);
                C::store(to, RK_E4M3, k, H, lane, y);
            }
        }
        if (a.stage_out) {
            const int size = size_of(a.out.type);
            team_sync<TEAM>();
            C::flush(stage, a.out.row(t), H * size, size, lane);
            if (ROWS > 1) team_sync<TEAM>();
        }
    }
}

// ---- launches ----

// Widest row, team, vectors of 8 a thread, rows a team, block and blocks per SM.  Narrow rows: teams of 8
// lanes for 2M rows of 64 columns took 173 us (residual, e4m3) where warps took 496, of 16 lanes for 1M
// of 128 167 and 252 (now, with rounded quotients, 202 and 199; to bf16 153 both).
#define RK_NORM_SHAPES(SHAPE)        \
    SHAPE(64, 8, 1, 4, 128, 8)       \
    SHAPE(128, 16, 1, 4, 128, 8)     \
    SHAPE(256, 32, 1, 4, 128, 8)     \
    SHAPE(512, 32, 2, 2, 128, 8)     \
    SHAPE(1024, 32, 4, 1, 128, 6)    \
    SHAPE(2048, 64, 4, 1, 64, 12)    \
    SHAPE(4096, 128, 4, 1, 128, 7)   \
    SHAPE(8192, 256, 4, 1, 256, 3)   \
    SHAPE(16384, 512, 4, 1, 512, 2)

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
#define SHAPE(MAX, TEAM, NV, ROWS, BLOCK, PER)                                                 \
    if (H <= MAX)                                                                              \
        return words  ? forward_launch<TEAM, NV, kWords, ROWS, BLOCK, PER>(a, di, st)          \
               : on16 ? forward_launch<TEAM, NV, kAligned, ROWS, BLOCK, (PER * 2 + 2) / 3>(a, di, st) \
                      : forward_launch<TEAM, NV, kFloats, ROWS, BLOCK, PER>(a, di, st);
    RK_NORM_SHAPES(SHAPE)
#undef SHAPE
    return cudaErrorInvalidValue;
}

}  // namespace rk
