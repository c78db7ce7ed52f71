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
// Both are bound by memory: 8 and 15 flop an element, against 7 to 12 bytes.
// A team of threads (a warp up to 512 columns, a block beyond) owns a run of
// consecutive rows and a ring of stages in shared memory; one of its warps
// copies whole rows into the ring with cp.async.bulk, several rows ahead, so
// that what is in flight does not depend on registers or on the rows' sums.
// Copies start and end on 16-byte boundaries around the row (the bytes beside
// it are not looked at), so a row may start on any element.
//
// The backward needs nothing but r: the sums of r^2 and of g * r come out of
// one reduction.  dweight: a team adds its rows in registers, in order; blocks
// leave partial sums that a last kernel adds in order.
//
// Which thread owns which column, and with it the order of every sum, depends
// on H alone: eight consecutive columns where H is a multiple of 8, columns
// TEAM apart otherwise (stores stay coalesced).  The team's run of rows
// depends on the number of canonical rows alone.  A sum of squares that
// leaves fp32 is formed again from r * 2^-80.
#include <algorithm>

#include "elements.cuh"
#include "rk_device.cuh"
#include "rk_internal.h"

namespace rk {
namespace {

constexpr int kMaxStages = 8;
constexpr int kMaxUnit = 16;           // rows of a stage
constexpr int kSharedPerSm = 227 * 1024;
constexpr float kShrink = 0x1p-80f;    // for rows whose sum of squares leaves fp32

// ---- rows on their way into shared memory ----

struct Input {
    const char *p;
    int64_t step;  // bytes from row to row
    int32_t bytes; // of a row
    int32_t wide;  // fp32 (else bf16)
    int32_t slot;  // bytes that a row may take in a stage
    int32_t offset;  // where the input's slots begin in a stage
};

struct Ring {
    Input in[3];
    int32_t inputs, stages, stage_bytes, unit;
    int32_t compact;  // rows follow one another without a gap, in every input
};

struct TeamHead {
    uint64_t full[kMaxStages];
    int32_t row[kMaxStages][kMaxUnit];  // of each row in a stage; -1: inactive, not copied
    int32_t merged[kMaxStages];         // the stage's rows came as one copy
    int32_t abort;
    int32_t pad[7];
};
static_assert(sizeof(TeamHead) % 16 == 0, "rings start on 16 bytes");

// Untiled bulk copy global -> shared; both addresses and the size are multiples of 16.
__device__ __forceinline__ void bulk_load(uint32_t dst, const void *src, uint32_t bytes, uint32_t bar) {
    asm volatile(
        "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst),
        "l"(src), "r"(bytes), "r"(bar)
        : "memory");
}

// The rows [begin, end) of a list, unit by unit; `row_of(i)` is the physical row
// of entry i, or -1.  Every unit completes one phase of its stage's barrier,
// whether or not it has anything to copy.
template <typename RowOf>
struct Feed {
    const Ring &g;
    TeamHead *head;
    unsigned char *ring;
    RowOf row_of;
    int64_t begin, end;
    int units;
    int next, next_stage;  // the unit to be issued, and its stage
    int pending;           // its rows, one a lane
    int stage;             // of the unit to be read
    unsigned phases;

    __device__ __forceinline__ Feed(const Ring &ring_, TeamHead *head_, unsigned char *at, RowOf f, int64_t b,
                                    int64_t e)
        : g(ring_), head(head_), ring(at), row_of(f), begin(b), end(e),
          units(e > b ? (int)((e - b + ring_.unit - 1) / ring_.unit) : 0), next(0), next_stage(0), stage(0),
          phases(0) {}

    __device__ __forceinline__ int rows_in(int unit) const {
        const int64_t left = end - begin - (int64_t)unit * g.unit;
        return left < g.unit ? (int)left : g.unit;
    }
    __device__ __forceinline__ int lookup(int unit, int lane) const {
        return unit < units && lane < rows_in(unit) ? row_of(begin + (int64_t)unit * g.unit + lane) : -1;
    }

    // By one warp: barriers, and the first stages on their way.
    __device__ __forceinline__ void start(int lane) {
        if (lane == 0) {
            head->abort = 0;
            for (int s = 0; s < g.stages; ++s) mbar_init(smem_u32(&head->full[s]), 1);
            fence_mbar_init();
        }
        __syncwarp();
        pending = lookup(0, lane);
        for (int s = 0; s < g.stages; ++s) issue(lane);
    }

    // By one warp: the next unit on its way; nobody reads its stage any more.
    __device__ __forceinline__ void issue(int lane) {
        if (next >= units) return;
        const int row = pending, s = next_stage;
        pending = lookup(next + 1, lane);
        const int count = rows_in(next);
        ++next;
        if (++next_stage == g.stages) next_stage = 0;
        const int first = __shfl_sync(0xffffffffu, row, 0);
        const bool merged = g.compact && count > 1 && first >= 0 &&
                            __all_sync(0xffffffffu, lane >= count || row == first + lane);
        if (lane < g.unit) head->row[s][lane] = row;
        if (lane == 0) head->merged[s] = merged;
        const uint32_t bar = smem_u32(&head->full[s]);
        uint32_t mine = 0;
        if (merged) {
            if (lane < g.inputs) mine = hull(g.in[lane], first, count * g.in[lane].bytes);
        } else if (row >= 0) {
            for (int k = 0; k < g.inputs; ++k) mine += hull(g.in[k], row, g.in[k].bytes);
        }
        const uint32_t all = __reduce_add_sync(0xffffffffu, mine);
        if (lane == 0) mbar_arrive_expect_tx(bar, all);
        __syncwarp();
        const uint32_t dst = smem_u32(ring + (size_t)s * g.stage_bytes);
        if (merged) {
            if (lane < g.inputs) copy(g.in[lane], first, count * g.in[lane].bytes, dst, bar);
        } else if (row >= 0) {
            for (int k = 0; k < g.inputs; ++k)
                copy(g.in[k], row, g.in[k].bytes, dst + lane * g.in[k].slot, bar);
        }
    }

    static __device__ __forceinline__ uint32_t hull(const Input &in, int row, int bytes) {
        const uintptr_t a = reinterpret_cast<uintptr_t>(in.p + row * in.step);
        return (uint32_t)(((a + bytes + 15) & ~uintptr_t(15)) - (a & ~uintptr_t(15)));
    }
    static __device__ __forceinline__ void copy(const Input &in, int row, int bytes, uint32_t dst, uint32_t bar) {
        const uintptr_t a = reinterpret_cast<uintptr_t>(in.p + row * in.step);
        bulk_load(dst + in.offset, reinterpret_cast<const void *>(a & ~uintptr_t(15)), hull(in, row, bytes), bar);
    }

    // The unit to be read has arrived (false: it has not, within the time limit).
    __device__ __forceinline__ bool wait(unsigned *err) {
        const bool mine = mbar_wait(smem_u32(&head->full[stage]), phases >> stage & 1u, &head->abort, err);
        const bool ok = __all_sync(0xffffffffu, mine);
        if (ok) phases ^= 1u << stage;
        return ok;
    }
    __device__ __forceinline__ int row(int j) const { return head->row[stage][j]; }
    // Row j of input k in shared memory.
    __device__ __forceinline__ const unsigned char *at(int k, int j) const {
        const Input &in = g.in[k];
        const unsigned char *base = ring + (size_t)stage * g.stage_bytes + in.offset;
        const bool merged = g.unit > 1 && head->merged[stage];
        const int from = head->row[stage][merged ? 0 : j];
        return base + (reinterpret_cast<uintptr_t>(in.p + from * in.step) & 15) + j * (merged ? in.bytes : in.slot);
    }
    __device__ __forceinline__ void advance() {
        if (++stage == g.stages) stage = 0;
    }
    // After a wait that gave up: copies still in flight must land before the block ends.
    __device__ __forceinline__ void drain() {
        for (int s = 0; s < g.stages; ++s)
            mbar_wait_drain(smem_u32(&head->full[s]), phases >> s & 1u, kWaitLimitNs / kMaxStages);
    }
};

// ---- a thread's columns of a row ----

// Thread `lane` of the team owns columns 8 (lane + TEAM k) .. + 7 (VEC: H is a multiple
// of 8) or lane + TEAM e; values past H are 0.
template <int TEAM, int NV, bool VEC>
struct Columns {
    static constexpr int kCount = 8 * NV;
    static __device__ __forceinline__ int at(int lane, int e) {
        return VEC ? 8 * (lane + TEAM * (e / 8)) + e % 8 : lane + TEAM * e;
    }

    // From shared memory, where the row may start on any element.
    static __device__ __forceinline__ void read(const unsigned char *row, bool wide, int H, int lane,
                                                float (&v)[kCount]) {
        __builtin_assume(__isShared(row));
        if constexpr (VEC) {
            const unsigned shift = smem_u32(row) & 15u;
#pragma unroll
            for (int k = 0; k < NV; ++k) {
                const int c = at(lane, 8 * k);
                float x[8];
#pragma unroll
                for (int j = 0; j < 8; ++j) x[j] = 0.f;
                if (c < H) {
                    if (shift == 0) {
                        if (wide)
                            get8(reinterpret_cast<const float *>(row) + c, x);
                        else
                            get8(reinterpret_cast<const uint16_t *>(row) + c, x);
                    } else if (wide) {
                        uint32_t w[12];
                        words<3>(row + 4 * c - shift, w);
                        shifted<8>(w, shift);
#pragma unroll
                        for (int j = 0; j < 8; ++j) x[j] = __uint_as_float(w[j]);
                    } else {
                        uint32_t w[8];
                        words<2>(row + 2 * c - shift, w);
                        shifted<4>(w, shift);
#pragma unroll
                        for (int j = 0; j < 4; ++j) {
                            x[2 * j] = bf16_lo(w[j]);
                            x[2 * j + 1] = bf16_hi(w[j]);
                        }
                    }
                }
#pragma unroll
                for (int j = 0; j < 8; ++j) v[8 * k + j] = x[j];
            }
        } else {
#pragma unroll
            for (int e = 0; e < kCount; ++e) {
                const int c = at(lane, e);
                v[e] = c >= H ? 0.f : wide ? get1(reinterpret_cast<const float *>(row) + c)
                                           : get1(reinterpret_cast<const uint16_t *>(row) + c);
            }
        }
    }
    template <int N>
    static __device__ __forceinline__ void words(const unsigned char *p, uint32_t (&w)[4 * N]) {
#pragma unroll
        for (int i = 0; i < N; ++i) {
            const uint4 q = reinterpret_cast<const uint4 *>(p)[i];
            w[4 * i] = q.x; w[4 * i + 1] = q.y; w[4 * i + 2] = q.z; w[4 * i + 3] = q.w;
        }
    }
    // The N words that begin `shift` (2 .. 14) bytes into w.
    template <int N>
    static __device__ __forceinline__ void shifted(uint32_t (&w)[N + 4], unsigned shift) {
        if (shift & 8u) {
#pragma unroll
            for (int i = 0; i < N + 2; ++i) w[i] = w[i + 2];
        }
        if (shift & 4u) {
#pragma unroll
            for (int i = 0; i < N + 1; ++i) w[i] = w[i + 1];
        }
        if (shift & 2u) {
#pragma unroll
            for (int i = 0; i < N; ++i) w[i] = __funnelshift_r(w[i], w[i + 1], 16);
        }
    }

    // From global memory (the weight).
    static __device__ __forceinline__ void load(const void *p, bool wide, int H, int lane, float (&v)[kCount]) {
#pragma unroll
        for (int e = 0; e < kCount; ++e) v[e] = 0.f;
        const bool vec = VEC && (reinterpret_cast<uintptr_t>(p) & 15) == 0;
#pragma unroll
        for (int k = 0; k < NV; ++k) {
            if (vec) {
                const int c = at(lane, 8 * k);
                if (c >= H) continue;
                float x[8];
                if (wide)
                    get8(static_cast<const float *>(p) + c, x);
                else
                    get8(static_cast<const uint16_t *>(p) + c, x);
#pragma unroll
                for (int j = 0; j < 8; ++j) v[8 * k + j] = x[j];
            } else {
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    const int c = at(lane, 8 * k + j);
                    if (c < H)
                        v[8 * k + j] = wide ? get1(static_cast<const float *>(p) + c)
                                            : get1(static_cast<const uint16_t *>(p) + c);
                }
            }
        }
    }

    // To global memory in fp32 or bf16.
    static __device__ __forceinline__ void store(void *p, bool wide, int H, int lane, const float (&v)[kCount]) {
        const bool vec = VEC && (reinterpret_cast<uintptr_t>(p) & 15) == 0;
#pragma unroll
        for (int k = 0; k < NV; ++k) {
            if (vec) {
                const int c = at(lane, 8 * k);
                if (c >= H) continue;
                float x[8];
#pragma unroll
                for (int j = 0; j < 8; ++j) x[j] = v[8 * k + j];
                if (wide)
                    put8(static_cast<float *>(p) + c, x);
                else
                    put8(static_cast<uint16_t *>(p) + c, x);
            } else {
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    const int c = at(lane, 8 * k + j);
                    if (c >= H) continue;
                    if (wide)
                        put1(static_cast<float *>(p) + c, v[8 * k + j]);
                    else
                        put1(static_cast<uint16_t *>(p) + c, v[8 * k + j]);
                }
            }
        }
    }
    // Eight of them (columns of at(lane, 8k ..)) as e4m3.
    static __device__ __forceinline__ void store_e4m3(uint8_t *p, int k, int H, int lane, const float (&x)[8]) {
        if (VEC && (reinterpret_cast<uintptr_t>(p) & 7) == 0) {
            const int c = at(lane, 8 * k);
            if (c < H) *reinterpret_cast<uint2 *>(p + c) = pack_e4m3x8(x);
        } else {
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const int c = at(lane, 8 * k + j);
                if (c < H) p[c] = (uint8_t)(pack_e4m3x2(x[j], 0.f) & 0xffu);
            }
        }
    }
};

// ---- sums and maxima over a team ----

struct TeamScratch {
    float2 sum[2][32];
    unsigned max[2][32];
    unsigned group[128];  // of 128 columns each, H <= 16384
};

template <int TEAM>
__device__ __forceinline__ void team_sync() {
    if constexpr (TEAM == 32)
        __syncwarp();
    else
        __syncthreads();
}

// Sums of a and b over the team, in an order that depends on TEAM alone.  Contains one
// team_sync; a buffer serves every other row.
template <int TEAM>
__device__ __forceinline__ float2 team_sum(float a, float b, float2 (&buffer)[32]) {
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) {
        a = __fadd_rn(a, __shfl_xor_sync(0xffffffffu, a, off));
        b = __fadd_rn(b, __shfl_xor_sync(0xffffffffu, b, off));
    }
    if constexpr (TEAM == 32) {
        __syncwarp();
    } else {
        const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
        if (lane == 0) buffer[warp] = make_float2(a, b);
        __syncthreads();
        constexpr int kWarps = TEAM / 32;
        const float2 v = buffer[lane % kWarps];
        a = v.x;
        b = v.y;
#pragma unroll
        for (int off = kWarps / 2; off > 0; off >>= 1) {
            a = __fadd_rn(a, __shfl_xor_sync(0xffffffffu, a, off));
            b = __fadd_rn(b, __shfl_xor_sync(0xffffffffu, b, off));
        }
    }
    return make_float2(a, b);
}

template <int TEAM>
__device__ __forceinline__ unsigned team_max(unsigned m, unsigned (&buffer)[32]) {
    m = __reduce_max_sync(0xffffffffu, m);
    if constexpr (TEAM > 32) {
        const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
        if (lane == 0) buffer[warp] = m;
        __syncthreads();
        m = __reduce_max_sync(0xffffffffu, buffer[lane % (TEAM / 32)]);
    }
    return m;
}

// ---- forward ----

struct Output {
    char *p;
    int64_t step;   // bytes from row to row
    int32_t type;   // rk_dtype
};

struct NormArgs {
    Ring ring;  // x, residual
    const void *weight;
    int32_t weight_wide;
    float eps;
    const int64_t *targets;
    const int32_t *cu;
    int32_t num_seqs;
    int64_t T;
    int32_t H;
    Output out, residual_out;
    float *scales;
    int32_t group;  // columns that share a scale: 128, or 0 for all
    unsigned *err;
};

// The active rows among 0 .. T-1; others are -1.
struct ActiveRows {
    const int64_t *targets;
    int64_t lo, hi;
    __device__ __forceinline__ int operator()(int64_t i) const {
        return i >= lo && i < hi && (!targets || targets[i] >= 0) ? (int)i : -1;
    }
};

__device__ __forceinline__ void row_range(const int32_t *cu, int num_seqs, int64_t T, int64_t *lo, int64_t *hi) {
    *lo = 0;
    *hi = T;
    if (cu) {
        *lo = max((int64_t)0, (int64_t)cu[0]);
        *hi = min(T, (int64_t)cu[num_seqs]);
    }
}

// A team's share of n list entries: whole units, the same for the same n and number of teams.
__device__ __forceinline__ int64_t team_share(int64_t n, int64_t teams, int unit) {
    const int64_t units = (n + unit - 1) / unit;
    return (units + teams - 1) / teams * unit;
}

// The scale of the largest magnitude `top` (as bits) and what to multiply with.  A scale is
// 2^-120 at least, so that its reciprocal is finite; 0 if there is nothing to scale.
__device__ __forceinline__ float scale_of(unsigned top, float *inverse) {
    const float m = __uint_as_float(top);
    if (m == 0.f) {
        *inverse = 0.f;
        return 0.f;
    }
    const float s = fmaxf(__fdiv_rn(m, 448.f), 0x1p-120f);
    *inverse = __frcp_rn(s);
    return s;
}

template <int TEAM, int NV, bool VEC, int BLOCK, int PER_SM>
__global__ void __launch_bounds__(BLOCK, PER_SM) rms_norm_forward(const __grid_constant__ NormArgs a) {
    using C = Columns<TEAM, NV, VEC>;
    constexpr int kTeams = BLOCK / TEAM;
    extern __shared__ __align__(128) unsigned char shared[];
    TeamScratch *scratch = reinterpret_cast<TeamScratch *>(shared) + threadIdx.x / TEAM;
    TeamHead *head =
        reinterpret_cast<TeamHead *>(shared + kTeams * sizeof(TeamScratch)) + threadIdx.x / TEAM;
    unsigned char *ring = shared + kTeams * (sizeof(TeamScratch) + sizeof(TeamHead)) +
                          (size_t)(threadIdx.x / TEAM) * a.ring.stages * a.ring.stage_bytes;
    const int lane = threadIdx.x % TEAM, wlane = threadIdx.x & 31;
    const bool feeder = lane < 32;
    const int H = a.H;
    wait_prior_grid();

    ActiveRows rows{a.targets, 0, 0};
    row_range(a.cu, a.num_seqs, a.T, &rows.lo, &rows.hi);
    const int64_t team = (int64_t)blockIdx.x * kTeams + threadIdx.x / TEAM;
    const int64_t share = team_share(a.T, (int64_t)gridDim.x * kTeams, a.ring.unit);
    Feed<ActiveRows> feed(a.ring, head, ring, rows, min(a.T, team * share), min(a.T, (team + 1) * share));
    if (feeder) feed.start(wlane);
    float w[C::kCount];
    C::load(a.weight, a.weight_wide, H, lane, w);
    if constexpr (TEAM > 32) __syncthreads();

    const float count = (float)H;
    bool dead = false;
    int parity = 0;
    for (int u = 0; u < feed.units; ++u) {
        if (!feed.wait(a.err)) dead = true;
        const int n = feed.rows_in(u);
        for (int j = 0; j < n; ++j, parity ^= 1) {
            const int row = feed.row(j);
            const int64_t t = feed.begin + (int64_t)u * a.ring.unit + j;
            float v[C::kCount];
            char *out = a.out.p + t * a.out.step, *stream = a.residual_out.p + t * a.residual_out.step;
            const bool with_residual = a.ring.inputs > 1;
            float k = 1.f, q = 0.f;  // rstd = k q
            if (row >= 0) {
                C::read(feed.at(0, j), a.ring.in[0].wide, H, lane, v);
                if (with_residual) {
                    float z[C::kCount];
                    C::read(feed.at(1, j), a.ring.in[1].wide, H, lane, z);
#pragma unroll
                    for (int e = 0; e < C::kCount; ++e) v[e] = __fadd_rn(v[e], z[e]);
                    if (a.residual_out.type == RK_BF16) {
                        // the sum as it is kept is what the norm, and a backward that reads it, sees
#pragma unroll
                        for (int e = 0; e < C::kCount; e += 2) {
                            const uint32_t b = pack_bf16x2(v[e], v[e + 1]);
                            v[e] = bf16_lo(b);
                            v[e + 1] = bf16_hi(b);
                        }
                    }
                }
                float ss = 0.f;
#pragma unroll
                for (int e = 0; e < C::kCount; ++e) ss = __fmaf_rn(v[e], v[e], ss);
                ss = team_sum<TEAM>(ss, 0.f, scratch->sum[parity]).x;
                if (!(ss < INFINITY)) {
                    k = kShrink;
                    ss = 0.f;
#pragma unroll
                    for (int e = 0; e < C::kCount; ++e) ss = __fmaf_rn(v[e] * k, v[e] * k, ss);
                    team_sync<TEAM>();
                    ss = team_sum<TEAM>(ss, 0.f, scratch->sum[parity]).x;
                }
                q = __frsqrt_rn(__fadd_rn(__fdiv_rn(ss, count), __fmul_rn(__fmul_rn(a.eps, k), k)));
            } else {
                team_sync<TEAM>();
#pragma unroll
                for (int e = 0; e < C::kCount; ++e) v[e] = 0.f;
            }
            // every thread has read the row: its stage is free
            if (TEAM > 32 && feeder && !dead) feed.issue(wlane);
            const int to = dead ? 0 : H;  // columns to write
            if (with_residual) C::store(stream, a.residual_out.type == RK_FP32, to, lane, v);
            const float rstd = q * k;
#pragma unroll
            for (int e = 0; e < C::kCount; ++e) v[e] = row >= 0 ? __fmul_rn(__fmul_rn(v[e], rstd), w[e]) : 0.f;
            if (a.out.type != RK_E4M3) {
                C::store(out, a.out.type == RK_FP32, to, lane, v);
                continue;
            }
            float inverse = 0.f;
            if (a.group == 0) {
                unsigned top = 0;
#pragma unroll
                for (int e = 0; e < C::kCount; ++e) top = max(top, __float_as_uint(fmaxf(fabsf(v[e]), 0.f)));
                top = team_max<TEAM>(top, scratch->max[parity]);
                const float s = scale_of(top, &inverse);
                if (lane == 0 && !dead) a.scales[t] = s;
            } else if (!VEC) {
                // a warp's columns of one e lie in one group of 128
                team_sync<TEAM>();
                for (int g = lane; g < 128; g += TEAM) scratch->group[g] = 0;
                team_sync<TEAM>();
#pragma unroll
                for (int e = 0; e < C::kCount; ++e) {
                    const unsigned top = __reduce_max_sync(0xffffffffu, __float_as_uint(fmaxf(fabsf(v[e]), 0.f)));
                    const int c = C::at(lane - wlane, e);
                    if (wlane == 0 && c < H) atomicMax(&scratch->group[c / 128], top);
                }
                team_sync<TEAM>();
            }
            const int groups = (H + 127) / 128;
#pragma unroll
            for (int m = 0; m < NV; ++m) {
                float x[8];
                if (a.group != 0 && VEC) {
                    unsigned top = 0;
#pragma unroll
                    for (int i = 0; i < 8; ++i) top = max(top, __float_as_uint(fmaxf(fabsf(v[8 * m + i]), 0.f)));
                    top = __reduce_max_sync(0xffffu << (wlane & 16), top);
                    const float s = scale_of(top, &inverse);
                    const int c = C::at(lane, 8 * m);
                    if ((wlane & 15) == 0 && c < to) a.scales[t * groups + c / 128] = s;
                }
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    if (a.group != 0 && !VEC) {
                        const int c = C::at(lane, 8 * m + i);
                        const float s = scale_of(scratch->group[min(c, H - 1) / 128], &inverse);
                        if (c % 128 == 0 && c < to) a.scales[t * groups + c / 128] = s;
                    }
                    x[i] = __fmul_rn(v[8 * m + i], inverse);
                }
                C::store_e4m3(reinterpret_cast<uint8_t *>(out), m, to, lane, x);
            }
        }
        feed.advance();
        if (TEAM == 32 && !dead) {
            __syncwarp();
            feed.issue(wlane);
        }
    }
    if (dead && lane == 0) feed.drain();
}

// ---- backward ----

struct NormBwdArgs {
    Ring ring;  // r, dout, dr
    const void *weight;
    int32_t weight_wide;
    float eps;
    const int32_t *cu;
    int32_t num_seqs;
    int64_t T;
    int32_t H;
    const int32_t *rows;      // the canonical rows, or NULL: those of the cu_seqlens range
    const int64_t *n_rows;    // how many
    const uint8_t *listed;    // which rows are among them
    Output dx;
    float *partial;  // [blocks, H], or NULL: no dweight
    unsigned *err;
};

struct ListedRows {
    const int32_t *rows;
    int64_t first;
    __device__ __forceinline__ int operator()(int64_t i) const { return rows ? rows[i] : (int)(first + i); }
};

template <int TEAM, int NV, bool VEC, int BLOCK, int PER_SM>
__global__ void __launch_bounds__(BLOCK, PER_SM) rms_norm_backward(const __grid_constant__ NormBwdArgs a) {
    using C = Columns<TEAM, NV, VEC>;
    constexpr int kTeams = BLOCK / TEAM;
    constexpr bool kKeep = TEAM < 1024;  // the weight and the row stay in registers
    extern __shared__ __align__(128) unsigned char shared[];
    TeamScratch *scratch = reinterpret_cast<TeamScratch *>(shared) + threadIdx.x / TEAM;
    TeamHead *head =
        reinterpret_cast<TeamHead *>(shared + kTeams * sizeof(TeamScratch)) + threadIdx.x / TEAM;
    unsigned char *rings = shared + kTeams * (sizeof(TeamScratch) + sizeof(TeamHead));
    unsigned char *ring = rings + (size_t)(threadIdx.x / TEAM) * a.ring.stages * a.ring.stage_bytes;
    const int lane = threadIdx.x % TEAM, wlane = threadIdx.x & 31;
    const bool feeder = lane < 32;
    const int H = a.H;
    wait_prior_grid();

    int64_t lo, hi;
    row_range(a.cu, a.num_seqs, a.T, &lo, &hi);
    const int64_t n = a.rows ? *a.n_rows : max((int64_t)0, hi - lo);
    const int64_t teams = (int64_t)gridDim.x * kTeams;
    const int64_t team = (int64_t)blockIdx.x * kTeams + threadIdx.x / TEAM;
    const int64_t share = team_share(n, teams, a.ring.unit);
    Feed<ListedRows> feed(a.ring, head, ring, ListedRows{a.rows, lo}, min(n, team * share),
                          min(n, (team + 1) * share));
    if (feeder) feed.start(wlane);
    float w[C::kCount], acc[C::kCount];
    if (kKeep) C::load(a.weight, a.weight_wide, H, lane, w);
#pragma unroll
    for (int e = 0; e < C::kCount; ++e) acc[e] = 0.f;
    if constexpr (TEAM > 32) __syncthreads();

    const float count = (float)H;
    const bool late = a.ring.stages > 1;  // a stage is refilled one row later
    bool dead = false;
    int parity = 0;
    for (int u = 0; u < feed.units; ++u) {
        if (!feed.wait(a.err)) dead = true;
        const int rows = feed.rows_in(u);
        for (int j = 0; j < rows; ++j, parity ^= 1) {
            const int64_t t = feed.row(j);
            float r[C::kCount], d[C::kCount];
            C::read(feed.at(0, j), a.ring.in[0].wide, H, lane, r);
            C::read(feed.at(1, j), a.ring.in[1].wide, H, lane, d);
            if (!kKeep) C::load(a.weight, a.weight_wide, H, lane, w);
            float s1 = 0.f, s2 = 0.f, k = 1.f;
#pragma unroll
            for (int e = 0; e < C::kCount; ++e) {
                s1 = __fmaf_rn(r[e], r[e], s1);
                s2 = __fmaf_rn(__fmul_rn(d[e], w[e]), r[e], s2);
            }
            float2 s = team_sum<TEAM>(s1, s2, scratch->sum[parity]);
            // every thread is done with the row before: its stage is free
            if (TEAM > 32 && feeder && late && u > 0 && !dead) feed.issue(wlane);
            if (!(s.x < INFINITY)) {
                k = kShrink;
                s1 = s2 = 0.f;
#pragma unroll
                for (int e = 0; e < C::kCount; ++e) {
                    s1 = __fmaf_rn(r[e] * k, r[e] * k, s1);
                    s2 = __fmaf_rn(__fmul_rn(d[e], w[e]), r[e] * k, s2);
                }
                team_sync<TEAM>();
                s = team_sum<TEAM>(s1, s2, scratch->sum[parity]);
            }
            // with z = k r:  rstd = k q,  n = r rstd,  mean(g n) = q mean(g z)
            const float q = __frsqrt_rn(__fadd_rn(__fdiv_rn(s.x, count), __fmul_rn(__fmul_rn(a.eps, k), k)));
            const float rstd = q * k, c = __fmul_rn(q, __fdiv_rn(s.y, count));
            float z[C::kCount];
            if (a.ring.inputs > 2) {
                C::read(feed.at(2, j), a.ring.in[2].wide, H, lane, z);
            } else {
#pragma unroll
                for (int e = 0; e < C::kCount; ++e) z[e] = 0.f;
            }
#pragma unroll
            for (int e = 0; e < C::kCount; ++e) {
                const float x = __fmul_rn(r[e], rstd);
                acc[e] = __fmaf_rn(d[e], x, acc[e]);
                z[e] = __fmaf_rn(rstd, __fmaf_rn(-x, c, __fmul_rn(d[e], w[e])), z[e]);
            }
            if (!dead) C::store(a.dx.p + t * a.dx.step, a.dx.type == RK_FP32, H, lane, z);
        }
        feed.advance();
        if (TEAM == 32) {
            __syncwarp();
            if (!dead) feed.issue(wlane);
        } else if (!late) {
            __syncthreads();
            if (feeder && !dead) feed.issue(wlane);
        }
    }
    if (dead && lane == 0) feed.drain();

    // 0 in the rows that are not among the canonical ones
    if (a.cu || a.listed) {
        float zero[C::kCount];
#pragma unroll
        for (int e = 0; e < C::kCount; ++e) zero[e] = 0.f;
        for (int64_t t = team; t < a.T; t += teams)
            if (a.listed ? !a.listed[t] : t < lo || t >= hi)
                C::store(a.dx.p + t * a.dx.step, a.dx.type == RK_FP32, H, lane, zero);
    }
    if (!a.partial) return;
    float *partial = a.partial + (int64_t)blockIdx.x * H;
    if constexpr (kTeams == 1) {
        C::store(partial, true, H, lane, acc);
    } else {
        // the block's teams one after the other, over the rings (every copy has landed)
        float *sum = reinterpret_cast<float *>(rings);
        __syncthreads();
        for (int i = 0; i < kTeams; ++i) {
            if ((int)(threadIdx.x / TEAM) == i) {
#pragma unroll
                for (int e = 0; e < C::kCount; ++e) {
                    const int col = C::at(lane, e);
                    if (col < H) sum[col] = i == 0 ? acc[e] : __fadd_rn(sum[col], acc[e]);
                }
            }
            __syncthreads();
        }
        for (int col = threadIdx.x; col < H; col += BLOCK) partial[col] = sum[col];
    }
}

// dweight[c] (+)= the blocks' partial sums: lane y takes blocks y, y + 32, ... in order,
// then the lanes' sums are added in order.
constexpr int kJoinLanes = 32;
__global__ void __launch_bounds__(32 * kJoinLanes)
    rms_norm_join(const float *partial, int blocks, int H, float *dweight, int accumulate) {
    __shared__ float sums[kJoinLanes][33];
    wait_prior_grid();
    const int x = threadIdx.x & 31, y = threadIdx.x >> 5, c = blockIdx.x * 32 + x;
    float s = 0.f;
    if (c < H) {
#pragma unroll 4
        for (int b = y; b < blocks; b += kJoinLanes) s = __fadd_rn(s, partial[(int64_t)b * H + c]);
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

__global__ void __launch_bounds__(kListThreads) norm_rows_count(Candidates c, int32_t *counts, uint8_t *listed) {
    __shared__ int scratch[32];
    wait_prior_grid();
    int64_t lo, hi;
    row_range(c.cu, c.num_seqs, c.T, &lo, &hi);
    for (int64_t t = (int64_t)blockIdx.x * kListThreads + threadIdx.x; t < c.T; t += (int64_t)gridDim.x * kListThreads)
        listed[t] = 0;
    int row[kListItems];
    const int total = block_sum(candidate_rows(c, lo, hi, row), scratch);
    if (threadIdx.x == 0) counts[blockIdx.x] = total;
}

__global__ void __launch_bounds__(kListThreads)
    norm_rows_write(Candidates c, const int32_t *counts, int32_t *rows, uint8_t *listed, int64_t *n_rows) {
    __shared__ int scratch[32], warps[32];
    wait_prior_grid();
    int64_t lo, hi;
    row_range(c.cu, c.num_seqs, c.T, &lo, &hi);
    int before = 0;  // rows of the blocks before this one (fewer than 2^31)
    for (int b = threadIdx.x; b < (int)blockIdx.x; b += kListThreads) before += counts[b];
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

int element_bytes(rk_dtype t) { return t == RK_E4M3 ? 1 : t == RK_BF16 ? 2 : 4; }

// Rows of a unit: about 1024 columns for a warp, one row for a block.
int unit_rows(int H, int team) {
    if (team > 32) return 1;
    int u = 1;
    while (u < kMaxUnit && 2 * u * H <= 1024) u *= 2;
    return u;
}

// Fills the ring's layout for blocks of `teams` teams, `per_sm` of them per SM; returns
// their shared memory, 0 if not even one stage fits into an SM.
size_t lay_out(Ring *g, int teams, int per_sm) {
    const size_t fixed = teams * (sizeof(TeamScratch) + sizeof(TeamHead));
    g->stage_bytes = 0;
    for (int k = 0; k < g->inputs; ++k) {
        g->in[k].slot = (g->in[k].bytes + 15) / 16 * 16 + 16;
        g->in[k].offset = g->stage_bytes;
        g->stage_bytes += g->in[k].slot * g->unit;
    }
    const size_t stage = (size_t)g->stage_bytes * teams;
    size_t room = kSharedPerSm / per_sm - 1024;
    if (fixed + stage > room) room = kSharedPerSm - 1024;
    if (fixed + stage > room) return 0;
    g->stages = (int)std::min<size_t>(kMaxStages, (room - fixed) / stage);
    return fixed + g->stages * stage;
}

Input input(const RulesMatrix &m, int64_t H) {
    Input in{};
    in.p = static_cast<const char *>(m.p);
    in.step = m.ld * element_bytes(m.type);
    in.bytes = (int32_t)(H * element_bytes(m.type));
    in.wide = m.type == RK_FP32;
    return in;
}

Output output(const RulesMatrix &m) {
    return Output{static_cast<char *>(const_cast<void *>(m.p)), m.ld * element_bytes(m.type), (int32_t)m.type};
}

// Team, vectors of 8 a thread, block, blocks per SM (forward, backward).
#define RK_NORM_SHAPES(SHAPE)         \
    SHAPE(256, 32, 1, 256, 4, 4)      \
    SHAPE(512, 32, 2, 256, 4, 3)      \
    SHAPE(1024, 128, 1, 128, 8, 6)    \
    SHAPE(2048, 128, 2, 128, 8, 4)    \
    SHAPE(4096, 256, 2, 256, 4, 2)    \
    SHAPE(8192, 512, 2, 512, 2, 1)    \
    SHAPE(16384, 1024, 2, 1024, 1, 1)

constexpr int kSmCount = 152;  // what the backward's partial sums are laid out for, on any device

template <int TEAM, int NV, bool VEC, int BLOCK, int PER_SM>
cudaError_t forward_launch(NormArgs &a, const DeviceInfo &di, cudaStream_t st) {
    auto *kernel = rms_norm_forward<TEAM, NV, VEC, BLOCK, PER_SM>;
    static std::atomic<uint64_t> allowed{0};
    const cudaError_t e = allow_shared(reinterpret_cast<const void *>(kernel), kSharedPerSm, di, allowed);
    if (e != cudaSuccess) return e;
    constexpr int kTeams = BLOCK / TEAM;
    a.ring.unit = unit_rows(a.H, TEAM);
    const size_t shared = lay_out(&a.ring, kTeams, PER_SM);
    if (!shared) return cudaErrorInvalidConfiguration;
    const int64_t per_block = (int64_t)kTeams * a.ring.unit;
    const int64_t grid = std::min((a.T + per_block - 1) / per_block, (int64_t)di.sm_count * PER_SM);
    return launch_dependent_smem(kernel, grid, BLOCK, shared, st, a);
}

template <int TEAM, int NV, bool VEC, int BLOCK, int PER_SM>
cudaError_t backward_launch(NormBwdArgs &a, const DeviceInfo &di, cudaStream_t st) {
    auto *kernel = rms_norm_backward<TEAM, NV, VEC, BLOCK, PER_SM>;
    static std::atomic<uint64_t> allowed{0};
    const cudaError_t e = allow_shared(reinterpret_cast<const void *>(kernel), kSharedPerSm, di, allowed);
    if (e != cudaSuccess) return e;
    constexpr int kTeams = BLOCK / TEAM;
    a.ring.unit = unit_rows(a.H, TEAM);
    size_t shared = lay_out(&a.ring, kTeams, PER_SM);
    if (!shared) return cudaErrorInvalidConfiguration;
    if (kTeams > 1) shared = std::max(shared, kTeams * (sizeof(TeamScratch) + sizeof(TeamHead)) + (size_t)a.H * 4);
    return launch_dependent_smem(kernel, (int64_t)kSmCount * PER_SM, BLOCK, shared, st, a);
}

int backward_blocks(int64_t H) {
#define SHAPE(MAX, TEAM, NV, BLOCK, FWD, BWD) \
    if (H <= MAX) return kSmCount * BWD;
    RK_NORM_SHAPES(SHAPE)
#undef SHAPE
    return 0;
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
    b.partial = static_cast<float *>(take((size_t)backward_blocks(H) * (size_t)H * 4));
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
    NormArgs a{};
    a.ring.in[0] = input(x, H);
    a.ring.inputs = 1;
    if (residual) {
        a.ring.in[a.ring.inputs++] = input(*residual, H);
        a.residual_out = output(*residual_out);
    }
    a.ring.compact = 1;
    for (int k = 0; k < a.ring.inputs; ++k) a.ring.compact &= a.ring.in[k].step == a.ring.in[k].bytes;
    a.weight = weight;
    a.weight_wide = weight_type == RK_FP32;
    a.eps = eps;
    a.targets = targets;
    a.cu = cu;
    a.num_seqs = num_seqs;
    a.T = T;
    a.H = (int32_t)H;
    a.out = output(out);
    a.scales = scales;
    a.group = group;
    a.err = di.err;
#define SHAPE(MAX, TEAM, NV, BLOCK, FWD, BWD)                                        \
    if (H <= MAX)                                                                    \
        return H % 8 == 0 ? forward_launch<TEAM, NV, true, BLOCK, FWD>(a, di, st)    \
                          : forward_launch<TEAM, NV, false, BLOCK, FWD>(a, di, st);
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
    NormBwdArgs a{};
    a.ring.in[0] = input(r, H);
    a.ring.in[1] = input(dout, H);
    a.ring.inputs = 2;
    if (dr) a.ring.in[a.ring.inputs++] = input(*dr, H);
    a.ring.compact = 1;
    for (int k = 0; k < a.ring.inputs; ++k) a.ring.compact &= a.ring.in[k].step == a.ring.in[k].bytes;
    a.weight = weight;
    a.weight_wide = weight_type == RK_FP32;
    a.eps = eps;
    a.cu = cu;
    a.num_seqs = num_seqs;
    a.T = T;
    a.H = (int32_t)H;
    a.dx = output(dx);
    a.partial = dweight ? b.partial : nullptr;
    a.err = di.err;
    if (targets || order) {
        const Candidates c{order, n, T, targets, cu, num_seqs};
        const int64_t tiles = std::max<int64_t>(1, (n + kListTile - 1) / kListTile);
        cudaError_t e = launch_dependent(norm_rows_count, tiles, kListThreads, st, c, b.counts, b.listed);
        if (e == cudaSuccess)
            e = launch_dependent(norm_rows_write, tiles, kListThreads, st, c, (const int32_t *)b.counts, b.rows,
                                 b.listed, b.n_rows);
        if (e != cudaSuccess) return e;
        a.rows = b.rows;
        a.n_rows = b.n_rows;
        a.listed = b.listed;
    }
    cudaError_t e = cudaErrorInvalidValue;
#define SHAPE(MAX, TEAM, NV, BLOCK, FWD, BWD)                                         \
    if (H <= MAX && e == cudaErrorInvalidValue)                                       \
        e = H % 8 == 0 ? backward_launch<TEAM, NV, true, BLOCK, BWD>(a, di, st)       \
                       : backward_launch<TEAM, NV, false, BLOCK, BWD>(a, di, st);     \
    else
    RK_NORM_SHAPES(SHAPE) {}
#undef SHAPE
    if (e != cudaSuccess || !dweight) return e;
    return launch_dependent(rms_norm_join, (H + 31) / 32, 32 * kJoinLanes, st, (const float *)a.partial,
                            backward_blocks(H), (int)H, dweight, (int)accumulate);
}

}  // namespace rk
