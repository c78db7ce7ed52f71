// preference.cu -- preference loss on selected logprobs: sums over the tokens
// of sequences, compared in pairs, and the gradient of every token's logprob
// (a loss beside grpo_loss, RL-Kernel issue #101, maintainer comment, P0
// operator list; end of the chain of PR #264, whose review asks for
// per-token outputs or a fixed normalisation: here a caller-given scale).
//
//   s_q = sum over the sequence's active tokens of (logp - logp_ref)   [/ their number]
//   d_p = s_chosen - s_rejected - margin_p
//   loss_p = scale * f(d_p),   grad_logp[t] = sum over p of the sequence: +-scale f'(d_p) [/ number]
//
// Bound by latency: 12 to 16 bytes a token, and five results that wait for one
// another (sums, ratios, pairs, coefficients, gradients).  One cluster of up to
// 16 blocks runs all of it, with the hardware's cluster barrier between the
// steps, up to kClusterTokens tokens; beyond, every step is a launch of its own
// over the whole device.
//
// The sums are integers, so that no order of tokens, blocks or atomic additions
// can change a bit: a logprob is rounded to a multiple of 2^-42 (logprobs of
// 2^-18 and more have no smaller bits) and added in two words.  A magnitude of
// 2^20 and more, which no probability of interest has, counts as infinite.
#include <algorithm>

#include "elements.cuh"
#include "rk_device.cuh"
#include "rk_internal.h"

namespace rk {
namespace {

constexpr int kThreads = 1024;
constexpr int kRun = 8;               // consecutive tokens of a thread
constexpr int kSharedOffsets = 8192;  // sequences whose offsets are searched in shared memory
constexpr float kQuantum = 0x1p-42f;
constexpr float kInfinite = 0x1p20f;

enum Flag : unsigned { kPlusInf = 1, kMinusInf = 2, kNaN = 4 };

struct Sequence {
    unsigned long long hi, lo;  // sum of the tokens' fixed-point words
    double s;
    float coef;                 // d (sum of losses) / d logp of each of its tokens
    int count;                  // active tokens
    unsigned flags;
    int pairs, first, last;     // how many times pairs name it, and the range they are in
};

struct Args {
    const float *logp, *ref;  // ref may be NULL
    const int64_t *targets;
    const int32_t *cu;
    int32_t Q;
    int64_t T;
    const int32_t *chosen, *rejected;
    int32_t P;
    const float *margin;  // or NULL
    int32_t kind, average;
    float beta, smoothing, scale;
    float *loss, *grad, *logratio;  // logratio may be NULL
    Sequence *seq;
    float *slope;  // [P] scale f'(d)
    unsigned *err;
};

// ---- steps; thread `i` of `n` ----

__device__ void step_clear(const Args &a, int64_t i, int64_t n) {
    for (int64_t q = i; q < a.Q; q += n) {
        Sequence z{};
        z.first = 0x7fffffff;
        z.last = -1;
        a.seq[q] = z;
        const int32_t b = a.cu[q], e = a.cu[q + 1];
        if (b < 0 || e < b || e > a.T) atomicOr(a.err, kErrRules);
    }
}

// The last sequence that begins at or before token t (-1: none); cu[0 .. Q] ascends.
__device__ __forceinline__ int sequence_of(const int32_t *cu, int Q, int64_t t) {
    int lo = 0, hi = Q;  // cu[lo - 1] <= t < cu[hi]
    while (lo < hi) {
        const int mid = (lo + hi) >> 1;
        if (cu[mid] <= t)
            lo = mid + 1;
        else
            hi = mid;
    }
    return lo - 1;
}

// Tokens t .. t + kRun - 1 of a thread: values, zeros past T.
template <typename T, typename V>
__device__ __forceinline__ void load_run(const T *p, int64_t t, int64_t n, bool vec, T fill, T (&v)[kRun]) {
    constexpr int kPer = 16 / sizeof(T);
    if (vec && t + kRun <= n) {
#pragma unroll
        for (int j = 0; j < kRun / kPer; ++j) {
            const V w = reinterpret_cast<const V *>(p + t)[j];
            const T *x = reinterpret_cast<const T *>(&w);
#pragma unroll
            for (int k = 0; k < kPer; ++k) v[j * kPer + k] = x[k];
        }
    } else {
#pragma unroll
        for (int j = 0; j < kRun; ++j) v[j] = t + j < n ? p[t + j] : fill;
    }
}

__device__ __forceinline__ bool aligned16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0; }

// Adds a thread's share of sequence q's sums.
__device__ __forceinline__ void add_to(const Args &a, int q, unsigned long long hi, unsigned long long lo, int count,
                                       unsigned flags) {
    if (count == 0) return;
    Sequence &s = a.seq[q];
    atomicAdd(&s.hi, hi);
    atomicAdd(&s.lo, lo);
    atomicAdd(&s.count, count);
    if (flags) atomicOr(&s.flags, flags);
}

__device__ void step_sums(const Args &a, const int32_t *cu, int64_t i, int64_t n) {
    const bool vec = aligned16(a.logp) && aligned16(a.targets) && (!a.ref || aligned16(a.ref));
    const int lane = threadIdx.x & 31;
    const int64_t runs = (a.T + kRun - 1) / kRun;
    // whole warps stay in the loop: i - lane is the warp's first run
    for (int64_t run = i; run - lane < runs; run += n) {
        const int64_t t = run * kRun;
        int64_t tg[kRun];
        float lp[kRun], rf[kRun];
        load_run<int64_t, longlong2>(a.targets, t, a.T, vec, -1, tg);
        load_run<float, float4>(a.logp, t, a.T, vec, 0.f, lp);
        if (a.ref) load_run<float, float4>(a.ref, t, a.T, vec, 0.f, rf);
        int q = sequence_of(cu, a.Q, t);
        int64_t end = q < 0 ? cu[0] : q < a.Q ? cu[q + 1] : a.T;  // where the next sequence begins
        unsigned long long hi = 0, lo = 0;
        int count = 0;
        unsigned flags = 0;
#pragma unroll
        for (int j = 0; j < kRun; ++j) {
            if (t + j >= end && q < a.Q) {  // a sequence begins inside the run
                add_to(a, q, hi, lo, count, flags);
                hi = lo = 0;
                count = 0;
                flags = 0;
                while (q < a.Q && t + j >= end) {
                    ++q;
                    end = q < a.Q ? cu[q + 1] : a.T;
                }
            }
            if (q < 0 || q >= a.Q || tg[j] < 0) continue;
            ++count;
            const float x = lp[j], y = a.ref ? rf[j] : 0.f;
            if (fabsf(x) < kInfinite && fabsf(y) < kInfinite) {
                const long long v = __float2ll_rn(x * (1.f / kQuantum)) - __float2ll_rn(y * (1.f / kQuantum));
                hi += (unsigned long long)(v >> 32);
                lo += (unsigned long long)v & 0xffffffffull;
            } else {
                const float d = (fabsf(x) < kInfinite ? 0.f : copysignf(INFINITY, x)) -
                                (fabsf(y) < kInfinite ? 0.f : copysignf(INFINITY, y));
                flags |= x != x || y != y || d != d ? kNaN : d > 0.f ? kPlusInf : kMinusInf;
            }
        }
        // the lanes' last sequences, added up from lane to lane where they are the same
        if (q < 0 || q >= a.Q) count = 0, hi = lo = 0, flags = 0;
        const int before = __shfl_up_sync(0xffffffffu, q, 1);
#pragma unroll
        for (int off = 1; off < 32; off <<= 1) {
            const int oq = __shfl_down_sync(0xffffffffu, q, off);
            const unsigned long long oh = __shfl_down_sync(0xffffffffu, hi, off);
            const unsigned long long ol = __shfl_down_sync(0xffffffffu, lo, off);
            const int oc = __shfl_down_sync(0xffffffffu, count, off);
            const unsigned of = __shfl_down_sync(0xffffffffu, flags, off);
            if (lane + off < 32 && oq == q) {
                hi += oh;
                lo += ol;
                count += oc;
                flags |= of;
            }
        }
        if (lane == 0 || before != q) add_to(a, q, hi, lo, count, flags);
    }
}

__device__ void step_ratios(const Args &a, int64_t i, int64_t n) {
    for (int64_t q = i; q < a.Q; q += n) {
        Sequence &s = a.seq[q];
        const long long hi = (long long)__ldcg(&s.hi);
        const unsigned long long lo = __ldcg(&s.lo);
        const int count = __ldcg(&s.count);
        const unsigned flags = __ldcg(&s.flags);
        double v = ((double)hi * 0x1p32 + (double)lo) * (double)kQuantum;
        if (a.average && count > 1) v /= (double)count;
        if (flags) v = flags == kPlusInf ? INFINITY : flags == kMinusInf ? -INFINITY : __longlong_as_double(0x7ff8000000000000ll);
        s.s = v;
        if (a.logratio) a.logratio[q] = (float)v;
    }
}

__device__ void step_pairs(const Args &a, int64_t i, int64_t n) {
    for (int64_t p = i; p < a.P; p += n) {
        const int c = a.chosen[p], r = a.rejected[p];
        float loss = 0.f, slope = 0.f;
        if (c >= a.Q || r >= a.Q) {
            atomicOr(a.err, kErrRules);
            loss = __int_as_float(0x7fc00000);
        } else if (c >= 0 && r >= 0) {
            double d = __ldcg(&a.seq[c].s) - __ldcg(&a.seq[r].s);
            if (a.margin) d -= (double)a.margin[p];
            if (a.kind == RK_PREFERENCE_IPO) {
                const double gap = d - 0.5 / (double)a.beta;
                loss = (float)(gap * gap);
                slope = (float)(2.0 * gap);
            } else {
                // x = beta d as a rounded number and what is left of it
                const double wide = (double)a.beta * d;
                const float x = (float)wide, rest = fabsf(x) < INFINITY ? (float)(wide - (double)x) : 0.f;
                if (a.kind == RK_PREFERENCE_HINGE) {
                    const float gap = (1.f - x) - rest;
                    loss = gap > 0.f || gap != gap ? gap : 0.f;
                    slope = wide < 1.0 ? -a.beta : wide != wide ? x : 0.f;
                } else {
                    // e = exp(-|x|): softplus(+-x) = max(+-x, 0) + log1p(e), sigmoid(|x|) = 1 / (1 + e)
                    const float sign = x < 0.f ? -1.f : 1.f;
                    const float m = expf(-fabsf(x)), e = m - m * (sign * rest);
                    const float tail = log1pf(e), minor = e / (1.f + e), major = 1.f / (1.f + e);
                    const float up = x < 0.f ? minor : major, down = x < 0.f ? major : minor;
                    const float keep = 1.f - a.smoothing;
                    loss = tail;
                    if (x < 0.f && keep > 0.f) loss += keep * -(x + rest);
                    if (x > 0.f && a.smoothing > 0.f) loss += a.smoothing * (x + rest);
                    if (x != x) loss = x;
                    slope = a.beta * (a.smoothing * up - keep * down);
                }
            }
            loss *= a.scale;
            slope *= a.scale;
            for (int side = 0; side < 2; ++side) {
                Sequence &s = a.seq[side ? r : c];
                atomicAdd(&s.pairs, 1);
                atomicMin(&s.first, (int)p);
                atomicMax(&s.last, (int)p);
            }
        }
        a.loss[p] = loss;
        a.slope[p] = slope;
    }
}

// A warp per sequence: its pairs' slopes in ascending order.
__device__ void step_coefs(const Args &a, int64_t i, int64_t n) {
    const int lane = threadIdx.x & 31;
    for (int64_t q = i >> 5; q < a.Q; q += n >> 5) {
        Sequence &s = a.seq[q];
        const int pairs = __ldcg(&s.pairs), first = __ldcg(&s.first), last = __ldcg(&s.last);
        float sum = 0.f;
        if (pairs > 0) {
            for (int64_t p0 = first; p0 <= last; p0 += 32) {
                const int64_t p = p0 + lane;
                int c = -1, r = -1;
                float slope = 0.f;
                if (p <= last) {
                    c = a.chosen[p];
                    r = a.rejected[p];
                    slope = __ldcg(&a.slope[p]);
                    if (c < 0 || r < 0 || c >= a.Q || r >= a.Q) c = r = -1;
                }
                const float mine = (c == q ? slope : 0.f) - (r == q ? slope : 0.f);
                unsigned named = __ballot_sync(0xffffffffu, c == q || r == q);
                for (; named; named &= named - 1)
                    sum = __fadd_rn(sum, __shfl_sync(0xffffffffu, mine, __ffs((int)named) - 1));
            }
            const int count = __ldcg(&s.count);
            if (a.average && count > 1) sum = __fdiv_rn(sum, (float)count);
        }
        if (lane == 0) s.coef = sum;
    }
}

__device__ void step_grads(const Args &a, const int32_t *cu, int64_t i, int64_t n) {
    const bool vec = aligned16(a.targets) && aligned16(a.grad);
    const int64_t runs = (a.T + kRun - 1) / kRun;
    for (int64_t run = i; run < runs; run += n) {
        const int64_t t = run * kRun;
        int64_t tg[kRun];
        load_run<int64_t, longlong2>(a.targets, t, a.T, vec, -1, tg);
        int q = sequence_of(cu, a.Q, t);
        int64_t end = q < 0 ? cu[0] : q < a.Q ? cu[q + 1] : a.T;
        float coef = q >= 0 && q < a.Q ? __ldcg(&a.seq[q].coef) : 0.f;
        float g[kRun];
#pragma unroll
        for (int j = 0; j < kRun; ++j) {
            if (t + j >= end && q < a.Q) {
                while (q < a.Q && t + j >= end) {
                    ++q;
                    end = q < a.Q ? cu[q + 1] : a.T;
                }
                coef = q < a.Q ? __ldcg(&a.seq[q].coef) : 0.f;
            }
            g[j] = tg[j] >= 0 ? coef : 0.f;
        }
        if (vec && t + kRun <= a.T) {
            put8(a.grad + t, g);
        } else {
#pragma unroll
            for (int j = 0; j < kRun; ++j)
                if (t + j < a.T) a.grad[t + j] = g[j];
        }
    }
}

enum Step { kClear, kSums, kRatios, kPairs, kCoefs, kGrads, kAll };

// Steps that read what other threads wrote have a barrier, or a launch, before them.
template <int STEP>
__global__ void __launch_bounds__(kThreads) preference_kernel(const __grid_constant__ Args a) {
    __shared__ int32_t offsets[kSharedOffsets + 1];
    wait_prior_grid();
    const int64_t n = (int64_t)gridDim.x * kThreads, i = (int64_t)blockIdx.x * kThreads + threadIdx.x;
    const int32_t *cu = a.cu;
    if ((STEP == kAll || STEP == kSums || STEP == kGrads) && a.Q <= kSharedOffsets) {
        for (int q = threadIdx.x; q <= a.Q; q += kThreads) offsets[q] = a.cu[q];
        cu = offsets;
        __syncthreads();
    }
    if (STEP == kAll || STEP == kClear) step_clear(a, i, n);
    if (STEP == kAll) cluster_sync();
    if (STEP == kAll || STEP == kSums) step_sums(a, cu, i, n);
    if (STEP == kAll) cluster_sync();
    if (STEP == kAll || STEP == kRatios) step_ratios(a, i, n);
    if (STEP == kAll) cluster_sync();
    if (STEP == kAll || STEP == kPairs) step_pairs(a, i, n);
    if (STEP == kAll) cluster_sync();
    if (STEP == kAll || STEP == kCoefs) step_coefs(a, i, n);
    if (STEP == kAll) cluster_sync();
    if (STEP == kAll || STEP == kGrads) step_grads(a, cu, i, n);
}

constexpr int kMaxCluster = 16;
constexpr int64_t kClusterTokens = int64_t(1) << 20;

size_t round256(size_t b) { return (b + 255) / 256 * 256; }

int64_t blocks_for(int64_t threads) { return (threads + kThreads - 1) / kThreads; }

template <int STEP>
cudaError_t launch_step(const Args &a, int64_t threads, const DeviceInfo &di, cudaStream_t st) {
    const int64_t grid = std::min(std::max<int64_t>(1, blocks_for(threads)), (int64_t)di.sm_count * 2);
    return launch_dependent(preference_kernel<STEP>, grid, kThreads, st, a);
}

cudaError_t launch_cluster(const Args &a, const DeviceInfo &di, cudaStream_t st) {
    auto *kernel = preference_kernel<kAll>;
    static std::atomic<uint64_t> allowed{0};
    const uint64_t bit = uint64_t(1) << di.device;
    if (!(allowed.load(std::memory_order_relaxed) & bit)) {
        const cudaError_t e = cudaFuncSetAttribute(reinterpret_cast<const void *>(kernel),
                                                   cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
        if (e != cudaSuccess) return e;
        allowed.fetch_or(bit, std::memory_order_relaxed);
    }
    const int64_t need = blocks_for(std::max({(a.T + kRun - 1) / kRun, (int64_t)a.Q, (int64_t)a.P}));
    int size = 1;
    while (size < kMaxCluster && size < need) size *= 2;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(size);
    cfg.blockDim = dim3(kThreads);
    cfg.stream = st;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = size;
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[1].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    return cudaLaunchKernelEx(&cfg, kernel, a);
}

}  // namespace

size_t preference_workspace_bytes(int64_t num_seqs, int64_t P) {
    return round256((size_t)num_seqs * sizeof(Sequence)) + round256((size_t)P * 4);
}

cudaError_t launch_preference(const float *logp, const float *ref, const int64_t *targets, const int32_t *cu,
                              int num_seqs, int64_t T, const int32_t *chosen, const int32_t *rejected, int64_t P,
                              const float *margin, int kind, float beta, float smoothing, bool average, float scale,
                              float *loss, float *grad, float *logratio, void *workspace, const DeviceInfo &di,
                              cudaStream_t st) {
    Args a{logp, ref, targets, cu, num_seqs, T, chosen, rejected, (int32_t)P, margin, kind, (int32_t)average, beta,
           smoothing, scale, loss, grad, logratio, static_cast<Sequence *>(workspace),
           reinterpret_cast<float *>(static_cast<char *>(workspace) + round256((size_t)num_seqs * sizeof(Sequence))),
           di.err};
    if (T <= kClusterTokens && num_seqs <= kSharedOffsets && P <= kClusterTokens / kRun)
        return launch_cluster(a, di, st);
    const int64_t runs = (T + kRun - 1) / kRun;
    cudaError_t e = launch_step<kClear>(a, num_seqs, di, st);
    if (e == cudaSuccess) e = launch_step<kSums>(a, runs, di, st);
    if (e == cudaSuccess) e = launch_step<kRatios>(a, num_seqs, di, st);
    if (e == cudaSuccess) e = launch_step<kPairs>(a, P, di, st);
    if (e == cudaSuccess) e = launch_step<kCoefs>(a, (int64_t)num_seqs * 32, di, st);
    if (e == cudaSuccess) e = launch_step<kGrads>(a, runs, di, st);
    return e;
}

}  // namespace rk
