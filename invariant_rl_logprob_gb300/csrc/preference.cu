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
// Bound by latency: 12 to 16 bytes a token, and results that wait for one another
// (sums, pairs, gradients).  Where a thread has at most one run of tokens and one
// pair, one cluster of up to 16 blocks does all of it with the hardware's cluster
// barrier between the steps, and every thread keeps its run and its pair in
// registers; beyond, every step is a launch of its own over the whole device.  The
// launches are what a caller waits for: at 131072 tokens the cluster takes 13.9 us
// on the device and one launch, the steps 10.4 us and four, some 9 us more on the
// host.  8 sequences of 128 tokens take 8.0 us, 512 of 1024 14.1, 1024 17.3.
//
// The sums are integers, so that no order of tokens, blocks or atomic additions
// can change a bit: a logprob is rounded to a multiple of 2^-42 (logprobs of
// 2^-18 and more have no smaller bits) and added in two words.  A magnitude of
// 2^20 and more, which no probability of interest has, counts as infinite.
#include <algorithm>
#include <cmath>

#include "elements.cuh"
#include "rk_device.cuh"
#include "rk_internal.h"

namespace rk {
namespace {

constexpr int kThreads = 1024;      // of a cluster's block
constexpr int kStepThreads = 256;   // of the steps as launches: over as many SMs as there are
constexpr int kRun = 8;               // consecutive tokens of a thread
constexpr int kSharedOffsets = 8192;  // sequences whose offsets are searched in shared memory
constexpr float kQuantum = 0x1p-42f;
constexpr float kInfinite = 0x1p20f;
constexpr float kFixed = 0x1p18f;  // what is below it is compared in fixed point

enum Flag : unsigned { kPlusInf = 1, kMinusInf = 2, kNaN = 4 };

struct Sequence {
    unsigned long long hi, lo;  // sum of the tokens' fixed-point words
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
    long long middle;  // 1 / (2 beta) as a multiple of 2^-42, unless it is kFixed and more
    int32_t middle_far;
    float *loss, *grad, *logratio;  // logratio may be NULL
    Sequence *seq;
    float *slope;  // [P] scale f'(d)
    unsigned *err;
};

__device__ __forceinline__ bool aligned16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0; }

// Elements t .. t + kRun - 1 of p, `fill` past n.
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

// ---- a thread's tokens ----

struct Run {
    int64_t t;      // the first one
    unsigned live;  // a bit for each that is active
    int q;          // the last sequence that begins at or before it (-1: none, Q: behind the last)
    int64_t end;    // where the next one begins

    __device__ __forceinline__ void load_targets(const Args &a, int64_t run) {
        t = run * kRun;
        int64_t tg[kRun];
        load_run<int64_t, longlong2>(a.targets, t, a.T, aligned16(a.targets), -1, tg);
        live = 0;
#pragma unroll
        for (int j = 0; j < kRun; ++j) live |= (tg[j] >= 0 ? 1u : 0u) << j;
    }
    // The last sequence that begins at or before token u; cu[0 .. Q] ascends, and whatever it holds
    // q stays in range.
    __device__ __forceinline__ void find(const int32_t *cu, int Q, int64_t u) {
        int lo = 0, hi = Q;  // cu[lo - 1] <= u < cu[hi]
        while (lo < hi) {
            const int mid = (lo + hi) >> 1;
            if (cu[mid] <= u)
                lo = mid + 1;
            else
                hi = mid;
        }
        q = lo - 1;
        end = cu[q + 1];
    }
    // On to the sequence of token u, at or behind `end`.
    __device__ __forceinline__ void advance(const int32_t *cu, int Q, int64_t T, int64_t u) {
        if (++q < Q) end = cu[q + 1];
        if (q < Q && u >= end) find(cu, Q, u);  // over empty ones, however many
        if (q >= Q || u >= end) {
            q = Q;
            end = T;
        }
    }
};

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

// ---- steps ----

__device__ __forceinline__ void clear(const Args &a, int64_t q) {
    Sequence z{};
    z.first = 0x7fffffff;
    z.last = -1;
    a.seq[q] = z;
    const int32_t b = a.cu[q], e = a.cu[q + 1];
    if (b < 0 || e < b || e > a.T) atomicOr(a.err, kErrRules);
}

// A run's logprobs into their sequences' sums; by whole warps, of consecutive runs.
__device__ __forceinline__ void add_run(const Args &a, const int32_t *cu, Run run, const float (&lp)[kRun],
                                        const float (&rf)[kRun]) {
    const int lane = threadIdx.x & 31;
    unsigned long long hi = 0, lo = 0;
    int count = 0;
    unsigned flags = 0;
#pragma unroll
    for (int j = 0; j < kRun; ++j) {
        if (run.t + j >= run.end && run.q < a.Q) {  // a sequence begins inside the run
            add_to(a, run.q, hi, lo, count, flags);
            hi = lo = 0;
            count = 0;
            flags = 0;
            run.advance(cu, a.Q, a.T, run.t + j);
        }
        if (run.q < 0 || run.q >= a.Q || !(run.live >> j & 1u)) continue;
        ++count;
        const float x = lp[j], y = rf[j];
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
    const int q = run.q;
    const int before = __shfl_up_sync(0xffffffffu, q, 1);
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
        const int oq = __shfl_down_sync(0xffffffffu, q, off);
        const unsigned long long oh = __shfl_down_sync(0xffffffffu, hi, off);
        const unsigned long long ol = __shfl_down_sync(0xffffffffu, lo, off);
        const unsigned both = __shfl_down_sync(0xffffffffu, (unsigned)count << 3 | flags, off);
        if (lane + off < 32 && oq == q) {
            hi += oh;
            lo += ol;
            count += (int)(both >> 3);
            flags |= both & 7u;
        }
    }
    if (lane == 0 || before != q) add_to(a, q, hi, lo, count, flags);
}

struct Pair {
    int c, r;  // -1 both: none
    float margin;
    bool bad;
    __device__ __forceinline__ void load(const Args &a, int64_t p) {
        c = a.chosen[p];
        r = a.rejected[p];
        margin = a.margin ? a.margin[p] : 0.f;
        bad = c >= a.Q || r >= a.Q;
        if (bad || c < 0 || r < 0) c = r = -1;
    }
};

// Which pairs name a sequence.
__device__ __forceinline__ void name(const Args &a, const Pair &pair, int64_t p) {
    if (pair.bad) atomicOr(a.err, kErrRules);
    if (pair.c < 0) return;
    for (int side = 0; side < 2; ++side) {
        Sequence &s = a.seq[side ? pair.r : pair.c];
        atomicAdd(&s.pairs, 1);
        atomicMin(&s.first, (int)p);
        atomicMax(&s.last, (int)p);
    }
}

// A sequence's s as a multiple of 2^-42, where that is one: finite and below 2^18, so that the
// difference of two, a margin and 1 / (2 beta) fit into 63 bits.
struct Ratio {
    long long fixed;
    double wide;  // the value where it is none
    bool far;
    __device__ __forceinline__ float rounded() const { return far ? (float)wide : __ll2float_rn(fixed) * kQuantum; }
    __device__ __forceinline__ double value() const { return far ? wide : (double)fixed * (double)kQuantum; }
};

__device__ __forceinline__ Ratio ratio_of(const Args &a, int q) {
    const Sequence *s = a.seq + q;
    const unsigned long long lo = __ldcg(&s->lo);
    const long long hi = (long long)__ldcg(&s->hi) + (long long)(lo >> 32);
    const int count = __ldcg(&s->count);
    const unsigned flags = __ldcg(&s->flags);
    Ratio r{};
    const long long limit = 1ll << 28;  // of the high word: 2^28 * 2^32 * 2^-42 = 2^18
    if (flags == 0 && hi > -limit && hi < limit) {
        r.fixed = hi * (1ll << 32) + (long long)(lo & 0xffffffffull);
        if (a.average && count > 1) {
            const long long half = count / 2;  // to the nearest
            r.fixed = (r.fixed + (r.fixed < 0 ? -half : half)) / count;
        }
        return r;
    }
    r.far = true;
    r.wide = ((double)hi * 0x1p32 + (double)(lo & 0xffffffffull)) * (double)kQuantum;
    if (a.average && count > 1) r.wide /= (double)count;
    if (flags) r.wide = flags == kPlusInf ? INFINITY : flags == kMinusInf ? -INFINITY : __longlong_as_double(0x7ff8000000000000ll);
    return r;
}

// loss and f' of x = beta d, given as a rounded number and what is left of it.  (Here and in `compare`
// every product says whether it is fused with the sum that it goes into: both kernels have the same bits.)
__device__ __forceinline__ void lose(const Args &a, float x, float rest, float *loss, float *slope) {
    if (a.kind == RK_PREFERENCE_HINGE) {
        const float gap = (1.f - x) - rest;
        *loss = gap > 0.f || gap != gap ? gap : 0.f;
        *slope = gap > 0.f ? -a.beta : gap != gap ? gap : 0.f;
        return;
    }
    // e = exp(-|x|): softplus(+-x) = max(+-x, 0) + log1p(e), sigmoid(|x|) = 1 / (1 + e)
    const float sign = x < 0.f ? -1.f : 1.f;
    const float m = expf(-fabsf(x)), e = __fmaf_rn(-m, sign * rest, m);
    const float tail = log1pf(e), minor = e / (1.f + e), major = 1.f / (1.f + e);
    const float up = x < 0.f ? minor : major, down = x < 0.f ? major : minor;
    const float keep = 1.f - a.smoothing;
    *loss = tail;
    if (x < 0.f && keep > 0.f) *loss = __fmaf_rn(keep, -(x + rest), *loss);
    if (x > 0.f && a.smoothing > 0.f) *loss = __fmaf_rn(a.smoothing, x + rest, *loss);
    if (x != x) *loss = x;
    *slope = a.beta * __fmaf_rn(-keep, down, __fmul_rn(a.smoothing, up));
}

// Differences are exact in multiples of 2^-42; 64-bit floating point, of which this GPU does two a
// cycle and SM, is left to values that are none (1792 pairs by mean logprobs in it: 19 us).
__device__ __forceinline__ void compare(const Args &a, const Pair &pair, int64_t p) {
    float loss = pair.bad ? __int_as_float(0x7fc00000) : 0.f, slope = 0.f;
    if (pair.c >= 0) {
        const Ratio c = ratio_of(a, pair.c), r = ratio_of(a, pair.r);
        const bool ipo = a.kind == RK_PREFERENCE_IPO;
        if (!c.far && !r.far && fabsf(pair.margin) < kFixed && !(ipo && a.middle_far)) {
            long long d = c.fixed - r.fixed - __float2ll_rn(pair.margin * (1.f / kQuantum));
            if (ipo) d -= a.middle;
            const float top = __ll2float_rn(d), low = __ll2float_rn(d - __float2ll_rn(top));
            const float unit = (ipo ? 1.f : a.beta) * kQuantum;
            const float x = __fmul_rn(top, unit);
            const float rest = fabsf(x) < INFINITY ? __fmaf_rn(low, unit, __fmaf_rn(top, unit, -x)) : 0.f;
            if (ipo) {
                loss = __fmaf_rn(x, x, __fmul_rn(2.f * x, rest));
                slope = 2.f * (x + rest);
            } else {
                lose(a, x, rest, &loss, &slope);
            }
        } else {
            const double d = c.value() - r.value() - (double)pair.margin;
            if (ipo) {
                const double gap = d - 0.5 / (double)a.beta;
                loss = (float)(gap * gap);
                slope = (float)(2.0 * gap);
            } else {
                const double wide = __dmul_rn((double)a.beta, d);
                const float x = (float)wide;
                lose(a, x, fabsf(x) < INFINITY ? (float)(wide - (double)x) : 0.f, &loss, &slope);
            }
        }
        loss *= a.scale;
        slope *= a.scale;
    }
    a.loss[p] = loss;
    a.slope[p] = slope;
}

// d (sum of the losses) / d logp of sequence q's tokens: the slopes of its pairs in ascending order, which
// are looked for between the first and the last, once for each tile: 4096 sequences of 64 tokens in 14336
// pairs take 21 us with a sequence's pairs together and 445 with all of them shuffled.
__device__ __forceinline__ float share_of(const Args &a, const Sequence &s, float sum) {
    const int count = __ldcg(&s.count);
    return a.average && count > 1 ? __fdiv_rn(sum, (float)count) : sum;
}
__device__ __forceinline__ float slope_at(const Args &a, int q, int64_t p, bool *named) {
    Pair pair;
    pair.load(a, p);
    const float slope = __ldcg(&a.slope[p]);
    *named = pair.c == q || pair.r == q;
    return (pair.c == q ? slope : 0.f) - (pair.r == q ? slope : 0.f);
}
// By a warp.
__device__ __forceinline__ float gather(const Args &a, int q) {
    const int lane = threadIdx.x & 31;
    const Sequence &s = a.seq[q];
    const int pairs = __ldcg(&s.pairs), first = __ldcg(&s.first), last = __ldcg(&s.last);
    float sum = 0.f;
    for (int64_t p0 = first; pairs > 0 && p0 <= last; p0 += 32) {
        bool named = false;
        const float mine = p0 + lane <= last ? slope_at(a, q, p0 + lane, &named) : 0.f;
        for (unsigned m = __ballot_sync(0xffffffffu, named); m; m &= m - 1)
            sum = __fadd_rn(sum, __shfl_sync(0xffffffffu, mine, __ffs((int)m) - 1));
    }
    return share_of(a, s, sum);
}
// By a thread, where a tile has more sequences than there is room for.
__device__ __noinline__ float gather_alone(const Args &a, int q) {
    const Sequence &s = a.seq[q];
    const int pairs = __ldcg(&s.pairs), first = __ldcg(&s.first), last = __ldcg(&s.last);
    float sum = 0.f;
    for (int64_t p = first; pairs > 0 && p <= last; ++p) {
        bool named;
        const float mine = slope_at(a, q, p, &named);
        if (named) sum = __fadd_rn(sum, mine);
    }
    return share_of(a, s, sum);
}

constexpr int kTileSequences = 1024;

struct Tile {
    int first, last;  // sequences that the block's tokens belong to
    float coef[kTileSequences];
};

// The gradients of a block's runs; `mine`: this thread has one.
template <int THREADS>
__device__ __forceinline__ void write_runs(const Args &a, const int32_t *cu, Run run, bool mine, Tile &tile) {
    const bool end = mine && (run.t + kRun >= a.T || threadIdx.x == THREADS - 1);
    if (threadIdx.x == 0) tile.first = mine ? max(run.q, 0) : 0;
    if (threadIdx.x == 0 && !mine) tile.last = -1;
    if (end) {
        Run last = run;
        last.find(cu, a.Q, min(a.T, run.t + kRun) - 1);
        tile.last = last.q;
    }
    __syncthreads();
    const int first = tile.first, count = tile.last - first + 1;
    const bool near = count <= kTileSequences;
    if (near)
        for (int k = threadIdx.x >> 5; k < count; k += THREADS / 32) {
            const float c = gather(a, first + k);
            if ((threadIdx.x & 31) == 0) tile.coef[k] = c;
        }
    __syncthreads();
    if (!mine) return;
    // offsets that do not ascend may lead out of the tile
    const auto coef_of = [&](int q) {
        if (q < 0 || q >= a.Q) return 0.f;
        return near && q >= first && q < first + count ? tile.coef[q - first] : gather_alone(a, q);
    };
    float coef = coef_of(run.q), g[kRun];
#pragma unroll
    for (int j = 0; j < kRun; ++j) {
        if (run.t + j >= run.end && run.q < a.Q) {
            run.advance(cu, a.Q, a.T, run.t + j);
            coef = coef_of(run.q);
        }
        g[j] = run.live >> j & 1u ? coef : 0.f;
    }
    if (aligned16(a.grad) && run.t + kRun <= a.T) {
        put8(a.grad + run.t, g);
    } else {
#pragma unroll
        for (int j = 0; j < kRun; ++j)
            if (run.t + j < a.T) a.grad[run.t + j] = g[j];
    }
}

// ---- kernels ----

template <int THREADS>
__device__ __forceinline__ const int32_t *offsets_near(const Args &a, int32_t (&offsets)[kSharedOffsets + 1]) {
    if (a.Q > kSharedOffsets) return a.cu;
    for (int q = threadIdx.x; q <= a.Q; q += THREADS) offsets[q] = a.cu[q];
    __syncthreads();
    return offsets;
}

__device__ __forceinline__ void load_logprobs(const Args &a, int64_t t, float (&lp)[kRun], float (&rf)[kRun]) {
    load_run<float, float4>(a.logp, t, a.T, aligned16(a.logp), 0.f, lp);
    if (a.ref) {
        load_run<float, float4>(a.ref, t, a.T, aligned16(a.ref), 0.f, rf);
    } else {
#pragma unroll
        for (int j = 0; j < kRun; ++j) rf[j] = 0.f;
    }
}

// All steps by one cluster whose threads have at most one run, one sequence and one pair each.
__global__ void __launch_bounds__(kThreads) preference_cluster(const __grid_constant__ Args a) {
    __shared__ int32_t offsets[kSharedOffsets + 1];
    __shared__ Tile tile;
    wait_prior_grid();
    const int64_t i = (int64_t)blockIdx.x * kThreads + threadIdx.x;
    const int64_t runs = (a.T + kRun - 1) / kRun;
    const bool mine = i - (threadIdx.x & 31) < runs;  // whole warps
    Run run{};
    float lp[kRun], rf[kRun];
    Pair pair{-1, -1, 0.f, false};
    if (mine) {
        run.load_targets(a, i);
        load_logprobs(a, run.t, lp, rf);
    }
    if (i < a.P) pair.load(a, i);
    if (i < a.Q) clear(a, i);
    const int32_t *cu = offsets_near<kThreads>(a, offsets);
    if (mine) run.find(cu, a.Q, run.t);
    cluster_sync();
    if (mine) add_run(a, cu, run, lp, rf);
    if (i < a.P) name(a, pair, i);
    cluster_sync();
    if (i < a.P) compare(a, pair, i);
    if (i < a.Q && a.logratio) a.logratio[i] = ratio_of(a, (int)i).rounded();
    cluster_sync();
    write_runs<kThreads>(a, cu, run, i < runs, tile);
}

// The same steps as launches of their own.
enum Step { kClear, kSums, kPairs, kGrads };

template <int STEP>
__global__ void __launch_bounds__(kStepThreads) preference_step(const __grid_constant__ Args a) {
    wait_prior_grid();
    const int64_t n = (int64_t)gridDim.x * kStepThreads, i = (int64_t)blockIdx.x * kStepThreads + threadIdx.x;
    const int64_t runs = (a.T + kRun - 1) / kRun, warp_first = i - (threadIdx.x & 31);
    if constexpr (STEP == kClear) {
        for (int64_t q = i; q < a.Q; q += n) clear(a, q);
    } else if constexpr (STEP == kSums) {
        __shared__ int32_t offsets[kSharedOffsets + 1];
        const int32_t *cu = offsets_near<kStepThreads>(a, offsets);
        for (int64_t r = i, w = warp_first; w < runs; r += n, w += n) {
            Run run;
            float lp[kRun], rf[kRun];
            run.load_targets(a, r);
            load_logprobs(a, run.t, lp, rf);
            run.find(cu, a.Q, run.t);
            add_run(a, cu, run, lp, rf);
        }
        for (int64_t p = i; p < a.P; p += n) {
            Pair pair;
            pair.load(a, p);
            name(a, pair, p);
        }
    } else if constexpr (STEP == kPairs) {
        for (int64_t p = i; p < a.P; p += n) {
            Pair pair;
            pair.load(a, p);
            compare(a, pair, p);
        }
        if (a.logratio)
            for (int64_t q = i; q < a.Q; q += n) a.logratio[q] = ratio_of(a, (int)q).rounded();
    } else {
        __shared__ int32_t offsets[kSharedOffsets + 1];
        const int32_t *cu = offsets_near<kStepThreads>(a, offsets);
        __shared__ Tile tile;
        for (int64_t r = i, b = (int64_t)blockIdx.x * kStepThreads; b < runs; r += n, b += n) {
            Run run{};
            if (r < runs) {
                run.load_targets(a, r);
                run.find(cu, a.Q, run.t);
            }
            write_runs<kStepThreads>(a, cu, run, r < runs, tile);
            __syncthreads();
        }
    }
}

constexpr int kMaxCluster = 16;

size_t round256(size_t b) { return (b + 255) / 256 * 256; }

int64_t blocks_for(int64_t threads, int block) { return std::max<int64_t>(1, (threads + block - 1) / block); }

template <int STEP>
cudaError_t launch_step(const Args &a, int64_t threads, const DeviceInfo &di, cudaStream_t st) {
    return launch_dependent(preference_step<STEP>, std::min(blocks_for(threads, kStepThreads), (int64_t)di.sm_count * 4),
                            kStepThreads, st, a);
}

cudaError_t launch_cluster(const Args &a, int64_t blocks, const DeviceInfo &di, cudaStream_t st) {
    static std::atomic<uint64_t> allowed{0};
    const uint64_t bit = uint64_t(1) << di.device;
    if (!(allowed.load(std::memory_order_relaxed) & bit)) {
        const cudaError_t e = cudaFuncSetAttribute(reinterpret_cast<const void *>(preference_cluster),
                                                   cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
        if (e != cudaSuccess) return e;
        allowed.fetch_or(bit, std::memory_order_relaxed);
    }
    int size = 1;
    while (size < blocks) size *= 2;
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
    return cudaLaunchKernelEx(&cfg, preference_cluster, a);
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
    const double middle = 0.5 / (double)beta;
    const bool far = !(middle < (double)kFixed);
    const Args a{logp, ref, targets, cu, num_seqs, T, chosen, rejected, (int32_t)P, margin, kind, (int32_t)average, beta,
                 smoothing, scale, far ? 0 : std::llrint(middle / (double)kQuantum), (int32_t)far, loss, grad, logratio,
                 static_cast<Sequence *>(workspace),
                 reinterpret_cast<float *>(static_cast<char *>(workspace) + round256((size_t)num_seqs * sizeof(Sequence))),
                 di.err};
    const int64_t runs = (T + kRun - 1) / kRun, most = std::max({runs, (int64_t)num_seqs, P});
    const int64_t blocks = blocks_for(most, kThreads);
    if (blocks <= kMaxCluster && num_seqs <= kSharedOffsets) return launch_cluster(a, blocks, di, st);
    cudaError_t e = launch_step<kClear>(a, num_seqs, di, st);
    if (e == cudaSuccess) e = launch_step<kSums>(a, std::max(runs, P), di, st);
    if (e == cudaSuccess) e = launch_step<kPairs>(a, std::max<int64_t>(P, num_seqs), di, st);
    if (e == cudaSuccess) e = launch_step<kGrads>(a, runs, di, st);
    return e;
}

}  // namespace rk
