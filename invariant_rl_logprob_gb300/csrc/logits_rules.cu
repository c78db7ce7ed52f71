// logits_rules.cu -- logits under sampling rules: repetition, frequency and
// presence penalties, per-request biases, grammar masks and temperature (the
// definition stands at rk_logits_rules in rk.h), applied (kApply), scored
// (kLogp: selected logprob and log-sum-exp) and differentiated (kBwd).
//
// Decomposition.  A block works on a slice of kSliceCols columns and a run of
// consecutive rows; each of its warps owns a segment of kSegCols columns of
// that slice, and each lane kGroups groups of 8 columns of the segment (group
// g of the segment = columns [8g, 8g + 8); lane l owns groups l, l + 32, ...).
// For a lane's 32 columns a bit set tells which of them the rules touch
// (seen before, or biased); the others need the temperature and the mask only.
//
// History.  The block counts a request's tokens of its slice in shared
// memory (one word per column: bit 31 in the prompt, bits 0-30 times
// produced).  Integer atomics only, so the order does not matter.  Rows of
// one request with growing prefixes (a packed training sequence) add the new
// token or two to the counts they have: each lane then updates its own
// columns, without a barrier.  Any other change counts anew.
//
// Batch invariance: a row's partial (max, sum) of a segment is formed by a
// tree fixed by the column index alone, and the segments' partials are merged
// in a fixed order: nothing depends on T, on where the row sits or on how the
// rows were cut into runs.
#include <algorithm>

#include "rk_device.cuh"
#include "rk_internal.h"

namespace rk {
namespace {

constexpr int kGroups = 4;                    // groups of 8 columns per lane
constexpr int kSegCols = 32 * 8 * kGroups;    // 1024 columns per warp
constexpr int kWarps = 8;
constexpr int kThreads = 32 * kWarps;
constexpr int kSliceCols = kSegCols * kWarps;  // 8192 columns per block
constexpr int kMaxRun = 64;                    // rows per block at most
constexpr int kInlineTokens = 4;  // new tokens that lanes add on their own
constexpr uint32_t kPromptBit = 0x80000000u;

enum RulesOp { kApply, kLogp, kBwd };

struct RulesIo {
    const void *logits;
    int64_t ld;
    const int64_t *targets;
    const int32_t *cu;
    int num_seqs;
    int64_t T, V;
    int run;         // rows per block
    int vec_in;      // 16-byte loads of a group are aligned
    const float *lse, *grad;  // kBwd
    void *out;       // kApply, kBwd
    int64_t ld_out;
    int vec_out;
    float2 *part;    // kLogp: [T][segments] (max of y, sum relative to it)
    float *ytgt;     // kLogp: [T] y of the target, -inf when it is masked
    unsigned *err;
};

// What a row says about itself.  `ok` is false when an index is out of range.
struct RowInfo {
    int64_t tgt;
    int32_t req, len, mrow;
    bool active, ok;
};

template <RulesOp OP>
__device__ __forceinline__ RowInfo row_info(const RulesIo &io, const rk_logits_rules &r, int64_t t) {
    RowInfo i;
    i.tgt = (OP == kApply) ? 0 : io.targets[t];
    i.active = OP == kApply || row_active(t, i.tgt, io.cu, io.num_seqs);
    i.req = r.row_request ? r.row_request[t] : (r.num_requests > 0 ? (int32_t)t : 0);
    if (r.row_request && i.req == -1) i.active = false;
    i.len = r.row_length ? max(r.row_length[t], 0) : 0x7fffffff;
    i.mrow = r.mask ? (r.row_mask ? r.row_mask[t] : (int32_t)t) : -1;
    i.ok = (r.num_requests == 0 && !r.row_request) || (i.req >= 0 && i.req < r.num_requests) ||
           (r.num_requests == 0 && i.req >= 0);
    i.ok = i.ok && (i.mrow < 0 || i.mrow < r.mask_rows);
    return i;
}

// A request's parameters.
struct Request {
    float tau, itau;   // temperature and its reciprocal
    float rep, irep, freq, pres;
    const int64_t *tokens;
    int32_t ntok, prompt;
    int64_t bias0;
    int32_t nbias;
    bool ok;
};

__device__ __forceinline__ bool in_range(float v) { return v >= 1e-6f && v <= 1e6f; }

__device__ __forceinline__ Request load_request(const rk_logits_rules &r, int32_t q) {
    Request s;
    const bool any = r.num_requests > 0;
    s.tau = any && r.temperature ? r.temperature[q] : 1.f;
    s.rep = any && r.repetition ? r.repetition[q] : 1.f;
    s.freq = any && r.frequency ? r.frequency[q] : 0.f;
    s.pres = any && r.presence ? r.presence[q] : 0.f;
    s.itau = __frcp_rn(s.tau);
    s.irep = __frcp_rn(s.rep);
    s.ok = in_range(s.tau) && in_range(s.rep);
    s.tokens = nullptr;
    s.ntok = 0;
    s.prompt = 0;
    if (any && r.tokens) {
        const int64_t a = r.token_offsets[q], b = r.token_offsets[q + 1];
        if (a >= 0 && b >= a && b <= r.num_tokens && b - a < 0x7fffffff) {
            s.tokens = r.tokens + a;
            s.ntok = (int32_t)(b - a);
            s.prompt = r.prompt_lengths ? r.prompt_lengths[q] : 0;
        } else {
            s.ok = false;
        }
    }
    s.bias0 = 0;
    s.nbias = 0;
    if (any && r.bias_ids) {
        const int64_t a = r.bias_offsets[q], b = r.bias_offsets[q + 1];
        if (a >= 0 && b >= a && b <= r.num_bias && b - a < 0x7fffffff) {
            s.bias0 = a;
            s.nbias = (int32_t)(b - a);
        } else {
            s.ok = false;
        }
    }
    return s;
}

// y of a touched column from z, its count word and its bias.
__device__ __forceinline__ float rule_y(float z, uint32_t w, float bias, const Request &q) {
    float y = z;
    if (w) y = __fmul_rn(z, z > 0.f ? q.irep : q.rep);
    const uint32_t n = w & ~kPromptBit;
    if (n) y = __fsub_rn(y, __fmaf_rn(q.freq, (float)n, q.pres));
    return __fadd_rn(y, bias);
}

__device__ __forceinline__ float load_elem(const uint16_t *p) { return bf16_bits_to_f32(*p); }
__device__ __forceinline__ float load_elem(const float *p) { return *p; }

// One group of 8 columns; columns without a bit in `live` are not read.
__device__ __forceinline__ void load_group(const uint16_t *p, bool vec, uint32_t live, float (&z)[8]) {
    if (vec && live == 0xffu) {
        const uint4 w = reinterpret_cast<const uint4 *>(p)[0];
        const uint32_t q[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            z[2 * j] = bf16_lo(q[j]);
            z[2 * j + 1] = bf16_hi(q[j]);
        }
    } else {
#pragma unroll
        for (int j = 0; j < 8; ++j) z[j] = (live >> j & 1u) ? load_elem(p + j) : -INFINITY;
    }
}
__device__ __forceinline__ void load_group(const float *p, bool vec, uint32_t live, float (&z)[8]) {
    if (vec && live == 0xffu) {
        const float4 a = reinterpret_cast<const float4 *>(p)[0];
        const float4 b = reinterpret_cast<const float4 *>(p)[1];
        z[0] = a.x; z[1] = a.y; z[2] = a.z; z[3] = a.w;
        z[4] = b.x; z[5] = b.y; z[6] = b.z; z[7] = b.w;
    } else {
#pragma unroll
        for (int j = 0; j < 8; ++j) z[j] = (live >> j & 1u) ? load_elem(p + j) : -INFINITY;
    }
}

__device__ __forceinline__ void store_elem(uint16_t *p, float v) {
    *p = (uint16_t)(pack_bf16x2(v, 0.f) & 0xffffu);
}
__device__ __forceinline__ void store_elem(float *p, float v) { *p = v; }

// One group of 8 columns; columns without a bit in `inside` are not written.
__device__ __forceinline__ void store_group(uint16_t *p, bool vec, uint32_t inside, const float (&x)[8]) {
    if (vec && inside == 0xffu) {
        *reinterpret_cast<uint4 *>(p) = make_uint4(pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3]),
                                                   pack_bf16x2(x[4], x[5]), pack_bf16x2(x[6], x[7]));
    } else {
#pragma unroll
        for (int j = 0; j < 8; ++j)
            if (inside >> j & 1u) store_elem(p + j, x[j]);
    }
}
__device__ __forceinline__ void store_group(float *p, bool vec, uint32_t inside, const float (&x)[8]) {
    if (vec && inside == 0xffu) {
        reinterpret_cast<float4 *>(p)[0] = make_float4(x[0], x[1], x[2], x[3]);
        reinterpret_cast<float4 *>(p)[1] = make_float4(x[4], x[5], x[6], x[7]);
    } else {
#pragma unroll
        for (int j = 0; j < 8; ++j)
            if (inside >> j & 1u) store_elem(p + j, x[j]);
    }
}

// exp(y / temperature - lse), 1 / temperature = itau + i1.  -inf stays out of
// the product with i1, whose sign it would take.
__device__ __forceinline__ float prob(float y, float itau, float i1, float lse) {
    const float v = y < -3.3e38f ? -3.3e38f : y;
    return ex2(__fmul_rn(__fmaf_rn(v, i1, __fmaf_rn(v, itau, -lse)), kLog2e));
}

__device__ __forceinline__ float warp_max(float v) {
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, off));
    return v;
}
__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) v = __fadd_rn(v, __shfl_xor_sync(0xffffffffu, v, off));
    return v;
}

// Shared memory: the slice's count words, its bias values when there are
// biases, and per lane the touched bits.
struct Shared {
    uint32_t *count;    // [kSliceCols]
    int32_t *bias;    // [kSliceCols], or null: first 1 + entry index, then the value's bits
    uint32_t *touched;  // [kThreads]
};

// Sets a slice column's touched bit (any thread).
__device__ __forceinline__ void mark(const Shared &sh, int c) {
    const int g = (c & (kSegCols - 1)) >> 3;
    atomicOr(&sh.touched[(c / kSegCols) * 32 + (g & 31)], 1u << ((g >> 5) * 8 + (c & 7)));
}

// The column of a segment that bit k of a lane stands for.
__device__ __forceinline__ int lane_column(int lane, int k) {
    return 8 * (lane + 32 * (k >> 3)) + (k & 7);
}

// Block-wide: tokens [from, to) of the request into the counts of columns
// [slice0, slice0 + width).
__device__ __forceinline__ void count_tokens(const Shared &sh, const Request &q, int32_t from,
                                             int32_t to, int64_t slice0, int width) {
    for (int32_t i = from + (int32_t)threadIdx.x; i < to; i += kThreads) {
        const int64_t c = q.tokens[i] - slice0;
        if (c >= 0 && c < width) {
            if (i < q.prompt)
                atomicOr(&sh.count[c], kPromptBit);
            else
                atomicAdd(&sh.count[c], 1u);
            mark(sh, (int)c);
        }
    }
}

template <RulesOp OP, typename TIn, typename TOut>
__global__ void __launch_bounds__(kThreads)
    rules_kernel(const __grid_constant__ RulesIo io, const __grid_constant__ rk_logits_rules rules) {
    extern __shared__ uint4 smem[];
    Shared sh;
    sh.count = reinterpret_cast<uint32_t *>(smem);
    sh.touched = sh.count + kSliceCols;
    sh.bias = rules.bias_ids ? reinterpret_cast<int32_t *>(sh.touched + kThreads) : nullptr;
    // Launched with programmatic stream serialisation: wait until the previous
    // kernel of the stream has completed before reading or writing anything.
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");

    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int64_t slices = (io.V + kSliceCols - 1) / kSliceCols;
    const int64_t slice0 = (int64_t)(blockIdx.x % slices) * kSliceCols;
    const int width = (int)min((int64_t)kSliceCols, io.V - slice0);
    const int64_t seg0 = slice0 + (int64_t)warp * kSegCols;
    const int64_t nseg = (io.V + kSegCols - 1) / kSegCols;
    const int64_t t0 = (int64_t)(blockIdx.x / slices) * io.run;
    const int64_t t1 = min(io.T, t0 + io.run);
    const bool first_thread = slice0 == 0 && threadIdx.x == 0;

    // this lane's columns that exist
    uint32_t inside = 0;
#pragma unroll
    for (int i = 0; i < kGroups; ++i) {
        const int64_t left = io.V - (seg0 + 8 * (lane + 32 * i));
        inside |= (left >= 8 ? 0xffu : left > 0 ? (1u << left) - 1u : 0u) << (8 * i);
    }
    const int64_t words = (io.V + 31) / 32;

    int32_t cur = -1, counted = 0;
    uint32_t touched = 0;
    Request q{};
    for (int64_t t = t0; t < t1; ++t) {
        const RowInfo row = row_info<OP>(io, rules, t);
        TOut *orow = reinterpret_cast<TOut *>(io.out) + t * io.ld_out;
        bool ok = row.ok && (OP == kApply || row.tgt < io.V);
        if (row.active && row.ok) {
            const bool other = row.req != cur;
            if (other) {
                q = load_request(rules, row.req);
                cur = row.req;
            }
            const int32_t len = min(row.len, q.ntok);
            if (q.ok && (other || len < counted)) {  // count from the start
                __syncthreads();
                for (int k = threadIdx.x; k < kSliceCols / 4; k += kThreads)
                    reinterpret_cast<uint4 *>(sh.count)[k] = make_uint4(0, 0, 0, 0);
                if (sh.bias)
                    for (int k = threadIdx.x; k < kSliceCols / 4; k += kThreads)
                        reinterpret_cast<uint4 *>(sh.bias)[k] = make_uint4(0, 0, 0, 0);
                sh.touched[threadIdx.x] = 0;
                __syncthreads();
                for (int k = threadIdx.x; k < q.nbias; k += kThreads) {
                    const int64_t c = rules.bias_ids[q.bias0 + k] - slice0;
                    if (c >= 0 && c < width) {
                        atomicMax(&sh.bias[c], k + 1);
                        mark(sh, (int)c);
                    }
                }
                count_tokens(sh, q, 0, len, slice0, width);
                __syncthreads();
                touched = sh.touched[threadIdx.x];
                if (sh.bias)  // entry indices to values, by each column's lane
                    for (uint32_t b = touched; b; b &= b - 1) {
                        int32_t *p = &sh.bias[warp * kSegCols + lane_column(lane, __ffs(b) - 1)];
                        if (*p > 0) *p = __float_as_int(rules.bias_values[q.bias0 + *p - 1]);
                    }
            } else if (q.ok && len - counted <= kInlineTokens) {  // each lane its own columns
                for (int32_t i = counted; i < len; ++i) {
                    const int64_t c = q.tokens[i] - seg0;
                    if (c >= 0 && c < kSegCols && seg0 + c < io.V && ((c >> 3) & 31) == lane) {
                        uint32_t *w = &sh.count[warp * kSegCols + c];
                        *w = i < q.prompt ? (*w | kPromptBit) : *w + 1u;
                        touched |= 1u << ((c >> 8) * 8 + (c & 7));
                    }
                }
            } else if (q.ok) {  // add the new tokens
                __syncthreads();
                sh.touched[threadIdx.x] = touched;
                __syncthreads();
                count_tokens(sh, q, counted, len, slice0, width);
                __syncthreads();
                touched = sh.touched[threadIdx.x];
            }
            if (q.ok) counted = len;
            ok = ok && q.ok;
        }
        if (!row.active) {
            if (OP == kBwd) {
                const float zero[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
#pragma unroll
                for (int i = 0; i < kGroups; ++i)
                    store_group(orow + seg0 + 8 * (lane + 32 * i), io.vec_out, inside >> (8 * i) & 0xffu,
                                zero);
            }
            continue;
        }
        if (!ok) {
            const float nan = __int_as_float(0x7fc00000);
            if (first_thread)
                atomicOr(io.err, OP != kApply && row.tgt >= io.V ? kErrTargetRange : kErrRules);
            if (OP == kLogp) {
                if (lane == 0 && seg0 < io.V) io.part[t * nseg + seg0 / kSegCols] = make_float2(0.f, nan);
                if (first_thread) io.ytgt[t] = nan;
            } else {
                const float x[8] = {nan, nan, nan, nan, nan, nan, nan, nan};
#pragma unroll
                for (int i = 0; i < kGroups; ++i)
                    store_group(orow + seg0 + 8 * (lane + 32 * i), io.vec_out, inside >> (8 * i) & 0xffu,
                                x);
            }
            continue;
        }

        // this lane's columns that the mask allows
        uint32_t live = inside;
        if (row.mrow >= 0) {
            const uint8_t *m = reinterpret_cast<const uint8_t *>(rules.mask + (int64_t)row.mrow * words);
            uint32_t allowed = 0;
#pragma unroll
            for (int i = 0; i < kGroups; ++i)
                if (inside >> (8 * i) & 0xffu)
                    allowed |= (uint32_t)m[(seg0 >> 3) + lane + 32 * i] << (8 * i);
            live &= allowed;
        }
        const TIn *zrow = reinterpret_cast<const TIn *>(io.logits) + t * io.ld;
        float z[kGroups][8];
#pragma unroll
        for (int i = 0; i < kGroups; ++i)
            load_group(zrow + seg0 + 8 * (lane + 32 * i), io.vec_in, inside >> (8 * i) & 0xffu, z[i]);

        const uint32_t special = touched & live;
        if (OP == kLogp) {
            const float c = __fmul_rn(kLog2e, q.itau);
            // untouched columns: one maximum, then the terms relative to it
            const uint32_t plain = live & ~touched;
            float m = -INFINITY;
#pragma unroll
            for (int i = 0; i < kGroups; ++i)
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    if (!(plain >> (8 * i + j) & 1u)) z[i][j] = -INFINITY;
                    m = fmaxf(m, z[i][j]);
                }
            // touched columns: running maximum and sum, in column order
            float mt = -INFINITY, st = 0.f;
            const int64_t tc = row.tgt - seg0;
            const bool mine = tc >= 0 && tc < kSegCols && ((tc >> 3) & 31) == lane;
            const int tbit = mine ? (int)((tc >> 8) * 8 + (tc & 7)) : -1;
            float yt = -INFINITY;
            uint32_t b = special;
            while (b) {
                const int k = __ffs(b) - 1;
                b &= b - 1;
                const int sc = warp * kSegCols + lane_column(lane, k);
                const float y = rule_y(load_elem(zrow + slice0 + sc), sh.count[sc],
                                       sh.bias ? __int_as_float(sh.bias[sc]) : 0.f, q);
                if (k == tbit) yt = y;
                if (y == -INFINITY) continue;  // banned by its bias
                if (y > mt) {
                    st = __fadd_rn(__fmul_rn(st, ex2(__fmul_rn(__fsub_rn(mt, y), c))),
                                   ex2(__fmul_rn(__fsub_rn(y, y), c)));  // 1, or NaN for inf
                    mt = y;
                } else {
                    st = __fadd_rn(st, ex2(__fmul_rn(__fsub_rn(y, mt), c)));
                }
            }
            if (mine && (plain >> tbit & 1u)) yt = load_elem(zrow + row.tgt);
            if (mine) io.ytgt[t] = yt;
            // terms relative to the segment's maximum: (z - m) c rather than one
            // fused z c - m c, whose product overflows next to the type's lowest
            // value, and with the maximum's own term exactly 1
            m = warp_max(fmaxf(m, mt));
            const float ref = m == -INFINITY ? 0.f : m;
            float s = 0.f;
#pragma unroll
            for (int i = 0; i < kGroups; ++i) {
                float e[8];
#pragma unroll
                for (int j = 0; j < 8; ++j) e[j] = ex2(__fmul_rn(__fsub_rn(z[i][j], ref), c));
                s = __fadd_rn(s, __fadd_rn(__fadd_rn(__fadd_rn(e[0], e[1]), __fadd_rn(e[2], e[3])),
                                           __fadd_rn(__fadd_rn(e[4], e[5]), __fadd_rn(e[6], e[7]))));
            }
            s = __fadd_rn(s, mt == -INFINITY ? st : __fmul_rn(st, ex2(__fmul_rn(__fsub_rn(mt, ref), c))));
            s = warp_sum(s);
            if (lane == 0 && seg0 < io.V) io.part[t * nseg + seg0 / kSegCols] = make_float2(m, s);
        } else if (OP == kApply) {
#pragma unroll
            for (int i = 0; i < kGroups; ++i) {
                float x[8];
#pragma unroll
                for (int j = 0; j < 8; ++j)
                    x[j] = (live >> (8 * i + j) & 1u) ? __fmul_rn(z[i][j], q.itau) : -INFINITY;
                store_group(orow + seg0 + 8 * (lane + 32 * i), io.vec_out, inside >> (8 * i) & 0xffu, x);
            }
            uint32_t b = special;
            while (b) {
                const int k = __ffs(b) - 1;
                b &= b - 1;
                const int sc = warp * kSegCols + lane_column(lane, k);
                const float y = rule_y(load_elem(zrow + slice0 + sc), sh.count[sc],
                                       sh.bias ? __int_as_float(sh.bias[sc]) : 0.f, q);
                store_elem(orow + slice0 + sc, __fmul_rn(y, q.itau));
            }
        } else {
            const float l = io.lse[t];
            const bool none = l == -INFINITY;  // the rules leave nothing
            const float g = none ? 0.f : __fmul_rn(io.grad[t], q.itau);
            // x - lse with 1 / temperature to 48 bits (itau + i1): the rounding of
            // 1 / temperature alone would weigh |x| times half a step
            const float i1 = __fmul_rn(__fmaf_rn(-q.tau, q.itau, 1.f), q.itau);
            const float a = -g;
#pragma unroll
            for (int i = 0; i < kGroups; ++i) {
                float d[8];
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    const float p = prob(z[i][j], q.itau, i1, l);
                    d[j] = (!none && (live >> (8 * i + j) & 1u)) ? __fmul_rn(a, p) : 0.f;
                }
                store_group(orow + seg0 + 8 * (lane + 32 * i), io.vec_out, inside >> (8 * i) & 0xffu, d);
            }
            const int64_t tc = row.tgt - seg0;
            uint32_t b = special;
            int tbit = -1;
            if (tc >= 0 && tc < kSegCols && ((tc >> 3) & 31) == lane) {
                tbit = (int)((tc >> 8) * 8 + (tc & 7));
                b |= (1u << tbit) & live;
            }
            if (none) b = 0;
            while (b) {
                const int k = __ffs(b) - 1;
                b &= b - 1;
                const int sc = warp * kSegCols + lane_column(lane, k);
                const bool tch = touched >> k & 1u;
                const float zv = load_elem(zrow + slice0 + sc);
                const uint32_t w = tch ? sh.count[sc] : 0u;
                const float y = tch ? rule_y(zv, w, sh.bias ? __int_as_float(sh.bias[sc]) : 0.f, q) : zv;
                const float p = prob(y, q.itau, i1, l);
                const float slope = w ? (zv > 0.f ? q.irep : q.rep) : 1.f;
                store_elem(orow + slice0 + sc,
                           __fmul_rn(__fmul_rn(g, __fsub_rn(k == tbit ? 1.f : 0.f, p)), slope));
            }
        }
    }
}

// (m, s) += (mo, so): s exp((m) / temperature) each, c = log2e / temperature.
// An empty partial is (-inf, 0); a NaN sum stays.
__device__ __forceinline__ void merge_y(float &m, float &s, float mo, float so, float c) {
    const float mn = fmaxf(m, mo);
    if (mn == -INFINITY) {
        s = __fadd_rn(s, so);
        return;
    }
    const float ea = ex2(__fmul_rn(__fsub_rn(m, mn), c));
    const float eb = ex2(__fmul_rn(__fsub_rn(mo, mn), c));
    s = __fadd_rn(__fmul_rn(s, ea), __fmul_rn(so, eb));
    m = mn;
}

// One warp per row: lane l folds segments l, l + 32, ... in order, then a
// fixed xor tree.
constexpr int kMergeRows = 8;
__global__ void __launch_bounds__(32 * kMergeRows)
    rules_merge(const __grid_constant__ RulesIo io, const __grid_constant__ rk_logits_rules rules,
                float *logp, float *lse) {
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    const int lane = threadIdx.x & 31;
    const int64_t t = (int64_t)blockIdx.x * kMergeRows + (threadIdx.x >> 5);
    if (t >= io.T) return;
    const RowInfo row = row_info<kLogp>(io, rules, t);
    if (!row.active) {
        if (lane == 0) {
            logp[t] = 0.f;
            if (lse) lse[t] = 0.f;
        }
        return;
    }
    const bool has_tau = row.ok && rules.num_requests > 0 && rules.temperature;
    const float tau = has_tau ? rules.temperature[row.req] : 1.f;
    const float c = __fmul_rn(kLog2e, __frcp_rn(tau));
    const int64_t nseg = (io.V + kSegCols - 1) / kSegCols;
    float m = -INFINITY, s = 0.f;
    for (int64_t k = lane; k < nseg; k += 32) {
        const float2 p = io.part[t * nseg + k];
        merge_y(m, s, p.x, p.y, c);
    }
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) {
        const float mo = __shfl_xor_sync(0xffffffffu, m, off);
        const float so = __shfl_xor_sync(0xffffffffu, s, off);
        merge_y(m, s, mo, so, c);
    }
    if (lane == 0) {
        const float nan = __int_as_float(0x7fc00000);
        float l, p;
        if (!row.ok || row.tgt >= io.V || s != s) {
            l = p = nan;
        } else if (s == 0.f) {
            l = p = -INFINITY;
        } else {
            const float ls = logf(s);
            l = __fadd_rn(__fdiv_rn(m, tau), ls);  // -inf where m / tau is past the type
            p = __fsub_rn(__fdiv_rn(__fsub_rn(io.ytgt[t], m), tau), ls);
            if (p > 0.f) p = 0.f;  // rounding alone can take it there
            if (l == -INFINITY) p = l;
        }
        logp[t] = p;
        if (lse) lse[t] = l;
    }
}

size_t smem_bytes(const rk_logits_rules &r) {
    return (size_t)(kSliceCols + kThreads + (r.bias_ids ? kSliceCols : 0)) * 4;
}

void dependent(cudaLaunchConfig_t *cfg, cudaLaunchAttribute *attr, unsigned grid, unsigned block,
               size_t smem, cudaStream_t st) {
    *cfg = cudaLaunchConfig_t{};
    cfg->gridDim = dim3(grid);
    cfg->blockDim = dim3(block);
    cfg->dynamicSmemBytes = smem;
    cfg->stream = st;
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg->attrs = attr;
    cfg->numAttrs = 1;
}

// Rows per block: about eight blocks per SM, so that a block counts a
// history as seldom as that allows.
int rows_per_block(int64_t T, int64_t V, const DeviceInfo &di) {
    const int64_t slices = (V + kSliceCols - 1) / kSliceCols;
    const int64_t want = T * slices / ((int64_t)di.sm_count * 8);
    return (int)std::max<int64_t>(1, std::min<int64_t>(kMaxRun, want));
}

template <RulesOp OP, typename TIn, typename TOut>
cudaError_t launch(RulesIo io, const rk_logits_rules &r, const DeviceInfo &di, cudaStream_t st) {
    auto *kernel = rules_kernel<OP, TIn, TOut>;
    const size_t smem = smem_bytes(r);
    if (smem > 48 * 1024) {
        const cudaError_t e =
            cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
        if (e != cudaSuccess) return e;
    }
    io.run = rows_per_block(io.T, io.V, di);
    const int64_t slices = (io.V + kSliceCols - 1) / kSliceCols;
    const int64_t blocks = slices * ((io.T + io.run - 1) / io.run);
    if (blocks > 0x7fffffff) return cudaErrorInvalidConfiguration;
    cudaLaunchConfig_t cfg;
    cudaLaunchAttribute attr[1];
    dependent(&cfg, attr, (unsigned)blocks, kThreads, smem, st);
    return cudaLaunchKernelEx(&cfg, kernel, io, r);
}

template <RulesOp OP>
cudaError_t launch_types(const RulesIo &io, const rk_logits_rules &r, int in, int out,
                         const DeviceInfo &di, cudaStream_t st) {
    if (in == RK_BF16)
        return out == RK_BF16 ? launch<OP, uint16_t, uint16_t>(io, r, di, st)
                              : launch<OP, uint16_t, float>(io, r, di, st);
    return out == RK_BF16 ? launch<OP, float, uint16_t>(io, r, di, st)
                          : launch<OP, float, float>(io, r, di, st);
}

bool vec16(const void *p, int64_t ld, rk_dtype type) {
    return aligned(p, 16) && (ld * (type == RK_BF16 ? 2 : 4)) % 16 == 0;
}

}  // namespace

size_t logp_rules_workspace_bytes(int64_t T, int64_t V) {
    const size_t nseg = (size_t)((V + kSegCols - 1) / kSegCols);
    return ((size_t)T * nseg * sizeof(float2) + (size_t)T * sizeof(float) + 255) / 256 * 256;
}

cudaError_t launch_rules_apply(const RulesMatrix &logits, const rk_logits_rules &rules, int64_t T,
                               int64_t V, const RulesMatrix &out, const DeviceInfo &di,
                               cudaStream_t st) {
    RulesIo io{};
    io.logits = logits.p;
    io.ld = logits.ld;
    io.vec_in = vec16(logits.p, logits.ld, logits.type);
    io.T = T;
    io.V = V;
    io.out = const_cast<void *>(out.p);
    io.ld_out = out.ld;
    io.vec_out = vec16(out.p, out.ld, out.type);
    io.err = di.err;
    return launch_types<kApply>(io, rules, logits.type, out.type, di, st);
}

cudaError_t launch_rules_logp(const RulesMatrix &logits, const int64_t *targets, const int32_t *cu,
                              int num_seqs, const rk_logits_rules &rules, int64_t T, int64_t V,
                              float *logp, float *lse, void *workspace, const DeviceInfo &di,
                              cudaStream_t st) {
    RulesIo io{};
    io.logits = logits.p;
    io.ld = logits.ld;
    io.vec_in = vec16(logits.p, logits.ld, logits.type);
    io.targets = targets;
    io.cu = cu;
    io.num_seqs = num_seqs;
    io.T = T;
    io.V = V;
    io.part = static_cast<float2 *>(workspace);
    io.ytgt = reinterpret_cast<float *>(io.part + T * ((V + kSegCols - 1) / kSegCols));
    io.err = di.err;
    cudaError_t e = logits.type == RK_BF16 ? launch<kLogp, uint16_t, float>(io, rules, di, st)
                                           : launch<kLogp, float, float>(io, rules, di, st);
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg;
    cudaLaunchAttribute attr[1];
    dependent(&cfg, attr, (unsigned)((T + kMergeRows - 1) / kMergeRows), 32 * kMergeRows, 0, st);
    return cudaLaunchKernelEx(&cfg, rules_merge, io, rules, logp, lse);
}

cudaError_t launch_rules_bwd(const RulesMatrix &logits, const int64_t *targets, const int32_t *cu,
                             int num_seqs, const rk_logits_rules &rules, int64_t T, int64_t V,
                             const float *lse, const float *grad, const RulesMatrix &dlogits,
                             const DeviceInfo &di, cudaStream_t st) {
    RulesIo io{};
    io.logits = logits.p;
    io.ld = logits.ld;
    io.vec_in = vec16(logits.p, logits.ld, logits.type);
    io.targets = targets;
    io.cu = cu;
    io.num_seqs = num_seqs;
    io.T = T;
    io.V = V;
    io.lse = lse;
    io.grad = grad;
    io.out = const_cast<void *>(dlogits.p);
    io.ld_out = dlogits.ld;
    io.vec_out = vec16(dlogits.p, dlogits.ld, dlogits.type);
    io.err = di.err;
    return launch_types<kBwd>(io, rules, logits.type, dlogits.type, di, st);
}

}  // namespace rk
