// logits_rules.cu -- logits under sampling rules: repetition, frequency and
// presence penalties, per-request biases, grammar masks and temperature (the
// definition stands at rk_logits_rules in rk.h), applied (kApply), scored
// (kLogp: selected logprob and log-sum-exp) and differentiated (kBwd).
//
// Decomposition.  A block works on a slice of kSliceCols columns and a run of
// consecutive rows; each of its warps owns a segment of kSegCols columns of
// that slice, and each lane 32 neighbouring columns of the segment: one word
// of a grammar mask, and one word that tells which of them the rules touch
// (seen before, or biased).  The others need the temperature and mask only.
//
// Data.  A warp copies its segment of the next rows into a ring of its own in
// shared memory (cp.async, 16 bytes a lane, or 4 where rows are not 16-byte
// aligned; the mask words with them) while it works on the present one, so no
// barrier stands between the rows.  What the rows say about themselves is read
// once per block.  Results of kApply and kBwd leave through the same stage, so
// that a warp writes whole lines although a lane owns 32 columns.  The lanes
// take their 16-byte pieces in rotated order, which spreads a quarter warp
// over all banks.
//
// History.  The block counts a request's tokens of its slice in shared
// memory (one word per column: bit 31 in the prompt, bits 0-30 times
// produced).  Integer atomics only, so the order does not matter.  A row that
// has one token more than the row before (a packed training sequence) adds it
// to the counts without a barrier: its column belongs to one lane.  Longer
// steps add their tokens block-wide; any other change counts anew.  Each warp
// lists its touched columns in ascending order, 32 of which its lanes take at
// a time: text is made of few tokens, which sit at the low ids, so lanes that
// looped over their own columns would wait for the first lane's 32.
//
// Batch invariance: a row's partial (max, sum) of a segment is formed by a
// tree fixed by the column index alone, and the segments' partials are merged
// in a fixed order: nothing depends on T, on where the row sits or on how the
// rows were cut into runs.
#include <algorithm>
#include <cfloat>

#include "rk_device.cuh"
#include "rk_internal.h"

namespace rk {
namespace {

constexpr int kLaneCols = 32;
constexpr int kSegCols = 32 * kLaneCols;       // 1024 columns per warp
constexpr int kWarps = 8;
constexpr int kThreads = 32 * kWarps;
constexpr int kSliceCols = kSegCols * kWarps;  // 8192 columns per block
constexpr int kMaxRun = 64;                    // rows per block at most
constexpr int kMaxBiases = 65534;  // per request: indices are kept in 16 bits
constexpr uint32_t kPromptBit = 0x80000000u;
constexpr uint32_t kNegInf2 = 0xFF80FF80u;  // two bf16 -inf
constexpr uint32_t kLowest2 = 0xFF7FFF7Fu;  // two bf16 lowest finite values

enum RulesOp { kApply, kLogp, kBwd };

struct RulesIo {
    const void *logits;
    int64_t ld;
    const int64_t *targets;
    const int32_t *cu;
    int num_seqs;
    int64_t T, V;
    int run;         // rows per block
    int vec_in;      // every row starts on a 16-byte boundary
    const float *lse, *grad;  // kBwd
    void *out;       // kApply, kBwd
    int64_t ld_out;
    int vec_out;
    float2 *part;    // kLogp: [T][segments] (max of y, sum relative to it)
    float *ytgt;     // kLogp: [T] y of the target, -inf when it is masked
    unsigned *err;
};

// What a row says about itself.
constexpr int32_t kInactive = -1, kBadTarget = -2, kBadRules = -3;
struct RowInfo {
    int32_t tgt;  // the target, or one of the codes above
    int32_t req, len, mrow;
    // how its history differs from the row before: by one token, by none, or
    // else (kAnew); a token outside the vocabulary counts as none
    int32_t step;
    int32_t step_prompt;
    float lse, g;
};
constexpr int32_t kNoToken = -1, kAnew = -2;

template <RulesOp OP>
__device__ __forceinline__ RowInfo row_info(const RulesIo &io, const rk_logits_rules &r, int64_t t) {
    const int64_t tgt = (OP == kApply) ? 0 : io.targets[t];
    RowInfo i;
    i.req = r.row_request ? r.row_request[t] : (r.num_requests > 0 ? (int32_t)t : 0);
    i.len = r.row_length ? max(r.row_length[t], 0) : 0x7fffffff;
    i.mrow = r.mask ? (r.row_mask ? r.row_mask[t] : (int32_t)t) : -1;
    i.tgt = (int32_t)tgt;
    i.step = kAnew;
    i.step_prompt = 0;
    i.lse = OP == kBwd ? io.lse[t] : 0.f;
    i.g = OP == kBwd ? io.grad[t] : 0.f;
    if ((OP != kApply && !row_active(t, tgt, io.cu, io.num_seqs)) || (r.row_request && i.req == -1))
        i.tgt = kInactive;
    else if (i.req < 0 || (r.num_requests > 0 && i.req >= r.num_requests) ||
             (i.mrow >= 0 && i.mrow >= r.mask_rows))
        i.tgt = kBadRules;
    else if (tgt >= io.V)
        i.tgt = kBadTarget;
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
        if (a >= 0 && b >= a && b <= r.num_bias && b - a <= kMaxBiases) {
            s.bias0 = a;
            s.nbias = (int32_t)(b - a);
        } else {
            s.ok = false;
        }
    }
    return s;
}

// row.step and row.step_prompt, given the row before.
__device__ __forceinline__ void find_step(const RulesIo &io, const rk_logits_rules &r,
                                          const RowInfo &before, RowInfo &row) {
    if (row.tgt < 0 || before.tgt < 0 || row.req != before.req) return;
    row.step = kNoToken;
    if (r.num_requests == 0 || !r.tokens) return;
    const int64_t a = r.token_offsets[row.req], b = r.token_offsets[row.req + 1];
    if (!(a >= 0 && b >= a && b <= r.num_tokens && b - a < 0x7fffffff)) return;  // refused by load_request
    const int32_t ntok = (int32_t)(b - a), len = min(row.len, ntok), was = min(before.len, ntok);
    if (len == was) return;
    if (len != was + 1) {
        row.step = kAnew;
        return;
    }
    const int64_t v = r.tokens[a + was];
    if (v >= 0 && v < io.V) row.step = (int32_t)v;
    row.step_prompt = r.prompt_lengths && was < r.prompt_lengths[row.req];
}

// y of a touched column from z, its count word and its bias.
__device__ __forceinline__ float rule_y(float z, uint32_t w, float bias, const Request &q) {
    float y = z;
    if (w) y = __fmul_rn(z, z > 0.f ? q.irep : q.rep);
    const uint32_t n = w & ~kPromptBit;
    if (n) y = __fsub_rn(y, __fmaf_rn(q.freq, (float)n, q.pres));
    return __fadd_rn(y, bias);
}

// ---- elements and 16-byte pieces in shared memory ----

__device__ __forceinline__ float elem(const uint16_t *p) { return bf16_bits_to_f32(*p); }
__device__ __forceinline__ float elem(const float *p) { return *p; }
__device__ __forceinline__ void put(uint16_t *p, float v) {
    *p = (uint16_t)(pack_bf16x2(v, 0.f) & 0xffffu);
}
__device__ __forceinline__ void put(float *p, float v) { *p = v; }

// Pairs of fp32 (one instruction for both).
__device__ __forceinline__ uint64_t pair(float a, float b) {
    uint64_t d;
    asm("mov.b64 %0, {%1, %2};" : "=l"(d) : "f"(a), "f"(b));
    return d;
}
__device__ __forceinline__ void unpair(uint64_t p, float &a, float &b) {
    asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(p));
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
    uint64_t d;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
    return d;
}
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
    uint64_t d;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
    return d;
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
    uint64_t d;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
    return d;
}
__device__ __forceinline__ uint32_t max_bf16x2(uint32_t a, uint32_t b) {
    uint32_t d;
    asm("max.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
    return d;
}
__device__ __forceinline__ uint32_t max_nan_bf16x2(uint32_t a, uint32_t b) {
    uint32_t d;
    asm("max.NaN.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
    return d;
}
__device__ __forceinline__ float max_nan(float a, float b) {
    float d;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(d) : "f"(a), "f"(b));
    return d;
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

// A lane's 32 columns as 16-byte pieces.  Piece register i holds piece
// order(i) of the lane: rotated by lane so that the eight lanes of a quarter
// warp read eight different bank groups.
template <typename T>
struct Lane;
template <>
struct Lane<uint16_t> {
    static constexpr int kPieces = 4, kCols = 8;  // pieces, columns of a piece
    static __device__ __forceinline__ int order(int lane, int i) { return (i + (lane >> 1)) & 3; }
    static __device__ __forceinline__ int bits(int lane) { return 8 * ((lane >> 1) & 3); }
};
template <>
struct Lane<float> {
    static constexpr int kPieces = 8, kCols = 4;
    static __device__ __forceinline__ int order(int lane, int i) { return (i + lane) & 7; }
    static __device__ __forceinline__ int bits(int lane) { return 4 * (lane & 7); }
};


__device__ __forceinline__ void cp_async16(uint32_t dst, const void *src, int bytes) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes)
                 : "memory");
}
__device__ __forceinline__ void cp_async4(uint32_t dst, const void *src) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// Whether a row starts on an odd 2-byte element.
__device__ __forceinline__ bool odd_start(const uint16_t *src) {
    return (reinterpret_cast<uintptr_t>(src) & 2) != 0;
}
__device__ __forceinline__ bool odd_start(const float *) { return false; }

// Starts the copy of `cols` columns from src into a stage (2 bytes into it
// after an odd start).  Nothing outside [src, src + cols) is read.
template <typename T>
__device__ __forceinline__ void start_copy(unsigned char *stage, const T *src, int cols, bool vec,
                                           int lane) {
    const uint32_t dst = smem_u32(stage);
    if (vec) {
        constexpr int kPer = 16 / (int)sizeof(T);
#pragma unroll
        for (int i = 0; i < kSegCols / kPer / 32; ++i) {
            const int c = (lane + 32 * i) * kPer;
            const int n = min(kPer, cols - c);
            if (n > 0) cp_async16(dst + c * (int)sizeof(T), src + c, n * (int)sizeof(T));
        }
    } else if constexpr (sizeof(T) == 4) {
#pragma unroll 8
        for (int c = lane; c < cols; c += 32) cp_async4(dst + 4 * c, src + c);
    } else {
        // words on 4-byte boundaries; a word that the row does not fill is
        // copied by element
        const int odd = odd_start(src) ? 1 : 0;
        uint16_t *d = reinterpret_cast<uint16_t *>(stage);
#pragma unroll 8
        for (int w = lane; 2 * w < cols + odd; w += 32) {
            const int c = 2 * w - odd;  // its first column
            if (c >= 0 && c + 1 < cols) {
                cp_async4(dst + 4 * w, src + c);
            } else {
                if (c >= 0) d[2 * w] = src[c];
                if (c + 1 < cols) d[2 * w + 1] = src[c + 1];
            }
        }
    }
}

// Piece i of a lane, from a stage; `odd`: it sits one element further in.
__device__ __forceinline__ uint4 load_piece(const unsigned char *p, bool odd) {
    const uint4 a = *reinterpret_cast<const uint4 *>(p);
    if (!odd) return a;
    const uint32_t b = *reinterpret_cast<const uint32_t *>(p + 16);
    return make_uint4(__funnelshift_r(a.x, a.y, 16), __funnelshift_r(a.y, a.z, 16),
                      __funnelshift_r(a.z, a.w, 16), __funnelshift_r(a.w, b, 16));
}

// ---- history ----

// Shared memory of a block.
struct Shared {
    uint32_t *count;    // [kSliceCols]
    uint32_t *touched;  // [kThreads]: bit c % 32 of word c / 32 for slice column c
    uint16_t *list;     // [kSliceCols]: each warp's touched columns, ascending
    uint16_t *bias;     // [kSliceCols], or null: 1 + the index of the column's bias, 0: none
};

__device__ __forceinline__ void mark(const Shared &sh, int c) {
    atomicOr(&sh.touched[c >> 5], 1u << (c & 31));
}

// Block-wide: tokens [from, to) of the request into the counts of columns
// [slice0, slice0 + width).
__device__ __forceinline__ void count_tokens(const Shared &sh, const Request &q, int32_t from,
                                             int32_t to, int64_t slice0, int width) {
    constexpr int kBatch = 8;  // loads in flight per thread
    for (int32_t i0 = from + (int32_t)threadIdx.x; i0 < to; i0 += kBatch * kThreads) {
        int64_t v[kBatch];
#pragma unroll
        for (int k = 0; k < kBatch; ++k) v[k] = i0 + k * kThreads < to ? q.tokens[i0 + k * kThreads] : -1;
#pragma unroll
        for (int k = 0; k < kBatch; ++k) {
            const int64_t c = v[k] - slice0;
            if (v[k] >= 0 && c >= 0 && c < width) {
                if (i0 + k * kThreads < q.prompt)
                    atomicOr(&sh.count[c], kPromptBit);
                else
                    atomicAdd(&sh.count[c], 1u);
                mark(sh, (int)c);
            }
        }
    }
}

// Block-wide: the request's first `len` tokens and its biases from scratch.
// Of biases for one column the last counts: the count words find it first.
__device__ __forceinline__ void count_request(const Shared &sh, const rk_logits_rules &rules,
                                              const Request &q, int32_t len, int64_t slice0, int width) {
    __syncthreads();
    for (int k = threadIdx.x; k < kSliceCols / 4; k += kThreads)
        reinterpret_cast<uint4 *>(sh.count)[k] = make_uint4(0, 0, 0, 0);
    sh.touched[threadIdx.x] = 0;
    if (sh.bias)
        for (int k = threadIdx.x; k < kSliceCols / 8; k += kThreads)
            reinterpret_cast<uint4 *>(sh.bias)[k] = make_uint4(0, 0, 0, 0);
    __syncthreads();
    if (q.nbias > 0) {
        for (int k = threadIdx.x; k < q.nbias; k += kThreads) {
            const int64_t v = rules.bias_ids[q.bias0 + k], c = v - slice0;
            if (v >= 0 && c >= 0 && c < width) {
                atomicMax(&sh.count[c], (uint32_t)(k + 1));
                mark(sh, (int)c);
            }
        }
        __syncthreads();
        for (uint32_t b = sh.touched[threadIdx.x]; b; b &= b - 1) {
            const int c = threadIdx.x * kLaneCols + __ffs(b) - 1;
            sh.bias[c] = (uint16_t)sh.count[c];
            sh.count[c] = 0;
        }
        __syncthreads();
    }
    count_tokens(sh, q, 0, len, slice0, width);
    __syncthreads();
}

// A warp's list of its touched columns (segment columns, ascending) from its
// lanes' bits; returns their number.
__device__ __forceinline__ int make_list(uint16_t *list, uint32_t touched, int lane) {
    const int mine = __popc(touched);
    int incl = mine;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, incl, off);
        if (lane >= off) incl += y;
    }
    int at = incl - mine;
    for (uint32_t b = touched; b; b &= b - 1)
        list[at++] = (uint16_t)(lane * kLaneCols + __ffs(b) - 1);
    return __shfl_sync(0xffffffffu, incl, 31);
}

// exp(y / temperature - lse), 1 / temperature = itau + i1.  -inf stays out of
// the product with i1, whose sign it would take.
__device__ __forceinline__ float prob(float y, float itau, float i1, float lse) {
    const float v = max_nan(y, -FLT_MAX);
    return ex2(__fmul_rn(__fmaf_rn(v, i1, __fmaf_rn(v, itau, -lse)), kLog2e));
}

// bf16 pieces: where a pair's two bits in `keep` are 0, -inf.  Byte i of `keep`
// belongs to piece i, bit j of it to column j.
__device__ __forceinline__ void keep_columns(uint4 (&w)[4], uint32_t keep) {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        // the sign bit of byte i of a (of b) is bit 2j (2j + 1) of piece i
        const uint32_t a = keep << (7 - 2 * j), b = keep << (6 - 2 * j);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            uint32_t m;  // each byte: the sign of byte i of a, twice, and of b, twice
            asm("prmt.b32 %0, %1, %2, %3;" : "=r"(m) : "r"(a), "r"(b), "r"(0xCC88 + 0x1111 * i));
            uint32_t &q = j == 0 ? w[i].x : j == 1 ? w[i].y : j == 2 ? w[i].z : w[i].w;
            q = (q & m) | (kNegInf2 & ~m);
        }
    }
}

__device__ __forceinline__ void unpack(const uint4 &w, uint64_t (&z)[4]) {
    const uint32_t q[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int j = 0; j < 4; ++j) z[j] = pair(bf16_lo(q[j]), bf16_hi(q[j]));
}

// Shared memory of a block: counts, touched words, rows, lists and bias
// indices, and a ring of stages per warp.  A stage holds the segment's logits
// (16 bytes more for rows that start on an odd element: they sit one element
// further in) and afterwards its results, and the segment's mask words.
// Blocks of up to 113 KB run two to an SM, which beats a second stage.
template <RulesOp OP, typename TIn, typename TOut>
struct Config {
    static constexpr int kElem = OP != kLogp && sizeof(TOut) > sizeof(TIn) ? sizeof(TOut) : sizeof(TIn);
    static constexpr int kStages = kElem == 2 ? 2 : 1;
    static constexpr int kMaskAt = kSegCols * kElem + 16;
    static constexpr int kStageBytes = kMaskAt + kSegCols / 8;
    // fp32 results of bf16 pieces: neighbouring lanes would write the same bank
    // group, so odd lanes swap neighbouring pieces
    static constexpr int kSwap = (sizeof(TIn) == 2 && sizeof(TOut) == 4) ? 1 : 0;
    static size_t smem(bool bias) {
        return (size_t)(kSliceCols + kThreads) * 4 + kMaxRun * sizeof(RowInfo) +
               (size_t)kSliceCols * (bias ? 4 : 2) + (size_t)kWarps * kStages * kStageBytes;
    }
};

// Writes `cols` results of a segment from the warp's staging area to dst.
template <int SWAP>
__device__ __forceinline__ void write_out(const unsigned char *stage, float *dst, int cols, bool vec,
                                          int lane) {
    const float4 *s4 = reinterpret_cast<const float4 *>(stage);
    if (vec && cols == kSegCols) {
#pragma unroll
        for (int i = 0; i < kSegCols / 128; ++i) {
            const int x = lane + 32 * i;
            reinterpret_cast<float4 *>(dst)[x] = s4[x ^ (SWAP ? (x >> 3) & 1 : 0)];
        }
    } else {
        const float *s = reinterpret_cast<const float *>(stage);
#pragma unroll 8
        for (int c = lane; c < cols; c += 32) dst[c] = s[c ^ (SWAP ? ((c >> 5) & 1) << 2 : 0)];
    }
}
template <int SWAP>
__device__ __forceinline__ void write_out(const unsigned char *stage, uint16_t *dst, int cols,
                                          bool vec, int lane) {
    if (vec && cols == kSegCols) {
#pragma unroll
        for (int i = 0; i < kSegCols / 256; ++i)
            reinterpret_cast<uint4 *>(dst)[lane + 32 * i] =
                reinterpret_cast<const uint4 *>(stage)[lane + 32 * i];
    } else {
        const uint16_t *s = reinterpret_cast<const uint16_t *>(stage);
#pragma unroll 8
        for (int c = lane; c < cols; c += 32) dst[c] = s[c];
    }
}

template <RulesOp OP, typename TIn, typename TOut>
__global__ void __launch_bounds__(kThreads)
    rules_kernel(const __grid_constant__ RulesIo io, const __grid_constant__ rk_logits_rules rules) {
    using C = Config<OP, TIn, TOut>;
    using L = Lane<TIn>;
    extern __shared__ uint4 smem[];
    Shared sh;
    sh.count = reinterpret_cast<uint32_t *>(smem);
    sh.touched = sh.count + kSliceCols;
    RowInfo *rows = reinterpret_cast<RowInfo *>(sh.touched + kThreads);
    sh.list = reinterpret_cast<uint16_t *>(rows + kMaxRun);
    sh.bias = rules.bias_ids ? sh.list + kSliceCols : nullptr;
    unsigned char *p = reinterpret_cast<unsigned char *>(sh.list + (rules.bias_ids ? 2 : 1) * kSliceCols);
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    unsigned char *ring = p + warp * C::kStages * C::kStageBytes;
    // Launched with programmatic stream serialisation: wait until the previous
    // kernel of the stream has completed before reading or writing anything.
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");

    const int64_t slices = (io.V + kSliceCols - 1) / kSliceCols;
    const int64_t slice0 = (int64_t)(blockIdx.x % slices) * kSliceCols;
    const int width = (int)min((int64_t)kSliceCols, io.V - slice0);
    const int64_t t0 = (int64_t)(blockIdx.x / slices) * io.run;
    const int n = (int)min((int64_t)io.run, io.T - t0);
    const int64_t seg0 = slice0 + (int64_t)warp * kSegCols;
    const int cols = (int)max((int64_t)0, min((int64_t)kSegCols, io.V - seg0));  // of this warp
    const int64_t nseg = (io.V + kSegCols - 1) / kSegCols;
    const int64_t words = (io.V + 31) / 32;
    const int own = lane * kLaneCols;  // the lane's first column in the segment
    const uint32_t inside =
        cols >= own + 32 ? 0xffffffffu : cols > own ? (1u << (cols - own)) - 1u : 0u;
    uint32_t *count = sh.count + warp * kSegCols;  // of the segment
    const uint16_t *bias = sh.bias ? sh.bias + warp * kSegCols : nullptr;
    uint16_t *list = sh.list + warp * kSegCols;

    for (int k = threadIdx.x; k < n; k += kThreads) rows[k] = row_info<OP>(io, rules, t0 + k);
    __syncthreads();

    const TIn *zseg = reinterpret_cast<const TIn *>(io.logits) + t0 * io.ld + seg0;
    auto prefetch = [&](int k) {
        if (k < n && rows[k].tgt >= 0) {
            unsigned char *stage = ring + (k % C::kStages) * C::kStageBytes;
            start_copy(stage, zseg + k * io.ld, cols, io.vec_in, lane);
            if (rows[k].mrow >= 0 && inside)
                cp_async4(smem_u32(stage + C::kMaskAt) + 4 * lane,
                          rules.mask + (int64_t)rows[k].mrow * words + (seg0 >> 5) + lane);
        }
        cp_commit();
    };
    for (int k = 0; k < C::kStages; ++k) prefetch(k);
    for (int k = threadIdx.x + 1; k < n; k += kThreads) find_step(io, rules, rows[k - 1], rows[k]);
    __syncthreads();

    int32_t cur = -1, counted = 0;
    uint32_t touched = 0;
    int listed = 0;  // touched columns of the warp
    Request q{};
    for (int k = 0; k < n; ++k) {
        const RowInfo row = rows[k];
        const int64_t t = t0 + k;
        bool ok = row.tgt >= 0;
        if (ok && (row.req != cur || (q.ok && row.step == kAnew))) {
            const bool other = row.req != cur;
            if (other) {
                q = load_request(rules, row.req);
                cur = row.req;
            }
            if (q.ok) {
                const int32_t len = min(row.len, q.ntok);
                if (other || len < counted) {
                    count_request(sh, rules, q, len, slice0, width);
                } else {
                    __syncthreads();
                    sh.touched[threadIdx.x] = touched;
                    __syncthreads();
                    count_tokens(sh, q, counted, len, slice0, width);
                    __syncthreads();
                }
                counted = len;
                touched = sh.touched[threadIdx.x];
                listed = make_list(list, touched, lane);
            }
        } else if (ok && q.ok) {
            counted = min(row.len, q.ntok);
            const int64_t c = row.step - seg0;  // negative where there is no token
            if (row.step >= 0 && c >= 0 && c < cols) {
                const uint32_t bit = (c >> 5) == lane ? 1u << (c & 31) : 0u;
                if (bit) count[c] = row.step_prompt ? (count[c] | kPromptBit) : count[c] + 1u;
                const bool fresh = (bit & ~touched) != 0;
                touched |= bit;
                if (__any_sync(0xffffffffu, fresh)) listed = make_list(list, touched, lane);
            }
        }
        ok = ok && q.ok;
        cp_wait<C::kStages - 1>();  // all copies but those of later rows
        __syncwarp();
        TOut *orow = reinterpret_cast<TOut *>(io.out) + t * io.ld_out + seg0;
        if (!ok) {
            const float fill = row.tgt == kInactive ? 0.f : __int_as_float(0x7fc00000);
            if (row.tgt != kInactive) {
                if (slice0 == 0 && threadIdx.x == 0)
                    atomicOr(io.err, row.tgt == kBadTarget ? kErrTargetRange : kErrRules);
                if (OP == kLogp && lane == 0 && cols > 0) {
                    io.part[t * nseg + seg0 / kSegCols] = make_float2(0.f, fill);
                    if (seg0 == 0) io.ytgt[t] = fill;
                }
            }
            if (OP == kBwd || (OP == kApply && row.tgt != kInactive))
                for (int c = lane; c < cols; c += 32) put(orow + c, fill);
            prefetch(k + C::kStages);
            continue;
        }
        unsigned char *stage = ring + (k % C::kStages) * C::kStageBytes;
        const bool odd = !io.vec_in && odd_start(zseg + k * io.ld);
        // single logits: from the stage, or, where results replace it, from the row
        const TIn *zs = OP == kLogp ? reinterpret_cast<const TIn *>(stage) + (odd ? 1 : 0) : zseg + k * io.ld;
        const uint32_t *masks = reinterpret_cast<const uint32_t *>(stage + C::kMaskAt);
        const bool masked = row.mrow >= 0;
        const uint32_t live = masked ? inside & masks[lane] : inside;  // columns the mask allows
        // a listed column's y from its logit z (false: masked)
        auto listed_y = [&](int j, float &z, uint32_t &cw, float &y) {
            if (masked && !(masks[j >> 5] >> (j & 31) & 1u)) return false;
            z = elem(zs + j);
            cw = count[j];
            const int bi = bias ? bias[j] : 0;
            y = rule_y(z, cw, bi ? rules.bias_values[q.bias0 + bi - 1] : 0.f, q);
            return true;
        };
        const int rot = L::bits(lane);
        uint4 w[L::kPieces];
#pragma unroll
        for (int i = 0; i < L::kPieces; ++i)
            w[i] = load_piece(stage + 16 * (lane * L::kPieces + L::order(lane, i)), odd);
        if (OP != kLogp) __syncwarp();  // the stage is read

        if (OP == kLogp) {
            const float c = __fmul_rn(kLog2e, q.itau);
            const int tcol = row.tgt >= seg0 && row.tgt < seg0 + cols ? row.tgt - (int)seg0 : -1;
            // touched columns: running maximum and sum, each lane its share of the list
            float mt = -INFINITY, st = 0.f;
            for (int e = lane; e < listed; e += 32) {
                const int j = list[e];
                float z, y = -INFINITY;
                uint32_t cw;
                const bool allowed = listed_y(j, z, cw, y);
                if (j == tcol) io.ytgt[t] = y;
                if (!allowed || y == -INFINITY) continue;  // masked, or banned by its bias
                const float mn = fmaxf(mt, y);
                st = __fmaf_rn(st, ex2(__fmul_rn(__fsub_rn(mt, mn), c)),
                               ex2(__fmul_rn(__fsub_rn(y, mn), c)));
                mt = mn;
            }
            // untouched columns: one maximum, then the terms relative to it
            const uint32_t plain = live & ~touched;
            if (tcol >= 0 && (tcol >> 5) == lane && !(touched >> (tcol & 31) & 1u))
                io.ytgt[t] = plain >> (tcol & 31) & 1u ? elem(zs + tcol) : -INFINITY;
            const uint32_t keep = __funnelshift_r(plain, plain, rot);
            float m;
            if constexpr (sizeof(TIn) == 2) {
                if (!__all_sync(0xffffffffu, plain == 0xffffffffu)) keep_columns(w, keep);
                uint32_t x[4];
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    x[i] = max_bf16x2(max_bf16x2(w[i].x, w[i].y), max_bf16x2(w[i].z, w[i].w));
                x[0] = max_bf16x2(max_bf16x2(x[0], x[1]), max_bf16x2(x[2], x[3]));
                m = fmaxf(bf16_lo(x[0]), bf16_hi(x[0]));
            } else {
                float x[8];
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    uint32_t *f = &w[i].x;
#pragma unroll
                    for (int j = 0; j < 4; ++j)
                        if ((int32_t)(keep << (31 - 4 * i - j)) >= 0) f[j] = 0xff800000u;
                    x[i] = fmaxf(fmaxf(__uint_as_float(w[i].x), __uint_as_float(w[i].y)),
                                 fmaxf(__uint_as_float(w[i].z), __uint_as_float(w[i].w)));
                }
                m = fmaxf(fmaxf(fmaxf(x[0], x[1]), fmaxf(x[2], x[3])),
                          fmaxf(fmaxf(x[4], x[5]), fmaxf(x[6], x[7])));
            }
            // terms relative to the segment's maximum: (z - m) c rather than one
            // fused z c - m c, whose product overflows next to the type's lowest
            // value, and with the maximum's own term exactly 1
            m = warp_max(fmaxf(m, mt));
            const float ref = m == -INFINITY ? 0.f : m;
            const uint64_t nref = pair(-ref, -ref), cc = pair(c, c);
            uint64_t acc[2] = {0, 0};  // pairs of +0
#pragma unroll
            for (int i = 0; i < L::kPieces; ++i) {
                uint64_t z[4];
                if constexpr (sizeof(TIn) == 2) {
                    unpack(w[i], z);
                } else {
                    z[0] = pair(__uint_as_float(w[i].x), __uint_as_float(w[i].y));
                    z[1] = pair(__uint_as_float(w[i].z), __uint_as_float(w[i].w));
                }
#pragma unroll
                for (int j = 0; j < L::kCols / 2; ++j) {
                    float a, b;
                    unpair(mul2(add2(z[j], nref), cc), a, b);
                    acc[j & 1] = add2(acc[j & 1], pair(ex2(a), ex2(b)));
                }
            }
            float s0, s1;
            unpair(add2(acc[0], acc[1]), s0, s1);
            float s = __fadd_rn(s0, s1);
            s = __fadd_rn(s, mt == -INFINITY ? st : __fmul_rn(st, ex2(__fmul_rn(__fsub_rn(mt, ref), c))));
            s = warp_sum(s);
            if (lane == 0 && cols > 0) io.part[t * nseg + seg0 / kSegCols] = make_float2(m, s);
        } else {
            const float l = row.lse;
            const bool none = OP == kBwd && l == -INFINITY;  // the rules leave nothing
            const float g = OP == kBwd && !none ? __fmul_rn(row.g, q.itau) : 0.f;
            // x - lse with 1 / temperature to 48 bits (itau + i1): the rounding of
            // 1 / temperature alone would weigh |x| times half a step
            const float i1 = __fmul_rn(__fmaf_rn(-q.tau, q.itau, 1.f), q.itau);
            const uint32_t shown = none ? 0u : live;
            const uint32_t keep = __funnelshift_r(shown, shown, rot);
            const uint64_t it2 = pair(q.itau, q.itau);
#pragma unroll
            for (int i = 0; i < L::kPieces; ++i) {
                constexpr int N = L::kCols;
                uint64_t z[4];
                float x[8];
                if constexpr (sizeof(TIn) == 2) {
                    if (OP == kBwd) {  // -inf out of the products (see prob)
                        w[i].x = max_nan_bf16x2(w[i].x, kLowest2);
                        w[i].y = max_nan_bf16x2(w[i].y, kLowest2);
                        w[i].z = max_nan_bf16x2(w[i].z, kLowest2);
                        w[i].w = max_nan_bf16x2(w[i].w, kLowest2);
                    }
                    unpack(w[i], z);
                } else {
                    float f[4] = {__uint_as_float(w[i].x), __uint_as_float(w[i].y),
                                  __uint_as_float(w[i].z), __uint_as_float(w[i].w)};
                    if (OP == kBwd)
#pragma unroll
                        for (int j = 0; j < 4; ++j) f[j] = max_nan(f[j], -FLT_MAX);
                    z[0] = pair(f[0], f[1]);
                    z[1] = pair(f[2], f[3]);
                }
#pragma unroll
                for (int j = 0; j < N / 2; ++j) {
                    uint64_t v;
                    if (OP == kApply) {
                        v = mul2(z[j], it2);
                    } else {
                        v = fma2(z[j], pair(i1, i1), fma2(z[j], it2, pair(-l, -l)));
                        v = mul2(v, pair(kLog2e, kLog2e));
                        float a, b;
                        unpair(v, a, b);
                        v = mul2(pair(ex2(a), ex2(b)), pair(-g, -g));
                    }
                    unpair(v, x[2 * j], x[2 * j + 1]);
                }
#pragma unroll
                for (int j = 0; j < N; ++j)
                    if ((int32_t)(keep << (31 - N * i - j)) >= 0) x[j] = OP == kApply ? -INFINITY : 0.f;
                const int piece = lane * L::kPieces + L::order(lane, i);  // of the segment
                if constexpr (sizeof(TOut) == 4) {
                    float4 *o = reinterpret_cast<float4 *>(stage);
#pragma unroll
                    for (int h = 0; h < N / 4; ++h)
                        o[(piece * (N / 4) + h) ^ (C::kSwap ? lane & 1 : 0)] =
                            make_float4(x[4 * h], x[4 * h + 1], x[4 * h + 2], x[4 * h + 3]);
                } else {
                    uint32_t *o = reinterpret_cast<uint32_t *>(stage) + piece * (N / 2);
                    if constexpr (N == 8)
                        *reinterpret_cast<uint4 *>(o) =
                            make_uint4(pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3]),
                                       pack_bf16x2(x[4], x[5]), pack_bf16x2(x[6], x[7]));
                    else
                        *reinterpret_cast<uint2 *>(o) =
                            make_uint2(pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3]));
                }
            }
            // the touched columns, and the target's, over what stands there
            __syncwarp();
            auto put_column = [&](int j, float v) {
                put(reinterpret_cast<TOut *>(stage) + (j ^ (C::kSwap ? (j >> 3) & 4 : 0)), v);
            };
            if (OP == kBwd && row.tgt >= seg0 && row.tgt < seg0 + cols) {
                const int j = row.tgt - (int)seg0;
                if ((j >> 5) == lane && ((shown & ~touched) >> (j & 31) & 1u))
                    put_column(j, __fmul_rn(g, __fsub_rn(1.f, prob(elem(zs + j), q.itau, i1, l))));
            }
            for (int e = lane; e < (none ? 0 : listed); e += 32) {
                const int j = list[e];
                float z, y;
                uint32_t cw;
                if (!listed_y(j, z, cw, y)) continue;
                if (OP == kApply) {
                    put_column(j, __fmul_rn(y, q.itau));
                } else {
                    const float slope = cw ? (z > 0.f ? q.irep : q.rep) : 1.f;
                    const float hot = j == row.tgt - seg0 ? 1.f : 0.f;
                    put_column(j, __fmul_rn(__fmul_rn(g, __fsub_rn(hot, prob(y, q.itau, i1, l))), slope));
                }
            }
            __syncwarp();
            write_out<C::kSwap>(stage, orow, cols, io.vec_out, lane);
        }
        __syncwarp();  // the stage is free again
        prefetch(k + C::kStages);
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
    if (row.tgt == kInactive) {
        if (lane == 0) {
            logp[t] = 0.f;
            if (lse) lse[t] = 0.f;
        }
        return;
    }
    const bool has_tau = row.tgt >= 0 && rules.num_requests > 0 && rules.temperature;
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
        if (row.tgt < 0 || s != s) {
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

// Rows per block: one wave of two blocks per SM where kMaxRun allows it, so
// that a block counts a history as seldom as possible.
int rows_per_block(int64_t T, int64_t V, const DeviceInfo &di) {
    const int64_t slices = (V + kSliceCols - 1) / kSliceCols, blocks = (int64_t)di.sm_count * 2;
    const int64_t want = (T * slices + blocks - 1) / blocks;
    return (int)std::max<int64_t>(1, std::min<int64_t>(kMaxRun, want));
}

template <RulesOp OP, typename TIn, typename TOut>
cudaError_t launch(RulesIo io, const rk_logits_rules &r, const DeviceInfo &di, cudaStream_t st) {
    auto *kernel = rules_kernel<OP, TIn, TOut>;
    const size_t smem = Config<OP, TIn, TOut>::smem(r.bias_ids != nullptr);
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
