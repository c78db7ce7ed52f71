// logits_rules.cu -- logits under sampling rules: repetition, frequency and
// presence penalties, per-request biases, grammar masks and temperature (the
// definition stands at rk_logits_rules in rk.h), applied (kApply), scored
// (kLogp: selected logprob and log-sum-exp) and differentiated (kBwd).
//
// Decomposition.  A block works on a slice of kSliceCols columns and a run of
// consecutive rows.  Its warps own 1024 neighbouring columns each; in the
// first slice they own blocks of 64 columns in turn instead, because text is
// made of few tokens and those sit at the low ids where a vocabulary is
// ordered by frequency, so that its warps share them.  In the first slice,
// nowhere, everywhere (us): logp of 2048 x 32000 49, 67, -; logp of 8192 x
// 128256 506, 512, -; gradient of 4096 x 128256 in bf16 399, 392, -, and in
// fp32 without rules 524, 506, 579 (a warp's writes are then in short pieces).
// Each lane owns 32 neighbouring columns: one word of a grammar mask, and one
// word that tells which of them the rules touch (seen before, or biased).  The
// others need the temperature and the mask only.
//
// Data.  A warp copies its columns of the next row into shared memory of its
// own (cp.async, 16 bytes a lane, the mask words with them) while it works on
// the present one, so no barrier stands between the rows.  Rows that do not
// start on 16-byte boundaries are copied from the boundary before them and
// shifted on the way into registers (300 x 50257 without rules: logp
// 23.2 us, fp32 gradient 31.2; 21.6 and 26.5 at 50264, where they do).  What the
// rows say about themselves is read once per block.  Results of kApply and kBwd
// leave through the same memory, so that a warp writes whole lines although a
// lane owns 32 columns.  Each lane's 32 columns are followed by 16 bytes: they
// spread a quarter warp's 16-byte accesses over all banks, and hold the end of
// columns that do not start on a 16-byte boundary.
//
// History.  The block (its warps, each for itself, if they are few) counts a
// request's tokens of its slice in shared memory (one word per column: bit 31 in
// the prompt, bits 0-30 times produced).  Integer atomics only, so the order does
// not matter.  A row that has one token more than the row before (a packed
// training sequence) adds it to the counts without a barrier: its column belongs
// to one lane.  Longer steps add their tokens in the way a request's are counted;
// any other change counts anew.  Each warp lists its touched columns in ascending
// order, 32 of which its lanes take at a time; lanes that looped over their own
// would wait for the one with the most.
//
// Measured, 4096 x 128256 bf16 (us; bytes at the copy rate: logp 157, gradient in
// bf16 314 and in fp32 471, applied to bf16 314 and to fp32 471): without rules
// 202, 361, 524, 341, 491; with histories 250, 391, 569, 363, 532; with masks and
// biases too 272, 416, 590, 377, 549.  fp32 logits (314, 471, 628, 471, 628): 325,
// 517, 638, 491, 630; 344, 561, 668, 517, 643; 364, 583, 686, 532, 653.  Without
// rules the gradient and apply are bound by memory; logp of bf16, and the touched
// columns of all, by instruction latency: 16 warps per SM are what 128 registers
// and counts of 32 bits leave room for.
//
// Batch invariance: a warp's partial (max, sum) of a row is formed by a tree
// fixed by the columns' indices and by which of them are touched, and the
// partials are merged in a fixed order: nothing depends on T, on where the row
// sits or on how the rows were cut into runs.
#include <algorithm>
#include <type_traits>

#include "rk_device.cuh"
#include "rk_internal.h"

namespace rk {
namespace {

constexpr int kLaneCols = 32;
constexpr int kWarps = 8;
constexpr int kThreads = 32 * kWarps;
constexpr int kSliceCols = kThreads * kLaneCols;  // 8192 columns per block
constexpr int kMaxRun = 40;                    // rows per block at most
constexpr int kWarpTokens = 256;    // up to here a warp counts by itself
constexpr int kMaxBiases = 65534;  // per request: indices are kept in 16 bits
constexpr uint32_t kPromptBit = 0x80000000u;
constexpr uint32_t kNegInf2 = 0xFF80FF80u;  // two bf16 -inf
constexpr float kLn2 = 0.69314718055994531f;
// Below this, m c rounds by r <= 2^-12, and 1 - r ln 2 is 2^-r to (r ln 2)^2 / 2 <
// 2^-26; far above it, it is not even positive.
constexpr float kNearExponent = 8192.f;

enum RulesOp { kApply, kLogp, kBwd };

// Which of a slice's columns a warp's lane owns (see above).
struct Columns {
    bool mixed;  // the first slice
    // the first of a lane's columns
    __device__ __forceinline__ int first(int warp, int lane) const {
        return mixed ? ((lane >> 1) * kWarps + warp) * 64 + (lane & 1) * kLaneCols
                     : (warp * 32 + lane) * kLaneCols;
    }
    // the owner of a column
    __device__ __forceinline__ int warp(int c) const { return mixed ? (c >> 6) & (kWarps - 1) : c >> 10; }
    __device__ __forceinline__ int lane(int c) const {
        return mixed ? (c >> 9 << 1) | (c >> 5 & 1) : c >> 5 & 31;
    }
};

struct RulesIo {
    const void *logits;
    int64_t ld;
    const int64_t *targets;
    const int32_t *cu;
    int num_seqs;
    int64_t T, V;
    int run0, run;   // rows per block, of the first slice and of the others
    unsigned blocks0;  // the first slice's blocks
    const float *lse, *grad;  // kBwd
    const double *lse64;      // kBwd: instead of lse, or null
    void *out;       // kApply, kBwd
    int64_t ld_out;
    float2 *part;    // kLogp: [T][kWarps per slice] (max of y, sum relative to it)
    float *ytgt;     // kLogp: [T] y of the target, -inf when it is masked
    unsigned *err;
};

// What a row says about itself, as far as it concerns a slice.
constexpr int32_t kOk = 0, kInactive = -1, kBadTarget = -2, kBadRules = -3;
constexpr int32_t kNoToken = -1, kAnew = -2;
struct __align__(16) RowInfo {
    int32_t state;   // kOk, or another of these codes
    int32_t mrow;    // the row of the mask, or negative
    // how its history differs from the row before in this slice: by one token
    // (where: see place), by none, or else (kAnew)
    int32_t step;
    int32_t target;  // where the target is, or -1: not in this slice
};
// A column of the slice with the warp that owns it, and a flag.
__device__ __forceinline__ int32_t place(const Columns &own, int c, bool flag) {
    return c | own.warp(c) << 16 | (flag ? 1 << 24 : 0);
}
__device__ __forceinline__ int place_column(int32_t p) { return p & 0xffff; }
__device__ __forceinline__ int place_warp(int32_t p) { return p >> 16 & 0xff; }
__device__ __forceinline__ bool place_flag(int32_t p) { return p >> 24 != 0; }

__device__ __forceinline__ int32_t row_request(const rk_logits_rules &r, int64_t t) {
    return r.row_request ? r.row_request[t] : (r.num_requests > 0 ? (int32_t)t : 0);
}
__device__ __forceinline__ int32_t row_length(const rk_logits_rules &r, int64_t t) {
    return r.row_length ? max(r.row_length[t], 0) : 0x7fffffff;
}

template <RulesOp OP>
__device__ __forceinline__ int32_t row_state(const RulesIo &io, const rk_logits_rules &r, int64_t t,
                                             int64_t tgt, int32_t mrow) {
    const int32_t req = row_request(r, t);
    if ((OP != kApply && !row_active(t, tgt, io.cu, io.num_seqs)) || (r.row_request && req == -1))
        return kInactive;
    if (req < 0 || (r.num_requests > 0 && req >= r.num_requests) || (mrow >= 0 && mrow >= r.mask_rows))
        return kBadRules;
    return OP != kApply && tgt >= io.V ? kBadTarget : kOk;
}
__device__ __forceinline__ int32_t row_mask(const rk_logits_rules &r, int64_t t) {
    return r.mask ? (r.row_mask ? r.row_mask[t] : (int32_t)t) : -1;
}

template <RulesOp OP>
__device__ __forceinline__ RowInfo row_info(const RulesIo &io, const rk_logits_rules &r, int64_t t,
                                            const Columns &own, int64_t slice0, int width) {
    const int64_t tgt = OP == kApply ? -1 : io.targets[t];
    RowInfo i;
    i.mrow = row_mask(r, t);
    i.state = row_state<OP>(io, r, t, tgt, i.mrow);
    i.step = kAnew;
    const int64_t c = tgt - slice0;
    i.target = tgt >= 0 && c >= 0 && c < width ? place(own, (int)c, false) : -1;
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
    int32_t ok;
};

// A row's, with how many of the tokens it has seen.
struct RowRequest {
    Request q;
    int32_t id, len;
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
            s.prompt = r.prompt_lengths ? max(r.prompt_lengths[q], 0) : 0;
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

// How a row's history differs from the row before: by the token *v, by none, or
// else (RowInfo::step before the token is placed: >= 0, kNoToken, kAnew).
__device__ __forceinline__ int32_t find_step(const RowInfo &before, const RowRequest &rb, const RowInfo &row,
                                             const RowRequest &rr, int64_t *v) {
    if (row.state != kOk || before.state != kOk || rr.id != rb.id || !rr.q.ok) return kAnew;
    if (rr.len == rb.len) return kNoToken;
    if (rr.len != rb.len + 1) return kAnew;
    *v = rr.q.tokens[rb.len];
    return 0;
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
__device__ __forceinline__ float warp_max(float v) {
    float d;
    asm volatile("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(d) : "f"(v));
    return d;
}
// A lane's 32 columns as 16-byte pieces, and the bytes from lane to lane.
template <typename T>
struct Lane {
    static constexpr int kCols = 16 / (int)sizeof(T), kPieces = kLaneCols / kCols;
    static constexpr int kPitch = kLaneCols * (int)sizeof(T) + 16;
    // Spread over a warp, lane l has pieces l, l + 32, ...: the lanes whose
    // pieces are had at a time, and the columns from one time to the next.
    static constexpr int kLanes = 32 / kPieces;
    static constexpr int kStep = kLanes * kLaneCols, kMixedStep = kLanes / 2 * kWarps * 64;
};

__device__ __forceinline__ void cp_async16(uint32_t dst, const void *src) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
// its first `bytes`, zeros behind them
__device__ __forceinline__ void cp_async16_part(uint32_t dst, const void *src, int bytes) {
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

// Bytes from the 16-byte boundary at or before p to p.
__device__ __forceinline__ int shift_of(const void *p) { return (int)(reinterpret_cast<uintptr_t>(p) & 15); }

// Copies of a warp's columns of a row's slice into a stage.  Nothing outside
// the slice (of `width` columns) is read.
//
// Rows on 16-byte boundaries: `from` and `dst` are those of the lane's first
// piece, which is piece `lane` of the warp's; it has pieces lane, lane + 32, ...
template <typename T>
__device__ __forceinline__ int first_piece(const Columns &own, int warp, int lane) {
    using L = Lane<T>;
    return own.first(warp, lane / L::kPieces) + lane % L::kPieces * L::kCols;
}
template <typename T>
__device__ __forceinline__ int first_piece_at(int lane) {
    using L = Lane<T>;
    return lane / L::kPieces * L::kPitch + lane % L::kPieces * 16;
}
template <typename T>
__device__ __forceinline__ void copy_pieces(uint32_t dst, const T *from, int left, bool whole, bool mixed) {
    using L = Lane<T>;
    if (!whole) {
        const int step = mixed ? L::kMixedStep : L::kStep;
#pragma unroll 1
        for (int i = 0; i < L::kPieces; ++i) {
            const int n = min(L::kCols, left - i * step);
            if (n > 0) cp_async16_part(dst + i * L::kLanes * L::kPitch, from + i * step, n * (int)sizeof(T));
        }
    } else if (mixed) {
#pragma unroll
        for (int i = 0; i < L::kPieces; ++i) cp_async16(dst + i * L::kLanes * L::kPitch, from + i * L::kMixedStep);
    } else {
#pragma unroll
        for (int i = 0; i < L::kPieces; ++i) cp_async16(dst + i * L::kLanes * L::kPitch, from + i * L::kStep);
    }
}

// Other rows (`src`: the slice's first element): every 64 columns (a pair of
// lanes') as the pieces from the 16-byte boundary before them on, one more than
// they fill, which goes behind the second lane's.  The columns sit
// shift_of(src) bytes further in.  Of the first piece the bytes before the
// columns belong to the columns or the row before; next to the tensor's first
// element (`top`) they may not, and it is copied by element.
template <typename T>
__device__ __forceinline__ void copy_shifted(unsigned char *stage, const T *src, int width, bool top,
                                             const Columns &own, int warp, int lane) {
    using L = Lane<T>;
    constexpr int kSize = (int)sizeof(T);
    const int shift = shift_of(src), end = shift + width * kSize;
    const char *base = reinterpret_cast<const char *>(src) - shift;
    const int first = first_piece<T>(own, warp, lane) * kSize, step = (own.mixed ? L::kMixedStep : L::kStep) * kSize;
    const uint32_t dst = smem_u32(stage) + first_piece_at<T>(lane);
#pragma unroll
    for (int i = 0; i < L::kPieces; ++i) {
        const int b = first + i * step, n = min(16, end - b);
        if (top && shift > 0 && b == 0) {
            for (int e = shift; e < n; e += kSize)
                *reinterpret_cast<T *>(stage + e) = *reinterpret_cast<const T *>(base + e);
        } else if (n > 0) {
            cp_async16_part(dst + i * L::kLanes * L::kPitch, base + b, n);
        }
    }
    if (shift > 0 && lane < 16) {
        const int o = 2 * lane + 1, b = (own.first(warp, o) + kLaneCols) * kSize, n = min(16, end - b);
        if (n > 0) cp_async16_part(smem_u32(stage) + o * L::kPitch + kLaneCols * kSize, base + b, n);
    }
}

// f(std::integral_constant<int, words>()), words = 0 .. 3 known at run time.
template <typename F>
__device__ __forceinline__ void with_words(int words, F f) {
    switch (words) {
    case 0: f(std::integral_constant<int, 0>{}); break;
    case 1: f(std::integral_constant<int, 1>{}); break;
    case 2: f(std::integral_constant<int, 2>{}); break;
    default: f(std::integral_constant<int, 3>{}); break;
    }
}

// A lane's columns out of what copy_shifted made.
template <typename T>
__device__ __forceinline__ void load_shifted(uint4 (&w)[Lane<T>::kPieces], const unsigned char *stage, int shift,
                                             int lane) {
    using L = Lane<T>;
    uint32_t r[4 * L::kPieces + 4];
    const unsigned char *p = stage + lane * L::kPitch;
#pragma unroll
    for (int i = 0; i <= L::kPieces; ++i) {
        const int next = lane & 1 ? 0 : 16;  // the second lane's first piece
        const uint4 v = *reinterpret_cast<const uint4 *>(p + 16 * i + (i == L::kPieces ? next : 0));
        r[4 * i] = v.x;
        r[4 * i + 1] = v.y;
        r[4 * i + 2] = v.z;
        r[4 * i + 3] = v.w;
    }
    const int bits = shift & 2 ? 16 : 0;
    with_words(shift >> 2, [&](auto words) {
        constexpr int S = decltype(words)::value;
        auto word = [&](int i) {
            return sizeof(T) == 2 ? __funnelshift_r(r[i + S], r[i + S + 1], bits) : r[i + S];
        };
#pragma unroll
        for (int i = 0; i < L::kPieces; ++i)
            w[i] = make_uint4(word(4 * i), word(4 * i + 1), word(4 * i + 2), word(4 * i + 3));
    });
}

// Where column j of lane l is in such a stage.
template <typename T>
__device__ __forceinline__ T *shifted_at(unsigned char *stage, int shift, int l, int j) {
    using L = Lane<T>;
    const int o = (j & 63) * (int)sizeof(T) + shift;
    return reinterpret_cast<T *>(stage + (l >> 1) * 2 * L::kPitch + o + (o >= kLaneCols * (int)sizeof(T) ? 16 : 0));
}

// ---- history ----

// Shared memory of a block.
struct Shared {
    uint32_t *count;    // [kSliceCols]
    uint32_t *touched;  // [kThreads]: bit c % 32 of word c / 32 for slice column c
    uint16_t *list;     // [kWarps][1024]: each warp's touched columns, ascending
    uint16_t *bias;     // [kSliceCols], or null: 1 + the index of the column's bias, 0: none
    RowInfo *rows;      // [kMaxRun]
    RowRequest *requests;  // [kMaxRun]
    unsigned char *rings;
};
constexpr int kWarpCols = 32 * kLaneCols;

extern __shared__ uint4 rules_smem[];

// Its layout: counts, touched words, rows and their requests, lists, bias indices
// if there are biases, and then the warps' rings.
__device__ __forceinline__ Shared shared_view(bool has_bias) {
    Shared sh;
    sh.count = reinterpret_cast<uint32_t *>(rules_smem);
    sh.touched = sh.count + kSliceCols;
    sh.rows = reinterpret_cast<RowInfo *>(sh.touched + kThreads);
    sh.requests = reinterpret_cast<RowRequest *>(sh.rows + kMaxRun);
    sh.list = reinterpret_cast<uint16_t *>(sh.requests + kMaxRun);
    sh.bias = has_bias ? sh.list + kSliceCols : nullptr;
    sh.rings = reinterpret_cast<unsigned char *>(sh.list + (has_bias ? 2 : 1) * kSliceCols);
    return sh;
}

__device__ __forceinline__ void mark(const Shared &sh, int c) {
    atomicOr(&sh.touched[c >> 5], 1u << (c & 31));
}

// The functions below run seldom: out of line, and with plain arguments, so
// that the row loop keeps its values in registers.

// Tokens into the counts of the columns [slice0, slice0 + width): a thread's
// N loads of v from i0 on, kThreads apart, and adding them.
template <int N, int STEP = kThreads>
__device__ __forceinline__ void load_tokens(int64_t (&v)[N], const int64_t *tokens, int32_t i0, int32_t to) {
#pragma unroll
    for (int k = 0; k < N; ++k) v[k] = k * STEP < to - i0 ? tokens[i0 + k * STEP] : -1;
}
template <int N>
__device__ __forceinline__ void add_tokens(const Shared &sh, const int64_t (&v)[N], int32_t i0, int32_t prompt,
                                           int64_t slice0, int width) {
#pragma unroll
    for (int k = 0; k < N; ++k) {
        const int64_t c = v[k] - slice0;
        if (v[k] >= 0 && c >= 0 && c < width) {
            if (k * kThreads < prompt - i0)
                atomicOr(&sh.count[c], kPromptBit);
            else
                atomicAdd(&sh.count[c], 1u);
            mark(sh, (int)c);
        }
    }
}
constexpr int kTokenBatch = 8;  // loads in flight per thread

// Block-wide: tokens [from, to) of a request into the counts.
__device__ __noinline__ void count_tokens(const int64_t *tokens, int32_t prompt, int32_t from, int32_t to,
                                          int64_t slice0, int width) {
    const Shared sh = shared_view(false);
    for (int64_t i0 = from + (int64_t)threadIdx.x; i0 < to; i0 += kTokenBatch * kThreads) {
        int64_t v[kTokenBatch];
        load_tokens(v, tokens, (int32_t)i0, to);
        add_tokens(sh, v, (int32_t)i0, prompt, slice0, width);
    }
}

__device__ __forceinline__ void clear_counts(const Shared &sh) {
    for (int k = threadIdx.x; k < kSliceCols / 4; k += kThreads)
        reinterpret_cast<uint4 *>(sh.count)[k] = make_uint4(0, 0, 0, 0);
    sh.touched[threadIdx.x] = 0;
    if (sh.bias)
        for (int k = threadIdx.x; k < kSliceCols / 8; k += kThreads)
            reinterpret_cast<uint4 *>(sh.bias)[k] = make_uint4(0, 0, 0, 0);
}

// Block-wide: a request's biases (`ids`) and its first `len` tokens.  Of biases
// for one column the last counts: the count words find it.  What memory held
// before goes, unless it is `clear` already; the first loads are on their way
// meanwhile.
__device__ __noinline__ void count_request(bool has_bias, bool clear, const int64_t *ids, int32_t nbias,
                                           const int64_t *tokens, int32_t prompt, int32_t len, int64_t slice0,
                                           int width) {
    const Shared sh = shared_view(has_bias);
    const int32_t i0 = (int32_t)threadIdx.x;
    const int64_t bias = i0 < nbias ? ids[i0] : -1;
    int64_t first[kTokenBatch];
    load_tokens(first, tokens, i0, len);
    if (!clear) {
        __syncthreads();
        clear_counts(sh);
        __syncthreads();
    }
    if (nbias > 0) {
        for (int k = i0; k < nbias; k += kThreads) {
            const int64_t v = k == i0 ? bias : ids[k], c = v - slice0;
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
    add_tokens(sh, first, i0, prompt, slice0, width);
    for (int64_t i = i0 + (int64_t)kTokenBatch * kThreads; i < len; i += kTokenBatch * kThreads) {
        load_tokens(first, tokens, (int32_t)i, len);
        add_tokens(sh, first, (int32_t)i, prompt, slice0, width);
    }
}

// A warp's part of that by itself, with no barrier: the biases (if the request is
// new) and tokens [from, to), of which it adds those of its own columns.
__device__ __noinline__ void count_warp(bool has_bias, const int64_t *ids, int32_t nbias, const int64_t *tokens,
                                        int32_t prompt, int32_t from, int32_t to, int64_t slice0, int width) {
    const Shared sh = shared_view(has_bias);
    const Columns own{slice0 == 0};
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    auto ours = [&](int64_t v) {
        const uint64_t c = (uint64_t)v - (uint64_t)slice0;
        return c < (uint64_t)width && own.warp((int)c) == warp;
    };
    int64_t v[kTokenBatch];
    load_tokens<kTokenBatch, 32>(v, tokens, from + lane, to);
    if (nbias > 0) {
        for (int k = lane; k < nbias; k += 32) {
            const int64_t b = ids[k];
            if (ours(b)) {
                atomicMax(&sh.count[b - slice0], (uint32_t)(k + 1));
                mark(sh, (int)(b - slice0));
            }
        }
        __syncwarp();
        const int mine = own.first(warp, lane);
        for (uint32_t b = sh.touched[mine >> 5]; b; b &= b - 1) {
            const int c = mine + __ffs(b) - 1;
            sh.bias[c] = (uint16_t)sh.count[c];
            sh.count[c] = 0;
        }
        __syncwarp();
    }
    for (int64_t i = from + lane;;) {
#pragma unroll
        for (int k = 0; k < kTokenBatch; ++k)
            if (ours(v[k])) {
                const int c = (int)(v[k] - slice0);
                if (32 * k < prompt - (int32_t)i)
                    atomicOr(&sh.count[c], kPromptBit);
                else
                    atomicAdd(&sh.count[c], 1u);
                mark(sh, c);
            }
        i += 32 * kTokenBatch;
        if (i - lane >= to) break;
        load_tokens<kTokenBatch, 32>(v, tokens, (int32_t)i, to);
    }
    __syncwarp();
}

// A warp's list of its touched columns (of the slice, ascending) from its
// lanes' bits, `own`: the lane's first column; returns their number.
__device__ __forceinline__ int make_list(uint16_t *list, uint32_t touched, int own, int lane) {
    const int mine = __popc(touched);
    int incl = mine;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, incl, off);
        if (lane >= off) incl += y;
    }
    int at = incl - mine;
    for (uint32_t b = touched; b; b &= b - 1)
        list[at++] = (uint16_t)(own + __ffs(b) - 1);
    return __shfl_sync(0xffffffffu, incl, 31);
}

// exp(y / temperature - lse), 1 / temperature = id + i1, i1 >= 0 (-inf stays -inf);
// `low`: -log2e times what of the log-sum-exp is not in lse.
__device__ __forceinline__ float prob(float y, float id, float i1, float lse, float low) {
    float x = __fmaf_rn(y, id, -lse);
    if (i1 > 0.f) x = __fmaf_rn(y, i1, x);
    return ex2(__fmaf_rn(x, kLog2e, low));
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

// fp32 pieces: bit 4 i + j of `keep` belongs to column j of piece i.
__device__ __forceinline__ void keep_columns(uint4 (&w)[8], uint32_t keep) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        if (!(keep >> (4 * i) & 1u)) w[i].x = 0xff800000u;
        if (!(keep >> (4 * i + 1) & 1u)) w[i].y = 0xff800000u;
        if (!(keep >> (4 * i + 2) & 1u)) w[i].z = 0xff800000u;
        if (!(keep >> (4 * i + 3) & 1u)) w[i].w = 0xff800000u;
    }
}

// A piece's columns as pairs of fp32.
template <typename T>
__device__ __forceinline__ void pairs_of(const uint4 &w, uint64_t (&z)[4]) {
    const uint32_t q[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int j = 0; j < 16 / (int)sizeof(T) / 2; ++j)
        z[j] = sizeof(T) == 2 ? pair(bf16_lo(q[j]), bf16_hi(q[j]))
                              : pair(__uint_as_float(q[(2 * j) & 3]), __uint_as_float(q[(2 * j + 1) & 3]));
}

// Shared memory of a block: what shared_view lays out, and a ring of stages
// per warp.  A stage holds the warp's logits and afterwards its results, and
// its mask words.  Two blocks run per SM, which leaves room for two stages of
// bf16 (logp of 4096 x 128256 without rules 219 us with one, 202 with two; its
// gradient in bf16 425 and 361).
template <RulesOp OP, typename TIn, typename TOut>
struct Config {
    static constexpr bool kWider = OP != kLogp && sizeof(TOut) > sizeof(TIn);
    static constexpr int kStages = sizeof(TIn) == 2 && !kWider ? 2 : 1;
    static constexpr int kMaskAt = 32 * (kWider ? Lane<TOut>::kPitch : Lane<TIn>::kPitch);
    static constexpr int kStageBytes = kMaskAt + 32 * 4;
    static size_t smem(bool bias) {
        return (size_t)(kSliceCols + kThreads) * 4 + kMaxRun * (sizeof(RowInfo) + sizeof(RowRequest)) +
               (size_t)kSliceCols * (bias ? 4 : 2) + (size_t)kWarps * kStages * kStageBytes;
    }
};

// Writes a warp's results from its stage to the row's slice, of `width` columns.
template <typename T>
__device__ __forceinline__ void write_part(T *to, const uint4 &v, int n) {  // n of a piece's columns
    if (n >= Lane<T>::kCols) {
        *reinterpret_cast<uint4 *>(to) = v;
    } else if (n > 0) {
        const uint32_t q[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int j = 0; j < Lane<T>::kCols; ++j)
            if (j < n) {
                if constexpr (sizeof(T) == 4)
                    to[j] = __uint_as_float(q[j]);
                else
                    to[j] = (uint16_t)(q[j >> 1] >> (16 * (j & 1)));
            }
    }
}

// dst on a 16-byte boundary.
template <typename T>
__device__ __forceinline__ void write_pieces(const unsigned char *stage, T *dst, int width, const Columns &own,
                                             int warp, int lane) {
    using L = Lane<T>;
    if (width == kSliceCols) {
        const int o = lane / L::kPieces, part = lane % L::kPieces;
        const unsigned char *from = stage + o * L::kPitch + 16 * part;
        T *to = dst + own.first(warp, o) + part * L::kCols;
        const int step = own.mixed ? L::kMixedStep : L::kStep;
#pragma unroll
        for (int i = 0; i < L::kPieces; ++i)
            *reinterpret_cast<uint4 *>(to + i * step) =
                *reinterpret_cast<const uint4 *>(from + i * L::kLanes * L::kPitch);
    } else {
#pragma unroll 4
        for (int o = 0; o < 32; ++o) {
            const int j = own.first(warp, o) + lane;
            if (j < width) dst[j] = reinterpret_cast<const T *>(stage + o * L::kPitch)[lane];
        }
    }
}

// Elsewhere.  Every 64 columns: the pieces that start on boundaries, and the
// columns before and behind them one by one.
template <typename T>
__device__ __forceinline__ void write_shifted(const unsigned char *stage, T *dst, int width, const Columns &own,
                                              int warp, int lane) {
    using L = Lane<T>;
    constexpr int kSize = (int)sizeof(T), kPair = 2 * L::kPieces;  // pieces of 64 columns
    const int head = (16 - shift_of(dst)) / kSize % L::kCols;      // columns before the first piece
    const int bits = head * kSize & 2 ? 16 : 0;
    with_words(head * kSize >> 2, [&](auto words) {
        constexpr int S = decltype(words)::value;
#pragma unroll
        for (int i = 0; i < L::kPieces; ++i) {
            const int x = lane + 32 * i, pair = x / kPair, p = x % kPair, q = head + p * L::kCols;
            if (q + L::kCols > 64) continue;
            const unsigned char *from = stage + 2 * pair * L::kPitch;
            const uint4 a = *reinterpret_cast<const uint4 *>(from + 16 * p + (p >= L::kPieces ? 16 : 0));
            const uint4 b = *reinterpret_cast<const uint4 *>(from + 16 * p + (p + 1 >= L::kPieces ? 32 : 16));
            const uint32_t r[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
            auto word = [&](int k) {
                return kSize == 2 ? __funnelshift_r(r[k + S], r[k + S + 1], bits) : r[k + S];
            };
            const int c = own.first(warp, 2 * pair) + q;
            write_part(dst + c, make_uint4(word(0), word(1), word(2), word(3)), width - c);
        }
    });
    if (head > 0) {
#pragma unroll
        for (int i = 0; i < L::kCols / 2; ++i) {
            const int x = lane + 32 * i, pair = x / L::kCols, e = x % L::kCols;
            const int q = e < head ? e : 64 - L::kCols + e, o = 2 * pair + (q >> 5);
            const int c = own.first(warp, o) + (q & 31);
            if (c < width) dst[c] = reinterpret_cast<const T *>(stage + o * L::kPitch)[q & 31];
        }
    }
}

// VEC: every row of the logits, and of what is written, starts on a 16-byte
// boundary.
template <RulesOp OP, typename TIn, typename TOut, bool VEC>
__global__ void __launch_bounds__(kThreads, 2)
    rules_kernel(const __grid_constant__ RulesIo io, const __grid_constant__ rk_logits_rules rules) {
    using C = Config<OP, TIn, TOut>;
    using L = Lane<TIn>;
    const Shared sh = shared_view(rules.bias_ids != nullptr);
    RowInfo *rows = sh.rows;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    unsigned char *ring = sh.rings + warp * C::kStages * C::kStageBytes;
    clear_counts(sh);
    // Launched with programmatic stream serialisation: wait until the previous
    // kernel of the stream has completed before reading or writing anything.
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");

    const int64_t slices = (io.V + kSliceCols - 1) / kSliceCols;
    int64_t slice = 0, t0 = (int64_t)blockIdx.x * io.run0;  // the first slice's blocks come first
    int run = io.run0;
    if (blockIdx.x >= io.blocks0) {
        const unsigned b = blockIdx.x - io.blocks0;
        slice = 1 + b % (slices - 1);
        t0 = b / (slices - 1) * io.run;
        run = io.run;
    }
    const int64_t slice0 = slice * kSliceCols;
    const int width = (int)min((int64_t)kSliceCols, io.V - slice0);
    const int n = (int)min((int64_t)run, io.T - t0);
    const int64_t words = (io.V + 31) / 32;
    const Columns own{slice == 0};
    const int mine = own.first(warp, lane);  // the lane's first column
    const uint32_t inside =
        width >= mine + 32 ? 0xffffffffu : width > mine ? (1u << (width - mine)) - 1u : 0u;
    uint32_t *my_word = sh.touched + (mine >> 5);
    uint16_t *list = sh.list + warp * kWarpCols;

    const TIn *zslice = reinterpret_cast<const TIn *>(io.logits) + t0 * io.ld + slice0;
    TOut *oslice = OP == kLogp ? nullptr : reinterpret_cast<TOut *>(io.out) + t0 * io.ld_out + slice0;
    float2 *parts = OP == kLogp ? io.part + (t0 * slices + slice) * kWarps + warp : nullptr;
    // Copies run ahead of the rows: the next row to copy, its logits (VEC: the
    // lane's first piece of them), and its stage.
    int ahead = 0;
    const TIn *from = zslice + (VEC ? first_piece<TIn>(own, warp, lane) : 0);
    unsigned char *into = ring;
    unsigned char *const both = ring + (C::kStages - 1) * C::kStageBytes;  // stage a + stage b - ring
    auto other_stage = [&](unsigned char *stage) { return both - (stage - ring); };
    const bool whole = width == kSliceCols;
    const int left = width - (VEC ? first_piece<TIn>(own, warp, lane) : 0);
    auto copy_logits = [&] {
        if constexpr (VEC)
            copy_pieces(smem_u32(into) + first_piece_at<TIn>(lane), from, left, whole, own.mixed);
        else
            copy_shifted(into, from, width, slice == 0 && (t0 + ahead) * io.ld < 16 / (int)sizeof(TIn), own, warp, lane);
    };
    auto next_copy = [&] {
        ++ahead;
        from += io.ld;
        into = other_stage(into);
    };
    auto prefetch = [&](bool logits) {
        if (ahead < n) {
            const int2 r = *reinterpret_cast<const int2 *>(&rows[ahead]);  // state, mrow
            if (r.x == kOk) {
                if (logits) copy_logits();
                if (r.y >= 0 && inside)
                    cp_async4(smem_u32(into + C::kMaskAt) + 4 * lane,
                              rules.mask + (int64_t)r.y * words + ((slice0 + mine) >> 5));
            }
        }
        cp_commit();
        next_copy();
    };
    // The first rows' logits are on their way before anything about the rows is known.
    for (int k = 0; k < C::kStages; ++k) {
        if (ahead < n) copy_logits();
        next_copy();
    }
    ahead = 0;
    from -= C::kStages * io.ld;
    into = ring;

    RowRequest *requests = sh.requests;
    for (int k = threadIdx.x; k < n; k += kThreads) {
        rows[k] = row_info<OP>(io, rules, t0 + k, own, slice0, width);
        if (rows[k].state == kOk) {
            const int32_t id = row_request(rules, t0 + k);
            const Request r = load_request(rules, id);
            requests[k] = RowRequest{r, id, min(row_length(rules, t0 + k), r.ntok)};
        }
    }
    __syncthreads();
    for (int k = 0; k < C::kStages; ++k) prefetch(false);

    int32_t cur = -1;
    int done = -1;      // the last row whose history is counted
    bool clear = true;  // nothing counted yet
    uint32_t touched = 0;
    int listed = 0;  // touched columns of the warp
    Request q{};
    // Row k's request, or a step of more than one token.  Short histories each
    // warp counts for itself, so that no barrier holds the rows back; long ones
    // the whole block (apply of 256 requests with up to 4096 tokens, warps alone up
    // to 0, 128, 256, 512, 1024, 2048 tokens: 80.0, 75.7, 74.7, 74.1, 76.7, 85.8 us;
    // logp of 64 on the device 15.5, 15.2, 15.4, 15.5, 21, 26; logp of 8192 packed
    // rows 506, 506, 506, 507, 514, 528).
    auto start_row = [&](int k) {
        const bool other = requests[k].id != cur;
        cur = requests[k].id;
        q = requests[k].q;
        if (!q.ok) return;
        const int32_t len = requests[k].len;
        const int32_t counted = other ? 0 : requests[done].len;
        const bool anew = other || len < counted;
        if (clear && q.ntok == 0 && q.nbias == 0) return;  // nothing touched, as before
        if ((int64_t)len + (anew ? q.nbias : -counted) <= kWarpTokens) {
            if (anew) {
                for (int e = lane; e < listed; e += 32) {
                    sh.count[list[e]] = 0;
                    if (sh.bias) sh.bias[list[e]] = 0;
                }
                touched = 0;
            }
            *my_word = touched;
            __syncwarp();
            count_warp(sh.bias != nullptr, rules.bias_ids + q.bias0, anew ? q.nbias : 0, q.tokens, q.prompt,
                       anew ? 0 : counted, len, slice0, width);
        } else {
            if (anew) {
                count_request(sh.bias != nullptr, clear, rules.bias_ids + q.bias0, q.nbias, q.tokens, q.prompt, len,
                              slice0, width);
            } else {
                __syncthreads();
                *my_word = touched;
                __syncthreads();
                count_tokens(q.tokens, q.prompt, counted, len, slice0, width);
            }
            __syncthreads();
        }
        clear = false;
        touched = *my_word;
        listed = make_list(list, touched, mine, lane);
    };
    {
        static_assert(kMaxRun <= kThreads);
        const int k = (int)threadIdx.x;
        int64_t v = -1;
        int32_t step = kAnew;
        if (k > 0 && k < n) step = find_step(rows[k - 1], requests[k - 1], rows[k], requests[k], &v);
        if (rows[0].state == kOk) start_row(0);
        if (step == 0) {
            const int64_t c = v - slice0;
            step = v >= 0 && c >= 0 && c < width ? place(own, (int)c, requests[k - 1].len < requests[k].q.prompt)
                                                 : kNoToken;
        }
        if (k < n) rows[k].step = k > 0 ? step : kNoToken;  // row 0 is started
        __syncthreads();
    }
    // kBwd: lse (and what a 64-bit one has beyond it, times -log2e) and gradient of
    // rows k & ~31 + lane
    float lse_of = 0.f, low_of = 0.f, grad_of = 0.f;
    int held = -1;
    unsigned char *now = ring;  // row k's stage
    for (int k = 0; k < n;) {
        if (rows[k].state == kOk && rows[k].step == kAnew) start_row(k);
        // A row without a result, or without usable rules.
        if (rows[k].state != kOk || !q.ok) {
            const int32_t state = rows[k].state;
            const float v = state == kInactive ? 0.f : __int_as_float(0x7fc00000);
            if (state != kInactive) {
                if (slice == 0 && threadIdx.x == 0) {
                    atomicOr(io.err, state == kBadTarget ? kErrTargetRange : kErrRules);
                    if (OP == kLogp) io.ytgt[t0 + k] = v;
                }
                if (OP == kLogp && lane == 0) *parts = make_float2(0.f, v);
            }
            if (OP == kBwd || (OP == kApply && state != kInactive))
#pragma unroll 1
                for (int o = 0; o < 32; ++o) {
                    const int c = own.first(warp, o) + lane;
                    if (c < width) put(oslice + c, v);
                }
            parts += slices * kWarps;
            oslice += io.ld_out;
            cp_wait<0>();
            prefetch(true);
            now = other_stage(now);
            ++k;
            continue;
        }
        // Rows of the request, each warp for itself.
        const float c = __fmul_rn(kLog2e, q.itau);
        // Single columns: a column's logit in a stage, a touched one's y from its
        // logit, and whether the mask allows a column.
        auto at = [&](unsigned char *stage, int shift, int j) {
            if constexpr (VEC)
                return reinterpret_cast<TIn *>(stage + own.lane(j) * L::kPitch) + (j & 31);
            else
                return shifted_at<TIn>(stage, shift, own.lane(j), j);
        };
        auto touched_y = [&](int j, float z) {
            const int bi = sh.bias ? sh.bias[j] : 0;
            return rule_y(z, sh.count[j], bi ? rules.bias_values[q.bias0 + bi - 1] : 0.f, q);
        };
        auto allowed = [&](const unsigned char *stage, int mrow, int j) {
            return mrow < 0 || (reinterpret_cast<const uint32_t *>(stage + C::kMaskAt)[own.lane(j)] >> (j & 31) & 1u);
        };
        auto load_pieces = [&](uint4 (&w)[L::kPieces], const unsigned char *stage, int shift) {
            if constexpr (VEC) {
#pragma unroll
                for (int i = 0; i < L::kPieces; ++i)
                    w[i] = *reinterpret_cast<const uint4 *>(stage + lane * L::kPitch + 16 * i);
            } else {
                load_shifted<TIn>(w, stage, shift, lane);
            }
        };

        // kLogp of rows k .. k + R - 1, whose histories are the same here.  Two
        // rows at a time share the list, and each fills the other's latencies.
        auto score = [&](auto rows_at_once) {
            constexpr int R = decltype(rows_at_once)::value;
            unsigned char *stage[R];
            int shift[R];
            RowInfo row[R];
            uint32_t live[R];  // columns the mask allows
#pragma unroll
            for (int r = 0; r < R; ++r) {
                stage[r] = r == 0 ? now : other_stage(now);
                shift[r] = VEC ? 0 : shift_of(zslice + (k + r) * io.ld);
                row[r] = rows[k + r];
                live[r] = inside;
                if (row[r].mrow >= 0)
                    live[r] &= reinterpret_cast<const uint32_t *>(stage[r] + C::kMaskAt)[lane];
                if (row[r].target >= 0 && place_warp(row[r].target) == warp) {
                    const int j = place_column(row[r].target);
                    if (own.lane(j) == lane) {
                        float y = -INFINITY;
                        if (live[r] >> (j & 31) & 1u) {
                            y = elem(at(stage[r], shift[r], j));
                            if (touched >> (j & 31) & 1u) y = touched_y(j, y);
                        }
                        io.ytgt[t0 + k + r] = y;
                    }
                    __syncwarp();
                }
            }
            // the touched columns, 32 at a time: their y are taken here (the first in
            // y0, the others as a running maximum and sum), and their logits become
            // -inf for the lanes that own them
            float mt[R], st[R], y0[R];
#pragma unroll
            for (int r = 0; r < R; ++r) {
                mt[r] = y0[r] = -INFINITY;
                st[r] = 0.f;
            }
            if (listed > 0) {
                if (lane < listed) {
                    const int j = list[lane];
#pragma unroll
                    for (int r = 0; r < R; ++r) {
                        TIn *zj = at(stage[r], shift[r], j);
                        if (allowed(stage[r], row[r].mrow, j)) y0[r] = touched_y(j, elem(zj));
                        put(zj, -INFINITY);
                    }
                }
                for (int e0 = 32 + lane; e0 - lane < listed; e0 += 128)
#pragma unroll
                    for (int r = 0; r < R; ++r) {
                        float y[4];
#pragma unroll
                        for (int u = 0; u < 4; ++u) {
                            y[u] = -INFINITY;
                            if (e0 + 32 * u < listed) {
                                const int j = list[e0 + 32 * u];
                                TIn *zj = at(stage[r], shift[r], j);
                                if (allowed(stage[r], row[r].mrow, j)) y[u] = touched_y(j, elem(zj));
                                put(zj, -INFINITY);
                            }
                        }
                        const float mn = fmaxf(fmaxf(mt[r], fmaxf(y[0], y[1])), fmaxf(y[2], y[3]));
                        const float ref = mn == -INFINITY ? 0.f : mn;
                        if (mt[r] != -INFINITY)
                            st[r] = __fmul_rn(st[r], ex2(__fmul_rn(__fsub_rn(mt[r], ref), c)));
#pragma unroll
                        for (int u = 0; u < 4; ++u)
                            st[r] = __fadd_rn(st[r], ex2(__fmul_rn(__fsub_rn(y[u], ref), c)));
                        mt[r] = mn;
                    }
                __syncwarp();
            }
            uint4 w[R][L::kPieces];
#pragma unroll
            for (int r = 0; r < R; ++r) load_pieces(w[r], stage[r], shift[r]);
            __syncwarp();  // the stages are free again
#pragma unroll
            for (int r = 0; r < R; ++r) prefetch(true);
            // the other columns: one maximum, then the terms relative to it
            float ref[R], rc[R], m[R];
            bool far = false;
#pragma unroll
            for (int r = 0; r < R; ++r) {
                if (!__all_sync(0xffffffffu, live[r] == 0xffffffffu)) keep_columns(w[r], live[r]);
                if constexpr (sizeof(TIn) == 2) {
                    uint32_t x[4];
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        x[i] = max_bf16x2(max_bf16x2(w[r][i].x, w[r][i].y), max_bf16x2(w[r][i].z, w[r][i].w));
                    x[0] = max_bf16x2(max_bf16x2(x[0], x[1]), max_bf16x2(x[2], x[3]));
                    m[r] = fmaxf(bf16_lo(x[0]), bf16_hi(x[0]));
                } else {
                    float x[8];
#pragma unroll
                    for (int i = 0; i < 8; ++i)
                        x[i] = fmaxf(fmaxf(__uint_as_float(w[r][i].x), __uint_as_float(w[r][i].y)),
                                     fmaxf(__uint_as_float(w[r][i].z), __uint_as_float(w[r][i].w)));
                    m[r] = fmaxf(fmaxf(fmaxf(x[0], x[1]), fmaxf(x[2], x[3])),
                                 fmaxf(fmaxf(x[4], x[5]), fmaxf(x[6], x[7])));
                }
                m[r] = fmaxf(m[r], fmaxf(mt[r], y0[r]));
            }
#pragma unroll
            for (int r = 0; r < R; ++r) {
                m[r] = warp_max(m[r]);
                ref[r] = m[r] == -INFINITY ? 0.f : m[r];
                rc[r] = __fmul_rn(ref[r], c);
                far = far || !(fabsf(rc[r]) < kNearExponent);
            }
            // Terms 2^(z c - m c), m c rounded: one rounding of the small difference
            // each, and one factor for the sum.  Where m c is large (a low temperature,
            // logits far from 0), 2^((z - m) c).
            uint64_t acc[R][4] = {};  // pairs of +0
            auto add_terms = [&](int r, int i, bool fused) {
                uint64_t z[4];
                pairs_of<TIn>(w[r][i], z);
#pragma unroll
                for (int j = 0; j < L::kCols / 2; ++j) {
                    float a, b;
                    if (fused)
                        unpair(fma2(z[j], pair(c, c), pair(-rc[r], -rc[r])), a, b);
                    else
                        unpair(mul2(add2(z[j], pair(-ref[r], -ref[r])), pair(c, c)), a, b);
                    const int to = (i * (L::kCols / 2) + j) & 3;
                    acc[r][to] = add2(acc[r][to], pair(ex2(a), ex2(b)));
                }
            };
            if (__builtin_expect(far, 0)) {
#pragma unroll
                for (int r = 0; r < R; ++r) {
                    const bool fused = fabsf(rc[r]) < kNearExponent;
#pragma unroll
                    for (int i = 0; i < L::kPieces; ++i) add_terms(r, i, fused);
                }
            } else {
#pragma unroll
                for (int i = 0; i < L::kPieces; ++i)
#pragma unroll
                    for (int r = 0; r < R; ++r) add_terms(r, i, true);
            }
            float s[R];
#pragma unroll
            for (int r = 0; r < R; ++r) {
                float s0, s1;
                unpair(add2(add2(acc[r][0], acc[r][1]), add2(acc[r][2], acc[r][3])), s0, s1);
                s[r] = __fadd_rn(s0, s1);
                // relative to m c itself rather than to its rounding, to first order
                if (!far || fabsf(rc[r]) < kNearExponent)
                    s[r] = __fmaf_rn(s[r], __fmul_rn(-kLn2, __fmaf_rn(ref[r], c, -rc[r])), s[r]);
                if (listed > 0) {
                    s[r] = __fadd_rn(s[r], ex2(__fmul_rn(__fsub_rn(y0[r], ref[r]), c)));
                    if (listed > 32)
                        s[r] = __fadd_rn(s[r], mt[r] == -INFINITY
                                                   ? st[r]
                                                   : __fmul_rn(st[r], ex2(__fmul_rn(__fsub_rn(mt[r], ref[r]), c))));
                }
            }
#pragma unroll
            for (int off = 16; off > 0; off >>= 1)
#pragma unroll
                for (int r = 0; r < R; ++r)
                    s[r] = __fadd_rn(s[r], __shfl_xor_sync(0xffffffffu, s[r], off));
            if (lane == 0)
#pragma unroll
                for (int r = 0; r < R; ++r) parts[r * slices * kWarps] = make_float2(m[r], s[r]);
            parts += R * slices * kWarps;
        };

        do {
            cp_wait<C::kStages - 1>();  // all copies but those of later rows
            __syncwarp();
            if constexpr (OP == kLogp) {
                bool two = false;
                if (C::kStages > 1 && k + 1 < n) {
                    const RowInfo next = rows[k + 1];
                    two = next.state == kOk && next.step != kAnew &&
                          !(next.step >= 0 && place_warp(next.step) == warp);
                }
                if (two) {
                    cp_wait<0>();
                    __syncwarp();
                    score(std::integral_constant<int, 2>{});
                    ++k;
                } else {
                    score(std::integral_constant<int, 1>{});
                    now = other_stage(now);
                }
            } else {
                unsigned char *stage = now;
                const RowInfo row = rows[k];
                const TIn *zrow = zslice + k * io.ld;
                const int shift = VEC ? 0 : shift_of(zrow);
                uint32_t live = inside;  // columns the mask allows
                if (row.mrow >= 0) live &= reinterpret_cast<const uint32_t *>(stage + C::kMaskAt)[lane];
                uint4 w[L::kPieces];
                load_pieces(w, stage, shift);
                // the list's first 32 columns, one to a lane
                int c0 = -1;
                float z0 = 0.f, y0 = 0.f;
                uint32_t cw0 = 0;
                if (listed > 0 && lane < listed) {
                    c0 = list[lane];
                    if (allowed(stage, row.mrow, c0)) {
                        z0 = elem(at(stage, shift, c0));
                        cw0 = sh.count[c0];
                        y0 = touched_y(c0, z0);
                    } else {
                        c0 = -1;
                    }
                }
                // the target, if it is one of this warp's columns
                const bool has_target = OP == kBwd && row.target >= 0 && place_warp(row.target) == warp;
                const int tcol = place_column(row.target);
                const float zt = has_target && own.lane(tcol) == lane ? elem(at(stage, shift, tcol)) : 0.f;
                if (OP == kBwd && k >> 5 != held) {
                    held = k >> 5;
                    const int64_t t = t0 + (held * 32 + lane);
                    if (io.lse64) {
                        const double d = t < io.T ? io.lse64[t] : 0.0;
                        lse_of = __double2float_rn(d);
                        low_of = fabsf(lse_of) < INFINITY
                                     ? __fmul_rn(-kLog2e, __double2float_rn(d - (double)lse_of))
                                     : 0.f;
                    } else {
                        lse_of = t < io.T ? io.lse[t] : 0.f;
                    }
                    grad_of = t < io.T ? io.grad[t] : 0.f;
                }
                __syncwarp();  // the stage is read
                const float lse = OP == kBwd ? __shfl_sync(0xffffffffu, lse_of, k & 31) : 0.f;
                const bool none = OP == kBwd && lse == -INFINITY;  // the rules leave nothing
                const float l = none ? 0.f : lse;
                const float low = OP == kBwd ? __shfl_sync(0xffffffffu, low_of, k & 31) : 0.f;
                const float g =
                    OP == kBwd && !none ? __fmul_rn(__shfl_sync(0xffffffffu, grad_of, k & 31), q.itau) : 0.f;
                // x - lse with 1 / temperature to 48 bits (id + i1): the rounding of
                // 1 / temperature alone would weigh |x| times half a step.  Rounded
                // down: i1 >= 0, so that -inf times i1 > 0 stays -inf, and i1 = 0 is left
                // out.
                const float id = __frcp_rd(q.tau);
                const float i1 = __fmul_rn(__fmaf_rn(-q.tau, id, 1.f), id);
                const uint32_t shown = none ? 0u : live;
                // other columns become -inf, whose result is -inf, or 0
                if (!__all_sync(0xffffffffu, shown == 0xffffffffu)) keep_columns(w, shown);
                // a touched column's result
                auto result = [&](float hot, float z, uint32_t cw, float y) {
                    if (OP == kApply) return __fmul_rn(y, q.itau);
                    const float slope = cw ? (z > 0.f ? q.irep : q.rep) : 1.f;
                    return __fmul_rn(__fmul_rn(g, __fsub_rn(hot, prob(y, id, i1, l, low))), slope);
                };
                auto transform = [&](auto is_split) {
                    const float f = OP == kApply ? q.itau : id;
                    const uint64_t f2 = pair(f, f), i2 = pair(i1, i1), nl = pair(-l, -l), ng = pair(-g, -g),
                                   lo = pair(low, low);
#pragma unroll
                    for (int i = 0; i < L::kPieces; ++i) {
                        constexpr int N = L::kCols;
                        uint64_t z[4];
                        float x[8];
                        pairs_of<TIn>(w[i], z);
#pragma unroll
                        for (int j = 0; j < N / 2; ++j) {
                            uint64_t v;
                            if constexpr (OP == kApply) {
                                v = mul2(z[j], f2);
                            } else {
                                float a, b;
                                v = fma2(z[j], f2, nl);
                                if constexpr (decltype(is_split)::value) v = fma2(z[j], i2, v);
                                unpair(fma2(v, pair(kLog2e, kLog2e), lo), a, b);
                                v = mul2(pair(ex2(a), ex2(b)), ng);
                            }
                            unpair(v, x[2 * j], x[2 * j + 1]);
                        }
                        unsigned char *o = stage + lane * Lane<TOut>::kPitch + N * i * (int)sizeof(TOut);
                        if constexpr (sizeof(TOut) == 4) {
#pragma unroll
                            for (int h = 0; h < N / 4; ++h)
                                reinterpret_cast<float4 *>(o)[h] =
                                    make_float4(x[4 * h], x[4 * h + 1], x[4 * h + 2], x[4 * h + 3]);
                        } else if constexpr (N == 8) {
                            *reinterpret_cast<uint4 *>(o) =
                                make_uint4(pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3]),
                                           pack_bf16x2(x[4], x[5]), pack_bf16x2(x[6], x[7]));
                        } else {
                            *reinterpret_cast<uint2 *>(o) =
                                make_uint2(pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3]));
                        }
                    }
                };
                if (OP == kBwd && i1 > 0.f)
                    transform(std::true_type{});
                else
                    transform(std::false_type{});
                __syncwarp();
                auto put_column = [&](int j, float v) {
                    put(reinterpret_cast<TOut *>(stage + own.lane(j) * Lane<TOut>::kPitch) + (j & 31), v);
                };
                if (listed > 0 && !none) {
                    // the touched columns over what stands there; the stage no longer
                    // has their logits, so past the list's first 32 they come from the row
                    if (c0 >= 0) put_column(c0, result(0.f, z0, cw0, y0));
                    for (int e0 = 32 + lane; e0 - lane < listed; e0 += 128) {
                        float z[4];
                        int cu[4];
#pragma unroll
                        for (int u = 0; u < 4; ++u) {
                            cu[u] = e0 + 32 * u < listed ? list[e0 + 32 * u] : -1;
                            if (cu[u] >= 0 && !allowed(stage, row.mrow, cu[u])) cu[u] = -1;
                            z[u] = cu[u] >= 0 ? elem(zrow + cu[u]) : 0.f;
                        }
#pragma unroll
                        for (int u = 0; u < 4; ++u)
                            if (cu[u] >= 0) {
                                const uint32_t cw = sh.count[cu[u]];
                                put_column(cu[u], result(0.f, z[u], cw, touched_y(cu[u], z[u])));
                            }
                    }
                    __syncwarp();
                }
                if (has_target) {
                    if (own.lane(tcol) == lane && (shown >> (tcol & 31) & 1u)) {
                        const bool t = touched >> (tcol & 31) & 1u;
                        const uint32_t cw = t ? sh.count[tcol] : 0u;
                        put_column(tcol, result(1.f, zt, cw, t ? touched_y(tcol, zt) : zt));
                    }
                    __syncwarp();
                }
                if constexpr (VEC)
                    write_pieces(stage, oslice, width, own, warp, lane);
                else
                    write_shifted(stage, oslice, width, own, warp, lane);
                oslice += io.ld_out;
                __syncwarp();  // the stage is free again
                prefetch(true);
                now = other_stage(now);
            }
            done = k;
            if (++k >= n) break;
            const RowInfo next = rows[k];
            if (next.state != kOk || next.step == kAnew) break;
            if (next.step >= 0 && place_warp(next.step) == warp) {  // one token more
                const int j = place_column(next.step);
                const uint32_t bit = own.lane(j) == lane ? 1u << (j & 31) : 0u;
                if (bit) sh.count[j] = place_flag(next.step) ? (sh.count[j] | kPromptBit) : sh.count[j] + 1u;
                const bool fresh = (bit & ~touched) != 0;
                touched |= bit;
                if (__any_sync(0xffffffffu, fresh)) listed = make_list(list, touched, mine, lane);
            }
        } while (true);
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

// One warp per row: lane l folds partials l, l + 32, ... in order, then a
// fixed xor tree.
constexpr int kMergeRows = 8;
__global__ void __launch_bounds__(32 * kMergeRows)
    rules_merge(const __grid_constant__ RulesIo io, const __grid_constant__ rk_logits_rules rules,
                float *logp, float *lse, double *lse64) {
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    const int lane = threadIdx.x & 31;
    const int64_t t = (int64_t)blockIdx.x * kMergeRows + (threadIdx.x >> 5);
    if (t >= io.T) return;
    const int32_t state = row_state<kLogp>(io, rules, t, io.targets[t], row_mask(rules, t));
    if (state == kInactive) {
        if (lane == 0) {
            logp[t] = 0.f;
            if (lse) lse[t] = 0.f;
            if (lse64) lse64[t] = 0.0;
        }
        return;
    }
    const bool has_tau = state != kBadRules && rules.num_requests > 0 && rules.temperature;
    const float tau = has_tau ? rules.temperature[row_request(rules, t)] : 1.f;
    const float c = __fmul_rn(kLog2e, __frcp_rn(tau));
    const int64_t parts = (io.V + kSliceCols - 1) / kSliceCols * kWarps;
    float m = -INFINITY, s = 0.f;
    for (int64_t k = lane; k < parts; k += 32) {
        const float2 p = io.part[t * parts + k];
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
        float l, p, ls = 0.f;
        if (state != kOk || s != s) {
            l = p = nan;
        } else if (s == 0.f) {
            l = p = -INFINITY;
        } else {
            ls = logf(s);
            l = __fadd_rn(__fdiv_rn(m, tau), ls);  // -inf where m / tau is past the type
            p = __fsub_rn(__fdiv_rn(__fsub_rn(io.ytgt[t], m), tau), ls);
            if (p > 0.f) p = 0.f;  // rounding alone can take it there
            if (l == -INFINITY) p = l;
        }
        logp[t] = p;
        if (lse) lse[t] = l;
        // past fp32 what l says (an infinity)
        if (lse64) lse64[t] = fabsf(l) < INFINITY ? (double)m / (double)tau + (double)ls : (double)l;
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

// Rows per block.  A long run counts a history seldom, a short one spreads the
// blocks evenly over the SMs: as few waves of two blocks per SM as kMaxRun
// allows, of equal runs.  kMaxRun at 24, 32, 40, 48, 64 (us): logp of 8192 rows
// with long histories 538, 525, 506, 500, 496; bwd of 4096 rows 395, 396, 398,
// 404, 414; 40 costs both little.
//
// The first slice has most of what a history touches, and a row takes up to
// twice the time there.  Its blocks come first, so that the others even out the
// end; in a single wave nothing follows that could, and their runs are shorter.
// By nothing, 3/4, 2/3, 3/5, 1/2: 57, 52, 49, 48.5, 50 us for logp of 2048 x
// 32000, 32, 30, 30, 30, 29.5 for the gradient of 300 x 50257, and no difference
// where runs are short.
constexpr int kFirstNum = 3, kFirstDen = 5;
void cut_rows(RulesIo &io, const rk_logits_rules &r, const DeviceInfo &di, int64_t *grid) {
    const int64_t slices = (io.V + kSliceCols - 1) / kSliceCols, wave = (int64_t)di.sm_count * 2;
    const int64_t waves = (io.T * slices + wave * kMaxRun - 1) / (wave * kMaxRun);
    const bool shorter = slices > 1 && waves == 1 && r.tokens;
    int64_t run = std::max<int64_t>(1, (io.T * slices + wave * waves - 1) / (wave * waves)), run0, blocks0;
    for (;; ++run) {
        run0 = shorter ? (run * kFirstNum + kFirstDen - 1) / kFirstDen : run;
        blocks0 = (io.T + run0 - 1) / run0;
        *grid = blocks0 + (slices - 1) * ((io.T + run - 1) / run);
        if (run >= kMaxRun || *grid <= wave * waves) break;
    }
    io.run0 = (int)run0;
    io.run = (int)run;
    io.blocks0 = (unsigned)std::min<int64_t>(blocks0, 0x7fffffff);
}

template <RulesOp OP, typename TIn, typename TOut, bool VEC>
cudaError_t launch_rows(RulesIo io, const rk_logits_rules &r, const DeviceInfo &di, cudaStream_t st) {
    auto *kernel = rules_kernel<OP, TIn, TOut, VEC>;
    using C = Config<OP, TIn, TOut>;
    static std::atomic<uint64_t> allowed{0};
    cudaError_t e = allow_shared(reinterpret_cast<const void *>(kernel), C::smem(true), di, allowed);
    if (e != cudaSuccess) return e;
    int64_t blocks;
    cut_rows(io, r, di, &blocks);
    if (blocks > 0x7fffffff) return cudaErrorInvalidConfiguration;
    cudaLaunchConfig_t cfg;
    cudaLaunchAttribute attr[1];
    dependent(&cfg, attr, (unsigned)blocks, kThreads, C::smem(r.bias_ids != nullptr), st);
    return cudaLaunchKernelEx(&cfg, kernel, io, r);
}

template <RulesOp OP, typename TIn, typename TOut>
cudaError_t launch(const RulesIo &io, const rk_logits_rules &r, const DeviceInfo &di, cudaStream_t st) {
    const auto rows_aligned = [](const void *p, int64_t ld, size_t size) {
        return aligned(p, 16) && ld * (int64_t)size % 16 == 0;
    };
    const bool vec = rows_aligned(io.logits, io.ld, sizeof(TIn)) &&
                     (OP == kLogp || rows_aligned(io.out, io.ld_out, sizeof(TOut)));
    return vec ? launch_rows<OP, TIn, TOut, true>(io, r, di, st)
               : launch_rows<OP, TIn, TOut, false>(io, r, di, st);
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

}  // namespace

size_t logp_rules_workspace_bytes(int64_t T, int64_t V) {
    const size_t parts = (size_t)((V + kSliceCols - 1) / kSliceCols * kWarps);
    return ((size_t)T * parts * sizeof(float2) + (size_t)T * sizeof(float) + 255) / 256 * 256;
}

cudaError_t launch_rules_apply(const RulesMatrix &logits, const rk_logits_rules &rules, int64_t T,
                               int64_t V, const RulesMatrix &out, const DeviceInfo &di,
                               cudaStream_t st) {
    RulesIo io{};
    io.logits = logits.p;
    io.ld = logits.ld;
    io.T = T;
    io.V = V;
    io.out = const_cast<void *>(out.p);
    io.ld_out = out.ld;
    io.err = di.err;
    return launch_types<kApply>(io, rules, logits.type, out.type, di, st);
}

cudaError_t launch_rules_logp(const RulesMatrix &logits, const int64_t *targets, const int32_t *cu,
                              int num_seqs, const rk_logits_rules &rules, int64_t T, int64_t V,
                              float *logp, float *lse, double *lse64, void *workspace,
                              const DeviceInfo &di, cudaStream_t st) {
    RulesIo io{};
    io.logits = logits.p;
    io.ld = logits.ld;
    io.targets = targets;
    io.cu = cu;
    io.num_seqs = num_seqs;
    io.T = T;
    io.V = V;
    io.part = static_cast<float2 *>(workspace);
    io.ytgt = reinterpret_cast<float *>(io.part + T * ((V + kSliceCols - 1) / kSliceCols * kWarps));
    io.err = di.err;
    cudaError_t e = logits.type == RK_BF16 ? launch<kLogp, uint16_t, float>(io, rules, di, st)
                                           : launch<kLogp, float, float>(io, rules, di, st);
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg;
    cudaLaunchAttribute attr[1];
    dependent(&cfg, attr, (unsigned)((T + kMergeRows - 1) / kMergeRows), 32 * kMergeRows, 0, st);
    return cudaLaunchKernelEx(&cfg, rules_merge, io, rules, logp, lse, lse64);
}

cudaError_t launch_rules_bwd(const RulesMatrix &logits, const int64_t *targets, const int32_t *cu,
                             int num_seqs, const rk_logits_rules &rules, int64_t T, int64_t V,
                             const float *lse, const double *lse64, const float *grad,
                             const RulesMatrix &dlogits, const DeviceInfo &di, cudaStream_t st) {
    RulesIo io{};
    io.logits = logits.p;
    io.ld = logits.ld;
    io.targets = targets;
    io.cu = cu;
    io.num_seqs = num_seqs;
    io.T = T;
    io.V = V;
    io.lse = lse;
    io.lse64 = lse64;
    io.grad = grad;
    io.out = const_cast<void *>(dlogits.p);
    io.ld_out = dlogits.ld;
    io.err = di.err;
    return launch_types<kBwd>(io, rules, logits.type, dlogits.type, di, st);
}

}  // namespace rk
