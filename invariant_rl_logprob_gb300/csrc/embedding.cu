// embedding.cu -- token embedding with scaling, and its gradient summed per
// token in canonical order ("embedding", RL-Kernel issue #101 P0 list; chain
// index 0 of PR #264; the embedding gradient belongs to the parameter
// gradients of issue #244, Workstream 3 #153: fixed order, no atomicAdd).
//
//   out[t, :] = scale * E[ids[t], :]
//   dE[v, :]  = scale * sum over canonical tokens i with ids[i] = v of dout[i, :]
//
// Both are memory bound.  The gradient runs in three stages:
//   sort    (id, row) pairs of the canonical tokens by id with a stable
//           least-significant-digit radix sort (digits of up to
//           kMaxDigitBits; inactive tokens get the key V and end up last):
//           in the shared memory of one block for up to kSmallSort tokens,
//           by tiles of kSortTile otherwise;
//   pieces  each id's run in the sorted list is cut into pieces of kPiece
//           occurrences, counted from the run's own start;
//   sum     a warp per (piece, 512 columns) adds the piece's rows in order in
//           fp32, with the loads of several rows and columns in flight.  An id
//           with one piece writes its row of dE; the others write partial
//           sums, which a last kernel adds in order.
//
// Measured (bytes at the copy rate in brackets): lookup of 65536 x 4096 bf16 115 us
// (104); gradient of 65536 x 4096 into a tied weight's 243 us (176): sums 194, sort
// and list of pieces 34, join 15; of 8192 x 3584 into 152064 rows 320 us (335;
// zeros leave faster than copies).
//
// The pieces of an id depend on its own occurrences alone, so its row of dE
// does too.  The order in which blocks find the pieces does not matter: no
// two write the same place.
#include <algorithm>
#include <utility>

#include "elements.cuh"
#include "rk_device.cuh"
#include "rk_internal.h"

namespace rk {
namespace {

// ---- lookup ----

constexpr int kLookupThreads = 128;

template <typename TE, typename TO, bool VEC>
__global__ void __launch_bounds__(kLookupThreads)
    embedding_kernel(const int64_t *ids, const int32_t *cu, int num_seqs,
                     const TE *E, int64_t H, int64_t V, float scale,
                     TO *out, unsigned *err) {
    wait_prior_grid();
    const int64_t t = blockIdx.x;
    const int64_t id = ids[t];
    const bool active = row_active(t, id, cu, num_seqs);
    const bool bad = active && id >= V;
    if (bad && threadIdx.x == 0) atomicOr(err, kErrTargetRange);
    const bool live = active && !bad;
    const float fill = bad ? __int_as_float(0x7fc00000) : 0.f;
    const TE *src = E + (live ? id : 0) * H;
    TO *dst = out + t * H;
    if (VEC) {
        for (int64_t c = 8 * (int64_t)threadIdx.x; c < H; c += 8 * kLookupThreads) {
            float v[8] = {fill, fill, fill, fill, fill, fill, fill, fill};
            if (live) {
                get8(src + c, v);
#pragma unroll
                for (int j = 0; j < 8; ++j) v[j] = __fmul_rn(scale, v[j]);
            }
            put8(dst + c, v);
        }
    } else {
        for (int64_t c = threadIdx.x; c < H; c += kLookupThreads)
            put1(dst + c, live ? __fmul_rn(scale, get1(src + c)) : fill);
    }
}

// ---- gradient: sort ----

constexpr int kSortThreads = 256;
constexpr int kSortWarps = kSortThreads / 32;
constexpr int kSortItems = 8;                                   // per lane
constexpr int kSortTile = kSortThreads * kSortItems;            // 2048
constexpr int kMaxDigitBits = 9;
constexpr int kMaxBins = 1 << kMaxDigitBits;
constexpr int kInlineScanTiles = 64;  // up to here each block scans the counts itself
constexpr int kTinyThreads = 128, kSmallThreads = 1024;         // blocks that sort alone
constexpr int kTinySort = kTinyThreads * kSortItems;            // 1024
constexpr int kSmallSort = kSmallThreads * kSortItems;          // 8192
constexpr int kPiece = 32;       // occurrences of an id summed by one warp
constexpr int kHalf = kPiece / 2;
constexpr int kScanThreads = 1024;
constexpr int kClasses = 6;      // pieces of 1, 2, 3..4, 5..8, 9..16, 17..32 rows
constexpr int kCounters = kClasses + 1;  // pieces of each class, joins
constexpr int kZeroAllShare = 8;

struct Canonical {  // the canonical tokens
    const int64_t *ids;
    const int32_t *cu;
    int num_seqs;
    int64_t T, V;
    const int64_t *order;
    int64_t n;
    unsigned *err;
};

// Key (the id, or V: inactive) and row of canonical token i.
__device__ __forceinline__ void canonical_token(const Canonical &c, int64_t i, int32_t &key, int32_t &row) {
    const int64_t r = c.order ? c.order[i] : i;
    int64_t k = c.V;
    if (r >= 0 && r < c.T) {
        const int64_t id = c.ids[r];
        if (row_active(r, id, c.cu, c.num_seqs)) {
            if (id < c.V)
                k = id;
            else
                atomicOr(c.err, kErrTargetRange);
        }
    }
    key = (int32_t)k;
    row = (int32_t)(k < c.V ? r : 0);
}

// Exclusive prefix sum of one int per thread over a block of 32 * WARPS
// threads; `total` gets the sum.
template <int WARPS>
__device__ __forceinline__ int block_scan(int x, int *total) {
    __shared__ int warp_sums[WARPS];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int incl = x;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, incl, off);
        if (lane >= off) incl += y;
    }
    if (lane == 31) warp_sums[warp] = incl;
    __syncthreads();
    int w = lane < WARPS ? warp_sums[lane] : 0;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, w, off);
        if (lane >= off) w += y;
    }
    *total = __shfl_sync(0xffffffffu, w, WARPS - 1);
    const int before = warp > 0 ? __shfl_sync(0xffffffffu, w, warp - 1) : 0;
    __syncthreads();
    return before + incl - x;
}

// Counts the digits of a tile's keys; a thread's items are strided by the
// block's size.
__device__ __forceinline__ void count_digits(const int32_t (&k)[kSortItems], int64_t first, int64_t n,
                                             int shift, int bins, int *cnt) {
#pragma unroll
    for (int j = 0; j < kSortItems; ++j)
        if (first + j * kSortThreads < n) atomicAdd(&cnt[(k[j] >> shift) & (bins - 1)], 1);
}

// Where digit d's count of tile b stands: rows of `pitch` tiles, the columns
// past the last tile 0.
__device__ __forceinline__ void write_counts(const int *cnt, int bins, int32_t *hist, int64_t tiles,
                                             int64_t pitch) {
    for (int d = threadIdx.x; d < bins; d += kSortThreads) {
        hist[d * pitch + blockIdx.x] = cnt[d];
        if (blockIdx.x == 0)
            for (int64_t b = tiles; b < pitch; ++b) hist[d * pitch + b] = 0;
    }
}

// Keys and rows of the canonical tokens, and the first pass's counts.
__global__ void __launch_bounds__(kSortThreads)
    emb_keys(const __grid_constant__ Canonical c, int32_t *key, int32_t *val, int bins, int32_t *hist,
             int64_t tiles, int64_t pitch, int32_t *counters) {
    __shared__ int cnt[kMaxBins];
    wait_prior_grid();
    for (int d = threadIdx.x; d < bins; d += kSortThreads) cnt[d] = 0;
    if (blockIdx.x == 0 && threadIdx.x < kCounters) counters[threadIdx.x] = 0;
    __syncthreads();
    const int64_t first = (int64_t)blockIdx.x * kSortTile + threadIdx.x;
    int32_t k[kSortItems];
#pragma unroll
    for (int j = 0; j < kSortItems; ++j) {
        const int64_t i = first + j * kSortThreads;
        if (i < c.n) {
            int32_t r;
            canonical_token(c, i, k[j], r);
            key[i] = k[j];
            val[i] = r;
        }
    }
    count_digits(k, first, c.n, 0, bins, cnt);
    __syncthreads();
    write_counts(cnt, bins, hist, tiles, pitch);
}

// A later pass's counts.
__global__ void __launch_bounds__(kSortThreads)
    emb_histogram(const int32_t *key, int64_t n, int shift, int bins, int32_t *hist, int64_t tiles,
                  int64_t pitch) {
    __shared__ int cnt[kMaxBins];
    wait_prior_grid();
    for (int d = threadIdx.x; d < bins; d += kSortThreads) cnt[d] = 0;
    const int64_t first = (int64_t)blockIdx.x * kSortTile + threadIdx.x;
    int32_t k[kSortItems];
#pragma unroll
    for (int j = 0; j < kSortItems; ++j)
        k[j] = first + j * kSortThreads < n ? key[first + j * kSortThreads] : 0;
    __syncthreads();
    count_digits(k, first, n, shift, bins, cnt);
    __syncthreads();
    write_counts(cnt, bins, hist, tiles, pitch);
}

// Exclusive prefix sums over cnt[0..len) in place, by one block (len a
// multiple of 4).
__global__ void __launch_bounds__(kScanThreads) emb_scan(int32_t *cnt, int64_t len) {
    wait_prior_grid();
    int carry = 0;
    for (int64_t base = 0; base < len; base += 16 * kScanThreads) {
        int4 v[4];
        const int64_t i0 = base + 16 * (int64_t)threadIdx.x;
        int sum = 0;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            v[j] = i0 + 4 * j < len ? *reinterpret_cast<const int4 *>(cnt + i0 + 4 * j)
                                    : make_int4(0, 0, 0, 0);
            sum += v[j].x + v[j].y + v[j].z + v[j].w;
        }
        int all;
        int run = carry + block_scan<kScanThreads / 32>(sum, &all);
        carry += all;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int4 o = make_int4(run, run + v[j].x, run + v[j].x + v[j].y, run + v[j].x + v[j].y + v[j].z);
            run = o.w + v[j].w;
            if (i0 + 4 * j < len) *reinterpret_cast<int4 *>(cnt + i0 + 4 * j) = o;
        }
    }
}

// A warp's kSortItems * 32 consecutive items, item j * 32 + lane in register
// j, to their digit's place, order kept: an item's rank is the number of
// earlier lanes with its digit plus the warp's running place of that digit.
template <typename Store>
__device__ __forceinline__ void place_items(const int32_t (&k)[kSortItems], int64_t left, int shift,
                                            int bins, int *place, int lane, Store store) {
#pragma unroll
    for (int j = 0; j < kSortItems; ++j) {
        const bool live = 32 * j + lane < left;
        const int d = live ? (k[j] >> shift) & (bins - 1) : 0;
        unsigned peers = __ballot_sync(0xffffffffu, live);  // live lanes with this digit
#pragma unroll
        for (int b = 0; b < kMaxDigitBits; ++b) {
            const bool set = d >> b & 1;
            const unsigned m = __ballot_sync(0xffffffffu, set);
            peers &= set ? m : ~m;
        }
        const int rank = __popc(peers & ((1u << lane) - 1u));
        const int at = live ? place[d] + rank : 0;
        __syncwarp();
        if (live) {
            if (rank == 0) place[d] = at + __popc(peers);
            store(j, at);
        }
        __syncwarp();
    }
}

// Radix pass, last part: a tile's items to their digit's place.  SCANNED: hist
// holds prefix sums; otherwise counts, which the block sums up itself.
template <bool SCANNED>
__global__ void __launch_bounds__(kSortThreads)
    emb_scatter(const int32_t *ks, const int32_t *vs, int32_t *kd, int32_t *vd, int64_t n, int shift,
                int bins, const int32_t *hist, int64_t pitch) {
    __shared__ int place[kSortWarps][kMaxBins];
    wait_prior_grid();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int64_t base = (int64_t)blockIdx.x * kSortTile + (int64_t)warp * 32 * kSortItems;
    int32_t k[kSortItems], v[kSortItems];
#pragma unroll
    for (int j = 0; j < kSortItems; ++j) {
        const int64_t i = base + 32 * j + lane;
        k[j] = i < n ? ks[i] : 0;
        v[j] = i < n ? vs[i] : 0;
    }
    for (int d = threadIdx.x; d < kSortWarps * kMaxBins; d += kSortThreads) (&place[0][0])[d] = 0;
    __syncthreads();
#pragma unroll
    for (int j = 0; j < kSortItems; ++j)
        if (base + 32 * j + lane < n) atomicAdd(&place[warp][(k[j] >> shift) & (bins - 1)], 1);
    // the tile's first place of digits 2 threadIdx and 2 threadIdx + 1
    constexpr int kPer = kMaxBins / kSortThreads;
    int first[kPer], sum = 0;
#pragma unroll
    for (int j = 0; j < kPer; ++j) {
        const int d = kPer * threadIdx.x + j;
        first[j] = 0;
        if (d >= bins) continue;
        if (SCANNED) {
            first[j] = hist[d * pitch + blockIdx.x];
        } else {
            int before = 0, all = 0;
#pragma unroll 4
            for (int b = 0; b < (int)pitch; b += 4) {
                const int4 h = *reinterpret_cast<const int4 *>(hist + d * pitch + b);
                all += h.x + h.y + h.z + h.w;
                const int m = (int)blockIdx.x - b;  // tiles before this one
                before += (m > 0 ? h.x : 0) + (m > 1 ? h.y : 0) + (m > 2 ? h.z : 0) + (m > 3 ? h.w : 0);
            }
            first[j] = sum + before;
            sum += all;
        }
    }
    int total;
    const int prefix = block_scan<kSortWarps>(sum, &total);  // a barrier too
#pragma unroll
    for (int j = 0; j < kPer; ++j) {
        const int d = kPer * threadIdx.x + j;
        int run = prefix + first[j];
#pragma unroll
        for (int w = 0; w < kSortWarps; ++w) {
            const int c = place[w][d];
            place[w][d] = run;
            run += c;
        }
    }
    __syncthreads();
    place_items(k, n - base, shift, bins, place[warp], lane, [&](int j, int at) {
        kd[at] = k[j];
        vd[at] = v[j];
    });
}

// ---- gradient: pieces ----

struct Piece {
    int32_t id, pos, len;  // rows val[pos .. pos + len) of id
    int32_t slot;          // partial sum, or -1: the id has this piece alone
};

// First position past the run of equal keys that starts at i.
template <typename K>
__device__ __forceinline__ int64_t run_end(const K *key, int64_t i, int64_t n, int32_t k) {
    int64_t lo = i + 1, hi = min(n, i + kPiece);
    if (hi < n && key[hi] == k) {
        lo = hi + 1;
        hi = n;
    }
    while (lo < hi) {
        const int64_t mid = (lo + hi) / 2;
        if (key[mid] == k)
            lo = mid + 1;
        else
            hi = mid;
    }
    return lo;
}

// Pieces are listed by size, the largest first, so that the warps that take them
// in turn get the same work (65536 x 4096: 243 us, and 258 to 284 in the order in
// which blocks found them).  Class c has its own part of the list: n / (its smallest size) + 1
// pieces at most.
__host__ __device__ inline int64_t class_pieces(int64_t n, int c) { return n / (c < 2 ? c + 1 : (1 << (c - 1)) + 1) + 1; }
__host__ __device__ inline int64_t class_first(int64_t n, int c) {  // c = -1: of all
    int64_t at = 0;
    for (int d = kClasses - 1; d > c; --d) at += class_pieces(n, d);
    return at;
}
__device__ __forceinline__ int class_of(int len) { return len > 1 ? 32 - __clz(len - 1) : 0; }

// The pieces of the run [i, end) of id k: all but the last are whole.  Where a
// block's pieces of each class are: `count` (shared) gives the places of this
// run's, at which write_pieces puts them behind base[class].
struct Places {
    int whole, last;
};
__device__ __forceinline__ int last_len(int np, int64_t i, int64_t end) {
    return (int)(end - i) - (np - 1) * kPiece;
}
__device__ __forceinline__ Places take_places(int *count, int np, int64_t i, int64_t end) {
    Places p;
    p.whole = np > 1 ? atomicAdd(&count[kClasses - 1], np - 1) : 0;
    p.last = atomicAdd(&count[class_of(last_len(np, i, end))], 1);
    return p;
}
// Their partial sums take slots ceil(i / kHalf), ...: a run of more than kPiece
// items has at least as many multiples of kHalf as pieces, so no two runs share a
// slot.
__device__ __forceinline__ void write_pieces(Piece *pieces, const int64_t *base, const Places &at, int np, int32_t k,
                                             int64_t i, int64_t end) {
    const int32_t slot = (int32_t)((i + kHalf - 1) / kHalf);
    Piece *whole = pieces + base[kClasses - 1] + at.whole;
    for (int j = 0; j < np - 1; ++j) whole[j] = Piece{k, (int32_t)(i + (int64_t)j * kPiece), kPiece, slot + j};
    const int len = last_len(np, i, end), c = class_of(len);
    pieces[base[c] + at.last] =
        Piece{k, (int32_t)(end - len), len, np > 1 ? slot + np - 1 : -1};
}
__device__ __forceinline__ Piece join_of(int np, int32_t k, int64_t i) {
    return Piece{k, (int32_t)i, np, (int32_t)((i + kHalf - 1) / kHalf)};
}

// The runs that start in a block of 256 sorted keys.  Only the last of them can
// reach beyond it; the block looks for its end together, 256 probes at a time.
constexpr int kPieceThreads = 256;
__global__ void __launch_bounds__(kPieceThreads)
    emb_pieces(const int32_t *key, int64_t n, int32_t V, Piece *pieces, Piece *joins, int32_t *counters) {
    __shared__ int count[kClasses];
    __shared__ int64_t place[kClasses];
    __shared__ unsigned starts[kPieceThreads / 32];  // bit per key: a run starts
    wait_prior_grid();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int64_t base = (int64_t)blockIdx.x * kPieceThreads, i = base + threadIdx.x;
    const int64_t stop = min(base + kPieceThreads, n);  // the end of the block's keys
    const int32_t k = i < n ? key[i] : V, last = key[stop - 1];
    const bool first = i < n && (i == 0 || key[i - 1] != k), start = first && k < V;
    const unsigned mine = __ballot_sync(0xffffffffu, first);
    if (lane == 0) starts[warp] = mine;
    if (threadIdx.x < kClasses) count[threadIdx.x] = 0;
    int64_t lo = stop, hi = last < V ? n : stop;  // the end of the last run is in [lo, hi]
    while (lo < hi) {
        const int64_t step = (hi - lo + kPieceThreads - 1) / kPieceThreads;
        const int64_t at = lo + ((int64_t)threadIdx.x + 1) * step - 1;  // the last of this thread's share
        const int same = __syncthreads_count(at < hi && key[at] == last);
        lo += same * step;
        hi = min(hi, lo + step - 1);
    }
    __syncthreads();
    int64_t end = lo;
    if (start) {
        unsigned rest = lane < 31 ? mine >> (lane + 1) << (lane + 1) : 0;
        int w = warp;
        while (rest == 0 && ++w < kPieceThreads / 32) rest = starts[w];
        if (rest) end = base + 32 * w + __ffs(rest) - 1;
    }
    const int np = start ? (int)((end - i + kPiece - 1) / kPiece) : 0;
    Places at{};
    if (start) at = take_places(count, np, i, end);
    __syncthreads();
    if (threadIdx.x < kClasses)
        place[threadIdx.x] = class_first(n, threadIdx.x) + atomicAdd(&counters[threadIdx.x], count[threadIdx.x]);
    __syncthreads();
    if (!start) return;
    write_pieces(pieces, place, at, np, k, i, end);
    if (np > 1) joins[atomicAdd(&counters[kClasses], 1)] = join_of(np, k, i);
}

// Keys, sort and pieces of up to kSortItems * THREADS tokens in one block.
template <int THREADS>
struct SmallSort {
    int32_t key[2][kSortItems * THREADS];
    uint16_t item[2][kSortItems * THREADS];  // canonical index
    int place[THREADS / 32][kMaxBins];
    int64_t base[kClasses];
    int count[kClasses], joins;
};

// Block `block` of THREADS * kZeroVectors * 16 bytes of zeros in dE, of n1 floats,
// the first 4 n4 as vectors.
constexpr int kZeroVectors = 4;
template <int THREADS>
__device__ __forceinline__ void zero_share(float *dE, int64_t n4, int64_t n1, int64_t block) {
    const int64_t first = block * THREADS * kZeroVectors + threadIdx.x;
#pragma unroll
    for (int k = 0; k < kZeroVectors; ++k) {
        const int64_t i = first + k * THREADS;
        if (i < n4)
            reinterpret_cast<float4 *>(dE)[i] = make_float4(0.f, 0.f, 0.f, 0.f);
        else if (4 * n4 + (i - n4) < n1)  // unaligned, or what is left
            dE[4 * n4 + (i - n4)] = 0.f;
    }
}

// The blocks behind the first write zeros over dE (n1 floats).
template <int THREADS>
__global__ void __launch_bounds__(THREADS)
    emb_sort_small(const __grid_constant__ Canonical c, int passes, int digit, int32_t *key, int32_t *val,
                   Piece *pieces, Piece *joins, int32_t *counters, float *dE, int64_t n4, int64_t n1) {
    constexpr int kWarps = THREADS / 32;
    constexpr int kPer = kMaxBins > THREADS ? kMaxBins / THREADS : 1;  // digits of a thread
    extern __shared__ uint4 raw[];
    SmallSort<THREADS> &s = *reinterpret_cast<SmallSort<THREADS> *>(raw);
    wait_prior_grid();
    if (blockIdx.x > 0) {
        zero_share<THREADS>(dE, n4, n1, (int64_t)blockIdx.x - 1);
        return;
    }
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int n = (int)c.n, base = warp * 32 * kSortItems, bins = 1 << digit;
    if (threadIdx.x < kClasses) {
        s.count[threadIdx.x] = 0;
        s.base[threadIdx.x] = class_first(n, threadIdx.x);
    }
    if (threadIdx.x == 0) s.joins = 0;
    int32_t k[kSortItems], v[kSortItems];
#pragma unroll
    for (int j = 0; j < kSortItems; ++j) {
        const int i = base + 32 * j + lane;
        v[j] = i;
        k[j] = 0;
        int32_t row;
        if (i < n) canonical_token(c, i, k[j], row);
    }
    for (int p = 0; p < passes; ++p) {
        const int shift = p * digit, to = p & 1;
        for (int d = threadIdx.x; d < kWarps * kMaxBins / 4; d += THREADS)
            reinterpret_cast<int4 *>(s.place)[d] = make_int4(0, 0, 0, 0);
        __syncthreads();
#pragma unroll
        for (int j = 0; j < kSortItems; ++j)
            if (base + 32 * j + lane < n) atomicAdd(&s.place[warp][(k[j] >> shift) & (bins - 1)], 1);
        __syncthreads();
        int sum = 0;
#pragma unroll
        for (int d = kPer * threadIdx.x; d < kPer * (threadIdx.x + 1); ++d)
            if (d < bins)
#pragma unroll
                for (int w = 0; w < kWarps; ++w) sum += s.place[w][d];
        int total;
        int run = block_scan<kWarps>(sum, &total);
#pragma unroll
        for (int d = kPer * threadIdx.x; d < kPer * (threadIdx.x + 1); ++d)
            if (d < bins)
#pragma unroll
                for (int w = 0; w < kWarps; ++w) {
                    const int x = s.place[w][d];
                    s.place[w][d] = run;
                    run += x;
                }
        __syncthreads();
        place_items(k, n - base, shift, bins, s.place[warp], lane, [&](int j, int at) {
            s.key[to][at] = k[j];
            s.item[to][at] = (uint16_t)v[j];
        });
        __syncthreads();
#pragma unroll
        for (int j = 0; j < kSortItems; ++j) {
            const int i = base + 32 * j + lane;
            if (i < n) {
                k[j] = s.key[to][i];
                v[j] = s.item[to][i];
            }
        }
    }
    const int32_t *sorted = s.key[(passes - 1) & 1];
#pragma unroll
    for (int j = 0; j < kSortItems; ++j) {
        const int i = base + 32 * j + lane;
        if (i >= n) continue;
        key[i] = k[j];
        val[i] = (int32_t)(k[j] < c.V ? (c.order ? c.order[v[j]] : (int64_t)v[j]) : 0);
        if (k[j] >= c.V || (i > 0 && sorted[i - 1] == k[j])) continue;
        const int64_t end = run_end(sorted, i, n, k[j]);
        const int np = (int)((end - i + kPiece - 1) / kPiece);
        write_pieces(pieces, s.base, take_places(s.count, np, i, end), np, k[j], i, end);
        if (np > 1) joins[atomicAdd(&s.joins, 1)] = join_of(np, k[j], i);
    }
    __syncthreads();
    if (threadIdx.x < kClasses) counters[threadIdx.x] = s.count[threadIdx.x];
    if (threadIdx.x == 0) counters[kClasses] = s.joins;
}

// ---- gradient: rows of dE without a token ----
//
// Zeros leave in many short blocks, in order: 2.2 GB took 281 us so (7.8 TB/s)
// and 332 to 342 us in resident blocks that loop, whose warps drift apart.

constexpr int kZeroThreads = 256;

// All of dE, beside the one block that sorts.  That block lets this grid start
// once the work before it is complete; the last block here waits for the sort,
// so that whoever waits for this grid has waited for both.
__global__ void __launch_bounds__(kZeroThreads) emb_zero_all(float *dE, int64_t n4, int64_t n1) {
    zero_share<kZeroThreads>(dE, n4, n1, blockIdx.x);
    if (blockIdx.x == gridDim.x - 1) asm volatile("griddepcontrol.wait;" ::: "memory");
}

// The rows that no sorted key names, a warp per row.
constexpr int kAbsentThreads = 128;
template <bool VEC>
__global__ void __launch_bounds__(kAbsentThreads)
    emb_zero_absent(const int32_t *key, int64_t n, int64_t H, int64_t V, float *dE) {
    wait_prior_grid();
    const int lane = threadIdx.x & 31;
    const int64_t v = (int64_t)blockIdx.x * (kAbsentThreads / 32) + (threadIdx.x >> 5);
    if (v >= V) return;
    int64_t lo = 0, hi = n;  // first key >= v
    while (lo < hi) {
        const int64_t mid = (lo + hi) / 2;
        if (key[mid] < v)
            lo = mid + 1;
        else
            hi = mid;
    }
    if (lo < n && key[lo] == v) return;
    float *row = dE + v * H;
    if (VEC) {
        for (int64_t c = 4 * lane; c < H; c += 128)
            *reinterpret_cast<float4 *>(row + c) = make_float4(0.f, 0.f, 0.f, 0.f);
    } else {
        for (int64_t c = lane; c < H; c += 32) row[c] = 0.f;
    }
}

// ---- gradient: sums ----

constexpr int kSumThreads = 128;
constexpr int kSumWarps = kSumThreads / 32;
constexpr int kSumBlocks = 5;  // per SM
constexpr int kLaneCols = 16;
constexpr int kSumCols = 32 * kLaneCols;  // columns of a warp: 512

// A lane's 16 columns of a warp's kSumCols: two vectors of 8 (VEC; vector k at
// column 8 (lane + 32 k)), or 16 single ones (k at lane + 32 k).
template <bool VEC>
struct Cols {
    static constexpr int kN = VEC ? 2 : kLaneCols;
    static __device__ __forceinline__ int at(int lane, int k) { return VEC ? 8 * (lane + 32 * k) : lane + 32 * k; }
};

template <bool VEC, typename T>
__device__ __forceinline__ void get_cols(const T *src, int64_t cols, int lane, float (&v)[kLaneCols]) {
    using C = Cols<VEC>;
#pragma unroll
    for (int k = 0; k < C::kN; ++k) {
        const int c = C::at(lane, k);
        if constexpr (VEC) {
            float x[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
            if (c < cols) get8(src + c, x);
#pragma unroll
            for (int j = 0; j < 8; ++j) v[8 * k + j] = x[j];
        } else {
            v[k] = c < cols ? get1(src + c) : 0.f;
        }
    }
}

template <bool VEC>
__device__ __forceinline__ void put_cols(float *dst, int64_t cols, int lane, const float (&v)[kLaneCols]) {
    using C = Cols<VEC>;
#pragma unroll
    for (int k = 0; k < C::kN; ++k) {
        const int c = C::at(lane, k);
        if (c >= cols) continue;
        if constexpr (VEC) {
            float x[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) x[j] = v[8 * k + j];
            put8(dst + c, x);
        } else {
            dst[c] = v[k];
        }
    }
}

// Warps take units in fixed strides (drawing them from a counter put a
// latency into every unit's chain, and a third more time, at 65536 x 4096).
template <typename T, bool VEC>
__global__ void __launch_bounds__(kSumThreads, VEC ? kSumBlocks : 3)
    emb_sum(const T *dout, int64_t H, float scale, const int32_t *val, const Piece *pieces, int64_t n,
            const int32_t *counters, int accumulate, float *dE, float *partial) {
    // the pieces before the end of each class, largest first, and where piece i of it
    // is in the list: i + shift
    __shared__ unsigned ends[kClasses];
    __shared__ int64_t shift[kClasses];
    wait_prior_grid();
    if (threadIdx.x < kClasses) {
        const int c = kClasses - 1 - (int)threadIdx.x;
        unsigned before = 0;
        for (int d = kClasses - 1; d > c; --d) before += (unsigned)counters[d];
        ends[threadIdx.x] = before + (unsigned)counters[c];
        shift[threadIdx.x] = class_first(n, c) - (int64_t)before;
    }
    __syncthreads();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int64_t ncb = (H + kSumCols - 1) / kSumCols;
    const unsigned count = ends[kClasses - 1], blocks = (unsigned)ncb;
    const unsigned u = blockIdx.x * kSumWarps + warp, step = gridDim.x * kSumWarps;
    // Unit u: piece u / ncb, columns from u % ncb * kSumCols on.  A unit's piece is
    // read two units ahead and its rows one ahead (kPiece == 32).
    const unsigned at_step = step / blocks, cb_step = step % blocks;
    unsigned at = u / blocks, cb = u % blocks;
    auto advance = [&](unsigned &a, unsigned &b) {
        a += at_step;
        b += cb_step;
        if (b >= blocks) {
            b -= blocks;
            ++a;
        }
    };
    unsigned at2 = at, cb2 = cb;  // two units ahead, in the end
    auto piece_ahead = [&] {
        Piece p{};
        if (at2 < count) {
            int c = 0;
#pragma unroll
            for (int d = 0; d < kClasses - 1; ++d) c += at2 >= ends[d];
            p = pieces[shift[c] + at2];
        }
        advance(at2, cb2);
        return p;
    };
    auto rows_of = [&](const Piece &p) { return lane < p.len ? val[p.pos + lane] : 0; };
    Piece next = piece_ahead();
    int next_row = rows_of(next);
    Piece after = piece_ahead();
    for (; at < count; advance(at, cb)) {
        const Piece p = next;
        const int row = next_row;
        next = after;
        next_row = rows_of(next);
        after = piece_ahead();
        const int64_t c0 = (int64_t)cb * kSumCols, cols = H - c0;
        const T *src = dout + c0;
        const bool last = p.slot < 0;
        float *dst = (last ? dE + (int64_t)p.id * H : partial + (int64_t)p.slot * H) + c0;
        float s[kLaneCols], old[kLaneCols];
        if (last && accumulate) get_cols<VEC>(dst, cols, lane, old);
        get_cols<VEC>(src + (int64_t)__shfl_sync(0xffffffffu, row, 0) * H, cols, lane, s);
        int i = 1;
        for (; i + 2 <= p.len; i += 2) {
            float a[kLaneCols], b[kLaneCols];
            get_cols<VEC>(src + (int64_t)__shfl_sync(0xffffffffu, row, i) * H, cols, lane, a);
            get_cols<VEC>(src + (int64_t)__shfl_sync(0xffffffffu, row, i + 1) * H, cols, lane, b);
#pragma unroll
            for (int j = 0; j < kLaneCols; ++j) s[j] = __fadd_rn(__fadd_rn(s[j], a[j]), b[j]);
        }
        if (i < p.len) {
            float a[kLaneCols];
            get_cols<VEC>(src + (int64_t)__shfl_sync(0xffffffffu, row, i) * H, cols, lane, a);
#pragma unroll
            for (int j = 0; j < kLaneCols; ++j) s[j] = __fadd_rn(s[j], a[j]);
        }
        if (last) {
#pragma unroll
            for (int j = 0; j < kLaneCols; ++j) {
                s[j] = __fmul_rn(scale, s[j]);
                if (accumulate) s[j] = __fadd_rn(old[j], s[j]);
            }
        }
        put_cols<VEC>(dst, cols, lane, s);
    }
}

// The ids with more than one piece: their partial sums, added in order.
constexpr int kJoinAhead = 16;  // loads in flight
__global__ void __launch_bounds__(kSumThreads)
    emb_join(int64_t H, float scale, const Piece *joins, const int32_t *counters, int accumulate,
             float *dE, const float *partial) {
    wait_prior_grid();
    const int64_t ncb = (H + kSumThreads - 1) / kSumThreads;  // a column per thread
    const int64_t units = (int64_t)counters[kClasses] * ncb;
    for (int64_t u = blockIdx.x; u < units; u += gridDim.x) {
        const Piece p = joins[u / ncb];
        const int64_t c = (u % ncb) * kSumThreads + threadIdx.x;
        if (c >= H) continue;
        const float *src = partial + (int64_t)p.slot * H + c;
        float s = 0.f;
        for (int i0 = 0; i0 < p.len; i0 += kJoinAhead) {
            float v[kJoinAhead];
#pragma unroll
            for (int j = 0; j < kJoinAhead; ++j) v[j] = i0 + j < p.len ? src[(int64_t)(i0 + j) * H] : 0.f;
#pragma unroll
            for (int j = 0; j < kJoinAhead; ++j)
                if (i0 + j < p.len) s = __fadd_rn(s, v[j]);
        }
        float *dst = dE + (int64_t)p.id * H + c;
        s = __fmul_rn(scale, s);
        *dst = accumulate ? __fadd_rn(*dst, s) : s;
    }
}

// ---- workspace ----

size_t round256(size_t b) { return (b + 255) / 256 * 256; }

struct BwdBuffers {
    int32_t *key[2], *val[2], *hist, *counters;
    Piece *pieces, *joins;
    float *partial;
    size_t bytes;
};

int key_bits(int64_t V) {  // keys are 0 .. V
    int bits = 1;
    while ((int64_t(1) << bits) <= V) ++bits;
    return bits;
}

int64_t tile_pitch(int64_t n) { return ((n + kSortTile - 1) / kSortTile + 3) / 4 * 4; }

BwdBuffers carve(void *base, int64_t n, int64_t H) {
    BwdBuffers b{};
    char *p = static_cast<char *>(base);
    size_t at = 0;
    auto take = [&](size_t bytes) {
        char *q = p + at;
        at += round256(bytes);
        return static_cast<void *>(q);
    };
    for (int i = 0; i < 2; ++i) {
        b.key[i] = static_cast<int32_t *>(take((size_t)n * 4));
        b.val[i] = static_cast<int32_t *>(take((size_t)n * 4));
    }
    b.hist = static_cast<int32_t *>(take((size_t)tile_pitch(n) * kMaxBins * 4));
    b.counters = static_cast<int32_t *>(take(kCounters * 4));
    b.pieces = static_cast<Piece *>(take((size_t)class_first(n, -1) * sizeof(Piece)));
    b.joins = static_cast<Piece *>(take((size_t)(n / kPiece + 1) * sizeof(Piece)));
    b.partial = static_cast<float *>(take((size_t)(n / kHalf + 1) * (size_t)H * 4));
    b.bytes = at;
    return b;
}

template <int THREADS>
cudaError_t launch_small(const Canonical &c, const BwdBuffers &b, int passes, int digit, float *dE,
                         int64_t zeros, const DeviceInfo &di, cudaStream_t st) {
    constexpr size_t smem = sizeof(SmallSort<THREADS>);
    static std::atomic<uint64_t> allowed{0};
    const cudaError_t e =
        allow_shared(reinterpret_cast<const void *>(emb_sort_small<THREADS>), smem, di, allowed);
    if (e != cudaSuccess) return e;
    const int64_t n4 = aligned(dE, 16) ? zeros / 4 : 0, per = THREADS * kZeroVectors;
    const int64_t blocks = (n4 + (zeros - 4 * n4) + per - 1) / per;
    if (blocks >= 0x7fffffff) return cudaErrorInvalidConfiguration;
    return launch_dependent_smem(emb_sort_small<THREADS>, 1 + blocks, THREADS, smem, st, c, passes, digit,
                                 b.key[0], b.val[0], b.pieces, b.joins, b.counters, dE, n4, zeros);
}

// Sorts the canonical tokens and finds their pieces; *where: which of the two
// buffers holds the sorted keys and rows.  Zeros over dE's first `zeros` floats,
// if there are any, come along with a sort of up to kTinyThreads * kSortItems
// tokens.
cudaError_t launch_sort(const Canonical &c, const BwdBuffers &b, int *where, float *dE, int64_t zeros,
                        const DeviceInfo &di, cudaStream_t st) {
    const int bits = key_bits(c.V);
    const int passes = (bits + kMaxDigitBits - 1) / kMaxDigitBits;
    const int digit = (bits + passes - 1) / passes;
    *where = 0;
    if (c.n <= kTinySort) return launch_small<kTinyThreads>(c, b, passes, digit, dE, zeros, di, st);
    if (c.n <= kSmallSort) return launch_small<kSmallThreads>(c, b, passes, digit, dE, 0, di, st);
    const int64_t tiles = (c.n + kSortTile - 1) / kSortTile, pitch = tile_pitch(c.n);
    const int bins = 1 << digit;
    cudaError_t e = launch_dependent(emb_keys, tiles, kSortThreads, st, c, b.key[0], b.val[0], bins, b.hist,
                                     tiles, pitch, b.counters);
    int src = 0;
    for (int p = 0; p < passes && e == cudaSuccess; ++p) {
        const int shift = p * digit;
        if (p > 0)
            e = launch_dependent(emb_histogram, tiles, kSortThreads, st, (const int32_t *)b.key[src], c.n, shift,
                                 bins, b.hist, tiles, pitch);
        if (e != cudaSuccess) return e;
        const bool scanned = tiles > kInlineScanTiles;
        if (scanned) e = launch_dependent(emb_scan, 1, kScanThreads, st, b.hist, pitch * bins);
        if (e != cudaSuccess) return e;
        e = launch_dependent(scanned ? emb_scatter<true> : emb_scatter<false>, tiles, kSortThreads, st,
                             (const int32_t *)b.key[src], (const int32_t *)b.val[src], b.key[1 - src],
                             b.val[1 - src], c.n, shift, bins, (const int32_t *)b.hist, pitch);
        src = 1 - src;
    }
    if (e != cudaSuccess) return e;
    *where = src;
    return launch_dependent(emb_pieces, (c.n + kPieceThreads - 1) / kPieceThreads, kPieceThreads, st,
                            (const int32_t *)b.key[src], c.n, (int32_t)c.V, b.pieces, b.joins, b.counters);
}

template <typename T, bool VEC>
cudaError_t launch_sums(const void *dout, int64_t H, float scale, int64_t n, int where, const BwdBuffers &b,
                        bool accumulate, float *dE, const DeviceInfo &di, cudaStream_t st) {
    cudaError_t e = launch_dependent(emb_sum<T, VEC>, (int64_t)di.sm_count * kSumBlocks, kSumThreads, st,
                                     static_cast<const T *>(dout), H, scale, (const int32_t *)b.val[where],
                                     (const Piece *)b.pieces, n, (const int32_t *)b.counters, (int)accumulate,
                                     dE, b.partial);
    if (e != cudaSuccess || n <= kPiece) return e;
    return launch_dependent(emb_join, (int64_t)di.sm_count * 16, kSumThreads, st, H, scale,
                            (const Piece *)b.joins, (const int32_t *)b.counters, (int)accumulate, dE,
                            (const float *)b.partial);
}

template <typename TE, typename TO>
cudaError_t launch_lookup(const int64_t *ids, const int32_t *cu, int num_seqs, const void *E, int64_t T,
                          int64_t H, int64_t V, float scale, void *out, const DeviceInfo &di,
                          cudaStream_t st) {
    const bool vec = H % 8 == 0 && aligned(E, 16) && aligned(out, 16);
    auto *kernel = vec ? embedding_kernel<TE, TO, true> : embedding_kernel<TE, TO, false>;
    return launch_dependent(kernel, T, kLookupThreads, st, ids, cu, num_seqs,
                            static_cast<const TE *>(E), H, V, scale, static_cast<TO *>(out), di.err);
}

}  // namespace

cudaError_t launch_embedding(const int64_t *ids, const int32_t *cu, int num_seqs, const void *E,
                             rk_dtype e_type, int64_t T, int64_t H, int64_t V, float scale,
                             void *out, rk_dtype out_type, const DeviceInfo &di, cudaStream_t st) {
    if (e_type == RK_BF16)
        return out_type == RK_BF16
                   ? launch_lookup<uint16_t, uint16_t>(ids, cu, num_seqs, E, T, H, V, scale, out, di, st)
                   : launch_lookup<uint16_t, float>(ids, cu, num_seqs, E, T, H, V, scale, out, di, st);
    return out_type == RK_BF16
               ? launch_lookup<float, uint16_t>(ids, cu, num_seqs, E, T, H, V, scale, out, di, st)
               : launch_lookup<float, float>(ids, cu, num_seqs, E, T, H, V, scale, out, di, st);
}

size_t embedding_bwd_workspace_bytes(int64_t n, int64_t H) { return carve(nullptr, n, H).bytes; }

cudaError_t launch_embedding_bwd(const void *dout, rk_dtype dout_type, const int64_t *ids,
                                 const int32_t *cu, int num_seqs, int64_t T, int64_t H, int64_t V,
                                 float scale, const int64_t *order, int64_t n, float *dE,
                                 bool accumulate, void *workspace, const DeviceInfo &di,
                                 cudaStream_t st) {
    if (n == 0)
        return accumulate ? cudaSuccess : cudaMemsetAsync(dE, 0, (size_t)V * (size_t)H * 4, st);
    const BwdBuffers b = carve(workspace, n, H);
    const Canonical c{ids, cu, num_seqs, T, V, order, n, di.err};
    // Zeros in the rows without a token.  While one block sorts, the rest of
    // the device writes zeros over all of dE, and the rows with a token are
    // written again, at most 1 / kZeroAllShare of them (8192 tokens, 152064 x
    // 3584: 34 us of sorting hidden for 8 us more to write).  Few tokens leave
    // the shared memory for it to be one launch.  Otherwise each row looks
    // itself up in the sorted keys.
    const bool zero_all = !accumulate && n <= kSmallSort && n * kZeroAllShare <= V, along = zero_all && n <= kTinySort;
    const int64_t n1 = V * H;
    int where;
    cudaError_t e = launch_sort(c, b, &where, dE, along ? n1 : 0, di, st);
    if (e != cudaSuccess) return e;
    if (zero_all && !along) {
        const int64_t n4 = aligned(dE, 16) ? n1 / 4 : 0;
        const int64_t per = kZeroThreads * kZeroVectors, blocks = (n4 + (n1 - 4 * n4) + per - 1) / per;
        if (blocks > 0x7fffffff) return cudaErrorInvalidConfiguration;
        e = launch_dependent(emb_zero_all, blocks, kZeroThreads, st, dE, n4, n1);
    } else if (!accumulate && !along) {
        const int64_t blocks = (V + kAbsentThreads / 32 - 1) / (kAbsentThreads / 32);
        const bool v4 = H % 4 == 0 && aligned(dE, 16);
        e = launch_dependent(v4 ? emb_zero_absent<true> : emb_zero_absent<false>, blocks, kAbsentThreads, st,
                             (const int32_t *)b.key[where], n, H, V, dE);
    }
    if (e != cudaSuccess) return e;
    const bool vec = H % 8 == 0 && aligned(dout, 16) && aligned(dE, 16);
    if (dout_type == RK_BF16)
        return vec ? launch_sums<uint16_t, true>(dout, H, scale, n, where, b, accumulate, dE, di, st)
                   : launch_sums<uint16_t, false>(dout, H, scale, n, where, b, accumulate, dE, di, st);
    return vec ? launch_sums<float, true>(dout, H, scale, n, where, b, accumulate, dE, di, st)
               : launch_sums<float, false>(dout, H, scale, n, where, b, accumulate, dE, di, st);
}

}  // namespace rk
