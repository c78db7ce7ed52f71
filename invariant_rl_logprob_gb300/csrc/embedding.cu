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
//           kMaxDigitBits; inactive tokens get the key V and end up last);
//   pieces  each id's run in the sorted list is cut into pieces of kPiece
//           occurrences, counted from the run's own start;
//   sum     a block per (piece, slice of columns) adds the piece's rows in
//           order in fp32.  An id with one piece writes its row of dE; the
//           others write partial sums, which a last kernel adds in order.
// The pieces of an id depend on its own occurrences alone, so its row of dE
// does too.  The order in which blocks find the pieces does not matter: no
// two write the same place.
#include <algorithm>
#include <utility>

#include "rk_device.cuh"
#include "rk_internal.h"

namespace rk {
namespace {

__device__ __forceinline__ void wait_prior_grid() {
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
}

// Launch with programmatic stream serialisation: the kernel's blocks may
// become resident while the previous kernel of the stream ends; each waits
// (wait_prior_grid) before it reads or writes anything.
template <typename... P, typename... A>
cudaError_t launch_dependent(void (*kernel)(P...), int64_t grid, int block, cudaStream_t st,
                             A... args) {
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3((unsigned)grid);
    cfg.blockDim = dim3((unsigned)block);
    cfg.stream = st;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, args...);
}

// ---- elements, eight at a time or one by one ----

__device__ __forceinline__ float get1(const uint16_t *p) { return bf16_bits_to_f32(*p); }
__device__ __forceinline__ float get1(const float *p) { return *p; }
__device__ __forceinline__ void get8(const uint16_t *p, float (&v)[8]) {
    const uint4 w = reinterpret_cast<const uint4 *>(p)[0];
    const uint32_t q[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        v[2 * j] = bf16_lo(q[j]);
        v[2 * j + 1] = bf16_hi(q[j]);
    }
}
__device__ __forceinline__ void get8(const float *p, float (&v)[8]) {
    const float4 a = reinterpret_cast<const float4 *>(p)[0];
    const float4 b = reinterpret_cast<const float4 *>(p)[1];
    v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
    v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
}
__device__ __forceinline__ void put1(uint16_t *p, float v) {
    *p = (uint16_t)(pack_bf16x2(v, 0.f) & 0xffffu);
}
__device__ __forceinline__ void put1(float *p, float v) { *p = v; }
__device__ __forceinline__ void put8(uint16_t *p, const float (&v)[8]) {
    *reinterpret_cast<uint4 *>(p) = make_uint4(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]),
                                               pack_bf16x2(v[4], v[5]), pack_bf16x2(v[6], v[7]));
}
__device__ __forceinline__ void put8(float *p, const float (&v)[8]) {
    reinterpret_cast<float4 *>(p)[0] = make_float4(v[0], v[1], v[2], v[3]);
    reinterpret_cast<float4 *>(p)[1] = make_float4(v[4], v[5], v[6], v[7]);
}

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
constexpr int kSortPerWarp = 512;                       // items per warp, in order
constexpr int kSortTile = kSortPerWarp * kSortWarps;    // 4096
constexpr int kMaxDigitBits = 9;
constexpr int kMaxBins = 1 << kMaxDigitBits;
constexpr int kPiece = 64;       // occurrences of an id summed by one block
constexpr int kHalf = kPiece / 2;
constexpr int kScanThreads = 1024;

// Keys and rows of the canonical tokens, in canonical order; row_end cleared.
__global__ void __launch_bounds__(256)
    emb_keys(const int64_t *ids, const int32_t *cu, int num_seqs,
             int64_t T, int64_t V, const int64_t *order, int64_t n,
             int32_t *key, int32_t *val, int32_t *row_end,
             int32_t *counters, unsigned *err) {
    wait_prior_grid();
    const int64_t step = (int64_t)gridDim.x * blockDim.x;
    const int64_t first = (int64_t)blockIdx.x * blockDim.x + threadIdx.x;
    if (first < 2) counters[first] = 0;
    for (int64_t v = first; v < V; v += step) row_end[v] = 0;
    for (int64_t i = first; i < n; i += step) {
        const int64_t r = order ? order[i] : i;
        int64_t k = V;
        if (r >= 0 && r < T) {
            const int64_t id = ids[r];
            if (row_active(r, id, cu, num_seqs)) {
                if (id < V)
                    k = id;
                else
                    atomicOr(err, kErrTargetRange);
            }
        }
        key[i] = (int32_t)k;
        val[i] = (int32_t)(k < V ? r : 0);
    }
}

// Radix pass, first part: hist[d * tiles + b] = items of tile b with digit d.
__global__ void __launch_bounds__(kSortThreads)
    emb_histogram(const int32_t *key, int64_t n, int shift, int bins,
                  int32_t *hist, int64_t tiles) {
    __shared__ int cnt[kMaxBins];
    wait_prior_grid();
    for (int d = threadIdx.x; d < bins; d += kSortThreads) cnt[d] = 0;
    __syncthreads();
    const int64_t base = (int64_t)blockIdx.x * kSortTile;
    for (int i = threadIdx.x; i < kSortTile; i += kSortThreads)
        if (base + i < n) atomicAdd(&cnt[(key[base + i] >> shift) & (bins - 1)], 1);
    __syncthreads();
    for (int d = threadIdx.x; d < bins; d += kSortThreads) hist[d * tiles + blockIdx.x] = cnt[d];
}

// Exclusive prefix sums over cnt[0..len) in place, by one block.
__global__ void __launch_bounds__(kScanThreads)
    emb_scan(int32_t *cnt, int64_t len) {
    __shared__ int warp_sums[32];
    wait_prior_grid();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int carry = 0;
    for (int64_t base = 0; base < len; base += 8 * kScanThreads) {
        const int64_t i0 = base + 8 * (int64_t)threadIdx.x;
        int v[8], sum = 0;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            v[j] = i0 + j < len ? cnt[i0 + j] : 0;
            sum += v[j];
        }
        int incl = sum;
#pragma unroll
        for (int off = 1; off < 32; off <<= 1) {
            const int y = __shfl_up_sync(0xffffffffu, incl, off);
            if (lane >= off) incl += y;
        }
        if (lane == 31) warp_sums[warp] = incl;
        __syncthreads();
        if (warp == 0) {
            int w = warp_sums[lane];
#pragma unroll
            for (int off = 1; off < 32; off <<= 1) {
                const int y = __shfl_up_sync(0xffffffffu, w, off);
                if (lane >= off) w += y;
            }
            warp_sums[lane] = w;
        }
        __syncthreads();
        int run = carry + (warp > 0 ? warp_sums[warp - 1] : 0) + incl - sum;
        carry += warp_sums[31];
        __syncthreads();
#pragma unroll
        for (int j = 0; j < 8; ++j)
            if (i0 + j < len) {
                cnt[i0 + j] = run;
                run += v[j];
            }
    }
}

// Radix pass, last part: a tile's items to their digit's place, order kept.
// Each warp walks its own kSortPerWarp consecutive items 32 at a time; an
// item's rank is the number of earlier lanes with its digit plus the warp's
// running count of that digit.
__global__ void __launch_bounds__(kSortThreads)
    emb_scatter(const int32_t *ks, const int32_t *vs,
                int32_t *kd, int32_t *vd, int64_t n, int shift, int bins,
                const int32_t *hist, int64_t tiles) {
    __shared__ int cnt[kSortWarps][kMaxBins];
    wait_prior_grid();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    for (int d = threadIdx.x; d < kSortWarps * kMaxBins; d += kSortThreads) (&cnt[0][0])[d] = 0;
    __syncthreads();
    const int64_t base = (int64_t)blockIdx.x * kSortTile + (int64_t)warp * kSortPerWarp;
    for (int i = lane; i < kSortPerWarp; i += 32)
        if (base + i < n) atomicAdd(&cnt[warp][(ks[base + i] >> shift) & (bins - 1)], 1);
    __syncthreads();
    for (int d = threadIdx.x; d < bins; d += kSortThreads) {
        int run = hist[d * tiles + blockIdx.x];
#pragma unroll
        for (int w = 0; w < kSortWarps; ++w) {
            const int c = cnt[w][d];
            cnt[w][d] = run;
            run += c;
        }
    }
    __syncthreads();
    for (int i0 = 0; i0 < kSortPerWarp; i0 += 32) {
        const bool live = base + i0 + lane < n;
        const int32_t k = live ? ks[base + i0 + lane] : 0;
        const int32_t v = live ? vs[base + i0 + lane] : 0;
        const int d = live ? (k >> shift) & (bins - 1) : -1;
        const unsigned peers = __match_any_sync(0xffffffffu, d);
        const int rank = __popc(peers & ((1u << lane) - 1u));
        const int at = live ? cnt[warp][d] + rank : 0;
        __syncwarp();
        if (live) {
            if (rank == 0) cnt[warp][d] += __popc(peers);
            kd[at] = k;
            vd[at] = v;
        }
        __syncwarp();
    }
}

// ---- gradient: pieces ----

struct Piece {
    int32_t id, pos, len;  // rows val[pos .. pos + len) of id
    int32_t slot;          // partial sum, or -1: the id has this piece alone
};

// For each run of equal ids below V: row_end[id] = its end, and its pieces.
// The partial sums of a run that starts at b take slots ceil(b / kHalf), ...:
// a run of more than kPiece items has at least as many multiples of kHalf as
// pieces, so no two runs share a slot.
__global__ void __launch_bounds__(256)
    emb_pieces(const int32_t *key, int64_t n, int32_t V, int32_t *row_end,
               Piece *pieces, Piece *joins, int32_t *counters) {
    __shared__ int block_base, warp_cnt[8];
    wait_prior_grid();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
    const int32_t k = i < n ? key[i] : V;
    const bool start = k < V && (i == 0 || key[i - 1] != k);
    int64_t end = 0;
    if (start) {
        int64_t lo = i + 1, hi = min(n, i + kPiece);  // first position past the run
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
        end = lo;
        row_end[k] = (int32_t)end;
    }
    const int np = start ? (int)((end - i + kPiece - 1) / kPiece) : 0;
    int incl = np;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, incl, off);
        if (lane >= off) incl += y;
    }
    if (lane == 31) warp_cnt[warp] = incl;
    __syncthreads();
    if (threadIdx.x == 0) {
        int all = 0;
        for (int w = 0; w < 8; ++w) {
            const int c = warp_cnt[w];
            warp_cnt[w] = all;
            all += c;
        }
        block_base = all ? atomicAdd(&counters[0], all) : 0;
    }
    __syncthreads();
    if (!start) return;
    Piece *p = pieces + block_base + warp_cnt[warp] + incl - np;
    const int32_t slot = (int32_t)((i + kHalf - 1) / kHalf);
    for (int j = 0; j < np; ++j) {
        const int64_t at = i + (int64_t)j * kPiece;
        p[j] = Piece{k, (int32_t)at, (int32_t)min((int64_t)kPiece, end - at), np > 1 ? slot + j : -1};
    }
    if (np > 1) joins[atomicAdd(&counters[1], 1)] = Piece{k, (int32_t)i, np, slot};
}

// ---- gradient: sums ----

constexpr int kSumThreads = 128;

// dE row and column c0.. of one id from its sum.
template <bool VEC>
__device__ __forceinline__ void put_row(float *p, bool accumulate, float scale, float (&s)[8]) {
    constexpr int N = VEC ? 8 : 1;
#pragma unroll
    for (int j = 0; j < N; ++j) s[j] = __fmul_rn(scale, s[j]);
    if (accumulate) {
        float old[8];
        if (VEC) {
            const float4 a = reinterpret_cast<const float4 *>(p)[0];
            const float4 b = reinterpret_cast<const float4 *>(p)[1];
            old[0] = a.x; old[1] = a.y; old[2] = a.z; old[3] = a.w;
            old[4] = b.x; old[5] = b.y; old[6] = b.z; old[7] = b.w;
        } else {
            old[0] = *p;
        }
#pragma unroll
        for (int j = 0; j < N; ++j) s[j] = __fadd_rn(old[j], s[j]);
    }
    if (VEC)
        put8(p, s);
    else
        *p = s[0];
}

template <typename T, bool VEC>
__global__ void __launch_bounds__(kSumThreads)
    emb_sum(const T *dout, int64_t H, int64_t V, float scale,
            const int32_t *val, const int32_t *row_end,
            const Piece *pieces, const int32_t *counters, int accumulate,
            float *dE, float *partial) {
    constexpr int N = VEC ? 8 : 1;
    constexpr int kCols = N * kSumThreads;
    wait_prior_grid();
    const int64_t ncb = (H + kCols - 1) / kCols;
    const int64_t units = (int64_t)counters[0] * ncb;
    for (int64_t u = blockIdx.x; u < units; u += gridDim.x) {
        const Piece p = pieces[u / ncb];
        const int64_t c = (u % ncb) * kCols + N * (int64_t)threadIdx.x;
        if (c >= H) continue;
        float s[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
        for (int i = 0; i < p.len; ++i) {
            const T *src = dout + (int64_t)val[p.pos + i] * H + c;
            if (VEC) {
                float v[8];
                get8(src, v);
#pragma unroll
                for (int j = 0; j < 8; ++j) s[j] = __fadd_rn(s[j], v[j]);
            } else {
                s[0] = __fadd_rn(s[0], get1(src));
            }
        }
        if (p.slot < 0) {
            put_row<VEC>(dE + (int64_t)p.id * H + c, accumulate, scale, s);
        } else if (VEC) {
            put8(partial + (int64_t)p.slot * H + c, s);
        } else {
            partial[(int64_t)p.slot * H + c] = s[0];
        }
    }
    if (accumulate) return;
    for (int64_t v = blockIdx.x; v < V; v += gridDim.x) {  // rows without a token
        if (row_end[v] != 0) continue;
        float *row = dE + v * H;
        if (VEC) {
            const float zero[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
            for (int64_t c = 8 * (int64_t)threadIdx.x; c < H; c += kCols) put8(row + c, zero);
        } else {
            for (int64_t c = threadIdx.x; c < H; c += kCols) row[c] = 0.f;
        }
    }
}

// The ids with more than one piece: their partial sums, added in order.
template <bool VEC>
__global__ void __launch_bounds__(kSumThreads)
    emb_join(int64_t H, float scale, const Piece *joins,
             const int32_t *counters, int accumulate, float *dE,
             const float *partial) {
    constexpr int N = VEC ? 8 : 1;
    constexpr int kCols = N * kSumThreads;
    wait_prior_grid();
    const int64_t ncb = (H + kCols - 1) / kCols;
    const int64_t units = (int64_t)counters[1] * ncb;
    for (int64_t u = blockIdx.x; u < units; u += gridDim.x) {
        const Piece p = joins[u / ncb];
        const int64_t c = (u % ncb) * kCols + N * (int64_t)threadIdx.x;
        if (c >= H) continue;
        float s[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
        for (int i = 0; i < p.len; ++i) {
            const float *src = partial + (int64_t)(p.slot + i) * H + c;
            if (VEC) {
                float v[8];
                get8(src, v);
#pragma unroll
                for (int j = 0; j < 8; ++j) s[j] = __fadd_rn(s[j], v[j]);
            } else {
                s[0] = __fadd_rn(s[0], *src);
            }
        }
        put_row<VEC>(dE + (int64_t)p.id * H + c, accumulate, scale, s);
    }
}

// ---- workspace ----

size_t round256(size_t b) { return (b + 255) / 256 * 256; }

struct BwdBuffers {
    int32_t *key[2], *val[2], *hist, *row_end, *counters;
    Piece *pieces, *joins;
    float *partial;
    size_t bytes;
};

int key_bits(int64_t V) {  // keys are 0 .. V
    int bits = 1;
    while ((int64_t(1) << bits) <= V) ++bits;
    return bits;
}

BwdBuffers carve(void *base, int64_t n, int64_t H, int64_t V) {
    BwdBuffers b{};
    char *p = static_cast<char *>(base);
    size_t at = 0;
    auto take = [&](size_t bytes) {
        char *q = p + at;
        at += round256(bytes);
        return static_cast<void *>(q);
    };
    const size_t tiles = (size_t)((n + kSortTile - 1) / kSortTile);
    for (int i = 0; i < 2; ++i) {
        b.key[i] = static_cast<int32_t *>(take((size_t)n * 4));
        b.val[i] = static_cast<int32_t *>(take((size_t)n * 4));
    }
    b.hist = static_cast<int32_t *>(take(tiles * kMaxBins * 4));
    b.row_end = static_cast<int32_t *>(take((size_t)V * 4));
    b.counters = static_cast<int32_t *>(take(2 * 4));
    b.pieces = static_cast<Piece *>(take((size_t)n * sizeof(Piece)));
    b.joins = static_cast<Piece *>(take((size_t)(n / kPiece + 1) * sizeof(Piece)));
    b.partial = static_cast<float *>(take((size_t)(n / kHalf + 1) * (size_t)H * 4));
    b.bytes = at;
    return b;
}

template <typename T, bool VEC>
cudaError_t launch_sums(const void *dout, int64_t H, int64_t V, float scale, const int32_t *val,
                        const BwdBuffers &b, bool accumulate, float *dE, const DeviceInfo &di,
                        cudaStream_t st) {
    cudaError_t e = launch_dependent(emb_sum<T, VEC>, (int64_t)di.sm_count * 16, kSumThreads, st,
                                     static_cast<const T *>(dout), H, V, scale, val, b.row_end,
                                     b.pieces, b.counters, (int)accumulate, dE, b.partial);
    if (e != cudaSuccess) return e;
    return launch_dependent(emb_join<VEC>, (int64_t)di.sm_count * 4, kSumThreads, st, H, scale,
                            b.joins, b.counters, (int)accumulate, dE, b.partial);
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

size_t embedding_bwd_workspace_bytes(int64_t n, int64_t H, int64_t V) {
    return carve(nullptr, n, H, V).bytes;
}

cudaError_t launch_embedding_bwd(const void *dout, rk_dtype dout_type, const int64_t *ids,
                                 const int32_t *cu, int num_seqs, int64_t T, int64_t H, int64_t V,
                                 float scale, const int64_t *order, int64_t n, float *dE,
                                 bool accumulate, void *workspace, const DeviceInfo &di,
                                 cudaStream_t st) {
    if (n == 0)
        return accumulate ? cudaSuccess : cudaMemsetAsync(dE, 0, (size_t)V * (size_t)H * 4, st);
    const BwdBuffers b = carve(workspace, n, H, V);
    const int64_t blocks = std::min<int64_t>((std::max(n, V) + 255) / 256, (int64_t)di.sm_count * 8);
    cudaError_t e = launch_dependent(emb_keys, blocks, 256, st, ids, cu, num_seqs, T, V, order, n,
                                     b.key[0], b.val[0], b.row_end, b.counters, di.err);
    if (e != cudaSuccess) return e;
    const int bits = key_bits(V);
    const int passes = (bits + kMaxDigitBits - 1) / kMaxDigitBits;
    const int digit = (bits + passes - 1) / passes;
    const int64_t tiles = (n + kSortTile - 1) / kSortTile;
    int src = 0;
    for (int p = 0; p < passes; ++p) {
        const int shift = p * digit, bins = 1 << digit;
        e = launch_dependent(emb_histogram, tiles, kSortThreads, st, b.key[src], n, shift, bins, b.hist,
                             tiles);
        if (e != cudaSuccess) return e;
        e = launch_dependent(emb_scan, 1, kScanThreads, st, b.hist, tiles * bins);
        if (e != cudaSuccess) return e;
        e = launch_dependent(emb_scatter, tiles, kSortThreads, st, b.key[src], b.val[src],
                             b.key[1 - src], b.val[1 - src], n, shift, bins, b.hist, tiles);
        if (e != cudaSuccess) return e;
        src = 1 - src;
    }
    e = launch_dependent(emb_pieces, (n + 255) / 256, 256, st, b.key[src], n, (int32_t)V, b.row_end,
                         b.pieces, b.joins, b.counters);
    if (e != cudaSuccess) return e;
    const bool vec = H % 8 == 0 && aligned(dout, 16) && aligned(dE, 16);
    const int32_t *val = b.val[src];
    if (dout_type == RK_BF16)
        return vec ? launch_sums<uint16_t, true>(dout, H, V, scale, val, b, accumulate, dE, di, st)
                   : launch_sums<uint16_t, false>(dout, H, V, scale, val, b, accumulate, dE, di, st);
    return vec ? launch_sums<float, true>(dout, H, V, scale, val, b, accumulate, dE, di, st)
               : launch_sums<float, false>(dout, H, V, scale, val, b, accumulate, dE, di, st);
}

}  // namespace rk
