// rms_norm_bwd.cu -- gradient of the root-mean-square norm (its weight's gradient
// belongs to the parameter gradients of issue #244, Workstream 3 #153: fixed
// order, no atomicAdd).
//
//   g = dout * weight,  n = r * rstd
//   dx = rstd * (g - n * mean(g * n)) + dr,   dweight (+)= sum over rows of dout * n
//
// Bound by memory: 15 flop an element, against 6 to 16 bytes.  It needs nothing but
// r: the sums of r^2 and of g * r come out of one reduction.  dweight: a team
// (rms_norm.cuh) adds its rows in registers, in order; blocks leave partial sums
// that a last kernel adds in order.  Teams therefore stay, and ask for their next row
// ahead, into the second cache (65536 x 4096, all bf16: 347 us without, 318 with, the
// copy rate).
//
// Which rows a team takes depends on the number of canonical rows and on the number of teams, which
// H, the types and whether there is a dr decide (`halved`).
#include <algorithm>

#include "rms_norm.cuh"

namespace rk {
namespace {

__device__ __forceinline__ float one(const void *p, int type, int c) {
    return type == RK_FP32 ? get1(static_cast<const float *>(p) + c) : get1(static_cast<const uint16_t *>(p) + c);
}

// ---- the canonical rows: the active ones among the candidates, order kept ----

constexpr int kListItems = 8;  // consecutive candidates of a thread

struct Candidates {
    const int64_t *order;  // or NULL: rows 0, 1, ...
    int64_t n, T;
    const int64_t *targets;  // or NULL: all active
    const int32_t *cu;
    int32_t num_seqs;
};

// Rows of candidates first .. first + 7 (-1: none), and how many there are.
__device__ __forceinline__ int candidate_rows(const Candidates &c, int64_t first, int64_t lo, int64_t hi,
                                              int (&row)[kListItems]) {
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

// The sum of `v` over the lanes up to this one.
__device__ __forceinline__ int sum_upto(int v) {
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, v, off);
        if ((threadIdx.x & 31) >= off) v += y;
    }
    return v;
}

// The list by every block for itself, in shared memory; returns how many.
template <int BLOCK>
__device__ __forceinline__ int list_rows(const Candidates &c, int64_t lo, int64_t hi, int32_t *rows, uint8_t *listed,
                                         int (&warps)[BLOCK / 32]) {
    for (int t = threadIdx.x; t < (int)c.T; t += BLOCK) listed[t] = 0;
    __syncthreads();
    int total = 0;
    for (int64_t base = 0; base < c.n; base += BLOCK * kListItems) {
        int row[kListItems];
        const int mine = candidate_rows(c, base + threadIdx.x * kListItems, lo, hi, row);
        const int upto = sum_upto(mine);
        if ((threadIdx.x & 31) == 31) warps[threadIdx.x >> 5] = upto;
        __syncthreads();
        int at = total + upto - mine;
#pragma unroll
        for (int w = 0; w < BLOCK / 32; ++w) {
            at += w < (int)threadIdx.x >> 5 ? warps[w] : 0;
            total += warps[w];
        }
#pragma unroll
        for (int i = 0; i < kListItems; ++i) {
            if (row[i] < 0) continue;
            rows[at++] = row[i];
            listed[row[i]] = 1;
        }
        __syncthreads();
    }
    return total;
}

struct NormBwdArgs {
    Matrix r, dout, dr;  // dr.p may be NULL
    const void *weight;
    int32_t weight_type;
    float eps, per_column;  // 1 / H
    const int32_t *cu;
    int32_t num_seqs;
    int64_t T;
    int32_t H;
    const int32_t *rows;    // the canonical rows, or NULL: those of the cu_seqlens range
    int64_t *n_rows;        // how many
    const uint8_t *listed;  // which rows are among them
    Matrix dx;
    int32_t stage_dx;  // its rows leave through shared memory
    float *partial;    // [blocks, pitch_of(H)], or NULL: no dweight
    Candidates from;   // LIST: what blocks take the rows from, and where in shared memory they keep them
    int32_t list_at;   // and, behind them, which are listed; rows and listed are NULL, n_rows is written
};

__host__ __device__ constexpr int64_t pitch_of(int64_t H) { return (H + 7) / 8 * 8; }

// What the backward keeps of a row between its sums and its results: with kWords (r, dout and dr in
// bf16) and kMixed (the same with dout in fp32) its words, with kAligned up to 16 columns a thread;
// otherwise nothing, it is read again, from the caches.  65536 x 4096: kWords 318 us, kMixed 398 (both
// the copy rate); without kMixed its case took 610.  32768 x 4096 all in fp32: 316, the copy rate, where
// 32 columns a thread, read again, take 417.
constexpr int kMixed = 3;

// LIST: every block lists the canonical rows for itself.  (A variant of its own: as a branch it cost
// the large cases 1 % in registers.)
template <int TEAM, int NV, int READ, int BLOCK, int PER_SM, bool LIST>
__global__ void __launch_bounds__(BLOCK, PER_SM) rms_norm_backward(const __grid_constant__ NormBwdArgs a) {
    using C = Columns<TEAM>;
    constexpr int kTeams = BLOCK / TEAM;
    __shared__ float2 sums[2][32];
    // the teams' stages, and in the end their sums of dweight
    extern __shared__ __align__(16) char stages[];
    const int lane = threadIdx.x % TEAM, H = a.H;
    char *stage = stages + (size_t)(threadIdx.x / TEAM) * stage_bytes(H);
    wait_prior_grid();

    int64_t lo, hi;
    row_range(a.cu, a.num_seqs, a.T, &lo, &hi);
    int64_t n;
    const int32_t *rows = a.rows;
    const uint8_t *listed = a.listed;
    if constexpr (LIST) {
        __shared__ int warps[BLOCK / 32];
        int32_t *const list = reinterpret_cast<int32_t *>(stages + a.list_at);
        uint8_t *const in_list = reinterpret_cast<uint8_t *>(list + a.from.n);
        n = list_rows<BLOCK>(a.from, lo, hi, list, in_list, warps);
        if (blockIdx.x == 0 && threadIdx.x == 0) *a.n_rows = n;  // for rms_norm_join
        rows = list;
        listed = in_list;
    } else {
        n = rows ? *a.n_rows : max((int64_t)0, hi - lo);
    }
    const int64_t teams = (int64_t)gridDim.x * kTeams;
    const int64_t team = (int64_t)blockIdx.x * kTeams + threadIdx.x / TEAM;
    float acc[NV][8];
#pragma unroll
    for (int k = 0; k < NV; ++k)
#pragma unroll
        for (int e = 0; e < 8; ++e) acc[k][e] = 0.f;

    int parity = 0;
    // fewer than 2^31 rows
    const int last = (int)n, step = (int)teams, first = (int)lo;
    const auto row_at = [&](int64_t i) { return i >= last ? 0 : rows ? rows[i] : first + (int)i; };
    // what is kept of a row between its sums and its results
    constexpr bool kKeep = READ == kAligned && NV <= 2;
    struct Held {
        uint4 r[NV], d[NV * (READ == kMixed ? 2 : 1)], z[NV];
        Raw raw_r[kKeep ? NV : 1], raw_d[kKeep ? NV : 1], raw_z[kKeep ? NV : 1];
    };
    const auto hold = [&](int t, Held &h) {
        const char *r = a.r.row(t), *d = a.dout.row(t), *z = a.dr.row(t);
        if constexpr (READ == kWords || READ == kMixed) {
#pragma unroll
            for (int k = 0; k < NV; ++k) {
                const int c = C::at(lane, k);
                h.r[k] = C::words(r, k, H, lane);
                if constexpr (READ == kWords) {
                    h.d[k] = C::words(d, k, H, lane);
                } else {
                    const uint4 *from = reinterpret_cast<const uint4 *>(d + 4 * c);
                    h.d[2 * k] = c < H ? from[0] : make_uint4(0, 0, 0, 0);
                    h.d[2 * k + 1] = c < H ? from[1] : make_uint4(0, 0, 0, 0);
                }
                h.z[k] = a.dr.p ? C::words(z, k, H, lane) : make_uint4(0, 0, 0, 0);
            }
        } else if constexpr (kKeep) {
#pragma unroll
            for (int k = 0; k < NV; ++k) {
                h.raw_r[k] = raw_vector<TEAM>(r, a.r.type == RK_FP32, true, k, H, lane);
                h.raw_d[k] = raw_vector<TEAM>(d, a.dout.type == RK_FP32, true, k, H, lane);
                h.raw_z[k] = raw_vector<TEAM>(z, a.dr.type == RK_FP32, a.dr.p, k, H, lane);
            }
        }
    };
    // A narrow row is asked for a row ahead in registers, not in the second cache: 2^27 elements of bf16 with
    // dr, 64 columns 227 us against 277, with the weight kept as well 186 (128 columns: 185 for 210, 256: 182 for
    // 190).
    constexpr bool kAhead = NV == 1 && (READ == kWords || READ == kMixed);
    Held h, ahead;
    // the weight, kept as well where there is room (512 columns 162 us for 187)
    constexpr bool kWeight = NV <= 2 && READ != kFloats;
    float kept[kWeight ? NV : 1][8];
    if constexpr (kWeight) {
#pragma unroll
        for (int k = 0; k < NV; ++k) weight_vector<TEAM, READ>(a.weight, a.weight_type, k, H, lane, kept[k]);
    }
    const auto weight = [&](int k, float (&w)[8]) {
        if constexpr (kWeight) {
#pragma unroll
            for (int e = 0; e < 8; ++e) w[e] = kept[k][e];
        } else {
            weight_vector<TEAM, READ>(a.weight, a.weight_type, k, H, lane, w);
        }
    };
    int next = row_at(team);
    if constexpr (kAhead) {
        if (team < last) hold(next, ahead);
    }
    for (int64_t i = team; i < last; i += step) {
        const int t = next;
        next = row_at(i + step);
        const auto r = [&] { return a.r.row(t); };
        const auto d = [&] { return a.dout.row(t); };
        const auto z = [&] { return a.dr.row(t); };
        if constexpr (kAhead) {
            h = ahead;
            if (i + step < last) hold(next, ahead);
        } else {
            if (lane < 3 && i + step < last) {
                // the team's next row, on its way into the second cache
                const Matrix &m = lane == 0 ? a.r : lane == 1 ? a.dout : a.dr;
                if (m.p) {
                    const uintptr_t from = reinterpret_cast<uintptr_t>(m.row(next)), to = from + H * size_of(m.type);
                    const uintptr_t first16 = from & ~uintptr_t(15);
                    asm volatile("cp.async.bulk.prefetch.L2.global [%0], %1;" ::"l"(first16),
                                 "r"((uint32_t)((to + 15 & ~uintptr_t(15)) - first16))
                                 : "memory");
                }
            }
            hold(t, h);
        }
        constexpr int kPair = NV > 1 ? 2 : 1;
        // vectors k .. k + kPair - 1 of r, dout and the weight
        const auto values = [&](int k, float (&x)[kPair][8], float (&g)[kPair][8], float (&w)[kPair][8]) {
            if constexpr (READ == kFloats) {
                C::load(r(), a.r.type, k, H, lane, x);
                C::load(d(), a.dout.type, k, H, lane, g);
                C::load(a.weight, a.weight_type, k, H, lane, w);
            } else if constexpr (READ == kAligned) {
                const bool r_wide = a.r.type == RK_FP32, d_wide = a.dout.type == RK_FP32;
                Raw p[kPair], q[kPair];
#pragma unroll
                for (int i = 0; i < kPair; ++i) {
                    p[i] = kKeep ? h.raw_r[kKeep ? k + i : 0] : raw_vector<TEAM>(r(), r_wide, true, k + i, H, lane);
                    q[i] = kKeep ? h.raw_d[kKeep ? k + i : 0] : raw_vector<TEAM>(d(), d_wide, true, k + i, H, lane);
                }
#pragma unroll
                for (int i = 0; i < kPair; ++i) {
                    weight(k + i, w[i]);
                    unpack(p[i], r_wide, x[i]);
                    unpack(q[i], d_wide, g[i]);
                }
            } else {
#pragma unroll
                for (int i = 0; i < kPair; ++i) {
                    weight(k + i, w[i]);
                    unpack(h.r[k + i], x[i]);
                    if constexpr (READ == kWords) {
                        unpack(h.d[k + i], g[i]);
                    } else {
                        const uint4 p = h.d[2 * (k + i)], q = h.d[2 * (k + i) + 1];
                        const uint32_t v[8] = {p.x, p.y, p.z, p.w, q.x, q.y, q.z, q.w};
#pragma unroll
                        for (int e = 0; e < 8; ++e) g[i][e] = __uint_as_float(v[e]);
                    }
                }
            }
        };

        // sums of z^2 and g z, z = k r
        float k1 = 1.f;
        float2 s;
        {
            float even1 = 0.f, odd1 = 0.f, even2 = 0.f, odd2 = 0.f;
#pragma unroll
            for (int k = 0; k < NV; k += kPair) {
                float x[kPair][8], g[kPair][8], w[kPair][8];
                values(k, x, g, w);
#pragma unroll
                for (int i = 0; i < kPair; ++i)
#pragma unroll
                    for (int e = 0; e < 8; e += 2) {
                        mul2(g[i][e], g[i][e + 1], w[i][e], w[i][e + 1]);
                        fma2(even1, odd1, x[i][e], x[i][e + 1], x[i][e], x[i][e + 1]);
                        fma2(even2, odd2, g[i][e], g[i][e + 1], x[i][e], x[i][e + 1]);
                    }
            }
            add2(even1, even2, odd1, odd2);
            s = team_sums<TEAM>(even1, even2, sums[parity]);
            parity ^= 1;
        }
        if (!(s.x < INFINITY)) {
            float squares = 0.f, products = 0.f;
#pragma unroll 1
            for (int k = 0; k < NV; ++k) {
#pragma unroll 1
                for (int e = 0; e < 8; ++e) {
                    const int c = C::at(lane, k) + e;
                    if (c >= H) continue;
                    const float x = kShrink * one(r(), a.r.type, c);
                    squares = __fmaf_rn(x, x, squares);
                    products = __fmaf_rn(__fmul_rn(one(d(), a.dout.type, c), one(a.weight, a.weight_type, c)), x, products);
                }
            }
            s = team_sums<TEAM>(squares, products, sums[parity]);
            parity ^= 1;
            k1 = kShrink;
        }
        // rstd = k q,  n = r rstd,  mean(g n) = q mean(g z)
        const float q = root(s.x, a.per_column, a.eps, k1), rstd = q * k1;
        float c = -__fmul_rn(q, __fmul_rn(s.y, a.per_column));
        if (!(fabsf(c) < INFINITY)) {
            // The products leave fp32: those of g n, or of g 2^-32 and n where g is so large that no more
            // than its mean fits.
            float whole = 0.f, part = 0.f;
#pragma unroll 1
            for (int k = 0; k < NV; ++k) {
#pragma unroll 1
                for (int e = 0; e < 8; ++e) {
                    const int col = C::at(lane, k) + e;
                    if (col >= H) continue;
                    const float up = one(d(), a.dout.type, col), w = one(a.weight, a.weight_type, col);
                    const float n = __fmul_rn(one(r(), a.r.type, col), rstd);
                    whole = __fmaf_rn(__fmul_rn(up, w), n, whole);
                    part = __fmaf_rn(__fmul_rn(__fmul_rn(up, 0x1p-32f), w), n, part);
                }
            }
            s = team_sums<TEAM>(whole, part, sums[parity]);
            parity ^= 1;
            c = fabsf(s.x) < INFINITY ? -__fmul_rn(s.x, a.per_column) : -__fmul_rn(s.y, a.per_column) * 0x1p32f;
        }
#pragma unroll
        for (int k = 0; k < NV; k += kPair) {
            float x[kPair][8], g[kPair][8], w[kPair][8], y[kPair][8];
            const bool z_wide = a.dr.type == RK_FP32;
            Raw zr[kPair];
            if constexpr (READ == kAligned) {
#pragma unroll
                for (int i = 0; i < kPair; ++i)
                    zr[i] = kKeep ? h.raw_z[kKeep ? k + i : 0] : raw_vector<TEAM>(z(), z_wide, a.dr.p, k + i, H, lane);
            }
            values(k, x, g, w);
            if constexpr (READ == kAligned) {
#pragma unroll
                for (int i = 0; i < kPair; ++i) unpack(zr[i], z_wide, y[i]);
            } else if constexpr (READ == kFloats) {
                if (a.dr.p) {
                    C::load(z(), a.dr.type, k, H, lane, y);
                } else {
#pragma unroll
                    for (int j = 0; j < 8 * kPair; ++j) y[j / 8][j % 8] = 0.f;
                }
            } else {
#pragma unroll
                for (int i = 0; i < kPair; ++i) unpack(h.z[k + i], y[i]);
            }
#pragma unroll
            for (int i = 0; i < kPair; ++i) {
#pragma unroll
                for (int e = 0; e < 8; e += 2) {
                    mul2(x[i][e], x[i][e + 1], rstd, rstd);
                    fma2(acc[k + i][e], acc[k + i][e + 1], g[i][e], g[i][e + 1], x[i][e], x[i][e + 1]);
                    mul2(g[i][e], g[i][e + 1], w[i][e], w[i][e + 1]);
                    fma2(g[i][e], g[i][e + 1], x[i][e], x[i][e + 1], c, c);
                    fma2(y[i][e], y[i][e + 1], rstd, rstd, g[i][e], g[i][e + 1]);
                }
                C::store(a.stage_dx ? stage : a.dx.row(t), a.dx.type, k + i, H, lane, y[i]);
            }
        }
        if (a.stage_dx) {
            const int size = size_of(a.dx.type);
            team_sync<TEAM>();
            C::flush(stage, a.dx.row(t), H * size, size, lane);
            team_sync<TEAM>();
        }
    }

    // 0 in the rows that are not among the canonical ones
    if (a.cu || listed) {
        const float zero[8] = {};
        for (int64_t u = team; u < a.T; u += teams) {
            if (listed ? listed[u] : u >= lo && u < hi) continue;
            char *row = a.dx.row(u);
            if (!a.stage_dx) {
#pragma unroll
                for (int k = 0; k < NV; ++k) C::store(row, a.dx.type, k, H, lane, zero);
            } else {
                for (int c = lane; c < H; c += TEAM) {
                    if (a.dx.type == RK_FP32)
                        reinterpret_cast<float *>(row)[c] = 0.f;
                    else
                        reinterpret_cast<uint16_t *>(row)[c] = 0;
                }
            }
        }
    }
    // a block without rows has nothing to leave, and rms_norm_join does not look for it
    if (!a.partial || (int64_t)blockIdx.x * kTeams >= n) return;
    float *partial = a.partial + (int64_t)blockIdx.x * pitch_of(H);
    if constexpr (kTeams == 1) {
#pragma unroll
        for (int k = 0; k < NV; ++k) C::store(reinterpret_cast<char *>(partial), RK_FP32, k, H, lane, acc[k]);
    } else {
        // the block's teams one after the other
        float *joined = reinterpret_cast<float *>(stages);
        __syncthreads();
        for (int j = 0; j < kTeams; ++j) {
            if ((int)(threadIdx.x / TEAM) == j) {
#pragma unroll
                for (int k = 0; k < NV; ++k) {
                    const int c = C::at(lane, k);
#pragma unroll
                    for (int e = 0; e < 8; ++e)
                        if (c < H) joined[c + e] = j == 0 ? acc[k][e] : __fadd_rn(joined[c + e], acc[k][e]);
                }
            }
            __syncthreads();
        }
        for (int c = threadIdx.x; c < H; c += BLOCK) partial[c] = joined[c];
    }
}

// dweight[c] (+)= the partial sums of the blocks that had rows: lane y takes blocks y, y + 32, ...
// in order, then the lanes' sums are added in order.
constexpr int kJoinLanes = 32;
__global__ void __launch_bounds__(32 * kJoinLanes)
    rms_norm_join(const float *partial, int blocks, int rows_of_block, const int64_t *n_rows, const int32_t *cu,
                  int num_seqs, int64_t T, int H, float *dweight, int accumulate) {
    __shared__ float sums[kJoinLanes][33];
    wait_prior_grid();
    int64_t lo, hi;
    row_range(cu, num_seqs, T, &lo, &hi);
    const int64_t n = n_rows ? *n_rows : max((int64_t)0, hi - lo);
    const int busy = (int)min((int64_t)blocks, (n + rows_of_block - 1) / rows_of_block);
    const int x = threadIdx.x & 31, y = threadIdx.x >> 5, c = blockIdx.x * 32 + x;
    float s = 0.f;
    if (c < H) {
#pragma unroll 4
        for (int b = y; b < busy; b += kJoinLanes) s = __fadd_rn(s, partial[b * pitch_of(H) + c]);
    }
    sums[y][x] = s;
    __syncthreads();
    if (y == 0 && c < H) {
        for (int i = 1; i < kJoinLanes; ++i) s = __fadd_rn(s, sums[i][x]);
        dweight[c] = accumulate ? __fadd_rn(dweight[c], s) : s;
    }
}

// ---- the canonical rows by launches of their own ----

constexpr int kListThreads = 1024;
constexpr int kListTile = kListThreads * kListItems;

__device__ __forceinline__ int64_t first_of_thread() {
    return (int64_t)blockIdx.x * kListTile + (int64_t)threadIdx.x * kListItems;
}

__device__ __forceinline__ int block_sum(int v, int *scratch) {
    v = __reduce_add_sync(0xffffffffu, v);
    if ((threadIdx.x & 31) == 0) scratch[threadIdx.x >> 5] = v;
    __syncthreads();
    v = __reduce_add_sync(0xffffffffu, scratch[threadIdx.x & 31]);
    __syncthreads();
    return v;
}

__global__ void __launch_bounds__(kListThreads) norm_rows_count(Candidates c, int32_t *counts) {
    __shared__ int scratch[32];
    wait_prior_grid();
    int64_t lo, hi;
    row_range(c.cu, c.num_seqs, c.T, &lo, &hi);
    int row[kListItems];
    const int total = block_sum(candidate_rows(c, first_of_thread(), lo, hi, row), scratch);
    if (threadIdx.x == 0) counts[blockIdx.x] = total;
}

__global__ void __launch_bounds__(kListThreads)
    norm_rows_write(Candidates c, const int32_t *counts, int32_t *rows, uint8_t *listed, int64_t *n_rows) {  // counts NULL: one block
    __shared__ int scratch[32], warps[32];
    wait_prior_grid();
    int64_t lo, hi;
    row_range(c.cu, c.num_seqs, c.T, &lo, &hi);
    if (!counts) {  // nobody has cleared `listed` either
        for (int64_t t = threadIdx.x; t < c.T; t += kListThreads) listed[t] = 0;
        __syncthreads();
    }
    int before = 0;  // rows of the blocks before this one (fewer than 2^31)
    for (int b = threadIdx.x; counts && b < (int)blockIdx.x; b += kListThreads) before += counts[b];
    before = block_sum(before, scratch);
    int row[kListItems];
    const int mine = candidate_rows(c, first_of_thread(), lo, hi, row);
    int upto = sum_upto(mine);
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
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

constexpr int kSmCount = 152;  // what the backward's partial sums are laid out for, on any device
// Up to so many candidates every block lists the rows for itself, beyond a launch does.  With targets,
// 64 / 2048 / 4096 columns: 300 rows 7.7 / 7.9 / 9.5 us against 9.4 / 9.2 / 11.2, 1000 rows 8.1 / 10.4 /
// 13.9 against 10.1 / 12.0 / 15.6; 2048 rows in an order, with 2048 columns, 25.2 against 19.5.
constexpr int kListed = 1024;

template <int TEAM, int NV, int READ, int BLOCK, int PER_SM, bool LIST>
cudaError_t backward_launch(NormBwdArgs &a, const DeviceInfo &di, cudaStream_t st) {
    auto *kernel = rms_norm_backward<TEAM, NV, READ, BLOCK, PER_SM, LIST>;
    size_t shared = a.stage_dx ? (size_t)(BLOCK / TEAM) * stage_bytes(a.H) : 0;
    if (BLOCK > TEAM) shared = std::max(shared, (size_t)pitch_of(a.H) * 4);
    if (LIST) {
        a.list_at = (int32_t)shared;  // a multiple of 16
        shared += (size_t)a.from.n * 4 + (size_t)a.from.T;
    }
    if (shared > 48 * 1024 - 1024) {
        static std::atomic<uint64_t> allowed{0};
        const cudaError_t e = allow_shared(reinterpret_cast<const void *>(kernel), kMostShared, di, allowed);
        if (e != cudaSuccess) return e;
    }
    return launch_dependent_smem(kernel, (int64_t)kSmCount * PER_SM, BLOCK, shared, st, a);
}
template <int TEAM, int NV, int BLOCK, int PER_SM, bool LIST>
cudaError_t whole_launch(int read, NormBwdArgs &a, const DeviceInfo &di, cudaStream_t st) {
    switch (read) {
        case kWords: return backward_launch<TEAM, NV, kWords, BLOCK, PER_SM, LIST>(a, di, st);
        case kMixed: return backward_launch<TEAM, NV, kMixed, BLOCK, PER_SM, LIST>(a, di, st);
        case kAligned:
            // (the one width whose rows are halved whenever they are read so)
            if constexpr (TEAM != 64 || NV != 4) return backward_launch<TEAM, NV, kAligned, BLOCK, PER_SM, LIST>(a, di, st);
            return cudaErrorInvalidValue;
        default: return backward_launch<TEAM, NV, kFloats, BLOCK, PER_SM, LIST>(a, di, st);
    }
}
template <int TEAM, int NV, int BLOCK, int PER_SM, bool LIST>
cudaError_t halved_launch(int read, NormBwdArgs &a, const DeviceInfo &di, cudaStream_t st) {
    if constexpr (TEAM == 128) {  // the one width that halves rows in bf16
        if (read == kWords) return backward_launch<TEAM, NV, kWords, BLOCK, PER_SM, LIST>(a, di, st);
        if (read == kMixed) return backward_launch<TEAM, NV, kMixed, BLOCK, PER_SM, LIST>(a, di, st);
    }
    return read == kAligned ? backward_launch<TEAM, NV, kAligned, BLOCK, PER_SM, LIST>(a, di, st)
                            : backward_launch<TEAM, NV, kFloats, BLOCK, PER_SM, LIST>(a, di, st);
}

// Whether a row of more than 1024 columns is kept by twice the threads, half the columns each.  2^27
// elements, halved against not:
//   up to 2048 columns, rows that are made of whole vectors: where r or dr is fp32 (all fp32 without dr, 1536
//   columns 248 us and 259, 1792 256 and 297), or where so many of the threads have work that it pays: in bf16
//   beyond 1792 columns (1536 with dr 194 and 184, 1792 173 and 170, 2048 161 and 182), with dout in fp32
//   beyond 1408 (1408 220 and 212, 1536 213 and 240).  Other rows are read twice in any case: with a wide dr
//   only (2047 columns, bf16 472 and 456, without dr 413 and 387, all fp32 without dr 499 and 472).
//   beyond: where r or dr is fp32 and there is a dr (all fp32, 4096 columns 315 and 417, 7168 335 and 385, 8192
//   325 and 409), but for 4097 to 6144 columns, where up to half of 512 threads would have none (5120 386 and 349;
//   6144 350 and 371, but 311 and 268 with r and dx in bf16).  Without dr there is a third less to wait for: r and
//   dx in fp32, 4096 columns 249 and 223, 8192 263 and 242 (all fp32 268 and 298, 286 and 278).
struct Kind {
    bool wide, dr, dout_wide;  // r or dr in fp32, dr given, dout in fp32
};
bool halved(int64_t H, const Kind &k) {
    if (H <= 1024) return false;
    if (H > 2048) return k.wide && k.dr && (H <= 4096 || H > 6144);
    if (H % 8 != 0) return k.wide && k.dr;
    return k.wide || H > (k.dout_wide ? 1408 : 1792);
}

// Widest row, and for rows as they are and halved ones team, vectors of 8 a thread, block and blocks per
// SM.  The blocks per SM are what leaves a team's sums in registers (but for 16 to 32 bytes a thread of bf16
// and mixed rows of four vectors): at 4096 columns of bf16 3, 4 and 5 blocks of 128 threads took 103, 96
// and 104 us for 16384 rows, before rows were asked for ahead.  Up to 1024 columns a thread has 16 (2^27
// elements of bf16 with dr, 1024 columns 163 us where 32 took 188).
#define RK_NORM_BWD_SHAPES(SHAPE)                  \
    SHAPE(64, 8, 1, 256, 3, 8, 1, 256, 3)          \
    SHAPE(128, 16, 1, 256, 3, 16, 1, 256, 3)       \
    SHAPE(256, 32, 1, 256, 3, 32, 1, 256, 3)       \
    SHAPE(512, 32, 2, 256, 2, 32, 2, 256, 2)       \
    SHAPE(1024, 64, 2, 64, 8, 64, 2, 64, 8)        \
    SHAPE(2048, 64, 4, 64, 8, 128, 2, 128, 4)      \
    SHAPE(4096, 128, 4, 128, 4, 256, 2, 256, 2)    \
    SHAPE(8192, 256, 4, 256, 2, 512, 2, 512, 1)    \
    SHAPE(16384, 512, 4, 512, 1, 512, 4, 512, 1)

// Blocks of the backward, and rows that a block takes at once.
struct Split {
    int blocks, rows;
};
Split split_of(int64_t H, bool half) {
#define SHAPE(MAX, TEAM, NV, BLOCK, PER, HTEAM, HNV, HBLOCK, HPER) \
    if (H <= MAX) return half ? Split{kSmCount * HPER, HBLOCK / HTEAM} : Split{kSmCount * PER, BLOCK / TEAM};
    RK_NORM_BWD_SHAPES(SHAPE)
#undef SHAPE
    return Split{0, 1};
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
    const int blocks = std::max(split_of(H, false).blocks, split_of(H, true).blocks);  // whatever the types
    b.partial = static_cast<float *>(take((size_t)blocks * (size_t)pitch_of(H) * 4));
    b.rows = static_cast<int32_t *>(take((size_t)n * 4));
    b.counts = static_cast<int32_t *>(take((size_t)(n / kListTile + 1) * 4));
    b.n_rows = static_cast<int64_t *>(take(8));
    b.listed = static_cast<uint8_t *>(take((size_t)T));
    return b;
}

}  // namespace

size_t rms_norm_bwd_workspace_bytes(int64_t T, int64_t n, int64_t H) { return carve(nullptr, T, n, H).bytes; }

cudaError_t launch_rms_norm_bwd(const RulesMatrix &dout, const RulesMatrix &r, const void *weight,
                                rk_dtype weight_type, float eps, const RulesMatrix *dr,
                                const int64_t *targets, const int32_t *cu, int num_seqs, int64_t T,
                                int64_t H, const int64_t *order, int64_t n, const RulesMatrix &dx,
                                float *dweight, bool accumulate, void *workspace, const DeviceInfo &di,
                                cudaStream_t st) {
    const BwdBuffers b = carve(workspace, T, n, H);
    NormBwdArgs a{matrix(&r), matrix(&dout), matrix(dr), weight, (int32_t)weight_type, eps, 1.f / (float)H, cu, num_seqs,
                  T, (int32_t)H, nullptr, nullptr, nullptr, matrix(&dx), 0, dweight ? b.partial : nullptr, Candidates{}, 0};
    a.stage_dx = !plain(a.dx, H);
    const Candidates c{order, n, T, targets, cu, num_seqs};
    const bool list = (targets || order) && n <= kListed && T <= kListed;
    if (list) {
        a.from = c;
        a.n_rows = b.n_rows;
    } else if (targets || order) {
        const int64_t tiles = std::max<int64_t>(1, (n + kListTile - 1) / kListTile);
        // one block does it all: a launch and a fill less (8192 rows of 1024: 26 us, 8200: 30)
        const bool one = tiles == 1 && T <= kListTile;
        cudaError_t e = one ? cudaSuccess : cudaMemsetAsync(b.listed, 0, (size_t)T, st);
        if (e == cudaSuccess && !one) e = launch_dependent(norm_rows_count, tiles, kListThreads, st, c, b.counts);
        if (e == cudaSuccess)
            e = launch_dependent(norm_rows_write, tiles, kListThreads, st, c, one ? (const int32_t *)nullptr : b.counts,
                                 b.rows, b.listed, b.n_rows);
        if (e != cudaSuccess) return e;
        a.rows = b.rows;
        a.n_rows = b.n_rows;
        a.listed = b.listed;
    }
    const bool on16 = plain(a.r, H) && plain(a.dout, H) && plain(a.dr, H) && aligned(weight, 16);
    const bool wide = a.r.type == RK_FP32 || (dr && a.dr.type == RK_FP32);
    const bool half = halved(H, Kind{wide, dr != nullptr, a.dout.type == RK_FP32});
    const int read = !on16 ? kFloats : wide ? kAligned : a.dout.type == RK_BF16 ? kWords : kMixed;
    const auto run = [&] {
#define SHAPE(MAX, TEAM, NV, BLOCK, PER, HTEAM, HNV, HBLOCK, HPER)                          \
    if (H <= MAX)                                                                           \
        return half   ? list ? halved_launch<HTEAM, HNV, HBLOCK, HPER, true>(read, a, di, st)  \
                             : halved_launch<HTEAM, HNV, HBLOCK, HPER, false>(read, a, di, st) \
               : list ? whole_launch<TEAM, NV, BLOCK, PER, true>(read, a, di, st)           \
                      : whole_launch<TEAM, NV, BLOCK, PER, false>(read, a, di, st);
        RK_NORM_BWD_SHAPES(SHAPE)
#undef SHAPE
        return cudaErrorInvalidValue;
    };
    const cudaError_t e = run();
    if (e != cudaSuccess || !dweight) return e;
    const Split split = split_of(H, half);
    return launch_dependent(rms_norm_join, (H + 31) / 32, 32 * kJoinLanes, st, (const float *)a.partial,
                            split.blocks, split.rows, (const int64_t *)a.n_rows, cu, num_seqs, T, (int)H, dweight,
                            (int)accumulate);
}

}  // namespace rk
