// adamw.cu -- one AdamW step over many tensors, with 32-bit states or states
// in 8 bits, and fp32 master weights beside bf16 parameters (what consumes
// the parameter gradients of issue #244, Workstream 3 #153: linear_logp_dw,
// embedding_bwd, rms_norm_bwd).
//
//   g = grad * grad_scale
//   m = beta1 m + (1 - beta1) g,   v = beta2 v + (1 - beta2) g^2
//   w = w - lr wd w - lr (m / (1 - beta1^step)) / (sqrt(v / (1 - beta2^step)) + eps)
//
// Bound by memory: 22 to 30 bytes an element with 32-bit states, 12 to 18 with
// 8-bit ones.  Every result depends on its own element (in 8 bits: on its block of 256
// elements) alone.  One launch takes up to kTensors tensors, described in the
// kernel's parameters (nothing to copy, nothing to keep alive for a graph);
// a block takes kChunk elements of one of them, a warp 256 at a time, a thread 8
// consecutive ones, so that a block of 8-bit states is a warp's.  525M elements with fp32
// gradients, masters and 32-bit states: 2237 us, 104 % of the copy rate; 545M with bf16
// gradients, masters and 8-bit states 1246 us, 103 %; 200 tensors of 150000 elements on average
// 83 us, 86 %, where one tensor of as many takes 76 and 200 of whole chunks 80: blocks look their tensor
// up, and 1.4 % of the chunks' room is empty.
//
// 8-bit states: m = e4m3 * scale, and for v its root, u = e4m3 * scale (e4m3
// spans 2^18, so v spans 2^36 within a block); scale = largest magnitude of
// the new block / 448.  A positive u takes the code 2^-9 at least: an element whose m
// is kept while its v is rounded away would be divided by eps alone.  Codes are those of
// the quotients where a block has an infinite value too: its scales are infinite, the other
// elements' codes 0 or 2^-9, and all of them NaN when they are read again.
#include <algorithm>
#include <cmath>

#include "elements.cuh"
#include "rk_device.cuh"
#include "rk_internal.h"

namespace rk {
namespace {

constexpr int kTensors = 256;    // of a launch
constexpr int kThreads = 256;
constexpr int kBlock = 256;      // elements that share a scale: a warp's, 8 a lane
constexpr int kChunk = 8 * kThreads * 2;  // elements of a block
// A block with 8-bit states asks for the chunk that comes this much later, into the second cache:
// 12 bytes an element and some 60 instructions do not keep enough loads in flight by themselves
// (64M elements 205 us without, 162 at 152 chunks, 164 at 304, 172 at 608, 232 at 1216; with 32-bit
// states 298 without, 353 with).
constexpr int kPrefetch = 152;

struct Tensor {
    void *param;
    float *master;
    const void *grad;
    void *m, *v;
    float *m_scale, *v_scale;
    int64_t n;
    float lr_scale, weight_decay;
    uint8_t param_wide, grad_wide, vec;
};

struct Table {
    int32_t first[kTensors + 1];  // chunks before each tensor
    int32_t count;
    float lr, rise, root;  // learning rate and the corrections of the host's step
    float beta1, rest1, log1, beta2, rest2, log2, eps;  // rest = 1 - beta, log = log(beta)
    float one;  // 1
    const float *lr_device;
    const int64_t *step_device;
    const float *grad_scale;
    unsigned *err;
    Tensor tensor[kTensors];
};
static_assert(sizeof(Table) <= 32764, "kernel parameters");

// ---- e4m3 ----

__device__ __forceinline__ void unpack_e4m3x8(uint2 w, float (&v)[8]) {
    const uint32_t q[2] = {w.x, w.y};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const uint16_t pair = (uint16_t)(q[i / 2] >> 16 * (i % 2));
        uint32_t h;
        asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"(pair));
        asm("{\n\t.reg .f16 a, b;\n\tmov.b32 {a, b}, %2;\n\tcvt.f32.f16 %0, a;\n\tcvt.f32.f16 %1, b;\n\t}"
            : "=f"(v[2 * i]), "=f"(v[2 * i + 1])
            : "r"(h));
    }
}

// The codes of a warp's block of values and, for its first lane to write, their scale.
template <bool FLOOR>
__device__ __forceinline__ uint2 encode(const float (&x)[8], float *scale) {
    float most = 0.f;  // fmaxf passes over NaN
#pragma unroll
    for (int i = 0; i < 8; ++i) most = fmaxf(most, fabsf(x[i]));
    const unsigned top = __reduce_max_sync(0xffffffffu, __float_as_uint(most));
    // 2^-120 at least, for a finite reciprocal
    const float s = top ? fmaxf(__fmul_rn(__uint_as_float(top), 1.f / 448.f), 0x1p-120f) : 0.f;
    *scale = s;
    float n[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) n[i] = x[i];
    Divisor(s).divide(n);
    if (FLOOR) {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (x[i] > 0.f) asm("max.NaN.f32 %0, %0, %1;" : "+f"(n[i]) : "f"(0x1p-9f));  // NaN stays NaN
    }
    return pack_e4m3x8(n);
}

// ---- 8 elements of a tensor ----

template <typename T>
__device__ __forceinline__ void get(const T *p, int64_t at, int left, bool vec, float (&v)[8]) {
    if (vec && left >= 8) {
        get8(p + at, v);
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = i < left ? get1(p + at + i) : 0.f;
    }
}
template <typename T>
__device__ __forceinline__ void put(T *p, int64_t at, int left, bool vec, const float (&v)[8]) {
    if (vec && left >= 8) {
        put8(p + at, v);
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (i < left) put1(p + at + i, v[i]);
    }
}
__device__ __forceinline__ uint2 get_codes(const void *p, int64_t at, int left, bool vec) {
    const uint8_t *q = static_cast<const uint8_t *>(p) + at;
    if (vec && left >= 8) return *reinterpret_cast<const uint2 *>(q);
    uint32_t w[2] = {0, 0};
#pragma unroll
    for (int i = 0; i < 8; ++i)
        if (i < left) w[i / 4] |= (uint32_t)q[i] << 8 * (i % 4);
    return make_uint2(w[0], w[1]);
}
__device__ __forceinline__ void put_codes(void *p, int64_t at, int left, bool vec, uint2 c) {
    uint8_t *q = static_cast<uint8_t *>(p) + at;
    if (vec && left >= 8) {
        *reinterpret_cast<uint2 *>(q) = c;
        return;
    }
#pragma unroll
    for (int i = 0; i < 8; ++i)
        if (i < left) q[i] = (uint8_t)((i < 4 ? c.x : c.y) >> 8 * (i % 4));
}

// ---- the step ----

// 1 - exp(x) for x <= 0, within two units in the last place and without a difference of numbers close to
// 1: x = k log 2 + r (Cody and Waite, 1980), e^r - 1 by its Taylor series up to r^7.  Every operation is
// one of IEEE 754, so that the host and the device get the same bits.
__host__ __device__ inline float one_minus_exp(float x) {
    x = fmaxf(x, -80.f);  // 1 from there on
    const float k = rintf(x * 1.44269504f);
    const float r = fmaf(k, -3.19461845e-5f, fmaf(k, -0.693115234375f, x));
    float p = fmaf(r, 1.f / 5040.f, 1.f / 720.f);
    p = fmaf(r, p, 1.f / 120.f);
    p = fmaf(r, p, 1.f / 24.f);
    p = fmaf(r, p, 1.f / 6.f);
    p = fmaf(r, p, 0.5f);
    const float power = ldexpf(1.f, (int)k);
    return fmaf(-power, fmaf(r * r, p, r), 1.f - power);
}

// What the moments' bias leaves of a step: 1 / (1 - beta1^step) and 1 / sqrt(1 - beta2^step), of log(beta).
struct Corrections {
    float rise, root;
    __host__ __device__ Corrections(int64_t step, float log1, float log2) {
        rise = 1.f / one_minus_exp((float)step * log1);
        root = 1.f / sqrtf(one_minus_exp((float)step * log2));
    }
};

struct Rates {
    float rate, root, decay, scale;  // lr / (1 - beta1^step), 1 / sqrt(1 - beta2^step), lr wd, grad_scale
};

// What a warp reads of 256 elements, 8 a lane, before it computes on them.
template <bool EIGHT>
struct States {
    float m[8], v[8];
    __device__ __forceinline__ void load(const Tensor &t, int64_t, int64_t at, int left) {
        get(static_cast<const float *>(t.m), at, left, t.vec, m);
        get(static_cast<const float *>(t.v), at, left, t.vec, v);
    }
};
template <>
struct States<true> {
    uint2 m, v;
    float ms, vs;
    __device__ __forceinline__ void load(const Tensor &t, int64_t block, int64_t at, int left) {
        m = get_codes(t.m, at, left, t.vec);
        v = get_codes(t.v, at, left, t.vec);
        ms = t.m_scale[block / kBlock];
        vs = t.v_scale[block / kBlock];
    }
};

template <bool EIGHT, typename G>
struct Elements {
    float g[8], w[8];
    States<EIGHT> s;
    int64_t at;
    int left;
    __device__ __forceinline__ void load(const Tensor &t, int64_t block) {
        at = block + 8 * (threadIdx.x & 31);
        left = (int)min((int64_t)8, max((int64_t)0, t.n - at));
        get(static_cast<const G *>(t.grad), at, left, t.vec, g);
        if (t.master)
            get(t.master, at, left, t.vec, w);
        else if (t.param_wide)
            get(static_cast<const float *>(t.param), at, left, t.vec, w);
        else
            get(static_cast<const uint16_t *>(t.param), at, left, t.vec, w);
        s.load(t, block, at, left);
    }
    __device__ __forceinline__ void update(const Table &a, const Tensor &t, const Rates &r, int64_t block) {
        float m[8], v[8];
        if constexpr (EIGHT) {
            unpack_e4m3x8(s.m, m);
            unpack_e4m3x8(s.v, v);
#pragma unroll
            for (int i = 0; i < 8; i += 2) {
                mul2(m[i], m[i + 1], s.ms, s.ms);
                mul2(v[i], v[i + 1], s.vs, s.vs);
                mul2(v[i], v[i + 1], v[i], v[i + 1]);
            }
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i) m[i] = s.m[i], v[i] = s.v[i];
        }
#pragma unroll
        for (int i = 0; i < 8; i += 2) {
            // Every product and sum of the states is rounded by itself: they are what elementary
            // fp32 operations give, and so are their codes.  (A packed product and the packed sum
            // that it goes into are compiled into one operation with one rounding; a product with a 1
            // that the compiler does not know keeps them apart.  In scalars 545M elements took 1252 us, so 1242.)
            float x0 = g[i], x1 = g[i + 1];
            mul2(x0, x1, r.scale, r.scale);
            float y0 = x0, y1 = x1;
            mul2(y0, y1, x0, x1);
            mul2(y0, y1, a.rest2, a.rest2);
            mul2(x0, x1, a.rest1, a.rest1);
            mul2(m[i], m[i + 1], a.beta1, a.beta1);
            mul2(v[i], v[i + 1], a.beta2, a.beta2);
            fma2(x0, x1, m[i], m[i + 1], a.one, a.one);
            fma2(y0, y1, v[i], v[i + 1], a.one, a.one);
            m[i] = x0, m[i + 1] = x1;
            v[i] = y0, v[i + 1] = y1;
            const float u0 = __fsqrt_rn(v[i]), u1 = __fsqrt_rn(v[i + 1]);
            float d0 = a.eps, d1 = a.eps, p0 = m[i], p1 = m[i + 1];
            fma2(d0, d1, u0, u1, r.root, r.root);
            mul2(p0, p1, r.rate, r.rate);
            fma2(w[i], w[i + 1], w[i], w[i + 1], -r.decay, -r.decay);
            // (the move's quotient within two units in its last place, of what is a correction to w; d0 stays
            // far below 2^126, where this one ends)
            w[i] = __fsub_rn(w[i], __fdividef(p0, d0));
            w[i + 1] = __fsub_rn(w[i + 1], __fdividef(p1, d1));
            if (EIGHT) v[i] = u0, v[i + 1] = u1;
        }
        if (t.master) put(t.master, at, left, t.vec, w);
        if (t.param_wide)
            put(static_cast<float *>(t.param), at, left, t.vec, w);
        else
            put(static_cast<uint16_t *>(t.param), at, left, t.vec, w);
        if constexpr (EIGHT) {
            float ms, vs;
            const uint2 mc = encode<false>(m, &ms), vc = encode<true>(v, &vs);
            put_codes(t.m, at, left, t.vec, mc);
            put_codes(t.v, at, left, t.vec, vc);
            if ((threadIdx.x & 31) == 0) {
                t.m_scale[block / kBlock] = ms;
                t.v_scale[block / kBlock] = vs;
            }
        } else {
            put(static_cast<float *>(t.m), at, left, t.vec, m);
            put(static_cast<float *>(t.v), at, left, t.vec, v);
        }
    }
};

template <bool EIGHT, typename G>
__device__ __forceinline__ void chunk_step(const Table &a, const Tensor &t, const Rates &r, int64_t chunk) {
#pragma unroll 1
    for (int64_t block = chunk + (threadIdx.x >> 5) * kBlock; block < min(t.n, chunk + kChunk);
         block += kThreads / 32 * kBlock) {
        Elements<EIGHT, G> e;
        e.load(t, block);
        e.update(a, t, r, block);
    }
}

// The tensor that a chunk belongs to.
__device__ __forceinline__ int tensor_of(const Table &a, int chunk) {
    int lo = 0, hi = a.count;
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (a.first[mid] <= chunk)
            lo = mid;
        else
            hi = mid;
    }
    return lo;
}

// By four threads: a chunk's gradient, weights and states, into the second cache.
__device__ __forceinline__ void prefetch(const Table &a, int chunk) {
    const int k = tensor_of(a, chunk);
    const Tensor &t = a.tensor[k];
    const int64_t from = (int64_t)(chunk - a.first[k]) * kChunk, n = min((int64_t)kChunk, t.n - from);
    const int weight = t.master || t.param_wide ? 4 : 2, grad = t.grad_wide ? 4 : 2;
    const void *p = threadIdx.x == 0 ? t.grad : threadIdx.x == 1 ? t.m : threadIdx.x == 2 ? t.v : t.master ? t.master : t.param;
    const int size = threadIdx.x == 0 ? grad : threadIdx.x < 3 ? 1 : weight;
    const char *q = static_cast<const char *>(p) + from * size;
    const uint32_t bytes = (uint32_t)(n * size) & ~15u;
    if (bytes && (reinterpret_cast<uintptr_t>(q) & 15) == 0)
        asm volatile("cp.async.bulk.prefetch.L2.global [%0], %1;" ::"l"(q), "r"(bytes) : "memory");
}

template <bool EIGHT>
__global__ void __launch_bounds__(kThreads, 4) adamw_kernel(const __grid_constant__ Table a) {
    wait_prior_grid();
    const int lo = tensor_of(a, (int)blockIdx.x);
    const Tensor &t = a.tensor[lo];
    float rise = a.rise, root = a.root;
    if (a.step_device) {
        const int64_t step = *a.step_device;
        if (step < 1) {
            if (threadIdx.x == 0) atomicOr(a.err, kErrRules);
            return;
        }
        const Corrections c(step, a.log1, a.log2);
        rise = c.rise;
        root = c.root;
    }
    const float lr = __fmul_rn(a.lr_device ? *a.lr_device : a.lr, t.lr_scale);
    const Rates r{__fmul_rn(lr, rise), root, __fmul_rn(lr, t.weight_decay), a.grad_scale ? *a.grad_scale : 1.f};
    const int64_t chunk = (int64_t)((int)blockIdx.x - a.first[lo]) * kChunk;
    if (EIGHT && threadIdx.x < 4 && (int)blockIdx.x < a.first[a.count] - kPrefetch) prefetch(a, (int)blockIdx.x + kPrefetch);
    if (t.grad_wide)
        chunk_step<EIGHT, float>(a, t, r, chunk);
    else
        chunk_step<EIGHT, uint16_t>(a, t, r, chunk);
}

}  // namespace

cudaError_t launch_adamw(const rk_adamw_tensor *tensors, int64_t count, const rk_adamw_options &o,
                         const DeviceInfo &di, cudaStream_t st) {
    Table a;
    a.lr = (float)o.lr;
    a.beta1 = (float)o.beta1;
    a.rest1 = (float)(1.0 - o.beta1);
    a.log1 = (float)std::log(o.beta1);
    a.beta2 = (float)o.beta2;
    a.rest2 = (float)(1.0 - o.beta2);
    a.log2 = (float)std::log(o.beta2);
    const Corrections c(o.step_device ? 1 : o.step, a.log1, a.log2);
    a.rise = c.rise;
    a.root = c.root;
    a.eps = (float)o.eps;
    a.one = 1.f;
    a.lr_device = o.lr_device;
    a.step_device = o.step_device;
    a.grad_scale = o.grad_scale;
    a.err = di.err;
    for (int64_t i = 0; i < count;) {
        // as many tensors with the same kind of states as fit
        const bool eight = tensors[i].m_scale != nullptr;
        a.count = 0;
        int64_t chunks = 0;
        for (; i < count && a.count < kTensors; ++i) {
            const rk_adamw_tensor &s = tensors[i];
            if (s.n == 0) continue;
            if ((s.m_scale != nullptr) != eight) break;
            const int64_t more = (s.n + kChunk - 1) / kChunk;
            if (chunks + more > 0x7fffffff) break;
            Tensor &t = a.tensor[a.count];
            t.param = s.param;
            t.master = s.master;
            t.grad = s.grad;
            t.m = s.m;
            t.v = s.v;
            t.m_scale = s.m_scale;
            t.v_scale = s.v_scale;
            t.n = s.n;
            t.lr_scale = s.lr_scale;
            t.weight_decay = s.weight_decay;
            t.param_wide = s.param_type == RK_FP32;
            t.grad_wide = s.grad_type == RK_FP32;
            const uintptr_t state = s.m_scale ? 8 : 16;
            t.vec = aligned(s.param, 16) && aligned(s.grad, 16) && aligned(s.master, 16) && aligned(s.m, state) &&
                    aligned(s.v, state);
            a.first[a.count++] = (int32_t)chunks;
            chunks += more;
        }
        if (a.count == 0) continue;  // empty ones, or one of the other kind next
        a.first[a.count] = (int32_t)chunks;
        const cudaError_t e = launch_dependent(eight ? adamw_kernel<true> : adamw_kernel<false>, chunks, kThreads, st, a);
        if (e != cudaSuccess) return e;
    }
    return cudaSuccess;
}

}  // namespace rk
