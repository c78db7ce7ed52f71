// elements.cuh -- elements of bf16 and fp32 matrices as floats, eight at a time
// or one by one, and launches that overlap the end of the kernel before them;
// shared by the memory-bound kernels (embedding.cu, rms_norm.cuh, adamw.cu,
// preference.cu).
#pragma once

#include "rk_device.cuh"

namespace rk {

__device__ __forceinline__ void wait_prior_grid() {
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
}

// Launch with programmatic stream serialisation: the kernel's blocks may
// become resident while the previous kernel of the stream ends; each waits
// (wait_prior_grid) before it reads or writes anything.
template <typename... P, typename... A>
cudaError_t launch_dependent_smem(void (*kernel)(P...), int64_t grid, int block, size_t smem,
                                  cudaStream_t st, A... args) {
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3((unsigned)grid);
    cfg.blockDim = dim3((unsigned)block);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, args...);
}

template <typename... P, typename... A>
cudaError_t launch_dependent(void (*kernel)(P...), int64_t grid, int block, cudaStream_t st,
                             A... args) {
    return launch_dependent_smem(kernel, grid, block, 0, st, args...);
}

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

// Two products, sums or fused sums of fp32 at once, each rounded as the single operation.
__device__ __forceinline__ void mul2(float &x0, float &x1, float y0, float y1) {
    asm("{\n\t.reg .b64 a, b;\n\tmov.b64 a, {%0, %1};\n\tmov.b64 b, {%2, %3};\n\t"
        "mul.rn.f32x2 a, a, b;\n\tmov.b64 {%0, %1}, a;\n\t}"
        : "+f"(x0), "+f"(x1)
        : "f"(y0), "f"(y1));
}
// A product of mul2 that goes into add2 is compiled into one fma2, with one rounding.
__device__ __forceinline__ void add2(float &x0, float &x1, float y0, float y1) {
    asm("{\n\t.reg .b64 a, b;\n\tmov.b64 a, {%0, %1};\n\tmov.b64 b, {%2, %3};\n\t"
        "add.rn.f32x2 a, a, b;\n\tmov.b64 {%0, %1}, a;\n\t}"
        : "+f"(x0), "+f"(x1)
        : "f"(y0), "f"(y1));
}
// z = x y + z
__device__ __forceinline__ void fma2(float &z0, float &z1, float x0, float x1, float y0, float y1) {
    asm("{\n\t.reg .b64 a, b, c;\n\tmov.b64 a, {%2, %3};\n\tmov.b64 b, {%4, %5};\n\tmov.b64 c, {%0, %1};\n\t"
        "fma.rn.f32x2 c, a, b, c;\n\tmov.b64 {%0, %1}, c;\n\t}"
        : "+f"(z0), "+f"(z1)
        : "f"(x0), "f"(x1), "f"(y0), "f"(y1));
}
// Two bf16 sums, each rounded once.
__device__ __forceinline__ uint32_t add_bf16x2(uint32_t a, uint32_t b) {
    uint32_t d;
    asm("add.rn.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
    return d;
}

// Two floats -> packed e4m3x2 (round to nearest even, saturating at 448; NaN
// stays NaN); `lo` in bits 0-7.
__device__ __forceinline__ uint32_t pack_e4m3x2(float lo, float hi) {
    uint16_t d;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(d) : "f"(hi), "f"(lo));
    return d;
}
// x / s, each correctly rounded (Markstein, 1990: a faithful quotient and its remainder times the
// rounded reciprocal), so that a code next to a border is that of the quotient.  s is 2^-120 at least and
// |x| at most 448 s; an infinite s leaves 0 of a finite x and NaN of an infinite one, and so does a 0
// (where x is 0 or NaN).
struct Divisor {
    float s, inverse;
    __device__ __forceinline__ explicit Divisor(float scale) {
        s = scale;
        inverse = __frcp_rn(scale);
    }
    __device__ __forceinline__ void divide(float (&x)[8]) const {
        if (s >= 0x1p-60f && s < INFINITY) {
            quotients(x, -s, inverse);
            return;
        }
        // below 2^-60 both are moved up, by a power of two: the remainder would leave the normal numbers
        const bool some = s > 0.f && s < INFINITY;
#pragma unroll
        for (int i = 0; i < 8; ++i) x[i] *= some ? 0x1p64f : 0.f;
        if (some) quotients(x, s * -0x1p64f, __frcp_rn(s * 0x1p64f));
    }

private:
    static __device__ __forceinline__ void quotients(float (&x)[8], float minus, float inverse) {
#pragma unroll
        for (int i = 0; i < 8; i += 2) {
            float n0 = x[i], n1 = x[i + 1];
            mul2(n0, n1, inverse, inverse);
            fma2(x[i], x[i + 1], n0, n1, minus, minus);
            fma2(n0, n1, x[i], x[i + 1], inverse, inverse);
            x[i] = n0;
            x[i + 1] = n1;
        }
    }
};

__device__ __forceinline__ uint2 pack_e4m3x8(const float (&v)[8]) {
    return make_uint2(pack_e4m3x2(v[0], v[1]) | pack_e4m3x2(v[2], v[3]) << 16,
                      pack_e4m3x2(v[4], v[5]) | pack_e4m3x2(v[6], v[7]) << 16);
}

}  // namespace rk
