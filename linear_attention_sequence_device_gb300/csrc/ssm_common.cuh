// Device pieces shared by the selective scan layer's kernels and the block norm.
#pragma once

#include "gdn_internal.cuh"

namespace gdn {

constexpr float kLog2e = 1.4426950408889634f;

// eight consecutive elements (16-byte aligned) <-> fp32
__device__ __forceinline__ void load8(const __nv_bfloat16* p, float (&f)[8]) {
    const uint4 raw = __ldg(reinterpret_cast<const uint4*>(p));
    const __nv_bfloat162* h = reinterpret_cast<const __nv_bfloat162*>(&raw);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float2 t = __bfloat1622float2(h[i]);
        f[2 * i] = t.x;
        f[2 * i + 1] = t.y;
    }
}
__device__ __forceinline__ void load8(const float* p, float (&f)[8]) {
    const float4 a = __ldg(reinterpret_cast<const float4*>(p)), b = __ldg(reinterpret_cast<const float4*>(p) + 1);
    f[0] = a.x; f[1] = a.y; f[2] = a.z; f[3] = a.w;
    f[4] = b.x; f[5] = b.y; f[6] = b.z; f[7] = b.w;
}
__device__ __forceinline__ void store8(__nv_bfloat16* p, const float (&f)[8]) {
    uint4 raw;
    __nv_bfloat162* h = reinterpret_cast<__nv_bfloat162*>(&raw);
#pragma unroll
    for (int i = 0; i < 4; ++i) h[i] = __floats2bfloat162_rn(f[2 * i], f[2 * i + 1]);
    *reinterpret_cast<uint4*>(p) = raw;
}
__device__ __forceinline__ void store8(float* p, const float (&f)[8]) {
    reinterpret_cast<float4*>(p)[0] = make_float4(f[0], f[1], f[2], f[3]);
    reinterpret_cast<float4*>(p)[1] = make_float4(f[4], f[5], f[6], f[7]);
}

// the same by ordinary loads, for arrays that the kernel may write in place
__device__ __forceinline__ void load8_rw(const __nv_bfloat16* p, float (&f)[8]) {
    const uint4 raw = *reinterpret_cast<const uint4*>(p);
    const __nv_bfloat162* h = reinterpret_cast<const __nv_bfloat162*>(&raw);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float2 t = __bfloat1622float2(h[i]);
        f[2 * i] = t.x;
        f[2 * i + 1] = t.y;
    }
}
__device__ __forceinline__ void load8_rw(const float* p, float (&f)[8]) {
    const float4 a = reinterpret_cast<const float4*>(p)[0], b = reinterpret_cast<const float4*>(p)[1];
    f[0] = a.x; f[1] = a.y; f[2] = a.z; f[3] = a.w;
    f[4] = b.x; f[5] = b.y; f[6] = b.z; f[7] = b.w;
}

// 2^v by the special function unit (relative error 2^-22; -inf gives 0)
__device__ __forceinline__ float exp2_fast(float v) {
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(v));
    return r;
}
// 1 / (1 + e^-v): an infinite e^-v gives 0
__device__ __forceinline__ float sigmoid_fast(float v) {
    return __fdividef(1.f, 1.f + exp2_fast(fminf(-kLog2e * v, 126.f)));
}
__device__ __forceinline__ float silu_fast(float v) { return v * sigmoid_fast(v); }
// log(1 + e^v), v above 20 (the gates' threshold).  The full-precision
// functions: delta enters every state's decay, and the hardware logarithm of
// 1 + e^v would leave it 20 bits where delta is small.
__device__ __forceinline__ float softplus_f(float v) { return v > 20.f ? v : log1pf(expf(v)); }

// the sequence that holds packed token t: the last n with cu[n] <= t, which is
// not empty; clamped to a sequence for a malformed cu
__device__ __forceinline__ int seq_of(const int32_t* cu, int num_seqs, int t) {
    const int n = upper_bound_minus1(cu, num_seqs, t);
    return n < num_seqs ? n : num_seqs - 1;
}

}  // namespace gdn
