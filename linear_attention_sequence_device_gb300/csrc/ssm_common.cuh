// Device pieces shared by the selective scan layer's kernels and the block norm.
#pragma once

#include "gdn_internal.cuh"

namespace gdn {

constexpr float kLog2e = 1.4426950408889634f;

// The most tokens of a call.  Rows are counted in 32 bits, and a strip's, a segment's
// or a grid's step beyond the last row stays below 2^31 with this much to spare (strips:
// 65535 of them, each rounded up to four rows).
constexpr int kMaxTokens = 0x7fffffff - (1 << 20);

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

// one element by a load that stays where it is written: the compiler would move
// an ordinary load down to its first use, a whole tile later
__device__ __forceinline__ __nv_bfloat16 load_now(const __nv_bfloat16* p) {
    unsigned short r;
    asm volatile("ld.global.nc.u16 %0, [%1];" : "=h"(r) : "l"(p));
    return __ushort_as_bfloat16(r);
}
__device__ __forceinline__ float load_now(const float* p) {
    float r;
    asm volatile("ld.global.nc.f32 %0, [%1];" : "=f"(r) : "l"(p));
    return r;
}

// 2^v by the special function unit (relative error 2^-22; -inf gives 0)
__device__ __forceinline__ float exp2_fast(float v) {
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(v));
    return r;
}
// 1 / (1 + e^-v): an infinite e^-v gives 0, a NaN goes through
__device__ __forceinline__ float rcp_fast(float v) {
    float r;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(v));
    return r;
}
__device__ __forceinline__ float sigmoid_fast(float v) { return rcp_fast(1.f + exp2_fast(-kLog2e * v)); }
__device__ __forceinline__ float silu_fast(float v) { return v * sigmoid_fast(v); }
// e^-|v| = t (1 + c).  The exponent h = |v| log2 e is off by half a step of its own size,
// which alone would put t, and with it a delta of 1e-3 (|v| = 7), off by 15 of its half
// steps; what the rounded h has too much comes back as a factor.  h is rounded up, so
// that c = h ln 2 - |v| lies in [0, |v| 2^-22]: the clamp to [0, 1] then costs nothing and
// takes the NaN of an infinite v, whose t is 0.  Measured: delta within 15 half steps, 30
// without (32768 x 4096: 893 -> 907 us).
__device__ __forceinline__ void exp_neg_abs_parts(float v, float& t, float& c) {
    const float h = __fmul_ru(fabsf(v), 1.44269514083862305f);  // the fp32 value above log2 e
    t = exp2_fast(-h);
    c = __saturatef(fmaf(h, 0.693147182464599609f, -fabsf(v)));
}
__device__ __forceinline__ float exp_neg_abs(float v) {
    float t, c;
    exp_neg_abs_parts(v, t, c);
    return fmaf(t, c, t);
}
// log(1 + e^v) = max(v, 0) + log(1 + t), t = e^-|v| in (0, 1]: the first term is
// all of it above 20, the gates' threshold.  log(1 + t) is t times a polynomial
// of degree 9 interpolated at the Chebyshev points of [0, 1] (relative error
// 5e-9, with fp32 coefficients and steps 1.6e-7), so that delta keeps its digits
// where it is small, which the hardware logarithm of 1 + t would not.
__device__ __forceinline__ float softplus_f(float v) {
    const float t = exp_neg_abs(v);
    float q = -0.0031760570127516985f;
    q = fmaf(q, t, 0.019542526453733444f);
    q = fmaf(q, t, -0.056373611092567444f);
    q = fmaf(q, t, 0.10543623566627502f);
    q = fmaf(q, t, -0.1526966691017151f);
    q = fmaf(q, t, 0.1966327428817749f);
    q = fmaf(q, t, -0.24951615929603577f);
    q = fmaf(q, t, 0.33329710364341736f);
    q = fmaf(q, t, -0.49999892711639404f);
    q = fmaf(q, t, 1.f);
    float m;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(m) : "f"(v), "f"(0.f));
    return fmaf(t, q, m);
}
// The decay 2^(d A2) of a step.  The special function unit's results lie below the
// value on average, by 0.6e-8 to 3.5e-8 with the argument's place in cells of 1/64
// (half a step is 3e-8 there), and a state multiplied a thousand times by the decay
// of its channel, whose arguments stay in a few cells, adds that up.  Two remedies
// that cost no operation per state:
//  - a constant in the argument, inside the product;
//  - shifts: tokens go in pairs, of which the first takes its decays 2^s too large
//    and the second 2^s too small, so that the state is 2^s times its value between
//    the two.  What enters and leaves there is scaled by 2^s per token, not per state.
//    Eight pairs' shifts spread the arguments over sixteen places in eight cells, on
//    average over which the error is between -0.8e-8 (arguments near 0) and -2.8e-8
//    (near -0.07); the constant takes back 1.1e-8.
// Measured on sequences of 8 to 1200 tokens with carried states (4096 channels of 16
// states, segments of 256 tokens), error in norm and of that in one direction: final
// states 3.4e-7 and -0.2e-7, A_log's gradient 5.2e-7 and -0.5e-7; without the constant
// 7.9e-7 and -4.8e-7, 15e-7 and -11e-7; without the shifts 6.0e-7 and -2.3e-7, 13e-7 and
// -8e-7; with a constant of 1.3e-8 3.3e-7 and -1.0e-7, 5.6e-7 and -2.6e-7, of 2.0e-8
// 4.5e-7 and 1.1e-7, 7.1e-7 and 2.4e-7.
constexpr float kDecayBias = 1.6e-8f;
constexpr int kShifts = 8;
__constant__ const float kShift[kShifts] = {0.00439453125f, 0.0131835938f, 0.0219726562f, 0.0307617188f, 0.0395507812f, 0.0483398438f, 0.0571289062f, 0.0659179688f};
__constant__ const float kShiftUp[kShifts] = {1.00305068f, 1.00918007f, 1.01534688f, 1.02155137f, 1.02779377f, 1.03407431f, 1.04039323f, 1.04675078f};  // 2^s
__constant__ const float kShiftDown[kShifts] = {0.996958554f, 0.990903437f, 0.984885097f, 0.978903294f, 0.97295785f, 0.967048526f, 0.961175025f, 0.955337226f};  // 2^-s

// Gradients that are sums over all tokens are added one by one within a block, in fp32,
// and the blocks' partial sums behind it; terms that are alike then put the sum off by up
// to half a step for every two of a block's.  So a block has this many tokens at most:
// above, `wave` blocks side by side become whole multiples of that many.
constexpr int kLongestSum = 1024;
inline int64_t blocks_for_sum(int64_t tokens, int64_t wave) {
    const int64_t least = (tokens + kLongestSum - 1) / kLongestSum;
    return wave >= least ? wave : (least + wave - 1) / wave * wave;
}

// Two fp32 values in a register pair, for the two-wide instructions: the pipe's
// rate is the same, the instructions are half.  Kept as 64 bits, so that the pair
// is not taken apart and put together again between operations.
struct F2 {
    unsigned long long b;
    __device__ __forceinline__ float x() const { return __uint_as_float((unsigned)b); }
    __device__ __forceinline__ float y() const { return __uint_as_float((unsigned)(b >> 32)); }
};
__device__ __forceinline__ F2 f2(float x, float y) {
    F2 r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r.b) : "f"(x), "f"(y));
    return r;
}
__device__ __forceinline__ F2 f2_fma(F2 a, F2 b, F2 c) {
    F2 r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r.b) : "l"(a.b), "l"(b.b), "l"(c.b));
    return r;
}
__device__ __forceinline__ F2 f2_mul(F2 a, F2 b) {
    F2 r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r.b) : "l"(a.b), "l"(b.b));
    return r;
}
__device__ __forceinline__ F2 f2_exp2(F2 a) {
    F2 r;
    asm("{\n\t.reg .f32 lo, hi;\n\tmov.b64 {lo, hi}, %1;\n\tex2.approx.ftz.f32 lo, lo;\n\tex2.approx.ftz.f32 hi, hi;\n\t"
        "mov.b64 %0, {lo, hi};\n\t}"
        : "=l"(r.b)
        : "l"(a.b));
    return r;
}
__device__ __forceinline__ F2 f2_dup(float v) { return f2(v, v); }
__device__ __forceinline__ F2 f2_decay(F2 d, F2 A2, F2 bias) { return f2_exp2(f2_fma(d, A2, bias)); }
__device__ __forceinline__ float f2_sum(F2 a) { return a.x() + a.y(); }
__device__ __forceinline__ F2 f2_add(F2 a, F2 b) {
    F2 r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r.b) : "l"(a.b), "l"(b.b));
    return r;
}
__device__ __forceinline__ F2 f2_sigmoid(F2 v) {
    const F2 e = f2_add(f2_exp2(f2_mul(v, f2_dup(-kLog2e))), f2_dup(1.f));
    return f2(rcp_fast(e.x()), rcp_fast(e.y()));
}
__device__ __forceinline__ F2 f2_silu(F2 v) { return f2_mul(v, f2_sigmoid(v)); }
__device__ __forceinline__ F2 f2_max0(F2 v) {
    float x, y;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(x) : "f"(v.x()), "f"(0.f));
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(y) : "f"(v.y()), "f"(0.f));
    return f2(x, y);
}
// softplus_f of pairs, step by step together: a coefficient is made once for all; t: their e^-|v|
template <int M>
__device__ __forceinline__ void f2_softplus(F2 (&v)[M], F2 (&t)[M]) {
    constexpr float c[9] = {0.019542526453733444f, -0.056373611092567444f, 0.10543623566627502f, -0.1526966691017151f,
                            0.1966327428817749f, -0.24951615929603577f, 0.33329710364341736f, -0.49999892711639404f, 1.f};
    F2 q[M];
#pragma unroll
    for (int i = 0; i < M; ++i) {
        float tx, ty, cx, cy;
        exp_neg_abs_parts(v[i].x(), tx, cx);
        exp_neg_abs_parts(v[i].y(), ty, cy);
        t[i] = f2(tx, ty);
        t[i] = f2_fma(t[i], f2(cx, cy), t[i]);
        q[i] = f2_dup(-0.0031760570127516985f);
    }
#pragma unroll
    for (int k = 0; k < 9; ++k) {
        const F2 ck = f2_dup(c[k]);
#pragma unroll
        for (int i = 0; i < M; ++i) q[i] = f2_fma(q[i], t[i], ck);
    }
#pragma unroll
    for (int i = 0; i < M; ++i) v[i] = f2_fma(t[i], q[i], f2_max0(v[i]));
}
// eight consecutive elements (16-byte aligned) as four pairs
__device__ __forceinline__ void f2_load8(const __nv_bfloat16* p, F2 (&f)[4]) {
    const uint4 r = *reinterpret_cast<const uint4*>(p);
    const unsigned w[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) f[i] = f2(__uint_as_float(w[i] << 16), __uint_as_float(w[i] & 0xffff0000u));
}
__device__ __forceinline__ void f2_load8(const float* p, F2 (&f)[4]) {
    const ulonglong2 a = reinterpret_cast<const ulonglong2*>(p)[0], b = reinterpret_cast<const ulonglong2*>(p)[1];
    f[0].b = a.x; f[1].b = a.y; f[2].b = b.x; f[3].b = b.y;
}
__device__ __forceinline__ void f2_store8(__nv_bfloat16* p, const F2 (&f)[4]) {
    uint4 raw;
    __nv_bfloat162* h = reinterpret_cast<__nv_bfloat162*>(&raw);
#pragma unroll
    for (int i = 0; i < 4; ++i) h[i] = __floats2bfloat162_rn(f[i].x(), f[i].y());
    *reinterpret_cast<uint4*>(p) = raw;
}
__device__ __forceinline__ void f2_store8(float* p, const F2 (&f)[4]) {
    reinterpret_cast<ulonglong2*>(p)[0] = make_ulonglong2(f[0].b, f[1].b);
    reinterpret_cast<ulonglong2*>(p)[1] = make_ulonglong2(f[2].b, f[3].b);
}
// two pairs from shared memory
__device__ __forceinline__ void f2_load2(const float* p, F2& a, F2& b) {
    const ulonglong2 v = *reinterpret_cast<const ulonglong2*>(p);
    a.b = v.x;
    b.b = v.y;
}
__device__ __forceinline__ void f2_store2(void* p, F2 a, F2 b) {
    *reinterpret_cast<ulonglong2*>(p) = make_ulonglong2(a.b, b.b);
}

// the sequence that holds packed token t: the last n with cu[n] <= t, which is
// not empty; clamped to a sequence for a malformed cu
__device__ __forceinline__ int seq_of(const int32_t* cu, int num_seqs, int t) {
    const int n = upper_bound_minus1(cu, num_seqs, t);
    return n < num_seqs ? n : num_seqs - 1;
}

}  // namespace gdn
