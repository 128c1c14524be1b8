// Epilogue of the linear layers: out = residual + act(c + bias), from the fp32
// accumulator c, rounded once to the output's type.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "kq_device.cuh"
#include "kq.h"

namespace kq {

__device__ __forceinline__ float ex2_approx(float x)
{
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// x * sigmoid(t ln 2) = x / (1 + 2^-t).  Where 2^-t overflows the quotient is
// zero, its limit; x = -inf gives NaN, as the formula read literally does.
__device__ __forceinline__ float times_sigmoid2(float x, float t)
{
    return __fdividef(x, 1.0f + ex2_approx(-t));
}

constexpr float kLog2e = 1.4426950408889634f;

// x (1 + erf(x / sqrt 2)) / 2 = max(x, 0) - |x| q / 2 with q = erfc(|x| / sqrt 2), by
// the rational approximation 7.1.26 of Abramowitz and Stegun, Handbook of
// Mathematical Functions: erfc(a) = (a1 t + ... + a5 t^5) exp(-a^2), t = 1 / (1 + p a),
// within 1.5e-7.  (erff took 1.3 times as long in the epilogue of short products.)
// |x| is capped where q is zero, so that an infinity does not meet it.
__device__ __forceinline__ float act_gelu(float x)
{
    const float a = fabsf(x) * 0.70710678118654752f;
    const float t = __fdividef(1.0f, fmaf(0.3275911f, a, 1.0f));
    float q = fmaf(1.061405429f, t, -1.453152027f);
    q = fmaf(q, t, 1.421413741f);
    q = fmaf(q, t, -0.284496736f);
    q = fmaf(q, t, 0.254829592f);
    q = q * t * ex2_approx(a * a * -kLog2e);
    return fmaf(-0.5f * fminf(fabsf(x), 64.0f), q, fmaxf(x, 0.0f));
}
__device__ __forceinline__ float act_gelu_tanh(float x)
{
    // 0.5 x (1 + tanh u) = x sigmoid(2 u), u = sqrt(2 / pi) (x + 0.044715 x^3)
    constexpr float a = 2.0f * 0.79788456080286536f * kLog2e;
    return times_sigmoid2(x, x * fmaf(a * 0.044715f, x * x, a));
}
__device__ __forceinline__ float act_silu(float x) { return times_sigmoid2(x, x * kLog2e); }

template <int N>
__device__ __forceinline__ void apply_act(float (&v)[N], int act)
{
    if (act == KQ_ACT_GELU) {
#pragma unroll
        for (int i = 0; i < N; ++i) v[i] = act_gelu(v[i]);
    } else if (act == KQ_ACT_GELU_TANH) {
#pragma unroll
        for (int i = 0; i < N; ++i) v[i] = act_gelu_tanh(v[i]);
    } else if (act == KQ_ACT_SILU) {
#pragma unroll
        for (int i = 0; i < N; ++i) v[i] = act_silu(v[i]);
    }
}

__device__ __forceinline__ uint32_t pack16(float lo, float hi, bool f16)
{
    if (f16) {
        const __half2 p = __floats2half2_rn(lo, hi);
        return *reinterpret_cast<const uint32_t *>(&p);
    }
    const __nv_bfloat162 p = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t *>(&p);
}

__device__ __forceinline__ float2 unpack16(uint32_t w, bool f16)
{
    return f16 ? make_float2(f16_lo(w), f16_hi(w)) : make_float2(bf16_lo(w), bf16_hi(w));
}

// One element of the residual (fmt) at element offset i; a plain load: the
// residual may be the output itself, read before it is written.
__device__ __forceinline__ float load_residual(const void *p, int64_t i, int fmt)
{
    if (fmt == KQ_F32) return *(static_cast<const volatile float *>(p) + i);
    const uint32_t w = *(static_cast<const volatile uint16_t *>(p) + i);
    return fmt == KQ_F16 ? f16_lo(w) : bf16_lo(w);
}

__device__ __forceinline__ void store_out(void *p, int64_t i, int fmt, float v)
{
    if (fmt == KQ_F32)
        static_cast<float *>(p)[i] = v;
    else
        static_cast<uint16_t *>(p)[i] = static_cast<uint16_t>(pack16(v, 0.f, fmt == KQ_F16));
}

}  // namespace kq
