// Packed fp32 arithmetic of sm_100: two values in one register pair.  A packed
// instruction takes the pipe as long as two scalar ones but one issue slot.
// And the SFU's reciprocal and SiLU without the range handling of the
// compiler's own forms, which costs more instructions than they do.
#pragma once

#include <cuda_runtime.h>

namespace la {
namespace sm100 {

typedef unsigned long long f2;
__device__ __forceinline__ f2 pack2(float a, float b)
{
    f2 r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
    return r;
}
__device__ __forceinline__ float2 unpack2(f2 v)
{
    float2 r;
    asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(v));
    return r;
}
__device__ __forceinline__ f2 mul2(f2 a, f2 b)
{
    f2 r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ f2 fma2(f2 a, f2 b, f2 c)
{
    f2 r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}
__device__ __forceinline__ f2 add2(f2 a, f2 b)
{
    f2 r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}

// 1 / x for x in [1, inf] (1 / inf = 0): one SFU instruction, relative error 2^-23
__device__ __forceinline__ float rcp_approx(float x)
{
    float r;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}

// y / (1 + e^-y), with e^-y as 2^(-y log2 e) flushed to zero where it is subnormal
__device__ __forceinline__ float silu_approx(float y)
{
    float e;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"(y * -1.4426950408889634f));
    return y * rcp_approx(1.f + e);
}

// y / (1 + e^-y) within about five steps of fp32 and without branches: with h =
// e^-|y| <= 1 it is y r or y h r, r = 1 / (1 + h).  The rounding of |y| log2 e is
// put back to first order, r gets a Newton step.  (A library exponential and
// division here took a third of the state-space scan's time in fp32.)
__device__ __forceinline__ float silu_f32(float y)
{
    constexpr float kLog2e = 1.4426950408889634f, kLog2eLow = 1.925962991e-8f, kLn2 = 0.6931471805599453f;
    const float w = fminf(fabsf(y), 256.f), t = w * kLog2e,   // e^-256 is zero already
                lo = fmaf(w, kLog2eLow, fmaf(w, kLog2e, -t));
    float h;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(h) : "f"(-t));
    h *= fmaf(-lo, kLn2, 1.f);
    const float d = 1.f + h;
    float r = rcp_approx(d);
    r = fmaf(fmaf(-d, r, 1.f), r, r);
    return y * (y < 0.f ? h * r : r);
}

}  // namespace sm100
}  // namespace la
