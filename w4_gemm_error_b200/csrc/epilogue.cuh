// What a layer's epilogue does after the W4 product and the Error Compensator:
//   y = act(Y + bias) * mul + residual
// in fp32, rounded once to bf16.  Shared by the forms of the forward kernels
// that have one (library-internal).
#pragma once
#include <cstdint>

#include "device_utils.cuh"

namespace spear {

// Activations, the values of SPEAR_ACT_*.
enum : int { kActNone = 0, kActRelu = 1, kActSilu = 2, kActGelu = 3, kActGeluTanh = 4 };

// Form of a forward kernel: kPlain is y = Y on bf16 activations; kEpi adds the
// epilogue; kQ8 reads e4m3 activations with one scale a token, and has the
// epilogue too.
enum : int { kPlain = 0, kEpi = 1, kQ8 = 2 };

struct Epilogue {
    const uint16_t *bias = nullptr;       // bf16 [N]
    const uint16_t *mul = nullptr;        // bf16 [M][N]
    const uint16_t *residual = nullptr;   // bf16 [M][N]; may be y itself
    int act = kActNone;
    const float *xs = nullptr;            // [M] scale of each token's e4m3 activations (kQ8)
};

// v / (1 + exp(-c)), by the hardware's exp2 and reciprocal:  with t = 2^-7 exp(-c / 2),
//   (2^-14 v) / (2^-14 + t^2).
// Both instructions flush what leaves the normal numbers, and exp(-c) itself does
// so from |c| = 88 on, where the result still is a bf16 value; t and the
// denominator do so from c = -97 on, where the result is below bf16's smallest
// value (2^-133).  The exponent of t, |c| log2(e) / 2 + 7, is off by a unit in its
// last place at most, so the result by a few units of 2^-23 max(8, |c|), far inside
// its bf16 rounding; 2^-14 v is inexact below |v| = 2^-112 and moves the result by
// less than 2^-135 there.  A large negative c gives t = inf and a zero.
__device__ __forceinline__ float ex2_approx(float x)
{
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ float rcp_approx(float x)
{
    float y;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
constexpr float kHalfLog2e = 0.7213475204444817f;
constexpr float kSig = 0x1p-14f;
constexpr float kGeluK = 1.5957691216057308f, kGeluK3 = 0.071354816272600f;   // 2 sqrt(2/pi), and times 0.044715
__device__ __forceinline__ float times_sigmoid(float v, float c)
{
    const float t = ex2_approx(fmaf(-kHalfLog2e, c, -7.0f));
    return kSig * v * rcp_approx(fmaf(t, t, kSig));
}

__device__ __forceinline__ float activate(float v, int act)
{
    switch (act) {
    case kActRelu: return v < 0.f ? 0.f : v;
    case kActSilu: return times_sigmoid(v, v);
    // v Phi(v), by erfc so that the negative tail keeps its relative accuracy
    case kActGelu: return 0.5f * v * erfcf(-0.70710678118654752f * v);
    // 0.5 (1 + tanh a) = 1 / (1 + exp(-2a)), a = sqrt(2/pi) (v + 0.044715 v^3)
    case kActGeluTanh: return times_sigmoid(v, v * fmaf(kGeluK3, v * v, kGeluK));
    default: return v;
    }
}

// The same as a call, for code that runs once.
static __device__ __noinline__ float activate_call(float v, int act) { return activate(v, act); }

// Two fp32 values in one register pair, and the packed fp32 instructions of
// sm_100 on them (each half rounded as the scalar instruction rounds it).
using f32x2 = unsigned long long;
__device__ __forceinline__ f32x2 f2_pack(float lo, float hi)
{
    f32x2 d;
    asm("mov.b64 %0, {%1, %2};" : "=l"(d) : "f"(lo), "f"(hi));
    return d;
}
__device__ __forceinline__ void f2_unpack(f32x2 v, float &lo, float &hi)
{
    asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(v));
}
__device__ __forceinline__ f32x2 f2_mul(f32x2 a, f32x2 b)
{
    f32x2 d;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
    return d;
}
__device__ __forceinline__ f32x2 f2_add(f32x2 a, f32x2 b)
{
    f32x2 d;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
    return d;
}
__device__ __forceinline__ f32x2 f2_fma(f32x2 a, f32x2 b, f32x2 c)
{
    f32x2 d;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
    return d;
}

// activate() of two values.
template <int ACT>
__device__ __forceinline__ f32x2 activate2(f32x2 v)
{
    if constexpr (ACT == kActNone) {
        return v;
    } else if constexpr (ACT == kActSilu || ACT == kActGeluTanh) {
        f32x2 c = v;
        if constexpr (ACT == kActGeluTanh)
            c = f2_mul(v, f2_fma(f2_pack(kGeluK3, kGeluK3), f2_mul(v, v), f2_pack(kGeluK, kGeluK)));
        float a, b;
        f2_unpack(f2_fma(c, f2_pack(-kHalfLog2e, -kHalfLog2e), f2_pack(-7.f, -7.f)), a, b);
        const f32x2 t = f2_pack(ex2_approx(a), ex2_approx(b));
        f2_unpack(f2_fma(t, t, f2_pack(kSig, kSig)), a, b);
        return f2_mul(f2_mul(v, f2_pack(kSig, kSig)), f2_pack(rcp_approx(a), rcp_approx(b)));
    } else {
        float a, b;
        f2_unpack(v, a, b);
        return f2_pack(activate(a, ACT), activate(b, ACT));
    }
}

// The operands of output (t, n): loaded apart from their use, so that the
// loads are in flight while the product is formed.  Plain loads: an earlier kernel
// that still runs may write them, and mul and residual may be the memory of y.
struct EpiOperands {
    float bias = 0.f, mul = 1.f, residual = 0.f;
};

__device__ __forceinline__ EpiOperands epi_load(const Epilogue &e, int64_t t, int64_t n, int64_t N)
{
    EpiOperands o;
    if (e.bias)
        o.bias = bf16_lo(e.bias[n]);
    if (e.mul)
        o.mul = bf16_lo(e.mul[t * N + n]);
    if (e.residual)
        o.residual = bf16_lo(e.residual[t * N + n]);
    return o;
}

__device__ __forceinline__ float epi_apply(const Epilogue &e, float v, const EpiOperands &o)
{
    return activate(v + o.bias, e.act) * o.mul + o.residual;
}

}  // namespace spear
