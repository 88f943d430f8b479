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

// v / (1 + exp(-c)).  The fast exponential and reciprocal are off by a few
// units of 2^-23 |c| at most, far inside the bf16 rounding of the result; a
// large negative c gives exp = inf and a result of zero.
__device__ __forceinline__ float times_sigmoid(float v, float c) { return __fdividef(v, 1.0f + __expf(-c)); }

__device__ __forceinline__ float activate(float v, int act)
{
    switch (act) {
    case kActRelu: return v < 0.f ? 0.f : v;
    case kActSilu: return times_sigmoid(v, v);
    // v Phi(v), by erfc so that the negative tail keeps its relative accuracy
    case kActGelu: return 0.5f * v * erfcf(-0.70710678118654752f * v);
    // 0.5 (1 + tanh a) = 1 / (1 + exp(-2a)), a = sqrt(2/pi) (v + 0.044715 v^3)
    case kActGeluTanh: return times_sigmoid(v, 1.5957691216057308f * (v + 0.044715f * v * v * v));
    default: return v;
    }
}

// The operands of output (t, n): loaded apart from their use, so that the
// loads are in flight while the product is formed.  mul and residual are read
// with plain loads, since either may be the memory of y.
struct EpiOperands {
    float bias = 0.f, mul = 1.f, residual = 0.f;
};

__device__ __forceinline__ EpiOperands epi_load(const Epilogue &e, int64_t t, int64_t n, int64_t N)
{
    EpiOperands o;
    if (e.bias)
        o.bias = bf16_lo(__ldg(e.bias + n));
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
