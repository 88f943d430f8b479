// Root-mean-square norm with the residual's addition, and 8-bit quantisation
// of activation rows with one scale a row.
//
//   h[t,k] = bf16(x[t,k] + residual[t,k])                 (h = x without a residual)
//   v[t,k] = h[t,k] w[k] * rinv_t,  rinv_t = 1 / sqrt(mean_k h[t,k]^2 + eps)
//   y[t,k] = bf16(v[t,k])
//   a_t    = max(max_k |v[t,k]|, 2^-100)
//   s[t]   = a_t / 448,   q[t,k] = e4m3(v[t,k] * (448 / a_t))
//
// (the quantisation alone: v = x).  The rows feed the W4 layers: y the bf16
// forward, (q, s) the 8-bit one.
//
// One CTA per row, the row in registers: it is read once and both outputs are
// formed from the copy held there.  rinv_t is one positive factor of the whole
// row, so max_k |v| = rinv_t max_k |h w| (rounding is monotonic: the largest
// product stays the largest), and the sum of squares and the maximum share one
// block reduction: one barrier between the last load and the first store.
// All sums are fp32; v is rounded once to each output type.
#include <cuda_runtime.h>

#include "device_utils.cuh"
#include "handle.h"
#include "norm.h"
#include "spear_w4ec.h"

namespace spear {
namespace {

constexpr float kE4m3Max = 448.0f;
constexpr float kAmaxFloor = 7.888609052210118e-31f;   // 2^-100: 448 / a stays finite

struct NormParams {
    const uint16_t *x;
    const uint16_t *residual;   // null: none
    const uint16_t *w;          // null: quantise x itself (no norm)
    float eps;
    uint16_t *h;                // the sum (null: not stored)
    uint16_t *y;                // null: none
    uint8_t *q;                 // null: none
    float *s;
    int64_t K;
};

// VEC consecutive elements from global memory, as bf16 bit patterns.
template <int VEC>
__device__ __forceinline__ void load_vec(const uint16_t *p, uint16_t (&e)[VEC])
{
    if constexpr (VEC == 8) {
        const uint4 v = *reinterpret_cast<const uint4 *>(p);
        const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            e[2 * i] = (uint16_t)w[i];
            e[2 * i + 1] = (uint16_t)(w[i] >> 16);
        }
    } else if constexpr (VEC == 2) {
        const uint32_t v = *reinterpret_cast<const uint32_t *>(p);
        e[0] = (uint16_t)v;
        e[1] = (uint16_t)(v >> 16);
    } else {
        e[0] = *p;
    }
}

template <int VEC>
__device__ __forceinline__ void store_bf16(uint16_t *p, const float (&v)[VEC])
{
    if constexpr (VEC == 8) {
        *reinterpret_cast<uint4 *>(p) = make_uint4(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]),
                                                   pack_bf16x2(v[4], v[5]), pack_bf16x2(v[6], v[7]));
    } else if constexpr (VEC == 2) {
        *reinterpret_cast<uint32_t *>(p) = pack_bf16x2(v[0], v[1]);
    } else {
        *p = __bfloat16_as_ushort(__float2bfloat16_rn(v[0]));
    }
}

template <int VEC>
__device__ __forceinline__ void store_e4m3(uint8_t *p, const float (&v)[VEC])
{
    if constexpr (VEC == 8) {
        *reinterpret_cast<uint2 *>(p) =
            make_uint2((uint32_t)pack_e4m3x2(v[0], v[1]) | ((uint32_t)pack_e4m3x2(v[2], v[3]) << 16),
                       (uint32_t)pack_e4m3x2(v[4], v[5]) | ((uint32_t)pack_e4m3x2(v[6], v[7]) << 16));
    } else if constexpr (VEC == 2) {
        *reinterpret_cast<uint16_t *>(p) = pack_e4m3x2(v[0], v[1]);
    } else {
        *p = (uint8_t)pack_e4m3x2(v[0], 0.f);
    }
}

__device__ __forceinline__ float bf16_f(uint16_t b) { return __uint_as_float((uint32_t)b << 16); }

// Sum and maximum over the CTA, the same in every thread.  The maximum is of
// non-negative values (or NaN) as bit patterns: unsigned order keeps a NaN,
// which is above every number, so that a bad row is seen.
__device__ __forceinline__ void block_reduce(float &sum, uint32_t &top)
{
    __shared__ float s_sum[32];
    __shared__ uint32_t s_top[32];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, nw = (int)(blockDim.x >> 5);
#pragma unroll
    for (int d = 16; d > 0; d >>= 1)
        sum += __shfl_xor_sync(0xffffffffu, sum, d);
    top = __reduce_max_sync(0xffffffffu, top);
    if (nw == 1)
        return;
    if (lane == 0) {
        s_sum[warp] = sum;
        s_top[warp] = top;
    }
    __syncthreads();
    sum = lane < nw ? s_sum[lane] : 0.f;
    top = lane < nw ? s_top[lane] : 0u;
#pragma unroll
    for (int d = 16; d > 0; d >>= 1)
        sum += __shfl_xor_sync(0xffffffffu, sum, d);
    top = __reduce_max_sync(0xffffffffu, top);
}

// NV vectors of VEC elements a thread; NV = 0: the row is longer than the
// registers hold and is read again for the outputs (h is rounded the same way
// both times; a sum stored over its residual is read back from h instead).
template <int VEC, int NV>
__global__ void __launch_bounds__(1024) norm_kernel(NormParams p)
{
    pdl_launch_dependents();
    pdl_wait();   // every operand may come from an earlier kernel in the stream
    const int64_t row = blockIdx.x;
    const int T = (int)blockDim.x, tid = (int)threadIdx.x;
    const int64_t nvec = p.K / VEC;
    const uint16_t *x = p.x + row * p.K;
    const uint16_t *res = p.residual ? p.residual + row * p.K : nullptr;
    uint16_t *h = p.h ? p.h + row * p.K : nullptr;
    constexpr bool kHeld = NV > 0;
    constexpr int kN = kHeld ? NV : 1;
    float hv[kN][VEC];   // h, then h w
    float sum = 0.f;
    uint32_t top = 0u;

    auto load_h = [&](int64_t c, float (&v)[VEC]) {
        uint16_t e[VEC];
        load_vec<VEC>(x + c * VEC, e);
#pragma unroll
        for (int i = 0; i < VEC; ++i)
            v[i] = bf16_f(e[i]);
        if (res) {
            load_vec<VEC>(res + c * VEC, e);
#pragma unroll
            for (int i = 0; i < VEC; ++i)
                v[i] = __bfloat162float(__float2bfloat16_rn(v[i] + bf16_f(e[i])));
        }
    };
    auto times_w = [&](int64_t c, float (&v)[VEC]) {
        if (!p.w)
            return;
        uint16_t e[VEC];
        load_vec<VEC>(p.w + c * VEC, e);
#pragma unroll
        for (int i = 0; i < VEC; ++i)
            v[i] *= bf16_f(e[i]);
    };
    auto count = [&](int64_t c, float (&v)[VEC]) {
        if (h)
            store_bf16<VEC>(h + c * VEC, v);
#pragma unroll
        for (int i = 0; i < VEC; ++i)
            sum += v[i] * v[i];
        times_w(c, v);
#pragma unroll
        for (int i = 0; i < VEC; ++i)
            top = max(top, __float_as_uint(fabsf(v[i])));
    };
    if constexpr (kHeld) {
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            const int64_t c = tid + (int64_t)j * T;
            if (c < nvec) {
                load_h(c, hv[j]);
                count(c, hv[j]);
            }
        }
    } else {
        for (int64_t c = tid; c < nvec; c += T) {
            load_h(c, hv[0]);
            count(c, hv[0]);
        }
    }
    block_reduce(sum, top);
    const float rinv = p.w ? 1.0f / sqrtf(sum / (float)p.K + p.eps) : 1.0f;
    uint32_t amax = __float_as_uint(__uint_as_float(top) * rinv);
    amax = max(amax & 0x7FFFFFFFu, __float_as_uint(kAmaxFloor));
    const float a = __uint_as_float(amax);
    const float inv = kE4m3Max / a;
    if (p.q && tid == 0)
        p.s[row] = a / kE4m3Max;
    auto emit = [&](int64_t c, float (&v)[VEC]) {
#pragma unroll
        for (int i = 0; i < VEC; ++i)
            v[i] *= rinv;
        if (p.y)
            store_bf16<VEC>(p.y + row * p.K + c * VEC, v);
        if (p.q) {
#pragma unroll
            for (int i = 0; i < VEC; ++i)
                v[i] *= inv;
            store_e4m3<VEC>(p.q + row * p.K + c * VEC, v);
        }
    };
    if constexpr (kHeld) {
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            const int64_t c = tid + (int64_t)j * T;
            if (c < nvec)
                emit(c, hv[j]);
        }
    } else {
        for (int64_t c = tid; c < nvec; c += T) {
            if (h) {   // written above by this thread; x or the residual may be the same memory
                uint16_t e[VEC];
                load_vec<VEC>(h + c * VEC, e);
#pragma unroll
                for (int i = 0; i < VEC; ++i)
                    hv[0][i] = bf16_f(e[i]);
            } else {
                load_h(c, hv[0]);
            }
            times_w(c, hv[0]);
            emit(c, hv[0]);
        }
    }
}

using NormFn = void (*)(NormParams);
template <int VEC>
NormFn norm_fn(int nv)
{
    switch (nv) {
    case 1: return norm_kernel<VEC, 1>;
    case 2: return norm_kernel<VEC, 2>;
    case 4: return norm_kernel<VEC, 4>;
    default: return norm_kernel<VEC, 0>;
    }
}

}  // namespace

cudaError_t launch_norm(const void *x, const void *residual, const void *w, float eps, int64_t M, int64_t K, void *h,
                        void *y, void *q, float *s, cudaStream_t st)
{
    if (M <= 0)
        return cudaSuccess;
    NormParams p;
    p.x = static_cast<const uint16_t *>(x);
    p.residual = static_cast<const uint16_t *>(residual);
    p.w = static_cast<const uint16_t *>(w);
    p.eps = eps;
    p.h = static_cast<uint16_t *>(h);
    p.y = static_cast<uint16_t *>(y);
    p.q = static_cast<uint8_t *>(q);
    p.s = s;
    p.K = K;
    // the widest access that every row starts on (the bases are 16-byte aligned)
    const int vec = K % 8 == 0 ? 8 : (K % 2 == 0 ? 2 : 1);
    const int64_t nvec = K / vec;
    int nv = 1;
    while (nv < 4 && nvec > (int64_t)256 * nv)
        nv *= 2;
    int64_t threads = (nvec + nv - 1) / nv;
    threads = (threads + 31) / 32 * 32;
    if (threads > 1024) {
        threads = 1024;
        nv = 0;
    }
    NormFn fn = vec == 8 ? norm_fn<8>(nv) : (vec == 2 ? norm_fn<2>(nv) : norm_fn<1>(nv));
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)M);
    cfg.blockDim = dim3((unsigned)threads);
    cfg.stream = st;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, fn, p);
}

}  // namespace spear

namespace {

bool aligned16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
constexpr int64_t kMaxRows = 0x7FFFFFFF;   // one CTA a row

// Whether [a, a + na) and [b, b + nb) share a byte.
bool overlap(const void *a, size_t na, const void *b, size_t nb)
{
    const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
    return a && b && x < y + nb && y < x + na;
}

// An output of the same shape and type may take the place of an input (each
// element is read by the thread that writes it, before it does), but no output
// may overlap another buffer in any other way.
bool clash(const void *out, const void *in, size_t n) { return out != in && overlap(out, n, in, n); }

}  // namespace

extern "C" {

int spear_w4ec_rmsnorm(const void *x, const void *residual, const void *weight, float eps, int64_t M, int64_t K,
                       void *sum, void *y, void *q, float *s, void *stream)
{
    if (M < 0 || M > kMaxRows || K <= 0 || K > kMaxRows || !(eps >= 0.0f && eps < 1e30f))
        return SPEAR_ERR_INVALID;
    if (M == 0)
        return SPEAR_OK;
    if (!x || !weight || (!y && !q) || (q != nullptr) != (s != nullptr) || (residual != nullptr) != (sum != nullptr))
        return SPEAR_ERR_INVALID;
    if (!aligned16(x) || !aligned16(residual) || !aligned16(weight) || !aligned16(sum) || !aligned16(y) ||
        !aligned16(q) || (reinterpret_cast<uintptr_t>(s) & 3u) != 0)
        return SPEAR_ERR_INVALID;
    const size_t n = (size_t)M * (size_t)K * 2, nw = (size_t)K * 2, ns = (size_t)M * 4;
    const void *ins[2] = {x, residual}, *outs[2] = {sum, y};
    for (const void *o : outs) {
        for (const void *i : ins)
            if (clash(o, i, n))
                return SPEAR_ERR_INVALID;
        if (overlap(o, n, weight, nw) || overlap(o, n, q, n / 2) || overlap(o, n, s, ns))
            return SPEAR_ERR_INVALID;
    }
    for (const void *i : ins)
        if (overlap(q, n / 2, i, n) || overlap(s, ns, i, n))
            return SPEAR_ERR_INVALID;
    if (overlap(sum, n, y, n) || overlap(q, n / 2, weight, nw) || overlap(s, ns, weight, nw) ||
        overlap(q, n / 2, s, ns))
        return SPEAR_ERR_INVALID;
    return spear::status_of(spear::launch_norm(x, residual, weight, eps, M, K, sum, y, q, s,
                                               static_cast<cudaStream_t>(stream)));
}

int spear_w4ec_quantize_q8(const void *x, int64_t M, int64_t K, void *q, float *s, void *stream)
{
    if (M < 0 || M > kMaxRows || K <= 0 || K > kMaxRows)
        return SPEAR_ERR_INVALID;
    if (M == 0)
        return SPEAR_OK;
    const size_t n = (size_t)M * (size_t)K;
    if (!x || !q || !s || !aligned16(x) || !aligned16(q) || (reinterpret_cast<uintptr_t>(s) & 3u) != 0 ||
        overlap(x, 2 * n, q, n) || overlap(x, 2 * n, s, (size_t)M * 4) || overlap(q, n, s, (size_t)M * 4))
        return SPEAR_ERR_INVALID;
    return spear::status_of(spear::launch_norm(x, nullptr, nullptr, 0.f, M, K, nullptr, nullptr, q, s,
                                               static_cast<cudaStream_t>(stream)));
}

}  // extern "C"
