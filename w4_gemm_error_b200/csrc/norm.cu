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
// A row is read once and held in registers as h in bf16 (exact); both outputs
// are formed from it.  rinv_t is one positive factor of the whole
// row, so max_k |v| = rinv_t max_k |h w| (rounding is monotonic: the largest
// product stays the largest), and the sum of squares and the maximum share one
// block reduction: one barrier between the last load and the first store.
// All sums are fp32; v is rounded once to each output type.
#include <cuda_runtime.h>

#include <atomic>

#include "async_utils.cuh"
#include "handle.h"
#include "norm.h"
#include "spear_w4ec.h"

namespace spear {
namespace {

constexpr float kE4m3Max = 448.0f;
constexpr int kWarpRows = 8;   // rows of a CTA with one warp a row
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
    int64_t M, K;
};

// VEC consecutive bf16 elements (8, 2 or 1) as packed pairs.
template <int VEC>
struct Vec {
    uint32_t w[(VEC + 1) / 2];
    __device__ __forceinline__ float get(int i) const { return i & 1 ? bf16_hi(w[i / 2]) : bf16_lo(w[i / 2]); }
};

template <int VEC>
__device__ __forceinline__ Vec<VEC> load_vec(const uint16_t *p)
{
    Vec<VEC> v;
    if constexpr (VEC == 8) {
        const uint4 u = *reinterpret_cast<const uint4 *>(p);
        v.w[0] = u.x, v.w[1] = u.y, v.w[2] = u.z, v.w[3] = u.w;
    } else if constexpr (VEC == 2) {
        v.w[0] = *reinterpret_cast<const uint32_t *>(p);
    } else {
        v.w[0] = *p;
    }
    return v;
}

template <int VEC>
__device__ __forceinline__ void store_vec(uint16_t *p, const Vec<VEC> &v)
{
    if constexpr (VEC == 8)
        *reinterpret_cast<uint4 *>(p) = make_uint4(v.w[0], v.w[1], v.w[2], v.w[3]);
    else if constexpr (VEC == 2)
        *reinterpret_cast<uint32_t *>(p) = v.w[0];
    else
        *p = (uint16_t)v.w[0];
}

// bf16(a + b), element by element.
template <int VEC>
__device__ __forceinline__ Vec<VEC> add_vec(const Vec<VEC> &a, const Vec<VEC> &b)
{
    Vec<VEC> v;
#pragma unroll
    for (int i = 0; i < (VEC + 1) / 2; ++i)
        v.w[i] = pack_bf16x2(bf16_lo(a.w[i]) + bf16_lo(b.w[i]), bf16_hi(a.w[i]) + bf16_hi(b.w[i]));
    return v;
}

template <int VEC>
__device__ __forceinline__ Vec<VEC> to_bf16(const float (&v)[VEC])
{
    Vec<VEC> o;
#pragma unroll
    for (int i = 0; i < (VEC + 1) / 2; ++i)
        o.w[i] = pack_bf16x2(v[2 * i], 2 * i + 1 < VEC ? v[(2 * i + 1) % VEC] : 0.f);
    return o;
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

// Sum and maximum over the nw warps of a row, the same in every thread.  The maximum is of
// non-negative values (or NaN) as bit patterns: unsigned order keeps a NaN,
// which is above every number, so that a bad row is seen.
struct Reduce {
    float sum[32];
    uint32_t top[32];
};
__device__ __forceinline__ void block_reduce(float &sum, float &most, Reduce &s, int nw)
{
    uint32_t top = __float_as_uint(most) & 0x7FFFFFFFu;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
    for (int d = 16; d > 0; d >>= 1)
        sum += __shfl_xor_sync(0xffffffffu, sum, d);
    top = __reduce_max_sync(0xffffffffu, top);
    most = __uint_as_float(top);
    if (nw == 1)
        return;
    if (lane == 0) {
        s.sum[warp] = sum;
        s.top[warp] = top;
    }
    __syncthreads();
    sum = lane < nw ? s.sum[lane] : 0.f;
    top = lane < nw ? s.top[lane] : 0u;
#pragma unroll
    for (int d = 16; d > 0; d >>= 1)
        sum += __shfl_xor_sync(0xffffffffu, sum, d);
    most = __uint_as_float(__reduce_max_sync(0xffffffffu, top));
}

// h w of one vector (h itself without a norm), in fp32.
template <int VEC, bool NORM>
__device__ __forceinline__ void times_w(const Vec<VEC> &h, const Vec<VEC> &w, float (&v)[VEC])
{
#pragma unroll
    for (int i = 0; i < VEC; ++i)
        v[i] = NORM ? h.get(i) * w.get(i) : h.get(i);
}

// max(|a|, |b|); NaN if either is.
__device__ __forceinline__ float max_abs(float a, float b)
{
    float d;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(d) : "f"(a), "f"(fabsf(b)));
    return d;
}

// One vector's share of the row's statistics: the sum of h^2 and the largest
// |h w| (needed for a quantised output alone).
template <int VEC, bool NORM>
__device__ __forceinline__ void count(const Vec<VEC> &h, const Vec<VEC> &w, bool q8, float &sum, float &top)
{
    if (NORM) {
#pragma unroll
        for (int i = 0; i < VEC; ++i)
            sum += h.get(i) * h.get(i);
    }
    if (!q8)
        return;
    float v[VEC];
    times_w<VEC, NORM>(h, w, v);
#pragma unroll
    for (int i = 0; i < VEC; ++i)
        top = max_abs(top, v[i]);
}

// The row's factors from its statistics: 1 / rms (1 without a norm), the
// quantisation's a and 448 / a.
struct Factors {
    float rinv, a, inv;
};
template <bool NORM>
__device__ __forceinline__ Factors factors(const NormParams &p, float sum, float top)
{
    Factors f;
    f.rinv = NORM ? rsqrtf(sum / (float)p.K + p.eps) : 1.0f;   // (2 ulp: a 2^14th of the bf16 rounding)
    const uint32_t amax = __float_as_uint(top * f.rinv) & 0x7FFFFFFFu;
    f.a = __uint_as_float(max(amax, __float_as_uint(kAmaxFloor)));
    f.inv = kE4m3Max / f.a;
    return f;
}

template <int VEC, bool NORM>
__device__ __forceinline__ void emit(const NormParams &p, int64_t at, const Vec<VEC> &h, const Vec<VEC> &w,
                                     const Factors &f)
{
    float v[VEC];
    times_w<VEC, NORM>(h, w, v);
    if (NORM) {
#pragma unroll
        for (int i = 0; i < VEC; ++i)
            v[i] *= f.rinv;
    }
    if (NORM && p.y)
        store_vec<VEC>(p.y + at, to_bf16<VEC>(v));
    if (p.q) {
#pragma unroll
        for (int i = 0; i < VEC; ++i)
            v[i] *= f.inv;
        store_e4m3<VEC>(p.q + at, v);
    }
}

// One CTA a row, or (WARP) one warp a row where a warp holds it: short rows cost
// a CTA's launch each otherwise (8192 rows of 512 quantised: 3.6 us instead of 8.9).
// HBM bounds many rows (8192 rows of 4096 with residual to 8 bits: 42.5 us, 5.5
// TB/s; 2047 of 14336 quantised: 14.8 us, 5.9 TB/s): enough CTAs an SM are resident
// that others load while one reduces and stores.  (Persistent CTAs with a ring of
// rows filled by bulk copies took 43.2 and 16.8 us.)
// NV vectors of VEC elements a thread;
// NV = 0: the row is longer than the registers hold and is read again for the
// outputs (a sum that was stored is read back, since x or the residual may be the
// same memory).
template <int VEC, int NV, bool NORM, bool WARP>
__global__ void __launch_bounds__(WARP ? 32 * kWarpRows : 1024) norm_kernel(NormParams p)
{
    __shared__ Reduce s_red;
    pdl_launch_dependents();
    pdl_wait();   // every operand may come from an earlier kernel in the stream
    const int64_t row = WARP ? (int64_t)blockIdx.x * kWarpRows + (threadIdx.x >> 5) : blockIdx.x;
    if (WARP && row >= p.M)
        return;
    const int64_t at = row * p.K;
    const int T = WARP ? 32 : (int)blockDim.x, tid = WARP ? (int)(threadIdx.x & 31) : (int)threadIdx.x;
    const int64_t nvec = p.K / VEC;
    const bool q8 = p.q != nullptr;
    constexpr int kN = NV > 0 ? NV : 1;
    Vec<VEC> h[kN] = {}, w[kN] = {};
    float sum = 0.f;
    float top = 0.f;
    auto load_h = [&](int64_t c) {
        Vec<VEC> v = load_vec<VEC>(p.x + at + c * VEC);
        if (p.residual)
            v = add_vec<VEC>(v, load_vec<VEC>(p.residual + at + c * VEC));
        return v;
    };
    if constexpr (NV > 0) {
        // every load is issued before the first is used
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            const int64_t c = tid + (int64_t)j * T;
            if (c < nvec) {
                h[j] = load_h(c);
                if (NORM)
                    w[j] = load_vec<VEC>(p.w + c * VEC);
            }
        }
#pragma unroll
        for (int j = 0; j < NV; ++j) {   // (a vector past the row is zero and counts for nothing)
            const int64_t c = tid + (int64_t)j * T;
            if (p.h && c < nvec)
                store_vec<VEC>(p.h + at + c * VEC, h[j]);
            count<VEC, NORM>(h[j], w[j], q8, sum, top);
        }
    } else {
        for (int64_t c = tid; c < nvec; c += T) {
            h[0] = load_h(c);
            if (NORM)
                w[0] = load_vec<VEC>(p.w + c * VEC);
            if (p.h)
                store_vec<VEC>(p.h + at + c * VEC, h[0]);
            count<VEC, NORM>(h[0], w[0], q8, sum, top);
        }
    }
    block_reduce(sum, top, s_red, WARP ? 1 : T >> 5);
    const Factors f = factors<NORM>(p, sum, top);
    if (q8 && tid == 0)
        p.s[row] = f.a / kE4m3Max;
    if constexpr (NV > 0) {
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            const int64_t c = tid + (int64_t)j * T;
            if (c < nvec)
                emit<VEC, NORM>(p, at + c * VEC, h[j], w[j], f);
        }
    } else {
        for (int64_t c = tid; c < nvec; c += T) {
            h[0] = p.h ? load_vec<VEC>(p.h + at + c * VEC) : load_h(c);
            if (NORM)
                w[0] = load_vec<VEC>(p.w + c * VEC);
            emit<VEC, NORM>(p, at + c * VEC, h[0], w[0], f);
        }
    }
}

// SMs of the current device (asked for once a device).
int sm_count()
{
    constexpr int kMaxDevices = 64;
    static std::atomic<int> known[kMaxDevices];
    int dev = 0, n = 0;
    if (cudaGetDevice(&dev) == cudaSuccess && dev < kMaxDevices)
        n = known[dev].load(std::memory_order_relaxed);
    if (n == 0) {
        if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || n <= 0)
            return 1;   // (the launch will report what is wrong)
        if (dev < kMaxDevices)
            known[dev].store(n, std::memory_order_relaxed);
    }
    return n;
}

using NormFn = void (*)(NormParams);
template <int VEC, bool NORM, bool WARP>
NormFn norm_fn(int nv)
{
    switch (nv) {
    case 1: return norm_kernel<VEC, 1, NORM, WARP>;
    case 2: return norm_kernel<VEC, 2, NORM, WARP>;
    case 4: return norm_kernel<VEC, 4, NORM, WARP>;
    default: return norm_kernel<VEC, 0, NORM, false>;
    }
}
template <bool NORM, bool WARP>
NormFn norm_fn_of(int vec, int nv)
{
    return vec == 8 ? norm_fn<8, NORM, WARP>(nv) : (vec == 2 ? norm_fn<2, NORM, WARP>(nv) : norm_fn<1, NORM, WARP>(nv));
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
    p.M = M;
    p.K = K;
    cudaLaunchConfig_t cfg = {};
    cfg.stream = st;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    // the widest access that every row starts on (the bases are 16-byte aligned)
    const int vec = K % 8 == 0 ? 8 : (K % 2 == 0 ? 2 : 1);
    const int64_t nvec = K / vec;
    // as few vectors a thread as 256 threads hold the row with, 512 where every row
    // has an SM (one row of 8192 with residual 2.3 us instead of 2.7; many of them
    // 95 us instead of 85: fewer CTAs an SM to fill each other's waits); a warp a
    // row from two CTAs of them an SM on (2048 rows of 512 normed with residual to 8
    // bits: 3.6 us with a CTA a row, 4.4 with a warp; 4096: 5.5 and 5.1)
    const int64_t sms = sm_count();
    const bool warp = nvec <= 32 * 4 && M >= 2 * sms * kWarpRows;
    const int span = warp ? 32 : (M <= sms ? 512 : 256);
    int nv = 1;
    while (nv < 4 && nvec > (int64_t)span * nv)
        nv *= 2;
    int64_t threads = warp ? 32 * kWarpRows : ((nvec + nv - 1) / nv + 31) / 32 * 32;
    if (threads > 1024) {
        threads = 1024;
        nv = 0;
    }
    cfg.gridDim = dim3((unsigned)(warp ? (M + kWarpRows - 1) / kWarpRows : M));
    cfg.blockDim = dim3((unsigned)threads);
    const NormFn fn = w ? (warp ? norm_fn_of<true, true>(vec, nv) : norm_fn_of<true, false>(vec, nv))
                        : (warp ? norm_fn_of<false, true>(vec, nv) : norm_fn_of<false, false>(vec, nv));
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
    return spear::guarded([&] {
        return spear::status_of(spear::launch_norm(x, residual, weight, eps, M, K, sum, y, q, s,
                                                   static_cast<cudaStream_t>(stream)));
    });
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
    return spear::guarded([&] {
        return spear::status_of(spear::launch_norm(x, nullptr, nullptr, 0.f, M, K, nullptr, nullptr, q, s,
                                                   static_cast<cudaStream_t>(stream)));
    });
}

}  // extern "C"
