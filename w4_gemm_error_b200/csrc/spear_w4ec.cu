// C ABI of the W4 + per-token-gated low-rank Error Compensator linear layer
// (declared in include/spear_w4ec.h): handle life cycle, argument checks,
// workspace, the adaptive fused/split dispatch and the kernel sequence of a
// forward pass.
#include <cuda_runtime.h>

#include <algorithm>
#include <cstdlib>
#include <cstring>
#include <mutex>
#include <new>
#include <vector>

#include "spear_w4ec.h"
#include "device_utils.cuh"
#include "epilogue.cuh"
#include "handle.h"
#include "kernels.h"
#include "tc_gemm.h"

using namespace spear;

namespace {


const char *env_fault()
{
    const char *f = std::getenv("SPEAR_FAULT");
    return f ? f : "";
}

int64_t round_up(int64_t a, int64_t b) { return (a + b - 1) / b * b; }

bool aligned16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

template <class T>
cudaError_t alloc_zero(T **p, size_t count)
{
    *p = nullptr;
    if (count == 0)
        return cudaSuccess;
    cudaError_t e = cudaMalloc(reinterpret_cast<void **>(p), count * sizeof(T));
    if (e != cudaSuccess)
        return e;
    return cudaMemset(*p, 0, count * sizeof(T));
}

void free_all(spear_w4ec *h)
{
    cudaFree(h->pk.codes);
    cudaFree(h->pk.s);
    cudaFree(h->pk.z);
    cudaFree(h->pk.G);
    cudaFree(h->pk.Bt);
    cudaFree(h->pk.Bts);
    cudaFree(h->v);
    cudaFree(h->gbuf);
    cudaFree(h->pre.part);
    cudaFree(h->pre.counters);
    cudaFree(h->dec.ws_u);
    cudaFree(h->dec.flags);
    cudaFree(h->dec.ws_stream);
    cudaFree(h->dec.cnt_stream);
    decode_free(h->dec);
    tc_free(h->tc);
    cudaFree(h->status);
    cudaFree(h->vready);
    cudaFree(h->x_stage);
    cudaFree(h->y_stage);
    cudaFree(h->xq_pad);
    cudaFree(h->rowc);
}

int from_cuda(cudaError_t e)
{
    if (e == cudaSuccess)
        return SPEAR_OK;
    if (e == cudaErrorMemoryAllocation)
        return SPEAR_ERR_NOMEM;
    return SPEAR_ERR_CUDA;
}

bool tc_supported(const spear_w4ec *h) { return tc_available(h->pk); }


// Kernel family and EC placement for M tokens: an explicit request, the tuned
// table entry, or the default (the split-K decode kernel for a few tokens,
// the tcgen05 tile kernel above, the EC fused in both).
// Untuned path: the decode kernel up to 32 tokens; beyond, the tcgen05
// kernel (which splits K on layers whose 128-row tiles fill at most half of
// the SMs).
uint32_t default_path(const spear_w4ec *h, int64_t M)
{
    const bool dec = decode_supported(h->pk, h->num_sms);
    if (!tc_supported(h) || (dec && M <= kDecodeMaxTokens))
        return SPEAR_FORCE_DECODE;
    return SPEAR_FORCE_TC;
}

// Path of the forms kEpi and kQ8 (the table's times are of the plain kernels,
// whose tcgen05 family is another one).  Measured in us per call, chained,
// decode against tcgen05 (bf16 / 8 bits):
//   4096 x 4096, r 32 (row-CTA kernel)   16 tokens  8.2 / 10.3 against 13.0 / 12.2
//                                        24 tokens 18.9 / 18.9 against 13.1 / 12.3
//   4096 x 14336, r 64 (split-K kernel)   8 tokens 15.2 / 16.7 against 22.3 / 18.1
//                                        16 tokens 20.2 / 21.5 against 22.7 / 18.6
//                                        24 tokens 31.2 / 33.0 against 23.1 / 19.0
//   14336 x 4096, r 64 (split-K kernel)   8 tokens 18.4 / 17.6 against 26.0 / 21.4
//                                        16 tokens 24.0 / 24.2 against 26.3 / 21.8
//   1032 x 2744, r 8 (split-K kernel)     8 tokens  7.1 /  8.3 against  8.5 / 11.1
//                                        16 tokens 10.4 / 11.7 against  8.8 / 11.5
// so: the decode kernels up to 16 tokens, but with 8 bits only up to 8 where
// the row-CTA kernel does not run (bf16 on narrow layers that it does not take
// loses up to 1.6 us from 9 to 16 tokens).
uint32_t form_path(const spear_w4ec *h, int64_t M, int form)
{
    int64_t most = 16;
    if (form == kQ8 && M > 8 && M <= 16 && !decode_rows_fits(h->pk, M, h->num_sms, form))
        most = 8;
    if (!tc_supported(h) || (M <= most && decode_supported(h->pk, h->num_sms)))
        return SPEAR_FORCE_DECODE;
    return SPEAR_FORCE_TC;
}

uint32_t resolve(const spear_w4ec *h, int64_t M, uint32_t flags)
{
    uint32_t path = flags & (SPEAR_FORCE_DECODE | SPEAR_FORCE_TC);
    uint32_t mode = flags & (SPEAR_FORCE_FUSED | SPEAR_FORCE_SPLIT);
    const uint32_t tuned = h->table[bucket_of(M)];
    if (!path)
        path = tuned ? (tuned & (SPEAR_FORCE_DECODE | SPEAR_FORCE_TC)) : default_path(h, M);
    if (!mode)
        mode = tuned ? (tuned & (SPEAR_FORCE_FUSED | SPEAR_FORCE_SPLIT)) : SPEAR_FORCE_FUSED;
    if (!mode)
        mode = SPEAR_FORCE_FUSED;
    return path | mode;
}

// Gate and v for M tokens: the tcgen05 kernel from 256 tokens on, the
// split-K mma.sync kernel below that.
// With `ready`, each CTA (tcgen05) or token tile (mma.sync) counts its v into
// ready[0]; *expected receives the number of counts.
cudaError_t run_prepass(const spear_w4ec *h, const void *x, int64_t M, bool tf32, cudaStream_t st,
                        unsigned *ready = nullptr, unsigned *expected = nullptr)
{
    if (M >= 256 && tc_prepass_supported(h->pk)) {
        if (expected)
            *expected = (unsigned)((M + 127) / 128);
        return launch_tc_prepass(h->pk, x, M, h->v, tf32, h->gbuf, h->tc, h->status, st, ready);
    }
    if (expected)
        *expected = (unsigned)((M + 15) / 16);
    // beside a tcgen05 kernel with tiles of at most 64 tokens (M <= 64), the
    // register-capped prepass shares the SMs with it instead of holding them
    return launch_prepass(h->pk, x, M, h->v, tf32, h->gbuf, h->pre, st, h->num_sms, ready, ready && M <= 64);
}

// The epilogue of tokens t0 and up.
Epilogue epi_rows(Epilogue e, int64_t t0, int64_t N)
{
    if (e.mul)
        e.mul += t0 * N;
    if (e.residual)
        e.residual += t0 * N;
    if (e.xs)
        e.xs += t0;
    return e;
}

// The forms kEpi and kQ8 of the forward pass on the tcgen05 kernels, rows of x
// ldx elements apart.  As in run_forward, with the EC the product's main stages
// start beside the prepass, which counts what it has written into vready.
int run_tc_form(const spear_w4ec *h, const void *x, int64_t ldx, void *y, int64_t M, bool ec, cudaStream_t st, int form,
                const Epilogue &epi)
{
    const Packed &pk = h->pk;
    if (h->fault_timeout) {
        // injected fault: report what a wait that ran out reports, launch nothing
        const int bits = kStatusTimeout;
        return from_cuda(cudaMemcpyAsync(h->status, &bits, sizeof(int), cudaMemcpyHostToDevice, st));
    }
    const bool pair = tc_use_pair(pk, M, ec, form, h->num_sms);
    unsigned *ready = ec ? h->vready : nullptr;
    unsigned expected = 0;
    cudaError_t e = cudaSuccess;
    // (without the EC only the pair kernel's 8-bit form needs one)
    if (ec || (pair && form == kQ8))
        e = launch_tc_prepass2(pk, x, ldx, epi.xs, M, ec, h->v, h->rowc, form, tc_map_g(h->tc), h->status, st,
                               h->num_sms, ready, &expected);
    if (e != cudaSuccess)
        return from_cuda(e);
    e = pair ? launch_tc_pair(pk, x, y, M, h->v, ec, tc_map_bt(h->tc), h->status, st, h->num_sms, ready, expected, form,
                              epi, ldx, h->rowc)
             : launch_tc_tile(pk, x, y, M, h->v, ec, tc_map_bt(h->tc), h->status, st, h->num_sms, ready, expected, form,
                              epi, ldx);
    if (e != cudaSuccess && ready)
        cudaMemsetAsync(h->vready, 0, 2 * sizeof(unsigned), st);   // nothing will reset the prepass's counts
    return from_cuda(e);
}

// form and epi: see epilogue.cuh.  The forms with an epilogue form the EC in
// the same kernel as the product: y is written once, after its last operand was
// read.
int run_forward(const spear_w4ec *h, const void *x, void *y, int64_t M, uint32_t flags, cudaStream_t st,
                int form = kPlain, const Epilogue &epi = Epilogue())
{
    const Packed &pk = h->pk;
    const bool ec = pk.r > 0 && !(flags & SPEAR_EC_OFF);
    uint32_t choice = resolve(h, M, flags);
    if (form != kPlain) {
        const uint32_t path = flags & (SPEAR_FORCE_DECODE | SPEAR_FORCE_TC);
        const uint32_t mode = flags & (SPEAR_FORCE_FUSED | SPEAR_FORCE_SPLIT);
        choice = (path ? path : form_path(h, M, form)) | (mode ? mode : (uint32_t)SPEAR_FORCE_FUSED);
    }
    if ((choice & SPEAR_FORCE_DECODE) && (choice & SPEAR_FORCE_TC))
        return SPEAR_ERR_INVALID;
    if ((choice & SPEAR_FORCE_FUSED) && (choice & SPEAR_FORCE_SPLIT))
        return SPEAR_ERR_INVALID;
    const bool fused = (choice & SPEAR_FORCE_FUSED) != 0;
    if (form != kPlain && !fused)
        return SPEAR_ERR_UNSUPPORTED;
    if (h->fault_launch)
        return SPEAR_ERR_CUDA;
    if (form != kPlain && (choice & SPEAR_FORCE_TC))
        return tc_supported(h) ? run_tc_form(h, x, pk.K, y, M, ec, st, form, epi) : SPEAR_ERR_UNSUPPORTED;
    cudaError_t e = cudaSuccess;
    const bool decode = (choice & SPEAR_FORCE_DECODE) != 0;
    if (decode && !decode_supported(pk, h->num_sms))
        return SPEAR_ERR_UNSUPPORTED;
    // the decode kernel computes its own gate and EC down-projection when fused;
    // before the fused tcgen05 kernel, the prepass counts its v into vready so
    // that the tcgen05 kernel can start its main stages alongside it
    const bool early = ec && fused && (choice & SPEAR_FORCE_TC) && tc_supported(h);
    unsigned expected = 0;
    if (ec && !(decode && fused)) {
        e = run_prepass(h, x, M, (choice & SPEAR_FORCE_TC) != 0 && fused, st, early ? h->vready : nullptr,
                        &expected);
        if (e != cudaSuccess)
            return from_cuda(e);
    }
    if (choice & SPEAR_FORCE_TC) {
        if (!tc_supported(h))
            return SPEAR_ERR_UNSUPPORTED;
        e = launch_tc(pk, x, y, M, h->v, ec && fused, h->tc, h->status, h->fault_timeout, st, h->num_sms,
                      early ? h->vready : nullptr, expected);
        if (e != cudaSuccess || (early && h->fault_timeout)) {
            // nothing will reset the prepass's counts: clear them for the next forward
            cudaMemsetAsync(h->vready, 0, 2 * sizeof(unsigned), st);
        }
        if (e != cudaSuccess)
            return from_cuda(e);
    } else {
        for (int64_t t0 = 0; t0 < M; t0 += kDecodeMaxTokens) {
            const int64_t m = std::min<int64_t>(kDecodeMaxTokens, M - t0);
            e = launch_decode_form(pk, static_cast<const uint16_t *>(x) + t0 * pk.K, pk.K,
                                   static_cast<uint16_t *>(y) + t0 * pk.N, m, ec && fused, h->dec, h->status, st,
                                   h->num_sms, form, epi_rows(epi, t0, pk.N));
            if (e != cudaSuccess)
                return from_cuda(e);
        }
    }
    if (ec && !fused) {
        e = launch_ec_apply(pk, h->v, y, M, st);
        if (e != cudaSuccess)
            return from_cuda(e);
    }
    return SPEAR_OK;
}

// Rows of 8-bit activations whose length is no multiple of 16 (it is one of 8)
// with the row pitch that the TMA copies need.
__global__ void __launch_bounds__(256) pad_rows_kernel(const uint2 *src, uint2 *dst, int64_t M, int units)
{
    pdl_launch_dependents();
    pdl_wait();
    const int64_t n = M * (units + 1);
    for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < n; i += (int64_t)gridDim.x * 256) {
        const int64_t t = i / (units + 1);
        const int u = (int)(i - t * (units + 1));
        dst[i] = u < units ? src[t * units + u] : make_uint2(0u, 0u);
    }
}

// The forward pass on e4m3 activations.
int run_forward_q8(const spear_w4ec *h, const void *xq, const float *xs, void *y, int64_t M, uint32_t flags,
                   cudaStream_t st, Epilogue epi)
{
    const Packed &pk = h->pk;
    const bool ec = pk.r > 0 && !(flags & SPEAR_EC_OFF);
    if ((flags & SPEAR_FORCE_DECODE) && (flags & SPEAR_FORCE_TC))
        return SPEAR_ERR_INVALID;
    if ((flags & SPEAR_FORCE_FUSED) && (flags & SPEAR_FORCE_SPLIT))
        return SPEAR_ERR_INVALID;
    if (flags & SPEAR_FORCE_SPLIT)
        return SPEAR_ERR_UNSUPPORTED;
    uint32_t path = flags & (SPEAR_FORCE_DECODE | SPEAR_FORCE_TC);
    if (!path)
        path = form_path(h, M, kQ8);
    if (!path_supported(h, path))
        return SPEAR_ERR_UNSUPPORTED;
    if (h->fault_launch)
        return SPEAR_ERR_CUDA;
    epi.xs = xs;
    int64_t ldx = pk.K;
    if (ldx % 16) {
        const int units = (int)(pk.K / 8);
        const int64_t blocks = std::min<int64_t>((M * (units + 1) + 255) / 256, 8 * h->num_sms);
        cudaLaunchConfig_t cfg = {};
        cfg.gridDim = dim3((unsigned)blocks);
        cfg.blockDim = dim3(256);
        cfg.stream = st;
        cudaLaunchAttribute attr[1];
        attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
        attr[0].val.programmaticStreamSerializationAllowed = 1;
        cfg.attrs = attr;
        cfg.numAttrs = 1;
        const cudaError_t e = cudaLaunchKernelEx(&cfg, pad_rows_kernel, static_cast<const uint2 *>(xq),
                                                 reinterpret_cast<uint2 *>(h->xq_pad), M, units);
        if (e != cudaSuccess)
            return from_cuda(e);
        xq = h->xq_pad;
        ldx = pk.K + 8;
    }
    if (path == SPEAR_FORCE_TC)
        return run_tc_form(h, xq, ldx, y, M, ec, st, kQ8, epi);
    for (int64_t t0 = 0; t0 < M; t0 += kDecodeMaxTokens) {
        const int64_t m = std::min<int64_t>(kDecodeMaxTokens, M - t0);
        const cudaError_t e = launch_decode_form(pk, static_cast<const uint8_t *>(xq) + t0 * ldx, ldx,
                                                 static_cast<uint16_t *>(y) + t0 * pk.N, m, ec, h->dec, h->status,
                                                 st, h->num_sms, kQ8, epi_rows(epi, t0, pk.N));
        if (e != cudaSuccess)
            return from_cuda(e);
    }
    return SPEAR_OK;
}

// Whether [a, a + na) and [b, b + nb) share a byte.
bool overlap(const void *a, size_t na, const void *b, size_t nb)
{
    const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
    return a && b && x < y + nb && y < x + na;
}

// Check a caller's epilogue and take it over.  mul and residual may be y
// itself (each output's operands are read by the thread that writes it, before
// it does); any other overlap with y is refused.
int take_epilogue(const spear_w4ec *h, const spear_w4ec_epilogue *ep, const void *y, int64_t M, Epilogue *out)
{
    *out = Epilogue();
    if (!ep)
        return SPEAR_OK;
    if (ep->act < SPEAR_ACT_NONE || ep->act > SPEAR_ACT_GELU_TANH || ep->reserved != 0)
        return SPEAR_ERR_INVALID;
    if (!aligned16(ep->bias) || !aligned16(ep->mul) || !aligned16(ep->residual))
        return SPEAR_ERR_INVALID;
    const size_t ny = (size_t)M * (size_t)h->pk.N * 2;
    if (overlap(ep->bias, (size_t)h->pk.N * 2, y, ny) || (ep->mul != y && overlap(ep->mul, ny, y, ny)) ||
        (ep->residual != y && overlap(ep->residual, ny, y, ny)))
        return SPEAR_ERR_INVALID;
    out->bias = static_cast<const uint16_t *>(ep->bias);
    out->mul = static_cast<const uint16_t *>(ep->mul);
    out->residual = static_cast<const uint16_t *>(ep->residual);
    out->act = ep->act;
    return SPEAR_OK;
}

// Pack (W given: symmetric or asymmetric RTN) or import (codes, s, z given)
// the layer, then the EC operands and the kernels' tensor maps.
int pack_layer(spear_w4ec *h, const void *W, const void *codes, const float *s, const uint8_t *z, const void *A,
               const void *B, const void *w_g, float b_g, void *stream, bool asym)
{
    if (!h || (W && !aligned16(W)) || (!W && !codes))
        return SPEAR_ERR_INVALID;
    if (h->pk.r > 0 && (!A || !B || !w_g))
        return SPEAR_ERR_INVALID;
    DeviceGuard guard(h->device);
    if (!guard.ok())
        return SPEAR_ERR_CUDA;
    h->pk.b_g = b_g;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    cudaError_t e = W ? launch_pack(h->pk, W, A, B, w_g, h->status, st, asym)
                      : launch_import(h->pk, codes, s, z, A, B, w_g, h->status, st);
    if (e != cudaSuccess)
        return from_cuda(e);
    e = tc_prepare(h->pk, h->tc);
    if (e == cudaSuccess)
        e = decode_prepare(h->pk, h->dec);
    if (e != cudaSuccess)
        return from_cuda(e);
    h->packed = true;
    return SPEAR_OK;
}

}  // namespace

namespace spear {

int status_of(cudaError_t e) { return from_cuda(e); }

int bucket_of(int64_t M)
{
    int b = 0;
    int64_t cap = 1;
    while (b < 8 && M > cap) {
        cap *= 2;
        ++b;
    }
    return b;  // 1,2,4,...,128 -> 0..7, >128 -> 8
}

bool path_supported(const spear_w4ec *h, uint32_t path)
{
    if (path == SPEAR_FORCE_TC)
        return tc_supported(h);
    if (path == SPEAR_FORCE_DECODE)
        return decode_supported(h->pk, h->num_sms);
    return false;
}

int forward_checked(const spear_w4ec *h, const void *x, void *y, int64_t M, uint32_t flags, cudaStream_t st)
{
    return run_forward(h, x, y, M, flags, st);
}

int forward_ep_checked(const spear_w4ec *h, const void *x, const float *xs, void *y, int64_t M, uint32_t flags,
                       cudaStream_t st, const Epilogue &epi)
{
    if (xs)
        return run_forward_q8(h, x, xs, y, M, flags, st, epi);
    // nothing after the layer: the plain forward, its EC in the product's kernel
    if (!epi.bias && !epi.mul && !epi.residual && epi.act == kActNone) {
        if (flags & SPEAR_FORCE_SPLIT)
            return SPEAR_ERR_UNSUPPORTED;
        return run_forward(h, x, y, M, flags | SPEAR_FORCE_FUSED, st);
    }
    return run_forward(h, x, y, M, flags, st, kEpi, epi);
}

}  // namespace spear

extern "C" {

const char *spear_w4ec_strerror(int status)
{
    switch (status) {
    case SPEAR_OK: return "ok";
    case SPEAR_ERR_INVALID: return "invalid argument";
    case SPEAR_ERR_UNSUPPORTED: return "unsupported shape or path";
    case SPEAR_ERR_NOMEM: return "out of memory";
    case SPEAR_ERR_CUDA: return "CUDA error";
    case SPEAR_ERR_TIMEOUT: return "device-side wait timed out";
    case SPEAR_ERR_DEVICE: return "kernel reported bad data (non-finite weights or scaled EC operand)";
    case SPEAR_ERR_STATE: return "call out of order (layer not packed)";
    default: return "unknown status";
    }
}

int spear_w4ec_create(spear_w4ec **out, int64_t K, int64_t N, int32_t r, const spear_w4ec_opts *opts)
{
    if (!out)
        return SPEAR_ERR_INVALID;
    *out = nullptr;
    if (K <= 0 || N <= 0 || K % 8 || N % 8 || r < 0 || r > 128)
        return SPEAR_ERR_INVALID;
    int dev = (opts && opts->device >= 0) ? opts->device : -1;
    if (dev < 0 && cudaGetDevice(&dev) != cudaSuccess)
        return SPEAR_ERR_CUDA;
    int ndev = 0;
    if (cudaGetDeviceCount(&ndev) != cudaSuccess || dev >= ndev)
        return SPEAR_ERR_INVALID;
    if (std::strcmp(env_fault(), "alloc") == 0)
        return SPEAR_ERR_NOMEM;
    DeviceGuard guard(dev);
    if (!guard.ok())
        return SPEAR_ERR_CUDA;

    spear_w4ec *h = new (std::nothrow) spear_w4ec();
    if (!h)
        return SPEAR_ERR_NOMEM;
    h->device = dev;
    h->max_M = (opts && opts->max_M > 0) ? opts->max_M : 4096;
    cudaDeviceGetAttribute(&h->num_sms, cudaDevAttrMultiProcessorCount, dev);
    for (auto &row : h->cost_us)
        for (float &c : row)
            c = -1.0f;
    h->fault_launch = std::strcmp(env_fault(), "launch") == 0;
    h->fault_timeout = std::strcmp(env_fault(), "timeout") == 0;

    Packed &pk = h->pk;
    pk.K = K;
    pk.N = N;
    pk.Kp = round_up(K, 256);
    pk.Np = round_up(N, 128);
    pk.r = r;
    pk.rp = r > 0 ? (int)round_up(r, 16) : 0;
    pk.R1p = r > 0 ? (int)round_up(r + 1, 16) : 0;
    pk.b_g = 0.f;

    cudaError_t e = cudaSuccess;
    auto chk = [&](cudaError_t x) {
        if (e == cudaSuccess)
            e = x;
    };
    chk(alloc_zero(&pk.codes, (size_t)pk.Np * pk.Kp / 8));
    chk(alloc_zero(&pk.s, (size_t)pk.Np));
    chk(alloc_zero(&pk.z, (size_t)pk.Np));
    if (r > 0) {
        chk(alloc_zero(&pk.G, (size_t)pk.R1p * pk.Kp));
        chk(alloc_zero(&pk.Bt, (size_t)pk.Np * pk.rp));
        chk(alloc_zero(&pk.Bts, (size_t)pk.Np * pk.rp));
        chk(alloc_zero(&h->v, (size_t)h->max_M * pk.rp));
        chk(alloc_zero(&h->gbuf, (size_t)h->max_M));
        h->pre.part_floats = prepass_part_floats(pk, h->max_M, h->num_sms);
        h->pre.n_counters = prepass_counters(h->max_M);
        chk(alloc_zero(&h->pre.part, h->pre.part_floats));
        chk(alloc_zero(&h->pre.counters, (size_t)h->pre.n_counters));
    }
    chk(alloc_zero(&h->dec.ws_u, decode_u_floats(pk)));
    chk(alloc_zero(&h->dec.flags, (size_t)kDecodeFlags));
    chk(alloc_zero(&h->dec.ws_stream, decode_stream_ws_floats(pk)));
    chk(alloc_zero(&h->dec.cnt_stream, (size_t)kDecodeStreamCounters));
    chk(tc_alloc(pk, h->max_M, h->num_sms, h->tc));
    chk(alloc_zero(&h->status, 1));
    chk(alloc_zero(&h->vready, 2));
    chk(alloc_zero(&h->rowc, rowc_floats(h->max_M)));
    if (K % 16)
        chk(alloc_zero(&h->xq_pad, (size_t)h->max_M * (size_t)(K + 8)));
    if (e == cudaSuccess)
        e = cudaDeviceSynchronize();
    if (e != cudaSuccess) {
        free_all(h);
        delete h;
        return from_cuda(e);
    }
    *out = h;
    return SPEAR_OK;
}

int spear_w4ec_pack(spear_w4ec *h, const void *W, const void *A, const void *B, const void *w_g, float b_g,
                    void *stream)
{
    return pack_layer(h, W, nullptr, nullptr, nullptr, A, B, w_g, b_g, stream, false);
}

int spear_w4ec_pack_asym(spear_w4ec *h, const void *W, const void *A, const void *B, const void *w_g, float b_g,
                         void *stream)
{
    return pack_layer(h, W, nullptr, nullptr, nullptr, A, B, w_g, b_g, stream, true);
}

int spear_w4ec_import(spear_w4ec *h, const void *codes, const float *s, const uint8_t *z, const void *A,
                      const void *B, const void *w_g, float b_g, void *stream)
{
    if (!codes || !s || !z)
        return SPEAR_ERR_INVALID;
    return pack_layer(h, nullptr, codes, s, z, A, B, w_g, b_g, stream, false);
}

int spear_w4ec_forward(const spear_w4ec *h, const void *x, void *y, int64_t M, uint32_t flags, void *stream)
{
    if (!h || M < 0)
        return SPEAR_ERR_INVALID;
    if (M == 0)
        return SPEAR_OK;
    if (!h->packed)
        return SPEAR_ERR_STATE;
    if (M > h->max_M || !x || !y || !aligned16(x) || !aligned16(y))
        return SPEAR_ERR_INVALID;
    DeviceGuard guard(h->device);
    if (!guard.ok())
        return SPEAR_ERR_CUDA;
    return run_forward(h, x, y, M, flags, static_cast<cudaStream_t>(stream));
}

int spear_w4ec_forward_ep(const spear_w4ec *h, const void *x, void *y, int64_t M, const spear_w4ec_epilogue *ep,
                          uint32_t flags, void *stream)
{
    if (!h || M < 0)
        return SPEAR_ERR_INVALID;
    if (M == 0)
        return SPEAR_OK;
    if (!h->packed)
        return SPEAR_ERR_STATE;
    if (M > h->max_M || !x || !y || !aligned16(x) || !aligned16(y) ||
        overlap(x, (size_t)M * (size_t)h->pk.K * 2, y, (size_t)M * (size_t)h->pk.N * 2))
        return SPEAR_ERR_INVALID;
    Epilogue epi;
    const int rc = take_epilogue(h, ep, y, M, &epi);
    if (rc != SPEAR_OK)
        return rc;
    DeviceGuard guard(h->device);
    if (!guard.ok())
        return SPEAR_ERR_CUDA;
    return guarded(
        [&] { return forward_ep_checked(h, x, nullptr, y, M, flags, static_cast<cudaStream_t>(stream), epi); });
}

int spear_w4ec_forward_q8(const spear_w4ec *h, const void *xq, const float *xs, void *y, int64_t M,
                          const spear_w4ec_epilogue *ep, uint32_t flags, void *stream)
{
    if (!h || M < 0)
        return SPEAR_ERR_INVALID;
    if (M == 0)
        return SPEAR_OK;
    if (!h->packed)
        return SPEAR_ERR_STATE;
    const size_t ny = (size_t)M * (size_t)h->pk.N * 2;
    if (M > h->max_M || !xq || !xs || !y || !aligned16(xq) || !aligned16(y) ||
        (reinterpret_cast<uintptr_t>(xs) & 3u) != 0 || overlap(xq, (size_t)M * (size_t)h->pk.K, y, ny) ||
        overlap(xs, (size_t)M * 4, y, ny))
        return SPEAR_ERR_INVALID;
    Epilogue epi;
    const int rc = take_epilogue(h, ep, y, M, &epi);
    if (rc != SPEAR_OK)
        return rc;
    DeviceGuard guard(h->device);
    if (!guard.ok())
        return SPEAR_ERR_CUDA;
    return guarded(
        [&] { return forward_ep_checked(h, xq, xs, y, M, flags, static_cast<cudaStream_t>(stream), epi); });
}

int spear_w4ec_forward_host(spear_w4ec *h, const void *x_host, void *y_host, int64_t M, uint32_t flags,
                            void *stream)
{
    if (!h || M < 0)
        return SPEAR_ERR_INVALID;
    if (M == 0)
        return SPEAR_OK;
    if (!h->packed)
        return SPEAR_ERR_STATE;
    if (M > h->max_M || !x_host || !y_host)
        return SPEAR_ERR_INVALID;
    DeviceGuard guard(h->device);
    if (!guard.ok())
        return SPEAR_ERR_CUDA;
    cudaError_t e = cudaSuccess;
    if (!h->x_stage) {
        e = cudaMalloc(&h->x_stage, (size_t)h->max_M * h->pk.K * 2);
        if (e == cudaSuccess)
            e = cudaMalloc(&h->y_stage, (size_t)h->max_M * h->pk.N * 2);
        if (e != cudaSuccess) {
            cudaFree(h->x_stage);
            h->x_stage = nullptr;
            h->y_stage = nullptr;
            return from_cuda(e);
        }
    }
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    e = cudaMemcpyAsync(h->x_stage, x_host, (size_t)M * h->pk.K * 2, cudaMemcpyHostToDevice, st);
    if (e != cudaSuccess)
        return from_cuda(e);
    int rc = run_forward(h, h->x_stage, h->y_stage, M, flags, st);
    if (rc != SPEAR_OK)
        return rc;
    e = cudaMemcpyAsync(y_host, h->y_stage, (size_t)M * h->pk.N * 2, cudaMemcpyDeviceToHost, st);
    if (e == cudaSuccess)
        e = cudaStreamSynchronize(st);
    return from_cuda(e);
}

int spear_w4ec_destroy(spear_w4ec *h)
{
    if (!h)
        return SPEAR_OK;
    DeviceGuard guard(h->device);
    cudaDeviceSynchronize();
    // no handle may go on prefetching this one's memory
    for (spear_w4ec *p : h->prev)
        if (p != h) {
            p->next = nullptr;
            p->dec.pf = nullptr;
            p->dec.pf_bytes = 0;
        }
    if (h->next && h->next != h) {
        auto &v = h->next->prev;
        v.erase(std::remove(v.begin(), v.end(), h), v.end());
    }
    free_all(h);
    delete h;
    return SPEAR_OK;
}

int spear_w4ec_set_next(spear_w4ec *h, spear_w4ec *next)
{
    if (!h || (next && next->device != h->device))
        return SPEAR_ERR_INVALID;
    if (h->next) {
        auto &v = h->next->prev;
        v.erase(std::remove(v.begin(), v.end(), h), v.end());
    }
    h->next = next;
    h->dec.pf = nullptr;
    h->dec.pf_bytes = 0;
    if (next) {
        next->prev.push_back(h);
        h->dec.pf = next->pk.codes;
        h->dec.pf_bytes = (size_t)next->pk.Np * (size_t)next->pk.Kp / 2;
    }
    return SPEAR_OK;
}

int spear_w4ec_get_packed(const spear_w4ec *h, void *codes, float *s, uint8_t *z, void *stream)
{
    if (!h)
        return SPEAR_ERR_INVALID;
    if (!h->packed)
        return SPEAR_ERR_STATE;
    DeviceGuard guard(h->device);
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    const Packed &pk = h->pk;
    cudaError_t e = cudaSuccess;
    if (codes)
        e = launch_untile_codes(pk, static_cast<uint32_t *>(codes), st);
    if (e == cudaSuccess && s)
        e = cudaMemcpyAsync(s, pk.s, (size_t)pk.N * sizeof(float), cudaMemcpyDeviceToDevice, st);
    if (e == cudaSuccess && z)
        e = cudaMemcpyAsync(z, pk.z, (size_t)pk.N, cudaMemcpyDeviceToDevice, st);
    return from_cuda(e);
}

int spear_w4ec_get_gate(const spear_w4ec *h, const void *x, float *g, int64_t M, void *stream)
{
    if (!h || M < 0 || !x || !g || !aligned16(x))
        return SPEAR_ERR_INVALID;
    if (h->pk.r == 0)
        return SPEAR_ERR_UNSUPPORTED;
    if (!h->packed)
        return SPEAR_ERR_STATE;
    if (M > h->max_M)
        return SPEAR_ERR_INVALID;
    if (M == 0)
        return SPEAR_OK;
    DeviceGuard guard(h->device);
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    cudaError_t e = run_prepass(h, x, M, false, st);
    if (e == cudaSuccess)
        e = cudaMemcpyAsync(g, h->gbuf, (size_t)M * sizeof(float), cudaMemcpyDeviceToDevice, st);
    return from_cuda(e);
}

int spear_w4ec_sync_status(spear_w4ec *h, void *stream)
{
    if (!h)
        return SPEAR_ERR_INVALID;
    DeviceGuard guard(h->device);
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    int bits = 0;
    cudaError_t e = cudaStreamSynchronize(st);
    if (e == cudaSuccess)
        e = cudaMemcpy(&bits, h->status, sizeof(int), cudaMemcpyDeviceToHost);
    if (e == cudaSuccess && bits)
        e = cudaMemset(h->status, 0, sizeof(int));
    if (e != cudaSuccess)
        return from_cuda(e);
    if (bits & kStatusTimeout)
        return SPEAR_ERR_TIMEOUT;
    if (bits & kStatusNonFinite)
        return SPEAR_ERR_DEVICE;
    return SPEAR_OK;
}

int spear_w4ec_dispatch(const spear_w4ec *h, int64_t M, uint32_t *choice)
{
    if (!h || M < 0 || !choice)
        return SPEAR_ERR_INVALID;
    *choice = resolve(h, M, 0);
    return SPEAR_OK;
}

int spear_w4ec_tune(spear_w4ec *h, const void *x, void *y, int64_t M, void *stream, uint32_t *choice)
{
    if (!h || M <= 0 || !x || !y || !aligned16(x) || !aligned16(y))
        return SPEAR_ERR_INVALID;
    if (!h->packed)
        return SPEAR_ERR_STATE;
    if (M > h->max_M)
        return SPEAR_ERR_INVALID;
    DeviceGuard guard(h->device);
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    // every legal choice with the EC (fused and split), and each path with the EC off
    std::vector<uint32_t> cands;
    const uint32_t paths[2] = {SPEAR_FORCE_DECODE, SPEAR_FORCE_TC};
    for (uint32_t path : paths) {
        if (!path_supported(h, path))
            continue;
        cands.push_back(path | SPEAR_FORCE_FUSED);
        if (h->pk.r > 0) {
            cands.push_back(path | SPEAR_FORCE_SPLIT);
            cands.push_back(path | SPEAR_FORCE_FUSED | SPEAR_EC_OFF);
        }
    }
    cudaEvent_t e0, e1;
    if (cudaEventCreate(&e0) != cudaSuccess)
        return SPEAR_ERR_CUDA;
    if (cudaEventCreate(&e1) != cudaSuccess) {
        cudaEventDestroy(e0);
        return SPEAR_ERR_CUDA;
    }
    const int b = bucket_of(M);
    float best_ms = 1e30f;
    uint32_t best = 0;
    int rc = SPEAR_OK;
    for (uint32_t cand : cands) {
        for (int i = 0; i < 3 && rc == SPEAR_OK; ++i)
            rc = run_forward(h, x, y, M, cand, st);
        if (rc != SPEAR_OK)
            break;
        std::vector<float> times;
        for (int i = 0; i < 9 && rc == SPEAR_OK; ++i) {
            cudaEventRecord(e0, st);
            rc = run_forward(h, x, y, M, cand, st);
            cudaEventRecord(e1, st);
            cudaEventSynchronize(e1);
            float ms = 0.f;
            cudaEventElapsedTime(&ms, e0, e1);
            times.push_back(ms);
        }
        if (rc != SPEAR_OK)
            break;
        std::sort(times.begin(), times.end());
        const float med = times[times.size() / 2];
        h->cost_us[b][cost_index(cand)] = med * 1000.0f;
        if (cand & SPEAR_EC_OFF) {
            h->cost_us[b][cost_index(cand | SPEAR_FORCE_SPLIT)] = med * 1000.0f;
            continue;   // a time without the EC, for the cost model only
        }
        if (med < best_ms) {
            best_ms = med;
            best = cand;
        }
    }
    cudaEventDestroy(e0);
    cudaEventDestroy(e1);
    if (rc != SPEAR_OK)
        return rc;
    h->table[bucket_of(M)] = best;
    if (choice)
        *choice = best;
    return from_cuda(cudaStreamSynchronize(st));
}

}  // extern "C"

namespace spear {

cudaError_t raise_smem_limit(const void *func, size_t bytes)
{
    struct Entry {
        const void *func;
        int device;
        size_t bytes;
    };
    static std::vector<Entry> done;
    static std::mutex mu;
    int dev = 0;
    cudaGetDevice(&dev);
    std::lock_guard<std::mutex> lock(mu);
    for (const Entry &e : done)
        if (e.func == func && e.device == dev && e.bytes >= bytes)
            return cudaSuccess;
    cudaError_t e = cudaFuncSetAttribute(func, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)bytes);
    if (e == cudaSuccess)
        done.push_back({func, dev, bytes});
    return e;
}

}  // namespace spear
