// What the tcgen05 form of the 8-bit forward needs of each token before its
// epilogue: the token's scale and code sum, and with the Error Compensator the
// gated down-projection.
//
//   X_t = sum_k xq[t,k]                     rowc: 2^9 xs[t] and 2^-9 X_t
//   u   = xq[t,:] . [w_g, A]                (of the codes; xs[t] times it is the layer's)
//   g_t = 1 / (1 + exp(-(xs[t] u_0 + b_g)))
//   v   = 2^-9 g_t u_j, rounded to tf32     [M][rp]
//
// The GEMM multiplies the 4-bit codes as 2^-9 q and leaves the zero point to
// its epilogue, hence X_t and the factor 2^-9 (a power of two: exact) of v.
//
// One CTA takes 16 tokens and a 1/S share of K; four warps each take every
// fourth 64-k block.  e4m3 activations are made bf16 in registers (exact) for
// mma.sync against the rows of G; one more MMA against a constant tile of ones
// gives X_t.  The S partials are summed in split order by the CTA that arrives
// last (no floating-point atomics: run-to-run identical).
#include <algorithm>

#include "async_utils.cuh"
#include "kernels.h"
#include "tc_gemm.h"

namespace spear {
namespace {

constexpr int kTok = 16;
constexpr int kMaxSplits = 32;

struct PrepassQ8Params {
    const uint16_t *G;      // [R1p][Kp]
    const uint8_t *x;       // e4m3, rows ldx apart
    int64_t ldx;
    const float *xs;
    int64_t M, K, Kp;
    int R1p, r, rp;
    float b_g;
    int S, bps;             // splits of K, 64-k blocks a split
    float *v;
    float *rowc;
    float *part;            // [tiles][S][(R1p + 1) x 16]
    unsigned *counters;     // [tiles], zero between calls
    unsigned *ready;        // counted (release) once per token tile; null for none
};

// MT 16-row groups of G (0: the code sums alone).
template <int MT>
__global__ void __launch_bounds__(128) prepass_q8_kernel(PrepassQ8Params p)
{
    pdl_wait();   // x is written by the previous kernel in the stream
    pdl_launch_dependents();   // (a tcgen05 kernel that starts early reads x without waiting)
    extern __shared__ float4 smem_f4[];
    float *red = reinterpret_cast<float *>(smem_f4);   // [4][R1p + 1][16]
    __shared__ int s_last;

    constexpr int kRowsG = 16 * MT;
    constexpr int kElems = (kRowsG + 1) * kTok;        // rows of G, then X
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, gid = lane >> 2, c = lane & 3;
    const int tile = blockIdx.x / p.S, ks = blockIdx.x - tile * p.S;
    const int64_t t0 = (int64_t)tile * kTok;
    const int nkb = (int)(p.Kp / 64);
    const int kb0 = ks * p.bps, kb1 = min(kb0 + p.bps, nkb);

    float acc[MT > 0 ? MT : 1][2][4], ax[2][4];
#pragma unroll
    for (int n = 0; n < 2; ++n)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            ax[n][i] = 0.f;
#pragma unroll
            for (int m = 0; m < MT; ++m)
                acc[m][n][i] = 0.f;
        }
    constexpr uint32_t kOnes = 0x3F803F80u;

    for (int kb = kb0 + warp; kb < kb1; kb += 4) {
        const int64_t k = (int64_t)kb * 64 + 16 * c;
        uint32_t xb[2][8];
#pragma unroll
        for (int n = 0; n < 2; ++n) {
            const int64_t t = t0 + 8 * n + gid;
            // (rows are padded to a multiple of 16, with zeros)
            const uint4 a = t < p.M && k < p.K ? __ldg(reinterpret_cast<const uint4 *>(p.x + t * p.ldx + k))
                                               : make_uint4(0u, 0u, 0u, 0u);
            const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                xb[n][2 * i] = f16x2_to_bf16x2(e4m3x2_to_f16x2((uint16_t)w[i]));
                xb[n][2 * i + 1] = f16x2_to_bf16x2(e4m3x2_to_f16x2((uint16_t)(w[i] >> 16)));
            }
        }
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int n = 0; n < 2; ++n)
                mma_bf16_16816(ax[n], kOnes, kOnes, kOnes, kOnes, xb[n][2 * i], xb[n][2 * i + 1]);
#pragma unroll
        for (int m = 0; m < MT; ++m) {
            const uint16_t *g0 = p.G + (int64_t)(16 * m + gid) * p.Kp + k;
            const uint16_t *g1 = g0 + 8 * p.Kp;
            const uint4 a0 = ld_nc(g0), a1 = ld_nc(g0 + 8), h0 = ld_nc(g1), h1 = ld_nc(g1 + 8);
            const uint32_t ga[8] = {a0.x, a0.y, a0.z, a0.w, a1.x, a1.y, a1.z, a1.w};
            const uint32_t ha[8] = {h0.x, h0.y, h0.z, h0.w, h1.x, h1.y, h1.z, h1.w};
            // step i covers k = 16c + 4i + {0,1} (first pair) and + {2,3} (second pair)
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int n = 0; n < 2; ++n)
                    mma_bf16_16816(acc[m][n], ga[2 * i], ha[2 * i], ga[2 * i + 1], ha[2 * i + 1], xb[n][2 * i],
                                   xb[n][2 * i + 1]);
        }
    }

    // the four warps' partial tiles, in warp order
    float *base = red + warp * kElems;
#pragma unroll
    for (int n = 0; n < 2; ++n) {
        const int col = 8 * n + 2 * c;
#pragma unroll
        for (int m = 0; m < MT; ++m) {
            const int r0 = 16 * m + gid;
            base[r0 * kTok + col] = acc[m][n][0];
            base[r0 * kTok + col + 1] = acc[m][n][1];
            base[(r0 + 8) * kTok + col] = acc[m][n][2];
            base[(r0 + 8) * kTok + col + 1] = acc[m][n][3];
        }
        if (gid == 0) {   // every row of the ones' product is X
            base[kRowsG * kTok + col] = ax[n][0];
            base[kRowsG * kTok + col + 1] = ax[n][1];
        }
    }
    __syncthreads();
    for (int e = tid; e < kElems; e += 128)
        red[e] = red[e] + red[kElems + e] + red[2 * kElems + e] + red[3 * kElems + e];
    __syncthreads();

    if (p.S > 1) {
        float *mine = p.part + ((size_t)tile * p.S + ks) * kElems;
        for (int e = tid; e < kElems; e += 128)
            mine[e] = red[e];
        __threadfence();
        __syncthreads();
        if (tid == 0)
            s_last = atomicAdd(&p.counters[tile], 1u) == (unsigned)(p.S - 1) ? 1 : 0;
        __syncthreads();
        if (!s_last)
            return;
        __threadfence();
        const float *src = p.part + (size_t)tile * p.S * kElems;
        for (int e = tid; e < kElems; e += 128) {
            float sum = 0.f;
            for (int q0 = 0; q0 < p.S; q0 += 8) {
                float w[8];
#pragma unroll
                for (int q = 0; q < 8; ++q)
                    w[q] = q0 + q < p.S ? __ldcg(src + (size_t)(q0 + q) * kElems + e) : 0.f;
#pragma unroll
                for (int q = 0; q < 8; ++q)
                    sum += w[q];
            }
            red[e] = sum;
        }
        if (tid == 0)
            p.counters[tile] = 0u;
        __syncthreads();
    }

    __shared__ float s_gate[kTok];
    if (tid < kTok && t0 + tid < p.M) {
        const float xs = __ldg(p.xs + t0 + tid);
        p.rowc[rowc_at(t0 + tid)] = 512.0f * xs;
        p.rowc[rowc_at(t0 + tid) + 2] = red[kRowsG * kTok + tid] * (1.0f / 512.0f);
        if (MT > 0)
            s_gate[tid] = 1.0f / (1.0f + expf(-(xs * red[tid] + p.b_g)));
    }
    __syncthreads();
    if constexpr (MT > 0)
        for (int e = tid; e < kTok * p.rp; e += 128) {
            const int tt = e / p.rp, j = e - tt * p.rp;
            if (t0 + tt < p.M)
                p.v[(t0 + tt) * p.rp + j] =
                    j < p.r ? to_tf32((1.0f / 512.0f) * s_gate[tt] * red[(1 + j) * kTok + tt]) : 0.f;
        }
    if (p.ready) {
        __syncthreads();
        if (tid == 0)
            red_release_gpu_add(p.ready, 1u);   // this tile's v and rowc are written
    }
}

int pick_splits(int64_t M, int64_t Kp, int num_sms)
{
    const int64_t tiles = (M + kTok - 1) / kTok;
    const int nkb = (int)(Kp / 64);
    const int S = (int)std::max<int64_t>(1, (2 * num_sms) / tiles);
    return std::min({S, std::max(1, nkb / 4), kMaxSplits});   // at least one k block a warp
}

using PrepassQ8Fn = void (*)(PrepassQ8Params);
PrepassQ8Fn prepass_q8_fn(int MT)
{
    switch (MT) {
    case 0: return prepass_q8_kernel<0>;
    case 1: return prepass_q8_kernel<1>;
    case 2: return prepass_q8_kernel<2>;
    case 3: return prepass_q8_kernel<3>;
    case 4: return prepass_q8_kernel<4>;
    case 5: return prepass_q8_kernel<5>;
    case 6: return prepass_q8_kernel<6>;
    case 7: return prepass_q8_kernel<7>;
    case 8: return prepass_q8_kernel<8>;
    case 9: return prepass_q8_kernel<9>;
    default: return nullptr;
    }
}

size_t part_floats(const Packed &pk, int64_t M, int num_sms)
{
    const int S = pick_splits(M, pk.Kp, num_sms);
    return S > 1 ? (size_t)((M + kTok - 1) / kTok) * S * (pk.R1p + 1) * kTok : 0;
}

}  // namespace

cudaError_t prepass_q8_alloc(const Packed &pk, int64_t max_M, int num_sms, PrepassQ8Work &w)
{
    const int64_t tiles = (max_M + kTok - 1) / kTok;
    size_t worst = 0;
    // a split needs two CTAs a tile at most 2 num_sms in all: fewer tiles than SMs
    for (int64_t i = 1; i <= std::min<int64_t>(tiles, num_sms); ++i)
        worst = std::max(worst, part_floats(pk, i * kTok, num_sms));
    w.part_floats = worst;
    w.n_counters = (int)tiles;
    // whole chunks of 32 tokens, zero where no token is (a copy of a chunk reads all of it)
    const size_t rowc_bytes = (size_t)((max_M + 31) / 32 * 32) * 2 * sizeof(float);
    cudaError_t e = cudaMalloc(&w.rowc, rowc_bytes);
    if (e == cudaSuccess)
        e = cudaMemset(w.rowc, 0, rowc_bytes);
    if (e == cudaSuccess && worst)
        e = cudaMalloc(&w.part, worst * sizeof(float));
    if (e == cudaSuccess)
        e = cudaMalloc(&w.counters, (size_t)tiles * sizeof(unsigned));
    if (e == cudaSuccess)
        e = cudaMemset(w.counters, 0, (size_t)tiles * sizeof(unsigned));
    return e;
}

void prepass_q8_free(PrepassQ8Work &w)
{
    cudaFree(w.rowc);
    cudaFree(w.part);
    cudaFree(w.counters);
    w = PrepassQ8Work();
}

cudaError_t launch_prepass_q8(const Packed &pk, const void *xq, int64_t ldx, const float *xs, int64_t M, bool ec,
                              float *v, const PrepassQ8Work &w, cudaStream_t st, int num_sms, unsigned *ready,
                              unsigned *expected)
{
    PrepassQ8Params p = {};
    p.G = pk.G;
    p.x = static_cast<const uint8_t *>(xq);
    p.ldx = ldx;
    p.xs = xs;
    p.M = M;
    p.K = pk.K;
    p.Kp = pk.Kp;
    p.R1p = ec ? pk.R1p : 0;
    p.r = pk.r;
    p.rp = pk.rp;
    p.b_g = pk.b_g;
    const int nkb = (int)(pk.Kp / 64);
    p.S = pick_splits(M, pk.Kp, num_sms);
    p.bps = (nkb + p.S - 1) / p.S;
    p.S = (nkb + p.bps - 1) / p.bps;   // no empty split
    p.v = v;
    p.rowc = w.rowc;
    p.part = w.part;
    p.counters = w.counters;
    p.ready = ready;
    const int64_t tiles = (M + kTok - 1) / kTok;
    if (expected)
        *expected = (unsigned)tiles;
    const size_t elems = (size_t)(p.R1p + 1) * kTok;
    if (tiles > w.n_counters || (p.S > 1 && (size_t)tiles * p.S * elems > w.part_floats))
        return cudaErrorInvalidValue;
    const PrepassQ8Fn fn = prepass_q8_fn(p.R1p / 16);
    if (!fn)
        return cudaErrorInvalidValue;
    const size_t smem = 4 * elems * sizeof(float);
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(tiles * p.S));
    cfg.blockDim = dim3(128);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, fn, p);
}

}  // namespace spear
