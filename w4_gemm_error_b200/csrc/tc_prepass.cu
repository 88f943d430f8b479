// Gate and EC down-projection of many tokens on the tensor cores, K split over
// a cluster: what the forms kEpi and kQ8 of the forward pass need of each token
// before their epilogue (see prepass.cu for g and v).
//
//   D[t, j] = x[t,:] . G[j,:],  G = [w_g; A^T] (R1p rows)
//   kEpi: v = g D[t,1+j],         g = 1 / (1 + exp(-(D[t,0] + b_g)))
//   kQ8:  v = 2^-9 g D[t,1+j],    g = 1 / (1 + exp(-(xs[t] D[t,0] + b_g))),
//         rowc: xs[t] and 2^-9 X_t,  X_t = sum_k xq[t,k]
//   (v rounded to tf32, half a unit of 2^-10: the correction enters the product's
//   accumulator by tf32 MMAs, and is small beside the product)
//
// A cluster of S CTAs takes 128 tokens; CTA q the 64-k blocks q, q + S, ...
// The tokens are the 128 rows (TMEM lanes) of the MMA and the rows of G its N.
// One CTA a tile leaves most SMs idle (16 of them work at 2048 tokens of K = 4096,
// 29 us alone and cold; S = 8 there: 14 us).  The loop runs at about 540 cycles a
// 64-k block (630 with the copies issued from a single lane's branch); at few
// tokens the exchange and what surrounds it take as long.
// (As first CTAs of tc_tile.cu's grid, their partials exchanged through global
// memory, the same work took longer by three more trips to L2: 33 tokens of
// 256 x 256 in 12.5 us instead of 9.2.)
// e4m3 activations are made bf16 on their way from the copied tile to the MMA's
// (exact), and sixteen rows of ones behind those of G make X_t one more column of
// D; a NaN code is a number here, but the product beside it is NaN.  The S partial
// accumulators meet in shared memory: CTA q sums its 128 / S tokens over the
// cluster in rank order (run-to-run identical), forms the gate and writes v.
#include <algorithm>

#include "async_utils.cuh"
#include "epilogue.cuh"
#include "tc_gemm.h"
#include "tensor_map.h"

namespace spear {
namespace {

constexpr int kTok = 128;
constexpr int kMaxStages = 8;
// Warps 2-17: two groups of eight, converting every second block (kQ8), then all
// reading the accumulator.  The ring has an even number of stages, so that a
// stage always belongs to one group: a group that skipped a phase of a barrier
// could take the phase before it, of the same parity, for its own.
constexpr int kGroups = 2;
constexpr int kThreads = 64 + 256 * kGroups;
constexpr int kMaxCluster = 8;
constexpr int kOnesRows = 16;      // kQ8: rows of ones after those of G, whose product is X_t

struct TcPrepass2Params {
    int64_t M;
    int n_k;              // 64-k blocks
    int S;                // CTAs a cluster
    int stages;
    int R1p, r, rp;
    float b_g;
    const float *xs;      // kQ8
    float *v;             // [M][rp]; null without the EC (kQ8: the code sums alone)
    float *rowc;          // kQ8
    int *status;
    unsigned *ready;      // counted (release) once per CTA; null for none
};

template <int FORM>
__host__ __device__ constexpr uint32_t xin_bytes() { return FORM == kQ8 ? kTok * 64 : 0; }

// Columns of D: the rows of G, then (kQ8) those of ones.
template <int FORM>
__host__ __device__ inline int columns(int R1p)
{
    return R1p + (FORM == kQ8 ? kOnesRows : 0);
}
// Stage: the MMA's tile of x (16 KB), the copied e4m3 tile (kQ8), the rows of G
// (and of ones).
template <int FORM>
__host__ __device__ inline uint32_t stage_bytes(int R1p)
{
    return kTok * 128 + xin_bytes<FORM>() + (((uint32_t)columns<FORM>(R1p) * 128 + 1023u) & ~1023u);
}

template <int FORM>
__global__ void __launch_bounds__(kThreads, 1)
tc_prepass2_kernel(const __grid_constant__ CUtensorMap tm_x, const __grid_constant__ CUtensorMap tm_g,
                   TcPrepass2Params p)
{
    extern __shared__ uint8_t smem_raw[];
    // copied, staged (converted) and empty of each stage; accumulator done; drain
    __shared__ __align__(8) uint64_t bars[3 * kMaxStages + 2];
    __shared__ uint32_t tmem_base_slot;
    __shared__ volatile int abort_flag;
    __shared__ float s_gate[kTok];

    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const uint32_t base = (smem_addr(smem_raw) + 1023u) & ~1023u;
    uint8_t *const bp = smem_raw + (base - smem_addr(smem_raw));
    const uint32_t full0 = smem_addr(&bars[0]), staged0 = smem_addr(&bars[kMaxStages]);
    const uint32_t empty0 = smem_addr(&bars[2 * kMaxStages]);
    const uint32_t done = smem_addr(&bars[3 * kMaxStages]), drain = smem_addr(&bars[3 * kMaxStages + 1]);
    const uint32_t g_bytes = (uint32_t)p.R1p * 128, sbytes = stage_bytes<FORM>(p.R1p);
    constexpr uint32_t kXin = kTok * 128;                 // offset of the copied e4m3 tile
    const uint32_t o_g = kTok * 128 + xin_bytes<FORM>();  // offset of the rows of G
    const int kStages = p.stages;
    const int ncol = columns<FORM>(p.R1p);
    const int S = p.S, rank = S > 1 ? (int)cluster_ctarank() : 0;
    const int t0 = (int)(blockIdx.x / S) * kTok;
    const int nkb = (p.n_k - rank + S - 1) / S;   // this CTA's blocks (at least one)
    const bool ec = p.R1p > 0;
    uint32_t tmem_cols = 32;
    while (tmem_cols < (uint32_t)ncol)
        tmem_cols <<= 1;

    if (tid == 0) {
        abort_flag = 0;
        for (int s = 0; s < kStages; ++s) {
            mbar_init(full0 + 8 * s, 1);
            mbar_init(staged0 + 8 * s, 8);
            mbar_init(empty0 + 8 * s, 1);
        }
        mbar_init(done, 1);
        mbar_init(drain, 1);
        fence_mbarrier_init_cluster();
    }
    if (warp == 1) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                         smem_addr(&tmem_base_slot)),
                     "r"(tmem_cols)
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    }
    // the rows of G do not depend on earlier kernels: on their way to L2 now
    if (ec && warp == 0)
        for (int i = lane; i < nkb; i += 32)
            tma_prefetch_2d(&tm_g, (rank + i * S) * 64, 0);
    if constexpr (FORM == kQ8) {
        // the rows of ones of every stage, once (any order of a row will do)
        for (int i = tid; i < kStages * kOnesRows * 8; i += kThreads) {
            const int s = i / (kOnesRows * 8), e = i - s * (kOnesRows * 8);
            *reinterpret_cast<uint4 *>(bp + s * sbytes + o_g + g_bytes + e * 16) =
                make_uint4(0x3F803F80u, 0x3F803F80u, 0x3F803F80u, 0x3F803F80u);
        }
        fence_proxy_async_smem();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = tmem_base_slot;
    pdl_wait();   // x and xs come from earlier kernels in the stream
    // the next kernel may start: x is complete (it may read x without waiting)
    // and this CTA holds its tensor memory
    pdl_launch_dependents();

    const int q = warp & 3, row = 32 * q + lane;   // warps 2 and up: TMEM lane = token of the tile
    if (warp == 0) {
        const bool elected = elect_one();
        uint32_t slot = 0, phase = 0;
        int issued = 0;
        for (int i = 0; i < nkb; ++i, ++issued) {
            if (!warp_wait(empty0 + 8 * slot, phase ^ 1, &abort_flag, p.status))
                break;
            const uint32_t sb = base + slot * sbytes, full = full0 + 8 * slot;
            const int k = (rank + i * S) * 64;
            if (elected) {
                mbar_expect_tx(full, (FORM == kQ8 ? xin_bytes<FORM>() : kTok * 128) + g_bytes);
                tma_load_2d(FORM == kQ8 ? sb + kXin : sb, &tm_x, k, t0, full);
                if (ec)
                    tma_load_2d(sb + o_g, &tm_g, k, 0, full);
            }
            if ((int)++slot == kStages) {
                slot = 0;
                phase ^= 1;
            }
        }
        if (abort_flag)
            for (int j = 0; j < kStages && j < issued; ++j) {
                const int i = issued - 1 - j;
                mbar_wait_final(full0 + 8 * (i % kStages), (i / kStages) & 1);
            }
    } else if (warp == 1) {
        const bool elected = elect_one();
        const uint32_t idesc = (1u << 4) | (1u << 7) | (1u << 10) | ((uint32_t)(ncol >> 3) << 17) |
                               ((uint32_t)(kTok >> 4) << 24);
        const uint64_t a0 = smem_desc_sw128(base), b0 = smem_desc_sw128(base + o_g);
        uint32_t slot = 0, phase = 0;
        bool ok = true;
        for (int i = 0; i < nkb; ++i) {
            if (!warp_wait((FORM == kQ8 ? staged0 : full0) + 8 * slot, phase, &abort_flag, p.status)) {
                ok = false;
                break;
            }
            tc_fence_after();
            const uint64_t a_desc = a0 + slot * (sbytes >> 4), b_desc = b0 + slot * (sbytes >> 4);
            if (elected) {
#pragma unroll
                for (int k = 0; k < 4; ++k)
                    mma_bf16(tmem, a_desc + 2 * k, b_desc + 2 * k, idesc, (i > 0 || k > 0) ? 1u : 0u);
                mma_commit(empty0 + 8 * slot);
            }
            __syncwarp();
            if ((int)++slot == kStages) {
                slot = 0;
                phase ^= 1;
            }
        }
        if (elected) {
            if (ok)
                mma_commit(done);
            mma_commit(drain);
        }
        __syncwarp();
        mbar_wait_final(drain, 0);
    } else if (FORM == kQ8) {
        // e4m3 -> bf16: half of one token's 64 k a thread
        const int grp = (warp - 2) >> 3, half = ((warp - 2) >> 2) & 1;
        int slot = grp;   // (the ring has at least two stages)
        uint32_t phase = 0;
        for (int i = grp; i < nkb; i += kGroups) {
            if (!warp_wait(full0 + 8 * slot, phase, &abort_flag, p.status))
                break;
            uint8_t *const sb = bp + slot * sbytes;
            const uint8_t *src = sb + kXin + row * 64;
            uint8_t *dst = sb + row * 128;
#pragma unroll
            for (int c = 2 * half; c < 2 * half + 2; ++c) {
                const uint4 w = *reinterpret_cast<const uint4 *>(src + ((c ^ ((row >> 1) & 3)) << 4));
                const uint32_t words[4] = {w.x, w.y, w.z, w.w};
                uint32_t o[8];
#pragma unroll
                for (int h = 0; h < 4; ++h)
                    e4m3x4_to_bf16(words[h], o[2 * h], o[2 * h + 1]);
                *reinterpret_cast<uint4 *>(dst + (((2 * c) ^ (row & 7)) << 4)) = make_uint4(o[0], o[1], o[2], o[3]);
                *reinterpret_cast<uint4 *>(dst + (((2 * c + 1) ^ (row & 7)) << 4)) = make_uint4(o[4], o[5], o[6], o[7]);
            }
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0)
                mbar_arrive(staged0 + 8 * slot);
            slot += kGroups;
            if (slot >= kStages) {   // (an even ring: back to this group's first)
                slot -= kStages;
                phase ^= 1;
            }
        }
    }

    // ---- this CTA's partial: [token][R1p columns of D, X], rows of whole 16 bytes
    const int ld = p.R1p + 4;
    const bool reader = warp >= 2;   // quarter q: the tokens 32 q ..; four warps a quarter, columns 16 at a time
    float *const part = reinterpret_cast<float *>(bp);
    const bool got = !reader || mbar_wait(done, 0, &abort_flag, p.status);
    __syncthreads();   // every copy and MMA of this CTA is over: the stages are free
    if (reader) {
        tc_fence_after();
        __syncwarp();
        for (int c = 16 * ((warp - 2) >> 2); c < ncol; c += 64) {
            uint32_t a[16];
            tmem_ld_32x32b_x16(tmem + ((uint32_t)(32 * q) << 16) + c, a);
#pragma unroll
            for (int j = 0; j < 16; j += 4)
                if (c + j < ld)   // (a few columns of the ones)
                    *reinterpret_cast<float4 *>(part + row * ld + c + j) =
                        got ? make_float4(__uint_as_float(a[j]), __uint_as_float(a[j + 1]), __uint_as_float(a[j + 2]),
                                          __uint_as_float(a[j + 3]))
                            : make_float4(0.f, 0.f, 0.f, 0.f);
        }
    }
    if (S > 1)
        cluster_sync();
    else
        __syncthreads();

    // ---- the cluster's sums of this CTA's tokens, four columns a thread, in rank order
    // (the tile's real tokens, shared out evenly)
    const int ntok = (int)min((int64_t)kTok, p.M - t0), per = (ntok + S - 1) / S;
    const int first = min(rank * per, ntok), mine = min(per, ntok - first), nv = ld / 4;
    const float *sums = part + first * ld;   // [mine][ld]
    if (S > 1) {
        float *const own = part + kTok * ld;
        for (int i = tid; i < mine * nv; i += kThreads) {
            const uint32_t a = base + (uint32_t)(first * ld + 4 * i) * 4;
            float4 v[kMaxCluster], sum = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
            for (int s = 0; s < kMaxCluster; ++s)   // (all loads in flight)
                v[s] = s < S ? ld_dsmem_f4(map_to_rank(a, (uint32_t)s)) : make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
            for (int s = 0; s < kMaxCluster; ++s) {
                sum.x += v[s].x;
                sum.y += v[s].y;
                sum.z += v[s].z;
                sum.w += v[s].w;
            }
            reinterpret_cast<float4 *>(own)[i] = sum;
        }
        sums = own;
        __syncthreads();
    }
    if (tid < mine) {
        const int64_t t = t0 + first + tid;
        float xs = 1.f;
        if constexpr (FORM == kQ8) {
            xs = p.xs[t];
            p.rowc[rowc_at(t)] = xs;
            p.rowc[rowc_at(t) + 2] = sums[tid * ld + p.R1p] * (1.0f / 512.0f);
        }
        if (ec)
            s_gate[tid] = 1.0f / (1.0f + expf(-(xs * sums[tid * ld] + p.b_g))) * (FORM == kQ8 ? 1.0f / 512.0f : 1.0f);
    }
    __syncthreads();
    if (ec)
        for (int tt = warp; tt < mine; tt += kThreads / 32)
            for (int j = lane; j < p.rp; j += 32)
                p.v[(int64_t)(t0 + first + tt) * p.rp + j] =
                    j < p.r ? to_tf32(s_gate[tt] * sums[tt * ld + 1 + j]) : 0.f;
    tc_fence_before();
    __syncthreads();
    if (tid == 0 && p.ready)
        red_release_gpu_add(p.ready, 1u);   // this CTA's v and rowc are written
    if (warp == 1) {
        tc_fence_after();
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(tmem_cols) : "memory");
    }
    if (S > 1)
        cluster_sync();   // no CTA leaves while another reads its partial
}

// As many CTAs a tile as keep one SM each, up to the portable cluster of 8.
int tc_prepass2_split(const Packed &pk, int64_t M, int num_sms)
{
    const int64_t tiles = (M + kTok - 1) / kTok;
    int S = 1;
    while (S < kMaxCluster && 2 * S <= (int)(pk.Kp / 64) && tiles * 2 * S <= num_sms)
        S *= 2;
    return S;
}

}  // namespace

int64_t tc_prepass2_room(const Packed &pk, int64_t M, int num_sms)
{
    return (M + kTok - 1) / kTok * tc_prepass2_split(pk, M, num_sms) * 5 / 4;
}

cudaError_t launch_tc_prepass2(const Packed &pk, const void *x, int64_t ldx, const float *xs, int64_t M, bool ec,
                               float *v, float *rowc, int form, const CUtensorMap *g, int *status, cudaStream_t st,
                               int num_sms, unsigned *ready, unsigned *expected)
{
    const bool q8 = form == kQ8;
    const uint64_t xd[2] = {(uint64_t)pk.K, (uint64_t)M};
    const uint64_t xst[1] = {(uint64_t)ldx * (q8 ? 1u : 2u)};
    const uint32_t xb[2] = {64, kTok};
    CUtensorMap tm_x;
    cudaError_t e = make_map_nd(&tm_x, x, q8 ? CU_TENSOR_MAP_DATA_TYPE_UINT8 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, xd,
                                xst, xb, q8 ? CU_TENSOR_MAP_SWIZZLE_64B : CU_TENSOR_MAP_SWIZZLE_128B);
    if (e != cudaSuccess)
        return e;
    TcPrepass2Params p;
    p.M = M;
    p.n_k = (int)(pk.Kp / 64);   // (a multiple of 4)
    p.R1p = ec ? pk.R1p : 0;
    p.r = pk.r;
    p.rp = pk.rp;
    p.b_g = pk.b_g;
    p.xs = xs;
    p.v = v;
    p.rowc = rowc;
    p.status = status;
    p.ready = ready;
    const int64_t tiles = (M + kTok - 1) / kTok;
    const int S = tc_prepass2_split(pk, M, num_sms);
    p.S = S;
    if (expected)
        *expected = (unsigned)(tiles * S);
    const size_t stage = q8 ? stage_bytes<kQ8>(p.R1p) : stage_bytes<kEpi>(p.R1p);
    p.stages = (int)std::min<size_t>(kMaxStages, 220 * 1024 / stage) & ~1;   // even
    const size_t ring = p.stages * stage;
    const size_t part = (size_t)(kTok + (kTok + S - 1) / S) * (p.R1p + 4) * sizeof(float);   // partials, then sums
    const size_t smem = std::max(ring, part) + 1024;
    using Fn = void (*)(CUtensorMap, CUtensorMap, TcPrepass2Params);
    const Fn fn = q8 ? tc_prepass2_kernel<kQ8> : tc_prepass2_kernel<kEpi>;
    e = raise_smem_limit(reinterpret_cast<const void *>(fn), smem);
    if (e != cudaSuccess)
        return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(tiles * S));
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = (unsigned)S;
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = S > 1 ? 2 : 1;
    return cudaLaunchKernelEx(&cfg, fn, tm_x, p.R1p ? *g : tm_x, p);
}

}  // namespace spear
