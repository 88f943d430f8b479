// W4 GEMM of a batch of tokens with an epilogue (tcgen05), K split over a
// cluster: the forms kEpi and kQ8 of the forward pass where the tiles of the
// pair kernel (tc_pair.cu, which has the formulas) would leave SMs idle.
//
// One CTA takes 128 weight rows x BN tokens (32, 64 or 128) and a 1/S share of
// K; the cluster of S CTAs of a tile sums its partial accumulators through
// distributed shared memory, in rank order (run-to-run identical).  At these
// sizes the layer is bound by reading the codes and by the length of one CTA's
// chain of stages, so S is the largest that still gives every CTA its own SM.
//
// Roles (24 warps): warp 0 copies the tokens (TMA; EC stages, on the last
// rank: v and B^T/e), warp 1 issues the MMAs, warp 2 asks for the CTA's codes
// from HBM to L2 (all of them at once, before anything else: they depend on no
// earlier kernel), warps 8-23 dequantise (four groups taking every fourth stage,
// tc_dequant.cuh), warps 4-7 read the accumulator at the end.  In form kQ8 every
// stage also multiplies its tokens with a constant tile of ones (64 rows, into
// TMEM columns of their own): the code sums that the zero points need, so that a
// layer without the Error Compensator needs no prepass.  (Summed by four warps
// with mma.sync instead, the sums lagged six stages behind the product.)
// Then all of them take the outputs of the CTA's 1/S of the tokens, two channels a
// thread: the S partials, the epilogue, 4-byte stores of whole lines.
// Measured in a chain of calls: 64 tokens of 14336 x 4096 in 8 bits 17.8 us
// (24 with the Error Compensator and its prepass), 128 of 4096 x 14336 23.2 (26),
// 333 of 2064 x 1000 9.6 (14), 33 of 256 x 256 5.0 (9).  About 590 cycles a stage;
// of the 33000 of the first case 6000 pass until the first stage is there and 7000
// from the last MMA to the end (partials, exchange, outputs), so that latency, not
// the 4.6 us of its HBM bytes, bounds it.
// Every wait is bounded (about a second); one that runs out sets the handle's
// status word and the kernel winds down.
#include <algorithm>

#include "async_utils.cuh"
#include "epilogue.cuh"
#include "tc_dequant.cuh"
#include "tc_gemm.h"
#include "tensor_map.h"

namespace spear {
namespace {

constexpr int BM = 128;
constexpr int A_BYTES = BM * kTcRowBytes;
constexpr int DEQ_WARP = 8, GROUPS = 4, GROUP_WARPS = 4;
constexpr int THREADS = 32 * (DEQ_WARP + GROUPS * GROUP_WARPS);
constexpr int kMaxSplit = 8;
__host__ __device__ constexpr int tile_stage_bytes(int BN) { return A_BYTES + BN * kTcRowBytes; }
__host__ __device__ constexpr int tile_stages(int BN) { return BN == 128 ? 6 : 8; }
constexpr int ONES_BYTES = 64 * kTcRowBytes;   // form kQ8: the tile of ones
__host__ __device__ constexpr int tile_smem_bytes(int BN)
{
    return tile_stages(BN) * tile_stage_bytes(BN) + ONES_BYTES + 1024;
}

struct TileParams {
    int64_t M, N, Np;
    int kchunks;             // Kp / 256
    int n_main, n_ec, rp;    // stages of the main product and of the EC; columns of v
    int S;                   // CTAs a tile
    int n_ttiles;
    const uint8_t *codes;
    const float *s;
    const uint8_t *z;
    uint16_t *y;
    int *status;
    unsigned *v_ready;       // as TcParams::v_ready (tc_gemm.cu)
    unsigned v_expected;
    Epilogue epi;
};

template <int FORM, int BN>
__global__ void __launch_bounds__(THREADS, 1)
tc_tile_kernel(const __grid_constant__ CUtensorMap tm_x, const __grid_constant__ CUtensorMap tm_bt,
               const __grid_constant__ CUtensorMap tm_v, TileParams p)
{
    constexpr int STAGES = tile_stages(BN);
    constexpr int B_BYTES = BN * kTcRowBytes;
    constexpr int STAGE_BYTES = tile_stage_bytes(BN);
    constexpr int TMEM_COLS = FORM == kQ8 ? 2 * BN : BN;   // the accumulator, the code sums
    constexpr uint32_t ONES = STAGES * STAGE_BYTES;        // byte offset of the tile of ones
    extern __shared__ uint8_t smem_raw[];
    __shared__ __align__(8) uint64_t bars[2 * STAGES + 2];   // ready and empty of each stage; done; drain
    __shared__ uint32_t tmem_base_slot;
    __shared__ volatile int abort_flag;
    __shared__ float2 s_const[FORM == kQ8 ? BN : 1];   // xs[t], 2^-9 sum_k xq[t,k] of this CTA's outputs

    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const uint32_t base = (smem_addr(smem_raw) + 1023u) & ~1023u;
    uint8_t *const bp = smem_raw + (base - smem_addr(smem_raw));
    const uint32_t ready0 = smem_addr(&bars[0]), empty0 = smem_addr(&bars[STAGES]);
    const uint32_t done = smem_addr(&bars[2 * STAGES]), drain = smem_addr(&bars[2 * STAGES + 1]);
    const int S = p.S, rank = (int)cluster_ctarank(), unit = (int)blockIdx.x / S;
    const int t0 = (unit % p.n_ttiles) * BN, n0 = (unit / p.n_ttiles) * BM;
    const int lo = rank * p.n_main / S, nm = (rank + 1) * p.n_main / S - lo;   // (S <= n_main: at least one)
    const int nst = nm + (rank == S - 1 ? p.n_ec : 0);

    if (tid == 0) {
        abort_flag = 0;
        for (int s = 0; s < STAGES; ++s) {
            mbar_init(ready0 + 8 * s, GROUP_WARPS + 1);
            mbar_init(empty0 + 8 * s, 1);
        }
        mbar_init(done, 1);
        mbar_init(drain, 1);
        fence_mbarrier_init_cluster();
    }
    if (warp == 2) {
        // the blocks of 256 k that hold this CTA's stages, of both 64-row block rows
        constexpr int SUB = tc_stages_per_block(FORM);
        const int b0 = lo / SUB, nb = (lo + nm - 1) / SUB + 1 - b0;
        for (int i = lane; i < 2 * nb; i += 32)
            bulk_prefetch_l2(p.codes + ((int64_t)(n0 / 64 + i / nb) * p.kchunks + b0 + i % nb) * 8192, 8192);
    }
    if (warp == 1) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                         smem_addr(&tmem_base_slot)),
                     "r"(TMEM_COLS)
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    }
    if constexpr (FORM == kQ8) {
        for (int i = tid; i < ONES_BYTES / 16; i += THREADS)   // (1.0 in e4m3; any order will do)
            reinterpret_cast<uint4 *>(bp + ONES)[i] = make_uint4(0x38383838u, 0x38383838u, 0x38383838u, 0x38383838u);
        fence_proxy_async_smem();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = tmem_base_slot;
    pdl_launch_dependents();   // (after the tensor memory is held: see the prepass)

    if (warp == 0) {
        const bool elected = elect_one();
        if (!p.v_ready)
            pdl_wait();   // x and v come from earlier kernels in the stream
        bool v_seen = p.v_ready == nullptr;
        uint32_t slot = 0, phase = 0;
        int issued = 0;
        for (int i = 0; i < nst; ++i, ++issued) {
            if (!warp_wait(empty0 + 8 * slot, phase ^ 1, &abort_flag, p.status))
                break;
            const uint32_t sb = base + slot * STAGE_BYTES, ready = ready0 + 8 * slot;
            if (i < nm) {
                if (elected) {
                    mbar_expect_tx(ready, B_BYTES);
                    tma_load_2d(sb + A_BYTES, &tm_x, (lo + i) * tc_stage_k(FORM), t0, ready);
                }
            } else {
                if (!v_seen) {
                    if (!__all_sync(0xffffffffu, wait_counted(p.v_ready, p.v_expected, &abort_flag, p.status)))
                        break;
                    v_seen = true;
                }
                if (elected) {
                    mbar_expect_tx(ready, A_BYTES + B_BYTES);
                    tma_load_2d(sb, &tm_bt, (i - nm) * 32, n0, ready);   // 32 tf32 values of j a stage
                    tma_load_2d(sb + A_BYTES, &tm_v, (i - nm) * 32, t0, ready);
                }
            }
            if (++slot == STAGES) {
                slot = 0;
                phase ^= 1;
            }
        }
        // do not leave while copies may still land (the MMA issuer waited for
        // every stage unless a wait gave up)
        if (abort_flag)
            for (int k = 0; k < STAGES && k < issued; ++k)
                mbar_wait_final(ready0 + 8 * ((issued - 1 - k) % STAGES), ((issued - 1 - k) / STAGES) & 1);
    } else if (warp == 1) {
        const bool elected = elect_one();
        const uint32_t shape = ((uint32_t)(BN >> 3) << 17) | ((uint32_t)(BM >> 4) << 24) | (1u << 4);
        const uint32_t idesc = shape | (FORM == kQ8 ? 0u : (1u << 7) | (1u << 10));
        const uint32_t idesc_tf32 = shape | (2u << 7) | (2u << 10);
        const uint32_t idesc_ones = ((uint32_t)(BN >> 3) << 17) | ((uint32_t)(64 >> 4) << 24) | (1u << 4);
        const uint64_t a0 = smem_desc_sw128(base), b0 = smem_desc_sw128(base + A_BYTES);
        const uint64_t ones = smem_desc_sw128(base + ONES);
        uint32_t slot = 0, phase = 0;
        bool ok = true;
        for (int i = 0; i < nst; ++i) {
            if (!warp_wait(ready0 + 8 * slot, phase, &abort_flag, p.status)) {
                ok = false;
                break;
            }
            tc_fence_after();
            const uint64_t a_desc = a0 + slot * (STAGE_BYTES >> 4), b_desc = b0 + slot * (STAGE_BYTES >> 4);
            if (i < nm) {
                if (elected) {
                    // 32 bytes of k an instruction
#pragma unroll
                    for (int k = 0; k < kTcRowBytes / 32; ++k) {
                        const uint32_t accumulate = (i > 0 || k > 0) ? 1u : 0u;
                        if constexpr (FORM == kQ8)
                            mma_e4m3(tmem, a_desc + 2 * k, b_desc + 2 * k, idesc, accumulate);
                        else
                            mma_bf16(tmem, a_desc + 2 * k, b_desc + 2 * k, idesc, accumulate);
                        if constexpr (FORM == kQ8)
                            mma_e4m3(tmem + BN, ones, b_desc + 2 * k, idesc_ones, accumulate);
                    }
                    mma_commit(empty0 + 8 * slot);
                }
            } else if (elected) {
                const int rem = p.rp - (i - nm) * 32;
                const int ksteps = (rem < 32 ? rem : 32) / 8;
                for (int k = 0; k < ksteps; ++k)
                    mma_tf32(tmem, a_desc + 2 * k, b_desc + 2 * k, idesc_tf32, 1u);
                mma_commit(empty0 + 8 * slot);
            }
            __syncwarp();
            if (++slot == STAGES) {
                slot = 0;
                phase ^= 1;
            }
        }
        if (elected) {
            if (ok)
                mma_commit(done);
            mma_commit(drain);   // every MMA this warp issued is complete before TMEM is released
        }
        __syncwarp();
        mbar_wait_final(drain, 0);
    } else if (warp >= DEQ_WARP) {
        const int grp = (warp - DEQ_WARP) / GROUP_WARPS, w = warp & 3;
        TcDequant<FORM> d(w, lane);
        const uint8_t *src = p.codes + (int64_t)(n0 / 64 + (w >> 1)) * p.kchunks * 8192 + d.offset();
        d.set_rows(p.s, p.z, n0, p.Np);
        if (grp < nm)
            d.fetch(src, lo + grp);
        uint32_t slot = (uint32_t)grp, phase = 0;
        for (int st = grp; st < nst; st += GROUPS) {
            if (st < nm) {
                d.convert();
                if (st + GROUPS < nm)
                    d.fetch(src, lo + st + GROUPS);
            }
            if (!warp_wait(empty0 + 8 * slot, phase ^ 1, &abort_flag, p.status))
                break;
            if (st < nm) {
                d.store(bp + slot * STAGE_BYTES);
                fence_proxy_async_smem();
                __syncwarp();
            }
            if (lane == 0)
                mbar_arrive(ready0 + 8 * slot);
            slot += GROUPS;
            if (slot >= STAGES) {
                slot -= STAGES;
                phase ^= 1;
            }
        }
    }

    // ---- the partial accumulator, [token][128 channels] fp32, over the stages
    bool ok = true;
    if (warp >= 4 && warp < 8)
        ok = warp_wait(done, 0, &abort_flag, p.status);
    __syncthreads();   // every copy and MMA of this CTA is over
    float *const part = reinterpret_cast<float *>(bp);
    if (warp >= 4 && warp < 8) {
        tc_fence_after();
        const int q = warp & 3;
        for (int c = 0; c < BN && t0 + c < p.M; c += 16) {
            uint32_t a[16];
            tmem_ld_32x32b_x16(tmem + ((uint32_t)(32 * q) << 16) + c, a);
#pragma unroll
            for (int j = 0; j < 16; ++j)
                part[(c + j) * BM + 32 * q + lane] = ok ? __uint_as_float(a[j]) : 0.f;
        }
        if (FORM == kQ8 && q == 0)   // (every row of the ones' product is the sums; the first is lane 0's)
            for (int c = 0; c < BN && t0 + c < p.M; c += 16) {
                uint32_t a[16];
                tmem_ld_32x32b_x16(tmem + BN + c, a);
                if (lane == 0)
#pragma unroll
                    for (int j = 0; j < 16; ++j)
                        part[BN * BM + c + j] = __uint_as_float(a[j]);
            }
        tc_fence_before();
    }
    // the prepass has finished (its constants are read below; and this grid
    // completes only after its predecessor)
    pdl_wait();
    if (S > 1)
        cluster_sync();
    else
        __syncthreads();
    if (warp == 1) {
        tc_fence_after();
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(TMEM_COLS)
                     : "memory");
    }

    // ---- outputs: this CTA's tokens, two channels a thread
    // (the tile's real tokens, shared out evenly)
    const int real = (int)min((int64_t)BN, p.M - t0), per = (real + S - 1) / S;
    const int first = min(rank * per, real), ntok = min(per, real - first);
    if constexpr (FORM == kQ8) {
        if (tid < ntok) {
            float x = 0.f;
            for (int s = 0; s < S; ++s)
                x += ld_dsmem_f32(map_to_rank(base + (uint32_t)(BN * BM + first + tid) * 4, (uint32_t)s));
            s_const[tid] = make_float2(p.epi.xs[t0 + first + tid], x * (1.0f / 512.0f));
        }
        __syncthreads();
    }
    // A thread's channels are the same for all its tokens (THREADS is a multiple
    // of BM / 2).  This code runs once per CTA, from a cold instruction cache, so
    // it is kept short: the loop is not unrolled and the activations are one
    // function (unrolled by four with them inlined, this phase took 10000 cycles).
    const int cp = tid & (BM / 2 - 1), n = n0 + 2 * cp;
    if (n < p.N) {
        const float2 sn = __ldg(reinterpret_cast<const float2 *>(p.s + n));
        const float e0 = sn.x != 0.f ? sn.x : 1.f, e1 = sn.y != 0.f ? sn.y : 1.f;   // (B^T was divided by it)
        float z0 = 0.f, z1 = 0.f;
        if (FORM == kQ8) {
            const uint32_t z = __ldg(reinterpret_cast<const uint16_t *>(p.z + n));
            z0 = sn.x != 0.f ? (float)(z & 255u) : 0.f;
            z1 = sn.y != 0.f ? (float)(z >> 8) : 0.f;
        }
        const uint32_t bias = p.epi.bias ? *reinterpret_cast<const uint32_t *>(p.epi.bias + n) : 0u;
#pragma unroll 1
        for (int tt = tid / (BM / 2); tt < ntok; tt += THREADS / (BM / 2)) {
            const int64_t at = (int64_t)(t0 + first + tt) * p.N + n;
            const uint32_t m = p.epi.mul ? *reinterpret_cast<const uint32_t *>(p.epi.mul + at) : 0x3F803F80u;
            const uint32_t r = p.epi.residual ? *reinterpret_cast<const uint32_t *>(p.epi.residual + at) : 0u;
            const uint32_t a = base + (uint32_t)((first + tt) * BM + 2 * cp) * 4;
            float2 v[kMaxSplit];
#pragma unroll
            for (int s = 0; s < kMaxSplit; ++s)   // (all S loads in flight; a cluster of one reads itself)
                v[s] = s < S ? ld_dsmem_f2(map_to_rank(a, (uint32_t)s)) : make_float2(0.f, 0.f);
            float v0 = v[0].x, v1 = v[0].y;
#pragma unroll
            for (int s = 1; s < kMaxSplit; ++s) {
                v0 += v[s].x;
                v1 += v[s].y;
            }
            if constexpr (FORM == kQ8) {
                const float2 c = s_const[tt];
                // (2^9 beside the sum: with a scale of 2^119 or more it would leave fp32)
                v0 = e0 * c.x * (512.0f * (v0 - z0 * c.y));
                v1 = e1 * c.x * (512.0f * (v1 - z1 * c.y));
            } else {
                v0 *= e0;
                v1 *= e1;
            }
            v0 += bf16_lo(bias);
            v1 += bf16_hi(bias);
            if (p.epi.act != kActNone) {
                v0 = activate_call(v0, p.epi.act);
                v1 = activate_call(v1, p.epi.act);
            }
            v0 = v0 * bf16_lo(m) + bf16_lo(r);
            v1 = v1 * bf16_hi(m) + bf16_hi(r);
            *reinterpret_cast<uint32_t *>(p.y + at) = pack_bf16x2(v0, v1);
        }
    }
    if (S > 1)
        cluster_sync();   // no CTA leaves while another reads its partial
    if (tid == 0 && p.v_ready && atomicAdd(p.v_ready + 1, 1u) == gridDim.x - 1) {
        // every CTA is past its waits for the prepass, which has finished: reset
        p.v_ready[0] = 0u;
        p.v_ready[1] = 0u;
    }
}

using TileFn = void (*)(CUtensorMap, CUtensorMap, CUtensorMap, TileParams);
template <int FORM>
TileFn tile_fn(int BN)
{
    return BN == 32 ? tc_tile_kernel<FORM, 32> : (BN == 64 ? tc_tile_kernel<FORM, 64> : tc_tile_kernel<FORM, 128>);
}

}  // namespace

cudaError_t launch_tc_tile(const Packed &pk, const void *x, void *y, int64_t M, const float *v, bool ec,
                           const CUtensorMap *bt, int *status, cudaStream_t st, int num_sms, unsigned *v_ready,
                           unsigned v_expected, int form, const Epilogue &epi, int64_t ldx)
{
    const int BN = M <= 32 ? 32 : (M <= 64 ? 64 : 128);
    const int BK = tc_stage_k(form);
    const uint64_t xd[2] = {(uint64_t)pk.K, (uint64_t)M};
    const uint64_t xst[1] = {(uint64_t)ldx * (uint64_t)(kTcRowBytes / BK)};
    const uint32_t xb[2] = {(uint32_t)BK, (uint32_t)BN};
    CUtensorMap tm_x, tm_v;
    cudaError_t e = make_map_nd(&tm_x, x, form == kQ8 ? CU_TENSOR_MAP_DATA_TYPE_UINT8
                                                      : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16,
                                2, xd, xst, xb, CU_TENSOR_MAP_SWIZZLE_128B);
    const bool use_ec = ec && pk.r > 0;
    tm_v = tm_x;   // unused without the EC
    if (e == cudaSuccess && use_ec)
        e = make_map(&tm_v, v, CU_TENSOR_MAP_DATA_TYPE_FLOAT32, 4, (uint64_t)pk.rp, (uint64_t)M, 32, (uint32_t)BN,
                     CU_TENSOR_MAP_SWIZZLE_128B);
    if (e != cudaSuccess)
        return e;
    TileParams p;
    p.M = M;
    p.N = pk.N;
    p.Np = pk.Np;
    p.kchunks = (int)(pk.Kp / 256);
    p.n_main = (int)(pk.Kp / BK);
    p.n_ec = use_ec ? (pk.rp + 31) / 32 : 0;
    p.rp = pk.rp;
    p.n_ttiles = (int)((M + BN - 1) / BN);
    const int64_t units = (int64_t)p.n_ttiles * (pk.Np / BM);
    const TileFn fn = form == kQ8 ? tile_fn<kQ8>(BN) : tile_fn<kEpi>(BN);
    const int smem = tile_smem_bytes(BN);
    e = raise_smem_limit(reinterpret_cast<const void *>(fn), smem);
    if (e != cudaSuccess)
        return e;
    // K over as many CTAs a tile as are all resident at once, at least four
    // stages a CTA, beside the prepass with the EC (clusters that have to wait for
    // it make the two run one after the other, 31 us instead of 24 at 64 tokens
    // of a 14336x4096 layer)
    const int64_t beside = use_ec ? tc_prepass2_room(pk, M, num_sms) : 0;
    int S = (int)std::min<int64_t>({kMaxSplit, std::max(1, p.n_main / 4), std::max<int64_t>(1, num_sms / units)});
    while (S > 1 && !grid_is_one_wave(reinterpret_cast<const void *>(fn), THREADS, smem, S, units * S + beside, num_sms))
        --S;
    p.S = S;
    p.codes = reinterpret_cast<const uint8_t *>(pk.codes);
    p.s = pk.s;
    p.z = pk.z;
    p.y = static_cast<uint16_t *>(y);
    p.status = status;
    p.v_ready = use_ec ? v_ready : nullptr;
    p.v_expected = v_expected;
    p.epi = epi;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(units * S));
    cfg.blockDim = dim3(THREADS);
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
    return cudaLaunchKernelEx(&cfg, fn, tm_x, use_ec ? *bt : tm_x, tm_v, p);
}

}  // namespace spear
