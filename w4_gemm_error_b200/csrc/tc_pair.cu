// W4 GEMM of many tokens with an epilogue, on pairs of CTAs (tcgen05,
// cta_group::2): the forms kEpi (bf16 activations) and kQ8 (e4m3) of the
// forward pass where there are many tiles (tc_use_pair).
//
//   D[n, t] = sum_k a[n,k] x[t,k] + sum_j (B[j,n] / e[n]) v[t,j]
//   form kEpi:  a = q - z,     Y = e[n] D                       (bf16 MMAs)
//   form kQ8:   a = 2^-9 q,    Y = xs[t] e[n] (2^9 D - z[n] X_t)   (e4m3 MMAs)
//   y[t, n] = act(Y + bias[n]) * mul[t,n] + residual[t,n]
//
// Why a pair: a 128 x 256 tile of one SM moves more bytes through its shared
// memory than the tensor core leaves time for (operands written by TMA and by
// the dequantisers, read by them and by the MMAs).  A pair works on 256 weight
// rows x 256 tokens; each CTA holds its own 128 weight rows and half of the
// tokens, and the MMAs read both halves of the activations from the two SMs,
// so each SM stages half the activations for the same products.
//
// Roles in each CTA (28 warps):
//   warp 0       TMA producer of the stages: its 128 tokens of x (EC stages: v
//                and B^T/e)
//   warp 1       TMEM allocation; in the pair's first CTA the issuer of the
//                MMAs of both
//   warp 2       loader of the epilogue's operands (multiplier, residual and
//                per-token constants) into slots of 32 tokens x 128 channels
//   warps 4-11   epilogue, two sets of four warps (each warp its 32 TMEM
//                lanes) taking alternate slots: accumulator from TMEM, the
//                formula above, y into the slot (over the residual, element by
//                element) and from there to HBM by one TMA store a slot
//   warps 12-27  dequantisers, four groups of four taking every fourth stage:
//                codes from global memory into registers four stages ahead,
//                from there into the stage as MMA operands
// The codes never pass through shared memory before they are dequantised, so
// that the ring of stages (5, or 6 without a multiplier) is deep enough to
// cover the latency from a TMA request to the MMA that frees its stage: with
// four stages that held the codes too, a 128-k stage took 1200 cycles instead
// of the 512 of its MMAs.  The producer and the MMA issuer run as whole warps
// with one elected lane in the asynchronous instructions, so that addresses
// and descriptors stay in uniform registers (issued from a single-lane branch,
// the four MMAs of a stage alone cost about 400 cycles).
// Measured in a short chain of calls (with the prepass): 4096 tokens of 4096 x 14336,
// 8 bits, SiLU: 205 us, 2390 TFLOP/s (the tensor pipe 73 % active, clocks at
// 1.4 GHz under the power limit); 2048 tokens, bf16, times a multiplier: 184 us,
// 1330 TFLOP/s (82 % active; 448 units on 74 pairs are 6.05 rounds, so that a
// seventh runs nearly empty).  In runs of seconds, at the clock that the power limit
// then leaves: 245 us (2000 TFLOP/s) and 217 us (1130 TFLOP/s).  What bounds it is shared memory: a stage is written
// by TMA and dequantisers and read by the MMAs, 64 KB or about 512 cycles of its
// 128 bytes a cycle, beside the epilogue's.
// Two accumulators of 256 columns in TMEM: the epilogue of a tile overlaps the
// main loop of the next.  Every wait is bounded (about a second); one that runs
// out sets the handle's status word and the kernel winds down.
#include <algorithm>

#include "async_utils.cuh"
#include "epilogue.cuh"
#include "tc_dequant.cuh"
#include "tc_gemm.h"
#include "tensor_map.h"

namespace spear {
namespace {

constexpr int BM = 128;                 // weight rows of a CTA (256 a pair)
constexpr int BN = 256;                 // tokens of a pair (128 staged by each CTA)
constexpr int ROW_BYTES = kTcRowBytes;
constexpr int A_BYTES = BM * ROW_BYTES;
constexpr int B_BYTES = (BN / 2) * ROW_BYTES;
constexpr int STAGE_BYTES = A_BYTES + B_BYTES;
constexpr int MAX_STAGES = 6;
constexpr int CHUNK = 32;               // tokens of an epilogue slot
constexpr int NSLOT = 4;
constexpr int HALF_SLOT = CHUNK * BM * 2;   // residual / y; a second one for the multiplier
constexpr int ROWC_BYTES = CHUNK * 8;
constexpr int EPI_WARP = 4, DEQ_WARP = 12, GROUP_WARPS = 4, GROUPS = 4;
constexpr int THREADS = 32 * (DEQ_WARP + GROUPS * GROUP_WARPS);
// What a CTA adds to an accumulator's hand-back: its epilogue warps and the prefetching
// warp, each when it has seen the accumulator full.  Whoever waits for a phase of
// `tfull` has to be counted, or that phase and the next could pass unseen, and the
// one after them, of the same parity, may never come.
constexpr int HAND_BACK = DEQ_WARP - EPI_WARP + 1;

// Ring depth and shared memory with and without a multiplier in the slots.
int pair_stages(bool mul) { return mul ? 5 : 6; }
int pair_smem_bytes(bool mul)
{
    return pair_stages(mul) * STAGE_BYTES + NSLOT * (HALF_SLOT * (mul ? 2 : 1) + ROWC_BYTES) + 1024;
}

struct PairParams {
    int64_t M, N, Np;
    int kchunks;             // Kp / 256
    int n_main, n_ec, rp;    // stages of the main loop and of the EC; columns of v
    int n_ttiles, n_units;
    int stages;
    const uint8_t *codes;    // the tiled codes (Packed::codes)
    const float *s;
    const uint8_t *z;
    int *status;
    unsigned *v_ready;       // as TcParams::v_ready (tc_gemm.cu)
    unsigned v_expected;
    Epilogue epi;
    const float *rowc;       // form kQ8: the constants of rowc_at, whole chunks
};

// One slot's outputs of this thread: channel n (row `row` of the CTA), the 32
// tokens of the chunk, the accumulator at tacc in TMEM.  mul and y are its columns of
// [32 tokens][128 channels] bf16.  Eight tokens at a time: every shared-memory
// read of a group comes before its first store.
template <int FORM, int ACT, bool MUL, bool RES>
__device__ __forceinline__ void emit_chunk(uint32_t tacc, float e_n, float z_n, float bias,
                                           const uint16_t *mul, uint16_t *y, const float4 *rc)
{
    const f32x2 e2 = f2_pack(e_n, e_n), nz2 = f2_pack(-z_n, -z_n), bias2 = f2_pack(bias, bias);
#pragma unroll
    for (int j0 = 0; j0 < CHUNK; j0 += 8) {
        uint32_t acc[8];
        tmem_ld_32x32b_x8(tacc + j0, acc);
        float4 c[4];   // per-token constants of two tokens: both first ones, both second ones
        uint32_t m[8], r[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            if (FORM == kQ8 && (j & 1) == 0)
                c[j / 2] = rc[(j0 + j) / 2];
            m[j] = MUL ? mul[(j0 + j) * BM] : 0u;
            r[j] = RES ? y[(j0 + j) * BM] : 0u;
        }
        uint32_t two[4];
#pragma unroll
        for (int j = 0; j < 8; j += 2) {
            f32x2 v = f2_pack(__uint_as_float(acc[j]), __uint_as_float(acc[j + 1]));
            f32x2 k = e2;
            if constexpr (FORM == kQ8) {
                k = f2_mul(e2, f2_pack(c[j / 2].x, c[j / 2].y));
                // (2^9 beside the sum: with a scale of 2^119 or more it would leave fp32)
                v = f2_mul(f2_fma(nz2, f2_pack(c[j / 2].z, c[j / 2].w), v), f2_pack(512.f, 512.f));
            }
            v = activate2<ACT>(f2_fma(k, v, bias2));
            if (MUL)
                v = f2_mul(v, f2_pack(bf16_lo(m[j]), bf16_lo(m[j + 1])));
            if (RES)
                v = f2_add(v, f2_pack(bf16_lo(r[j]), bf16_lo(r[j + 1])));
            float lo, hi;
            f2_unpack(v, lo, hi);
            two[j / 2] = pack_bf16x2(lo, hi);
        }
#pragma unroll
        for (int j = 0; j < 8; j += 2) {
            y[(j0 + j) * BM] = (uint16_t)two[j / 2];
            y[(j0 + j + 1) * BM] = (uint16_t)(two[j / 2] >> 16);
        }
    }
}

template <int FORM, int ACT>
__device__ __forceinline__ void emit_chunk_of(uint32_t tacc, float e_n, float z_n, float bias,
                                              const uint16_t *mul, uint16_t *y, const float4 *rc, bool has_mul,
                                              bool has_res)
{
    if (has_mul)
        has_res ? emit_chunk<FORM, ACT, true, true>(tacc, e_n, z_n, bias, mul, y, rc)
                : emit_chunk<FORM, ACT, true, false>(tacc, e_n, z_n, bias, mul, y, rc);
    else
        has_res ? emit_chunk<FORM, ACT, false, true>(tacc, e_n, z_n, bias, mul, y, rc)
                : emit_chunk<FORM, ACT, false, false>(tacc, e_n, z_n, bias, mul, y, rc);
}

template <int FORM>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(THREADS, 1)
tc_pair_kernel(const __grid_constant__ CUtensorMap tm_x, const __grid_constant__ CUtensorMap tm_bt, const __grid_constant__ CUtensorMap tm_v,
               const __grid_constant__ CUtensorMap tm_mul, const __grid_constant__ CUtensorMap tm_res,
               const __grid_constant__ CUtensorMap tm_y, PairParams p)
{
    constexpr int BK = tc_stage_k(FORM);
    extern __shared__ uint8_t smem_raw[];
    // ready and empty of each stage; accumulator full and empty; slot full and empty; drain
    __shared__ __align__(8) uint64_t bars[2 * MAX_STAGES + 4 + 2 * NSLOT + 1];
    __shared__ uint32_t tmem_base_slot;
    __shared__ volatile int abort_flag;

    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const uint32_t base = (smem_addr(smem_raw) + 1023u) & ~1023u;
    uint8_t *const base_ptr = smem_raw + (base - smem_addr(smem_raw));
    const uint32_t rank = cluster_ctarank();
    // first CTA's: both CTAs' operands of the stage are there (the copies of both
    // count their bytes on it, the dequantising warps of both arrive on it)
    const uint32_t ready0 = smem_addr(&bars[0]);
    const uint32_t empty0 = smem_addr(&bars[MAX_STAGES]);
    const uint32_t tfull0 = smem_addr(&bars[2 * MAX_STAGES]);
    const uint32_t tempty0 = smem_addr(&bars[2 * MAX_STAGES + 2]);   // first CTA's: HAND_BACK arrivals of each CTA
    const uint32_t sfull0 = smem_addr(&bars[2 * MAX_STAGES + 4]);
    const uint32_t sempty0 = smem_addr(&bars[2 * MAX_STAGES + 4 + NSLOT]);
    const uint32_t drain = smem_addr(&bars[2 * MAX_STAGES + 4 + 2 * NSLOT]);
    const uint32_t S = (uint32_t)p.stages;
    const bool has_mul = p.epi.mul != nullptr, has_res = p.epi.residual != nullptr;
    // byte offsets: residual / y halves of the slots, multiplier halves, per-token constants
    const uint32_t o_y = S * STAGE_BYTES, o_mul = o_y + NSLOT * HALF_SLOT;
    const uint32_t o_rowc = o_mul + (has_mul ? NSLOT * HALF_SLOT : 0);

    if (tid == 0) {
        abort_flag = 0;
        for (uint32_t s = 0; s < S; ++s) {
            mbar_init(ready0 + 8 * s, 2 * GROUP_WARPS + 1);
            mbar_init(empty0 + 8 * s, 1);
        }
        for (int b = 0; b < 2; ++b) {
            mbar_init(tfull0 + 8 * b, 1);
            mbar_init(tempty0 + 8 * b, 2 * HAND_BACK);
        }
        for (int s = 0; s < NSLOT; ++s) {
            mbar_init(sfull0 + 8 * s, 1);
            mbar_init(sempty0 + 8 * s, 1);
        }
        mbar_init(drain, 1);
        fence_mbarrier_init_cluster();
    }
    if (warp == 1) {
        asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                         smem_addr(&tmem_base_slot)),
                     "r"(2 * BN)
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
    }
    tc_fence_before();
    __syncthreads();
    cluster_sync();   // both CTAs' barriers are initialised and both hold their tensor memory
    tc_fence_after();
    const uint32_t tmem_base = tmem_base_slot;
    pdl_launch_dependents();

    const int cluster = blockIdx.x >> 1, n_clusters = gridDim.x >> 1;
    const int nst = p.n_main + p.n_ec;

    if (warp == 0) {
        // ------------------------------------------------ TMA producer
        const bool elected = elect_one();
        if (!p.v_ready)
            pdl_wait();   // x and v come from earlier kernels in the stream
        bool v_seen = p.v_ready == nullptr;
        const uint32_t lead0 = map_to_rank(ready0, 0);
        uint32_t slot = 0, phase = 0, issued = 0;
        bool ok = true;
        for (int u = cluster; u < p.n_units && ok; u += n_clusters) {
            const int t0 = (u % p.n_ttiles) * BN + (int)rank * (BN / 2);
            const int n0 = (u / p.n_ttiles) * 2 * BM + (int)rank * BM;
            for (int i = 0; i < nst; ++i) {
                if (!warp_wait(empty0 + 8 * slot, phase ^ 1, &abort_flag, p.status)) {
                    ok = false;
                    break;
                }
                const uint32_t sb = base + slot * STAGE_BYTES, ready = lead0 + 8 * slot;
                if (i < p.n_main) {
                    if (elected) {
                        if (rank == 0)
                            mbar_expect_tx(ready0 + 8 * slot, 2 * B_BYTES);
                        tma_load_2d_pair(sb + A_BYTES, &tm_x, i * BK, t0, ready);
                    }
                } else {
                    if (!v_seen && !__all_sync(0xffffffffu, wait_counted(p.v_ready, p.v_expected, &abort_flag, p.status))) {
                        ok = false;
                        break;
                    }
                    v_seen = true;
                    if (elected) {
                        const int e = i - p.n_main;   // 32 tf32 values of j a stage
                        if (rank == 0)
                            mbar_expect_tx(ready0 + 8 * slot, 2 * (A_BYTES + B_BYTES));
                        tma_load_2d_pair(sb, &tm_bt, e * 32, n0, ready);
                        tma_load_2d_pair(sb + A_BYTES, &tm_v, e * 32, t0, ready);
                    }
                }
                ++issued;
                if (++slot == S) {
                    slot = 0;
                    phase ^= 1;
                }
            }
        }
        // the pair does not leave while copies may still land (the MMA issuer
        // waited for every stage of both CTAs unless a wait gave up; the second
        // CTA waits for the first in the cluster barrier at the end)
        if (abort_flag && rank == 0)
            for (uint32_t k = 0; k < S && k < issued; ++k) {
                const uint32_t g = issued - 1 - k;
                mbar_wait_final(ready0 + 8 * (g % S), (g / S) & 1);
            }
        // early start: this grid completes only after its predecessor
        if (p.v_ready)
            pdl_wait();
    } else if (warp == 1) {
        // ------------------------------------------------ MMA issuer of the pair
        if (rank == 0) {
            const bool elected = elect_one();
            const uint32_t shape = ((uint32_t)(BN >> 3) << 17) | ((uint32_t)(2 * BM >> 4) << 24) | (1u << 4);
            const uint32_t idesc = shape | (FORM == kQ8 ? 0u : (1u << 7) | (1u << 10));
            const uint32_t idesc_tf32 = shape | (2u << 7) | (2u << 10);
            const uint64_t a0 = smem_desc_sw128(base), b0 = smem_desc_sw128(base + A_BYTES);
            uint32_t slot = 0, phase = 0;
            int lt = 0;
            bool ok = true;
            for (int u = cluster; u < p.n_units && ok; u += n_clusters, ++lt) {
                const uint32_t buf = lt & 1;
                if (!warp_wait(tempty0 + 8 * buf, ((lt >> 1) & 1) ^ 1, &abort_flag, p.status))
                    break;
                tc_fence_after();
                const uint32_t d_tmem = tmem_base + buf * BN;
                for (int i = 0; i < nst; ++i) {
                    if (!warp_wait(ready0 + 8 * slot, phase, &abort_flag, p.status)) {
                        ok = false;
                        break;
                    }
                    tc_fence_after();
                    const uint64_t a_desc = a0 + slot * (STAGE_BYTES >> 4), b_desc = b0 + slot * (STAGE_BYTES >> 4);
                    if (i < p.n_main) {
                        if (elected) {
                            // 32 bytes of k an instruction
#pragma unroll
                            for (int k = 0; k < ROW_BYTES / 32; ++k) {
                                const uint32_t accumulate = (i > 0 || k > 0) ? 1u : 0u;
                                if constexpr (FORM == kQ8)
                                    mma2_e4m3(d_tmem, a_desc + 2 * k, b_desc + 2 * k, idesc, accumulate);
                                else
                                    mma2_bf16(d_tmem, a_desc + 2 * k, b_desc + 2 * k, idesc, accumulate);
                            }
                            mma2_commit_both(empty0 + 8 * slot);
                        }
                    } else {
                        const int rem = p.rp - (i - p.n_main) * 32;
                        const int ksteps = (rem < 32 ? rem : 32) / 8;
                        if (elected) {
                            for (int k = 0; k < ksteps; ++k)
                                mma2_tf32(d_tmem, a_desc + 2 * k, b_desc + 2 * k, idesc_tf32, 1u);
                            mma2_commit_both(empty0 + 8 * slot);
                        }
                    }
                    __syncwarp();
                    if (++slot == S) {
                        slot = 0;
                        phase ^= 1;
                    }
                }
                if (ok && elected)
                    mma2_commit_both(tfull0 + 8 * buf);
                __syncwarp();
            }
            // every MMA this warp issued is complete before TMEM is released
            if (elected)
                mma2_commit(drain);
            __syncwarp();
            mbar_wait_final(drain, 0);
        }
    } else if (warp == 2) {
        // ------------------------------------------------ loader of the epilogue's operands
        if (lane == 0) {
            bool ready = p.v_ready == nullptr || FORM != kQ8;
            if (!p.v_ready)
                pdl_wait();
            uint32_t g = 0;
            bool ok = true;
            const uint32_t bytes = (has_mul ? HALF_SLOT : 0u) + (has_res ? HALF_SLOT : 0u) +
                                   (FORM == kQ8 ? (uint32_t)ROWC_BYTES : 0u);
            for (int u = cluster; u < p.n_units && ok; u += n_clusters) {
                const int t0 = (u % p.n_ttiles) * BN;
                const int n0 = (u / p.n_ttiles) * 2 * BM + (int)rank * BM;
                if (n0 >= p.N)
                    continue;
                for (int c = 0; c < BN / CHUNK && t0 + c * CHUNK < p.M; ++c, ++g) {
                    const uint32_t slot = g % NSLOT, phase = (g / NSLOT) & 1;
                    if (!mbar_wait(sempty0 + 8 * slot, phase ^ 1, &abort_flag, p.status)) {
                        ok = false;
                        break;
                    }
                    const uint32_t bar = sfull0 + 8 * slot;
                    if (bytes == 0) {
                        mbar_arrive(bar);
                        continue;
                    }
                    if (!ready && !wait_counted(p.v_ready, p.v_expected, &abort_flag, p.status)) {
                        ok = false;
                        break;
                    }
                    ready = true;
                    mbar_expect_tx(bar, bytes);
                    if (has_mul)
                        tma_load_2d(base + o_mul + slot * HALF_SLOT, &tm_mul, n0, t0 + c * CHUNK, bar);
                    if (has_res)
                        tma_load_2d(base + o_y + slot * HALF_SLOT, &tm_res, n0, t0 + c * CHUNK, bar);
                    if (FORM == kQ8)
                        bulk_load(base + o_rowc + slot * ROWC_BYTES, p.rowc + 2 * (t0 + c * CHUNK), ROWC_BYTES, bar);
                }
            }
            // (the epilogue waited for every slot unless a wait gave up)
            if (abort_flag && bytes)
                for (uint32_t k = 0; k < NSLOT && k < g; ++k)
                    mbar_wait_final(sfull0 + 8 * ((g - 1 - k) % NSLOT), ((g - 1 - k) / NSLOT) & 1);
        }
    } else if (warp == 3) {
        // ------------------------------------------------ codes from HBM to L2, one unit ahead.  The clusters
        // that share a row of tiles read its codes at about the same time, so without this all of
        // them wait for HBM; the cluster that has the row's first token tile asks for all
        if (lane == 0) {
            const uint32_t row_bytes = (uint32_t)p.kchunks * 8192u;   // codes of 64 rows
            auto prefetch = [&](int u) {
                if (u >= p.n_units || (u % p.n_ttiles != 0 && u >= n_clusters))
                    return;
                const int64_t nb = (int64_t)(u / p.n_ttiles) * 4 + (int)rank * 2;
                if (nb * 64 >= p.Np)
                    return;
                for (uint32_t at = 0; at < 2 * row_bytes; at += 16384)   // (Np is a multiple of 128)
                    bulk_prefetch_l2(p.codes + nb * row_bytes + at, 16384);
            };
            prefetch(cluster);
            int lt = 0;
            for (int u = cluster; u < p.n_units; u += n_clusters, ++lt) {
                prefetch(u + n_clusters);
                if (!mbar_wait(tfull0 + 8 * (lt & 1), (lt >> 1) & 1, &abort_flag, p.status))
                    break;
                mbar_arrive_remote(tempty0 + 8 * (lt & 1), 0);
            }
        }
    } else if (warp >= EPI_WARP && warp < DEQ_WARP) {
        // ------------------------------------------------ epilogue: set `set` takes slots g with g % 2 == set,
        // warp quarter q owns TMEM lanes 32q .. 32q + 31 (channels)
        const int q = warp & 3, set = (warp - EPI_WARP) >> 2;
        const int row = 32 * q + lane;
        const bool storer = q == 0 && lane == 0;
        uint32_t g = 0;
        int lt = 0, stores = 0;
        if (!p.v_ready)
            pdl_wait();   // the bias may come from an earlier kernel (early start: the prepass waited for it)
        // a wait that gives up ends this warp's waits and stores, but not its
        // loops: the warps of a set meet in a barrier at every slot
        bool ok = true;
        for (int u = cluster; u < p.n_units; u += n_clusters, ++lt) {
            const uint32_t buf = lt & 1;
            const int t0 = (u % p.n_ttiles) * BN;
            const int n0 = (u / p.n_ttiles) * 2 * BM + (int)rank * BM;
            const int n = n0 + row;
            const float sn = n < p.N ? p.s[n] : 0.f;
            const float e_n = sn != 0.0f ? sn : 1.0f;   // the EC operand was divided by it
            const float z_n = FORM == kQ8 && sn != 0.0f ? (float)p.z[n] : 0.f;
            const float bias = p.epi.bias && n < p.N ? bf16_lo(p.epi.bias[n]) : 0.f;
            ok = ok && mbar_wait(tfull0 + 8 * buf, (lt >> 1) & 1, &abort_flag, p.status);
            tc_fence_after();
            for (int c = 0; n0 < p.N && c < BN / CHUNK && t0 + c * CHUNK < p.M; ++c, ++g) {
                if ((int)(g & 1u) != set)
                    continue;
                const uint32_t slot = g % NSLOT;
                ok = ok && mbar_wait(sfull0 + 8 * slot, (g / NSLOT) & 1, &abort_flag, p.status);
                __syncwarp();
                const uint32_t acc = tmem_base + ((uint32_t)(32 * q) << 16) + buf * BN + CHUNK * c;
                const uint16_t *mul = reinterpret_cast<const uint16_t *>(base_ptr + o_mul + slot * HALF_SLOT) + row;
                uint16_t *y = reinterpret_cast<uint16_t *>(base_ptr + o_y + slot * HALF_SLOT) + row;
                const float4 *rc = reinterpret_cast<const float4 *>(base_ptr + o_rowc + slot * ROWC_BYTES);
                switch (p.epi.act) {
                case kActRelu:
                    emit_chunk_of<FORM, kActRelu>(acc, e_n, z_n, bias, mul, y, rc, has_mul, has_res);
                    break;
                case kActSilu:
                    emit_chunk_of<FORM, kActSilu>(acc, e_n, z_n, bias, mul, y, rc, has_mul, has_res);
                    break;
                case kActGelu:
                    emit_chunk_of<FORM, kActGelu>(acc, e_n, z_n, bias, mul, y, rc, has_mul, has_res);
                    break;
                case kActGeluTanh:
                    emit_chunk_of<FORM, kActGeluTanh>(acc, e_n, z_n, bias, mul, y, rc, has_mul, has_res);
                    break;
                default:
                    emit_chunk_of<FORM, kActNone>(acc, e_n, z_n, bias, mul, y, rc, has_mul, has_res);
                    break;
                }
                fence_proxy_async_smem();
                asm volatile("bar.sync %0, 128;" ::"r"(1 + set) : "memory");   // the set's four warps
                if (storer && ok) {
                    tma_store_2d(&tm_y, base + o_y + slot * HALF_SLOT, n0, t0 + c * CHUNK);
                    bulk_commit();
                    // the set's slot before this one has been read out: free it
                    if (stores++ > 0) {
                        bulk_wait_read<1>();
                        mbar_arrive(sempty0 + 8 * ((g - 2) % NSLOT));
                    }
                }
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0)
                mbar_arrive_remote(tempty0 + 8 * buf, 0);
        }
        if (storer)
            bulk_wait_all();   // the stores are complete (and the slots read) before the CTA leaves
    } else if (warp >= DEQ_WARP) {
        // ------------------------------------------------ dequantisers: group `grp` takes every fourth stage
        const int grp = (warp - DEQ_WARP) / GROUP_WARPS, w = warp & 3;
        TcDequant<FORM> d(w, lane);
        // this group's stages in order, GROUPS apart: (u, st) the one at work, (fu, fst)
        // the one whose codes are fetched, `src` its unit's codes (null: none)
        int u = cluster, st = grp, fu = 0, fst = 0;
        const uint8_t *src = nullptr;
        auto enter = [&]() {   // the fetching side's unit is fu
            const int nb = (fu / p.n_ttiles) * 4 + (int)rank * 2 + (w >> 1);   // 64-row block of this warp's rows
            src = fu < p.n_units && (int64_t)nb * 64 < p.Np
                      ? p.codes + (int64_t)nb * p.kchunks * 8192 + d.offset() : nullptr;
        };
        auto fetch = [&]() {   // (the codes do not depend on earlier kernels: no wait)
            d.fetch(fst < p.n_main ? src : nullptr, fst);
            fst += GROUPS;
            if (fst >= nst) {
                while (fst >= nst && fu < p.n_units) {
                    fst -= nst;
                    fu += n_clusters;
                }
                enter();
            }
        };
        while (st >= nst && u < p.n_units) {
            st -= nst;
            u += n_clusters;
        }
        fu = u;
        fst = st;
        enter();
        fetch();
        uint32_t slot = (uint32_t)grp, phase = 0;   // (the ring has more stages than there are groups)
        int unit = -1;
        bool ok = true;
        while (u < p.n_units && ok) {
            if (unit != u) {
                unit = u;
                d.set_rows(p.s, p.z, (int64_t)(u / p.n_ttiles) * 2 * BM + rank * BM, p.Np);
            }
            // dequantise before the stage is free
            d.convert();
            fetch();
            // the stage is free once the MMAs of its last round are done
            ok = warp_wait(empty0 + 8 * slot, phase ^ 1, &abort_flag, p.status);
            if (ok && st < p.n_main) {
                d.store(base_ptr + slot * STAGE_BYTES);
                fence_proxy_async_smem();
                __syncwarp();
            }
            if (lane == 0 && ok)
                mbar_arrive_remote(ready0 + 8 * slot, 0);
            st += GROUPS;
            while (st >= nst && u < p.n_units) {
                st -= nst;
                u += n_clusters;
            }
            slot += GROUPS;
            if (slot >= S) {
                slot -= S;
                phase ^= 1;
            }
        }
    }

    tc_fence_before();
    __syncthreads();
    cluster_sync();   // the pair's MMAs and remote arrivals are over
    if (warp == 1) {
        tc_fence_after();
        asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(tmem_base), "r"(2 * BN)
                     : "memory");
    }
    if (tid == 0 && p.v_ready && atomicAdd(p.v_ready + 1, 1u) == gridDim.x - 1) {
        // every CTA is past its waits for the prepass, which has finished: reset
        p.v_ready[0] = 0u;
        p.v_ready[1] = 0u;
    }
}

using PairFn = void (*)(CUtensorMap, CUtensorMap, CUtensorMap, CUtensorMap, CUtensorMap, CUtensorMap, PairParams);

}  // namespace

// Whether the forms with an epilogue take these kernels' 256 x 256 tiles or the
// 128 x 128 ones of tc_tile.cu.  Those read twice as much per product and a stage
// takes longer, but they can split K: they win while they can split it at least
// in two (of equal work the pairs finish first).  Measured in us, tile against
// pair, bf16 / 8 bits:
//   4096 x 4096, r 32    256 tokens (K in 2)  20.5 / 18.4 against 30.5 / 22.2
//                        512 tokens (whole)   36.5 / 32.4 against 31.8 / 23.0
//   14336 x 4096, r 64   256 tokens (K in 2)  47.5 / 36.7 against 76.9 / 47.8
//                        512 tokens (whole)   92.4 / 73.9 against 80.4 / 49.5
//   4096 x 14336, r 64   128 tokens (whole)   32.4 / 27.0 against 30.7 / 21.3
//                         64 tokens (whole)   26.7 / 22.3 against 28.9 / 19.8
//   8192 x 512, r 64    1024 tokens (K in 2)  31.2 / 24.9 against 49.3 / 32.2
//                       1536 tokens (whole)   52.4 / 40.2 against 51.1 / 33.1
//   2048 x 512, no EC   4096 tokens (whole)   21.6 / 17.5 against 18.5 / 22.2
// In 8 bits without the EC the pairs alone need a prepass (of the code sums).  It
// reads all the tokens, so its cost grows with them, and what the pairs win with the
// channels: there they are taken, while the tiles have an SM each, up to as many
// blocks of 128 tokens as of 128 channels.  Tile against pair:
//   14336 x 4096   256 tokens (K in 2) 33.6 against 52.3, 320 55.9 / 53.1, 512 58.3 / 54.2, 640 110.2 / 55.5
//    4096 x 4096   256 tokens (K in 2) 17.1 against 22.4, 320 24.1 / 22.6, 512 25.6 / 23.2
//     512 x 4096   384 tokens 13.3 against 12.6, 512 13.7 / 12.6
//    4096 x 14336   40 tokens 18.8 against 19.7, 64 20.2 / 19.8, 128 25.1 / 21.0
//     512 x 14336  128 tokens 13.5 against 10.2
//    1032 x 2744   400 tokens 16.7 against 16.8, 513 17.2 / 17.6, 700 19.2 / 18.4
//   28672 x 1024  1300 tokens 100.9 against 95.5, 2000 101.6 / 117.0
//    8192 x 512   4096 tokens 39.2 against 44.4
//    2048 x 512   4096 tokens 18.9 against 21.8, 5000 (more tiles than SMs) 35.1 / 23.4
bool tc_use_pair(const Packed &pk, int64_t M, bool ec, int form, int num_sms)
{
    if (M <= (form == kQ8 ? 32 : 64))
        return false;
    const int64_t tok = M <= 64 ? 64 : 128, tiles = (M + tok - 1) / tok * (pk.Np / 128);
    if (form == kQ8 && !ec)
        return tiles > num_sms || (2 * tiles > num_sms && (M + 127) / 128 <= pk.Np / 128);
    return 2 * tiles + (ec ? tc_prepass2_room(pk, M, num_sms) : 0) > num_sms;
}

cudaError_t launch_tc_pair(const Packed &pk, const void *x, void *y, int64_t M, const float *v, bool ec,
                           const CUtensorMap *bt, int *status, cudaStream_t st, int num_sms,
                           unsigned *v_ready, unsigned v_expected, int form, const Epilogue &epi, int64_t ldx,
                           const float *rowc)
{
    const int BK = tc_stage_k(form);
    const uint64_t xd[2] = {(uint64_t)pk.K, (uint64_t)M};
    const uint64_t xst[1] = {(uint64_t)ldx * (uint64_t)(ROW_BYTES / BK)};
    const uint32_t xb[2] = {(uint32_t)BK, (uint32_t)(BN / 2)};
    CUtensorMap tm_x, tm_v, tm_y, tm_mul, tm_res;
    cudaError_t e = make_map_nd(&tm_x, x, form == kQ8 ? CU_TENSOR_MAP_DATA_TYPE_UINT8
                                                      : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16,
                                2, xd, xst, xb, CU_TENSOR_MAP_SWIZZLE_128B);
    const bool use_ec = ec && pk.r > 0;
    tm_v = tm_x;   // unused without the EC
    if (e == cudaSuccess && use_ec)
        e = make_map(&tm_v, v, CU_TENSOR_MAP_DATA_TYPE_FLOAT32, 4, (uint64_t)pk.rp, (uint64_t)M, 32, BN / 2,
                     CU_TENSOR_MAP_SWIZZLE_128B);
    auto out_map = [&](CUtensorMap *m, const void *ptr) {
        if (e == cudaSuccess)
            e = make_map(m, ptr, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, (uint64_t)pk.N, (uint64_t)M, BM, CHUNK,
                         CU_TENSOR_MAP_SWIZZLE_NONE);
    };
    out_map(&tm_y, y);
    tm_mul = tm_y;   // unused without one
    tm_res = tm_y;
    if (epi.mul)
        out_map(&tm_mul, epi.mul);
    if (epi.residual)
        out_map(&tm_res, epi.residual);
    if (e != cudaSuccess)
        return e;
    PairParams p;
    p.M = M;
    p.N = pk.N;
    p.Np = pk.Np;
    p.kchunks = (int)(pk.Kp / 256);
    p.n_main = (int)(pk.Kp / BK);
    p.n_ec = use_ec ? (pk.rp + 31) / 32 : 0;
    p.rp = pk.rp;
    p.n_ttiles = (int)((M + BN - 1) / BN);
    p.n_units = p.n_ttiles * (int)((pk.Np + 2 * BM - 1) / (2 * BM));
    p.stages = pair_stages(epi.mul != nullptr);
    p.codes = reinterpret_cast<const uint8_t *>(pk.codes);
    p.s = pk.s;
    p.z = pk.z;
    p.status = status;
    p.v_ready = use_ec ? v_ready : nullptr;
    p.v_expected = v_expected;
    p.epi = epi;
    p.rowc = rowc;
    const PairFn fn = form == kQ8 ? tc_pair_kernel<kQ8> : tc_pair_kernel<kEpi>;
    const int smem = pair_smem_bytes(epi.mul != nullptr);
    e = raise_smem_limit(reinterpret_cast<const void *>(fn), smem);
    if (e != cudaSuccess)
        return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(2 * std::min(p.n_units, num_sms / 2)));
    cfg.blockDim = dim3(THREADS);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, fn, tm_x, use_ec ? *bt : tm_x, tm_v, tm_mul, tm_res, tm_y, p);
}

}  // namespace spear
