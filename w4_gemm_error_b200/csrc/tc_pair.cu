// W4 GEMM of many tokens with an epilogue, on pairs of CTAs (tcgen05,
// cta_group::2): the forms kEpi (bf16 activations) and kQ8 (e4m3) of the
// forward pass from 129 tokens on.
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
// Roles in each CTA (20 warps):
//   warp 0       TMA producer of the stages: its 128 tokens of x and its 128
//                rows of codes (EC stages: v and B^T/e instead)
//   warp 1       TMEM allocation; in the pair's first CTA the one thread that
//                issues the MMAs of both
//   warp 2       loader of the epilogue's operands (multiplier, residual and
//                per-token constants) into slots of 32 tokens x 128 channels
//   warps 4-11   epilogue, two sets of four warps (each warp its 32 TMEM
//                lanes) taking alternate slots: accumulator from TMEM, the
//                formula above, y into the slot (over the residual, element by
//                element) and from there to HBM by one TMA store a slot
//   warps 12-19  dequantisers, two groups of four taking alternate stages,
//                one weight row a thread
// Two accumulators of 256 columns in TMEM: the epilogue of a tile overlaps the
// main loop of the next.  Every wait is bounded (about a second); one that runs
// out sets the handle's status word and the kernel winds down.
#include <algorithm>

#include "async_utils.cuh"
#include "epilogue.cuh"
#include "tc_gemm.h"
#include "tensor_map.h"

namespace spear {
namespace {

constexpr int BM = 128;                 // weight rows of a CTA (256 a pair)
constexpr int BN = 256;                 // tokens of a pair (128 staged by each CTA)
constexpr int ROW_BYTES = 128;
constexpr int A_BYTES = BM * ROW_BYTES;
constexpr int B_BYTES = (BN / 2) * ROW_BYTES;
constexpr int STAGES = 4;
constexpr int CHUNK = 32;               // tokens of an epilogue slot
constexpr int NSLOT = 4;
constexpr int SLOT_BYTES = 2 * CHUNK * BM * 2;   // multiplier, then residual / y
constexpr int ROWC_BYTES = CHUNK * 8;
constexpr int THREADS = 640;
constexpr int EPI_WARP = 4, DEQ_WARP = 12;

__host__ __device__ constexpr int pair_bk(int form) { return form == kQ8 ? 128 : 64; }
__host__ __device__ constexpr int pair_c_bytes(int form) { return BM * pair_bk(form) / 2; }
__host__ __device__ constexpr int pair_stage_bytes(int form) { return A_BYTES + B_BYTES + pair_c_bytes(form); }
__host__ __device__ constexpr int pair_smem_bytes(int form)
{
    return STAGES * pair_stage_bytes(form) + NSLOT * (SLOT_BYTES + ROWC_BYTES) + 1024;
}

struct PairParams {
    int64_t M, N, Np;
    int kchunks;             // Kp / 256
    int n_main, n_ec, rp;    // stages of the main loop and of the EC; columns of v
    int n_ttiles, n_units;
    const float *s;
    const uint8_t *z;
    int *status;
    unsigned *v_ready;       // as TcParams::v_ready (tc_gemm.cu)
    unsigned v_expected;
    Epilogue epi;
    const float2 *rowc;      // form kQ8: as TcParams::rowc, padded to whole chunks
};

// Bounded wait with cluster scope (arrivals from the other CTA of the pair).
__device__ __forceinline__ bool mbar_wait_cluster(uint32_t bar, uint32_t parity, volatile int *abort_flag,
                                                  int *status)
{
    const long long t0 = clock64();
    while (!mbar_try_wait_cluster(bar, parity, kWaitSleepNs)) {
        if (*abort_flag)
            return false;
        if (clock64() - t0 > kWaitBudgetCycles) {
            *abort_flag = 1;
            atomicOr(status, kStatusTimeout);
            return false;
        }
    }
    return true;
}

// Bounded wait until the prepass has counted everything it writes.
__device__ __forceinline__ bool wait_prepass(const PairParams &p, volatile int *abort_flag)
{
    const long long t0 = clock64();
    while (ld_acquire_gpu(p.v_ready) < p.v_expected) {
        if (*abort_flag || clock64() - t0 > kWaitBudgetCycles) {
            *abort_flag = 1;
            atomicOr(p.status, kStatusTimeout);
            return false;
        }
        __nanosleep(64);
    }
    asm volatile("fence.proxy.async;" ::: "memory");   // the copies that follow read what it wrote
    return true;
}

// One slot's outputs of this thread: channel n (row `row` of the CTA), the 32
// tokens of the chunk, the accumulator in acc.  mul and y are its columns of
// the slot's two halves ([32 tokens][128 channels] bf16).
template <int FORM, int ACT>
__device__ __forceinline__ void emit_chunk(const uint32_t (&acc)[CHUNK], float e_n, float z_n, float bias,
                                           const uint16_t *mul, uint16_t *y, const float2 *rc, bool has_mul,
                                           bool has_res)
{
#pragma unroll
    for (int j = 0; j < CHUNK; ++j) {
        float v = __uint_as_float(acc[j]);
        if constexpr (FORM == kQ8) {
            const float2 c = rc[j];
            v = c.x * e_n * (v - z_n * c.y);
        } else {
            v = e_n * v;
        }
        v = activate(v + bias, ACT);
        if (has_mul)
            v *= bf16_lo(mul[j * BM]);
        if (has_res)
            v += bf16_lo(y[j * BM]);
        y[j * BM] = __bfloat16_as_ushort(__float2bfloat16_rn(v));
    }
}

template <int FORM>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(THREADS, 1)
tc_pair_kernel(const __grid_constant__ CUtensorMap tm_x, const __grid_constant__ CUtensorMap tm_codes,
               const __grid_constant__ CUtensorMap tm_bt, const __grid_constant__ CUtensorMap tm_v,
               const __grid_constant__ CUtensorMap tm_mul, const __grid_constant__ CUtensorMap tm_res,
               const __grid_constant__ CUtensorMap tm_y, PairParams p)
{
    constexpr int BK = pair_bk(FORM);
    constexpr int C_BYTES = pair_c_bytes(FORM);
    constexpr int STAGE_BYTES = pair_stage_bytes(FORM);
    constexpr int SUB = 256 / BK;
    constexpr int GROUP_WARPS = 4;
    extern __shared__ uint8_t smem_raw[];
    // full, ready and empty of each stage; accumulator full and empty; slot full and empty; drain
    __shared__ __align__(8) uint64_t bars[3 * STAGES + 4 + 2 * NSLOT + 1];
    __shared__ uint32_t tmem_base_slot;
    __shared__ volatile int abort_flag;

    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const uint32_t base = (smem_addr(smem_raw) + 1023u) & ~1023u;
    uint8_t *const base_ptr = smem_raw + (base - smem_addr(smem_raw));
    const uint32_t rank = cluster_ctarank();
    const uint32_t full0 = smem_addr(&bars[0]);
    const uint32_t ready0 = smem_addr(&bars[STAGES]);         // first CTA's: both CTAs' operands are staged
    const uint32_t empty0 = smem_addr(&bars[2 * STAGES]);
    const uint32_t tfull0 = smem_addr(&bars[3 * STAGES]);
    const uint32_t tempty0 = smem_addr(&bars[3 * STAGES + 2]);   // first CTA's: both epilogues are done
    const uint32_t sfull0 = smem_addr(&bars[3 * STAGES + 4]);
    const uint32_t sempty0 = smem_addr(&bars[3 * STAGES + 4 + NSLOT]);
    const uint32_t drain = smem_addr(&bars[3 * STAGES + 4 + 2 * NSLOT]);
    constexpr uint32_t kSlots = STAGES * STAGE_BYTES, kRowc = kSlots + NSLOT * SLOT_BYTES;

    if (tid == 0) {
        abort_flag = 0;
        for (int s = 0; s < STAGES; ++s) {
            mbar_init(full0 + 8 * s, 1);
            mbar_init(ready0 + 8 * s, 2 * GROUP_WARPS);
            mbar_init(empty0 + 8 * s, 1);
        }
        for (int b = 0; b < 2; ++b) {
            mbar_init(tfull0 + 8 * b, 1);
            mbar_init(tempty0 + 8 * b, 2 * 8);
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
        if (lane == 0) {
            if (!p.v_ready)
                pdl_wait();   // x and v come from earlier kernels in the stream
            bool v_seen = p.v_ready == nullptr;
            uint32_t g = 0;
            bool ok = true;
            for (int u = cluster; u < p.n_units && ok; u += n_clusters) {
                const int t0 = (u % p.n_ttiles) * BN + (int)rank * (BN / 2);
                const int n0 = (u / p.n_ttiles) * 2 * BM + (int)rank * BM;
                for (int i = 0; i < nst; ++i, ++g) {
                    const uint32_t slot = g % STAGES, phase = (g / STAGES) & 1;
                    if (!mbar_wait(empty0 + 8 * slot, phase ^ 1, &abort_flag, p.status)) {
                        ok = false;
                        break;
                    }
                    const uint32_t sb = base + slot * STAGE_BYTES, full = full0 + 8 * slot;
                    if (i < p.n_main) {
                        mbar_expect_tx(full, B_BYTES + C_BYTES);
                        tma_load_2d(sb + A_BYTES, &tm_x, i * BK, t0, full);
                        const int blk = (n0 / 64) * p.kchunks + i / SUB, sub = i % SUB;
                        tma_load_4d(sb + A_BYTES + B_BYTES, &tm_codes, 0, sub, 0, blk, full);
                        tma_load_4d(sb + A_BYTES + B_BYTES + C_BYTES / 2, &tm_codes, 0, sub, 0, blk + p.kchunks,
                                    full);
                    } else {
                        if (!v_seen && !wait_prepass(p, &abort_flag)) {
                            ok = false;
                            break;
                        }
                        v_seen = true;
                        const int e = i - p.n_main;   // 32 tf32 values of j a stage
                        mbar_expect_tx(full, A_BYTES + B_BYTES);
                        tma_load_2d(sb, &tm_bt, e * 32, n0, full);
                        tma_load_2d(sb + A_BYTES, &tm_v, e * 32, t0, full);
                    }
                }
            }
            // do not leave while copies this CTA issued may still land (the
            // dequantisers waited for every stage unless a wait gave up)
            if (abort_flag)
                for (uint32_t k = 0; k < STAGES && k < g; ++k)
                    mbar_wait_final(full0 + 8 * ((g - 1 - k) % STAGES), ((g - 1 - k) / STAGES) & 1);
            // early start: this grid completes only after its predecessor
            if (p.v_ready)
                pdl_wait();
        }
    } else if (warp == 1) {
        // ------------------------------------------------ MMA issuer of the pair
        if (lane == 0 && rank == 0) {
            const uint32_t shape = ((uint32_t)(BN >> 3) << 17) | ((uint32_t)(2 * BM >> 4) << 24) | (1u << 4);
            const uint32_t idesc = shape | (FORM == kQ8 ? 0u : (1u << 7) | (1u << 10));
            const uint32_t idesc_tf32 = shape | (2u << 7) | (2u << 10);
            uint32_t g = 0;
            int lt = 0;
            bool ok = true;
            for (int u = cluster; u < p.n_units && ok; u += n_clusters, ++lt) {
                const uint32_t buf = lt & 1;
                if (!mbar_wait_cluster(tempty0 + 8 * buf, ((lt >> 1) & 1) ^ 1, &abort_flag, p.status))
                    break;
                tc_fence_after();
                const uint32_t d_tmem = tmem_base + buf * BN;
                for (int i = 0; i < nst; ++i, ++g) {
                    const uint32_t slot = g % STAGES, phase = (g / STAGES) & 1;
                    if (!mbar_wait_cluster(ready0 + 8 * slot, phase, &abort_flag, p.status)) {
                        ok = false;
                        break;
                    }
                    tc_fence_after();
                    const uint32_t sb = base + slot * STAGE_BYTES;
                    const uint64_t a_desc = smem_desc_sw128(sb), b_desc = smem_desc_sw128(sb + A_BYTES);
                    if (i < p.n_main) {
                        // 32 bytes of k an instruction
                        for (int k = 0; k < ROW_BYTES / 32; ++k) {
                            const uint32_t accumulate = (i > 0 || k > 0) ? 1u : 0u;
                            if constexpr (FORM == kQ8)
                                mma2_e4m3(d_tmem, a_desc + 2 * k, b_desc + 2 * k, idesc, accumulate);
                            else
                                mma2_bf16(d_tmem, a_desc + 2 * k, b_desc + 2 * k, idesc, accumulate);
                        }
                    } else {
                        const int rem = p.rp - (i - p.n_main) * 32;
                        const int ksteps = (rem < 32 ? rem : 32) / 8;
                        for (int k = 0; k < ksteps; ++k)
                            mma2_tf32(d_tmem, a_desc + 2 * k, b_desc + 2 * k, idesc_tf32, 1u);
                    }
                    mma2_commit_both(empty0 + 8 * slot);
                }
                if (ok)
                    mma2_commit_both(tfull0 + 8 * buf);
            }
            // every MMA this thread issued is complete before TMEM is released
            mma2_commit(drain);
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
            const uint32_t bytes = (p.epi.mul ? CHUNK * BM * 2u : 0u) + (p.epi.residual ? CHUNK * BM * 2u : 0u) +
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
                    const uint32_t bar = sfull0 + 8 * slot, dst = base + kSlots + slot * SLOT_BYTES;
                    if (bytes == 0) {
                        mbar_arrive(bar);
                        continue;
                    }
                    if (!ready && !wait_prepass(p, &abort_flag)) {
                        ok = false;
                        break;
                    }
                    ready = true;
                    mbar_expect_tx(bar, bytes);
                    if (p.epi.mul)
                        tma_load_2d(dst, &tm_mul, n0, t0 + c * CHUNK, bar);
                    if (p.epi.residual)
                        tma_load_2d(dst + SLOT_BYTES / 2, &tm_res, n0, t0 + c * CHUNK, bar);
                    if (FORM == kQ8)
                        bulk_load(base + kRowc + slot * ROWC_BYTES, p.rowc + t0 + c * CHUNK, ROWC_BYTES, bar);
                }
            }
            // (the epilogue waited for every slot unless a wait gave up)
            if (abort_flag && bytes)
                for (uint32_t k = 0; k < NSLOT && k < g; ++k)
                    mbar_wait_final(sfull0 + 8 * ((g - 1 - k) % NSLOT), ((g - 1 - k) / NSLOT) & 1);
        }
    } else if (warp >= EPI_WARP && warp < DEQ_WARP) {
        // ------------------------------------------------ epilogue: set `set` takes slots g with g % 2 == set,
        // warp quarter q owns TMEM lanes 32q .. 32q + 31 (channels)
        const int q = warp & 3, set = (warp - EPI_WARP) >> 2;
        const int row = 32 * q + lane;
        const bool storer = q == 0 && lane == 0;
        const bool has_mul = p.epi.mul != nullptr, has_res = p.epi.residual != nullptr;
        uint32_t g = 0;
        int lt = 0, stores = 0;
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
            const float bias = p.epi.bias && n < p.N ? bf16_lo(__ldg(p.epi.bias + n)) : 0.f;
            ok = ok && mbar_wait(tfull0 + 8 * buf, (lt >> 1) & 1, &abort_flag, p.status);
            tc_fence_after();
            for (int c = 0; n0 < p.N && c < BN / CHUNK && t0 + c * CHUNK < p.M; ++c, ++g) {
                if ((int)(g & 1u) != set)
                    continue;
                const uint32_t slot = g % NSLOT;
                ok = ok && mbar_wait(sfull0 + 8 * slot, (g / NSLOT) & 1, &abort_flag, p.status);
                __syncwarp();
                uint32_t acc[CHUNK];
                tmem_ld_32x32b_x32(tmem_base + ((uint32_t)(32 * q) << 16) + buf * BN + CHUNK * c, acc);
                uint8_t *const sp = base_ptr + kSlots + slot * SLOT_BYTES;
                const uint16_t *mul = reinterpret_cast<const uint16_t *>(sp) + row;
                uint16_t *y = reinterpret_cast<uint16_t *>(sp + SLOT_BYTES / 2) + row;
                const float2 *rc = reinterpret_cast<const float2 *>(base_ptr + kRowc + slot * ROWC_BYTES);
                switch (p.epi.act) {
                case kActRelu: emit_chunk<FORM, kActRelu>(acc, e_n, z_n, bias, mul, y, rc, has_mul, has_res); break;
                case kActSilu: emit_chunk<FORM, kActSilu>(acc, e_n, z_n, bias, mul, y, rc, has_mul, has_res); break;
                case kActGelu: emit_chunk<FORM, kActGelu>(acc, e_n, z_n, bias, mul, y, rc, has_mul, has_res); break;
                case kActGeluTanh:
                    emit_chunk<FORM, kActGeluTanh>(acc, e_n, z_n, bias, mul, y, rc, has_mul, has_res);
                    break;
                default: emit_chunk<FORM, kActNone>(acc, e_n, z_n, bias, mul, y, rc, has_mul, has_res); break;
                }
                fence_proxy_async_smem();
                asm volatile("bar.sync %0, 128;" ::"r"(1 + set) : "memory");   // the set's four warps
                if (storer && ok) {
                    tma_store_2d(&tm_y, base + kSlots + slot * SLOT_BYTES + SLOT_BYTES / 2, n0, t0 + c * CHUNK);
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
        // ------------------------------------------------ dequantisers: group `grp` takes the stages g with
        // g % 2 == grp, one weight row a thread
        const uint32_t grp = (uint32_t)(warp - DEQ_WARP) / GROUP_WARPS;
        const int i = 32 * (warp & 3) + lane;
        uint32_t g = 0;
        bool ok = true;
        for (int u = cluster; u < p.n_units && ok; u += n_clusters) {
            const int64_t n = (int64_t)(u / p.n_ttiles) * 2 * BM + rank * BM + i;
            // a row whose s is 0 has weights 0, whatever its codes (the epilogue scales it by 1)
            const bool live = n < p.Np && p.s[n] != 0.0f;
            const uint32_t negz = live ? dequant_bias<false>(p.z[n]) : 0u;
            const uint32_t mulz = live ? 0x3F803F80u : 0u;
            const uint32_t nib = live ? 0x0F0F0F0Fu : 0u;
            for (int st = 0; st < nst; ++st, ++g) {
                if ((g & 1u) != grp)
                    continue;
                const uint32_t slot = g % STAGES, phase = (g / STAGES) & 1;
                if (!mbar_wait(full0 + 8 * slot, phase, &abort_flag, p.status)) {
                    ok = false;
                    break;
                }
                if (st < p.n_main) {
                    uint8_t *sb = base_ptr + slot * STAGE_BYTES;
                    uint8_t *arow = sb + i * ROW_BYTES;
                    if constexpr (FORM == kQ8) {
                        // 64 bytes of codes (128 k): four 16-byte pieces permuted by row bits 1 and 2
                        // (64-byte TMA swizzle), each 32 e4m3 values
                        const uint8_t *crow = sb + A_BYTES + B_BYTES + i * 64;
                        uint4 w[4];
#pragma unroll
                        for (int c = 0; c < 4; ++c)
                            w[c] = *reinterpret_cast<const uint4 *>(crow + ((c ^ ((i >> 1) & 3)) << 4));
#pragma unroll
                        for (int c = 0; c < 4; ++c) {
                            uint4 o;
                            nibbles_to_e4m3(w[c].x, nib, o.x, o.y);
                            nibbles_to_e4m3(w[c].y, nib, o.z, o.w);
                            *reinterpret_cast<uint4 *>(arow + (((2 * c) ^ (i & 7)) << 4)) = o;
                            nibbles_to_e4m3(w[c].z, nib, o.x, o.y);
                            nibbles_to_e4m3(w[c].w, nib, o.z, o.w);
                            *reinterpret_cast<uint4 *>(arow + (((2 * c + 1) ^ (i & 7)) << 4)) = o;
                        }
                    } else {
                        // 32 bytes of codes (64 k): two 16-byte pieces swapped in rows with bit 2
                        // set (32-byte TMA swizzle), each 32 bf16 values
                        const uint8_t *crow = sb + A_BYTES + B_BYTES + i * 32;
#pragma unroll
                        for (int h = 0; h < 2; ++h) {
                            const uint4 w = *reinterpret_cast<const uint4 *>(crow + ((h ^ ((i >> 2) & 1)) << 4));
                            const uint32_t words[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
                            for (int jj = 0; jj < 4; ++jj) {
                                uint4 o;
                                o.x = dequant_pair_mul(words[jj], mulz, negz);
                                o.y = dequant_pair_mul(words[jj] >> 4, mulz, negz);
                                o.z = dequant_pair_mul(words[jj] >> 8, mulz, negz);
                                o.w = dequant_pair_mul(words[jj] >> 12, mulz, negz);
                                *reinterpret_cast<uint4 *>(arow + (((4 * h + jj) ^ (i & 7)) << 4)) = o;
                            }
                        }
                    }
                    fence_proxy_async_smem();
                }
                __syncwarp();
                if (lane == 0)
                    mbar_arrive_remote(ready0 + 8 * slot, 0);
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

using PairFn = void (*)(CUtensorMap, CUtensorMap, CUtensorMap, CUtensorMap, CUtensorMap, CUtensorMap, CUtensorMap,
                        PairParams);

}  // namespace

cudaError_t launch_tc_pair(const Packed &pk, const void *x, void *y, int64_t M, const float *v, bool ec,
                           const CUtensorMap &codes, const CUtensorMap &bt, int *status, cudaStream_t st, int num_sms,
                           unsigned *v_ready, unsigned v_expected, int form, const Epilogue &epi, int64_t ldx,
                           const float2 *rowc)
{
    const int BK = pair_bk(form);
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
    p.s = pk.s;
    p.z = pk.z;
    p.status = status;
    p.v_ready = use_ec ? v_ready : nullptr;
    p.v_expected = v_expected;
    p.epi = epi;
    p.rowc = rowc;
    const PairFn fn = form == kQ8 ? tc_pair_kernel<kQ8> : tc_pair_kernel<kEpi>;
    const int smem = pair_smem_bytes(form);
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
    return cudaLaunchKernelEx(&cfg, fn, tm_x, codes, use_ec ? bt : codes, tm_v, tm_mul, tm_res, tm_y, p);
}

}  // namespace spear
