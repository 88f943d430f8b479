// tcgen05 / TMEM tile kernel for larger token counts (library-internal).
#pragma once
#include <cuda_runtime.h>
#include <cstdint>

#include "kernels.h"

namespace spear {

struct TcWork {
    void *maps = nullptr;        // host-side tensor maps of the packed operands
    float *part = nullptr;       // split-K partials
    size_t part_floats = 0;
    unsigned *counters = nullptr;
    int n_counters = 0;
};

bool tc_available(const Packed &pk);
cudaError_t tc_alloc(const Packed &pk, int64_t max_M, int num_sms, TcWork &w);
void tc_free(TcWork &w);
cudaError_t tc_prepare(const Packed &pk, TcWork &w);
// Gate and v = g * (x . A) for many tokens on the tensor cores (128 tokens per CTA).
// `ready` (may be null): counted once per CTA (release) when its v is written;
// ceil(M / 128) counts in all.
bool tc_prepass_supported(const Packed &pk);
cudaError_t launch_tc_prepass(const Packed &pk, const void *x, int64_t M, float *v, bool tf32, float *g,
                              const TcWork &w, int *status, cudaStream_t st, unsigned *ready);
// v: the prepass output in fp32 rounded to tf32 ([M][rp]), read when `ec` is set.
// v_ready (may be null; used only with `ec`): the kernel starts its main stages
// without waiting for its predecessor, which must be a prepass that counts
// v_expected completions into v_ready[0] and starts its dependents only once x is
// complete; v_ready[0..1] are zero between calls.
cudaError_t launch_tc(const Packed &pk, const void *x, void *y, int64_t M, const float *v, bool ec,
                      const TcWork &w, int *status, bool zero_wait_budget, cudaStream_t st, int num_sms,
                      unsigned *v_ready, unsigned v_expected);

// ---- the forms kEpi and kQ8 of epilogue.cuh

// Two constants a token of form kQ8, xs[t] and 2^-9 sum_k xq[t,k], pairs of
// tokens together (c0[2i], c0[2i+1], c1[2i], c1[2i+1]); whole chunks of 32
// tokens are allocated.  Index of c0; c1 is 2 on.
__host__ __device__ constexpr int64_t rowc_at(int64_t t) { return 4 * (t / 2) + (t & 1); }
inline size_t rowc_floats(int64_t max_M) { return (size_t)((max_M + 31) / 32 * 32) * 2; }

struct Epilogue;
const CUtensorMap *tc_map_g(const TcWork &w);    // tensor maps of G and of B^T/e
const CUtensorMap *tc_map_bt(const TcWork &w);   // (of a packed layer with an EC)

// Prepass on the tensor cores, K split over a cluster (tc_prepass.cu): v with
// `ec`, rowc in form kQ8 (xs: its scales).  Rows of x are ldx elements apart.
// `ready` (may be null) is counted *expected times in all, once per CTA when
// what it writes is there.
// SMs to leave free for a kernel that is to start beside it: its CTAs and a
// quarter more, since whole clusters of up to 8 need their places.
int64_t tc_prepass2_room(const Packed &pk, int64_t M, int num_sms);
cudaError_t launch_tc_prepass2(const Packed &pk, const void *x, int64_t ldx, const float *xs, int64_t M, bool ec,
                               float *v, float *rowc, int form, const CUtensorMap *g, int *status, cudaStream_t st,
                               int num_sms, unsigned *ready, unsigned *expected);

// The product and epilogue: pairs of CTAs on 256 x 256 tiles (tc_pair.cu, which
// reads rowc), or one CTA on 128 x up to 128 with K split over a cluster
// (tc_tile.cu, which sums the codes itself).  v_ready, v_expected: as launch_tc.
bool tc_use_pair(const Packed &pk, int64_t M, bool ec, int form, int num_sms);
cudaError_t launch_tc_pair(const Packed &pk, const void *x, void *y, int64_t M, const float *v, bool ec,
                           const CUtensorMap *bt, int *status, cudaStream_t st, int num_sms, unsigned *v_ready,
                           unsigned v_expected, int form, const Epilogue &epi, int64_t ldx, const float *rowc);
cudaError_t launch_tc_tile(const Packed &pk, const void *x, void *y, int64_t M, const float *v, bool ec,
                           const CUtensorMap *bt, int *status, cudaStream_t st, int num_sms, unsigned *v_ready,
                           unsigned v_expected, int form, const Epilogue &epi, int64_t ldx);

}  // namespace spear
