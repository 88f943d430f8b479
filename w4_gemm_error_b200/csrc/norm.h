// Row norm and 8-bit quantisation of activations (library-internal).
#pragma once
#include <cuda_runtime.h>
#include <cstdint>

namespace spear {

// Argument meanings as spear_w4ec_rmsnorm; w = null: quantise x itself.
cudaError_t launch_norm(const void *x, const void *residual, const void *w, float eps, int64_t M, int64_t K, void *h,
                        void *y, void *q, float *s, cudaStream_t st);

}  // namespace spear
