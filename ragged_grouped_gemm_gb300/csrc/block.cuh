// The pre-norm block around the MoE layer: layer norm with its backward, and
// the residual dropout fused into the combine.
#pragma once
#include <cstddef>
#include <cstdint>
#include <cuda_runtime.h>

namespace moe {

// Widest row of the layer norm kernels (their rows live in registers).
constexpr int kNormMaxCols = 32768;

// The waits for rows that arrive in shared memory.  One that runs out ends the block's (or
// cluster's) work: the rows it has left, and every sum over them, are NaN, and the status
// words, where there are any, say DEV_TIMEOUT.
struct RowWait {
  uint64_t limit_ns = 2000000000ull;
  int64_t withheld = -1;        // a self-test's row that is never asked for
  int32_t* status = nullptr;
};

// y = (x - mean) * rstd * gamma + beta over rows of d elements (d % 8 == 0);
// x bf16 or fp32, y bf16, mean and rstd nullable.
cudaError_t launch_layernorm(int64_t rows, int d, const void* x, bool x_f32, const float* gamma, const float* beta,
                             float eps, void* y, float* mean, float* rstd, cudaStream_t st, const RowWait& wait = {});
// Floats of scratch launch_layernorm_bwd needs for its partial sums.
size_t layernorm_bwd_floats(int64_t rows, int d);
// dx = rstd (g - mean(g) - xhat mean(g xhat)) + dres with g = dy gamma;
// dgamma = sum dy xhat, dbeta = sum dy (nullable), added in a fixed order.
cudaError_t launch_layernorm_bwd(int64_t rows, int d, const void* dy, const void* x, bool x_f32, const float* gamma,
                                 const float* mean, const float* rstd, const void* dres, void* dx, float* dgamma,
                                 float* dbeta, float* scratch, cudaStream_t st, const RowWait& wait = {});

// out = resid + keep * scale * (sum_k w y_perm[row] + y_shared); out and resid
// (nullable) bf16 or fp32.  An element is kept when its random word is at
// least `threshold`; threshold 0 keeps all without drawing any.
cudaError_t launch_combine_dropout(int n_tok, int d, int top_k, const void* y_perm, const int32_t* row_of_copy,
                                   const float* topk_w, const void* y_shared, const void* resid, bool f32,
                                   const int64_t* rng, uint32_t threshold, float scale, void* out, cudaStream_t st);
// dy = bf16(keep * scale * dout), n elements (n % 8 == 0).
cudaError_t launch_dropout_bwd(int64_t n, const void* dout, bool f32, const int64_t* rng, uint32_t threshold,
                               float scale, void* dy, cudaStream_t st);

}  // namespace moe
