// The router's balance loss over ragged sequences, with its z-loss, and the
// dense router gradient (see seq_balance.cu).
#pragma once
#include <algorithm>
#include <cstddef>
#include <cstdint>
#include <cuda_runtime.h>

namespace moe {

struct SeqBalanceArgs {
  int n_tok, n_exp, top_k, gate;
  int n_seq;
  const float* logits;         // [N, E]
  const int32_t* topk_idx;     // [N, K]
  const int32_t* seq_offsets;  // [S + 1]
  float coef, z_coef;
  const float* dloss;          // one float (nullable: 1)
  int32_t* counts;             // [S, E]
  float* loss;                 // [2]
  float* dlogits;              // [N, E], nullable
  float4* part;                // one a block of the launch (seq_balance_parts), 16-byte aligned
  int32_t* head;               // 4 int32: sequences that are not empty, their tokens, offsets that decrease
  int32_t* ticket;             // zero before the launch, left zero
  int32_t* status;
};
// Blocks of a launch at most: 8 tokens a block, or one cluster for few.
constexpr int kSeqBalanceCluster = 8;
inline int64_t seq_balance_parts(int n_tok) {
  return n_tok > 0 ? std::max<int64_t>(kSeqBalanceCluster, (static_cast<int64_t>(n_tok) + 7) / 8) : 0;
}
cudaError_t launch_seq_balance(const SeqBalanceArgs& a, cudaStream_t st);

// dlogits [N, E] fp32 as a sum of three bf16 terms [N, 3 * E8], E8 = E rounded up to 8, term i in the columns
// from i * E8 (zero past E): what remains of a number after its terms is below 2^-24 of it.  Also
// offsets = {0, N} and the starts of `slices` runs of `slice_rows` tokens.
inline int router_term_cols(int n_exp) { return (n_exp + 7) / 8 * 8; }
cudaError_t launch_router_terms(const float* dl, int n_tok, int n_exp, void* terms, int32_t* dense, int32_t* slices,
                                int n_slices, int slice_rows, cudaStream_t st);
// dw[e, :] = dw_in[e, :] + the sum over the slices and terms (1 or 3) of part[slice][term * E8 + e][d].
cudaError_t launch_router_dw(const float* part, int n_slices, int terms, int n_exp, int d, const float* dw_in,
                             float* dw, cudaStream_t st);

// The whole dense router gradient of up to kRouterFew experts; `part` holds part_bytes: as many runs of tokens as partial
// products of E * D floats fit, one (which needs none) at least.
constexpr int kRouterFew = 16;
constexpr int kRouterFewRuns = 48;
cudaError_t launch_router_few(const float* dl, const void* x, const void* w_gate, const void* dx_in, void* dx,
                              float* part, size_t part_bytes, int n_tok, int d, int n_exp, const float* dw_in,
                              float* dw, cudaStream_t st);

// And of any number of experts where there is little to do in all.  What it reads again grows with tokens x columns x
// experts: beside the tensor cores' four launches 256 x 2048 x 128 takes 9.1 us a call for 17.6, 512 x 2048 x 64 11.8 for 18.5,
// 512 x 7168 x 24 9.6 for 20.7, 64 x 256 x 256 7.9 for 16; 64 x 7168 x 256 21.1 for 20.7, 256 x 4096 x 256 24.1 for
// 22.7.  Beside the pass over 16 experts at most and the sums of its runs, 257 x 512 x 16 7.3 for 9.5,
// 300 x 7168 x 8 7.4 for 7.7, 512 x 4096 x 16 10.5 for 9.8.  One run of tokens, so not too many: 768 x 1024 x 64 16.5 for
// 16.5, 2048 x 512 x 32 24.7 for 16.1.
constexpr int kRouterShort = 512;
inline bool router_short(int n_tok, int d, int n_exp) {
  return n_tok <= kRouterShort && static_cast<int64_t>(n_tok) * d * n_exp <= (n_exp <= kRouterFew ? 30000000 : 100000000);
}
cudaError_t launch_router_short(const float* dl, const void* x, const void* w_gate, const void* dx_in, void* dx, int n_tok,
                                int d, int n_exp, const float* dw_in, float* dw, cudaStream_t st);

}  // namespace moe
