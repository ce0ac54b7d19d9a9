// FP8 products with one fp32 scale per block of 128: launchers of the row
// quantisers and of the grouped GEMM on E4M3 codes.
//
// A block of 128 consecutive elements of an activation row (the contraction
// dimension) has the scale s = amax * (1 / 448), an fp32 product (1 where that is
// zero), and the codes E4M3(x / s), the exact quotient rounded once to nearest
// even.  Weights have
// one scale per 128 x 128 tile (launch_fp8_tile_quant).
#pragma once
#include <cstddef>
#include <cstdint>
#include <cuda_runtime.h>

namespace moe {

// Floats between two rows of an activation's scales: one per block of 128
// columns, rounded up to 4 so that every row starts on 16 bytes.
inline int64_t fp8_scale_ld(int64_t cols) { return ((cols + 127) / 128 + 3) / 4 * 4; }

// bf16 src [rows, cols] -> codes [rows, cols], scales [rows, ld].  cols % 16 == 0.
cudaError_t launch_fp8_quant_rows(const void* src, int64_t rows, int64_t cols, uint8_t* codes, float* scales,
                                  int64_t ld, cudaStream_t st);
// The same of the token rows x [n_tok, d], each written to its top_k permuted
// rows row_of_copy[t * top_k + k] (a negative row is skipped) and, with
// tok_codes, to token row t.
cudaError_t launch_fp8_quant_scatter(const void* x, int n_tok, int d, int top_k, const int32_t* row_of_copy,
                                     uint8_t* codes, float* scales, int64_t ld, uint8_t* tok_codes,
                                     float* tok_scales, cudaStream_t st);

enum Fp8Epi : int {
  FP8_EPI_BF16 = 0,        // out0[row, col] = bf16(acc)
  FP8_EPI_SWIGLU_FWD = 1,  // dual N: acc = [a1 | a3] -> h = silu(a1) * a3 quantised per 128 columns: out0 = codes,
                           // hs = scales; optional bf16 out1 = a1, out2 = a3, out3 = h
  FP8_EPI_SWIGLU_BWD = 2,  // acc = dh; in0 = a1, in1 = a3 -> out0 = da1, out1 = da3 (bf16)
};

// For every group g and its rows r in [offsets[g], offsets[g + 1]):
//   acc[r, n] = sum over k-blocks b of a_scale[r, b] * b_scale[g, n / 128, b] * sum_{k in b} a[r, k] b[g, n, k]
// over the contraction sources (b[1] is instead the second half of the N tile
// with `dual`), in the order of the k-blocks, or, where a cluster of 2, 4 or 8 CTAs shares a
// tile, each CTA's run of them in that order and then the runs' sums in order.  B is stored
// [N, K] per group, or [K, N] with b_mn.  Offsets that decrease: no row is written.
struct Fp8GemmArgs {
  Fp8Epi epi = FP8_EPI_BF16;
  bool b_mn = false;
  bool dual = false;
  const uint8_t* a[2] = {nullptr, nullptr};
  const float* a_scale[2] = {nullptr, nullptr};
  const uint8_t* b[2] = {nullptr, nullptr};
  const float* b_scale[2] = {nullptr, nullptr};
  int sources = 1;             // contraction sources, each of length k
  int64_t k = 0, n = 0;
  int64_t a_scale_ld = 0;
  const int32_t* offsets = nullptr;   // device, [groups + 1]
  int groups = 1;
  int64_t rows = 0;            // rows of A; offsets outside 0 .. rows are cut to it (DEV_BAD_OFFSETS)
  void* out0 = nullptr;
  void* out1 = nullptr;
  void* out2 = nullptr;
  void* out3 = nullptr;
  float* hs = nullptr;
  int64_t hs_ld = 0;
  const void* in0 = nullptr;
  const void* in1 = nullptr;
  int32_t* status = nullptr;
};

cudaError_t launch_fp8_gemm(const Fp8GemmArgs& args, cudaStream_t st);

}  // namespace moe
