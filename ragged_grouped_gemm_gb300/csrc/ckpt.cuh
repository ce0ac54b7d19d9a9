// Activation checkpoints in 8 bits (MXFP8 rows) on the backward's side: decoding rows and the
// row weights' gradient (see ckpt.cu).
#pragma once
#include <cstdint>
#include <cuda.h>
#include <cuda_runtime.h>

namespace moe {

// out [rows, cols] bf16 = the values of MXFP8 rows: row r is row row_map[r] / row_div of the codes [src_rows, cols]
// and their scales [cols/32][ld] (row_map null: row r).  An index outside [0, src_rows) gives a zero row and
// DEV_BAD_INDEX.  cols % 32 == 0.
struct KeptOperand {
  const uint8_t* codes;
  const uint8_t* scales;
  int64_t src_rows;
  int cols;
  int64_t ld;
  const int32_t* row_map;
  int row_div;
  int64_t rows;
  void* out;
};
// The per-group tensor maps of a product over groups of rows whose offsets come from outside the layer: each
// offset is cut to 0 .. rows into `checked` (groups + 1 entries), all of them to zero where they decrease
// (DEV_BAD_OFFSETS either way); out [0, G) and [G, 2G) receive copies of ta and tb (encoded for one row) at the
// group's rows.  groups <= 1024.
struct GroupMaps {
  CUtensorMap ta, tb;
  CUtensorMap* out;
  const int32_t* offsets;
  int32_t* checked;
  int32_t groups, rows;
  const char* a;
  int64_t a_ld;
  const char* b;
  int64_t b_ld;
};
// maps (host, nullable): written by one more block of the same launch.
cudaError_t launch_mx_dequant_rows(const KeptOperand& k, int32_t* status, cudaStream_t st,
                                   const GroupMaps* maps = nullptr);
// dg[r] = sum over the slices, in a fixed order, of part[slice][ld] for the rows of [offsets[0], offsets[groups]).
cudaError_t launch_row_dot_sum(const float* part, int64_t slices, int64_t ld, const int32_t* offsets, int groups,
                               int64_t rows, float* dg, cudaStream_t st);
// Per token: dg[t, k] = dg_row[row_of_copy[t K + k]] (0 for a row of -1) and the router's logit gradient dl[t, k],
// as launch_combine_bwd forms it.
cudaError_t launch_gate_bwd(int n_tok, int top_k, int gate, const float* dg_row, const int32_t* row_of_copy,
                            const float* topk_w, const float* logits, int n_exp, const int32_t* topk_idx, float* dg,
                            float* dl, cudaStream_t st);

}  // namespace moe
