// Activation checkpoints in 8 bits, on the backward's side.  What is kept of a
// layer's forward is MXFP8 (E4M3 codes, a power-of-two scale per 32 elements of
// a row): every value is a bf16 number, so decoding rounds nothing and the
// bf16 products on the decoded rows are the products of the kept values.
#include "ckpt.cuh"

#include <cuda_bf16.h>
#include <cuda_fp8.h>

#include <algorithm>

#include "pdl.cuh"
#include "sm100_ptx.cuh"

namespace moe {
int num_sms();
namespace {

// 16 codes a thread, a warp 512 consecutive codes of one row: the codes and the
// bf16 values move in whole 128-byte lines.  The scale bytes of a row lie ld apart
// (the layout the products read), 16 of them for a warp; they come from L2, where
// the whole array (1/32 of the codes) stays.  Bound by the bf16 rows it writes.
__global__ void __launch_bounds__(256) mx_dequant_rows_kernel(const uint8_t* __restrict__ codes,
                                                              const uint8_t* __restrict__ scales, int64_t src_rows,
                                                              int c16, int64_t ld, const int32_t* __restrict__ row_map,
                                                              int row_div, int64_t rows, uint4* __restrict__ out,
                                                              int32_t* status) {
  pdl_trigger();
  pdl_wait();
  const int64_t items = rows * c16;
  for (int64_t i = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x; i < items;
       i += static_cast<int64_t>(gridDim.x) * 256) {
    const int64_t r = i / c16;
    const int c = static_cast<int>(i - r * c16);
    int64_t src = r;
    if (row_map) {
      const int m = __ldg(row_map + r);
      src = m < 0 ? -1 : m / row_div;
    }
    uint32_t w[8] = {0, 0, 0, 0, 0, 0, 0, 0};
    if (src >= 0 && src < src_rows) {
      const uint4 v = __ldg(reinterpret_cast<const uint4*>(codes) + src * c16 + c);
      const uint32_t b = __ldg(scales + static_cast<int64_t>(c >> 1) * ld + src);
      const float sc = __uint_as_float(b ? b << 23 : 0x00400000u);   // byte 0: 2^-127
      const uint32_t cw[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const __half2_raw hr = __nv_cvt_fp8x2_to_halfraw2(
            static_cast<__nv_fp8x2_storage_t>(cw[j >> 1] >> (16 * (j & 1))), __NV_E4M3);
        __half2 h2;
        *reinterpret_cast<__half2_raw*>(&h2) = hr;
        const float2 f = __half22float2(h2);
        const __nv_bfloat162 o = __floats2bfloat162_rn(f.x * sc, f.y * sc);
        w[j] = *reinterpret_cast<const uint32_t*>(&o);
      }
    } else if (status && c == 0) {
      atomicOr(status, DEV_BAD_INDEX);
    }
    uint4* dst = out + 2 * i;
    dst[0] = make_uint4(w[0], w[1], w[2], w[3]);
    dst[1] = make_uint4(w[4], w[5], w[6], w[7]);
  }
}

__global__ void __launch_bounds__(256) check_offsets_kernel(const int32_t* __restrict__ offsets, int groups, int rows,
                                                            int32_t* __restrict__ dst, int32_t* status) {
  __shared__ int s_less, s_out;
  pdl_trigger();
  if (threadIdx.x == 0) s_less = s_out = 0;
  __syncthreads();
  pdl_wait();
  for (int i = threadIdx.x; i <= groups; i += 256) {
    const int o = offsets[i];
    if (o < 0 || o > rows) s_out = 1;
    if (i > 0 && o < offsets[i - 1]) s_less = 1;
  }
  __syncthreads();
  for (int i = threadIdx.x; i <= groups; i += 256) dst[i] = s_less ? 0 : min(max(offsets[i], 0), rows);
  if (threadIdx.x == 0 && (s_less || s_out)) atomicOr(status, DEV_BAD_OFFSETS);
}

__global__ void __launch_bounds__(256) row_dot_sum_kernel(const float* __restrict__ part, int64_t slices, int64_t ld,
                                                          const int32_t* __restrict__ offsets, int groups,
                                                          float* __restrict__ dg) {
  const int64_t r = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x;
  if (r < offsets[0] || r >= offsets[groups]) return;
  float s = 0.0f;
#pragma unroll 8
  for (int64_t j = 0; j < slices; ++j) s += part[j * ld + r];
  dg[r] = s;
}

// A warp a token, a lane a copy.
__global__ void __launch_bounds__(256) gate_bwd_kernel(int n_tok, int K, int gate, const float* __restrict__ dg_row,
                                                       const int32_t* __restrict__ row_of_copy,
                                                       const float* __restrict__ topk_w,
                                                       const float* __restrict__ logits, int E,
                                                       const int32_t* __restrict__ topk_idx, float* __restrict__ dg,
                                                       float* __restrict__ dl) {
  const int64_t t = static_cast<int64_t>(blockIdx.x) * 8 + (threadIdx.x >> 5);
  const int lane = threadIdx.x & 31;
  if (t >= n_tok) return;
  const bool on = lane < K;
  const int64_t c = t * K + lane;
  float d = 0.0f, g = 0.0f, sg = 0.0f;
  if (on) {
    const int r = row_of_copy[c];
    d = r >= 0 ? dg_row[r] : 0.0f;
    g = topk_w[c];
    if (gate == 1) sg = 1.0f / (1.0f + expf(-logits[t * E + topk_idx[c]]));
  }
  float inner = g * d, ssum = sg;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    inner += __shfl_xor_sync(0xffffffffu, inner, o);
    ssum += __shfl_xor_sync(0xffffffffu, ssum, o);
  }
  if (!on) return;
  dg[c] = d;
  dl[c] = gate == 0 ? g * (d - inner) : sg * (1.0f - sg) / ssum * (d - inner);
}

}  // namespace

cudaError_t launch_mx_dequant_rows(const uint8_t* codes, const uint8_t* scales, int64_t src_rows, int cols, int64_t ld,
                                   const int32_t* row_map, int row_div, int64_t rows, void* out, int32_t* status,
                                   cudaStream_t st) {
  if (rows <= 0) return cudaSuccess;
  if (cols <= 0 || cols % 32 || row_div < 1) return cudaErrorInvalidValue;
  const int64_t items = rows * (cols / 16);
  const int64_t blocks = std::min<int64_t>((items + 255) / 256, static_cast<int64_t>(num_sms()) * 16);
  return launch_pdl(mx_dequant_rows_kernel, static_cast<unsigned>(blocks), 256, 0, st, codes, scales, src_rows,
                    cols / 16, ld, row_map, row_div, rows, static_cast<uint4*>(out), status);
}

cudaError_t launch_check_offsets(const int32_t* offsets, int groups, int64_t rows, int32_t* dst, int32_t* status,
                                 cudaStream_t st) {
  return launch_pdl(check_offsets_kernel, 1, 256, 0, st, offsets, groups, static_cast<int>(rows), dst, status);
}

cudaError_t launch_row_dot_sum(const float* part, int64_t slices, int64_t ld, const int32_t* offsets, int groups,
                               int64_t rows, float* dg, cudaStream_t st) {
  if (rows <= 0) return cudaSuccess;
  row_dot_sum_kernel<<<static_cast<unsigned>((rows + 255) / 256), 256, 0, st>>>(part, slices, ld, offsets, groups, dg);
  return cudaGetLastError();
}

cudaError_t launch_gate_bwd(int n_tok, int top_k, int gate, const float* dg_row, const int32_t* row_of_copy,
                            const float* topk_w, const float* logits, int n_exp, const int32_t* topk_idx, float* dg,
                            float* dl, cudaStream_t st) {
  if (n_tok <= 0) return cudaSuccess;
  if (top_k > 32) return cudaErrorInvalidValue;
  gate_bwd_kernel<<<static_cast<unsigned>((n_tok + 7) / 8), 256, 0, st>>>(n_tok, top_k, gate, dg_row, row_of_copy,
                                                                          topk_w, logits, n_exp, topk_idx, dg, dl);
  return cudaGetLastError();
}

}  // namespace moe
