// Activation checkpoints in 8 bits, on the backward's side.  What is kept of a
// layer's forward is MXFP8 (E4M3 codes, a power-of-two scale per 32 elements of
// a row): every value is a bf16 number, so decoding rounds nothing and the
// bf16 products on the decoded rows are the products of the kept values.
#include "ckpt.cuh"

#include <cuda_bf16.h>
#include <cuda_fp8.h>

#include "pdl.cuh"
#include "sm100_ptx.cuh"

namespace moe {
namespace {

// Rows over the y threads of a block, 8 codes a lane and turn: a warp reads 256
// and writes 512 consecutive bytes at a time (32 codes a lane, which writes 64
// bytes apart, took 38 us for 8192 x 7168 rows where this takes less).  The scale
// bytes of a row lie ld apart (the layout the products read); they come from L2,
// where the whole array (1/32 of the codes) stays.  A thread asks for the codes of
// kTurns turns before it decodes the first.  Bound by the bf16 rows it writes.
constexpr int kTurns = 8;

__device__ __forceinline__ void dequant_rows(const KeptOperand& k, int64_t block, int32_t* status) {
  const int64_t r = block * blockDim.y + threadIdx.y;
  if (r >= k.rows) return;
  const int n8 = k.cols / 8;
  const auto* codes = reinterpret_cast<const uint2*>(k.codes);
  int64_t src = r;
  if (k.row_map) {
    const int m = __ldg(k.row_map + r);
    src = m < 0 ? -1 : m / k.row_div;
  }
  const bool ok = src >= 0 && src < k.src_rows;
  if (!ok && threadIdx.x == 0 && status) atomicOr(status, DEV_BAD_INDEX);
  const uint2* in = codes + src * n8;
  uint4* dst = static_cast<uint4*>(k.out) + r * n8;
  for (int c0 = threadIdx.x; c0 < n8; c0 += kTurns * blockDim.x) {
    uint2 v[kTurns];
    uint32_t e[kTurns];
#pragma unroll
    for (int i = 0; i < kTurns; ++i) {
      const int c = c0 + i * blockDim.x;
      v[i] = make_uint2(0, 0);
      e[i] = 0;
      if (ok && c < n8) {
        v[i] = __ldg(in + c);
        e[i] = __ldg(k.scales + (c >> 2) * k.ld + src);
      }
    }
#pragma unroll
    for (int i = 0; i < kTurns; ++i) {
      const int c = c0 + i * blockDim.x;
      if (c >= n8) break;
      const float sc = __uint_as_float(e[i] ? e[i] << 23 : 0x00400000u);   // byte 0: 2^-127
      uint32_t w[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const __half2_raw hr = __nv_cvt_fp8x2_to_halfraw2(
            static_cast<__nv_fp8x2_storage_t>((j < 2 ? v[i].x : v[i].y) >> (16 * (j & 1))), __NV_E4M3);
        __half2 h2;
        *reinterpret_cast<__half2_raw*>(&h2) = hr;
        const float2 f = __half22float2(h2);
        const __nv_bfloat162 o = __floats2bfloat162_rn(f.x * sc, f.y * sc);
        w[j] = *reinterpret_cast<const uint32_t*>(&o);
      }
      dst[c] = make_uint4(w[0], w[1], w[2], w[3]);
    }
  }
}

// By the 256 threads of one block.
__device__ __forceinline__ void group_maps(const GroupMaps& m, int32_t* status) {
  const int tid = threadIdx.y * blockDim.x + threadIdx.x;
  bool less = false, out = false;
  for (int g = tid; g < m.groups; g += 256) {
    const int o0 = m.offsets[g], o1 = m.offsets[g + 1];
    less |= o1 < o0;
    out |= o0 < 0 || o0 > m.rows || o1 < 0 || o1 > m.rows;
  }
  less = __syncthreads_or(less);
  out = __syncthreads_or(out);
  if (tid == 0 && (less || out) && status) atomicOr(status, DEV_BAD_OFFSETS);
  for (int g = tid; g < m.groups; g += 256) {
    const int o0 = less ? 0 : min(max(m.offsets[g], 0), m.rows), o1 = less ? 0 : min(max(m.offsets[g + 1], 0), m.rows);
    m.checked[g] = o0;
    if (g == m.groups - 1) m.checked[m.groups] = o1;
    const uint32_t n = static_cast<uint32_t>(max(o1 - o0, 1));   // an empty group is never loaded
    tensormap_rebase_rows(m.out + g, &m.ta, reinterpret_cast<uint64_t>(m.a + o0 * m.a_ld), n);
    tensormap_rebase_rows(m.out + m.groups + g, &m.tb, reinterpret_cast<uint64_t>(m.b + o0 * m.b_ld), n);
  }
}

__global__ void __launch_bounds__(256) mx_dequant_rows_kernel(const KeptOperand k, int32_t* status) {
  pdl_trigger();
  pdl_wait();
  dequant_rows(k, blockIdx.x, status);
}

// The first block writes the maps (in a launch of their own 16 groups of 256 x 512 over 3108 rows took 16.8 us
// where they take 14.6).
__global__ void __launch_bounds__(256) mx_dequant_rows_maps_kernel(const KeptOperand k, int32_t* status,
                                                                   const __grid_constant__ GroupMaps m) {
  pdl_trigger();
  pdl_wait();
  if (blockIdx.x == 0) group_maps(m, status);
  else dequant_rows(k, blockIdx.x - 1, status);
}

// 32 rows a block; its eight warps take every eighth slice, and their sums are added in order.
__global__ void __launch_bounds__(256) row_dot_sum_kernel(const float* __restrict__ part, int64_t slices, int64_t ld,
                                                          const int32_t* __restrict__ offsets, int groups, int64_t rows,
                                                          float* __restrict__ dg) {
  __shared__ float s_sum[8][32];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  pdl_trigger();
  pdl_wait();
  const int64_t r = static_cast<int64_t>(blockIdx.x) * 32 + lane;
  const bool in = r >= offsets[0] && r < offsets[groups] && r < rows;
  float s = 0.0f;
  if (in) {
#pragma unroll 8
    for (int64_t j = warp; j < slices; j += 8) s += part[j * ld + r];
  }
  s_sum[warp][lane] = s;
  __syncthreads();
  if (warp != 0 || !in) return;
  for (int w = 1; w < 8; ++w) s += s_sum[w][lane];
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

cudaError_t launch_mx_dequant_rows(const KeptOperand& k, int32_t* status, cudaStream_t st, const GroupMaps* maps) {
  if (k.rows <= 0 && !maps) return cudaSuccess;
  if (k.cols <= 0 || k.cols % 32 || k.row_div < 1) return cudaErrorInvalidValue;
  // lanes along a row: as many as it has turns of 8, up to 32
  const int n8 = k.cols / 8;
  int x = 4;
  while (x < 32 && x < n8) x *= 2;
  const int y = 256 / x;
  cudaLaunchConfig_t cfg{};
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.gridDim = dim3(static_cast<unsigned>((k.rows + y - 1) / y + (maps ? 1 : 0)));
  cfg.blockDim = dim3(x, y);
  cfg.stream = st;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  if (maps) return cudaLaunchKernelEx(&cfg, mx_dequant_rows_maps_kernel, k, status, *maps);
  return cudaLaunchKernelEx(&cfg, mx_dequant_rows_kernel, k, status);
}

cudaError_t launch_row_dot_sum(const float* part, int64_t slices, int64_t ld, const int32_t* offsets, int groups,
                               int64_t rows, float* dg, cudaStream_t st) {
  if (rows <= 0) return cudaSuccess;
  return launch_pdl(row_dot_sum_kernel, static_cast<unsigned>((rows + 31) / 32), 256, 0, st, part, slices, ld, offsets,
                    groups, rows, dg);
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
