// The router's balance loss over ragged sequences, its z-loss and their
// gradient; and the pieces of the dense router gradient around the tensor
// cores.
//
// Sequence s holds the tokens [o_s, o_{s+1}), T_s of them; S' sequences are not
// empty, T = sum T_s.  With c_si the copies of sequence s routed to expert i,
// f_si = c_si / T_s and q_t the gate's distribution over all experts (softmax,
// or the sigmoids normalised over the experts):
//   balance = coef E / S' sum_s sum_i f_si (1 / T_s) sum_{t in s} q_ti
//   z       = z_coef / T sum_t lse_t^2,   lse_t = log sum_i exp(l_ti)
// The sum over i needs no table of mean probabilities: it is the sum over the
// tokens of inner_t = sum_i f_si q_ti, and the gradient (f held fixed, the
// selection is discrete) has that number anyway:
//   d balance / d l_tj = coef E / (S' T_s) w_tj (f_sj - inner_t)
//   d z / d l_tj       = 2 z_coef / T lse_t p_tj
// with w = q for softmax and s_j (1 - s_j) / sum_i s_i for sigmoid, p the
// softmax.  So one pass over the logits gives loss and gradient once the counts
// are known, and those come from the indices alone: two launches.
#include "seq_balance.cuh"

#include <cooperative_groups.h>
#include <cuda_bf16.h>

#include <algorithm>

#include "pdl.cuh"
#include "sm100_ptx.cuh"

namespace cg = cooperative_groups;

namespace moe {
int num_sms();
namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;

// Sequence offset i, cut to [0, n].
__device__ __forceinline__ int seq_at(const int32_t* __restrict__ off, int i, int n) {
  return min(max(__ldg(off + i), 0), n);
}

// counts[s][e] of one sequence by a cluster of C blocks: each counts its run of
// the sequence's indices, one histogram a warp (few experts meet in one word
// otherwise), and the blocks' sums are joined through the cluster's shared
// memory, so no count is zeroed first or added by atomics in global memory.
// The last cluster counts the sequences and their tokens instead.
template <int C>
__global__ void __launch_bounds__(kThreads) seq_counts_kernel(int n_tok, int E, int K, int S,
                                                              const int32_t* __restrict__ idx,
                                                              const int32_t* __restrict__ off,
                                                              int32_t* __restrict__ counts, int32_t* __restrict__ head,
                                                              int32_t* status) {
  extern __shared__ int s_hist[];   // [kWarps][E]
  __shared__ int s_sum[3];
  __shared__ int s_bad;
  const int s = blockIdx.x / C, rank = blockIdx.x % C;
  const int warp = threadIdx.x >> 5;
  pdl_trigger();
  if (s < S)
    for (int i = threadIdx.x; i < kWarps * E; i += kThreads) s_hist[i] = 0;
  if (threadIdx.x < 3) s_sum[threadIdx.x] = 0;
  if (threadIdx.x == 0) s_bad = 0;
  __syncthreads();
  pdl_wait();
  if (s == S) {
    if (rank != 0) return;   // nobody of this cluster meets at a barrier
    int full = 0, used = 0, less = 0, out = 0;
    for (int i = threadIdx.x; i < S; i += kThreads) {
      const int a = off[i], b = off[i + 1];
      const int len = seq_at(off, i + 1, n_tok) - seq_at(off, i, n_tok);
      full += len > 0;
      used += max(len, 0);
      less |= b < a;
      out |= a < 0 || a > n_tok || b < 0 || b > n_tok;
    }
    if (full) atomicAdd(&s_sum[0], full);
    if (used) atomicAdd(&s_sum[1], used);
    if (less) atomicOr(&s_sum[2], 1);
    if (less | out) atomicOr(&s_bad, 1);
    __syncthreads();
    if (threadIdx.x < 3) head[threadIdx.x] = s_sum[threadIdx.x];
    if (threadIdx.x == 0 && s_bad) atomicOr(status, DEV_BAD_OFFSETS);
    return;
  }
  const int64_t lo = static_cast<int64_t>(seq_at(off, s, n_tok)) * K;
  const int64_t n = max(static_cast<int64_t>(seq_at(off, s + 1, n_tok)) * K - lo, int64_t{0});
  const int64_t per = (n + C - 1) / C;
  const int64_t a = lo + min(n, per * rank), b = lo + min(n, per * (rank + 1));
  int* mine = s_hist + warp * E;
  bool bad = false;
  for (int64_t i = a + threadIdx.x; i < b; i += 4 * kThreads) {
    int e[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) e[j] = i + j * kThreads < b ? __ldg(idx + i + j * kThreads) : E;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      if (e[j] >= 0 && e[j] < E) atomicAdd(mine + e[j], 1);
      else bad |= i + j * kThreads < b;
    }
  }
  if (bad) s_bad = 1;
  __syncthreads();
  if (threadIdx.x == 0 && s_bad) atomicOr(status, DEV_BAD_INDEX);
  for (int e = threadIdx.x; e < E; e += kThreads) {
    int v = 0;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) v += s_hist[w * E + e];
    s_hist[e] = v;   // row 0, read above by this thread alone
  }
  int32_t* dst = counts + static_cast<int64_t>(s) * E;
  if (C == 1) {
    __syncthreads();
    for (int e = threadIdx.x; e < E; e += kThreads) dst[e] = s_hist[e];
    return;
  }
  cg::cluster_group cl = cg::this_cluster();
  cl.sync();
  const int eper = (E + C - 1) / C;
  for (int e = rank * eper + threadIdx.x; e < min(E, (rank + 1) * eper); e += kThreads) {
    int v = 0;
#pragma unroll
    for (int r = 0; r < C; ++r) v += cl.map_shared_rank(s_hist, r)[e];
    dst[e] = v;
  }
  cl.sync();   // no block leaves while its sums are read
}

__device__ __forceinline__ float warp_max(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, o));
  return v;
}
__device__ __forceinline__ float warp_add(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

struct RowsParams {
  const float* logits;
  const int32_t* counts;
  const int32_t* off;
  const float* dloss;
  const int32_t* head;
  float* dl;
  float* loss;
  double* part;
  int32_t* ticket;
  int32_t* counts_out;
  float coef, z_coef;
  int n_tok, E, gate, S, per;
};

// A warp a token, its experts over the lanes (NPER registers), tokens of a
// warp consecutive so that a sequence's f stays in registers from one to the
// next.  Each block's sums leave as two doubles, and the last block to finish
// adds them in a fixed order: equal calls give equal bits.
template <int NPER>
__global__ void __launch_bounds__(kThreads) seq_rows_kernel(const RowsParams p) {
  __shared__ double s_red[2][kThreads];
  __shared__ int s_last;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int E = p.E, N = p.n_tok;
  pdl_wait();
  const int full = __ldg(p.head), used = __ldg(p.head + 1), wrong = __ldg(p.head + 2);
  const float up = p.dloss ? __ldg(p.dloss) : 1.0f;
  const float zf = used > 0 ? p.z_coef / static_cast<float>(used) : 0.0f;
  double bal = 0.0, zz = 0.0;
  const int64_t w0 = (static_cast<int64_t>(blockIdx.x) * kWarps + warp) * p.per;
  const int t0 = static_cast<int>(min(static_cast<int64_t>(N), w0));
  const int t1 = static_cast<int>(min(static_cast<int64_t>(N), w0 + p.per));
  if (wrong) {   // overlapping sequences: no loss, no gradient, no counts
    const int64_t all = static_cast<int64_t>(p.S) * E;
    for (int64_t i = static_cast<int64_t>(blockIdx.x) * kThreads + threadIdx.x; i < all;
         i += static_cast<int64_t>(gridDim.x) * kThreads)
      p.counts_out[i] = 0;
  }
  int end = t0;         // the first token that the sequence at hand does not hold
  bool inside = false;
  float factor = 0.0f;
  float f[NPER];
#pragma unroll
  for (int j = 0; j < NPER; ++j) f[j] = 0.0f;
  for (int t = t0; t < t1; ++t) {
    if (t >= end) {
      int lo = -1, hi = p.S;   // lo: the last sequence that starts at or before t (-1: none)
      while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (seq_at(p.off, mid, N) <= t) lo = mid; else hi = mid;
      }
      const int a = lo < 0 ? 0 : seq_at(p.off, lo, N);
      const int b = seq_at(p.off, lo + 1, N);
      inside = lo >= 0 && t < b && !wrong;
      end = lo < 0 ? b : (t < b ? b : N);
      if (inside) {
        const float len = static_cast<float>(b - a);
        factor = p.coef * static_cast<float>(E) / (static_cast<float>(full) * len);
        const int32_t* c = p.counts + static_cast<int64_t>(lo) * E;
#pragma unroll
        for (int j = 0; j < NPER; ++j)
          f[j] = lane + 32 * j < E ? static_cast<float>(__ldg(c + lane + 32 * j)) / len : 0.0f;
      }
    }
    const int64_t row = static_cast<int64_t>(t) * E;
    if (!inside) {
      if (p.dl) {
#pragma unroll
        for (int j = 0; j < NPER; ++j)
          if (lane + 32 * j < E) p.dl[row + lane + 32 * j] = 0.0f;
      }
      continue;
    }
    float l[NPER], q[NPER];
#pragma unroll
    for (int j = 0; j < NPER; ++j) l[j] = lane + 32 * j < E ? __ldg(p.logits + row + lane + 32 * j) : -INFINITY;
    float m = l[0];
    bool nan = false;   // fmaxf passes a NaN over
#pragma unroll
    for (int j = 0; j < NPER; ++j) {
      m = fmaxf(m, l[j]);
      nan |= l[j] != l[j];
    }
    m = warp_max(m);
    if (m == -INFINITY) m = 0.0f;   // every expert masked: no probability, no z
    if (__any_sync(0xffffffffu, nan)) m = NAN;
    const bool soft = p.gate == 0 || p.z_coef != 0.0f;
    float z = 0.0f;
#pragma unroll
    for (int j = 0; j < NPER; ++j) {
      q[j] = soft ? expf(l[j] - m) : 0.0f;
      z += q[j];
    }
    float lse = 0.0f, invz = 0.0f;
    if (soft) {
      z = warp_add(z);
      if (z != 0.0f) {
        lse = m + logf(z);
        invz = 1.0f / z;
      }
    }
    float inner = 0.0f, invs = 0.0f;
    const float g2 = 2.0f * zf * lse * invz * up;
    if (p.gate == 0) {
#pragma unroll
      for (int j = 0; j < NPER; ++j) inner = fmaf(f[j], q[j], inner);
      inner = warp_add(inner) * invz;
      if (p.dl) {
        const float g1 = factor * invz * up;
#pragma unroll
        for (int j = 0; j < NPER; ++j)
          if (lane + 32 * j < E) p.dl[row + lane + 32 * j] = q[j] * fmaf(g1, f[j] - inner, g2);
      }
    } else {
      float sum = 0.0f, sg[NPER];
#pragma unroll
      for (int j = 0; j < NPER; ++j) {
        sg[j] = 1.0f / (1.0f + expf(-l[j]));
        sum += sg[j];
        inner = fmaf(f[j], sg[j], inner);
      }
      sum = warp_add(sum);
      if (sum != 0.0f) invs = 1.0f / sum;
      inner = warp_add(inner) * invs;
      if (p.dl) {
        const float g1 = factor * invs * up;
#pragma unroll
        for (int j = 0; j < NPER; ++j)
          if (lane + 32 * j < E)
            p.dl[row + lane + 32 * j] = fmaf(g1 * (sg[j] * (1.0f - sg[j])), f[j] - inner, g2 * q[j]);
      }
    }
    bal += static_cast<double>(factor) * inner;
    zz += static_cast<double>(lse) * lse;
  }
  if (lane == 0) {
    s_red[0][warp] = bal;
    s_red[1][warp] = zz;
  }
  __syncthreads();
  if (threadIdx.x == 0) {
    double a = 0.0, b = 0.0;
    for (int w = 0; w < kWarps; ++w) {
      a += s_red[0][w];
      b += s_red[1][w];
    }
    p.part[2 * blockIdx.x] = a;
    p.part[2 * blockIdx.x + 1] = b;
    __threadfence();
    s_last = atomicAdd(p.ticket, 1) == static_cast<int>(gridDim.x) - 1;
  }
  __syncthreads();
  if (!s_last) return;
  __threadfence();
  double a = 0.0, b = 0.0;
  for (int i = threadIdx.x; i < static_cast<int>(gridDim.x); i += kThreads) {
    a += __ldcg(p.part + 2 * i);
    b += __ldcg(p.part + 2 * i + 1);
  }
  s_red[0][threadIdx.x] = a;
  s_red[1][threadIdx.x] = b;
  __syncthreads();
  for (int n = kThreads / 2; n > 0; n >>= 1) {
    if (threadIdx.x < n) {
      s_red[0][threadIdx.x] += s_red[0][threadIdx.x + n];
      s_red[1][threadIdx.x] += s_red[1][threadIdx.x + n];
    }
    __syncthreads();
  }
  if (threadIdx.x == 0) {
    p.loss[0] = static_cast<float>(s_red[0][0]);
    p.loss[1] = used > 0 ? static_cast<float>(s_red[1][0] * (static_cast<double>(p.z_coef) / used)) : 0.0f;
    *p.ticket = 0;
  }
}

// Blocks of the rows kernel: a warp a token, at most eight blocks an SM.
int rows_grid(int n_tok) {
  return static_cast<int>(std::min<int64_t>((static_cast<int64_t>(n_tok) + kWarps - 1) / kWarps,
                                            static_cast<int64_t>(num_sms()) * 8));
}

// 8 columns of a row a thread.
__global__ void __launch_bounds__(256) router_terms_kernel(const float* __restrict__ dl, int n_tok, int E, int e8,
                                                           uint4* __restrict__ terms, int32_t* __restrict__ dense,
                                                           int32_t* __restrict__ slices, int n_slices, int slice_rows) {
  pdl_trigger();
  pdl_wait();
  const int64_t i = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x;
  if (blockIdx.x == 0) {
    if (threadIdx.x == 0) {
      dense[0] = 0;
      dense[1] = n_tok;
    }
    for (int j = threadIdx.x; j <= n_slices; j += 256)
      slices[j] = static_cast<int>(min(static_cast<int64_t>(n_tok), static_cast<int64_t>(j) * slice_rows));
  }
  const int c8 = e8 / 8;
  const int64_t row = i / c8;
  if (row >= n_tok) return;
  const int c = static_cast<int>(i - row * c8) * 8;
  const float* src = dl + row * E + c;
  float v[8];
  if (E % 4 == 0 && c + 8 <= E) {
    const float4 a = __ldg(reinterpret_cast<const float4*>(src)), b = __ldg(reinterpret_cast<const float4*>(src) + 1);
    v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
    v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] = c + j < E ? __ldg(src + j) : 0.0f;
  }
  uint4* dst = terms + row * 3 * c8 + c / 8;
#pragma unroll
  for (int k = 0; k < 3; ++k) {
    uint32_t w[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const __nv_bfloat162 h = __floats2bfloat162_rn(v[2 * j], v[2 * j + 1]);
      w[j] = *reinterpret_cast<const uint32_t*>(&h);
      const float2 r = __bfloat1622float2(h);
      // a number that is not finite is its first term alone
      v[2 * j] = isfinite(r.x) ? v[2 * j] - r.x : 0.0f;
      v[2 * j + 1] = isfinite(r.y) ? v[2 * j + 1] - r.y : 0.0f;
    }
    dst[static_cast<int64_t>(k) * c8] = make_uint4(w[0], w[1], w[2], w[3]);
  }
}

__global__ void __launch_bounds__(256) router_dw_kernel(const float4* __restrict__ part, int n_slices, int E, int e8,
                                                        int d4, const float4* dw_in, float4* dw) {
  pdl_wait();
  const int e = blockIdx.x;
  const int i = blockIdx.y * 256 + threadIdx.x;
  if (i >= d4) return;
  const int64_t o = static_cast<int64_t>(e) * d4 + i;
  float4 acc = dw_in ? dw_in[o] : make_float4(0.f, 0.f, 0.f, 0.f);
  for (int s = 0; s < n_slices; ++s) {
    const float4* src = part + static_cast<int64_t>(s) * 3 * e8 * d4 + o;
    const float4 h = __ldcg(src), m = __ldcg(src + static_cast<int64_t>(e8) * d4),
                 l = __ldcg(src + 2 * static_cast<int64_t>(e8) * d4);
    acc.x += h.x + (m.x + l.x);
    acc.y += h.y + (m.y + l.y);
    acc.z += h.z + (m.z + l.z);
    acc.w += h.w + (m.w + l.w);
  }
  dw[o] = acc;
}

}  // namespace

int64_t seq_balance_partials(int n_tok) { return rows_grid(n_tok); }

cudaError_t launch_seq_balance(const SeqBalanceArgs& a, cudaStream_t st) {
  if (a.n_tok < 1 || a.n_exp < 1 || a.n_exp > 1024 || a.n_seq < 1) return cudaErrorInvalidValue;
  // A cluster of eight blocks a sequence where one block's share of the indices would be long
  // (16384 tokens, top 8, 8 sequences: 16384 indices a sequence), one block where they are few.
  const int64_t copies = static_cast<int64_t>(a.n_tok) * a.top_k;
  const bool wide = copies >= 4096 && a.n_seq <= 4096;
  const size_t smem = static_cast<size_t>(kWarps) * a.n_exp * sizeof(int);
  cudaError_t e;
  if (wide)
    e = launch_pdl<8>(seq_counts_kernel<8>, static_cast<unsigned>(a.n_seq + 1) * 8, kThreads, smem, st, a.n_tok,
                      a.n_exp, a.top_k, a.n_seq, a.topk_idx, a.seq_offsets, a.counts, a.head, a.status);
  else
    e = launch_pdl(seq_counts_kernel<1>, static_cast<unsigned>(a.n_seq + 1), kThreads, smem, st, a.n_tok, a.n_exp,
                   a.top_k, a.n_seq, a.topk_idx, a.seq_offsets, a.counts, a.head, a.status);
  if (e != cudaSuccess) return e;
  const int grid = rows_grid(a.n_tok);
  RowsParams p;
  p.logits = a.logits;
  p.counts = a.counts;
  p.counts_out = a.counts;
  p.off = a.seq_offsets;
  p.dloss = a.dloss;
  p.head = a.head;
  p.dl = a.dlogits;
  p.loss = a.loss;
  p.part = a.part;
  p.ticket = a.ticket;
  p.coef = a.coef;
  p.z_coef = a.z_coef;
  p.n_tok = a.n_tok;
  p.E = a.n_exp;
  p.gate = a.gate;
  p.S = a.n_seq;
  p.per = static_cast<int>((static_cast<int64_t>(a.n_tok) + static_cast<int64_t>(grid) * kWarps - 1) /
                           (static_cast<int64_t>(grid) * kWarps));
  auto kern = a.n_exp <= 32 ? seq_rows_kernel<1>
              : a.n_exp <= 64 ? seq_rows_kernel<2>
              : a.n_exp <= 128 ? seq_rows_kernel<4>
              : a.n_exp <= 256 ? seq_rows_kernel<8>
              : a.n_exp <= 512 ? seq_rows_kernel<16> : seq_rows_kernel<32>;
  return launch_pdl(kern, static_cast<unsigned>(grid), kThreads, 0, st, p);
}

cudaError_t launch_router_terms(const float* dl, int n_tok, int n_exp, void* terms, int32_t* dense, int32_t* slices,
                                int n_slices, int slice_rows, cudaStream_t st) {
  const int e8 = router_term_cols(n_exp);
  const int64_t items = static_cast<int64_t>(n_tok) * (e8 / 8);
  return launch_pdl(router_terms_kernel, static_cast<unsigned>((items + 255) / 256), 256, 0, st, dl, n_tok, n_exp, e8,
                    static_cast<uint4*>(terms), dense, slices, n_slices, slice_rows);
}

cudaError_t launch_router_dw(const float* part, int n_slices, int n_exp, int d, const float* dw_in, float* dw,
                             cudaStream_t st) {
  const dim3 grid(static_cast<unsigned>(n_exp), static_cast<unsigned>((d / 4 + 255) / 256));
  router_dw_kernel<<<grid, 256, 0, st>>>(reinterpret_cast<const float4*>(part), n_slices, n_exp,
                                         router_term_cols(n_exp), d / 4, reinterpret_cast<const float4*>(dw_in),
                                         reinterpret_cast<float4*>(dw));
  return cudaGetLastError();
}

}  // namespace moe
