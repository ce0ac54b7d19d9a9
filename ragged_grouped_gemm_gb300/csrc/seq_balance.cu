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
// are known, and those come from the indices alone: two launches, or one for a few tokens.
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
static_assert(kWarps == 8, "a block of rows takes 8 tokens at least");

// Sequence offset i, cut to [0, n].
__device__ __forceinline__ int seq_at(const int32_t* __restrict__ off, int i, int n) {
  return min(max(__ldg(off + i), 0), n);
}

// counts[s][e] of one sequence by one block, or by a cluster of C: each counts its
// run of the sequence's indices in nh histograms (its warps in turn; few experts
// meet in one word otherwise), and the blocks' sums are joined through the
// cluster's shared memory, so no count is zeroed first or added by atomics in
// global memory.  The last block or cluster counts the sequences and their tokens.
template <int C, int T>
__global__ void __launch_bounds__(T) seq_counts_kernel(int n_tok, int E, int K, int S, int nh,
                                                       const int32_t* __restrict__ idx,
                                                       const int32_t* __restrict__ off,
                                                       int32_t* __restrict__ counts, int32_t* __restrict__ head,
                                                       int32_t* status) {
  extern __shared__ int s_hist[];   // [nh][E]
  __shared__ int s_sum[3];
  __shared__ int s_bad;
  const int s = blockIdx.x / C, rank = blockIdx.x % C;
  const int warp = threadIdx.x >> 5;
  pdl_trigger();
  if (s < S)
    for (int i = threadIdx.x; i < nh * E; i += T) s_hist[i] = 0;
  if (threadIdx.x < 3) s_sum[threadIdx.x] = 0;
  if (threadIdx.x == 0) s_bad = 0;
  __syncthreads();
  pdl_wait();
  if (s == S) {
    if (rank != 0) return;   // nobody of this cluster meets at a barrier
    int full = 0, used = 0, less = 0, out = 0;
    for (int i = threadIdx.x; i < S; i += T) {
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
  int* mine = s_hist + (warp & (nh - 1)) * E;
  bool bad = false;
  for (int64_t i = a + threadIdx.x; i < b; i += 8 * T) {
    int e[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) e[j] = i + j * T < b ? __ldg(idx + i + j * T) : E;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      if (e[j] >= 0 && e[j] < E) atomicAdd(mine + e[j], 1);
      else bad |= i + j * T < b;
    }
  }
  if (bad) s_bad = 1;
  __syncthreads();
  if (threadIdx.x == 0 && s_bad) atomicOr(status, DEV_BAD_INDEX);
  int32_t* dst = counts + static_cast<int64_t>(s) * E;
  for (int e = threadIdx.x; e < E; e += T) {
    int v = 0;
#pragma unroll 8
    for (int w = 0; w < nh; ++w) v += s_hist[w * E + e];
    if (C == 1) dst[e] = v;
    else s_hist[e] = v;   // row 0, read above by this thread alone
  }
  if (C == 1) return;
  cg::cluster_group cl = cg::this_cluster();
  cl.sync();
  const int eper = (E + C - 1) / C;
  for (int e = rank * eper + threadIdx.x; e < min(E, (rank + 1) * eper); e += T) {
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
  float4* part;
  int32_t* ticket;
  int32_t* counts_out;
  const int32_t* idx;   // ALL: the rest
  int32_t* status;
  int K;
  float coef, z_coef;
  int n_tok, E, S, per;
};

// acc += v with what the addition lost kept in acc.y: 48 bits from 32-bit additions (64-bit ones, by every warp and
// then in a tree of the last block, took 9 of 21 us).  An infinite or NaN sum has no rest.
__device__ __forceinline__ void add_kept(float2& acc, float v, float rest = 0.0f) {
  const float s = acc.x + v;
  const float b = s - acc.x;
  const float e = (acc.x - (s - b)) + (v - b);
  acc.y = isfinite(s) ? acc.y + rest + e : 0.0f;
  acc.x = s;
}

// The warps' sums (of lane 0) added in warp order by thread 0.
__device__ __forceinline__ void block_sum(float2& bal, float2& zz, float4* s_red, int warp, int lane) {
  __syncthreads();
  if (lane == 0) s_red[warp] = make_float4(bal.x, bal.y, zz.x, zz.y);
  __syncthreads();
  if (threadIdx.x != 0) return;
#pragma unroll
  for (int w = 1; w < kWarps; ++w) {
    const float4 v = s_red[w];
    add_kept(bal, v.x, v.y);
    add_kept(zz, v.z, v.w);
  }
}

// 1 / x to the unit's one ulp, for normal x and 1 / x.
__device__ __forceinline__ float rcp_fast(float x) {
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}

// Resident blocks an SM by the registers a row takes: all blocks run at once, so that the look-up of a warp's
// sequence and a block's end are paid once.
template <int NPER>
constexpr int kRowBlocks = NPER <= 4 ? 4 : NPER <= 8 ? 3 : NPER <= 16 ? 2 : 1;

// Register j of a lane holds expert e_of(lane, j): VEC consecutive experts a lane, so that rows move in 16-byte
// words where E and the arrays allow it.
template <int VEC>
__device__ __forceinline__ int e_of(int lane, int j) {
  return VEC * lane + j % VEC + 32 * VEC * (j / VEC);
}
template <int NPER, int VEC>
__device__ __forceinline__ void load_row(const float* __restrict__ row, int E, int lane, float (&v)[NPER]) {
#pragma unroll
  for (int j = 0; j < NPER; j += VEC) {
    const int e = e_of<VEC>(lane, j);
    if (VEC == 4) {
      const float4 x = e < E ? __ldg(reinterpret_cast<const float4*>(row + e))
                             : make_float4(-INFINITY, -INFINITY, -INFINITY, -INFINITY);
      v[j] = x.x;
      v[j + 1 < NPER ? j + 1 : j] = x.y;
      v[j + 2 < NPER ? j + 2 : j] = x.z;
      v[j + 3 < NPER ? j + 3 : j] = x.w;
    } else {
      v[j] = e < E ? __ldg(row + e) : -INFINITY;
    }
  }
}
template <int NPER, int VEC>
__device__ __forceinline__ void store_row(float* __restrict__ row, int E, int lane, const float (&v)[NPER]) {
#pragma unroll
  for (int j = 0; j < NPER; j += VEC) {
    const int e = e_of<VEC>(lane, j);
    if (e >= E) continue;
    if (VEC == 4)
      *reinterpret_cast<float4*>(row + e) = make_float4(v[j], v[j + 1 < NPER ? j + 1 : j], v[j + 2 < NPER ? j + 2 : j],
                                                        v[j + 3 < NPER ? j + 3 : j]);
    else
      row[e] = v[j];
  }
}

// Few tokens: one cluster counts too, each copy looking up its sequence and adding to counts in global memory
// (whole numbers, so the order does not matter), which the cluster's barriers zero before and close behind.
// s_head: sequences that are not empty, their tokens, decreasing offsets.
constexpr int kAllBlocks = kSeqBalanceCluster;
__device__ __forceinline__ void count_all(const RowsParams& p, int (&s_head)[3]) {
  const int N = p.n_tok, tid = static_cast<int>(blockIdx.x) * kThreads + threadIdx.x;
  if (threadIdx.x < 3) s_head[threadIdx.x] = 0;
  __syncthreads();
  int full = 0, used = 0, less = 0, out = 0;
  for (int i = threadIdx.x; i < p.S; i += kThreads) {
    const int a = __ldg(p.off + i), b = __ldg(p.off + i + 1);
    const int len = seq_at(p.off, i + 1, N) - seq_at(p.off, i, N);
    full += len > 0;
    used += max(len, 0);
    less |= b < a;
    out |= a < 0 || a > N || b < 0 || b > N;
  }
  if (full) atomicAdd(&s_head[0], full);
  if (used) atomicAdd(&s_head[1], used);
  if (less) atomicOr(&s_head[2], 1);
  if ((less | out) && blockIdx.x == 0) atomicOr(p.status, DEV_BAD_OFFSETS);
  const int64_t all = static_cast<int64_t>(p.S) * p.E;
  for (int64_t i = tid; i < all; i += kAllBlocks * kThreads) p.counts_out[i] = 0;
  cg::cluster_group cl = cg::this_cluster();
  cl.sync();
  if (!s_head[2]) {
    bool bad = false;
    for (int i = tid; i < N * p.K; i += kAllBlocks * kThreads) {
      const int e = __ldg(p.idx + i), t = i / p.K;
      int lo = -1, hi = p.S;   // start[lo] <= t < start[hi]
      while (hi - lo > 1) {
        const int mid = (lo + hi) / 2;
        if (seq_at(p.off, mid, N) <= t) lo = mid;
        else hi = mid;
      }
      if (lo < 0 || t >= seq_at(p.off, lo + 1, N)) continue;
      if (e >= 0 && e < p.E) atomicAdd(p.counts_out + static_cast<int64_t>(lo) * p.E + e, 1);
      else bad = true;
    }
    if (bad) atomicOr(p.status, DEV_BAD_INDEX);
  }
  cl.sync();
}

// A warp a token, its experts over the lanes (NPER registers), tokens of a
// warp consecutive so that a sequence's f stays in registers from one to the
// next.  Each block's sums leave as two numbers with their rests, and the last
// block to finish adds them in a fixed order: equal calls give equal bits.
// Bound by latency: a row is one chain of loads, an exponential, two sums over the warp, a reciprocal and a logarithm, and
// with a token a warp at a time an SM issues on a third of its cycles (16384 x 256: 17 us alone, DRAM 13 % busy).
template <int NPER, int VEC, int GATE, bool ALL = false>
__global__ void __launch_bounds__(kThreads, kRowBlocks<NPER>) seq_rows_kernel(const RowsParams p) {
  __shared__ float4 s_red[kWarps];
  __shared__ int s_last;
  __shared__ int s_head[3];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int E = p.E, N = p.n_tok;
  pdl_wait();
  if (ALL) count_all(p, s_head);
  const int full = ALL ? s_head[0] : __ldg(p.head), used = ALL ? s_head[1] : __ldg(p.head + 1);
  const int wrong = ALL ? s_head[2] : __ldg(p.head + 2);
  const float up = p.dloss ? __ldg(p.dloss) : 1.0f;
  const float zf = used > 0 ? p.z_coef / static_cast<float>(used) : 0.0f;
  float2 bal = make_float2(0.0f, 0.0f), zz = bal;
  const int64_t w0 = (static_cast<int64_t>(blockIdx.x) * kWarps + warp) * p.per;
  const int t0 = static_cast<int>(min(static_cast<int64_t>(N), w0));
  const int t1 = static_cast<int>(min(static_cast<int64_t>(N), w0 + p.per));
  if (wrong && !ALL) {   // overlapping sequences: no loss, no gradient, no counts
    const int64_t all = static_cast<int64_t>(p.S) * E;
    for (int64_t i = static_cast<int64_t>(blockIdx.x) * kThreads + threadIdx.x; i < all;
         i += static_cast<int64_t>(gridDim.x) * kThreads)
      p.counts_out[i] = 0;
  }
  int end = t0;         // the first token that the sequence at hand does not hold
  bool inside = false;
  float factor = 0.0f;
  float f[NPER], nxt[NPER];
#pragma unroll
  for (int j = 0; j < NPER; ++j) f[j] = 0.0f;
  // the first row is on its way while its sequence is looked up, every later one while the one before is worked on
  if (t0 < t1) load_row<NPER, VEC>(p.logits + static_cast<int64_t>(t0) * E, E, lane, nxt);
  for (int t = t0; t < t1; ++t) {
    float l[NPER];
#pragma unroll
    for (int j = 0; j < NPER; ++j) l[j] = nxt[j];
    if (t + 1 < t1) load_row<NPER, VEC>(p.logits + static_cast<int64_t>(t + 1) * E, E, lane, nxt);
    if (t >= end) {
      // the last sequence that starts at or before t (-1: none), 32 starts a look
      int lo = -1, hi = p.S;   // start[lo] <= t < start[hi]
      while (hi - lo > 1) {
        const int step = (hi - lo + 31) / 32;
        const int i = lo + 1 + lane * step;
        const unsigned le = __ballot_sync(0xffffffffu, i < hi && seq_at(p.off, min(i, p.S), N) <= t);
        const int c = __popc(le);   // starts do not decrease (or `wrong` is set): a run of lanes from the first
        const int base = lo;
        if (c > 0) lo = base + 1 + (c - 1) * step;
        hi = min(hi, base + 1 + c * step);
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
        for (int j = 0; j < NPER; ++j) {
          const int e = e_of<VEC>(lane, j);
          f[j] = e < E ? static_cast<float>(ALL ? __ldcg(c + e) : __ldg(c + e)) / len : 0.0f;
        }
      }
    }
    const int64_t row = static_cast<int64_t>(t) * E;
    if (!inside) {
      if (p.dl) {
#pragma unroll
        for (int j = 0; j < NPER; ++j) l[j] = 0.0f;
        store_row<NPER, VEC>(p.dl + row, E, lane, l);
      }
      continue;
    }
    float inner, lse = 0.0f;
    // q: the softmax before its division by z; w: the slope of the gate's distribution before its own
    float q[NPER], w[NPER];
    float z = 0.0f, sum = 0.0f, fs = 0.0f;
#pragma unroll
    for (int j = 0; j < NPER; ++j) {
      q[j] = expf(l[j]);
      z += q[j];
      if (GATE == 0) {
        fs = fmaf(f[j], q[j], fs);
      } else {
        // sigmoid = v / (1 + v) and its slope v / (1 + v)^2 for v = e^l: the softmax's exponential serves both
        const float r = rcp_fast(1.0f + q[j]);
        const float sg = q[j] * r;
        sum += sg;
        fs = fmaf(f[j], sg, fs);
        w[j] = sg * r;
      }
    }
    z = warp_add(z);
    fs = warp_add(fs);
    if (GATE != 0) sum = warp_add(sum);
    float invz, invq;
    // Exponentials of the logits as they are, without the largest taken off: right while their sum is not so small that
    // terms that matter were lost (the largest is above -28 then, what e^l loses below -87 is 1e-25 of it), nor so
    // large that the gradient's factors, of which 1 / z is one, leave the normal numbers (with coef E / T of 1e-12
    // there are 1e10 left; up to 1e34 rows near 74 lost 1e-4 of the gradient to 5 %).  Else row by row the long way.
    if (z < 1e15f && z > 1e-9f) {
      invz = rcp_fast(z);
      lse = logf(z);
      invq = GATE == 0 ? invz : rcp_fast(sum);
      inner = fs * invq;
    } else {
      float m = l[0];
      bool nan = false;   // a NaN, which fmaxf passes over, or +inf
#pragma unroll
      for (int j = 0; j < NPER; ++j) {
        m = fmaxf(m, l[j]);
        nan |= !(l[j] < INFINITY);
      }
      m = warp_max(m);
      if (m == -INFINITY) m = 0.0f;   // every expert masked: no probability, no z
      if (__any_sync(0xffffffffu, nan)) m = NAN;
      // Every logit below zero: the sigmoids without their common factor e^m, which may be below the smallest number,
      // e^(l - m) / (1 + e^l).  Quotients and slopes over their sum are the same.
      const bool low = m < 0.0f;
      z = sum = fs = 0.0f;
#pragma unroll
      for (int j = 0; j < NPER; ++j) {
        q[j] = expf(l[j] - m);
        z += q[j];
        float d = q[j];
        if (GATE != 0) {
          const float v = expf(-fabsf(l[j]));   // sigmoid(|l|) = 1 / (1 + v), the other side v / (1 + v)
          const float big = 1.0f / (1.0f + v), small = (low ? q[j] : v) * big;
          d = l[j] > 0.0f ? big : small;
          w[j] = big * small;
          if (l[j] == -INFINITY) d = w[j] = 0.0f;
          sum += d;
        }
        fs = fmaf(f[j], d, fs);
      }
      z = warp_add(z);
      sum = warp_add(sum);
      fs = warp_add(fs);
      if (m != m) fs = m;   // sigmoids are finite: the row is to be NaN as the softmax makes it
      invz = z != 0.0f ? 1.0f / z : 0.0f;
      lse = z != 0.0f ? m + logf(z) : 0.0f;
      invq = GATE == 0 ? invz : sum != 0.0f ? 1.0f / sum : 0.0f;
      inner = fs * invq;
    }
    if (p.dl) {
      const float g1 = factor * invq * up, g2 = 2.0f * zf * lse * invz * up;
#pragma unroll
      for (int j = 0; j < NPER; ++j)
        l[j] = GATE == 0 ? q[j] * fmaf(g1, f[j] - inner, g2) : fmaf(g1 * w[j], f[j] - inner, g2 * q[j]);
      store_row<NPER, VEC>(p.dl + row, E, lane, l);
    }
    add_kept(bal, factor * inner);
    if (p.z_coef != 0.0f) add_kept(zz, lse * lse);   // a row of the type's lowest value is infinite here
  }
  block_sum(bal, zz, s_red, warp, lane);
  if (threadIdx.x == 0) {
    p.part[blockIdx.x] = make_float4(bal.x, bal.y, zz.x, zz.y);
    __threadfence();
    s_last = atomicAdd(p.ticket, 1) == static_cast<int>(gridDim.x) - 1;
  }
  __syncthreads();
  if (!s_last) return;
  __threadfence();
  bal = zz = make_float2(0.0f, 0.0f);
  for (int i = threadIdx.x; i < static_cast<int>(gridDim.x); i += kThreads) {
    const float4 v = __ldcg(p.part + i);
    add_kept(bal, v.x, v.y);
    add_kept(zz, v.z, v.w);
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    const float4 v = make_float4(__shfl_xor_sync(0xffffffffu, bal.x, o), __shfl_xor_sync(0xffffffffu, bal.y, o),
                                 __shfl_xor_sync(0xffffffffu, zz.x, o), __shfl_xor_sync(0xffffffffu, zz.y, o));
    add_kept(bal, v.x, v.y);
    add_kept(zz, v.z, v.w);
  }
  block_sum(bal, zz, s_red, warp, lane);
  if (threadIdx.x == 0) {
    p.loss[0] = bal.x + bal.y;
    p.loss[1] = p.z_coef != 0.0f ? (zz.x + zz.y) * zf : 0.0f;
    *p.ticket = 0;
  }
}

int row_blocks(int n_exp) {
  return n_exp <= 128 ? kRowBlocks<4> : n_exp <= 256 ? kRowBlocks<8> : n_exp <= 512 ? kRowBlocks<16> : kRowBlocks<32>;
}
template <int GATE>
auto rows_kernel(int n_exp, bool vec) {
  return n_exp <= 32 ? seq_rows_kernel<1, 1, GATE>
         : n_exp <= 64 ? seq_rows_kernel<2, 1, GATE>
         : n_exp <= 128 ? (vec ? seq_rows_kernel<4, 4, GATE> : seq_rows_kernel<4, 1, GATE>)
         : n_exp <= 256 ? (vec ? seq_rows_kernel<8, 4, GATE> : seq_rows_kernel<8, 1, GATE>)
         : n_exp <= 512 ? (vec ? seq_rows_kernel<16, 4, GATE> : seq_rows_kernel<16, 1, GATE>)
                        : (vec ? seq_rows_kernel<32, 4, GATE> : seq_rows_kernel<32, 1, GATE>);
}
template <int GATE>
auto all_kernel(int n_exp) {   // up to 64 experts
  return n_exp <= 32 ? seq_rows_kernel<1, 1, GATE, true> : seq_rows_kernel<2, 1, GATE, true>;
}
// Blocks of the rows kernel: a warp a token, no more than are resident.
int rows_grid(int n_tok, int n_exp) {
  return static_cast<int>(std::min<int64_t>((static_cast<int64_t>(n_tok) + kWarps - 1) / kWarps,
                                            static_cast<int64_t>(num_sms()) * row_blocks(n_exp)));
}

__device__ __forceinline__ float plus(float a, float b) { return a + b; }
__device__ __forceinline__ float4 plus(const float4& a, const float4& b) {
  return make_float4(a.x + b.x, a.y + b.y, a.z + b.z, a.w + b.w);
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

// V numbers a thread: four where that leaves every SM its threads, one where few experts would not.
template <int TERMS, typename V>
__global__ void __launch_bounds__(256) router_dw_kernel(const V* __restrict__ part, int n_slices, int64_t n,
                                                        int64_t term, const V* dw_in, V* dw) {
  pdl_trigger();
  pdl_wait();
  const int64_t o = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x;
  if (o >= n) return;
  V acc{};
  if (dw_in) acc = dw_in[o];
#pragma unroll 4
  for (int s = 0; s < n_slices; ++s) {
    const V* src = part + s * TERMS * term + o;
    V v = __ldcg(src);
    if (TERMS == 3) v = plus(v, plus(__ldcg(src + term), __ldcg(src + 2 * term)));
    acc = plus(acc, v);
  }
  dw[o] = acc;
}

// ---- few experts: the dense router gradient in one pass
// D (16 x 8, fp32) += A (16 x 16) B (16 x 8), bf16; lane l holds rows l / 4 and l / 4 + 8 of A and D, column l / 4 of B.
__device__ __forceinline__ void mma_16x8x16(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
               : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
               : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
// The transpose of an 8 x 8 matrix of bf16 across the warp: lane l holds row l / 4, columns 2 (l % 4) and the next.
__device__ __forceinline__ uint32_t transpose8(uint32_t v) {
  uint32_t r;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(v));
  return r;
}
// The next bf16 term of two numbers, which keep what remains; a number that is not finite is its first term alone.
__device__ __forceinline__ uint32_t next_term(float2& v) {
  const __nv_bfloat162 h = __floats2bfloat162_rn(v.x, v.y);
  const float2 r = __bfloat1622float2(h);
  v.x = isfinite(r.x) ? v.x - r.x : 0.0f;
  v.y = isfinite(r.y) ? v.y - r.y : 0.0f;
  return *reinterpret_cast<const uint32_t*>(&h);
}

// The B of dlogits W for eight experts from e0 and 64 columns: rows of W, transposed (tile t's columns as below).
__device__ __forceinline__ void expert_columns(const __nv_bfloat16* __restrict__ wg, int e0, int E, int D, int col0,
                                               bool on, int lane, uint32_t (&f)[8]) {
  const int e = e0 + lane / 4;
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    uint4 v = make_uint4(0, 0, 0, 0);
    if (on && e < E)
      v = __ldg(reinterpret_cast<const uint4*>(wg + static_cast<int64_t>(e) * D + col0 + 32 * k + lane % 4 * 8));
#pragma unroll
    for (int i = 0; i < 4; ++i) f[4 * k + i] = transpose8(reinterpret_cast<const uint32_t*>(&v)[i]);
  }
}

//   dx_t = dx_in_t + sum_e dl_te W_e,   dw_e = dw_in_e + sum_t dl_te x_t   for up to 8 * H experts (H 1, 2)
// tcgen05's tiles of 128 rows would be an eighth full at most, and its two products read x, the addend and dl (as
// bf16 terms that a third kernel makes) in launches of their own; here each is read once and what bounds it is
// that traffic (4096 x 4096, 8 experts: 100 MB).  The same on the FMA units took 30 us with 8 experts
// and 50 with 16, by their instructions.
//
// A warp takes 16 tokens x 64 columns a turn: x and the addend come straight into the layout of D, 16 bytes a lane,
// the columns of the eight 16 x 8 tiles being dealt so that a lane's lie together (column c of the 64 in tile
// t = c / 32 * 4 + c % 8 / 2, as column c % 32 / 8 * 2 + c % 2); a transpose in registers makes x the
// B of the second product, and dl's terms their A's.  dx, which bf16 holds to 2^-9, takes two terms of dl (a third: 26 us
// for 24), dw three; K of the first product is terms and experts, the first term of the second has an accumulator of its
// own (rows or registers).  W stays in registers.  The block's warps
// lie cw along the columns, the others take other tokens and are joined at the end.
// warps of a block and blocks an SM: 128 registers a thread, or 168
template <int H> constexpr int kFewWarps = H == 1 ? 8 : 4;
template <int H> constexpr int kFewBlocks = H == 1 ? 2 : 3;
constexpr int kFewTurns = 56;   // of a warp, about, that one accumulator adds (1.5e-8 of a sum is cut at each)
// The block's dw of 8 * H experts from e0, eight at a time: the terms' sums, then the warps', in order.
template <int H, int WARPS>
__device__ __forceinline__ void few_join(const float (&acc)[H][8][4], float (&s_sum)[WARPS][16][33], int cw, int E, int e0,
                                         int D, int64_t at, const float* dw_in, float* dw) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, tw = WARPS / cw;
#pragma unroll
  for (int h = 0; h < H; ++h) {
    __syncthreads();
#pragma unroll
    for (int t = 0; t < 8; ++t)
#pragma unroll
      for (int i = 0; i < 2; ++i)
        s_sum[warp][2 * t + i][lane] = H == 1 ? acc[0][t][i] + acc[0][t][2 + i] : acc[0][t][2 * h + i] + acc[H - 1][t][2 * h + i];
    __syncthreads();
    for (int o = threadIdx.x; o < cw * 512; o += WARPS * 32) {
      const int c = o % 64, e = e0 + 8 * h + o / 64 % 8, w = o / 512, col = (static_cast<int>(blockIdx.x) * cw + w) * 64 + c;
      const int t = c / 32 * 4 + c % 8 / 2;
      float v = 0.0f;
      for (int k = 0; k < tw; ++k) v += s_sum[k * cw + w][2 * t + c % 2][o / 64 % 8 * 4 + c % 32 / 8];
      if (e < E && col < D) {
        const int64_t i = at + static_cast<int64_t>(e) * D + col;
        dw[i] = dw_in ? dw_in[i] + v : v;
      }
    }
  }
}

template <int H>
__global__ void __launch_bounds__(kFewWarps<H> * 32, kFewBlocks<H>) router_few_kernel(
    const float* __restrict__ dl, const __nv_bfloat16* __restrict__ x, const __nv_bfloat16* __restrict__ wg,
    const __nv_bfloat16* dx_in, __nv_bfloat16* dx, const float* dw_in, float* dw, int N, int D, int E, int per, int cw) {
  __shared__ float s_sum[kFewWarps<H>][16][33];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, q = lane & 3;
  const int tw = kFewWarps<H> / cw, wc = warp % cw, wt = warp / cw;
  const int col0 = (static_cast<int>(blockIdx.x) * cw + wc) * 64;
  const bool on = col0 < D;
  pdl_trigger();
  pdl_wait();
  uint32_t wf[8][H];
#pragma unroll
  for (int h = 0; h < H; ++h) {
    uint32_t f[8];
    expert_columns(wg, 8 * h, E, D, col0, on, lane, f);
#pragma unroll
    for (int t = 0; t < 8; ++t) wf[t][h] = f[t];
  }
  float acc[H][8][4];   // H 1: rows 0-7 the first term, 8-15 the others; H 2: [0] the first, [1] the others
#pragma unroll
  for (int h = 0; h < H; ++h)
#pragma unroll
    for (int t = 0; t < 8; ++t)
#pragma unroll
      for (int i = 0; i < 4; ++i) acc[h][t][i] = 0.0f;
  const int64_t t0 = static_cast<int64_t>(blockIdx.y) * per;
  const int64_t t1 = min(static_cast<int64_t>(N), t0 + per);
  for (int64_t base = t0 + 16 * wt; on && base < t1; base += 16 * tw) {
    uint4 xv[2][2], av[2][2];   // [rows g, g + 8][columns 8q.., 32 + 8q..]
    float2 v[2][H];
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      const int64_t t = base + g + 8 * r;
      const bool in = t < t1;
      const int64_t o = t * D + col0 + 8 * q;
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        xv[r][k] = av[r][k] = make_uint4(0, 0, 0, 0);
        if (in) xv[r][k] = __ldg(reinterpret_cast<const uint4*>(x + o + 32 * k));
        if (in && dx_in) av[r][k] = *reinterpret_cast<const uint4*>(dx_in + o + 32 * k);
      }
#pragma unroll
      for (int h = 0; h < H; ++h) {
        const int e = 8 * h + 2 * q;
        v[r][h].x = in && e < E ? __ldg(dl + t * E + e) : 0.0f;
        v[r][h].y = in && e + 1 < E ? __ldg(dl + t * E + e + 1) : 0.0f;
      }
    }
    uint32_t term[3][2][H];
#pragma unroll
    for (int i = 0; i < 3; ++i)
#pragma unroll
      for (int r = 0; r < 2; ++r)
#pragma unroll
        for (int h = 0; h < H; ++h) term[i][r][h] = next_term(v[r][h]);
    // dx: the addend and two terms
#pragma unroll
    for (int t = 0; t < 8; ++t) {
      uint32_t* p0 = reinterpret_cast<uint32_t*>(&av[0][t / 4]) + t % 4;
      uint32_t* p1 = reinterpret_cast<uint32_t*>(&av[1][t / 4]) + t % 4;
      float c[4] = {__uint_as_float(*p0 << 16), __uint_as_float(*p0 & 0xffff0000u), __uint_as_float(*p1 << 16),
                    __uint_as_float(*p1 & 0xffff0000u)};
      if (H == 1) {
        const uint32_t a[4] = {term[0][0][0], term[0][1][0], term[1][0][0], term[1][1][0]};
        mma_16x8x16(c, a, wf[t][0], wf[t][0]);
      } else {
#pragma unroll
        for (int i = 1; i >= 0; --i) {
          const uint32_t a[4] = {term[i][0][0], term[i][1][0], term[i][0][H - 1], term[i][1][H - 1]};
          mma_16x8x16(c, a, wf[t][0], wf[t][H - 1]);
        }
      }
      const __nv_bfloat162 r0 = __floats2bfloat162_rn(c[0], c[1]), r1 = __floats2bfloat162_rn(c[2], c[3]);
      *p0 = *reinterpret_cast<const uint32_t*>(&r0);
      *p1 = *reinterpret_cast<const uint32_t*>(&r1);
    }
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      const int64_t t = base + g + 8 * r;
      if (t < t1) {
#pragma unroll
        for (int k = 0; k < 2; ++k) *reinterpret_cast<uint4*>(dx + t * D + col0 + 8 * q + 32 * k) = av[r][k];
      }
    }
    // dw: three terms, x and they transposed
#pragma unroll
    for (int i = 0; i < 3; ++i)
#pragma unroll
      for (int r = 0; r < 2; ++r)
#pragma unroll
        for (int h = 0; h < H; ++h) term[i][r][h] = transpose8(term[i][r][h]);
#pragma unroll
    for (int t = 0; t < 8; ++t) {
      const uint32_t b0 = transpose8(reinterpret_cast<const uint32_t*>(&xv[0][t / 4])[t % 4]);
      const uint32_t b1 = transpose8(reinterpret_cast<const uint32_t*>(&xv[1][t / 4])[t % 4]);
      if (H == 1) {
        const uint32_t a[4] = {term[0][0][0], term[1][0][0], term[0][1][0], term[1][1][0]};
        const uint32_t a2[4] = {0u, term[2][0][0], 0u, term[2][1][0]};
        mma_16x8x16(acc[0][t], a, b0, b1);
        mma_16x8x16(acc[0][t], a2, b0, b1);
      } else {
#pragma unroll
        for (int i = 0; i < 3; ++i) {
          const uint32_t a[4] = {term[i][0][0], term[i][0][H - 1], term[i][1][0], term[i][1][H - 1]};
          mma_16x8x16(acc[i > 0 ? H - 1 : 0][t], a, b0, b1);
        }
      }
    }
  }
  few_join<H, kFewWarps<H>>(acc, s_sum, cw, E, 0, D, static_cast<int64_t>(blockIdx.y) * E * D, dw_in, dw);
}

// The same for few tokens of any number of experts, in one launch: blocks of z < G =
// ceil(E / 16) form dw of 16 experts each, 64 columns over all tokens, those behind them dx of 64 tokens each over
// all experts.  x is read G times and W once for every 64 tokens, from L2, which little work allows.
constexpr int kShortWarps = 4;
__global__ void __launch_bounds__(kShortWarps * 32, 3) router_short_kernel(
    const float* __restrict__ dl, const __nv_bfloat16* __restrict__ x, const __nv_bfloat16* __restrict__ wg,
    const __nv_bfloat16* dx_in, __nv_bfloat16* dx, const float* dw_in, float* dw, int N, int D, int E) {
  __shared__ float s_sum[kShortWarps][16][33];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, q = lane & 3;
  const int G = (E + 15) / 16, col0 = static_cast<int>(blockIdx.x) * 64;
  pdl_trigger();
  pdl_wait();
  // two (dx) or three terms of dlogits: rows g, g + 8, experts e0 + 2q, e0 + 8 + 2q and the next
  auto terms_of = [&](int base, int e0, auto& term) {
    constexpr int T = sizeof(term) / sizeof(term[0]);
#pragma unroll
    for (int r = 0; r < 2; ++r)
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int t = base + g + 8 * r, e = e0 + 8 * h + 2 * q;
        const float* p = dl + static_cast<int64_t>(t) * E + e;
        float2 v = make_float2(t < N && e < E ? __ldg(p) : 0.0f, t < N && e + 1 < E ? __ldg(p + 1) : 0.0f);
#pragma unroll
        for (int i = 0; i < T; ++i) term[i][r][h] = next_term(v);
      }
  };
  if (static_cast<int>(blockIdx.z) >= G) {
    const int base = 16 * ((static_cast<int>(blockIdx.z) - G) * kShortWarps + warp);
    if (base < N) {
      float c[8][4];
      uint4 av[2][2];
#pragma unroll
      for (int r = 0; r < 2; ++r)
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          const int t = base + g + 8 * r;
          av[r][k] = make_uint4(0, 0, 0, 0);
          if (t < N && dx_in)
            av[r][k] = *reinterpret_cast<const uint4*>(dx_in + static_cast<int64_t>(t) * D + col0 + 8 * q + 32 * k);
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const uint32_t w = reinterpret_cast<const uint32_t*>(&av[r][k])[i];
            c[4 * k + i][2 * r] = __uint_as_float(w << 16);
            c[4 * k + i][2 * r + 1] = __uint_as_float(w & 0xffff0000u);
          }
        }
      for (int e0 = 0; e0 < E; e0 += 16) {
        uint32_t w0[8], w1[8], term[2][2][2];
        terms_of(base, e0, term);
        expert_columns(wg, e0, E, D, col0, true, lane, w0);
        expert_columns(wg, e0 + 8, E, D, col0, true, lane, w1);
#pragma unroll
        for (int i = 1; i >= 0; --i) {
          const uint32_t a[4] = {term[i][0][0], term[i][1][0], term[i][0][1], term[i][1][1]};
#pragma unroll
          for (int t = 0; t < 8; ++t) mma_16x8x16(c[t], a, w0[t], w1[t]);
        }
      }
#pragma unroll
      for (int r = 0; r < 2; ++r)
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          const int t = base + g + 8 * r;
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const __nv_bfloat162 o = __floats2bfloat162_rn(c[4 * k + i][2 * r], c[4 * k + i][2 * r + 1]);
            reinterpret_cast<uint32_t*>(&av[r][k])[i] = *reinterpret_cast<const uint32_t*>(&o);
          }
          if (t < N) *reinterpret_cast<uint4*>(dx + static_cast<int64_t>(t) * D + col0 + 8 * q + 32 * k) = av[r][k];
        }
    }
    return;
  }
  const int e0 = 16 * static_cast<int>(blockIdx.z);
  float acc[2][8][4];   // [0] the first term, [1] the others
#pragma unroll
  for (int h = 0; h < 2; ++h)
#pragma unroll
    for (int t = 0; t < 8; ++t)
#pragma unroll
      for (int i = 0; i < 4; ++i) acc[h][t][i] = 0.0f;
  for (int base = 16 * warp; base < N; base += 16 * kShortWarps) {
    uint4 xv[2][2];
    uint32_t term[3][2][2];
#pragma unroll
    for (int r = 0; r < 2; ++r)
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        const int t = base + g + 8 * r;
        xv[r][k] = make_uint4(0, 0, 0, 0);
        if (t < N) xv[r][k] = __ldg(reinterpret_cast<const uint4*>(x + static_cast<int64_t>(t) * D + col0 + 8 * q + 32 * k));
      }
    terms_of(base, e0, term);
#pragma unroll
    for (int i = 0; i < 3; ++i)
#pragma unroll
      for (int r = 0; r < 2; ++r)
#pragma unroll
        for (int h = 0; h < 2; ++h) term[i][r][h] = transpose8(term[i][r][h]);
#pragma unroll
    for (int t = 0; t < 8; ++t) {
      const uint32_t b0 = transpose8(reinterpret_cast<const uint32_t*>(&xv[0][t / 4])[t % 4]);
      const uint32_t b1 = transpose8(reinterpret_cast<const uint32_t*>(&xv[1][t / 4])[t % 4]);
#pragma unroll
      for (int i = 0; i < 3; ++i) {
        const uint32_t a[4] = {term[i][0][0], term[i][0][1], term[i][1][0], term[i][1][1]};
        mma_16x8x16(acc[i > 0 ? 1 : 0][t], a, b0, b1);
      }
    }
  }
  few_join<2, kShortWarps>(acc, s_sum, 1, E, e0, D, 0, dw_in, dw);
}

// dw = dw_in + the runs' partial products: 32 numbers a block, its warps take the runs in turn and are joined in order.
__global__ void __launch_bounds__(256) router_few_sum_kernel(const float* __restrict__ part, int runs, int64_t n,
                                                             const float* dw_in, float* dw) {
  __shared__ float s_sum[8][32];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int64_t o = static_cast<int64_t>(blockIdx.x) * 32 + lane;   // n is a multiple of 32
  pdl_trigger();
  pdl_wait();
  float s = 0.0f;
#pragma unroll 4
  for (int r = warp; r < runs; r += 8) s += __ldcg(part + r * n + o);
  s_sum[warp][lane] = s;
  __syncthreads();
  if (warp != 0) return;
  for (int k = 1; k < 8; ++k) s += s_sum[k][lane];
  dw[o] = (dw_in ? dw_in[o] : 0.0f) + s;
}

}  // namespace

cudaError_t launch_seq_balance(const SeqBalanceArgs& a, cudaStream_t st) {
  if (a.n_tok < 1 || a.n_exp < 1 || a.n_exp > 1024 || a.n_seq < 1) return cudaErrorInvalidValue;
  const int64_t copies = static_cast<int64_t>(a.n_tok) * a.top_k;
  // Little enough: one launch of one cluster instead of two.  Enqueueing the second costs more than 2 us, and the
  // kernels' own time is level: 256 x 8, top-2, 1 sequence 7.6 us a call for 9.8 (captured 6.2 for 6.0), 64 x 60 in 8
  // sequences 7.6 for 9.7 (5.8 for 6.4).  Beyond, eight blocks take longer than a grid: 512 x 8 7.5 us captured
  // for 6.6, 128 x 64 in 8 sequences 7.6 for 6.2, 128 x 256 13.2 for 7.4
  const bool one = copies <= 512 && a.n_seq <= 8 && a.n_exp <= 64 && static_cast<int64_t>(a.n_tok) * a.n_exp <= 4096;
  const int grid = one ? kAllBlocks : rows_grid(a.n_tok, a.n_exp);
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
  p.S = a.n_seq;
  p.idx = a.topk_idx;
  p.status = a.status;
  p.K = a.top_k;
  p.per = static_cast<int>((static_cast<int64_t>(a.n_tok) + static_cast<int64_t>(grid) * kWarps - 1) /
                           (static_cast<int64_t>(grid) * kWarps));
  if (one)
    return launch_pdl<kAllBlocks>(a.gate == 0 ? all_kernel<0>(a.n_exp) : all_kernel<1>(a.n_exp), kAllBlocks, kThreads, 0,
                                  st, p);
  // One block counts a sequence of up to about 8192 indices in one turn of its 1024 threads; longer
  // ones, on average, take a cluster of eight (16384 of them: 12 thousand cycles in one block, 9 in eight).
  cudaError_t e;
  if (copies / a.n_seq > 8192) {
    e = launch_pdl<8>(seq_counts_kernel<8, 256>, static_cast<unsigned>(a.n_seq + 1) * 8, 256,
                      8 * static_cast<size_t>(a.n_exp) * sizeof(int), st, a.n_tok, a.n_exp, a.top_k, a.n_seq, 8,
                      a.topk_idx, a.seq_offsets, a.counts, a.head, a.status);
  } else if (copies / a.n_seq > 512 || copies > 32768) {   // lengths may be uneven: one sequence may hold most
    const int nh = a.n_exp <= 256 ? 32 : 8;
    e = launch_pdl(seq_counts_kernel<1, 1024>, static_cast<unsigned>(a.n_seq + 1), 1024,
                   nh * static_cast<size_t>(a.n_exp) * sizeof(int), st, a.n_tok, a.n_exp, a.top_k, a.n_seq, nh,
                   a.topk_idx, a.seq_offsets, a.counts, a.head, a.status);
  } else {
    e = launch_pdl(seq_counts_kernel<1, 256>, static_cast<unsigned>(a.n_seq + 1), 256,
                   8 * static_cast<size_t>(a.n_exp) * sizeof(int), st, a.n_tok, a.n_exp, a.top_k, a.n_seq, 8,
                   a.topk_idx, a.seq_offsets, a.counts, a.head, a.status);
  }
  if (e != cudaSuccess) return e;
  // 16-byte words above 64 experts (below, lanes would idle), where every row starts on one
  const bool vec = a.n_exp > 64 && a.n_exp % 4 == 0 && ((reinterpret_cast<uintptr_t>(a.logits) |
                                                        reinterpret_cast<uintptr_t>(a.dlogits)) & 15u) == 0;
  auto kern = a.gate == 0 ? rows_kernel<0>(a.n_exp, vec) : rows_kernel<1>(a.n_exp, vec);
  return launch_pdl(kern, static_cast<unsigned>(grid), kThreads, 0, st, p);
}

cudaError_t launch_router_terms(const float* dl, int n_tok, int n_exp, void* terms, int32_t* dense, int32_t* slices,
                                int n_slices, int slice_rows, cudaStream_t st) {
  const int e8 = router_term_cols(n_exp);
  const int64_t items = static_cast<int64_t>(n_tok) * (e8 / 8);
  return launch_pdl(router_terms_kernel, static_cast<unsigned>((items + 255) / 256), 256, 0, st, dl, n_tok, n_exp, e8,
                    static_cast<uint4*>(terms), dense, slices, n_slices, slice_rows);
}

cudaError_t launch_router_dw(const float* part, int n_slices, int terms, int n_exp, int d, const float* dw_in,
                             float* dw, cudaStream_t st) {
  const int64_t n = static_cast<int64_t>(n_exp) * d, term = static_cast<int64_t>(router_term_cols(n_exp)) * d;
  if (n / 4 >= static_cast<int64_t>(num_sms()) * 512)
    return launch_pdl(terms == 3 ? router_dw_kernel<3, float4> : router_dw_kernel<1, float4>,
                      static_cast<unsigned>((n / 4 + 255) / 256), 256, 0, st, reinterpret_cast<const float4*>(part),
                      n_slices, n / 4, term / 4, reinterpret_cast<const float4*>(dw_in), reinterpret_cast<float4*>(dw));
  return launch_pdl(terms == 3 ? router_dw_kernel<3, float> : router_dw_kernel<1, float>,
                    static_cast<unsigned>((n + 255) / 256), 256, 0, st, part, n_slices, n, term, dw_in, dw);
}

cudaError_t launch_router_few(const float* dl, const void* x, const void* w_gate, const void* dx_in, void* dx,
                              float* part, size_t part_bytes, int n_tok, int d, int n_exp, const float* dw_in,
                              float* dw, cudaStream_t st) {
  if (n_exp > kRouterFew || n_tok < 1 || d % 64) return cudaErrorInvalidValue;
  // Warps along the columns and runs of tokens: about 2.2 us a turn of all the warps' 16 tokens x 64 columns;
  // partial products are written and read again by a launch of its own
  const bool two = n_exp > 8;
  const int strips64 = d / 64, warps = two ? kFewWarps<2> : kFewWarps<1>;
  const int at_once = num_sms() * (two ? kFewBlocks<2> : kFewBlocks<1>);
  const int64_t fit = std::min<int64_t>(kRouterFewRuns, static_cast<int64_t>(part_bytes / (sizeof(float) * n_exp * d)));
  int cw = 1;
  int64_t per = n_tok, runs = 1;
  double best = 0;
  for (int w = 1; w <= warps; w *= 2) {
    const int64_t strips = (strips64 + w - 1) / w, tile = 16 * (warps / w);   // tokens of a block's turn
    const int64_t turns_all = (n_tok + tile - 1) / tile;
    for (int64_t r = 1; r <= std::max<int64_t>(1, std::min(fit, turns_all)); ++r) {
      const int64_t turns = (turns_all + r - 1) / r, n = (turns_all + turns - 1) / turns;
      const int64_t waves = (strips * n + at_once - 1) / at_once;
      const double t = waves * (2.2 * turns + 1) + (n > 1 ? 3 + n * n_exp * d * 8.0 / 5e6 : 0) +
                       (turns > kFewTurns ? turns - kFewTurns : 0);
      if (best == 0 || t < best) {
        best = t;
        cw = w;
        runs = n;
        per = turns * tile;
      }
    }
  }
  const int strips = (strips64 + cw - 1) / cw;
  auto kern = two ? router_few_kernel<2> : router_few_kernel<1>;
  cudaLaunchConfig_t cfg{};
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.gridDim = dim3(static_cast<unsigned>(strips), static_cast<unsigned>(runs));
  cfg.blockDim = dim3(warps * 32);
  cfg.stream = st;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  const auto* xb = static_cast<const __nv_bfloat16*>(x);
  const cudaError_t e = cudaLaunchKernelEx(
      &cfg, kern, dl, xb, static_cast<const __nv_bfloat16*>(w_gate), static_cast<const __nv_bfloat16*>(dx_in),
      static_cast<__nv_bfloat16*>(dx), runs > 1 ? nullptr : dw_in, runs > 1 ? part : dw, n_tok, d, n_exp,
      static_cast<int>(per), cw);
  if (e != cudaSuccess || runs == 1) return e;
  const int64_t n = static_cast<int64_t>(n_exp) * d;
  return launch_pdl(router_few_sum_kernel, static_cast<unsigned>(n / 32), 256, 0, st, const_cast<const float*>(part),
                    static_cast<int>(runs), n, dw_in, dw);
}

cudaError_t launch_router_short(const float* dl, const void* x, const void* w_gate, const void* dx_in, void* dx, int n_tok,
                                int d, int n_exp, const float* dw_in, float* dw, cudaStream_t st) {
  if (n_tok < 1 || n_tok > kRouterShort || d % 64) return cudaErrorInvalidValue;
  cudaLaunchConfig_t cfg{};
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.gridDim = dim3(static_cast<unsigned>(d / 64), 1,
                     static_cast<unsigned>((n_exp + 15) / 16 + (n_tok + 16 * kShortWarps - 1) / (16 * kShortWarps)));
  cfg.blockDim = dim3(kShortWarps * 32);
  cfg.stream = st;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, router_short_kernel, dl, static_cast<const __nv_bfloat16*>(x),
                            static_cast<const __nv_bfloat16*>(w_gate), static_cast<const __nv_bfloat16*>(dx_in),
                            static_cast<__nv_bfloat16*>(dx), dw_in, dw, n_tok, d, n_exp);
}

}  // namespace moe
