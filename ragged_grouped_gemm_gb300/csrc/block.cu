// Layer norm (forward, backward with the reduction of the weight gradients)
// and the residual dropout of a pre-norm MoE block.
#include "block.cuh"
#include "grouped_gemm.cuh"
#include "pdl.cuh"
#include "sm100_ptx.cuh"

#include <cuda_bf16.h>

#include <algorithm>

namespace moe {
namespace {

__device__ __forceinline__ uint32_t pack2(float a, float b) {
  __nv_bfloat162 v = __floats2bfloat162_rn(a, b);
  return *reinterpret_cast<uint32_t*>(&v);
}

// Eight consecutive elements of a bf16 or fp32 row, kept packed as loaded.
template <bool F32>
struct Vec8;
template <>
struct Vec8<false> {
  uint4 a;
  __device__ __forceinline__ void load(const void* p, int64_t i) { a = __ldg(static_cast<const uint4*>(p) + i); }
  __device__ __forceinline__ void zero() { a = make_uint4(0, 0, 0, 0); }
  __device__ __forceinline__ float get(int j) const {
    const uint32_t w = (j >> 1) == 0 ? a.x : (j >> 1) == 1 ? a.y : (j >> 1) == 2 ? a.z : a.w;
    return (j & 1) ? __uint_as_float(w & 0xFFFF0000u) : __uint_as_float(w << 16);
  }
  __device__ __forceinline__ static void store(void* p, int64_t i, const float (&f)[8]) {
    static_cast<uint4*>(p)[i] = make_uint4(pack2(f[0], f[1]), pack2(f[2], f[3]), pack2(f[4], f[5]), pack2(f[6], f[7]));
  }
};
template <>
struct Vec8<true> {
  float4 a, b;
  __device__ __forceinline__ void load(const void* p, int64_t i) {
    a = __ldg(static_cast<const float4*>(p) + 2 * i);
    b = __ldg(static_cast<const float4*>(p) + 2 * i + 1);
  }
  __device__ __forceinline__ void zero() { a = b = make_float4(0.f, 0.f, 0.f, 0.f); }
  __device__ __forceinline__ float get(int j) const {
    return j == 0 ? a.x : j == 1 ? a.y : j == 2 ? a.z : j == 3 ? a.w : j == 4 ? b.x : j == 5 ? b.y : j == 6 ? b.z : b.w;
  }
  __device__ __forceinline__ static void store(void* p, int64_t i, const float (&f)[8]) {
    static_cast<float4*>(p)[2 * i] = make_float4(f[0], f[1], f[2], f[3]);
    static_cast<float4*>(p)[2 * i + 1] = make_float4(f[4], f[5], f[6], f[7]);
  }
};

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}
// Sum over the T threads of a block; s holds one value per warp, and a caller
// alternates between two of them, so that one barrier a sum is enough.
template <int T>
__device__ __forceinline__ float block_sum(float v, float* s) {
  v = warp_sum(v);
  if ((threadIdx.x & 31) == 0) s[threadIdx.x >> 5] = v;
  __syncthreads();
  float t = 0.0f;
#pragma unroll
  for (int w = 0; w < T / 32; ++w) t += s[w];
  return t;
}

// ---- clusters: C blocks of a cluster hold the columns of a row between them
template <int C>
__device__ __forceinline__ uint32_t cluster_rank() {
  return C > 1 ? cluster_ctarank() : 0u;
}
__device__ __forceinline__ void st_cluster_f32(const void* at, uint32_t rank, float v) {
  asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(mapa_shared(smem_u32(at), rank)), "f"(v) : "memory");
}
__device__ __forceinline__ void st_cluster_f32x2(const void* at, uint32_t rank, float v, float w) {
  asm volatile("st.shared::cluster.v2.f32 [%0], {%1, %2};" ::"r"(mapa_shared(smem_u32(at), rank)), "f"(v), "f"(w)
               : "memory");
}

// N sums (2 or 4) over the T threads of each of C blocks at once.  While two lanes
// have more than one sum between them, each passes the half that the other goes on
// with; in one block the warps' sums are joined the same way (16 warps: 5 + 6 shuffles for
// two sums, 7 + 12 for four).  In a cluster each warp leaves its sums with every block.  s
// holds N values a warp of the cluster, and a caller alternates between two of them.
template <int T, int N, int C>
__device__ __forceinline__ void block_sums(float (&v)[N], float (*s)[N]) {
  constexpr int W = T / 32;
  const int lane = threadIdx.x & 31;
  float a;
  if constexpr (N == 4) {
    const bool up = lane & 16;
    const float k0 = (up ? v[2] : v[0]) + __shfl_xor_sync(0xffffffffu, up ? v[0] : v[2], 16);
    const float k1 = (up ? v[3] : v[1]) + __shfl_xor_sync(0xffffffffu, up ? v[1] : v[3], 16);
    const bool up2 = lane & 8;
    a = (up2 ? k1 : k0) + __shfl_xor_sync(0xffffffffu, up2 ? k0 : k1, 8);
  } else {
    const bool up = lane & 16;
    a = (up ? v[1] : v[0]) + __shfl_xor_sync(0xffffffffu, up ? v[0] : v[1], 16);
  }
#pragma unroll
  for (int o = 16 / N; o > 0; o >>= 1) a += __shfl_xor_sync(0xffffffffu, a, o);
  const int warp = threadIdx.x >> 5, which = lane / (32 / N);
  const bool mine = lane % (32 / N) == 0;
  if constexpr (C > 1) {
    static_assert(C * W % 32 == 0);
    const uint32_t me = cluster_rank<C>();
    if (mine)
#pragma unroll
      for (int c = 0; c < C; ++c) st_cluster_f32(&s[me * W + warp][which], c, a);
    cluster_sync_all();
#pragma unroll
    for (int j = 0; j < N; ++j) {
      v[j] = 0.0f;
#pragma unroll
      for (int w = 0; w < C * W; w += 32) v[j] += s[w + lane][j];
      v[j] = warp_sum(v[j]);
    }
  } else {
    if (mine) s[warp][which] = a;
    __syncthreads();
    // lane l takes Q sums of warp l % W
    constexpr int P = 32 / W, Q = N > P ? N / P : 1;
    float q[Q];
#pragma unroll
    for (int j = 0; j < Q; ++j) {
      q[j] = s[lane % W][lane / W % (N / Q) * Q + j];
#pragma unroll
      for (int o = W / 2; o > 0; o >>= 1) q[j] += __shfl_xor_sync(0xffffffffu, q[j], o);
    }
#pragma unroll
    for (int j = 0; j < N; ++j) v[j] = N == Q ? q[j] : __shfl_sync(0xffffffffu, q[j % Q], j / Q * W);
  }
}

// A warp a row of at most 1024 elements, V vectors of eight columns a lane.  The mean
// and then the squared deviations from it are summed over the registers that hold the
// row, so the variance loses nothing to a large mean.
constexpr int kRowWarps = 8;   // rows of a block
template <bool F32, int V>
__global__ void __launch_bounds__(kRowWarps * 32) layernorm_kernel(int64_t rows, int d8, const void* __restrict__ x,
                                                                   const float* __restrict__ gamma,
                                                                   const float* __restrict__ beta, float eps,
                                                                   void* __restrict__ y, float* __restrict__ mean,
                                                                   float* __restrict__ rstd) {
  pdl_trigger();
  pdl_wait();
  const int lane = threadIdx.x & 31;
  const float inv_d = 1.0f / static_cast<float>(d8 * 8);
  for (int64_t r = static_cast<int64_t>(blockIdx.x) * kRowWarps + threadIdx.x / 32; r < rows;
       r += static_cast<int64_t>(gridDim.x) * kRowWarps) {
    Vec8<F32> v[V];
    float sum = 0.0f;
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int c = lane + i * 32;
      if (c < d8) v[i].load(x, r * d8 + c);
      else v[i].zero();
    }
#pragma unroll
    for (int i = 0; i < V; ++i)
#pragma unroll
      for (int j = 0; j < 8; ++j) sum += v[i].get(j);
    const float mu = warp_sum(sum) * inv_d;
    float sq = 0.0f;
#pragma unroll
    for (int i = 0; i < V; ++i)
      if (lane + i * 32 < d8) {
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const float e = v[i].get(j) - mu;
          sq = fmaf(e, e, sq);
        }
      }
    const float rs = 1.0f / sqrtf(warp_sum(sq) * inv_d + eps);
    if (lane == 0) {
      if (mean) mean[r] = mu;
      if (rstd) rstd[r] = rs;
    }
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int c = lane + i * 32;
      if (c < d8) {
        Vec8<true> g, b;
        g.load(gamma, c);
        if (beta) b.load(beta, c);
        else b.zero();
        float o[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) o[j] = fmaf((v[i].get(j) - mu) * rs, g.get(j), b.get(j));
        Vec8<false>::store(y, r * d8 + c, o);
      }
    }
  }
}

// ---- rows through shared memory
// For rows of more than 1024 elements the inputs arrive by bulk copies in a ring
// of row buffers, so that the loads of the next rows run under the arithmetic
// and the block sums of this one; gamma, beta and the gradients' sums stay in
// registers.  4096 rows of 7168 bf16 numbers: 25.8 us forward, 41 us backward with
// its sums (17.3 and 34.6 at the rate of a plain copy); straight from global
// memory, two blocks of 256 threads an SM, 27.2 and 66; one row 2.5 against 2.9.
// What bounds it is a row's way through a block: two (backward: one) block sums
// and 16 elements a thread, about 1.7 us.  Forward, one sum a row by taking the next
// row's mean along needs twice the registers, one block an SM: 31.9 us; two rows
// together spill at two blocks an SM: 40.8.
// Above 8192 elements a cluster of two blocks, above 16384 one of four, shares the row,
// each with a ring of its own columns.  2730 rows of 12288 bf16 numbers: 40 us forward,
// 64 backward; 1024 of 32768 40 and 68 (all 19.8 and 39.6 at the rate of a plain copy).
// From global memory with 1024 threads a row they were 64, 88, 47 and 147: no loads under
// the sums, and the backward's sums did not fit the registers.
constexpr int kRingBytes = 200 * 1024;   // of an SM's shared memory, over its blocks

__device__ __forceinline__ void bulk_load(void* dst, const void* src, uint32_t bytes, uint64_t* bar) {
  asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(
                   smem_u32(dst)),
               "l"(src), "r"(bytes), "r"(smem_u32(bar))
               : "memory");
}

// Vector c of a row in shared memory, packed.
template <bool F32>
__device__ __forceinline__ Vec8<F32> smem_vec8(const uint8_t* row, int c) {
  Vec8<F32> v;
  if constexpr (F32) {
    v.a = reinterpret_cast<const float4*>(row)[2 * c];
    v.b = reinterpret_cast<const float4*>(row)[2 * c + 1];
  } else {
    v.a = reinterpret_cast<const uint4*>(row)[c];
  }
  return v;
}
__device__ __forceinline__ void load_f32x8(const float* p, int c, float (&f)[8]) {
  Vec8<true> v;
  v.load(p, c);
#pragma unroll
  for (int j = 0; j < 8; ++j) f[j] = v.get(j);
}

// Waits for a row.  A wait that runs out raises `stop` in every block of the cluster, at which
// no later wait of the turn begins; a caller looks at it behind the row's next barrier, which
// no thread passes before the row's waits, and takes turns between two of them where there is one
// barrier a turn, so that all threads find the same.  It leaves at the turn's end, so that nothing
// waits for the look, and what the turn stored is overwritten.
constexpr int kRowWaitSite = 900;
__device__ __forceinline__ bool stopped(const int* stop) { return *static_cast<const volatile int*>(stop) != 0; }
template <int C>
__device__ __forceinline__ void wait_row(uint64_t* bar, uint32_t parity, int* stop, const RowWait& w) {
  if (mbar_try_wait(bar, parity)) return;
  if (!stopped(stop) && mbar_wait_drain(bar, parity, w.limit_ns)) return;
  *static_cast<volatile int*>(stop) = 1;
  if (w.status) {
    atomicOr(w.status, DEV_TIMEOUT);
    atomicExch(w.status + 1, kRowWaitSite);
  }
  if constexpr (C > 1)
    for (int c = 0; c < C; ++c)
      asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(mapa_shared(smem_u32(stop), c)), "r"(1) : "memory");
}
__device__ __forceinline__ float not_a_number() { return __uint_as_float(0x7FC00000u); }
// What a block does that gives up at row r: one thread waits, with a limit too, for the copies
// under way, those of `stages` rows; vectors first .. first + n8 - 1 of the rows left are not a number.
template <bool F32>
__device__ __noinline__ void give_up(uint64_t* full, int stages, int64_t r, int64_t row0, int64_t step, int64_t rows,
                                     int d8, int first, int n8, void* out, float* mean, float* rstd,
                                     uint64_t limit_ns) {
  if (threadIdx.x == 0) {
    int64_t j = (r - row0) / step, at = r;
    for (int k = 0; k < stages && at < rows; ++k, ++j, at += step)
      mbar_wait_drain(&full[j % stages], static_cast<uint32_t>(j / stages) & 1u, limit_ns / 8);
  }
  float f[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) f[j] = not_a_number();
  for (; r < rows; r += step) {
    for (int c = threadIdx.x; c < n8; c += blockDim.x) Vec8<F32>::store(out, r * d8 + first + c, f);
    if (threadIdx.x == 0 && first == 0) {
      if (mean) mean[r] = not_a_number();
      if (rstd) rstd[r] = not_a_number();
    }
  }
}

// A block's share of the rows: vectors first .. first + n8 - 1 of rows row0, row0 + step, ...
struct Part {
  int first, n8;
  int64_t row0, step;
};
template <int C>
__device__ __forceinline__ Part part_of(int d8) {
  if constexpr (C == 1) return {0, d8, blockIdx.x, gridDim.x};
  const int per = (d8 + C - 1) / C, first = per * static_cast<int>(cluster_rank<C>());
  return {first, min(per, d8 - first), blockIdx.x / C, gridDim.x / C};
}
// Columns of a row that warp w of block `rank` holds.
template <int T, int V, int C>
__device__ __forceinline__ float warp_columns(int d8, int rank, int w) {
  const int per = (d8 + C - 1) / C, n8 = min(per, d8 - per * rank);
  int n = 0;
#pragma unroll
  for (int i = 0; i < V; ++i) n += max(0, min(32, n8 - i * T - w * 32));
  return static_cast<float>(8 * n);
}

// T threads share a row, V vectors of eight columns each; `stages` row buffers.
template <bool F32, int T, int V>
__global__ void __launch_bounds__(T, 1024 / T) layernorm_ring_kernel(
    int64_t rows, int d8, int stages, const uint8_t* __restrict__ x, const float* __restrict__ gamma,
    const float* __restrict__ beta, float eps, void* __restrict__ y, float* __restrict__ mean,
    float* __restrict__ rstd, const RowWait wait) {
  extern __shared__ __align__(128) uint8_t ring[];
  __shared__ uint64_t full[8];
  __shared__ int stop;
  __shared__ float s_red[2][T / 32];
  const int tid = threadIdx.x;
  const uint32_t xb = static_cast<uint32_t>(d8) * (F32 ? 32 : 16);
  const float inv_d = 1.0f / static_cast<float>(d8 * 8);
  if (tid == 0) {
    for (int s = 0; s < stages; ++s) mbar_init(&full[s], 1);
    stop = 0;
    fence_mbar_init();
  }
  pdl_trigger();
  pdl_wait();
  float g[V][8], b[V][8];
#pragma unroll
  for (int i = 0; i < V; ++i) {
    const int c = min(tid + i * T, d8 - 1);
    load_f32x8(gamma, c, g[i]);
    if (beta) load_f32x8(beta, c, b[i]);
    else
#pragma unroll
      for (int j = 0; j < 8; ++j) b[i][j] = 0.0f;
  }
  __syncthreads();
  auto fetch = [&](int s, int64_t r) {
    if (r == wait.withheld) return;
    mbar_arrive_expect_tx(&full[s], xb);
    bulk_load(ring + static_cast<size_t>(s) * xb, x + r * xb, xb, &full[s]);
  };
  if (tid == 0)
    for (int s = 0; s < stages; ++s) {
      const int64_t r = blockIdx.x + static_cast<int64_t>(s) * gridDim.x;
      if (r < rows) fetch(s, r);
    }
  int s = 0;
  uint32_t ph = 0;
  int64_t r = blockIdx.x;
  for (; r < rows; r += gridDim.x) {
    wait_row<1>(&full[s], ph, &stop, wait);
    const uint8_t* row = ring + static_cast<size_t>(s) * xb;
    float v[V][8];
    float sum = 0.0f;
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int c = tid + i * T;
      if (c < d8) {
        const Vec8<F32> p = smem_vec8<F32>(row, c);
#pragma unroll
        for (int j = 0; j < 8; ++j) v[i][j] = p.get(j);
      } else {
#pragma unroll
        for (int j = 0; j < 8; ++j) v[i][j] = 0.0f;
      }
#pragma unroll
      for (int j = 0; j < 8; ++j) sum += v[i][j];
    }
    const float mu = block_sum<T>(sum, s_red[0]) * inv_d;
    const bool halt = stopped(&stop);
    // every thread has read the buffer: the row after next `stages` may land in it
    const int64_t next = r + static_cast<int64_t>(stages) * gridDim.x;
    if (tid == 0 && !halt && next < rows) fetch(s, next);
    float sq = 0.0f;
#pragma unroll
    for (int i = 0; i < V; ++i)
      if (tid + i * T < d8) {
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const float e = v[i][j] - mu;
          sq = fmaf(e, e, sq);
        }
      }
    const float rs = 1.0f / sqrtf(block_sum<T>(sq, s_red[1]) * inv_d + eps);
    if (tid == 0) {
      if (mean) mean[r] = mu;
      if (rstd) rstd[r] = rs;
    }
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int c = tid + i * T;
      if (c < d8) {
        float o[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) o[j] = fmaf((v[i][j] - mu) * rs, g[i][j], b[i][j]);
        Vec8<false>::store(y, r * d8 + c, o);
      }
    }
    if (halt) break;
    if (++s == stages) {
      s = 0;
      ph ^= 1u;
    }
  }
  if (r < rows)
    give_up<false>(full, stages, r, blockIdx.x, gridDim.x, rows, d8, 0, d8, y, mean, rstd, wait.limit_ns);
}

// T threads of C blocks share a row, V vectors of eight columns each; `stages` row
// buffers.  R rows an exchange between the blocks, which costs about 0.6 us: every warp
// takes its columns' mean m_w and the squares about it, q_w, and mean = sum n_w m_w / n,
// variance = sum (q_w + n_w (m_w - mean)^2) / n, which like two passes over the row loses
// nothing to a large mean.  Two exchanges of one row each, two blocks an SM: 2730 x 12288
// 54.7 us, one 43.7; four bf16 (two fp32) rows an exchange, one block an SM, 40.2.
template <bool F32, int T, int V, int R, int C>
__global__ void __launch_bounds__(T, 512 / T) layernorm_cluster_kernel(
    int64_t rows, int d8, int stages, const uint8_t* __restrict__ x, const float* __restrict__ gamma,
    const float* __restrict__ beta, float eps, void* __restrict__ y, float* __restrict__ mean,
    float* __restrict__ rstd, const RowWait wait) {
  extern __shared__ __align__(128) uint8_t ring[];
  __shared__ uint64_t full[8];
  __shared__ int stop[2];
  constexpr int W = C * T / 32, K = W / 32;   // warps of a row; a lane joins K of them
  static_assert(W % 32 == 0);
  __shared__ float2 s_red[2][W][R];
  const int tid = threadIdx.x, lane = tid & 31;
  const Part part = part_of<C>(d8);
  const int n8 = part.n8;
  const uint32_t xb = static_cast<uint32_t>(n8) * (F32 ? 32 : 16);
  const float inv_d = 1.0f / static_cast<float>(d8 * 8);
  if (tid == 0) {
    for (int s = 0; s < stages; ++s) mbar_init(&full[s], 1);
    stop[0] = stop[1] = 0;
    fence_mbar_init();
  }
  pdl_trigger();
  pdl_wait();
  float g[V][8], b[V][8];
#pragma unroll
  for (int i = 0; i < V; ++i) {
    const int c = part.first + min(tid + i * T, n8 - 1);
    load_f32x8(gamma, c, g[i]);
    if (beta) load_f32x8(beta, c, b[i]);
    else
#pragma unroll
      for (int j = 0; j < 8; ++j) b[i][j] = 0.0f;
  }
  cluster_sync_all();   // every block of the cluster has started
  const int me = static_cast<int>(cluster_rank<C>()) * (T / 32) + (tid >> 5);
  const float own_n = warp_columns<T, V, C>(d8, me / (T / 32), me % (T / 32));
  const float own_inv = own_n > 0.0f ? 1.0f / own_n : 0.0f;
  float wn[K], winv[K];
#pragma unroll
  for (int k = 0; k < K; ++k) {
    const int w = lane + 32 * k;
    wn[k] = warp_columns<T, V, C>(d8, w / (T / 32), w % (T / 32));
    winv[k] = wn[k] > 0.0f ? 1.0f / wn[k] : 0.0f;
  }
  auto fetch = [&](int s, int64_t r) {
    if (r == wait.withheld) return;
    mbar_arrive_expect_tx(&full[s], xb);
    bulk_load(ring + static_cast<size_t>(s) * xb, x + (r * d8 + part.first) * (F32 ? 32 : 16), xb, &full[s]);
  };
  if (tid == 0)
    for (int s = 0; s < stages; ++s) {
      const int64_t r = part.row0 + static_cast<int64_t>(s) * part.step;
      if (r < rows) fetch(s, r);
    }
  int s = 0, flip = 0;
  uint32_t ph = 0;
  int64_t r = part.row0;
  for (; r < rows; r += R * part.step, flip ^= 1) {
    Vec8<F32> v[R][V];
    float sum[R], sq[R];
    int freed[R];
#pragma unroll
    for (int h = 0; h < R; ++h) {
      const bool have = h == 0 || r + h * part.step < rows;
      const uint8_t* row = ring + static_cast<size_t>(s) * xb;
      sum[h] = sq[h] = 0.0f;
      if (have) wait_row<C>(&full[s], ph, &stop[flip], wait);
#pragma unroll
      for (int i = 0; i < V; ++i) {
        const int c = tid + i * T;
        if (have && c < n8) v[h][i] = smem_vec8<F32>(row, c);
        else v[h][i].zero();
#pragma unroll
        for (int j = 0; j < 8; ++j) sum[h] += v[h][i].get(j);
      }
      freed[h] = s;
      if (++s == stages) {
        s = 0;
        ph ^= 1u;
      }
    }
#pragma unroll
    for (int h = 0; h < R; ++h) {
      sum[h] = warp_sum(sum[h]);
      const float wmean = sum[h] * own_inv;
#pragma unroll
      for (int i = 0; i < V; ++i)
        if (tid + i * T < n8) {
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            const float e = v[h][i].get(j) - wmean;
            sq[h] = fmaf(e, e, sq[h]);
          }
        }
    }
#pragma unroll
    for (int h = 0; h < R; ++h) {
      sq[h] = warp_sum(sq[h]);
      if (lane < C) st_cluster_f32x2(&s_red[flip][me][h], lane, sum[h], sq[h]);
    }
    cluster_sync_all();
    const bool halt = stopped(&stop[flip]);
    // every thread has read the buffers: later rows may land in them
    if (tid == 0 && !halt)
#pragma unroll
      for (int h = 0; h < R; ++h) {
        const int64_t next = r + (h + stages) * part.step;
        if (next < rows) fetch(freed[h], next);
      }
#pragma unroll
    for (int h = 0; h < R; ++h) {
      const int64_t row = r + h * part.step;
      if (h > 0 && row >= rows) break;
      float2 p[K];
      float mu = 0.0f, var = 0.0f;
#pragma unroll
      for (int k = 0; k < K; ++k) {
        p[k] = s_red[flip][lane + 32 * k][h];
        mu += p[k].x;
      }
      mu = warp_sum(mu) * inv_d;
#pragma unroll
      for (int k = 0; k < K; ++k) {
        const float e = fmaf(p[k].x, winv[k], -mu);
        var += fmaf(wn[k] * e, e, p[k].y);
      }
      const float rs = 1.0f / sqrtf(warp_sum(var) * inv_d + eps);
      if (tid == 0 && part.first == 0) {
        if (mean) mean[row] = mu;
        if (rstd) rstd[row] = rs;
      }
#pragma unroll
      for (int i = 0; i < V; ++i) {
        const int c = tid + i * T;
        if (c < n8) {
          float o[8];
#pragma unroll
          for (int j = 0; j < 8; ++j) o[j] = fmaf((v[h][i].get(j) - mu) * rs, g[i][j], b[i][j]);
          Vec8<false>::store(y, row * d8 + part.first + c, o);
        }
      }
    }
    if (halt) break;
  }
  if (r < rows)
    give_up<false>(full, stages, r, part.row0, part.step, rows, d8, part.first, n8, y, mean, rstd, wait.limit_ns);
}

// R rows pass through a block together, packed: two bf16 rows
// share the block sum, 41 us against 46; fp32 rows have no registers for it.
template <bool F32, int T, int V, int R, int C>
__global__ void __launch_bounds__(T, 512 / T) layernorm_bwd_ring_kernel(
    int64_t rows, int d8, int stages, const uint8_t* __restrict__ dy, const uint8_t* __restrict__ x,
    const float* __restrict__ gamma, const float* __restrict__ mean, const float* __restrict__ rstd,
    const uint8_t* __restrict__ dres, void* __restrict__ dx, float* __restrict__ part, const RowWait wait) {
  extern __shared__ __align__(128) uint8_t ring[];
  __shared__ uint64_t full[8];
  __shared__ int stop[2];
  __shared__ __align__(16) float s_red[2][C * T / 32][2 * R];
  const int tid = threadIdx.x;
  const Part own = part_of<C>(d8);
  const int n8 = own.n8;
  const uint32_t xb = static_cast<uint32_t>(n8) * (F32 ? 32 : 16), yb = static_cast<uint32_t>(n8) * 16;
  const float inv_d = 1.0f / static_cast<float>(d8 * 8);
  if (tid == 0) {
    for (int s = 0; s < stages; ++s) mbar_init(&full[s], 1);
    stop[0] = stop[1] = 0;
    fence_mbar_init();
  }
  pdl_trigger();
  pdl_wait();
  float g[V][8], dg[V][8], db[V][8];
#pragma unroll
  for (int i = 0; i < V; ++i) {
    load_f32x8(gamma, own.first + min(tid + i * T, n8 - 1), g[i]);
#pragma unroll
    for (int j = 0; j < 8; ++j) dg[i][j] = db[i][j] = 0.0f;
  }
  if constexpr (C > 1) cluster_sync_all();   // every block of the cluster has started
  else __syncthreads();
  const uint32_t sb = xb + yb + (dres ? xb : 0);   // a row's x, dy and dres
  auto fetch = [&](int s, int64_t r) {
    uint8_t* dst = ring + static_cast<size_t>(s) * sb;
    if (r == wait.withheld) return;
    mbar_arrive_expect_tx(&full[s], sb);
    const int64_t at = r * d8 + own.first;
    bulk_load(dst, x + at * (F32 ? 32 : 16), xb, &full[s]);
    bulk_load(dst + xb, dy + at * 16, yb, &full[s]);
    if (dres) bulk_load(dst + xb + yb, dres + at * (F32 ? 32 : 16), xb, &full[s]);
  };
  if (tid == 0)
    for (int s = 0; s < stages; ++s) {
      const int64_t r = own.row0 + static_cast<int64_t>(s) * own.step;
      if (r < rows) fetch(s, r);
    }
  int s = 0, flip = 0;
  uint32_t ph = 0;
  const int64_t step = own.step;
  int64_t r = own.row0;
  for (; r < rows; r += R * step, flip ^= 1) {
    Vec8<F32> xv[R][V], res[R][V];
    Vec8<false> ev[R][V];
    float mu[R], rs[R], sum[2 * R];   // of g dy and of g dy x^, row by row
    int freed[R];
#pragma unroll
    for (int h = 0; h < R; ++h) {
      const int64_t at = min(r + h * step, rows - 1);
      mu[h] = __ldg(mean + at);
      rs[h] = __ldg(rstd + at);
    }
#pragma unroll
    for (int h = 0; h < R; ++h) {
      const bool have = h == 0 || r + h * step < rows;
      const uint8_t* row = ring + static_cast<size_t>(s) * sb;
      sum[2 * h] = sum[2 * h + 1] = 0.0f;
      if (have) {
        wait_row<C>(&full[s], ph, &stop[flip], wait);
#pragma unroll
        for (int i = 0; i < V; ++i) {
          const int c = tid + i * T;
          if (c < n8) {
            xv[h][i] = smem_vec8<F32>(row, c);
            ev[h][i] = smem_vec8<false>(row + xb, c);
            if (dres) res[h][i] = smem_vec8<F32>(row + xb + yb, c);
            else res[h][i].zero();
#pragma unroll
            for (int j = 0; j < 8; ++j) {
              const float e = ev[h][i].get(j), xh = (xv[h][i].get(j) - mu[h]) * rs[h], ge = g[i][j] * e;
              sum[2 * h] += ge;
              sum[2 * h + 1] = fmaf(ge, xh, sum[2 * h + 1]);
              dg[i][j] = fmaf(e, xh, dg[i][j]);
              db[i][j] += e;
            }
          }
        }
      }
      freed[h] = s;
      if (++s == stages) {
        s = 0;
        ph ^= 1u;
      }
    }
    block_sums<T, 2 * R, C>(sum, s_red[flip]);
    const bool halt = stopped(&stop[flip]);
    // every thread has read the buffers
    if (tid == 0 && !halt)
#pragma unroll
      for (int h = 0; h < R; ++h) {
        const int64_t next = r + (h + stages) * step;
        if (next < rows) fetch(freed[h], next);
      }
#pragma unroll
    for (int h = 0; h < R; ++h) {
      const int64_t row = r + h * step;
      if (h > 0 && row >= rows) break;
      const float m1 = sum[2 * h] * inv_d, m2 = sum[2 * h + 1] * inv_d;
#pragma unroll
      for (int i = 0; i < V; ++i) {
        const int c = tid + i * T;
        if (c < n8) {
          float o[8];
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            const float xh = (xv[h][i].get(j) - mu[h]) * rs[h];
            o[j] = fmaf(rs[h], g[i][j] * ev[h][i].get(j) - m1 - xh * m2, res[h][i].get(j));
          }
          Vec8<F32>::store(dx, row * d8 + own.first + c, o);
        }
      }
    }
    if (halt) break;
  }
  if (r < rows) {
    give_up<F32>(full, stages, r, own.row0, step, rows, d8, own.first, n8, dx, nullptr, nullptr, wait.limit_ns);
#pragma unroll
    for (int i = 0; i < V; ++i)
#pragma unroll
      for (int j = 0; j < 8; ++j) dg[i][j] = db[i][j] = not_a_number();
  }
  float* p = part + (own.row0 * 2 * d8 + own.first) * 8;
#pragma unroll
  for (int i = 0; i < V; ++i) {
    const int c = tid + i * T;
    if (c < n8) {
      Vec8<true>::store(p, c, dg[i]);
      Vec8<true>::store(p + 8 * d8, c, db[i]);
    }
  }
}

// Blocks of the backward, each of which leaves one partial sum of dgamma and
// dbeta: two per SM.
constexpr int kNormBlocks = 304;

template <bool F32, int V>
__global__ void __launch_bounds__(kRowWarps * 32) layernorm_bwd_kernel(
    int64_t rows, int d8, const uint4* __restrict__ dy, const void* __restrict__ x, const float* __restrict__ gamma,
    const float* __restrict__ mean, const float* __restrict__ rstd, const void* __restrict__ dres,
    void* __restrict__ dx, float* __restrict__ part) {
  __shared__ float s_part[kRowWarps][V * 256];
  pdl_trigger();
  pdl_wait();
  const int lane = threadIdx.x & 31, w = threadIdx.x / 32;
  const float inv_d = 1.0f / static_cast<float>(d8 * 8);
  float dg[V][8], db[V][8];
#pragma unroll
  for (int i = 0; i < V; ++i)
#pragma unroll
    for (int j = 0; j < 8; ++j) dg[i][j] = db[i][j] = 0.0f;
  for (int64_t r = static_cast<int64_t>(blockIdx.x) * kRowWarps + w; r < rows;
       r += static_cast<int64_t>(gridDim.x) * kRowWarps) {
    Vec8<F32> xv[V];
    Vec8<false> dv[V];
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int c = lane + i * 32;
      if (c < d8) {
        xv[i].load(x, r * d8 + c);
        dv[i].load(dy, r * d8 + c);
      } else {
        xv[i].zero();
        dv[i].zero();
      }
    }
    const float mu = __ldg(mean + r), rs = __ldg(rstd + r);
    float2 sum = make_float2(0.0f, 0.0f);
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int c = lane + i * 32;
      if (c < d8) {
        Vec8<true> g;
        g.load(gamma, c);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const float xh = (xv[i].get(j) - mu) * rs, e = dv[i].get(j);
          const float ge = g.get(j) * e;
          sum.x += ge;
          sum.y = fmaf(ge, xh, sum.y);
          dg[i][j] = fmaf(e, xh, dg[i][j]);
          db[i][j] += e;
        }
      }
    }
    const float m1 = warp_sum(sum.x) * inv_d, m2 = warp_sum(sum.y) * inv_d;
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int c = lane + i * 32;
      if (c < d8) {
        Vec8<true> g;
        g.load(gamma, c);
        Vec8<F32> res;
        if (dres) res.load(dres, r * d8 + c);
        else res.zero();
        float o[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const float xh = (xv[i].get(j) - mu) * rs;
          o[j] = fmaf(rs, g.get(j) * dv[i].get(j) - m1 - xh * m2, res.get(j));
        }
        Vec8<F32>::store(dx, r * d8 + c, o);
      }
    }
  }
  // this block's partial sums [2][d]; rows of a block are added in order
  const int d = d8 * 8;
  float* p = part + static_cast<int64_t>(blockIdx.x) * 2 * d;
#pragma unroll
  for (int which = 0; which < 2; ++which) {
    __syncthreads();
#pragma unroll
    for (int i = 0; i < V; ++i)
#pragma unroll
      for (int j = 0; j < 8; ++j) s_part[w][(lane + i * 32) * 8 + j] = which ? db[i][j] : dg[i][j];
    __syncthreads();
    for (int c = threadIdx.x; c < d; c += kRowWarps * 32) {
      float t = 0.0f;
#pragma unroll
      for (int k = 0; k < kRowWarps; ++k) t += s_part[k][c];
      p[which * d + c] = t;
    }
  }
}

// dgamma, dbeta = the blocks' partial sums [blocks][2][d] added: 32 columns a
// block, 32 threads a column (a handful of loads in a row each), joined in order.
__global__ void __launch_bounds__(1024) layernorm_reduce_kernel(int blocks, int d, const float* __restrict__ part,
                                                                float* __restrict__ dgamma,
                                                                float* __restrict__ dbeta) {
  __shared__ float s[32][33];
  pdl_trigger();
  pdl_wait();
  const int lane = threadIdx.x & 31, k = threadIdx.x >> 5;
  const int c = blockIdx.x * 32 + lane;
  float t = 0.0f;
  if (c < 2 * d) {
#pragma unroll 4
    for (int b = k; b < blocks; b += 32) t += __ldg(part + static_cast<int64_t>(b) * 2 * d + c);
  }
  s[k][lane] = t;
  __syncthreads();
  // warp k adds column k of the 32 by a shuffle tree
  t = s[lane][k];
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) t += __shfl_xor_sync(0xffffffffu, t, o);
  const int ck = blockIdx.x * 32 + k;
  if (lane == 0 && ck < 2 * d) {
    if (ck < d) dgamma[ck] = t;
    else if (dbeta) dbeta[ck - d] = t;
  }
}

// Four random words of counter `ctr`: Philox-4x32 with ten rounds (J. Salmon,
// M. Moraes, R. Dror, D. Shaw, "Parallel random numbers: as easy as 1, 2, 3",
// 2011): each round multiplies two words by constants and mixes the high
// halves with the others and the key, which steps by constants of its own.
__device__ __forceinline__ uint4 random_words(uint64_t key, uint64_t ctr) {
  uint32_t k0 = static_cast<uint32_t>(key), k1 = static_cast<uint32_t>(key >> 32);
  uint4 c = make_uint4(static_cast<uint32_t>(ctr), static_cast<uint32_t>(ctr >> 32), 0u, 0u);
#pragma unroll
  for (int i = 0; i < 10; ++i) {
    const uint64_t a = static_cast<uint64_t>(c.x) * 0xD2511F53u;
    const uint64_t b = static_cast<uint64_t>(c.z) * 0xCD9E8D57u;
    c = make_uint4(static_cast<uint32_t>(b >> 32) ^ c.y ^ k0, static_cast<uint32_t>(b),
                   static_cast<uint32_t>(a >> 32) ^ c.w ^ k1, static_cast<uint32_t>(a));
    k0 += 0x9E3779B9u;
    k1 += 0xBB67AE85u;
  }
  return c;
}
// Whether elements 8 i .. 8 i + 7 are kept, one bit each.
__device__ __forceinline__ uint32_t keep8(uint64_t key, uint64_t first, int64_t i, uint32_t threshold) {
  const uint4 a = random_words(key, first + 2 * static_cast<uint64_t>(i));
  const uint4 b = random_words(key, first + 2 * static_cast<uint64_t>(i) + 1);
  return (a.x >= threshold ? 1u : 0u) | (a.y >= threshold ? 2u : 0u) | (a.z >= threshold ? 4u : 0u) |
         (a.w >= threshold ? 8u : 0u) | (b.x >= threshold ? 16u : 0u) | (b.y >= threshold ? 32u : 0u) |
         (b.z >= threshold ? 64u : 0u) | (b.w >= threshold ? 128u : 0u);
}

// A thread takes eight columns of a token: KB copies' loads in flight.  Bound by
// the copies' rows: 4096 x 7168 with K = 8 and a shared expert 105 us, 99 without
// random words, 95 at the rate of a plain copy (646 MB); eight loads in flight 126.
template <bool F32, int KB>
__global__ void __launch_bounds__(256) combine_dropout_kernel(
    int64_t items, int d8, int K, const uint4* __restrict__ y_perm, const int32_t* __restrict__ row_of_copy,
    const float* __restrict__ topk_w, const uint4* __restrict__ y_shared, const void* __restrict__ resid,
    const int64_t* __restrict__ rng, uint32_t threshold, float scale, void* __restrict__ out) {
  pdl_trigger();
  pdl_wait();
  uint64_t key = 0, first = 0;
  if (threshold) {
    key = static_cast<uint64_t>(__ldg(rng));
    first = static_cast<uint64_t>(__ldg(rng + 1));
  }
  for (int64_t it = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x; it < items;
       it += static_cast<int64_t>(gridDim.x) * 256) {
    const int64_t t = it / d8;
    const int c = static_cast<int>(it - t * d8);
    float acc[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
    Vec8<F32> res;
    if (resid) res.load(resid, it);
    else res.zero();
    Vec8<false> sh;
    if (y_shared) sh.load(y_shared, it);
    else sh.zero();
    for (int k0 = 0; k0 < K; k0 += KB) {
      Vec8<false> v[KB];
      float w[KB];
#pragma unroll
      for (int j = 0; j < KB; ++j) {
        const int64_t r = k0 + j < K ? __ldg(row_of_copy + t * K + k0 + j) : -1;   // -1: a dropped copy
        w[j] = r >= 0 ? __ldg(topk_w + t * K + k0 + j) : 0.0f;
        if (r >= 0) v[j].load(y_perm, r * d8 + c);
        else v[j].zero();
      }
#pragma unroll
      for (int j = 0; j < KB; ++j)
#pragma unroll
        for (int e = 0; e < 8; ++e) acc[e] = fmaf(w[j], v[j].get(e), acc[e]);
    }
    const uint32_t keep = threshold ? keep8(key, first, it, threshold) : 0xFFu;
    float o[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const float m = acc[e] + sh.get(e);
      o[e] = (keep >> e) & 1u ? fmaf(scale, m, res.get(e)) : res.get(e);
    }
    Vec8<F32>::store(out, it, o);
  }
}

// Bound by the random words: 4096 x 7168 bf16 35 us, 23 without them (117 MB, 17
// at the rate of a plain copy).  A word an element is what lets the mask be drawn
// from the position alone.
template <bool F32>
__global__ void __launch_bounds__(256) dropout_bwd_kernel(int64_t items, const void* __restrict__ dout,
                                                          const int64_t* __restrict__ rng, uint32_t threshold,
                                                          float scale, void* __restrict__ dy) {
  pdl_trigger();
  pdl_wait();
  uint64_t key = 0, first = 0;
  if (threshold) {
    key = static_cast<uint64_t>(__ldg(rng));
    first = static_cast<uint64_t>(__ldg(rng + 1));
  }
  // the loads of a turn's items are in flight together, under the random words of the last
  const int64_t stride = static_cast<int64_t>(gridDim.x) * 256;
  for (int64_t it = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x; it < items; it += 2 * stride) {
    Vec8<F32> v[2];
    const bool two = it + stride < items;
    v[0].load(dout, it);
    if (two) v[1].load(dout, it + stride);
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      if (h && !two) break;
      const int64_t i = it + h * stride;
      const uint32_t keep = threshold ? keep8(key, first, i, threshold) : 0xFFu;
      float o[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) o[e] = (keep >> e) & 1u ? scale * v[h].get(e) : 0.0f;
      Vec8<false>::store(dy, i, o);
    }
  }
}

// Row buffers of a ring kernel with `blocks` blocks an SM and buffers of
// `bytes`, at most 8 and no more than there are rows for; 0: rows too wide.
int ring_stages(int64_t bytes, int blocks) {
  const int64_t n = std::min<int64_t>(8, kRingBytes / blocks / bytes);
  return n < 2 ? 0 : static_cast<int>(n);
}
// Launches K on `clusters` clusters of C blocks.
template <auto K, int C, class... A>
cudaError_t launch_ring(int64_t clusters, unsigned block, size_t smem, cudaStream_t st, A... args) {
  // a ring's dynamic shared memory, allowed once a kernel
  static const cudaError_t e = cudaFuncSetAttribute(K, cudaFuncAttributeMaxDynamicSharedMemorySize, kRingBytes);
  return e != cudaSuccess ? e : launch_pdl<C>(K, static_cast<unsigned>(clusters * C), block, smem, st, args...);
}
// How many clusters of C blocks of K run at once, with `blocks` an SM.
template <auto K, int C>
int resident(int block, int blocks) {
  if (C == 1) return num_sms() * blocks;
  static const int n = [&] {
    cudaLaunchConfig_t cfg{};
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeClusterDimension;
    at[0].val.clusterDim = {C, 1, 1};
    cfg.gridDim = dim3(C * num_sms());
    cfg.blockDim = dim3(block);
    cfg.dynamicSmemBytes = kRingBytes / blocks;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    int clusters = 0;
    if (cudaFuncSetAttribute(K, cudaFuncAttributeMaxDynamicSharedMemorySize, kRingBytes) != cudaSuccess ||
        cudaOccupancyMaxActiveClusters(&clusters, K, &cfg) != cudaSuccess || clusters < 1) {
      cudaGetLastError();
      return 1;
    }
    return clusters;
  }();
  return n;
}
template <bool F32, int T, int V, int C>
constexpr auto forward_kernel() {
  if constexpr (C > 1) return layernorm_cluster_kernel<F32, T, V, F32 ? 2 : 4, C>;
  else return layernorm_ring_kernel<F32, T, V>;
}
// Calls f(threads, vectors, blocks) with the ring kernels' shape of a row of more than
// 1024 elements: a cluster of 2 or 4 blocks shares a row of more than 8192 or 16384.
template <class F>
cudaError_t with_ring_shape(int d, F&& f) {
  using std::integral_constant;
  if (d <= 2048) return f(integral_constant<int, 256>(), integral_constant<int, 1>(), integral_constant<int, 1>());
  if (d <= 4096) return f(integral_constant<int, 256>(), integral_constant<int, 2>(), integral_constant<int, 1>());
  if (d <= 8192) return f(integral_constant<int, 512>(), integral_constant<int, 2>(), integral_constant<int, 1>());
  if (d <= 16384) return f(integral_constant<int, 512>(), integral_constant<int, 2>(), integral_constant<int, 2>());
  return f(integral_constant<int, 512>(), integral_constant<int, 2>(), integral_constant<int, 4>());
}

// Calls f(vectors) with the warp kernels' shape of a row of at most 1024 elements.
template <class F>
cudaError_t with_row_shape(int d, F&& f) {
  switch ((d / 8 + 31) / 32) {
    case 1: return f(std::integral_constant<int, 1>());
    case 2: return f(std::integral_constant<int, 2>());
    case 3: return f(std::integral_constant<int, 3>());
    default: return f(std::integral_constant<int, 4>());
  }
}

}  // namespace

cudaError_t launch_layernorm(int64_t rows, int d, const void* x, bool x_f32, const float* gamma, const float* beta,
                             float eps, void* y, float* mean, float* rstd, cudaStream_t st, const RowWait& wait) {
  if (rows <= 0) return cudaSuccess;
  if (d <= 0 || d % 8 || d > kNormMaxCols) return cudaErrorInvalidValue;
  if (d > 1024)
    return with_ring_shape(d, [&](auto t, auto v, auto c) {
      constexpr int T = decltype(t)::value, V = decltype(v)::value, C = decltype(c)::value;
      constexpr int per_sm = C > 1 ? 1 : 1024 / T;
      const int64_t bytes = static_cast<int64_t>((d / 8 + C - 1) / C) * (x_f32 ? 32 : 16);
      const int stages = ring_stages(bytes, per_sm);
      const auto* px = static_cast<const uint8_t*>(x);
      auto run = [&](auto f32) {
        constexpr bool F = decltype(f32)::value;
        constexpr auto K = forward_kernel<F, T, V, C>();
        return launch_ring<K, C>(std::min<int64_t>(rows, resident<K, C>(T, per_sm)), T, stages * bytes, st, rows, d / 8,
                                 stages, px, gamma, beta, eps, y, mean, rstd, wait);
      };
      return x_f32 ? run(std::true_type()) : run(std::false_type());
    });
  return with_row_shape(d, [&](auto v) {
    constexpr int V = decltype(v)::value;
    const int grid = static_cast<int>(std::min<int64_t>((rows + kRowWarps - 1) / kRowWarps, 1 << 20));
    const auto kern = x_f32 ? layernorm_kernel<true, V> : layernorm_kernel<false, V>;
    return launch_pdl(kern, grid, kRowWarps * 32, 0, st, rows, d / 8, x, gamma, beta, eps, y, mean, rstd);
  });
}

size_t layernorm_bwd_floats(int64_t rows, int d) {
  return static_cast<size_t>(std::min<int64_t>(std::max<int64_t>(rows, 1), kNormBlocks)) * 2 * d;
}

cudaError_t launch_layernorm_bwd(int64_t rows, int d, const void* dy, const void* x, bool x_f32, const float* gamma,
                                 const float* mean, const float* rstd, const void* dres, void* dx, float* dgamma,
                                 float* dbeta, float* scratch, cudaStream_t st, const RowWait& wait) {
  if (d <= 0 || d % 8 || d > kNormMaxCols) return cudaErrorInvalidValue;
  int grid = 0;
  if (rows > 0 && d > 1024) {
    const cudaError_t e = with_ring_shape(d, [&](auto t, auto v, auto c) {
      constexpr int T = decltype(t)::value, V = decltype(v)::value, C = decltype(c)::value;
      constexpr int per_sm = 512 / T;
      const int64_t bytes = static_cast<int64_t>((d / 8 + C - 1) / C) * 8 * ((x_f32 ? 4 : 2) * (dres ? 2 : 1) + 2);
      const int stages = ring_stages(bytes, per_sm);
      auto run = [&](auto f32) {
        constexpr auto K = layernorm_bwd_ring_kernel<decltype(f32)::value, T, V, decltype(f32)::value ? 1 : 2, C>;
        grid = static_cast<int>(std::min<int64_t>({rows, kNormBlocks, resident<K, C>(T, per_sm)}));
        return launch_ring<K, C>(grid, T, stages * bytes, st, rows, d / 8, stages, static_cast<const uint8_t*>(dy),
                                 static_cast<const uint8_t*>(x), gamma, mean, rstd, static_cast<const uint8_t*>(dres),
                                 dx, scratch, wait);
      };
      return x_f32 ? run(std::true_type()) : run(std::false_type());
    });
    if (e != cudaSuccess) return e;
  } else if (rows > 0) {
    const cudaError_t e = with_row_shape(d, [&](auto v) {
      constexpr int V = decltype(v)::value;
      grid = static_cast<int>(std::min<int64_t>((rows + kRowWarps - 1) / kRowWarps, kNormBlocks));
      const auto kern = x_f32 ? layernorm_bwd_kernel<true, V> : layernorm_bwd_kernel<false, V>;
      return launch_pdl(kern, grid, kRowWarps * 32, 0, st, rows, d / 8, static_cast<const uint4*>(dy), x, gamma, mean,
                        rstd, dres, dx, scratch);
    });
    if (e != cudaSuccess) return e;
  }
  return launch_pdl(layernorm_reduce_kernel, (2 * d + 31) / 32, 1024, 0, st, grid, d, scratch, dgamma, dbeta);
}

cudaError_t launch_combine_dropout(int n_tok, int d, int top_k, const void* y_perm, const int32_t* row_of_copy,
                                   const float* topk_w, const void* y_shared, const void* resid, bool f32,
                                   const int64_t* rng, uint32_t threshold, float scale, void* out, cudaStream_t st) {
  const int64_t items = static_cast<int64_t>(n_tok) * (d / 8);
  if (items <= 0) return cudaSuccess;
  // eight blocks an SM, each thread several items: 105 us at 4096 x 7168, K = 8, a block per 256 items 117
  const int grid = static_cast<int>(std::min<int64_t>((items + 255) / 256, static_cast<int64_t>(num_sms()) * 8));
  auto run = [&](auto kern) {
    return launch_pdl(kern, grid, 256, 0, st, items, d / 8, top_k, static_cast<const uint4*>(y_perm), row_of_copy,
                      topk_w, static_cast<const uint4*>(y_shared), resid, rng, threshold, scale, out);
  };
  if (top_k <= 1) return f32 ? run(combine_dropout_kernel<true, 1>) : run(combine_dropout_kernel<false, 1>);
  if (top_k <= 2) return f32 ? run(combine_dropout_kernel<true, 2>) : run(combine_dropout_kernel<false, 2>);
  return f32 ? run(combine_dropout_kernel<true, 4>) : run(combine_dropout_kernel<false, 4>);
}

cudaError_t launch_dropout_bwd(int64_t n, const void* dout, bool f32, const int64_t* rng, uint32_t threshold,
                               float scale, void* dy, cudaStream_t st) {
  const int64_t items = n / 8;
  if (items <= 0) return cudaSuccess;
  const int grid = static_cast<int>(std::min<int64_t>((items + 255) / 256, static_cast<int64_t>(num_sms()) * 8));
  return launch_pdl(f32 ? dropout_bwd_kernel<true> : dropout_bwd_kernel<false>, grid, 256, 0, st, items, dout, rng,
                    threshold, scale, dy);
}

}  // namespace moe
