// FP8 row quantisers and the grouped GEMM on E4M3 codes with one fp32 scale
// per 1 x 128 block of A and per 128 x 128 tile of B.
//
// The scales are arbitrary fp32 numbers, so the tensor cores cannot apply
// them: each k-block of 128 gives an unscaled fp32 partial product in tensor
// memory (four K = 32 MMAs, kind::f8f6f4), and the epilogue warps add
// a_scale * b_scale times it to fp32 accumulators they keep in registers.
// The partial products take turns in the 512 columns of tensor memory, so the
// MMAs of one k-block run while the previous one is being added.
#include "fp8_block.cuh"
#include "grouped_gemm.cuh"
#include "pdl.cuh"
#include "sm100_ptx.cuh"

#include <cuda_bf16.h>
#include <cuda_fp8.h>

#include <algorithm>
#include <mutex>

namespace moe {
namespace {

// ------------------------------------------------------------ quantisation
// A float whose E4M3 rounding is that of the exact quotient x / s.  |x| * inv
// (inv = 1 / s rounded) is within 2 ulp of the quotient, which is enough to find
// the border b between the two codes around it: low 20 mantissa bits 0x80000, or,
// below 2^-6 where the codes are subnormal and as far apart as in [2^-6, 2^-5),
// the same after adding 2^-6 (truncated: a sum rounded up to 2^-5 would give a border of
// the next binade).  The sign of |x| - b s, exact in one FMA, says on
// which side of b the quotient lies: quotients of bf16 numbers do fall on borders,
// where a rounded one would round a second time.  All in fp32: with 64-bit
// divisions near the borders 8192 x 4096 took 125 us instead of 30.
__device__ __forceinline__ float fp8_quotient(float x, float s, float inv) {
  const float q = fabsf(x) * inv;
  const float up = q < 0.015625f ? 0.015625f : 0.0f;
  const float b = __uint_as_float((__float_as_uint(__fadd_rz(q, up)) & 0xFFF00000u) | 0x80000u) - up;
  const float r = fmaf(-b, s, fabsf(x));
  const uint32_t u = __float_as_uint(b) + (r > 0.0f ? 1u : 0u) - (r < 0.0f ? 1u : 0u);
  return __uint_as_float(u | (__float_as_uint(x) & 0x80000000u));
}

__device__ __forceinline__ uint32_t fp8_pack4(float a, float b, float c, float d) {
  const uint32_t lo = __nv_cvt_float2_to_fp8x2(make_float2(a, b), __NV_SATFINITE, __NV_E4M3);
  const uint32_t hi = __nv_cvt_float2_to_fp8x2(make_float2(c, d), __NV_SATFINITE, __NV_E4M3);
  return lo | (hi << 16);
}

// s: the block's scale.  d, inv: divisor and its reciprocal for values times f
// (2^64 where the scale is so small that products with it would lose bits).
struct BlockScale {
  float s, d, inv, f;
};
__device__ __forceinline__ BlockScale block_scale(float amax) {
  BlockScale b;
  const float s = amax * (1.0f / 448.0f);
  b.s = s > 0.0f ? s : 1.0f;
  b.f = b.s < 5.421010862427522e-20f ? 18446744073709551616.0f : 1.0f;   // 2^-64, 2^64
  b.d = b.s * b.f;
  b.inv = 1.0f / b.d;
  return b;
}
__device__ __forceinline__ uint32_t fp8_encode4(float a, float b, float c, float d, const BlockScale& k) {
  return fp8_pack4(fp8_quotient(a * k.f, k.d, k.inv), fp8_quotient(b * k.f, k.d, k.inv),
                   fp8_quotient(c * k.f, k.d, k.inv), fp8_quotient(d * k.f, k.d, k.inv));
}

__device__ __forceinline__ float lo16(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float hi16(uint32_t w) { return __uint_as_float(w & 0xFFFF0000u); }
__device__ __forceinline__ uint32_t bf2(float a, float b) {
  __nv_bfloat162 v = __floats2bfloat162_rn(a, b);
  return *reinterpret_cast<uint32_t*>(&v);
}

// Sixteen elements of a 128-element block per lane, eight lanes a block: the
// block's scale and this lane's sixteen codes.
__device__ __forceinline__ uint4 quant16(const uint4 v0, const uint4 v1, float& scale) {
  const uint32_t w[8] = {v0.x, v0.y, v0.z, v0.w, v1.x, v1.y, v1.z, v1.w};
  float m = 0.0f;
#pragma unroll
  for (int i = 0; i < 8; ++i) m = fmaxf(m, fmaxf(fabsf(lo16(w[i])), fabsf(hi16(w[i]))));
#pragma unroll
  for (int o = 1; o < 8; o <<= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
  const BlockScale b = block_scale(m);
  scale = b.s;
  uint32_t c[4];
#pragma unroll
  for (int i = 0; i < 4; ++i)
    c[i] = fp8_encode4(lo16(w[2 * i]), hi16(w[2 * i]), lo16(w[2 * i + 1]), hi16(w[2 * i + 1]), b);
  return make_uint4(c[0], c[1], c[2], c[3]);
}

// A warp takes four blocks of a row at a time.
__global__ void __launch_bounds__(256) fp8_quant_rows_kernel(const uint4* __restrict__ src, int64_t rows, int c16,
                                                             uint4* __restrict__ codes, float* __restrict__ scales,
                                                             int64_t ld) {
  pdl_trigger();
  pdl_wait();
  const int lane = threadIdx.x & 31;
  const int segs = (c16 + 31) / 32;
  const int64_t items = rows * segs;
  const int64_t stride = static_cast<int64_t>(gridDim.x) * 8;
  for (int64_t it = static_cast<int64_t>(blockIdx.x) * 8 + (threadIdx.x >> 5); it < items; it += stride) {
    const int64_t r = it / segs;
    const int c = static_cast<int>(it - r * segs) * 32 + lane;
    uint4 v0 = make_uint4(0, 0, 0, 0), v1 = v0;
    if (c < c16) {
      v0 = __ldg(src + (r * c16 + c) * 2);
      v1 = __ldg(src + (r * c16 + c) * 2 + 1);
    }
    float s;
    const uint4 q = quant16(v0, v1, s);
    if (c < c16) {
      codes[r * c16 + c] = q;
      if ((lane & 7) == 0) scales[r * ld + (c >> 3)] = s;
    }
  }
}

__global__ void __launch_bounds__(256) fp8_quant_scatter_kernel(const uint4* __restrict__ x, int n_tok, int c16,
                                                                int top_k, const int32_t* __restrict__ row_of_copy,
                                                                uint4* __restrict__ codes, float* __restrict__ scales,
                                                                int64_t ld, uint4* __restrict__ tok_codes,
                                                                float* __restrict__ tok_scales) {
  pdl_trigger();
  pdl_wait();
  const int lane = threadIdx.x & 31;
  const int segs = (c16 + 31) / 32;
  const int64_t items = static_cast<int64_t>(n_tok) * segs;
  const int64_t stride = static_cast<int64_t>(gridDim.x) * 8;
  for (int64_t it = static_cast<int64_t>(blockIdx.x) * 8 + (threadIdx.x >> 5); it < items; it += stride) {
    const int64_t t = it / segs;
    const int c = static_cast<int>(it - t * segs) * 32 + lane;
    const int my_row = lane < top_k ? __ldg(row_of_copy + t * top_k + lane) : -1;
    uint4 v0 = make_uint4(0, 0, 0, 0), v1 = v0;
    if (c < c16) {
      v0 = __ldg(x + (t * c16 + c) * 2);
      v1 = __ldg(x + (t * c16 + c) * 2 + 1);
    }
    float s;
    const uint4 q = quant16(v0, v1, s);
    for (int k = 0; k < top_k; ++k) {
      const int64_t r = __shfl_sync(0xffffffffu, my_row, k);
      if (r >= 0 && c < c16) {
        codes[r * c16 + c] = q;
        if ((lane & 7) == 0) scales[r * ld + (c >> 3)] = s;
      }
    }
    if (tok_codes && c < c16) {
      tok_codes[t * c16 + c] = q;
      if ((lane & 7) == 0) tok_scales[t * ld + (c >> 3)] = s;
    }
  }
}

// -------------------------------------------------------------------- GEMM
// Roles (384 threads, one CTA per SM): warp 0 TMA producer, warp 1 MMA issuer,
// warps 2-3 scale products, warps 4-11 epilogue (warp w reads tensor-memory
// lanes 32 (w % 4) .. + 31 and half of the columns: 128 accumulators a thread).
// Tiles of 128 rows x BN columns per CTA, 512 / BN partial products in tensor
// memory.
//
// What bounds it: a k-block's operands are written to shared memory once and
// read once by the MMAs (96 KB, about 750 clocks), and the chain from one k-block
// to the next (the MMAs' completion seen through a barrier, 128 tensor-memory
// words added by each epilogue thread, the buffer's release seen by the MMA
// warp) takes about 850.  8192 rows x 4096 columns x 14336: 357 us (2.70 PFLOP/s).
// Measured against it on that shape: 16 epilogue warps of 64 columns 413; the
// two-product multiply-add 448; tensor-memory loads of 32 columns 438, of the next
// 16 columns ahead of the multiply-adds 400; 128-column tiles with four
// partial products 622, since the issue of a k-block (four MMAs, two commits,
// two waits) takes 400 clocks whatever its size; CTA pairs sharing 256 x 256
// tiles 352, and no faster than this within an expert layer (1.42 ms both).
//
// GEMM1 (SwiGLU): a tile holds 128 columns of w1 and the same 128 of w3, which
// is one scale block of h.
//
// Few tiles: one CTA takes about 0.35 us a k-block of a long contraction while other SMs
// idle.  Where 2, 4 or 8 CTAs a tile still all run at once and have eight k-blocks
// each, a cluster shares the tile; the CTAs leave their sums in shared memory and add each
// other's, row by row, in the order of the k-blocks.  8 rows of 2048 x 7168: 11.1 us
// (one CTA a tile 20.5), a row of 7168 x 7168 15.1 (21.1), two groups of one row of
// 4096 x 14336 25.8 (36.8); a token through one expert of 7168 x 2048, whole layer, 35.9 (50.7).
constexpr int BM = 128;
constexpr int BK = 128;              // contraction elements (bytes) of a k-block
constexpr int kAuxThreads = 128;
constexpr int kEpiWarps = 8;
constexpr int kThreads = kAuxThreads + kEpiWarps * 32;
constexpr int kMaxGroups = 1024;
constexpr int kABytes = BM * BK;     // A of a stage
// A block launches with 384 x 168 = 64512 registers; the split hands 96 of them a
// thread from the first warpgroup to the two that accumulate: 128 x 72 + 256 x 216 = 64512.
constexpr int kAuxRegs = 72, kEpiRegs = 216;

__host__ __device__ constexpr uint32_t idesc_e4m3_f32(int m, int n, bool b_mn) {
  // D format fp32 (bits 4-5 = 1), A and B E4M3 (7-9, 10-12 = 0), B major (16), N >> 3 (17-22), M >> 4 (24-28)
  return (1u << 4) | ((b_mn ? 1u : 0u) << 16) | (static_cast<uint32_t>(n >> 3) << 17) |
         (static_cast<uint32_t>(m >> 4) << 24);
}
__device__ __forceinline__ void tc_mma_e4m3(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc, uint32_t idesc,
                                            uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
      "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate)
      : "memory");
}

// acc += s * v.  Volatile, which keeps it behind the wait for the tensor-memory
// load whose register it reads; naming the registers in the wait costs a copy
// of each.  (The instruction for two products runs at half the rate.)
__device__ __forceinline__ void fma_after_wait(float& acc, float s, uint32_t v) {
  asm volatile("fma.rn.f32 %0, %1, %2, %0;" : "+f"(acc) : "f"(s), "f"(__uint_as_float(v)));
}
__device__ __forceinline__ float ld_shared_f32(uint32_t addr) {
  float r;
  asm volatile("ld.shared.f32 %0, [%1];" : "=f"(r) : "r"(addr) : "memory");
  return r;
}
__device__ __forceinline__ void st_shared_f32(uint32_t addr, float x) {
  asm volatile("st.shared.f32 [%0], %1;" ::"r"(addr), "f"(x) : "memory");
}

__device__ __forceinline__ uint32_t cluster_nctarank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_nctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ float4 ld_cluster_f32x4(uint32_t addr) {
  float4 v;
  asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
               : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
               : "r"(addr)
               : "memory");
  return v;
}

// Zero below a1 = -87, where 1 + e^-a1 is past 2^126 and silu smaller than 2^-119.
__device__ __forceinline__ float swiglu(float a1, float a3) { return __fdividef(a1, 1.0f + __expf(-a1)) * a3; }
// What a block of h with the scale s is multiplied by before the scale's reciprocal, which
// is beyond fp32's range for the smallest scales: the reciprocal is that of h_factor(s) * s.
__device__ __forceinline__ float h_factor(float s) {
  return s < 5.421010862427522e-20f ? 18446744073709551616.0f : 1.0f;   // 2^-64, 2^64
}
__device__ __forceinline__ float scale_of_h(float m) {
  const float s = m * (1.0f / 448.0f);
  return s > 0.0f ? s : 1.0f;
}

// One lane of a converged warp.  The compiler knows this form: operands of the
// TMA and tcgen05 instructions behind it go to uniform registers at once, where a
// `lane == 0` branch makes each a loop over the lanes (four MMAs 250 clocks).
__device__ __forceinline__ bool elect_one() {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "elect.sync _|p, 0xFFFFFFFF;\n\t"
      "selp.b32 %0, 1, 0, p;\n\t}"
      : "=r"(r));
  return r != 0;
}

// mbar_wait_bounded for a whole warp, with the same answer in every lane.  The
// abort flag and the limit are looked at now and then: the polls of the
// waiting warps take issue slots from the others.
__device__ __forceinline__ bool warp_wait(uint64_t* bar, uint32_t parity, volatile int* abort_flag, int32_t* status,
                                          int site) {
  if (__all_sync(0xffffffffu, mbar_try_wait(bar, parity))) return true;
  uint64_t t0 = 0;
  uint32_t n = 0;
#pragma unroll 1
  while (true) {
#pragma unroll 1
    for (int i = 0; i < 64; ++i)
      if (__all_sync(0xffffffffu, mbar_try_wait(bar, parity))) return true;
    if (__any_sync(0xffffffffu, *abort_flag)) return false;
    const uint64_t now = __shfl_sync(0xffffffffu, globaltimer_ns(), 0);
    if (n++ == 0) {
      t0 = now;
    } else if (now - t0 > kSpinTimeoutNs) {
      if ((threadIdx.x & 31) == 0) {
        *abort_flag = 1;
        if (status) {
          atomicOr(status, DEV_TIMEOUT);
          atomicExch(status + 1, site);
        }
      }
      return false;
    }
  }
}

// Whether the phase has completed, for a whole warp.
__device__ __forceinline__ bool try_wait_all(uint32_t addr, uint32_t parity) {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t"
      "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
      "vote.sync.all.pred q, p, 0xFFFFFFFF;\n\t"
      "selp.u32 %0, 1, 0, q;\n\t}"
      : "=r"(r)
      : "r"(addr), "r"(parity)
      : "memory");
  return r != 0;
}

struct Fp8Params {
  CUtensorMap tmA[2];
  CUtensorMap tmA32[2];   // boxes of 32 rows
  CUtensorMap tmB[2];
  const float* a_scale[2];
  const float* b_scale[2];
  int64_t a_scale_ld;
  const int32_t* offsets;
  int32_t groups;
  int32_t rows;
  int32_t n;
  int32_t ntiles;      // column tiles of the output
  int32_t n128;        // 128-column tiles of a weight matrix's N
  int32_t kb;          // k-blocks of one source
  int32_t sources;
  void* out0;
  void* out1;
  void* out2;
  void* out3;
  float* hs;
  int64_t hs_ld;
  const void* in0;
  const void* in1;
  int32_t* status;
};

template <int BN>
struct Cfg {
  static constexpr int kBufs = 512 / BN;             // partial products in tensor memory
  static constexpr int kBBytes = BN * BK;
  static constexpr int kStageBytes = kABytes + kBBytes;
  static constexpr int kStages = 196608 / kStageBytes;
  static constexpr int kEpiOff = kStages * kStageBytes;        // 2 KB of output staging a warp
  static constexpr int kMaxOff = kEpiOff + kEpiWarps * 2048;   // row maxima [2][4][128]
  static constexpr int kScaleOff = kMaxOff + 4096;             // scale products [2][4 k-blocks][2][128]
  static constexpr int kBarOff = kScaleOff + 8192;
  static constexpr int kBars = 2 * kStages + 2 * kBufs + 4 + 4 + 1;
  static constexpr int kMiscOff = kBarOff + kBars * 8;
  static constexpr int kTabOff = kMiscOff + 16;
  static constexpr size_t smem_bytes(int groups) { return 1024 + kTabOff + 4 * (groups + 1); }
  static_assert(smem_bytes(kMaxGroups) <= 232448, "shared memory above 227 KB");
};

struct Tile {
  int g, nt, row0, valid;   // valid: rows of the 128
};

// An offset cut to the rows there are, so that no tile reaches outside them.
__device__ __forceinline__ int cut_offset(const Fp8Params& p, int i) {
  return min(max(__ldg(p.offsets + i), 0), p.rows);
}

__device__ __forceinline__ Tile find_tile(int tile, const Fp8Params& p, const int* s_pre) {
  int lo = 0, hi = p.groups;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (s_pre[mid] <= tile) lo = mid; else hi = mid;
  }
  // M tiles innermost: the CTAs that run at once share an expert's weight blocks
  const int first = cut_offset(p, lo), last = cut_offset(p, lo + 1);
  const int mtiles = (last - first + BM - 1) / BM;
  const int rem = tile - s_pre[lo];
  Tile t;
  t.g = lo;
  t.nt = rem / mtiles;
  t.row0 = first + (rem - t.nt * mtiles) * BM;
  t.valid = min(BM, last - t.row0);
  return t;
}

// Sixteen 32-bit words of each lane's row (64 bytes) written to global memory
// as whole 64-byte row segments, through 2 KB of shared memory.
// dst: row 0 of the warp's 32; chunks: 16-byte chunks inside the output's columns.
__device__ __forceinline__ void store_rows64(uint32_t stg, int lane, const uint32_t (&w)[16], uint8_t* dst,
                                             int64_t ld_bytes, int rows, int chunks) {
  __syncwarp();
#pragma unroll
  for (int j = 0; j < 4; ++j)   // chunk j of row l at j ^ ((l >> 1) & 3): eight rows span the banks twice
    st_shared_v4(stg + lane * 64 + ((j ^ ((lane >> 1) & 3)) << 4), w[4 * j], w[4 * j + 1], w[4 * j + 2],
                 w[4 * j + 3]);
  __syncwarp();
  const int c = lane & 3, r0 = lane >> 2;
  uint8_t* p = dst + r0 * ld_bytes + c * 16;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int r = i * 8 + r0;
    uint4 v;
    ld_shared_v4(stg + r * 64 + ((c ^ ((r >> 1) & 3)) << 4), v.x, v.y, v.z, v.w);
    if (r < rows && c < chunks) *reinterpret_cast<uint4*>(p) = v;
    p += 8 * ld_bytes;
  }
}

template <int BN, bool B_MN, int EPI, bool SPLIT>
__global__ void __launch_bounds__(kThreads, 1) fp8_gemm_kernel(const __grid_constant__ Fp8Params p) {
  using C = Cfg<BN>;
  constexpr int S = C::kStages, kBufs = C::kBufs;
  constexpr bool DUAL = EPI == FP8_EPI_SWIGLU_FWD;
  constexpr int NS = BN / 128;        // scale products a row and k-block: 128-column blocks, or w1 and w3
  constexpr int CG = kEpiWarps / 4;   // column groups of the epilogue warps
  constexpr int COLS = BN / CG;       // columns of an epilogue warp
  constexpr int CW = 16;              // columns of a tensor-memory load
  static_assert(!DUAL || BN == 256, "w1 and w3 halves of a 256-column tile");
  static_assert(!SPLIT || EPI == FP8_EPI_SWIGLU_FWD || (EPI == FP8_EPI_BF16 && BN == 128), "forms of partial sums");
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + C::kBarOff);
  uint64_t* empty = full + S;
  uint64_t* tfull = empty + S;
  uint64_t* tempty = tfull + kBufs;
  uint64_t* xbar = tempty + kBufs;    // the warps of a lane quarter exchanging row maxima
  uint64_t* sfull = xbar + 4;         // scale products of four k-blocks written
  uint64_t* sempty = sfull + 2;
  uint64_t* mma_done = sempty + 2;
  uint32_t* s_tmem = reinterpret_cast<uint32_t*>(smem + C::kMiscOff);
  volatile int* s_abort = reinterpret_cast<volatile int*>(smem + C::kMiscOff + 4);
  int* s_pre = reinterpret_cast<int*>(smem + C::kTabOff);
  const uint32_t s_scale = smem_u32(smem + C::kScaleOff);

  const int warp = __shfl_sync(0xffffffffu, static_cast<int>(threadIdx.x) >> 5, 0);
  const int lane = threadIdx.x & 31;
  const int G = p.groups;
  // SPLIT: a cluster has one tile (or none) and each CTA a share of its k-blocks, in fours
  const int ranks = SPLIT ? static_cast<int>(cluster_nctarank()) : 1;
  const int rank = SPLIT ? static_cast<int>(cluster_ctarank()) : 0;
  const int unit0 = blockIdx.x / ranks, ustride = gridDim.x / ranks;
  const int fours = (p.kb + 3) / 4;
  const int kbeg = SPLIT ? fours * rank / ranks * 4 : 0;
  const int kend = SPLIT ? min(p.kb, fours * (rank + 1) / ranks * 4) : p.kb;

  if (threadIdx.x == 0) {
    for (int s = 0; s < S; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
    }
    for (int b = 0; b < kBufs; ++b) {
      mbar_init(&tfull[b], 1);
      mbar_init(&tempty[b], kEpiWarps);
    }
    for (int q = 0; q < 4; ++q) mbar_init(&xbar[q], CG);
    for (int b = 0; b < 2; ++b) {
      mbar_init(&sfull[b], 2);
      mbar_init(&sempty[b], kEpiWarps);
    }
    mbar_init(mma_done, 1);
    *s_abort = 0;
    fence_mbar_init();
    tma_prefetch_desc(&p.tmA[0]);
    tma_prefetch_desc(&p.tmB[0]);
  }
  if (warp == 1) {
    tmem_alloc(s_tmem, 512);
    tmem_relinquish();
  }
  // all of the above needs nothing of the kernels before this one
  pdl_trigger();
  pdl_wait();
  bool descend = false;
  for (int i = threadIdx.x; i <= G; i += kThreads) {
    const int o = cut_offset(p, i);
    const bool less = i < G && cut_offset(p, i + 1) < o;
    descend |= less;
    if ((less || o != __ldg(p.offsets + i)) && p.status) atomicOr(p.status, DEV_BAD_OFFSETS);
  }
  if (warp == 0) {
    auto tiles_of = [&](int g) { return max(0, cut_offset(p, g + 1) - cut_offset(p, g) + BM - 1) / BM * p.ntiles; };
    const int per = (G + 31) / 32;
    const int lo = min(G, lane * per), hi = min(G, lo + per);
    int sum = 0;
    for (int g = lo; g < hi; ++g) sum += tiles_of(g);
    int incl = sum;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const int v = __shfl_up_sync(0xffffffffu, incl, d);
      if (lane >= d) incl += v;
    }
    int run = incl - sum;
    for (int g = lo; g < hi; ++g) {
      s_pre[g] = run;
      run += tiles_of(g);
    }
    if (lane == 31) s_pre[G] = incl;
  }
  tc_fence_before();
  descend = __syncthreads_or(descend);
  tc_fence_after();
  const uint32_t tmem_base = *s_tmem;
  // groups of descending offsets overlap, and two tiles would write the same rows: then none is written
  const int total = descend ? 0 : s_pre[G];
  const int nkb = (kend - kbeg) * p.sources;

  if (warp < kAuxThreads / 32) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kAuxRegs));
    if (warp == 0) {
      // ---------------------------------------------------------- producer
      uint32_t it = 0, s = 0, ph = 1;
      bool ok = true;
      for (int tile = unit0; ok && tile < total; tile += ustride) {
        const Tile t = find_tile(tile, p, s_pre);
        // a tile of at most 32 rows loads no others (47.8 -> 40.4 us for 2 rows of 16 groups
        // of 7168 x 2048): what the rest of its stage holds reaches accumulator rows that
        // nothing reads
        const bool few = t.valid <= 32;
        const uint32_t bytes = few ? C::kStageBytes - kABytes * 3 / 4 : C::kStageBytes;
        for (int src = 0; ok && src < p.sources; ++src) {
          const CUtensorMap* ma = few ? &p.tmA32[src] : &p.tmA[src];
          const CUtensorMap* mb = &p.tmB[src];
          const int n0 = DUAL ? t.nt * 128 : t.nt * BN;
          for (int k0 = kbeg * BK; k0 < kend * BK; k0 += BK, ++it) {
            ok = warp_wait(&empty[s], ph, s_abort, p.status, 800);
            if (!ok) break;
            uint8_t* sA = smem + s * C::kStageBytes;
            uint8_t* sB = sA + kABytes;
            if (elect_one()) {
              mbar_arrive_expect_tx(&full[s], bytes);
              tma_load_2d(sA, ma, &full[s], k0, t.row0);
              if (B_MN) {
                tma_load_3d(sB, mb, &full[s], n0, k0, t.g);
                if (BN == 256) tma_load_3d(sB + 16384, mb, &full[s], n0 + 128, k0, t.g);
              } else {
                tma_load_3d(sB, mb, &full[s], k0, n0, t.g);
                if (DUAL) tma_load_3d(sB + 16384, &p.tmB[1], &full[s], k0, n0, t.g);
              }
            }
            __syncwarp();
            if (++s == S) {
              s = 0;
              ph ^= 1u;
            }
          }
        }
      }
      // no copy and no stage release may still be under way when the CTA exits
      for (uint32_t i = 0; i < S; ++i) {
        if (it > i) {
          const uint32_t uses = (it - 1 - i) / S + 1;   // of stage i
          mbar_wait_drain(&full[i], (uses - 1) & 1u);
          if (ok) mbar_wait_drain(&empty[i], (uses - 1) & 1u);
        }
      }
      __syncwarp();
    } else if (warp == 1) {
      // -------------------------------------------------------- MMA issuer
      constexpr uint32_t idesc = idesc_e4m3_f32(BM, BN, B_MN);
      int64_t left = 0;   // k-blocks of this CTA's tiles
      for (int tile = unit0; tile < total; tile += ustride) left += nkb;
      // K-major: rows of 128 bytes, 32 bytes on per K = 32; MN-major: 128 columns a row of
      // 128 bytes, 32 rows on, the next 128 columns a whole region further
      constexpr uint32_t kAdvB = (B_MN ? 4096 : 32) >> 4;
      const uint64_t ad0 = smem_desc_sw128(smem_u32(smem), 16, 1024);
      const uint64_t bd0 = smem_desc_sw128(smem_u32(smem) + kABytes, B_MN ? 16384 : 16, 1024);
      uint32_t s = 0, ph = 0, buf = 0, bph = 1;
      for (; left > 0; --left) {
        // the operands are there long before the buffer is
        if (!warp_wait(&full[s], ph, s_abort, p.status, 840) || !warp_wait(&tempty[buf], bph, s_abort, p.status, 820))
          break;
        tc_fence_after();
        if (elect_one()) {
          const uint64_t ad = ad0 + s * (C::kStageBytes >> 4), bd = bd0 + s * (C::kStageBytes >> 4);
#pragma unroll
          for (int kk = 0; kk < 4; ++kk)
            tc_mma_e4m3(tmem_base + buf * BN, ad + kk * 2, bd + kk * kAdvB, idesc, kk > 0 ? 1u : 0u);
          tc_commit(&empty[s]);
          tc_commit(&tfull[buf]);
        }
        __syncwarp();
        if (++s == S) {
          s = 0;
          ph ^= 1u;
        }
        if (++buf == kBufs) {
          buf = 0;
          bph ^= 1u;
        }
      }
      // every MMA has completed before tensor memory is released
      if (elect_one()) {
        tc_commit(mma_done);
        mbar_wait_drain(mma_done, 0);
      }
    } else if (warp >= 2) {
      // -------------------------------------------------------- scales
      // The products a_scale[r, k-block] * b_scale[n / 128, k-block] of a tile's
      // rows and its 128-column blocks (or w1 and w3), four k-blocks at a time, up to
      // eight ahead of the epilogue, which then reads one number per row and block.
      const int at = static_cast<int>(threadIdx.x) - 64;    // rows at and at + 64
      const int64_t wtiles = static_cast<int64_t>(p.n128) * p.kb;
      const int64_t bstep = B_MN ? p.n128 : 1;
      float4 a[2];
      float b[NS][4];
      // the factors of k-blocks k4 .. k4 + 3 of a tile
      auto load = [&](const Tile& t, int src, int k4) {
#pragma unroll
        for (int h = 0; h < 2; ++h)
          a[h] = __ldg(reinterpret_cast<const float4*>(
              p.a_scale[src] + static_cast<int64_t>(min(t.row0 + at + 64 * h, p.rows - 1)) * p.a_scale_ld + k4));
#pragma unroll
        for (int j = 0; j < NS; ++j) {
          const int nb = DUAL ? t.nt : min(t.nt * NS + j, p.n128 - 1);
          const float* pb = p.b_scale[DUAL ? j : src] + t.g * wtiles + (B_MN ? nb : static_cast<int64_t>(nb) * p.kb);
#pragma unroll
          for (int u = 0; u < 4; ++u) b[j][u] = __ldg(pb + min(k4 + u, p.kb - 1) * bstep);
        }
      };
      uint32_t gi = 0;
      bool ok = true;
      int tile = unit0, src = 0, k4 = kbeg;
      Tile t{};
      if (tile < total) {
        t = find_tile(tile, p, s_pre);
        load(t, 0, kbeg);
      }
      while (tile < total) {
        float prod[2][NS][4];
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
          for (int j = 0; j < NS; ++j) {
            prod[h][j][0] = a[h].x * b[j][0];
            prod[h][j][1] = a[h].y * b[j][1];
            prod[h][j][2] = a[h].z * b[j][2];
            prod[h][j][3] = a[h].w * b[j][3];
          }
        // the next four's factors are on their way while these are handed over
        k4 += 4;
        if (k4 >= kend) {
          k4 = kbeg;
          if (++src == p.sources) {
            src = 0;
            tile += ustride;
            if (tile < total) t = find_tile(tile, p, s_pre);
          }
        }
        if (tile < total) load(t, src, k4);
        ok = warp_wait(&sempty[gi & 1u], ((gi >> 1) & 1u) ^ 1u, s_abort, p.status, 870);
        if (!ok) break;
        const uint32_t dst = s_scale + ((gi & 1u) * 1024 + at) * 4;
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
          for (int j = 0; j < NS; ++j)
#pragma unroll
            for (int u = 0; u < 4; ++u) st_shared_f32(dst + (u * 256 + j * 128 + h * 64) * 4, prod[h][j][u]);
        __syncwarp();
        if (lane == 0) mbar_arrive(&sfull[gi & 1u]);
        ++gi;
      }
    }
    __syncwarp();
    if constexpr (SPLIT) {
      cluster_sync_all();
      cluster_sync_all();
    }
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kEpiRegs));
    // -------------------------------------------------------------- epilogue
    const int ew = warp - kAuxThreads / 32;
    const int q = warp & 3;           // lane quarter of tensor memory this warp may read
    const int cg = ew >> 2;           // column group
    const uint32_t lane_base = tmem_base + (static_cast<uint32_t>(q * 32) << 16);
    // tile column of this warp's chunk c (w1 | w3: half of the chunks each)
    auto chunk_col = [&](int c) { constexpr int H = COLS / 32;
      return DUAL ? (c / H) * 128 + cg * (COLS / 2) + (c % H) * 16 : cg * COLS + c * 16; };
    const uint32_t stg = smem_u32(smem + C::kEpiOff + ew * 2048);
    float* s_max = reinterpret_cast<float*>(smem + C::kMaxOff);
    const uint32_t tfull_addr = smem_u32(tfull);
    const int r = q * 32 + lane;
    // this warp has read a partial product
    auto release = [&](uint32_t buf) {
      tc_fence_before();
      __syncwarp();
      if (elect_one()) mbar_arrive(&tempty[buf]);
    };
    uint32_t buf = 0, bph = 0, gi = 0, tcount = 0;
    bool ok = true;
    for (int tile = unit0; ok && tile < total; tile += ustride, ++tcount) {
      const Tile t = find_tile(tile, p, s_pre);
      const bool mine = q * 32 < t.valid;   // whether this warp has rows of the tile
      const int rows = t.valid - q * 32;
      const int64_t row = t.row0 + q * 32;
      float acc[COLS];                      // DUAL: half of them a1, the same columns of a3 the rest
#pragma unroll
      for (int i = 0; i < COLS; ++i) acc[i] = 0.0f;
      for (int src = 0; ok && src < p.sources; ++src) {
        for (int k4 = kbeg; ok && k4 < kend; k4 += 4, ++gi) {
          ok = warp_wait(&sfull[gi & 1u], (gi >> 1) & 1u, s_abort, p.status, 880);
          uint32_t ps = s_scale + ((gi & 1u) * 1024 + (DUAL ? 0 : cg * COLS / 128 * 128) + r) * 4;
          const uint32_t pe = ps + min(4, kend - k4) * 1024;
#pragma unroll 1   // four copies of the body miss the instruction cache: 410 us against 358
          for (; ok && ps != pe; ps += 1024) {
            const float sa = ld_shared_f32(ps), sb = DUAL ? ld_shared_f32(ps + 512) : sa;
            if (!try_wait_all(tfull_addr + buf * 8, bph)) {
              ok = warp_wait(&tfull[buf], bph, s_abort, p.status, 860);
              if (!ok) break;
            }
            if (mine) {
              tc_fence_after();
              const uint32_t tb = lane_base + buf * BN;
#pragma unroll
              for (int c = 0; c < COLS / CW; ++c) {
                uint32_t v[CW];
                tmem_ld_32x32b_x16(tb + chunk_col(c), v);
                tmem_wait_ld();
                if (c + 1 == COLS / CW) release(buf);
#pragma unroll
                for (int i = 0; i < CW; ++i) fma_after_wait(acc[c * CW + i], DUAL && c >= COLS / CW / 2 ? sb : sa, v[i]);
              }
            } else {
              release(buf);
            }
            if (++buf == kBufs) {
              buf = 0;
              bph ^= 1u;
            }
          }
          __syncwarp();
          if (elect_one()) mbar_arrive(&sempty[gi & 1u]);
        }
      }
      if (!ok) break;

      auto rows_bf16 = [&](const float* f, void* out, int col) {   // 32 columns of the warp's rows
        uint32_t w[16];
#pragma unroll
        for (int j = 0; j < 16; ++j) w[j] = bf2(f[2 * j], f[2 * j + 1]);
        if (mine && col < p.n)
          store_rows64(stg, lane, w, static_cast<uint8_t*>(out) + (row * p.n + col) * 2, static_cast<int64_t>(p.n) * 2,
                       rows, (p.n - col) / 8);
      };
      if constexpr (SPLIT) {
        // this CTA's sums over the operands' stages, which no load and no MMA uses any
        // more; 16-byte chunk c of row r at c ^ (r & 31)
        if (r < t.valid) {
#pragma unroll
          for (int i = 0; i < COLS / 4; ++i) {
            const int c = chunk_col(i / 4) / 4 + i % 4;
            st_shared_v4(smem_u32(smem) + r * (BN * 4) + ((c ^ (r & 31)) << 4), __float_as_uint(acc[4 * i]),
                         __float_as_uint(acc[4 * i + 1]), __float_as_uint(acc[4 * i + 2]),
                         __float_as_uint(acc[4 * i + 3]));
          }
        }
      } else if constexpr (EPI == FP8_EPI_BF16) {
#pragma unroll
        for (int c = 0; c < COLS / 32; ++c) rows_bf16(acc + 32 * c, p.out0, t.nt * BN + cg * COLS + c * 32);
      } else if constexpr (EPI == FP8_EPI_SWIGLU_BWD) {
        // dh -> da1 = dh a3 silu'(a1), da3 = dh silu(a1); n is a multiple of 64
#pragma unroll
        for (int c = 0; c < COLS / 32; ++c) {
          const int col = t.nt * BN + cg * COLS + c * 32;
          if (mine && col < p.n) {
            const int64_t base = static_cast<int64_t>(min(t.row0 + r, p.rows - 1)) * p.n + col;
            float d1[32];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const uint4 x1 = __ldg(reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(p.in0) + base) + i);
              const uint4 x3 = __ldg(reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(p.in1) + base) + i);
              const uint32_t u1[4] = {x1.x, x1.y, x1.z, x1.w}, u3[4] = {x3.x, x3.y, x3.z, x3.w};
#pragma unroll
              for (int e = 0; e < 8; ++e) {
                const float dh = acc[c * 32 + i * 8 + e];
                const float a = (e & 1) ? hi16(u1[e >> 1]) : lo16(u1[e >> 1]);
                const float b = (e & 1) ? hi16(u3[e >> 1]) : lo16(u3[e >> 1]);
                const float sg = 1.0f / (1.0f + __expf(-a));
                d1[i * 8 + e] = dh * b * sg * (1.0f + a * (1.0f - sg));
                acc[c * 32 + i * 8 + e] = dh * a * sg;
              }
            }
            rows_bf16(d1, p.out0, col);
            rows_bf16(acc + 32 * c, p.out1, col);
          }
        }
      } else {
        // columns past F hold zero (their weights are read as zero)
        constexpr int HC = COLS / 2;
        const int f = t.nt * 128 + cg * HC;
#pragma unroll
        for (int c = 0; c < HC / 32; ++c) {
          if (p.out1) rows_bf16(acc + 32 * c, p.out1, f + 32 * c);
          if (p.out2) rows_bf16(acc + HC + 32 * c, p.out2, f + 32 * c);
        }
        float m = 0.0f;
#pragma unroll
        for (int i = 0; i < HC; ++i) {
          acc[i] = swiglu(acc[i], acc[HC + i]);
          m = fmaxf(m, fabsf(acc[i]));
        }
        if (p.out3) {
#pragma unroll
          for (int c = 0; c < HC / 32; ++c) rows_bf16(acc + 32 * c, p.out3, f + 32 * c);
        }
        // the other column groups' maxima of the same rows; two buffers, since a
        // warp is at most one exchange ahead of the others
        float* mx = s_max + (tcount & 1u) * 512 + r;
        mx[cg * 128] = m;
        __syncwarp();
        if (lane == 0) mbar_arrive(&xbar[q]);
        ok = warp_wait(&xbar[q], tcount & 1u, s_abort, p.status, 890 + q);
        if (!ok) break;
#pragma unroll
        for (int g = 0; g < CG; ++g) m = fmaxf(m, mx[g * 128]);
        const float hscale = scale_of_h(m), hf = h_factor(hscale), rs = 1.0f / (hscale * hf);
        if (hf != 1.0f) {
#pragma unroll
          for (int i = 0; i < HC; ++i) acc[i] *= hf;
        }
        if (cg == 0 && r < t.valid) p.hs[(row + lane) * p.hs_ld + t.nt] = hscale;
        uint4* dst = reinterpret_cast<uint4*>(static_cast<uint8_t*>(p.out0) + (row + lane) * p.n + f);
#pragma unroll
        for (int k = 0; k < HC / 16; ++k) {
          uint32_t w[4];
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            // times the reciprocal: h carries a thousand such roundings already, and the exact
            // quotient (ten instructions an element) made this launch a quarter longer
            const float* h = acc + k * 16 + 4 * i;
            w[i] = fp8_pack4(h[0] * rs, h[1] * rs, h[2] * rs, h[3] * rs);
          }
          if (r < t.valid && f + k * 16 < p.n) dst[k] = make_uint4(w[0], w[1], w[2], w[3]);
        }
      }
    }
    __syncwarp();
    if constexpr (SPLIT) {
      cluster_sync_all();
      // a warp a row: the CTAs' sums added in the order of their k-blocks
      if (unit0 < total) {
        const Tile t = find_tile(unit0, p, s_pre);
        const int col = t.nt * 128 + lane * 4;
        for (int r = rank * kEpiWarps + ew; r < t.valid; r += ranks * kEpiWarps) {
          const uint32_t at = smem_u32(smem) + r * (BN * 4) + ((lane ^ (r & 31)) << 4);
          float a[NS][4] = {};
          for (int c = 0; c < ranks; ++c)
#pragma unroll
            for (int j = 0; j < NS; ++j) {
              const float4 v = ld_cluster_f32x4(mapa_shared(at + j * 512, c));
              a[j][0] += v.x;
              a[j][1] += v.y;
              a[j][2] += v.z;
              a[j][3] += v.w;
            }
          const int64_t row = t.row0 + r;
          auto row_bf16 = [&](const float* f, void* out) {
            if (out && col < p.n)
              *reinterpret_cast<uint2*>(static_cast<uint8_t*>(out) + (row * p.n + col) * 2) =
                  make_uint2(bf2(f[0], f[1]), bf2(f[2], f[3]));
          };
          if constexpr (DUAL) {
            row_bf16(a[0], p.out1);
            row_bf16(a[1], p.out2);
            float m = 0.0f;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              a[0][i] = swiglu(a[0][i], a[1][i]);
              m = fmaxf(m, fabsf(a[0][i]));
            }
            row_bf16(a[0], p.out3);
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
            const float hscale = scale_of_h(m), hf = h_factor(hscale), rs = 1.0f / (hscale * hf);
            if (lane == 0) p.hs[row * p.hs_ld + t.nt] = hscale;
            if (col < p.n)
              *reinterpret_cast<uint32_t*>(static_cast<uint8_t*>(p.out0) + row * p.n + col) =
                  fp8_pack4(a[0][0] * hf * rs, a[0][1] * hf * rs, a[0][2] * hf * rs, a[0][3] * hf * rs);
          } else {
            row_bf16(a[0], p.out0);
          }
        }
      }
      cluster_sync_all();   // no CTA's sums go away while another reads them
    }
  }

  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 1) tmem_dealloc(tmem_base, 512);
}

// -------------------------------------------------------------------- host
using EncodeFn = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                              const cuuint64_t*, const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave,
                              CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeFn encode_fn() {
  static EncodeFn fn = nullptr;
  static std::once_flag once;
  std::call_once(once, [] {
    void* ptr = nullptr;
    cudaDriverEntryPointQueryResult q{};
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &ptr, 12000, cudaEnableDefault, &q) ==
            cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      fn = reinterpret_cast<EncodeFn>(ptr);
  });
  return fn;
}

// Codes {inner, rows, groups} (2-D without groups) in boxes of 128 bytes x
// box_rows, 128-byte swizzle, zero outside.
bool code_map(CUtensorMap* map, const void* base, int64_t inner, int64_t rows, int64_t groups, uint32_t box_rows) {
  EncodeFn enc = encode_fn();
  if (!enc || !base || (reinterpret_cast<uintptr_t>(base) & 15u) || inner % 16) return false;
  cuuint64_t dims[3] = {static_cast<cuuint64_t>(inner), static_cast<cuuint64_t>(rows),
                        static_cast<cuuint64_t>(groups > 0 ? groups : 1)};
  cuuint64_t strides[2] = {static_cast<cuuint64_t>(inner), static_cast<cuuint64_t>(inner * rows)};
  cuuint32_t box[3] = {128, box_rows, 1};
  cuuint32_t one[3] = {1, 1, 1};
  return enc(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, groups > 0 ? 3 : 2, const_cast<void*>(base), dims, strides, box, one,
             CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Allows the kernel its shared memory, once.
template <auto K, int BN>
cudaError_t prepare() {
  static const cudaError_t err = cudaFuncSetAttribute(K, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                                      static_cast<int>(Cfg<BN>::smem_bytes(kMaxGroups)));
  return err;
}

template <int BN, bool B_MN, int EPI>
cudaError_t launch_form(const Fp8Params& p, int64_t units, cudaStream_t st) {
  constexpr auto K = fp8_gemm_kernel<BN, B_MN, EPI, false>;
  const cudaError_t err = prepare<K, BN>();
  if (err != cudaSuccess) return err;
  return launch_pdl(K, static_cast<unsigned>(std::min<int64_t>(units, num_sms())), kThreads,
                    Cfg<BN>::smem_bytes(p.groups), st, p);
}

// Clusters of S CTAs of a split kernel that run at once.
template <auto K, int BN, int S>
int resident_clusters() {
  static const int n = [] {
    cudaLaunchConfig_t cfg{};
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeClusterDimension;
    at[0].val.clusterDim = {S, 1, 1};
    cfg.gridDim = dim3(S * num_sms());
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = Cfg<BN>::smem_bytes(kMaxGroups);
    cfg.attrs = at;
    cfg.numAttrs = 1;
    int clusters = 0;
    if (prepare<K, BN>() != cudaSuccess || cudaOccupancyMaxActiveClusters(&clusters, K, &cfg) != cudaSuccess) {
      cudaGetLastError();
      return 0;
    }
    return clusters;
  }();
  return n;
}
// Launches `units` tiles on clusters of S, or of fewer where they would not all run at
// once or a CTA would have fewer than eight k-blocks; false: not split.
template <int BN, bool B_MN, int EPI, int S>
bool launch_split(const Fp8Params& p, int64_t units, cudaStream_t st, cudaError_t* err) {
  if constexpr (S == 1) {
    return false;
  } else {
    constexpr auto K = fp8_gemm_kernel<BN, B_MN, EPI, true>;
    if (p.sources > 1 || p.kb < 8 * S || units * S > num_sms() || units > resident_clusters<K, BN, S>())
      return launch_split<BN, B_MN, EPI, S / 2>(p, units, st, err);
    *err = launch_pdl<S>(K, static_cast<unsigned>(units * S), kThreads, Cfg<BN>::smem_bytes(p.groups), st, p);
    return true;
  }
}

template <bool B_MN, int EPI>
cudaError_t launch_pick(const Fp8Params& p, int bn, int64_t units, cudaStream_t st) {
  cudaError_t err;
  if constexpr (EPI == FP8_EPI_BF16)
    if (bn == 128)
      return launch_split<128, B_MN, EPI, 8>(p, units, st, &err) ? err : launch_form<128, B_MN, EPI>(p, units, st);
  if constexpr (EPI == FP8_EPI_SWIGLU_FWD)
    if (launch_split<256, B_MN, EPI, 8>(p, units, st, &err)) return err;
  return launch_form<256, B_MN, EPI>(p, units, st);
}

}  // namespace

cudaError_t launch_fp8_quant_rows(const void* src, int64_t rows, int64_t cols, uint8_t* codes, float* scales,
                                  int64_t ld, cudaStream_t st) {
  if (rows <= 0) return cudaSuccess;
  const int64_t warps = rows * ((cols / 16 + 31) / 32);
  const int grid = static_cast<int>(std::min<int64_t>((warps + 7) / 8, static_cast<int64_t>(num_sms()) * 32));
  return launch_pdl(fp8_quant_rows_kernel, grid, 256, 0, st, static_cast<const uint4*>(src), rows,
                    static_cast<int>(cols / 16), reinterpret_cast<uint4*>(codes), scales, ld);
}

cudaError_t launch_fp8_quant_scatter(const void* x, int n_tok, int d, int top_k, const int32_t* row_of_copy,
                                     uint8_t* codes, float* scales, int64_t ld, uint8_t* tok_codes,
                                     float* tok_scales, cudaStream_t st) {
  if (n_tok <= 0) return cudaSuccess;
  const int64_t warps = static_cast<int64_t>(n_tok) * ((d / 16 + 31) / 32);
  const int grid = static_cast<int>(std::min<int64_t>((warps + 7) / 8, static_cast<int64_t>(num_sms()) * 32));
  return launch_pdl(fp8_quant_scatter_kernel, grid, 256, 0, st, static_cast<const uint4*>(x), n_tok, d / 16, top_k,
                    row_of_copy, reinterpret_cast<uint4*>(codes), scales, ld, reinterpret_cast<uint4*>(tok_codes),
                    tok_scales);
}

cudaError_t launch_fp8_gemm(const Fp8GemmArgs& a, cudaStream_t st) {
  if (a.rows <= 0 || a.n <= 0 || a.groups <= 0) return cudaSuccess;
  if (a.groups > kMaxGroups || a.k <= 0 || a.k % 16 || a.n % 16 || a.sources < 1 || a.sources > 2 ||
      a.rows > 0x7fffff00LL || a.n > 0x3fffffffLL || a.k > 0x3fffffffLL)
    return cudaErrorInvalidValue;
  // most M tiles of any split of the rows into groups
  const int64_t mtiles = a.rows / BM + std::min<int64_t>(a.groups, a.rows);
  // 128 columns a tile where 256 would leave SMs without one: a row for each of 8
  // groups of 2048 x 7168 24.7 us (256: 28.8), 8 rows of one group 20.7 (26.8); with
  // tiles enough 256: 64 groups of 128 rows of 7168 x 2048 164 us (128: 174), 8 of 1024
  // rows of 4096 x 4096 116 (172)
  const int bn = a.epi == FP8_EPI_BF16 && mtiles * ((a.n + 255) / 256) < num_sms() ? 128 : 256;
  Fp8Params p{};
  for (int s = 0; s < a.sources; ++s) {
    if (!code_map(&p.tmA[s], a.a[s], a.k, a.rows, 0, 128)) return cudaErrorInvalidValue;
    if (!code_map(&p.tmA32[s], a.a[s], a.k, a.rows, 0, 32)) return cudaErrorInvalidValue;
    p.a_scale[s] = a.a_scale[s];
  }
  for (int s = 0; s < (a.dual ? 2 : a.sources); ++s) {
    if (!(a.b_mn ? code_map(&p.tmB[s], a.b[s], a.n, a.k, a.groups, 128)
                 : code_map(&p.tmB[s], a.b[s], a.k, a.n, a.groups, a.dual ? 128 : bn)))
      return cudaErrorInvalidValue;
    p.b_scale[s] = a.b_scale[s];
  }
  p.a_scale_ld = a.a_scale_ld;
  p.offsets = a.offsets;
  p.groups = a.groups;
  p.rows = static_cast<int32_t>(a.rows);
  p.n = static_cast<int32_t>(a.n);
  p.kb = static_cast<int32_t>((a.k + BK - 1) / BK);
  p.sources = a.sources;
  p.n128 = static_cast<int32_t>((a.n + 127) / 128);
  p.ntiles = a.dual ? p.n128 : static_cast<int32_t>((a.n + bn - 1) / bn);
  p.out0 = a.out0;
  p.out1 = a.out1;
  p.out2 = a.out2;
  p.out3 = a.out3;
  p.hs = a.hs;
  p.hs_ld = a.hs_ld;
  p.in0 = a.in0;
  p.in1 = a.in1;
  p.status = a.status;
  const int64_t units = mtiles * p.ntiles;
  if (a.epi == FP8_EPI_SWIGLU_FWD) return launch_pick<false, FP8_EPI_SWIGLU_FWD>(p, bn, units, st);
  if (a.epi == FP8_EPI_SWIGLU_BWD) return launch_pick<true, FP8_EPI_SWIGLU_BWD>(p, bn, units, st);
  return a.b_mn ? launch_pick<true, FP8_EPI_BF16>(p, bn, units, st)
                : launch_pick<false, FP8_EPI_BF16>(p, bn, units, st);
}

}  // namespace moe
