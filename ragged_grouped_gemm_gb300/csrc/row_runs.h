// The runs of rows that a long weight gradient is summed in (grouped_gemm.cu), for host compilers too.
#pragma once
#include <cstdint>

#ifdef __CUDACC__
#define MOE_HOST_DEVICE __host__ __device__ __forceinline__
#else
#define MOE_HOST_DEVICE inline
#endif

namespace moe {

constexpr int kRowChunk = 1792;   // rows of a run, about

// The runs of a group of `rows` rows (one for none).
MOE_HOST_DEVICE int row_runs(int rows) { return rows > kRowChunk ? (rows - 1) / kRowChunk + 1 : 1; }

// The first of num_kb k-blocks that run `run` of `runs` takes; num_kb itself for run == runs.  The product passes 32 bits
// from about 16 million rows in a group.
MOE_HOST_DEVICE int run_begin(int run, int runs, int num_kb) {
  return static_cast<int>(static_cast<int64_t>(run) * num_kb / runs);
}

}  // namespace moe
