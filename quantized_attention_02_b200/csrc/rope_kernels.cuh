// rope_kernels.cuh -- launcher of the query / key norm + rotation kernel (rope_kernels.cu).
#pragma once
#include <cstdint>
#include <cuda_runtime.h>

#include "sage_attn.h"

namespace sage {

// One of the up to three tensors a launch walks.
struct RopeTensor {
  const void* in;
  void* out;
  const void* weight;       // null: no norm
  sage_strides in_st, out_st;
};

struct RopeArgs {
  RopeTensor q, k, v;       // v: copied into the cache (append), unused otherwise
  const float* cos;
  const float* sin;
  const int32_t* positions; // null: row n of the table
  const int32_t* slots;     // null: k goes to k.out; else k and v go to the cache slots
  int positions_stride_b;
  int B, N, Hq, Hk, Hv;
  int d, rot, table_rows;
  int page_shift;           // log2 of the page size (append)
  int slot_count;           // pages * page size (append)
  float eps;
  bool interleaved, bf16;
};

cudaError_t launch_qk_norm_rope(const RopeArgs& a, cudaStream_t st);

}  // namespace sage
