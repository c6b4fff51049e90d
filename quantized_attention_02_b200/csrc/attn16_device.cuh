// attn16_device.cuh -- device helpers of the 16-bit attention kernels: a sequence's place and length, the
// keys a query sees, packing.
#pragma once
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "attn16_kernels.cuh"

namespace sage {

struct Sequence {
  int b, token0, nq, kv;  // token0: first token in the query tensor (paged) or 0 (dense)
};

__device__ __forceinline__ int keys_of(const Attn16Args& a, int b) {
  return a.kv_len ? min(max(__ldg(a.kv_len + b), 0), a.Nk) : a.Nk;
}

// Keys that query `tok` of the sequence sees.
__device__ __forceinline__ int visible(const Attn16Args& a, const Sequence& s, int tok) {
  return a.causal ? min(max(s.kv - s.nq + tok + 1, 0), s.kv) : s.kv;
}

// Sequence b: its tokens and keys, taken into range.
__device__ __forceinline__ Sequence sequence(const Attn16Args& a, int b) {
  Sequence s;
  s.b = b;
  if (a.cu_q) {
    s.token0 = min(max(__ldg(a.cu_q + b), 0), a.Nq);
    s.nq = max(0, min(max(__ldg(a.cu_q + b + 1), 0), a.Nq) - s.token0);
  } else {
    s.token0 = 0;
    s.nq = a.Nq;
  }
  s.kv = keys_of(a, b);
  return s;
}

// Key tiles that `tokens` tokens from tok0 on see together: those of the last one.
__device__ __forceinline__ int key_tiles(const Attn16Args& a, const Sequence& s, int tok0, int tokens) {
  return (visible(a, s, min(s.nq, tok0 + tokens) - 1) + 127) / 128;
}

// Element offset of head h of the sequence's token `tok` in O.
__device__ __forceinline__ long long out_offset(const Attn16Args& a, const Sequence& s, int tok, int h) {
  return (a.cu_q ? 0 : s.b * a.o_sb) + h * a.o_sh + static_cast<long long>(s.token0 + tok) * a.o_sn;
}

template <bool BF16>
__device__ __forceinline__ uint32_t pack16(float lo, float hi) {
  if constexpr (BF16) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&h);
  } else {
    const __half2 h = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&h);
  }
}

// One row's parts c0 .. c1 joined by a warp, in their order: acc[e] = sum_c 2^(m_c - m) O_c, l likewise, m the largest
// m_c.  ml(c): (m, l) of part c; o(c): where this lane's C channels of its O stand.  The lanes take the parts'
// factors first, 32 at a time, so that the loads of O follow each other without waiting.
template <int C, typename ML, typename O>
__device__ __forceinline__ void join_parts(float (&acc)[C], float& l, int c0, int c1, ML ml, O o) {
  const int lane = threadIdx.x & 31;
  float m = -INFINITY;
  for (int c = c0 + lane; c <= c1; c += 32) m = fmaxf(m, ml(c).x);
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, off));
  const float base = m == -INFINITY ? 0.f : m;
  for (int first = c0; first <= c1; first += 32) {
    const int n = min(32, c1 - first + 1);
    const float2 mine = lane < n ? ml(first + lane) : make_float2(-INFINITY, 0.f);
    const float w = exp2f(mine.x - base);
    float part_l = mine.y * w;
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) part_l += __shfl_xor_sync(0xffffffffu, part_l, off);
    l += part_l;
#pragma unroll 8
    for (int i = 0; i < n; ++i) {
      const float f = __shfl_sync(0xffffffffu, w, i);
      const float* src = o(first + i);
#pragma unroll
      for (int e = 0; e < C; e += 2) {
        const float2 y = *reinterpret_cast<const float2*>(src + e);
        acc[e] = fmaf(y.x, f, acc[e]);
        acc[e + 1] = fmaf(y.y, f, acc[e + 1]);
      }
    }
  }
}

}  // namespace sage
