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

}  // namespace sage
