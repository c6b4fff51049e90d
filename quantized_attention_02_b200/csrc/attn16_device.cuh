// attn16_device.cuh -- device helpers of the 16-bit attention kernels: a sequence's place and length, the
// keys a query sees, packing.
#pragma once
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "attn16_kernels.cuh"
#include "attn_common.cuh"

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

// Paged: how many sequences own slots up to `slot`, where sequence b owns those from cu_q[b] / tokens + b on (tokens: of
// a slot).  That leaves room for its ceil(nq / tokens) slots before the next one's and needs no sum over the sequences.
// By a whole warp.  The places ascend, so each look at 32 of them leaves one piece in 32: a look at every place took
// 700 cycles per 32 sequences, and a walk past many empty ones could then outlast the waits for it (the square of their
// number: 30 ms for 20000, 0.5 ms now).  (Places that do not ascend give some number in [0, B].)
__device__ __forceinline__ int sequences_upto(const Attn16Args& a, int tokens, int slot) {
  const int lane = threadIdx.x & 31;
  int lo = 0, n = a.B;  // the number is in [lo, lo + n]
  while (n > 0) {
    const int piece = (n + 31) >> 5, at = lane * piece;
    const int last = lo + min(n, at + piece) - 1;  // of this lane's piece
    const bool in = at < n && min(max(__ldg(a.cu_q + last), 0), a.Nq) / tokens + last <= slot;
    const int skip = min(n, __popc(__ballot_sync(0xffffffffu, in)) * piece);
    lo += skip;
    n = max(0, min(piece, n - skip) - 1);  // the next piece, whose last is past the slot
  }
  return lo;
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

// What a row's O is multiplied with at the end: 0 for a row without a key, NaN for a sum that is NaN.
__device__ __forceinline__ float weight_sum_inverse(float l) { return l == 0.f ? 0.f : 1.f / l; }

// Two means of an output row as a pair, in fp16's range.  The weights' rounding moves a mean by up to 2^-11 of the values'
// size, which their unrounded sum does not follow: next to 65504 the mean would round to infinity.  (bf16's range is
// that of the accumulator.)
template <bool BF16>
__device__ __forceinline__ uint32_t pack_in_range(float lo, float hi) {
  if constexpr (!BF16) {
    if (fabsf(lo) < INFINITY) lo = fminf(fmaxf(lo, -65504.f), 65504.f);
    if (fabsf(hi) < INFINITY) hi = fminf(fmaxf(hi, -65504.f), 65504.f);
  }
  return pack16<BF16>(lo, hi);
}
// 32 of a row's means, unnormalised, times `scale` into pairs, and the largest of them into `most` (four chains).
template <bool BF16>
__device__ __forceinline__ void pack_means(const uint32_t (&o)[32], float scale, uint32_t (&w)[16], __half2 (&most)[4]) {
#pragma unroll
  for (int i = 0; i < 16; ++i) {
    w[i] = pack16<BF16>(__uint_as_float(o[2 * i]) * scale, __uint_as_float(o[2 * i + 1]) * scale);
    if constexpr (!BF16) most[i & 3] = __hmax2(most[i & 3], __habs2(*reinterpret_cast<const __half2*>(&w[i])));
  }
}
// Whether one of the warp's rows has an infinite mean, so that they have to be packed again, in range.
template <bool BF16>
__device__ __forceinline__ bool out_of_range(const __half2 (&most)[4]) {
  if constexpr (BF16) return false;
  const __half2 m = __hmax2(__hmax2(most[0], most[1]), __hmax2(most[2], most[3]));
  const uint32_t bits = *reinterpret_cast<const uint32_t*>(&m);
  return __any_sync(0xffffffffu, (bits & 0xffffu) == 0x7c00u || bits >> 16 == 0x7c00u);
}

// Parts c0 .. c1 of ROWS rows joined by a warp, in the parts' order: acc[k][e] = sum_c 2^(m_c - m) O_c of row k, l
// likewise, m the largest m_c.  at(k, c): the place of part c of row k in ml and in o (rows of D = 32 C fp32).
// The lanes take the parts' factors first, 32 at a time, so that the loads of O follow each other without
// waiting.
template <int ROWS, int C, typename At>
__device__ __forceinline__ void join_parts(float (&acc)[ROWS][C], float (&l)[ROWS], int c0, int c1, const float2* ml,
                                           const float* o, At at) {
  const int lane = threadIdx.x & 31;
  float m[ROWS];
#pragma unroll
  for (int k = 0; k < ROWS; ++k) {
    m[k] = -INFINITY;
    l[k] = 0.f;
#pragma unroll
    for (int e = 0; e < C; ++e) acc[k][e] = 0.f;
  }
  for (int c = c0 + lane; c <= c1; c += 32) {
#pragma unroll
    for (int k = 0; k < ROWS; ++k) m[k] = fmaxf(m[k], ml[at(k, c)].x);
  }
#pragma unroll
  for (int k = 0; k < ROWS; ++k) {
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) m[k] = fmaxf(m[k], __shfl_xor_sync(0xffffffffu, m[k], off));
    if (m[k] == -INFINITY) m[k] = 0.f;
  }
  for (int first = c0; first <= c1; first += 32) {
    const int n = min(32, c1 - first + 1);
    float w[ROWS];
#pragma unroll
    for (int k = 0; k < ROWS; ++k) {
      const float2 mine = lane < n ? ml[at(k, first + lane)] : make_float2(-INFINITY, 0.f);
      w[k] = exp2f(mine.x - m[k]);
      float part = mine.y * w[k];
#pragma unroll
      for (int off = 16; off > 0; off >>= 1) part += __shfl_xor_sync(0xffffffffu, part, off);
      l[k] += part;
    }
#pragma unroll 4
    for (int i = 0; i < n; ++i) {
#pragma unroll
      for (int k = 0; k < ROWS; ++k) {
        const float f = __shfl_sync(0xffffffffu, w[k], i);
        const float* src = o + at(k, first + i) * (32 * C) + lane * C;
#pragma unroll
        for (int e = 0; e < C; e += 2) {
          const float2 y = *reinterpret_cast<const float2*>(src + e);
          acc[k][e] = fmaf(y.x, f, acc[k][e]);
          acc[k][e + 1] = fmaf(y.y, f, acc[k][e + 1]);
        }
      }
    }
  }
}

// A joined row into O: this lane's C channels from `dst` on.
template <bool BF16, int C>
__device__ __forceinline__ void store_joined(uint16_t* dst, const float (&acc)[C], float l) {
  const float inv = weight_sum_inverse(l);
#pragma unroll
  for (int e = 0; e < C; e += 2)
    *reinterpret_cast<uint32_t*>(dst + e) = pack_in_range<BF16>(acc[e] * inv, acc[e + 1] * inv);
}

}  // namespace sage
