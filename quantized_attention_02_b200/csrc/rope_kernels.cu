// rope_kernels.cu -- norm of every query and key head, position rotation, and the append into a paged
// cache, in one pass over the projection's output.
//
// Mathematics, per token and head (x of d channels, all in fp32, one rounding at the end):
//   y = x * rsqrt(mean(x^2) + eps) * w          (w null: y = x)
//   (a, b) -> (a c - b s, b c + a s)            on the pairs of the first rot channels, c and s from row
//                                               `position` of the tables; pairs (i, i + rot/2), or
//                                               (2i, 2i + 1) when interleaved; channels past rot: y
// Bound: device memory (each element read once, written once: 4 bytes; about 10 operations).
// Layout: a row of d channels belongs to d/8 lanes, 8 channels (16 bytes) each, so a row is one coalesced
// 16-byte access per lane, the sum of squares a shuffle over those lanes, and a half-split pair's partner
// a shuffle too.  A lane works on HEADS heads of one token, all loads first: the rotation's 16 floats are
// read once per token and channel block, and HEADS 16-byte loads are in flight per thread.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "rope_kernels.cuh"

namespace sage {
namespace {

template <bool BF16>
__device__ __forceinline__ void unpack8(const uint4& u, float (&x)[8]) {
  const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    float2 f;
    if constexpr (BF16) {
      f = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(&w[i]));
    } else {
      f = __half22float2(*reinterpret_cast<const __half2*>(&w[i]));
    }
    x[2 * i] = f.x;
    x[2 * i + 1] = f.y;
  }
}

template <bool BF16>
__device__ __forceinline__ uint4 pack8(const float (&x)[8]) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if constexpr (BF16) {
      const __nv_bfloat162 h = __floats2bfloat162_rn(x[2 * i], x[2 * i + 1]);
      w[i] = *reinterpret_cast<const uint32_t*>(&h);
    } else {
      const __half2 h = __floats2half2_rn(x[2 * i], x[2 * i + 1]);
      w[i] = *reinterpret_cast<const uint32_t*>(&h);
    }
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}

constexpr int kRopeThreads = 256;

template <int D, bool BF16, int HEADS>
__global__ void __launch_bounds__(kRopeThreads) qk_norm_rope_kernel(const __grid_constant__ RopeArgs a) {
  constexpr int LANES = D / 8;  // lanes per row
  const int heads = a.Hq + a.Hk + a.Hv;
  const unsigned groups = static_cast<unsigned>((heads + HEADS - 1) / HEADS);
  const unsigned tokens = static_cast<unsigned>(a.B) * a.N;
  const unsigned item = (blockIdx.x * kRopeThreads + threadIdx.x) / LANES;
  const int l = threadIdx.x % LANES;
  // rows of a warp past the end still take part in its shuffles
  const unsigned token = min(item / groups, tokens - 1);
  const bool live = item / groups < tokens;
  const int h0 = static_cast<int>(item % groups) * HEADS;
  const int b = static_cast<int>(token) / a.N, n = static_cast<int>(token) % a.N;
  const int c0 = 8 * l;

  // where this token's K and V go
  long long page = b, row = n;
  bool keep = true;
  if (a.slots) {
    const int slot = __ldg(a.slots + token);
    keep = slot >= 0 && slot < a.slot_count;
    page = slot >> a.page_shift;
    row = slot & ((1 << a.page_shift) - 1);
  }

  // ---- all loads of the thread's heads first
  uint4 raw[HEADS];
#pragma unroll
  for (int i = 0; i < HEADS; ++i) {
    const int h = h0 + i;
    raw[i] = make_uint4(0, 0, 0, 0);
    if (live && h < heads) {
      const RopeTensor& t = h < a.Hq ? a.q : h < a.Hq + a.Hk ? a.k : a.v;
      const int hh = h < a.Hq ? h : h < a.Hq + a.Hk ? h - a.Hq : h - a.Hq - a.Hk;
      raw[i] = *reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(t.in) + b * t.in_st.b + hh * t.in_st.h +
                                               n * t.in_st.n + c0);
    }
  }

  // ---- the rotation of this lane's channels: 8 pairs (half split) or 4 (interleaved)
  const int half = a.rot >> 1;
  float cs[8], sn[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) cs[i] = 1.f, sn[i] = 0.f;
  const int pos = a.positions ? __ldg(a.positions + static_cast<long long>(b) * a.positions_stride_b + n) : n;
  // a position outside the tables has no rotation: the token's rows become NaN, nothing is read
  const bool bad = pos < 0 || pos >= a.table_rows;
  if (c0 < a.rot && !bad) {
    const float* pc = a.cos + static_cast<long long>(pos) * half;
    const float* ps = a.sin + static_cast<long long>(pos) * half;
    const int at = a.interleaved ? c0 >> 1 : (c0 < half ? c0 : c0 - half);
    *reinterpret_cast<float4*>(cs) = __ldg(reinterpret_cast<const float4*>(pc + at));
    *reinterpret_cast<float4*>(sn) = __ldg(reinterpret_cast<const float4*>(ps + at));
    if (!a.interleaved) {
      *reinterpret_cast<float4*>(cs + 4) = __ldg(reinterpret_cast<const float4*>(pc + at + 4));
      *reinterpret_cast<float4*>(sn + 4) = __ldg(reinterpret_cast<const float4*>(ps + at + 4));
    }
  }
  // half split: the partner channels sit half/8 lanes up (first half) or down (second half)
  const int lane = threadIdx.x & 31;
  const int partner = c0 >= a.rot ? lane : c0 < half ? lane + (half >> 3) : lane - (half >> 3);

#pragma unroll
  for (int i = 0; i < HEADS; ++i) {
    const int h = h0 + i;
    const bool is_q = h < a.Hq, is_k = !is_q && h < a.Hq + a.Hk;
    uint4 res = raw[i];  // V: copied as it is
    float x[8];
    unpack8<BF16>(raw[i], x);
    float ss = 0.f;
#pragma unroll
    for (int c = 0; c < 8; ++c) ss = fmaf(x[c], x[c], ss);
#pragma unroll
    for (int off = LANES / 2; off > 0; off >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, off);
    const void* weight = is_q ? a.q.weight : is_k ? a.k.weight : nullptr;
    if (weight) {
      const float r = rsqrtf(ss * (1.f / D) + a.eps);
      float w[8];
      unpack8<BF16>(__ldg(reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(weight) + c0)), w);
#pragma unroll
      for (int c = 0; c < 8; ++c) x[c] = x[c] * r * w[c];
    }
    float y[8];
    if (a.interleaved) {
#pragma unroll
      for (int p = 0; p < 4; ++p) {
        y[2 * p] = x[2 * p] * cs[p] - x[2 * p + 1] * sn[p];
        y[2 * p + 1] = x[2 * p + 1] * cs[p] + x[2 * p] * sn[p];
      }
    } else {
      // first half: a c - b s; second half: b c + a s
      const float sign = c0 < half ? -1.f : 1.f;
#pragma unroll
      for (int c = 0; c < 8; ++c) {
        const float o = __shfl_sync(0xffffffffu, x[c], partner);
        y[c] = x[c] * cs[c] + sign * (o * sn[c]);
      }
    }
    if (c0 >= a.rot) {
#pragma unroll
      for (int c = 0; c < 8; ++c) y[c] = x[c];
    }
    if (bad) {
#pragma unroll
      for (int c = 0; c < 8; ++c) y[c] = __int_as_float(0x7fc00000);
    }
    if (is_q || is_k) res = pack8<BF16>(y);
    if (live && h < heads && (is_q || keep)) {
      const RopeTensor& t = is_q ? a.q : is_k ? a.k : a.v;
      const int hh = is_q ? h : is_k ? h - a.Hq : h - a.Hq - a.Hk;
      const long long ob = is_q ? b : page, on = is_q ? n : row;
      *reinterpret_cast<uint4*>(static_cast<uint16_t*>(t.out) + ob * t.out_st.b + hh * t.out_st.h + on * t.out_st.n +
                                c0) = res;
    }
  }
}

template <int D, bool BF16, int HEADS>
cudaError_t launch_t(const RopeArgs& a, cudaStream_t st) {
  const long long groups = (a.Hq + a.Hk + a.Hv + HEADS - 1) / HEADS;
  const long long items = groups * a.B * a.N;
  const long long per_block = kRopeThreads / (D / 8);
  qk_norm_rope_kernel<D, BF16, HEADS><<<static_cast<unsigned>((items + per_block - 1) / per_block), kRopeThreads, 0, st>>>(a);
  return cudaGetLastError();
}

template <int D, bool BF16>
cudaError_t launch_d(const RopeArgs& a, cudaStream_t st) {
  return launch_t<D, BF16, 4>(a, st);
}

}  // namespace

cudaError_t launch_qk_norm_rope(const RopeArgs& a, cudaStream_t st) {
  if (a.d == 128) return a.bf16 ? launch_d<128, true>(a, st) : launch_d<128, false>(a, st);
  return a.bf16 ? launch_d<64, true>(a, st) : launch_d<64, false>(a, st);
}

}  // namespace sage
