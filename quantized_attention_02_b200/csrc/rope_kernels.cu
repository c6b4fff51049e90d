// rope_kernels.cu -- norm of every query and key head, position rotation, and the append into a paged
// cache, in one pass over the projection's output.
//
// Mathematics, per token and head (x of d channels, all in fp32, one rounding at the end):
//   y = x * rsqrt(mean(x^2) + eps) * w          (w null: y = x)
//   (a, b) -> (a c - b s, b c + a s)            on the pairs of the first rot channels, c and s from row
//                                               `position` of the tables; pairs (i, i + rot/2), or
//                                               (2i, 2i + 1) when interleaved; channels past rot: y
// Bound: device memory (each element read once, written once: 4 bytes), if the instructions are kept down: at
// 6.5 TB/s an SM has about 90 issue slots for the 16 bytes of a lane.
// Layout: a row of d channels belongs to d/8 lanes, 8 channels (16 bytes) each, so a row is one coalesced
// 16-byte access per lane and the sum of squares a shuffle over those lanes.  A block works on eight heads of
// one tensor for its tokens (all eight loads first), so that what a lane needs besides -- weight and rotation,
// multiplied together once -- is the same for all of them: y = r (x cw + x' sw), x' the pair's other channel
// (its neighbour, or, half split, from another lane: shuffled as 16-bit pairs), r the row's norm.
// 2 x (48 + 48) heads of 64 channels, 16384 tokens, fp16, interleaved: 123 us in the profiler, 6.56 TB/s; 128 us a call
// (224 us with the norm, the weights and both pair layouts worked out per head: 213 instructions per 16 bytes; 141 us
// with four heads and 256 threads, 168 us with two heads).
// Half split pairs cost more: four shuffles per row and, at 64 registers (eight blocks per SM), 44 to 48 bytes of spills
// a thread where the interleaved form has 8 at most.  8192 tokens of 32 + 8 + 8 heads of 128 into a cache: 37 us in the
// profiler, 5.5 TB/s, with 67 % of the issue slots taken (62 % above).
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

constexpr int kRopeThreads = 128;
constexpr int kHeads = 8;  // heads per thread

__host__ __device__ constexpr int head_groups(int heads) { return (heads + kHeads - 1) / kHeads; }

template <int D, bool BF16, bool INTERLEAVED>
__global__ void __launch_bounds__(kRopeThreads, 8) qk_norm_rope_kernel(const __grid_constant__ RopeArgs a) {
  constexpr int LANES = D / 8;  // lanes per row
  constexpr int TOKENS = kRopeThreads / LANES;
  // ---- the block's tensor and heads, this thread's token and channels
  const int gq = head_groups(a.Hq), gk = head_groups(a.Hk), groups = gq + gk + head_groups(a.Hv);
  const int group = static_cast<int>(blockIdx.x) % groups;
  const unsigned tokens = static_cast<unsigned>(a.B) * a.N;
  const unsigned item = blockIdx.x / groups * TOKENS + threadIdx.x / LANES;
  // rows of a warp past the end still take part in its shuffles
  const bool live = item < tokens;
  const unsigned token = live ? item : tokens - 1;
  const int b = static_cast<int>(token / a.N), n = static_cast<int>(token) - b * a.N;
  const int l = threadIdx.x % LANES, c0 = 8 * l;
  const bool is_q = group < gq, is_v = group >= gq + gk;
  const RopeTensor& t = is_q ? a.q : is_v ? a.v : a.k;
  const int h0 = (is_q ? group : is_v ? group - gq - gk : group - gq) * kHeads;
  const int heads = (is_q ? a.Hq : is_v ? a.Hv : a.Hk) - h0;  // of them, kHeads at most

  // ---- all loads first
  const uint16_t* src = static_cast<const uint16_t*>(t.in) + b * t.in_st.b + h0 * t.in_st.h + n * t.in_st.n + c0;
  uint4 raw[kHeads];
#pragma unroll
  for (int i = 0; i < kHeads; ++i, src += t.in_st.h)
    raw[i] = live && i < heads ? *reinterpret_cast<const uint4*>(src) : make_uint4(0, 0, 0, 0);

  // ---- where the token's rows go
  long long ob = b, on = n;
  bool keep = live;
  if (a.slots && !is_q) {
    const int slot = __ldg(a.slots + token);
    keep = live && slot >= 0 && slot < a.slot_count;
    ob = slot >> a.page_shift;
    on = slot & ((1 << a.page_shift) - 1);
  }
  uint16_t* dst = static_cast<uint16_t*>(t.out) + ob * t.out_st.b + h0 * t.out_st.h + on * t.out_st.n + c0;
  if (is_v) {  // copied as it is
#pragma unroll
    for (int i = 0; i < kHeads; ++i, dst += t.out_st.h)
      if (keep && i < heads) *reinterpret_cast<uint4*>(dst) = raw[i];
    return;
  }

  // ---- factors of this lane's channels: cw of the channel itself, sw of the pair's other one
  const int half = a.rot >> 1;
  const bool turned = c0 < a.rot;
  // half split: the other channels sit half/8 lanes up (first half) or down (second half)
  const int lane = threadIdx.x & 31;
  const int away = INTERLEAVED || !turned ? 0 : c0 < half ? half >> 3 : -(half >> 3);
  float cw[8], sw[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) cw[i] = 1.f, sw[i] = 0.f;
  const int pos = a.positions ? __ldg(a.positions + static_cast<long long>(b) * a.positions_stride_b + n) : n;
  if (pos < 0 || pos >= a.table_rows) {  // no rotation in the tables: the token's rows become NaN, nothing is read
#pragma unroll
    for (int i = 0; i < 8; ++i) cw[i] = __int_as_float(0x7fc00000);
  } else if (turned) {
    const float* pc = a.cos + static_cast<long long>(pos) * half;
    const float* ps = a.sin + static_cast<long long>(pos) * half;
    if constexpr (INTERLEAVED) {
      const float4 c = __ldg(reinterpret_cast<const float4*>(pc + (c0 >> 1)));
      const float4 s = __ldg(reinterpret_cast<const float4*>(ps + (c0 >> 1)));
      const float cv[4] = {c.x, c.y, c.z, c.w}, sv[4] = {s.x, s.y, s.z, s.w};
#pragma unroll
      for (int p = 0; p < 4; ++p) {
        cw[2 * p] = cw[2 * p + 1] = cv[p];
        sw[2 * p] = -sv[p];
        sw[2 * p + 1] = sv[p];
      }
    } else {
      const int at = c0 < half ? c0 : c0 - half;
      const float sign = c0 < half ? -1.f : 1.f;
#pragma unroll
      for (int k = 0; k < 8; k += 4) {
        *reinterpret_cast<float4*>(cw + k) = __ldg(reinterpret_cast<const float4*>(pc + at + k));
        *reinterpret_cast<float4*>(sw + k) = __ldg(reinterpret_cast<const float4*>(ps + at + k));
      }
#pragma unroll
      for (int k = 0; k < 8; ++k) sw[k] *= sign;
    }
  }
  const bool norm = t.weight != nullptr;
  if (norm) {
    const uint16_t* weight = static_cast<const uint16_t*>(t.weight);
    float w[8], wo[8];  // of the channels, of the pairs' other ones
    unpack8<BF16>(__ldg(reinterpret_cast<const uint4*>(weight + c0)), w);
    if constexpr (INTERLEAVED) {
#pragma unroll
      for (int k = 0; k < 8; ++k) wo[k] = w[k ^ 1];
    } else {
      unpack8<BF16>(__ldg(reinterpret_cast<const uint4*>(weight + c0 + 8 * away)), wo);
    }
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      cw[k] *= w[k];
      sw[k] *= wo[k];
    }
  }

#pragma unroll
  for (int i = 0; i < kHeads; ++i, dst += t.out_st.h) {
    if (i >= heads) break;  // the same for the whole block
    float x[8];
    unpack8<BF16>(raw[i], x);
    float r = 1.f;
    if (norm) {
      float2 ss = make_float2(0.f, 0.f);
#pragma unroll
      for (int k = 0; k < 8; k += 2) ss = __ffma2_rn(make_float2(x[k], x[k + 1]), make_float2(x[k], x[k + 1]), ss);
      float sum = ss.x + ss.y;
#pragma unroll
      for (int off = LANES / 2; off > 0; off >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, off);
      r = rsqrtf(sum * (1.f / D) + a.eps);
    }
    float y[8];
    if constexpr (INTERLEAVED) {
#pragma unroll
      for (int k = 0; k < 8; ++k) y[k] = turned ? fmaf(x[k ^ 1], sw[k], x[k] * cw[k]) : x[k] * cw[k];
    } else {
      uint4 other;
      other.x = __shfl_sync(0xffffffffu, raw[i].x, lane + away);
      other.y = __shfl_sync(0xffffffffu, raw[i].y, lane + away);
      other.z = __shfl_sync(0xffffffffu, raw[i].z, lane + away);
      other.w = __shfl_sync(0xffffffffu, raw[i].w, lane + away);
      float o[8];
      unpack8<BF16>(other, o);
#pragma unroll
      for (int k = 0; k < 8; k += 2) {
        float2 v = __fmul2_rn(make_float2(x[k], x[k + 1]), make_float2(cw[k], cw[k + 1]));
        if (turned) v = __ffma2_rn(make_float2(o[k], o[k + 1]), make_float2(sw[k], sw[k + 1]), v);
        y[k] = v.x;
        y[k + 1] = v.y;
      }
    }
    if (norm) {
#pragma unroll
      for (int k = 0; k < 8; k += 2) {
        const float2 v = __fmul2_rn(make_float2(y[k], y[k + 1]), make_float2(r, r));
        y[k] = v.x;
        y[k + 1] = v.y;
      }
    }
    if (keep) *reinterpret_cast<uint4*>(dst) = pack8<BF16>(y);
  }
}

template <int D, bool BF16>
cudaError_t launch_t(const RopeArgs& a, cudaStream_t st) {
  const long long groups = head_groups(a.Hq) + head_groups(a.Hk) + head_groups(a.Hv);
  const long long per_block = kRopeThreads / (D / 8);
  const unsigned grid = static_cast<unsigned>((static_cast<long long>(a.B) * a.N + per_block - 1) / per_block * groups);
  if (a.interleaved) qk_norm_rope_kernel<D, BF16, true><<<grid, kRopeThreads, 0, st>>>(a);
  else qk_norm_rope_kernel<D, BF16, false><<<grid, kRopeThreads, 0, st>>>(a);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_qk_norm_rope(const RopeArgs& a, cudaStream_t st) {
  if (a.d == 128) return a.bf16 ? launch_t<128, true>(a, st) : launch_t<128, false>(a, st);
  return a.bf16 ? launch_t<64, true>(a, st) : launch_t<64, false>(a, st);
}

}  // namespace sage
