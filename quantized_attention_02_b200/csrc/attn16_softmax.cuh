// attn16_softmax.cuh -- one 128-key tile of the online softmax with query rows on the TMEM lanes, shared by the
// kernels of attn_tile_kernels.cu and attn_pair_kernels.cu.
#pragma once
#include <type_traits>

#include "attn16_device.cuh"
#include "attn_common.cuh"
#include "sm100_ptx.cuh"

namespace sage {

// d = 64 leaves TMEM columns for the weights beside the scores, so that the next scores can be computed as
// soon as these are in registers; d = 128: the weights overwrite the scores
template <int D>
constexpr bool kOwnWeights = D == 64;

// TMEM columns of stream t: scores, accumulator, 16-bit weights
template <int D>
struct Columns {
  __host__ __device__ static constexpr uint32_t s(int t) { return 128u * t; }
  __host__ __device__ static constexpr uint32_t o(int t) { return 256u + static_cast<uint32_t>(D) * t; }
  __host__ __device__ static constexpr uint32_t p(int t) { return kOwnWeights<D> ? 384u + 64u * t : 128u * t; }
};

// A row's running offset (log2 units) and the sum of its weights.
struct RowState {
  float m_use;
  float2 lsum[4];
  __device__ __forceinline__ void clear() {
    m_use = -INFINITY;
#pragma unroll
    for (int i = 0; i < 4; ++i) lsum[i] = make_float2(0.f, 0.f);
  }
  // NaN where a score was NaN or +inf (the accumulator may have missed it).  0 where no score was above -inf: what the
  // polynomial's 2^-126 left in the sum, and in the accumulator, does not count.
  __device__ __forceinline__ float sum() const {
    const float2 l2 = __fadd2_rn(__fadd2_rn(lsum[0], lsum[1]), __fadd2_rn(lsum[2], lsum[3]));
    const float l = l2.x + l2.y;
    return m_use > -INFINITY || l != l ? l : 0.f;
  }
};

// fp16 weights carry a factor 2^7, so that a row's small weights keep their bits (2^8 * 2^7 fits)
template <bool BF16>
constexpr float kWeightShift = BF16 ? 0.f : 7.f;

// Weights 2^(s * scale - offset) of 32 scores into TMEM at tP, one pair in POLY by the polynomial (0: none; the
// MUFU pipe alone would hold up the rest, more of it costs more issue slots than it saves), and their sums.
// NaN and +inf make the sum NaN: on the MUFU pipe by the weight (inf - inf is NaN once the offset has followed), beside the
// polynomial, whose result for them is some number, by adding 0 * u.
template <bool BF16, int POLY>
__device__ __forceinline__ void weights32(const uint32_t* x, uint32_t tP, float scale_log2, float off, float2 (&sum)[4]) {
  const float2 sc2 = make_float2(scale_log2, scale_log2), off2 = make_float2(off, off);
  uint32_t pk[16];
#pragma unroll
  for (int i = 0; i < 32; i += 2) {
    const float2 u = __ffma2_rn(make_float2(__uint_as_float(x[i]), __uint_as_float(x[i + 1])), sc2, off2);
    float2 p;
    if (POLY > 0 && (i >> 1) % (POLY > 0 ? POLY : 1) == POLY - 1) {
      const float2 t = make_float2(max_nan(u.x, -126.f), max_nan(u.y, -126.f));
      p = exp2_poly2_above(t);
      sum[(i >> 1) & 3] = __ffma2_rn(t, make_float2(0.f, 0.f), sum[(i >> 1) & 3]);
    } else {
      p = make_float2(fast_exp2(u.x), fast_exp2(u.y));
    }
    sum[(i >> 1) & 3] = __fadd2_rn(sum[(i >> 1) & 3], p);
    pk[i >> 1] = pack16<BF16>(p.x, p.y);
  }
  tmem_st16(tP, pk);
}

// The largest of N scores.
template <int N>
__device__ __forceinline__ float scores_max(const uint32_t* x) {
  float mx[8];
#pragma unroll
  for (int k = 0; k < 8; ++k) mx[k] = fmaxf(__uint_as_float(x[k]), __uint_as_float(x[8 + k]));
#pragma unroll
  for (int c = 16; c < N; c += 16) {
#pragma unroll
    for (int k = 0; k < 8; ++k) mx[k] = max3f(mx[k], __uint_as_float(x[c + k]), __uint_as_float(x[c + 8 + k]));
  }
  return fmaxf(max3f(mx[0], mx[1], mx[2]), fmaxf(max3f(mx[3], mx[4], mx[5]), fmaxf(mx[6], mx[7])));
}

// This thread's row of a score tile (TMEM column base tS) -> its weights (tP).  The row sees the tile's keys
// below `seen`; the warp's rows that count see seen_warp of them at least and seen_most at most.  `fresh`: the
// row's first tile.  s_free (kOwnWeights): receives an arrival once the scores are read for the last time; prior:
// waits until the product that read the last weights is done, false if that wait gave up.  On return the
// weights are stored but not yet waited for (tcgen05.wait::st).
// Scores that are not finite: NaN and +inf make the row NaN, -inf has no weight, in every tile and at every place of it.
template <int D, bool BF16, typename Prior>
__device__ __forceinline__ bool softmax_tile(RowState& row, uint32_t tS, uint32_t tO, uint32_t tP, int seen, int seen_warp,
                                             int seen_most, bool fresh, float scale_log2, uint64_t* s_free, Prior prior) {
  // The offset moves when the maximum has passed it by 8 (also at the first finite maximum).  The last
  // product is complete, and the next one waits for this tile's weights: O may be rescaled here.
  auto move_offset = [&](float mx) {
    const bool move = mx > row.m_use + 8.f;
    const float alpha = move ? fast_exp2(row.m_use - mx) : 1.f;
    if (move) row.m_use = mx;
#pragma unroll
    for (int i = 0; i < 4; ++i) row.lsum[i] = __fmul2_rn(row.lsum[i], make_float2(alpha, alpha));
#pragma unroll 1
    for (int cb = 0; cb < D; cb += 32) {
      uint32_t ov[32];
      tmem_ld32_sync(tO + cb, ov);
#pragma unroll
      for (int i = 0; i < 32; ++i) ov[i] = __float_as_uint(__uint_as_float(ov[i]) * alpha);
      tmem_st32(tO + cb, ov);
    }
  };
  auto offset = [&]() { return kWeightShift<BF16> - (row.m_use == -INFINITY ? 0.f : row.m_use); };
  if (fresh || seen_warp < 128) {
    // A first tile, whose maximum has to be known before its weights, or one with masked keys.  Rolled loops over 32
    // keys that read the scores twice: beside the pass below this is little code, and where keys are few,
    // so that every tile comes here, it is the instruction fetch that counts.  Masked weights are exactly 0 on
    // the MUFU pipe (ex2(-inf)); the polynomial bottoms out at 2^-126 instead and is not used.
    const int most = min(seen_most, 128);
    auto scores = [&](int cb, uint32_t (&x)[32]) {
      tmem_ld32_sync(tS + cb, x);
      if (seen_warp < cb + 32) {
#pragma unroll
        for (int c = 0; c < 32; ++c) x[c] = cb + c < seen ? x[c] : 0xFF800000u;
      }
    };
    float mx = -INFINITY;
#pragma unroll 1
    for (int cb = 0; cb < most; cb += 32) {
      uint32_t x[32];
      scores(cb, x);
      mx = fmaxf(mx, scores_max<32>(x));
    }
    mx *= scale_log2;
    if (!prior()) return false;
    if (fresh) row.m_use = mx;
    else if (__any_sync(0xffffffffu, mx > row.m_use + 8.f)) move_offset(mx);
    const float off = offset();
    // (d = 128: the weights of 32 keys overwrite scores of keys before them, which are read)
#pragma unroll 1
    for (int cb = 0; cb < 128; cb += 32) {
      uint32_t x[32];
      if (cb < most) {
        scores(cb, x);
      } else {
#pragma unroll
        for (int c = 0; c < 32; ++c) x[c] = 0xFF800000u;
      }
      if (kOwnWeights<D> && cb == 96) {
        tc_fence_before();
        mbar_arrive(s_free);
      }
      weights32<BF16, 0>(x, tP + (cb >> 1), scale_log2, off, row.lsum);
    }
    return true;
  }
  uint32_t x[128];
  tmem_ld64_sync(tS + 0, *reinterpret_cast<uint32_t(*)[64]>(x + 0));
  tmem_ld64_sync(tS + 64, *reinterpret_cast<uint32_t(*)[64]>(x + 64));
  if constexpr (kOwnWeights<D>) {
    tc_fence_before();
    mbar_arrive(s_free);
  }
  if (!prior()) return false;
  // The offset hardly ever moves after the first tiles: the first 64 weights are taken at the old one while the
  // maximum is found beside them, and taken again if it did move.
  float2 sum[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) sum[i] = row.lsum[i];
  float off = offset();
  weights32<BF16, 8>(x, tP, scale_log2, off, sum);
  weights32<BF16, 8>(x + 32, tP + 16, scale_log2, off, sum);
  const float mx = scores_max<128>(x) * scale_log2;
  if (__any_sync(0xffffffffu, mx > row.m_use + 8.f)) {
    move_offset(mx);
    off = offset();
#pragma unroll
    for (int i = 0; i < 4; ++i) sum[i] = row.lsum[i];
    weights32<BF16, 0>(x, tP, scale_log2, off, sum);
    weights32<BF16, 0>(x + 32, tP + 16, scale_log2, off, sum);
  }
  weights32<BF16, 8>(x + 64, tP + 32, scale_log2, off, sum);
  weights32<BF16, 8>(x + 96, tP + 48, scale_log2, off, sum);
#pragma unroll
  for (int i = 0; i < 4; ++i) row.lsum[i] = sum[i];
  return true;
}

// V rows [valid, 128) of a tile (boxes of 128 rows of 128 bytes) to zero, by one warp: keys past the
// sequence's end have no weight, but what stands in their rows (stale or unwritten memory) may be NaN or
// infinite, and the product would carry that on.
template <int D>
__device__ __forceinline__ void zero_v_tail(uint8_t* v_tile, int valid, int lane) {
#pragma unroll
  for (int c = 0; c < D / 64; ++c)
    for (int at = valid * 128 + lane * 16; at < 128 * 128; at += 512)
      *reinterpret_cast<uint4*>(v_tile + c * (128 * 128) + at) = make_uint4(0, 0, 0, 0);
  fence_proxy_async_shared();
  __syncwarp();
}

}  // namespace sage
