// attn_common.cuh -- device helpers shared by the attention kernels: exp2 on either pipe, packing,
// register redistribution between warpgroups, the exit paths' bounded wait.
#pragma once
#include <cuda_fp16.h>
#include <cstdint>

#include "sm100_ptx.cuh"

namespace sage {

__device__ __forceinline__ float fast_exp2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

__device__ __forceinline__ float fast_log2(float x) {
  float y;
  asm("lg2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

__device__ __forceinline__ uint32_t pack_half2(float lo, float hi) {
  const __half2 h = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}

// Magic-number integer -> float: for |S| < 2^22 the bits of S + 0x4B400000 are the float
// 1.5 * 2^23 + S exactly.
constexpr uint32_t kMagicBits = 0x4B400000u;
constexpr float kMagicF = 12582912.0f;

__device__ __forceinline__ float max3f(float a, float b, float c) {
  float r;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}

// The larger of two, NaN if one of them is.
__device__ __forceinline__ float max_nan(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}

// exp2 on the FMA pipe for a pair of arguments (Cody-Waite style range reduction plus a
// polynomial), to take part of the exp2 work off the MUFU unit:
//   t -> max(t, -126); n = round_to_nearest(t) via the 1.5 * 2^23 add; f = t - n in [-1/2, 1/2];
//   2^f ~ c0 + c1 f + c2 f^2 + c3 f^3 with coefficients fitted here to the minimax relative error on
//   [-1/2, 1/2] (max relative error 7.5e-5, below half an fp16 ulp); 2^n by adding n to the
//   exponent field (n << 23, taken from the low bits of the magic sum).
// exp2_poly2_above: for arguments of -126 at least (a NaN gives some number).
__device__ __forceinline__ float2 exp2_poly2_above(float2 t) {
  constexpr float c0 = 0.9999281167984009f, c1 = 0.6932609677314758f, c2 = 0.2426108568906784f,
                  c3 = 0.055171459913253784f;
  const float2 y = __fadd2_rn(t, make_float2(kMagicF, kMagicF));
  const float2 n = __fadd2_rn(y, make_float2(-kMagicF, -kMagicF));
  const float2 f = __ffma2_rn(n, make_float2(-1.f, -1.f), t);
  float2 p = __ffma2_rn(f, make_float2(c3, c3), make_float2(c2, c2));
  p = __ffma2_rn(p, f, make_float2(c1, c1));
  p = __ffma2_rn(p, f, make_float2(c0, c0));
  return make_float2(__int_as_float(__float_as_int(p.x) + (__float_as_int(y.x) << 23)),
                     __int_as_float(__float_as_int(p.y) + (__float_as_int(y.y) << 23)));
}

__device__ __forceinline__ float2 exp2_poly2(float2 t) {
  return exp2_poly2_above(make_float2(fmaxf(t.x, -126.f), fmaxf(t.y, -126.f)));
}

template <uint32_t N>
__device__ __forceinline__ void reg_alloc() {
  asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N));
}
template <uint32_t N>
__device__ __forceinline__ void reg_dealloc() {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N));
}

// The bounded wait of a role that runs ahead of the others (loads, bookkeeping): it sleeps between two looks,
// so that it takes no issue slots from the warps that compute.
__device__ __forceinline__ bool mbar_wait_idle(uint64_t* bar, uint32_t parity, volatile int* abort) {
  if (mbar_try_wait(bar, parity)) return true;
  const long long t0 = clock64();
  while (true) {
    __nanosleep(200);
    if (mbar_try_wait(bar, parity)) return true;
    if (*abort) return false;
    if (clock64() - t0 > kWaitLimitCycles) {
      *abort = 1;
      atomicExch(&g_device_error, kDevTimeoutBarrier);
      return false;
    }
  }
}

// Bounded wait used on exit paths: ignores the abort flag, records a timeout.
__device__ __forceinline__ void mbar_drain(uint64_t* bar, uint32_t parity) {
  const long long t0 = clock64();
  while (!mbar_try_wait(bar, parity)) {
    if (clock64() - t0 > kWaitLimitCycles) {
      atomicExch(&g_device_error, kDevTimeoutBarrier);
      return;
    }
  }
}

}  // namespace sage
