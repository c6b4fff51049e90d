// attn_step_kernels.cu -- 16-bit attention of few query rows (single tokens, very short chunks) over many
// keys: paged or strided keys, grouped heads.
//
// Mathematics: as attn_pair_kernels.cu (online softmax in log2 units), with each weight p = 2^(u - m) split into
// two 16-bit parts, p = hi + lo, and two products: the matrix instructions take 16-bit operands, they
// are far from busy here, and the weights then carry about twice the operand type's bits.
//
// Bound: device memory.  Each key and value is read once and meets at most 16 rows (the query heads of a
// group, times a few tokens), so what counts is bytes in flight and no idle SM:
//   - All key tiles (128 keys) of all (sequence, token tile, key head) items form one axis that is cut into
//     equal shares, two per SM, whatever the lengths are; each CTA finds its share from the lengths on the
//     device and walks through it.  An item that a cut goes through is joined from its parts
//     (attn_step_join_kernel).
//   - The products are taken transposed, with the keys on the tensor memory's 128 lanes and the 16 rows as
//     the narrow side: S^T = K Q^T (N = 16) and O^T = V^T P^T (N = 32: the columns of hi, then of lo), so
//     that a tile costs 16 short MMAs and a thread computes the few weights of one key.  With the rows on
//     the lanes 112 of them would idle in the products and, worse, in the softmax: measured 125 us in this
//     kernel's frame against 97 us for a token of 32 heads over 131072 keys of 8 heads of 128 channels, both with the
//     joining (86 us of it this kernel, 6.2 TB/s); 48 tokens over 5300 keys each on average take 163 us, 6.3 TB/s.
//   - A row's offset is common to all lanes; it is taken from the first tile and moves only when a lane sees
//     a score 8 above it (one vote per tile), so no tile but the first needs a maximum over lanes.
//
// CTA: 192 threads, two per SM.  Warps 0-3: softmax (thread = key of the tile = TMEM lane) and output
// (thread = channel), warp 4: MMA issuer (and TMEM: S^T of two tiles [0, 32), O^T [32, 64)), warp 5: TMA, Q and
// the ring of K and V tiles, filled across the items' borders.
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <cstdint>
#include <type_traits>

#include "attn16_device.cuh"
#include "attn16_kernels.cuh"
#include "attn16_softmax.cuh"
#include "attn_common.cuh"
#include "sm100_ptx.cuh"
#include "workspace.cuh"

namespace sage {
namespace {

constexpr int kUnit = 128;     // keys per unit: one tile
constexpr int kWarps = 6;
constexpr int kThreads = 32 * kWarps;
constexpr int kMinShare = 1;   // units per CTA at least
constexpr int R = kStepRows;

template <int D>
struct StepLayout {
  static constexpr int BOX = 128 * 128;         // 128 keys of 64 channels (128-byte rows)
  static constexpr int TILE = BOX * (D / 64);
  static constexpr int NS = D == 128 ? 3 : 5;   // ring stages: K0 V0 K1 ...
  static constexpr int Q_BOX = R * 128;         // 16 rows of 64 channels
  static constexpr int P_ATOM = 2 * R * 128;    // 64 keys of hi (16 rows), then lo
  static constexpr int OFF_RING = 0;
  static constexpr int OFF_Q = NS * TILE;
  static constexpr int OFF_P = OFF_Q + Q_BOX * (D / 64);
  static constexpr int OFF_RED = OFF_P + 2 * P_ATOM;  // [4 warps][16 rows] fp32
  static constexpr int OFF_BAR = OFF_RED + 4 * R * 4;
  static constexpr int NUM_BARS = 2 * NS + 7;
  static constexpr int OFF_MISC = OFF_BAR + NUM_BARS * 8;
  // d = 64: the V^T operand is 128 rows high, its upper 64 rows are whatever the 16 KB behind the tile hold
  // (their products land in lanes that are not read)
  static constexpr int USED = OFF_MISC + 16;
  static constexpr int SMEM = (D == 64 && USED < OFF_Q + BOX ? OFF_Q + BOX : USED) + 1024;
  static_assert(2 * (SMEM + 2048) <= 228 * 1024, "two CTAs per SM");
};

// (p0, p1) -> the 16-bit pair nearest to them, and the pair nearest to what is left
template <bool BF16>
__device__ __forceinline__ void split16(float2 p, uint32_t& hi, uint32_t& lo) {
  hi = pack16<BF16>(p.x, p.y);
  float2 f;
  if constexpr (BF16) {
    f = make_float2(__uint_as_float(hi << 16), __uint_as_float(hi & 0xffff0000u));
  } else {
    f = __half22float2(*reinterpret_cast<const __half2*>(&hi));
  }
  f = __fadd2_rn(p, make_float2(-f.x, -f.y));
  lo = pack16<BF16>(f.x, f.y);
}

// ---- the axis of units: sequence b has items(b) items (token tile, key head) of units(b) units each
struct Items {
  Sequence seq;
  int items, units;
};
__device__ __forceinline__ Items items_of(const StepArgs& s, int b) {
  Items r;
  r.seq = sequence(s.a, b);
  r.items = (r.seq.nq + s.tile_tokens - 1) / s.tile_tokens * s.a.Hk;
  r.units = max(1, (r.seq.kv + kUnit - 1) / kUnit);
  return r;
}
__device__ __forceinline__ long long length_of(const Items& r) { return static_cast<long long>(r.items) * r.units; }

// a / b for a >= 0, b > 0; by the short division where it fits
__device__ __forceinline__ long long quotient(long long a, int b) {
  return a >> 32 == 0 ? static_cast<unsigned>(a) / static_cast<unsigned>(b) : a / b;
}

__device__ __forceinline__ long long share_of(long long total, int ctas) {
  const long long even = quotient(total + ctas - 1, ctas);
  return even > kMinShare ? even : kMinShare;
}

// Barrier of the 128 softmax threads, counted per thread.
__device__ __forceinline__ void group_sync() { asm volatile("barrier.sync 1, 128;" ::: "memory"); }
// Whether p holds in any of them; a barrier too.
__device__ __forceinline__ bool group_any(bool p) {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t"
      "setp.ne.u32 p, %1, 0;\n\t"
      "barrier.red.or.pred q, 1, 128, p;\n\t"
      "selp.u32 %0, 1, 0, q;\n\t}"
      : "=r"(r)
      : "r"(p ? 1u : 0u)
      : "memory");
  return r != 0;
}
__device__ __forceinline__ void st_shared_u16(uint32_t addr, uint32_t v) {
  asm volatile("st.shared.u16 [%0], %1;" ::"r"(addr), "h"(static_cast<uint16_t>(v)) : "memory");
}

// The largest of a warp's values, in every lane.
__device__ __forceinline__ float warp_max(float v) {
  float r;
  asm volatile("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(r) : "f"(v));
  return r;
}

// One item's part of a share: key tiles [first, last) of it.
struct Segment {
  Sequence seq;
  int tok0, hk, first, last, part;
  bool whole;
};

// A CTA's walk through its share; every warp takes it for itself, with the same result.
struct Walk {
  long long u, end, prefix;
  int b;
  Items it;
  bool first_item = true;
  __device__ __forceinline__ bool next(const StepArgs& s, Segment& g) {
    if (u >= end) return false;
    while (u >= prefix + length_of(it)) {  // u < end <= the axis' length: there is such a sequence
      prefix += length_of(it);
      it = items_of(s, ++b);
    }
    const long long at = u - prefix;
    const int item = static_cast<int>(quotient(at, it.units));
    g.first = static_cast<int>(at - static_cast<long long>(item) * it.units);
    g.last = static_cast<int>(min(static_cast<long long>(it.units), g.first + (end - u)));
    g.whole = g.first == 0 && g.last == it.units;
    g.tok0 = item / s.a.Hk * s.tile_tokens;
    g.hk = item % s.a.Hk;
    g.seq = it.seq;
    g.part = 2 * static_cast<int>(blockIdx.x) + (first_item ? 0 : 1);  // at most two: of the first item and the last
    u += g.last - g.first;
    if (g.seq.kv == 0) g.last = g.first;  // nothing to read: the rows are 0
    first_item = false;
    return true;
  }
};

template <int D, bool BF16>
__global__ void __launch_bounds__(kThreads, 2)
    attn_step_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
                     const __grid_constant__ CUtensorMap tm_v, const __grid_constant__ StepArgs s) {
  using L = StepLayout<D>;
  constexpr int NS = L::NS, NB = D / 64;
  const Attn16Args& a = s.a;
  extern __shared__ uint8_t smem_raw[];
  __shared__ long long scratch[kWarps];
  __shared__ long long found_prefix;
  __shared__ int found_b;
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* sQ = smem + L::OFF_Q;
  uint8_t* sRing = smem + L::OFF_RING;
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + L::OFF_BAR);
  uint64_t* bar_full = bars;
  uint64_t* bar_empty = bar_full + NS;
  uint64_t* bar_q_full = bar_empty + NS;
  uint64_t* bar_q_free = bar_q_full + 1;  // the item's last K Q^T is done
  uint64_t* bar_s_full = bar_q_full + 2;  // [2] S^T of a tile (in buffer tile & 1)
  uint64_t* bar_p_full = bar_q_full + 4;  // the tile's weights are in shared memory
  uint64_t* bar_pv = bar_q_full + 5;      // the tile's V^T P^T is done
  uint64_t* bar_drain = bar_q_full + 6;
  uint8_t* sP = smem + L::OFF_P;
  float* sRed = reinterpret_cast<float*>(smem + L::OFF_RED);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + L::OFF_MISC);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + L::OFF_MISC + 4);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  // ---- this CTA's share of the units, and the sequence in which it begins: a scan over the sequences' lengths,
  // kThreads at a time (twice when there are more)
  Walk walk;
  long long share = 0;
  {
    long long before = 0, len = 0, incl = 0;
    auto scan = [&](int base) {  // incl: length up to this thread's sequence, before: of all so far
      const int b = base + static_cast<int>(threadIdx.x);
      len = b < a.B ? length_of(items_of(s, b)) : 0;
      incl = len;
#pragma unroll
      for (int off = 1; off < 32; off <<= 1) {
        const long long v = __shfl_up_sync(0xffffffffu, incl, off);
        if (lane >= off) incl += v;
      }
      __syncthreads();
      if (lane == 31) scratch[warp] = incl;
      __syncthreads();
      incl += before;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) {
        const long long v = scratch[w];
        if (w < warp) incl += v;
        before += v;
      }
    };
    for (int base = 0; base < a.B; base += kThreads) scan(base);
    const long long total = before;
    share = share_of(total, gridDim.x);
    walk.u = blockIdx.x * share;
    walk.end = min(total, walk.u + share);
    if (walk.u >= walk.end) {
      if (threadIdx.x == 0 && a.cuts) a.cuts[blockIdx.x] = CutNote{};  // no cut
      return;
    }
    if (a.B > kThreads) before = 0;
    for (int base = 0; base < a.B; base += kThreads) {
      if (a.B > kThreads) scan(base);
      if (walk.u >= incl - len && walk.u < incl) {
        found_b = base + static_cast<int>(threadIdx.x);
        found_prefix = incl - len;
      }
    }
  }

  if (threadIdx.x == 0) {
    for (int i = 0; i < NS; ++i) {
      mbar_init(bar_full + i, 1);
      mbar_init(bar_empty + i, 1);
    }
    mbar_init(bar_q_full, 1);
    mbar_init(bar_q_free, 1);
    mbar_init(bar_s_full, 1);
    mbar_init(bar_s_full + 1, 1);
    mbar_init(bar_p_full, 128);
    mbar_init(bar_pv, 1);
    mbar_init(bar_drain, 1);
    *abort_flag = 0;
    fence_barrier_init();
    tma_prefetch_desc(&tm_q);
    tma_prefetch_desc(&tm_k);
    tma_prefetch_desc(&tm_v);
  }
  if (warp == 4) {
    tmem_alloc(tmem_slot, 64);
    tmem_relinquish();
  }
  tc_fence_before();
  cta_sync();  // lane 0 of warp 0 initialised the barriers alone; found_b is written
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  walk.b = found_b;
  walk.prefix = found_prefix;
  walk.it = items_of(s, walk.b);
  if (threadIdx.x == 0 && a.cuts) {
    const long long at = walk.u - walk.prefix;
    const int item = static_cast<int>(quotient(at, walk.it.units));
    const int off = static_cast<int>(at - static_cast<long long>(item) * walk.it.units);
    a.cuts[blockIdx.x] = CutNote{walk.u - off, share, walk.b, walk.it.seq.token0, walk.it.seq.nq,
                                 item / a.Hk * s.tile_tokens, item % a.Hk, off, walk.it.units};
  }
  Segment seg;
  auto wait = [&](uint64_t* bar, uint32_t parity) {
    return __all_sync(0xffffffffu, mbar_wait(bar, parity, abort_flag));
  };

  if (warp == 5) {
    // ============================================================ TMA: Q of each item, K and V tiles (lane i:
    // the tile's page i).  A later item's Q is asked for behind its first K and V: its buffer is free only when
    // the item before it has used it, and the ring goes on meanwhile.
    const int page = 1 << a.page_shift;
    const int pages_per_tile = a.page_table && page < 128 ? 128 >> a.page_shift : 1;
    const int rows_per_copy = 128 / pages_per_tile;
    int fill = 0, n = 0, q_asked = 0;
    bool ok = true;
    while (ok && walk.next(s, seg)) {
      // (outer coordinate) of this lane's copy of key tile kt; pages past the sequence or outside the
      // cache take a coordinate past the tensor, which reads as zeros and counts its bytes
      auto page_of = [&](int kt) -> int {
        if (!a.page_table) return seg.seq.b;
        const int key = kt * 128 + lane * rows_per_copy;
        int p = -1;
        if (lane < pages_per_tile && key < seg.seq.kv)
          p = __ldg(a.page_table + static_cast<long long>(seg.seq.b) * a.pages_per_seq + (key >> a.page_shift));
        return p < 0 || p >= a.num_pages ? a.num_pages : p;
      };
      auto load_q = [&]() -> bool {
        if (n > 0 && !wait(bar_q_free, (n - 1) & 1)) return false;
        if (lane == 0) {
          mbar_arrive_expect_tx(bar_q_full, static_cast<uint32_t>(s.tile_tokens * a.G * NB * 128));
          for (int c = 0; c < NB; ++c)
            tma_load_5d(sQ + c * L::Q_BOX, &tm_q, bar_q_full, 64 * c, 0, seg.seq.token0 + seg.tok0, seg.hk,
                        a.cu_q ? 0 : seg.seq.b);
        }
        __syncwarp();
        q_asked = n + 1;
        return true;
      };
      int outer = seg.first < seg.last ? page_of(seg.first) : 0;
      if (seg.first < seg.last && n == 0) load_q();
      for (int kt = seg.first; ok && kt < seg.last; ++kt) {
        const int next = kt + 1 < seg.last ? page_of(kt + 1) : 0;  // in flight during this tile's waits
        const int row = a.page_table ? (kt * 128) & (page - 1) : kt * 128;
        for (int kind = 0; kind < 2; ++kind, ++fill) {
          const int st = fill % NS;
          if (fill >= NS && !wait(bar_empty + st, (fill / NS - 1) & 1)) {
            ok = false;
            break;
          }
          if (lane == 0) mbar_arrive_expect_tx(bar_full + st, L::TILE);
          __syncwarp();
          if (lane < pages_per_tile) {
            uint8_t* dst = sRing + st * L::TILE + lane * rows_per_copy * 128;
            const CUtensorMap* map = kind == 0 ? &tm_k : &tm_v;
#pragma unroll
            for (int c = 0; c < NB; ++c)
              tma_load_4d(dst + c * L::BOX, map, bar_full + st, 64 * c, pages_per_tile > 1 ? 0 : row, seg.hk, outer);
          }
          __syncwarp();
        }
        outer = next;
        if (ok && kt == seg.first && n > 0) ok = load_q();
      }
      if (seg.first < seg.last) ++n;
    }
    if (*abort_flag && lane == 0) {  // let copies in flight land before the CTA exits
      for (int f = max(0, fill - NS); f < fill; ++f) mbar_drain(bar_full + f % NS, (f / NS) & 1);
      if (q_asked > 0) mbar_drain(bar_q_full, (q_asked - 1) & 1);
    }
  } else if (warp == 4) {
    // ============================================================ MMA issuer
    constexpr uint32_t FMT = BF16 ? 1u : 0u;
    constexpr uint32_t IDESC_QK = make_idesc(1 /*f32*/, FMT, FMT, 0, 0, 128, R);
    constexpr uint32_t IDESC_PV = make_idesc(1 /*f32*/, FMT, FMT, 1 /*V^T is MN-major*/, 0, 128, 2 * R);
    const uint32_t q_base = smem_u32(sQ), ring = smem_u32(sRing), p_base = smem_u32(sP);
    int n = 0, fill = 0, tile = 0;  // fill: of the item's next K that has not been used
    auto full = [&](int f) { return wait(bar_full + f % NS, (f / NS) & 1); };
    auto issue_qk = [&](int f, int buf) {
      const uint32_t k_base = ring + (f % NS) * L::TILE;
#pragma unroll
      for (int c = 0; c < NB; ++c)  // 16 channels per product: 32 bytes inside a 128-byte swizzled row
        mma_f16_ss_x4_warp<2, 2>(tmem + R * buf, make_smem_desc(k_base + c * L::BOX, 16, 1024, kSwizzle128B),
                                 make_smem_desc(q_base + c * L::Q_BOX, 16, 1024, kSwizzle128B), IDESC_QK, c > 0 ? 1u : 0u);
      mma_commit_warp(bar_empty + f % NS);
      mma_commit_warp(bar_s_full + buf);
    };
    bool ok = true;
    while (ok && walk.next(s, seg)) {
      if (seg.first == seg.last) continue;
      ok = full(fill) && wait(bar_q_full, n & 1);
      ++n;
      if (!ok) break;
      tc_fence_after();
      issue_qk(fill, tile & 1);
      for (int kt = seg.first; ok && kt < seg.last; ++kt, ++tile, fill += 2) {
        // the next tile's scores first: their buffer was read before the weights of the tile before this
        // one were written, which this warp has waited for
        if (kt + 1 < seg.last) {
          if (!full(fill + 2)) { ok = false; break; }
          tc_fence_after();
          issue_qk(fill + 2, (tile + 1) & 1);
        } else {
          mma_commit_warp(bar_q_free);
        }
        if (!full(fill + 1)) { ok = false; break; }
        const int st = (fill + 1) % NS;
        // keys past the sequence's end have no weight, but what stands in their rows (stale or unwritten
        // memory) may be NaN or infinite: zero those V rows before the product reads them
        const int valid = seg.seq.kv - kt * 128;
        if (valid < 128) {
          zero_v_tail<D>(sRing + st * L::TILE, valid, lane);
        }
        if (!wait(bar_p_full, tile & 1)) { ok = false; break; }
        tc_fence_after();
#pragma unroll
        for (int half = 0; half < 2; ++half)  // 16 keys per product: 16 rows of the V tile, 32 bytes of a weight row
          mma_f16_ss_x4_warp<16 * 128 / 16, 2>(tmem + 2 * R, make_smem_desc(ring + st * L::TILE + half * 64 * 128, L::BOX, 1024, kSwizzle128B),
                                               make_smem_desc(p_base + half * L::P_ATOM, 16, 1024, kSwizzle128B), IDESC_PV,
                                               kt == seg.first && half == 0 ? 0u : 1u);
        mma_commit_warp(bar_empty + st);
        mma_commit_warp(bar_pv);
      }
    }
    // all MMAs must finish before TMEM is released
    mma_commit_warp(bar_drain);
    mbar_drain(bar_drain, 0);
  } else {
    // ============================================================ softmax: thread = key, output: thread = channel
    constexpr float kShift = BF16 ? 0.f : 7.f;  // fp16: small weights keep their bits (2^8 * 2^7 fits)
    const int c = threadIdx.x;
    const uint32_t lanes = tmem + (static_cast<uint32_t>(warp * 32) << 16);
    const uint32_t p_key = smem_u32(sP) + (c >> 6) * L::P_ATOM + (c & 7) * 2;  // this key's place in a weight row
    const uint32_t chunk = (c & 63) >> 3;
    // The 128 threads meet at barriers; a warp whose bounded wait gave up goes on taking part until the next
    // tile's vote, where all four warps leave together, so that none is left at a barrier.
    bool ok = true, stop = false;
    int tile = 0;
    while (walk.next(s, seg)) {
      const int rows = min(s.tile_tokens, seg.seq.nq - seg.tok0) * a.G;
      const int lim_min = visible(a, seg.seq, seg.tok0);  // the item's first token sees the fewest keys
      float m[R], l[R];
#pragma unroll
      for (int r = 0; r < R; ++r) m[r] = -INFINITY, l[r] = 0.f;
      for (int kt = seg.first; kt < seg.last; ++kt, ++tile) {
        ok = ok && wait(bar_s_full + (tile & 1), (tile >> 1) & 1);
        tc_fence_after();
        uint32_t xr[R];
        tmem_ld16_sync(lanes + R * (tile & 1), xr);
        float x[R];
#pragma unroll
        for (int r = 0; r < R; ++r) x[r] = __uint_as_float(xr[r]) * a.scale_log2;
        const int key = kt * 128 + c;
        if (kt * 128 + 128 > lim_min) {
          int tok = seg.tok0, h = 0;
#pragma unroll
          for (int r = 0; r < R; ++r) {
            if (key >= visible(a, seg.seq, tok)) x[r] = -INFINITY;
            if (++h == a.G) h = 0, ++tok;
          }
        }
        bool over = kt == seg.first;
#pragma unroll
        for (int r = 0; r < R; ++r) over |= r < rows && x[r] > m[r] + 8.f;
        if (group_any(over || !ok)) {
          if (group_any(!ok)) {
            stop = true;
            break;
          }
          // ---- new offsets: maxima over the tile's keys
          // (rows in fours, without a branch per row, so that their loads and maxima overlap; rows past `rows`
          // compute on whatever there is)
          float4* red4 = reinterpret_cast<float4*>(sRed);  // [4 warps][rows / 4]
#pragma unroll
          for (int r = 0; r < R; r += 4) {
            if (r < rows) {
              const float4 v = make_float4(warp_max(x[r]), warp_max(x[r + 1]), warp_max(x[r + 2]), warp_max(x[r + 3]));
              if (lane == 0) red4[(warp * R + r) / 4] = v;
            }
          }
          group_sync();
          float f[R];
          bool moved = false;
#pragma unroll
          for (int r = 0; r < R; r += 4) {
            f[r] = f[r + 1] = f[r + 2] = f[r + 3] = 1.f;
            if (r < rows) {
              const float4 v0 = red4[r / 4], v1 = red4[(R + r) / 4], v2 = red4[(2 * R + r) / 4], v3 = red4[(3 * R + r) / 4];
              const float v[4] = {fmaxf(fmaxf(v0.x, v1.x), fmaxf(v2.x, v3.x)), fmaxf(fmaxf(v0.y, v1.y), fmaxf(v2.y, v3.y)),
                                  fmaxf(fmaxf(v0.z, v1.z), fmaxf(v2.z, v3.z)), fmaxf(fmaxf(v0.w, v1.w), fmaxf(v2.w, v3.w))};
#pragma unroll
              for (int k = 0; k < 4; ++k) {
                const bool move = v[k] > m[r + k] + 8.f;  // also the first finite maximum
                f[r + k] = move ? fast_exp2(m[r + k] - v[k]) : 1.f;
                m[r + k] = move ? v[k] : m[r + k];
                l[r + k] *= f[r + k];
                moved |= move;
              }
            }
          }
          group_sync();  // sRed is read
          if (moved && kt > seg.first) {  // the same in every thread
            ok = wait(bar_pv, (tile - 1) & 1) && ok;  // O^T is complete up to the tile before
            tc_fence_after();
#pragma unroll
            for (int part = 0; part < 2; ++part) {
              uint32_t o[R];
              tmem_ld16_sync(lanes + 2 * R + R * part, o);
#pragma unroll
              for (int r = 0; r < R; ++r) o[r] = __float_as_uint(__uint_as_float(o[r]) * f[r]);
              tmem_st16(lanes + 2 * R + R * part, o);
            }
            tmem_wait_st();
          }
        }
        // ---- weights: hi and lo into the two atoms (the product of the tile before has read them)
        uint32_t hi[R / 2], lo[R / 2];
#pragma unroll
        for (int g = 0; g < R; g += 4) {
          if (g < rows) {
#pragma unroll
            for (int r = g; r < g + 4; r += 2) {
              const float2 p = make_float2(fast_exp2(x[r] + (kShift - (m[r] == -INFINITY ? 0.f : m[r]))),
                                           fast_exp2(x[r + 1] + (kShift - (m[r + 1] == -INFINITY ? 0.f : m[r + 1]))));
              l[r] += p.x;
              l[r + 1] += p.y;
              split16<BF16>(p, hi[r / 2], lo[r / 2]);
            }
          }
        }
        if (tile > 0) ok = wait(bar_pv, (tile - 1) & 1) && ok;
#pragma unroll
        for (int g = 0; g < R; g += 4) {
          if (g < rows) {
#pragma unroll
            for (int r = g; r < g + 4; r += 2) {
              const uint32_t p0 = p_key + r * 128 + ((chunk ^ (r & 7)) << 4), p1 = p_key + (r + 1) * 128 + ((chunk ^ ((r + 1) & 7)) << 4);
              st_shared_u16(p0, hi[r / 2]);
              st_shared_u16(p1, hi[r / 2] >> 16);
              st_shared_u16(p0 + R * 128, lo[r / 2]);
              st_shared_u16(p1 + R * 128, lo[r / 2] >> 16);
            }
          }
        }
        fence_proxy_async_shared();
        tc_fence_before();
        mbar_arrive(bar_p_full);
      }
      if (stop) break;
      // ---- row sums over the 128 keys' threads (through the weights' memory, whose product is done), then the
      // output of the item or its part
      const bool some = seg.first < seg.last;
      if (some) ok = wait(bar_pv, (tile - 1) & 1) && ok;
      tc_fence_after();
      float* sums = reinterpret_cast<float*>(sP);  // [row][key]
      static_assert(R * 128 * 4 <= 2 * L::P_ATOM, "a row's 128 partial sums fit the weights' memory");
#pragma unroll
      for (int g = 0; g < R; g += 4) {
        if (g < rows) {
#pragma unroll
          for (int r = g; r < g + 4; ++r) sums[r * 128 + c] = l[r];
        }
      }
      uint32_t o[2 * R];
      if (some) {
        tmem_ld32_sync(lanes + 2 * R, o);
      } else {
#pragma unroll
        for (int r = 0; r < 2 * R; ++r) o[r] = 0u;
      }
      group_sync();
      for (int r = warp; r < rows; r += 4) {
        const float4 y = *reinterpret_cast<const float4*>(sums + r * 128 + 4 * lane);
        float v = (y.x + y.y) + (y.z + y.w);
#pragma unroll
        for (int off = 16; off > 0; off >>= 1) v += __shfl_xor_sync(0xffffffffu, v, off);
        if (lane == 0) sRed[r] = seg.whole ? weight_sum_inverse(v) : v;
      }
      group_sync();
      if (c < D && ok && !*abort_flag) {
        uint16_t* dst = static_cast<uint16_t*>(a.o) + out_offset(a, seg.seq, seg.tok0, seg.hk * a.G) + c;
        const long long next_token = a.o_sn - (a.G - 1) * a.o_sh;
        float* part = a.part_o + static_cast<long long>(seg.part) * R * D + c;
        int h = 0;
#pragma unroll
        for (int g = 0; g < R; g += 4) {
          if (g < rows) {
            const float4 y = *reinterpret_cast<const float4*>(sRed + g);
            const float sum[4] = {y.x, y.y, y.z, y.w};
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              const int r = g + k;
              const float acc = __uint_as_float(o[r]) + __uint_as_float(o[R + r]);
              if (seg.whole) {
                if (r < rows) *dst = static_cast<uint16_t>(pack16<BF16>(acc * sum[k], 0.f));
              } else if (r < rows) {
                part[r * D] = acc;
                if (c == 0) a.part_ml[seg.part * R + r] = make_float2(m[r], sum[k]);
              }
              const bool wrap = ++h == a.G;
              dst += wrap ? next_token : a.o_sh;
              h = wrap ? 0 : h;
            }
          }
        }
      }
      group_sync();  // sRed and the sums are read; O^T too: the arrivals of the next item's weights order what follows
      tc_fence_before();
    }
  }

  // roles diverge inside warps (single-lane producers): the thread-counting barrier holds the TMEM
  // release until every thread of the CTA is done
  tc_fence_before();
  cta_sync();
  if (warp == 4) {
    tc_fence_after();
    tmem_dealloc(tmem, 64);
  }
}

// Joins the items that a cut went through, in the order of their parts.  One CTA per cut between two shares, a
// warp per row; an item that more than one cut goes through is joined by its first one.
constexpr int kJoinThreads = 32 * R;

template <int D, bool BF16>
__global__ void __launch_bounds__(kJoinThreads) attn_step_join_kernel(const __grid_constant__ StepArgs s) {
  const Attn16Args& a = s.a;
  const int r = static_cast<int>(threadIdx.x >> 5), lane = threadIdx.x & 31;
  cudaGridDependencySynchronize();  // the parts are written
  const CutNote cut = a.cuts[blockIdx.x + 1];
  if (cut.off == 0) return;  // no such share, or it begins with an item
  const int c0 = static_cast<int>(cut.first / cut.share), c1 = static_cast<int>((cut.first + cut.units - 1) / cut.share);
  if (c0 != static_cast<int>(blockIdx.x)) return;
  // in its first CTA the item is the last one (part 1) unless the CTA begins with it
  const bool late = cut.first % cut.share != 0;
  const int tok = cut.tok0 + r / a.G;
  if (r >= s.tile_tokens * a.G || tok >= cut.nq) return;
  constexpr int C = D / 32;  // channels per lane
  float acc[1][C], l[1];
  join_parts(acc, l, c0, c1, a.part_ml, a.part_o,
             [&](int, int c) { return static_cast<long long>(2 * c + (c == c0 && late ? 1 : 0)) * R + r; });
  store_joined<BF16>(static_cast<uint16_t*>(a.o) + lane * C +
                         out_offset(a, Sequence{cut.b, cut.token0, cut.nq, 0}, tok, cut.hk * a.G + r % a.G),
                     acc[0], l[0]);
}

template <int D, bool BF16>
cudaError_t launch_step_t(const StepLaunch& l, int ctas, cudaStream_t st) {
  const StepArgs& s = l.s;
  using L = StepLayout<D>;
  auto kern = attn_step_kernel<D, BF16>;
  static std::atomic<unsigned long long> allowed{0};
  cudaError_t e = allow_shared_memory(allowed, reinterpret_cast<const void*>(kern), L::SMEM);
  if (e != cudaSuccess) return e;
  kern<<<ctas, kThreads, L::SMEM, st>>>(l.tm_q, l.tm_k, l.tm_v, s);
  e = cudaGetLastError();
  if (e != cudaSuccess || ctas == 1) return e;
  // launched early, while the attention drains: it waits on the device for the parts
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(static_cast<unsigned>(ctas) - 1);
  cfg.blockDim = dim3(kJoinThreads);
  cfg.stream = st;
  cudaLaunchAttribute attr{};
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, attn_step_join_kernel<D, BF16>, s);
}

}  // namespace

int step_ctas(const StepArgs& s, int sms) {
  // two CTAs per SM; fewer when the whole axis, at its longest, has not kMinShare units for each
  const long long tiles = (s.a.Nq + s.tile_tokens - 1) / s.tile_tokens;
  const long long items = s.a.cu_q ? (tiles + s.a.B) * s.a.Hk : tiles * s.a.B * s.a.Hk;
  const long long units = s.a.Nk > kUnit ? (s.a.Nk + kUnit - 1ll) / kUnit : 1;
  const long long most = (items * units + kMinShare - 1) / kMinShare;
  return static_cast<int>(most < 2ll * sms ? most : 2ll * sms);
}

size_t step_part_rows(int ctas) { return static_cast<size_t>(ctas) * 2 * R; }

cudaError_t launch_attn_step(const StepLaunch& l, int ctas, cudaStream_t st) {
  if (l.D == 128) return l.bf16 ? launch_step_t<128, true>(l, ctas, st) : launch_step_t<128, false>(l, ctas, st);
  return l.bf16 ? launch_step_t<64, true>(l, ctas, st) : launch_step_t<64, false>(l, ctas, st);
}

int read_and_clear_step_error(cudaStream_t st, cudaError_t* err) {
  *err = cudaStreamSynchronize(st);
  if (*err != cudaSuccess) return -1;
  int h = 0;
  *err = cudaMemcpyFromSymbol(&h, g_device_error, sizeof(int));
  if (*err != cudaSuccess) return -1;
  const int zero = 0;
  *err = cudaMemcpyToSymbol(g_device_error, &zero, sizeof(int));
  return *err == cudaSuccess ? h : -1;
}

}  // namespace sage
