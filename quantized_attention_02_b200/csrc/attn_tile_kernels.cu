// attn_tile_kernels.cu -- 16-bit attention for sm_100a behind the paged attention and the cross attention, where a
// sequence has one tile of query rows (17 to 128): short chunks, wide head groups.
//
// Mathematics as attn_pair_kernels.cu.  Bound: device memory at the lower end, the softmax at the upper: what
// counts is that the key axis is read fast, so the CTA's two streams are one query tile with every other
// key tile each, with a ring of their own, and the two (m, l, O) are joined at the end.  As
// pairs of tiles, with one stream in use (replays of a graph, cold L2): 32 rows over 32768 keys of 8 heads of 128 73 us
// instead of 48, 100 rows over 4 x 1500 keys of 16 heads of 64 34 instead of 26, 120 rows over 20 x 3000 keys of 8 heads
// of 128 87 instead of 84.
// Few CTAs: the key axis is cut into parts, joined by attn_tile_join_kernel.  The last of these, 160 CTAs for 148
// SMs, is not cut: its second round holds 12 CTAs (73 us in the profiler, 3.4 TB/s of keys and values; its bytes
// alone would take 37).
//
// CTA: 12 warps, 512 TMEM columns, about 226 KB of shared memory.
//   warp 0      TMA: Q once, then K and V tiles of 128 keys, K0 V0 K1 V1 ... in each stream's ring
//   warp 1      MMA issuer of both streams; allocates TMEM
//   warps 4-7   softmax of stream 0 (thread = query row = TMEM lane), then the output; warps 8-11 of stream 1
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <cstdint>
#include <type_traits>

#include "attn16_device.cuh"
#include "attn16_kernels.cuh"
#include "attn16_softmax.cuh"
#include "workspace.cuh"

namespace sage {
namespace {

constexpr int kThreads = 384;

template <int D>
struct TileLayout {
  static constexpr int BOX = 128 * 128;        // 128 rows of 64 channels (128-byte rows)
  static constexpr int TILE = BOX * (D / 64);  // one Q, K or V tile
  // Stages of each stream's ring.  A stage's barrier only tells one fill from the next (phase parity), so
  // whoever waits for a fill must have waited for the one before it in that stage too: in a ring that both
  // streams drew from by turns, one could take the other's late fill for its own.
  static constexpr int NS = D == 128 ? 3 : 6;
  static constexpr int OFF_Q = 0;
  static constexpr int OFF_RING = TILE;
  static constexpr int OFF_ML = OFF_RING + 2 * NS * TILE;  // [128] (m, l) of stream 1
  static constexpr int OFF_BAR = OFF_ML + 128 * 8;
  static constexpr int NUM_BARS = 1 + 2 * 2 * NS + 4 * 2 + 1;
  static constexpr int OFF_MISC = OFF_BAR + NUM_BARS * 8;
  static constexpr int SMEM = OFF_MISC + 16 + 1024;
  static_assert(SMEM <= 227 * 1024, "shared memory budget");
  static_assert(SMEM > 114 * 1024, "one CTA per SM: each allocates all of TMEM");
  static_assert(128 * D * 4 <= 2 * NS * TILE, "stream 1's O fits the rings");
};

// The part s of a key axis of nt tiles: tiles [first, last); parts = how many of them are used.  The
// same arithmetic in the attention kernel and in the one that joins the parts.
struct KeyRange {
  int first, last, parts;
};
__device__ __forceinline__ KeyRange key_range(int nt, int splits, int min_chunk, int s) {
  const int chunk = max(min_chunk, (nt + splits - 1) / splits);
  KeyRange r;
  r.parts = max(1, (nt + chunk - 1) / chunk);
  r.first = min(nt, s * chunk);
  r.last = min(nt, r.first + chunk);
  return r;
}

// Tile slot -> sequence and first token; some slots have no tile (false).  By a whole warp.
__device__ __forceinline__ bool tile_of_slot(const Attn16Args& a, int slot, Sequence& seq, int& tok0) {
  if (a.cu_q) {
    const int upto = sequences_upto(a, a.tile_tokens, slot);
    if (upto == 0) return false;
    seq = sequence(a, upto - 1);
    tok0 = (slot - (seq.token0 / a.tile_tokens + seq.b)) * a.tile_tokens;
  } else {
    const int per_b = (a.Nq + a.tile_tokens - 1) / a.tile_tokens;
    seq = sequence(a, slot / per_b);
    tok0 = slot % per_b * a.tile_tokens;
  }
  return tok0 >= 0 && tok0 < seq.nq;  // (negative: cu_q is not ascending)
}

template <int D, bool BF16>
__global__ void __launch_bounds__(kThreads, 1)
    attn_tile_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
                  const __grid_constant__ CUtensorMap tm_v, const __grid_constant__ Attn16Args a) {
  using L = TileLayout<D>;
  using C = Columns<D>;
  constexpr int NS = L::NS, NB = D / 64;
  constexpr bool OWN_P = kOwnWeights<D>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* sQ = smem + L::OFF_Q;
  uint8_t* sRing = smem + L::OFF_RING;
  float2* sML = reinterpret_cast<float2*>(smem + L::OFF_ML);
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + L::OFF_BAR);
  uint64_t* bar_q = bars;
  uint64_t* bar_full = bar_q + 1;
  uint64_t* bar_empty = bar_full + 2 * NS;
  uint64_t* bar_s_full = bar_empty + 2 * NS;  // [2] S_t of the next key tile (and every product before it) done
  uint64_t* bar_s_free = bar_s_full + 2;  // [2] S_t is in registers (OWN_P)
  uint64_t* bar_p_full = bar_s_free + 2;  // [2] the tile's weights written
  uint64_t* bar_pv = bar_p_full + 2;      // [2] the tile's second product done (OWN_P; else: the last tile's)
  uint64_t* bar_drain = bar_pv + 2;       // all MMAs done at exit
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + L::OFF_MISC);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + L::OFF_MISC + 4);

  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;

  // ---- work unit: (query tile slot, key part, key head), tiles of one head next to each other (their
  // keys stay in L2), the last (causal: longest) first
  int rest = static_cast<int>(blockIdx.x);
  const int slot = a.slots - 1 - rest % a.slots;
  rest /= a.slots;
  const int split = rest % a.splits;
  const int hk = rest / a.splits;
  Sequence seq;
  int tok0;  // first token (within the sequence) of the CTA
  if (!tile_of_slot(a, slot, seq, tok0)) return;  // a slot without a tile
  const KeyRange range = key_range(key_tiles(a, seq, tok0, a.tile_tokens), a.splits, a.min_chunk, split);
  if (split >= range.parts) return;
  const int n_kv = range.last - range.first;  // key tiles of this CTA
  auto n_iter = [&](int t) { return (n_kv + 1 - t) >> 1; };  // those of stream t: 2 it + t
  // fill f of stream t's ring (K of step it: f = 2 it, V: 2 it + 1) -> stage
  auto stage = [&](int t, int f) { return t * NS + f % NS; };

  if (threadIdx.x == 0) {
    mbar_init(bar_q, 1);
    for (int s = 0; s < 2 * NS; ++s) {
      mbar_init(bar_full + s, 1);
      mbar_init(bar_empty + s, 1);
    }
    for (int t = 0; t < 2; ++t) {
      mbar_init(bar_s_full + t, 1);
      mbar_init(bar_s_free + t, 128);
      mbar_init(bar_p_full + t, 128);
      mbar_init(bar_pv + t, 1);
    }
    mbar_init(bar_drain, 1);
    *abort_flag = 0;
    fence_barrier_init();
    tma_prefetch_desc(&tm_q);
    tma_prefetch_desc(&tm_k);
    tma_prefetch_desc(&tm_v);
  }
  if (warp == 1) {
    tmem_alloc(tmem_slot, 512);
    tmem_relinquish();
  }
  tc_fence_before();
  cta_sync();  // lane 0 of warp 0 initialised the barriers alone
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  auto wait = [&](uint64_t* bar, uint32_t parity) {
    return __all_sync(0xffffffffu, mbar_wait(bar, parity, abort_flag));
  };

  // Registers: launched with 168 per thread (384 x 168); 128 x 72 + 256 x 216 is the same total.  Each
  // setmaxnreg is executed by a whole warpgroup and dominates that group's code.
  if (warp < 4) {
    reg_dealloc<72>();
    if (warp == 0) {
      // ============================================================ TMA producer (the whole warp; lane
      // i issues the copies of the tile's page i)
      const int page = 1 << a.page_shift;
      const int pages_per_tile = a.page_table && page < 128 ? 128 >> a.page_shift : 1;
      const int rows_per_copy = 128 / pages_per_tile;
      // (outer coordinate, row) of this lane's copy of key tile kt; pages past the sequence or outside
      // the cache take a coordinate past the tensor, which reads as zeros and counts its bytes
      auto page_of = [&](int kt) -> int {
        if (!a.page_table) return seq.b;
        const int key = kt * 128 + lane * rows_per_copy;
        int p = -1;
        if (lane < pages_per_tile && key < seq.kv)
          p = __ldg(a.page_table + static_cast<long long>(seq.b) * a.pages_per_seq + (key >> a.page_shift));
        return p < 0 || p >= a.num_pages ? a.num_pages : p;
      };
      int issued[2] = {0, 0};  // fills of each ring so far
      if (n_kv > 0 && lane == 0) {
        mbar_arrive_expect_tx(bar_q, static_cast<uint32_t>(a.tile_tokens * a.G * NB * 128));
        for (int c = 0; c < NB; ++c)
          tma_load_5d(sQ + c * L::BOX, &tm_q, bar_q, 64 * c, 0, seq.token0 + tok0, hk, a.cu_q ? 0 : seq.b);
      }
      __syncwarp();
      int outer = n_kv > 0 ? page_of(range.first) : 0;
      bool ok = true;
      for (int j = 0; ok && j < n_kv; ++j) {
        const int kt = range.first + j;
        const int next = j + 1 < n_kv ? page_of(kt + 1) : 0;  // in flight during this tile's waits
        const int row = a.page_table ? (kt * 128) & (page - 1) : kt * 128;
        const int ring = j & 1;
        for (int kind = 0; kind < 2; ++kind) {
          const int fill = (j & ~1) + kind, s = stage(ring, fill);
          if (fill >= NS && !wait(bar_empty + s, (fill / NS - 1) & 1)) {
            ok = false;
            break;
          }
          if (lane == 0) mbar_arrive_expect_tx(bar_full + s, L::TILE);
          __syncwarp();
          if (lane < pages_per_tile) {
            uint8_t* dst = sRing + s * L::TILE + lane * rows_per_copy * 128;
            const CUtensorMap* map = kind == 0 ? &tm_k : &tm_v;
#pragma unroll
            for (int c = 0; c < NB; ++c)
              tma_load_4d(dst + c * L::BOX, map, bar_full + s, 64 * c, pages_per_tile > 1 ? 0 : row, hk, outer);
          }
          __syncwarp();
          if (ring == 0) issued[0] = fill + 1;
          else issued[1] = fill + 1;
        }
        outer = next;
      }
      if (*abort_flag && lane == 0) {  // let copies in flight land before the CTA exits
        if (n_kv > 0) mbar_drain(bar_q, 0);
#pragma unroll
        for (int g = 0; g < 2; ++g)
          for (int f = max(0, issued[g] - NS); f < issued[g]; ++f) mbar_drain(bar_full + stage(g, f), (f / NS) & 1);
      }
    } else if (warp == 1 && n_kv > 0) {
      // ============================================================ MMA issuer of both streams, in turn
      constexpr uint32_t FMT = BF16 ? 1u : 0u;
      constexpr uint32_t IDESC_QK = make_idesc(1 /*f32*/, FMT, FMT, 0, 0, 128, 128);
      constexpr uint32_t IDESC_PV = make_idesc(1 /*f32*/, FMT, FMT, 0, 1 /*V is MN-major*/, 128, D);
      const uint32_t ring = smem_u32(sRing);
      auto full = [&](int t, int fill) { return wait(bar_full + stage(t, fill), (fill / NS) & 1); };
      auto issue_qk = [&](int t, int it) -> bool {
        if (!full(t, 2 * it)) return false;
        if (OWN_P && it > 0 && !wait(bar_s_free + t, (it - 1) & 1)) return false;
        tc_fence_after();
        const uint32_t q_base = smem_u32(sQ);
        const uint32_t k_base = ring + stage(t, 2 * it) * L::TILE;
#pragma unroll
        for (int c = 0; c < NB; ++c)  // 16 channels per product: 32 bytes inside a 128-byte swizzled row
          mma_f16_ss_x4_warp<2, 2>(tmem + C::s(t), make_smem_desc(q_base + c * L::BOX, 16, 1024, kSwizzle128B),
                                   make_smem_desc(k_base + c * L::BOX, 16, 1024, kSwizzle128B), IDESC_QK, c > 0 ? 1u : 0u);
        mma_commit_warp(bar_s_full + t);
        mma_commit_warp(bar_empty + stage(t, 2 * it));
        return true;
      };
      auto issue_pv = [&](int t, int it) -> bool {
        const int fill = 2 * it + 1;
        if (!full(t, fill)) return false;
        const int valid = seq.kv - (range.first + 2 * it + t) * 128;
        if (valid < 128) zero_v_tail<D>(sRing + stage(t, fill) * L::TILE, valid, lane);
        if (!wait(bar_p_full + t, it & 1)) return false;
        tc_fence_after();
        const uint32_t v_base = ring + stage(t, fill) * L::TILE;
#pragma unroll
        for (int half = 0; half < 2; ++half)  // 64 keys, 16 per product
          mma_f16_ts_x4_warp<8, 16 * 128 / 16>(tmem + C::o(t), tmem + C::p(t) + half * 32,
                                               make_smem_desc(v_base + half * 64 * 128, L::BOX, 1024, kSwizzle128B),
                                               IDESC_PV, it == 0 && half == 0 ? 0u : 1u);
        mma_commit_warp(bar_empty + stage(t, fill));
        if (OWN_P || it + 1 == n_iter(t)) mma_commit_warp(bar_pv + t);
        return true;
      };
      bool ok = wait(bar_q, 0);
      for (int t = 0; ok && t < 2; ++t)
        if (n_iter(t) > 0) ok = issue_qk(t, 0);
      for (int it = 0; ok && it < n_iter(0); ++it) {
        for (int t = 0; ok && t < 2; ++t) {
          if (it >= n_iter(t)) continue;
          if constexpr (OWN_P) {
            if (it + 1 < n_iter(t)) ok = issue_qk(t, it + 1);
            ok = ok && issue_pv(t, it);
          } else {
            ok = issue_pv(t, it);
            if (ok && it + 1 < n_iter(t)) ok = issue_qk(t, it + 1);
          }
        }
      }
      // all MMAs must finish before TMEM is released
      mma_commit_warp(bar_drain);
      mbar_drain(bar_drain, 0);
    }
  } else {
    reg_alloc<216>();
    // ============================================================ softmax warpgroups
    const int t = (warp - 4) >> 2;
    const int quad = warp & 3;  // TMEM lane quadrant this warp may access
    const int r = quad * 32 + lane;
    const uint32_t lane_addr = static_cast<uint32_t>(quad * 32) << 16;
    const uint32_t tS = tmem + lane_addr + C::s(t), tO = tmem + lane_addr + C::o(t), tP = tmem + lane_addr + C::p(t);
    const int tok = tok0 + r / a.G;
    const bool row_valid = r < a.tile_tokens * a.G && tok < seq.nq;
    const int lim = visible(a, seq, tok) - range.first * 128;  // the row sees keys [0, lim) of the CTA's
    const int lim_warp = __reduce_min_sync(0xffffffffu, row_valid ? lim : 0x7fffffff);
    const int lim_most = __reduce_max_sync(0xffffffffu, row_valid ? lim : 0);
    const bool warp_live = __any_sync(0xffffffffu, row_valid);  // else what stands in its lanes is never stored
    RowState row;
    row.clear();
    bool ok = true;
    int it = 0;
    auto prior = [&]() -> bool {  // (d = 128: the last product precedes these scores)
      if (!OWN_P || it == 0) return true;
      const bool w = wait(bar_pv + t, (it - 1) & 1);
      tc_fence_after();
      return w;
    };
    for (; ok && it < n_iter(t); ++it) {
      if (!wait(bar_s_full + t, it & 1)) { ok = false; break; }
      tc_fence_after();
      const int k0 = (2 * it + t) * 128;
      if (warp_live) {
        ok = softmax_tile<D, BF16>(row, tS, tO, tP, lim - k0, lim_warp - k0, lim_most - k0, it == 0, a.scale_log2, bar_s_free + t, prior);
        tmem_wait_st();
        tc_fence_before();
      } else if (OWN_P) {
        // one arrival per tile: the next scores may come before the other warps' weights of this tile
        mbar_arrive(bar_s_free + t);
        ok = prior();
      }
      mbar_arrive(bar_p_full + t);
    }

    // ---- output
    float l = row.sum();
    if (ok && n_iter(t) > 0) ok = wait(bar_pv + t, OWN_P ? (n_iter(t) - 1) & 1 : 0);
    tc_fence_after();
    // Stream 1 hands its (m, l, O) over through shared memory: the rings, once both streams' products are
    // complete, as [4 channels][row] so that a warp's accesses are contiguous.
    const bool join = n_iter(1) > 0;
    float keep = 1.f, take = 0.f;  // factors of this stream's O and of stream 1's
    float4* sO = reinterpret_cast<float4*>(sRing);
    if (join) {
      if (t == 1) {
        ok = wait(bar_drain, 0) && ok;
        if (ok && warp_live) {
          sML[r] = make_float2(row.m_use, l);
#pragma unroll
          for (int cb = 0; cb < D; cb += 32) {
            uint32_t ov[32];
            tmem_ld32_sync(tO + cb, ov);
#pragma unroll
            for (int i = 0; i < 32; i += 4)
              sO[(cb + i) / 4 * 128 + r] = make_float4(__uint_as_float(ov[i]), __uint_as_float(ov[i + 1]),
                                                      __uint_as_float(ov[i + 2]), __uint_as_float(ov[i + 3]));
          }
        }
      }
      asm volatile("barrier.sync 1, 256;" ::: "memory");
      if (t == 0) {
        const float2 other = sML[r];
        const float m = fmaxf(row.m_use, other.x);
        const float base = m == -INFINITY ? 0.f : m;
        keep = fast_exp2(row.m_use - base);
        take = fast_exp2(other.x - base);
        l = l * keep + other.y * take;
        row.m_use = m;
      }
    }
    if (ok && !*abort_flag && t == 0 && warp_live) {
      const bool whole = range.parts == 1;  // else: a part, joined by attn_tile_join_kernel
      const float scale = whole ? weight_sum_inverse(l) : 1.f;
      uint16_t* orow = static_cast<uint16_t*>(a.o) + out_offset(a, seq, tok, hk * a.G + r % a.G);
      const long long part = static_cast<long long>(blockIdx.x) * 128 + r;
      if (!whole && row_valid) a.part_ml[part] = make_float2(row.m_use, l);
#pragma unroll
      for (int cb = 0; cb < D; cb += 32) {
        float o[32];
        if (n_kv > 0) {
          uint32_t ov[32];
          tmem_ld32_sync(tO + cb, ov);
#pragma unroll
          for (int i = 0; i < 32; ++i) o[i] = __uint_as_float(ov[i]);
        } else {
#pragma unroll
          for (int i = 0; i < 32; ++i) o[i] = 0.f;
        }
        if (join) {
#pragma unroll
          for (int i = 0; i < 32; i += 4) {
            const float4 y = sO[(cb + i) / 4 * 128 + r];
            o[i] = o[i] * keep + y.x * take;
            o[i + 1] = o[i + 1] * keep + y.y * take;
            o[i + 2] = o[i + 2] * keep + y.z * take;
            o[i + 3] = o[i + 3] * keep + y.w * take;
          }
        }
        if (row_valid) {
          if (whole) {
#pragma unroll
            for (int i = 0; i < 32; i += 8)
              *reinterpret_cast<uint4*>(orow + cb + i) =
                  make_uint4(pack_in_range<BF16>(o[i] * scale, o[i + 1] * scale), pack_in_range<BF16>(o[i + 2] * scale, o[i + 3] * scale),
                             pack_in_range<BF16>(o[i + 4] * scale, o[i + 5] * scale), pack_in_range<BF16>(o[i + 6] * scale, o[i + 7] * scale));
          } else {
            float4* dst = reinterpret_cast<float4*>(a.part_o + part * D + cb);
#pragma unroll
            for (int i = 0; i < 32; i += 4) dst[i / 4] = make_float4(o[i], o[i + 1], o[i + 2], o[i + 3]);
          }
        }
      }
    }
  }

  // roles diverge inside warps (single-lane producers): the thread-counting barrier holds the TMEM
  // release until every thread of the CTA is done
  tc_fence_before();
  cta_sync();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

// Joins the key parts of each row, in their order.  Grid: (tile slot, key head) x eight rows at a time, a warp per row; tiles whose key axis was one part have their result already.
constexpr int kJoinThreads = 256;

template <int D, bool BF16>
__global__ void __launch_bounds__(kJoinThreads) attn_tile_join_kernel(const __grid_constant__ Attn16Args a) {
  const int lane = threadIdx.x & 31;
  const int place = static_cast<int>(blockIdx.x) % a.slots, hk = static_cast<int>(blockIdx.x) / a.slots;
  cudaGridDependencySynchronize();  // the parts are written
  Sequence seq;
  int tok0;
  if (!tile_of_slot(a, a.slots - 1 - place, seq, tok0)) return;
  const int parts = key_range(key_tiles(a, seq, tok0, a.tile_tokens), a.splits, a.min_chunk, 0).parts;
  if (parts == 1) return;
  const int r = static_cast<int>(blockIdx.y) * (kJoinThreads / 32) + static_cast<int>(threadIdx.x >> 5);
  const int tok = tok0 + r / a.G;
  if (r >= a.tile_tokens * a.G || tok >= seq.nq) return;
  constexpr int PER = D / 32;  // channels per lane
  float acc[1][PER], l[1];
  join_parts(acc, l, 0, parts - 1, a.part_ml, a.part_o,
             [&](int, int s) { return (static_cast<long long>(hk * a.splits + s) * a.slots + place) * 128 + r; });
  store_joined<BF16>(static_cast<uint16_t*>(a.o) + out_offset(a, seq, tok, hk * a.G + r % a.G) + lane * PER, acc[0], l[0]);
}

template <int D, bool BF16>
cudaError_t launch_t(const Attn16Launch& l, cudaStream_t st) {
  using L = TileLayout<D>;
  auto kern = attn_tile_kernel<D, BF16>;
  static std::atomic<unsigned long long> allowed{0};
  cudaError_t e = allow_shared_memory(allowed, reinterpret_cast<const void*>(kern), L::SMEM);
  if (e != cudaSuccess) return e;
  kern<<<static_cast<unsigned>(l.a.slots) * l.a.splits * l.a.Hk, kThreads, L::SMEM, st>>>(l.tm_q, l.tm_k, l.tm_v, l.a);
  e = cudaGetLastError();
  if (e != cudaSuccess || l.a.splits == 1) return e;
  // launched early, while the attention drains: it waits on the device for the parts
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(static_cast<unsigned>(l.a.slots) * l.a.Hk, (l.a.tile_tokens * l.a.G + kJoinThreads / 32 - 1) / (kJoinThreads / 32));
  cfg.blockDim = dim3(kJoinThreads);
  cfg.stream = st;
  cudaLaunchAttribute attr{};
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, attn_tile_join_kernel<D, BF16>, l.a);
}

}  // namespace

size_t tile_part_rows(const Attn16Args& a) { return static_cast<size_t>(a.slots) * a.splits * a.Hk * 128; }

cudaError_t launch_attn_tile(const Attn16Launch& l, cudaStream_t st) {
  if (l.D == 128) return l.bf16 ? launch_t<128, true>(l, st) : launch_t<128, false>(l, st);
  return l.bf16 ? launch_t<64, true>(l, st) : launch_t<64, false>(l, st);
}

int read_and_clear_tile_error(cudaStream_t st, cudaError_t* err) {
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
