// attn16_kernels.cu -- 16-bit attention for sm_100a behind the paged attention and the cross attention:
// grouped query heads, chunks of queries of ragged length, keys from pages or from strided tensors.
//
// Mathematics, per query row i and key j of its sequence and head group (log2 units):
//   u_ij = (q_i . k_j) * sm_scale * log2(e)        16-bit operands, fp32 accumulation (tcgen05 kind::f16)
//   m = a running maximum of u, l = sum_j 2^(u_ij - m), O = sum_j 2^(u_ij - m) v_j    over the keys the row sees
//   o_i = O / l, rounded once; a row that sees no key gives 0
// The weights 2^(u - m) are rounded to the operands' type for the second product (kind::f16 takes no
// fp32 operand): half a step each, in sums where the errors average out; l adds the unrounded weights.
// m follows the maximum only when it grew by more than 8 (weights <= 2^8, O rescaled then and only
// then); in fp16 the weights carry a factor 2^7 besides, so that a row's small weights keep their bits.
//
// Rows: the query heads that share a key head are rows of the same tile (row = token * G + head in
// group), so a tile of 128 rows reads the keys once for all of them.
//
// CTA organisation (one per SM: 512 TMEM columns, about 226 KB of shared memory), 12 warps:
//   warp 0      TMA producer: Q once, then K and V tiles of 128 keys through rings, K0 V0 K1 V1 ...
//   warp 1      MMA issuer of both streams; allocates TMEM
//   warps 4-7   softmax of stream 0 (thread = query row = TMEM lane), warps 8-11 of stream 1
// NQT = 2: the streams are two query tiles that share each key tile.  NQT = 1: one query tile, stream t
// takes every other key tile, and the two (m, l, O) are joined at the end: single tokens and short
// chunks, where a second tile would be empty and the key axis is what has to be read fast.
// TMEM: S_t [128 t, +128), O_t [256 + D t, +D); the 16-bit weights of stream t overwrite the first 64
// columns of S_t (a thread holds its row of S in registers by then), and the next S_t is issued behind
// the product that reads them.
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <cstdint>
#include <type_traits>

#include "attn16_device.cuh"
#include "attn16_kernels.cuh"
#include "attn_common.cuh"
#include "sm100_ptx.cuh"
#include "workspace.cuh"

namespace sage {
namespace {

template <int D, int NQT>
struct Layout16 {
  static constexpr int BOX = 128 * 128;           // 128 rows of 64 channels (128-byte rows)
  static constexpr int TILE = BOX * (D / 64);     // one Q, K or V tile
  // Ring stages: with Q, 7 tiles fit (d = 128), or 14 (d = 64).  NQT = 1 gives each stream a ring of its
  // own: a stage's barrier only tells one fill from the next (phase parity), so whoever waits for a
  // fill must have waited for the one before it in that stage too.  In a ring that both streams draw
  // from by turns, one of them could take the other's late fill for its own.
  static constexpr int RINGS = NQT == 2 ? 1 : 2;
  static constexpr int NS = (7 * 128 / D - NQT) / RINGS;  // stages per ring
  static constexpr int OFF_Q = 0;
  static constexpr int OFF_RING = NQT * TILE;
  static constexpr int OFF_ML = OFF_RING + RINGS * NS * TILE;  // [128] (m, l) of stream 1 (NQT = 1)
  static constexpr int OFF_BAR = OFF_ML + 128 * 8;
  static constexpr int NUM_BARS = 1 + 2 * RINGS * NS + 4 * 2 + 1;
  // d = 64 leaves TMEM columns for the weights beside the scores, so that the next scores can be computed as
  // soon as these are in registers
  static constexpr bool OWN_P = D == 64;
  static constexpr int OFF_MISC = OFF_BAR + NUM_BARS * 8;
  static constexpr int SMEM = OFF_MISC + 16 + 1024;
  static constexpr int THREADS = 384;
  static_assert(SMEM <= 227 * 1024, "shared memory budget");
  static_assert(SMEM > 114 * 1024, "one CTA per SM: each allocates all of TMEM");
  static_assert(128 * D * 4 <= RINGS * NS * TILE, "stream 1's O fits the ring");
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

template <int D, bool BF16, int NQT>
__global__ void __launch_bounds__(384, 1)
    attn16_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
                  const __grid_constant__ CUtensorMap tm_v, const __grid_constant__ Attn16Args a) {
  using L = Layout16<D, NQT>;
  constexpr int NS = L::NS, STAGES = L::RINGS * L::NS;
  constexpr int NB = D / 64;  // 64-channel boxes per tile
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* sQ = smem + L::OFF_Q;
  uint8_t* sRing = smem + L::OFF_RING;
  float2* sML = reinterpret_cast<float2*>(smem + L::OFF_ML);
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + L::OFF_BAR);
  uint64_t* bar_q = bars;
  uint64_t* bar_full = bar_q + 1;
  uint64_t* bar_empty = bar_full + STAGES;
  uint64_t* bar_s_full = bar_empty + STAGES;  // [2] S_t of the next key tile (and every product before it) done
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
  const int cta_tokens = NQT * a.tile_tokens;
  int rest = static_cast<int>(blockIdx.x);
  const int slot = a.slots - 1 - rest % a.slots;
  rest /= a.slots;
  const int split = rest % a.splits;
  const int hk = rest / a.splits;
  Sequence seq;
  int tok0;  // first token (within the sequence) of the CTA
  if (a.cu_q) {
    // slot -> sequence: sequence b owns the slots from cu_q[b] / cta_tokens + b on, which leaves room for
    // its ceil(nq / cta_tokens) tiles before the next one's and needs no sum over the sequences
    int upto = 0;
    for (int base = 0; base < a.B; base += L::THREADS) {
      const int i = base + static_cast<int>(threadIdx.x);
      upto += __syncthreads_count(i < a.B && min(max(__ldg(a.cu_q + i), 0), a.Nq) / cta_tokens + i <= slot);
    }
    if (upto == 0) return;
    seq.b = upto - 1;
    seq.token0 = min(max(__ldg(a.cu_q + seq.b), 0), a.Nq);
    seq.nq = min(max(__ldg(a.cu_q + seq.b + 1), 0), a.Nq) - seq.token0;
    tok0 = (slot - (seq.token0 / cta_tokens + seq.b)) * cta_tokens;
  } else {
    const int per_b = (a.Nq + cta_tokens - 1) / cta_tokens;
    seq.b = slot / per_b;
    seq.token0 = 0;
    seq.nq = a.Nq;
    tok0 = (slot % per_b) * cta_tokens;
  }
  if (tok0 >= seq.nq) return;  // a slot without a tile
  seq.kv = keys_of(a, seq.b);
  const KeyRange range = key_range(key_tiles(a, seq, tok0, cta_tokens), a.splits, a.min_chunk, split);
  if (split >= range.parts) return;
  const int n_kv = range.last - range.first;  // key tiles of this CTA
  int n_iter[2];                              // key tiles of stream 0 and 1
  if constexpr (NQT == 2) {
    for (int t = 0; t < 2; ++t) {
      const int tk = tok0 + t * a.tile_tokens;
      const int nt = tk < seq.nq ? key_tiles(a, seq, tk, a.tile_tokens) : 0;
      n_iter[t] = max(0, min(nt, range.last) - range.first);
    }
  } else {
    n_iter[0] = (n_kv + 1) / 2;
    n_iter[1] = n_kv / 2;
  }
  const int q_tiles = NQT == 2 && tok0 + a.tile_tokens < seq.nq ? 2 : 1;
  auto tile_of = [&](int t, int it) { return NQT == 2 ? it : 2 * it + t; };  // stream step -> CTA key tile
  // fill f of stream t's ring (K of step it: f = 2 it, V: 2 it + 1; NQT = 2: one ring, both streams) -> stage
  auto stage = [&](int t, int f) { return (NQT == 2 ? 0 : t * NS) + f % NS; };

  if (threadIdx.x == 0) {
    mbar_init(bar_q, 1);
    for (int s = 0; s < STAGES; ++s) {
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
  auto s_col = [](int t) { return 128u * t; };
  auto o_col = [](int t) { return 256u + static_cast<uint32_t>(D) * t; };
  auto p_col = [&](int t) { return L::OWN_P ? 384u + 64u * t : s_col(t); };

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
      int q_issued = 0, issued[L::RINGS] = {};  // fills of each ring so far
      if (n_kv > 0) {
        if (lane == 0) {
          const uint32_t bytes = static_cast<uint32_t>(q_tiles * a.tile_tokens * a.G * NB * 128);
          mbar_arrive_expect_tx(bar_q, bytes);
          for (int t = 0; t < q_tiles; ++t)
            for (int c = 0; c < NB; ++c)
              tma_load_5d(sQ + t * L::TILE + c * L::BOX, &tm_q, bar_q, 64 * c, 0,
                          seq.token0 + tok0 + t * a.tile_tokens, hk, a.cu_q ? 0 : seq.b);
        }
        q_issued = 1;
        __syncwarp();
      }
      int outer = n_kv > 0 ? page_of(range.first) : 0;
      bool ok = true;
      for (int j = 0; ok && j < n_kv; ++j) {
        const int kt = range.first + j;
        const int next = j + 1 < n_kv ? page_of(kt + 1) : 0;  // in flight during this tile's waits
        const int row = a.page_table ? (kt * 128) & (page - 1) : kt * 128;
        const int ring = NQT == 2 ? 0 : j & 1;
        for (int kind = 0; kind < 2; ++kind) {
          const int fill = (NQT == 2 ? 2 * j : j & ~1) + kind, s = stage(ring, fill);
          if (fill >= NS && !__all_sync(0xffffffffu, mbar_wait(bar_empty + s, (fill / NS - 1) & 1, abort_flag))) {
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
          else issued[L::RINGS - 1] = fill + 1;
        }
        outer = next;
      }
      if (*abort_flag && lane == 0) {  // let copies in flight land before the CTA exits
        if (q_issued) mbar_drain(bar_q, 0);
#pragma unroll
        for (int g = 0; g < L::RINGS; ++g)
          for (int f = max(0, issued[g] - NS); f < issued[g]; ++f) mbar_drain(bar_full + stage(g, f), (f / NS) & 1);
      }
    } else if (warp == 1 && n_kv > 0) {
      // ============================================================ MMA issuer of both streams, in turn: the
      // second product of one and its next scores, then the other's.  The tensor core so finishes one
      // stream's scores a whole turn before the other's, and the streams' softmax work falls into each
      // other's product time.  (Issued by a warp per stream, the products of both finish together and the
      // softmax warps work at the same time and wait at the same time: 4470 cycles a turn of two 128 x 128
      // tiles of d = 128 instead of 3330.)  The whole warp runs the loop; see mma_f16_ss_x4_warp.
      constexpr uint32_t FMT = BF16 ? 1u : 0u;
      constexpr uint32_t IDESC_QK = make_idesc(1 /*f32*/, FMT, FMT, 0, 0, 128, 128);
      constexpr uint32_t IDESC_PV = make_idesc(1 /*f32*/, FMT, FMT, 0, 1 /*V is MN-major*/, 128, D);
      const uint32_t ring = smem_u32(sRing);
      auto wait = [&](uint64_t* bar, uint32_t parity) {
        return __all_sync(0xffffffffu, mbar_wait(bar, parity, abort_flag));
      };
      auto full = [&](int t, int fill) { return wait(bar_full + stage(t, fill), (fill / NS) & 1); };
      // a shared ring's tile `it` is waited for in its first stream's turn and freed in its last one's
      auto first_user = [&](int t, int it) { return NQT == 1 || t == 0 || it >= n_iter[0]; };
      auto last_user = [&](int t, int it) { return NQT == 1 || t == 1 || it >= n_iter[1]; };
      auto issue_qk = [&](int t, int it) -> bool {
        if (first_user(t, it) && !full(t, 2 * it)) return false;
        if (L::OWN_P && it > 0 && !wait(bar_s_free + t, (it - 1) & 1)) return false;
        tc_fence_after();
        const uint32_t q_base = smem_u32(sQ) + (NQT == 2 ? t * L::TILE : 0);
        const uint32_t k_base = ring + stage(t, 2 * it) * L::TILE;
#pragma unroll
        for (int c = 0; c < NB; ++c)  // 16 channels per product: 32 bytes inside a 128-byte swizzled row
          mma_f16_ss_x4_warp<2, 2>(tmem + s_col(t), make_smem_desc(q_base + c * L::BOX, 16, 1024, kSwizzle128B),
                                   make_smem_desc(k_base + c * L::BOX, 16, 1024, kSwizzle128B), IDESC_QK, c > 0 ? 1u : 0u);
        mma_commit_warp(bar_s_full + t);
        if (last_user(t, it)) mma_commit_warp(bar_empty + stage(t, 2 * it));
        return true;
      };
      auto issue_pv = [&](int t, int it) -> bool {
        const int fill = 2 * it + 1;
        if (first_user(t, it)) {
          if (!full(t, fill)) return false;
          // Keys past the sequence's end have no weight, but what stands in their rows (stale or unwritten
          // memory) may be NaN or infinite: zero those V rows before a product reads them.
          const int valid = seq.kv - (range.first + tile_of(t, it)) * 128;
          if (valid < 128) {
            uint8_t* v_tile = sRing + stage(t, fill) * L::TILE;
            for (int i = lane; i < (128 - valid) * 8 * NB; i += 32) {
              const int c = i / ((128 - valid) * 8), in_box = i % ((128 - valid) * 8);
              *reinterpret_cast<uint4*>(v_tile + c * L::BOX + valid * 128 + in_box * 16) = make_uint4(0, 0, 0, 0);
            }
            fence_proxy_async_shared();
            __syncwarp();
          }
        }
        if (!wait(bar_p_full + t, it & 1)) return false;
        tc_fence_after();
        const uint32_t v_base = ring + stage(t, fill) * L::TILE;
#pragma unroll
        for (int half = 0; half < 2; ++half)  // 64 keys, 16 per product
          mma_f16_ts_x4_warp<8, 16 * 128 / 16>(tmem + o_col(t), tmem + p_col(t) + half * 32,
                                               make_smem_desc(v_base + half * 64 * 128, L::BOX, 1024, kSwizzle128B),
                                               IDESC_PV, it == 0 && half == 0 ? 0u : 1u);
        if (last_user(t, it)) mma_commit_warp(bar_empty + stage(t, fill));
        if (L::OWN_P || it + 1 == n_iter[t]) mma_commit_warp(bar_pv + t);
        return true;
      };
      bool ok = wait(bar_q, 0);
      for (int t = 0; ok && t < 2; ++t)
        if (n_iter[t] > 0) ok = issue_qk(t, 0);
      for (int it = 0; ok && it < max(n_iter[0], n_iter[1]); ++it) {
        for (int t = 0; ok && t < 2; ++t) {
          if (it >= n_iter[t]) continue;
          if constexpr (L::OWN_P) {
            if (it + 1 < n_iter[t]) ok = issue_qk(t, it + 1);
            ok = ok && issue_pv(t, it);
          } else {
            ok = issue_pv(t, it);
            if (ok && it + 1 < n_iter[t]) ok = issue_qk(t, it + 1);
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
    const uint32_t tS = tmem + lane_addr + s_col(t);
    const uint32_t tO = tmem + lane_addr + o_col(t);
    const uint32_t tP = tmem + lane_addr + p_col(t);
    const int tok = tok0 + (NQT == 2 ? t * a.tile_tokens : 0) + r / a.G;
    const bool row_valid = r < a.tile_tokens * a.G && tok < seq.nq;
    const int lim = visible(a, seq, tok);  // this row's keys: [0, lim)
    const int lim_warp = __reduce_min_sync(0xffffffffu, row_valid ? lim : 0x7fffffff);
    const bool warp_live = __any_sync(0xffffffffu, row_valid);
    constexpr float kShift = BF16 ? 0.f : 7.f;
    float m_use = -INFINITY;  // offset (log2 units) of the weights so far
    float2 lsum[4] = {{0.f, 0.f}, {0.f, 0.f}, {0.f, 0.f}, {0.f, 0.f}};
    bool ok = true;
    for (int it = 0; it < n_iter[t]; ++it) {
      if (!__all_sync(0xffffffffu, mbar_wait(bar_s_full + t, it & 1, abort_flag))) { ok = false; break; }
      tc_fence_after();
      if (!warp_live) {  // no row of this warp exists: whatever stands in its lanes is never stored
        if (L::OWN_P) {
          // one arrival per tile: S of the next tile may come before the other warps' weights of this one
          mbar_arrive(bar_s_free + t);
          if (it > 0 && !__all_sync(0xffffffffu, mbar_wait(bar_pv + t, (it - 1) & 1, abort_flag))) { ok = false; break; }
        }
        mbar_arrive(bar_p_full + t);
        continue;
      }
      const int k0 = (range.first + tile_of(t, it)) * 128;
      uint32_t x[128];
      tmem_ld64_sync(tS + 0, *reinterpret_cast<uint32_t(*)[64]>(x + 0));
      tmem_ld64_sync(tS + 64, *reinterpret_cast<uint32_t(*)[64]>(x + 64));
      if (L::OWN_P) {
        tc_fence_before();
        mbar_arrive(bar_s_free + t);
      }
      const bool masked = lim_warp < k0 + 128;
      if (masked) {
        const int seen = lim - k0;
#pragma unroll
        for (int c = 0; c < 128; ++c) x[c] = c < seen ? x[c] : 0xFF800000u;
      }
      auto row_max = [&]() {  // log2 units
        float mx[8];
#pragma unroll
        for (int k = 0; k < 8; ++k) mx[k] = fmaxf(__uint_as_float(x[k]), __uint_as_float(x[8 + k]));
#pragma unroll
        for (int c = 16; c < 128; c += 16) {
#pragma unroll
          for (int k = 0; k < 8; ++k)
            mx[k] = max3f(mx[k], __uint_as_float(x[c + k]), __uint_as_float(x[c + 8 + k]));
        }
        return fmaxf(max3f(mx[0], mx[1], mx[2]), fmaxf(max3f(mx[3], mx[4], mx[5]), fmaxf(mx[6], mx[7]))) * a.scale_log2;
      };
      // The offset moves when the maximum has passed it by 8 (also at the first finite maximum).  The next
      // product waits for the arrival below, so O may be rescaled here once the last one is complete.
      auto move_offset = [&](float mx) {
        const bool move = mx > m_use + 8.f;
        const float alpha = move ? fast_exp2(m_use - mx) : 1.f;
        if (move) m_use = mx;
#pragma unroll
        for (int i = 0; i < 4; ++i) lsum[i] = __fmul2_rn(lsum[i], make_float2(alpha, alpha));
#pragma unroll
        for (int cb = 0; cb < D; cb += 32) {
          uint32_t ov[32];
          tmem_ld32_sync(tO + cb, ov);
#pragma unroll
          for (int i = 0; i < 32; ++i) ov[i] = __float_as_uint(__uint_as_float(ov[i]) * alpha);
          tmem_st32(tO + cb, ov);
        }
      };
      // Weights of 64 keys into TMEM, one pair in eight by the polynomial (the MUFU pipe alone would hold up
      // the rest; more of it costs more issue slots than it saves).  Masked weights are exactly 0 on the MUFU
      // pipe (ex2(-inf)); the polynomial bottoms out at 2^-126 instead, so tiles with masked keys do not use it.
      auto weights = [&](int half, auto poly, float2 (&sum)[4]) {
        const float off = kShift - (m_use == -INFINITY ? 0.f : m_use);
        const float2 sc2 = make_float2(a.scale_log2, a.scale_log2), off2 = make_float2(off, off);
#pragma unroll
        for (int cb = 0; cb < 64; cb += 32) {
          uint32_t pk[16];
#pragma unroll
          for (int i = 0; i < 32; i += 2) {
            const int c = 64 * half + cb + i;
            const float2 u = __ffma2_rn(make_float2(__uint_as_float(x[c]), __uint_as_float(x[c + 1])), sc2, off2);
            float2 p;
            if (decltype(poly)::value && ((i >> 1) & 7) == 7) p = exp2_poly2(u);
            else p = make_float2(fast_exp2(u.x), fast_exp2(u.y));
            sum[(i >> 1) & 3] = __fadd2_rn(sum[(i >> 1) & 3], p);
            pk[i >> 1] = pack16<BF16>(p.x, p.y);
          }
          tmem_st16(tP + 32 * half + (cb >> 1), pk);
        }
      };
      if (L::OWN_P && it > 0) {  // the product of the tile before has read its weights (else: it precedes this S)
        if (!__all_sync(0xffffffffu, mbar_wait(bar_pv + t, (it - 1) & 1, abort_flag))) { ok = false; break; }
        tc_fence_after();
      }
      if (it == 0 || masked) {
        const float mx = row_max();
        if (it == 0) m_use = mx;
        else if (__any_sync(0xffffffffu, mx > m_use + 8.f)) move_offset(mx);
        weights(0, std::false_type{}, lsum);
        weights(1, std::false_type{}, lsum);
      } else {
        // The offset hardly ever moves after the first tiles: the first 64 weights are taken at the old
        // one while the maximum is found beside them, and taken again if it did move.
        float2 sum[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) sum[i] = lsum[i];
        weights(0, std::true_type{}, sum);
        const float mx = row_max();
        if (__any_sync(0xffffffffu, mx > m_use + 8.f)) {
          move_offset(mx);
          weights(0, std::true_type{}, lsum);
        } else {
#pragma unroll
          for (int i = 0; i < 4; ++i) lsum[i] = sum[i];
        }
        weights(1, std::true_type{}, lsum);
      }
      tmem_wait_st();
      tc_fence_before();
      mbar_arrive(bar_p_full + t);
    }

    // ---- epilogue
    const float2 l2 = __fadd2_rn(__fadd2_rn(lsum[0], lsum[1]), __fadd2_rn(lsum[2], lsum[3]));
    float l = l2.x + l2.y;
    if (ok && n_iter[t] > 0)
      ok = __all_sync(0xffffffffu, mbar_wait(bar_pv + t, L::OWN_P ? (n_iter[t] - 1) & 1 : 0, abort_flag));
    tc_fence_after();
    float keep = 1.f, take = 0.f;  // factors of this stream's O and of stream 1's (NQT = 1)
    bool join = false;
    if constexpr (NQT == 1) {
      // stream 1 hands its (m, l, O) over through shared memory: the ring, once both streams' products
      // are complete, as [4 channels][row] so that a warp's accesses are contiguous
      join = n_iter[1] > 0;
      float4* sO = reinterpret_cast<float4*>(sRing);
      if (join) {
        if (t == 1) {
          ok = __all_sync(0xffffffffu, mbar_wait(bar_drain, 0, abort_flag)) && ok;
          if (ok && warp_live) {
            sML[r] = make_float2(m_use, l);
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
          const float m = fmaxf(m_use, other.x);
          const float base = m == -INFINITY ? 0.f : m;
          keep = fast_exp2(m_use - base);
          take = fast_exp2(other.x - base);
          l = l * keep + other.y * take;
          m_use = m;
        }
      }
    }
    const bool writer = NQT == 2 ? t < q_tiles : t == 0;
    if (ok && !*abort_flag && writer && warp_live) {
      const int h = hk * a.G + r % a.G;
      const bool whole = range.parts == 1;  // else: a part, joined by attn16_join_kernel
      const float scale = whole ? (l > 0.f ? 1.f / l : 0.f) : 1.f;
      const long long token = static_cast<long long>(a.cu_q ? seq.token0 : seq.b * static_cast<long long>(a.Nq)) + tok;
      const long long part = (token * (a.Hk * a.G) + h) * a.splits + split;
      uint16_t* orow = static_cast<uint16_t*>(a.o) + (a.cu_q ? 0 : seq.b * a.o_sb) + h * a.o_sh +
                       static_cast<long long>((a.cu_q ? seq.token0 : 0) + tok) * a.o_sn;
      if (!whole && row_valid) a.part_ml[part] = make_float2(m_use, l);
#pragma unroll
      for (int cb = 0; cb < D; cb += 32) {
        float o[32];
        if (n_iter[t] > 0) {
          uint32_t ov[32];
          tmem_ld32_sync(tO + cb, ov);
#pragma unroll
          for (int i = 0; i < 32; ++i) o[i] = __uint_as_float(ov[i]);
        } else {
#pragma unroll
          for (int i = 0; i < 32; ++i) o[i] = 0.f;
        }
        if (NQT == 1 && join) {
          const float4* sO = reinterpret_cast<const float4*>(sRing);
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
                  make_uint4(pack16<BF16>(o[i] * scale, o[i + 1] * scale), pack16<BF16>(o[i + 2] * scale, o[i + 3] * scale),
                             pack16<BF16>(o[i + 4] * scale, o[i + 5] * scale), pack16<BF16>(o[i + 6] * scale, o[i + 7] * scale));
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

// Joins the key parts of each row: o = sum_s 2^(m_s - m) O_s / sum_s 2^(m_s - m) l_s, in the order of the
// parts.  One warp per (token, head); rows whose key axis was one part have their result already.
constexpr int kJoinThreads = 256;

template <int D, bool BF16>
__global__ void __launch_bounds__(kJoinThreads) attn16_join_kernel(const __grid_constant__ Attn16Args a, int cta_tokens) {
  const int heads = a.Hk * a.G;
  const int per_token = (heads + kJoinThreads / 32 - 1) / (kJoinThreads / 32);
  const int token = static_cast<int>(blockIdx.x) / per_token;
  const int h = (static_cast<int>(blockIdx.x) % per_token) * (kJoinThreads / 32) + static_cast<int>(threadIdx.x >> 5);
  const int lane = threadIdx.x & 31;
  Sequence seq;
  int tok;
  if (a.cu_q) {
    int upto = 0;  // sequences that begin at or before this token
    for (int base = 0; base < a.B; base += kJoinThreads) {
      const int i = base + static_cast<int>(threadIdx.x);
      upto += __syncthreads_count(i < a.B && min(max(__ldg(a.cu_q + i), 0), a.Nq) <= token);
    }
    if (upto == 0) return;
    seq.b = upto - 1;
    seq.token0 = min(max(__ldg(a.cu_q + seq.b), 0), a.Nq);
    seq.nq = min(max(__ldg(a.cu_q + seq.b + 1), 0), a.Nq) - seq.token0;
    tok = token - seq.token0;
    if (tok >= seq.nq) return;  // behind the last sequence
  } else {
    seq.b = token / a.Nq;
    seq.token0 = 0;
    seq.nq = a.Nq;
    tok = token % a.Nq;
  }
  seq.kv = keys_of(a, seq.b);
  const int nt = key_tiles(a, seq, tok / cta_tokens * cta_tokens, cta_tokens);
  const int parts = key_range(nt, a.splits, a.min_chunk, 0).parts;
  if (parts == 1 || h >= heads) return;
  const long long first = (static_cast<long long>(token) * heads + h) * a.splits;
  float m = -INFINITY;
  for (int s = lane; s < parts; s += 32) m = fmaxf(m, a.part_ml[first + s].x);
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, off));
  const float base = m == -INFINITY ? 0.f : m;
  constexpr int C = D / 32;  // channels per lane
  float acc[C] = {}, l = 0.f;
  for (int s = 0; s < parts; ++s) {
    const float2 ml = a.part_ml[first + s];
    const float w = fast_exp2(ml.x - base);
    l = fmaf(ml.y, w, l);
    const float* src = a.part_o + (first + s) * D + lane * C;
#pragma unroll
    for (int c = 0; c < C; c += 2) {
      const float2 y = *reinterpret_cast<const float2*>(src + c);
      acc[c] = fmaf(y.x, w, acc[c]);
      acc[c + 1] = fmaf(y.y, w, acc[c + 1]);
    }
  }
  const float inv = l > 0.f ? 1.f / l : 0.f;
  uint16_t* orow = static_cast<uint16_t*>(a.o) + (a.cu_q ? 0 : seq.b * a.o_sb) + h * a.o_sh +
                   static_cast<long long>(a.cu_q ? token : tok) * a.o_sn + lane * C;
#pragma unroll
  for (int c = 0; c < C; c += 2) *reinterpret_cast<uint32_t*>(orow + c) = pack16<BF16>(acc[c] * inv, acc[c + 1] * inv);
}

template <int D, bool BF16, int NQT>
cudaError_t launch_t(const Attn16Launch& l, cudaStream_t st) {
  using L = Layout16<D, NQT>;
  auto kern = attn16_kernel<D, BF16, NQT>;
  static std::atomic<unsigned long long> allowed{0};
  cudaError_t e = allow_shared_memory(allowed, reinterpret_cast<const void*>(kern), L::SMEM);
  if (e != cudaSuccess) return e;
  const unsigned grid = static_cast<unsigned>(l.a.slots) * l.a.splits * l.a.Hk;
  kern<<<grid, L::THREADS, L::SMEM, st>>>(l.tm_q, l.tm_k, l.tm_v, l.a);
  e = cudaGetLastError();
  if (e != cudaSuccess || l.a.splits == 1) return e;
  const int per_token = (l.a.Hk * l.a.G + kJoinThreads / 32 - 1) / (kJoinThreads / 32);
  const unsigned tokens = static_cast<unsigned>(l.a.cu_q ? l.a.Nq : l.a.B * l.a.Nq);
  attn16_join_kernel<D, BF16><<<tokens * per_token, kJoinThreads, 0, st>>>(l.a, NQT * l.a.tile_tokens);
  return cudaGetLastError();
}

template <int D, bool BF16>
cudaError_t launch_d(const Attn16Launch& l, cudaStream_t st) {
  return l.pair ? launch_t<D, BF16, 2>(l, st) : launch_t<D, BF16, 1>(l, st);
}

}  // namespace

cudaError_t launch_attn16(const Attn16Launch& l, cudaStream_t st) {
  if (l.D == 128) return l.bf16 ? launch_d<128, true>(l, st) : launch_d<128, false>(l, st);
  return l.bf16 ? launch_d<64, true>(l, st) : launch_d<64, false>(l, st);
}

int read_and_clear_attn16_error(cudaStream_t st, cudaError_t* err) {
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
