// attn_pair_kernels.cu -- 16-bit attention for sm_100a behind the paged attention and the cross attention, for
// many query rows: chunks of ragged length, grouped query heads, keys from pages or strided tensors.
//
// Mathematics, per query row i and key j of its sequence and head group (log2 units):
//   u_ij = (q_i . k_j) * sm_scale * log2(e)        16-bit operands, fp32 accumulation (tcgen05 kind::f16)
//   m = a running maximum of u, l = sum_j 2^(u_ij - m), O = sum_j 2^(u_ij - m) v_j    over the keys the row sees
//   o_i = O / l, rounded once; a row that sees no key gives 0
// The weights 2^(u - m) are rounded to the operands' type for the second product (kind::f16 takes no
// fp32 operand): half a step each, in sums where the errors average out; l adds the unrounded weights.
//
// Bound: the softmax's exp2 work and the tensor cores about equally (a 128 x 128 score tile of d = 128 takes
// 1024 tensor cycles and about 1300 of exp2, sums and conversions on the other pipes).
//
// Rows: the query heads that share a key head are rows of the same tile (row = token * G + head in
// group).  An item is a pair of 128-row tiles of one (sequence, key head) that share each key tile; the
// two are the streams 0 and 1 of a CTA, and while the tensor core works on one the softmax of the other runs.
// One CTA per SM walks through its share of all items' key tiles (PairWalk): no start-up, no empty pipeline
// between items, and the last product of one item is followed by the first scores of the next.
//
// CTA: 12 warps, 512 TMEM columns, about 226 KB of shared memory.
//   warp 0      TMA: Q tiles, K and V tiles of 128 keys through one ring, K0 V0 K1 V1 ...
//   warp 1      MMA issuer of both streams; allocates TMEM
//   warp 2      walks through the share and posts its segments to the other warps (PairSegment)
//   warps 4-7   softmax and output of stream 0 (thread = query row = TMEM lane), warps 8-11 of stream 1
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <cstdint>

#include "attn16_device.cuh"
#include "attn16_kernels.cuh"
#include "attn16_softmax.cuh"
#include "workspace.cuh"

namespace sage {
namespace {

constexpr int kThreads = 384;
constexpr int kWarps = kThreads / 32;
constexpr int kRows = 256;  // rows of an item
constexpr int kPosts = 8;    // segments posted ahead
constexpr int kReaders = 10;  // warps that read them

template <int D>
struct PairLayout {
  static constexpr int BOX = 128 * 128;      // 128 rows of 64 channels (128-byte rows)
  static constexpr int TILE = BOX * (D / 64);  // one Q, K or V tile
  static constexpr int NS = D == 128 ? 5 : 8;   // ring stages
  static constexpr int QB = D == 128 ? 1 : 2;   // Q buffers per stream: few keys leave no time to fetch one in between
  static constexpr bool STAGED = D == 64;       // O leaves through shared memory (there is none left at d = 128)
  static constexpr int OFF_Q = 0;
  static constexpr int OFF_RING = 2 * QB * TILE;
  static constexpr int OFF_STAGE = OFF_RING + NS * TILE;  // 32 rows of 128 bytes for each softmax warp
  static constexpr int OFF_BAR = OFF_STAGE + (STAGED ? 8 * 4096 : 0);
  static constexpr int NUM_BARS = 2 * NS + 2 * 2 * QB + 4 * 2 + 1 + 2 * kPosts;
  static constexpr int OFF_POSTS = (OFF_BAR + NUM_BARS * 8 + 15) / 16 * 16;
  static constexpr int OFF_MISC = OFF_POSTS + kPosts * 64;
  static constexpr int SMEM = OFF_MISC + 16 + 1024;
  static_assert(SMEM <= 227 * 1024, "shared memory budget");
  static_assert(SMEM > 114 * 1024, "one CTA per SM: each allocates all of TMEM");
};

// ---- the axis of key tiles: items in the order sequence, key head, pair
__device__ __forceinline__ int pair_units(const Attn16Args& a, const Sequence& s, int p) {
  return max(1, key_tiles(a, s, 2 * a.tile_tokens * p, 2 * a.tile_tokens));
}
__device__ __forceinline__ int pairs_of(const Attn16Args& a, const Sequence& s) {
  return (s.nq + 2 * a.tile_tokens - 1) / (2 * a.tile_tokens);
}
// key tiles of one key head of a sequence
__device__ __forceinline__ long long head_units(const Attn16Args& a, const Sequence& s) {
  const int pairs = pairs_of(a, s);
  if (!a.causal) return pairs > 0 ? static_cast<long long>(pairs) * pair_units(a, s, 0) : 0;
  long long sum = 0;
  for (int p = 0; p < pairs; ++p) sum += pair_units(a, s, p);
  return sum;
}
__device__ __forceinline__ long long share_of(const Attn16Args& a, long long total, int ctas) {
  const long long even = (total + ctas - 1) / ctas;
  return max(even, static_cast<long long>(a.min_chunk));
}

// Part of an item: key tiles [first, first + steps), n0 and n1 of them for the two streams (n1 >= n0 where both
// exist: its tokens see further).  64 bytes, as posted in shared memory.
struct __align__(16) PairSegment {
  int b, token0, nq, kv;              // the sequence
  int tok0, hk, q_tiles, first;
  int n0, n1, steps, part;
  int whole, end, unused0, unused1;   // end: no segment, the share is done
  __device__ __forceinline__ int n(int t) const { return t ? n1 : n0; }
  __device__ __forceinline__ Sequence seq() const { return Sequence{b, token0, nq, kv}; }
};
static_assert(sizeof(PairSegment) == 64, "posted as four 16-byte pieces");

// Slot -> pair p of sequence b; some slots have no pair (false).  By a whole warp.
__device__ __forceinline__ bool slot_pair(const Attn16Args& a, int slot, Sequence& seq, int& p) {
  const int cta_tokens = 2 * a.tile_tokens;
  if (!a.cu_q) {
    const int per_b = (a.Nq + cta_tokens - 1) / cta_tokens;
    seq = sequence(a, slot / per_b);
    p = slot % per_b;
    return true;
  }
  const int upto = sequences_upto(a, cta_tokens, slot);
  if (upto == 0) return false;
  seq = sequence(a, upto - 1);
  p = slot - (seq.token0 / cta_tokens + seq.b);
  return p >= 0 && p < pairs_of(a, seq);  // (negative: cu_q is not ascending)
}

// A CTA's walk through its share.
// a.cut (few items): all items' key tiles form one axis, cut into equal shares wherever that falls; items that
// a cut goes through are joined from parts.  Else the items are dealt out in turn, the last (causal: longest)
// pairs first, so that neighbouring CTAs work on the same keys.
struct PairWalk {
  long long u, end;  // cut: place on the axis, end of the share; else: number of the next item, number of items
  Sequence seq;
  int pairs, p, hk, off;
  bool started, first_item;

  __device__ __forceinline__ void step(const Attn16Args& a) {
    off = 0;
    if (++p < pairs) return;
    p = 0;
    if (++hk < a.Hk) return;
    hk = 0;
    do {  // the walk goes on only where there is another item
      seq = sequence(a, seq.b + 1);
      pairs = pairs_of(a, seq);
    } while (pairs == 0);
  }

  // cut: u is a place in sequence b, which begins at `prefix`
  __device__ __forceinline__ void start(const Attn16Args& a, int b, long long prefix) {
    started = false;
    first_item = true;
    if (!a.cut) return;
    seq = sequence(a, b);
    pairs = pairs_of(a, seq);
    const long long head = head_units(a, seq);
    long long rest = u - prefix;
    hk = static_cast<int>(rest / head);
    rest -= hk * head;
    p = 0;
    if (a.causal) {
      for (int n; rest >= (n = pair_units(a, seq, p)); ++p) rest -= n;
    } else {
      const int n = pair_units(a, seq, 0);
      p = static_cast<int>(rest / n);
      rest -= static_cast<long long>(p) * n;
    }
    off = static_cast<int>(rest);
  }

  __device__ __forceinline__ bool next(const Attn16Args& a, PairSegment& g) {
    int take;
    if (a.cut) {
      if (u >= end) return false;
      if (started) step(a);
      started = true;
      const int n = pair_units(a, seq, p);
      take = static_cast<int>(min(static_cast<long long>(n - off), end - u));
      g.whole = take == n;
      u += take;
    } else {
      do {
        if (u >= end) return false;
        hk = static_cast<int>(u / a.slots);
        const int slot = a.slots - 1 - static_cast<int>(u % a.slots);
        u += gridDim.x;
        if (slot_pair(a, slot, seq, p)) break;
      } while (true);
      off = 0;
      take = pair_units(a, seq, p);
      g.whole = true;
    }
    g.b = seq.b, g.token0 = seq.token0, g.nq = seq.nq, g.kv = seq.kv;
    g.end = 0;
    g.tok0 = 2 * a.tile_tokens * p;
    g.hk = hk;
    g.first = off;
    g.q_tiles = g.tok0 + a.tile_tokens < seq.nq ? 2 : 1;
    const int last = off + take;
    g.n0 = max(0, min(last, key_tiles(a, seq, g.tok0, a.tile_tokens)) - off);
    g.n1 = g.q_tiles == 2 ? max(0, min(last, key_tiles(a, seq, g.tok0 + a.tile_tokens, a.tile_tokens)) - off) : 0;
    g.steps = max(g.n0, g.n1);
    // a CTA has at most two parts: of its first item and of its last
    g.part = 2 * static_cast<int>(blockIdx.x) + (first_item ? 0 : 1);
    first_item = false;
    return true;
  }
};

template <int WARPS>
__device__ __forceinline__ long long block_sum(long long v, long long* scratch) {
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) v += __shfl_xor_sync(0xffffffffu, v, off);
  __syncthreads();
  if ((threadIdx.x & 31) == 0) scratch[threadIdx.x >> 5] = v;
  __syncthreads();
  long long sum = 0;
#pragma unroll
  for (int w = 0; w < WARPS; ++w) sum += scratch[w];
  return sum;
}

// This CTA's share of the axis into walk.u and walk.end, with the sequence it begins in and that one's place on
// the axis; false: there is no such share.  scratch: kWarps + 2 values.
__device__ __forceinline__ bool find_share(const Attn16Args& a, long long* scratch, PairWalk& walk, long long& share,
                                           int& first_b, long long& prefix) {
  constexpr int WARPS = kWarps;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  long long mine = 0;
  for (int b = threadIdx.x; b < a.B; b += 32 * WARPS) mine += head_units(a, sequence(a, b)) * a.Hk;
  const long long total = block_sum<WARPS>(mine, scratch);
  share = share_of(a, total, gridDim.x);
  walk.u = blockIdx.x * share;
  walk.end = min(total, walk.u + share);
  if (walk.u >= walk.end) return false;
  first_b = 0;
  prefix = 0;
  if (a.B > 1) {  // a scan over the sequences, a block at a time
    long long before = 0;
    for (int base = 0; base < a.B; base += 32 * WARPS) {
      const int b = base + static_cast<int>(threadIdx.x);
      const long long len = b < a.B ? head_units(a, sequence(a, b)) * a.Hk : 0;
      long long incl = len;
#pragma unroll
      for (int off = 1; off < 32; off <<= 1) {
        const long long v = __shfl_up_sync(0xffffffffu, incl, off);
        if (lane >= off) incl += v;
      }
      __syncthreads();
      if (lane == 31) scratch[warp] = incl;
      __syncthreads();
      long long sum = before;
      for (int w = 0; w < WARPS; ++w) {
        if (w < warp) incl += scratch[w];
        sum += scratch[w];
      }
      const long long at = before + incl - len;
      if (walk.u >= at && walk.u < at + len) {
        scratch[WARPS] = b;
        scratch[WARPS + 1] = at;
      }
      before = sum;
      if (before > walk.u) break;
    }
    __syncthreads();
    first_b = static_cast<int>(scratch[WARPS]);
    prefix = scratch[WARPS + 1];
  }
  return true;
}

template <int D, bool BF16>
__global__ void __launch_bounds__(kThreads, 1)
    attn_pair_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
                     const __grid_constant__ CUtensorMap tm_v, const __grid_constant__ Attn16Args a) {
  using L = PairLayout<D>;
  using C = Columns<D>;
  constexpr int NS = L::NS, NB = D / 64, QB = L::QB;
  constexpr bool OWN_P = kOwnWeights<D>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* sQ = smem + L::OFF_Q;
  uint8_t* sRing = smem + L::OFF_RING;
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + L::OFF_BAR);
  uint64_t* bar_full = bars;
  uint64_t* bar_empty = bar_full + NS;
  uint64_t* bar_q_full = bar_empty + NS;       // [2 streams][QB]
  uint64_t* bar_q_free = bar_q_full + 2 * QB;  // [2 streams][QB] the segment's last scores are computed
  // [2], one per stream:
  uint64_t* bar_s_full = bar_q_free + 2 * QB;  // scores of a key tile (and every product before them) done
  uint64_t* bar_s_free = bar_s_full + 2;  // scores in registers (OWN_P)
  uint64_t* bar_p_full = bar_s_free + 2;  // weights written
  uint64_t* bar_pv = bar_p_full + 2;      // second product done (OWN_P: each; else: the segment's last)
  uint64_t* bar_drain = bar_pv + 2;
  uint64_t* bar_posted = bar_drain + 1;       // [kPosts] a segment is posted
  uint64_t* bar_read = bar_posted + kPosts;   // [kPosts] all readers have it
  PairSegment* posts = reinterpret_cast<PairSegment*>(smem + L::OFF_POSTS);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + L::OFF_MISC);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + L::OFF_MISC + 4);
  // the start-up's scratch lies in the ring, which the TMA fills only later
  long long* scratch = reinterpret_cast<long long*>(sRing);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  // ---- this CTA's share
  PairWalk walk;
  int first_b = 0;
  long long prefix = 0, share;
  if (a.cut) {
    if (!find_share(a, scratch, walk, share, first_b, prefix)) {
      if (threadIdx.x == 0 && a.cuts) a.cuts[blockIdx.x] = CutNote{};  // no cut
      return;
    }
  } else {
    walk.u = blockIdx.x;
    walk.end = static_cast<long long>(a.slots) * a.Hk;
  }
  walk.start(a, first_b, prefix);
  if (a.cut && threadIdx.x == 0 && a.cuts)
    a.cuts[blockIdx.x] = CutNote{walk.u - walk.off, share, walk.seq.b, walk.seq.token0, walk.seq.nq,
                                 2 * a.tile_tokens * walk.p, walk.hk, walk.off, pair_units(a, walk.seq, walk.p)};

  if (threadIdx.x == 0) {
    for (int i = 0; i < NS; ++i) {
      mbar_init(bar_full + i, 1);
      mbar_init(bar_empty + i, 1);
    }
    for (int t = 0; t < 2; ++t) {
      for (int i = 0; i < QB; ++i) {
        mbar_init(bar_q_full + t * QB + i, 1);
        mbar_init(bar_q_free + t * QB + i, 1);
      }
      mbar_init(bar_s_full + t, 1);
      mbar_init(bar_s_free + t, 128);
      mbar_init(bar_p_full + t, 128);
      mbar_init(bar_pv + t, 1);
    }
    mbar_init(bar_drain, 1);
    for (int i = 0; i < kPosts; ++i) {
      mbar_init(bar_posted + i, 1);
      mbar_init(bar_read + i, kReaders);
    }
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
  fence_proxy_async_shared();  // the scratch was written and read by ordinary accesses; the TMA writes there next
  tc_fence_before();
  cta_sync();  // lane 0 of warp 0 initialised the barriers alone
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  auto wait = [&](uint64_t* bar, uint32_t parity) {
    return __all_sync(0xffffffffu, mbar_wait(bar, parity, abort_flag));
  };

  auto wait_idle = [&](uint64_t* bar, uint32_t parity) {
    return __all_sync(0xffffffffu, mbar_wait_idle(bar, parity, abort_flag));
  };
  // segment i of the share into the registers of a reading warp; false: the share is done (or a wait gave up)
  auto read_post = [&](int i, PairSegment& g) -> bool {
    if (!wait(bar_posted + i % kPosts, (i / kPosts) & 1)) {
      g.end = 1;
      return false;
    }
    g = posts[i % kPosts];
    __syncwarp();
    if (lane == 0) mbar_arrive(bar_read + i % kPosts);
    return g.end == 0;
  };

  // Registers: launched with 168 per thread (384 x 168); 128 x 72 + 256 x 216 is the same total.  Each
  // setmaxnreg is executed by a whole warpgroup and dominates that group's code.
  if (warp < 4) {
    reg_dealloc<72>();
    if (warp == 0) {
      // ============================================================ TMA (the whole warp; lane i issues the
      // copies of the tile's page i).  A stream's Q is asked for behind the segment's first K and V: its
      // buffer is free only when the segment before has used it, and the ring goes on meanwhile.
      const int page = 1 << a.page_shift;
      const int pages_per_tile = a.page_table && page < 128 ? 128 >> a.page_shift : 1;
      const int rows_per_copy = 128 / pages_per_tile;
      PairSegment seg;
      int fill = 0, nq[2] = {0, 0};
      bool ok = true;
      for (int i = 0; ok && read_post(i, seg); ++i) {
        if (seg.steps == 0) continue;
        // outer coordinate of this lane's copy of key tile kt; pages past the sequence or outside the
        // cache take a coordinate past the tensor, which reads as zeros and counts its bytes
        auto page_of = [&](int kt) -> int {
          if (!a.page_table) return seg.b;
          const int key = kt * 128 + lane * rows_per_copy;
          int p = -1;
          if (lane < pages_per_tile && key < seg.kv)
            p = __ldg(a.page_table + static_cast<long long>(seg.b) * a.pages_per_seq + (key >> a.page_shift));
          return p < 0 || p >= a.num_pages ? a.num_pages : p;
        };
        int outer = page_of(seg.first);
        for (int j = 0; ok && j < seg.steps; ++j) {
          const int kt = seg.first + j;
          const int next = j + 1 < seg.steps ? page_of(kt + 1) : 0;  // in flight during this tile's waits
          const int row = a.page_table ? (kt * 128) & (page - 1) : kt * 128;
          for (int kind = 0; kind < 2; ++kind, ++fill) {
            const int st = fill % NS;
            if (fill >= NS && !wait_idle(bar_empty + st, (fill / NS - 1) & 1)) {
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
          if (j > 0) continue;
#pragma unroll
          for (int t = 0; t < 2; ++t) {
            if (!ok || seg.n(t) == 0) continue;
            const int buf = t * QB + nq[t] % QB;
            if (nq[t] >= QB && !wait(bar_q_free + buf, (nq[t] / QB - 1) & 1)) {
              ok = false;
              continue;
            }
            if (lane == 0) {
              mbar_arrive_expect_tx(bar_q_full + buf, static_cast<uint32_t>(a.tile_tokens * a.G * NB * 128));
              for (int c = 0; c < NB; ++c)
                tma_load_5d(sQ + buf * L::TILE + c * L::BOX, &tm_q, bar_q_full + buf, 64 * c, 0,
                            seg.token0 + seg.tok0 + t * a.tile_tokens, seg.hk, a.cu_q ? 0 : seg.b);
            }
            __syncwarp();
            ++nq[t];
          }
        }
      }
      if (*abort_flag && lane == 0) {  // let copies in flight land before the CTA exits
        for (int f = max(0, fill - NS); f < fill; ++f) mbar_drain(bar_full + f % NS, (f / NS) & 1);
#pragma unroll
        for (int t = 0; t < 2; ++t)
          for (int i = max(0, nq[t] - QB); i < nq[t]; ++i) mbar_drain(bar_q_full + t * QB + i % QB, (i / QB) & 1);
      }
    } else if (warp == 1) {
      // ============================================================ MMA issuer of both streams, in turn: the
      // second product of one and its next scores (of the next segment after the last), then the other's.
      // The tensor core so finishes one stream's scores a whole turn before the other's, and the streams'
      // softmax work falls into each other's product time.  (Issued by a warp per stream, the products of both
      // finish together and the softmax warps work at the same time and wait at the same time: 4470 cycles a turn
      // of two 128 x 128 tiles of d = 128 instead of 3330.)
      constexpr uint32_t FMT = BF16 ? 1u : 0u;
      constexpr uint32_t IDESC_QK = make_idesc(1 /*f32*/, FMT, FMT, 0, 0, 128, 128);
      constexpr uint32_t IDESC_PV = make_idesc(1 /*f32*/, FMT, FMT, 0, 1 /*V is MN-major*/, 128, D);
      const uint32_t q_base = smem_u32(sQ), ring = smem_u32(sRing);
      struct Steps {  // what this warp needs of a segment
        int n0, n1, steps, keys;  // keys: of the sequence, from the segment's first tile on
        __device__ __forceinline__ int n(int t) const { return t ? n1 : n0; }
      };
      int posted = 0;
      // The next segment, whether or not it has keys to read.  (Not the next one that has: the posts in between come
      // only when those before are free, and the softmax warps hold on to theirs until this warp has gone on.)
      auto next_steps = [&](Steps& g) -> bool {
        PairSegment x;
        if (!read_post(posted, x)) {
          g = Steps{0, 0, 0, 0};
          return false;
        }
        ++posted;
        g = Steps{x.n0, x.n1, x.steps, x.kv - x.first * 128};
        return true;
      };
      Steps seg{0, 0, 0, 0}, ahead;
      int base = 0;                // ring fill of the segment's first K; step it: K base + 2 it, V base + 2 it + 1
      int scores[2] = {0, 0};      // score tiles issued for each stream so far
      int weights[2] = {0, 0};     // weight tiles used
      int nq[2] = {0, 0};          // Q tiles used
      auto full = [&](int fill) { return wait(bar_full + fill % NS, (fill / NS) & 1); };
      // the products themselves; t is a compile-time value
      auto mma_qk = [&](auto t, int fill) {
        tc_fence_after();
#pragma unroll
        for (int c = 0; c < NB; ++c)  // 16 channels per product: 32 bytes inside a 128-byte swizzled row
          mma_f16_ss_x4_warp<2, 2>(tmem + C::s(t), make_smem_desc(q_base + (t * QB + (nq[t] - 1) % QB) * L::TILE + c * L::BOX, 16, 1024, kSwizzle128B),
                                   make_smem_desc(ring + (fill % NS) * L::TILE + c * L::BOX, 16, 1024, kSwizzle128B),
                                   IDESC_QK, c > 0 ? 1u : 0u);
        mma_commit_warp(bar_s_full + t);
      };
      auto mma_pv = [&](auto t, int fill, bool first) {
        tc_fence_after();
#pragma unroll
        for (int half = 0; half < 2; ++half)  // 64 keys, 16 per product
          mma_f16_ts_x4_warp<8, 16 * 128 / 16>(tmem + C::o(t), tmem + C::p(t) + half * 32,
                                               make_smem_desc(ring + (fill % NS) * L::TILE + half * 64 * 128, L::BOX, 1024, kSwizzle128B),
                                               IDESC_PV, first && half == 0 ? 0u : 1u);
      };
      // scores of stream t, step it of segment g whose first K is fill b.  A key tile is waited for in its
      // first stream's turn and freed in its last one's.
      auto issue_qk = [&](const Steps& g, int b, auto t, int it) -> bool {
        const int fill = b + 2 * it;
        if ((t == 0 || it >= g.n0) && !full(fill)) return false;
        if (it == 0) {
          const int i = nq[t]++;
          if (!wait(bar_q_full + t * QB + i % QB, (i / QB) & 1)) return false;
        }
        if (OWN_P && scores[t] > 0 && !wait(bar_s_free + t, (scores[t] - 1) & 1)) return false;
        ++scores[t];
        mma_qk(t, fill);
        if (t == 1 || it >= g.n1) mma_commit_warp(bar_empty + fill % NS);
        if (it + 1 == g.n(t)) mma_commit_warp(bar_q_free + t * QB + (nq[t] - 1) % QB);
        return true;
      };
      auto issue_pv = [&](const Steps& g, int b, auto t, int it) -> bool {
        const int fill = b + 2 * it + 1;
        if (t == 0 || it >= g.n0) {
          if (!full(fill)) return false;
          const int valid = g.keys - it * 128;
          if (valid < 128) zero_v_tail<D>(sRing + (fill % NS) * L::TILE, valid, lane);
        }
        if (!wait(bar_p_full + t, weights[t]++ & 1)) return false;
        mma_pv(t, fill, it == 0);
        if (t == 1 || it >= g.n1) mma_commit_warp(bar_empty + fill % NS);
        if (OWN_P || it + 1 == g.n(t)) mma_commit_warp(bar_pv + t);
        return true;
      };
      const std::integral_constant<int, 0> s0{};
      const std::integral_constant<int, 1> s1{};
      // (a segment without steps still has a turn, which issues the first scores of the one behind it)
      bool more = next_steps(seg), ok = true;
      if (more && seg.n0 > 0) ok = issue_qk(seg, base, s0, 0);
      if (more && ok && seg.n1 > 0) ok = issue_qk(seg, base, s1, 0);
      while (more && ok) {
        more = next_steps(ahead);
        int it = 0;
        // the bulk of a segment: both streams have this tile and the next two, none of the rest applies
        for (; ok && it + 2 < min(seg.n0, seg.n1); ++it) {
          const int kf = base + 2 * it + 2, vf = kf - 1;
          auto qk = [&](auto t) -> bool {
            if (t == 0 && !full(kf)) return false;
            if (OWN_P && !wait(bar_s_free + t, (scores[t] - 1) & 1)) return false;
            ++scores[t];
            mma_qk(t, kf);
            if (t == 1) mma_commit_warp(bar_empty + kf % NS);
            return true;
          };
          auto pv = [&](auto t) -> bool {
            if (t == 0 && !full(vf)) return false;
            if (!wait(bar_p_full + t, weights[t]++ & 1)) return false;
            mma_pv(t, vf, it == 0);
            if (t == 1) mma_commit_warp(bar_empty + vf % NS);
            if (OWN_P) mma_commit_warp(bar_pv + t);
            return true;
          };
          if constexpr (OWN_P) ok = qk(s0) && pv(s0) && qk(s1) && pv(s1);
          else ok = pv(s0) && qk(s0) && pv(s1) && qk(s1);
        }
        for (; ok && it < max(seg.steps, 1); ++it) {
          const bool last = it + 1 >= seg.steps;
          auto turn = [&](auto t) -> bool {
            // what follows: the stream's next step, or, in the segment's last step, the next segment's first
            auto follow = [&]() -> bool {
              if (it + 1 < seg.n(t)) return issue_qk(seg, base, t, it + 1);
              if (last && more && ahead.n(t) > 0) return issue_qk(ahead, base + 2 * seg.steps, t, 0);
              return true;
            };
            const bool has = it < seg.n(t);
            // (the next segment's Q may be on its way still: the last product goes first)
            if (OWN_P && !last) return follow() && (!has || issue_pv(seg, base, t, it));
            return (!has || issue_pv(seg, base, t, it)) && follow();
          };
          ok = turn(s0) && turn(s1);
        }
        base += 2 * seg.steps;
        seg = ahead;
      }
      // all MMAs must finish before TMEM is released
      mma_commit_warp(bar_drain);
      mbar_drain(bar_drain, 0);
    } else if (warp == 2) {
      // ============================================================ the walk
      PairSegment seg;
      for (int i = 0;; ++i) {
        if (!walk.next(a, seg)) seg.end = 1;
        if (i >= kPosts && !wait_idle(bar_read + i % kPosts, (i / kPosts - 1) & 1)) break;
        if (lane == 0) {
          posts[i % kPosts] = seg;
          mbar_arrive(bar_posted + i % kPosts);
        }
        __syncwarp();
        if (seg.end) break;
      }
    }
  } else {
    reg_alloc<216>();
    // ============================================================ softmax and output: thread = query row
    const int t = (warp - 4) >> 2;
    const int quad = warp & 3;  // TMEM lane quadrant this warp may access
    const int r = quad * 32 + lane;
    const uint32_t lane_addr = static_cast<uint32_t>(quad * 32) << 16;
    const uint32_t tS = tmem + lane_addr + C::s(t), tO = tmem + lane_addr + C::o(t), tP = tmem + lane_addr + C::p(t);
    const int r_tok = t * a.tile_tokens + r / a.G, r_head = r % a.G;  // the row's token within an item, its head in the group
    int tiles = 0, done = 0;  // score tiles taken, segments with keys finished
    bool ok = true;
    for (int i = 0; ok && wait(bar_posted + i % kPosts, (i / kPosts) & 1); ++i) {
      // the post is held until the output: of its numbers only these few live through the tiles
      const PairSegment* seg = posts + i % kPosts;
      if (seg->end) break;
      const int n = seg->n(t);
      RowState row;
      row.clear();
      bool warp_live;  // else what stands in the warp's lanes is never stored
      {
        const Sequence sq = seg->seq();
        const int tok = seg->tok0 + r_tok;
        const bool row_valid = r < a.tile_tokens * a.G && tok < sq.nq;
        warp_live = __any_sync(0xffffffffu, row_valid);
        int lim = visible(a, sq, tok) - seg->first * 128;  // the row sees keys [0, lim) of the segment's
        const int lim_warp = __reduce_min_sync(0xffffffffu, row_valid ? lim : 0x7fffffff);
        const int lim_most = __reduce_max_sync(0xffffffffu, row_valid ? lim : 0);
        auto prior = [&]() -> bool {  // (d = 128: the last product precedes these scores)
          if (!OWN_P || tiles == 0) return true;
          const bool w = wait(bar_pv + t, (tiles - 1) & 1);
          tc_fence_after();
          return w;
        };
        for (int it = 0; ok && it < n; ++it, ++tiles) {
          if (!wait(bar_s_full + t, tiles & 1)) { ok = false; break; }
          tc_fence_after();
          if (warp_live) {
            ok = softmax_tile<D, BF16>(row, tS, tO, tP, lim - it * 128, lim_warp - it * 128, lim_most - it * 128, it == 0, a.scale_log2,
                                       bar_s_free + t, prior);
            tmem_wait_st();
            tc_fence_before();
          } else if (OWN_P) {
            // one arrival per tile: the next scores may come before the other warps' weights of this tile
            mbar_arrive(bar_s_free + t);
            ok = prior();
          }
          mbar_arrive(bar_p_full + t);
        }
      }
      if (!ok) break;
      // ---- output of the item, or its part
      const float l = row.sum();
      if (n > 0) {
        if (!wait(bar_pv + t, (OWN_P ? tiles - 1 : done) & 1)) break;
        tc_fence_after();
        ++done;
      }
      if (warp_live && t < seg->q_tiles) {
        const Sequence sq = seg->seq();
        const int tok = seg->tok0 + r_tok;
        const bool row_valid = r < a.tile_tokens * a.G && tok < sq.nq;
        const bool whole = seg->whole;
        const float scale = whole ? weight_sum_inverse(l) : 1.f;
        uint16_t* orow = static_cast<uint16_t*>(a.o) + out_offset(a, sq, tok, seg->hk * a.G + r_head);
        const long long part = static_cast<long long>(seg->part) * kRows + t * 128 + r;
        if (!whole && row_valid) a.part_ml[part] = make_float2(row.m_use, l);
        uint8_t* stage = smem + L::OFF_STAGE + (warp - 4) * 4096;  // [32 rows][8 pieces], piece p of row i at p ^ (i & 7)
        __half2 most[4] = {};
#pragma unroll
        for (int cb = 0; cb < D; cb += 32) {
          uint32_t ov[32];
          if (n > 0) {
            tmem_ld32_sync(tO + cb, ov);
          } else {
#pragma unroll
            for (int i = 0; i < 32; ++i) ov[i] = 0u;
          }
          if (whole) {
            uint32_t w[16];
            pack_means<BF16>(ov, scale, w, most);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const uint4 v = make_uint4(w[4 * i], w[4 * i + 1], w[4 * i + 2], w[4 * i + 3]);
              if constexpr (L::STAGED) *reinterpret_cast<uint4*>(stage + lane * 128 + (((cb / 8 + i) ^ (lane & 7)) << 4)) = v;
              else if (row_valid) *reinterpret_cast<uint4*>(orow + cb + 8 * i) = v;
            }
          } else if (row_valid) {
            {
              uint4* dst = reinterpret_cast<uint4*>(a.part_o + part * D + cb);
#pragma unroll
              for (int i = 0; i < 8; ++i) dst[i] = make_uint4(ov[4 * i], ov[4 * i + 1], ov[4 * i + 2], ov[4 * i + 3]);
            }
          }
        }
        if (out_of_range<BF16>(most)) {  // (parts have none)
#pragma unroll 1
          for (int cb = 0; cb < D; cb += 8) {
            uint32_t ov[8], w[4];
            tmem_ld8_sync(tO + cb, ov);
#pragma unroll
            for (int i = 0; i < 4; ++i) w[i] = pack_in_range<BF16>(__uint_as_float(ov[2 * i]) * scale, __uint_as_float(ov[2 * i + 1]) * scale);
            const uint4 v = make_uint4(w[0], w[1], w[2], w[3]);
            if constexpr (L::STAGED) *reinterpret_cast<uint4*>(stage + lane * 128 + (((cb / 8) ^ (lane & 7)) << 4)) = v;
            else if (row_valid) *reinterpret_cast<uint4*>(orow + cb) = v;
          }
        }
        if (L::STAGED && whole) {
          // four whole rows per instruction (a row per lane would be 32 lines each: 8 of them hold up the
          // load-store unit for 256 cycles a warp)
          __syncwarp();
          const unsigned long long at = row_valid ? reinterpret_cast<unsigned long long>(orow) : 0ull;
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const int row = 4 * i + (lane >> 3);
            const unsigned long long dst = __shfl_sync(0xffffffffu, at, row);
            const uint4 v = *reinterpret_cast<const uint4*>(stage + row * 128 + (((lane & 7) ^ (row & 7)) << 4));
            if (dst) reinterpret_cast<uint4*>(dst)[lane & 7] = v;
          }
          __syncwarp();
        }
      }
      tc_fence_before();  // O is read: the arrivals of the next segment's weights order what follows
      __syncwarp();
      if (lane == 0) mbar_arrive(bar_read + i % kPosts);
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

// Joins the items that a cut went through: o = sum_s 2^(m_s - m) O_s / sum_s 2^(m_s - m) l_s, in the order of the
// parts.  Grid: the cuts between two shares x eighths of an item's rows, a warp for four rows; an item that more
// than one cut goes through is joined by its first one.
constexpr int kJoinThreads = 256;
constexpr int kJoinSplit = 8;

template <int D, bool BF16>
__global__ void __launch_bounds__(kJoinThreads) attn_pair_join_kernel(const __grid_constant__ Attn16Args a, int ctas) {
  const int lane = threadIdx.x & 31;
  cudaGridDependencySynchronize();  // the parts are written
  const CutNote cut = a.cuts[blockIdx.x + 1];
  if (cut.off == 0) return;  // no such share, or it begins with an item
  const int c0 = static_cast<int>(cut.first / cut.share), c1 = static_cast<int>((cut.first + cut.units - 1) / cut.share);
  if (c0 != static_cast<int>(blockIdx.x)) return;
  // in its first CTA the item is the last one (part 1) unless the CTA begins with it
  const bool late = cut.first % cut.share != 0;
  constexpr int PER = D / 32;  // channels per lane
  const int first_row = static_cast<int>(blockIdx.y) * (kRows / kJoinSplit) + 4 * static_cast<int>(threadIdx.x >> 5);
  static_assert(kRows / kJoinSplit == 4 * (kJoinThreads / 32), "four rows per warp");
  float acc[4][PER], l[4];
  join_parts(acc, l, c0, c1, a.part_ml, a.part_o, [&](int k, int c) {
    return static_cast<long long>(2 * c + (c == c0 && late ? 1 : 0)) * kRows + first_row + k;
  });
#pragma unroll
  for (int k = 0; k < 4; ++k) {  // (rows that do not exist joined whatever stands in their places)
    const int row = first_row + k, t = row >> 7, r = row & 127;
    const int tok = cut.tok0 + t * a.tile_tokens + r / a.G;
    if (r < a.tile_tokens * a.G && tok < cut.nq)
      store_joined<BF16>(static_cast<uint16_t*>(a.o) + lane * PER +
                             out_offset(a, Sequence{cut.b, cut.token0, cut.nq, 0}, tok, cut.hk * a.G + r % a.G),
                         acc[k], l[k]);
  }
}

template <int D, bool BF16>
cudaError_t launch_t(const Attn16Launch& l, int ctas, cudaStream_t st) {
  using L = PairLayout<D>;
  auto kern = attn_pair_kernel<D, BF16>;
  static std::atomic<unsigned long long> allowed{0};
  cudaError_t e = allow_shared_memory(allowed, reinterpret_cast<const void*>(kern), L::SMEM);
  if (e != cudaSuccess) return e;
  kern<<<ctas, kThreads, L::SMEM, st>>>(l.tm_q, l.tm_k, l.tm_v, l.a);
  e = cudaGetLastError();
  if (e != cudaSuccess || !l.a.cut || ctas == 1) return e;
  // launched early, while the attention drains: it waits on the device for the parts
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(static_cast<unsigned>(ctas) - 1, kJoinSplit);
  cfg.blockDim = dim3(kJoinThreads);
  cfg.stream = st;
  cudaLaunchAttribute attr{};
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, attn_pair_join_kernel<D, BF16>, l.a, ctas);
}

}  // namespace

size_t pair_part_rows(int ctas) { return static_cast<size_t>(ctas) * 2 * kRows; }

cudaError_t launch_attn_pair(const Attn16Launch& l, int ctas, cudaStream_t st) {
  if (l.D == 128) return l.bf16 ? launch_t<128, true>(l, ctas, st) : launch_t<128, false>(l, ctas, st);
  return l.bf16 ? launch_t<64, true>(l, ctas, st) : launch_t<64, false>(l, ctas, st);
}

int read_and_clear_pair_error(cudaStream_t st, cudaError_t* err) {
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
