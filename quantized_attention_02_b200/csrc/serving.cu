// serving.cu -- C ABI of the serving operators declared in include/sage_attn.h: argument checks and
// launches of the query / key norm with rotation, the append into a paged cache, the attention over
// it and the cross attention.
#include <cuda_runtime.h>

#include <algorithm>
#include <atomic>
#include <cmath>
#include <cstdint>

#include "attn16_kernels.cuh"
#include "rope_kernels.cuh"
#include "sage_attn.h"
#include "tensor_map.cuh"
#include "workspace.cuh"

namespace {

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

bool stride_ok(int64_t s, int64_t extent) { return extent <= 1 || (s > 0 && s % 8 == 0); }

// A view [B][H][N][d]: present, aligned, strides usable.
bool view_ok(const void* p, const sage_strides* s, int64_t B, int64_t H, int64_t N) {
  return p && s && aligned16(p) && stride_ok(s->b, B) && stride_ok(s->h, H) && stride_ok(s->n, N);
}

int check_common(int Hq, int Hk, int d, int dtype) {
  if (Hq <= 0 || Hk < 0 || d <= 0) return SAGE_ERR_INVALID;
  if (dtype != SAGE_F16 && dtype != SAGE_BF16) return SAGE_ERR_INVALID;
  if (d != 64 && d != 128) return SAGE_ERR_UNSUPPORTED;
  return SAGE_OK;
}

int check_rope(const float* cos, const float* sin, const void* qw, const void* kw, int d, int rot, int table_rows,
               bool by_token, int N, float eps) {
  if (!cos || !sin || !aligned16(cos) || !aligned16(sin) || !aligned16(qw) || !aligned16(kw)) return SAGE_ERR_INVALID;
  if (rot < 16 || rot > d || rot % 16 != 0 || table_rows <= 0) return SAGE_ERR_INVALID;
  if (by_token && table_rows < N) return SAGE_ERR_INVALID;
  return std::isfinite(eps) && eps >= 0.f ? SAGE_OK : SAGE_ERR_INVALID;
}

// log2 of a supported page size, -1 for the others
int page_shift(int page_size) {
  for (int s = 4; s <= 8; ++s)
    if (page_size == 1 << s) return s;
  return -1;
}

int check_pages(int num_pages, int page_size) {
  if (num_pages <= 0 || page_size <= 0) return SAGE_ERR_INVALID;
  if (page_shift(page_size) < 0 || static_cast<int64_t>(num_pages) * page_size >= (1ll << 31))
    return SAGE_ERR_UNSUPPORTED;
  return SAGE_OK;
}

int cuda_status(cudaError_t e) { return e == cudaSuccess ? SAGE_OK : SAGE_ERR_CUDA; }

// ---------------------------------------------------------------- 16-bit attention
int check_attn(int Hq, int Hk, int d, float sm_scale, int dtype) {
  if (Hk <= 0) return SAGE_ERR_INVALID;
  const int rc = check_common(Hq, Hk, d, dtype);
  if (rc) return rc;
  if (Hq % Hk != 0 || !(std::isfinite(sm_scale) && sm_scale > 0.f)) return SAGE_ERR_INVALID;
  return Hq / Hk <= 128 ? SAGE_OK : SAGE_ERR_UNSUPPORTED;  // a group's heads are rows of one query tile
}

// Byte stride of a dimension for a tensor map: any valid value where the extent is 1.
uint64_t map_stride(int64_t elems, int64_t extent, int d) {
  return static_cast<uint64_t>(extent > 1 ? elems : d) * 2;
}

// Strides of a view [B][H][N][d] that a tensor map takes: below 2^40 bytes, that from one group of G heads to the next
// too.  Of a dimension of one entry any stride does.
bool strides_fit(const sage_strides* s, int64_t B, int64_t H, int64_t N, int64_t G) {
  constexpr int64_t kLimit = 1ll << 38;
  return (B == 1 || s->b < kLimit) && (N == 1 || s->n < kLimit) && (H == 1 || s->h < kLimit / G);
}

// queries [B][Hk][N][G][d] from a [B][Hq][N][d] view
bool query_map(CUtensorMap* m, bool bf16, const void* q, const sage_strides& st, int B, int Hk, int G, int N, int d,
               int tile_tokens) {
  const uint64_t dims[5] = {static_cast<uint64_t>(d), static_cast<uint64_t>(G), static_cast<uint64_t>(N),
                            static_cast<uint64_t>(Hk), static_cast<uint64_t>(B)};
  const uint64_t strides[4] = {map_stride(st.h, G, d), map_stride(st.n, N, d), map_stride(st.h * G, Hk, d),
                               map_stride(st.b, B, d)};
  const uint32_t box[5] = {64u, static_cast<uint32_t>(G), static_cast<uint32_t>(tile_tokens), 1u, 1u};
  return sage::encode_tiled_16bit(m, bf16, q, 5, dims, strides, box);
}

// keys or values [outer][Hk][rows][d]: outer = batch entries, or a cache's pages
bool key_map(CUtensorMap* m, bool bf16, const void* k, const sage_strides& st, int outer, int Hk, int rows, int d,
             int box_rows) {
  const uint64_t dims[4] = {static_cast<uint64_t>(d), static_cast<uint64_t>(rows), static_cast<uint64_t>(Hk),
                            static_cast<uint64_t>(outer)};
  const uint64_t strides[3] = {map_stride(st.n, rows, d), map_stride(st.h, Hk, d), map_stride(st.b, outer, d)};
  const uint32_t box[4] = {64u, static_cast<uint32_t>(box_rows), 1u, 1u};
  return sage::encode_tiled_16bit(m, bf16, k, 4, dims, strides, box);
}

int sm_count() {
  static std::atomic<int> counts[64];
  int dev = 0, sms = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return 0;
  if (dev < 64 && (sms = counts[dev].load(std::memory_order_relaxed)) > 0) return sms;
  if (cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) return 0;
  if (dev < 64) counts[dev].store(sms, std::memory_order_relaxed);
  return sms;
}

// fp32 parts of `rows` rows: O, then (m, l), then the notes of `ctas` shares.  Stream-ordered, freed by part_free.
int part_alloc(sage::Attn16Args& a, void** ws, int64_t rows, int ctas, int d, cudaStream_t st) {
  const size_t o_bytes = static_cast<size_t>(rows) * d * sizeof(float), ml_bytes = static_cast<size_t>(rows) * sizeof(float2);
  if (sage::workspace_alloc(ws, o_bytes + ml_bytes + ctas * sizeof(sage::CutNote), st) != cudaSuccess) {
    cudaGetLastError();
    return SAGE_ERR_NOMEM;
  }
  a.part_o = static_cast<float*>(*ws);
  a.part_ml = reinterpret_cast<float2*>(static_cast<uint8_t*>(*ws) + o_bytes);
  a.cuts = reinterpret_cast<sage::CutNote*>(static_cast<uint8_t*>(*ws) + o_bytes + ml_bytes);
  return SAGE_OK;
}
int part_free(void* ws, int rc, cudaStream_t st) {
  if (!ws) return rc;
  const cudaError_t fe = cudaFreeAsync(ws, st);
  return !rc && fe != cudaSuccess ? SAGE_ERR_CUDA : rc;
}

// Few rows: one axis of key units over all sequences, cut into equal shares.
int run_step(const sage::Attn16Launch& t, cudaStream_t st) {
  const int sms = sm_count();
  if (sms <= 0) return SAGE_ERR_CUDA;
  sage::StepLaunch l{{t.a, t.a.tile_tokens}, t.tm_q, t.tm_k, t.tm_v, t.D, t.bf16};
  const int ctas = sage::step_ctas(l.s, sms);
  void* ws = nullptr;
  int rc = SAGE_OK;
  if (ctas > 1 && (rc = part_alloc(l.s.a, &ws, static_cast<int64_t>(sage::step_part_rows(ctas)), ctas, l.D, st))) return rc;
  return part_free(ws, cuda_status(sage::launch_attn_step(l, ctas, st)), st);
}

// Pairs of query tiles: many items are dealt out whole, few have their key tiles cut into equal shares (of 512
// keys at least).  Replays of a graph, cold L2: 16 sequences of up to 333 tokens over up to 4099 keys, 2.4 items per SM,
// 161 us cut, 180 whole (the last round is not full); a chunk of 2048 tokens over 16384 keys, 1.8 per SM, 434 cut, 455
// whole; 2 x 4096 tokens over 6001 keys, 6.9 per SM, 663 cut (parts and joins), 635 whole.
int run_pair(sage::Attn16Launch& l, cudaStream_t st) {
  sage::Attn16Args& a = l.a;
  const int sms = sm_count();
  if (sms <= 0) return SAGE_ERR_CUDA;
  const int64_t items = static_cast<int64_t>(a.slots) * a.Hk;
  if (items >= (1ll << 31)) return SAGE_ERR_UNSUPPORTED;
  a.cut = items < 4ll * sms;
  a.min_chunk = 4;
  const int64_t units = items * std::max<int64_t>(1, (a.Nk + 127ll) / 128);
  const int ctas = static_cast<int>(std::min<int64_t>(sms, a.cut ? (units + a.min_chunk - 1) / a.min_chunk : items));
  void* ws = nullptr;
  int rc = SAGE_OK;
  if (a.cut && ctas > 1 && (rc = part_alloc(a, &ws, static_cast<int64_t>(sage::pair_part_rows(ctas)), ctas, l.D, st))) return rc;
  return part_free(ws, cuda_status(sage::launch_attn_pair(l, ctas, st)), st);
}

// One tile of query rows per CTA.  Fewer CTAs than SMs: the key axis is split so that each SM has a part, of 512 keys
// at least.  How many parts a sequence really has follows on the device from its length.
int run_tile(sage::Attn16Launch& l, int64_t ctas, cudaStream_t st) {
  sage::Attn16Args& a = l.a;
  const int sms = sm_count();
  if (sms <= 0) return SAGE_ERR_CUDA;
  a.min_chunk = 4;
  const int64_t tiles = (a.Nk + 127ll) / 128;
  a.splits = static_cast<int>(std::max<int64_t>(1, std::min<int64_t>(sms / std::max<int64_t>(ctas, 1),
                                                                     (tiles + a.min_chunk - 1) / a.min_chunk)));
  if (static_cast<int64_t>(a.slots) * a.splits * a.Hk >= (1ll << 31)) return SAGE_ERR_UNSUPPORTED;
  void* ws = nullptr;
  int rc = SAGE_OK;
  if (a.splits > 1 && (rc = part_alloc(a, &ws, static_cast<int64_t>(sage::tile_part_rows(a)), 0, l.D, st))) return rc;
  return part_free(ws, cuda_status(sage::launch_attn_tile(l, st)), st);
}

// Keys of a sequence, and sequences: no wait inside the kernels then comes near their limit of 2^30 cycles.  2^24 keys are
// 2^17 key tiles of 1500 to 4000 cycles; a role that walks past 2^20 empty sequences takes at most 600 for each.
constexpr int64_t kMaxKeys = 1 << 24;
constexpr int kMaxSequences = 1 << 20;

// Which kernel: by the rows (tokens x group) that a key head of an average sequence has.  Single tokens in the kernel for
// few rows and in that for one tile, heads of 128, replays of a graph, cold L2: 48 of 32/8 heads over up to 8192 keys 180
// and 203 us, one over 131072 keys 118 and 114, 16 of 16 heads of 64 over up to 1500 keys 34 and 38.
// One choice for the call: a chunk among single tokens runs in the kernel that suits the average.  With 63 single tokens
// over 4000 keys, 32/8 heads, and a chunk of 190 tokens (few rows) or 4096 (pairs) over as many keys, one call takes
// 196 and 342 us, two calls 210 and 360.  Where the chunk has many more keys than the rest, two are better: 256 single tokens
// over 200 keys and 700 tokens over 30000, 2150 us in one call (the kernel for few rows reads the keys once for every four
// tokens), 365 in two.
bool few_rows(int64_t tokens, int64_t sequences, int G) {
  return G <= sage::kStepRows && tokens * G <= sequences * sage::kStepRows;
}
constexpr int kTileRows = 128;  // one query tile

}  // namespace

extern "C" {

int sage_qk_norm_rope(const void* q, const void* k, void* q_out, void* k_out, const sage_strides* q_st,
                      const sage_strides* k_st, const sage_strides* q_out_st, const sage_strides* k_out_st,
                      const void* q_weight, const void* k_weight, const float* cos, const float* sin,
                      const int32_t* positions, int positions_per_batch, int B, int Hq, int Hk, int N, int d,
                      int rot_dim, int table_rows, int interleaved, float eps, int dtype, void* stream) {
  if (B < 0 || N < 0) return SAGE_ERR_INVALID;
  int rc = check_common(Hq, Hk, d, dtype);
  if (rc) return rc;
  if ((rc = check_rope(cos, sin, q_weight, k_weight, d, rot_dim, table_rows, !positions, N, eps))) return rc;
  if (B == 0 || N == 0) return SAGE_OK;
  if (!view_ok(q, q_st, B, Hq, N) || !view_ok(q_out, q_out_st, B, Hq, N)) return SAGE_ERR_INVALID;
  if (Hk > 0 && (!view_ok(k, k_st, B, Hk, N) || !view_ok(k_out, k_out_st, B, Hk, N))) return SAGE_ERR_INVALID;
  if (static_cast<int64_t>(B) * N * (Hq + static_cast<int64_t>(Hk)) >= (1ll << 31)) return SAGE_ERR_UNSUPPORTED;
  sage::RopeArgs a{};
  a.q = {q, q_out, q_weight, *q_st, *q_out_st};
  if (Hk > 0) a.k = {k, k_out, k_weight, *k_st, *k_out_st};
  a.cos = cos;
  a.sin = sin;
  a.positions = positions;
  a.positions_stride_b = positions_per_batch ? N : 0;
  a.B = B, a.N = N, a.Hq = Hq, a.Hk = Hk;
  a.d = d, a.rot = rot_dim, a.table_rows = table_rows;
  a.eps = eps;
  a.interleaved = interleaved != 0;
  a.bf16 = dtype == SAGE_BF16;
  return cuda_status(sage::launch_qk_norm_rope(a, static_cast<cudaStream_t>(stream)));
}

int sage_qk_norm_rope_append(const void* q, const void* k, const void* v, void* q_out, void* k_cache, void* v_cache,
                             const sage_strides* q_st, const sage_strides* k_st, const sage_strides* v_st,
                             const sage_strides* q_out_st, const sage_strides* k_cache_st,
                             const sage_strides* v_cache_st, const void* q_weight, const void* k_weight,
                             const float* cos, const float* sin, const int32_t* positions, const int32_t* slots,
                             int T, int Hq, int Hk, int d, int rot_dim, int table_rows, int num_pages, int page_size,
                             int interleaved, float eps, int dtype, void* stream) {
  if (T < 0 || Hk <= 0) return SAGE_ERR_INVALID;
  int rc = check_common(Hq, Hk, d, dtype);
  if (rc) return rc;
  if ((rc = check_rope(cos, sin, q_weight, k_weight, d, rot_dim, table_rows, !positions, T, eps))) return rc;
  if ((rc = check_pages(num_pages, page_size))) return rc;
  if (T == 0) return SAGE_OK;
  if (!slots || !view_ok(q, q_st, 1, Hq, T) || !view_ok(q_out, q_out_st, 1, Hq, T) || !view_ok(k, k_st, 1, Hk, T) ||
      !view_ok(v, v_st, 1, Hk, T) || !view_ok(k_cache, k_cache_st, num_pages, Hk, page_size) ||
      !view_ok(v_cache, v_cache_st, num_pages, Hk, page_size))
    return SAGE_ERR_INVALID;
  if (static_cast<int64_t>(T) * (Hq + 2ll * Hk) >= (1ll << 31)) return SAGE_ERR_UNSUPPORTED;
  sage::RopeArgs a{};
  a.q = {q, q_out, q_weight, *q_st, *q_out_st};
  a.k = {k, k_cache, k_weight, *k_st, *k_cache_st};
  a.v = {v, v_cache, nullptr, *v_st, *v_cache_st};
  a.cos = cos;
  a.sin = sin;
  a.positions = positions;
  a.slots = slots;
  a.B = 1, a.N = T, a.Hq = Hq, a.Hk = Hk, a.Hv = Hk;
  a.d = d, a.rot = rot_dim, a.table_rows = table_rows;
  a.page_shift = page_shift(page_size);
  a.slot_count = num_pages * page_size;
  a.eps = eps;
  a.interleaved = interleaved != 0;
  a.bf16 = dtype == SAGE_BF16;
  return cuda_status(sage::launch_qk_norm_rope(a, static_cast<cudaStream_t>(stream)));
}

int sage_paged_attn(const void* q, const void* k_cache, const void* v_cache, void* o, const sage_strides* q_st,
                    const sage_strides* k_cache_st, const sage_strides* v_cache_st, const sage_strides* o_st,
                    const int32_t* page_table, const int32_t* cu_q, const int32_t* kv_len, int B, int T, int Hq,
                    int Hk, int d, int num_pages, int page_size, int pages_per_seq, int causal, float sm_scale,
                    int dtype, void* stream) {
  if (B < 0 || T < 0 || pages_per_seq < 0) return SAGE_ERR_INVALID;
  int rc = check_attn(Hq, Hk, d, sm_scale, dtype);
  if (rc) return rc;
  if ((rc = check_pages(num_pages, page_size))) return rc;
  if (B == 0 || T == 0) return SAGE_OK;
  if (!cu_q || !kv_len || (pages_per_seq > 0 && !page_table) || !view_ok(q, q_st, 1, Hq, T) ||
      !view_ok(o, o_st, 1, Hq, T) || !view_ok(k_cache, k_cache_st, num_pages, Hk, page_size) ||
      !view_ok(v_cache, v_cache_st, num_pages, Hk, page_size))
    return SAGE_ERR_INVALID;
  const int G = Hq / Hk;
  if (static_cast<int64_t>(pages_per_seq) * page_size > kMaxKeys || B > kMaxSequences ||
      static_cast<int64_t>(T) * Hq >= (1ll << 31) || !strides_fit(q_st, 1, Hq, T, G) ||
      !strides_fit(k_cache_st, num_pages, Hk, page_size, 1) || !strides_fit(v_cache_st, num_pages, Hk, page_size, 1))
    return SAGE_ERR_UNSUPPORTED;
  sage::Attn16Launch l{};
  sage::Attn16Args& a = l.a;
  a.o = o;
  a.o_sh = o_st->h, a.o_sn = o_st->n;
  a.cu_q = cu_q;
  a.kv_len = kv_len;
  a.page_table = page_table;
  a.pages_per_seq = pages_per_seq, a.num_pages = num_pages, a.page_shift = page_shift(page_size);
  a.B = B, a.Nq = T, a.Nk = pages_per_seq * page_size;
  a.Hk = Hk, a.G = G;
  a.scale_log2 = sm_scale * 1.4426950408889634f;
  a.causal = causal != 0;
  l.D = d;
  l.bf16 = dtype == SAGE_BF16;
  const bool step = few_rows(T, B, G);
  a.tile_tokens = (step ? sage::kStepRows : kTileRows) / G;
  if (!query_map(&l.tm_q, l.bf16, q, *q_st, 1, Hk, G, T, d, a.tile_tokens) ||
      !key_map(&l.tm_k, l.bf16, k_cache, *k_cache_st, num_pages, Hk, page_size, d, std::min(128, page_size)) ||
      !key_map(&l.tm_v, l.bf16, v_cache, *v_cache_st, num_pages, Hk, page_size, d, std::min(128, page_size)))
    return SAGE_ERR_CUDA;
  if (step) return run_step(l, static_cast<cudaStream_t>(stream));
  // pairs of query tiles when the average sequence has more rows than one tile holds
  l.pair = static_cast<int64_t>(T) * G > static_cast<int64_t>(B) * kTileRows;
  const int cta_tokens = (l.pair ? 2 : 1) * a.tile_tokens;
  a.slots = T / cta_tokens + B;
  if (l.pair) return run_pair(l, static_cast<cudaStream_t>(stream));
  const int64_t tiles = std::max(std::min(B, T), (T + cta_tokens - 1) / cta_tokens);
  return run_tile(l, tiles * Hk, static_cast<cudaStream_t>(stream));
}

int sage_cross_attn(const void* q, const void* k, const void* v, void* o, const sage_strides* q_st,
                    const sage_strides* k_st, const sage_strides* v_st, const sage_strides* o_st,
                    const int32_t* key_len, int B, int Hq, int Hk, int Nq, int Nk, int d, float sm_scale, int dtype,
                    void* stream) {
  if (B < 0 || Nq < 0 || Nk < 0) return SAGE_ERR_INVALID;
  int rc = check_attn(Hq, Hk, d, sm_scale, dtype);
  if (rc) return rc;
  if (B == 0 || Nq == 0) return SAGE_OK;
  if (!view_ok(q, q_st, B, Hq, Nq) || !view_ok(o, o_st, B, Hq, Nq)) return SAGE_ERR_INVALID;
  if (Nk > 0 && (!view_ok(k, k_st, B, Hk, Nk) || !view_ok(v, v_st, B, Hk, Nk))) return SAGE_ERR_INVALID;
  const int G = Hq / Hk;
  if (static_cast<int64_t>(B) * Nq * Hq >= (1ll << 31) || Nk > kMaxKeys || !strides_fit(q_st, B, Hq, Nq, G) ||
      (Nk > 0 && (!strides_fit(k_st, B, Hk, Nk, 1) || !strides_fit(v_st, B, Hk, Nk, 1))))
    return SAGE_ERR_UNSUPPORTED;
  sage::Attn16Launch l{};
  sage::Attn16Args& a = l.a;
  a.o = o;
  a.o_sb = o_st->b, a.o_sh = o_st->h, a.o_sn = o_st->n;
  a.kv_len = Nk > 0 ? key_len : nullptr;
  a.B = B, a.Nq = Nq, a.Nk = Nk;
  a.Hk = Hk, a.G = G;
  a.scale_log2 = sm_scale * 1.4426950408889634f;
  l.D = d;
  l.bf16 = dtype == SAGE_BF16;
  const bool step = few_rows(Nq, 1, G);
  a.tile_tokens = (step ? sage::kStepRows : kTileRows) / G;
  if (!query_map(&l.tm_q, l.bf16, q, *q_st, B, Hk, G, Nq, d, a.tile_tokens)) return SAGE_ERR_CUDA;
  if (Nk > 0) {
    if (!key_map(&l.tm_k, l.bf16, k, *k_st, B, Hk, Nk, d, 128) || !key_map(&l.tm_v, l.bf16, v, *v_st, B, Hk, Nk, d, 128))
      return SAGE_ERR_CUDA;
  } else {
    l.tm_k = l.tm_v = l.tm_q;  // no key: nothing is loaded, every row is 0
  }
  if (step) return run_step(l, static_cast<cudaStream_t>(stream));
  l.pair = Nq > a.tile_tokens;
  const int cta_tokens = (l.pair ? 2 : 1) * a.tile_tokens;
  const int64_t slots = static_cast<int64_t>(B) * ((Nq + cta_tokens - 1) / cta_tokens);
  if (slots >= (1ll << 31)) return SAGE_ERR_UNSUPPORTED;
  a.slots = static_cast<int>(slots);
  if (l.pair) return run_pair(l, static_cast<cudaStream_t>(stream));
  return run_tile(l, slots * Hk, static_cast<cudaStream_t>(stream));
}

}  // extern "C"
