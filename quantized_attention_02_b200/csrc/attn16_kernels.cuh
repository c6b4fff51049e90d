// attn16_kernels.cuh -- launchers of the 16-bit attention kernels behind the paged attention and the cross
// attention, by the query rows of a sequence and key head: attn_step_kernels.cu (16 at most),
// attn_tile_kernels.cu (one tile) and attn_pair_kernels.cu (more).
#pragma once
#include <cuda.h>
#include <cuda_runtime.h>
#include <cstdint>

namespace sage {

// Where a CTA's share of the axis of key tiles begins, for the kernel that joins the parts: `off` tiles into an item
// of `units` tiles that begins at `first` (off 0: with an item, or there is no share).
struct CutNote {
  long long first, share;
  int b, token0, nq, tok0, hk, off, units;
};

struct Attn16Args {
  void* o;
  long long o_sb, o_sh, o_sn;   // element strides of O
  const int32_t* cu_q;          // paged: [B+1] first token of each sequence; null: dense, Nq tokens each
  const int32_t* kv_len;        // keys of each sequence; null (dense): Nk
  const int32_t* page_table;    // paged: [B][pages_per_seq]; null: dense
  int pages_per_seq, num_pages, page_shift;
  int B, Nq, Nk;                // paged: Nq = all tokens, Nk = pages_per_seq * page size
  int Hk, G;                    // key heads, query heads per key head
  int tile_tokens;              // tokens of a query tile: its rows / G
  int slots;                    // places for query tiles (or pairs of them), see tile_of_slot
  int splits, min_chunk;        // key axis: at most splits parts of at least min_chunk key tiles
  float* part_o;                // fp32, unnormalised: rows of D channels of the parts that are joined
  float2* part_ml;              // their (row maximum in log2 units, row sum)
  CutNote* cuts;                // [CTA], where the axis is cut into shares (a workspace too)
  float scale_log2;             // sm_scale * log2(e)
  bool causal;
  bool cut;                     // pairs of tiles: cut the key axis into equal shares (attn_pair_kernels.cu)
};

// The tensor maps (16-bit, 128-byte swizzle, boxes of 64 channels):
//   q: [B][Hk][tokens][G][D], box {64, G, tile_tokens, 1, 1}
//   k, v: [B or pages][Hk][rows][D], box {64, min(128, page size), 1, 1}
struct Attn16Launch {
  Attn16Args a;
  CUtensorMap tm_q, tm_k, tm_v;
  int D;
  bool bf16;
  bool pair;  // items of two query tiles (else tiles alone)
};

// One tile of query rows per CTA (attn_tile_kernels.cu): slots, splits and min_chunk say how the grid is laid out;
// with splits > 1 part_o and part_ml hold tile_part_rows rows.
size_t tile_part_rows(const Attn16Args& a);
cudaError_t launch_attn_tile(const Attn16Launch& l, cudaStream_t st);

// Many rows: pairs of query tiles, ctas CTAs; with a.cut part_o and part_ml hold pair_part_rows(ctas) rows.
size_t pair_part_rows(int ctas);
cudaError_t launch_attn_pair(const Attn16Launch& l, int ctas, cudaStream_t st);
int read_and_clear_pair_error(cudaStream_t st, cudaError_t* err);

// The same for few query rows (attn_step_kernels.cu): items of at most kStepRows rows, tile_tokens =
// kStepRows / G tokens.  Of a, slots, splits and min_chunk are not used; part_o and part_ml hold
// step_part_rows(ctas) rows.
constexpr int kStepRows = 16;
struct StepArgs {
  Attn16Args a;
  int tile_tokens;
};
struct StepLaunch {
  StepArgs s;
  CUtensorMap tm_q, tm_k, tm_v;  // as Attn16Launch, the q box with this tile_tokens
  int D;
  bool bf16;
};
int step_ctas(const StepArgs& s, int sms);
size_t step_part_rows(int ctas);
cudaError_t launch_attn_step(const StepLaunch& l, int ctas, cudaStream_t st);
int read_and_clear_step_error(cudaStream_t st, cudaError_t* err);
int read_and_clear_tile_error(cudaStream_t st, cudaError_t* err);

}  // namespace sage
