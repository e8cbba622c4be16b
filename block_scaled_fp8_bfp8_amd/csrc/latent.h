// Sizes and launchers of latent attention (internal to libbfp8; arguments are validated by the C-ABI
// layer before any launcher is called).
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace bfp8 {

constexpr int kLatentDim = 512;                            // latents of a token
constexpr int kRopeDim = 64;                               // its rotary key
constexpr int kLatentRow = kLatentDim + 2 * kRopeDim;      // bytes of a cache row
constexpr uint32_t kLatentMinCode = 127 - 42, kLatentMaxCode = 127 + 40;  // scale codes the writer makes

// A paged cache and (for readers) its page table.
struct LatentCache {
  const uint8_t* rows;    // row r of page p at p * page_stride + r * kLatentRow
  const uint8_t* scales;  // its scale code at p * scale_stride + r
  int64_t page_stride, scale_stride;
  int pages, page_size;
  const int32_t* table;  // [B][table_stride] pages of a sequence in order, the first table_width entries
  int64_t table_stride;
  int table_width;
};

hipError_t launch_latent_write(const uint16_t* kv, int64_t T, int64_t ld_kv, const uint16_t* w, float eps,
                               const int64_t* slots, const LatentCache& cache, uint8_t* rows, uint8_t* scales,
                               hipStream_t stream);
hipError_t launch_latent_read(const LatentCache& cache, const int32_t* cu, int64_t B, int64_t T, uint16_t* out,
                              int64_t ld_out, hipStream_t stream);
hipError_t launch_latent_gather(const LatentCache& cache, const int32_t* cu, int64_t B, int64_t T, uint8_t* q,
                                int64_t ldq, uint8_t* e, int64_t ld_e, uint16_t* rope, int64_t ld_rope,
                                hipStream_t stream);

// Attention over the cache in the absorbed form. Strides of q and out in elements.
struct LatentAttnArgs {
  const uint16_t* q;  // [T][H][576] bf16
  int64_t q_tok, q_head;
  uint16_t* out;  // [T][H][512] bf16
  int64_t o_tok, o_head;
  LatentCache cache;
  const int32_t* lens;  // [B] keys of a sequence, its new tokens among them
  const int32_t* cu_q;  // [B + 1] first query token of a sequence, or NULL: token b is sequence b's
  int T, B, H;
  float scale;
  int target_parts, min_tiles, max_tiles, max_slots, max_cuts;  // how the work is cut (LatentAttnPlan)
  int* counts;    // workspace: number of cut blocks, then their descriptors from byte 16
  float* stats;   // running maximum and sum of every row of every part of a cut block
  float* states;  // its accumulator
};
struct LatentAttnPlan {
  int64_t blocks, parts, slots, cuts;
  int pairs, target_parts, min_tiles, max_tiles;
  bool join;        // blocks may be cut: a second launch joins their parts
  bool split_join;  // eight waves join a row
  size_t counts_bytes, stats_bytes, states_bytes;
};
// max_keys: no sequence's page table reaches further.
LatentAttnPlan plan_latent_attn(int64_t T, int64_t B, int64_t H, int64_t max_keys);
hipError_t launch_latent_attn(const LatentAttnArgs& args, const LatentAttnPlan& plan, hipStream_t stream);

// Attention in the expanded form, ragged and causal. Strides in elements.
struct LatentExpandedArgs {
  const uint16_t* q;  // [Tq][H][192]
  int64_t q_tok, q_head;
  const uint16_t* kv;  // [Tk][H][256]: 128 key dimensions, 128 value dimensions
  int64_t kv_tok, kv_head;
  const uint16_t* rope;  // [Tk][64], shared by the heads
  int64_t ld_rope;
  uint16_t* out;  // [Tq][H][128]
  int64_t o_tok, o_head;
  const int32_t* cu_q;  // [B + 1]
  const int32_t* cu_k;  // [B + 1]
  int Tq, Tk, B, H;
  float scale;
  bool longest_first;  // set by the launch
};
// The most blocks of query rows that B sequences of Tq rows in all can have, a head.
int64_t latent_expanded_blocks(int64_t Tq, int64_t B);
hipError_t launch_latent_expanded(const LatentExpandedArgs& args, bool f16, hipStream_t stream);

// Accumulated attention weights of cached tokens.
struct LatentMassArgs {
  LatentAttnArgs work;   // the rows, the keys and how the work is cut (out, counts, stats and states are not used)
  const float* mass_in;  // [B][in_stride], or NULL: zeros
  int64_t in_stride;
  float* mass;  // [B][out_stride]
  int64_t out_stride;
  int width;        // columns of mass that are written, at least the page table's reach
  int each;         // workgroups a sequence of the last launch (set by the launch)
  int ids;          // parts of all blocks, at most
  int2* first;      // workspace [B]: of a sequence's first block the first part, and its parts
  float2* stats;    // workspace [ids][128]: maximum and sum of the rows of a part
  float* scores;    // workspace [T * H][pitch]: scores times log2(e)
  float* partial;   // workspace [T * H / 128 + B + 1][pitch]: weights summed over a block of rows
  int64_t pitch;
};
struct LatentMassPlan {
  int target_parts, min_tiles, max_tiles;
  int64_t ids, pitch;
  bool keeps_scores;
  size_t first_bytes, stats_bytes, rest_bytes;
};
LatentMassPlan plan_latent_mass(int64_t T, int64_t B, int64_t H, int64_t max_keys);
hipError_t launch_latent_mass(LatentMassArgs args, const LatentMassPlan& plan, hipStream_t stream);

// Eviction by accumulated weight.
struct LatentEvictArgs {
  LatentCache cache;  // its table names the pages that tokens lie on
  uint8_t* rows;      // the same cache, to write
  uint8_t* scales;
  const int32_t* to;  // [B][to_stride] pages the kept tokens go to, or NULL: in place
  int64_t to_stride;
  int to_width;
  const int32_t* lens;
  const float* mass;
  int64_t mass_stride;
  int width;  // columns of mass
  int B, budget, recent;
  int32_t* kept;  // [B][budget]
  int32_t* lens_out;
  float* mass_out;  // [B][mass_out_stride]; may be mass
  int64_t mass_out_stride;
};
hipError_t launch_latent_evict(const LatentEvictArgs& args, hipStream_t stream);

}  // namespace bfp8
