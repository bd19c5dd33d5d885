// Parameter blocks and launchers of the operators of a batch that shares
// prefixes and lives within a budget.  Internal to the library.
#pragma once

#include <cstddef>
#include <cstdint>
#include <cuda.h>
#include <cuda_bf16.h>

#include "../../include/locks.h"

namespace locks {

constexpr int kBatchSms = 152;         // blocks of a persistent launch: one per SM
constexpr size_t kMaxSmemBlock = 227 * 1024;
constexpr int kBatchMaxGroup = 16;     // query heads a KV head
constexpr int kTileRows = 128;         // query rows of a matrix instruction
constexpr int kStageTok = 128;         // tokens of a stage of the attention

struct PrefixParams {
  const int32_t* block_table;    // [batch][max_pages]
  const int32_t* seq_lens;       // [batch]
  const int32_t* group_starts;   // [n_groups + 1]
  const int32_t* prefix_pages;   // [n_groups]
  __nv_bfloat16* out;            // [batch][n_rows][H_q][d]
  float* out_lse;                // nullable [batch][n_rows][H_q]
  int32_t* status;               // nullable
  // workspace (see prefix_layout)
  float4* acc;                   // [32 chunks of 4 dims][parts]: [2 kinds][2 parts][rows] first pieces,
                                 // rows as [KV head][query token][head of the group], then
                                 // [blocks][256] pieces continued from the block before
  float4* sums;                  // [parts][2 halves of the columns] (m, l, l of the rounded weights, -)
  int4* entry_info;              // [n_groups + batch + 1] of each entry of the list: see join_kernel
  int32_t* longest;              // [blocks][n_groups] of many groups: see Groups
  int batch, n_groups, n_rows, n_kv_heads, group, max_pages, num_blocks, page_size, page_shift;
  int tile_tokens;               // query tokens of a tile: floor(128 / group)
  uint64_t tile_magic;           // ceil(2^32 / (2 tile_tokens)): n / (2 tile_tokens) = n * magic >> 32 below 2^24
  int64_t rows, parts;           // batch * n_rows * n_q_heads; 4 rows + 256 blocks
  float scale_log2;
};

struct PrefixLayout {
  size_t acc, sums, entry_info, longest, total;
  int64_t parts;
};
PrefixLayout prefix_layout(int64_t rows, int64_t batch, int64_t groups);
int launch_prefix(const PrefixParams& p, const CUtensorMap& q_group, const CUtensorMap& q_own,
                  const CUtensorMap& k, const CUtensorMap& v, cudaStream_t stream);

struct WeighParams {
  const float* lse;              // [batch][n_rows][H_q]
  const int32_t* block_table;    // [batch][max_pages]
  const int32_t* seq_lens;       // [batch]
  const int32_t* fixed;          // nullable [batch]
  const float* weights;          // nullable [num_blocks][H_kv][B]
  float* out;                    // [num_blocks][H_kv][B]
  int32_t* positions;            // nullable [num_blocks][H_kv][B]
  const int32_t* evicted;        // nullable [batch]
  int32_t* status;               // nullable
  int batch, n_rows, n_kv_heads, group, max_pages, num_blocks, page_size, page_shift, n_new;
  float decay, scale_log2;
  int q_half, n_cols, tmem_cols, ring;   // set by the launch: see launch_weigh
};
int launch_weigh(WeighParams p, const CUtensorMap& q, const CUtensorMap& k, cudaStream_t stream);

struct EvictParams {
  __nv_bfloat16* k_cache;        // [num_blocks][H_kv][B][d]
  __nv_bfloat16* v_cache;
  const int32_t* block_table;    // [batch][max_pages]
  int32_t* seq_lens;             // [batch], lowered
  const int32_t* fixed;          // nullable [batch]
  float* weights;                // [num_blocks][H_kv][B]
  int32_t* positions;            // [num_blocks][H_kv][B]
  int32_t* evicted;              // [batch], raised
  int32_t* tickets;              // [batch] zeros, left as zeros
  int64_t* lists;                // [batch * H_kv][2][list_len] pool rows
  int32_t* status;               // nullable
  int batch, n_kv_heads, max_pages, num_blocks, page_size, page_shift, budget, recent, list_len;
  int keys;                      // set by the launch: keys a block holds
};
int evict_list_len(int budget, int64_t slots);
constexpr int kEvictMostBlocks = 16;
// Blocks of the cluster that has one of `units` heads of so many slots; fit[c]: clusters of c blocks
// that run at once, a block an SM (0: the device has no room for one, or refuses the size).
// As many as fill the SMs with two each, while each still has a thousand slots.  Where
// one block an SM is all there is, as many as have an SM each: two clusters in one part of the chip while
// others are idle (16 blocks a head of eight) took 57 us where 12 blocks take 53.6.
template <typename Fit>
int evict_blocks(int units, int64_t slots, const Fit& fit) {
  int c = 1;
  while (2 * c <= kEvictMostBlocks && int64_t(units) * c <= kBatchSms && slots / (2 * c) >= 1024) c *= 2;
  const int least = units <= kBatchSms / c ? units : 1;
  while (c > 1 && fit[c] < least) --c;
  return c;
}
int launch_evict(EvictParams p, cudaStream_t stream);

}  // namespace locks
