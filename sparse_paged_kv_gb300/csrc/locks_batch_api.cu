// C-ABI entry points of the operators of a batch that shares prefixes and lives
// within a budget (declared in include/locks.h): argument validation, tensor
// maps and dispatch.  Nothing here allocates, frees or synchronises.
#include <cmath>
#include <cstdint>
#include <mutex>

#include <cudaTypedefs.h>

#include "locks_batch.h"
#include "locks_common.cuh"

namespace {

using locks::kHeadDim;

bool misaligned(const void* p) { return reinterpret_cast<uintptr_t>(p) & 15; }

int check_batch_cfg(const locks_cfg_t* c) {
  if (!c) return LOCKS_ERR_INVALID_ARG;
  if (c->batch < 0 || c->n_q_heads <= 0 || c->n_kv_heads <= 0 || c->head_dim <= 0 ||
      c->page_size <= 0 || c->max_pages <= 0 || c->num_blocks <= 0)
    return LOCKS_ERR_INVALID_ARG;
  if (c->n_q_heads % c->n_kv_heads != 0) return LOCKS_ERR_INVALID_ARG;
  if (c->head_dim != kHeadDim ||
      (c->page_size != 64 && c->page_size != 32 && c->page_size != 16))
    return LOCKS_ERR_UNSUPPORTED;
  if (c->n_q_heads / c->n_kv_heads > locks::kBatchMaxGroup) return LOCKS_ERR_UNSUPPORTED;
  // slots and (block, head) indices are ints
  if (c->max_pages >= (1 << 24) || int64_t(c->max_pages) * c->page_size >= (int64_t(1) << 30) ||
      int64_t(c->num_blocks) * c->n_kv_heads >= (int64_t(1) << 31) ||
      int64_t(c->batch) * c->n_q_heads >= (1 << 24))
    return LOCKS_ERR_UNSUPPORTED;
  return LOCKS_OK;
}

int page_shift(const locks_cfg_t* c) { return c->page_size == 64 ? 6 : c->page_size == 32 ? 5 : 4; }
int group_size(const locks_cfg_t* c) { return c->n_q_heads / c->n_kv_heads; }
int tile_tokens(const locks_cfg_t* c) { return locks::kTileRows / group_size(c); }

int check_rows(const locks_cfg_t* c, int32_t n_rows) {
  if (n_rows <= 0) return LOCKS_ERR_INVALID_ARG;
  return n_rows > 2 * tile_tokens(c) ? LOCKS_ERR_UNSUPPORTED : LOCKS_OK;
}

int check_prefix(const locks_cfg_t* c, int32_t n_groups, int32_t n_rows) {
  int rc = check_batch_cfg(c);
  if (rc != LOCKS_OK || (rc = check_rows(c, n_rows)) != LOCKS_OK) return rc;
  if (n_groups < 0 || n_groups > c->batch) return LOCKS_ERR_INVALID_ARG;
  // what the whole list costs (up to 11 a stage, 8 a unit), and rows, are ints: every sequence's own pages and every group's
  // (at most one unit of two tiles more than the sequences fill) over all of the table's pages
  const int64_t stages = (int64_t(c->max_pages) * c->page_size + locks::kStageTok - 1) / locks::kStageTok;
  const int64_t units = int64_t(c->batch) + n_groups +
                        int64_t(c->batch) * n_rows / (2 * tile_tokens(c)) + 1;
  if ((stages * 11 + 8) * units * c->n_kv_heads >= (int64_t(1) << 31) ||
      int64_t(c->batch) * n_rows * c->n_q_heads >= (int64_t(1) << 28) ||
      int64_t(c->batch) * n_rows >= (1 << 24) - 256)
    return LOCKS_ERR_UNSUPPORTED;
  return LOCKS_OK;
}

// the stages of every sequence's pages are counted in an int
int check_stages(const locks_cfg_t* c) {
  const int64_t stages = (int64_t(c->max_pages) * c->page_size + locks::kStageTok - 1) / locks::kStageTok;
  return (stages + 1) * c->batch * c->n_kv_heads >= (int64_t(1) << 31) ? LOCKS_ERR_UNSUPPORTED : LOCKS_OK;
}

int check_evict(const locks_cfg_t* c, int32_t budget) {
  const int rc = check_batch_cfg(c);
  if (rc != LOCKS_OK) return rc;
  if (budget < 1) return LOCKS_ERR_INVALID_ARG;
  return LOCKS_OK;
}
int evict_list(const locks_cfg_t* c, int32_t budget) {
  return locks::evict_list_len(budget, int64_t(c->max_pages) * c->page_size);
}
size_t evict_list_offset(const locks_cfg_t* c) { return (size_t(c->batch) * 4 + 255) / 256 * 256; }

// cuTensorMapEncodeTiled through the runtime's driver entry point (no link
// against the driver library)
PFN_cuTensorMapEncodeTiled_v12000 tensor_map_encoder() {
  static PFN_cuTensorMapEncodeTiled_v12000 fn = nullptr;
  static std::once_flag once;
  std::call_once(once, [] {
    void* f = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault,
                                         &q) == cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      fn = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(f);
  });
  return fn;
}

// A contiguous bf16 tensor [n2][n1][128], read in boxes [b2][b1][64] with 128-byte swizzle.
bool encode_map(CUtensorMap* m, const void* base, uint64_t n1, uint64_t n2, uint32_t b1, uint32_t b2) {
  auto enc = tensor_map_encoder();
  if (!enc) return false;
  const cuuint64_t dims[3] = {cuuint64_t(kHeadDim), n1, n2};
  const cuuint64_t strides[2] = {cuuint64_t(kHeadDim) * 2, n1 * kHeadDim * 2};
  const cuuint32_t box[3] = {64, b1, b2};
  const cuuint32_t estr[3] = {1, 1, 1};
  return enc(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(base), dims, strides, box,
             estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
             CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// pages [num_blocks * n_kv_heads][page_size][128], a page a box
bool encode_pool(CUtensorMap* m, const void* pool, const locks_cfg_t* c) {
  return encode_map(m, pool, c->page_size, uint64_t(c->num_blocks) * c->n_kv_heads, c->page_size, 1);
}

// queries [batch * n_rows][n_q_heads][128], `tokens` of one KV head's group a box
bool encode_queries(CUtensorMap* m, const void* q, const locks_cfg_t* c, int n_rows, int tokens) {
  return encode_map(m, q, c->n_q_heads, uint64_t(c->batch) * n_rows, group_size(c), tokens);
}

float logit_scale_log2() { return float(1.4426950408889634 / std::sqrt(double(kHeadDim))); }

}  // namespace

extern "C" {

size_t locks_prefix_workspace_bytes(const locks_cfg_t* cfg, int32_t n_groups, int32_t n_rows) {
  if (check_prefix(cfg, n_groups, n_rows) != LOCKS_OK) return 0;
  return locks::prefix_layout(int64_t(cfg->batch) * n_rows * cfg->n_q_heads, cfg->batch, n_groups).total;
}

int locks_prefix_decode(const locks_cfg_t* cfg, const void* q, int32_t n_rows, const void* k_cache,
                        const void* v_cache, const int32_t* block_table, const int32_t* seq_lens,
                        const int32_t* group_starts, const int32_t* prefix_pages, int32_t n_groups,
                        void* out, float* out_lse, void* workspace, size_t workspace_bytes,
                        int32_t* status, void* stream) {
  const int rc = check_prefix(cfg, n_groups, n_rows);
  if (rc != LOCKS_OK) return rc;
  if (cfg->batch == 0) return LOCKS_OK;
  if (!q || !k_cache || !v_cache || !block_table || !seq_lens || !out || !workspace ||
      (n_groups > 0 && (!group_starts || !prefix_pages)))
    return LOCKS_ERR_INVALID_ARG;
  if (misaligned(q) || misaligned(k_cache) || misaligned(v_cache) || misaligned(out) ||
      misaligned(workspace))
    return LOCKS_ERR_INVALID_ARG;
  locks::PrefixParams p;
  p.rows = int64_t(cfg->batch) * n_rows * cfg->n_q_heads;
  const locks::PrefixLayout L = locks::prefix_layout(p.rows, cfg->batch, n_groups);
  if (workspace_bytes < L.total) return LOCKS_ERR_WORKSPACE;
  p.block_table = block_table;
  p.seq_lens = seq_lens;
  p.group_starts = group_starts;
  p.prefix_pages = prefix_pages;
  p.out = static_cast<__nv_bfloat16*>(out);
  p.out_lse = out_lse;
  p.status = status;
  unsigned char* ws = static_cast<unsigned char*>(workspace);
  p.acc = reinterpret_cast<float4*>(ws + L.acc);
  p.parts = L.parts;
  p.sums = reinterpret_cast<float4*>(ws + L.sums);
  p.entry_info = reinterpret_cast<int4*>(ws + L.entry_info);
  p.longest = reinterpret_cast<int32_t*>(ws + L.longest);
  p.batch = cfg->batch;
  p.n_groups = n_groups;
  p.n_rows = n_rows;
  p.n_kv_heads = cfg->n_kv_heads;
  p.group = group_size(cfg);
  p.max_pages = cfg->max_pages;
  p.num_blocks = cfg->num_blocks;
  p.page_size = cfg->page_size;
  p.page_shift = page_shift(cfg);
  p.tile_tokens = tile_tokens(cfg);
  p.tile_magic = ((uint64_t(1) << 32) + 2 * p.tile_tokens - 1) / (2 * p.tile_tokens);
  p.scale_log2 = logit_scale_log2();
  CUtensorMap qg, qo, mk, mv;
  const int own = n_rows < p.tile_tokens ? n_rows : p.tile_tokens;
  if (!encode_queries(&qg, q, cfg, n_rows, p.tile_tokens) || !encode_queries(&qo, q, cfg, n_rows, own) ||
      !encode_pool(&mk, k_cache, cfg) || !encode_pool(&mv, v_cache, cfg))
    return LOCKS_ERR_CUDA;
  return locks::launch_prefix(p, qg, qo, mk, mv, static_cast<cudaStream_t>(stream));
}

int locks_weigh(const locks_cfg_t* cfg, const void* q, int32_t n_rows, const float* lse,
                const void* k_cache, const int32_t* block_table, const int32_t* seq_lens,
                const int32_t* fixed, const float* weights, float* out, int32_t n_new, float decay,
                int32_t* positions, const int32_t* evicted, int32_t* status, void* stream) {
  int rc = check_batch_cfg(cfg);
  if (rc != LOCKS_OK || (rc = check_rows(cfg, n_rows)) != LOCKS_OK) return rc;
  if (n_new < 0 || !(decay >= 0.f) || !std::isfinite(decay)) return LOCKS_ERR_INVALID_ARG;
  if ((rc = check_stages(cfg)) != LOCKS_OK) return rc;
  if (cfg->batch == 0) return LOCKS_OK;
  if (!q || !lse || !k_cache || !block_table || !seq_lens || !out) return LOCKS_ERR_INVALID_ARG;
  if (misaligned(q) || misaligned(k_cache)) return LOCKS_ERR_INVALID_ARG;
  locks::WeighParams p = {};
  p.lse = lse;
  p.block_table = block_table;
  p.seq_lens = seq_lens;
  p.fixed = fixed;
  p.weights = weights;
  p.out = out;
  p.positions = positions;
  p.evicted = evicted;
  p.status = status;
  p.batch = cfg->batch;
  p.n_rows = n_rows;
  p.n_kv_heads = cfg->n_kv_heads;
  p.group = group_size(cfg);
  p.max_pages = cfg->max_pages;
  p.num_blocks = cfg->num_blocks;
  p.page_size = cfg->page_size;
  p.page_shift = page_shift(cfg);
  p.n_new = n_new;
  p.decay = decay;
  p.scale_log2 = logit_scale_log2();
  CUtensorMap mq, mk;
  if (!encode_queries(&mq, q, cfg, n_rows, n_rows) || !encode_pool(&mk, k_cache, cfg))
    return LOCKS_ERR_CUDA;
  return locks::launch_weigh(p, mq, mk, static_cast<cudaStream_t>(stream));
}

size_t locks_evict_workspace_bytes(const locks_cfg_t* cfg, int32_t budget) {
  if (check_evict(cfg, budget) != LOCKS_OK) return 0;
  return evict_list_offset(cfg) + size_t(cfg->batch) * cfg->n_kv_heads * 2 * evict_list(cfg, budget) * 8;
}

int locks_evict(const locks_cfg_t* cfg, int32_t budget, int32_t recent, void* k_cache, void* v_cache,
                const int32_t* block_table, int32_t* seq_lens, const int32_t* fixed, float* weights,
                int32_t* positions, int32_t* evicted, void* workspace, size_t workspace_bytes,
                int32_t* status, void* stream) {
  const int rc = check_evict(cfg, budget);
  if (rc != LOCKS_OK) return rc;
  if (recent < 0 || recent > budget) return LOCKS_ERR_INVALID_ARG;
  if (cfg->batch == 0) return LOCKS_OK;
  if (!k_cache || !v_cache || !block_table || !seq_lens || !weights || !positions || !evicted || !workspace)
    return LOCKS_ERR_INVALID_ARG;
  if (misaligned(k_cache) || misaligned(v_cache) || misaligned(weights) || misaligned(positions) ||
      misaligned(workspace))
    return LOCKS_ERR_INVALID_ARG;                     // rows, and four slots' records, move as 16-byte words
  if (workspace_bytes < locks_evict_workspace_bytes(cfg, budget)) return LOCKS_ERR_WORKSPACE;
  locks::EvictParams p = {};
  p.k_cache = static_cast<__nv_bfloat16*>(k_cache);
  p.v_cache = static_cast<__nv_bfloat16*>(v_cache);
  p.block_table = block_table;
  p.seq_lens = seq_lens;
  p.fixed = fixed;
  p.weights = weights;
  p.positions = positions;
  p.evicted = evicted;
  p.tickets = static_cast<int32_t*>(workspace);
  p.lists = reinterpret_cast<int64_t*>(static_cast<unsigned char*>(workspace) + evict_list_offset(cfg));
  p.status = status;
  p.batch = cfg->batch;
  p.n_kv_heads = cfg->n_kv_heads;
  p.max_pages = cfg->max_pages;
  p.num_blocks = cfg->num_blocks;
  p.page_size = cfg->page_size;
  p.page_shift = page_shift(cfg);
  p.budget = budget;
  p.recent = recent;
  p.list_len = evict_list(cfg, budget);
  return locks::launch_evict(p, static_cast<cudaStream_t>(stream));
}

}  // extern "C"
