// C-ABI entry points of the quantised cache (declared in include/locks.h):
// argument validation and dispatch.  Nothing here allocates, frees or
// synchronises.
#include <cstdint>

#include "locks_kv.cuh"

namespace {

using locks::kHeadDim;

constexpr int64_t kMaxWriteRows = 1 << 16;     // of a token: query, key and value heads

bool misaligned(const void* p) { return reinterpret_cast<uintptr_t>(p) & 15; }

int check_kv_cfg(const locks_kv_cfg_t* c) {
  if (!c) return LOCKS_ERR_INVALID_ARG;
  if (c->batch < 0 || c->n_q_heads <= 0 || c->n_kv_heads <= 0 || c->head_dim <= 0 ||
      c->page_size <= 0 || c->max_pages <= 0 || c->num_blocks <= 0)
    return LOCKS_ERR_INVALID_ARG;
  if (c->n_q_heads % c->n_kv_heads != 0) return LOCKS_ERR_INVALID_ARG;
  if (c->kv_dtype != LOCKS_KV_F8 && c->kv_dtype != LOCKS_KV_I8 && c->kv_dtype != LOCKS_KV_I4)
    return LOCKS_ERR_INVALID_ARG;
  if (c->head_dim != kHeadDim ||
      (c->page_size != 64 && c->page_size != 32 && c->page_size != 16))
    return LOCKS_ERR_UNSUPPORTED;
  if (c->n_q_heads / c->n_kv_heads > locks::kKvMaxGroup) return LOCKS_ERR_UNSUPPORTED;
  // page ids are kept in 24 bits, positions and (block, head) indices in an int
  if (c->max_pages >= (1 << 24) || int64_t(c->num_blocks) * c->n_kv_heads >= (int64_t(1) << 31) ||
      int64_t(c->batch) * c->n_kv_heads >= (1 << 24))
    return LOCKS_ERR_UNSUPPORTED;
  return LOCKS_OK;
}

int check_rope(const locks_rope_table_t* r, int head_dim) {
  if (!r || !r->turns || r->rotary_dim < 2 || r->rotary_dim % 2 || r->rotary_dim > head_dim ||
      (r->layout != LOCKS_ROPE_HALF && r->layout != LOCKS_ROPE_INTERLEAVED) || !(r->mscale > 0.f))
    return LOCKS_ERR_INVALID_ARG;
  return LOCKS_OK;
}

locks::RopeArgs rope_args(const locks_rope_table_t* r) {
  locks::RopeArgs a = {nullptr, 0, LOCKS_ROPE_HALF, 1.f};
  if (r) {
    a.turns = r->turns;
    a.rotary_dim = r->rotary_dim;
    a.layout = r->layout;
    a.mscale = r->mscale;
  }
  return a;
}

}  // namespace

extern "C" {

size_t locks_kv_record_bytes(const locks_kv_cfg_t* cfg) {
  if (check_kv_cfg(cfg) != LOCKS_OK) return 0;
  return size_t(locks::kv_rec_bytes(cfg->kv_dtype, cfg->page_size));
}

size_t locks_kv_decode_workspace_bytes(const locks_kv_cfg_t* cfg) {
  if (check_kv_cfg(cfg) != LOCKS_OK) return 0;
  return locks::kv_decode_workspace(cfg->n_q_heads / cfg->n_kv_heads);
}

int locks_rope(const locks_rope_table_t* rope, int32_t dtype, int32_t head_dim, const void* x,
               int64_t x_token_stride, int64_t x_head_stride, const int32_t* positions,
               int32_t n_tokens, int32_t n_heads, void* out, int64_t out_token_stride,
               int64_t out_head_stride, int32_t inverse, void* stream) {
  if (head_dim < 2 || head_dim % 2 || n_tokens < 0 || n_heads < 0) return LOCKS_ERR_INVALID_ARG;
  if (dtype != LOCKS_BF16 && dtype != LOCKS_F16 && dtype != LOCKS_F32) return LOCKS_ERR_INVALID_ARG;
  const int rc = check_rope(rope, head_dim);
  if (rc != LOCKS_OK) return rc;
  // (a thread's next head is as many heads on as the others take: an int)
  if (head_dim > 512 || n_heads > (1 << 24)) return LOCKS_ERR_UNSUPPORTED;
  if (n_tokens == 0 || n_heads == 0) return LOCKS_OK;
  if (!x || !positions || !out) return LOCKS_ERR_INVALID_ARG;
  const uintptr_t size = dtype == LOCKS_F32 ? 4 : 2;
  if ((reinterpret_cast<uintptr_t>(x) | reinterpret_cast<uintptr_t>(out)) % size)
    return LOCKS_ERR_INVALID_ARG;
  locks::RopeParams p;
  p.rope = rope_args(rope);
  p.x = x;
  p.out = out;
  p.positions = positions;
  p.x_ts = x_token_stride;
  p.x_hs = x_head_stride;
  p.o_ts = out_token_stride;
  p.o_hs = out_head_stride;
  p.n_tokens = n_tokens;
  p.n_heads = n_heads;
  p.head_dim = head_dim;
  p.inverse = inverse != 0;
  p.n_chunks = 1;
  return locks::launch_rope(p, dtype, static_cast<cudaStream_t>(stream));
}

int locks_kv_write(const locks_kv_cfg_t* cfg, const void* k_new, int64_t k_stride,
                   const void* v_new, int64_t v_stride, const void* q_new, int64_t q_stride,
                   void* q_out, const int32_t* token_seq, const int32_t* token_pos,
                   int32_t n_tokens, const locks_rope_table_t* rope, void* k_pool, void* v_pool,
                   const int32_t* block_table, int32_t* seq_lens, int32_t* completed,
                   int32_t* status, void* stream) {
  int rc = check_kv_cfg(cfg);
  if (rc != LOCKS_OK) return rc;
  if (n_tokens < 0) return LOCKS_ERR_INVALID_ARG;
  if (rope) {
    if ((rc = check_rope(rope, cfg->head_dim)) != LOCKS_OK) return rc;
    if (rope->rotary_dim % 16) return LOCKS_ERR_UNSUPPORTED;
  }
  if (n_tokens == 0) return LOCKS_OK;
  if (!k_new || !v_new || !token_pos || !k_pool || !v_pool || !block_table ||
      (q_new == nullptr) != (q_out == nullptr) || token_pos == seq_lens)
    return LOCKS_ERR_INVALID_ARG;
  if (!token_seq && n_tokens > cfg->batch) return LOCKS_ERR_INVALID_ARG;
  if (n_tokens > (1 << 30)) return LOCKS_ERR_UNSUPPORTED;     // token numbers are ints, rounded up to groups
  // and so are a token's rows and their shares, rows * shares of 16 rows
  if ((q_new ? int64_t(cfg->n_q_heads) : 0) + 2 * int64_t(cfg->n_kv_heads) > kMaxWriteRows)
    return LOCKS_ERR_UNSUPPORTED;
  if (misaligned(k_new) || misaligned(v_new) || misaligned(k_pool) || misaligned(v_pool) ||
      misaligned(q_new) || misaligned(q_out) || k_stride % 8 || v_stride % 8 ||
      (q_new && q_stride % 8))
    return LOCKS_ERR_INVALID_ARG;                     // rows move as 16-byte words
  // rotating in place needs q_out's own layout
  if (q_new && q_new == q_out && q_stride != int64_t(cfg->n_q_heads) * kHeadDim)
    return LOCKS_ERR_INVALID_ARG;
  locks::KvWriteParams p;
  p.k_new = static_cast<const __nv_bfloat16*>(k_new);
  p.v_new = static_cast<const __nv_bfloat16*>(v_new);
  p.q_new = static_cast<const __nv_bfloat16*>(q_new);
  p.q_out = static_cast<__nv_bfloat16*>(q_out);
  p.k_stride = k_stride;
  p.v_stride = v_stride;
  p.q_stride = q_stride;
  p.token_seq = token_seq;
  p.token_pos = token_pos;
  p.rope = rope_args(rope);
  p.k_pool = static_cast<unsigned char*>(k_pool);
  p.v_pool = static_cast<unsigned char*>(v_pool);
  p.block_table = block_table;
  p.seq_lens = seq_lens;
  p.completed = completed;
  p.status = status;
  p.n_tokens = n_tokens;
  p.batch = cfg->batch;
  p.n_q_heads = cfg->n_q_heads;
  p.n_kv_heads = cfg->n_kv_heads;
  p.max_pages = cfg->max_pages;
  p.num_blocks = cfg->num_blocks;
  p.page_size = cfg->page_size;
  p.n_chunks = 1;
  return locks::launch_kv_write(p, cfg->kv_dtype, static_cast<cudaStream_t>(stream));
}

int locks_kv_read(const locks_kv_cfg_t* cfg, const void* k_pool, const void* v_pool,
                  const int32_t* block_ids, int32_t n_blocks, void* k_out, void* v_out,
                  int32_t* status, void* stream) {
  const int rc = check_kv_cfg(cfg);
  if (rc != LOCKS_OK) return rc;
  if (n_blocks < 0) return LOCKS_ERR_INVALID_ARG;
  if (n_blocks == 0) return LOCKS_OK;
  if (!block_ids || (!k_out && !v_out) || (k_out && !k_pool) || (v_out && !v_pool))
    return LOCKS_ERR_INVALID_ARG;
  if (misaligned(k_pool) || misaligned(v_pool) || misaligned(k_out) || misaligned(v_out))
    return LOCKS_ERR_INVALID_ARG;
  locks::KvReadParams p;
  p.k_pool = static_cast<const unsigned char*>(k_pool);
  p.v_pool = static_cast<const unsigned char*>(v_pool);
  p.block_ids = block_ids;
  p.k_out = static_cast<__nv_bfloat16*>(k_out);
  p.v_out = static_cast<__nv_bfloat16*>(v_out);
  p.status = status;
  p.n_blocks = n_blocks;
  p.n_kv_heads = cfg->n_kv_heads;
  p.num_blocks = cfg->num_blocks;
  p.page_size = cfg->page_size;
  return locks::launch_kv_read(p, cfg->kv_dtype, static_cast<cudaStream_t>(stream));
}

int locks_kv_decode(const locks_kv_cfg_t* cfg, const void* q, const void* k_pool,
                    const void* v_pool, const int32_t* block_table, const int32_t* seq_lens,
                    const int32_t* selected, int32_t k, int32_t window, void* out, float* out_lse,
                    void* workspace, size_t workspace_bytes, int32_t* status, void* stream) {
  const int rc = check_kv_cfg(cfg);
  if (rc != LOCKS_OK) return rc;
  if (window < 0 || (selected && k <= 0)) return LOCKS_ERR_INVALID_ARG;
  // the kernel counts the 64-token stages of all units (and 8 more a unit) in an int
  if (selected && k >= (1 << 24)) return LOCKS_ERR_UNSUPPORTED;
  const int64_t pages = selected ? k : cfg->max_pages;
  if (((pages * cfg->page_size + 63) / 64 + 8) * cfg->batch * cfg->n_kv_heads >= (int64_t(1) << 31))
    return LOCKS_ERR_UNSUPPORTED;
  if (cfg->batch == 0) return LOCKS_OK;
  if (!q || !k_pool || !v_pool || !block_table || !seq_lens || !out || !workspace)
    return LOCKS_ERR_INVALID_ARG;
  if (misaligned(q) || misaligned(k_pool) || misaligned(v_pool) || misaligned(out) ||
      misaligned(workspace))
    return LOCKS_ERR_INVALID_ARG;
  if (workspace_bytes < locks_kv_decode_workspace_bytes(cfg)) return LOCKS_ERR_WORKSPACE;
  locks::KvDecodeParams p;
  p.q = static_cast<const __nv_bfloat16*>(q);
  p.k_pool = static_cast<const unsigned char*>(k_pool);
  p.v_pool = static_cast<const unsigned char*>(v_pool);
  p.block_table = block_table;
  p.seq_lens = seq_lens;
  p.selected = selected;
  p.out = static_cast<__nv_bfloat16*>(out);
  p.out_lse = out_lse;
  p.status = status;
  p.ws = static_cast<unsigned char*>(workspace);
  p.batch = cfg->batch;
  p.n_kv_heads = cfg->n_kv_heads;
  p.group = cfg->n_q_heads / cfg->n_kv_heads;
  p.max_pages = cfg->max_pages;
  p.num_blocks = cfg->num_blocks;
  p.page_size = cfg->page_size;
  p.k = selected ? k : 0;
  p.window = window;
  return locks::launch_kv_decode(p, cfg->kv_dtype, static_cast<cudaStream_t>(stream));
}

}  // extern "C"
