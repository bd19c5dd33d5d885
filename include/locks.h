/*
 * locks.h -- C ABI of the Locks decode-attention hot path on one GB300 (sm_103a).
 *
 * The method is the one of "Locks: Page-Local Compact Key Summaries for
 * Efficient Long-Context Decoding" (arXiv 2607.24555): every completed page of
 * a paged KV cache gets its own rank-r spectral key summary (section 4,
 * "Build"); each decode step scores every candidate page by the log-sum-exp of
 * its reconstructed within-page logits (section 4, Eq. (1)), normalises the
 * scores into per-head page-mass shares, averages the shares over the GQA
 * group, keeps the sink page and the most recent page and the top-(k-2)
 * remaining pages under the token budget (section 2; section 4; Cor. 3), and
 * attends only the selected pages.
 *
 * Conventions shared by every call
 * --------------------------------
 *  - All pointers named *_cache, q, summaries, block_table, seq_lens, selected,
 *    out*, page_*, workspace, status, tail_energy and block_ids are DEVICE
 *    pointers owned by the caller.  The library never allocates, frees or
 *    synchronises; every call only enqueues kernels on `stream` (a
 *    cudaStream_t passed as void*, NULL = legacy default stream).
 *  - The return value reports argument validation and launch errors only
 *    (LOCKS_ERR_*).  Conditions found on the device (a block id outside the
 *    pool, a page id outside the sequence, a bounded wait that ran out, a
 *    Jacobi solve that did not converge) are OR-ed as LOCKS_DEV_* bits into the
 *    caller's `status` word(s) when that pointer is non-NULL; the offending
 *    page is skipped.  Read them after synchronising the stream.
 *  - bf16 is IEEE bfloat16 stored as 16-bit words.
 *  - KV pools are [num_blocks][n_kv_heads][page_size][head_dim] bf16: each
 *    (block, KV head) page is contiguous.  Logical page j of sequence b lives
 *    in physical block block_table[b * max_pages + j].  Only the first
 *    seq_lens[b] tokens of a sequence are ever read; the rest of its tail page
 *    may hold anything (NaN included).
 *  - Query head h uses KV head h / G, with G = n_q_heads / n_kv_heads
 *    (contiguous grouping).  Logits are scaled by 1/sqrt(head_dim)
 *    (section 2).
 *  - Calls that use a workspace require it to be zero-filled before its first
 *    use (cudaMemset once); every call leaves it ready for the next call, so
 *    the same workspace can be replayed inside a CUDA graph.  Calls that share
 *    a workspace must not overlap on the GPU.
 *
 * Supported shapes: head_dim = 128; page_size = 64 or 16; 1 <= rank <= 16;
 * G in {1, 2, 4, 8}; max_pages < 2^24; num_blocks * n_kv_heads < 2^31.
 * Other values return LOCKS_ERR_UNSUPPORTED.
 */
#ifndef LOCKS_H_
#define LOCKS_H_

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

#define LOCKS_ABI_VERSION 1

/* host return codes */
#define LOCKS_OK               0
#define LOCKS_ERR_INVALID_ARG (-1)   /* null pointer, bad size, k < 2, ...        */
#define LOCKS_ERR_UNSUPPORTED (-2)   /* shape outside the supported set           */
#define LOCKS_ERR_WORKSPACE   (-3)   /* workspace smaller than the size query     */
#define LOCKS_ERR_CUDA        (-4)   /* a CUDA launch failed                       */

/* device status bits, OR-ed into *status */
#define LOCKS_DEV_BAD_BLOCK_ID   0x1  /* block id < 0 or >= num_blocks: page skipped      */
#define LOCKS_DEV_WAIT_TIMEOUT   0x2  /* a bounded wait on a copy ran out: page skipped   */
#define LOCKS_DEV_NOT_CONVERGED  0x4  /* Jacobi hit max_sweeps before its tolerance       */
#define LOCKS_DEV_BAD_PAGE_ID    0x8  /* selected page id outside [0, n): entry skipped   */
#define LOCKS_DEV_BAD_SEQ_LEN    0x10 /* seq_len > max_pages * page_size: clamped         */
#define LOCKS_DEV_BAD_GROUP      0x20 /* group_starts not ascending: no group; prefix_pages: clamped */

/* summary record element type */
#define LOCKS_SUMMARY_F32  0
#define LOCKS_SUMMARY_BF16 1
#define LOCKS_SUMMARY_I4   2   /* int4 basis, int8 coefficients and centroid */

typedef struct locks_cfg {
  int32_t batch;          /* sequences in the decode batch (>= 0)                     */
  int32_t n_q_heads;      /* query heads H_q                                           */
  int32_t n_kv_heads;     /* KV heads H_kv; H_q % H_kv == 0                            */
  int32_t head_dim;       /* d                                                         */
  int32_t page_size;      /* B, tokens per page                                        */
  int32_t rank;           /* r, modes kept per page summary                            */
  int32_t max_pages;      /* row stride of block_table (pages per sequence, at most)  */
  int32_t num_blocks;     /* physical blocks in the KV / summary pools                 */
  int32_t summary_dtype;  /* LOCKS_SUMMARY_F32, LOCKS_SUMMARY_BF16 or LOCKS_SUMMARY_I4  */
} locks_cfg_t;

/*
 * Summary record (one per (physical block, KV head)), written by
 * locks_build_summaries and read by locks_select.  Element type T is float
 * (LOCKS_SUMMARY_F32) or bf16 (LOCKS_SUMMARY_BF16).  With d = head_dim,
 * B = page_size and R = the smallest power of two >= max(rank, 4):
 *
 *   T W[R + 1][d];      W[0] = page centroid mu; W[1 + k] = basis column v_k
 *   T C[R / 4][B][4];   C[c][i][e] = coefficient c_{i, 4c + e} of token i
 *
 * Columns k >= rank and dropped (zero) modes hold zeros.  Records of one
 * KV head follow each other: record (blk, h) starts at byte
 * (blk * n_kv_heads + h) * locks_summary_record_bytes(cfg) of the pool.  The
 * basis is orthonormal (v_k^T v_l = delta_kl up to rounding), modes are in
 * descending eigenvalue order, and c_i = V^T (k_i - mu) (section 4, "Build").
 *
 * LOCKS_SUMMARY_I4 is the quantised record the paper deploys (section 4
 * "Build": the basis in int4, the coefficients and centroid in int8, with
 * per-column and per-row scales).  Each group is quantised symmetrically:
 * scale = max|x| / qmax (qmax 7 for int4, 127 for int8), code =
 * round-half-even(x / scale) clamped to [-qmax, qmax], in float32; an
 * all-zero group has scale 0.  Codes are stored biased (int4 + 8 as an
 * unsigned nibble, int8 + 128 as an unsigned byte), in the order the
 * scorer's tensor-core fragments read them.  With HDR = (R + 1) * 4 rounded
 * up to 16 bytes, KK = ceil(R / 8), and for a lane l = 4g + t (g < 8, t < 4):
 *
 *   float    vscale[R], mscale;      scale of basis column k; of the centroid
 *   uint32_t vq[R][4][4]       @HDR  word vq[k][t][j] holds, for the k-steps
 *                                    s = 2j and 2j + 1 (columns 16s + c):
 *                                    nibbles 0 / 4 = v_k at c = 2t / 2t + 1,
 *                                    nibbles 1 / 5 = c = 2t + 8 / 2t + 9 (k-step
 *                                    2j), nibbles 2 / 6 and 3 / 7 the same for
 *                                    k-step 2j + 1
 *   uint8_t  mq[32][4]         @HDR + 64R   mq[l] = mu at 16g + 2t, 16g + 2t + 1,
 *                                    16g + 2t + 8, 16g + 2t + 9
 *   uint8_t  cq[B/16][KK][32][4]  @HDR + 64R + 128   cq[m][kk][l] = c_{i,k} at
 *                                    (i, k) = (16m + g, 8kk + 2t), (16m + g,
 *                                    8kk + 2t + 1), (16m + g + 8, 8kk + 2t),
 *                                    (16m + g + 8, 8kk + 2t + 1)
 *   float    cscale[B]         @HDR + 64R + 128 + 8 B KK   scale of row c_i
 *
 * (nibble n of a word is bits 4n..4n+3; codes of columns k >= rank are 0), so
 * that v_k[x] = vscale[k] * (nibble - 8), mu[x] = mscale * (byte - 128) and
 * c_{i,k} = cscale[i] * (byte - 128).  The quantised values are those of the
 * float record's basis, coefficients and centroid.
 */
size_t locks_summary_record_bytes(const locks_cfg_t* cfg);

/* Same value as locks_summary_record_bytes (the shorter name). */
size_t locks_summary_bytes(const locks_cfg_t* cfg);

/* Bytes of workspace locks_select needs for this cfg and token budget. */
size_t locks_select_workspace_bytes(const locks_cfg_t* cfg, int32_t budget_tokens);

/* Bytes of workspace locks_sparse_decode (n_pages = its k) or
 * locks_dense_decode (n_pages = cfg->max_pages) needs. */
size_t locks_decode_workspace_bytes(const locks_cfg_t* cfg, int32_t n_pages);

/*
 * locks_build_summaries -- section 4 "Build" (and the blog review's Algorithm 1).
 *
 * For every listed block and every KV head: centre the page's B keys
 * (k_i = mu + delta_i), form the B x B Gram D D^T of the deviations, find its
 * eigenpairs with a cyclic Jacobi solver (fp32), keep the top-`rank` modes in
 * descending order (modes with sigma^2 <= 1e-5 sigma_1^2 are dropped: zero
 * basis column and coefficients), and write V = D^T U_r S_r^-1 and C = U_r S_r
 * with the centroid into the summary record.  Only complete pages (all B
 * tokens valid) may be listed.
 *
 *   k_cache      bf16 [num_blocks][n_kv_heads][B][d]
 *   block_ids    int32 [n_blocks]: physical blocks to summarise
 *   summaries    record pool, num_blocks * n_kv_heads records (see above)
 *   tail_energy  nullable float [n_blocks][n_kv_heads]: tau = sum_{k>r} sigma_k^2
 *   status       nullable int32 [n_blocks][n_kv_heads]: Jacobi sweeps used,
 *                OR-ed with LOCKS_DEV_NOT_CONVERGED << 16 / LOCKS_DEV_BAD_BLOCK_ID << 16
 *   max_sweeps   Jacobi sweep cap (>= 1; 0 selects the default, 20)
 */
int locks_build_summaries(const locks_cfg_t* cfg, const void* k_cache, const int32_t* block_ids,
                          int32_t n_blocks, void* summaries, float* tail_energy, int32_t* status,
                          int32_t max_sweeps, void* stream);

/*
 * locks_append_kv -- the cache write of one decode step, and the page
 * completions it causes (section 4 "Build": a page is summarised once, when it
 * completes; App. E (ii): one incremental build per finalised page).
 *
 * For every sequence b with t = seq_lens[b] on entry: the token's key and
 * value rows of every KV head go to slot t % B of physical block
 * block_table[b * max_pages + t / B]; seq_lens[b] becomes t + 1; and
 * completed[b] is that block when t + 1 is a multiple of B (the token
 * completed its page), else -1.  Allocating a block for a sequence's next
 * page (writing the block-table entry before the step that starts the page)
 * stays with the caller.  A sequence already holding max_pages * B tokens
 * (LOCKS_DEV_BAD_SEQ_LEN) or whose entry is not a valid block
 * (LOCKS_DEV_BAD_BLOCK_ID) is left unchanged, with completed[b] = -1.
 *
 *   k_new, v_new  bf16 [batch][n_kv_heads][d], 16-byte aligned
 *   k_cache, v_cache  the pools, 16-byte aligned; written
 *   seq_lens      int32 [batch]: read, then advanced
 *   completed     nullable int32 [batch]: written
 *   status        nullable int32[1]
 * Pass `completed` to locks_build_completed (for example on a second stream
 * that waits for this call): the page completed at step s is first a
 * selection candidate at step s + 1, so its build may overlap step s's
 * selection and decode and must finish before step s + 1's locks_select.
 */
int locks_append_kv(const locks_cfg_t* cfg, const void* k_new, const void* v_new, void* k_cache,
                    void* v_cache, const int32_t* block_table, int32_t* seq_lens,
                    int32_t* completed, int32_t* status, void* stream);

/*
 * locks_build_completed -- locks_build_summaries over a list in which an entry
 * < 0 means "no page" and is skipped without a flag (its status entries are
 * set to 0): the `completed` list that locks_append_kv writes, used as it
 * stands on the device, so no host round trip decides which pages to build.
 * Arguments as for locks_build_summaries, with block_ids = completed and
 * n_blocks = n (the batch).
 */
int locks_build_completed(const locks_cfg_t* cfg, const void* k_cache, const int32_t* completed,
                          int32_t n, void* summaries, float* tail_energy, int32_t* status,
                          int32_t max_sweeps, void* stream);

/*
 * locks_select -- section 4 "Score" (Eq. (1)), the page-mass share, the
 * share-average, and the forced-page top-(k-2) rule (section 2; Cor. 3).
 *
 * With n = ceil(seq_len / B) pages, the forced pages are {0, n-1} (page n-1 is
 * the tail, complete or not) and the candidates are the complete pages other
 * than those.  For every candidate j and query head g of the group:
 *   s_hat[g][j] = log sum_{i<B} exp((q_g^T mu_j + (V_j^T q_g)^T c_i) / sqrt(d)),
 * then m_hat_g(j) = exp(s_hat[g][j]) / sum_{j' candidate} exp(s_hat[g][j']),
 * m_bar_j = mean_g m_hat_g(j), and the selection is the forced pages plus the
 * k-2 candidates with the largest m_bar (ties: smaller page id), k = ceil(b/B).
 * If n <= k every page is selected.  Selection reads only summaries.
 *
 *   q            bf16 [batch][n_q_heads][d]
 *   summaries    record pool written by locks_build_summaries (read through block_table)
 *   block_table  int32 [batch][max_pages]
 *   seq_lens     int32 [batch]
 *   budget_tokens b >= B + 1 (k >= 2), else LOCKS_ERR_INVALID_ARG
 *   selected     int32 [batch][n_kv_heads][k]: logical page ids ascending, -1 padded
 *   page_lse     nullable float [batch][n_q_heads][max_pages]: s_hat of candidates
 *                (other entries untouched)
 *   page_share   nullable float [batch][n_kv_heads][max_pages]: m_bar of candidates
 *   workspace    >= locks_select_workspace_bytes(cfg, budget_tokens) bytes
 *   status       nullable int32[1]
 */
int locks_select(const locks_cfg_t* cfg, const void* q, const void* summaries,
                 const int32_t* block_table, const int32_t* seq_lens, int32_t budget_tokens,
                 int32_t* selected, float* page_lse, float* page_share, void* workspace,
                 size_t workspace_bytes, int32_t* status, void* stream);

/*
 * locks_sparse_decode -- attention restricted to the selected pages with the
 * softmax renormalised over them (section 2, o_S; Lemma 1), computed as
 * split-K flash decoding: each split keeps a running max, sum and weighted
 * value sum over its pages, and the splits are merged by their log-sum-exp.
 * The tail page contributes only its valid tokens.  Entries < 0 in `selected`
 * are skipped.
 *
 *   selected     int32 [batch][n_kv_heads][k] logical page ids (as locks_select writes)
 *   out          bf16 [batch][n_q_heads][d]
 *   out_lse      nullable float [batch][n_q_heads]: natural-log log-sum-exp of
 *                the scaled logits over the attended tokens (-inf if none)
 *   workspace    >= locks_decode_workspace_bytes(cfg, k) bytes
 * A sequence with no attended token gets out = 0.
 */
int locks_sparse_decode(const locks_cfg_t* cfg, const void* q, const void* k_cache,
                        const void* v_cache, const int32_t* block_table, const int32_t* seq_lens,
                        const int32_t* selected, int32_t k, void* out, float* out_lse,
                        void* workspace, size_t workspace_bytes, int32_t* status, void* stream);

/*
 * locks_dense_decode -- full-cache paged decode attention (section 2, o), the
 * comparison point: the same split-K kernel over every page of each sequence.
 *   workspace    >= locks_decode_workspace_bytes(cfg, cfg->max_pages) bytes
 */
int locks_dense_decode(const locks_cfg_t* cfg, const void* q, const void* k_cache,
                       const void* v_cache, const int32_t* block_table, const int32_t* seq_lens,
                       void* out, float* out_lse, void* workspace, size_t workspace_bytes,
                       int32_t* status, void* stream);

/*
 * locks_select_noalloc -- the page selection of locks_select for callers that
 * cannot allocate device memory.  The paper has no counterpart: this is a
 * packaging variant, not a step of the method.
 *
 * Callers such as a serving engine whose memory pool already owns all of the
 * GPU, a plugin whose host forbids cudaMalloc on the decode path (it can
 * synchronise the device and fragment the pool), or an embedded user without
 * an allocator get the same selection without passing a workspace: the
 * scratch lives in one fixed device array of LOCKS_SELECT_NOALLOC_MAX_BYTES
 * inside the library, which every GPU that loads the library keeps until the
 * process exits.  The call itself allocates and frees nothing.
 *
 * Arguments and outputs are those of locks_select, minus the workspace.
 * Shapes whose locks_select_workspace_bytes(cfg, budget_tokens) exceeds
 * LOCKS_SELECT_NOALLOC_MAX_BYTES are rejected with LOCKS_ERR_WORKSPACE (for
 * example, with G = 4, batch x n_kv_heads x max_pages must stay below about
 * 250,000 pages).  The array's device address is looked up by the first call
 * on a device (with that device current) and again by the first call after
 * that device's context was destroyed and re-created (cudaDeviceReset): make
 * those calls before any stream capture.  Every call clears the scratch it uses on `stream` before selecting.
 * All calls share the one array: calls that can overlap on the GPU race.
 */
#define LOCKS_SELECT_NOALLOC_MAX_BYTES (4u << 20)
int locks_select_noalloc(const locks_cfg_t* cfg, const void* q, const void* summaries,
                         const int32_t* block_table, const int32_t* seq_lens,
                         int32_t budget_tokens, int32_t* selected, float* page_lse,
                         float* page_share, int32_t* status, void* stream);

/* ===========================================================================
 * The quantised cache: rotary positions, writing and reading a paged KV cache
 * in 8 or 4 bits, and decode attention over it.
 *
 * The conventions above hold (device pointers, no allocation, no
 * synchronisation, status bits).  The calls take their own configuration:
 * supported are head_dim = 128; page_size 64, 32 or 16; any G from 1 to 16;
 * max_pages < 2^24; num_blocks * n_kv_heads < 2^31; batch * n_kv_heads < 2^24;
 * and for the attention batch * n_kv_heads * (ceil(max_pages * page_size / 64) + 8)
 * < 2^31 (with a page list, k in place of max_pages, k < 2^24); at most 2^30
 * tokens a write, of at most 2^16 rows each (2 n_kv_heads, and n_q_heads where
 * queries are passed).
 * =========================================================================== */

/* element type of a quantised cache */
#define LOCKS_KV_F8 0   /* e4m3 codes, one scale per token and KV head              */
#define LOCKS_KV_I8 1   /* 8-bit integers, one scale per token and KV head          */
#define LOCKS_KV_I4 2   /* 4-bit integers, e4m3 scales of 32 dims, a scale per token */

typedef struct locks_kv_cfg {
  int32_t batch;          /* sequences (rows of block_table, >= 0)                     */
  int32_t n_q_heads;      /* query heads H_q                                           */
  int32_t n_kv_heads;     /* KV heads H_kv; H_q % H_kv == 0                            */
  int32_t head_dim;       /* d                                                         */
  int32_t page_size;      /* B, tokens per page                                        */
  int32_t max_pages;      /* row stride of block_table (pages per sequence, at most)  */
  int32_t num_blocks;     /* physical blocks in the pools                              */
  int32_t kv_dtype;       /* LOCKS_KV_F8, LOCKS_KV_I8 or LOCKS_KV_I4                   */
} locks_kv_cfg_t;

/*
 * Cache record: one per (physical block, KV head) in each of the K and the V
 * pool, at byte (block * n_kv_heads + h) * locks_kv_record_bytes(cfg).  With
 * B = page_size:
 *
 *   uint8_t codes[B][R]        R = 128 (F8, I8) or 64 (I4)
 *   uint8_t group[B][4]        I4 only: e4m3 scale of dims 32j .. 32j + 31
 *   float   scale[B]           scale of the token's row
 *
 * The 16-byte chunk c of row r is stored at byte r R + 16 (c ^ x(r)), with
 * x(r) = r & 7 for R = 128 and (r >> 1) & 3 for R = 64 (the order in which the
 * attention reads rows from shared memory without bank conflicts).  Before
 * that permutation byte i of a row is the code of dim i (F8: e4m3 bits; I8:
 * code + 128) or, in I4, of dims 2i (low nibble) and 2i + 1 (high nibble),
 * code + 8.  A dim stands for
 *
 *   F8, I8:  code * scale         I4:  code * group[dim / 32] * scale
 *
 * A row x is quantised in float32, every operation rounded to nearest even:
 *   scale = max|x| * (1 / t), t = 448 (F8), 127 (I8), 7 * 448 (I4);
 *   y = x * (1 / scale);  F8: code = e4m3(y);  I8: code = rint(y);
 *   I4: group = e4m3(max|y| over the group * (1 / 7)),
 *       code = rint(y * (1 / group)) within -7 .. 7 (0 where group is 0).
 * A row whose largest magnitude is below 2^-96 is stored as zeros with scale
 * 0; a row that holds an infinity or a NaN is stored with scale NaN, reads
 * back as NaN and makes the attention over it NaN.
 */
size_t locks_kv_record_bytes(const locks_kv_cfg_t* cfg);

/* rotary layouts: which elements of a head form the pair i < rotary_dim / 2 */
#define LOCKS_ROPE_HALF        0   /* (i, i + rotary_dim / 2) */
#define LOCKS_ROPE_INTERLEAVED 1   /* (2 i, 2 i + 1)          */

/* rotary frequency scalings */
#define LOCKS_ROPE_SCALE_NONE   0
#define LOCKS_ROPE_SCALE_LINEAR 1  /* w / factor                                          */
#define LOCKS_ROPE_SCALE_NTK    2  /* base theta * factor^(r / (r - 2)), r = rotary_dim   */
#define LOCKS_ROPE_SCALE_LLAMA3 3  /* by wavelength bands of the original context         */
#define LOCKS_ROPE_SCALE_YARN   4  /* ramp between two dims, and a factor on cos and sin   */

typedef struct locks_rope_spec {
  int32_t rotary_dim;         /* even, 2 .. 512                                          */
  int32_t scaling;            /* LOCKS_ROPE_SCALE_*                                      */
  double theta;               /* base, > 1                                               */
  double factor;              /* context extension, >= 1 (not read by SCALE_NONE)         */
  double low_freq_factor;     /* LLAMA3                                                  */
  double high_freq_factor;    /* LLAMA3, > low_freq_factor                               */
  double original_positions;  /* LLAMA3, YARN: original context, > 0                     */
  double beta_fast;           /* YARN: turns in the original context (usually 32)        */
  double beta_slow;           /* YARN (usually 1)                                        */
} locks_rope_spec_t;

/*
 * locks_rope_frequencies -- the rotation rate of each pair, on the HOST.
 *
 * w_i = theta^(-2 i / rotary_dim) radians per position, scaled by the spec:
 *   LINEAR  w / factor
 *   NTK     theta' = theta * factor^(rotary_dim / (rotary_dim - 2))
 *   LLAMA3  wavelength 2 pi / w above original / low_freq_factor: w / factor;
 *           below original / high_freq_factor: w; between: interpolated by
 *           (original / wavelength - low) / (high - low)
 *   YARN    w / factor * z + w * (1 - z), z = clamp((i - a) / (b - a), 0, 1),
 *           a = floor(D(beta_fast)), b = ceil(D(beta_slow)), clamped to
 *           [0, rotary_dim - 1], D(t) = rotary_dim ln(original / (2 pi t)) /
 *           (2 ln theta); mscale = 0.1 ln(factor) + 1
 * turns[i] = w_i / (2 pi) as a 64-bit binary fraction of a turn: the kernels
 * multiply it by the position modulo 2^64, which loses nothing, and keep the
 * top 32 bits.  The rate itself is computed in double and off by about 2^-55 of
 * a turn at most, so the angle at position p is within 2^-32 + |p| 2^-55 of a
 * turn: 2^-31 up to 8 million positions, 2^-24 at 2^31.
 *
 *   turns    HOST uint64 [rotary_dim / 2]: written
 *   mscale   HOST float: written, the factor on cos and sin (1 but for YARN)
 */
int locks_rope_frequencies(const locks_rope_spec_t* spec, uint64_t* turns, float* mscale);

/* a rotary table as the kernels take it */
typedef struct locks_rope_table {
  const uint64_t* turns;      /* DEVICE uint64 [rotary_dim / 2]                          */
  int32_t rotary_dim;         /* leading dims of a head that are rotated                 */
  int32_t layout;             /* LOCKS_ROPE_HALF or LOCKS_ROPE_INTERLEAVED               */
  float mscale;               /* factor on cos and sin                                   */
} locks_rope_table_t;

/* element types of locks_rope */
#define LOCKS_BF16 0
#define LOCKS_F16  1
#define LOCKS_F32  2

/*
 * locks_rope -- rotary positions: the pair (u, v) of a head at position p
 * becomes (u c - v s, v c + u s) with c, s = mscale * cos, sin(p w_i); dims
 * from rotary_dim on are copied.  `inverse` != 0 rotates by -p: the transposed
 * map, which is the gradient of the forward call with respect to x.  Computed
 * in float32 (cos and sin of the angle within 2^-23), rounded once.
 *
 *   head_dim          even, 2 .. 512; rope->rotary_dim <= head_dim
 *   n_heads           at most 2^24
 *   x, out            [n_tokens][n_heads][head_dim] of dtype, strides in
 *                     elements between tokens and between heads (the last dim
 *                     is contiguous); out may be x with the same strides, and
 *                     may not overlap it otherwise
 *   positions         int32 [n_tokens], any values
 */
int locks_rope(const locks_rope_table_t* rope, int32_t dtype, int32_t head_dim, const void* x,
               int64_t x_token_stride, int64_t x_head_stride, const int32_t* positions,
               int32_t n_tokens, int32_t n_heads, void* out, int64_t out_token_stride,
               int64_t out_head_stride, int32_t inverse, void* stream);

/*
 * locks_kv_write -- tokens (of a prompt, a chunk of one, or a decode step)
 * into a quantised cache, with the rotation of their queries and keys.
 *
 * Token i belongs to sequence token_seq[i] (i itself when token_seq is NULL)
 * at position token_pos[i]; its key rows, rotated by `rope`, and its value
 * rows go, quantised, to slot pos % B of block
 * block_table[seq * max_pages + pos / B] of the pools.  Keys are quantised
 * from the float32 rotation, without a rounding to bf16 in between.  Its query
 * rows, rotated and rounded to bf16, go to q_out.
 *
 *   k_new, v_new  bf16 rows: element e of head h of token i is at
 *                 i * stride + h * d + e; 16-byte aligned, strides multiples
 *                 of 8 elements (slices of one projection's output will do)
 *   q_new, q_out  nullable (both or neither); q_new as k_new, q_out bf16
 *                 [n_tokens][n_q_heads][d]; q_out may be q_new
 *   token_seq     nullable int32 [n_tokens]; a token with an entry < 0 is
 *                 padding: nothing of it is written
 *   token_pos     int32 [n_tokens]; no two tokens of a call may share a slot
 *   rope          nullable: no rotation; rotary_dim a multiple of 16, <= d
 *   seq_lens      nullable int32 [batch]: raised to at least pos + 1 (may not
 *                 be the array passed as token_pos)
 *   completed     nullable int32 [n_tokens]: the block whose last slot the
 *                 token took, else -1
 *   status        nullable int32[1]
 * A position outside [0, max_pages * B) (LOCKS_DEV_BAD_SEQ_LEN), a sequence
 * >= batch (LOCKS_DEV_BAD_PAGE_ID) or an invalid block (LOCKS_DEV_BAD_BLOCK_ID)
 * leaves the cache and seq_lens as they are, with completed -1; the query is
 * rotated all the same.
 */
int locks_kv_write(const locks_kv_cfg_t* cfg, const void* k_new, int64_t k_stride,
                   const void* v_new, int64_t v_stride, const void* q_new, int64_t q_stride,
                   void* q_out, const int32_t* token_seq, const int32_t* token_pos,
                   int32_t n_tokens, const locks_rope_table_t* rope, void* k_pool, void* v_pool,
                   const int32_t* block_table, int32_t* seq_lens, int32_t* completed,
                   int32_t* status, void* stream);

/*
 * locks_kv_read -- listed blocks of a quantised cache as bf16 pages, in the
 * layout of a bf16 pool of n_blocks blocks (locks_build_summaries reads it as
 * it stands).  Entries < 0 are skipped; an entry >= num_blocks is skipped with
 * LOCKS_DEV_BAD_BLOCK_ID.  Slots that were never written read as whatever
 * their bytes stand for.
 *
 *   block_ids     int32 [n_blocks]
 *   k_out, v_out  bf16 [n_blocks][n_kv_heads][B][d], 16-byte aligned; each
 *                 nullable (not both): only the other pool is read
 */
int locks_kv_read(const locks_kv_cfg_t* cfg, const void* k_pool, const void* v_pool,
                  const int32_t* block_ids, int32_t n_blocks, void* k_out, void* v_out,
                  int32_t* status, void* stream);

/* Bytes of workspace locks_kv_decode needs for this cfg: one of two sizes, by
 * whether G exceeds 8.  Configurations may share a workspace that is large
 * enough for each (calls on it one after the other). */
size_t locks_kv_decode_workspace_bytes(const locks_kv_cfg_t* cfg);

/*
 * locks_kv_decode -- attention of one new token per sequence over a quantised
 * cache: out = sum_t p_t v_t, p = softmax(q^T k_t / sqrt(d)) over the attended
 * tokens: those of every page or of the listed pages, and with window > 0 only
 * the last `window` positions.  The codes are read once, and scales multiply
 * logits and weights.  Logits, running maxima and sums are float32.  A weight
 * (p_t times the value's scale) is rounded to f16 before its product with the
 * codes: by 2^-11 of itself, or 2^-31 of the largest where it is smaller than
 * that; the products are summed in float32 and rounded to bf16 once.  Against 64
 * bits that adds about 1% to the error of the output's own rounding.
 *
 *   q             bf16 [batch][n_q_heads][d], 16-byte aligned
 *   seq_lens      int32 [batch], the new token included; a length of 0 gives
 *                 out = 0 and out_lse = -inf
 *   selected, k   nullable int32 [batch][n_kv_heads][k] logical page ids, each
 *                 at most once (as locks_select writes them); entries < 0 are
 *                 skipped.  NULL: every page (k is not read)
 *   window        0: no window
 *   out           bf16 [batch][n_q_heads][d], 16-byte aligned
 *   out_lse       nullable float [batch][n_q_heads]: natural-log log-sum-exp
 *   workspace     >= locks_kv_decode_workspace_bytes(cfg) bytes, 16-byte
 *                 aligned, zero-filled before its first use
 *   status        nullable int32[1]
 */
int locks_kv_decode(const locks_kv_cfg_t* cfg, const void* q, const void* k_pool,
                    const void* v_pool, const int32_t* block_table, const int32_t* seq_lens,
                    const int32_t* selected, int32_t k, int32_t window, void* out, float* out_lse,
                    void* workspace, size_t workspace_bytes, int32_t* status, void* stream);

/* ===========================================================================
 * A batch that shares prefixes and lives within a budget, over the bf16 pools.
 *
 * The conventions at the top hold (device pointers, no allocation, no
 * synchronisation, status bits).  The calls take a locks_cfg_t of which rank
 * and summary_dtype are not read; supported are head_dim = 128; page_size 64,
 * 32 or 16; any G from 1 to 16; max_pages < 2^24, max_pages * page_size < 2^30;
 * num_blocks * n_kv_heads < 2^31; batch * n_q_heads < 2^24.  locks_weigh takes
 * batch * n_kv_heads * (s + 1) < 2^31 with s = ceil(max_pages * page_size / 128), and
 * locks_prefix_decode (11 s + 8) * n_kv_heads * (batch + n_groups + 1 +
 * floor(batch * n_rows / (2 floor(128 / G)))) < 2^31, batch * n_rows < 2^24 - 256 and
 * batch * n_rows * n_q_heads < 2^28 (LOCKS_ERR_UNSUPPORTED otherwise).
 *
 * The newest tokens of a sequence: the calls take the queries of the last
 * n_rows tokens of every sequence, q [batch][n_rows][n_q_heads][d]: 1 in a
 * decode step, more for drafted tokens or the last tokens of a prompt.  Query
 * row r of a sequence of t tokens is that of slot t - n_rows + r and sees the
 * slots up to it.  A row whose slot would be negative sees nothing.  (Eviction
 * moves rows: several rows are the newest tokens' if they were appended since.)
 * n_rows <= 2 * floor(128 / G).
 * =========================================================================== */

/* Bytes of workspace locks_prefix_decode needs (0: refused arguments). */
size_t locks_prefix_workspace_bytes(const locks_cfg_t* cfg, int32_t n_groups, int32_t n_rows);

/*
 * locks_prefix_decode -- attention of the newest tokens of a batch whose
 * sequences share prefixes: out = sum_t p_t v_t, p = softmax(q^T k_t / sqrt(d))
 * over every slot the row sees.  Sequences group_starts[g] ..
 * group_starts[g + 1] - 1 have their first prefix_pages[g] pages in common; the
 * call reads them once for all of the group's queries (256 rows at a time),
 * through the block-table row of the group's first sequence, and each sequence's
 * further pages through its own row.  The entries of the other rows for shared
 * pages are not read.
 *
 *   q             bf16 [batch][n_rows][n_q_heads][d], 16-byte aligned
 *   k_cache, v_cache  the pools, 16-byte aligned
 *   seq_lens      int32 [batch], the new tokens included.  A sequence may end
 *                 inside its group's prefix
 *   group_starts  int32 [n_groups + 1], ascending, within 0 .. batch; sequences
 *                 outside every group share nothing.  If they are not, every
 *                 sequence is read through its own row (LOCKS_DEV_BAD_GROUP)
 *   prefix_pages  int32 [n_groups], each 0 .. max_pages
 *   n_groups      0 .. batch (0: the two arrays are not read and may be NULL)
 *   out           bf16 [batch][n_rows][n_q_heads][d], 16-byte aligned; a row
 *                 that sees nothing gets 0
 *   out_lse       nullable float [batch][n_rows][n_q_heads]: natural-log
 *                 log-sum-exp (-inf for a row that sees nothing)
 *   workspace     >= locks_prefix_workspace_bytes bytes, 16-byte aligned
 *
 * Logits, maxima, sums and accumulators are float32.  Weights are rounded to
 * bf16 before their product with the values (2^-8 of each at most), and the
 * output divides by their sum.  Slots that no row of a sequence (of a group,
 * within the prefix) sees may hold anything; a NaN or an infinity in the value of a token that only some
 * of the rows see (one of the last n_rows tokens, or a token of the prefix behind
 * a shorter sequence's end) may reach the others.
 * Pages of a block id outside the pool are left out (LOCKS_DEV_BAD_BLOCK_ID).
 */
int locks_prefix_decode(const locks_cfg_t* cfg, const void* q, int32_t n_rows, const void* k_cache,
                        const void* v_cache, const int32_t* block_table, const int32_t* seq_lens,
                        const int32_t* group_starts, const int32_t* prefix_pages, int32_t n_groups,
                        void* out, float* out_lse, void* workspace, size_t workspace_bytes,
                        int32_t* status, void* stream);

/*
 * locks_weigh -- the attention weight that each cached token has received:
 *
 *   out[slot] = decay * weights[slot] + sum over the query rows of the KV head
 *               that see the slot of exp(q^T k_slot / sqrt(d) - lse_row)
 *
 * for every slot from fixed[b] up to the sequence's length, with lse the rows'
 * log-sum-exp from the attention call before.  Weights (and positions) lie in
 * pools [num_blocks][n_kv_heads][page_size] beside the K/V pools, through the
 * same block table; a weighed page belongs to one sequence (fixed keeps a
 * shared prefix out).  The last n_new slots have no weight yet: their old one
 * counts as 0, and their entry of `positions` becomes slot + evicted[b].
 *
 *   q             bf16 [batch][n_rows][n_q_heads][d], 16-byte aligned
 *   lse           float [batch][n_rows][n_q_heads]; infinite: the row adds
 *                 nothing, whatever its query holds
 *   k_cache       the K pool, 16-byte aligned
 *   fixed         nullable int32 [batch], >= 0 (NULL: 0)
 *   weights       nullable float pool (NULL: every slot is new)
 *   out           float pool; may be weights.  Slots before fixed and behind the
 *                 sequence stay as they are
 *   n_new         >= 0
 *   decay         >= 0, 1 to accumulate
 *   positions     nullable int32 pool
 *   evicted       nullable int32 [batch]: tokens that locks_evict took so far
 * All of it in float32.  A key that is not finite may give its slot a NaN.  Slots of
 * a block id outside the pool are left out (LOCKS_DEV_BAD_BLOCK_ID).
 */
int locks_weigh(const locks_cfg_t* cfg, const void* q, int32_t n_rows, const float* lse,
                const void* k_cache, const int32_t* block_table, const int32_t* seq_lens,
                const int32_t* fixed, const float* weights, float* out, int32_t n_new, float decay,
                int32_t* positions, const int32_t* evicted, int32_t* status, void* stream);

/* Bytes of workspace locks_evict needs (0: refused arguments). */
size_t locks_evict_workspace_bytes(const locks_cfg_t* cfg, int32_t budget);

/*
 * locks_evict -- every sequence with more than `budget` slots behind its fixed
 * ones is cut to fixed[b] + budget slots, each KV head for itself: the slots
 * whose position is among the `recent` newest (position >= seq_lens[b] +
 * evicted[b] - recent) stay, then those of the largest weights; of equal ones the
 * lower slot stays.  A NaN weighs more than any number.
 *
 * Kept slots from fixed + budget on move into the holes before it, the lowest
 * into the lowest: rows of K and V, weights and positions.  So the order of slots
 * is lost, which attention does not depend on (keys are rotated before they are
 * cached); positions says where a slot's token stood.  Page summaries of pages
 * behind the fixed ones no longer describe them.  Everything behind the new
 * length stays as it is.  Then seq_lens[b] becomes fixed + budget, and
 * evicted[b] grows by what was dropped: the next token's position is
 * seq_lens[b] + evicted[b].
 *
 *   budget        >= 1
 *   recent        0 .. budget
 *   k_cache, v_cache  the pools, 16-byte aligned; written
 *   seq_lens      int32 [batch]; written
 *   fixed         nullable int32 [batch], >= 0 (NULL: 0): slots that are kept
 *                 where they are (a shared prefix, the first tokens)
 *   weights, positions  pools as for locks_weigh, 16-byte aligned; written
 *   evicted       int32 [batch]; written
 *   workspace     >= locks_evict_workspace_bytes bytes, 16-byte aligned,
 *                 zero-filled before its first use; shared only by calls of this
 *                 kind with the same batch (any budget)
 * A slot of a block id outside the pool weighs less than any other; moves from
 * or to one are left out (LOCKS_DEV_BAD_BLOCK_ID).
 */
int locks_evict(const locks_cfg_t* cfg, int32_t budget, int32_t recent, void* k_cache, void* v_cache,
                const int32_t* block_table, int32_t* seq_lens, const int32_t* fixed, float* weights,
                int32_t* positions, int32_t* evicted, void* workspace, size_t workspace_bytes,
                int32_t* status, void* stream);

/* Static string for a LOCKS_* return code. */
const char* locks_status_string(int code);

/* LOCKS_ABI_VERSION of the loaded library. */
int locks_abi_version(void);

#ifdef __cplusplus
}
#endif

#endif /* LOCKS_H_ */
