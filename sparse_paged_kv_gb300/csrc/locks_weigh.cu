// The attention weight that each cached token receives (locks_weigh):
//
//   w'[slot] = decay w[slot] + sum over the KV head's query rows that see the slot of
//              exp(q^T k_slot / sqrt(d) - lse_row).
//
// Every key is read once (256 bytes against 8 of weights), so memory bounds it
// while a sequence's rows are few.  The product is taken with the tokens as the
// rows of the matrix instruction: S^T (128 tokens x rows) = K Q^T, so that a
// thread holds one token, sums over its own registers and writes one float; no
// reduction across threads, no atomics, any number of rows up to 256 in one
// pass over the keys.  A list of stages of 128 tokens is shared out equally
// over 152 blocks (a stage's result is complete, so pieces need no joining).  A
// block's 10 warps: one loads keys (tensor maps, a ring of 32 KB tiles) and the
// unit's queries (two buffers), one issues the products, and two
// groups of four take stages in turn, thread = token, each with an accumulator
// of its own in tensor memory.  Weights and block ids of a stage are loaded
// before the wait for its product.  A step of 32 sequences of 4224 tokens (248 MB) takes 44 us, 5.65
// TB/s; the last 32 tokens of four 32K prompts (128 rows, 241 MB) 45.8 us, 5.25 TB/s.
#include "locks_batch.h"
#include "locks_batch.cuh"
#include "locks_kv.cuh"
#include "locks_tc.cuh"

namespace locks {

namespace {

constexpr int kThreads = 320;
constexpr int kProducerWarp = 8, kMmaWarp = 9;
constexpr int kTileBytes = 128 * 256;
constexpr int kHalfBytes = kTileBytes / 2;
constexpr int kMaxRing = 6;

struct Shared {
  uint64_t full[kMaxRing], empty[kMaxRing];
  uint64_t q_full[2], q_empty[2];
  uint64_t d_full[2], d_empty[2];
  uint64_t lse_full;
  uint64_t done;
  uint32_t tmem;
  int dead;
  ListPlace place;
  int off[2][8];                                      // a row of the warp's part has no weight; units in turn
  alignas(16) float minus_lse[2][256];                // of the unit, times log2 e; units in turn
};

struct Unit {
  int b, head, first, page0, len;                     // slots [first, len), from page page0 on
  int s0, s1;                                         // stages of this block
};

__device__ __forceinline__ int length_of(const WeighParams& p, int b) {
  return min(max(p.seq_lens[b], 0), p.max_pages * p.page_size);
}
__device__ __forceinline__ int first_of(const WeighParams& p, int b) {
  return p.fixed ? max(p.fixed[b], 0) : 0;
}
__device__ __forceinline__ int stages_of(const WeighParams& p, int b) {
  const int t = length_of(p, b), f = first_of(p, b);
  return f >= t ? 0 : (t - (f >> p.page_shift << p.page_shift) + kStageTok - 1) / kStageTok;
}

struct Walk {
  int b, offset, left, n;
  __device__ Walk(const WeighParams& p, const Shared& sh, int share)
      : b(sh.place.entry), offset(sh.place.offset), left(share), n(stages_of(p, b)) {}
  __device__ bool next(const WeighParams& p, Unit& u) {
    if (left <= 0) return false;
    while (offset >= n * p.n_kv_heads) {
      offset = 0;
      if (++b >= p.batch) return false;
      n = stages_of(p, b);
    }
    u.b = b;
    u.head = offset / n;
    u.len = length_of(p, b);
    u.first = first_of(p, b);
    u.page0 = u.first >> p.page_shift;
    u.s0 = offset - u.head * n;
    u.s1 = min(n, u.s0 + left);
    offset += u.s1 - u.s0;
    left -= u.s1 - u.s0;
    return true;
  }
};

__device__ void load_role(const WeighParams& p, Shared& sh, unsigned char* qbuf, unsigned char* ring,
                          const CUtensorMap* map_q, const CUtensorMap* map_k, int share) {
  const int lane = threadIdx.x & 31;
  const int per_stage = kStageTok >> p.page_shift;
  Walk walk(p, sh, share);
  Unit u;
  int qn = 0, stage = 0;
  bool ok = true;
  while (ok && walk.next(p, u)) {
    const int qs = qn & 1;
    ok = warp_wait_or_dead(&sh.q_empty[qs], ((qn >> 1) & 1) ^ 1, &sh.dead);
    if (!ok) break;
    if (lane == 0) {
      mbar_arrive_expect_tx(&sh.q_full[qs], p.n_rows * p.group * 256);
      unsigned char* dst = qbuf + qs * 2 * p.q_half;
      tma_load3(dst, map_q, 0, u.head * p.group, u.b * p.n_rows, &sh.q_full[qs]);
      tma_load3(dst + p.q_half, map_q, 64, u.head * p.group, u.b * p.n_rows, &sh.q_full[qs]);
    }
    ++qn;
    const int32_t* table = p.block_table + int64_t(u.b) * p.max_pages + u.page0;
    const int tokens = u.len - (u.page0 << p.page_shift);
    for (int s = u.s0; s < u.s1; ++s) {
      const int page = s * per_stage + lane;
      bool want = lane < per_stage && page << p.page_shift < tokens;
      int block = 0;
      if (want) {
        block = table[page];
        if (block < 0 || block >= p.num_blocks) {
          flag_status(p.status, LOCKS_DEV_BAD_BLOCK_ID);
          want = false;
        }
      }
      const int n = __popc(__ballot_sync(kFull, want));
      const int slot = stage % p.ring;
      ok = warp_wait_or_dead(&sh.empty[slot], ((stage / p.ring) & 1) ^ 1, &sh.dead);
      if (!ok) break;
      if (lane == 0) mbar_arrive_expect_tx(&sh.full[slot], (n << p.page_shift) * 256);
      __syncwarp();
      if (want) {
        unsigned char* dst = ring + slot * kTileBytes + (lane << p.page_shift) * 128;
        const int z = block * p.n_kv_heads + u.head;
        tma_load3(dst, map_k, 0, 0, z, &sh.full[slot]);
        tma_load3(dst + kHalfBytes, map_k, 64, 0, z, &sh.full[slot]);
      }
      ++stage;
    }
  }
  // no block leaves while copies into its memory are in flight
  if (!ok) {
    for (int c = max(0, stage - p.ring); c < stage; ++c)
      mbar_wait_bounded(&sh.full[c % p.ring], (c / p.ring) & 1);
    for (int t = max(0, qn - 2); t < qn; ++t)
      mbar_wait_bounded(&sh.q_full[t & 1], (t >> 1) & 1);
  }
}

__device__ void issue_role(const WeighParams& p, Shared& sh, unsigned char* qbuf, unsigned char* ring,
                           int share) {
  const uint32_t idesc = mma_idesc(128, p.n_cols, false), half = p.q_half >> 4;
  const uint32_t q_desc = smem_desc_lo(smem_u32(qbuf), 16), k_desc = smem_desc_lo(smem_u32(ring), 16);
  const uint32_t tmem = sh.tmem;
  Walk walk(p, sh, share);
  Unit u;
  int qn = 0, stage = 0;
  bool ok = true;
  while (ok && walk.next(p, u)) {
    const int qs = qn & 1;
    ok = warp_wait_or_dead(&sh.q_full[qs], (qn >> 1) & 1, &sh.dead);
    ++qn;
    const uint32_t db = warp_uniform(q_desc + qs * 2 * half);
    for (int s = u.s0; ok && s < u.s1; ++s, ++stage) {
      const int slot = stage % p.ring, w = stage & 1;
      ok = warp_wait_or_dead(&sh.full[slot], (stage / p.ring) & 1, &sh.dead) &&
           warp_wait_or_dead(&sh.d_empty[w], ((stage >> 1) & 1) ^ 1, &sh.dead);
      if (!ok) break;
      tc_fence_after();
      const uint32_t da = warp_uniform(k_desc + slot * (kTileBytes >> 4));
      const uint32_t d = warp_uniform(tmem + w * p.n_cols);
      if (elect_one()) {
#pragma unroll
        for (int k = 0; k < 8; ++k)                   // 16 of the 128 dims each, 64 in a half
          mma_ss(d, da + (((k >> 2) * kHalfBytes + (k & 3) * 32) >> 4),
                 db + (k >> 2) * half + (k & 3) * 2, idesc, k > 0);
        mma_commit(&sh.d_full[w]);
        mma_commit(&sh.empty[slot]);
        if (s == u.s1 - 1) mma_commit(&sh.q_empty[qs]);
      }
      __syncwarp();
    }
  }
  if (elect_one()) mma_commit(&sh.done);
  __syncwarp();
  mbar_wait_bounded(&sh.done, 0);
}

__device__ __forceinline__ void add_weights(const float* x, const float* minus, float2 scale, float2& a0,
                                            float2& a1) {
#pragma unroll
  for (int k = 0; k < 16; k += 4) {
    const float4 m = *reinterpret_cast<const float4*>(minus + k);
    float2 y = ffma2(make_float2(x[k], x[k + 1]), scale, make_float2(m.x, m.y));
    float2 z = ffma2(make_float2(x[k + 2], x[k + 3]), scale, make_float2(m.z, m.w));
    a0 = fadd2(a0, make_float2(ex2_approx(y.x), ex2_approx(y.y)));
    a1 = fadd2(a1, make_float2(ex2_approx(z.x), ex2_approx(z.y)));
  }
}

__device__ void weigh_role(const WeighParams& p, Shared& sh, int w, int share) {
  const int tid = threadIdx.x & 127, lane = tid & 31;
  const uint32_t d = sh.tmem + (uint32_t(tid >> 5 << 5) << 16) + w * p.n_cols;
  const int rows = p.n_rows * p.group;
  Walk walk(p, sh, share);
  Unit u;
  int stage = 0, units = 0;
  while (walk.next(p, u)) {
    // This unit's log-sum-exps, a part a warp.  (A row that sees nothing has -inf, and gives no weight: as
    // the columns behind the rows, whose queries are zeros, it gets the factor 2^-inf.  Its own query may
    // hold anything, NaN included, so a unit that has such a row takes the loop that looks at each.)
    // A warp that gets here has finished the unit before, so once all have arrived for
    // unit n, nobody reads the buffer of unit n - 1, which unit n + 1 takes.
    float* minus = sh.minus_lse[units & 1];
    bool off = false;
    for (int c = threadIdx.x; c < p.n_cols; c += 256) {
      const int r = c / p.group;
      float x = -INFINITY;
      if (c < rows)
        x = p.lse[(int64_t(u.b) * p.n_rows + r) * (p.n_kv_heads * p.group) + u.head * p.group +
                  c - r * p.group];
      minus[c] = x == -INFINITY ? -INFINITY : -x * kLog2e;
      off |= c < rows && minus[c] == -INFINITY;
    }
    off = __any_sync(kFull, off);
    __syncwarp();
    if (lane == 0) {
      sh.off[units & 1][threadIdx.x >> 5] = off;
      mbar_arrive(&sh.lse_full);
    }
    if (!warp_wait_or_dead(&sh.lse_full, units & 1, &sh.dead)) return;
    off = __any_sync(kFull, sh.off[units & 1][lane & 7]);
    ++units;
    const int32_t* table = p.block_table + int64_t(u.b) * p.max_pages;
    for (int s = u.s0; s < u.s1; ++s, ++stage) {
      if ((stage & 1) != w) continue;
      const int slot = (u.page0 << p.page_shift) + s * kStageTok + tid;
      const bool there = slot >= u.first && slot < u.len;
      const bool fresh = !p.weights || slot >= u.len - p.n_new;
      int64_t at = -1;
      float old = 0.f;
      if (there) {
        const int block = table[slot >> p.page_shift];
        if (block >= 0 && block < p.num_blocks) {
          at = (int64_t(block) * p.n_kv_heads + u.head) * p.page_size + (slot & (p.page_size - 1));
          if (!fresh) old = p.weights[at];
        }
      }
      if (!warp_wait_or_dead(&sh.d_full[w], (stage >> 1) & 1, &sh.dead)) return;
      tc_fence_after();
      // rows from c0 on see this slot
      const int c0 = max(0, slot - (u.len - p.n_rows)) * p.group;
      const float2 scale = make_float2(p.scale_log2, p.scale_log2);
      float2 a0 = make_float2(0.f, 0.f), a1 = a0;
      if (off || __any_sync(kFull, there && c0 > 0)) {
        for (int c = 0; c < p.n_cols; c += 16) {
          float x[16];
          tmem_ld16(d + c, x);
          tmem_wait_ld();
#pragma unroll
          for (int k = 0; k < 16; ++k) {
            const float y = ex2_approx(fmaf(x[k], p.scale_log2, minus[c + k]));
            if (c + k >= c0 && minus[c + k] != -INFINITY) a0.x += y;
          }
        }
      } else {
        // two columns an instruction, sixteen loaded while sixteen are added up
        float x[2][16];
        tmem_ld16(d, x[0]);
        for (int c = 0; c < p.n_cols; c += 32) {
          tmem_wait_ld();
          if (c + 16 < p.n_cols) tmem_ld16(d + c + 16, x[1]);
          add_weights(x[0], minus + c, scale, a0, a1);
          if (c + 16 >= p.n_cols) break;
          tmem_wait_ld();
          if (c + 32 < p.n_cols) tmem_ld16(d + c + 32, x[0]);
          add_weights(x[1], minus + c + 16, scale, a0, a1);
        }
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&sh.d_empty[w]);
      if (at >= 0) {
        p.out[at] = fmaf(p.decay, old, (a0.x + a0.y) + (a1.x + a1.y));
        if (fresh && p.positions) p.positions[at] = slot + (p.evicted ? p.evicted[u.b] : 0);
      }
    }
  }
}

__global__ void __launch_bounds__(kThreads, 1)
    weigh_kernel(const WeighParams p, const __grid_constant__ CUtensorMap map_q,
                 const __grid_constant__ CUtensorMap map_k) {
  extern __shared__ __align__(1024) unsigned char smem[];
  unsigned char* ring = smem;
  unsigned char* qbuf = ring + p.ring * kTileBytes;
  Shared& sh = *reinterpret_cast<Shared*>(qbuf + 4 * p.q_half);
  const int tid = threadIdx.x, warp = tid >> 5;

  if (warp == kMmaWarp) tmem_alloc(&sh.tmem, p.tmem_cols);
  if (tid == 0) {
    for (int i = 0; i < p.ring; ++i) {
      mbar_init(&sh.full[i], 1);
      mbar_init(&sh.empty[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&sh.q_full[i], 1);
      mbar_init(&sh.q_empty[i], 1);
      mbar_init(&sh.d_full[i], 1);
      mbar_init(&sh.d_empty[i], 4);
    }
    mbar_init(&sh.lse_full, 8);
    mbar_init(&sh.done, 1);
    mbar_fence_init();
    sh.dead = 0;
    prefetch_map(&map_q);
    prefetch_map(&map_k);
  }
  // the rows behind the queries' last, which no load writes, become zeros
  for (int i = tid; i < 4 * p.q_half / 16; i += kThreads)
    reinterpret_cast<uint4*>(qbuf)[i] = make_uint4(0, 0, 0, 0);
  proxy_fence_smem();
  griddep_wait();
  tc_fence_before();
  const int share = locate<kThreads>(
      [&](int b) { return stages_of(p, b) * p.n_kv_heads; }, p.batch, blockIdx.x, 1, kBatchSms, sh.place);
  tc_fence_after();
  if (blockIdx.x == 0)
    for (int b = tid; b < p.batch; b += kThreads)
      if (p.seq_lens[b] < 0 || p.seq_lens[b] > p.max_pages * p.page_size)
        flag_status(p.status, LOCKS_DEV_BAD_SEQ_LEN);
  if (share > 0) {
    if (warp < kProducerWarp) weigh_role(p, sh, warp >> 2, share);
    else if (warp == kProducerWarp) load_role(p, sh, qbuf, ring, &map_q, &map_k, share);
    else if (warp == kMmaWarp) issue_role(p, sh, qbuf, ring, share);
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (tid == 0 && sh.dead) flag_status(p.status, LOCKS_DEV_WAIT_TIMEOUT);
  if (warp == kMmaWarp) tmem_free(sh.tmem, p.tmem_cols);
}

}  // namespace

int launch_weigh(WeighParams p, const CUtensorMap& q, const CUtensorMap& k, cudaStream_t stream) {
  const int rows = p.n_rows * p.group;
  p.n_cols = (rows + 15) / 16 * 16;
  p.q_half = p.n_cols * 128;                          // 64 columns of the unit's queries, and zeros
  p.tmem_cols = 32;
  while (p.tmem_cols < 2 * p.n_cols) p.tmem_cols *= 2;
  const int fixed = 4 * p.q_half + int(sizeof(Shared));
  p.ring = (int(kMaxSmemBlock) - fixed) / kTileBytes;
  if (p.ring > kMaxRing) p.ring = kMaxRing;
  static LaunchOnce once;
  if (!once.run([] {
        return cudaFuncSetAttribute(weigh_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                    int(kMaxSmemBlock)) == cudaSuccess;
      }))
    return LOCKS_ERR_CUDA;
  cudaLaunchConfig_t lc = {};
  lc.gridDim = dim3(kBatchSms);
  lc.blockDim = dim3(kThreads);
  lc.dynamicSmemBytes = size_t(p.ring) * kTileBytes + fixed;
  lc.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  lc.attrs = attr;
  lc.numAttrs = 1;
  return cudaLaunchKernelEx(&lc, weigh_kernel, p, q, k) == cudaSuccess ? LOCKS_OK : LOCKS_ERR_CUDA;
}

}  // namespace locks
