// Eviction of the tokens of least weight (locks_evict).
//
// Of a (sequence, KV head)'s n = len - fixed slots behind the fixed ones, the
// `budget` of the largest keys stay: key = the weight's bits in order (the
// newest positions above all, a NaN above every number), ties to the lower slot.
// The kept ones among the slots behind the first `budget` then move into the
// holes among those, in ascending order on both sides; nothing else moves.  What
// is moved is read behind fixed + budget and written before it, so rows never
// overlap and any block may move any of them.
//
// A cluster of 1 to 16 blocks takes one (sequence, KV head); each block has a
// neighbouring share of its slots and keeps their keys in shared memory.  The
// budget-th largest key is found digit by digit (11, 11 and 10 bits), with
// a histogram a block, added up over the cluster through distributed shared
// memory.  Counts of ties, holes and movers are scanned over the block's
// threads and then over the cluster, which gives every hole and every mover its
// number; the lists go through the workspace, and all warps of the cluster move
// rows, 16 bytes a lane: lanes 0-15 the key, 16-31 the value.
// Bound: long prompts by the moves' traffic, a decode step by latency.
#include <cooperative_groups.h>

#include "locks_batch.h"
#include "locks_kv.cuh"

namespace cg = cooperative_groups;

namespace locks {

namespace {

constexpr int kThreads = 512;
constexpr int kBins = 2048;
constexpr int kMaxKeys = 40 * 1024;                   // kept in shared memory by a block
constexpr uint32_t kKeyRecent = 0xFFFFFFFFu, kKeyNaN = 0xFFFFFFFEu;

struct Shared {
  int hist[kBins];
  int warp[kThreads / 32][2];
  int ties, holes, movers;                            // of this block
  int digit, above;
};

// exclusive sums of two values over the block's threads; totals in t0, t1
__device__ __forceinline__ void scan2(Shared& sh, int v0, int v1, int& e0, int& e1, int& t0, int& t1) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int a = v0, b = v1;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int x = __shfl_up_sync(kFull, a, o), y = __shfl_up_sync(kFull, b, o);
    if (lane >= o) {
      a += x;
      b += y;
    }
  }
  __syncthreads();
  if (lane == 31) {
    sh.warp[warp][0] = a;
    sh.warp[warp][1] = b;
  }
  __syncthreads();
  t0 = t1 = 0;
  e0 = a - v0;
  e1 = b - v1;
#pragma unroll
  for (int i = 0; i < kThreads / 32; ++i) {
    if (i < warp) {
      e0 += sh.warp[i][0];
      e1 += sh.warp[i][1];
    }
    t0 += sh.warp[i][0];
    t1 += sh.warp[i][1];
  }
}

__device__ __forceinline__ uint32_t weight_key(float w) {
  if (w != w) return kKeyNaN;
  const uint32_t u = __float_as_uint(w + 0.f);        // (-0 is 0)
  return u & 0x80000000u ? ~u : u | 0x80000000u;
}

__global__ void __launch_bounds__(kThreads) evict_kernel(const EvictParams p) {
  extern __shared__ __align__(16) unsigned char smem[];
  Shared& sh = *reinterpret_cast<Shared*>(smem);
  uint32_t* keys = reinterpret_cast<uint32_t*>(smem + sizeof(Shared));
  cg::cluster_group cluster = cg::this_cluster();
  const int C = int(cluster.num_blocks()), rank = int(cluster.block_rank());
  const int tid = threadIdx.x;
  const int unit = blockIdx.x / C, b = unit / p.n_kv_heads, h = unit - b * p.n_kv_heads;
  griddep_wait();

  const int raw = p.seq_lens[b], gone = p.evicted[b];
  const int len = min(max(raw, 0), p.max_pages * p.page_size);
  if (tid == 0 && rank == 0 && h == 0 && len != raw) flag_status(p.status, LOCKS_DEV_BAD_SEQ_LEN);
  const int first = min(p.fixed ? max(p.fixed[b], 0) : 0, len);
  const int n = len - first;
  if (n <= p.budget) return;                          // (the whole cluster, and every head)
  const int64_t newest = int64_t(len) + gone - p.recent;   // positions from here on are recent
  const int32_t* table = p.block_table + int64_t(b) * p.max_pages;

  // this block's slots [lo, hi) of the n, and of them a run a thread
  const int lo = int(int64_t(n) * rank / C), hi = int(int64_t(n) * (rank + 1) / C), m = hi - lo;
  const bool held = m <= p.keys;
  auto place = [&](int i) -> int64_t {                // where slot i (of the n) lies in the pools, or -1
    const int slot = first + i, block = table[slot >> p.page_shift];
    if (block < 0 || block >= p.num_blocks) return -1;
    return (int64_t(block) * p.n_kv_heads + h) * p.page_size + (slot & (p.page_size - 1));
  };
  auto make_key = [&](int i) -> uint32_t {
    const int64_t at = place(i);
    if (at < 0) return 0;
    return p.positions[at] >= newest ? kKeyRecent : weight_key(p.weights[at]);
  };
  auto key = [&](int i) { return held ? keys[i - lo] : make_key(i); };
  if (held) {
    for (int i = tid; i < m; i += kThreads) keys[i] = make_key(lo + i);
  }

  // ---- the budget-th largest key, T; `need` slots of that key stay ----
  uint32_t T = 0;
  int need = p.budget;
  int shift = 32;
#pragma unroll 1
  for (int pass = 0; pass < 3; ++pass) {
    const int bits = pass < 2 ? 11 : 10, top = shift;
    shift -= bits;
    for (int i = tid; i < kBins; i += kThreads) sh.hist[i] = 0;
    __syncthreads();
    for (int i = lo + tid; i < hi; i += kThreads) {
      const uint32_t k = key(i);
      if (pass == 0 || k >> top == T >> top) atomicAdd(&sh.hist[(k >> shift) & ((1u << bits) - 1)], 1);
    }
    if (C > 1) cluster.sync();
    else __syncthreads();
    // thread t has bins 4t .. 4t + 3 from the top down
    int v[4], sum = 0;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const int bin = kBins - 1 - (4 * tid + k);
      v[k] = 0;
      for (int r = 0; r < C; ++r) v[k] += C > 1 ? cluster.map_shared_rank(sh.hist, r)[bin] : sh.hist[bin];
      sum += v[k];
    }
    int before, unused, t0, t1;
    scan2(sh, sum, 0, before, unused, t0, t1);
    if (need > before && need <= before + sum) {
      int at = before;
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        if (need > at && need <= at + v[k]) {
          sh.digit = kBins - 1 - (4 * tid + k);
          sh.above = at;
        }
        at += v[k];
      }
    }
    if (C > 1) cluster.sync();                        // (the histograms are cleared next)
    else __syncthreads();
    T |= uint32_t(sh.digit) << shift;
    need -= sh.above;
  }

  // ---- ties, holes and movers ----
  const int run = (m + kThreads - 1) / kThreads;
  const int r_lo = min(hi, lo + tid * run), r_hi = min(hi, r_lo + run);
  int ties = 0;
  for (int i = r_lo; i < r_hi; ++i) ties += key(i) == T;
  int tie_at, unused, total, t1;
  scan2(sh, ties, 0, tie_at, unused, total, t1);
  if (C > 1) {
    if (tid == 0) sh.ties = total;
    cluster.sync();
    for (int r = 0; r < rank; ++r) tie_at += *cluster.map_shared_rank(&sh.ties, r);
  }
  int holes = 0, movers = 0, tie = tie_at;
  for (int i = r_lo; i < r_hi; ++i) {
    const uint32_t k = key(i);
    const bool keep = k > T || (k == T && tie < need);
    tie += k == T;
    if (i < p.budget) holes += !keep;
    else movers += keep;
  }
  int hole_at, mover_at, all_holes, all_movers;
  scan2(sh, holes, movers, hole_at, mover_at, all_holes, all_movers);
  int moves = all_movers;
  if (C > 1) {
    if (tid == 0) {
      sh.holes = all_holes;
      sh.movers = all_movers;
    }
    cluster.sync();
    moves = 0;
    for (int r = 0; r < C; ++r) {
      const int x = *cluster.map_shared_rank(&sh.holes, r), y = *cluster.map_shared_rank(&sh.movers, r);
      if (r < rank) {
        hole_at += x;
        mover_at += y;
      }
      moves += y;
    }
  }
  int32_t* to = p.lists + int64_t(unit) * 2 * p.list_len;
  int32_t* from = to + p.list_len;
  tie = tie_at;
  for (int i = r_lo; i < r_hi; ++i) {
    const uint32_t k = key(i);
    const bool keep = k > T || (k == T && tie < need);
    tie += k == T;
    if (i < p.budget) {
      if (!keep) to[hole_at++] = i;
    } else if (keep) {
      from[mover_at++] = i;
    }
  }
  __threadfence();
  if (C > 1) cluster.sync();
  else __syncthreads();

  // every block of this head is past its reads of the length: the last head writes it
  if (rank == 0 && tid == 0) {
    if (atomicAdd(p.tickets + b, 1) == p.n_kv_heads - 1) {
      p.tickets[b] = 0;
      p.seq_lens[b] = first + p.budget;
      p.evicted[b] = gone + (n - p.budget);
    }
  }

  // ---- moves ----
  constexpr int kAhead = 4;
  const int lane = tid & 31, warps = kThreads / 32 * C, warp = rank * (kThreads / 32) + (tid >> 5);
  const __nv_bfloat16* src_pool = lane < 16 ? p.k_cache : p.v_cache;
  for (int i0 = warp; i0 < moves; i0 += warps * kAhead) {
    int64_t src[kAhead], dst[kAhead];
    uint4 row[kAhead];
    float wt[kAhead];
    int32_t ps[kAhead];
#pragma unroll
    for (int a = 0; a < kAhead; ++a) {
      const int i = i0 + a * warps;
      src[a] = dst[a] = -1;
      if (i < moves) {
        src[a] = place(__ldcg(from + i));
        dst[a] = place(__ldcg(to + i));
        if (src[a] < 0 || dst[a] < 0) {
          src[a] = -1;
          if (lane == 0) flag_status(p.status, LOCKS_DEV_BAD_BLOCK_ID);
        }
      }
    }
#pragma unroll
    for (int a = 0; a < kAhead; ++a)
      if (src[a] >= 0) {
        row[a] = *reinterpret_cast<const uint4*>(src_pool + src[a] * kHeadDim + (lane & 15) * 8);
        if (lane == 0) wt[a] = p.weights[src[a]];
        if (lane == 1) ps[a] = p.positions[src[a]];
      }
#pragma unroll
    for (int a = 0; a < kAhead; ++a)
      if (src[a] >= 0) {
        __nv_bfloat16* out = lane < 16 ? p.k_cache : p.v_cache;
        *reinterpret_cast<uint4*>(out + dst[a] * kHeadDim + (lane & 15) * 8) = row[a];
        if (lane == 0) p.weights[dst[a]] = wt[a];
        if (lane == 1) p.positions[dst[a]] = ps[a];
      }
  }
}

}  // namespace

int evict_list_len(int budget, int64_t slots) { return int(budget < slots / 2 ? budget : slots / 2) + 1; }

int launch_evict(EvictParams p, cudaStream_t stream) {
  const int units = p.batch * p.n_kv_heads;
  const int64_t slots = int64_t(p.max_pages) * p.page_size;
  // Blocks a head: as many as fill the SMs, while each still has some thousand slots.
  int C = 1;
  while (C < 16 && units * C * 2 <= kBatchSms && slots / (2 * C) >= 1024) C *= 2;
  const int64_t share = (slots + C - 1) / C;
  p.keys = int(share < kMaxKeys ? share : kMaxKeys);
  static LaunchOnce once;
  constexpr int kMost = int(sizeof(Shared)) + kMaxKeys * 4;
  static_assert(kMost <= int(kMaxSmemBlock), "shared memory of a block");
  if (!once.run([] {
        return cudaFuncSetAttribute(evict_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kMost) ==
                   cudaSuccess &&
               cudaFuncSetAttribute(evict_kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1) ==
                   cudaSuccess;
      }))
    return LOCKS_ERR_CUDA;
  cudaLaunchConfig_t lc = {};
  lc.gridDim = dim3(unsigned(units) * C);
  lc.blockDim = dim3(kThreads);
  lc.dynamicSmemBytes = sizeof(Shared) + size_t(p.keys) * 4;
  lc.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = C;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  lc.attrs = attr;
  lc.numAttrs = 2;
  return cudaLaunchKernelEx(&lc, evict_kernel, p) == cudaSuccess ? LOCKS_OK : LOCKS_ERR_CUDA;
}

}  // namespace locks
