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
// neighbouring share of its slots and keeps their keys in shared memory (a share
// larger than that goes through it in chunks, made anew each time).  The
// budget-th largest key is found digit by digit (11, 11 and 10 bits), with
// a histogram a block, added up over the cluster through distributed shared
// memory.  Thread = slot, so 32 neighbouring slots are a warp's: their holes and
// movers (and, where not all of them stay, ties) are counted by votes, the counts
// of 32s scanned over the block and the cluster, which gives every hole and every
// mover its number.  The lists of pool rows go through the workspace, and all warps of the
// cluster move rows, 16 bytes a lane: lanes 0-15 the key, 16-31 the value.
// Bound: long prompts by the chain of phases and then the moves' traffic (four 32K prompts cut to 4096
// tokens, on the device: 44 us, of which 16 for 117 MB read and written at 7.3 TB/s; one of 128K to 8192:
// 46), a decode step by latency (7 us).
#include <atomic>
#include <climits>

#include <cooperative_groups.h>

#include "locks_batch.h"
#include "locks_kv.cuh"

namespace cg = cooperative_groups;

namespace locks {

namespace {

constexpr int kThreads = 512;
constexpr int kBins = 2048;
constexpr int kMostCluster = kEvictMostBlocks;
constexpr int kMaxKeys = 40 * 1024;                   // kept in shared memory by a block
constexpr int kAhead = 2, kMoveAhead = 4;             // loads ahead: four slots of a thread, rows of a warp
// Up to so many slots to evict are found one after another, as least keys (a decode step evicts as many
// as it added: 4097 slots in 7 to 8 us on the device, by digits 28).
constexpr int kFew = 8;
constexpr uint32_t kKeyRecent = 0xFFFFFFFFu, kKeyNaN = 0xFFFFFFFEu;

struct Shared {
  alignas(16) int hist[kBins];
  int2 warp[kThreads / 32];
  int2 count[kMaxKeys / 32];                          // (holes or ties, movers) of 32 slots; then before them
  int2 total[3];                                      // of this block, a count each
  int digit, above, equal;
  int4 found;                                         // T, need and equal, from the cluster's first block
  uint64_t least[2][kThreads / 32], block_least[2];   // by rounds
  int hole[kFew], mover[kFew], few_moves;
};

// exclusive sum of v over the block's threads (two values at once); the total in t
__device__ __forceinline__ int2 scan(Shared& sh, int2 v, int2& t) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int2 a = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int x = __shfl_up_sync(kFull, a.x, o), y = __shfl_up_sync(kFull, a.y, o);
    if (lane >= o) {
      a.x += x;
      a.y += y;
    }
  }
  __syncthreads();
  if (lane == 31) sh.warp[warp] = a;
  __syncthreads();
  // the warps' sums, one a lane
  int2 w = lane < kThreads / 32 ? sh.warp[lane] : make_int2(0, 0);
  const int2 own = w;
#pragma unroll
  for (int o = 1; o < kThreads / 32; o <<= 1) {
    const int x = __shfl_up_sync(kFull, w.x, o), y = __shfl_up_sync(kFull, w.y, o);
    if (lane >= o) {
      w.x += x;
      w.y += y;
    }
  }
  t = make_int2(__shfl_sync(kFull, w.x, kThreads / 32 - 1), __shfl_sync(kFull, w.y, kThreads / 32 - 1));
  const int bx = __shfl_sync(kFull, w.x - own.x, warp), by = __shfl_sync(kFull, w.y - own.y, warp);
  return make_int2(bx + a.x - v.x, by + a.y - v.y);
}

__device__ __forceinline__ uint64_t least_of_warp(uint64_t x) {
  const uint32_t hi = __reduce_min_sync(kFull, uint32_t(x >> 32));
  const uint32_t lo = __reduce_min_sync(kFull, uint32_t(x >> 32) == hi ? uint32_t(x) : 0xFFFFFFFFu);
  return uint64_t(hi) << 32 | lo;
}

__device__ __forceinline__ uint32_t weight_key(float w) {
  if (w != w) return kKeyNaN;
  const uint32_t u = __float_as_uint(w + 0.f);        // (-0 is 0)
  return u & 0x80000000u ? ~u : u | 0x80000000u;
}

__global__ void __launch_bounds__(kThreads, 2) evict_kernel(const EvictParams p) {
  extern __shared__ __align__(16) unsigned char smem[];
  Shared& sh = *reinterpret_cast<Shared*>(smem);
  uint32_t* keys = reinterpret_cast<uint32_t*>(smem + sizeof(Shared));
  cg::cluster_group cluster = cg::this_cluster();
  const int C = int(cluster.num_blocks()), rank = int(cluster.block_rank());
  const int tid = threadIdx.x, lane = tid & 31;
  const int unit = blockIdx.x / C, b = unit / p.n_kv_heads, h = unit - b * p.n_kv_heads;
  auto meet = [&]() {                                 // all threads of the cluster
    if (C > 1) cluster.sync();
    else __syncthreads();
  };
  griddep_wait();

  const int raw = p.seq_lens[b], gone = p.evicted[b];
  const int len = min(max(raw, 0), p.max_pages * p.page_size);
  if (tid == 0 && rank == 0 && h == 0 && len != raw) flag_status(p.status, LOCKS_DEV_BAD_SEQ_LEN);
  const int first = min(p.fixed ? max(p.fixed[b], 0) : 0, len);
  const int n = len - first;
  if (n <= p.budget) return;                          // (the whole cluster, and every head)
  const int64_t newest = int64_t(len) + gone - p.recent;   // positions from here on are recent
  const int32_t* table = p.block_table + int64_t(b) * p.max_pages;

  // this block's slots [lo, hi) of the n, in chunks of p.keys
  const int lo = int(int64_t(n) * rank / C), hi = int(int64_t(n) * (rank + 1) / C);
  // once every block of this head is past its reads of the length: the last head writes it
  auto finish = [&]() {
    if (rank == 0 && tid == 0) {
      __threadfence();
      if (atomicAdd(p.tickets + b, 1) == p.n_kv_heads - 1) {
        p.tickets[b] = 0;
        p.seq_lens[b] = first + p.budget;
        p.evicted[b] = gone + (n - p.budget);
      }
    }
  };
  auto place = [&](int i) -> int64_t {                // where slot i (of the n) lies in the pools, or -1
    const int slot = first + i, block = table[slot >> p.page_shift];
    if (block < 0 || block >= p.num_blocks) return -1;
    return (int64_t(block) * p.n_kv_heads + h) * p.page_size + (slot & (p.page_size - 1));
  };
  // Keys of the chunk that begins at c0: four neighbouring slots a load, so from up to three slots before c0
  // on (those, and the ones behind the chunk's end, are never looked at).
  int loaded = -1, shifted = 0;                       // the chunk whose keys are there
  auto key = [&](int i) { return keys[i - loaded + shifted]; };
  auto load = [&](int c0, int c1) {                   // ends with the keys visible to the block
    if (loaded == c0) return;
    if (loaded >= 0) __syncthreads();                 // (the chunk before is still looked at)
    loaded = c0;
    shifted = (first + c0) & 3;
    const int fours = (c1 - c0 + shifted + 3) / 4;
    for (int f0 = tid; f0 < fours; f0 += kThreads * kAhead) {
      int64_t at[kAhead];
      int4 pos[kAhead];
      float4 w[kAhead];
#pragma unroll
      for (int k = 0; k < kAhead; ++k) {
        const int f = f0 + k * kThreads;
        at[k] = f < fours ? place(c0 - shifted + 4 * f) : -1;
      }
#pragma unroll
      for (int k = 0; k < kAhead; ++k)
        if (at[k] >= 0) {
          pos[k] = *reinterpret_cast<const int4*>(p.positions + at[k]);
          w[k] = *reinterpret_cast<const float4*>(p.weights + at[k]);
        }
#pragma unroll
      for (int k = 0; k < kAhead; ++k) {
        const int f = f0 + k * kThreads;
        uint4 x = make_uint4(0, 0, 0, 0);
        if (at[k] >= 0) {
          x.x = pos[k].x >= newest ? kKeyRecent : weight_key(w[k].x);
          x.y = pos[k].y >= newest ? kKeyRecent : weight_key(w[k].y);
          x.z = pos[k].z >= newest ? kKeyRecent : weight_key(w[k].z);
          x.w = pos[k].w >= newest ? kKeyRecent : weight_key(w[k].w);
        }
        if (f < fours) *reinterpret_cast<uint4*>(keys + 4 * f) = x;
      }
    }
    __syncthreads();
  };

  // ---- a few slots to evict ----
  if (n - p.budget <= kFew && (n + C - 1) / C <= p.keys) {
    load(lo, hi);
    // (key, ~slot) of the one evicted last: of equal keys the higher slot goes first
    uint64_t last = 0;
    int gone_slot[kFew];
    for (int round = 0; round < n - p.budget; ++round) {
      const int at = round & 1;
      uint64_t best = ~uint64_t(0);
      for (int i = lo + tid; i < hi; i += kThreads) {
        const uint64_t x = uint64_t(key(i)) << 32 | uint32_t(~i);
        if (x < best && (round == 0 || x > last)) best = x;
      }
      best = least_of_warp(best);
      if (lane == 0) sh.least[at][tid >> 5] = best;
      __syncthreads();
      best = least_of_warp(lane < kThreads / 32 ? sh.least[at][lane] : ~uint64_t(0));
      if (C > 1) {
        if (tid == 0) sh.block_least[at] = best;
        cluster.sync();
        best = least_of_warp(lane < C ? *cluster.map_shared_rank(&sh.block_least[at], lane) : ~uint64_t(0));
      }
      last = best;
#pragma unroll
      for (int k = 0; k < kFew; ++k)
        if (k == round) gone_slot[k] = ~uint32_t(best);
    }
    if (rank == 0) {
      if (tid == 0) {
        // holes before the budget and kept slots behind it, ascending: both are few
        int holes = 0, movers = 0;
        for (int round = 0; round < n - p.budget; ++round) {
          int next = INT_MAX;                         // the least hole above the one before
#pragma unroll
          for (int k = 0; k < kFew; ++k)
            if (k < n - p.budget && gone_slot[k] < p.budget && gone_slot[k] < next &&
                (holes == 0 || gone_slot[k] > sh.hole[holes - 1]))
              next = gone_slot[k];
          if (next == INT_MAX) break;
          sh.hole[holes++] = next;
        }
        for (int i = p.budget; i < n; ++i) {
          bool stays = true;
#pragma unroll
          for (int k = 0; k < kFew; ++k) stays = stays && !(k < n - p.budget && gone_slot[k] == i);
          if (stays) sh.mover[movers++] = i;
        }
        sh.few_moves = movers;
      }
      __syncthreads();
      const int i = tid >> 5;
      if (i < sh.few_moves) {
        const int64_t src = place(sh.mover[i]), dst = place(sh.hole[i]);
        if (src >= 0 && dst >= 0) {
          __nv_bfloat16* pool = (lane < 16 ? p.k_cache : p.v_cache) + (lane & 15) * 8;
          *reinterpret_cast<uint4*>(pool + dst * kHeadDim) = *reinterpret_cast<const uint4*>(pool + src * kHeadDim);
          if (lane == 0) p.weights[dst] = p.weights[src];
          if (lane == 1) p.positions[dst] = p.positions[src];
        } else if (lane == 0) {
          flag_status(p.status, LOCKS_DEV_BAD_BLOCK_ID);
        }
      }
    }
    if (C > 1) cluster.sync();                        // (nobody leaves while its candidate may be read)
    finish();
    return;
  }

  // ---- the budget-th largest key, T; `need` slots of that key stay, of `equal` ----
  uint32_t T = 0;
  int need = p.budget, equal = 0;
  // the digit at `shift` of T, from the block's histogram or its cluster's first block's: thread t has
  // bins 4t .. 4t + 3 from the top down
  auto take = [&](const int* hist) {
    const int bin = kBins - 4 - 4 * tid;
    const int4 bins = *reinterpret_cast<const int4*>(hist + bin);
    const int v[4] = {bins.w, bins.z, bins.y, bins.x}, sum = v[0] + v[1] + v[2] + v[3];
    int2 unused;
    const int before = scan(sh, make_int2(sum, 0), unused).x;
    if (need > before && need <= before + sum) {
      int at = before;
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        if (need > at && need <= at + v[k]) {
          sh.digit = bin + 3 - k;
          sh.above = at;
          sh.equal = v[k];
        }
        at += v[k];
      }
    }
  };
  auto taken = [&](int shift) {
    T |= uint32_t(sh.digit) << shift;
    need -= sh.above;
    equal = sh.equal;
  };
  constexpr int kShift[3] = {21, 10, 0}, kDigits[3] = {2047, 2047, 1023};
  uint32_t* few = reinterpret_cast<uint32_t*>(sh.count);
  if (tid == 0) sh.few_moves = 0;                     // (how many keys are in `few`)
#pragma unroll 1
  for (int pass = 0; pass < 3; ++pass) {
    const int shift = kShift[pass], top = pass ? kShift[pass - 1] : 0;
    for (int i = tid; i < kBins; i += kThreads) sh.hist[i] = 0;
    __syncthreads();
    if (C > 1) asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
    for (int c0 = lo; c0 < hi; c0 += p.keys) {
      const int c1 = min(hi, c0 + p.keys);
      load(c0, c1);
      const int from = shifted, to = c1 - c0 + shifted;        // of the keys held
      for (int i = 4 * tid; i < to; i += 4 * kThreads) {
        const uint4 four = *reinterpret_cast<const uint4*>(keys + i);
        const uint32_t k4[4] = {four.x, four.y, four.z, four.w};
#pragma unroll
        for (int j = 0; j < 4; ++j)
          if (i + j >= from && i + j < to && (pass == 0 || k4[j] >> top == T >> top))
            atomicAdd(&sh.hist[(k4[j] >> shift) & kDigits[pass]], 1);
      }
    }
    __syncthreads();
    // a cluster's counts are added up in its first block, where few bins hold anything
    if (C > 1) {
      asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");   // (the first block's bins are cleared)
      const int bin = 4 * tid;
      if (rank > 0) {
        int* sum = cluster.map_shared_rank(sh.hist, 0) + bin;
#pragma unroll
        for (int k = 0; k < 4; ++k)
          if (sh.hist[bin + k]) atomicAdd(sum + k, sh.hist[bin + k]);
      }
      cluster.sync();
    }
    take(C > 1 ? cluster.map_shared_rank(sh.hist, 0) : sh.hist);
    meet();                                           // (and the histograms are cleared next)
    taken(shift);
    if (pass == 0 && equal <= int(sizeof(sh.count) / 4)) {
      // The keys of T's first digit are few: the first block takes them and the other two digits
      // alone, which spares the cluster six meetings.
      uint32_t* all = C > 1 ? cluster.map_shared_rank(few, 0) : few;
      int* used = C > 1 ? cluster.map_shared_rank(&sh.few_moves, 0) : &sh.few_moves;
      for (int c0 = lo; c0 < hi; c0 += p.keys) {
        const int c1 = min(hi, c0 + p.keys);
        load(c0, c1);
        const int from = shifted, to = c1 - c0 + shifted;
        for (int i = 4 * tid; i < to; i += 4 * kThreads) {
          const uint4 four = *reinterpret_cast<const uint4*>(keys + i);
          const uint32_t k4[4] = {four.x, four.y, four.z, four.w};
#pragma unroll
          for (int j = 0; j < 4; ++j)
            if (i + j >= from && i + j < to && k4[j] >> shift == T >> shift) all[atomicAdd(used, 1)] = k4[j];
        }
      }
      meet();
      if (rank == 0) {
        const int n_few = equal;
#pragma unroll 1
        for (int digit = 1; digit < 3; ++digit) {
          for (int i = tid; i < kBins; i += kThreads) sh.hist[i] = 0;
          __syncthreads();
          for (int i = tid; i < n_few; i += kThreads)
            if (few[i] >> kShift[digit - 1] == T >> kShift[digit - 1])
              atomicAdd(&sh.hist[(few[i] >> kShift[digit]) & kDigits[digit]], 1);
          __syncthreads();
          take(sh.hist);
          __syncthreads();
          taken(kShift[digit]);
        }
        if (tid < C) *(C > 1 ? cluster.map_shared_rank(&sh.found, tid) : &sh.found) = make_int4(int(T), need, equal, 0);
      }
      meet();
      T = uint32_t(sh.found.x);
      need = sh.found.y;
      equal = sh.found.z;
      break;
    }
  }

  // ---- numbers of ties, holes and movers ----
  // what is before this block of the cluster, of two counts; their sums over the cluster in all
  auto before_block = [&](int which, int2 mine, int2& all) {
    all = mine;
    if (C == 1) return make_int2(0, 0);
    if (tid == 0) sh.total[which] = mine;
    cluster.sync();
    // (a block's counts a lane: one after another the 128K prompt took 59 us, not 57.5)
    const int2 x = lane < C ? *cluster.map_shared_rank(&sh.total[which], lane) : make_int2(0, 0);
    const bool before = lane < rank;
    all = make_int2(__reduce_add_sync(kFull, x.x), __reduce_add_sync(kFull, x.y));
    return make_int2(__reduce_add_sync(kFull, before ? x.x : 0), __reduce_add_sync(kFull, before ? x.y : 0));
  };
  // Counts f(slot of the n, key) -> (first, second) over the block's chunk by 32 slots, and turns the counts
  // into what is before each 32 within the chunk; the chunk's sums
  auto count = [&](int c0, int c1, auto f) {
    const int m = c1 - c0, groups = (m + 31) / 32;
    for (int i = tid; i < groups * 32; i += kThreads) {
      const int2 x = i < m ? f(c0 + i, key(c0 + i)) : make_int2(0, 0);
      const unsigned vx = __ballot_sync(kFull, x.x), vy = __ballot_sync(kFull, x.y);
      if (lane == 0) sh.count[i >> 5] = make_int2(__popc(vx), __popc(vy));
    }
    __syncthreads();
    int2 sum = make_int2(0, 0);
    for (int g0 = 0; g0 < groups; g0 += kThreads) {
      const int2 v = g0 + tid < groups ? sh.count[g0 + tid] : make_int2(0, 0);
      int2 t, at = scan(sh, v, t);
      if (g0 + tid < groups) sh.count[g0 + tid] = make_int2(sum.x + at.x, sum.y + at.y);
      sum.x += t.x;
      sum.y += t.y;
    }
    __syncthreads();
    return sum;
  };

  // With every slot of the key T kept, or none missing before, ties need no numbers.  Else the cut among
  // them is a slot: the first one of that key that goes.
  int cut = need == equal ? INT_MAX : -1;
  if (cut < 0) {
    auto tie = [&](int, uint32_t k) { return make_int2(k == T, 0); };
    int2 mine = make_int2(0, 0), all;
    for (int c0 = lo; c0 < hi; c0 += p.keys) {
      const int c1 = min(hi, c0 + p.keys);
      load(c0, c1);
      mine.x += count(c0, c1, tie).x;
    }
    int at = before_block(0, mine, all).x;
    if (tid == 0) sh.digit = INT_MAX;
    __syncthreads();
    for (int c0 = lo; c0 < hi; c0 += p.keys) {
      const int c1 = min(hi, c0 + p.keys), groups = (c1 - c0 + 31) / 32;
      load(c0, c1);
      const int2 sum = count(c0, c1, tie);
      for (int i = tid; i < groups * 32; i += kThreads) {
        const bool mark = i < c1 - c0 && key(c0 + i) == T;
        const unsigned v = __ballot_sync(kFull, mark);
        if (mark && at + sh.count[i >> 5].x + __popc(v & ((1u << lane) - 1)) == need) sh.digit = c0 + i;
      }
      at += sum.x;
      __syncthreads();
    }
    cut = sh.digit;                                   // of this block's slots
    // (blocks before the cut's keep all of theirs, blocks behind it none)
    const int here = cut != INT_MAX;
    int2 found;
    const int2 past = before_block(1, make_int2(here, 0), found);
    if (!here) cut = past.x ? lo : INT_MAX;
  }
  auto stays = [&](int i, uint32_t k) { return k > T || (k == T && i < cut); };
  auto moved = [&](int i, uint32_t k) {
    const bool keep = stays(i, k);
    return make_int2(i < p.budget && !keep, i >= p.budget && keep);
  };
  int2 mine = make_int2(0, 0), all;
  for (int c0 = lo; c0 < hi; c0 += p.keys) {
    const int c1 = min(hi, c0 + p.keys);
    load(c0, c1);
    const int2 sum = count(c0, c1, moved);
    mine.x += sum.x;
    mine.y += sum.y;
  }
  int2 at = before_block(2, mine, all);
  const int moves = all.y;
  int64_t* to = p.lists + int64_t(unit) * 2 * p.list_len;
  int64_t* from = to + p.list_len;
  const bool chunks = hi - lo > p.keys;
  for (int c0 = lo; c0 < hi; c0 += p.keys) {
    const int c1 = min(hi, c0 + p.keys), groups = (c1 - c0 + 31) / 32;
    load(c0, c1);
    int2 sum = make_int2(0, 0);
    if (chunks) sum = count(c0, c1, moved);           // (a single chunk's counts are still there)
    for (int i = tid; i < groups * 32; i += kThreads) {
      const int2 x = i < c1 - c0 ? moved(c0 + i, key(c0 + i)) : make_int2(0, 0);
      const unsigned vx = __ballot_sync(kFull, x.x), vy = __ballot_sync(kFull, x.y);
      const unsigned less = (1u << lane) - 1;
      if (x.x | x.y) {
        const int2 before = sh.count[i >> 5];
        int64_t* entry = x.x ? to + at.x + before.x + __popc(vx & less) : from + at.y + before.y + __popc(vy & less);
        *entry = place(c0 + i);
      }
    }
    at.x += sum.x;
    at.y += sum.y;
    if (chunks) __syncthreads();
  }
  meet();                                             // (orders the lists in global memory too)

  finish();

  // ---- moves ----
  const int warps = kThreads / 32 * C, warp = rank * (kThreads / 32) + (tid >> 5);
  __nv_bfloat16* pool = (lane < 16 ? p.k_cache : p.v_cache) + (lane & 15) * 8;
  int64_t src[kMoveAhead], dst[kMoveAhead];           // of the round at hand; the next one's are loaded ahead
  auto listed = [&](int i0) {
#pragma unroll
    for (int k = 0; k < kMoveAhead; ++k) {
      const int i = i0 + k * warps;
      src[k] = i < moves ? __ldcg(from + i) : -2;
      dst[k] = i < moves ? __ldcg(to + i) : -2;
    }
  };
  listed(warp);
  for (int i0 = warp; i0 < moves; i0 += warps * kMoveAhead) {
    uint4 row[kMoveAhead];
    uint32_t word[kMoveAhead];                        // lane 0: the weight, lane 1: the position
    int64_t here[kMoveAhead];
#pragma unroll
    for (int k = 0; k < kMoveAhead; ++k) {
      here[k] = dst[k];
      if (src[k] < 0 || dst[k] < 0) {
        if (lane == 0 && src[k] != -2) flag_status(p.status, LOCKS_DEV_BAD_BLOCK_ID);
        here[k] = -1;
        continue;
      }
      row[k] = *reinterpret_cast<const uint4*>(pool + src[k] * kHeadDim);
      if (lane == 0) word[k] = reinterpret_cast<const uint32_t*>(p.weights)[src[k]];
      if (lane == 1) word[k] = reinterpret_cast<const uint32_t*>(p.positions)[src[k]];
    }
    listed(i0 + warps * kMoveAhead);
#pragma unroll
    for (int k = 0; k < kMoveAhead; ++k)
      if (here[k] >= 0) {
        *reinterpret_cast<uint4*>(pool + here[k] * kHeadDim) = row[k];
        if (lane == 0) reinterpret_cast<uint32_t*>(p.weights)[here[k]] = word[k];
        if (lane == 1) reinterpret_cast<uint32_t*>(p.positions)[here[k]] = word[k];
      }
  }
}

}  // namespace

int evict_list_len(int budget, int64_t slots) { return int(budget < slots / 2 ? budget : slots / 2) + 1; }

int launch_evict(EvictParams p, cudaStream_t stream) {
  const int units = p.batch * p.n_kv_heads;
  const int64_t slots = int64_t(p.max_pages) * p.page_size;
  static LaunchOnce once;
  static std::atomic<int> fit[kMostCluster + 1];      // clusters of so many blocks that run at once, a block an SM
  constexpr int kMost = int(sizeof(Shared)) + (kMaxKeys + 4) * 4;
  static_assert(kMost <= int(kMaxSmemBlock) && kMost > int(kMaxSmemBlock) / 2, "shared memory of a block");
  if (!once.run([] {
        if (cudaFuncSetAttribute(evict_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kMost) != cudaSuccess ||
            cudaFuncSetAttribute(evict_kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1) != cudaSuccess)
          return false;
        for (int c = 1; c <= kMostCluster; ++c) {
          cudaLaunchConfig_t lc = {};
          lc.gridDim = dim3(c);
          lc.blockDim = dim3(kThreads);
          lc.dynamicSmemBytes = kMost;
          cudaLaunchAttribute attr[1];
          attr[0].id = cudaLaunchAttributeClusterDimension;
          attr[0].val.clusterDim.x = c;
          attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
          lc.attrs = attr;
          lc.numAttrs = 1;
          int n = 0;
          const bool asked = cudaOccupancyMaxActiveClusters(&n, evict_kernel, &lc) == cudaSuccess;
          if (!asked) cudaGetLastError();             // (a refusal is an answer)
          fit[c] = asked ? n : 0;
        }
        return true;
      }))
    return LOCKS_ERR_CUDA;
  const int C = evict_blocks(units, slots, fit);
  const int64_t share = (slots + C - 1) / C;
  p.keys = int(share < kMaxKeys ? (share + 31) / 32 * 32 : kMaxKeys);
  cudaLaunchConfig_t lc = {};
  lc.gridDim = dim3(unsigned(units) * C);
  lc.blockDim = dim3(kThreads);
  lc.dynamicSmemBytes = sizeof(Shared) + size_t(p.keys + 4) * 4;
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
