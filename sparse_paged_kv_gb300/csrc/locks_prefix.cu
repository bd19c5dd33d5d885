// Attention of the newest tokens of a batch whose sequences share prefixes
// (locks_prefix_decode).
//
//   out[q] = sum_{t < n_q} p_t v_t,  p = softmax_t(q^T k_t / sqrt(d)),
//
// n_q the slots that query q sees.  The softmax over a sequence splits into its
// group's shared pages and its own: each part keeps a running maximum m, a sum
// l = sum 2^(x_t - m) and an accumulator sum 2^(x_t - m) v_t, and parts are
// joined by their m.  So the shared pages are read once for the queries of the
// whole group, 256 rows (query token, head of the KV head's group) at a time.
//
// Work is a list of stages of 128 tokens: first every (group, KV head, 256 rows)
// over the group's pages, as far as the longest of its sequences sees them, then
// every (sequence, KV head) over its own.  152
// blocks, one per SM, take equal shares of the list, so that any mix of lengths
// fills the chip; a unit cut by a share's border leaves a piece in either block.
// A block's warps are: one that loads (tensor maps, a ring of five 32 KB
// tiles, K and V of a stage in turn), two whose first lanes issue the matrix
// instructions, and two groups of eight for the softmax, two warps to 32 rows:
//   S (128 x 128, tensor memory) = Q K^T    both operands in shared memory
//   P (bf16, over S's columns)   = 2^(S - m)
//   O (128 x 128, tensor memory) += P V     P from tensor memory
// A stage's product for one group runs while the other group exponentiates:
// with more than 128 rows the groups are the two halves of them, both on every
// stage; with fewer rows they take stages in turn, each with its own m, l and O
// (two parts of a piece, joined as pieces are).  The accumulator is brought to
// a new maximum only where a row's maximum grew by more than 2^8, so rarely.
// A second kernel joins the pieces of each row.
//
// 64 sequences behind a 32K prompt (32 heads on 8, 202 MB): 63 us, 3.2 TB/s with everything, memory
// busy at 4 TB/s while stages run; 256 samples of a 16K prompt (64 heads on 8, 138 GFLOP): 158 us, 875
// TFLOP/s.  A stage's chain (S, softmax, P V) bounds both, the tensor cores half busy; few rows are
// bound by memory but for the 4 us before the first key and as many behind the last.
//
// P is rounded to bf16 because V is bf16 and both operands of a matrix
// instruction have one type: each weight is off by 2^-8 of itself at most (the
// output's own rounding is as large).  The output divides by the sum of the
// rounded weights, so that a row with one dominant token keeps that token's
// value exactly; the log-sum-exp comes from the unrounded sum.
#include <climits>

#include "locks_batch.h"
#include "locks_batch.cuh"
#include "locks_kv.cuh"
#include "locks_tc.cuh"

namespace locks {

namespace {

constexpr int kSoftmaxWarps = 16;                     // two groups, two halves of the columns, four quarters of the rows
constexpr int kThreads = (kSoftmaxWarps + 4) * 32;
// (Two issuing warps.  With few rows the softmax works on the first scheduler's warps alone, so none
// of the others is there.)
constexpr int kMmaWarp = kSoftmaxWarps + 1, kProducerWarp = kSoftmaxWarps + 3;
// registers a thread after the split: 512 * 104 + 128 * 64 = 640 * 96, the launch's
constexpr int kSoftmaxRegs = 104, kOtherRegs = 64;
constexpr int kTileBytes = 128 * 256;                 // 128 rows of 128 bf16
constexpr int kHalfBytes = kTileBytes / 2;
constexpr int kRing = 5;
// Pieces handed on.  When piece n is written, the queries of piece n - 2 have had their last use in
// both groups, so each group's products with the values are issued up to its piece before that
// (n - 5 at the earliest, if every piece has one stage), and the softmax has read that piece's entry.
constexpr int kPieces = 16;
constexpr int kGroupsHeld = 64;                       // groups whose bounds a block holds
// What the list counts: a stage, one that both groups work on, and a unit's beginning and end, in
// eighths of the first.  (A pair's stage takes 1.4 to 2 times as long, more where memory does not bound
// either; of 14 settings tried these were best or within 2% in all cases: 256 samples of a 16K prompt 161
// us, with 8, 12, 6 178, with 8, 8, 6 167.)
constexpr int kCostStage = 8, kCostPair = 11, kCostUnit = 8;
constexpr uint32_t kTmemCols = 512;                   // S0 S1 O0 O1
constexpr float kLazy = 8.f;                          // log2 growth of a maximum that is left alone

// A unit's stages [s0, s0 + stages) that this block has, as the loading warp hands them to the others.
struct Piece {
  int stages;             // 0: no more pieces
  int pair;               // two tiles: a group each, both on every stage; else stages in turn
  int group_pages;        // the unit is a group's (else a sequence's own pages)
  int head, tokens, row, page0;
  int q0, nq;             // query tokens of the unit (at most two tiles)
  int s0;
};

struct Shared {
  Piece piece[kPieces];
  uint64_t piece_full[kPieces];
  uint64_t full[kRing], empty[kRing];
  uint64_t q_full[2], q_empty[2];
  uint64_t s_full[2], p_full[2], o_full[2], o_empty[2];
  uint64_t done[2];
  uint32_t tmem;
  float top[2][128];                                  // a row's new maximum, between the halves
  int lock;                                           // of the tensor cores, between the groups
  int flag[2][2][4][2];                               // what a softmax warp tells its partner
  int dead;                                           // a wait ran out: every role leaves
  int group_start[kGroupsHeld + 1], group_pages[kGroupsHeld], group_longest[kGroupsHeld];
  int bad[8];                                         // pages of a stage whose block is invalid, by stage & 7
  ListPlace place;
};
constexpr size_t kSmemBytes = size_t(kRing + 2) * kTileBytes + sizeof(Shared);
static_assert(kSmemBytes <= kMaxSmemBlock, "shared memory of a block");

// ---- the list of work -----------------------------------------------------------
__device__ __forceinline__ int clamp_int(int x, int lo, int hi) { return min(max(x, lo), hi); }

// bounds and pages of the groups, held in shared memory or (many of them) as given, and the length of each
// group's longest sequence, there or in this block's part of the workspace
struct Groups {
  const int32_t *start, *pages;
  int32_t* longest;       // INT_MAX: some sequence sees the whole prefix; 0: none found so far
  bool bounded;           // prefixes end at the longest sequence (else all are seen whole)
  bool ascending;         // else no group counts (two could claim a sequence, and the list outgrow an int)
  __device__ __forceinline__ int start_of(const PrefixParams& p, int g) const {
    return clamp_int(start[g], 0, p.batch);
  }
  __device__ __forceinline__ int pages_of(const PrefixParams& p, int g) const {
    return clamp_int(pages[g], 0, p.max_pages);
  }
  // the group of sequence b, or -1
  __device__ int of(const PrefixParams& p, int b) const {
    int lo = 0, hi = ascending ? p.n_groups : 0;      // the groups that start at or before b
    while (lo < hi) {
      const int mid = (lo + hi) >> 1;
      if (start_of(p, mid) <= b) lo = mid + 1;
      else hi = mid;
    }
    return lo > 0 && b < start_of(p, lo) ? lo - 1 : -1;
  }
};
__device__ __forceinline__ int length_of(const PrefixParams& p, int b) {
  return clamp_int(p.seq_lens[b], 0, p.max_pages * p.page_size);
}

// Entry e < n_groups: the shared pages of group e; else the own pages of sequence e - n_groups.  Its
// units: a KV head, and of a group 2 * tile_tokens query tokens.
struct Entry {
  int stages, tokens, row, page0;   // tokens; the block table's row and its first page
  int q0, nq, tiles;                // first query token (of all), how many, in how many units a head
  int cost, last_cost;              // of a unit; of a head's last one
  int group;                        // of a sequence that sees its whole prefix, else -1
  __device__ __forceinline__ int head_cost() const { return (tiles - 1) * cost + last_cost; }
};
// how many of a unit's stages begin before `cost` of it
__device__ __forceinline__ int stages_before(int cost, bool pair) {
  const int c = cost - kCostUnit;
  return c <= 0 ? 0 : pair ? (c + kCostPair - 1) / kCostPair : (c + kCostStage - 1) / kCostStage;
}

__device__ Entry load_entry(const PrefixParams& p, const Groups& groups, int e) {
  Entry n;
  if (e < p.n_groups) {
    const int a = groups.start_of(p, e), seqs = max(0, groups.start_of(p, e + 1) - a);
    n.tokens = groups.pages_of(p, e) * p.page_size;
    // (what no row of the group sees is neither read nor multiplied: it may hold anything)
    if (groups.bounded) n.tokens = min(n.tokens, groups.longest[e]);
    n.group = -1;
    n.row = a;
    n.page0 = 0;
    n.q0 = a * p.n_rows;
    n.nq = seqs * p.n_rows;
    if (n.nq == 0 || !groups.ascending) n.tokens = 0;
  } else {
    const int b = e - p.n_groups, len = length_of(p, b), g = groups.of(p, b);
    n.page0 = g >= 0 ? groups.pages_of(p, g) : 0;
    n.tokens = max(0, len - n.page0 * p.page_size);
    n.group = len < n.page0 * p.page_size ? -1 : g;
    n.row = b;
    n.q0 = b * p.n_rows;
    n.nq = p.n_rows;
  }
  n.stages = (n.tokens + kStageTok - 1) / kStageTok;
  n.tiles = int(uint64_t(uint32_t(n.nq + 2 * p.tile_tokens - 1)) * p.tile_magic >> 32);
  n.cost = n.last_cost = 0;
  if (n.stages > 0) {
    n.cost = n.stages * kCostPair + kCostUnit;
    const bool pair = n.nq - (n.tiles - 1) * 2 * p.tile_tokens > p.tile_tokens;
    n.last_cost = n.stages * (pair ? kCostPair : kCostStage) + kCostUnit;
  }
  return n;
}

// The pieces of this block's share, in the list's order.
struct Walk {
  int e, offset, left;
  Groups groups;
  Entry n;
  __device__ Walk(const PrefixParams& p, const Groups& groups, const Shared& sh, int share)
      : e(sh.place.entry), offset(sh.place.offset), left(share), groups(groups),
        n(load_entry(p, groups, e)) {}
  __device__ bool next(const PrefixParams& p, Piece& u) {
    while (left > 0) {
      const int head_cost = n.head_cost();
      if (offset >= head_cost * p.n_kv_heads) {
        offset = 0;
        if (++e >= p.n_groups + p.batch) return false;
        n = load_entry(p, groups, e);
        continue;
      }
      const int head = offset / head_cost, in_head = offset - head * head_cost;
      const int tile = n.tiles == 1 ? 0 : min(in_head / n.cost, n.tiles - 1);
      const int at = in_head - tile * n.cost, end = min(at + left, tile == n.tiles - 1 ? n.last_cost : n.cost);
      offset += end - at;
      left -= end - at;
      u.group_pages = e < p.n_groups;
      u.head = head;
      u.tokens = n.tokens;
      u.row = n.row;
      u.page0 = n.page0;
      u.q0 = n.q0 + tile * 2 * p.tile_tokens;
      u.nq = min(n.nq - tile * 2 * p.tile_tokens, 2 * p.tile_tokens);
      u.pair = u.nq > p.tile_tokens;
      u.s0 = stages_before(at, u.pair);
      u.stages = stages_before(end, u.pair) - u.s0;
      if (u.stages > 0) return true;
    }
    return false;
  }
};

// ---- the softmax warps ------------------------------------------------------------
// Warp (w, h, quarter): 32 rows of group w's tile, columns 64 h .. 64 h + 63 of S and of O, so that a
// row's exponentials are shared by two warps, and four warps are on a scheduler to hide one
// another's latency.  The two tell each other once a stage whether the row's maximum has to move.
__device__ void softmax_role(const PrefixParams& p, Shared& sh, unsigned char* ring, int w, int h) {
  const int tid = threadIdx.x & 127, lane = tid & 31, quarter = tid >> 5;
  const uint32_t base = sh.tmem + (uint32_t(quarter * 32) << 16) + w * 128;
  const uint32_t t_s = base + 64 * h, t_o = t_s + 256;
  const int rt = tid / p.group;
  uint32_t jobs = 0, units = 0;                       // of this group
  int stage0 = 0;

  auto pair_sync = [&]() { asm volatile("bar.sync %0, 64;" ::"r"(1 + w * 4 + quarter) : "memory"); };
  // The partners meet: what the other one says.  A warp that leaves says so at the meeting that the
  // other is at or comes to next; every way out of here has exactly one such last meeting.
  constexpr int kLeft = 2;
  volatile int* mine = sh.flag[w][h][quarter];
  volatile int* theirs = sh.flag[w][h ^ 1][quarter];
  auto meet = [&](int say) {
    if (lane == 0) mine[jobs & 1] = say;
    pair_sync();
    return theirs[jobs & 1];
  };

  // columns that the row does not see, or of pages whose block is invalid (col0: of the stage)
  auto mask_scores = [&](float* s, int seen, int bad, int col0) {
#pragma unroll
    for (int k = 0; k < 64; ++k) s[k] = k < seen ? s[k] : -INFINITY;
    if (bad) {
#pragma unroll
      for (int k = 0; k < 64; ++k)
        if (bad >> ((col0 + k) >> p.page_shift) & 1) s[k] = -INFINITY;
    }
  };

  for (int n = 0;; ++n) {
    if (!warp_wait_or_dead(&sh.piece_full[n % kPieces], (n / kPieces) & 1, &sh.dead)) break;
    const Piece u = sh.piece[n % kPieces];
    if (u.stages == 0) break;
    const int first = u.pair ? 0 : (stage0 ^ w) & 1, step = u.pair ? 1 : 2;
    if (first < u.stages) {
      const int tq = (u.pair ? w * p.tile_tokens : 0) + rt;
      const bool valid = rt < p.tile_tokens && tq < u.nq;
      int lim = 1 << 30;                              // tokens of the unit that this row sees
      const int qt = u.q0 + tq;                       // query token among the batch's
      if (valid) {
        if (u.group_pages) {
          const int b = p.n_rows == 1 ? qt : qt / p.n_rows;
          lim = length_of(p, b) - p.n_rows + (qt - b * p.n_rows) + 1;
        } else {
          lim = u.tokens - p.n_rows + tq + 1;
        }
        lim = clamp_int(lim, 0, u.tokens);
      }
      const bool any = __any_sync(kFull, valid);
      float m = -INFINITY, l = 0.f, lr = 0.f;
      bool ok = true;
      for (int i = first; i < u.stages; i += step) {
        const int tok = (u.s0 + i) * kStageTok, nv = min(kStageTok, u.tokens - tok);
        ok = warp_wait_or_dead(&sh.s_full[w], jobs & 1, &sh.dead);
        if (!ok) break;
        tc_fence_after();
        const int bad = *static_cast<volatile int*>(&sh.bad[(stage0 + i) & 7]);
        if (any) {
          const int seen = lim - tok - 64 * h;
          const bool masked = __any_sync(kFull, seen < 64) || bad;
          float s[64], x0 = -INFINITY, x1 = -INFINITY;
          tmem_ld32(t_s, s);
          tmem_ld32(t_s + 32, s + 32);
          tmem_wait_ld();
          if (masked) mask_scores(s, seen, bad, 64 * h);
#pragma unroll
          for (int k = 0; k < 64; k += 4) {
            x0 = fmaxf(fmaxf(x0, s[k]), s[k + 1]);
            x1 = fmaxf(fmaxf(x1, s[k + 2]), s[k + 3]);
          }
          const float top = fmaxf(x0, x1) * p.scale_log2;
          // (rows past the unit's last hold whatever the tile held, and decide nothing)
          const int need = __any_sync(kFull, valid && top > m + kLazy);
          const int other = meet(need);
          if (other == kLeft) return;                 // (that was the last meeting)
          if (need | other) {
            // both halves' maximum, by way of the second one's
            float mn;
            if (h == 1) sh.top[w][tid] = top;
            pair_sync();
            if (h == 0) {
              mn = fmaxf(m, fmaxf(top, sh.top[w][tid]));
              sh.top[w][tid] = mn;
            }
            pair_sync();
            if (h == 1) mn = sh.top[w][tid];
            const float f = m == -INFINITY ? 0.f : ex2_approx(m - mn);
            m = mn;
            l *= f;
            lr *= f;
            if (i != first) {                         // (the first product overwrites O)
#pragma unroll 1
              for (int c = 0; c < 64; c += 16) {
                float o[16];
                tmem_ld16(t_o + c, o);
                tmem_wait_ld();
#pragma unroll
                for (int k = 0; k < 16; ++k) o[k] *= f;
                tmem_st16(t_o + c, reinterpret_cast<uint32_t*>(o));
              }
            }
          }
          const float mu = m == -INFINITY ? 0.f : m;
          const float2 sc = make_float2(p.scale_log2, p.scale_log2), off = make_float2(-mu, -mu);
          float2 a0 = make_float2(0.f, 0.f), a1 = a0;
#pragma unroll
          for (int c = 0; c < 64; c += 32) {
            uint32_t pk[16];
#pragma unroll
            for (int k = 0; k < 16; ++k) {
              float2 x = ffma2(make_float2(s[c + 2 * k], s[c + 2 * k + 1]), sc, off);
              x.x = ex2_approx(x.x);
              x.y = ex2_approx(x.y);
              const __nv_bfloat162 r = __floats2bfloat162_rn(x.x, x.y);
              pk[k] = *reinterpret_cast<const uint32_t*>(&r);
              a0 = fadd2(a0, x);
              a1 = fadd2(a1, make_float2(bf16_lo(pk[k]), bf16_hi(pk[k])));
            }
            tmem_st16(t_s + c / 2, pk);
          }
          l += a0.x + a0.y;
          lr += a1.x + a1.y;
          tmem_wait_st();
        }
        ++jobs;
        if (nv < kStageTok || bad) {
          // rows of V that no query sees (behind the unit's end, or of an invalid page) may hold
          // anything, NaN included, which a weight of 0 would not keep out
          const int c = 2 * (stage0 + i) + 1, slot = c % kRing;
          ok = warp_wait_or_dead(&sh.full[slot], (c / kRing) & 1, &sh.dead);
          if (!ok) break;
          if (tid >= nv || (bad >> (tid >> p.page_shift) & 1)) {
            uint4* row = reinterpret_cast<uint4*>(ring + slot * kTileBytes + h * kHalfBytes + tid * 128);
#pragma unroll
            for (int k = 0; k < 8; ++k) row[k] = make_uint4(0, 0, 0, 0);
          }
          proxy_fence_smem();
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&sh.p_full[w]);
      }
      // this group's part of the piece
      if (!ok || !warp_wait_or_dead(&sh.o_full[w], units & 1, &sh.dead)) break;
      ++units;
      tc_fence_after();
      if (any) {
        const int part = u.pair ? 0 : first;          // (of the piece's stages, in turn)
        // the first piece of a unit by the row, one continued from the block before by the block
        const int64_t row = (int64_t(u.head) * p.batch * p.n_rows + u.q0 + (u.pair ? w * p.tile_tokens : 0)) *
                                p.group + tid;
        const int64_t at = u.s0 == 0 ? ((u.group_pages ? 0 : 2) + part) * p.rows + row
                                     : 4 * p.rows + int64_t(blockIdx.x) * 256 + (u.pair ? w : part) * 128 + tid;
        if (valid) p.sums[2 * at + h] = make_float4(m, l, lr, 0.f);
        float4* acc = p.acc + (16 * h) * p.parts + at;
#pragma unroll 1
        for (int c = 0; c < 64; c += 32) {
          float o[32];
          tmem_ld32(t_o + c, o);
          tmem_wait_ld();
          if (valid) {
#pragma unroll
            for (int k = 0; k < 32; k += 4)
              acc[(c + k) / 4 * p.parts] = make_float4(o[k], o[k + 1], o[k + 2], o[k + 3]);
          }
        }
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&sh.o_empty[w]);
    }
    stage0 += u.stages;
  }
  meet(kLeft);
}

// ---- the loading warp -------------------------------------------------------------
__device__ void load_role(const PrefixParams& p, const Groups& groups, Shared& sh, unsigned char* qtile,
                          unsigned char* ring, const CUtensorMap* map_qg, const CUtensorMap* map_qo,
                          const CUtensorMap* map_k, const CUtensorMap* map_v, int share) {
  const int lane = threadIdx.x & 31;
  const int per_stage = kStageTok >> p.page_shift;
  Walk walk(p, groups, sh, share);
  Piece u;
  int qn = 0, stage = 0, piece = 0;
  bool ok = true;
  for (; ok && walk.next(p, u); ++piece) {
    const int32_t* table = p.block_table + int64_t(u.row) * p.max_pages + u.page0;
    auto page_of = [&](int s) {                       // lane i has the stage's page i: its block
      const int page = s * per_stage + lane;
      return lane < per_stage && page << p.page_shift < u.tokens ? table[page] : INT_MIN;
    };
    int next = page_of(u.s0);
    const int box_tokens = u.group_pages ? p.tile_tokens : min(p.n_rows, p.tile_tokens);
    const CUtensorMap* map_q = u.group_pages ? map_qg : map_qo;
    for (int t = 0; ok && t < (u.pair ? 2 : 1); ++t, ++qn) {
      const int slot = qn & 1;
      ok = warp_wait_or_dead(&sh.q_empty[slot], ((qn >> 1) & 1) ^ 1, &sh.dead);
      if (ok && lane == 0) {
        if (t == 0) {
          sh.piece[piece % kPieces] = u;
          mbar_arrive(&sh.piece_full[piece % kPieces]);
        }
        mbar_arrive_expect_tx(&sh.q_full[slot], box_tokens * p.group * 256);
        unsigned char* dst = qtile + slot * kTileBytes;
        tma_load3(dst, map_q, 0, u.head * p.group, u.q0 + t * p.tile_tokens, &sh.q_full[slot]);
        tma_load3(dst + kHalfBytes, map_q, 64, u.head * p.group, u.q0 + t * p.tile_tokens,
                  &sh.q_full[slot]);
      }
    }
    for (int s = u.s0; ok && s < u.s0 + u.stages; ++s, ++stage) {
      const int block = next;
      if (s + 1 < u.s0 + u.stages) next = page_of(s + 1);
      bool want = block != INT_MIN;
      const bool there = block >= 0 && block < p.num_blocks;
      if (want && !there) flag_status(p.status, LOCKS_DEV_BAD_BLOCK_ID);
      const int bad = __ballot_sync(kFull, want && !there);
      want = want && there;
      const int n = __popc(__ballot_sync(kFull, want));
      const int z = block * p.n_kv_heads + u.head;
#pragma unroll
      for (int kv = 0; kv < 2; ++kv) {
        const int c = 2 * stage + kv, slot = c % kRing;
        ok = ok && warp_wait_or_dead(&sh.empty[slot], ((c / kRing) & 1) ^ 1, &sh.dead);
        if (!ok) break;
        if (lane == 0) {
          if (kv == 0) *static_cast<volatile int*>(&sh.bad[stage & 7]) = bad;
          mbar_arrive_expect_tx(&sh.full[slot], (n << p.page_shift) * 256);
        }
        __syncwarp();
        if (want) {
          unsigned char* dst = ring + slot * kTileBytes + (lane << p.page_shift) * 128;
          const CUtensorMap* map = kv ? map_v : map_k;
          tma_load3(dst, map, 0, 0, z, &sh.full[slot]);
          tma_load3(dst + kHalfBytes, map, 64, 0, z, &sh.full[slot]);
        }
      }
    }
  }
  if (ok && lane == 0) {
    sh.piece[piece % kPieces].stages = 0;
    mbar_arrive(&sh.piece_full[piece % kPieces]);
  }
  // no block leaves while copies into its memory are in flight: after a wait that ran out, each
  // slot's last copy is waited for once more
  if (!ok) {
    for (int c = max(0, 2 * stage - kRing); c < 2 * stage; ++c)
      mbar_wait_bounded(&sh.full[c % kRing], (c / kRing) & 1);
    for (int t = max(0, qn - 2); t < qn; ++t)
      mbar_wait_bounded(&sh.q_full[t & 1], (t >> 1) & 1);
  }
}

// ---- the issuing threads ------------------------------------------------------------
// One a softmax group w: its latency, one instruction after another, is as long as the products, so a
// single one for both groups would bound the kernel.  Each goes S, (softmax), O += P V, next S; the
// products of the two meet in the tensor cores' queue.  A wait tells phases apart by one bit, so
// whoever waits for a phase has to know that the one before is over: each thread waits for every
// tile and every piece's queries, also for those that only the other group uses, and each tile is
// free when both have been there.
__device__ void issue_role(Shared& sh, unsigned char* qtile, unsigned char* ring, int w) {
  constexpr uint32_t kIdescS = mma_idesc(128, 128, false), kIdescO = mma_idesc(128, 128, true);
  const uint32_t t_s = sh.tmem + w * 128, t_o = t_s + 256;
  const uint32_t q_desc = smem_desc_lo(smem_u32(qtile), 16);
  const uint32_t k_desc = smem_desc_lo(smem_u32(ring), 16);
  // 64 columns of V (a half) follow each other at kHalfBytes, 8 tokens at 1024 bytes
  const uint32_t v_desc = smem_desc_lo(smem_u32(ring), kHalfBytes);
  uint32_t jobs = 0, units = 0;                       // of this group
  int stage0 = 0, tile0 = 0;
  bool ok = true;
  for (int n = 0; ok; ++n) {
    if (!mbar_wait_or_dead(&sh.piece_full[n % kPieces], (n / kPieces) & 1, &sh.dead)) break;
    const int stages = sh.piece[n % kPieces].stages, pair = sh.piece[n % kPieces].pair;
    if (stages == 0) break;
    const int first = pair ? 0 : (stage0 ^ w) & 1, step = 2 - pair;
    const uint32_t t = tile0 + (w & pair), qs = t & 1;
    const uint32_t da = q_desc + qs * (kTileBytes >> 4);
    if (first >= stages) {
      ok = mbar_wait_or_dead(&sh.q_full[qs], t >> 1 & 1, &sh.dead);
      if (ok) mbar_arrive(&sh.q_empty[qs]);
    }
    bool scored = false;                              // S of stage i is issued
    for (int i = 0; ok && i < stages; ++i) {
      const uint32_t c = 2 * (stage0 + i), ks = c % kRing, kp = c / kRing & 1;
      const uint32_t vs = (c + 1) % kRing, vp = (c + 1) / kRing & 1;
      if (!pair && ((stage0 + i) ^ w) & 1) {          // the other group's stage
        ok = mbar_wait_or_dead(&sh.full[ks], kp, &sh.dead);
        if (!ok) break;
        mbar_arrive(&sh.empty[ks]);
        ok = mbar_wait_or_dead(&sh.full[vs], vp, &sh.dead);
        if (!ok) break;
        mbar_arrive(&sh.empty[vs]);
        continue;
      }
      // (a pair's query tiles are used by one group each, which gives both arrivals)
      auto scores = [&](uint32_t slot, bool last) {
        mma_ss_128(t_s, da, k_desc + slot * (kTileBytes >> 4), kIdescS);
        mma_commit(&sh.s_full[w]);
        mma_commit(&sh.empty[slot]);
        if (last) {
          mma_commit(&sh.q_empty[qs]);
          if (pair) mma_commit(&sh.q_empty[qs]);
        }
      };
      const bool last = i + step >= stages;
      if (!scored) {
        ok = (i != first || mbar_wait_or_dead(&sh.q_full[qs], t >> 1 & 1, &sh.dead)) &&
             mbar_wait_or_dead(&sh.full[ks], kp, &sh.dead);
        if (!ok) break;
        scores(ks, last);
      }
      ok = mbar_wait_or_dead(&sh.full[vs], vp, &sh.dead) &&
           (i != first || mbar_wait_or_dead(&sh.o_empty[w], (units & 1) ^ 1, &sh.dead));
      if (!ok) break;
      const uint32_t ns = (c + 2) % kRing;
      scored = pair && !last && mbar_try_wait(&sh.full[ns], (c + 2) / kRing & 1);
      // With both groups on every stage, P V and the next S go to the tensor cores as one block: two
      // groups in step would wait for their products together and then crowd the schedulers together
      // (a stage took 4000 cycles); one block after the other, each group's exponentials meet the other's
      // products.  The lock is taken before the wait for P, so that nothing is left to do after it;
      // it is a courtesy: after a while the block goes without it.
      if (scored)
        for (int tries = 0; tries < 64 && atomicCAS_block(&sh.lock, 0, 1); ++tries) {}
      ok = mbar_wait_or_dead(&sh.p_full[w], jobs & 1, &sh.dead);
      if (!ok) break;
      ++jobs;
      tc_fence_after();
      mma_ts_128(t_o, t_s, v_desc + vs * (kTileBytes >> 4), kIdescO, i != first);
      mma_commit(&sh.empty[vs]);
      if (last) {
        mma_commit(&sh.o_full[w]);
        ++units;
      }
      if (scored) {
        scores(ns, i + 2 >= stages);
        atomicExch_block(&sh.lock, 0);
      }
    }
    stage0 += stages;
    tile0 += 1 + pair;
  }
  // everything issued is done before the block frees its tensor memory
  mma_commit(&sh.done[w]);
  mbar_wait_bounded(&sh.done[w], 0);
}

__global__ void __launch_bounds__(kThreads, 1)
    prefix_kernel(const PrefixParams p, const __grid_constant__ CUtensorMap map_qg,
                  const __grid_constant__ CUtensorMap map_qo,
                  const __grid_constant__ CUtensorMap map_k,
                  const __grid_constant__ CUtensorMap map_v) {
  extern __shared__ __align__(1024) unsigned char smem[];
  unsigned char* qtile = smem;
  unsigned char* ring = smem + 2 * kTileBytes;
  Shared& sh = *reinterpret_cast<Shared*>(smem + (kRing + 2) * kTileBytes);
  const int tid = threadIdx.x, warp = tid >> 5;

  if (warp == kMmaWarp) tmem_alloc(&sh.tmem, kTmemCols);
  if (tid == 0) {
    for (int i = 0; i < kRing; ++i) {
      mbar_init(&sh.full[i], 1);
      mbar_init(&sh.empty[i], 2);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&sh.q_full[i], 1);
      mbar_init(&sh.q_empty[i], 2);
      mbar_init(&sh.s_full[i], 1);
      mbar_init(&sh.p_full[i], 8);
      mbar_init(&sh.o_full[i], 1);
      mbar_init(&sh.o_empty[i], 8);
      mbar_init(&sh.done[i], 1);
    }
    for (int i = 0; i < kPieces; ++i) mbar_init(&sh.piece_full[i], 1);
    mbar_fence_init();
    sh.dead = sh.lock = 0;
    prefetch_map(&map_qg);
    prefetch_map(&map_qo);
    prefetch_map(&map_k);
    prefetch_map(&map_v);
  }
  // what follows reads memory that the kernel before this one may write
  griddep_wait();
  const bool held = p.n_groups <= kGroupsHeld;
  Groups groups = {p.group_starts, p.prefix_pages,
                   held ? sh.group_longest : p.longest + int64_t(blockIdx.x) * p.n_groups, false, true};
  if (tid < p.batch) asm volatile("prefetch.global.L1 [%0];" ::"l"(p.seq_lens + tid));
  bool out_of_order = false;
  for (int i = tid; i < p.n_groups; i += kThreads) {
    const int a = p.group_starts[i], z = p.group_starts[i + 1];
    out_of_order |= a < 0 || z < a || z > p.batch;
    groups.longest[i] = 0;
    if (held) {
      sh.group_start[i] = a;
      sh.group_pages[i] = p.prefix_pages[i];
      if (i == p.n_groups - 1) sh.group_start[i + 1] = z;
    }
  }
  if (held) {
    groups.start = sh.group_start;
    groups.pages = sh.group_pages;
  }
  groups.ascending = !__syncthreads_or(out_of_order);
  tc_fence_before();
  const int entries = p.n_groups + p.batch;
  int total, share;
  for (;;) {
    bool unseen = false;
    share = locate<kThreads>(
        [&](int e) {
          const Entry n = load_entry(p, groups, e);
          if (n.group >= 0) groups.longest[n.group] = INT_MAX;
          return n.head_cost() * p.n_kv_heads;
        },
        entries, blockIdx.x, kCostStage, kBatchSms, sh.place, total,
        [&](int e, int first) {
          // (called once every thread's entries have been asked for their stages)
          if (e < p.n_groups && groups.longest[e] == 0) unseen |= load_entry(p, groups, e).tokens > 0;
          if (blockIdx.x) return;
          // for the kernel that joins the pieces; and the arguments' check
          const Entry n = load_entry(p, groups, e);
          if (e >= p.n_groups) {
            const int t = p.seq_lens[e - p.n_groups];
            p.entry_info[e] = make_int4(first, n.stages, groups.of(p, e - p.n_groups), 0);
            if (t < 0 || t > p.max_pages * p.page_size) flag_status(p.status, LOCKS_DEV_BAD_SEQ_LEN);
          } else {
            p.entry_info[e] = make_int4(first, n.stages, n.q0, n.nq);
            if (!groups.ascending || groups.pages[e] < 0 || groups.pages[e] > p.max_pages)
              flag_status(p.status, LOCKS_DEV_BAD_GROUP);
          }
        });
    if (groups.bounded || !__syncthreads_or(unseen)) break;
    // Some prefix is seen whole by none of its sequences (only then is this worth 0.3 us): the longest of
    // each group, a sequence a thread, and the list once more.  A warp in one group adds one number.
    groups.bounded = true;
    for (int b0 = tid & ~31; b0 < p.batch; b0 += kThreads) {
      const int b = b0 + (tid & 31), g = b < p.batch ? groups.of(p, b) : -1;
      const int len = g >= 0 ? length_of(p, b) : 0;
      if (__all_sync(kFull, g == __shfl_sync(kFull, g, 0))) {
        const int most = __reduce_max_sync(kFull, len);
        if (g >= 0 && (tid & 31) == 0) atomicMax(groups.longest + g, most);
      } else if (g >= 0) {
        atomicMax(groups.longest + g, len);
      }
    }
    __syncthreads();
  }
  if (blockIdx.x == 0 && tid == 0) p.entry_info[entries] = make_int4(total, 0, 0, 0);
  tc_fence_after();
  griddep_launch();

  if (share > 0) {
    if (warp < kSoftmaxWarps) {
      asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kSoftmaxRegs));
      softmax_role(p, sh, ring, warp >> 3, warp >> 2 & 1);
    } else {
      asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kOtherRegs));
      if (warp == kProducerWarp) load_role(p, groups, sh, qtile, ring, &map_qg, &map_qo, &map_k, &map_v, share);
      else if (warp >= kMmaWarp && elect_one()) issue_role(sh, qtile, ring, warp - kMmaWarp);
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (tid == 0 && sh.dead) flag_status(p.status, LOCKS_DEV_WAIT_TIMEOUT);
  if (warp == kMmaWarp) tmem_free(sh.tmem, kTmemCols);
}

// ---- joining the pieces ---------------------------------------------------------------
// A block has RB rows (of [KV head][query token][head of the group], as the parts lie).  First a thread
// per row and kind (the group's pages, the sequence's own) finds the unit's place in the list, from which
// it follows where the row's parts are (a piece, for either softmax group): all threads write that down,
// kListed pieces a unit at a time.  Then thread = (row, chunks of 4 dims): neighbouring threads have
// neighbouring rows, whose parts lie side by side.  With fewer than 8 rows the threads left over split
// the parts, and are joined in shared memory.
// (Few loads ahead and four blocks an SM: with twice the loads and two blocks 16384 rows took 18 us, not 14.)
constexpr int kJoinThreads = 256, kListed = 32;

struct UnitParts {
  int first, end, c0, pieces;                         // its place in the list; blocks from c0 on
  int pair;
  int64_t base, carry;                                // the row's index in a first part; in block 0's

  // how many parts a piece may have, and where the row is in part `which` of piece i (-1: it has none)
  __device__ __forceinline__ int each() const { return pair ? 1 : 2; }
  __device__ __forceinline__ int64_t part(int i, int which, const Split& split, int64_t rows) const {
    const int c = c0 + i;
    const int s0 = stages_before(max(first, split.begin(c)) - first, pair);
    const int s1 = stages_before(min(end, split.begin(c + 1)) - first, pair);
    if (s1 - s0 <= which) return -1;
    return s0 == 0 ? base + which * rows : carry + int64_t(c) * 256 + which * 128;
  }
};

template <int RB>
__global__ void __launch_bounds__(kJoinThreads, 4) join_kernel(const PrefixParams p) {
  constexpr int kChunkThreads = RB >= 8 ? kJoinThreads / RB : 32, kChunks = 32 / kChunkThreads;
  constexpr int kSplits = kJoinThreads / (RB * kChunkThreads);
  __shared__ UnitParts s_unit[2 * RB];
  __shared__ int s_part[2 * RB][2 * kListed];         // (parts are fewer than 2^31)
  __shared__ int s_most;                              // pieces of the block's unit that has most
  const int tid = threadIdx.x;
  const int64_t row0 = int64_t(blockIdx.x) * RB;
  const int qts = p.batch * p.n_rows;
  if (tid == 0) s_most = 0;
  __syncthreads();
  griddep_wait();
  const Split split(p.entry_info[p.n_groups + p.batch].x, kCostStage, kBatchSms);
  if (tid < 2 * RB) {
    const int64_t row = row0 + (tid >> 1);
    const int kind = tid & 1;
    UnitParts u = {};
    if (row < p.rows) {
      const int item = int(row) / p.group, head = item / qts, qt = item - head * qts;   // (rows < 2^31)
      const int b = p.n_rows == 1 ? qt : qt / p.n_rows;
      // (place in the list, stages, then of a group: first query token and how many; of a sequence: its group)
      int4 info = p.entry_info[p.n_groups + b];
      int q0 = b * p.n_rows, nq = p.n_rows;
      if (kind == 0) {
        if (info.z >= 0) info = p.entry_info[info.z];
        else info.y = 0;
        q0 = info.z;
        nq = info.w;
      }
      if (info.y > 0) {
        const int step = 2 * p.tile_tokens;
        const int tiles = int(uint64_t(uint32_t(nq + step - 1)) * p.tile_magic >> 32);
        const int tq = qt - q0, tile = int(uint64_t(uint32_t(tq)) * p.tile_magic >> 32);
        const int in = tq - tile * step, w = in >= p.tile_tokens;
        const bool last_pair = nq - (tiles - 1) * step > p.tile_tokens;
        const int cost = info.y * kCostPair + kCostUnit;
        const int last_cost = info.y * (last_pair ? kCostPair : kCostStage) + kCostUnit;
        u.pair = nq - tile * step > p.tile_tokens;
        u.first = info.x + head * ((tiles - 1) * cost + last_cost) + tile * cost;
        u.end = u.first + (tile == tiles - 1 ? last_cost : cost);
        u.c0 = split.block_of(u.first);
        u.pieces = split.block_of(u.end - 1) - u.c0 + 1;
        u.base = 2 * kind * p.rows + row;
        u.carry = 4 * p.rows + (u.pair ? w * 128 : 0) + (in - w * p.tile_tokens) * p.group + int(row) - item * p.group;
      }
    }
    s_unit[tid] = u;
    if (u.pieces) atomicMax(&s_most, u.pieces);
  }
  __syncthreads();

  const int r = tid % RB, chunk0 = tid / RB % kChunkThreads * kChunks, sub = tid / (RB * kChunkThreads);
  const int64_t row = row0 + r;
  float M = -INFINITY, L = 0.f, LR = 0.f;
  float4 A[kChunks];
#pragma unroll
  for (int c = 0; c < kChunks; ++c) A[c] = make_float4(0.f, 0.f, 0.f, 0.f);
  auto add = [&](float4 s, const float4* a) {
    // (a part in which the row sees nothing has no sum, and an accumulator of no account)
    if (s.y == 0.f) return;
    const float mn = fmaxf(M, s.x);
    const float f = M == -INFINITY ? 0.f : ex2_approx(M - mn), h = ex2_approx(s.x - mn);
#pragma unroll
    for (int c = 0; c < kChunks; ++c) {
      A[c].x = A[c].x * f + a[c].x * h;
      A[c].y = A[c].y * f + a[c].y * h;
      A[c].z = A[c].z * f + a[c].z * h;
      A[c].w = A[c].w * f + a[c].w * h;
    }
    L = L * f + s.y * h;
    LR = LR * f + s.z * h;
    M = mn;
  };
  const int most = s_most, each0 = s_unit[2 * r].each(), each1 = s_unit[2 * r + 1].each();
  for (int i0 = 0; i0 < most; i0 += kListed) {
    if (i0) __syncthreads();
    const int round = min(kListed, most - i0);
    for (int j = tid; j < 2 * RB * round; j += kJoinThreads) {
      const int unit = j % (2 * RB), i = j / (2 * RB);
      const UnitParts& u = s_unit[unit];
      for (int which = 0; which < u.each(); ++which)
        s_part[unit][i * u.each() + which] =
            i0 + i < u.pieces ? int(u.part(i0 + i, which, split, p.rows)) : -1;
    }
    __syncthreads();
    const int n0 = each0 * round, n = n0 + each1 * round;
    constexpr int kAhead = kChunks > 1 ? 1 : 3;
    for (int t0 = sub; t0 < n; t0 += kSplits * kAhead) {
      float4 s[kAhead], z[kAhead], a[kAhead][kChunks];
#pragma unroll
      for (int k = 0; k < kAhead; ++k) {
        const int t = t0 + k * kSplits;
        s[k].y = z[k].y = 0.f;
        const int at = t >= n ? -1 : t < n0 ? s_part[2 * r][t] : s_part[2 * r + 1][t - n0];
        if (at >= 0) {
          s[k] = p.sums[2 * int64_t(at)];             // (l and the rounded l of the two halves of the
          z[k] = p.sums[2 * int64_t(at) + 1];         // columns, which share m)
#pragma unroll
          for (int c = 0; c < kChunks; ++c) a[k][c] = p.acc[(chunk0 + c) * p.parts + at];
        }
      }
#pragma unroll
      for (int k = 0; k < kAhead; ++k) {
        s[k].y += z[k].y;
        s[k].z += z[k].z;
        add(s[k], a[k]);
      }
    }
  }
  if constexpr (kSplits > 1) {
    __shared__ float4 s_acc[kJoinThreads], s_sum[kJoinThreads];
    s_acc[tid] = A[0];
    s_sum[tid] = make_float4(M, L, LR, 0.f);
    __syncthreads();
    if (sub == 0)
      for (int k = 1; k < kSplits; ++k) add(s_sum[tid + k * RB * kChunkThreads], &s_acc[tid + k * RB * kChunkThreads]);
  }
  if (sub != 0 || row >= p.rows) return;
  const int g = int(row) % p.group, item = int(row) / p.group, head = item / qts, qt = item - head * qts;
  const int64_t out = int64_t(qt) * (p.n_kv_heads * p.group) + head * p.group + g;
  const float inv = LR == 0.f ? 0.f : 1.f / LR;
  uint2 ow[kChunks];
#pragma unroll
  for (int c = 0; c < kChunks; ++c) {
    const __nv_bfloat162 o01 = __floats2bfloat162_rn(A[c].x * inv, A[c].y * inv);
    const __nv_bfloat162 o23 = __floats2bfloat162_rn(A[c].z * inv, A[c].w * inv);
    ow[c].x = *reinterpret_cast<const uint32_t*>(&o01);
    ow[c].y = *reinterpret_cast<const uint32_t*>(&o23);
  }
  __nv_bfloat16* o = p.out + out * kHeadDim + 4 * chunk0;
  if constexpr (kChunks >= 2) {
#pragma unroll
    for (int c = 0; c < kChunks; c += 2)
      *reinterpret_cast<uint4*>(o + 4 * c) = make_uint4(ow[c].x, ow[c].y, ow[c + 1].x, ow[c + 1].y);
  } else {
    *reinterpret_cast<uint2*>(o) = ow[0];
  }
  if (chunk0 == 0 && p.out_lse) p.out_lse[out] = L == 0.f ? -INFINITY : kLn2 * (M + log2f(L));
}

template <int RB>
int launch_join(const PrefixParams& p, cudaStream_t stream) {
  return launch_dependent(join_kernel<RB>, dim3(unsigned((p.rows + RB - 1) / RB)), kJoinThreads, 0, p, stream);
}

}  // namespace

PrefixLayout prefix_layout(int64_t rows, int64_t batch, int64_t groups) {
  PrefixLayout L;
  const auto up = [](size_t x) { return (x + 255) / 256 * 256; };
  const size_t parts = size_t(4) * rows + size_t(kBatchSms) * 256;
  L.parts = int64_t(parts);
  L.acc = 0;
  L.sums = up(L.acc + parts * kHeadDim * sizeof(float));
  L.entry_info = up(L.sums + 2 * parts * sizeof(float4));
  L.longest = up(L.entry_info + size_t(groups + batch + 1) * sizeof(int4));
  L.total = L.longest + (groups > kGroupsHeld ? up(size_t(kBatchSms) * groups * sizeof(int32_t)) : 0);
  return L;
}

int launch_prefix(const PrefixParams& p, const CUtensorMap& q_group, const CUtensorMap& q_own,
                  const CUtensorMap& k, const CUtensorMap& v, cudaStream_t stream) {
  static LaunchOnce once;
  if (!once.run([] {
        return cudaFuncSetAttribute(prefix_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                    int(kSmemBytes)) == cudaSuccess;
      }))
    return LOCKS_ERR_CUDA;
  cudaLaunchConfig_t lc = {};
  lc.gridDim = dim3(kBatchSms);
  lc.blockDim = dim3(kThreads);
  lc.dynamicSmemBytes = kSmemBytes;
  lc.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  lc.attrs = attr;
  lc.numAttrs = 1;
  if (cudaLaunchKernelEx(&lc, prefix_kernel, p, q_group, q_own, k, v) != cudaSuccess)
    return LOCKS_ERR_CUDA;
  // Rows a block: 32 (parts are read 512 bytes at a time) where that leaves two blocks an SM, or 4 (2048
  // rows of 16 parts: 11 us, with 8 rows 17 us, with 2 15 us);
  // a few rows of a long sequence have up to 600 parts each, which four threads split.
  if (p.rows >= 32 * 2 * kBatchSms) return launch_join<32>(p, stream);
  if (p.rows >= 8 * kBatchSms) return launch_join<4>(p, stream);
  return launch_join<2>(p, stream);
}

}  // namespace locks
