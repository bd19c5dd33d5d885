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
// over the group's pages, then every (sequence, KV head) over its own.  152
// blocks, one per SM, take equal shares of the list, so that any mix of lengths
// fills the chip; a unit cut by a share's border leaves a piece in either block.
// A block's warps are: one that loads (tensor maps, a ring of five 32 KB
// tiles, K and V of a stage in turn), one that issues the matrix
// instructions, and two groups of four for the softmax, thread = query row:
//   S (128 x 128, tensor memory) = Q K^T    both operands in shared memory
//   P (bf16, over S's columns)   = 2^(S - m)
//   O (128 x 128, tensor memory) += P V     P from tensor memory
// A stage's product for one group runs while the other group exponentiates:
// with more than 128 rows the groups are the two halves of them, both on every
// stage; with fewer rows they take stages in turn, each with its own m, l and O
// (two halves of a piece, joined as pieces are).  The accumulator is brought to
// a new maximum only where a row's maximum grew by more than 2^8, so rarely.
// A second kernel joins the pieces of each row.
//
// P is rounded to bf16 because V is bf16 and both operands of a matrix
// instruction have one type: each weight is off by 2^-9 of itself at most (the
// output's own rounding is as large).  The output divides by the sum of the
// rounded weights, so that a row with one dominant token keeps that token's
// value exactly; the log-sum-exp comes from the unrounded sum.
#include "locks_batch.h"
#include "locks_batch.cuh"
#include "locks_kv.cuh"
#include "locks_tc.cuh"

namespace locks {

namespace {

constexpr int kThreads = 384;                         // three warpgroups: two of softmax, one of the others
constexpr int kProducerWarp = 8, kMmaWarp = 9;
// registers a thread after the split: 256 * 208 + 128 * 88 = 384 * 168, the launch's
constexpr int kSoftmaxRegs = 208, kOtherRegs = 88;
constexpr int kTileBytes = 128 * 256;                 // 128 rows of 128 bf16
constexpr int kHalfBytes = kTileBytes / 2;
constexpr int kRing = 5;
// Pieces handed on: when piece n is written the queries of piece n - 2 have had their last use, so
// (two products ahead, at least one stage a piece) the softmax groups are past piece n - 8.
constexpr int kPieces = 16;
constexpr uint32_t kTmemCols = 512;                   // S0 S1 O0 O1
constexpr float kLazy = 8.f;                          // log2 growth of a maximum that is left alone

// A unit's stages [s0, s0 + stages) that this block has, as the loading warp hands them to the others.
struct Piece {
  int stages;
  int pair;               // two tiles: both on every stage; else stages in turn
  int group_pages;        // the unit is a group's (else a sequence's own pages)
  int head, tokens, row, page0;
  int q0, nq;             // query tokens of the unit (at most two tiles)
  int s0;
  __device__ __forceinline__ int jobs() const { return pair ? 2 * stages : stages; }
};

struct Shared {
  Piece piece[kPieces];
  uint64_t piece_full[kPieces];
  uint64_t full[kRing], empty[kRing];
  uint64_t q_full[2], q_empty[2];
  uint64_t s_full[2], p_full[2], o_full[2], o_empty[2];
  uint64_t done;
  uint32_t tmem;
  int dead;                                           // a wait ran out: every role leaves
  int bad[8];                                         // pages of a stage whose block is invalid, by stage & 7
  ListPlace place;
};
constexpr size_t kSmemBytes = size_t(kRing + 2) * kTileBytes + 1024 + sizeof(Shared);
static_assert(kSmemBytes <= kMaxSmemBlock, "shared memory of a block");

// ---- the list of work -----------------------------------------------------------
__device__ __forceinline__ int clamp_int(int x, int lo, int hi) { return min(max(x, lo), hi); }

__device__ __forceinline__ int start_of(const PrefixParams& p, int g) {
  return clamp_int(p.group_starts[g], 0, p.batch);
}
__device__ __forceinline__ int pages_of(const PrefixParams& p, int g) {
  return clamp_int(p.prefix_pages[g], 0, p.max_pages);
}
__device__ __forceinline__ int length_of(const PrefixParams& p, int b) {
  return clamp_int(p.seq_lens[b], 0, p.max_pages * p.page_size);
}
// the group of sequence b, or -1
__device__ int group_of(const PrefixParams& p, int b) {
  int lo = 0, hi = p.n_groups;                        // the last group that starts at or before b
  while (lo < hi) {
    const int mid = (lo + hi) >> 1;
    if (start_of(p, mid) <= b) lo = mid + 1;
    else hi = mid;
  }
  return lo > 0 && b < start_of(p, lo) ? lo - 1 : -1;
}

// Entry e < n_groups: the shared pages of group e; else the own pages of sequence e - n_groups.
struct Entry {
  int units, stages;      // units (KV head, and of a group 256 query rows) of so many stages each
  int tokens, row, page0; // tokens; the block table's row and its first page
  int q0, nq, tiles;      // first query token (of all), how many, in units of two tiles a head
};

__device__ Entry load_entry(const PrefixParams& p, int e) {
  Entry n;
  if (e < p.n_groups) {
    const int a = start_of(p, e), seqs = max(0, start_of(p, e + 1) - a);
    n.tokens = pages_of(p, e) * p.page_size;
    n.row = a;
    n.page0 = 0;
    n.q0 = a * p.n_rows;
    n.nq = seqs * p.n_rows;
    if (n.nq == 0) n.tokens = 0;
  } else {
    const int b = e - p.n_groups, g = group_of(p, b);
    n.page0 = g >= 0 ? pages_of(p, g) : 0;
    n.tokens = max(0, length_of(p, b) - n.page0 * p.page_size);
    n.row = b;
    n.q0 = b * p.n_rows;
    n.nq = p.n_rows;
  }
  n.stages = (n.tokens + kStageTok - 1) / kStageTok;
  n.tiles = (n.nq + 2 * p.tile_tokens - 1) / (2 * p.tile_tokens);
  n.units = n.tiles * p.n_kv_heads;
  return n;
}

// The pieces of this block's share, in the list's order.
struct Walk {
  int e, offset, left;
  Entry n;
  __device__ Walk(const PrefixParams& p, const Shared& sh, int share)
      : e(sh.place.entry), offset(sh.place.offset), left(share), n(load_entry(p, e)) {}
  __device__ bool next(const PrefixParams& p, Piece& u) {
    if (left <= 0) return false;
    while (offset >= n.units * n.stages) {
      offset = 0;
      if (++e >= p.n_groups + p.batch) return false;
      n = load_entry(p, e);
    }
    const int unit = offset / n.stages, tile = unit % n.tiles;
    u.group_pages = e < p.n_groups;
    u.head = unit / n.tiles;
    u.tokens = n.tokens;
    u.row = n.row;
    u.page0 = n.page0;
    u.q0 = n.q0 + tile * 2 * p.tile_tokens;
    u.nq = min(n.nq - tile * 2 * p.tile_tokens, 2 * p.tile_tokens);
    u.pair = u.nq > p.tile_tokens;
    u.s0 = offset - unit * n.stages;
    u.stages = min(n.stages - u.s0, left);
    offset += u.stages;
    left -= u.stages;
    return true;
  }
};

// ---- the softmax groups ---------------------------------------------------------
__device__ void softmax_role(const PrefixParams& p, Shared& sh, unsigned char* ring, int w,
                             int share) {
  const int tid = threadIdx.x & 127, lane = tid & 31;
  const uint32_t lanes = sh.tmem + (uint32_t(tid >> 5 << 5) << 16);
  const uint32_t t_s = lanes + w * 128, t_o = lanes + 256 + w * 128;
  const int rt = tid / p.group, head_in_group = tid % p.group;
  const int npg_shift = p.page_shift;
  int job0 = 0, stage0 = 0, units = 0;
  for (int n = 0; stage0 < share; ++n) {
    if (!warp_wait_or_dead(&sh.piece_full[n % kPieces], (n / kPieces) & 1, &sh.dead)) return;
    const Piece u = sh.piece[n % kPieces];
    const int njobs = u.jobs();
    const int first = (job0 & 1) == w ? 0 : 1;
    if (first < njobs) {
      const int tq = (u.pair ? w * p.tile_tokens : 0) + rt;
      const bool valid = rt < p.tile_tokens && tq < u.nq;
      int lim = 1 << 30;                              // tokens of the unit that this row sees
      const int qt = u.q0 + tq;                       // query token among the batch's
      if (valid) {
        const int b = qt / p.n_rows, r = qt - b * p.n_rows;
        lim = clamp_int(length_of(p, b) - p.n_rows + r + 1 - u.page0 * p.page_size, 0, u.tokens);
      }
      const bool any = __any_sync(kFull, valid);
      float m = -INFINITY, l = 0.f, lr = 0.f;
      for (int job = first; job < njobs; job += 2) {
        const int i = u.pair ? job >> 1 : job;
        const int tok = (u.s0 + i) * kStageTok, nv = min(kStageTok, u.tokens - tok);
        if (!warp_wait_or_dead(&sh.s_full[w], ((job0 + job) >> 1) & 1, &sh.dead)) return;
        tc_fence_after();
        const int bad = *static_cast<volatile int*>(&sh.bad[(stage0 + i) & 7]);
        if (any) {
          float s[128];
#pragma unroll
          for (int c = 0; c < 128; c += 32) tmem_ld32(t_s + c, s + c);
          tmem_wait_ld();
          const int seen = lim - tok;
          if (__any_sync(kFull, seen < 128) || bad) {
#pragma unroll
            for (int c = 0; c < 128; ++c)
              if (c >= seen || (bad >> (c >> npg_shift) & 1)) s[c] = -INFINITY;
          }
          float mx[4] = {s[0], s[1], s[2], s[3]};
#pragma unroll
          for (int c = 4; c < 128; c += 4) {
#pragma unroll
            for (int k = 0; k < 4; ++k) mx[k] = fmaxf(mx[k], s[c + k]);
          }
          const float top = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])) * p.scale_log2;
          // (rows past the unit's last hold whatever the tile held, and decide nothing)
          if (__any_sync(kFull, valid && top > m + kLazy)) {
            const float mn = fmaxf(m, top);
            const float f = m == -INFINITY ? 0.f : ex2_approx(m - mn);
            m = mn;
            l *= f;
            lr *= f;
            if (job >= 2) {                           // (the first product overwrites O)
#pragma unroll 1
              for (int c = 0; c < 128; c += 16) {
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
          for (int c = 0; c < 128; c += 32) {
            uint32_t pk[16];
#pragma unroll
            for (int k = 0; k < 16; ++k) {
              float2 x = ffma2(make_float2(s[c + 2 * k], s[c + 2 * k + 1]), sc, off);
              x.x = ex2_approx(x.x);
              x.y = ex2_approx(x.y);
              const __nv_bfloat162 h = __floats2bfloat162_rn(x.x, x.y);
              pk[k] = *reinterpret_cast<const uint32_t*>(&h);
              a0 = fadd2(a0, x);
              a1 = fadd2(a1, make_float2(bf16_lo(pk[k]), bf16_hi(pk[k])));
            }
            tmem_st16(t_s + c / 2, pk);
          }
          l += a0.x + a0.y;
          lr += a1.x + a1.y;
          tmem_wait_st();
        }
        if (nv < kStageTok || bad) {
          // rows of V that no query sees (behind the unit's end, or of an invalid page) may hold
          // anything, NaN included, which a weight of 0 would not keep out
          const int n = 2 * (stage0 + i) + 1, slot = n % kRing;
          if (!warp_wait_or_dead(&sh.full[slot], (n / kRing) & 1, &sh.dead)) return;
          if (tid >= nv || (bad >> (tid >> npg_shift) & 1)) {
            uint4* row = reinterpret_cast<uint4*>(ring + slot * kTileBytes + tid * 128);
#pragma unroll
            for (int c = 0; c < 8; ++c) {
              row[c] = make_uint4(0, 0, 0, 0);
              row[c + kHalfBytes / 16] = make_uint4(0, 0, 0, 0);
            }
          }
          proxy_fence_smem();
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&sh.p_full[w]);
      }
      // this group's half of the piece
      if (!warp_wait_or_dead(&sh.o_full[w], units & 1, &sh.dead)) return;
      ++units;
      tc_fence_after();
      if (any) {
        const int half = u.pair ? 0 : first;
        const int64_t row = int64_t(qt) * (p.n_kv_heads * p.group) + u.head * p.group + head_in_group;
        float* acc;
        float4* sums;
        if (u.s0 == 0) {
          const int64_t at = (u.group_pages ? 0 : 2 * p.rows) + half * p.rows + row;
          acc = p.acc + at * kHeadDim;
          sums = p.sums + at;
        } else {
          const int64_t at = int64_t(blockIdx.x) * 256 + (u.pair ? w : half) * 128 + tid;
          acc = p.carry_acc + at * kHeadDim;
          sums = p.carry_sums + at;
        }
        if (valid) *sums = make_float4(m, l, lr, 0.f);
#pragma unroll
        for (int c = 0; c < 128; c += 32) {
          float o[32];
          tmem_ld32(t_o + c, o);
          tmem_wait_ld();
          if (valid) {
#pragma unroll
            for (int k = 0; k < 32; k += 4)
              *reinterpret_cast<float4*>(acc + c + k) = make_float4(o[k], o[k + 1], o[k + 2], o[k + 3]);
          }
        }
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&sh.o_empty[w]);
    }
    job0 += njobs;
    stage0 += u.stages;
  }
}

// ---- the loading warp -------------------------------------------------------------
__device__ void load_role(const PrefixParams& p, Shared& sh, unsigned char* qtile,
                          unsigned char* ring, const CUtensorMap* map_qg, const CUtensorMap* map_qo,
                          const CUtensorMap* map_k, const CUtensorMap* map_v, int share) {
  const int lane = threadIdx.x & 31;
  const int per_stage = kStageTok >> p.page_shift;
  Walk walk(p, sh, share);
  Piece u;
  int qn = 0, stage = 0;
  bool ok = true;
  for (int piece = 0; ok && walk.next(p, u); ++piece) {
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
    const int32_t* table = p.block_table + int64_t(u.row) * p.max_pages + u.page0;
    for (int s = u.s0; ok && s < u.s0 + u.stages; ++s, ++stage) {
      // lane i has the stage's page i
      const int page = s * per_stage + lane;
      bool want = lane < per_stage && page << p.page_shift < u.tokens;
      int block = 0;
      if (want) {
        block = table[page];
        if (block < 0 || block >= p.num_blocks) {
          flag_status(p.status, LOCKS_DEV_BAD_BLOCK_ID);
          block = -1;
        }
      }
      const int bad = __ballot_sync(kFull, want && block < 0);
      want = want && block >= 0;
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
  // no block leaves while copies into its memory are in flight: after a wait that ran out, each
  // slot's last copy is waited for once more
  if (!ok) {
    for (int c = max(0, 2 * stage - kRing); c < 2 * stage; ++c)
      mbar_wait_bounded(&sh.full[c % kRing], (c / kRing) & 1);
    for (int t = max(0, qn - 2); t < qn; ++t)
      mbar_wait_bounded(&sh.q_full[t & 1], (t >> 1) & 1);
  }
}

// ---- the issuing warp (one lane issues) -------------------------------------------------------------
// Job J (counted over the block's pieces) is one stage for one softmax group, J & 1.  The products
// Q K^T run two jobs ahead of the products P V, each with a cursor like this.  The loop is kept
// short: it shares the instruction cache with the softmax, and the latency of its own instructions,
// one after another, has to stay below the products' time.
struct Cursor {
  uint32_t J = 0, job = 0, njobs = 0, pair = 0;
  uint32_t slot, phase = 0;                           // of the ring, for the stage's tile
  uint32_t tile = 0;                                  // query tiles of the pieces before
  int stages = 0, n = 0;                              // stages up to and with this piece; the next piece
  bool more = true;
  __device__ __forceinline__ explicit Cursor(uint32_t s) : slot(s) {}
  __device__ __forceinline__ bool open(Shared& sh, int share) {
    more = stages < share;
    if (!more) return true;
    if (!mbar_wait_or_dead(&sh.piece_full[n % kPieces], (n / kPieces) & 1, &sh.dead)) return false;
    const Piece& u = sh.piece[n % kPieces];
    ++n;
    stages += u.stages;
    pair = u.pair;
    njobs = u.jobs();
    job = 0;
    return true;
  }
  __device__ __forceinline__ bool first_of_stage() const { return !(job & pair); }
  __device__ __forceinline__ bool last_of_stage() const { return !pair || (job & 1); }
  __device__ __forceinline__ bool advance(Shared& sh, int share) {
    if (last_of_stage()) {
      slot += 2;                                      // (keys and values take slots in turn)
      if (slot >= kRing) {
        slot -= kRing;
        phase ^= 1;
      }
    }
    ++J;
    if (++job < njobs) return true;
    tile += 1 + pair;
    return open(sh, share);
  }
};

__device__ void issue_role(Shared& sh, unsigned char* qtile, unsigned char* ring, int share) {
  constexpr uint32_t kIdescS = mma_idesc(128, 128, false), kIdescO = mma_idesc(128, 128, true);
  const uint32_t tmem = sh.tmem;
  const uint32_t q_desc = smem_desc_lo(smem_u32(qtile), 16);
  const uint32_t k_desc = smem_desc_lo(smem_u32(ring), 16);
  // 64 columns of V (a half) follow each other at kHalfBytes, 8 tokens at 1024 bytes
  const uint32_t v_desc = smem_desc_lo(smem_u32(ring), kHalfBytes);
  Cursor a(0), b(1);
  uint32_t opened = 0;                                // accumulators begun, modulo 2, a bit a group
  int ahead = 0;
  bool ok = a.open(sh, share) && b.open(sh, share);
  while (ok && b.more) {
    if (ahead == 2) {                                 // P V of job b.J
      const uint32_t w = b.J & 1;
      ok = mbar_wait_or_dead(&sh.p_full[w], (b.J >> 1) & 1, &sh.dead);
      if (ok && b.first_of_stage()) ok = mbar_wait_or_dead(&sh.full[b.slot], b.phase, &sh.dead);
      uint32_t add = 1;
      if (ok && b.job < 2) {                          // the first of this unit for this group
        add = 0;
        ok = mbar_wait_or_dead(&sh.o_empty[w], (opened >> w & 1) ^ 1, &sh.dead);
        opened ^= 1u << w;
      }
      if (!ok) break;
      tc_fence_after();
      uint32_t db = v_desc + b.slot * (kTileBytes >> 4), p = tmem + w * 128;
      const uint32_t d = p + 256;
#pragma unroll
      for (int k = 0; k < 8; ++k)                     // 16 of the 128 tokens each
        mma_ts(d, p + 8 * k, db + k * (2048 >> 4), kIdescO, k > 0 ? 1u : add);
      if (b.last_of_stage()) mma_commit(&sh.empty[b.slot]);
      if (b.job + 2 >= b.njobs) mma_commit(&sh.o_full[w]);
      ok = b.advance(sh, share);
    } else {
      ++ahead;
    }
    if (ok && a.more) {                               // Q K^T of job a.J
      const uint32_t w = a.J & 1, t = a.tile + (w & a.pair), qs = t & 1;
      if (a.job <= a.pair) ok = mbar_wait_or_dead(&sh.q_full[qs], t >> 1 & 1, &sh.dead);
      if (ok && a.first_of_stage()) ok = mbar_wait_or_dead(&sh.full[a.slot], a.phase, &sh.dead);
      if (!ok) break;
      const uint32_t da = q_desc + qs * (kTileBytes >> 4), db = k_desc + a.slot * (kTileBytes >> 4);
      const uint32_t d = tmem + w * 128;
#pragma unroll
      for (int k = 0; k < 8; ++k) {                   // 16 of the 128 dims each, 64 in a half
        const uint32_t o = ((k >> 2) * kHalfBytes + (k & 3) * 32) >> 4;
        mma_ss(d, da + o, db + o, kIdescS, k > 0);
      }
      mma_commit(&sh.s_full[w]);
      if (a.last_of_stage()) mma_commit(&sh.empty[a.slot]);
      if (a.job + 1 + a.pair >= a.njobs) mma_commit(&sh.q_empty[qs]);
      ok = a.advance(sh, share);
    }
  }
  // everything issued is done before the block frees its tensor memory
  mma_commit(&sh.done);
  mbar_wait_bounded(&sh.done, 0);
}

__global__ void __launch_bounds__(kThreads, 1)
    prefix_kernel(const PrefixParams p, const __grid_constant__ CUtensorMap map_qg,
                  const __grid_constant__ CUtensorMap map_qo,
                  const __grid_constant__ CUtensorMap map_k,
                  const __grid_constant__ CUtensorMap map_v) {
  extern __shared__ unsigned char smem_raw[];
  unsigned char* smem = smem_raw + (-smem_u32(smem_raw) & 1023);
  unsigned char* qtile = smem;
  unsigned char* ring = smem + 2 * kTileBytes;
  Shared& sh = *reinterpret_cast<Shared*>(smem + (kRing + 2) * kTileBytes);
  const int tid = threadIdx.x, warp = tid >> 5;

  if (warp == kMmaWarp) tmem_alloc(&sh.tmem, kTmemCols);
  if (tid == 0) {
    for (int i = 0; i < kRing; ++i) {
      mbar_init(&sh.full[i], 1);
      mbar_init(&sh.empty[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&sh.q_full[i], 1);
      mbar_init(&sh.q_empty[i], 1);
      mbar_init(&sh.s_full[i], 1);
      mbar_init(&sh.p_full[i], 4);
      mbar_init(&sh.o_full[i], 1);
      mbar_init(&sh.o_empty[i], 4);
    }
    for (int i = 0; i < kPieces; ++i) mbar_init(&sh.piece_full[i], 1);
    mbar_init(&sh.done, 1);
    mbar_fence_init();
    sh.dead = 0;
    prefetch_map(&map_qg);
    prefetch_map(&map_qo);
    prefetch_map(&map_k);
    prefetch_map(&map_v);
  }
  // what follows reads memory that the kernel before this one may write
  griddep_wait();

  tc_fence_before();
  const int entries = p.n_groups + p.batch;
  int total;
  const int share = locate<kThreads>(
      [&](int e) {
        const Entry n = load_entry(p, e);
        return n.units * n.stages;
      },
      entries, blockIdx.x, kBatchSms, sh.place, total,
      [&](int e, int first) {
        if (blockIdx.x) return;
        // for the kernel that joins the pieces; and the arguments' check
        p.entry_start[e] = first;
        if (e >= p.n_groups) {
          const int t = p.seq_lens[e - p.n_groups];
          if (t < 0 || t > p.max_pages * p.page_size) flag_status(p.status, LOCKS_DEV_BAD_SEQ_LEN);
        } else {
          const int a = p.group_starts[e], z = p.group_starts[e + 1], n_pages = p.prefix_pages[e];
          if (a < 0 || z < a || z > p.batch || n_pages < 0 || n_pages > p.max_pages)
            flag_status(p.status, LOCKS_DEV_BAD_GROUP);
        }
      });
  if (blockIdx.x == 0 && tid == 0) p.entry_start[entries] = total;
  tc_fence_after();
  griddep_launch();

  if (share > 0) {
    if (warp < kProducerWarp) {
      asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kSoftmaxRegs));
      softmax_role(p, sh, ring, warp >> 2, share);
    } else {
      asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kOtherRegs));
      if (warp == kProducerWarp) load_role(p, sh, qtile, ring, &map_qg, &map_qo, &map_k, &map_v, share);
      else if (warp == kMmaWarp && elect_one()) issue_role(sh, qtile, ring, share);
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (tid == 0 && sh.dead) flag_status(p.status, LOCKS_DEV_WAIT_TIMEOUT);
  if (warp == kMmaWarp) tmem_free(sh.tmem, kTmemCols);
}

// ---- joining the pieces: a warp per (query token, head) row -------------------------
constexpr int kJoinWarps = 8;

__global__ void __launch_bounds__(kJoinWarps * 32) join_kernel(const PrefixParams p) {
  griddep_wait();
  const int lane = threadIdx.x & 31;
  const int64_t row = int64_t(blockIdx.x) * kJoinWarps + (threadIdx.x >> 5);
  if (row >= p.rows) return;
  const int hq = p.n_kv_heads * p.group;
  const int qt = int(row / hq), head_q = int(row - int64_t(qt) * hq);
  const int b = qt / p.n_rows, head = head_q / p.group;
  const int entries = p.n_groups + p.batch;
  const int total = p.entry_start[entries];
  float M = -INFINITY, L = 0.f, LR = 0.f;
  float4 A = make_float4(0.f, 0.f, 0.f, 0.f);

  auto add = [&](const float* acc, const float4* sums) {
    const float4 s = *sums;
    // (a part in which the row sees nothing has no sum, and an accumulator of no account)
    if (s.y == 0.f) return;
    const float mn = fmaxf(M, s.x);
    const float f = M == -INFINITY ? 0.f : exp2f(M - mn), g = exp2f(s.x - mn);
    const float4 a = *reinterpret_cast<const float4*>(acc + 4 * lane);
    A.x = A.x * f + a.x * g;
    A.y = A.y * f + a.y * g;
    A.z = A.z * f + a.z * g;
    A.w = A.w * f + a.w * g;
    L = L * f + s.y * g;
    LR = LR * f + s.z * g;
    M = mn;
  };
  auto unit = [&](int e, int kind) {
    const Entry n = load_entry(p, e);
    if (n.units * n.stages == 0) return;
    const int tq = qt - n.q0, tile = tq / (2 * p.tile_tokens), in = tq - tile * 2 * p.tile_tokens;
    const bool pair = n.nq - tile * 2 * p.tile_tokens > p.tile_tokens;
    const int w = in / p.tile_tokens;
    const int r = (in - w * p.tile_tokens) * p.group + head_q - head * p.group;
    const int first = p.entry_start[e] + (head * n.tiles + tile) * n.stages;
    int at = first;
    while (at < first + n.stages) {
      const int c = int(((int64_t(at) + 1) * kBatchSms - 1) / total);
      const int end = min(first + n.stages, share_begin(total, c + 1, kBatchSms));
      for (int half = 0; half < (pair ? 1 : min(2, end - at)); ++half) {
        if (at == first) {
          const int64_t i = (2 * kind + half) * p.rows + row;
          add(p.acc + i * kHeadDim, p.sums + i);
        } else {
          const int64_t i = int64_t(c) * 256 + (pair ? w : half) * 128 + r;
          add(p.carry_acc + i * kHeadDim, p.carry_sums + i);
        }
      }
      at = end;
    }
  };
  const int g = group_of(p, b);
  if (g >= 0) unit(g, 0);
  unit(p.n_groups + b, 1);

  const float inv = LR == 0.f ? 0.f : 1.f / LR;
  const __nv_bfloat162 o01 = __floats2bfloat162_rn(A.x * inv, A.y * inv);
  const __nv_bfloat162 o23 = __floats2bfloat162_rn(A.z * inv, A.w * inv);
  uint2 ow;
  ow.x = *reinterpret_cast<const uint32_t*>(&o01);
  ow.y = *reinterpret_cast<const uint32_t*>(&o23);
  *reinterpret_cast<uint2*>(p.out + row * kHeadDim + 4 * lane) = ow;
  if (lane == 0 && p.out_lse) p.out_lse[row] = L == 0.f ? -INFINITY : kLn2 * (M + log2f(L));
}

}  // namespace

PrefixLayout prefix_layout(int64_t rows, int64_t entries) {
  PrefixLayout L;
  const auto up = [](size_t x) { return (x + 255) / 256 * 256; };
  L.acc = 0;
  L.sums = up(L.acc + size_t(4) * rows * kHeadDim * sizeof(float));
  L.carry_acc = up(L.sums + size_t(4) * rows * sizeof(float4));
  L.carry_sums = up(L.carry_acc + size_t(kBatchSms) * 256 * kHeadDim * sizeof(float));
  L.entry_start = up(L.carry_sums + size_t(kBatchSms) * 256 * sizeof(float4));
  L.total = up(L.entry_start + size_t(entries + 1) * sizeof(int32_t));
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
  const int64_t blocks = (p.rows + kJoinWarps - 1) / kJoinWarps;
  return launch_dependent(join_kernel, dim3(unsigned(blocks)), kJoinWarps * 32, 0, p, stream);
}

}  // namespace locks
