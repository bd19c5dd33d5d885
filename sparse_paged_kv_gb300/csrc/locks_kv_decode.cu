// locks_kv_decode: attention of one new token per sequence over a quantised
// paged cache,
//   out = sum_t p_t v_t,   p = softmax(q^T k_t / sqrt(d)).
//
// Mathematics.  A row is k_t = s_t c_t (codes c, scale s), so q^T k_t =
// s_t (q^T c_t): the scale multiplies a logit and not 128 elements; likewise
// sum_t p_t v_t = sum_t (p_t s'_t) c'_t.  The codes (times their group scale,
// in 4 bits) are exact in f16, as is the bf16 query scaled by a power of two,
// so q^T c_t is a float32 sum of exact products on the tensor cores.  The
// weights p_t s'_t are rounded to f16 (2^-11, an eighth of the output's own
// rounding, and about 1% of the error where the two are together; a second f16 for
// the rest of a weight would double the second product); the sum of p_t that
// divides the result is kept in float32.
//
// Work split.  The 64-token stages of all (sequence, KV head) units form one
// list, each unit preceded by its fixed cost; block c of 152 (one per SM) takes
// the c-th part of it, whatever the lengths of the sequences, so that ragged
// batches load every SM alike.  (Units of one length that so many blocks each
// nearly fill the SMs are cut in equal parts instead.)  A unit that lies in one block is finished there;
// one that is cut is left as partials (running maximum, sum, weighted values) in
// the workspace, and the last of its blocks to arrive (atomic ticket) merges them
// in the blocks' order, so results do not depend on the order of arrival.  The
// workspace is a megabyte or two whatever the shape, and shapes may share it.
//
// Block.  Four producer warps take the stages in turn: each looks up its next
// pages (one a lane) and copies their K and V records (cp.async.bulk, one
// contiguous piece each) into a ring of 64-token stages; the last of them also
// brings the next unit's query.  Consumer warps take 16-token chunks of the
// stages in turn and keep everything in registers:
//   S^T (16 tokens x 8 heads)  = K (16 x 128) . Q^T      8 mma m16n8k16
//   O^T (128 dims x 8 heads)  += V^T (128 x 16) . P^T    8 mma m16n8k16
// Tokens and dims are the long sides of the products, so the short one, the
// heads, fills its 8 columns twice as well as it would 16 rows.  K's fragments
// are rows as they lie in memory (the dims of a product may come in any order
// that Q shares); V's are two tokens' bytes interleaved by a byte permute; P is
// turned from S^T's layout into an operand by movmatrix.
//
// Measured (one GB300, of 6.78 TB/s copy): e4m3 1M tokens 314 us (7.05 TB/s), 8 x
// 32K 86 us (6.4 TB/s): memory.  int4 4 x 128K 121 us (5.0 TB/s): 370 instructions
// for 16 tokens of a head, over half of them unpacking codes, issue in 65% of the
// cycles; the ALU (50%) and memory (55%) are further from their limits, and forms
// that spill 88, 100 or 212 bytes take the same time.  One sequence of 1000 tokens
// 9.6 us: a chain of latencies.
#include "locks_kv.cuh"

namespace locks {

namespace {

// One block per SM.  For up to 8 heads a group 16 consumer warps of 104
// registers; for up to 16, whose accumulators are twice as large, 12 of 136 (2 KV
// heads of 16 heads, us, with 12 and with 8 warps of 168: 16 x 128K tokens int4
// 190, 216, e4m3 171, 186; 4 x 20000 e4m3 23.2, 22.5; 1 x 1000 13.0, 11.6: long
// caches have the most to gain).
constexpr int kSms = 152;
__host__ __device__ constexpr int kv_warps(int nt) { return nt == 1 ? 16 : 12; }
// And a warpgroup of producers: among busy consumers a warp issues an instruction
// in about seven cycles, and one producer could not keep up with the stages (1M
// e4m3: 415 us).  All four copy; with 12 consumers three do, as the ring's length
// has to suit both.
__host__ __device__ constexpr int kv_threads(int nt) { return kv_warps(nt) * 32 + 128; }
constexpr int kv_copiers(int nt) { return nt == 1 ? 4 : 3; }
constexpr int kv_consumer_regs(int nt) { return nt == 1 ? 104 : 136; }   // of a thread
constexpr int kv_producer_regs(int nt) { return nt == 1 ? 64 : 96; }
// the launch has 65536 / threads, rounded down to 8
constexpr bool kv_regs_fit(int nt) {
  return kv_warps(nt) * 32 * kv_consumer_regs(nt) + 128 * kv_producer_regs(nt) <=
         kv_threads(nt) * (65536 / kv_threads(nt) / 8 * 8);
}
static_assert(kv_regs_fit(1) && kv_regs_fit(2), "registers of the launch");
constexpr int kStageTok = 64;
constexpr float kNone = -3.402823466e38f;         // running maximum before any token
// merge buffer: the warps' states of 8 heads x 128 floats
constexpr int kv_merge_bytes(int nt) { return kv_warps(nt) * 4096; }

// workspace: a ticket and two partials a block
constexpr size_t kTicketBytes = 1024;
static_assert(kSms * sizeof(int) <= kTicketBytes, "tickets");
__host__ __device__ constexpr size_t kv_part_bytes(int nt) { return size_t(nt) * (4096 + 64); }

__host__ __device__ constexpr int kv_stage_bytes(int fmt) {
  return 2 * kStageTok * (kv_row_bytes(fmt) + (fmt == LOCKS_KV_I4 ? 8 : 4));
}
// 16-token chunks a warp takes at a time: two in 4 bits, where instructions bind
// (int4 4 x 128K: 144 -> 122 us); one in 8 bits, where two would hold the whole
// ring while they are computed on (e4m3 1M: 316 -> 320 us).
constexpr int kv_chunks(int fmt, int nt) { return nt == 1 && fmt == LOCKS_KV_I4 ? 2 : 1; }
// Stages of the ring, beside the merge buffer.  The number has to make a ring of
// jobs a whole number of rounds of the warps: a warp then comes back to a ring
// slot at every use of it, as waiting by the barrier's parity requires (copies
// land out of order, so having seen a later stage full says nothing about a
// slot's earlier use).
constexpr int kv_stages(int fmt, int nt) {
  return nt == 1 ? (fmt == LOCKS_KV_I4 ? 16 : 8) : (fmt == LOCKS_KV_I4 ? 12 : 9);
}
constexpr bool kv_rounds(int fmt, int nt) {
  return 4 / kv_chunks(fmt, nt) * kv_stages(fmt, nt) % kv_warps(nt) == 0 &&
         kv_stages(fmt, nt) % kv_copiers(nt) == 0;     // (and a slot belongs to one producer warp)
}
static_assert(kv_rounds(LOCKS_KV_F8, 1) && kv_rounds(LOCKS_KV_I4, 1) && kv_rounds(LOCKS_KV_F8, 2) &&
                  kv_rounds(LOCKS_KV_I4, 2),
              "every warp must see every use of the ring slots it visits");

__device__ __forceinline__ uint32_t prmt(uint32_t a, uint32_t b, uint32_t sel) {
  uint32_t r;
  asm("prmt.b32 %0, %1, %2, %3;" : "=r"(r) : "r"(a), "r"(b), "r"(sel));
  return r;
}
__device__ __forceinline__ uint32_t hfma2(uint32_t a, uint32_t b, uint32_t c) {
  uint32_t r;
  asm("fma.rn.f16x2 %0, %1, %2, %3;" : "=r"(r) : "r"(a), "r"(b), "r"(c));
  return r;
}
__device__ __forceinline__ uint32_t hmul2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
__device__ __forceinline__ uint32_t hadd2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("add.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
__device__ __forceinline__ uint32_t f16x2(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
__device__ __forceinline__ uint32_t transpose8x8(uint32_t a) {
  uint32_t r;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(a));
  return r;
}
__device__ __forceinline__ void mma_f16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                        uint32_t a3, uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
      "{%8,%9}, {%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint4 lds128(uint32_t a) {
  uint4 v;
  asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "r"(a));
  return v;
}
__device__ __forceinline__ uint2 lds64(uint32_t a) {
  uint2 v;
  asm volatile("ld.shared.v2.u32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(a));
  return v;
}
__device__ __forceinline__ float lds_f(uint32_t a) {
  float v;
  asm volatile("ld.shared.f32 %0, [%1];" : "=f"(v) : "r"(a));
  return v;
}
__device__ __forceinline__ uint32_t lds_u8(uint32_t a) {
  uint32_t v;
  asm volatile("ld.shared.u8 %0, [%1];" : "=r"(v) : "r"(a));
  return v;
}
template <int NT>
__device__ __forceinline__ void consumers_sync() {
  asm volatile("bar.sync 1, %0;" ::"n"(kv_warps(NT) * 32) : "memory");
}

// (a & b) | c as one instruction: left to itself the compiler makes two of it
// when both b and c are constants (int4, 4 x 128K: 166 -> 154 us)
__device__ __forceinline__ uint32_t and_or(uint32_t a, uint32_t b, uint32_t c) {
  uint32_t r;
  asm("lop3.b32 %0, %1, %2, %3, 0xEA;" : "=r"(r) : "r"(a), "r"(b), "r"(c));
  return r;
}

// 4-bit codes: nibbles n and n + 4 of a word as f16x2 of c * s, exact.  A nibble
// under the exponent bits of 1024 is 1024 + u (u = c + 8), or 1024 + 16 u where
// it lies four bits higher; one fma takes the offset off and the scale on.
// s = e4m3 * 2^-8 keeps 1032 s inside f16's range (the 2^8 is made up for in float32).
struct I4Scale {
  uint32_t s, off, s16, off16;   // s, -1032 s, s / 16, -72 s
};
__device__ __forceinline__ I4Scale i4_scale(uint32_t s) {
  I4Scale r;
  r.s = hmul2(s, 0x1c001c00u);            // 2^-8
  r.off = hmul2(r.s, 0xe408e408u);        // -1032
  r.s16 = hmul2(r.s, 0x2c002c00u);        // 2^-4
  r.off16 = hmul2(r.s, 0xd480d480u);      // -72
  return r;
}
__device__ __forceinline__ void i4_pairs(uint32_t w, const I4Scale& s, uint32_t (&x)[4]) {
  const uint32_t v = w >> 8;
  x[0] = hfma2(and_or(w, 0x000f000fu, 0x64006400u), s.s, s.off);
  x[1] = hfma2(and_or(w, 0x00f000f0u, 0x64006400u), s.s16, s.off16);
  x[2] = hfma2(and_or(v, 0x000f000fu, 0x64006400u), s.s, s.off);
  x[3] = hfma2(and_or(v, 0x00f000f0u, 0x64006400u), s.s16, s.off16);
}
// two 8-bit codes in bytes (0, 1) or (2, 3) of w -> f16x2, exact
template <int FMT, int HI>
__device__ __forceinline__ uint32_t pair8(uint32_t w) {
  if constexpr (FMT == LOCKS_KV_F8) {
    return e4m3x2_to_f16x2(HI ? w >> 16 : w & 0xffffu);
  } else {
    // byte u = c + 128 under 1024's exponent, minus 1152
    return hadd2(prmt(w, 0x64646464u, HI ? 0x4342u : 0x4140u), 0xe480e480u);
  }
}

// Per-head softmax state of a lane's 2 NT head columns.
template <int NT>
struct State {
  float m[2 * NT];       // reference of the exponent (log2), within 8 of the running maximum
  float l[2 * NT];       // this lane's part of sum 2^(z - m)
  float f[2 * NT];       // factor that brings the weights to f16: largest seen -> 2^7 .. 2^15
  float acc[NT][8][4];   // O^T, times f
};

// Where a lane finds its part of 16 tokens: shared-memory byte offsets from the
// tokens' codes, or from their scales, in a stage (V's records are half a stage
// further on).  Rows 8 apart share a permutation, so the other addresses are
// these plus constants, or with bit 4 flipped (the neighbouring chunk).
struct LaneOff {
  uint32_t k;            // K: row g, first chunk
  uint32_t v;            // V: row 2t, this lane's dims
  uint32_t scale;        // scale of row g
  uint32_t gk, gv;       // I4: group scales of K's row g and of V's row 2t
};
template <int FMT>
__device__ __forceinline__ LaneOff lane_off(int B, int g, int t) {
  constexpr uint32_t kV = kv_stage_bytes(FMT) / 2;
  LaneOff o;
  o.k = kv_chunk_off<FMT>(g, FMT == LOCKS_KV_I4 ? t : 2 * t);
  o.v = kV + (FMT == LOCKS_KV_I4 ? kv_chunk_off<FMT>(2 * t, g >> 1) + 8 * (g & 1)
                                 : kv_chunk_off<FMT>(2 * t, g));
  o.scale = kv_scale_off(FMT, B) + 4 * g;
  o.gk = kv_group_off(FMT, B) + 4 * g + t;
  o.gv = kV + kv_group_off(FMT, B) + 8 * t + (g >> 1);
  return o;
}

// C chunks of 16 tokens of a stage, whose codes and scales are at shared-memory
// addresses base[c] and sbase[c] (plus LaneOff), of which rows lo .. hi - 1
// (range[c] = lo | hi << 8) are attended.
template <int FMT, int NT, int C>
__device__ __forceinline__ void attend(const uint32_t (&base)[C], const uint32_t (&sbase)[C],
                                       const int (&range)[C], const LaneOff& off, int g, int t,
                                       uint32_t qa, const float (&qs)[2 * NT], State<NT>& st) {
  constexpr uint32_t kV = kv_stage_bytes(FMT) / 2;
  constexpr uint32_t kRow = kv_row_bytes(FMT);
  constexpr int kWhole = 16 << 8;
  bool whole = true;
#pragma unroll
  for (int c = 0; c < C; ++c) whole = whole && range[c] == kWhole;
  // ---- S^T = K Q^T ----
  float sa[C][NT][4];
#pragma unroll
  for (int c = 0; c < C; ++c) {
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int e = 0; e < 4; ++e) sa[c][n][e] = 0.f;
    const uint32_t ka = base[c] + off.k;
    if constexpr (FMT == LOCKS_KV_I4) {
      const uint4 A = lds128(ka), D = lds128(ka + 8 * kRow);
      const uint32_t ga = lds_u8(sbase[c] + off.gk), gb = lds_u8(sbase[c] + off.gk + 32);
      const I4Scale s0 = i4_scale(e4m3x2_to_f16x2(ga | (ga << 8)));
      const I4Scale s1 = i4_scale(e4m3x2_to_f16x2(gb | (gb << 8)));
      const uint32_t aw[4] = {A.x, A.y, A.z, A.w}, dw[4] = {D.x, D.y, D.z, D.w};
#pragma unroll
      for (int w = 0; w < 4; ++w) {
        uint32_t x[4], y[4];
        i4_pairs(aw[w], s0, x);
        i4_pairs(dw[w], s1, y);
#pragma unroll
        for (int n = 0; n < NT; ++n) {
          const uint4 q = lds128(qa + (n * 4 + w) * 512);
          mma_f16(sa[c][n], x[0], y[0], x[1], y[1], q.x, q.y);
          mma_f16(sa[c][n], x[2], y[2], x[3], y[3], q.z, q.w);
        }
      }
    } else {
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const uint32_t kc = ka ^ (16 * h);
        const uint4 A = lds128(kc), D = lds128(kc + 8 * kRow);
        const uint32_t aw[4] = {A.x, A.y, A.z, A.w}, dw[4] = {D.x, D.y, D.z, D.w};
#pragma unroll
        for (int w = 0; w < 4; w += 2) {
          const uint32_t a0 = pair8<FMT, 0>(aw[w]), a2 = pair8<FMT, 1>(aw[w]);
          const uint32_t a1 = pair8<FMT, 0>(dw[w]), a3 = pair8<FMT, 1>(dw[w]);
          const uint32_t b0 = pair8<FMT, 0>(aw[w + 1]), b2 = pair8<FMT, 1>(aw[w + 1]);
          const uint32_t b1 = pair8<FMT, 0>(dw[w + 1]), b3 = pair8<FMT, 1>(dw[w + 1]);
#pragma unroll
          for (int n = 0; n < NT; ++n) {
            const uint4 q = lds128(qa + (n * 4 + 2 * h + w / 2) * 512);
            mma_f16(sa[c][n], a0, a1, a2, a3, q.x, q.y);
            mma_f16(sa[c][n], b0, b1, b2, b3, q.z, q.w);
          }
        }
      }
    }
  }
  // ---- weights: z = logit in log2 units, p = 2^(z - m), w = p v_scale f ----
  float vs[C][2], z[C][2 * NT][2], w[C][2 * NT][2], sum[2 * NT];
#pragma unroll
  for (int c = 0; c < C; ++c)
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      const float ks = lds_f(sbase[c] + off.scale + 32 * r);
      vs[c][r] = lds_f(sbase[c] + off.scale + kV + 32 * r);
#pragma unroll
      for (int j = 0; j < 2 * NT; ++j) z[c][j][r] = sa[c][j >> 1][2 * r + (j & 1)] * (qs[j] * ks);
    }
  if (!whole) {
    // rows outside the attended range may hold anything: no value of theirs is used
#pragma unroll
    for (int c = 0; c < C; ++c)
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        const int row = g + 8 * r;
        if (row < (range[c] & 255) || row >= (range[c] >> 8)) {
          vs[c][r] = 0.f;
#pragma unroll
          for (int j = 0; j < 2 * NT; ++j) z[c][j][r] = -INFINITY;
        }
      }
  }
  float pmax = 0.f, wmax = 0.f;
#pragma unroll
  for (int j = 0; j < 2 * NT; ++j) {
    sum[j] = 0.f;
#pragma unroll
    for (int c = 0; c < C; ++c)
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        const float p = ex2_approx(z[c][j][r] - st.m[j]);
        sum[j] += p;
        w[c][j][r] = p * vs[c][r] * st.f[j];
        wmax = fmaxf(wmax, fabsf(w[c][j][r]));
      }
    pmax = fmaxf(pmax, sum[j]);
  }
  // The references move only when a logit passes its reference by about 2^8 or a
  // weight leaves f16's range: a few times per sequence, so most chunks do no
  // rescaling.  (Before the first token m is the lowest float and p infinite.)
  if (__any_sync(kFull, pmax > 256.f || wmax > 32768.f)) {
#pragma unroll
    for (int j = 0; j < 2 * NT; ++j) {
      const int n = j >> 1, e = j & 1;
      float mx = kNone, xm = 0.f;
#pragma unroll
      for (int c = 0; c < C; ++c) mx = fmaxf(mx, fmaxf(z[c][j][0], z[c][j][1]));
#pragma unroll
      for (int o = 4; o < 32; o <<= 1) mx = fmaxf(mx, __shfl_xor_sync(kFull, mx, o));
      mx = fmaxf(mx, st.m[j]);
      const float alpha = ex2_approx(st.m[j] - mx);
      st.m[j] = mx;
      st.l[j] *= alpha;
      sum[j] = 0.f;
#pragma unroll
      for (int c = 0; c < C; ++c)
#pragma unroll
        for (int r = 0; r < 2; ++r) {
          const float p = ex2_approx(z[c][j][r] - mx);
          sum[j] += p;
          w[c][j][r] = p * vs[c][r];
          xm = fmaxf(xm, fabsf(w[c][j][r]));
        }
#pragma unroll
      for (int o = 4; o < 32; o <<= 1) xm = fmaxf(xm, __shfl_xor_sync(kFull, xm, o));
      const float f = st.f[j];
      xm = fmaxf(xm, f > 0.f ? alpha * 128.f / f : 0.f);
      // (weights that are all zero so far leave the largest factor: any that is not will move it)
      const float fn = fminf(128.f / xm, 1.2676506e30f);
      const float up = f > 0.f ? alpha * (fn / f) : 0.f;
      st.f[j] = fn;
#pragma unroll
      for (int c = 0; c < C; ++c) {
        w[c][j][0] *= fn;
        w[c][j][1] *= fn;
      }
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        st.acc[n][i][e] *= up;
        st.acc[n][i][2 + e] *= up;
      }
    }
  }
  // ---- P^T as the second operand ----
  uint32_t pb[C][NT][2];
#pragma unroll
  for (int j = 0; j < 2 * NT; ++j) st.l[j] += sum[j];
#pragma unroll
  for (int c = 0; c < C; ++c)
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int r = 0; r < 2; ++r)
        pb[c][n][r] = transpose8x8(f16x2(w[c][2 * n][r], w[c][2 * n + 1][r]));
  // ---- O^T += V^T P^T: this lane's tokens 2t, 2t+1, 2t+8, 2t+9, dims 16g .. 16g+15 ----
  constexpr int kTok[4] = {0, 1, 8, 9};            // beyond 2t
#pragma unroll
  for (int c = 0; c < C; ++c) {
    const uint32_t va = base[c] + off.v;
    if constexpr (FMT == LOCKS_KV_I4) {
      uint2 T[4];
      uint32_t gs[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        T[i] = lds64(va + kTok[i] * kRow);
        gs[i] = lds_u8(sbase[c] + off.gv + 4 * kTok[i]);
      }
      if (!whole) {                                // 0 x NaN must not enter the sum
#pragma unroll
        for (int i = 0; i < 4; ++i)
          if (2 * t + kTok[i] < (range[c] & 255) || 2 * t + kTok[i] >= (range[c] >> 8)) gs[i] = 0;
      }
      const I4Scale s01 = i4_scale(e4m3x2_to_f16x2(gs[0] | (gs[1] << 8)));
      const I4Scale s23 = i4_scale(e4m3x2_to_f16x2(gs[2] | (gs[3] << 8)));
#pragma unroll
      for (int q = 0; q < 4; ++q) {       // dims 4q .. 4q + 3: half a word of each token
        const uint32_t sel = (q & 1) ? 0x7632u : 0x5410u;
        const uint32_t a = prmt(q < 2 ? T[0].x : T[0].y, q < 2 ? T[1].x : T[1].y, sel);
        const uint32_t d = prmt(q < 2 ? T[2].x : T[2].y, q < 2 ? T[3].x : T[3].y, sel);
        uint32_t x[4], y[4];
        i4_pairs(a, s01, x);
        i4_pairs(d, s23, y);
#pragma unroll
        for (int n = 0; n < NT; ++n) {
          mma_f16(st.acc[n][2 * q], x[0], x[1], y[0], y[1], pb[c][n][0], pb[c][n][1]);
          mma_f16(st.acc[n][2 * q + 1], x[2], x[3], y[2], y[3], pb[c][n][0], pb[c][n][1]);
        }
      }
    } else {
      uint4 T[4];
      T[0] = lds128(va);
      T[1] = lds128((va ^ 16) + kRow);             // odd rows: the neighbouring chunk place
      T[2] = lds128(va + 8 * kRow);
      T[3] = lds128((va ^ 16) + 9 * kRow);
      if (FMT == LOCKS_KV_F8 && !whole) {          // e4m3 NaN codes
#pragma unroll
        for (int i = 0; i < 4; ++i)
          if (2 * t + kTok[i] < (range[c] & 255) || 2 * t + kTok[i] >= (range[c] >> 8))
            T[i] = make_uint4(0, 0, 0, 0);
      }
      const uint32_t T0[4] = {T[0].x, T[0].y, T[0].z, T[0].w}, T1[4] = {T[1].x, T[1].y, T[1].z, T[1].w};
      const uint32_t T2[4] = {T[2].x, T[2].y, T[2].z, T[2].w}, T3[4] = {T[3].x, T[3].y, T[3].z, T[3].w};
#pragma unroll
      for (int q = 0; q < 4; ++q) {
#pragma unroll
        for (int e = 0; e < 2; ++e) {     // dims 4q + 2e, 4q + 2e + 1
          const uint32_t sel = e ? 0x7362u : 0x5140u;
          const uint32_t x = prmt(T0[q], T1[q], sel), y = prmt(T2[q], T3[q], sel);
          const uint32_t a0 = pair8<FMT, 0>(x), a1 = pair8<FMT, 1>(x);
          const uint32_t a2 = pair8<FMT, 0>(y), a3 = pair8<FMT, 1>(y);
#pragma unroll
          for (int n = 0; n < NT; ++n)
            mma_f16(st.acc[n][2 * q + e], a0, a1, a2, a3, pb[c][n][0], pb[c][n][1]);
        }
      }
    }
  }
}

// What a unit costs a block beside its stages, in stages: the warps wait for one
// another at its end and merge their states.  (16 ragged sequences up to 16K in
// int8: 69.3 us with 0, 65.3 with 3, 62.5 with 6; equal lengths do not care.)
constexpr int kUnitCost = 6;
// What a block's second end costs against parts that are shorter by so many
// stages.  (Lists and contexts of one length: equal parts are 4 to 20% faster below
// 37 stages a unit's idle share, 5% slower at 46 in int4; measured for 40 to 144 units,
// taken for any number.)
constexpr float kEndCost = 36.f;

// A sequence as the kernel walks it: its length, the first attended position,
// its first stage and its number of stages (the same for every KV head).
struct Seq {
  int n, lo, first, stages;
  // cost of each of its units, the fixed part first
  __device__ __forceinline__ int cost(int fixed) const { return stages > 0 ? stages + fixed : 0; }
};
__device__ __forceinline__ Seq seq_of(const KvDecodeParams& p, int b) {
  Seq s;
  const int most = p.max_pages * p.page_size;
  s.n = min(max(p.seq_lens[b], 0), most);
  s.lo = p.window > 0 ? max(0, s.n - p.window) : 0;
  if (p.selected) {
    s.first = 0;
    s.stages = s.n > 0 ? (p.k * p.page_size + kStageTok - 1) / kStageTok : 0;
  } else {
    s.first = s.lo / kStageTok;
    s.stages = (s.n + kStageTok - 1) / kStageTok - s.first;
  }
  return s;
}

// Outputs of the sequences with nothing to attend, this block's share of them (one warp).
__device__ __forceinline__ void zero_empty(const KvDecodeParams& p, int lane) {
  const size_t rows = size_t(p.n_kv_heads) * p.group;
  for (int b = blockIdx.x; b < p.batch; b += gridDim.x) {
    if (seq_of(p, b).stages > 0) continue;
    const size_t row0 = b * rows;
    for (size_t i = lane; i < rows * (kHeadDim / 8); i += 32)
      reinterpret_cast<uint4*>(p.out + row0 * kHeadDim)[i] = make_uint4(0, 0, 0, 0);
    if (p.out_lse)
      for (size_t i = lane; i < rows; i += 32) p.out_lse[row0 + i] = -INFINITY;
  }
}

// x / y for 0 <= x < 2^19, y > 0, in floats: half a step off the borders, where
// the approximate quotient is certain
__device__ __forceinline__ int small_div(int x, int y) {
  return int(__fdividef(float(x) + 0.5f, float(y)));
}

// The block whose share [W c / N, W (c + 1) / N) holds x < W: the largest c with
// W c <= (x + 1) N - 1.  The float quotient (N <= 152) is off by less than one,
// and is put right in integers; a 64-bit division takes about a thousand cycles.
__device__ __forceinline__ int block_of(int x, int N, int W) {
  const int64_t most = int64_t(x + 1) * N - 1;
  int c = int(__fdividef(float(most), float(W)));
  if (int64_t(W) * c > most) --c;
  if (int64_t(W) * (c + 1) <= most) ++c;
  return c;
}

// The unit after (b, h), which starts at u in the list.  Shares end where the list
// does, so there is one; should the lengths change under the call, the walk still
// ends with the batch.
__device__ __forceinline__ void next_unit(const KvDecodeParams& p, int& b, Seq& sq, int& h, int& u,
                                          int end, int fixed) {
  u += sq.cost(fixed);
  if (++h < p.n_kv_heads || u >= end) return;     // (beyond `end` there may be no sequence)
  h = 0;
  ++b;
  while (b < p.batch && p.seq_lens[b] <= 0) ++b;
  if (b < p.batch) sq = seq_of(p, b);
  else u = end;
}

// A unit's query for heads h0 .. h0 + 7 (lane 4g + t: head h0 + g, dims 32t ..
// 32t + 31): brought to a largest magnitude in [2^14, 2^15) by a power of two,
// rounded to f16 (exact but for elements below 2^-28 of it) and laid out as the
// second operand of the eight k-steps.
__device__ __forceinline__ void load_query(const KvDecodeParams& p, int unit, int h0, int lane,
                                           uint4 (&raw)[4]) {
  const int head = h0 + (lane >> 2), t = lane & 3;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    raw[i] = make_uint4(0, 0, 0, 0);
    if (head < p.group)
      raw[i] = *reinterpret_cast<const uint4*>(p.q + (size_t(unit) * p.group + head) * kHeadDim +
                                               32 * t + 8 * i);
  }
}
template <int FMT>
__device__ __forceinline__ void put_query(const uint4 (&raw)[4], int h0, int lane, uint4 (*to)[32],
                                          float* scale) {
  const int head = h0 + (lane >> 2), t = lane & 3;
  uint32_t mx = 0;                                // largest magnitude, as bf16 bits
#pragma unroll
  for (int i = 0; i < 4; ++i)
    mx = __vmaxu2(__vmaxu2(__vmaxu2(raw[i].x & 0x7fff7fffu, raw[i].y & 0x7fff7fffu),
                           __vmaxu2(raw[i].z & 0x7fff7fffu, raw[i].w & 0x7fff7fffu)), mx);
  mx = max(mx & 0xffffu, mx >> 16);
  mx = max(mx, __shfl_xor_sync(kFull, mx, 1));
  mx = max(mx, __shfl_xor_sync(kFull, mx, 2));
  const int ex = int(mx >> 7);                    // biased exponent
  // factor 2^(14 - (ex - 127)), at most 2^126; infinities and NaN stay what they are
  const int up = ex == 255 ? 0 : min(126, 141 - ex);
  const float f = __uint_as_float(uint32_t(127 + up) << 23);
  constexpr float kScale = 0.08838834764831845f * kLog2e * (FMT == LOCKS_KV_I4 ? 256.f : 1.f);
  if (t == 0) scale[head] = __uint_as_float(uint32_t(127 - up) << 23) * kScale;
#pragma unroll
  for (int w = 0; w < 4; ++w) {                   // k-steps 2w, 2w + 1: dims 8w .. 8w + 7 of the lane's
    const float x0 = bf16_lo(raw[w].x) * f, x1 = bf16_hi(raw[w].x) * f;
    const float x2 = bf16_lo(raw[w].y) * f, x3 = bf16_hi(raw[w].y) * f;
    const float x4 = bf16_lo(raw[w].z) * f, x5 = bf16_hi(raw[w].z) * f;
    const float x6 = bf16_lo(raw[w].w) * f, x7 = bf16_hi(raw[w].w) * f;
    // 4 bits: nibbles (n, n + 4) of word w; 8 bits: bytes (0, 1), (2, 3) of words 2w, 2w + 1
    to[w][lane] = FMT == LOCKS_KV_I4
                      ? make_uint4(f16x2(x0, x4), f16x2(x1, x5), f16x2(x2, x6), f16x2(x3, x7))
                      : make_uint4(f16x2(x0, x1), f16x2(x2, x3), f16x2(x4, x5), f16x2(x6, x7));
  }
}

__device__ __forceinline__ int ticket_add(int* t) {
  int old;
  asm volatile("atom.add.acq_rel.gpu.global.s32 %0, [%1], 1;" : "=r"(old) : "l"(t) : "memory");
  return old;
}

// Two dims of an output row from sum p v, the reference and sum p.
__device__ __forceinline__ void store_out(const KvDecodeParams& p, size_t row, int dim, float2 A,
                                          float M, float L) {
  const float inv = L != 0.f ? 1.f / L : 0.f;
  *reinterpret_cast<__nv_bfloat162*>(p.out + row * kHeadDim + dim) =
      __floats2bfloat162_rn(A.x * inv, A.y * inv);
  if (p.out_lse && dim == 0) p.out_lse[row] = L != 0.f ? M * kLn2 + logf(L) : -INFINITY;
}

// The partials of blocks c_lo .. c_hi of a unit, in that order, K loaded at a
// time: item x (two dims of a head) of each.  The unit starts in block c_lo,
// whose second partial it is; in the others it is the first.
template <int NT, int K>
__device__ __forceinline__ void join_partials(const float* parts, int c_lo, int c_hi, int head, int x,
                                              float2& A, float& M, float& L) {
  for (int c = c_lo; c <= c_hi; c += K) {
    float2 ml[K], a[K];
#pragma unroll
    for (int k = 0; k < K; ++k) {
      ml[k] = make_float2(kNone, 0.f);
      a[k] = make_float2(0.f, 0.f);
      if (c + k <= c_hi) {
        const float* src = parts + (size_t(c + k) * 2 + (c + k == c_lo)) * (kv_part_bytes(NT) / 4);
        ml[k] = __ldcg(reinterpret_cast<const float2*>(src + NT * 1024 + 2 * head));
        a[k] = __ldcg(reinterpret_cast<const float2*>(src) + x);
      }
    }
    float Mn = M;
#pragma unroll
    for (int k = 0; k < K; ++k) Mn = fmaxf(Mn, ml[k].x);
    const float f0 = ex2_approx(M - Mn);
    L *= f0;
    A.x *= f0;
    A.y *= f0;
    M = Mn;
#pragma unroll
    for (int k = 0; k < K; ++k) {
      const float f = ex2_approx(ml[k].x - Mn);
      L += ml[k].y * f;
      A.x += a[k].x * f;
      A.y += a[k].y * f;
    }
  }
}

template <int FMT, int NT>
__global__ void __launch_bounds__(kv_threads(NT), 1) kv_decode_kernel(const KvDecodeParams p) {
  constexpr int STAGES = kv_stages(FMT, NT);
  constexpr int C = kv_chunks(FMT, NT), JOBS = 4 / C;   // chunks of a job, jobs of a stage
  constexpr int kStageBytes = kv_stage_bytes(FMT);
  constexpr int kKvWarps = kv_warps(NT), kCopiers = kv_copiers(NT);
  constexpr int kItems = (512 + kKvWarps * 32 - 1) / (kKvWarps * 32);   // float2 items of 8 heads a thread
  extern __shared__ __align__(1024) unsigned char smem[];
  unsigned char* ring = smem;
  float4* mbuf = reinterpret_cast<float4*>(smem + STAGES * kStageBytes);    // [warp][8][32]
  __shared__ uint64_t s_full[STAGES], s_empty[STAGES];
  __shared__ uint2 s_chunk[4];                    // a chunk's codes and scales in a stage
  __shared__ int s_range[STAGES][4];              // valid rows of each 16-token chunk: lo | hi << 8
  // of this unit and the next: query operands of the k-steps, and what brings their
  // products to log2 units
  __shared__ uint4 s_q[2][NT][4][32];
  __shared__ float s_qs[2][8 * NT];
  __shared__ uint64_t s_qfull[2], s_qempty[2];
  __shared__ __align__(16) float s_m[kKvWarps][8 * NT], s_l[kKvWarps][8 * NT];   // of each warp's state
  __shared__ float s_ref[8 * NT];                 // their largest m
  __shared__ int2 s_join;                         // blocks whose partials this block merges

  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int B = p.page_size, pps = kStageTok / B, hk = p.n_kv_heads;
  if (tid == 0) {
    for (int s = 0; s < STAGES; ++s) {
      mbar_init(s_full + s, 1);
      mbar_init(s_empty + s, JOBS);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(s_qfull + i, NT);
      mbar_init(s_qempty + i, kKvWarps);
    }
    mbar_fence_init();
  }
  if (tid < 4) {
    const int e = 16 * tid / B, r0 = 16 * tid - e * B;
    s_chunk[tid] = make_uint2(e * uint32_t(kv_rec_bytes(FMT, B)) + r0 * kv_row_bytes(FMT),
                              e * uint32_t(kv_rec_bytes(FMT, B)) + 4 * r0);
  }
  __syncthreads();
  griddep_launch();
  griddep_wait();

  // ---- this block's share of the units' cost, which every warp works out for itself ----
  const int per = (p.batch + 31) / 32;
  const int b_lo = min(p.batch, lane * per), b_hi = min(p.batch, b_lo + per);
  int stages = 0, units = 0, least = 0x7fffffff, most = 0;   // of this lane's sequences; units: with stages
#pragma unroll 4
  for (int i = b_lo; i < b_hi; ++i) {
    const int n = seq_of(p, i).stages;
    stages += n;
    units += n > 0;
    least = min(least, n > 0 ? n : least);
    most = max(most, n);
  }
  least = __reduce_min_sync(kFull, least);
  most = __reduce_max_sync(kFull, most);
  int stages_to = stages, units_to = units;       // up to and with this lane
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int x = __shfl_up_sync(kFull, stages_to, o), y = __shfl_up_sync(kFull, units_to, o);
    if (lane >= o) {
      stages_to += x;
      units_to += y;
    }
  }
  const int all_stages = __shfl_sync(kFull, stages_to, 31) * hk;   // below 2^31: the host has checked
  const int all_units = __shfl_sync(kFull, units_to, 31) * hk;
  // Units of one length that m blocks each come close to filling the SMs: equal
  // parts, no block with two units' ends (64 lists of 32 pages in int4: 16.1 -> 13.7
  // us with 128 blocks).  Taken when a part's extra stages cost less than the second
  // end that a block has on average otherwise.
  int m = least == most ? min(small_div(kSms, all_units), most) : 0;
  if (float(most) * float(kSms - m * all_units) > kEndCost * float(m * all_units)) m = 0;
  const int fixed = m ? 0 : kUnitCost;
  const int W = all_stages + fixed * all_units;
  // blocks with a share: none when every sequence is empty (W = 0)
  const int N = m ? m * all_units : min(kSms, W);
  int w_lo = 0, w_hi = 0;
  if (int(blockIdx.x) < N) {
    if (m) {
      const int unit = small_div(blockIdx.x, m), part = int(blockIdx.x) - unit * m;
      // most = each * m + rest, with an `each` a little below the quotient (the float one is
      // within 2^-22 of it): 0 <= rest < 16 m
      const int each = max(int(__fdividef(float(most), float(m)) * (1.f - 4.8e-7f)) - 1, 0);
      const int rest = most - each * m;
      w_lo = unit * most + part * each + small_div(part * rest, m);
      w_hi = unit * most + (part + 1) * each + small_div((part + 1) * rest, m);
    } else if (N == kSms) {                       // W c / kSms
      const unsigned c = blockIdx.x, each = unsigned(W) / kSms, rest = unsigned(W) % kSms;
      w_lo = each * c + rest * c / kSms;
      w_hi = each * (c + 1) + rest * (c + 1) / kSms;
    } else {
      w_lo = blockIdx.x;                          // W = N
      w_hi = blockIdx.x + 1;
    }
  }
  // the sequence of w_lo and where it starts in the list
  int b = b_lo, u = (stages_to - stages + fixed * (units_to - units)) * hk;
  const bool here = u <= w_lo && w_lo < (stages_to + fixed * units_to) * hk;
  if (here) {
    for (int c; u + (c = seq_of(p, b).cost(fixed) * hk) <= w_lo; ++b) u += c;
  }
  const int who = __ffs(__ballot_sync(kFull, here)) - 1;
  b = __shfl_sync(kFull, b, max(who, 0));
  u = __shfl_sync(kFull, u, max(who, 0));
  if (blockIdx.x == 0 && warp == 0)
    for (int i = b_lo; i < b_hi; ++i)
      if (p.seq_lens[i] < 0 || p.seq_lens[i] > p.max_pages * B) flag_status(p.status, LOCKS_DEV_BAD_SEQ_LEN);
  if (w_lo >= w_hi) {
    if (warp == 0) zero_empty(p, lane);
    return;
  }

  const size_t rec = size_t(kv_rec_bytes(FMT, B));
  Seq sq = seq_of(p, b);
  int h = (w_lo - u) / sq.cost(fixed);
  u += h * sq.cost(fixed);                             // where unit (b, h) starts in the list
  int it = 0;                                     // stages of this block so far

  if (warp >= kKvWarps) {
    // ---------------- producer ----------------
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kv_producer_regs(NT)));
    const uint64_t pol = l2_evict_first();
    const int pw = warp - kKvWarps;
    const int e = lane & (pps - 1), mine = lane / pps;   // this lane's page of a stage, and its stage
    const int cpp = B / 16;                       // chunks of a page
    const int looked = 32 / pps;                  // stages looked up at a time
    int s = pw, phase = 1;                        // ring slot of the warp's next stage; nothing to wait for yet
    bool ok = true;
    for (int seg = 0; ok; next_unit(p, b, sq, h, u, w_hi, fixed)) {
      if (u >= w_hi) break;
      const int i0 = max(0, w_lo - u - fixed);
      const int cnt = min(sq.stages, w_hi - u - fixed) - i0;
      if (cnt <= 0) continue;
      // the last warps also bring the unit's query, whose loads are on their way
      // while the first pages are looked up
      bool bring = pw >= 4 - NT;
      uint4 raw[4];
      if (bring) load_query(p, b * hk + h, 8 * (pw - (4 - NT)), lane, raw);
      const auto bring_query = [&] {
        const int n = pw - (4 - NT);
        bring = false;
        if (!__all_sync(kFull, mbar_wait_bounded(s_qempty + (seg & 1), ((seg >> 1) & 1) ^ 1))) {
          if (lane == 0) flag_status(p.status, LOCKS_DEV_WAIT_TIMEOUT);
          ok = false;
          return;
        }
        put_query<FMT>(raw, 8 * n, lane, s_q[seg & 1][n], s_qs[seg & 1]);
        __syncwarp();
        if (lane == 0) mbar_arrive(s_qfull + (seg & 1));
      };
      const int32_t* row = p.block_table + size_t(b) * p.max_pages;
      const int32_t* sel = p.selected ? p.selected + (size_t(b) * hk + h) * p.k : nullptr;
      const int pages = (sq.n + B - 1) / B;
      // this warp's stages of the segment: those whose number in the block is pw mod kCopiers
      const int first = pw < kCopiers ? (pw + kCopiers - it % kCopiers) % kCopiers : cnt;
      for (int s0 = first; s0 < cnt && ok; s0 += kCopiers * looked) {
        const int st = s0 + kCopiers * mine;
        int blk = -1, r_lo = 0, r_hi = 0;
        if (st < cnt) {
          const int slot = (sq.first + i0 + st) * pps + e;
          int j = slot;
          if (sel) j = slot < p.k ? sel[slot] : -1;
          if (j >= pages) {
            if (sel) flag_status(p.status, LOCKS_DEV_BAD_PAGE_ID);
            j = -1;
          }
          if (j >= 0) {
            blk = row[j];
            if (blk < 0 || blk >= p.num_blocks) {
              flag_status(p.status, LOCKS_DEV_BAD_BLOCK_ID);
              blk = -1;
            } else {
              r_lo = max(0, sq.lo - j * B);
              r_hi = min(B, sq.n - j * B);
              if (r_lo >= r_hi) blk = -1;         // before the window
            }
          }
          if (blk < 0) r_lo = r_hi = 0;
        }
        const size_t src = (size_t(max(blk, 0)) * hk + h) * rec;
        const unsigned char *ksrc = p.k_pool + src, *vsrc = p.v_pool + src;
        int range[4];
#pragma unroll
        for (int c = 0; c < 4; ++c)
          range[c] = min(16, max(0, r_lo - 16 * c)) | (min(16, max(0, r_hi - 16 * c)) << 8);
        const unsigned live = __ballot_sync(kFull, blk >= 0);
        if (bring) bring_query();
        const int todo = min(looked, (cnt - s0 + kCopiers - 1) / kCopiers);
        for (int x = 0; x < todo; ++x) {
          if (!mbar_wait_bounded(s_empty + s, phase)) ok = false;
          if (!__all_sync(kFull, ok)) {
            if (lane == 0) flag_status(p.status, LOCKS_DEV_WAIT_TIMEOUT);
            ok = false;
            break;
          }
          if (mine == x) {
            int* r = s_range[s] + e * cpp;
            r[0] = range[0];
            if (cpp > 1) r[1] = range[1];
            if (cpp > 2) {
              r[2] = range[2];
              r[3] = range[3];
            }
          }
          __syncwarp();
          if (lane == 0) {
            const int n = __popc((live >> (x * pps)) & ((1u << pps) - 1));
            if (n) mbar_arrive_expect_tx(s_full + s, uint32_t(n * 2 * rec));
            else mbar_arrive(s_full + s);
          }
          __syncwarp();
          if (mine == x && blk >= 0) {
            unsigned char* dst = ring + s * kStageBytes + e * rec;
            bulk_g2s_hint(dst, ksrc, uint32_t(rec), s_full + s, pol);
            bulk_g2s_hint(dst + kStageBytes / 2, vsrc, uint32_t(rec), s_full + s, pol);
          }
          s += kCopiers;
          if (s >= STAGES) {
            s -= STAGES;
            phase ^= 1;
          }
        }
      }
      if (bring) bring_query();                   // (no stage of the segment was this warp's)
      it += cnt;
      ++seg;
    }
    if (pw == 0) zero_empty(p, lane);
    return;
  }

  // ---------------- consumers ----------------
  asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kv_consumer_regs(NT)));
  const int g = lane >> 2, t = lane & 3, G = p.group;
  const LaneOff off = lane_off<FMT>(B, g, t);
  const uint32_t ring_at = smem_u32(ring);
  bool ok = true;
  // jobs of C 16-token chunks go round the warps: job `job` of this block, in ring slot s
  int job = warp, s = warp / JOBS, phase = 0;
  while (s >= STAGES) {
    s -= STAGES;
    phase ^= 1;
  }
  for (int seg = 0; u < w_hi; next_unit(p, b, sq, h, u, w_hi, fixed)) {
    const int i0 = max(0, w_lo - u - fixed);
    const int cnt = min(sq.stages, w_hi - u - fixed) - i0;
    if (cnt <= 0) continue;
    const int unit = b * hk + h;
    if (ok && !__all_sync(kFull, mbar_wait_bounded(s_qfull + (seg & 1), (seg >> 1) & 1))) {
      if (lane == 0) flag_status(p.status, LOCKS_DEV_WAIT_TIMEOUT);
      ok = false;
    }
    const uint32_t q_at = smem_u32(s_q[seg & 1]) + 16 * lane;
    float qs[2 * NT];
#pragma unroll
    for (int j = 0; j < 2 * NT; ++j) qs[j] = s_qs[seg & 1][8 * (j >> 1) + 2 * t + (j & 1)];
    State<NT> st;
#pragma unroll
    for (int j = 0; j < 2 * NT; ++j) {
      st.m[j] = kNone;
      st.l[j] = st.f[j] = 0.f;
    }
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int i = 0; i < 8; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e) st.acc[n][i][e] = 0.f;

    it += cnt;
    for (; job / JOBS < it; job += kKvWarps) {
      const int c0 = job % JOBS * C;
      if (ok && !__all_sync(kFull, mbar_wait_bounded(s_full + s, phase))) {
        if (lane == 0) flag_status(p.status, LOCKS_DEV_WAIT_TIMEOUT);
        ok = false;                               // the rest counts as empty: tickets stay right
      }
      if (ok) {
        uint32_t base[C], sbase[C];
        int range[C];
        bool any = false;
#pragma unroll
        for (int c = 0; c < C; ++c) {
          const uint2 at = s_chunk[c0 + c];
          base[c] = ring_at + s * kStageBytes + at.x;
          sbase[c] = ring_at + s * kStageBytes + at.y;
          range[c] = s_range[s][c0 + c];
          any |= (range[c] >> 8) > (range[c] & 255);
        }
        if (any) attend<FMT, NT, C>(base, sbase, range, off, g, t, q_at, qs, st);
        __syncwarp();
        if (lane == 0) mbar_arrive(s_empty + s);
      }
      s += (job + kKvWarps) / JOBS - job / JOBS;
      if (s >= STAGES) {
        s -= STAGES;
        phase ^= 1;
      }
    }

    // ---- merge the warps' states; finish the unit or leave a partial ----
    const int u_lo = u + fixed, u_hi = u_lo + sq.stages;     // its stages in the list
    const bool alone = u_lo >= w_lo && u_hi <= w_hi;
    float* parts = reinterpret_cast<float*>(p.ws + kTicketBytes);
    // a block's first partial goes on with an earlier block's unit, its second begins one
    float* part = parts + (size_t(blockIdx.x) * 2 + (u_lo >= w_lo)) * (kv_part_bytes(NT) / 4);
    __syncwarp();
    if (lane == 0) mbar_arrive(s_qempty + (seg & 1));
    // every warp brings its sums to the block's reference M, then they are added up item by item
    if (g == 0) {
#pragma unroll
      for (int j = 0; j < 2 * NT; ++j) s_m[warp][8 * (j >> 1) + 2 * t + (j & 1)] = st.m[j];
    }
    consumers_sync<NT>();                         // (and the buffer's last readers are done)
    if (!alone && tid == 0)                       // the blocks of the unit's first and last stage
      s_join = m ? make_int2(u / most * m, u / most * m + m - 1)
                 : make_int2(block_of(u_lo, N, W), block_of(u_hi - 1, N, W));
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      float2 M = make_float2(kNone, kNone);
#pragma unroll
      for (int w = 0; w < kKvWarps; ++w) {
        const float2 m = *reinterpret_cast<const float2*>(&s_m[w][8 * n + 2 * t]);
        M.x = fmaxf(M.x, m.x);
        M.y = fmaxf(M.y, m.y);
      }
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int j = 2 * n + e;
        const float a = ex2_approx(st.m[j] - (e ? M.y : M.x));
        const float f = st.f[j] > 0.f ? __fdividef(a * (FMT == LOCKS_KV_I4 ? 256.f : 1.f), st.f[j]) : 0.f;
        float l = st.l[j] * a;
#pragma unroll
        for (int o = 4; o < 32; o <<= 1) l += __shfl_xor_sync(kFull, l, o);
        if (g == 0) {
          s_l[warp][8 * n + 2 * t + e] = l;
          if (warp == 0) s_ref[8 * n + 2 * t + e] = e ? M.y : M.x;
        }
        // float4 x of a lane: head parity e = x / 4, dims 4 (x % 4) .. + 3 of its 16
#pragma unroll
        for (int x = 0; x < 4; ++x)
          mbuf[warp * 256 + (4 * e + x) * 32 + lane] =
              make_float4(st.acc[n][2 * x][e] * f, st.acc[n][2 * x][2 + e] * f,
                          st.acc[n][2 * x + 1][e] * f, st.acc[n][2 * x + 1][2 + e] * f);
      }
      consumers_sync<NT>();
      // a thread's items: float2 pairs of the 1024 floats, as the lanes laid them out
#pragma unroll
      for (int i = 0; i < kItems; ++i) {
        const int x = i * kKvWarps * 32 + tid;
        if (512 % (kKvWarps * 32) != 0 && x >= 512) break;
        const int q4 = x >> 6, l2 = (x >> 1) & 31;
        const int head = 8 * n + 2 * (l2 & 3) + (q4 >> 2);
        const int dim = 16 * (l2 >> 2) + 4 * (q4 & 3) + 2 * (x & 1);
        const float M = s_ref[head];
        float L = 0.f;
        float2 A = make_float2(0.f, 0.f);
#pragma unroll
        for (int w = 0; w < kKvWarps; ++w) {
          const float2 a = reinterpret_cast<const float2*>(mbuf + w * 256)[x];
          L += s_l[w][head];
          A.x += a.x;
          A.y += a.y;
        }
        if (alone) {
          if (head < G) store_out(p, size_t(unit) * G + head, dim, A, M, L);
        } else {
          reinterpret_cast<float2*>(part)[n * 512 + x] = A;
          if (dim == 0) *reinterpret_cast<float2*>(part + NT * 1024 + 2 * head) = make_float2(M, L);
        }
      }
      if (n + 1 < NT) consumers_sync<NT>();
    }
    if (!alone) {
      consumers_sync<NT>();
      if (tid == 0) {
        // at most one unit begins in a block and goes on beyond it: its ticket is that block's.
        // Releases this block's partial (ordered before by the barrier), acquires the others'
        const int before = ticket_add(reinterpret_cast<int*>(p.ws) + s_join.x);
        if (before != s_join.y - s_join.x) s_join.y = -1;
      }
      consumers_sync<NT>();
      const int c_lo = s_join.x, c_hi = s_join.y;
      if (c_hi >= 0) {
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
          for (int i = 0; i < kItems; ++i) {
            const int x = i * kKvWarps * 32 + tid;
            if (512 % (kKvWarps * 32) != 0 && x >= 512) break;
            const int q4 = x >> 6, l2 = (x >> 1) & 31;
            const int head = 8 * n + 2 * (l2 & 3) + (q4 >> 2);
            const int dim = 16 * (l2 >> 2) + 4 * (q4 & 3) + 2 * (x & 1);
            float M = kNone, L = 0.f;
            float2 A = make_float2(0.f, 0.f);
            // (a unit cut in two or three is the usual case, one cut in many the latency-bound one)
            if (c_hi - c_lo < 4) join_partials<NT, 4>(parts, c_lo, c_hi, head, n * 512 + x, A, M, L);
            else join_partials<NT, 16>(parts, c_lo, c_hi, head, n * 512 + x, A, M, L);
            if (head < G) store_out(p, size_t(unit) * G + head, dim, A, M, L);
          }
        if (tid == 0) reinterpret_cast<int*>(p.ws)[c_lo] = 0;
      }
    }
    ++seg;
  }
  // a wait ran out: the copies asked for are waited for once more, until one fails again
  // (no block should leave while copies into its memory are in flight)
  if (!ok)
    for (int i = 0; i < STAGES && mbar_wait_bounded(s_full + s, phase); ++i)
      if (++s == STAGES) {
        s = 0;
        phase ^= 1;
      }
}

template <int FMT, int NT>
int launch_nt(const KvDecodeParams& p, cudaStream_t stream) {
  constexpr size_t smem = size_t(kv_stages(FMT, NT)) * kv_stage_bytes(FMT) + kv_merge_bytes(NT);
  static LaunchOnce once;
  if (!once.run([] {
        return cudaFuncSetAttribute(kv_decode_kernel<FMT, NT>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                    int(smem)) == cudaSuccess;
      }))
    return LOCKS_ERR_CUDA;
  return launch_dependent(kv_decode_kernel<FMT, NT>, dim3(kSms), kv_threads(NT), smem, p, stream);
}

template <int FMT>
int launch_fmt(const KvDecodeParams& p, cudaStream_t stream) {
  return p.group <= 8 ? launch_nt<FMT, 1>(p, stream) : launch_nt<FMT, 2>(p, stream);
}

}  // namespace

size_t kv_decode_workspace(int group) {
  return kTicketBytes + size_t(kSms) * 2 * kv_part_bytes(group <= 8 ? 1 : 2);
}

int launch_kv_decode(const KvDecodeParams& p, int fmt, cudaStream_t stream) {
  switch (fmt) {
    case LOCKS_KV_F8: return launch_fmt<LOCKS_KV_F8>(p, stream);
    case LOCKS_KV_I8: return launch_fmt<LOCKS_KV_I8>(p, stream);
    case LOCKS_KV_I4: return launch_fmt<LOCKS_KV_I4>(p, stream);
    default: return LOCKS_ERR_INVALID_ARG;
  }
}

}  // namespace locks
