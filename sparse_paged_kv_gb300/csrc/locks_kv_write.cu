// locks_kv_write and locks_kv_read: tokens into a quantised paged cache, with
// the rotation of their queries and keys, and pages back out of it.
//
// Both move every byte once.  Measured (one GB300, 32 / 8 heads, e4m3, half
// layout): 8192 tokens written in 35 us (5.3 TB/s of 6.78 copy; the blocks of a
// wave load and compute in step), read back in 10 us (issue slots); 5001 tokens in
// int4 written in 24 us and read back in 8; 16 tokens of a decode step in 7 us
// (latency).  Half a warp (16 lanes of 8 dims) owns a row of 128 dims: its largest
// magnitude is four shuffles, a group of 32 dims is four lanes, and its codes
// leave as one 128-byte (or 64-byte) line.
//
// Write: a block takes a few tokens and a run of their rows (queries, then keys,
// then values).  One thread asks for all of them (cp.async.bulk: a token's heads
// are contiguous), so that 50 KB a block are on their way at once and no register
// waits for them; meanwhile the tokens' cos and sin are computed once, one pair a
// thread.  Then every half-warp takes rows in turn; in the half layout it reads a
// lane's partner elements (dims +- r/2) from shared memory a second time, which
// keeps every lane's 8 dims contiguous for the codes.
#include "locks_kv.cuh"

namespace locks {

namespace {

constexpr int kWriteThreads = 256;
constexpr int kHalfWarps = kWriteThreads / 16;
constexpr int kMaxWriteSmem = 52 * 1024;              // of rows a block: four blocks an SM

__device__ __forceinline__ void unpack8(const uint4& w, float (&x)[8]) {
  x[0] = bf16_lo(w.x); x[1] = bf16_hi(w.x);
  x[2] = bf16_lo(w.y); x[3] = bf16_hi(w.y);
  x[4] = bf16_lo(w.z); x[5] = bf16_hi(w.z);
  x[6] = bf16_lo(w.w); x[7] = bf16_hi(w.w);
}
__device__ __forceinline__ uint32_t bf16x2(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
// two float32 sums, each rounded to nearest
__device__ __forceinline__ float2 fadd2(float2 a, float2 b) {
  unsigned long long r;
  asm("add.rn.f32x2 %0, %1, %2;"
      : "=l"(r)
      : "l"(*reinterpret_cast<unsigned long long*>(&a)), "l"(*reinterpret_cast<unsigned long long*>(&b)));
  return *reinterpret_cast<float2*>(&r);
}
__device__ __forceinline__ uint4 pack8(const float (&x)[8]) {
  return make_uint4(bf16x2(x[0], x[1]), bf16x2(x[2], x[3]), bf16x2(x[4], x[5]), bf16x2(x[6], x[7]));
}

// largest of magnitudes, a NaN if there is one
__device__ __forceinline__ float max_abs(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(fabsf(a)), "f"(fabsf(b)));
  return r;
}
__device__ __forceinline__ float magnitude(const float (&x)[8]) {
  return max_abs(max_abs(max_abs(x[0], x[1]), max_abs(x[2], x[3])),
                 max_abs(max_abs(x[4], x[5]), max_abs(x[6], x[7])));
}

// rint(y) + k in the low bits of the result, for |y| + k < 2^22: the sum with
// 1.5 * 2^23 has a unit of 1, and rounds ties to even as rint does (k even).
// (A conversion to an integer runs at a quarter of an addition's rate.)
__device__ __forceinline__ uint32_t round_bits(float y, float k) {
  return __float_as_uint(__fadd_rn(y, 12582912.f + k));
}
__device__ __forceinline__ float round_float(float y) {
  return __fadd_rn(__fadd_rn(y, 12582912.f), -12582912.f);
}

// N rows (8 dims a lane each) quantised into row `r` of their records.  Every
// lane of the warp calls it; `live` says whether this half-warp's row is stored.
// The rows go side by side through each step, whose latencies then overlap.
template <int FMT, int N>
__device__ __forceinline__ void store_rows(const float (&x)[N][8], unsigned char* const (&rec)[N], int r,
                                           int B, int l16, const bool (&live)[N]) {
  float m[N], y[N][8];
#pragma unroll
  for (int n = 0; n < N; ++n) m[n] = magnitude(x[n]);
#pragma unroll
  for (int o = 8; o; o >>= 1)
#pragma unroll
    for (int n = 0; n < N; ++n) m[n] = max_abs(m[n], __shfl_xor_sync(kFull, m[n], o));
  constexpr float kInvTop = FMT == LOCKS_KV_F8 ? float(1.0 / 448.0)
                            : FMT == LOCKS_KV_I8 ? float(1.0 / 127.0)
                                                 : float(1.0 / (7.0 * 448.0));
#pragma unroll
  for (int n = 0; n < N; ++n) {
    const bool odd = !(m[n] <= 3.402823466e38f);      // an infinity or a NaN in the row
    const bool dead = odd || m[n] < kKvTiny;
    const float scale = __fmul_rn(m[n], kInvTop);
    const float inv = __frcp_rn(scale);
#pragma unroll
    for (int i = 0; i < 8; i += 2) {
      const float2 t = fmul2(make_float2(x[n][i], x[n][i + 1]), make_float2(inv, inv));
      y[n][i] = t.x;
      y[n][i + 1] = t.y;
    }
    if (dead) {                                       // (rare)
#pragma unroll
      for (int i = 0; i < 8; ++i) y[n][i] = 0.f;
    }
    if (live[n] && l16 == 0)
      *reinterpret_cast<float*>(rec[n] + kv_scale_off(FMT, B) + 4 * r) =
          odd ? __int_as_float(0x7fffffff) : (dead ? 0.f : scale);
  }
  if constexpr (FMT == LOCKS_KV_I4) {
    float gm[N];
#pragma unroll
    for (int n = 0; n < N; ++n) gm[n] = magnitude(y[n]);
#pragma unroll
    for (int o = 2; o; o >>= 1)                       // dims 32j .. 32j + 31
#pragma unroll
      for (int n = 0; n < N; ++n) gm[n] = max_abs(gm[n], __shfl_xor_sync(kFull, gm[n], o));
#pragma unroll
    for (int n = 0; n < N; ++n) {
      const uint32_t gbits = e4m3x2(__fmul_rn(gm[n], float(1.0 / 7.0)), 0.f) & 0xff;
      const float g = e4m3x2_to_f2(gbits).x;
      const float ginv = g > 0.f ? __frcp_rn(g) : 0.f;
      float c[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) c[i] = __fmul_rn(y[n][i], ginv);
      // e4m3 rounds a normal scale down by at most 2^-4, which leaves 7 * 16 / 15 < 7.5;
      // only below its normal range can a code pass 7
      if (gbits < 8) {
#pragma unroll
        for (int i = 0; i < 8; ++i) c[i] = fminf(7.f, fmaxf(-7.f, c[i]));
      }
#pragma unroll
      for (int i = 0; i < 8; ++i) c[i] = round_float(c[i]);
      // four codes + 8 as hexadecimal digits of an exact float sum (0x8888 = 34952)
      float lo = fmaf(fmaf(fmaf(c[3], 16.f, c[2]), 16.f, c[1]), 16.f, c[0]);
      float hi = fmaf(fmaf(fmaf(c[7], 16.f, c[6]), 16.f, c[5]), 16.f, c[4]);
      const uint32_t w = __byte_perm(round_bits(lo, 34952.f), round_bits(hi, 34952.f), 0x5410);
      if (live[n]) {
        *reinterpret_cast<uint32_t*>(rec[n] + kv_chunk_off<FMT>(r, l16 >> 2) + 4 * (l16 & 3)) = w;
        if ((l16 & 3) == 0) rec[n][kv_group_off(FMT, B) + 4 * r + (l16 >> 2)] = (unsigned char)gbits;
      }
    }
  } else {
#pragma unroll
    for (int n = 0; n < N; ++n) {
      uint2 w;
      if constexpr (FMT == LOCKS_KV_F8) {
        w.x = e4m3x2(y[n][0], y[n][1]) | (e4m3x2(y[n][2], y[n][3]) << 16);
        w.y = e4m3x2(y[n][4], y[n][5]) | (e4m3x2(y[n][6], y[n][7]) << 16);
      } else {
        // |y| <= 127 (1 + 2^-22): codes + 128 are bytes
        uint32_t c[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) c[i] = round_bits(y[n][i], 128.f);
        w.x = __byte_perm(__byte_perm(c[0], c[1], 0x0040), __byte_perm(c[2], c[3], 0x0040), 0x5410);
        w.y = __byte_perm(__byte_perm(c[4], c[5], 0x0040), __byte_perm(c[6], c[7], 0x0040), 0x5410);
      }
      if (live[n])
        *reinterpret_cast<uint2*>(rec[n] + kv_chunk_off<FMT>(r, l16 >> 1) + 8 * (l16 & 1)) = w;
    }
  }
}

enum { kNoTurn = 0, kHalf = 1, kInterleaved = 2 };

// What a lane needs to rotate its 8 dims: cos and sin of its pairs (in the half
// layout the sine's sign says which of a pair its dims are).
struct Turn {
  float c[8], s[8];
  bool on;                                            // its dims are rotated ones
};

// `table`: cos and sin of the token's pairs
template <int LAYOUT>
__device__ __forceinline__ Turn make_turn(const float2* table, int rot, int e0) {
  Turn t;
  t.on = LAYOUT != kNoTurn && e0 < rot;
  if (t.on) {
    if constexpr (LAYOUT == kHalf) {
      const bool second = e0 >= rot / 2;
      const float2* at = table + (second ? e0 - rot / 2 : e0);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        t.c[i] = at[i].x;
        t.s[i] = second ? at[i].y : -at[i].y;
      }
    } else if constexpr (LAYOUT == kInterleaved) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        t.c[i] = table[e0 / 2 + i].x;
        t.s[i] = table[e0 / 2 + i].y;
      }
    }
  }
  return t;
}

// first dim of the other elements of a lane's pairs (half layout)
template <int LAYOUT>
__device__ __forceinline__ int partner_dim(int rot, int e0) {
  return LAYOUT != kHalf || e0 >= rot ? e0 : (e0 >= rot / 2 ? e0 - rot / 2 : e0 + rot / 2);
}

// own and other: this lane's 8 elements and (half layout) their partners
template <int LAYOUT>
__device__ __forceinline__ void rotate8(float (&x)[8], const uint4& own, const uint4& other,
                                        const Turn& t) {
  unpack8(own, x);
  if constexpr (LAYOUT == kHalf) {
    float z[8];
    unpack8(other, z);
    if (t.on) {
#pragma unroll
      for (int i = 0; i < 8; i += 2) {                // u c - v s and v c + u s
        const float2 r = fadd2(fmul2(make_float2(x[i], x[i + 1]), make_float2(t.c[i], t.c[i + 1])),
                               fmul2(make_float2(z[i], z[i + 1]), make_float2(t.s[i], t.s[i + 1])));
        x[i] = r.x;
        x[i + 1] = r.y;
      }
    }
  } else if constexpr (LAYOUT == kInterleaved) {
    if (t.on) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float u = x[2 * i], v = x[2 * i + 1];
        x[2 * i] = rope_u(u, v, t.c[i], t.s[i]);
        x[2 * i + 1] = rope_v(u, v, t.c[i], t.s[i]);
      }
    }
  }
}

constexpr int kWriteWarps = kWriteThreads / 32;
constexpr int kRowBytes = kHeadDim * 2;

// TOKENS tokens a block: 8 / TOKENS warps a token
template <int FMT, int LAYOUT, int TOKENS>
__global__ void __launch_bounds__(kWriteThreads, 4) kv_write_kernel(const KvWriteParams p) {
  extern __shared__ __align__(128) unsigned char rows_in[];   // [TOKENS][run][128] bf16
  __shared__ float2 table[TOKENS][kHeadDim / 2 + 1];
  __shared__ uint64_t landed;
  constexpr int kPer = kWriteWarps / TOKENS;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int l16 = lane & 15, hw = 2 * (warp % kPer) + (lane >> 4), e0 = 8 * l16;   // hw: this half-warp of the token's
  const int group = blockIdx.x / p.n_chunks, chunk = blockIdx.x % p.n_chunks;
  // this block's run of each token's rows
  const int hq = p.q_out ? p.n_q_heads : 0, hk = p.n_kv_heads;
  const int rows = hq + 2 * hk;
  const int lo = rows * chunk / p.n_chunks, hi = rows * (chunk + 1) / p.n_chunks, run = hi - lo;
  if (threadIdx.x == 0) {
    mbar_init(&landed, 1);
    mbar_fence_init();
  }
  __syncthreads();
  griddep_launch();
  griddep_wait();
  if (threadIdx.x == 0) {
    const int n = min(TOKENS, p.n_tokens - group * TOKENS);
    mbar_arrive_expect_tx(&landed, uint32_t(n * run * kRowBytes));
    for (int t = 0; t < n; ++t) {
      const int64_t token = group * TOKENS + t;
      unsigned char* to = rows_in + t * run * kRowBytes;
      const int q_end = min(hi, hq), k_lo = max(lo, hq), k_end = min(hi, hq + hk), v_lo = max(lo, hq + hk);
      if (lo < q_end)
        bulk_g2s(to, p.q_new + token * p.q_stride + lo * kHeadDim, (q_end - lo) * kRowBytes, &landed);
      if (k_lo < k_end)
        bulk_g2s(to + (k_lo - lo) * kRowBytes, p.k_new + token * p.k_stride + (k_lo - hq) * kHeadDim,
                 (k_end - k_lo) * kRowBytes, &landed);
      if (v_lo < hi)
        bulk_g2s(to + (v_lo - lo) * kRowBytes, p.v_new + token * p.v_stride + (v_lo - hq - hk) * kHeadDim,
                 (hi - v_lo) * kRowBytes, &landed);
    }
  }
  const int rot = p.rope.rotary_dim;
  if constexpr (LAYOUT != kNoTurn) {
    for (int i = threadIdx.x; i < TOKENS * (kHeadDim / 2); i += kWriteThreads) {
      const int t = i / (kHeadDim / 2), pair = i % (kHeadDim / 2), tok = group * TOKENS + t;
      if (tok < p.n_tokens && pair < rot / 2) {
        float c, s;
        rope_cos_sin(__ldg(p.rope.turns + pair), p.token_pos[tok], p.rope.mscale, c, s);
        table[t][pair] = make_float2(c, s);
      }
    }
  }
  const int token = group * TOKENS + warp / kPer;
  const bool exists = token < p.n_tokens;
  const int seq = !exists ? -1 : (p.token_seq ? p.token_seq[token] : token);
  const int pos = exists ? p.token_pos[token] : 0;
  const int B = p.page_size, shift = __ffs(B) - 1;    // B is a power of two
  const bool first = exists && chunk == 0 && hw == 0 && l16 == 0;
  int blk = -1;
  if (seq >= 0) {
    int32_t bits = 0;
    if (seq >= p.batch) {
      bits = LOCKS_DEV_BAD_PAGE_ID;
    } else if (pos < 0 || (pos >> shift) >= p.max_pages) {
      bits = LOCKS_DEV_BAD_SEQ_LEN;
    } else {
      blk = p.block_table[size_t(seq) * p.max_pages + (pos >> shift)];
      if (blk < 0 || blk >= p.num_blocks) {
        bits = LOCKS_DEV_BAD_BLOCK_ID;
        blk = -1;
      }
    }
    if (first) {
      if (bits) flag_status(p.status, bits);
      if (p.seq_lens && blk >= 0) atomicMax(p.seq_lens + seq, pos + 1);
    }
  }
  const int slot = pos & (B - 1);
  if (first && p.completed) p.completed[token] = (blk >= 0 && slot == B - 1) ? blk : -1;

  // every thread waits (no block may end before its copies have landed)
  const bool here = mbar_wait_bounded(&landed, 0);
  if (__syncthreads_or(!here)) {
    if (threadIdx.x == 0) flag_status(p.status, LOCKS_DEV_WAIT_TIMEOUT);
    mbar_wait_bounded(&landed, 0);                    // once more, for what is still in flight
    return;
  }
  if (seq < 0) return;                                // (whole warps)
  constexpr int kStep = 2 * kPer;                     // a half-warp takes every kStep-th row
  const Turn turn = make_turn<LAYOUT>(table[warp / kPer], rot, e0);
  const unsigned char* mine = rows_in + (warp / kPer) * run * kRowBytes + e0 * 2;
  const int away = 2 * (partner_dim<LAYOUT>(rot, e0) - e0);   // bytes to the partner elements

  // queries
  {
    __nv_bfloat16* dst = p.q_out + int64_t(token) * hq * kHeadDim + e0;
    const int end = min(hi, hq);
#pragma unroll 4
    for (int r = lo + hw; r < end; r += kStep) {
      const unsigned char* at = mine + (r - lo) * kRowBytes;
      float x[8];
      rotate8<LAYOUT>(x, *reinterpret_cast<const uint4*>(at), *reinterpret_cast<const uint4*>(at + away), turn);
      *reinterpret_cast<uint4*>(dst + r * kHeadDim) = pack8(x);
    }
  }
  if (blk < 0) return;
  // keys and values, two rows at a time (the shuffles of store_rows name every
  // lane: a row past the end is not stored)
  const size_t rec_bytes = size_t(kv_rec_bytes(FMT, B));
  const size_t page = size_t(blk) * hk * rec_bytes;
  for (int r0 = max(lo, hq) + hw; r0 - (hw & 1) < hi; r0 += 2 * kStep) {
    float x[2][8];
    unsigned char* rec[2];
    bool live[2];
#pragma unroll
    for (int n = 0; n < 2; ++n) {
      const int r = min(r0 + n * kStep, hi - 1);
      live[n] = r == r0 + n * kStep;
      const unsigned char* at = mine + (r - lo) * kRowBytes;
      const uint4 own = *reinterpret_cast<const uint4*>(at);
      if (r < hq + hk) {
        rotate8<LAYOUT>(x[n], own, *reinterpret_cast<const uint4*>(at + away), turn);
        rec[n] = p.k_pool + page + (r - hq) * rec_bytes;
      } else {
        unpack8(own, x[n]);
        rec[n] = p.v_pool + page + (r - hq - hk) * rec_bytes;
      }
    }
    store_rows<FMT, 2>(x, rec, slot, B, l16, live);
  }
}

// Read: a block of 256 threads converts 64 rows of one pool (one page of 64,
// two of 32, four of 16), four rows a half-warp, all loaded before any is stored.
constexpr int kReadRows = 64;

template <int FMT>
__global__ void __launch_bounds__(kWriteThreads) kv_read_kernel(const KvReadParams p) {
  const int l16 = threadIdx.x & 15, hw = threadIdx.x >> 4;
  const bool vals = blockIdx.y == (p.k_out ? 1u : 0u);
  const unsigned char* pool = vals ? p.v_pool : p.k_pool;
  __nv_bfloat16* out = vals ? p.v_out : p.k_out;
  const int B = p.page_size, shift = __ffs(B) - 1;
  const int pages = p.n_blocks * p.n_kv_heads;        // below 2^31: the host has checked
  const size_t rec_bytes = size_t(kv_rec_bytes(FMT, B));
  griddep_launch();
  griddep_wait();
  constexpr int kPer = kReadRows / kHalfWarps;
  uint2 w[kPer];
  float scale[kPer], grp[kPer];
  bool on[kPer];
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    // 16 rows lie in one page, the same for the whole block
    const int r = ((i * kHalfWarps) & (B - 1)) + hw;
    const int page = int(blockIdx.x) * (kReadRows >> shift) + ((i * kHalfWarps) >> shift);
    on[i] = page < pages;
    if (!on[i]) continue;
    const int entry = page / p.n_kv_heads, h = page - entry * p.n_kv_heads;
    const int blk = p.block_ids[entry];
    on[i] = blk >= 0 && blk < p.num_blocks;
    if (!on[i]) {
      if (blk >= p.num_blocks && l16 == 0) flag_status(p.status, LOCKS_DEV_BAD_BLOCK_ID);
      continue;
    }
    const unsigned char* rec = pool + (size_t(blk) * p.n_kv_heads + h) * rec_bytes;
    scale[i] = *reinterpret_cast<const float*>(rec + kv_scale_off(FMT, B) + 4 * r);
    if constexpr (FMT == LOCKS_KV_I4) {
      w[i].x = *reinterpret_cast<const uint32_t*>(rec + kv_chunk_off<FMT>(r, l16 >> 2) + 4 * (l16 & 3));
      grp[i] = e4m3x2_to_f2(rec[kv_group_off(FMT, B) + 4 * r + (l16 >> 2)]).x;
    } else {
      w[i] = *reinterpret_cast<const uint2*>(rec + kv_chunk_off<FMT>(r, l16 >> 1) + 8 * (l16 & 1));
    }
  }
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    if (!on[i]) continue;
    const int64_t row = int64_t(blockIdx.x) * kReadRows + i * kHalfWarps + hw;
    float x[8];
    if constexpr (FMT == LOCKS_KV_F8) {
      const float2 a = e4m3x2_to_f2(w[i].x & 0xffff), b = e4m3x2_to_f2(w[i].x >> 16);
      const float2 c = e4m3x2_to_f2(w[i].y & 0xffff), d = e4m3x2_to_f2(w[i].y >> 16);
      x[0] = a.x; x[1] = a.y; x[2] = b.x; x[3] = b.y;
      x[4] = c.x; x[5] = c.y; x[6] = d.x; x[7] = d.y;
    } else if constexpr (FMT == LOCKS_KV_I8) {
      // the byte u = code + 128 as the low mantissa bits of 2^23, less 2^23 + 128: exact
#pragma unroll
      for (int e = 0; e < 8; ++e)
        x[e] = __uint_as_float(__byte_perm(e < 4 ? w[i].x : w[i].y, 0x4b000000u, 0x7440 + (e & 3))) -
               8388736.f;
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e)
        x[e] = __fmul_rn(__uint_as_float(((w[i].x >> (4 * e)) & 15u) | 0x4b000000u) - 8388616.f,
                         grp[i]);                     // exact
    }
#pragma unroll
    for (int e = 0; e < 8; ++e) x[e] = __fmul_rn(x[e], scale[i]);
    *reinterpret_cast<uint4*>(out + row * kHeadDim + 8 * l16) = pack8(x);
  }
}

template <int FMT, int LAYOUT, int TOKENS>
int launch_write_tokens(KvWriteParams p, int rows, int chunks, cudaStream_t stream) {
  p.n_chunks = chunks;
  const int64_t blocks = (int64_t(p.n_tokens) + TOKENS - 1) / TOKENS * chunks;
  if (blocks > 0x7fffffff) return LOCKS_ERR_UNSUPPORTED;
  const size_t smem = size_t(TOKENS) * ((rows + chunks - 1) / chunks) * kRowBytes;
  // above 48 KB a kernel has to be told, once a device
  auto kern = kv_write_kernel<FMT, LAYOUT, TOKENS>;
  static LaunchOnce once;
  if (!once.run([&] {
        return cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, kMaxWriteSmem) ==
               cudaSuccess;
      }))
    return LOCKS_ERR_CUDA;
  return launch_dependent(kern, dim3(unsigned(blocks)), kWriteThreads, smem, p, stream);
}

template <int FMT, int LAYOUT>
int launch_write_layout(const KvWriteParams& p, cudaStream_t stream) {
  // A prompt: all rows of four tokens a block (or of as many as leave room for
  // four blocks an SM), when that gives every SM four blocks.  A decode step:
  // one token a block and its rows spread over blocks of a row per half-warp.
  const int rows = (p.q_out ? p.n_q_heads : 0) + 2 * p.n_kv_heads;
  const int fits = kMaxWriteSmem / (rows * kRowBytes);
  if (p.n_tokens >= 4 * 4 * 152 && fits >= 4) return launch_write_tokens<FMT, LAYOUT, 4>(p, rows, 1, stream);
  if (p.n_tokens >= 2 * 4 * 152 && fits >= 2) return launch_write_tokens<FMT, LAYOUT, 2>(p, rows, 1, stream);
  return launch_write_tokens<FMT, LAYOUT, 1>(p, rows, (rows + kHalfWarps - 1) / kHalfWarps, stream);
}

template <int FMT>
int launch_write_fmt(const KvWriteParams& p, cudaStream_t stream) {
  if (!p.rope.turns) return launch_write_layout<FMT, kNoTurn>(p, stream);
  if (p.rope.layout == LOCKS_ROPE_HALF) return launch_write_layout<FMT, kHalf>(p, stream);
  return launch_write_layout<FMT, kInterleaved>(p, stream);
}

template <int FMT>
int launch_read_fmt(const KvReadParams& p, cudaStream_t stream) {
  const int64_t rows = int64_t(p.n_blocks) * p.n_kv_heads * p.page_size;
  const int64_t blocks = (rows + kReadRows - 1) / kReadRows;
  if (rows / p.page_size > 0x7fffffff) return LOCKS_ERR_UNSUPPORTED;
  const unsigned pools = (p.k_out ? 1 : 0) + (p.v_out ? 1 : 0);
  return launch_dependent(kv_read_kernel<FMT>, dim3(unsigned(blocks), pools), kWriteThreads, 0, p,
                          stream);
}

}  // namespace

int launch_kv_write(KvWriteParams p, int fmt, cudaStream_t stream) {
  switch (fmt) {
    case LOCKS_KV_F8: return launch_write_fmt<LOCKS_KV_F8>(p, stream);
    case LOCKS_KV_I8: return launch_write_fmt<LOCKS_KV_I8>(p, stream);
    case LOCKS_KV_I4: return launch_write_fmt<LOCKS_KV_I4>(p, stream);
    default: return LOCKS_ERR_INVALID_ARG;
  }
}

int launch_kv_read(const KvReadParams& p, int fmt, cudaStream_t stream) {
  switch (fmt) {
    case LOCKS_KV_F8: return launch_read_fmt<LOCKS_KV_F8>(p, stream);
    case LOCKS_KV_I8: return launch_read_fmt<LOCKS_KV_I8>(p, stream);
    case LOCKS_KV_I4: return launch_read_fmt<LOCKS_KV_I4>(p, stream);
    default: return LOCKS_ERR_INVALID_ARG;
  }
}

}  // namespace locks
