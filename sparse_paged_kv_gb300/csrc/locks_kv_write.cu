// locks_kv_write and locks_kv_read: tokens into a quantised paged cache, with
// the rotation of their queries and keys, and pages back out of it.
//
// Both move every byte once and are bound by memory.  Half a warp (16 lanes of
// 8 dims) owns a row of 128 dims: its largest magnitude is four shuffles, a
// group of 32 dims is four lanes, and its codes leave as one 128-byte (or
// 64-byte) line.
//
// Write: a block takes a few tokens and a run of their rows (queries, then keys,
// then values), computes the tokens' cos and sin once, one pair a thread, into
// shared memory, and its half-warps take a row each, the loads of several rows
// ahead of their arithmetic.  In the half layout a lane's partner elements (dims
// +- r/2) belong to another lane; it loads them itself (they are in L1 already),
// which keeps every lane's 8 dims contiguous for the codes.
#include "locks_kv.cuh"

namespace locks {

namespace {

constexpr int kWriteThreads = 256;
constexpr int kHalfWarps = kWriteThreads / 16;

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

// largest over the aligned group of W lanes
template <int W>
__device__ __forceinline__ uint32_t lanes_max(uint32_t m) {
#pragma unroll
  for (int o = W / 2; o; o >>= 1) m = max(m, __shfl_xor_sync(kFull, m, o));
  return m;
}

// largest magnitude of 8 floats, as bits (ordered like the magnitudes, a NaN above infinity)
__device__ __forceinline__ uint32_t magnitude(const float (&x)[8]) {
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) m = max(m, __float_as_uint(x[i]) & 0x7fffffffu);
  return m;
}

// The row x (8 dims a lane) quantised into row `r` of record `rec`.  Every lane
// of the warp calls it; `live` says whether this half-warp's row is stored.
template <int FMT>
__device__ __forceinline__ void store_row(const float (&x)[8], unsigned char* rec, int r, int B,
                                          int l16, bool live) {
  const uint32_t mb = lanes_max<16>(magnitude(x));
  const float m = __uint_as_float(mb);
  const bool odd = mb >= 0x7f800000u;                 // an infinity or a NaN
  const bool dead = odd || m < kKvTiny;
  constexpr float kInvTop = FMT == LOCKS_KV_F8 ? float(1.0 / 448.0)
                            : FMT == LOCKS_KV_I8 ? float(1.0 / 127.0)
                                                 : float(1.0 / (7.0 * 448.0));
  const float scale = __fmul_rn(m, kInvTop);
  const float inv = __frcp_rn(scale);
  float y[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) y[i] = __fmul_rn(x[i], inv);
  if (dead) {                                         // (rare: the whole half-warp)
#pragma unroll
    for (int i = 0; i < 8; ++i) y[i] = 0.f;
  }
  if constexpr (FMT == LOCKS_KV_F8) {
    uint2 w;
    w.x = e4m3x2(y[0], y[1]) | (e4m3x2(y[2], y[3]) << 16);
    w.y = e4m3x2(y[4], y[5]) | (e4m3x2(y[6], y[7]) << 16);
    if (live) *reinterpret_cast<uint2*>(rec + kv_chunk_off<FMT>(r, l16 >> 1) + 8 * (l16 & 1)) = w;
  } else if constexpr (FMT == LOCKS_KV_I8) {
    // |y| <= 127 (1 + 2^-22): rounding to integers keeps to -127 .. 127
    uint32_t c[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) c[i] = uint32_t(__float2int_rn(y[i]) + 128);
    uint2 w;
    w.x = c[0] | (c[1] << 8) | (c[2] << 16) | (c[3] << 24);
    w.y = c[4] | (c[5] << 8) | (c[6] << 16) | (c[7] << 24);
    if (live) *reinterpret_cast<uint2*>(rec + kv_chunk_off<FMT>(r, l16 >> 1) + 8 * (l16 & 1)) = w;
  } else {
    const float gm = __uint_as_float(lanes_max<4>(magnitude(y)));   // dims 32j .. 32j + 31
    const uint32_t gbits = e4m3x2(__fmul_rn(gm, float(1.0 / 7.0)), 0.f) & 0xff;
    const float g = e4m3x2_to_f2(gbits).x;
    const float ginv = g > 0.f ? __frcp_rn(g) : 0.f;
    uint32_t w = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      // (the group's scale may be rounded down by 2^-4: codes up to 7.47)
      const int c = min(7, max(-7, __float2int_rn(__fmul_rn(y[i], ginv))));
      w |= uint32_t(c + 8) << (4 * i);
    }
    if (live) {
      *reinterpret_cast<uint32_t*>(rec + kv_chunk_off<FMT>(r, l16 >> 2) + 4 * (l16 & 3)) = w;
      if ((l16 & 3) == 0) rec[kv_group_off(FMT, B) + 4 * r + (l16 >> 2)] = (unsigned char)gbits;
    }
  }
  if (live && l16 == 0)
    *reinterpret_cast<float*>(rec + kv_scale_off(FMT, B) + 4 * r) =
        odd ? __int_as_float(0x7fffffff) : (dead ? 0.f : scale);
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

// N rows of 128 dims, STEP apart from `row` on, those before `end`: this lane's
// 8 dims and their partners
template <int LAYOUT, int N, int STEP>
__device__ __forceinline__ void load_rows(const __nv_bfloat16* src, int row, int end, int e0,
                                          int partner, uint4 (&own)[N], uint4 (&other)[N]) {
#pragma unroll
  for (int i = 0; i < N; ++i) {
    own[i] = other[i] = make_uint4(0, 0, 0, 0);
    if (row + STEP * i < end) {
      const __nv_bfloat16* at = src + (row + STEP * i) * kHeadDim;
      own[i] = *reinterpret_cast<const uint4*>(at + e0);
      if (LAYOUT == kHalf) other[i] = *reinterpret_cast<const uint4*>(at + partner);
    }
  }
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

constexpr int kAhead = 3;                             // rows a half-warp loads at a time
constexpr int kWriteWarps = kWriteThreads / 32;

// TOKENS tokens a block: 8 / TOKENS warps a token
template <int FMT, int LAYOUT, int TOKENS>
__global__ void __launch_bounds__(kWriteThreads, 4) kv_write_kernel(const KvWriteParams p) {
  __shared__ float2 table[TOKENS][kHeadDim / 2 + 1];
  constexpr int kPer = kWriteWarps / TOKENS;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int l16 = lane & 15, hw = 2 * (warp % kPer) + (lane >> 4), e0 = 8 * l16;   // hw: this half-warp of the token's
  const int group = blockIdx.x / p.n_chunks, chunk = blockIdx.x % p.n_chunks;
  griddep_launch();
  griddep_wait();
  const int rot = p.rope.rotary_dim;
  const int token = group * TOKENS + warp / kPer;
  // this block's run of the token's rows; a half-warp takes every (2 kPer)-th
  constexpr int kStep = 2 * kPer;
  const int hq = p.q_out ? p.n_q_heads : 0, hk = p.n_kv_heads;
  const int rows = hq + 2 * hk;
  const int lo = rows * chunk / p.n_chunks, hi = rows * (chunk + 1) / p.n_chunks;
  // the first queries are on their way while the angles are computed
  const int q_end = token < p.n_tokens ? min(hi, hq) : 0;
  const int partner = partner_dim<LAYOUT>(rot, e0);
  const __nv_bfloat16* q_src = p.q_new + int64_t(token) * p.q_stride;
  uint4 own[kAhead], other[kAhead];
  load_rows<LAYOUT, kAhead, kStep>(q_src, lo + hw, q_end, e0, partner, own, other);
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
  if (LAYOUT != kNoTurn) __syncthreads();
  if (token >= p.n_tokens) return;                    // (whole warps)
  const int seq = p.token_seq ? p.token_seq[token] : token;
  const int pos = p.token_pos[token];
  const int B = p.page_size, shift = __ffs(B) - 1;    // B is a power of two
  const bool first = chunk == 0 && hw == 0 && l16 == 0;
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
  if (seq < 0) return;

  const Turn turn = make_turn<LAYOUT>(table[warp / kPer], rot, e0);

  // queries
  {
    __nv_bfloat16* dst = p.q_out + int64_t(token) * hq * kHeadDim + e0;
    for (int r = lo; r < q_end; r += kStep * kAhead) {
      if (r > lo) load_rows<LAYOUT, kAhead, kStep>(q_src, r + hw, q_end, e0, partner, own, other);
      __syncwarp();                                   // q_out may be q_new: a row's loads, then its stores
#pragma unroll
      for (int i = 0; i < kAhead; ++i) {
        const int row = r + kStep * i + hw;
        if (row < q_end) {
          float x[8];
          rotate8<LAYOUT>(x, own[i], other[i], turn);
          *reinterpret_cast<uint4*>(dst + row * kHeadDim) = pack8(x);
        }
      }
    }
  }
  if (blk < 0) return;
  // keys, then values (the shuffles of store_row name every lane: rows past the end are not stored)
  const size_t rec_bytes = size_t(kv_rec_bytes(FMT, B));
  {
    const __nv_bfloat16* src = p.k_new + int64_t(token) * p.k_stride;
    unsigned char* dst = p.k_pool + size_t(blk) * hk * rec_bytes;
    const int end = min(hi, hq + hk) - hq;
    for (int r = max(lo - hq, 0); r < end; r += 2 * kStep) {
      uint4 own[2], other[2];
      load_rows<LAYOUT, 2, kStep>(src, r + hw, end, e0, partner, own, other);
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int h = r + kStep * i + hw;
        if (r + kStep * i + (hw & ~1) >= end) break;  // neither half of the warp has a row
        float x[8];
        rotate8<LAYOUT>(x, own[i], other[i], turn);
        store_row<FMT>(x, dst + (h < end ? h : 0) * rec_bytes, slot, B, l16, h < end);
      }
    }
  }
  {
    const __nv_bfloat16* src = p.v_new + int64_t(token) * p.v_stride;
    unsigned char* dst = p.v_pool + size_t(blk) * hk * rec_bytes;
    const int end = hi - hq - hk;
    for (int r = max(lo - hq - hk, 0); r < end; r += 2 * kStep) {
      uint4 own[2], other[2];
      load_rows<kNoTurn, 2, kStep>(src, r + hw, end, e0, e0, own, other);
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int h = r + kStep * i + hw;
        if (r + kStep * i + (hw & ~1) >= end) break;
        float x[8];
        unpack8(own[i], x);
        store_row<FMT>(x, dst + (h < end ? h : 0) * rec_bytes, slot, B, l16, h < end);
      }
    }
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
int launch_write_tokens(KvWriteParams p, int chunks, cudaStream_t stream) {
  p.n_chunks = chunks;
  const int64_t blocks = (int64_t(p.n_tokens) + TOKENS - 1) / TOKENS * chunks;
  if (blocks > 0x7fffffff) return LOCKS_ERR_UNSUPPORTED;
  return launch_dependent(kv_write_kernel<FMT, LAYOUT, TOKENS>, dim3(unsigned(blocks)), kWriteThreads,
                          0, p, stream);
}

template <int FMT, int LAYOUT>
int launch_write_layout(const KvWriteParams& p, cudaStream_t stream) {
  // Four tokens a block and all their rows when that gives every SM four blocks
  // (a prompt); otherwise (a decode step) one token a block and its rows spread
  // over blocks of a row per half-warp.
  const int rows = (p.q_out ? p.n_q_heads : 0) + 2 * p.n_kv_heads;
  if (p.n_tokens >= 4 * 4 * 152) return launch_write_tokens<FMT, LAYOUT, 4>(p, 1, stream);
  return launch_write_tokens<FMT, LAYOUT, 1>(p, (rows + kHalfWarps - 1) / kHalfWarps, stream);
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
