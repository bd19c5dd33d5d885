// locks_kv_write and locks_kv_read: tokens into a quantised paged cache, with
// the rotation of their queries and keys, and pages back out of it.
//
// Both move every byte once and are bound by memory.  Half a warp (16 lanes of
// 8 dims) owns a row of 128 dims: its largest magnitude is four shuffles, a
// group of 32 dims is four lanes, and its codes leave as one 128-byte (or
// 64-byte) line.
//
// Write: a task is a token and a chunk of its rows (queries, then keys, then
// values).  The half-warp computes the cos and sin of its lanes' pairs once for
// the chunk.  In the half layout a lane's partner elements (dims + r/2) belong
// to another lane; it loads them itself (they are in L1 already), which keeps
// every lane's 8 dims contiguous for the codes, at the price of computing each
// pair's angle in two lanes.
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
__device__ __forceinline__ uint4 pack8(const float (&x)[8]) {
  return make_uint4(bf16x2(x[0], x[1]), bf16x2(x[2], x[3]), bf16x2(x[4], x[5]), bf16x2(x[6], x[7]));
}

// max over the aligned group of W lanes
template <int W>
__device__ __forceinline__ float lanes_max(float m) {
#pragma unroll
  for (int o = W / 2; o; o >>= 1) m = fmaxf(m, __shfl_xor_sync(kFull, m, o));
  return m;
}

// The row x (8 dims a lane) quantised into row `r` of record `rec`.  Every lane
// of the warp calls it; `live` says whether this half-warp's row is stored.
template <int FMT>
__device__ __forceinline__ void store_row(const float (&x)[8], unsigned char* rec, int r, int B,
                                          int l16, bool live) {
  float m = 0.f;
  bool odd = false;                                   // an infinity or a NaN
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float a = fabsf(x[i]);
    odd |= !(a <= 3.402823466e38f);
    m = fmaxf(m, a);
  }
  m = lanes_max<16>(odd ? INFINITY : m);
  odd = m == INFINITY;
  const bool dead = odd || m < kKvTiny;
  constexpr float kInvTop = FMT == LOCKS_KV_F8 ? float(1.0 / 448.0)
                            : FMT == LOCKS_KV_I8 ? float(1.0 / 127.0)
                                                 : float(1.0 / (7.0 * 448.0));
  const float scale = __fmul_rn(m, kInvTop);
  const float inv = __frcp_rn(scale);
  float y[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) y[i] = dead ? 0.f : __fmul_rn(x[i], inv);
  if constexpr (FMT == LOCKS_KV_F8) {
    uint2 w;
    w.x = e4m3x2(y[0], y[1]) | (e4m3x2(y[2], y[3]) << 16);
    w.y = e4m3x2(y[4], y[5]) | (e4m3x2(y[6], y[7]) << 16);
    if (live) *reinterpret_cast<uint2*>(rec + kv_chunk_off<FMT>(r, l16 >> 1) + 8 * (l16 & 1)) = w;
  } else if constexpr (FMT == LOCKS_KV_I8) {
    uint32_t c[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) c[i] = uint32_t(min(127, max(-127, __float2int_rn(y[i]))) + 128);
    uint2 w;
    w.x = c[0] | (c[1] << 8) | (c[2] << 16) | (c[3] << 24);
    w.y = c[4] | (c[5] << 8) | (c[6] << 16) | (c[7] << 24);
    if (live) *reinterpret_cast<uint2*>(rec + kv_chunk_off<FMT>(r, l16 >> 1) + 8 * (l16 & 1)) = w;
  } else {
    float gm = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) gm = fmaxf(gm, fabsf(y[i]));
    gm = lanes_max<4>(gm);                            // dims 32j .. 32j + 31
    const uint32_t gbits = e4m3x2(__fmul_rn(gm, float(1.0 / 7.0)), 0.f) & 0xff;
    const float g = e4m3x2_to_f2(gbits).x;
    const float ginv = __frcp_rn(g);
    uint32_t w = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int c = g > 0.f ? min(7, max(-7, __float2int_rn(__fmul_rn(y[i], ginv)))) : 0;
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

template <int FMT>
__global__ void __launch_bounds__(kWriteThreads) kv_write_kernel(const KvWriteParams p) {
  const int l16 = threadIdx.x & 15;
  const int64_t task = int64_t(blockIdx.x) * kHalfWarps + (threadIdx.x >> 4);
  griddep_launch();
  griddep_wait();
  // a warp's two half-warps run the same number of rounds (shuffles below name
  // every lane); one without a task stores nothing
  const bool has_task = task < int64_t(p.n_tokens) * p.n_chunks;
  const int64_t token = has_task ? task / p.n_chunks : 0;
  const int chunk = has_task ? int(task % p.n_chunks) : 0;
  const int seq = has_task ? (p.token_seq ? p.token_seq[token] : int(token)) : -1;
  const int pos = p.token_pos[token];
  const int B = p.page_size;
  int blk = -1;
  if (seq >= 0) {
    int32_t bits = 0;
    if (seq >= p.batch) {
      bits = LOCKS_DEV_BAD_PAGE_ID;
    } else if (pos < 0 || pos / B >= p.max_pages) {
      bits = LOCKS_DEV_BAD_SEQ_LEN;
    } else {
      blk = p.block_table[size_t(seq) * p.max_pages + pos / B];
      if (blk < 0 || blk >= p.num_blocks) {
        bits = LOCKS_DEV_BAD_BLOCK_ID;
        blk = -1;
      }
    }
    if (chunk == 0 && l16 == 0) {
      if (bits) flag_status(p.status, bits);
      if (p.seq_lens && blk >= 0) atomicMax(p.seq_lens + seq, pos + 1);
    }
  }
  if (has_task && chunk == 0 && l16 == 0 && p.completed)
    p.completed[token] = (blk >= 0 && (pos + 1) % B == 0) ? blk : -1;

  // cos and sin of this lane's 8 dims: element e of them uses c[e], s[e]
  const int rot = p.rope.turns ? p.rope.rotary_dim : 0;
  const int e0 = 8 * l16;
  const bool half = p.rope.layout == LOCKS_ROPE_HALF;
  const bool turn = e0 < rot;
  const bool upper = half && e0 >= rot / 2;           // second of its pairs
  const int partner = half ? (upper ? e0 - rot / 2 : e0 + rot / 2) : e0;
  float c[8], s[8];
  if (turn) {
    if (half) {
      const int pair = upper ? e0 - rot / 2 : e0;
#pragma unroll
      for (int i = 0; i < 8; ++i)
        rope_cos_sin(__ldg(p.rope.turns + pair + i), pos, p.rope.mscale, c[i], s[i]);
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i)
        rope_cos_sin(__ldg(p.rope.turns + e0 / 2 + i), pos, p.rope.mscale, c[i], s[i]);
    }
  }

  const int hq = p.q_out ? p.n_q_heads : 0, hk = p.n_kv_heads;
  const int rows = hq + 2 * hk;
  const size_t rec_bytes = size_t(kv_rec_bytes(FMT, B));
  const int slot = pos & (B - 1);                     // B is a power of two
  for (int base = 0; base < rows; base += p.n_chunks) {
    const int row = base + chunk;
    const bool is_q = row < hq, is_k = !is_q && row < hq + hk;
    const int h = is_q ? row : (is_k ? row - hq : row - hq - hk);
    const bool on = has_task && seq >= 0 && row < rows && (is_q || blk >= 0);
    float x[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
    if (on) {
      const __nv_bfloat16* src = is_q ? p.q_new + token * p.q_stride
                                      : (is_k ? p.k_new + token * p.k_stride
                                              : p.v_new + token * p.v_stride);
      src += h * kHeadDim;
      unpack8(*reinterpret_cast<const uint4*>(src + e0), x);
      if (turn && (is_q || is_k)) {
        if (half) {
          float z[8];
          unpack8(*reinterpret_cast<const uint4*>(src + partner), z);
#pragma unroll
          for (int i = 0; i < 8; ++i)
            x[i] = upper ? rope_v(z[i], x[i], c[i], s[i]) : rope_u(x[i], z[i], c[i], s[i]);
        } else {
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const float u = x[2 * i], v = x[2 * i + 1];
            x[2 * i] = rope_u(u, v, c[i], s[i]);
            x[2 * i + 1] = rope_v(u, v, c[i], s[i]);
          }
        }
      }
    }
    __syncwarp();                                     // q_out may be q_new: all loads, then stores
    if (on && is_q)
      *reinterpret_cast<uint4*>(p.q_out + (token * hq + h) * kHeadDim + e0) = pack8(x);
    const bool live = on && !is_q;
    if (__any_sync(kFull, live)) {
      unsigned char* rec = (is_k ? p.k_pool : p.v_pool) +
                           (size_t(live ? blk : 0) * hk + (live ? h : 0)) * rec_bytes;
      store_row<FMT>(x, rec, slot, B, l16, live);
    }
  }
}

// Read: a block of 256 threads converts 64 rows of one pool (one page of 64,
// two of 32, four of 16), four rows a half-warp, all loaded before any is stored.
constexpr int kReadRows = 64;

template <int FMT>
__global__ void __launch_bounds__(kWriteThreads) kv_read_kernel(const KvReadParams p) {
  const int l16 = threadIdx.x & 15, hw = threadIdx.x >> 4;
  const bool values = blockIdx.y == (p.k_out ? 1u : 0u);
  const unsigned char* pool = values ? p.v_pool : p.k_pool;
  __nv_bfloat16* out = values ? p.v_out : p.k_out;
  const int B = p.page_size;
  const int64_t n_rows = int64_t(p.n_blocks) * p.n_kv_heads * B;
  const size_t rec_bytes = size_t(kv_rec_bytes(FMT, B));
  griddep_launch();
  griddep_wait();
  constexpr int kPer = kReadRows / kHalfWarps;
  uint2 w[kPer];
  float scale[kPer], grp[kPer];
  bool on[kPer];
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    const int64_t row = int64_t(blockIdx.x) * kReadRows + i * kHalfWarps + hw;
    on[i] = row < n_rows;
    if (!on[i]) continue;
    const int64_t page = row / B;
    const int r = int(row % B), h = int(page % p.n_kv_heads);
    const int blk = p.block_ids[page / p.n_kv_heads];
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
#pragma unroll
      for (int e = 0; e < 8; ++e)
        x[e] = float(int(((e < 4 ? w[i].x : w[i].y) >> (8 * (e & 3))) & 255) - 128);
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e)
        x[e] = __fmul_rn(float(int((w[i].x >> (4 * e)) & 15) - 8), grp[i]);   // exact
    }
#pragma unroll
    for (int e = 0; e < 8; ++e) x[e] = __fmul_rn(x[e], scale[i]);
    *reinterpret_cast<uint4*>(out + row * kHeadDim + 8 * l16) = pack8(x);
  }
}

template <int FMT>
int launch_write_fmt(KvWriteParams p, cudaStream_t stream) {
  // Row chunks per token: one half-warp walks all rows of a token (its angles
  // computed once) when that still gives 8 blocks per SM; with fewer tokens the
  // rows are spread, down to one row a half-warp.
  const int rows = (p.q_out ? p.n_q_heads : 0) + 2 * p.n_kv_heads;
  int64_t per = int64_t(p.n_tokens) * rows / (int64_t(152) * 8 * kHalfWarps);
  per = per < 1 ? 1 : (per > rows ? rows : per);
  p.n_chunks = int((rows + per - 1) / per);
  const int64_t blocks = (int64_t(p.n_tokens) * p.n_chunks + kHalfWarps - 1) / kHalfWarps;
  if (blocks > 0x7fffffff) return LOCKS_ERR_UNSUPPORTED;
  return launch_dependent(kv_write_kernel<FMT>, dim3(unsigned(blocks)), kWriteThreads, 0, p, stream);
}

template <int FMT>
int launch_read_fmt(const KvReadParams& p, cudaStream_t stream) {
  const int64_t rows = int64_t(p.n_blocks) * p.n_kv_heads * p.page_size;
  const int64_t blocks = (rows + kReadRows - 1) / kReadRows;
  if (blocks > 0x7fffffff) return LOCKS_ERR_UNSUPPORTED;
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
