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
// rounding); the sum of p_t that divides the result is kept in float32.
//
// Work split.  The 64-token stages of all (sequence, KV head) units form one
// list; block c of N takes the c-th N-th of it, whatever the lengths of the
// sequences, so that ragged batches load every SM alike.  A unit that lies in
// one block is finished there; one that is cut is left as partials (running
// maximum, sum, weighted values) in the workspace, and the last of its blocks
// to arrive (atomic ticket) merges them in the blocks' order, so results do not
// depend on the order of arrival.  The workspace is a few MB for any shape.
//
// Block.  Warp 8 is a producer: it looks up 32 pages at a time (one a lane) and
// copies each page's K and V records (cp.async.bulk, one contiguous piece each)
// into a ring of 64-token stages.  Consumer warps 0-7 take 16 tokens of every
// other stage and keep everything in registers:
//   S^T (16 tokens x 8 heads)  = K (16 x 128) . Q^T      8 mma m16n8k16
//   O^T (128 dims x 8 heads)  += V^T (128 x 16) . P^T    8 mma m16n8k16
// Tokens and dims are the long sides of the products, so the short one, the
// heads, fills its 8 columns twice as well as it would 16 rows.  K's fragments
// are rows as they lie in memory (the dims of a product may come in any order
// that Q shares); V's are two tokens' bytes interleaved by a byte permute; P is
// turned from S^T's layout into an operand by movmatrix.
#include "locks_kv.cuh"

namespace locks {

namespace {

constexpr int kKvWarps = 8;                       // consumer warps
constexpr int kKvConsumers = kKvWarps * 32;
constexpr int kKvThreads = kKvConsumers + 32;
constexpr int kStageTok = 64;
constexpr float kNone = -3.402823466e38f;         // running maximum before any token
constexpr int kKvMergeBytes = kKvWarps * 4096;    // a warp's 8 heads x 128 floats

// Blocks: two per SM (one for more than 8 heads, whose accumulators fill the registers).
constexpr int kSms = 152;
__host__ __device__ constexpr int kv_blocks(int nt) { return kSms * (nt == 1 ? 2 : 1); }
__host__ __device__ constexpr size_t kv_part_bytes(int nt) { return size_t(nt) * (4096 + 64); }

__host__ __device__ constexpr int kv_stage_bytes(int fmt) {
  return 2 * kStageTok * (kv_row_bytes(fmt) + (fmt == LOCKS_KV_I4 ? 8 : 4));
}
// stages of the ring: what two blocks per SM (one for NT = 2) leave beside the merge buffer
constexpr int kv_stages(int fmt, int nt) {
  const int budget = (nt == 1 ? 115712 : 232448) - kKvMergeBytes - 4096;
  const int n = budget / kv_stage_bytes(fmt);
  return n > 16 ? 16 : n;
}

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
__device__ __forceinline__ uint4 lds128(const unsigned char* p) {
  return *reinterpret_cast<const uint4*>(p);
}
__device__ __forceinline__ float lds_f(const unsigned char* p) {
  return *reinterpret_cast<const float*>(p);
}
__device__ __forceinline__ void consumers_sync() {
  asm volatile("bar.sync 1, %0;" ::"n"(kKvConsumers) : "memory");
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
  x[0] = hfma2((w & 0x000f000fu) | 0x64006400u, s.s, s.off);
  x[1] = hfma2((w & 0x00f000f0u) | 0x64006400u, s.s16, s.off16);
  x[2] = hfma2((v & 0x000f000fu) | 0x64006400u, s.s, s.off);
  x[3] = hfma2((v & 0x00f000f0u) | 0x64006400u, s.s16, s.off16);
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
  float lim[2 * NT];     // weights above it need a new factor
  float acc[NT][8][4];   // O^T, times f
};

// One warp's 16 tokens: records k, v (rows r0 ..), valid rows [lo, hi) of them.
template <int FMT, int NT>
__device__ __forceinline__ void attend16(const unsigned char* k, const unsigned char* v, int B,
                                         int r0, int lo, int hi, int g, int t,
                                         const uint32_t (&qb)[NT][8][2], const float (&qs)[2 * NT],
                                         State<NT>& st) {
  // ---- S^T = K Q^T ----
  float sa[NT][4], sb[NT][4];
#pragma unroll
  for (int n = 0; n < NT; ++n)
#pragma unroll
    for (int e = 0; e < 4; ++e) sa[n][e] = sb[n][e] = 0.f;
  const int ra = r0 + g, rb = r0 + g + 8;
  if constexpr (FMT == LOCKS_KV_I4) {
    const uint4 A = lds128(k + kv_chunk_off<FMT>(ra, t)), C = lds128(k + kv_chunk_off<FMT>(rb, t));
    const uint32_t ga = k[kv_group_off(FMT, B) + 4 * ra + t], gb = k[kv_group_off(FMT, B) + 4 * rb + t];
    const I4Scale s0 = i4_scale(e4m3x2_to_f16x2(ga | (ga << 8)));
    const I4Scale s1 = i4_scale(e4m3x2_to_f16x2(gb | (gb << 8)));
    const uint32_t aw[4] = {A.x, A.y, A.z, A.w}, cw[4] = {C.x, C.y, C.z, C.w};
#pragma unroll
    for (int w = 0; w < 4; ++w) {
      uint32_t x[4], y[4];
      i4_pairs(aw[w], s0, x);
      i4_pairs(cw[w], s1, y);
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        mma_f16(sa[n], x[0], y[0], x[1], y[1], qb[n][2 * w][0], qb[n][2 * w][1]);
        mma_f16(sb[n], x[2], y[2], x[3], y[3], qb[n][2 * w + 1][0], qb[n][2 * w + 1][1]);
      }
    }
  } else {
#pragma unroll
    for (int c = 0; c < 2; ++c) {
      const uint4 A = lds128(k + kv_chunk_off<FMT>(ra, 2 * t + c));
      const uint4 C = lds128(k + kv_chunk_off<FMT>(rb, 2 * t + c));
      const uint32_t aw[4] = {A.x, A.y, A.z, A.w}, cw[4] = {C.x, C.y, C.z, C.w};
#pragma unroll
      for (int w = 0; w < 4; ++w) {
        const uint32_t a0 = pair8<FMT, 0>(aw[w]), a2 = pair8<FMT, 1>(aw[w]);
        const uint32_t a1 = pair8<FMT, 0>(cw[w]), a3 = pair8<FMT, 1>(cw[w]);
#pragma unroll
        for (int n = 0; n < NT; ++n)
          mma_f16((w & 1) ? sb[n] : sa[n], a0, a1, a2, a3, qb[n][4 * c + w][0], qb[n][4 * c + w][1]);
      }
    }
  }
  // ---- logits in log2 units, masked; weights ----
  const bool on0 = g >= lo && g < hi, on1 = g + 8 >= lo && g + 8 < hi;
  const float ks0 = lds_f(k + kv_scale_off(FMT, B) + 4 * ra), ks1 = lds_f(k + kv_scale_off(FMT, B) + 4 * rb);
  const float vs0 = on0 ? lds_f(v + kv_scale_off(FMT, B) + 4 * ra) : 0.f;
  const float vs1 = on1 ? lds_f(v + kv_scale_off(FMT, B) + 4 * rb) : 0.f;
  float z0[2 * NT], z1[2 * NT], p0[2 * NT], p1[2 * NT];
  bool over = false;
#pragma unroll
  for (int n = 0; n < NT; ++n)
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const int j = 2 * n + e;
      z0[j] = on0 ? (sa[n][e] + sb[n][e]) * qs[j] * ks0 : -INFINITY;
      z1[j] = on1 ? (sa[n][2 + e] + sb[n][2 + e]) * qs[j] * ks1 : -INFINITY;
      p0[j] = ex2_approx(z0[j] - st.m[j]);
      p1[j] = ex2_approx(z1[j] - st.m[j]);
      over |= fmaxf(z0[j], z1[j]) > st.m[j] + 8.f ||
              fmaxf(fabsf(p0[j] * vs0), fabsf(p1[j] * vs1)) > st.lim[j];
    }
  // The reference moves only when a logit passes it by 2^8 or a weight leaves
  // f16's range: a few times per sequence, so most chunks do no rescaling.
  if (__any_sync(kFull, over)) {
#pragma unroll
    for (int j = 0; j < 2 * NT; ++j) {
      float mx = fmaxf(z0[j], z1[j]);
#pragma unroll
      for (int o = 4; o < 32; o <<= 1) mx = fmaxf(mx, __shfl_xor_sync(kFull, mx, o));
      mx = fmaxf(st.m[j], mx);
      const float alpha = ex2_approx(st.m[j] - mx);
      st.m[j] = mx;
      st.l[j] *= alpha;
      p0[j] = ex2_approx(z0[j] - mx);
      p1[j] = ex2_approx(z1[j] - mx);
      float xm = fmaxf(fabsf(p0[j] * vs0), fabsf(p1[j] * vs1));
#pragma unroll
      for (int o = 4; o < 32; o <<= 1) xm = fmaxf(xm, __shfl_xor_sync(kFull, xm, o));
      const float f = st.f[j];
      xm = fmaxf(xm, f > 0.f ? alpha * 128.f / f : 0.f);
      const float fn = xm > 0.f ? fminf(128.f / xm, 1.2676506e30f) : 0.f;
      const float up = f > 0.f ? alpha * (fn / f) : 0.f;
      st.f[j] = fn;
      st.lim[j] = fn > 0.f ? 32768.f / fn : 0.f;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        st.acc[j >> 1][i][j & 1] *= up;
        st.acc[j >> 1][i][2 + (j & 1)] *= up;
      }
    }
  }
  // ---- P^T as the second operand ----
  uint32_t pb[NT][2];
#pragma unroll
  for (int n = 0; n < NT; ++n) {
    const int j = 2 * n;
    st.l[j] += p0[j] + p1[j];
    st.l[j + 1] += p0[j + 1] + p1[j + 1];
    pb[n][0] = transpose8x8(f16x2(p0[j] * vs0 * st.f[j], p0[j + 1] * vs0 * st.f[j + 1]));
    pb[n][1] = transpose8x8(f16x2(p1[j] * vs1 * st.f[j], p1[j + 1] * vs1 * st.f[j + 1]));
  }
  // ---- O^T += V^T P^T: this lane's tokens 2t, 2t+1, 2t+8, 2t+9, dims 16g .. 16g+15 ----
  const int tok[4] = {2 * t, 2 * t + 1, 2 * t + 8, 2 * t + 9};
  const bool whole = lo == 0 && hi == 16;
  if constexpr (FMT == LOCKS_KV_I4) {
    uint2 T[4];
    uint32_t gs[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int r = r0 + tok[i];
      T[i] = *reinterpret_cast<const uint2*>(v + kv_chunk_off<FMT>(r, g >> 1) + 8 * (g & 1));
      gs[i] = v[kv_group_off(FMT, B) + 4 * r + (g >> 1)];
      // a row outside the sequence may hold NaN scales: 0 x NaN must not enter the sum
      if (!whole && (tok[i] < lo || tok[i] >= hi)) gs[i] = 0;
    }
    const I4Scale s01 = i4_scale(e4m3x2_to_f16x2(gs[0] | (gs[1] << 8)));
    const I4Scale s23 = i4_scale(e4m3x2_to_f16x2(gs[2] | (gs[3] << 8)));
#pragma unroll
    for (int w = 0; w < 4; ++w) {       // dims 4w .. 4w + 3: half a word of each token
      const uint32_t sel = (w & 1) ? 0x7632u : 0x5410u;
      const uint32_t a = prmt(w < 2 ? T[0].x : T[0].y, w < 2 ? T[1].x : T[1].y, sel);
      const uint32_t c = prmt(w < 2 ? T[2].x : T[2].y, w < 2 ? T[3].x : T[3].y, sel);
      uint32_t x[4], y[4];
      i4_pairs(a, s01, x);
      i4_pairs(c, s23, y);
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        mma_f16(st.acc[n][2 * w], x[0], x[1], y[0], y[1], pb[n][0], pb[n][1]);
        mma_f16(st.acc[n][2 * w + 1], x[2], x[3], y[2], y[3], pb[n][0], pb[n][1]);
      }
    }
  } else {
    uint4 T[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      T[i] = lds128(v + kv_chunk_off<FMT>(r0 + tok[i], g));
      // a row outside the sequence may hold e4m3 NaN codes
      if (FMT == LOCKS_KV_F8 && !whole && (tok[i] < lo || tok[i] >= hi)) T[i] = make_uint4(0, 0, 0, 0);
    }
    const uint32_t T0[4] = {T[0].x, T[0].y, T[0].z, T[0].w}, T1[4] = {T[1].x, T[1].y, T[1].z, T[1].w};
    const uint32_t T2[4] = {T[2].x, T[2].y, T[2].z, T[2].w}, T3[4] = {T[3].x, T[3].y, T[3].z, T[3].w};
#pragma unroll
    for (int w = 0; w < 4; ++w) {
#pragma unroll
      for (int e = 0; e < 2; ++e) {     // dims 4w + 2e, 4w + 2e + 1
        const uint32_t sel = e ? 0x7362u : 0x5140u;
        const uint32_t x = prmt(T0[w], T1[w], sel), y = prmt(T2[w], T3[w], sel);
        const uint32_t a0 = pair8<FMT, 0>(x), a1 = pair8<FMT, 1>(x);
        const uint32_t a2 = pair8<FMT, 0>(y), a3 = pair8<FMT, 1>(y);
#pragma unroll
        for (int n = 0; n < NT; ++n)
          mma_f16(st.acc[n][2 * w + e], a0, a1, a2, a3, pb[n][0], pb[n][1]);
      }
    }
  }
}

// A sequence as the kernel walks it: its length, the first attended position,
// its first stage and its number of stages (the same for every KV head).
struct Seq {
  int n, lo, first, stages;
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

template <int FMT, int NT>
__global__ void __launch_bounds__(kKvThreads, NT == 1 ? 2 : 1) kv_decode_kernel(const KvDecodeParams p) {
  constexpr int STAGES = kv_stages(FMT, NT);
  constexpr int kStageBytes = kv_stage_bytes(FMT);
  extern __shared__ __align__(1024) unsigned char smem[];
  unsigned char* ring = smem;
  float4* mbuf = reinterpret_cast<float4*>(smem + STAGES * kStageBytes);    // [warp][8][32]
  __shared__ uint64_t s_full[STAGES], s_empty[STAGES];
  __shared__ int s_range[STAGES][4];              // valid rows of each 16-token chunk: lo | hi << 8
  __shared__ float s_m[kKvWarps][8 * NT], s_l[kKvWarps][8 * NT];
  __shared__ long long s_scan[kKvThreads / 32], s_base;
  __shared__ int s_first, s_last;

  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int B = p.page_size, pps = kStageTok / B, hk = p.n_kv_heads;
  if (tid == 0) {
    for (int s = 0; s < STAGES; ++s) {
      mbar_init(s_full + s, 1);
      mbar_init(s_empty + s, 4);
    }
    mbar_fence_init();
  }
  griddep_launch();
  griddep_wait();

  // ---- this block's share of the stages of all units ----
  const int per = (p.batch + kKvThreads - 1) / kKvThreads;
  const int b_lo = min(p.batch, tid * per), b_hi = min(p.batch, b_lo + per);
  long long mine = 0;
  for (int b = b_lo; b < b_hi; ++b) {
    mine += seq_of(p, b).stages;
    if (blockIdx.x == 0 && (p.seq_lens[b] < 0 || p.seq_lens[b] > p.max_pages * B))
      flag_status(p.status, LOCKS_DEV_BAD_SEQ_LEN);
  }
  long long incl = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long x = __shfl_up_sync(kFull, incl, o);
    if (lane >= o) incl += x;
  }
  if (lane == 31) s_scan[warp] = incl;
  __syncthreads();
  long long total = 0;
#pragma unroll
  for (int w = 0; w < kKvThreads / 32; ++w) {
    if (w == warp) incl += total;
    total += s_scan[w];
  }
  const long long W = total * hk;
  const int N = int(min((long long)gridDim.x, max(W, 1ll)));
  const long long w_lo = int(blockIdx.x) < N ? W * blockIdx.x / N : 0;
  const long long w_hi = int(blockIdx.x) < N ? W * (blockIdx.x + 1) / N : 0;
  if (w_lo < w_hi && (incl - mine) * hk <= w_lo && w_lo < incl * hk) {
    long long at = (incl - mine) * hk;
    for (int b = b_lo; b < b_hi; ++b) {
      const long long n = (long long)seq_of(p, b).stages * hk;
      if (w_lo < at + n) {
        s_first = b;
        s_base = at;
        break;
      }
      at += n;
    }
  }
  // sequences with nothing to attend: their outputs are written here
  for (int b = blockIdx.x; b < p.batch; b += gridDim.x) {
    if (seq_of(p, b).stages > 0) continue;
    const size_t rows = size_t(hk) * p.group, row0 = size_t(b) * rows;
    for (size_t i = tid; i < rows * (kHeadDim / 8); i += kKvThreads)
      reinterpret_cast<uint4*>(p.out + row0 * kHeadDim)[i] = make_uint4(0, 0, 0, 0);
    if (p.out_lse)
      for (size_t i = tid; i < rows; i += kKvThreads) p.out_lse[row0 + i] = -INFINITY;
  }
  __syncthreads();
  if (w_lo >= w_hi) return;

  const size_t rec = size_t(kv_rec_bytes(FMT, B));
  int b = s_first;
  Seq sq = seq_of(p, b);
  long long base = s_base;                        // first stage of sequence b in the list
  int h = int((w_lo - base) / sq.stages);
  int i0 = int((w_lo - base) % sq.stages);
  long long left = w_hi - w_lo;
  int it = 0;                                     // stages of this block so far

  if (warp == kKvWarps) {
    // ---------------- producer ----------------
    const uint64_t pol = l2_evict_first();
    bool ok = true;
    while (left > 0 && ok) {
      const int cnt = int(min((long long)(sq.stages - i0), left));
      const int32_t* row = p.block_table + size_t(b) * p.max_pages;
      const int32_t* sel = p.selected ? p.selected + (size_t(b) * hk + h) * p.k : nullptr;
      const int pages = (sq.n + B - 1) / B;
      const int batch_st = 32 / pps;              // stages looked up at a time
      for (int s0 = 0; s0 < cnt && ok; s0 += batch_st) {
        const int e = lane & (pps - 1), st = s0 + lane / pps;
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
        const int todo = min(batch_st, cnt - s0);
        for (int x = 0; x < todo; ++x, ++it) {
          const int s = it % STAGES;
          if (it >= STAGES &&
              !__all_sync(kFull, mbar_wait_bounded(s_empty + s, ((it / STAGES) - 1) & 1))) {
            if (lane == 0) flag_status(p.status, LOCKS_DEV_WAIT_TIMEOUT);
            ok = false;
            break;
          }
          const bool me = lane / pps == x;
          if (me)
            for (int c = 0; c < B / 16; ++c)
              s_range[s][e * (B / 16) + c] =
                  min(16, max(0, r_lo - 16 * c)) | (min(16, max(0, r_hi - 16 * c)) << 8);
          const unsigned live = __ballot_sync(kFull, me && blk >= 0);
          // (the ballot does not order the lanes' stores of s_range)
          __syncwarp();
          if (lane == 0) {
            if (live) mbar_arrive_expect_tx(s_full + s, uint32_t(__popc(live) * 2 * rec));
            else mbar_arrive(s_full + s);
          }
          __syncwarp();
          if (me && blk >= 0) {
            unsigned char* dst = ring + s * kStageBytes + e * rec;
            const size_t src = (size_t(blk) * hk + h) * rec;
            bulk_g2s_hint(dst, p.k_pool + src, uint32_t(rec), s_full + s, pol);
            bulk_g2s_hint(dst + kStageBytes / 2, p.v_pool + src, uint32_t(rec), s_full + s, pol);
          }
        }
      }
      left -= cnt;
      i0 = 0;
      if (++h == hk && left > 0) {
        h = 0;
        do {
          base += (long long)sq.stages * hk;
          sq = seq_of(p, ++b);
        } while (sq.stages == 0);
      }
    }
    return;
  }

  // ---------------- consumers ----------------
  const int g = lane >> 2, t = lane & 3, G = p.group;
  const int half = warp >> 2, chunk = warp & 3;   // stages of this parity, this 16-token chunk
  bool ok = true;
  float* parts = reinterpret_cast<float*>(p.ws + (size_t(p.batch) * hk * 4 + 255) / 256 * 256);
  int* tickets = reinterpret_cast<int*>(p.ws);
  while (left > 0) {
    const int cnt = int(min((long long)(sq.stages - i0), left));
    const size_t unit = size_t(b) * hk + h;
    // ---- the query: head 8n + g, dims 32t .. 32t + 31, brought to a largest magnitude in
    // [2^14, 2^15) by a power of two and rounded to f16 (exact but for elements 2^-28 of it) ----
    uint32_t qb[NT][8][2];
    float qs[2 * NT];
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      const int head = 8 * n + g;
      float x[32];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        uint4 w = make_uint4(0, 0, 0, 0);
        if (head < G)
          w = *reinterpret_cast<const uint4*>(p.q + (unit * G + head) * kHeadDim + 32 * t + 8 * i);
        const uint32_t ww[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          x[8 * i + 2 * e] = bf16_lo(ww[e]);
          x[8 * i + 2 * e + 1] = bf16_hi(ww[e]);
        }
      }
      float mx = 0.f;
#pragma unroll
      for (int i = 0; i < 32; ++i) mx = fmaxf(mx, fabsf(x[i]));
      mx = fmaxf(mx, __shfl_xor_sync(kFull, mx, 1));
      mx = fmaxf(mx, __shfl_xor_sync(kFull, mx, 2));
      const int ex = int(__float_as_uint(mx) >> 23);          // biased exponent
      // factor 2^(14 - (ex - 127)), at most 2^126; an infinity keeps its value
      const int up = ex == 255 ? 0 : min(126, 141 - ex);
      const float factor = __uint_as_float(uint32_t(127 + up) << 23);
      const float back = __uint_as_float(uint32_t(127 - up) << 23);
#pragma unroll
      for (int i = 0; i < 32; ++i) x[i] *= factor;
#pragma unroll
      for (int ks = 0; ks < 8; ++ks) {
        if constexpr (FMT == LOCKS_KV_I4) {
          // word ks / 2, nibbles (n, n + 4) with n = 0, 1 or 2, 3
          const int d = 8 * (ks >> 1) + 2 * (ks & 1);
          qb[n][ks][0] = f16x2(x[d], x[d + 4]);
          qb[n][ks][1] = f16x2(x[d + 1], x[d + 5]);
        } else {
          const int d = 4 * ks;
          qb[n][ks][0] = f16x2(x[d], x[d + 1]);
          qb[n][ks][1] = f16x2(x[d + 2], x[d + 3]);
        }
      }
      constexpr float kScale = 0.08838834764831845f * kLog2e * (FMT == LOCKS_KV_I4 ? 256.f : 1.f);
      qs[2 * n] = __shfl_sync(kFull, back, 8 * t) * kScale;       // heads 8n + 2t, 8n + 2t + 1
      qs[2 * n + 1] = __shfl_sync(kFull, back, 8 * t + 4) * kScale;
    }
    State<NT> st;
#pragma unroll
    for (int j = 0; j < 2 * NT; ++j) {
      st.m[j] = kNone;
      st.l[j] = st.f[j] = st.lim[j] = 0.f;
    }
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int i = 0; i < 8; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e) st.acc[n][i][e] = 0.f;

    for (const int end = it + cnt; it < end; ++it) {
      if ((it & 1) != half) continue;
      const int s = it % STAGES;
      if (ok && !__all_sync(kFull, mbar_wait_bounded(s_full + s, (it / STAGES) & 1))) {
        if (lane == 0) flag_status(p.status, LOCKS_DEV_WAIT_TIMEOUT);
        ok = false;                               // the rest counts as empty: tickets stay right
      }
      if (!ok) continue;
      const int range = s_range[s][chunk];
      if ((range >> 8) > (range & 255)) {
        const int tok0 = chunk * 16, e = tok0 / B;
        const unsigned char* k = ring + s * kStageBytes + e * rec;
        attend16<FMT, NT>(k, k + kStageBytes / 2, B, tok0 - e * B, range & 255, range >> 8, g, t, qb,
                          qs, st);
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(s_empty + s);
    }

    // ---- merge the warps' states; finish the unit or leave a partial ----
    const long long u_lo = base + (long long)h * sq.stages, u_hi = u_lo + sq.stages;
    const int c_lo = int(((u_lo + 1) * N - 1) / W), c_hi = int((u_hi * N - 1) / W);
    const bool alone = c_lo == c_hi;
    const int slot = int(blockIdx.x) == c_lo ? 1 : 0;
    float* part = parts + (size_t(blockIdx.x) * 2 + slot) * (kv_part_bytes(NT) / 4);
#pragma unroll
    for (int j = 0; j < 2 * NT; ++j) {
      float l = st.l[j];
#pragma unroll
      for (int o = 4; o < 32; o <<= 1) l += __shfl_xor_sync(kFull, l, o);
      if (g == 0) {
        s_m[warp][8 * (j >> 1) + 2 * t + (j & 1)] = st.m[j];
        s_l[warp][8 * (j >> 1) + 2 * t + (j & 1)] = l;
      }
    }
    // item of this thread: head parity and 4 dims of a lane's 16
    const int q4 = warp, odd = q4 >> 2, dq = q4 & 3;
#pragma unroll
    for (int n = 0; n < NT; ++n) {
#pragma unroll
      for (int x = 0; x < 8; ++x) {
        const int j = 2 * n + (x >> 2), i = 2 * (x & 3), e = x >> 2;
        const float f = st.f[j] > 0.f ? (FMT == LOCKS_KV_I4 ? 256.f : 1.f) / st.f[j] : 0.f;
        mbuf[(warp * 8 + x) * 32 + lane] =
            make_float4(st.acc[n][i][e] * f, st.acc[n][i][2 + e] * f, st.acc[n][i + 1][e] * f,
                        st.acc[n][i + 1][2 + e] * f);
      }
      consumers_sync();
      const int head = 8 * n + 2 * t + odd;
      float M = kNone, L = 0.f;
      float4 A = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int w = 0; w < kKvWarps; ++w) M = fmaxf(M, s_m[w][head]);
#pragma unroll
      for (int w = 0; w < kKvWarps; ++w) {
        const float f = exp2f(s_m[w][head] - M);
        const float4 a = mbuf[(w * 8 + q4) * 32 + lane];
        L += s_l[w][head] * f;
        A.x += a.x * f; A.y += a.y * f; A.z += a.z * f; A.w += a.w * f;
      }
      if (alone) {
        if (head < G) {
          const float inv = L != 0.f ? 1.f / L : 0.f;
          uint2 o;
          const __nv_bfloat162 o0 = __floats2bfloat162_rn(A.x * inv, A.y * inv);
          const __nv_bfloat162 o1 = __floats2bfloat162_rn(A.z * inv, A.w * inv);
          o.x = *reinterpret_cast<const uint32_t*>(&o0);
          o.y = *reinterpret_cast<const uint32_t*>(&o1);
          *reinterpret_cast<uint2*>(p.out + (unit * G + head) * kHeadDim + 16 * g + 4 * dq) = o;
          if (p.out_lse && g == 0 && dq == 0)
            p.out_lse[unit * G + head] = L != 0.f ? M * kLn2 + logf(L) : -INFINITY;
        }
      } else {
        reinterpret_cast<float4*>(part)[(n * 8 + q4) * 32 + lane] = A;
        if (g == 0 && dq == 0)
          *reinterpret_cast<float2*>(part + NT * 1024 + 2 * head) = make_float2(M, L);
      }
      consumers_sync();                           // mbuf is free again
    }
    if (!alone) {
      __threadfence();
      consumers_sync();
      if (tid == 0) s_last = atomicAdd(tickets + unit, 1) == c_hi - c_lo;
      consumers_sync();
      if (s_last) {
        __threadfence();
#pragma unroll
        for (int n = 0; n < NT; ++n) {
          const int head = 8 * n + 2 * t + odd;
          float M = kNone, L = 0.f;
          float4 A = make_float4(0.f, 0.f, 0.f, 0.f);
          for (int c = c_lo; c <= c_hi; c += 8) {
            float2 ml[8];
            float4 a[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              ml[i] = make_float2(kNone, 0.f);
              a[i] = make_float4(0.f, 0.f, 0.f, 0.f);
              if (c + i <= c_hi) {
                const float* src = parts + (size_t(c + i) * 2 + (c + i == c_lo)) * (kv_part_bytes(NT) / 4);
                ml[i] = __ldcg(reinterpret_cast<const float2*>(src + NT * 1024 + 2 * head));
                a[i] = __ldcg(reinterpret_cast<const float4*>(src) + (n * 8 + q4) * 32 + lane);
              }
            }
            float Mn = M;
#pragma unroll
            for (int i = 0; i < 8; ++i) Mn = fmaxf(Mn, ml[i].x);
            const float f0 = exp2f(M - Mn);
            L *= f0;
            A.x *= f0; A.y *= f0; A.z *= f0; A.w *= f0;
            M = Mn;
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              const float f = exp2f(ml[i].x - Mn);
              L += ml[i].y * f;
              A.x += a[i].x * f; A.y += a[i].y * f; A.z += a[i].z * f; A.w += a[i].w * f;
            }
          }
          if (head < G) {
            const float inv = L != 0.f ? 1.f / L : 0.f;
            uint2 o;
            const __nv_bfloat162 o0 = __floats2bfloat162_rn(A.x * inv, A.y * inv);
            const __nv_bfloat162 o1 = __floats2bfloat162_rn(A.z * inv, A.w * inv);
            o.x = *reinterpret_cast<const uint32_t*>(&o0);
            o.y = *reinterpret_cast<const uint32_t*>(&o1);
            *reinterpret_cast<uint2*>(p.out + (unit * G + head) * kHeadDim + 16 * g + 4 * dq) = o;
            if (p.out_lse && g == 0 && dq == 0)
              p.out_lse[unit * G + head] = L != 0.f ? M * kLn2 + logf(L) : -INFINITY;
          }
        }
        if (tid == 0) tickets[unit] = 0;
      }
    }
    left -= cnt;
    i0 = 0;
    if (++h == hk && left > 0) {
      h = 0;
      do {
        base += (long long)sq.stages * hk;
        sq = seq_of(p, ++b);
      } while (sq.stages == 0);
    }
  }
  // a wait that ran out: no block leaves while copies into its memory may be in flight
  if (!ok)
    for (int s = 0; s < STAGES; ++s) mbar_wait_bounded(s_full + s, 1);
}

template <int FMT, int NT>
int launch_nt(const KvDecodeParams& p, cudaStream_t stream) {
  constexpr size_t smem = size_t(kv_stages(FMT, NT)) * kv_stage_bytes(FMT) + kKvMergeBytes;
  if (cudaFuncSetAttribute(kv_decode_kernel<FMT, NT>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                           int(smem)) != cudaSuccess)
    return LOCKS_ERR_CUDA;
  return launch_dependent(kv_decode_kernel<FMT, NT>, dim3(kv_blocks(NT)), kKvThreads, smem, p, stream);
}

template <int FMT>
int launch_fmt(const KvDecodeParams& p, cudaStream_t stream) {
  return p.group <= 8 ? launch_nt<FMT, 1>(p, stream) : launch_nt<FMT, 2>(p, stream);
}

}  // namespace

size_t kv_decode_workspace(int batch, int n_kv_heads, int group) {
  const int nt = group <= 8 ? 1 : 2;
  return (size_t(batch) * n_kv_heads * 4 + 255) / 256 * 256 +
         size_t(kv_blocks(nt)) * 2 * kv_part_bytes(nt);
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
