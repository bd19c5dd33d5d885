// locks_kv_decode: attention of one new token per sequence over a quantised
// paged cache,
//   out = sum_t p_t v_t,   p = softmax(q^T k_t / sqrt(d)).
// A row is k_t = s_t c_t (codes c, scale s), so q^T k_t = s_t (q^T c_t), and
// the values enter as (p_t s'_t) c'_t.
//
// One block per (sequence, KV head); its warps take tokens in turn, four dims a
// lane, each with a running maximum and sum per query head, and merge at the end.
#include "locks_kv.cuh"

namespace locks {

namespace {

constexpr int kKvWarps = 8;
constexpr int kKvThreads = kKvWarps * 32;

template <int FMT>
__device__ __forceinline__ void load4(const unsigned char* rec, int B, int r, int lane,
                                      float (&x)[4]) {
  const float s = *reinterpret_cast<const float*>(rec + kv_scale_off(FMT, B) + 4 * r);
  if constexpr (FMT == LOCKS_KV_I4) {
    const uint32_t w = *reinterpret_cast<const uint16_t*>(rec + kv_chunk_off<FMT>(r, lane >> 3) +
                                                          2 * (lane & 7));
    const float g = e4m3x2_to_f2(rec[kv_group_off(FMT, B) + 4 * r + (lane >> 3)]).x;
#pragma unroll
    for (int e = 0; e < 4; ++e) x[e] = float(int((w >> (4 * e)) & 15) - 8) * g * s;
  } else {
    const uint32_t w = *reinterpret_cast<const uint32_t*>(rec + kv_chunk_off<FMT>(r, lane >> 2) +
                                                          4 * (lane & 3));
    if constexpr (FMT == LOCKS_KV_F8) {
      const float2 a = e4m3x2_to_f2(w & 0xffff), b = e4m3x2_to_f2(w >> 16);
      x[0] = a.x * s; x[1] = a.y * s; x[2] = b.x * s; x[3] = b.y * s;
    } else {
#pragma unroll
      for (int e = 0; e < 4; ++e) x[e] = float(int((w >> (8 * e)) & 255) - 128) * s;
    }
  }
}

template <int FMT, int GM>
__global__ void __launch_bounds__(kKvThreads) kv_decode_kernel(const KvDecodeParams p) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int b = blockIdx.x / p.n_kv_heads, h = blockIdx.x % p.n_kv_heads;
  const int G = p.group, B = p.page_size;
  __shared__ float s_m[kKvWarps][GM], s_l[kKvWarps][GM];
  __shared__ float s_acc[kKvWarps][kHeadDim];
  griddep_launch();
  griddep_wait();
  int n = p.seq_lens[b];
  if (n < 0 || n > p.max_pages * B) {
    if (threadIdx.x == 0) flag_status(p.status, LOCKS_DEV_BAD_SEQ_LEN);
    n = n < 0 ? 0 : p.max_pages * B;
  }
  const int lo = p.window > 0 ? max(0, n - p.window) : 0;
  const int pages = (n + B - 1) / B;
  const size_t row0 = (size_t(b) * p.n_kv_heads + h) * G;
  float q[GM][4], acc[GM][4], m[GM], l[GM];
  const float scale = rsqrtf(float(kHeadDim)) * kLog2e;
#pragma unroll
  for (int g = 0; g < GM; ++g) {
    m[g] = -INFINITY;
    l[g] = 0.f;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      acc[g][e] = 0.f;
      q[g][e] = g < G ? __bfloat162float(p.q[(row0 + g) * kHeadDim + 4 * lane + e]) * scale : 0.f;
    }
  }
  const int n_list = p.selected ? p.k : pages;
  for (int i = 0; i < n_list; ++i) {
    const int j = p.selected ? p.selected[(size_t(b) * p.n_kv_heads + h) * p.k + i] : i;
    if (j < 0) continue;
    if (j >= pages) {
      if (threadIdx.x == 0) flag_status(p.status, LOCKS_DEV_BAD_PAGE_ID);
      continue;
    }
    const int blk = p.block_table[size_t(b) * p.max_pages + j];
    if (blk < 0 || blk >= p.num_blocks) {
      if (threadIdx.x == 0) flag_status(p.status, LOCKS_DEV_BAD_BLOCK_ID);
      continue;
    }
    const size_t at = (size_t(blk) * p.n_kv_heads + h) * kv_rec_bytes(FMT, B);
    for (int r = warp; r < B; r += kKvWarps) {
      const int t = j * B + r;
      if (t < lo || t >= n) continue;
      float k[4], v[4];
      load4<FMT>(p.k_pool + at, B, r, lane, k);
      load4<FMT>(p.v_pool + at, B, r, lane, v);
#pragma unroll
      for (int g = 0; g < GM; ++g) {
        float d = q[g][0] * k[0] + q[g][1] * k[1] + q[g][2] * k[2] + q[g][3] * k[3];
        d = group_sum<32>(d);
        const float mn = fmaxf(m[g], d);
        const float a = exp2f(m[g] - mn), w = exp2f(d - mn);
        l[g] = l[g] * a + w;
        m[g] = mn;
#pragma unroll
        for (int e = 0; e < 4; ++e) acc[g][e] = acc[g][e] * a + w * v[e];
      }
    }
  }
#pragma unroll
  for (int g = 0; g < GM; ++g) {
    s_m[warp][g] = m[g];
    s_l[warp][g] = l[g];
  }
#pragma unroll
  for (int g = 0; g < GM; ++g) {
    __syncthreads();
#pragma unroll
    for (int e = 0; e < 4; ++e) s_acc[warp][4 * lane + e] = acc[g][e];
    __syncthreads();
    if (g < G && threadIdx.x < kHeadDim) {
      float M = -INFINITY, L = 0.f, A = 0.f;
      for (int w = 0; w < kKvWarps; ++w) M = fmaxf(M, s_m[w][g]);
      for (int w = 0; w < kKvWarps; ++w) {
        const float f = s_m[w][g] == -INFINITY ? 0.f : exp2f(s_m[w][g] - M);
        L += s_l[w][g] * f;
        A += s_acc[w][threadIdx.x] * f;
      }
      p.out[(row0 + g) * kHeadDim + threadIdx.x] = __float2bfloat16_rn(L == 0.f ? 0.f : A / L);
      if (threadIdx.x == 0 && p.out_lse)
        p.out_lse[row0 + g] = L == 0.f ? -INFINITY : M * kLn2 + logf(L);
    }
  }
}

template <int FMT>
int launch_fmt(const KvDecodeParams& p, cudaStream_t stream) {
  const dim3 grid(unsigned(p.batch) * p.n_kv_heads);
  if (p.group <= 4) return launch_dependent(kv_decode_kernel<FMT, 4>, grid, kKvThreads, 0, p, stream);
  return launch_dependent(kv_decode_kernel<FMT, 16>, grid, kKvThreads, 0, p, stream);
}

}  // namespace

size_t kv_decode_workspace(int, int, int) { return 256; }

int launch_kv_decode(const KvDecodeParams& p, int fmt, cudaStream_t stream) {
  switch (fmt) {
    case LOCKS_KV_F8: return launch_fmt<LOCKS_KV_F8>(p, stream);
    case LOCKS_KV_I8: return launch_fmt<LOCKS_KV_I8>(p, stream);
    case LOCKS_KV_I4: return launch_fmt<LOCKS_KV_I4>(p, stream);
    default: return LOCKS_ERR_INVALID_ARG;
  }
}

}  // namespace locks
