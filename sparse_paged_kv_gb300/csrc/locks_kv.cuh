// Shared by the quantised-cache kernels: record geometry, the parameter blocks
// of the launchers, the rotary angle and the conversions between codes and
// floats.  Internal to the library; the record is described in locks.h.
#pragma once

#include <atomic>

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "locks_common.cuh"

namespace locks {

constexpr int kKvMaxGroup = 16;
// rows with no larger magnitude are stored as zeros: 1 / scale stays finite
constexpr float kKvTiny = 1.2621774483536189e-29f;   // 2^-96

__host__ __device__ constexpr int kv_row_bytes(int fmt) { return fmt == LOCKS_KV_I4 ? 64 : 128; }
// byte offsets in a record of page_size rows
__host__ __device__ constexpr int kv_group_off(int fmt, int B) { return B * kv_row_bytes(fmt); }
__host__ __device__ constexpr int kv_scale_off(int fmt, int B) {
  return kv_group_off(fmt, B) + (fmt == LOCKS_KV_I4 ? 4 * B : 0);
}
__host__ __device__ constexpr int kv_rec_bytes(int fmt, int B) { return kv_scale_off(fmt, B) + 4 * B; }
// byte of 16-byte chunk c of row r
template <int FMT>
__host__ __device__ constexpr int kv_chunk_off(int r, int c) {
  return FMT == LOCKS_KV_I4 ? r * 64 + 16 * (c ^ ((r >> 1) & 3)) : r * 128 + 16 * (c ^ (r & 7));
}

struct RopeArgs {
  const uint64_t* turns;         // [rotary_dim / 2]; NULL: no rotation
  int rotary_dim, layout;
  float mscale;
};

struct RopeParams {
  RopeArgs rope;
  const void* x;
  void* out;
  const int32_t* positions;
  int64_t x_ts, x_hs, o_ts, o_hs;   // strides in elements
  int n_tokens, n_heads, head_dim;
  int inverse;
  int n_chunks;                  // head chunks per token (set by the launcher)
};

struct KvWriteParams {
  const __nv_bfloat16 *k_new, *v_new, *q_new;
  __nv_bfloat16* q_out;
  int64_t k_stride, v_stride, q_stride;
  const int32_t *token_seq, *token_pos;
  RopeArgs rope;
  unsigned char *k_pool, *v_pool;
  const int32_t* block_table;
  int32_t *seq_lens, *completed, *status;
  int n_tokens, batch, n_q_heads, n_kv_heads, max_pages, num_blocks, page_size;
  int n_chunks;                  // runs of a token's rows (set by the launcher)
};

struct KvReadParams {
  const unsigned char *k_pool, *v_pool;
  const int32_t* block_ids;
  __nv_bfloat16 *k_out, *v_out;
  int32_t* status;
  int n_blocks, n_kv_heads, num_blocks, page_size;
};

struct KvDecodeParams {
  const __nv_bfloat16* q;        // [batch][H_q][d]
  const unsigned char *k_pool, *v_pool;
  const int32_t* block_table;    // [batch][max_pages]
  const int32_t* seq_lens;       // [batch]
  const int32_t* selected;       // nullable: [batch][H_kv][k]
  __nv_bfloat16* out;            // [batch][H_q][d]
  float* out_lse;                // nullable [batch][H_q]
  int32_t* status;               // nullable
  unsigned char* ws;
  int batch, n_kv_heads, group, max_pages, num_blocks, page_size;
  int k, window;
};

int launch_rope(RopeParams p, int dtype, cudaStream_t stream);
int launch_kv_write(KvWriteParams p, int fmt, cudaStream_t stream);
int launch_kv_read(const KvReadParams& p, int fmt, cudaStream_t stream);
size_t kv_decode_workspace(int group);
int launch_kv_decode(const KvDecodeParams& p, int fmt, cudaStream_t stream);

// A kernel attribute holds for the device it was set on: `run` calls set() on
// the first launch there (and again after a failure).
struct LaunchOnce {
  std::atomic<uint64_t> ready{0};
  template <typename F>
  bool run(F set) {
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return false;
    const uint64_t bit = dev < 64 ? uint64_t(1) << dev : 0;
    if (ready.load(std::memory_order_acquire) & bit) return true;
    if (!set()) return false;
    ready.fetch_or(bit, std::memory_order_release);
    return true;
  }
};

// Launches with the programmatic-serialization attribute: the kernel may start
// while the one before it on the stream drains, and waits (griddep_wait) before
// it touches memory that one may write.
template <typename P>
int launch_dependent(void (*kern)(P), dim3 grid, int threads, size_t smem, const P& p,
                     cudaStream_t stream) {
  cudaLaunchConfig_t lc = {};
  lc.gridDim = grid;
  lc.blockDim = dim3(threads);
  lc.dynamicSmemBytes = smem;
  lc.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  lc.attrs = attr;
  lc.numAttrs = 1;
  return cudaLaunchKernelEx(&lc, kern, p) == cudaSuccess ? LOCKS_OK : LOCKS_ERR_CUDA;
}

#ifdef __CUDACC__
__device__ __forceinline__ void griddep_wait() {
  asm volatile("griddepcontrol.wait;" ::: "memory");
}
__device__ __forceinline__ void griddep_launch() {
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
}

// cos and sin of position * w, times mscale.  `turns` is w / 2 pi as a 64-bit
// fraction of a turn: the product modulo 2^64 is the fractional turn, with no
// error but the rate's own (a double's: 2^-55 of a turn a position).  (A float32
// product position * w would be off by 2^-24 of up to 10^6 radians.)  Its top 32 bits are split, as integers, into the nearest
// quarter turn and a remainder within an eighth, whose angle |a| <= pi / 4 goes
// through the Taylor series of sine and cosine: the first terms left out are
// a^11 / 11! < 2e-9 and a^12 / 12! < 2e-10, and with float32's roundings both are
// within 2^-23.  About 30 instructions, half of what
// sincospi takes, which has to find the quarter turn in floating point.
__device__ __forceinline__ void rope_cos_sin(uint64_t turns, int32_t pos, float mscale, float& c,
                                             float& s) {
  const uint64_t ph = turns * static_cast<uint64_t>(static_cast<int64_t>(pos));
  const uint32_t hi = static_cast<uint32_t>(ph >> 32);
  const uint32_t quarter = (hi + 0x20000000u) >> 30;
  const float a = static_cast<float>(static_cast<int32_t>(hi - (quarter << 30))) *
                  1.4629180792671596e-9f;          // 2 pi / 2^32
  const float t = a * a;
  float ps = fmaf(t, 1.f / 362880.f, -1.f / 5040.f);
  ps = fmaf(t, ps, 1.f / 120.f);
  ps = fmaf(t, ps, -1.f / 6.f);
  ps = fmaf(a * t, ps, a);
  float pc = fmaf(t, -1.f / 3628800.f, 1.f / 40320.f);
  pc = fmaf(t, pc, -1.f / 720.f);
  pc = fmaf(t, pc, 1.f / 24.f);
  pc = fmaf(t, pc, -0.5f);
  pc = fmaf(t, pc, 1.f);
  const bool odd = quarter & 1;
  const float cc = odd ? ps : pc, ss = odd ? pc : ps;
  // cos is negative in quarters 1 and 2, sin in 2 and 3
  c = __uint_as_float(__float_as_uint(cc) ^ (((quarter + 1) & 2u) << 30)) * mscale;
  s = __uint_as_float(__float_as_uint(ss) ^ ((quarter & 2u) << 30)) * mscale;
}

// u c - v s and v c + u s with every product rounded (no contraction), so that
// what is quantised from them does not depend on how the code was compiled
__device__ __forceinline__ float rope_u(float u, float v, float c, float s) {
  return __fsub_rn(__fmul_rn(u, c), __fmul_rn(v, s));
}
__device__ __forceinline__ float rope_v(float u, float v, float c, float s) {
  return __fadd_rn(__fmul_rn(v, c), __fmul_rn(u, s));
}

// two e4m3 codes (lo in bits 0-7, hi in bits 8-15) <-> floats
__device__ __forceinline__ uint32_t e4m3x2(float lo, float hi) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
  return r;
}
__device__ __forceinline__ uint32_t e4m3x2_to_f16x2(uint32_t codes) {
  uint32_t r;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"(static_cast<uint16_t>(codes)));
  return r;
}
__device__ __forceinline__ float2 e4m3x2_to_f2(uint32_t codes) {
  const uint32_t h = e4m3x2_to_f16x2(codes);
  return __half22float2(*reinterpret_cast<const __half2*>(&h));
}
#endif

}  // namespace locks
