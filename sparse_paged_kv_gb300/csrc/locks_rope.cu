// locks_rope: rotary positions of query and key rows, and the rotation rates.
//
//   (u, v) -> (u c - v s, v c + u s),   c, s = mscale * cos, sin(p w_i)
//
// One read and one write of every element: bound by memory (32768 tokens x 40
// heads of 128 in bf16: 100 us, 0.99 of the copy rate).  A thread owns VEC
// pairs of a token (the same pairs in every head), computes their cos and sin
// once, and walks the heads of its chunk; neighbouring threads own neighbouring
// pairs, so a row's loads and stores are whole 128-byte lines.
#include <algorithm>
#include <cmath>

#include "locks_kv.cuh"

namespace locks {

namespace {

constexpr int kRopeThreads = 256;
constexpr int64_t kRopeStreamBytes = int64_t(64) << 20;   // read and written, half of L2

template <typename T>
__device__ __forceinline__ float to_f(T x);
template <>
__device__ __forceinline__ float to_f(float x) { return x; }
template <>
__device__ __forceinline__ float to_f(__half x) { return __half2float(x); }
template <>
__device__ __forceinline__ float to_f(__nv_bfloat16 x) { return __bfloat162float(x); }
template <typename T>
__device__ __forceinline__ T from_f(float x);
template <>
__device__ __forceinline__ float from_f(float x) { return x; }
template <>
__device__ __forceinline__ __half from_f(float x) { return __float2half_rn(x); }
template <>
__device__ __forceinline__ __nv_bfloat16 from_f(float x) { return __float2bfloat16_rn(x); }

// N consecutive elements, N * sizeof(T) a multiple of 4 or one element.  STREAM:
// with the hint that the line is used once.
template <typename T, int N>
struct Pack {
  static constexpr int kBytes = N * int(sizeof(T));
  T e[N];
  template <bool STREAM>
  __device__ __forceinline__ void load(const T* p) {
    if constexpr (kBytes % 16 == 0) {
#pragma unroll
      for (int i = 0; i < kBytes / 16; ++i) {
        const uint4* at = reinterpret_cast<const uint4*>(p) + i;
        reinterpret_cast<uint4*>(e)[i] = STREAM ? __ldcs(at) : *at;
      }
    } else if constexpr (kBytes % 8 == 0) {
      const uint2* at = reinterpret_cast<const uint2*>(p);
      *reinterpret_cast<uint2*>(e) = STREAM ? __ldcs(at) : *at;
    } else if constexpr (kBytes % 4 == 0) {
      const uint32_t* at = reinterpret_cast<const uint32_t*>(p);
      *reinterpret_cast<uint32_t*>(e) = STREAM ? __ldcs(at) : *at;
    } else {
#pragma unroll
      for (int i = 0; i < N; ++i) e[i] = p[i];
    }
  }
  template <bool STREAM>
  __device__ __forceinline__ void store(T* p) const {
    if constexpr (kBytes % 16 == 0) {
#pragma unroll
      for (int i = 0; i < kBytes / 16; ++i) {
        uint4* at = reinterpret_cast<uint4*>(p) + i;
        if (STREAM) __stcs(at, reinterpret_cast<const uint4*>(e)[i]);
        else *at = reinterpret_cast<const uint4*>(e)[i];
      }
    } else if constexpr (kBytes % 8 == 0) {
      uint2* at = reinterpret_cast<uint2*>(p);
      if (STREAM) __stcs(at, *reinterpret_cast<const uint2*>(e));
      else *at = *reinterpret_cast<const uint2*>(e);
    } else if constexpr (kBytes % 4 == 0) {
      uint32_t* at = reinterpret_cast<uint32_t*>(p);
      if (STREAM) __stcs(at, *reinterpret_cast<const uint32_t*>(e));
      else *at = *reinterpret_cast<const uint32_t*>(e);
    } else {
#pragma unroll
      for (int i = 0; i < N; ++i) p[i] = e[i];
    }
  }
};

// u and v in place: VEC pairs, in the half layout (u, v) element by element, in
// the interleaved one neighbours
template <typename T, int VEC>
__device__ __forceinline__ void turn_pairs(Pack<T, VEC>& u, Pack<T, VEC>& v, const float (&c)[VEC],
                                           const float (&s)[VEC], bool half) {
  if (half || VEC == 1) {
#pragma unroll
    for (int i = 0; i < VEC; ++i) {
      const float fu = to_f(u.e[i]), fv = to_f(v.e[i]);
      u.e[i] = from_f<T>(rope_u(fu, fv, c[i], s[i]));
      v.e[i] = from_f<T>(rope_v(fu, fv, c[i], s[i]));
    }
  } else {
    constexpr int kHalfVec = VEC / 2;
#pragma unroll
    for (int i = 0; i < kHalfVec; ++i) {
      float fu = to_f(u.e[2 * i]), fv = to_f(u.e[2 * i + 1]);
      u.e[2 * i] = from_f<T>(rope_u(fu, fv, c[i], s[i]));
      u.e[2 * i + 1] = from_f<T>(rope_v(fu, fv, c[i], s[i]));
      fu = to_f(v.e[2 * i]);
      fv = to_f(v.e[2 * i + 1]);
      v.e[2 * i] = from_f<T>(rope_u(fu, fv, c[kHalfVec + i], s[kHalfVec + i]));
      v.e[2 * i + 1] = from_f<T>(rope_v(fu, fv, c[kHalfVec + i], s[kHalfVec + i]));
    }
  }
}

template <typename T, int VEC, bool STREAM>
__global__ void __launch_bounds__(kRopeThreads) rope_kernel(const RopeParams p) {
  const int n = p.rope.rotary_dim / 2;
  const int items = n / VEC + (p.head_dim - 2 * n) / (2 * VEC);
  const int slots = kRopeThreads / items;
  const int item = threadIdx.x % items, slot = threadIdx.x / items;
  const int64_t task = int64_t(blockIdx.x) * slots + slot;
  griddep_launch();
  griddep_wait();
  if (slot >= slots || task >= int64_t(p.n_tokens) * p.n_chunks) return;
  const int64_t token = task / p.n_chunks;
  const int first = int(task % p.n_chunks);
  const bool turn = item < n / VEC;
  // element offsets of the two packs this thread moves
  int a, b;
  if (!turn) {
    a = 2 * n + (item - n / VEC) * 2 * VEC;
    b = a + VEC;
  } else if (p.rope.layout == LOCKS_ROPE_HALF) {
    a = item * VEC;
    b = a + n;
  } else {
    a = item * 2 * VEC;
    b = a + VEC;
  }
  alignas(16) float c[VEC], s[VEC];
  if (turn) {
    const int32_t pos = p.positions[token];
#pragma unroll
    for (int i = 0; i < VEC; ++i) {
      rope_cos_sin(__ldg(p.rope.turns + item * VEC + i), pos, p.rope.mscale, c[i], s[i]);
      if (p.inverse) s[i] = -s[i];
    }
  }
  const T* x = static_cast<const T*>(p.x) + token * p.x_ts;
  T* o = static_cast<T*>(p.out) + token * p.o_ts;
  const bool half = p.rope.layout == LOCKS_ROPE_HALF;
  constexpr int kAhead = STREAM ? 4 : 1;          // heads loaded before any is stored
#pragma unroll 1
  for (int h0 = first; h0 < p.n_heads; h0 += kAhead * p.n_chunks) {
    alignas(16) Pack<T, VEC> u[kAhead], v[kAhead];
#pragma unroll
    for (int i = 0; i < kAhead; ++i) {
      const int h = h0 + i * p.n_chunks;
      if (h < p.n_heads) {
        u[i].template load<STREAM>(x + h * p.x_hs + a);
        v[i].template load<STREAM>(x + h * p.x_hs + b);
      }
    }
#pragma unroll
    for (int i = 0; i < kAhead; ++i) {
      const int h = h0 + i * p.n_chunks;
      if (h < p.n_heads) {
        if (turn) turn_pairs(u[i], v[i], c, s, half);
        u[i].template store<STREAM>(o + h * p.o_hs + a);
        v[i].template store<STREAM>(o + h * p.o_hs + b);
      }
    }
  }
}

template <typename T, int VEC>
int launch_rope_vec(RopeParams p, cudaStream_t stream) {
  const int n = p.rope.rotary_dim / 2;
  const int items = n / VEC + (p.head_dim - 2 * n) / (2 * VEC);
  const int slots = kRopeThreads / items;
  // heads a thread walks: as many as leave 8 blocks per SM, at most 8 (the
  // angles are then a small share of the work)
  const int64_t rows = int64_t(p.n_tokens) * p.n_heads;
  int64_t per = rows / (int64_t(152) * 8 * slots);
  per = per < 1 ? 1 : (per > 8 ? 8 : per);
  p.n_chunks = int((p.n_heads + per - 1) / per);
  const int64_t blocks = (int64_t(p.n_tokens) * p.n_chunks + slots - 1) / slots;
  if (blocks > 0x7fffffff) return LOCKS_ERR_UNSUPPORTED;
  // Tensors too large to stay in L2: four heads in flight a thread, and every
  // line marked as used once.  Smaller ones are left in L2 for the call that reads
  // them next.  40 heads of 128 in bf16, us with and without: 32768 tokens 100.4,
  // 104.7 (the copy rate is 99); 8192 28.3, 30.3; 4096 (84 MB) 15.9, 17.3; 2048
  // (42 MB) 11.2, 10.8; 1024 9.0, 7.2.
  const int64_t bytes = 2 * rows * p.head_dim * int64_t(sizeof(T));
  auto kern = bytes > kRopeStreamBytes ? rope_kernel<T, VEC, true> : rope_kernel<T, VEC, false>;
  return launch_dependent(kern, dim3(unsigned(blocks)), kRopeThreads, 0, p, stream);
}

// Widest pack that divides the pairs, the copied rest and the addresses.
template <typename T>
int launch_rope_t(const RopeParams& p, cudaStream_t stream) {
  const int n = p.rope.rotary_dim / 2, rest = p.head_dim - 2 * n;
  auto fits = [&](int vec) {
    const int64_t unit = std::min(16, vec * int(sizeof(T)));   // bytes a load must be aligned to
    const int64_t el = unit / int(sizeof(T));
    return n % vec == 0 && rest % (2 * vec) == 0 && p.x_ts % el == 0 && p.x_hs % el == 0 &&
           p.o_ts % el == 0 && p.o_hs % el == 0 && reinterpret_cast<uintptr_t>(p.x) % unit == 0 &&
           reinterpret_cast<uintptr_t>(p.out) % unit == 0;
  };
  if (fits(8)) return launch_rope_vec<T, 8>(p, stream);
  if (fits(4)) return launch_rope_vec<T, 4>(p, stream);
  if (fits(2)) return launch_rope_vec<T, 2>(p, stream);
  return launch_rope_vec<T, 1>(p, stream);
}

}  // namespace

int launch_rope(RopeParams p, int dtype, cudaStream_t stream) {
  switch (dtype) {
    case LOCKS_BF16: return launch_rope_t<__nv_bfloat16>(p, stream);
    case LOCKS_F16: return launch_rope_t<__half>(p, stream);
    case LOCKS_F32: return launch_rope_t<float>(p, stream);
    default: return LOCKS_ERR_INVALID_ARG;
  }
}

}  // namespace locks

extern "C" int locks_rope_frequencies(const locks_rope_spec_t* spec, uint64_t* turns,
                                      float* mscale) {
  if (!spec || !turns || !mscale) return LOCKS_ERR_INVALID_ARG;
  const int r = spec->rotary_dim, kind = spec->scaling;
  if (r < 2 || r % 2 || !(spec->theta > 1.0) || !std::isfinite(spec->theta))
    return LOCKS_ERR_INVALID_ARG;
  if (kind < LOCKS_ROPE_SCALE_NONE || kind > LOCKS_ROPE_SCALE_YARN) return LOCKS_ERR_INVALID_ARG;
  if (kind != LOCKS_ROPE_SCALE_NONE && !(spec->factor >= 1.0 && std::isfinite(spec->factor)))
    return LOCKS_ERR_INVALID_ARG;
  if (kind == LOCKS_ROPE_SCALE_NTK && r == 2) return LOCKS_ERR_INVALID_ARG;
  if ((kind == LOCKS_ROPE_SCALE_LLAMA3 || kind == LOCKS_ROPE_SCALE_YARN) &&
      !(spec->original_positions > 0.0))
    return LOCKS_ERR_INVALID_ARG;
  if (kind == LOCKS_ROPE_SCALE_LLAMA3 &&
      !(spec->low_freq_factor > 0.0 && spec->high_freq_factor > spec->low_freq_factor))
    return LOCKS_ERR_INVALID_ARG;
  if (kind == LOCKS_ROPE_SCALE_YARN && !(spec->beta_fast > 0.0 && spec->beta_slow > 0.0))
    return LOCKS_ERR_INVALID_ARG;
  if (r > 512) return LOCKS_ERR_UNSUPPORTED;
  constexpr double kPi = 3.14159265358979323846;
  double theta = spec->theta;
  if (kind == LOCKS_ROPE_SCALE_NTK) theta *= std::pow(spec->factor, double(r) / (r - 2));
  double lo = 0.0, hi = 0.0;
  if (kind == LOCKS_ROPE_SCALE_YARN) {
    auto dim_of = [&](double t) {
      return r * std::log(spec->original_positions / (2 * kPi * t)) / (2 * std::log(theta));
    };
    lo = std::fmax(0.0, std::floor(dim_of(spec->beta_fast)));
    hi = std::fmin(double(r - 1), std::ceil(dim_of(spec->beta_slow)));
  }
  *mscale = kind == LOCKS_ROPE_SCALE_YARN ? float(0.1 * std::log(spec->factor) + 1.0) : 1.f;
  for (int i = 0; i < r / 2; ++i) {
    double w = std::pow(theta, -2.0 * i / r);
    if (kind == LOCKS_ROPE_SCALE_LINEAR) {
      w /= spec->factor;
    } else if (kind == LOCKS_ROPE_SCALE_LLAMA3) {
      // share kept at the original rate: 0 below low_freq_factor turns of the
      // original context, 1 above high_freq_factor
      const double turns_ctx = spec->original_positions * w / (2 * kPi);
      double z = (turns_ctx - spec->low_freq_factor) /
                 (spec->high_freq_factor - spec->low_freq_factor);
      z = std::fmin(1.0, std::fmax(0.0, z));
      w = (1 - z) * w / spec->factor + z * w;
    } else if (kind == LOCKS_ROPE_SCALE_YARN) {
      double z = (i - lo) / std::fmax(hi - lo, 1e-3);
      z = std::fmin(1.0, std::fmax(0.0, z));
      w = w / spec->factor * z + w * (1 - z);
    }
    // w <= 1: below 2^62.  (The half rounds the slow pairs; the fast ones' doubles end above it.)
    turns[i] = uint64_t(std::ldexp(w / (2 * kPi), 64) + 0.5);
  }
  return LOCKS_OK;
}
