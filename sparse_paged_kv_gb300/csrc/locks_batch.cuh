// The list of work of a persistent launch: entries (sequences, groups) of so many stages each, one
// behind another, of which every block takes an equal share.
#pragma once

#include <cstdint>

#include "locks_common.cuh"

namespace locks {

struct ListPlace {
  int entry, offset;      // where the block's share begins: entry, and stages into it
  int scan[32];
};

// A list of `total` in equal parts for as many blocks as get `least` of it each, up to `most`: block b
// begins at floor(total * b / blocks), in 32 bits.
struct Split {
  int total, blocks, each, rest;
  float inv;
  __device__ __forceinline__ Split(int total, int least, int most)
      : total(total), blocks(min(max(total / least, 1), most)), each(total / blocks),
        rest(total - each * blocks), inv(1.f / float(blocks)) {}
  // (b * rest < 2^15, at least half a 152nd away from the next integer)
  __device__ __forceinline__ int begin(int b) const {
    return b >= blocks ? total : b * each + int((float(b * rest) + 0.5f) * inv);
  }
  // the block at a place of the list: an estimate, put right
  __device__ __forceinline__ int block_of(int x) const {
    int b = min(blocks - 1, int(float(x) * float(blocks) / float(total)));
    while (begin(b + 1) <= x) ++b;
    while (begin(b) > x) --b;
    return b;
  }
};

// Every thread of the block calls it; returns the block's share and fills place.  stages(e) is asked for
// every entry: a thread has ceil(entries / THREADS) neighbouring ones.  `visit(e, first)` is called
// for each entry by the thread that has it.  Ends with a __syncthreads().
template <int THREADS, typename Stages, typename Visit>
__device__ int locate(Stages stages, int entries, int block, int least, int most, ListPlace& place,
                      int& total, Visit visit) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int each = (entries + THREADS - 1) / THREADS;
  const int e_lo = min(entries, tid * each), e_hi = min(entries, e_lo + each);
  int sum = 0;
  for (int e = e_lo; e < e_hi; ++e) sum += stages(e);
  int before = sum;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int x = __shfl_up_sync(kFull, before, o);
    if (lane >= o) before += x;
  }
  if (lane == 31) place.scan[warp] = before;
  before -= sum;
  __syncthreads();
  total = 0;
  for (int i = 0; i < THREADS / 32; ++i) {
    if (i < warp) before += place.scan[i];
    total += place.scan[i];
  }
  const Split split(total, least, most);
  const int lo = split.begin(block), share = split.begin(block + 1) - lo;
  int at = before;
  for (int e = e_lo; e < e_hi; ++e) {
    const int n = each == 1 ? sum : stages(e);
    if (share > 0 && lo >= at && lo < at + n) {
      place.entry = e;
      place.offset = lo - at;
    }
    visit(e, at);
    at += n;
  }
  __syncthreads();
  return share;
}

template <int THREADS, typename Stages>
__device__ int locate(Stages stages, int entries, int block, int least, int most, ListPlace& place) {
  int total;
  return locate<THREADS>(stages, entries, block, least, most, place, total, [](int, int) {});
}

}  // namespace locks
