// What the products grouped by expert share: the groups' rows, checked, and the map from row tiles to groups.
#pragma once

#include "common.hpp"

namespace moe {

constexpr int kMaxGroups = 1024;

struct GroupedArgs {
  const void* x;
  const void* w;
  void* y;
  const int32_t* offsets;
  int32_t* status;
  int64_t rows, ldx, ldy;
  int G, K, N;
};

// The row tiles of all groups, by one workgroup of THREADS (a multiple of 64) threads: base[g] is the first of group g's
// ceil(rows / BM) tiles, base[G] their number (returned in every thread).  Offsets that descend or leave [0, rows] give
// no tiles at all, and *bad is set.  base: G + 1 words of LDS, part: THREADS / 64 + 1.
template <int THREADS>
__device__ __forceinline__ int group_tiles(const int32_t* __restrict__ offsets, int G, int64_t rows, int bm_log2,
                                           int32_t* base, int32_t* part, bool* bad) {
  constexpr int kPer = (kMaxGroups + THREADS - 1) / THREADS;
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  int n[kPer], sum = 0, wrong = 0;
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    const int g = tid * kPer + i;
    n[i] = 0;
    if (g < G) {
      const int a = offsets[g], b = offsets[g + 1];
      if (a < 0 || b < a || b > rows) wrong = 1;
      else n[i] = (b - a + (1 << bm_log2) - 1) >> bm_log2;
    }
    sum += n[i];
  }
  if (tid == 0) part[THREADS / 64] = 0;
  __syncthreads();
  if (wrong) part[THREADS / 64] = 1;
  int upto = sum;                                   // inclusive over the wave
#pragma unroll
  for (int o = 1; o < 64; o <<= 1) {
    const int t = __shfl_up(upto, o);
    if (lane >= o) upto += t;
  }
  if (lane == 63) part[wave] = upto;
  __syncthreads();
  wrong = part[THREADS / 64];
  int before = upto - sum, total = 0;
#pragma unroll
  for (int w = 0; w < THREADS / 64; ++w) {
    if (w < wave) before += part[w];
    total += part[w];
  }
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    const int g = tid * kPer + i;
    if (g < G) base[g] = before;
    before += n[i];
  }
  if (tid == 0) base[G] = total;
  __syncthreads();
  *bad = wrong != 0;
  return wrong ? 0 : total;
}

}  // namespace moe
