// The layer for given expert choices and gate weights (any router) on gfx950: the layout of
// the choices, the expert rows back at their tokens, and the gradients of both moves.
//
// Operations (the moves themselves: MoK article, kucoin.com/es "Cursor's MoK logra un aumento
// del 2.37x ...", sections 01-03: one expert's rows contiguous, results returned to their
// tokens, the weighted merge):
//   layout:  slot(p) = offsets[l] + rank of pair p among the pairs of local expert l, in
//            (rank, token, j) order
//   merge:   y[t]   = sum_j w[t][j] ye[slot(t, j)]
//   its gradient:        dye[slot(t, j)] = w[t][j] dy[t],   dw[t][j] = <dy[t], ye[slot(t, j)]>
//   the pull's gradient: dx[t] = sum_j dxe[slot(t, j)]
// Every source lies on this GPU, so merge reads the expert rows where the FFN left them: no
// receive buffer, which the push of moe_combine_push writes and its merge reads again.
//
// merge and both gradients are HBM-bound and iterate by token, so each token's row (y, dy,
// dx) moves once whatever k is, and each expert row once.
#include "common.hpp"

namespace moe {

// Histogram of one block's kTokPerLayoutBlock tokens.  A choice outside [-1, E) or an expert
// named twice by one token marks the block in `bad` (one word per block): rows are counted on
// at most one pair per token and expert, so such choices could overrun the tables.
__global__ __launch_bounds__(256) void choices_hist_kernel(const int32_t* __restrict__ idx, int64_t RT, int E, int k,
                                                           int32_t* __restrict__ blockhist, int32_t* __restrict__ bad,
                                                           int bad_stride) {
  __shared__ int hist[1024];
  __shared__ int wrong;
  const int tid = threadIdx.x;
  for (int e = tid; e < E; e += 256) hist[e] = 0;
  if (tid == 0) wrong = 0;
  __syncthreads();
  const int64_t g0 = int64_t(blockIdx.x) * kTokPerLayoutBlock;
  const int64_t p0 = g0 * k, p1 = min(g0 + kTokPerLayoutBlock, RT) * k;
  for (int64_t p = p0 + tid; p < p1; p += 256) {
    const int e = idx[p];
    if (e < -1 || e >= E) {
      wrong = 1;
    } else if (e >= 0) {
      const int64_t first = p - p % k;
      bool twice = false;
      for (int64_t q = first; q < p; ++q) twice |= idx[q] == e;
      if (twice) wrong = 1;
      else atomicAdd(&hist[e], 1);
    }
  }
  __syncthreads();
  for (int e = tid; e < E; e += 256) blockhist[size_t(blockIdx.x) * E + e] = hist[e];
  if (tid == 0) bad[size_t(blockIdx.x) * bad_stride] = wrong;
}

namespace {

__device__ __forceinline__ float wave_sum(float v) {
#pragma unroll
  for (int off = 32; off >= 1; off >>= 1) v += __shfl_xor(v, off, 64);
  return v;
}

template <bool BF16>
__device__ __forceinline__ void unpack(const u32x4 v, float* f) {
  if constexpr (BF16) {
#pragma unroll
    for (int w = 0; w < 4; ++w) {
      f[2 * w] = __uint_as_float(v[w] << 16);
      f[2 * w + 1] = __uint_as_float(v[w] & 0xFFFF0000u);
    }
  } else {
#pragma unroll
    for (int w = 0; w < 4; ++w) f[w] = __uint_as_float(v[w]);
  }
}

// rounds once to the row type (nearest even)
template <bool BF16>
__device__ __forceinline__ u32x4 pack(const float* f) {
  if constexpr (BF16)
    return u32x4{pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]), pack_bf16x2(f[4], f[5]), pack_bf16x2(f[6], f[7])};
  else
    return u32x4{__float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]), __float_as_uint(f[3])};
}

}  // namespace

// y[r][t] = sum over ascending j with slot >= 0 of w[r][t][j] rows[slot] (w = 1 when null); a
// token with none gets zeros.  A wave task is one column segment of 64 * VPL vectors.
template <bool BF16, int VPL>
__global__ __launch_bounds__(256) void merge_rows_kernel(const char* __restrict__ rows, RankPtrs<char*> y,
                                                         const int32_t* __restrict__ slot_of,
                                                         const float* __restrict__ w, int R, int T, int k, int d) {
  constexpr int EPV = BF16 ? 8 : 4;      // elements per 16-byte vector
  const int lane = threadIdx.x & 63;
  const int64_t row_bytes = int64_t(d) * (BF16 ? 2 : 4);
  const int n16 = int(row_bytes >> 4);
  const int nseg = (n16 + 64 * VPL - 1) / (64 * VPL);
  const int64_t tasks = int64_t(R) * T * nseg;
  const int64_t nw = int64_t(gridDim.x) * 4;
  for (int64_t task = int64_t(blockIdx.x) * 4 + (threadIdx.x >> 6); task < tasks; task += nw) {
    const int64_t g = task / nseg;
    const int cb = int(task - g * nseg) * 64 * VPL;
    const int r = int(g / T);
    const int t = int(g - int64_t(r) * T);
    const int slot = lane < k ? slot_of[g * k + lane] : -1;
    const float wl = (w && lane < k) ? w[g * k + lane] : 1.0f;
    float acc[VPL][EPV];
#pragma unroll
    for (int u = 0; u < VPL; ++u)
#pragma unroll
      for (int e = 0; e < EPV; ++e) acc[u][e] = 0.0f;
    for (unsigned long long m = __ballot(slot >= 0); m; m &= m - 1) {
      const int j = __builtin_ctzll(m);
      const int sj = __shfl(slot, j, 64);
      const float wj = __shfl(wl, j, 64);
      const u32x4* src = reinterpret_cast<const u32x4*>(rows + int64_t(sj) * row_bytes);
      u32x4 v[VPL];
#pragma unroll
      for (int u = 0; u < VPL; ++u) {
        const int i = cb + u * 64 + lane;
        if (i < n16) v[u] = __builtin_nontemporal_load(src + i);
      }
#pragma unroll
      for (int u = 0; u < VPL; ++u) {
        if (cb + u * 64 + lane < n16) {
          float f[EPV];
          unpack<BF16>(v[u], f);
#pragma unroll
          for (int e = 0; e < EPV; ++e) acc[u][e] = fmaf(wj, f[e], acc[u][e]);
        }
      }
    }
    u32x4* yrow = reinterpret_cast<u32x4*>(y.p[r] + int64_t(t) * row_bytes);
#pragma unroll
    for (int u = 0; u < VPL; ++u) {
      const int i = cb + u * 64 + lane;
      if (i < n16) __builtin_nontemporal_store(pack<BF16>(acc[u]), yrow + i);
    }
  }
}

// dye[slot] = w dy (rounded once), dw = <dy, ye[slot]> (fp32): one wave per token.  The row goes
// in segments of 64 * VPL vectors; each holds its part of dy in registers for all the token's
// rows, and lane j collects the dot product of pair j.
template <bool BF16, int VPL>
__global__ __launch_bounds__(256) void merge_rows_bwd_kernel(RankPtrs<const char*> dy, const char* __restrict__ ye,
                                                             const int32_t* __restrict__ slot_of,
                                                             const float* __restrict__ w, char* __restrict__ dye,
                                                             float* __restrict__ dw, int R, int T, int k, int d) {
  constexpr int EPV = BF16 ? 8 : 4;
  const int lane = threadIdx.x & 63;
  const int64_t row_bytes = int64_t(d) * (BF16 ? 2 : 4);
  const int n16 = int(row_bytes >> 4);
  const int64_t RT = int64_t(R) * T;
  const int64_t nw = int64_t(gridDim.x) * 4;
  for (int64_t g = int64_t(blockIdx.x) * 4 + (threadIdx.x >> 6); g < RT; g += nw) {
    const int r = int(g / T);
    const int t = int(g - int64_t(r) * T);
    const int slot = lane < k ? slot_of[g * k + lane] : -1;
    const float wl = lane < k ? w[g * k + lane] : 0.0f;
    const unsigned long long local = __ballot(slot >= 0);
    float mine = 0.0f;                      // lane j: the dot product of pair j
    const u32x4* dyr = reinterpret_cast<const u32x4*>(dy.p[r] + int64_t(t) * row_bytes);
    if (local) {
      for (int cb = 0; cb < n16; cb += 64 * VPL) {
        u32x4 dv[VPL];
#pragma unroll
        for (int u = 0; u < VPL; ++u) {
          const int i = cb + u * 64 + lane;
          dv[u] = u32x4{0, 0, 0, 0};
          if (i < n16) dv[u] = __builtin_nontemporal_load(dyr + i);
        }
        for (unsigned long long m = local; m; m &= m - 1) {
          const int j = __builtin_ctzll(m);
          const int64_t at = int64_t(__shfl(slot, j, 64)) * row_bytes;
          const float wj = __shfl(wl, j, 64);
          const u32x4* src = reinterpret_cast<const u32x4*>(ye + at);
          u32x4* dst = reinterpret_cast<u32x4*>(dye + at);
          u32x4 v[VPL];
#pragma unroll
          for (int u = 0; u < VPL; ++u) {
            const int i = cb + u * 64 + lane;
            v[u] = u32x4{0, 0, 0, 0};
            if (i < n16) v[u] = __builtin_nontemporal_load(src + i);
          }
          float dot = 0.0f;
#pragma unroll
          for (int u = 0; u < VPL; ++u) {
            const int i = cb + u * 64 + lane;
            float a[EPV], b[EPV];
            unpack<BF16>(dv[u], a);
            unpack<BF16>(v[u], b);
#pragma unroll
            for (int e = 0; e < EPV; ++e) {
              dot = fmaf(a[e], b[e], dot);
              a[e] *= wj;
            }
            if (i < n16) dst[i] = pack<BF16>(a);
          }
          dot = wave_sum(dot);
          if (lane == j) mine += dot;
        }
      }
    }
    if (lane < k) dw[g * k + lane] = mine;
  }
}

constexpr int kMergeRowsBlocksPerCU = 16, kMergeBwdBlocksPerCU = 8;

hipError_t launch_choices_hist(const moe_shape_t& s, const int32_t* idx, int32_t* blockhist, int32_t* bad, int El,
                               int nb, hipStream_t st) {
  hipLaunchKernelGGL(choices_hist_kernel, dim3(nb), dim3(256), 0, st, idx, int64_t(s.R) * s.T, s.E, s.k, blockhist, bad,
                     El);
  return hipGetLastError();
}

hipError_t launch_merge_rows(const moe_shape_t& s, const void* rows, const int32_t* slot_of, const float* w,
                             void* const* y, int cus, hipStream_t st) {
  RankPtrs<char*> yp{};
  for (int r = 0; r < s.R; ++r) yp.p[r] = static_cast<char*>(y[r]);
  const dim3 grid(cus * kMergeRowsBlocksPerCU);
  if (s.dtype != MOE_F32)
    hipLaunchKernelGGL((merge_rows_kernel<true, 4>), grid, dim3(256), 0, st, static_cast<const char*>(rows), yp, slot_of,
                       w, s.R, s.T, s.k, s.d);
  else
    hipLaunchKernelGGL((merge_rows_kernel<false, 4>), grid, dim3(256), 0, st, static_cast<const char*>(rows), yp, slot_of,
                       w, s.R, s.T, s.k, s.d);
  return hipGetLastError();
}

hipError_t launch_merge_rows_bwd(const moe_shape_t& s, const void* const* dy, const void* ye, const int32_t* slot_of,
                                 const float* w, void* dye, float* dw, int cus, hipStream_t st) {
  RankPtrs<const char*> dp{};
  for (int r = 0; r < s.R; ++r) dp.p[r] = static_cast<const char*>(dy[r]);
  const dim3 grid(cus * kMergeBwdBlocksPerCU);
  if (s.dtype != MOE_F32)
    hipLaunchKernelGGL((merge_rows_bwd_kernel<true, 4>), grid, dim3(256), 0, st, dp, static_cast<const char*>(ye),
                       slot_of, w, static_cast<char*>(dye), dw, s.R, s.T, s.k, s.d);
  else
    hipLaunchKernelGGL((merge_rows_bwd_kernel<false, 4>), grid, dim3(256), 0, st, dp, static_cast<const char*>(ye),
                       slot_of, w, static_cast<char*>(dye), dw, s.R, s.T, s.k, s.d);
  return hipGetLastError();
}

}  // namespace moe
