// The layer for given expert choices and gate weights (any router) on gfx950: the expert rows
// back at their tokens, and the gradients of both moves (the layout of the choices itself is in
// layout.hip).
//
// Operations (the moves themselves: MoK article, kucoin.com/es "Cursor's MoK logra un aumento
// del 2.37x ...", sections 01-03: results returned to their tokens, the weighted merge):
//   merge:               y[t] = sum_j w[t][j] ye[slot(t, j)]
//   its gradient:        dye[slot(t, j)] = w[t][j] dy[t],   dw[t][j] = <dy[t], ye[slot(t, j)]>
//   the pull's gradient: dx[t] = sum_j dxe[slot(t, j)]
// Every source lies on this GPU, so merge reads the expert rows where the FFN left them: no
// receive buffer, which the push of moe_combine_push writes and its merge reads again.
//
// merge and both gradients are HBM-bound and iterate by token, so each token's row (y, dy,
// dx) moves once whatever k is, and each expert row once.  32768 tokens and expert rows of 7168 bf16:
// merge and pull's gradient 141 us (0.94 GB, 6.7 TB/s), merge's gradient 187 us (1.25 GB, 6.7 TB/s).
#include "common.hpp"

namespace moe {

namespace {

__device__ __forceinline__ float wave_sum(float v) {
#pragma unroll
  for (int off = 32; off >= 1; off >>= 1) v += __shfl_xor(v, off, 64);
  return v;
}

// lane j's value, j the same in every lane
__device__ __forceinline__ float read_lane(float v, int j) {
  return __uint_as_float(uint32_t(__builtin_amdgcn_readlane(int(__float_as_uint(v)), j)));
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
// token with none gets zeros.  A wave task is one column segment of 64 * VPL vectors of one
// token's row; JB of the token's expert rows are in flight at once.  BF16: bf16 rows and y; else fp32 rows,
// and fp32 or (Y16) bf16 y.
template <bool BF16, int VPL, int JB, bool Y16 = BF16>
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
    for (unsigned long long m = __ballot(slot >= 0); m;) {
      const int n = __popcll(m);             // rows left (the same in every lane)
      u32x4 v[JB][VPL];
      float wj[JB];
#pragma unroll
      for (int b = 0; b < JB; ++b) {
        if (b >= n) continue;
        const int j = __builtin_ctzll(m);
        m &= m - 1;
        wj[b] = read_lane(wl, j);
        const u32x4* src = reinterpret_cast<const u32x4*>(rows + int64_t(__builtin_amdgcn_readlane(slot, j)) * row_bytes);
#pragma unroll
        for (int u = 0; u < VPL; ++u) {
          const int i = cb + u * 64 + lane;
          if (i < n16) v[b][u] = __builtin_nontemporal_load(src + i);
        }
      }
#pragma unroll
      for (int b = 0; b < JB; ++b) {
        if (b >= n) continue;
#pragma unroll
        for (int u = 0; u < VPL; ++u) {
          if (cb + u * 64 + lane < n16) {
            float f[EPV];
            unpack<BF16>(v[b][u], f);
#pragma unroll
            for (int e = 0; e < EPV; ++e) acc[u][e] = fmaf(wj[b], f[e], acc[u][e]);
          }
        }
      }
    }
    char* const yrow = y.p[r] + int64_t(t) * d * (Y16 ? 2 : 4);
#pragma unroll
    for (int u = 0; u < VPL; ++u) {
      const int i = cb + u * 64 + lane;
      if (i >= n16) continue;
      if constexpr (Y16 && !BF16)
        reinterpret_cast<uint2*>(yrow)[i] = make_uint2(pack_bf16x2(acc[u][0], acc[u][1]), pack_bf16x2(acc[u][2], acc[u][3]));
      else
        __builtin_nontemporal_store(pack<BF16>(acc[u]), reinterpret_cast<u32x4*>(yrow) + i);
    }
  }
}

// dye[slot] = w dy (rounded once), dw = <dy, ye[slot]> (fp32).  WPT waves (1 or the workgroup's 4)
// share a token; the row goes in segments of 64 * VPL vectors, wave after wave; a segment of dy
// stays in registers for all the token's rows, JB of which are in flight at once, and lane j
// collects the dot product of pair j.
template <bool BF16, int VPL, int JB, int WPT>
__global__ __launch_bounds__(256) void merge_rows_bwd_kernel(RankPtrs<const char*> dy, const char* __restrict__ ye,
                                                             const int32_t* __restrict__ slot_of,
                                                             const float* __restrict__ w, char* __restrict__ dye,
                                                             float* __restrict__ dw, int R, int T, int k, int d) {
  constexpr int EPV = BF16 ? 8 : 4;
  __shared__ float part[4][16];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int64_t row_bytes = int64_t(d) * (BF16 ? 2 : 4);
  const int n16 = int(row_bytes >> 4);
  const int64_t RT = int64_t(R) * T;
  const int first = WPT == 1 ? 0 : wave;
  const int64_t step = int64_t(gridDim.x) * (4 / WPT);
  for (int64_t g = WPT == 1 ? int64_t(blockIdx.x) * 4 + wave : int64_t(blockIdx.x); g < RT; g += step) {
    const int r = int(g / T);
    const int t = int(g - int64_t(r) * T);
    const int slot = lane < k ? slot_of[g * k + lane] : -1;
    const float wl = lane < k ? w[g * k + lane] : 0.0f;
    const unsigned long long local = __ballot(slot >= 0);
    float mine = 0.0f;                      // lane j: the dot product of pair j
    const u32x4* dyr = reinterpret_cast<const u32x4*>(dy.p[r] + int64_t(t) * row_bytes);
    for (int cb = first * 64 * VPL; local && cb < n16; cb += WPT * 64 * VPL) {
      u32x4 dv[VPL];
#pragma unroll
      for (int u = 0; u < VPL; ++u) {
        const int i = cb + u * 64 + lane;
        dv[u] = u32x4{0, 0, 0, 0};
        if (i < n16) dv[u] = __builtin_nontemporal_load(dyr + i);
      }
      for (unsigned long long m = local; m;) {
        const int n = __popcll(m);
        u32x4 v[JB][VPL];
        int js[JB];
        int64_t at[JB];
#pragma unroll
        for (int b = 0; b < JB; ++b) {
          if (b >= n) continue;
          js[b] = __builtin_ctzll(m);
          m &= m - 1;
          at[b] = int64_t(__builtin_amdgcn_readlane(slot, js[b])) * row_bytes;
          const u32x4* src = reinterpret_cast<const u32x4*>(ye + at[b]);
#pragma unroll
          for (int u = 0; u < VPL; ++u) {
            const int i = cb + u * 64 + lane;
            v[b][u] = u32x4{0, 0, 0, 0};
            if (i < n16) v[b][u] = __builtin_nontemporal_load(src + i);
          }
        }
#pragma unroll
        for (int b = 0; b < JB; ++b) {
          if (b >= n) continue;
          const float wj = read_lane(wl, js[b]);
          u32x4* dst = reinterpret_cast<u32x4*>(dye + at[b]);
          float dot = 0.0f;
#pragma unroll
          for (int u = 0; u < VPL; ++u) {
            const int i = cb + u * 64 + lane;
            float x[EPV], z[EPV];
            unpack<BF16>(dv[u], x);
            unpack<BF16>(v[b][u], z);
#pragma unroll
            for (int e = 0; e < EPV; ++e) {
              dot = fmaf(x[e], z[e], dot);
              x[e] *= wj;
            }
            if (i < n16) __builtin_nontemporal_store(pack<BF16>(x), dst + i);
          }
          dot = wave_sum(dot);
          if (lane == js[b]) mine += dot;
        }
      }
    }
    if constexpr (WPT > 1) {
      if (lane < k) part[wave][lane] = mine;
      __syncthreads();
      if (wave == 0 && lane < k) dw[g * k + lane] = (part[0][lane] + part[1][lane]) + (part[2][lane] + part[3][lane]);
      __syncthreads();
    } else {
      if (lane < k) dw[g * k + lane] = mine;
    }
  }
}

// One task per wave: a capped grid whose waves loop over tasks is slower (16 workgroups a CU 165 us,
// 64 a CU 151, uncapped 145 for the merge below; 8 a CU 243 us, uncapped 216 for its gradient).
// The cap that is left keeps a launch below 2^32 threads; the waves loop beyond it.
static int grid_of(int64_t n) { return int(n < (1 << 22) ? n : 1 << 22); }

// rows32: fp32 rows whatever the dtype (and y of the row type)
hipError_t launch_merge_rows(const moe_shape_t& s, const void* rows, bool rows32, const int32_t* slot_of, const float* w,
                             void* const* y, int cus, hipStream_t st) {
  RankPtrs<char*> yp{};
  for (int r = 0; r < s.R; ++r) yp.p[r] = static_cast<char*>(y[r]);
  const char* src = static_cast<const char*>(rows);
  const int64_t RT = int64_t(s.R) * s.T;
  const int64_t n16 = int64_t(s.d) * (s.dtype == MOE_F32 || rows32 ? 4 : 2) / 16;
  // Segments of 2 KiB with two rows in flight once 4-KiB ones would give every SIMD a wave (32768 tokens
  // of 7168 bf16: 142 us; 1-KiB ones with eight rows 179); below that short ones with all
  // rows in flight (61 tokens of 2048 fp32: 3.8 us against 4.7).
  const bool few = RT * ((n16 + 255) / 256) < int64_t(cus) * 4;
  const int64_t seg = few ? 64 : 128;
  const dim3 grid(grid_of((RT * ((n16 + seg - 1) / seg) + 3) / 4));
  auto launch = [&](auto kernel) {
    hipLaunchKernelGGL(kernel, grid, dim3(256), 0, st, src, yp, slot_of, w, s.R, s.T, s.k, s.d);
  };
  if (s.dtype == MOE_F32) launch(few ? merge_rows_kernel<false, 1, 8> : merge_rows_kernel<false, 2, 2>);
  else if (rows32) launch(few ? merge_rows_kernel<false, 1, 8, true> : merge_rows_kernel<false, 2, 2, true>);
  else launch(few ? merge_rows_kernel<true, 1, 8> : merge_rows_kernel<true, 2, 2>);
  return hipGetLastError();
}

hipError_t launch_merge_rows_bwd(const moe_shape_t& s, const void* const* dy, const void* ye, const int32_t* slot_of,
                                 const float* w, void* dye, float* dw, int cus, hipStream_t st) {
  RankPtrs<const char*> dp{};
  for (int r = 0; r < s.R; ++r) dp.p[r] = static_cast<const char*>(dy[r]);
  const char* src = static_cast<const char*>(ye);
  char* dst = static_cast<char*>(dye);
  const int64_t RT = int64_t(s.R) * s.T;
  // A wave per token once that gives every SIMD two, with the whole row in registers up to 14 KiB (32768
  // tokens of 7168 bf16: 187 us; segments of 4 KiB 216, of 7 KiB 194); below that a workgroup
  // per token (258 tokens of 1408 fp32: 6.5 us against 8.2).  Other widths, 16384 tokens with 16400 rows,
  // whole rows and segments of 4 KiB: rows of 14 KiB 116 and 130 us, 10 KiB 82 and 92, 8 KiB 66 and 75, 7 KiB 63.6
  // and 63.4, 5.5 KiB 52.5 and 51.2, 4.5 KiB 50 and 48, 4.1 KiB 48 and 42; 16 KiB 148 and 162.
  const bool few = RT < int64_t(cus) * 8;
  const bool wide = int64_t(s.d) * (s.dtype == MOE_F32 ? 4 : 2) > 4096;
  const dim3 grid(grid_of(few ? RT : (RT + 3) / 4));
  auto launch = [&](auto kernel) {
    hipLaunchKernelGGL(kernel, grid, dim3(256), 0, st, dp, src, slot_of, w, dst, dw, s.R, s.T, s.k, s.d);
  };
  if (s.dtype != MOE_F32) {
    if (few) launch(merge_rows_bwd_kernel<true, 1, 4, 4>);
    else if (wide) launch(merge_rows_bwd_kernel<true, 14, 1, 1>);
    else launch(merge_rows_bwd_kernel<true, 4, 1, 1>);
  } else {
    if (few) launch(merge_rows_bwd_kernel<false, 1, 4, 4>);
    else if (wide) launch(merge_rows_bwd_kernel<false, 14, 1, 1>);
    else launch(merge_rows_bwd_kernel<false, 4, 1, 1>);
  }
  return hipGetLastError();
}

}  // namespace moe
