// Products grouped by expert with ragged row counts, for experts of any form:
//   y[s] = x[s] W_g^T (W_g stored [N][K]) or x[s] W_g (stored [K][N]) for the rows s of group g;
//   dW_g = sum over s of dy[s]^T x[s] (or its transpose), the gradient by the weights.
// The gradient by the rows is the first product in the weights' other orientation.
#include "grouped.hpp"

namespace moe {

// A 64 x 64 tile of C = A B^T summed over K, A and B each stored with K contiguous (element (r, k) at r * ld + k) or with
// the row index contiguous (at k * ld + r).  256 threads, wave w owns the 32 x 32 block (w >> 1, w & 1); K steps of 32
// staged in LDS with K contiguous, rows padded so that 16 lanes' reads touch all banks.
constexpr int kSmallBM = 64, kSmallBK = 32;

template <typename T>
struct SmallTile;
template <>
struct SmallTile<float> {
  static constexpr int V = 4, kPitch = kSmallBK + 4;
};
template <>
struct SmallTile<uint16_t> {
  static constexpr int V = 8, kPitch = kSmallBK + 8;
};

template <typename T>
struct SmallOperand {
  const T* p;
  int64_t ld;
  int rows, k;         // valid rows of the tile and valid K (multiples of V along the contiguous axis, or cut there)
};

// 64 x 32 values from k0 on into LDS; zeros past the valid ones
template <typename T, bool MN>
__device__ __forceinline__ void small_fill(const SmallOperand<T>& o, int k0, T* lds) {
  using S = SmallTile<T>;
  constexpr int V = S::V;
  if constexpr (!MN) {
    constexpr int kPerRow = kSmallBK / V;
#pragma unroll
    for (int i = 0; i < kSmallBM * kPerRow / 256; ++i) {
      const int v = threadIdx.x + i * 256, r = v / kPerRow, k = (v % kPerRow) * V;
      u32x4 q = {0, 0, 0, 0};
      if (r < o.rows && k0 + k < o.k) q = *reinterpret_cast<const u32x4*>(o.p + int64_t(r) * o.ld + k0 + k);
      *reinterpret_cast<u32x4*>(lds + r * S::kPitch + k) = q;
    }
  } else {
    constexpr int kPerRow = kSmallBM / V;
#pragma unroll
    for (int i = 0; i < kSmallBK * kPerRow / 256; ++i) {
      const int v = threadIdx.x + i * 256, k = v / kPerRow, r = (v % kPerRow) * V;
      union {
        u32x4 q;
        T t[V];
      } u;
      u.q = u32x4{0, 0, 0, 0};
      if (r < o.rows && k0 + k < o.k) u.q = *reinterpret_cast<const u32x4*>(o.p + int64_t(k0 + k) * o.ld + r);
#pragma unroll
      for (int j = 0; j < V; ++j) lds[(r + j) * S::kPitch + k] = u.t[j];
    }
  }
}

template <typename T, bool A_MN, bool B_MN>
__device__ __forceinline__ f32x16 small_tile(const SmallOperand<T>& A, const SmallOperand<T>& B, int K, T* sa, T* sb) {
  using S = SmallTile<T>;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int wm = wave >> 1, wn = wave & 1, r32 = lane & 31, hi = lane >> 5;
  f32x16 acc;
#pragma unroll
  for (int e = 0; e < 16; ++e) acc[e] = 0.0f;
  for (int k0 = 0; k0 < K; k0 += kSmallBK) {
    small_fill<T, A_MN>(A, k0, sa);
    small_fill<T, B_MN>(B, k0, sb);
    __syncthreads();
    const T* pa = sa + (wm * 32 + r32) * S::kPitch;
    const T* pb = sb + (wn * 32 + r32) * S::kPitch;
    if constexpr (sizeof(T) == 2) {
#pragma unroll
      for (int c = 0; c < kSmallBK / 16; ++c) {
        const bf16x8 a = *reinterpret_cast<const bf16x8*>(pa + c * 16 + hi * 8);
        const bf16x8 b = *reinterpret_cast<const bf16x8*>(pb + c * 16 + hi * 8);
        acc = __builtin_amdgcn_mfma_f32_32x32x16_bf16(a, b, acc, 0, 0, 0);
      }
    } else {
#pragma unroll
      for (int c = 0; c < kSmallBK / 8; ++c) {
        const f32x4 a = *reinterpret_cast<const f32x4*>(pa + c * 8 + hi * 4);
        const f32x4 b = *reinterpret_cast<const f32x4*>(pb + c * 8 + hi * 4);
#pragma unroll
        for (int s = 0; s < 4; ++s) acc = __builtin_amdgcn_mfma_f32_32x32x2f32(a[s], b[s], acc, 0, 0, 0);
      }
    }
    __syncthreads();
  }
  return acc;
}

__device__ __forceinline__ void put(float* p, float v) { *p = v; }
__device__ __forceinline__ void put(uint16_t* p, float v) { *p = uint16_t(pack_bf16x2(v, 0.0f)); }

struct GroupedArgs {
  const void* x;
  const void* w;
  void* y;
  const int32_t* offsets;
  int32_t* status;
  int64_t rows, ldx, ldy;
  int G, K, N;
};

template <typename T, bool W_KN>
__global__ __launch_bounds__(256) void grouped_small_kernel(GroupedArgs g) {
  using S = SmallTile<T>;
  __shared__ __attribute__((aligned(16))) T sa[kSmallBM * S::kPitch];
  __shared__ __attribute__((aligned(16))) T sb[kSmallBM * S::kPitch];
  __shared__ int32_t base[kMaxGroups + 1], part[5];
  bool bad;
  const int mtiles = group_tiles<256>(g.offsets, g.G, g.rows, 6, base, part, &bad);
  if (g.status && blockIdx.x == 0 && threadIdx.x == 0) *g.status = bad ? MOE_EINVAL : MOE_OK;
  const int NT = (g.N + kSmallBM - 1) / kSmallBM;
  const int64_t total = int64_t(mtiles) * NT;
  for (int64_t tau = blockIdx.x; tau < total; tau += gridDim.x) {
    const int mtg = int(tau / NT), nt = int(tau - int64_t(mtg) * NT);
    const int l = find_expert(base, g.G, mtg);
    const int64_t row0 = g.offsets[l] + int64_t(mtg - base[l]) * kSmallBM;
    const int rows = int(min(int64_t(kSmallBM), g.offsets[l + 1] - row0));
    const int c0 = nt * kSmallBM, cols = min(kSmallBM, g.N - c0);
    const T* w = static_cast<const T*>(g.w) + int64_t(l) * g.N * g.K;
    const SmallOperand<T> A{static_cast<const T*>(g.x) + row0 * g.ldx, g.ldx, rows, g.K};
    const SmallOperand<T> B{W_KN ? w + c0 : w + int64_t(c0) * g.K, W_KN ? g.N : g.K, cols, g.K};
    const f32x16 acc = small_tile<T, false, W_KN>(A, B, g.K, sa, sb);
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int col = (wave & 1) * 32 + (lane & 31);
    T* out = static_cast<T*>(g.y) + row0 * g.ldy + c0 + col;
#pragma unroll
    for (int e = 0; e < 16; ++e) {
      const int row = (wave >> 1) * 32 + 8 * (e >> 2) + 4 * (lane >> 5) + (e & 3);
      if (row < rows && col < cols) put(out + row * g.ldy, acc[e]);
    }
  }
}

struct WgradArgs {
  const void* a;               // the rows whose columns become the gradient's rows
  const void* b;
  void* dw;                    // [G][M][N]
  const int32_t* offsets;
  int32_t* status;
  int64_t rows, lda, ldb;
  int G, M, N;
};

template <typename T, typename O, bool ADD>
__global__ __launch_bounds__(256) void grouped_small_wgrad_kernel(WgradArgs g) {
  using S = SmallTile<T>;
  __shared__ __attribute__((aligned(16))) T sa[kSmallBM * S::kPitch];
  __shared__ __attribute__((aligned(16))) T sb[kSmallBM * S::kPitch];
  __shared__ int32_t base[kMaxGroups + 1], part[5];
  bool bad;
  group_tiles<256>(g.offsets, g.G, g.rows, 6, base, part, &bad);
  if (g.status && blockIdx.x == 0 && threadIdx.x == 0) *g.status = bad ? MOE_EINVAL : MOE_OK;
  if (bad) return;
  const int MT = (g.M + kSmallBM - 1) / kSmallBM, NT = (g.N + kSmallBM - 1) / kSmallBM;
  const int64_t total = int64_t(g.G) * MT * NT;
  for (int64_t tau = blockIdx.x; tau < total; tau += gridDim.x) {
    const int l = int(tau / (int64_t(MT) * NT));
    const int rem = int(tau - int64_t(l) * MT * NT);
    const int m0 = (rem % MT) * kSmallBM, c0 = (rem / MT) * kSmallBM;
    const int mr = min(kSmallBM, g.M - m0), cols = min(kSmallBM, g.N - c0);
    const int64_t r0 = g.offsets[l];
    const int n = int(g.offsets[l + 1] - r0);
    const SmallOperand<T> A{static_cast<const T*>(g.a) + r0 * g.lda + m0, g.lda, mr, n};
    const SmallOperand<T> B{static_cast<const T*>(g.b) + r0 * g.ldb + c0, g.ldb, cols, n};
    const f32x16 acc = small_tile<T, true, true>(A, B, n, sa, sb);
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int col = (wave & 1) * 32 + (lane & 31);
    O* out = static_cast<O*>(g.dw) + (int64_t(l) * g.M + m0) * g.N + c0 + col;
#pragma unroll
    for (int e = 0; e < 16; ++e) {
      const int row = (wave >> 1) * 32 + 8 * (e >> 2) + 4 * (lane >> 5) + (e & 3);
      if (row < mr && col < cols) {
        if constexpr (ADD) out[int64_t(row) * g.N] += acc[e];
        else put(out + int64_t(row) * g.N, acc[e]);
      }
    }
  }
}

hipError_t launch_grouped(const moe_gemm_t& s, const void* x, const void* w, const int32_t* offsets, void* y,
                          int32_t* status, int cus, hipStream_t st) {
  const GroupedArgs g{x, w, y, offsets, status, s.rows, s.ldx ? s.ldx : s.K, s.ldy ? s.ldy : s.N, s.groups, s.K, s.N};
  const dim3 grid(cus * 4), threads(256);
  if (s.dtype == MOE_F32) {
    if (s.w_layout) hipLaunchKernelGGL((grouped_small_kernel<float, true>), grid, threads, 0, st, g);
    else hipLaunchKernelGGL((grouped_small_kernel<float, false>), grid, threads, 0, st, g);
  } else {
    if (s.w_layout) hipLaunchKernelGGL((grouped_small_kernel<uint16_t, true>), grid, threads, 0, st, g);
    else hipLaunchKernelGGL((grouped_small_kernel<uint16_t, false>), grid, threads, 0, st, g);
  }
  return hipGetLastError();
}

hipError_t launch_grouped_wgrad(const moe_gemm_t& s, const void* x, const void* dy, const int32_t* offsets, void* dw,
                                int dw_dtype, bool accumulate, int32_t* status, int cus, hipStream_t st) {
  const int64_t ldx = s.ldx ? s.ldx : s.K, ldy = s.ldy ? s.ldy : s.N;
  const WgradArgs g = s.w_layout ? WgradArgs{x, dy, dw, offsets, status, s.rows, ldx, ldy, s.groups, s.K, s.N}
                                 : WgradArgs{dy, x, dw, offsets, status, s.rows, ldy, ldx, s.groups, s.N, s.K};
  const dim3 grid(cus * 4), threads(256);
  if (s.dtype == MOE_F32) {
    if (accumulate) hipLaunchKernelGGL((grouped_small_wgrad_kernel<float, float, true>), grid, threads, 0, st, g);
    else hipLaunchKernelGGL((grouped_small_wgrad_kernel<float, float, false>), grid, threads, 0, st, g);
  } else if (dw_dtype == MOE_F32) {
    if (accumulate) hipLaunchKernelGGL((grouped_small_wgrad_kernel<uint16_t, float, true>), grid, threads, 0, st, g);
    else hipLaunchKernelGGL((grouped_small_wgrad_kernel<uint16_t, float, false>), grid, threads, 0, st, g);
  } else {
    hipLaunchKernelGGL((grouped_small_wgrad_kernel<uint16_t, uint16_t, false>), grid, threads, 0, st, g);
  }
  return hipGetLastError();
}

}  // namespace moe
