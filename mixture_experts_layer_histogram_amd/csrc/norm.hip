// RMS norm of token rows with the residual's addition ahead of it, rows out in their own type and in MXFP8, and its
// gradients.
//
//   s = x + residual;  rstd = (mean(s^2) + eps)^-1/2;  y = s rstd gamma;  h = s rounded;  codes = MXFP8(y).
//   With u = gamma dy:  dx = dh + rstd (u - h rstd^2 <u, h> / d);  dgamma = sum over rows of dy h rstd.
//
// Both are bound by the rows' bytes: a row is read once, stays in registers as fp32 (E values a lane, W waves a row) and is
// written once.  A workgroup takes consecutive rows, so a lane keeps its columns: gamma is read once a workgroup, the
// gradient of gamma adds up in registers, and the scale words of a chunk of rows leave through LDS as runs.  32768 x 7168 bf16 with residual, both
// rows out and MXFP8: 379 us (5.6 TB/s); its gradients 345 us (5.4 TB/s); 37 x 1408 fp32 5.4 us, a launch's submission.
#include <type_traits>

#include "mx.hpp"

namespace moe {

constexpr int kNormChunk = 16;          // rows of one workgroup whose scale words go to LDS together

// E values of a row held by a lane, 16 bytes of the row type at a time: vector u of a lane is vector u * 64 W + its index
template <bool BF16>
struct RowVec {
  static constexpr int N = BF16 ? 8 : 4;
  __device__ static __forceinline__ void unpack(const u32x4 v, float* f) {
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
  __device__ static __forceinline__ u32x4 pack(const float* f) {
    if constexpr (BF16)
      return u32x4{pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]), pack_bf16x2(f[4], f[5]), pack_bf16x2(f[6], f[7])};
    else
      return u32x4{__float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]), __float_as_uint(f[3])};
  }
};

// Rows from kNormPast bytes on go past the caches, which do not hold them until somebody reads them.  us of two norms on end, bf16, past
// them and through them: 4096 x 7168 80.7 and 76.7, 8192 x 7168 124 and 114, 32768 x 7168 393 and 413 (with residual and MXFP8 398 and 449).
constexpr int64_t kNormPast = int64_t(256) << 20;

// (a template: of two stores in the arms of a branch the compiler makes one, through the caches)
template <bool PAST>
__device__ __forceinline__ void put_row(u32x4* p, const u32x4 v) {
  if constexpr (PAST) __builtin_nontemporal_store(v, p);
  else *p = v;
}

__device__ __forceinline__ float wave_sum(float v) {
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) v += __shfl_xor(v, o);
  return v;
}

// Sum over the W waves of a row (all lanes get it); red: W floats of LDS a row, free again after the next call's barrier
template <int W>
__device__ __forceinline__ float row_sum(float v, float* red, int wave) {
  v = wave_sum(v);
  if constexpr (W > 1) {
    if ((threadIdx.x & 63) == 0) red[wave] = v;
    __syncthreads();
    float t = red[0];
#pragma unroll
    for (int w = 1; w < W; ++w) t += red[w];
    v = t;
  }
  return v;
}

// MXFP8 of N consecutive fp32 values of a lane; the 32 / N lanes of a block agree on its scale code.  A block with a NaN
// or an infinity gets E8M0's NaN and zero codes.
template <int N>
__device__ __forceinline__ uint2 mx_quant(const float* f, uint32_t* scale) {
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < N; ++i) m = max(m, __float_as_uint(f[i]) & 0x7FFFFFFFu);
  m = quad_max(m);
  // the other quad of eight lanes: the half row mirrored
  if constexpr (N == 4) m = max(m, uint32_t(__builtin_amdgcn_update_dpp(int(m), int(m), 0x141, 0xF, 0xF, false)));
  if (m == 0 || m >= 0x7F800000u) {
    *scale = m ? 255u : 0u;
    return make_uint2(0, 0);
  }
  const int e = mx_block_exp(m);
  const float inv = mx_inv_scale(e);
  *scale = uint32_t(e + 127);
  uint2 q = make_uint2(mx_pack4(f[0], f[1], f[2], f[3], inv), 0);
  if constexpr (N == 8) q.y = mx_pack4(f[4], f[5], f[6], f[7], inv);
  return q;
}

struct NormArgs {
  const char* x;
  const char* residual;      // or null
  const float* gamma;        // or null: ones
  char* h;                   // or null
  char* y;                   // or null
  uint8_t* codes;            // or null
  uint8_t* scales;
  int64_t rows;
  int d;
  float eps;
};

template <bool BF16, int W, int E, bool PAST>
__global__ __launch_bounds__(W < 4 ? 256 : 64 * W) void norm_kernel(NormArgs a) {
  using R = RowVec<BF16>;
  constexpr int V = E / R::N, PER = W < 4 ? 4 / W : 1;            // vectors a lane, rows a workgroup at a time
  extern __shared__ uint32_t s_sc[];                              // [kNormChunk][nq + 1] scale words
  __shared__ float red[2][16];
  const int part = W < 4 ? threadIdx.x / (64 * W) : 0;
  const int lane = threadIdx.x - part * 64 * W, wave = lane >> 6;
  const int nv = a.d / R::N, nq = a.d >> 7;
  const int64_t row_bytes = int64_t(a.d) * (BF16 ? 2 : 4);
  float gam[E];
#pragma unroll
  for (int u = 0; u < V; ++u) {
    const int i = u * 64 * W + lane;
#pragma unroll
    for (int j = 0; j < R::N; ++j) gam[u * R::N + j] = (a.gamma && i < nv) ? a.gamma[i * R::N + j] : 1.0f;
  }
  // rows of a workgroup's turn: what gives every workgroup one, at most a chunk
  const int64_t even = (a.rows + gridDim.x - 1) / gridDim.x;
  const int per_wg = even >= kNormChunk ? kNormChunk : int(even + PER - 1) / PER * PER;
  const int64_t tasks = (a.rows + per_wg - 1) / per_wg;
  int turn = 0;
  for (int64_t c = blockIdx.x; c < tasks; c += gridDim.x) {
    const int64_t r0 = c * per_wg;
    const int nr = int(min(int64_t(per_wg), a.rows - r0));
    for (int rr = part; rr - part < nr; rr += PER) {              // the same number of turns in every wave
      const bool on = rr < nr;
      const int64_t base = (r0 + (on ? rr : 0)) * row_bytes;
      float s[E];
      float sq = 0.0f;
      u32x4 vx[V], vr[V];
#pragma unroll
      for (int u = 0; u < V; ++u) {
        const int i = u * 64 * W + lane;
        vx[u] = vr[u] = u32x4{0, 0, 0, 0};
        if (on && i < nv) {
          vx[u] = __builtin_nontemporal_load(reinterpret_cast<const u32x4*>(a.x + base) + i);
          if (a.residual) vr[u] = __builtin_nontemporal_load(reinterpret_cast<const u32x4*>(a.residual + base) + i);
        }
      }
#pragma unroll
      for (int u = 0; u < V; ++u) {
        float fr[R::N];
        R::unpack(vx[u], s + u * R::N);
        R::unpack(vr[u], fr);
#pragma unroll
        for (int j = 0; j < R::N; ++j) {
          if (a.residual) s[u * R::N + j] += fr[j];
          sq = fmaf(s[u * R::N + j], s[u * R::N + j], sq);
        }
      }
      const float mean = row_sum<W>(sq, red[turn], wave) / float(a.d);
      turn ^= 1;
      const float rstd = 1.0f / sqrtf(mean + a.eps);
#pragma unroll
      for (int u = 0; u < V; ++u) {
        const int i = u * 64 * W + lane;
        const bool in = on && i < nv;
        if (a.h && in) put_row<PAST>(reinterpret_cast<u32x4*>(a.h + base) + i, R::pack(s + u * R::N));
#pragma unroll
        for (int j = 0; j < R::N; ++j) s[u * R::N + j] = s[u * R::N + j] * rstd * gam[u * R::N + j];
        if (a.y && in) put_row<PAST>(reinterpret_cast<u32x4*>(a.y + base) + i, R::pack(s + u * R::N));
        if (a.codes) {                                            // lanes past the row hold zeros or whole blocks of their own
          uint32_t sc;
          const uint2 q = mx_quant<R::N>(s + u * R::N, &sc);
          if (in) {
            uint8_t* dst = a.codes + (r0 + rr) * a.d + int64_t(i) * R::N;
            if constexpr (BF16) *reinterpret_cast<uint2*>(dst) = q;
            else *reinterpret_cast<uint32_t*>(dst) = q.x;
            const int k = i * R::N;
            if ((k & 31) == 0) reinterpret_cast<uint8_t*>(s_sc)[(rr * (nq + 1) + (k >> 7)) * 4 + ((k >> 5) & 3)] = uint8_t(sc);
          }
        }
      }
    }
    if (a.codes) {
      __syncthreads();
      uint32_t* out = reinterpret_cast<uint32_t*>(a.scales);
      for (int e = threadIdx.x; e < nq * per_wg; e += blockDim.x) {
        const int q = e / per_wg, rr = e - q * per_wg;
        if (rr < nr) out[a.rows * q + r0 + rr] = s_sc[rr * (nq + 1) + q];
      }
      __syncthreads();                                            // the next rows' scales overwrite these
    }
  }
}

struct NormBwdArgs {
  const char* dy;
  const char* h;
  const float* gamma;        // or null
  const char* dh;            // or null
  char* dx;                  // or null
  float* parts;              // [gridDim.x][d] sums of dy h rstd over a workgroup's rows, or null
  int64_t rows;
  int d;
  float eps;
};

template <bool BF16, int W, int E, bool PAST>
__global__ __launch_bounds__(W < 4 ? 256 : 64 * W) void norm_bwd_kernel(NormBwdArgs a) {
  using R = RowVec<BF16>;
  constexpr int V = E / R::N, PER = W < 4 ? 4 / W : 1;
  __shared__ float red[2][2][16];
  extern __shared__ float s_part[];                               // W < 4: [PER][d]
  const int part = W < 4 ? threadIdx.x / (64 * W) : 0;
  const int lane = threadIdx.x - part * 64 * W, wave = lane >> 6;
  const int nv = a.d / R::N;
  const int64_t row_bytes = int64_t(a.d) * (BF16 ? 2 : 4);
  float gam[E], acc[E];
#pragma unroll
  for (int u = 0; u < V; ++u) {
    const int i = u * 64 * W + lane;
#pragma unroll
    for (int j = 0; j < R::N; ++j) {
      gam[u * R::N + j] = (a.gamma && i < nv) ? a.gamma[i * R::N + j] : 1.0f;
      acc[u * R::N + j] = 0.0f;
    }
  }
  int turn = 0;
  for (int64_t r0 = int64_t(blockIdx.x) * PER; r0 < a.rows; r0 += int64_t(gridDim.x) * PER) {
    const bool on = r0 + part < a.rows;
    const int64_t base = (r0 + (on ? part : 0)) * row_bytes;
    u32x4 vy[V], vh[V], vd[V];
#pragma unroll
    for (int u = 0; u < V; ++u) {
      const int i = u * 64 * W + lane;
      vy[u] = vh[u] = vd[u] = u32x4{0, 0, 0, 0};
      if (on && i < nv) {
        vy[u] = __builtin_nontemporal_load(reinterpret_cast<const u32x4*>(a.dy + base) + i);
        vh[u] = __builtin_nontemporal_load(reinterpret_cast<const u32x4*>(a.h + base) + i);
        if (a.dh) vd[u] = __builtin_nontemporal_load(reinterpret_cast<const u32x4*>(a.dh + base) + i);
      }
    }
    float dy[E], h[E], sq = 0.0f, uh = 0.0f;
#pragma unroll
    for (int u = 0; u < V; ++u) {
      R::unpack(vy[u], dy + u * R::N);
      R::unpack(vh[u], h + u * R::N);
#pragma unroll
      for (int j = 0; j < R::N; ++j) {
        const int e = u * R::N + j;
        sq = fmaf(h[e], h[e], sq);
        uh = fmaf(dy[e] * gam[e], h[e], uh);
      }
    }
    sq = wave_sum(sq);
    uh = wave_sum(uh);
    if constexpr (W > 1) {
      if ((lane & 63) == 0) {
        red[turn][0][wave] = sq;
        red[turn][1][wave] = uh;
      }
      __syncthreads();
      sq = red[turn][0][0];
      uh = red[turn][1][0];
#pragma unroll
      for (int w = 1; w < W; ++w) {
        sq += red[turn][0][w];
        uh += red[turn][1][w];
      }
      turn ^= 1;
    }
    const float rstd = 1.0f / sqrtf(sq / float(a.d) + a.eps);
    const float k = rstd * rstd * (uh / float(a.d));
#pragma unroll
    for (int u = 0; u < V; ++u) {
      const int i = u * 64 * W + lane;
      float o[R::N];
      R::unpack(vd[u], o);
#pragma unroll
      for (int j = 0; j < R::N; ++j) {
        const int e = u * R::N + j;
        acc[e] = on ? fmaf(dy[e], h[e] * rstd, acc[e]) : acc[e];
        const float g = rstd * (dy[e] * gam[e] - h[e] * k);
        o[j] = a.dh ? o[j] + g : g;
      }
      if (a.dx && on && i < nv) put_row<PAST>(reinterpret_cast<u32x4*>(a.dx + base) + i, R::pack(o));
    }
  }
  if (!a.parts) return;
  if constexpr (W < 4) {
#pragma unroll
    for (int u = 0; u < V; ++u) {
      const int i = u * 64 * W + lane;
#pragma unroll
      for (int j = 0; j < R::N; ++j)
        if (i < nv) s_part[part * a.d + i * R::N + j] = acc[u * R::N + j];
    }
    __syncthreads();
    for (int c = threadIdx.x; c < a.d; c += blockDim.x) {
      float t = s_part[c];
#pragma unroll
      for (int p = 1; p < PER; ++p) t += s_part[p * a.d + c];
      a.parts[int64_t(blockIdx.x) * a.d + c] = t;
    }
  } else {
#pragma unroll
    for (int u = 0; u < V; ++u) {
      const int i = u * 64 * W + lane;
#pragma unroll
      for (int j = 0; j < R::N; ++j)
        if (i < nv) a.parts[int64_t(blockIdx.x) * a.d + i * R::N + j] = acc[u * R::N + j];
    }
  }
}

// dgamma[c] = sum over p of parts[p][c]: a workgroup takes 64 columns, its 16 waves every sixteenth part, eight of them in flight
__global__ __launch_bounds__(1024) void norm_gamma_kernel(const float* __restrict__ parts, int n_parts, int d,
                                                          float* __restrict__ dgamma) {
  __shared__ float s[16][64];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int c = blockIdx.x * 64 + lane;
  float t = 0.0f;
  if (c < d)
    for (int p0 = wave; p0 < n_parts; p0 += 128) {
      float v[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] = p0 + 16 * i < n_parts ? parts[int64_t(p0 + 16 * i) * d + c] : 0.0f;
#pragma unroll
      for (int i = 0; i < 8; ++i) t += v[i];
    }
  s[wave][lane] = t;
  __syncthreads();
  if (wave == 0 && c < d) {
#pragma unroll
    for (int w = 1; w < 16; ++w) t += s[w][lane];
    dgamma[c] = t;
  }
}

// Waves a row.  Few values a lane keep enough rows in flight, many waves a row wait for each other.  us of two norms on end and of the
// gradients, bf16: 4096 x 2048, one wave 39.2 and 31.5, four 29.7 and 22.5; 2048 x 4096, four 39.0, eight 27.8 (gradients 21.0, 21.1); 4096 x 7168,
// four 76.7 and 43.5, eight 65.0 and 41.7, sixteen 66.1 and 47.4; 32768 x 7168, four 393 and 256, eight 387 and 250, sixteen 443 and 291.
int norm_waves(int d) { return d <= 512 ? 1 : d <= 2048 ? 4 : d <= 8192 ? 8 : 16; }

// Workgroups of the backward, each of which leaves one partial sum of dgamma: 4096 waves.  Twice as many write and read those sums for longer
// (4096 x 7168 51.5 us instead of 43.5, with four waves a row), half as many leave too few rows in flight (48.1 instead of 41.7, 32768 x 7168
// 296 instead of 250).
int norm_bwd_grid(int64_t rows, int d) {
  const int W = norm_waves(d), per = W == 1 ? 4 : 1, most = W <= 4 ? 1024 : 4096 / W;
  const int64_t need = (rows + per - 1) / per;
  return int(need < most ? need : most);
}

template <bool BF16, int W, int E, bool PAST>
static void norm_launch(const NormArgs& a, int grid, size_t lds, hipStream_t st) {
  hipLaunchKernelGGL((norm_kernel<BF16, W, E, PAST>), dim3(grid), dim3(W < 4 ? 256 : 64 * W), lds, st, a);
}
template <bool BF16, int W, int E, bool PAST>
static void norm_launch(const NormBwdArgs& a, int grid, size_t lds, hipStream_t st) {
  hipLaunchKernelGGL((norm_bwd_kernel<BF16, W, E, PAST>), dim3(grid), dim3(W < 4 ? 256 : 64 * W), lds, st, a);
}

template <typename ARGS>
static hipError_t norm_pick(const ARGS& a, int dtype, int grid, size_t lds, hipStream_t st) {
  const int W = norm_waves(a.d), lane = (a.d + 64 * W - 1) / (64 * W);           // values a lane: 8, 16 or 32
  auto pick = [&](auto bf16, auto past) {
    constexpr bool B = decltype(bf16)::value, P = decltype(past)::value;
    if (W == 1) norm_launch<B, 1, 8, P>(a, grid, lds, st);
    else if (W == 4) norm_launch<B, 4, 8, P>(a, grid, lds, st);
    else if (W == 8 && lane <= 8) norm_launch<B, 8, 8, P>(a, grid, lds, st);
    else if (W == 8) norm_launch<B, 8, 16, P>(a, grid, lds, st);
    else if (lane <= 16) norm_launch<B, 16, 16, P>(a, grid, lds, st);
    else norm_launch<B, 16, 32, P>(a, grid, lds, st);
  };
  const bool past = a.rows * a.d * (dtype == MOE_BF16 ? 2 : 4) >= kNormPast;
  if (dtype == MOE_BF16 && past) pick(std::true_type{}, std::true_type{});
  else if (dtype == MOE_BF16) pick(std::true_type{}, std::false_type{});
  else if (past) pick(std::false_type{}, std::true_type{});
  else pick(std::false_type{}, std::false_type{});
  return hipGetLastError();
}

hipError_t launch_norm(const moe_norm_t& n, const void* x, const void* residual, const float* gamma, void* h, void* y,
                       uint8_t* codes, uint8_t* scales, int cus, hipStream_t st) {
  if (n.rows == 0) return hipSuccess;
  const NormArgs a{static_cast<const char*>(x), static_cast<const char*>(residual), gamma, static_cast<char*>(h),
                   static_cast<char*>(y), codes, scales, n.rows, n.d, n.eps};
  const int W = norm_waves(n.d), per = W == 1 ? 4 : 1;
  const int64_t need = (n.rows + per - 1) / per, most = int64_t(cus) * (W <= 4 ? 8 : 32 / W);      // 32 waves a CU
  const int grid = int(need < most ? need : most);
  const size_t lds = codes ? size_t(kNormChunk) * ((n.d >> 7) + 1) * 4 : 0;
  return norm_pick(a, n.dtype, grid, lds, st);
}

hipError_t launch_norm_bwd(const moe_norm_t& n, const void* dy, const void* h, const float* gamma, const void* dh, void* dx,
                           float* dgamma, float* parts, hipStream_t st) {
  const int grid = norm_bwd_grid(n.rows, n.d);
  const NormBwdArgs a{static_cast<const char*>(dy), static_cast<const char*>(h), gamma, static_cast<const char*>(dh),
                      static_cast<char*>(dx), dgamma ? parts : nullptr, n.rows, n.d, n.eps};
  if (grid) {
    const size_t lds = norm_waves(n.d) == 1 && a.parts ? size_t(4) * n.d * 4 : 0;
    const hipError_t e = norm_pick(a, n.dtype, grid, lds, st);
    if (e != hipSuccess) return e;
  }
  if (!dgamma) return hipSuccess;
  hipLaunchKernelGGL(norm_gamma_kernel, dim3((n.d + 63) / 64), dim3(1024), 0, st, parts, grid, n.d, dgamma);
  return hipGetLastError();
}

}  // namespace moe
