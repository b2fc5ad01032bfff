// MXFP4 quantiser, the dequantiser of both MX formats, and the pull dispatch that quantises
// each gathered token row to MXFP4 (the pull itself: MoK article, kucoin.com/es "Cursor's MoK
// logra un aumento del 2.37x ...", section 02).
//
// All are HBM-bound: per value the quantiser reads 2 (bf16) or 4 (fp32) bytes and writes
// 17/32; the dequantiser the reverse.  A wave takes 512 consecutive values of one row at a
// time (16 bytes of bf16 per lane, an aligned lane quad holds one 32-value block), a workgroup
// 32 rows x 512 values, so that its scale words -- four K-tile planes of 32 rows -- leave as
// four runs of 128 bytes instead of single words (each a partial write of its own line).
// Measured on 229376 rows of 2048 bf16 values: quantise 185 to 188 us, dequantise 177 to 194 us by the card
// (1.19 GB: 6.3 and 6.1 to 6.7 TB/s; a device copy of 2 GiB reaches 4.8 to 4.9); the gather of 32768 rows of
// 7168, 111 us (5.3 TB/s).  2^28 values: from bf16 106 to 121 us at K = 256 to 7168, from fp32 221 to 242 us
// (5.0 to 5.5 TB/s); to bf16 113 to 128, to fp32 298 to 316 (4.0 TB/s).  K = 128 uses 16 of a wave's 64
// lanes: 214 us from bf16, 199 back.
#include "mx4.hpp"

namespace moe {

constexpr int kQuantRows = 32, kQuantCols = 512;

template <bool BF16>
__global__ __launch_bounds__(256) void mx4_quantize_kernel(const void* __restrict__ src, int64_t rows, int K,
                                                           uint8_t* __restrict__ codes, uint8_t* __restrict__ scales) {
  __shared__ uint32_t s_sc[4][kQuantRows];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int nct = int((uint32_t(K) + kQuantCols - 1) / kQuantCols);
  const int64_t tasks = (rows + kQuantRows - 1) / kQuantRows * nct;
  uint32_t* const words = reinterpret_cast<uint32_t*>(scales);
  for (int64_t task = blockIdx.x; task < tasks; task += gridDim.x) {
    const int64_t r0 = task / nct * kQuantRows;
    const int ct = int(task % nct);
    const uint32_t k = uint32_t(ct) * kQuantCols + lane * 8;   // K % 128 == 0: whole 16-lane groups are in or out
    const bool in = k < uint32_t(K);
    const int nr = int(min(int64_t(kQuantRows), rows - r0));
    constexpr int U = 8;                                   // rows in flight per wave
    u32x4 v[U][BF16 ? 1 : 2];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int rr = u * 4 + wave;
#pragma unroll
      for (int h = 0; h < (BF16 ? 1 : 2); ++h) {
        v[u][h] = u32x4{0, 0, 0, 0};
        if (in && rr < nr)
          v[u][h] = __builtin_nontemporal_load(
              reinterpret_cast<const u32x4*>(static_cast<const char*>(src) + ((r0 + rr) * K + k) * (BF16 ? 2 : 4)) + h);
      }
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int rr = u * 4 + wave;
      uint32_t sc;
      uint32_t q;
      if constexpr (BF16) q = mx4_quant8_bf16(v[u][0], &sc);          // all lanes: quad permutations inside
      else q = mx4_quant8_f32(__builtin_bit_cast(f32x4, v[u][0]), __builtin_bit_cast(f32x4, v[u][1]), &sc);
      const uint32_t sw = mx_scale_word(sc);
      if (in && rr < nr) *reinterpret_cast<uint32_t*>(codes + ((r0 + rr) * K + k) / 2) = q;
      if ((lane & 15) == 0) s_sc[lane >> 4][rr] = sw;
    }
    __syncthreads();
    if (threadIdx.x < 4 * kQuantRows) {
      const int p = threadIdx.x >> 5, rr = threadIdx.x & 31;
      const int plane = ct * 4 + p;
      if (plane < (K >> 7) && rr < nr) words[int64_t(plane) * rows + r0 + rr] = s_sc[p][rr];
    }
    __syncthreads();
  }
}

// FP4: 4-bit codes, else E4M3 codes; BF16: bf16 values out, else fp32
template <bool FP4, bool BF16>
__global__ __launch_bounds__(256) void mx_dequantize_kernel(const uint8_t* __restrict__ codes,
                                                            const uint8_t* __restrict__ scales, int64_t rows, int K,
                                                            void* __restrict__ dst) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int nct = int((uint32_t(K) + kQuantCols - 1) / kQuantCols);
  const int64_t tasks = (rows + kQuantRows - 1) / kQuantRows * nct;
  const uint32_t* const words = reinterpret_cast<const uint32_t*>(scales);
  for (int64_t task = blockIdx.x; task < tasks; task += gridDim.x) {
    const int64_t r0 = task / nct * kQuantRows;
    const int ct = int(task % nct);
    const uint32_t k = uint32_t(ct) * kQuantCols + lane * 8;
    if (k >= uint32_t(K)) continue;
    const int nr = int(min(int64_t(kQuantRows), rows - r0));
    constexpr int U = 8;
    uint2 q[U];
    uint32_t sw[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int rr = u * 4 + wave;
      q[u] = make_uint2(0, 0);
      sw[u] = 0;
      if (rr < nr) {
        const int64_t at = (r0 + rr) * K + k;
        if (FP4) q[u].x = __builtin_nontemporal_load(reinterpret_cast<const uint32_t*>(codes + at / 2));
        else {
          q[u].x = __builtin_nontemporal_load(reinterpret_cast<const uint32_t*>(codes + at));
          q[u].y = __builtin_nontemporal_load(reinterpret_cast<const uint32_t*>(codes + at) + 1);
        }
        sw[u] = words[int64_t(k >> 7) * rows + r0 + rr];
      }
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int rr = u * 4 + wave;
      if (rr >= nr) continue;
      const float f = e8m0_f32((sw[u] >> (8 * ((k >> 5) & 3))) & 0xFFu);
      float o[8];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        f32v2 p;
        if constexpr (FP4) {
          p = i == 0   ? __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(q[u].x, 1.0f, 0)
              : i == 1 ? __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(q[u].x, 1.0f, 1)
              : i == 2 ? __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(q[u].x, 1.0f, 2)
                       : __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(q[u].x, 1.0f, 3);
        } else {
          const int w = int(i < 2 ? q[u].x : q[u].y);
          p = (i & 1) ? __builtin_amdgcn_cvt_pk_f32_fp8(w, true) : __builtin_amdgcn_cvt_pk_f32_fp8(w, false);
        }
        o[2 * i] = p[0] * f;              // exact, or an infinity past the type's range
        o[2 * i + 1] = p[1] * f;
      }
      char* d = static_cast<char*>(dst) + ((r0 + rr) * K + k) * (BF16 ? 2 : 4);
      if constexpr (BF16) {
        const u32x4 w = {pack_bf16x2(o[0], o[1]), pack_bf16x2(o[2], o[3]), pack_bf16x2(o[4], o[5]),
                         pack_bf16x2(o[6], o[7])};
        __builtin_nontemporal_store(w, reinterpret_cast<u32x4*>(d));
      } else {
        __builtin_nontemporal_store(f32x4{o[0], o[1], o[2], o[3]}, reinterpret_cast<f32x4*>(d));
        __builtin_nontemporal_store(f32x4{o[4], o[5], o[6], o[7]}, reinterpret_cast<f32x4*>(d) + 1);
      }
    }
  }
}

// xe[s] / xe_scales[s] = MXFP4(x[pull_src[s].rank][pull_src[s].token]); one wave per ROWS rows, UNROLL
// 16-byte vectors of each in flight per lane (the whole row for the widths below).  A workgroup
// takes up to `most` consecutive rows at a time -- fewer when there are not enough rows to give
// every workgroup that many, since one row alone takes two microseconds of waiting -- keeps
// their scale words in LDS and writes each K-tile plane's words as one run.  With no more rows than
// workgroups each takes one, its waves a quarter of the row each (512 rows of 7168: 5.6 us against 8.4).
template <int UNROLL, int ROWS>
__global__ __launch_bounds__(256) __attribute__((amdgpu_waves_per_eu(4, 8))) void dispatch_pull_mx4_kernel(
    RankPtrs<const char*> x, const int32_t* __restrict__ pull_src, const int32_t* __restrict__ ctrl,
    uint8_t* __restrict__ xe, uint8_t* __restrict__ xes, int d, int64_t nmax, int most) {
  extern __shared__ uint32_t s_sc[];           // [most][nq + 1]
  const int N = ctrl[kCtrlN];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int n16 = d >> 3;            // 16-byte source vectors per row (d % 128 == 0: whole 16-lane groups)
  const int nq = d >> 7;             // scale words (K-tile planes) per row
  uint32_t* xw = reinterpret_cast<uint32_t*>(xes);
  if (N <= int(gridDim.x)) {         // a row for a workgroup: its waves share it, a quarter of its vectors each
    const int row = blockIdx.x;
    if (row >= N) return;
    const u32x4* src = reinterpret_cast<const u32x4*>(x.p[pull_src[2 * row]] + int64_t(pull_src[2 * row + 1]) * d * 2);
    uint32_t* dst = reinterpret_cast<uint32_t*>(xe + int64_t(row) * (d >> 1));
    constexpr int U = 4;
    for (int base = int(threadIdx.x); base - int(threadIdx.x) < n16; base += 256 * U) {
      u32x4 v[U];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        v[u] = u32x4{0, 0, 0, 0};
        if (base + u * 256 < n16) v[u] = src[base + u * 256];
      }
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int q = base + u * 256;
        uint32_t sc;
        const uint32_t code = mx4_quant8_bf16(v[u], &sc);       // all lanes: quad permutations inside
        const uint32_t sw = mx_scale_word(sc);                   // all lanes: row shifts inside
        if (q < n16) {
          dst[q] = code;
          if ((q & 15) == 0) xw[nmax * (q >> 4) + row] = sw;
        }
      }
    }
    return;
  }
  const int even = (N + int(gridDim.x) - 1) / int(gridDim.x);
  const int cr = min(most, max(4, (even + 3) & ~3));
  const int nchunks = (N + cr - 1) / cr;
  for (int c = blockIdx.x; c < nchunks; c += gridDim.x) {
    const int s0 = c * cr, rows = min(cr, N - s0);
    // where this wave's rows (wave, wave + 4, ...: at most 8) come from, one load for all
    const int mine = s0 + wave + 4 * (lane & 7);
    int2 from = make_int2(0, 0);
    if (mine < s0 + rows) from = reinterpret_cast<const int2*>(pull_src)[mine];
    for (int i = 0; wave + 4 * i < rows; i += ROWS) {
      const u32x4* src[ROWS];
#pragma unroll
      for (int j = 0; j < ROWS; ++j) {
        const int r = __builtin_amdgcn_readlane(from.x, i + j), t = __builtin_amdgcn_readlane(from.y, i + j);
        src[j] = reinterpret_cast<const u32x4*>(x.p[r] + int64_t(t) * d * 2);
      }
      for (int base = 0; base < n16; base += 64 * UNROLL) {
        u32x4 v[ROWS][UNROLL];
#pragma unroll
        for (int j = 0; j < ROWS; ++j)
#pragma unroll
          for (int u = 0; u < UNROLL; ++u) {
            const int q = base + u * 64 + lane;
            v[j][u] = u32x4{0, 0, 0, 0};
            if (q < n16 && wave + 4 * (i + j) < rows) v[j][u] = __builtin_nontemporal_load(src[j] + q);
          }
#pragma unroll
        for (int j = 0; j < ROWS; ++j) {
          const int rr = wave + 4 * (i + j);
          if (rr >= rows) break;                               // the same in every lane
          uint32_t* dst = reinterpret_cast<uint32_t*>(xe + int64_t(s0 + rr) * (d >> 1));
#pragma unroll
          for (int u = 0; u < UNROLL; ++u) {
            const int q = base + u * 64 + lane;
            uint32_t sc;
            const uint32_t code = mx4_quant8_bf16(v[j][u], &sc);   // all lanes: quad permutations inside
            const uint32_t sw = mx_scale_word(sc);                 // all lanes: row shifts inside
            if (q < n16) {
              dst[q] = code;
              if ((q & 15) == 0) s_sc[rr * (nq + 1) + (q >> 4)] = sw;
            }
          }
        }
      }
    }
    __syncthreads();
    for (int e = threadIdx.x; e < nq * cr; e += 256) {
      const int q = e / cr, rr = e - q * cr;
      if (rr < rows) xw[nmax * q + s0 + rr] = s_sc[rr * (nq + 1) + q];
    }
    __syncthreads();                 // the next chunk's waves overwrite s_sc
  }
}

// a task per workgroup: 189 us for 229376 rows of 2048 bf16; 8 workgroups a CU that loop take 204
static int quant_grid(int64_t rows, int K) {
  const int64_t tasks = (rows + kQuantRows - 1) / kQuantRows * ((int64_t(K) + kQuantCols - 1) / kQuantCols);
  return int(tasks < (1 << 22) ? tasks : 1 << 22);        // a launch has less than 2^32 threads
}

hipError_t launch_mx4_quantize(const void* src, int src_dtype, int64_t rows, int K, uint8_t* codes, uint8_t* scales,
                               hipStream_t st) {
  const dim3 grid(quant_grid(rows, K));
  if (src_dtype == MOE_BF16)
    hipLaunchKernelGGL(mx4_quantize_kernel<true>, grid, dim3(256), 0, st, src, rows, K, codes, scales);
  else
    hipLaunchKernelGGL(mx4_quantize_kernel<false>, grid, dim3(256), 0, st, src, rows, K, codes, scales);
  return hipGetLastError();
}

hipError_t launch_mx_dequantize(const uint8_t* codes, const uint8_t* scales, int format, int64_t rows, int K, void* dst,
                                int dst_dtype, hipStream_t st) {
  const dim3 grid(quant_grid(rows, K));
  if (format == MOE_MXFP4) {
    if (dst_dtype == MOE_BF16)
      hipLaunchKernelGGL((mx_dequantize_kernel<true, true>), grid, dim3(256), 0, st, codes, scales, rows, K, dst);
    else
      hipLaunchKernelGGL((mx_dequantize_kernel<true, false>), grid, dim3(256), 0, st, codes, scales, rows, K, dst);
  } else {
    if (dst_dtype == MOE_BF16)
      hipLaunchKernelGGL((mx_dequantize_kernel<false, true>), grid, dim3(256), 0, st, codes, scales, rows, K, dst);
    else
      hipLaunchKernelGGL((mx_dequantize_kernel<false, false>), grid, dim3(256), 0, st, codes, scales, rows, K, dst);
  }
  return hipGetLastError();
}

hipError_t launch_dispatch_mx4(const moe_shape_t& s, const void* const* x, const int32_t* pull_src, uint8_t* xe,
                               uint8_t* xe_scales, int64_t nmax, const int32_t* ctrl, int cus, hipStream_t st) {
  RankPtrs<const char*> xp{};
  for (int r = 0; r < s.R; ++r) xp.p[r] = static_cast<const char*>(x[r]);
  // From d = 524288 on the words of the four rows that a workgroup takes at least pass the 64 KiB of LDS a
  // launch may ask for: then as many workgroups as rows there can be, which each take one row without LDS.
  const int64_t row_words = (s.d >> 7) + 1;
  const bool wide = 4 * row_words * 4 > 65536;
  const int cr = wide ? 4 : mx_chunk_rows(s.d);
  const size_t lds = wide ? 0 : cr * row_words * 4;
  const int n16 = s.d >> 3;
  // 32700 rows of 7168: 111 us; 8 workgroups a CU 114, 4 a CU 125.  No more of them than rows there can be
  // (no row: 1.7 us, and 2.1 with all of them).
  const dim3 grid(wide || nmax < cus * 16 ? int(nmax) : cus * 16);
  // two short rows at a time: 24.0 us against 26.6 for 23300 rows of 2048
  if (n16 <= 64 * 4)
    hipLaunchKernelGGL((dispatch_pull_mx4_kernel<4, 2>), grid, dim3(256), lds, st, xp, pull_src, ctrl, xe, xe_scales, s.d, nmax, cr);
  else if (n16 <= 64 * 8)
    hipLaunchKernelGGL((dispatch_pull_mx4_kernel<8, 1>), grid, dim3(256), lds, st, xp, pull_src, ctrl, xe, xe_scales, s.d, nmax, cr);
  else
    hipLaunchKernelGGL((dispatch_pull_mx4_kernel<14, 1>), grid, dim3(256), lds, st, xp, pull_src, ctrl, xe, xe_scales, s.d, nmax, cr);
  return hipGetLastError();
}

}  // namespace moe
