// Pull dispatch of token rows that are in MXFP8 or MXFP4 already (moe_norm's codes, moe_mx_quantize_to's): codes and scale
// words in expert order.
//
//   xe[s] = xq[r][t], xe_scales[:, s] = xq_scales[r][:, t] with (r, t) = pull_src[s].
//
// Half (a quarter) of the bytes that the bf16 rows would cost on the way to their experts, and a token is quantised once
// instead of at every expert that it goes to.  Bound by bytes: a wave copies a row's codes in 16-byte vectors, four a lane
// in flight at once.  The scale words of a row lie in d / 128 planes; a workgroup collects those of its chunk of
// rows in LDS and writes each plane's words as one run.  32700 rows of 7168 codes 71 us (6.8 TB/s, tokens partly in the caches), 512 rows 4.9 us.
#include "common.hpp"

namespace moe {

constexpr int kCodesRows = 32;            // rows of a workgroup's chunk
// Vectors that a lane has in flight: 16384 rows of 7168 bytes to two experts each 70.7 us with two, 70.0 with four, 73 with seven (a whole row)
constexpr int U = 4;

__global__ __launch_bounds__(256) void dispatch_codes_kernel(RankPtrs<const char*> xq, RankPtrs<const uint32_t*> xs,
                                                             const int32_t* __restrict__ pull_src,
                                                             const int32_t* __restrict__ ctrl, char* __restrict__ xe,
                                                             uint32_t* __restrict__ xes, int row_bytes, int nq, int T,
                                                             int64_t nmax) {
  __shared__ int2 s_src[kCodesRows];
  const int N = ctrl[kCtrlN];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int n16 = row_bytes >> 4;
  // fewer rows than every workgroup could take: shorter chunks
  const int cr = min(kCodesRows, max(4, ((N + int(gridDim.x) - 1) / int(gridDim.x) + 3) & ~3));
  const int chunks = (N + cr - 1) / cr;
  for (int c = blockIdx.x; c < chunks; c += gridDim.x) {
    const int s0 = c * cr, rows = min(cr, N - s0);
    if (int(threadIdx.x) < rows) s_src[threadIdx.x] = reinterpret_cast<const int2*>(pull_src)[s0 + threadIdx.x];
    __syncthreads();
    for (int rr = wave; rr < rows; rr += 4) {
      const int2 from = s_src[rr];
      const u32x4* src = reinterpret_cast<const u32x4*>(xq.p[from.x] + int64_t(from.y) * row_bytes);
      u32x4* dst = reinterpret_cast<u32x4*>(xe + int64_t(s0 + rr) * row_bytes);
      for (int base = 0; base < n16; base += 64 * U) {
        u32x4 v[U];
#pragma unroll
        for (int u = 0; u < U; ++u)
          if (base + u * 64 + lane < n16) v[u] = __builtin_nontemporal_load(src + base + u * 64 + lane);
#pragma unroll
        for (int u = 0; u < U; ++u)
          if (base + u * 64 + lane < n16) dst[base + u * 64 + lane] = v[u];
      }
    }
    for (int e = threadIdx.x; e < nq * rows; e += 256) {
      const int q = e / rows, rr = e - q * rows;
      const int2 from = s_src[rr];
      xes[nmax * q + s0 + rr] = xs.p[from.x][int64_t(q) * T + from.y];
    }
    __syncthreads();                      // the next chunk's sources overwrite these
  }
}

hipError_t launch_dispatch_codes(const moe_shape_t& s, const uint8_t* const* xq, const uint8_t* const* xq_scales,
                                 const int32_t* pull_src, uint8_t* xe, uint8_t* xe_scales, int64_t nmax,
                                 const int32_t* ctrl, int cus, hipStream_t st) {
  RankPtrs<const char*> q{};
  RankPtrs<const uint32_t*> w{};
  for (int r = 0; r < s.R; ++r) {
    q.p[r] = reinterpret_cast<const char*>(xq[r]);
    w.p[r] = reinterpret_cast<const uint32_t*>(xq_scales[r]);
  }
  const int row_bytes = s.dtype == MOE_MXFP8 ? s.d : s.d / 2;
  const int64_t need = (nmax + 3) / 4;
  const dim3 grid(int(need < cus * 8 ? need : cus * 8));
  char* out = reinterpret_cast<char*>(xe);
  uint32_t* words = reinterpret_cast<uint32_t*>(xe_scales);
  hipLaunchKernelGGL(dispatch_codes_kernel, grid, dim3(256), 0, st, q, w, pull_src, ctrl, out, words, row_bytes, s.d >> 7, s.T, nmax);
  return hipGetLastError();
}

}  // namespace moe
