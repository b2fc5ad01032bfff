// Grouped SwiGLU expert FFN in MXFP4 on gfx950 (v_mfma_scale_f32_32x32x64_f8f6f4, both
// operands FP4).
//
// Operation (grouped GEMM over expert-contiguous rows and SwiGLU: MoK article, kucoin.com/es
// "Cursor's MoK logra un aumento del 2.37x ...", sections 01 and 02):
//   GEMM1: h = MX4(silu(X W1^T) * (X W3^T))   X, W1, W3 in MXFP4 (blocks of 32 along d)
//   GEMM2: y = h W2^T (bf16 out)               h, W2 in MXFP4 (blocks of 32 along F)
// h is quantised in GEMM1's epilogue, so it reaches HBM once, at half a byte per value.
//
// The tile keeps the byte geometry of the MXFP8 one (256 x 256, 8 waves as 4 x 2, 128-byte LDS
// rows with the same XOR swizzle, direct global->LDS fills), so a stage holds 256 K values and
// two scale words per row, and four MFMA sub-steps of 64.  K is a multiple of 128: the last
// stage may hold only half, whose second half is neither read past the rows' ends nor used.
#include "gemm_mx4_tile.hpp"

namespace moe {

// MODE 0: A = xe codes [*][d/2], B0/B1 = W1/W3 -> h codes [*][F/2] + scales   (256 rows x 128 f)
// MODE 1: A = h codes [*][F/2],  B0 = W2 -> bf16 [*][d]                        (256 x 256)
// Tile enumeration as in the other grouped GEMMs: a persistent grid walks 8 contiguous
// per-XCD ranges of the expert-major tile list.
template <int MODE>
__global__ __launch_bounds__(kGemmThreads, 1) void grouped_gemm_mx4_kernel(
    const uint8_t* __restrict__ A, const uint8_t* __restrict__ As, const uint8_t* __restrict__ B0,
    const uint8_t* __restrict__ B1, const uint8_t* __restrict__ Bs0, const uint8_t* __restrict__ Bs1,
    void* __restrict__ C, uint8_t* __restrict__ Cs, const int32_t* __restrict__ offsets,
    const int32_t* __restrict__ mtile_base, const int32_t* __restrict__ ctrl, int El, int K, int Nout,
    int64_t nmax, const uint64_t* __restrict__ RowDst, int min_rows) {
  extern __shared__ __attribute__((aligned(16))) char smem[];
  if (min_rows > 0) {      // few rows expected: often the streaming kernel has taken every expert
    int any = 0;
    for (int l = threadIdx.x; l < El; l += kGemmThreads) any |= offsets[l + 1] - offsets[l] >= min_rows;
    if (!__syncthreads_or(any)) return;
  }
  const int cols_per_tile = (MODE == 0) ? kGemmBN / 2 : kGemmBN;
  const int NT = (Nout + cols_per_tile - 1) / cols_per_tile;
  const int total = ctrl[kCtrlMTiles] * NT;
  const int per_xcd = (total + 7) >> 3;
  const int xcd = blockIdx.x & 7;
  const int wg_per_xcd = gridDim.x >> 3;
  const int64_t bs_plane = 4 * int64_t(El) * Nout;    // weight scale planes hold every expert's rows

  for (int tt = blockIdx.x >> 3; tt < per_xcd; tt += wg_per_xcd) {
    const int tau = xcd * per_xcd + tt;
    if (tau >= total) break;
    const int mtg = tau / NT;
    const int l = find_expert(mtile_base, El, mtg);
    const int mt0 = mtile_base[l];
    if (offsets[l + 1] - offsets[l] < min_rows) continue;      // the streaming kernel's
    const int mtl = mtile_base[l + 1] - mt0;
    const int i_in = tau - mt0 * NT;
    const int nt = i_in / mtl, mt = i_in - nt * mtl;
    const int row0 = offsets[l] + mt * kGemmBM;
    TileMX4 io;
    io.a = A + size_t(row0) * (K >> 1);
    io.as = As + 4 * size_t(row0);
    io.as_plane = 4 * nmax;
    io.rows = min(kGemmBM, offsets[l + 1] - row0);
    if (MODE == 0) {
      io.o = static_cast<uint8_t*>(C) + size_t(row0) * (Nout >> 1);
      io.os = Cs + 4 * size_t(row0);
      io.os_plane = 4 * nmax;
      io.row_dst = nullptr;
    } else {
      io.o = C ? static_cast<uint16_t*>(C) + size_t(row0) * Nout : nullptr;   // null C: with RowDst
      io.os = nullptr;
      io.os_plane = 0;
      io.row_dst = RowDst ? RowDst + row0 : nullptr;
    }
    const size_t wb = size_t(l) * Nout * (K >> 1);
    const uint8_t* bs0 = Bs0 + 4 * size_t(l) * Nout;
    const uint8_t* bs1 = (MODE == 0) ? Bs1 + 4 * size_t(l) * Nout : bs0;
    gemm_mx4_tile<MODE>(io, B0 + wb, (MODE == 0) ? B1 + wb : B0 + wb, bs0, bs1, bs_plane, nt * cols_per_tile, Nout, K,
                        smem);
  }
}

hipError_t launch_thin_mx4(bool gate_up, const uint8_t* a, const uint8_t* as, const uint8_t* b0, const uint8_t* b1,
                           const uint8_t* bs0, const uint8_t* bs1, void* o, uint8_t* os, const int32_t* offsets,
                           const uint64_t* row_dst, int64_t nmax, int El, int64_t experts, int K, int Nout, int cus,
                           hipStream_t st);

hipError_t launch_ffn_mx4(const moe_shape_t& s, int El, const uint8_t* xe, const uint8_t* xe_scales,
                          const int32_t* offsets, const uint8_t* w1, const uint8_t* w3, const uint8_t* w2,
                          const moe_mx_scales_t& w_scales, void* ye, char* ws, const WsLayout& L, int cus,
                          hipStream_t st, const uint64_t* row_dst) {
  static std::atomic<uint64_t> attr_set{0};
  const hipError_t ea = once_per_device(attr_set, [] {
    hipError_t e = hipFuncSetAttribute(reinterpret_cast<const void*>(grouped_gemm_mx4_kernel<0>),
                                       hipFuncAttributeMaxDynamicSharedMemorySize, kMx4Lds);
    if (e == hipSuccess)
      e = hipFuncSetAttribute(reinterpret_cast<const void*>(grouped_gemm_mx4_kernel<1>),
                              hipFuncAttributeMaxDynamicSharedMemorySize, kMx4Lds);
    return e;
  });
  if (ea != hipSuccess) return ea;
  const int32_t* ctrl = reinterpret_cast<const int32_t*>(ws + L.ctrl);
  const int32_t* mtb = reinterpret_cast<const int32_t*>(ws + L.mtile_base);
  uint8_t* hq = reinterpret_cast<uint8_t*>(ws + L.hbuf);
  uint8_t* hs = hq + mx4_h_scales_offset(L.max_pairs, s.F);
  const int grid = (cus / 8) * 8;
  // Which experts have few rows is known on the device only.  An expert has at most R T rows (a
  // token names it once) and, under an even load, R T k / E.  So with at most kThinRows tokens the
  // streaming kernel does it all; with kThinRows rows expected of an expert or more the tile
  // kernel does; in between both run, each on its experts.
  const int64_t tokens = int64_t(s.R) * s.T;
  const bool thin = tokens <= kThinRows || tokens * s.k <= int64_t(kThinRows) * s.E;
  const bool wide = tokens > kThinRows;
  const int min_rows = thin ? kThinRows + 1 : 0;
  const int64_t nmax = L.max_pairs;
  const int64_t experts = El < nmax ? El : nmax;             // with a row, at most
  if (thin) {
    const hipError_t e = launch_thin_mx4(true, xe, xe_scales, w1, w3, w_scales.w1, w_scales.w3, hq, hs, offsets, nullptr,
                                         nmax, El, experts, s.d, s.F, cus, st);
    if (e != hipSuccess) return e;
  }
  if (wide)
    hipLaunchKernelGGL(grouped_gemm_mx4_kernel<0>, dim3(grid), dim3(kGemmThreads), kMx4Lds, st, xe, xe_scales, w1, w3,
                       w_scales.w1, w_scales.w3, static_cast<void*>(hq), hs, offsets, mtb, ctrl, El, s.d, s.F, nmax,
                       nullptr, min_rows);
  if (thin) {
    const hipError_t e = launch_thin_mx4(false, hq, hs, w2, w2, w_scales.w2, w_scales.w2, ye, nullptr, offsets, row_dst,
                                         nmax, El, experts, s.F, s.d, cus, st);
    if (e != hipSuccess) return e;
  }
  if (wide)
    hipLaunchKernelGGL(grouped_gemm_mx4_kernel<1>, dim3(grid), dim3(kGemmThreads), kMx4Lds, st, hq, hs, w2, nullptr,
                       w_scales.w2, nullptr, ye, nullptr, offsets, mtb, ctrl, El, s.F, s.d, nmax, row_dst, min_rows);
  return hipGetLastError();
}

}  // namespace moe
