// The MXFP4 expert FFN for experts with few rows (decoding): the weights stream once from HBM,
// each wave on its own.
//
// The formulas are gemm_mx4.hip's.  With at most kThinRows rows per expert the products are
// bound by the weights' bytes (17/32 a value), so the kernel is built to keep enough of them in
// flight: an item is 64 weight rows (32 f of W1 and of W3; 64 columns of W2) of one expert, and a
// wave streams units of 256 K values of those rows and of the expert's token rows through LDS
// stages of its own, filled by direct global->LDS loads that take whole 128-byte lines (8 rows a
// load).  No wave waits for another, and the fills run on across items, so the memory never idles
// at an item's end.  (Fragments loaded straight into registers take 32 bytes of each line per
// load; the four loads of a line are not merged, and the GEMM1 of 32 experts of 2048 x 7168 took
// 137 us that way instead of 89, both with cached weights.)
//
// Weights are the MFMA's A operand and the token rows its B operand, so a lane ends up with 16
// of the 32 f values (or columns) of one token row, and its partner in the other half with the
// rest: the block maximum of h is one exchange.
//
// SPLIT 1: a wave takes an item alone, three stages.  SPLIT 4: the workgroup's four waves share
// an item's units and add up through LDS in wave order (two stages), for so few items that waves
// alone would leave most of the card idle (GEMM2 of 6 experts of 1408 x 2048: 5.1 us against 8.1; of 32
// experts of 2048 x 7168: 57 against 52).
//
// 32 experts of 2048 x 7168, 512 rows: 80.6 us + 48.1 us for 749 MB, 5.8 TB/s.  Six experts of 1408 x 2048,
// one row each: 10.0 us + 5.1 us, bound by the latency of offsets, loads and sums.
#include "gemm_tile.hpp"
#include "mx4.hpp"

namespace moe {

constexpr int kThinWaves = 4;
constexpr int kUnitW = 64 * 128, kUnitX = 32 * 128;          // bytes of a unit's weight and token codes
constexpr int kUnitBytes = kUnitW + kUnitX + 2 * 256 + 256;  // + scale words of two K tiles
constexpr int kUnitFills = 8 + 4 + 2 + 1;                    // loads of a unit
constexpr int kPartBytes = 64 * 32 * 4;                      // a wave's accumulators

constexpr int thin_stages(int split) { return split == 1 ? 3 : 2; }
constexpr int thin_lds(int split) {
  return kThinWaves * (thin_stages(split) * kUnitBytes + (split == 1 ? 0 : kPartBytes));
}

struct ThinArgs {
  const uint8_t* a;       // token rows' codes, row stride K / 2; scales as, planes of 4 * nmax bytes
  const uint8_t* as;
  const uint8_t* b0;      // weight codes [El][Nout][K / 2] (MODE 0: W1 and W3, MODE 1 and 2: W2 for both)
  const uint8_t* b1;
  const uint8_t* bs0;     // their scales, planes of 4 * El * Nout bytes
  const uint8_t* bs1;
  void* o;                // MODE 0: h codes, row stride Nout / 2; MODE 1: bf16 rows, stride Nout (or row_dst); MODE 2: fp32 rows
  uint8_t* os;            // MODE 0: h scales, planes of 4 * nmax bytes
  const int32_t* offsets;
  const uint64_t* row_dst;
  int64_t nmax;
  int El, K, Nout;
};

// An item's place, the same in every lane
struct ThinItem {
  const uint8_t *w0, *w1, *s0, *s1, *x, *xs;
  int row0, rows, cb;
};

template <int MODE, int SPLIT>
__global__ __launch_bounds__(256, 1) void thin_mx4_kernel(ThinArgs g) {
  extern __shared__ __attribute__((aligned(16))) char smem[];
  __shared__ int16_t list[1024];          // the experts with 1..kThinRows rows, ascending
  __shared__ int n_list;
  constexpr int kStages = thin_stages(SPLIT);
  // Many items: the weights pass by once and would only push each other and the token rows out of the
  // caches (non-temporal: 151 us for the layer on 32 experts of 2048 x 7168, 512 rows, instead of
  // 167; the scale words stay cached, their lines serve two loads: 149 against 154).  Few: they may well be there still from the last token (27.5 us against 28.4).
  constexpr int kWeightPolicy = SPLIT == 1 ? 2 : 0;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int r32 = lane & 31, hi = lane >> 5;
  if (wave == 0) {
    int n = 0;
    for (int l0 = 0; l0 < g.El; l0 += 64) {
      const int l = l0 + lane;
      const int rows = l < g.El ? g.offsets[l + 1] - g.offsets[l] : 0;
      const unsigned long long on = __ballot(rows > 0 && rows <= kThinRows);
      if ((on >> lane) & 1) list[n + __popcll(on & ((1ull << lane) - 1))] = int16_t(l);
      n += __popcll(on);
    }
    if (lane == 0) n_list = n;
  }
  __syncthreads();
  const int np = g.K >> 7, nu = (np + 1) >> 1;                // K tiles of 128, units of 256
  const int ncb = MODE == 0 ? g.Nout >> 5 : g.Nout >> 6;
  const int items = n_list * ncb;                             // at most 1024 * 2^25 / 2^5: d * F < 2^32
  const uint32_t rb = uint32_t(g.K >> 1);
  const size_t splane = 4 * size_t(g.El) * g.Nout, xplane = 4 * size_t(g.nmax);
  const int it0 = SPLIT == 1 ? __builtin_amdgcn_readfirstlane(int(blockIdx.x) * kThinWaves + wave) : int(blockIdx.x);
  const int it_step = SPLIT == 1 ? int(gridDim.x) * kThinWaves : int(gridDim.x);
  const int u0 = SPLIT == 1 ? 0 : __builtin_amdgcn_readfirstlane(wave);

  // scalar loads: a vector load's wait would drain the fills in flight
  const auto* const offs = (const __attribute__((address_space(4))) int32_t*)reinterpret_cast<uintptr_t>(g.offsets);
  auto place = [&](int it) -> ThinItem {
    ThinItem t;
    const int l = __builtin_amdgcn_readfirstlane(int(list[it / ncb]));
    t.cb = it % ncb;
    t.row0 = offs[l];
    t.rows = offs[l + 1] - t.row0;
    // MODE 0: weight rows cb * 32 .. + 31 of W1 and of W3; MODE 1: rows cb * 64 .. + 31 and + 32 .. + 63 of W2
    const size_t n = size_t(l) * g.Nout + (MODE == 0 ? t.cb * 32 : t.cb * 64);
    const size_t n1 = MODE == 0 ? n : n + 32;
    t.w0 = g.b0 + n * rb;
    t.w1 = g.b1 + n1 * rb;
    t.s0 = g.bs0 + 4 * n;
    t.s1 = g.bs1 + 4 * n1;
    t.x = g.a + size_t(t.row0) * rb;
    t.xs = g.as + 4 * size_t(t.row0);
    return t;
  };

  // fills of one unit: lane -> row lrow of an 8-row group, LDS chunk lpos of its 128-byte line, which
  // holds logical chunk lpos ^ ((row >> 1) & 7) (the swizzle the fragment reads undo)
  const int lrow = lane >> 3, lpos = lane & 7;
  const int lch_even = lpos ^ (lrow >> 1), lch_odd = lpos ^ (4 + (lrow >> 1));
  const uint32_t even = uint32_t(lrow) * rb + lch_even * 16, odd = uint32_t(lrow) * rb + lch_odd * 16;
  const uint32_t lds0 = __builtin_amdgcn_readfirstlane(lds_addr(smem + wave * kStages * kUnitBytes));
  auto fill = [&](const ThinItem& t, int u, int stage) {
    const uint32_t dst = lds0 + uint32_t(stage * kUnitBytes);
    const bool tail = 2 * u + 1 >= np;          // only half a unit is left: re-read its first half (never used)
    const uint32_t te = tail ? uint32_t(lch_even & 4) * 16 : 0, to = tail ? uint32_t(lch_odd & 4) * 16 : 0;
    const size_t koff = size_t(u) * 128;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const uint8_t* base = (i < 4 ? t.w0 : t.w1) + size_t((i & 3) * 8) * rb + koff;
      __builtin_amdgcn_global_load_lds(static_cast<const void*>(base + ((i & 1) ? odd - to : even - te)),
                                       (lds_void_ptr)(uintptr_t)(dst + uint32_t(i * 1024)), 16, 0, kWeightPolicy);
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {               // token rows past the last re-read it, are not stored
      const uint32_t at = uint32_t(min(i * 8 + lrow, t.rows - 1)) * rb + ((i & 1) ? lch_odd * 16 - to : lch_even * 16 - te);
      __builtin_amdgcn_global_load_lds(static_cast<const void*>(t.x + koff + at),
                                       (lds_void_ptr)(uintptr_t)(dst + uint32_t(kUnitW + i * 1024)), 16, 0, 0);
    }
    const size_t p0 = 2 * u, p1 = tail ? p0 : p0 + 1;
    const uint8_t* sw = (hi ? t.s1 : t.s0) + 4 * r32;
    __builtin_amdgcn_global_load_lds(static_cast<const void*>(sw + p0 * splane),
                                     (lds_void_ptr)(uintptr_t)(dst + uint32_t(kUnitW + kUnitX)), 4, 0, 0);
    __builtin_amdgcn_global_load_lds(static_cast<const void*>(sw + p1 * splane),
                                     (lds_void_ptr)(uintptr_t)(dst + uint32_t(kUnitW + kUnitX + 256)), 4, 0, 0);
    __builtin_amdgcn_global_load_lds(static_cast<const void*>(t.xs + (hi ? p1 : p0) * xplane + 4 * min(r32, t.rows - 1)),
                                     (lds_void_ptr)(uintptr_t)(dst + uint32_t(kUnitW + kUnitX + 512)), 4, 0, 0);
  };

  // the fill cursor runs kStages - 1 units ahead of the products, across items
  int fit = it0, fu = u0, fstage = 0, ahead = 0;
  ThinItem ft;
  if (u0 >= nu) fit = items;                    // a wave without units (SPLIT 4, short K)
  if (fit < items) ft = place(fit);
  auto fill_next = [&]() {
    if (fit >= items) return;
    fill(ft, fu, fstage);
    fstage = fstage + 1 == kStages ? 0 : fstage + 1;
    ++ahead;
    fu += SPLIT;
    if (fu >= nu) {
      fu = u0;
      fit += it_step;
      if (fit < items) ft = place(fit);
    }
  };
#pragma unroll
  for (int i = 0; i < kStages - 1; ++i) fill_next();

  const char* const mine = smem + wave * kStages * kUnitBytes;
  int offW[4], offX[4];
#pragma unroll
  for (int st = 0; st < 4; ++st) {
    offW[st] = swz_off(r32, 2 * st + hi);
    offX[st] = kUnitW + swz_off(r32, 2 * st + hi);
  }
  auto frag = [&](const char* s, int off) -> i32x8 {
    const i32x4 v = *reinterpret_cast<const i32x4*>(s + off);
    return i32x8{v[0], v[1], v[2], v[3], 0, 0, 0, 0};
  };
  auto word = [&](const char* s, int off) -> int {       // byte 2 st + hi is the block of this half in step st
    return int(*reinterpret_cast<const uint32_t*>(s + kUnitW + kUnitX + off + 4 * r32) >> (8 * hi));
  };

  int stage = 0;
  for (int it = it0; it < items; it += it_step) {
    f32x16 acc[2];
#pragma unroll
    for (int q = 0; q < 2; ++q)
#pragma unroll
      for (int e = 0; e < 16; ++e) acc[q][e] = 0.0f;
    for (int u = u0; u < nu; u += SPLIT) {
      fill_next();                              // into the stage read last
      --ahead;                                  // units filled behind this one
      if (ahead >= 2) asm volatile("s_waitcnt vmcnt(%0)" ::"n"(2 * kUnitFills) : "memory");
      else if (ahead == 1) asm volatile("s_waitcnt vmcnt(%0)" ::"n"(kUnitFills) : "memory");
      else asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
      const char* s = mine + stage * kUnitBytes;
      stage = stage + 1 == kStages ? 0 : stage + 1;
      const bool both = 2 * u + 1 < np;
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        if (h == 1 && !both) break;
        const int sx = word(s, 512 + 128 * h), s0 = word(s, 256 * h), s1 = word(s, 256 * h + 128);
        const i32x8 x0 = frag(s, offX[2 * h]), x1 = frag(s, offX[2 * h + 1]);
        acc[0] = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(frag(s, offW[2 * h]), x0, acc[0], 4, 4, 0, s0, 0, sx);
        acc[1] = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(frag(s, offW[2 * h] + 4096), x0, acc[1], 4, 4, 0, s1, 0, sx);
        acc[0] = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(frag(s, offW[2 * h + 1]), x1, acc[0], 4, 4, 2, s0, 2, sx);
        acc[1] = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(frag(s, offW[2 * h + 1] + 4096), x1, acc[1], 4, 4, 2, s1, 2, sx);
      }
      asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");      // the stage is read: its next fill may come
    }
    if constexpr (SPLIT > 1) {                  // add the waves' parts in wave order
      f32x4* part = reinterpret_cast<f32x4*>(smem + kThinWaves * kStages * kUnitBytes);      // [wave][q][4][64]
#pragma unroll
      for (int q = 0; q < 2; ++q)
#pragma unroll
        for (int c = 0; c < 4; ++c)
          part[((wave * 2 + q) * 4 + c) * 64 + lane] =
              f32x4{acc[q][4 * c], acc[q][4 * c + 1], acc[q][4 * c + 2], acc[q][4 * c + 3]};
      __syncthreads();
      if (wave == 0) {
#pragma unroll
        for (int q = 0; q < 2; ++q)
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            f32x4 s = part[(q * 4 + c) * 64 + lane];
#pragma unroll
            for (int w = 1; w < kThinWaves; ++w) s += part[((w * 2 + q) * 4 + c) * 64 + lane];
#pragma unroll
            for (int e = 0; e < 4; ++e) acc[q][4 * c + e] = s[e];
          }
      }
      __syncthreads();                          // the next item's parts may come
    }
    if (SPLIT == 1 || wave == 0) {
      const ThinItem t = place(it);
      const int64_t row = t.row0 + r32;
      // value 4 c + e of a lane is weight row 8 c + 4 hi + e of the block of 32
      if (MODE == 0) {
        uint32_t mx = 0;
        float h[16];
#pragma unroll
        for (int e = 0; e < 16; ++e) {
          h[e] = mx4_silu(acc[0][e]) * acc[1][e];
          mx = max(mx, __float_as_uint(h[e]) & 0x7FFFFFFFu);
        }
        mx = max(mx, uint32_t(__shfl_xor(int(mx), 32, 64)));
        const uint32_t sc = mx4_scale_code(mx);
        if (r32 < t.rows) {
          uint8_t* hrow = static_cast<uint8_t*>(g.o) + size_t(row) * (g.Nout >> 1) + t.cb * 16 + hi * 2;
          const float f = e8m0_f32(sc);
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            uint32_t code = 0;
            if (!mx4_blank(mx)) {
              code = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(code, h[4 * c], h[4 * c + 1], f, 0);
              code = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(code, h[4 * c + 2], h[4 * c + 3], f, 1);
            }
            *reinterpret_cast<uint16_t*>(hrow + 4 * c) = uint16_t(code);
          }
          if (hi == 0) g.os[(t.cb >> 2) * 4 * g.nmax + 4 * row + (t.cb & 3)] = uint8_t(sc);
        }
      } else if (MODE == 2) {
        f32x4* dst = reinterpret_cast<f32x4*>(static_cast<float*>(g.o) + size_t(row) * g.Nout + t.cb * 64 + hi * 4);
        if (r32 < t.rows) {
#pragma unroll
          for (int q = 0; q < 2; ++q)
#pragma unroll
            for (int c = 0; c < 4; ++c)
              dst[8 * q + 2 * c] = f32x4{acc[q][4 * c], acc[q][4 * c + 1], acc[q][4 * c + 2], acc[q][4 * c + 3]};
        }
      } else if (r32 < t.rows) {
        uint16_t* orow = g.row_dst ? reinterpret_cast<uint16_t*>(g.row_dst[row])
                                   : static_cast<uint16_t*>(g.o) + size_t(row) * g.Nout;
        uint2* dst = reinterpret_cast<uint2*>(orow + t.cb * 64 + hi * 4);
#pragma unroll
        for (int q = 0; q < 2; ++q)
#pragma unroll
          for (int c = 0; c < 4; ++c)
            dst[8 * q + 2 * c] = make_uint2(pack_bf16x2(acc[q][4 * c], acc[q][4 * c + 1]),
                                            pack_bf16x2(acc[q][4 * c + 2], acc[q][4 * c + 3]));
      }
    }
  }
}

// `experts`: how many may have rows at most (the host's bound: local experts and pairs)
hipError_t launch_thin_mx4(bool gate_up, const uint8_t* a, const uint8_t* as, const uint8_t* b0, const uint8_t* b1,
                           const uint8_t* bs0, const uint8_t* bs1, void* o, uint8_t* os, const int32_t* offsets,
                           const uint64_t* row_dst, bool rows32, int64_t nmax, int El, int64_t experts, int K, int Nout,
                           int cus, hipStream_t st) {
  static std::atomic<uint64_t> attr_set{0};
  const hipError_t ea = once_per_device(attr_set, [] {
    const struct {
      const void* f;
      int lds;
    } ks[] = {{reinterpret_cast<const void*>(thin_mx4_kernel<0, 1>), thin_lds(1)},
              {reinterpret_cast<const void*>(thin_mx4_kernel<0, 4>), thin_lds(4)},
              {reinterpret_cast<const void*>(thin_mx4_kernel<1, 1>), thin_lds(1)},
              {reinterpret_cast<const void*>(thin_mx4_kernel<1, 4>), thin_lds(4)},
              {reinterpret_cast<const void*>(thin_mx4_kernel<2, 1>), thin_lds(1)},
              {reinterpret_cast<const void*>(thin_mx4_kernel<2, 4>), thin_lds(4)}};
    for (const auto& k : ks) {
      const hipError_t e = hipFuncSetAttribute(k.f, hipFuncAttributeMaxDynamicSharedMemorySize, k.lds);
      if (e != hipSuccess) return e;
    }
    return hipSuccess;
  });
  if (ea != hipSuccess) return ea;
  const ThinArgs g{a, as, b0, b1, bs0, bs1, o, os, offsets, row_dst, nmax, El, K, Nout};
  const int64_t items = experts * (gate_up ? Nout >> 5 : Nout >> 6);
  const bool alone = items >= int64_t(cus) * kThinWaves;     // a wave per item fills the card
  const int64_t wgs = alone ? (items + kThinWaves - 1) / kThinWaves : items;
  const dim3 grid(int(wgs < cus ? wgs : cus));               // one workgroup per CU (LDS)
  if (gate_up && alone) hipLaunchKernelGGL((thin_mx4_kernel<0, 1>), grid, dim3(256), thin_lds(1), st, g);
  else if (gate_up) hipLaunchKernelGGL((thin_mx4_kernel<0, 4>), grid, dim3(256), thin_lds(4), st, g);
  else if (rows32 && alone) hipLaunchKernelGGL((thin_mx4_kernel<2, 1>), grid, dim3(256), thin_lds(1), st, g);
  else if (rows32) hipLaunchKernelGGL((thin_mx4_kernel<2, 4>), grid, dim3(256), thin_lds(4), st, g);
  else if (alone) hipLaunchKernelGGL((thin_mx4_kernel<1, 1>), grid, dim3(256), thin_lds(1), st, g);
  else hipLaunchKernelGGL((thin_mx4_kernel<1, 4>), grid, dim3(256), thin_lds(4), st, g);
  return hipGetLastError();
}

}  // namespace moe
