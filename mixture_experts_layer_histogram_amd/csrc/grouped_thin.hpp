// Products grouped by expert where a group has few rows (decoding): the weights stream once from HBM, each wave on its own.
//
// An item is 64 output columns of up to 32 rows of one group.  A wave streams 64 K values of them at a time through LDS stages of its own,
// 8 KiB of weights and 4 KiB of rows, filled by direct global->LDS loads that take whole 128-byte lines, with two stages in flight
// while a third is at work; the fills run on across items.  Weights are the MFMA's first operand (v_mfma_f32_16x16x32_bf16), so a lane
// ends up with four consecutive columns of one row.  32 groups of 7168 x 2048, 509 rows: 147 us, 6.4 TB/s of weights.
//
// SPLIT 1: a wave takes an item alone.  SPLIT 4: the workgroup's four waves share an item's K and add up through LDS in wave order (two
// stages each), where the items do not come out even on the waves; thin_alone has the figures.
#pragma once

#include "grouped.hpp"
#include "grouped_tile.hpp"

namespace moe {

constexpr int kThinCols = 64, kThinRows = 32, kThinK = 64;
constexpr int kThinW = kThinCols * kThinK * 2, kThinStage = kThinW + kThinRows * kThinK * 2;
constexpr int kThinFills = kThinStage / 1024;                       // loads of a stage
constexpr int kThinPart = kThinCols * kThinRows * 4;                // a wave's sums

constexpr int thin_ring(int split) { return split == 1 ? 3 : 2; }
constexpr int thin_lds_bytes(int split) { return 4 * (thin_ring(split) * kThinStage + (split == 1 ? 0 : kThinPart)); }
constexpr int kThinLds = thin_lds_bytes(1) > thin_lds_bytes(4) ? thin_lds_bytes(1) : thin_lds_bytes(4);

// Whether waves take items alone: turns of all waves against turns of all workgroups, which are a quarter as long and lose a tenth (weights
// stored [N][K]) to a quarter ([K][N], where four waves far apart in K read 128 bytes of a row each) to sums and shorter queues.  32 groups of
// 7168 x 2048, us alone and split: 1024 items 149 and 159, in the other layout 163 and 205; 1056 items 237 and 181; 3584 items 202
// and 169; 64 groups of 2048 x 1408, one row each (1408 items): 84 and 69; 132 items: 16 and 9.
// Of few K steps there is little to share: always alone below 8 (us split and alone: 91 groups of 16 x 5040, 438 rows 64 and 22, 64 of 128 x 2048,
// 1024 rows 23 and 13, of 448 x 2048 31 and 27).
__device__ __forceinline__ bool thin_alone(int items, int wgs, int steps, bool w_kn) {
  if (steps < 8) return true;
  const int one = (items + 4 * wgs - 1) / (4 * wgs), four = (items + wgs - 1) / wgs;
  return one * (w_kn ? 16 : 37) <= four * (w_kn ? 5 : 10);
}

// The LDS place of 16-byte chunk c of K row k where the columns are contiguous (128 bytes a K row) is c ^ this
__device__ __forceinline__ int thin_swz(int k) { return 2 * (((k >> 1) & 1) | (((k >> 3) & 1) << 1)); }

template <bool W_KN, int SPLIT>
__device__ __forceinline__ void thin_run(const GroupedArgs& g, const int32_t* base, int mtiles, char* smem) {
  constexpr int S = thin_ring(SPLIT);
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int r16 = lane & 15, q = lane >> 4;
  const int ncb = (g.N + kThinCols - 1) / kThinCols, nst = (g.K + kThinK - 1) / kThinK;
  const int items = mtiles * ncb;                     // below 2^29: rows a group are few here, and the weights, 16 bytes a column at least, fit in memory
  const int it0 = SPLIT == 1 ? int(blockIdx.x) * 4 + wave : int(blockIdx.x);
  const int it_step = SPLIT == 1 ? int(gridDim.x) * 4 : int(gridDim.x);
  const int s0 = SPLIT == 1 ? 0 : nst * wave / 4, s1 = SPLIT == 1 ? nst : nst * (wave + 1) / 4;

  // an item's place, the same in every lane
  struct Item {
    int l, rows, c0;
    int64_t row0;
  };
  const auto* const offs = (const __attribute__((address_space(4))) int32_t*)reinterpret_cast<uintptr_t>(g.offsets);
  auto place = [&](int it) -> Item {
    Item t;
    const int mtg = __builtin_amdgcn_readfirstlane(int(uint32_t(it) / uint32_t(ncb)));
    t.l = __builtin_amdgcn_readfirstlane(find_expert(base, g.G, mtg));
    const int b0 = __builtin_amdgcn_readfirstlane(base[t.l]), mtl = __builtin_amdgcn_readfirstlane(base[t.l + 1]) - b0;
    const uint32_t i_in = uint32_t(it - b0 * ncb);
    const int nt = int(i_in / uint32_t(mtl)), mt = int(i_in) - nt * mtl;
    t.row0 = int64_t(offs[t.l]) + mt * kThinRows;
    t.rows = min(kThinRows, int(offs[t.l + 1] - t.row0));
    t.c0 = nt * kThinCols;
    return t;
  };

  // ---- fills
  const uint32_t lds0 = __builtin_amdgcn_readfirstlane(lds_addr(smem)) + uint32_t(wave * S * kThinStage);
  const int frow = lane >> 3, fpos = lane & 7;
  int f_it = it0;
  int f_s = s0;
  const char *f_w = nullptr, *f_x = nullptr;
  uint32_t f_wo[8], f_xo[4];
  auto f_place = [&]() {
    const Item t = place(f_it);
    const uint16_t* w = static_cast<const uint16_t*>(g.w) + int64_t(t.l) * g.N * g.K;
    const int cols = min(kThinCols, g.N - t.c0);
    f_w = reinterpret_cast<const char*>(wave_uniform(W_KN ? w + t.c0 + int64_t(s0) * kThinK * g.N : w + int64_t(t.c0) * g.K + s0 * kThinK));
    f_x = reinterpret_cast<const char*>(wave_uniform(static_cast<const uint16_t*>(g.x) + t.row0 * g.ldx + s0 * kThinK));
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int r = 8 * i + frow;                      // a column of W, or a K row
      if constexpr (W_KN) f_wo[i] = (uint32_t(r) * uint32_t(g.N) + uint32_t(min((fpos ^ thin_swz(r)) * 8, cols - 8))) * 2u;
      else f_wo[i] = (uint32_t(min(r, cols - 1)) * uint32_t(g.K) + uint32_t((fpos ^ ((r >> 1) & 7)) * 8)) * 2u;
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int r = 8 * i + frow;
      f_xo[i] = (uint32_t(min(r, t.rows - 1)) * uint32_t(g.ldx) + uint32_t((fpos ^ ((r >> 1) & 7)) * 8)) * 2u;
    }
  };
  auto fill = [&](uint32_t to, const char* p, uint32_t off, int k, int left, bool nt) {
    const lds_void_ptr d = (lds_void_ptr)(uintptr_t)to;
    const char* s = p + off;
    if (left < kThinK) s = k < left ? s : reinterpret_cast<const char*>(&kBigZeros);   // zeros past K, in both operands
    if (nt) __builtin_amdgcn_global_load_lds(static_cast<const void*>(s), d, 16, 0, 2);
    else __builtin_amdgcn_global_load_lds(static_cast<const void*>(s), d, 16, 0, 0);
  };
  auto issue = [&](int slot) {
    const uint32_t to = lds0 + uint32_t(slot * kThinStage);
    const int left = g.K - f_s * kThinK;
    if (left >= kThinK) {
#pragma unroll
      for (int i = 0; i < 8; ++i) fill(to + i * 1024, f_w, f_wo[i], 0, kThinK, SPLIT == 1);
#pragma unroll
      for (int i = 0; i < 4; ++i) fill(to + kThinW + i * 1024, f_x, f_xo[i], 0, kThinK, false);
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const int r = 8 * i + frow;
        fill(to + i * 1024, f_w, f_wo[i], W_KN ? r : (fpos ^ ((r >> 1) & 7)) * 8, left, SPLIT == 1);
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) fill(to + kThinW + i * 1024, f_x, f_xo[i], (fpos ^ (((8 * i + frow) >> 1) & 7)) * 8, left, false);
    }
    f_w += W_KN ? int64_t(g.N) * (kThinK * 2) : int64_t(kThinK * 2);
    f_x += kThinK * 2;
    if (++f_s == s1) {
      f_s = s0;
      f_it += it_step;
      if (f_it < items) f_place();
    }
  };

  // ---- fragment addresses
  uint32_t w_rd, x_rd[2];
  if constexpr (W_KN) {
    const int a = r16 & 3, k = 8 * q + (r16 >> 2);
    w_rd = k * 128 + (((a >> 1) ^ thin_swz(k)) << 4) + (a & 1) * 8;
  } else {
    w_rd = 0;
  }
#pragma unroll
  for (int h = 0; h < 2; ++h) x_rd[h] = r16 * 128 + (((h * 4 + q) ^ ((r16 >> 1) & 7)) << 4);

  int slot = 0, ahead = 0;                             // stages issued and not yet used
  if (s0 < s1 && it0 < items) {
    f_place();
    for (; ahead < S - 1 && f_it < items; ++ahead) issue(ahead);
  }
  for (int it = it0; it < items; it += it_step) {
    const Item t = place(it);
    f32x4 acc[4][2];
#pragma unroll
    for (int n = 0; n < 4; ++n) acc[n][0] = acc[n][1] = f32x4{0, 0, 0, 0};
    for (int s = s0; s < s1; ++s) {
      if (f_it < items) {
        issue(slot + S - 1 >= S ? slot - 1 : slot + S - 1);
        // all but the stages behind this one have landed
        if constexpr (S == 3) __builtin_amdgcn_s_waitcnt(0x4F78);       // vmcnt(24)
        else __builtin_amdgcn_s_waitcnt(0x0F7C);                        // vmcnt(12)
      } else {
        MOE_VMCNT0();
      }
      asm volatile("" ::: "memory");
      const uint32_t st = lds0 + uint32_t(slot * kThinStage);
      bf16x8 fw[2][4], fx[2][2];
#pragma unroll
      for (int h = 0; h < 2; ++h) {
#pragma unroll
        for (int n = 0; n < 4; ++n) {
          if constexpr (W_KN) {
            const uint32_t p = (w_rd ^ (n << 5)) + st + h * 4096;
            const s16x4 lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4_ptr)(uintptr_t)p);
            const s16x4 up = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4_ptr)(uintptr_t)(p + 512));
            fw[h][n] = __builtin_bit_cast(bf16x8, __builtin_shufflevector(lo, up, 0, 1, 2, 3, 4, 5, 6, 7));
          } else {
            fw[h][n] = *(const __attribute__((address_space(3))) bf16x8*)(uintptr_t)(x_rd[h] + st + n * 2048);
          }
        }
#pragma unroll
        for (int r = 0; r < 2; ++r)
          fx[h][r] = *(const __attribute__((address_space(3))) bf16x8*)(uintptr_t)(x_rd[h] + st + kThinW + r * 2048);
      }
      MOE_LGKM0();                                     // read before the next fill of this stage is issued
      asm volatile("" ::: "memory");
      __builtin_amdgcn_sched_barrier(0);
#pragma unroll
      for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int n = 0; n < 4; ++n) acc[n][0] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(fw[h][n], fx[h][0], acc[n][0], 0, 0, 0);
      if (t.rows > 16) {
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
          for (int n = 0; n < 4; ++n) acc[n][1] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(fw[h][n], fx[h][1], acc[n][1], 0, 0, 0);
      }
      slot = slot + 1 == S ? 0 : slot + 1;
    }
    uint16_t* out = static_cast<uint16_t*>(g.y) + t.row0 * g.ldy + t.c0;
    if constexpr (SPLIT == 1) {
#pragma unroll
      for (int r = 0; r < 2; ++r)
#pragma unroll
        for (int n = 0; n < 4; ++n) {
          const int row = r * 16 + r16, col = n * 16 + 4 * q;
          if (row < t.rows && t.c0 + col < g.N)
            *reinterpret_cast<uint2*>(out + row * g.ldy + col) =
                make_uint2(pack_bf16x2(acc[n][r][0], acc[n][r][1]), pack_bf16x2(acc[n][r][2], acc[n][r][3]));
        }
    } else {
      // [wave][row][column], four columns a vector
      f32x4* const sums = reinterpret_cast<f32x4*>(smem + 4 * S * kThinStage);
#pragma unroll
      for (int r = 0; r < 2; ++r)
#pragma unroll
        for (int n = 0; n < 4; ++n) sums[wave * (kThinPart / 16) + (r * 16 + r16) * 16 + ((n * 4 + q) ^ r16)] = acc[n][r];
      __syncthreads();
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int v = threadIdx.x + 256 * i, row = v >> 4, c4 = v & 15;
        if (row < t.rows && t.c0 + c4 * 4 < g.N) {
          f32x4 sum = sums[row * 16 + (c4 ^ (row & 15))];
#pragma unroll
          for (int w = 1; w < 4; ++w) sum += sums[w * (kThinPart / 16) + row * 16 + (c4 ^ (row & 15))];
          *reinterpret_cast<uint2*>(out + row * g.ldy + c4 * 4) =
              make_uint2(pack_bf16x2(sum[0], sum[1]), pack_bf16x2(sum[2], sum[3]));
        }
      }
      __syncthreads();
    }
  }
}

template <bool W_KN>
__global__ __launch_bounds__(256, 1) void grouped_thin_kernel(GroupedArgs g) {
  extern __shared__ __attribute__((aligned(16))) char smem[];
  __shared__ int32_t base[kMaxGroups + 1], part[5];
  bool bad;
  const int mtiles = group_tiles<256>(g.offsets, g.G, g.rows, 5, base, part, &bad);
  if (g.status && blockIdx.x == 0 && threadIdx.x == 0) *g.status = bad ? MOE_EINVAL : MOE_OK;
  const int items = mtiles * ((g.N + kThinCols - 1) / kThinCols);
  if (thin_alone(items, gridDim.x, (g.K + kThinK - 1) / kThinK, W_KN)) thin_run<W_KN, 1>(g, base, mtiles, smem);
  else thin_run<W_KN, 4>(g, base, mtiles, smem);
}

}  // namespace moe
