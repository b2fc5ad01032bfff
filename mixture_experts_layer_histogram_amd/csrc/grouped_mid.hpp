// 128 x 128 tiles of C = A B^T on gfx950, for products of so few 256 x 256 tiles that those would leave CUs idle, or whose groups' rows would
// fill them badly.
//
// 4 waves as 2 x 2, each with 64 x 64 outputs (4 x 4 blocks of v_mfma_f32_16x16x32_bf16).  K goes by steps of 64 through a ring of four stages
// of 32 KiB, filled by direct global->LDS loads two to three steps ahead, one barrier a step.  With one wave a SIMD nothing else covers an LDS
// read, so the fragments of the next half step are read beside the products of this one: 33.4 -> 28.8 us for 2048 x 2048 x 2048 (597 TFLOP/s; 46.8 us
// with the tiles of 256, which leave 192 of 256 CUs idle).  A step takes 0.5 to 0.6 us however few the tiles are, 0.25 of it products: the latency
// of the loads bounds it, and LDS holds no deeper ring.  Twice the bytes a product of the large tiles, so those win wherever they fill the card.
#pragma once

#include <type_traits>

#include "grouped_tile.hpp"

namespace moe {

constexpr int kMid = 128, kMidThreads = 256;
constexpr int kMidPanel = kMid * kBigBK * 2, kMidStage = 2 * kMidPanel, kMidRing = 4;
constexpr int kMidLds = kMidRing * kMidStage;

// This lane's four fills of a panel
template <bool MN>
struct MidFill {
  const char* p;              // the first value of the step (K contiguous), or its first K row; the same in every lane
  int64_t ld;
  uint32_t off[4];            // byte offsets from it
  int kb;                     // K of the first fill within a step

  __device__ __forceinline__ void at(int wave, int lane, const BigOperand& o) {
    p = reinterpret_cast<const char*>(wave_uniform(o.p));
    ld = o.ld;
    if constexpr (!MN) {
      kb = ((lane & 7) ^ (lane >> 4)) * 8;
#pragma unroll
      for (int i = 0; i < 4; ++i)
        off[i] = (uint32_t(min((wave * 4 + i) * 8 + (lane >> 3), o.rows - 1)) * uint32_t(ld) + uint32_t(kb ^ ((i & 1) * 32))) * 2u;
    } else {                  // 256 bytes a K row, four K rows a load
      kb = 16 * wave + (lane >> 4);
#pragma unroll
      for (int i = 0; i < 4; ++i)
        off[i] = (uint32_t(kb + 4 * i) * uint32_t(ld) + uint32_t(min(((lane & 15) ^ big_mn_swz(kb + 4 * i)) * 8, o.rows - 8))) * 2u;
    }
  }
  __device__ __forceinline__ void fill(uint32_t lds, int left) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const lds_void_ptr to = (lds_void_ptr)(uintptr_t)(lds + uint32_t(i * 1024));
      if (left >= kBigBK) {
        __builtin_amdgcn_global_load_lds(static_cast<const void*>(p + off[i]), to, 16, 0, 0);
      } else {                // zeros past K, in both operands
        const int k = MN ? kb + 4 * i : kb ^ ((i & 1) * 32);
        const char* q = k < left ? p + off[i] : reinterpret_cast<const char*>(&kBigZeros);
        __builtin_amdgcn_global_load_lds(static_cast<const void*>(q), to, 16, 0, 0);
      }
    }
    p += MN ? ld * (kBigBK * 2) : int64_t(kBigBK * 2);
  }
};

template <bool A_MN, bool B_MN, typename TILES>
struct MidWalk {
  static constexpr int kBlocks = 4;
  int lane, wave, row_base, col_base;
  f32x4 acc[4][4];            // lane: row row_base + m * 16 + lane % 16, columns col_base + n * 16 + 4 (lane / 16) + 0..3

  __device__ __forceinline__ void run(const TILES& tiles, char* smem) {
    lane = threadIdx.x & 63;
    wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int wm = wave >> 1, wn = wave & 1, r16 = lane & 15, g = lane >> 4;
    row_base = wm * 64;
    col_base = wn * 64;
    const uint32_t l0 = __builtin_amdgcn_readfirstlane(lds_addr(smem)), mine = l0 + wave * 4096;
    const int a = r16 & 3, kr = 8 * g + (r16 >> 2);
    uint32_t a_rd[2], b_rd[2];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const uint32_t sw = ((h * 4 + g) ^ ((r16 >> 1) & 7)) << 4;
      a_rd[h] = A_MN ? kr * 256 + (((wm * 8 + (a >> 1)) ^ big_mn_swz(kr)) << 4) + (a & 1) * 8 : (wm * 64 + r16) * 128 + sw;
      b_rd[h] = B_MN ? kr * 256 + (((wn * 8 + (a >> 1)) ^ big_mn_swz(kr)) << 4) + (a & 1) * 8 : (wn * 64 + r16) * 128 + sw;
    }
    auto read_tr = [](uint32_t p) {
      const s16x4 lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4_ptr)(uintptr_t)p);
      const s16x4 up = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4_ptr)(uintptr_t)(p + 1024));
      return __builtin_bit_cast(bf16x8, __builtin_shufflevector(lo, up, 0, 1, 2, 3, 4, 5, 6, 7));
    };
    MidFill<A_MN> fa;
    MidFill<B_MN> fb;
    for (int i = 0; i < tiles.count(); ++i) {
      const int K = tiles.K(i), nk = (K + kBigBK - 1) / kBigBK;
      fa.at(wave, lane, tiles.a(i));
      fb.at(wave, lane, tiles.b(i));
      auto issue = [&](int ks) {
        const uint32_t to = mine + uint32_t((ks & 3) * kMidStage);
        fa.fill(to, K - ks * kBigBK);
        fb.fill(to + kMidPanel, K - ks * kBigBK);
      };
      for (int ks = 0; ks < 3 && ks < nk; ++ks) issue(ks);
#pragma unroll
      for (int m = 0; m < 4; ++m)
#pragma unroll
        for (int n = 0; n < 4; ++n) acc[m][n] = f32x4{0, 0, 0, 0};
      const bool idle = row_base >= tiles.rows(i) || col_base >= tiles.cols(i);      // none of the tile's outputs are this wave's
      bf16x8 va[2][4], vb[2][4];
      auto read = [&](int ks, auto hc) {
        constexpr int h = decltype(hc)::value;
        const uint32_t st = l0 + uint32_t((ks & 3) * kMidStage);
#pragma unroll
        for (int m = 0; m < 4; ++m) {
          if constexpr (A_MN) va[h][m] = read_tr((a_rd[0] ^ (m << 5)) + st + h * 8192);
          else va[h][m] = *(const __attribute__((address_space(3))) bf16x8*)(uintptr_t)(a_rd[h] + st + m * 2048);
        }
#pragma unroll
        for (int n = 0; n < 4; ++n) {
          if constexpr (B_MN) vb[h][n] = read_tr((b_rd[0] ^ (n << 5)) + st + kMidPanel + h * 8192);
          else vb[h][n] = *(const __attribute__((address_space(3))) bf16x8*)(uintptr_t)(b_rd[h] + st + kMidPanel + n * 2048);
        }
      };
      auto turn = [&](auto hc) {
        constexpr int h = decltype(hc)::value;
#pragma unroll
        for (int m = 0; m < 4; ++m)
#pragma unroll
          for (int n = 0; n < 4; ++n) acc[m][n] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(vb[h][n], va[h][m], acc[m][n], 0, 0, 0);
      };
      const std::integral_constant<int, 0> h0;
      const std::integral_constant<int, 1> h1;
      // the step's first half is in registers when it begins, and the second's reads and the next step's first half go beside the products
      for (int ks = -1; ks < nk; ++ks) {
        // this wave's fills of the next step have landed: all but those of the one behind it
        if (ks + 2 < nk) __builtin_amdgcn_s_waitcnt(0x0F78);             // vmcnt(8)
        else MOE_VMCNT0();
        MOE_LGKM0();                                                     // done with the step before
        asm volatile("" ::: "memory");
        __builtin_amdgcn_s_barrier();
        asm volatile("" ::: "memory");
        if (ks + 3 < nk && ks >= 0) issue(ks + 3);
        if (ks >= 0 && !idle) {
          read(ks, h1);
          __builtin_amdgcn_sched_barrier(0);
          turn(h0);
        }
        if (!idle && ks + 1 < nk) read(ks + 1, h0);
        __builtin_amdgcn_sched_barrier(0);
        if (ks >= 0 && !idle) turn(h1);
      }
      __builtin_amdgcn_s_barrier();                                      // the next tile's first fills overwrite the stages
      asm volatile("" ::: "memory");
      if (!idle) tiles.store(i, *this);
    }
  }
};

}  // namespace moe
