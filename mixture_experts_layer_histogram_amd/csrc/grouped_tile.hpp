// 256 x 256 tiles of C = A B^T on gfx950 (v_mfma_f32_16x16x32_bf16), A and B each stored with K contiguous or with the row
// index contiguous; one workgroup a CU walks a list of tiles without ever letting its loads run dry.
//
// 8 waves as 2 (rows) x 4 (columns), each with 128 x 64 outputs: 8 x 4 blocks of 16 x 16 in 128 accumulators.  K goes by
// steps of 64.  The waves of the upper and of the lower half of the tile share SIMDs in pairs (w and w + 4) and take
// turns, half a step (32 of K) at a time: while one reads its fragments from LDS, the other has the matrix unit, and a
// barrier ends every turn (turns are about 512 cycles: 32 MFMAs of 16).
//
//   turn        4k          4k + 1      4k + 2      4k + 3      4k + 4
//   half 0   reads k.0     MFMA k.0    reads k.1   MFMA k.1    reads (k+1).0
//   half 1   MFMA (k-1).1  reads k.0   MFMA k.0    reads k.1   MFMA k.1
//
// A step's operands are two panels of 32 KiB, and a CU's 160 KiB of LDS hold five: a ring A0 B0 A1 B1 A2 | B2 ...,
// filled by direct global->LDS loads, two of them a wave and turn.  In step k the places of A and B of step k - 1 take B of
// step k + 1 (in the first two turns; it has the other two to land) and A of step k + 2 (in the last two).  What this
// is about: a CU takes in one 1 KiB load in 16 to 23 cycles, 64 of them a step of 2048, and a wave that finds
// the queue full waits at its issue, MFMAs and all.  8192^3 (rows and columns of K contiguous): two stages of 64 KiB with eight
// loads at once at a step's start 971 us, spread over three turns 869, the ring of five with two a turn 764 (1440 TFLOP/s; a
// library's product of that size 670 to 687).
//
// The loads know nothing of tiles: a cursor for A (two steps ahead) and one for B (one step) walk the list by
// themselves, so the next tile's first panels land while this one's last products and its stores are on their way.
// 32 groups of 7168 x 2048 (bf16): 32749 rows from 2048 values to 7168 845 us (1.1 PFLOP/s; one group of 32768 rows 699: the tiles at the
// groups' ends), 16381 rows back to 7168 values 497, their weight gradients 551 (8 steps a tile and 128 KiB stored); some 3 % more on other cards.  Not faster: workgroups set
// off by parts of a tile, other places for the short tiles, bands over the longer axis in the products.
#pragma once

#include "gemm_tile.hpp"

namespace moe {

typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef short s16x8 __attribute__((ext_vector_type(8)));
typedef __attribute__((address_space(3))) s16x4* lds_s16x4_ptr;

constexpr int kBig = 256, kBigBK = 64;
constexpr int kBigPanel = kBig * kBigBK * 2;          // bytes of one operand's step
constexpr int kBigLds = 5 * kBigPanel;                // all of a CU's LDS
constexpr int kBigThreads = 512;
constexpr int kBigBand = 8;                           // row tiles whose column tiles are walked together

// K contiguous: element (r, k) at p + r * ld + k.  Otherwise at p + k * ld + r.  rows: valid ones of the tile (of the row index
// contiguous: a multiple of 8).
struct BigOperand {
  const uint16_t* p;
  int64_t ld;
  int rows;
};

// Tile i of mt x nt: bands of at most kBigBand row tiles (even ones), in a band by column tile, row tiles innermost.  The 32 CUs
// of an XCD then work on about 8 row and 4 column panels at a time, which its L2 gives 64 times (hit rate 81 %; row tiles
// innermost over all of 8192 rows 50 %).
__device__ __forceinline__ void big_place(int64_t i, int mt, int nt, int* m, int* n) {
  const int bands = (mt + kBigBand - 1) / kBigBand, per = (mt + bands - 1) / bands;
  const int band = int(i / (int64_t(per) * nt));
  const int in = int(i - int64_t(band) * per * nt), high = min(per, mt - band * per);
  *n = in / high;
  *m = band * per + in - *n * high;
}

// The LDS place of 16-byte chunk c of K row k where the row index is contiguous (512 bytes a K row) is c ^ this: the eight K rows
// that half a wave reads at once lie in eight different 32-byte slots of the 64 banks.
__device__ __forceinline__ int big_mn_swz(int k) { return 2 * ((k & 3) | (((k >> 3) & 1) << 2)); }

#define MOE_VMCNT0() __builtin_amdgcn_s_waitcnt(0x0F70)          // vmcnt(0), the other counters at their largest
#define MOE_VMCNT4() __builtin_amdgcn_s_waitcnt(0x0F74)
#define MOE_LGKM0() __builtin_amdgcn_s_waitcnt(0xC07F)           // lgkmcnt(0)

// What a tile's last step reads past K: sixteen zero bytes, again and again.
__device__ const u32x4 kBigZeros = {0, 0, 0, 0};

// This lane's four fills of a panel
template <bool MN>
struct BigFill {
  const char* p;              // the first value of the cursor's step (K contiguous), or its first K row; the same in every lane
  int64_t ld;
  uint32_t off[4];            // byte offsets from it
  int kb;                     // K of the first fill within a step
  int tile, left;             // the cursor's tile, and K from its step on

  __device__ __forceinline__ void at(int wave, int lane, const BigOperand& o, int K) {
    p = reinterpret_cast<const char*>(wave_uniform(o.p));
    ld = o.ld;
    left = K;
    if constexpr (!MN) {
      kb = ((lane & 7) ^ (lane >> 4)) * 8;
#pragma unroll
      for (int i = 0; i < 4; ++i)
        off[i] = (uint32_t(min((wave * 4 + i) * 8 + (lane >> 3), o.rows - 1)) * uint32_t(ld) + uint32_t(kb ^ ((i & 1) * 32))) * 2u;
    } else {
      kb = 8 * wave + (lane >> 5);
#pragma unroll
      for (int i = 0; i < 4; ++i)
        off[i] = (uint32_t(kb + 2 * i) * uint32_t(ld) + uint32_t(min(((lane & 31) ^ big_mn_swz(kb + 2 * i)) * 8, o.rows - 8))) * 2u;
    }
  }
  template <int I, bool CUT>
  __device__ __forceinline__ void fill(uint32_t lds) const {
    const lds_void_ptr to = (lds_void_ptr)(uintptr_t)(lds + uint32_t(I * 1024));
    if (!CUT || left >= kBigBK) {
      __builtin_amdgcn_global_load_lds(static_cast<const void*>(p + off[I]), to, 16, 0, 0);
    } else {                  // zeros past K, in both operands: what lies there could be a NaN
      const int k = MN ? kb + 2 * I : kb ^ ((I & 1) * 32);
      const char* q = k < left ? p + off[I] : reinterpret_cast<const char*>(&kBigZeros);
      __builtin_amdgcn_global_load_lds(static_cast<const void*>(q), to, 16, 0, 0);
    }
  }
  __device__ __forceinline__ void step() {
    p += MN ? ld * (kBigBK * 2) : int64_t(kBigBK * 2);
    left -= kBigBK;
  }
};

// TILES: int count(); K of tile i; its operands a(i) and b(i); rows(i), cols(i) of its output; store(i, walk);
// kCut: 0 where every K is a multiple of 64; 1: the check at every fill; 2: at every step (few steps, and the code is there twice).
template <bool A_MN, bool B_MN, typename TILES>
struct BigWalk {
  static constexpr int kBlocks = 8;
  TILES& tiles;
  int lane, wave, half, wn, r16, g, n_tiles, row_base, col_base;
  uint32_t lds_fill;                        // LDS address of this wave's first fill of a panel
  uint32_t l0, a_rd[A_MN ? 1 : 2], b_rd[B_MN ? 1 : 2];
  uint32_t pa;                              // the ring's place of A of the step at work
  BigFill<A_MN> fa_;
  BigFill<B_MN> fb_;
  bf16x8 fa[8], fb[4];
  f32x4 acc[8][4];                          // lane: row half * 128 + m * 16 + r16, columns wn * 64 + n * 16 + 4 g + 0..3

  __device__ __forceinline__ BigWalk(TILES& t, char* smem) : tiles(t) {
    lane = threadIdx.x & 63;
    wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    half = wave >> 2;
    wn = wave & 3;
    row_base = half * 128;
    col_base = wn * 64;
    r16 = lane & 15;
    g = lane >> 4;
    l0 = __builtin_amdgcn_readfirstlane(lds_addr(smem));
    lds_fill = l0 + wave * 4096;
    pa = 0;
    // transposing reads: lane 4 c + a of 16 addresses K row c, columns 4 a .. 4 a + 3, and gets four K values of column 4 c + a
    const int a = r16 & 3, k = 8 * g + (r16 >> 2);
    if constexpr (!A_MN) {
#pragma unroll
      for (int h = 0; h < 2; ++h) a_rd[h] = l0 + (half * 128 + r16) * 128 + (((h * 4 + g) ^ ((r16 >> 1) & 7)) << 4);
    } else {
      a_rd[0] = k * 512 + half * 256 + (((a >> 1) ^ big_mn_swz(k)) << 4) + (a & 1) * 8;
    }
    if constexpr (!B_MN) {
#pragma unroll
      for (int h = 0; h < 2; ++h) b_rd[h] = l0 + (wn * 64 + r16) * 128 + (((h * 4 + g) ^ ((r16 >> 1) & 7)) << 4);
    } else {
      b_rd[0] = k * 512 + (wn >> 1) * 256 + (((wn & 1) * 8 + (a >> 1)) ^ big_mn_swz(k)) * 16 + (a & 1) * 8;
    }
  }

  // ---- the cursors
  __device__ __forceinline__ bool on_a() const { return fa_.tile < n_tiles; }
  __device__ __forceinline__ bool on_b() const { return fb_.tile < n_tiles; }
  template <bool A, int I, bool CUT>
  __device__ __forceinline__ void fill(uint32_t place) {
    if constexpr (A) fa_.template fill<I, CUT>(lds_fill + place);
    else fb_.template fill<I, CUT>(lds_fill + place);
    if constexpr (I == 3) {
      if constexpr (A) {
        fa_.step();
        if (fa_.left <= 0 && ++fa_.tile < n_tiles) fa_.at(wave, lane, tiles.a(fa_.tile), tiles.K(fa_.tile));
      } else {
        fb_.step();
        if (fb_.left <= 0 && ++fb_.tile < n_tiles) fb_.at(wave, lane, tiles.b(fb_.tile), tiles.K(fb_.tile));
      }
    }
  }
  template <bool A, int I, bool CUT>
  __device__ __forceinline__ void fill2(uint32_t place) {
    fill<A, I, CUT>(place);
    fill<A, I + 1, CUT>(place);
  }

  // ---- half a step's fragments from LDS, all landed at the end
  template <int MV>
  __device__ __forceinline__ void read(uint32_t pb, int h) {
    if constexpr (MV > 0) {
      uint32_t ar = a_rd[0], br = b_rd[0];
      if constexpr (A_MN) asm volatile("" : "+v"(ar));      // the blocks' addresses are not kept in registers of their own
      if constexpr (B_MN) asm volatile("" : "+v"(br));
#pragma unroll
      for (int m = 0; m < MV; ++m) {
        if constexpr (A_MN) fa[m] = read_tr((ar ^ (m << 5)) + (l0 + pa) + h * 16384);       // block m: 32 bytes on, swizzled
        else fa[m] = *(const __attribute__((address_space(3))) bf16x8*)(uintptr_t)(a_rd[h] + pa + m * 2048);
      }
#pragma unroll
      for (int n = 0; n < 4; ++n) {
        if constexpr (B_MN) fb[n] = read_tr((br ^ (n << 5)) + (l0 + pb) + h * 16384);
        else fb[n] = *(const __attribute__((address_space(3))) bf16x8*)(uintptr_t)(b_rd[h] + pb + n * 2048);
      }
    }
    __builtin_amdgcn_sched_barrier(0);
  }
  __device__ static __forceinline__ bf16x8 read_tr(uint32_t p) {
    const s16x4 lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4_ptr)(uintptr_t)p);
    const s16x4 up = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4_ptr)(uintptr_t)(p + 2048));
    return __builtin_bit_cast(bf16x8, __builtin_shufflevector(lo, up, 0, 1, 2, 3, 4, 5, 6, 7));
  }

  // ---- half a step's products, with two fills between them.  The weights' (columns') fragment comes first, so that a lane ends up
  // with four consecutive columns of one row.
  template <int MV, bool A, int I, bool CUT>
  __device__ __forceinline__ void mfma(uint32_t place, bool on) {
    __builtin_amdgcn_s_setprio(1);
#pragma unroll
    for (int m = 0; m < MV; ++m) {
#pragma unroll
      for (int n = 0; n < 4; ++n) acc[m][n] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(fb[n], fa[m], acc[m][n], 0, 0, 0);
      if (m == 0 || m == 3) {
        __builtin_amdgcn_sched_barrier(0);
        if (on) {
          if (m == 0) fill<A, I, CUT>(place);
          else fill<A, I + 1, CUT>(place);
        }
        __builtin_amdgcn_sched_barrier(0);
      }
    }
    if (MV == 0 && on) fill2<A, I, CUT>(place);
    __builtin_amdgcn_s_setprio(0);
  }
  __device__ static __forceinline__ void turn() {
    asm volatile("" ::: "memory");                    // no access to LDS moves over the barrier
    __builtin_amdgcn_sched_barrier(0);
    __builtin_amdgcn_s_barrier();
    __builtin_amdgcn_sched_barrier(0);
    asm volatile("" ::: "memory");
  }
  static __device__ __forceinline__ uint32_t next(uint32_t p, int by) {       // `by` places on in the ring
    p += uint32_t(by * kBigPanel);
    return p >= uint32_t(kBigLds) ? p - uint32_t(kBigLds) : p;
  }

  // ---- one step of a tile, and a tile.  CUT: some fill of the step may be of a tile's last, cut step (a branch at each fill: it costs
  // 8192^3 a tenth).
  template <int MV, int HALF, bool CUT>
  __device__ __forceinline__ void step() {
    const uint32_t pb = next(pa, 1), pb1 = next(pa, 3), pa2 = next(pa, 4);
    read<MV>(pb, 0);
    const bool b = on_b();
    if (b) fill2<false, HALF == 0 ? 0 : 2, CUT>(pb1);
    MOE_LGKM0();
    turn();
    const bool a = on_a();
    if constexpr (HALF == 0) mfma<MV, false, 2, CUT>(pb1, b);
    else mfma<MV, true, 0, CUT>(pa2, a);
    turn();
    read<MV>(pb, 1);
    if (a) fill2<true, HALF == 0 ? 0 : 2, CUT>(pa2);
    MOE_LGKM0();
    if constexpr (HALF == 1) {                       // B of the next step has landed: all but this step's four fills of A
      if (a) MOE_VMCNT4();
      else MOE_VMCNT0();
    }
    turn();
    if constexpr (HALF == 0) {
      mfma<MV, true, 2, CUT>(pa2, a);
      if (a) MOE_VMCNT4();
      else MOE_VMCNT0();
    } else {
      mfma<MV, false, 0, CUT>(pa, on_b());         // B of the step after next comes where A of this one lay
    }
    turn();
    pa = next(pa, 2);
  }
  template <int MV, int HALF>
  __device__ __forceinline__ void steps(int K) {
    for (int left = K; left > 0; left -= kBigBK) {
      // a step without cut fills needs two whole steps ahead of both cursors
      if (TILES::kCut == 0 || (TILES::kCut == 2 && min(fa_.left, fb_.left) >= 2 * kBigBK)) step<MV, HALF, false>();
      else step<MV, HALF, true>();
    }
  }
  template <int HALF>
  __device__ __forceinline__ void tile(int i) {
#pragma unroll
    for (int m = 0; m < 8; ++m)
#pragma unroll
      for (int n = 0; n < 4; ++n) acc[m][n] = f32x4{0, 0, 0, 0};
    // 16-row blocks of this wave that hold any of the tile's rows (and columns): the others' products are left out
    const int mv = wn * 64 >= tiles.cols(i) ? 0 : (tiles.rows(i) - HALF * 128 + 15) >> 4;
    const int K = tiles.K(i);
    if (mv > 4) steps<8, HALF>(K);
    else if (mv > 0) steps<4, HALF>(K);
    else steps<0, HALF>(K);
    if (mv > 0) tiles.store(i, *this);
  }

  // The whole list, every tile with K > 0.  LDS is free before and after.
  __device__ __forceinline__ void run() {
    n_tiles = tiles.count();
    if (n_tiles == 0) return;
    fa_.tile = fb_.tile = 0;
    fa_.at(wave, lane, tiles.a(0), tiles.K(0));
    fb_.at(wave, lane, tiles.b(0), tiles.K(0));
    fill2<true, 0, true>(pa);
    fill2<true, 2, true>(pa);
    fill2<false, 0, true>(next(pa, 1));
    fill2<false, 2, true>(next(pa, 1));
    if (on_a()) {
      fill2<true, 0, true>(next(pa, 2));
      fill2<true, 2, true>(next(pa, 2));
      MOE_VMCNT4();
    } else {
      MOE_VMCNT0();
    }
    turn();
    if (half == 0) {
      for (int i = 0; i < n_tiles; ++i) tile<0>(i);
      turn();
    } else {
      if (on_b()) fill2<false, 0, true>(next(pa, 3));
      turn();
      for (int i = 0; i < n_tiles; ++i) tile<1>(i);
    }
  }
};

// Output rows of a tile from the accumulators, in 16-byte vectors.  bf16: two 16-column blocks exchange halves between lane groups, so
// that a lane has eight consecutive columns, and lanes 8 apart exchange vectors, so that a store covers 128 bytes of each of eight
// rows.  fp32: added to what is there with ADD.  NT: past the caches.
template <bool NT>
__device__ __forceinline__ void big_put(void* p, const u32x4 v) {
  if constexpr (NT) __builtin_nontemporal_store(v, static_cast<u32x4*>(p));
  else *static_cast<u32x4*>(p) = v;
}

template <typename O, bool ADD, bool NT, typename WALK>
__device__ __forceinline__ void big_store(const WALK& w, O* out, int64_t ld, int rows, int cols) {
  int lane = w.lane;
  asm volatile("" : "+v"(lane));            // the compiler would keep these indices in registers all along the products
  const int r16 = lane & 15, g = lane >> 4;
#pragma unroll
  for (int m = 0; m < WALK::kBlocks; ++m) {
    const int row = w.row_base + m * 16 + r16;
    if (sizeof(O) == 4 && row >= rows) continue;
    O* p = out + row * ld;
    if constexpr (sizeof(O) == 2) {
      u32x4 v[2];
#pragma unroll
      for (int n = 0; n < 2; ++n)
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          const auto s = __builtin_amdgcn_permlane16_swap(pack_bf16x2(w.acc[m][2 * n][2 * j], w.acc[m][2 * n][2 * j + 1]),
                                                          pack_bf16x2(w.acc[m][2 * n + 1][2 * j], w.acc[m][2 * n + 1][2 * j + 1]), false, false);
          v[n][j] = s[0];
          v[n][2 + j] = s[1];
        }
      // lanes r16 and r16 ^ 8 exchange: then a lane's first vector is of row r16 & 7 and its second of row (r16 & 7) + 8
      const bool up = r16 >= 8;
      u32x4 a, b;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const uint32_t send = up ? v[0][j] : v[1][j];
        const uint32_t got = uint32_t(__builtin_amdgcn_update_dpp(int(send), int(send), 0x128, 0xF, 0xF, false));
        a[j] = up ? got : v[0][j];
        b[j] = up ? v[1][j] : got;
      }
      const int col = w.col_base + (up ? 32 : 0) + (g & 1) * 16 + (g >> 1) * 8;
      const int ra = w.row_base + m * 16 + (r16 & 7);
      O* q = out + ra * ld + col;
      if (col < cols && ra < rows) big_put<NT>(q, a);
      if (col < cols && ra + 8 < rows) big_put<NT>(q + 8 * ld, b);
    } else {
#pragma unroll
      for (int n = 0; n < 4; ++n) {
        const int col = w.col_base + n * 16 + 4 * g;
        if (col >= cols) continue;
        f32x4 v = w.acc[m][n];
        if constexpr (ADD) v += *reinterpret_cast<const f32x4*>(p + col);
        big_put<NT>(p + col, __builtin_bit_cast(u32x4, v));
      }
    }
  }
}

}  // namespace moe
