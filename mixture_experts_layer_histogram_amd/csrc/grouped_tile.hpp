// One 256 x 256 tile of C = A B^T on gfx950 (v_mfma_f32_16x16x32_bf16), A and B each stored with K contiguous or with the
// row index contiguous.
//
// 8 waves as 2 (rows) x 4 (columns), each with 128 x 64 outputs: 8 x 4 blocks of 16 x 16 in 128 accumulators.  K goes by
// steps of 64 through two LDS stages of 64 KiB, filled by direct global->LDS loads.  The waves of the upper and of the
// lower half of the tile share SIMDs in pairs (w and w + 4) and take turns, half a step (32 of K) at a time: while one
// reads its fragments from LDS, the other has the matrix unit, and a barrier ends every turn.  So neither waits for its own
// reads, and a fill has four turns (about 2000 cycles) to land.
//
//   turn        4k          4k + 1      4k + 2      4k + 3      4k + 4
//   half 0   reads k.0     MFMA k.0    reads k.1   MFMA k.1    reads (k+1).0
//   half 1   MFMA (k-1).1  reads k.0   MFMA k.0    reads k.1   MFMA k.1
//
// Both halves fill stage k + 1 in turn 4k (its last readers were half 1 in turn 4k - 1), and both wait for their fills before
// the barrier that ends turn 4k + 3.
#pragma once

#include "gemm_tile.hpp"

namespace moe {

typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef short s16x8 __attribute__((ext_vector_type(8)));
typedef __attribute__((address_space(3))) s16x4* lds_s16x4_ptr;

constexpr int kBig = 256, kBigBK = 64;
constexpr int kBigPanel = kBig * kBigBK * 2;          // bytes of one operand's stage
constexpr int kBigStage = 2 * kBigPanel;
constexpr int kBigLds = 2 * kBigStage;
constexpr int kBigThreads = 512;

// K contiguous: element (r, k) at p + r * ld + k.  Otherwise at p + k * ld + r.  rows: valid ones of the tile (of the row index
// contiguous: a multiple of 8).
struct BigOperand {
  const uint16_t* p;
  int64_t ld;
  int rows;
};

// The LDS place of 16-byte chunk c of K row k where the row index is contiguous (512 bytes a K row): the eight K rows that half a
// wave reads at once lie in eight different 32-byte slots of the 64 banks.
__device__ __forceinline__ int big_mn_swz(int k) { return 2 * ((k & 3) | (((k >> 3) & 1) << 2)); }

#define MOE_VMCNT0() __builtin_amdgcn_s_waitcnt(0x0F70)          // vmcnt(0), the others at their largest
#define MOE_LGKM0() __builtin_amdgcn_s_waitcnt(0xC07F)           // lgkmcnt(0)

template <bool A_MN, bool B_MN>
struct BigTile {
  // lane and wave
  int lane, wave, half, wn, r16, g;
  uint32_t a_off[4], b_off[4];              // byte offsets of this lane's fills
  int a_k[4], b_k[4];                       // K of them within a step
  uint32_t lds_fill;                        // LDS address of this wave's first fill
  uint32_t a_rd[A_MN ? 8 : 2], b_rd[B_MN ? 4 : 2];
  const char* abase;
  const char* bbase;
  int64_t lda, ldb;
  int K;
  bf16x8 fa[8], fb[4];
  f32x4 acc[8][4];

  template <bool MN>
  __device__ __forceinline__ void fill_offsets(const BigOperand& o, uint32_t* off, int* kk) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if constexpr (!MN) {
        const int row = (wave * 4 + i) * 8 + (lane >> 3);
        const int ch = (lane & 7) ^ ((row >> 1) & 7);
        kk[i] = ch * 8;
        off[i] = (uint32_t(min(row, o.rows - 1)) * uint32_t(o.ld) + uint32_t(ch * 8)) * 2u;
      } else {
        const int k = 8 * wave + 2 * i + (lane >> 5);
        const int ch = (lane & 31) ^ big_mn_swz(k);
        kk[i] = k;
        off[i] = uint32_t(min(ch * 8, o.rows - 8)) * 2u;
      }
    }
  }

  __device__ __forceinline__ void start(char* smem, const BigOperand& A, const BigOperand& B, int K_) {
    lane = threadIdx.x & 63;
    wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    half = wave >> 2;
    wn = wave & 3;
    r16 = lane & 15;
    g = lane >> 4;
    K = K_;
    lda = A.ld;
    ldb = B.ld;
    abase = reinterpret_cast<const char*>(wave_uniform(A.p));
    bbase = reinterpret_cast<const char*>(wave_uniform(B.p));
    fill_offsets<A_MN>(A, a_off, a_k);
    fill_offsets<B_MN>(B, b_off, b_k);
    lds_fill = __builtin_amdgcn_readfirstlane(lds_addr(smem + wave * 4 * 1024));
    const uint32_t l0 = lds_addr(smem);
    if constexpr (!A_MN) {
#pragma unroll
      for (int h = 0; h < 2; ++h) a_rd[h] = l0 + (half * 128 + r16) * 128 + (((h * 4 + g) ^ ((r16 >> 1) & 7)) << 4);
    } else {
      const int a = r16 & 3, c = r16 >> 2, k = 8 * g + c;
      const uint32_t b0 = k * 512 + half * 256 + (((a >> 1) ^ big_mn_swz(k)) << 4) + (a & 1) * 8;
#pragma unroll
      for (int m = 0; m < 8; ++m) a_rd[m] = l0 + (b0 ^ (m << 5));
    }
    if constexpr (!B_MN) {
#pragma unroll
      for (int h = 0; h < 2; ++h)
        b_rd[h] = l0 + kBigPanel + (wn * 64 + r16) * 128 + (((h * 4 + g) ^ ((r16 >> 1) & 7)) << 4);
    } else {
      const int a = r16 & 3, c = r16 >> 2, k = 8 * g + c;
      const uint32_t b0 = kBigPanel + k * 512 + (wn >> 1) * 256 + ((((wn & 1) * 8 + (a >> 1)) ^ big_mn_swz(k)) << 4) + (a & 1) * 8;
#pragma unroll
      for (int n = 0; n < 4; ++n) b_rd[n] = l0 + (b0 ^ (n << 5));
    }
  }

  // fills of step ks
  __device__ __forceinline__ void issue(int ks) {
    const uint32_t da = lds_fill + uint32_t((ks & 1) * kBigStage), db = da + uint32_t(kBigPanel);
    const int k0 = ks * kBigBK;
    const bool tail = k0 + kBigBK > K;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      fill_one<A_MN>(abase, lda, a_off[i], a_k[i], k0, tail, da + uint32_t(i * 1024));
      fill_one<B_MN>(bbase, ldb, b_off[i], b_k[i], k0, tail, db + uint32_t(i * 1024));
    }
  }
  template <bool MN>
  __device__ __forceinline__ void fill_one(const char* base, int64_t ld, uint32_t off, int kk, int k0, bool tail, uint32_t lds) {
    const lds_void_ptr to = (lds_void_ptr)(uintptr_t)lds;
    if constexpr (!MN) {
      uint32_t o = off;
      if (tail) o -= 2u * uint32_t(max(0, k0 + kk - (K - 8)));          // past K: the row's last values again, masked later
      __builtin_amdgcn_global_load_lds(static_cast<const void*>(base + int64_t(k0) * 2 + o), to, 16, 0, 0);
    } else {
      const int k = tail ? min(kk, K - 1 - k0) : kk;
      __builtin_amdgcn_global_load_lds(static_cast<const void*>(base + int64_t(k0) * ld * 2 + (uint32_t(k) * uint32_t(ld) * 2u + off)),
                                       to, 16, 0, 0);
    }
  }

  // fragments of half a step (32 of K) from LDS, all landed at the end
  template <int MV>
  __device__ __forceinline__ void read(int ks, int h, int klim) {
    const uint32_t st = uint32_t((ks & 1) * kBigStage);
    if constexpr (!A_MN) {
      const uint32_t p = a_rd[h] + st;
      if constexpr (MV > 4)
        asm volatile("ds_read_b128 %0, %8\n\tds_read_b128 %1, %8 offset:2048\n\tds_read_b128 %2, %8 offset:4096\n\t"
                     "ds_read_b128 %3, %8 offset:6144\n\tds_read_b128 %4, %8 offset:8192\n\tds_read_b128 %5, %8 offset:10240\n\t"
                     "ds_read_b128 %6, %8 offset:12288\n\tds_read_b128 %7, %8 offset:14336\n\ts_waitcnt lgkmcnt(0)"
                     : "=&v"(fa[0]), "=&v"(fa[1]), "=&v"(fa[2]), "=&v"(fa[3]), "=&v"(fa[4]), "=&v"(fa[5]), "=&v"(fa[6]), "=&v"(fa[7])
                     : "v"(p) : "memory");
      else if constexpr (MV > 0)
        asm volatile("ds_read_b128 %0, %4\n\tds_read_b128 %1, %4 offset:2048\n\tds_read_b128 %2, %4 offset:4096\n\t"
                     "ds_read_b128 %3, %4 offset:6144\n\ts_waitcnt lgkmcnt(0)"
                     : "=&v"(fa[0]), "=&v"(fa[1]), "=&v"(fa[2]), "=&v"(fa[3]) : "v"(p) : "memory");
    } else if constexpr (MV > 0) {
#pragma unroll
      for (int m = 0; m < MV; ++m) fa[m] = read_tr(a_rd[m] + st + h * 16384);
    }
    if constexpr (MV > 0) {
      if constexpr (!B_MN) {
        const uint32_t p = b_rd[h] + st;
        asm volatile("ds_read_b128 %0, %4\n\tds_read_b128 %1, %4 offset:2048\n\tds_read_b128 %2, %4 offset:4096\n\t"
                     "ds_read_b128 %3, %4 offset:6144\n\ts_waitcnt lgkmcnt(0)"
                     : "=&v"(fb[0]), "=&v"(fb[1]), "=&v"(fb[2]), "=&v"(fb[3]) : "v"(p) : "memory");
      } else {
#pragma unroll
        for (int n = 0; n < 4; ++n) fb[n] = read_tr(b_rd[n] + st + h * 16384);
      }
      if (klim < h * 32 + 32) {                       // the last step: zeros past K, in both (a NaN there must not count)
#pragma unroll
        for (int m = 0; m < MV; ++m) fa[m] = mask(fa[m], klim - h * 32 - 8 * g);
#pragma unroll
        for (int n = 0; n < 4; ++n) fb[n] = mask(fb[n], klim - h * 32 - 8 * g);
      }
    }
  }
  __device__ static __forceinline__ bf16x8 read_tr(uint32_t p) {
    const s16x4 lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4_ptr)(uintptr_t)p);
    const s16x4 up = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4_ptr)(uintptr_t)(p + 2048));
    return __builtin_bit_cast(bf16x8, __builtin_shufflevector(lo, up, 0, 1, 2, 3, 4, 5, 6, 7));
  }
  __device__ static __forceinline__ bf16x8 mask(bf16x8 f, int n) {     // the first n values
    s16x8 v = __builtin_bit_cast(s16x8, f);
#pragma unroll
    for (int e = 0; e < 8; ++e)
      if (e >= n) v[e] = 0;
    return __builtin_bit_cast(bf16x8, v);
  }

  template <int MV>
  __device__ __forceinline__ void mfma() {
    __builtin_amdgcn_s_setprio(1);
#pragma unroll
    for (int m = 0; m < MV; ++m)
#pragma unroll
      for (int n = 0; n < 4; ++n) acc[m][n] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(fb[n], fa[m], acc[m][n], 0, 0, 0);
    __builtin_amdgcn_s_setprio(0);
  }
  __device__ static __forceinline__ void turn() {
    asm volatile("" ::: "memory");                    // no access to LDS moves over the barrier
    __builtin_amdgcn_sched_barrier(0);
    __builtin_amdgcn_s_barrier();
    __builtin_amdgcn_sched_barrier(0);
    asm volatile("" ::: "memory");
  }

  template <int MV>
  __device__ __forceinline__ void loop(int nk) {
    for (int ks = 0; ks < nk; ++ks) {
      const int klim = K - ks * kBigBK;
      if (half == 0 && ks + 1 < nk) issue(ks + 1);
      read<MV>(ks, 0, klim);
      MOE_LGKM0();
      turn();
      mfma<MV>();
      turn();
      read<MV>(ks, 1, klim);
      MOE_LGKM0();
      if (half == 1) MOE_VMCNT0();
      turn();
      if (half == 1 && ks + 2 < nk) issue(ks + 2);
      mfma<MV>();
      if (half == 0) MOE_VMCNT0();
      turn();
    }
  }

  __device__ __forceinline__ void zero() {
#pragma unroll
    for (int m = 0; m < 8; ++m)
#pragma unroll
      for (int n = 0; n < 4; ++n) acc[m][n] = f32x4{0, 0, 0, 0};
  }

  // The sums of the tile in acc: lane holds row half * 128 + m * 16 + r16, columns wn * 64 + n * 16 + 4 g + 0..3.  Ends on a barrier.
  __device__ __forceinline__ void run(int rows, int cols) {
    const int nk = (K + kBigBK - 1) / kBigBK;
    zero();
    issue(0);
    MOE_VMCNT0();
    turn();
    if (half == 1) {
      if (nk > 1) issue(1);
      turn();
    }
    // 16-row blocks of this wave that hold any of the tile's rows (and columns): the others' products are left out
    const int mv = wn * 64 >= cols ? 0 : (rows - half * 128 + 15) >> 4;
    if (mv > 4) loop<8>(nk);
    else if (mv > 0) loop<4>(nk);
    else loop<0>(nk);
    if (half == 0) turn();
  }
};

}  // namespace moe
