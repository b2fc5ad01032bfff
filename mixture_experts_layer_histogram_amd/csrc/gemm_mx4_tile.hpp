// One 256-row x 256-column tile of the grouped SwiGLU FFN in MXFP4 on gfx950
// (v_mfma_scale_f32_32x32x64_f8f6f4 with both operands FP4); the operation and the tile's
// design are described at the top of gemm_mx4.hip.
#pragma once

#include "gemm_tile.hpp"
#include "mx4.hpp"

namespace moe {

constexpr int kMx4BK = 256;                                               // K values per stage: 128-byte LDS rows
constexpr int kMx4RowBytes = kMx4BK / 2;
constexpr int kMx4DataBytes = (kGemmBM + kGemmBN) * kMx4RowBytes;         // 64 KiB
constexpr int kMx4ScaleBytes = 2 * (kGemmBM + kGemmBN) * 4;               // two K-tile planes of a word per row
constexpr int kMx4StageBytes = kMx4DataBytes + kMx4ScaleBytes;
constexpr int kMx4Lds = 2 * kMx4StageBytes;                               // 136 KiB

struct TileMX4 {
  const uint8_t* a;     // the tile's first A row; row stride K / 2 bytes
  const uint8_t* as;    // the scale word of its first row in K-tile plane 0
  int64_t as_plane;     // bytes between K-tile planes of the A scales (4 * total A rows)
  void* o;              // MODE 0: h codes (row stride Nout / 2 bytes), MODE 1: bf16 rows (row stride Nout)
  uint8_t* os;          // MODE 0: the h scale word of the tile's first row in plane 0
  int64_t os_plane;     // MODE 0: bytes between planes of the h scales
  int rows;             // valid rows, 1..256; rows beyond re-read row rows-1 and are not stored
  const uint64_t* row_dst;  // MODE 1: null, or per tile row the address its output row goes to
};

// The order the scheduler is asked for in a sub-step of eight MFMAs: a read after each, so that the
// eight waves' LDS requests do not arrive in bursts.
#define MOE_MX4_PAIR                             \
  __builtin_amdgcn_sched_group_barrier(0x008, 1, 0); \
  __builtin_amdgcn_sched_group_barrier(0x100, 1, 0)
#define MOE_MX4_SPREAD \
  MOE_MX4_PAIR;        \
  MOE_MX4_PAIR;        \
  MOE_MX4_PAIR;        \
  MOE_MX4_PAIR;        \
  MOE_MX4_PAIR;        \
  MOE_MX4_PAIR;        \
  MOE_MX4_PAIR;        \
  MOE_MX4_PAIR

// MODE 0: h = MX4(silu(A B0^T) * (A B1^T)), 128 f columns of Nout = F per tile; MODE 1: bf16 A B0^T, 256
// columns.  b0/b1: this expert's weight codes ([Nout][K / 2]); bs0/bs1: the scale word of its row 0 in
// plane 0; bs_plane: bytes between the weights' K-tile planes.
template <int MODE>
__device__ __forceinline__ void gemm_mx4_tile(const TileMX4& io, const uint8_t* __restrict__ b0,
                                              const uint8_t* __restrict__ b1, const uint8_t* __restrict__ bs0,
                                              const uint8_t* __restrict__ bs1, int64_t bs_plane, int c0, int Nout,
                                              int K, char* smem) {
  const int tid = threadIdx.x;
  const int lane = tid & 63, wave = tid >> 6;
  const int wm = wave >> 1, wn = wave & 1;
  const int r32 = lane & 31, hi = lane >> 5;
  const int lrow = lane >> 3, lpos = lane & 7;
  const int lch_even = lpos ^ (lrow >> 1);
  const int lch_odd = lpos ^ (4 + (lrow >> 1));
  const int nk = (K + kMx4BK - 1) / kMx4BK;
  const bool half_tail = (K & 128) != 0;      // the last stage holds 128 K values
  const uint32_t rb = uint32_t(K >> 1);       // bytes of a row
  const int rows = io.rows;

  // fills: this wave's row groups g = wave*4 + i (rows g*8 + lrow) of the A and B tiles, as in
  // the bf16 and MXFP8 tiles (wave-uniform bases, 32-bit offsets)
  const uint8_t* abase = wave_uniform(io.a);
  const uint8_t* bbase = wave_uniform((MODE == 0 && (wave & 1)) ? b1 : b0);
  uint32_t aoff[4], boff[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int row = (wave * 4 + i) * 8 + lrow;
    const int lch = (i & 1) ? lch_odd : lch_even;
    aoff[i] = uint32_t(min(row, rows - 1)) * rb + lch * 16;
    const int n = (MODE == 0) ? min(c0 + (row >> 6) * 32 + (row & 31), Nout - 1) : min(c0 + row, Nout - 1);
    boff[i] = uint32_t(n) * rb + lch * 16;
  }
  // scale words: waves 0-3 fetch A rows 64*wave + lane, waves 4-7 B rows 64*(wave-4) + lane
  const uint8_t* sp;
  int64_t splane;
  {
    const int row = (wave & 3) * 64 + lane;
    if (wave < 4) {
      sp = io.as + 4 * size_t(min(row, rows - 1));
      splane = io.as_plane;
    } else {
      const int n = (MODE == 0) ? min(c0 + (row >> 6) * 32 + (row & 31), Nout - 1) : min(c0 + row, Nout - 1);
      sp = ((MODE == 0 && ((row >> 5) & 1)) ? bs1 : bs0) + 4 * size_t(n);
      splane = bs_plane;
    }
  }
  const uint32_t lds_dst0 = __builtin_amdgcn_readfirstlane(lds_addr(smem + wave * 4 * 1024));
  const uint32_t lds_sc0 = __builtin_amdgcn_readfirstlane(lds_addr(smem + kMx4DataBytes + wave * 256));
  auto issue = [&](int ks) {
    const uint32_t stage = uint32_t((ks & 1) * kMx4StageBytes);
    const uint32_t da = lds_dst0 + stage, db = da + uint32_t(kGemmBM * kMx4RowBytes);
    const uint32_t ls = lds_sc0 + stage;
    // the K offset goes into the scalar bases: no vector address work per fill
    const uint8_t* ak = abase + size_t(ks) * kMx4RowBytes;
    const uint8_t* bk = bbase + size_t(ks) * kMx4RowBytes;
    const uint8_t* s0 = sp + (2 * ks) * splane;
    const uint8_t* s1 = s0 + splane;
    uint32_t te = 0, to = 0;
    if (half_tail && ks == nk - 1) {  // chunks 4..7 lie past the row's end: re-read chunks 0..3 (never used)
      te = uint32_t(lch_even & 4) * 16;
      to = uint32_t(lch_odd & 4) * 16;
      s1 = s0;
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint32_t t = (i & 1) ? to : te;
      __builtin_amdgcn_global_load_lds(static_cast<const void*>(ak + (aoff[i] - t)),
                                       (lds_void_ptr)(uintptr_t)(da + uint32_t(i * 1024)), 16, 0, 0);
      __builtin_amdgcn_global_load_lds(static_cast<const void*>(bk + (boff[i] - t)),
                                       (lds_void_ptr)(uintptr_t)(db + uint32_t(i * 1024)), 16, 0, 0);
    }
    __builtin_amdgcn_global_load_lds(static_cast<const void*>(s0), (lds_void_ptr)(uintptr_t)ls, 4, 0, 0);
    __builtin_amdgcn_global_load_lds(static_cast<const void*>(s1),
                                     (lds_void_ptr)(uintptr_t)(ls + uint32_t(4 * (kGemmBM + kGemmBN))), 4, 0, 0);
  };

  f32x16 acc[2][4];
#pragma unroll
  for (int a = 0; a < 2; ++a)
#pragma unroll
    for (int b = 0; b < 4; ++b)
#pragma unroll
      for (int e = 0; e < 16; ++e) acc[a][b][e] = 0.0f;

  // Software pipeline over K, four sub-steps of 64 per 256-value stage.  The fragments of the
  // next sub-step are read while this one's MFMAs run (an FP4 fragment is 4 registers, so both
  // sets fit).  The stage's barrier sits before its last sub-step, whose fragments are in
  // registers by then: the fill two stages ahead goes into the stage nobody reads any more, and
  // the last sub-step's MFMAs cover the reads of the next stage's first fragments and scales.
  // Lane (row r32, half hi) supplies the 32 K values of block hi of the 64-value step (16 bytes)
  // and that block's scale: byte 2 (st & 1) + hi of the row's word st >> 1.
  int offA[4], offB[4];
#pragma unroll
  for (int st = 0; st < 4; ++st) {
    offA[st] = swz_off(wm * 64 + r32, 2 * st + hi);
    offB[st] = kGemmBM * kMx4RowBytes + swz_off(wn * 128 + r32, 2 * st + hi);
  }
  int offSA = kMx4DataBytes + 4 * (wm * 64 + r32);
  int offSB = kMx4DataBytes + 4 * (kGemmBM + wn * 128 + r32);
  auto frag = [&](const char* stg, int off, int m) -> i32x4 {
    return *reinterpret_cast<const i32x4*>(stg + off + m * 4096);
  };
  auto scl = [&](const char* stg, int off, int w, int m) -> int {
    return int(*reinterpret_cast<const uint32_t*>(stg + off + w * 4 * (kGemmBM + kGemmBN) + 128 * m) >> (8 * hi));
  };
  auto wide = [](const i32x4& v) -> i32x8 { return i32x8{v[0], v[1], v[2], v[3], 0, 0, 0, 0}; };

  __syncthreads();                               // the previous tile's epilogue is done with the stages
  issue(0);
  if (nk > 1) issue(1);
  if (nk > 1) asm volatile("s_waitcnt vmcnt(10)" ::: "memory");   // stage 0 landed (10 fills a stage)
  else asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
  __syncthreads();

  // Row padding: a wave whose 32-row blocks lie wholly past the tile's valid rows skips their
  // fragment reads and MFMAs; it still fills and meets every barrier.
  const int mv = __builtin_amdgcn_readfirstlane(min(2, max(0, (rows - wm * 64 + 31) >> 5)));
  auto kloop = [&](auto mvc) {
    constexpr int MV = decltype(mvc)::value;
    i32x4 fa[2][2], fb[2][4];            // fragments, two sets
    int sa[2][2], sb[2][4];              // scale words of a stage's two halves
    auto load = [&](int buf, const char* stg, int st) {
#pragma unroll
      for (int m = 0; m < MV; ++m) fa[buf][m] = frag(stg, offA[st], m);
#pragma unroll
      for (int n = 0; n < 4; ++n) fb[buf][n] = frag(stg, offB[st], n);
    };
    auto scales = [&](const char* stg, int w) {
#pragma unroll
      for (int m = 0; m < MV; ++m) sa[w][m] = scl(stg, offSA, w, m);
#pragma unroll
      for (int n = 0; n < 4; ++n) sb[w][n] = scl(stg, offSB, w, n);
    };
    auto mfmas = [&](int st) {           // sub-step st: fragment set st & 1, scale word st >> 1
      const int buf = st & 1, w = st >> 1;
#pragma unroll
      for (int m = 0; m < MV; ++m)
#pragma unroll
        for (int n = 0; n < 4; ++n) {
          if (st & 1)
            acc[m][n] = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(wide(fa[buf][m]), wide(fb[buf][n]), acc[m][n], 4,
                                                                        4, 2, sa[w][m], 2, sb[w][n]);
          else
            acc[m][n] = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(wide(fa[buf][m]), wide(fb[buf][n]), acc[m][n], 4,
                                                                        4, 0, sa[w][m], 0, sb[w][n]);
        }
    };
    // this wave's fills of the next stage and its reads of this one are done; then everyone's.
    // The accumulators pass through the statement, so no MFMA moves across the barrier.
    auto meet = [&]() {
      asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)\n\ts_barrier"
                   : "+v"(acc[0][0]), "+v"(acc[0][1]), "+v"(acc[0][2]), "+v"(acc[0][3]), "+v"(acc[1][0]),
                     "+v"(acc[1][1]), "+v"(acc[1][2]), "+v"(acc[1][3])
                   :
                   : "memory");
    };
    if constexpr (MV > 0) {
      load(0, smem, 0);
      scales(smem, 0);
    }
    const int nfull = half_tail ? nk - 1 : nk;
    for (int ks = 0; ks < nfull; ++ks) {
      const char* cs = smem + (ks & 1) * kMx4StageBytes;
      const char* ns = smem + ((ks + 1) & 1) * kMx4StageBytes;   // after the last stage: stale, unused
      asm volatile("" : "+v"(offA[0]), "+v"(offA[1]), "+v"(offA[2]), "+v"(offA[3]), "+v"(offB[0]), "+v"(offB[1]),
                   "+v"(offB[2]), "+v"(offB[3]), "+v"(offSA), "+v"(offSB));
      if constexpr (MV > 0) {
        load(1, cs, 1);
        mfmas(0);
        load(0, cs, 2);
        scales(cs, 1);
        mfmas(1);
        load(1, cs, 3);
        mfmas(2);
        if constexpr (MV == 2) {
          MOE_MX4_SPREAD;
          MOE_MX4_SPREAD;
          MOE_MX4_SPREAD;
        }
      }
      meet();
      if (ks + 2 < nk) issue(ks + 2);     // into stage ks, which nobody reads any more
      if constexpr (MV > 0) {
        load(0, ns, 0);
        scales(ns, 0);
        mfmas(3);
        if constexpr (MV == 2) MOE_MX4_SPREAD;
      }
    }
    if (half_tail) {                      // the last stage's first half: sub-steps 0 and 1
      if constexpr (MV > 0) {
        load(1, smem + (nfull & 1) * kMx4StageBytes, 1);
        mfmas(0);
        mfmas(1);
      }
    }
  };
  if (mv == 2) kloop(std::integral_constant<int, 2>{});
  else if (mv == 1) kloop(std::integral_constant<int, 1>{});
  else kloop(std::integral_constant<int, 0>{});
  __syncthreads();                        // the epilogues reuse the stages

  // The epilogue's lane indices are re-derived through an opaque copy, so the compiler cannot
  // hoist its store offsets above the main loop, where they would hold registers.
  int lane_o = lane;
  asm volatile("" : "+v"(lane_o));
  const int r32o = lane_o & 31, hio = lane_o >> 5;
  const int tido = wave * 64 + lane_o;

  // Epilogue through LDS, as the MXFP8 tile: a row-major tile whose rows are padded by 16 bytes;
  // the lane layout of the accumulators is column r32, rows 8*(e/4) + 4*hi + e%4 of each block.
  //  MODE 0: the fp32 h tile [256][128]; then every thread quantises whole 32-value blocks of it
  //          and writes 16 code bytes and the scale.  h is rounded once, from fp32 to E2M1 under
  //          its block's scale: 4-bit activations are what this dtype means.
  //  MODE 1: the bf16 output tile [256][256] (rounded once from fp32, the row type of this
  //          library's expert outputs); then 16-byte row segments go to global memory.
  constexpr int kPitch = 528;                                   // 512 bytes of data + 16
  static_assert(kGemmBM * kPitch <= kMx4Lds, "staged tile exceeds the LDS stages");
  char* ot = smem;
#pragma unroll
  for (int m = 0; m < 2; ++m) {
    const int rb0 = wm * 64 + m * 32;
    if (MODE == 0) {
#pragma unroll
      for (int q = 0; q < 2; ++q) {
        const int fc = (wn * 2 + q) * 32 + r32o;
#pragma unroll
        for (int e = 0; e < 16; ++e) {
          const int row = rb0 + 8 * (e >> 2) + 4 * hio + (e & 3);
          *reinterpret_cast<float*>(ot + row * kPitch + fc * 4) = mx4_silu(acc[m][2 * q][e]) * acc[m][2 * q + 1][e];
        }
      }
    } else {
#pragma unroll
      for (int n = 0; n < 4; ++n) {
        const int cc = wn * 128 + n * 32 + r32o;
#pragma unroll
        for (int e = 0; e < 16; ++e) {
          const int row = rb0 + 8 * (e >> 2) + 4 * hio + (e & 3);
          *reinterpret_cast<uint16_t*>(ot + row * kPitch + cc * 2) = uint16_t(pack_bf16x2(acc[m][n][e], 0.0f));
        }
      }
    }
  }
  __syncthreads();
  if (MODE == 0) {
    uint8_t* hq = static_cast<uint8_t*>(io.o);
    for (int b = tido; b < kGemmBM * 4; b += kGemmThreads) {    // 4 blocks of 32 f per row
      const int row = b >> 2, blk = b & 3;
      if (row >= rows) continue;
      const f32x4* src = reinterpret_cast<const f32x4*>(ot + row * kPitch + blk * 128);
      f32x4 v[8];
      uint32_t mx = 0;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        v[i] = src[i];
#pragma unroll
        for (int w = 0; w < 4; ++w) mx = max(mx, __float_as_uint(v[i][w]) & 0x7FFFFFFFu);
      }
      const uint32_t sc = mx4_scale_code(mx);
      u32x4 c = {0, 0, 0, 0};
      if (!mx4_blank(mx)) {
        const float f = e8m0_f32(sc);
#pragma unroll
        for (int w = 0; w < 4; ++w) c[w] = mx4_pack8(v[2 * w], v[2 * w + 1], f);
      }
      *reinterpret_cast<u32x4*>(hq + size_t(row) * (Nout >> 1) + ((c0 + blk * 32) >> 1)) = c;
      io.os[(c0 >> 7) * io.os_plane + 4 * size_t(row) + blk] = uint8_t(sc);
    }
  } else {
    uint16_t* orow0 = static_cast<uint16_t*>(io.o);
    const int ncols = min(kGemmBN, Nout - c0);
    for (int v = tido; v < kGemmBM * (kGemmBN / 8); v += kGemmThreads) {
      const int row = v >> 5, cv = v & 31;                   // 32 vectors of 8 bf16 per row
      if (row < rows && cv * 8 < ncols) {
        uint16_t* orow = io.row_dst ? reinterpret_cast<uint16_t*>(io.row_dst[row]) : orow0 + size_t(row) * Nout;
        *reinterpret_cast<u32x4*>(orow + c0 + cv * 8) = *reinterpret_cast<const u32x4*>(ot + row * kPitch + cv * 16);
      }
    }
  }
}

}  // namespace moe
