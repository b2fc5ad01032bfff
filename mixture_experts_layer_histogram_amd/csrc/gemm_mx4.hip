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
//
// Weights are the MFMA's first operand and token rows its second, so a lane ends up with 16 of 32
// columns of one token row and its partner in the other half with the rest: the epilogues work in
// registers (half exchanges instead of a tile in LDS), and the next tile's first two stages fill
// while they run; the waits for those fills leave the epilogue's stores in flight.
//
// Bound by both its schedule and power.  32 experts of 2048 x 7168, 32768 rows: GEMM1 504 to 539 us by the card
// and the clock (3.6 to 3.8 PFLOP/s), GEMM2 348 to 369 us (2.6 to 2.8 PFLOP/s; its rows' stores are 470 MB).
// On all-zero codes, with the same fills, reads and stores, they take 440 and 315 us: 13 and 9 % are power
// (the clock is 2.4 GHz there and 1.8 on random codes).  The rest is the schedule: the MFMA pipes are
// busy in 49 % and 35 % of the cycles on random codes (42 and 31 % on zeros), although GEMM1's MFMAs with the
// LDS reads and the epilogue but without fills take four fifths of its time.  MFMAs of this shape alone
// sustain 6.6 PFLOP/s on random operands and 9.8 on zeros.  A tile staged in LDS by the epilogue took 1224 us for the
// layer where this one takes 1092; 16x16x128 MFMAs, operands laid out by block, and token rows read
// straight into registers were no faster.
#include "gemm_tile.hpp"
#include "mx4.hpp"

namespace moe {

constexpr int kMx4BK = 256;                                               // K values per stage: 128-byte LDS rows
constexpr int kMx4RowBytes = kMx4BK / 2;
constexpr int kMx4DataBytes = (kGemmBM + kGemmBN) * kMx4RowBytes;         // 64 KiB
constexpr int kMx4ScaleBytes = 2 * (kGemmBM + kGemmBN) * 4;               // two K-tile planes of a word per row
constexpr int kMx4StageBytes = kMx4DataBytes + kMx4ScaleBytes;
constexpr int kMx4Lds = 2 * kMx4StageBytes;                               // 136 KiB

// The ten loads of a stage's fill in two parts (bits 0-3 A, 4-7 B, 8-9 scales): the token rows in the
// last sub-step of the stage before the one before, the weights and scales in the first sub-step
// after it.  All ten in one sub-step: 1146 us for the share of 32 experts of 2048 x 7168 (32700 rows)
// instead of 1105; other splits, or three parts, 1115 to 1175.
constexpr int kFirst = 0x00F, kSecond = 0x3F0;

// The order the scheduler is asked for in a sub-step of eight MFMAs: the LDS reads of the next
// fragments behind the first four, two each, so that the eight waves' requests do not arrive in one
// burst (one each 1139 us, three 1123, in front of the MFMAs 1113), then this part's fills behind the
// last four.
template <int PART>
__device__ __forceinline__ void spread() {
  constexpr int kPer = (__builtin_popcount(PART) + 3) / 4;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
    __builtin_amdgcn_sched_group_barrier(0x100, 2, 0);
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
    __builtin_amdgcn_sched_group_barrier(0x020, kPer, 0);
  }
}

// exchanges: the upper half (odd 16-lane rows) of `a` with the lower half (even rows) of `b`
__device__ __forceinline__ void swap_halves(uint32_t& a, uint32_t& b) {
  const auto r = __builtin_amdgcn_permlane32_swap(a, b, false, false);
  a = r[0];
  b = r[1];
}
__device__ __forceinline__ void swap_rows16(uint32_t& a, uint32_t& b) {
  const auto r = __builtin_amdgcn_permlane16_swap(a, b, false, false);
  a = r[0];
  b = r[1];
}

// MODE 0: A = xe codes [*][d/2], B0/B1 = W1/W3 -> h codes [*][F/2] + scales   (256 rows x 128 f)
// MODE 1: A = h codes [*][F/2],  B0 = W2 -> bf16 [*][d]                        (256 x 256)
// MODE 2: the same, each row to the address that RowDst holds for it (the fused push)
// MODE 3: the same, fp32 rows
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
  constexpr int kCols = (MODE == 0) ? kGemmBN / 2 : kGemmBN;
  const int NT = (Nout + kCols - 1) / kCols;
  const int total = ctrl[kCtrlMTiles] * NT;
  const int per_xcd = (total + 7) >> 3;
  const int xcd = blockIdx.x & 7;
  const int wg_per_xcd = gridDim.x >> 3;

  const int tid = threadIdx.x;
  const int lane = tid & 63, wave = tid >> 6;
  const int wm = wave >> 1, wn = wave & 1;
  const int r32 = lane & 31, hi = lane >> 5;
  const int lch_even = (lane & 7) ^ (lane >> 4);     // fill lane: row lane / 8 of eight, chunk lane % 8 swizzled
  const int nk = (K + kMx4BK - 1) / kMx4BK;
  const bool half_tail = (K & 128) != 0;      // the last stage holds 128 K values
  const uint32_t rb = uint32_t(K >> 1);       // bytes of a row

  // the tiles of this workgroup, in ascending order
  struct Tile {
    int l, row0, rows, c0;                    // expert, first row, valid rows (1..256), first column (f)
  };
  typedef const __attribute__((address_space(4))) int32_t* sload_t;     // scalar loads: a vector load's wait
  const sload_t mbase = (sload_t)reinterpret_cast<uintptr_t>(mtile_base);   // would drain the fills in flight
  const sload_t offs = (sload_t)reinterpret_cast<uintptr_t>(offsets);
  int tt = int(blockIdx.x >> 3) - wg_per_xcd;
  Tile next{-1, 0, 0, 0};
  auto advance = [&]() -> bool {
    for (;;) {
      tt += wg_per_xcd;
      const int tau = xcd * per_xcd + tt;
      if (tt >= per_xcd || tau >= total) return false;
      const int mtg = tau / NT;
      int l = next.l;
      if (l < 0) l = __builtin_amdgcn_readfirstlane(find_expert(mtile_base, El, mtg));
      while (l + 1 < El && mbase[l + 1] <= mtg) ++l;
      next.l = l;
      const int mt0 = mbase[l], mtl = mbase[l + 1] - mt0;
      const int o0 = offs[l], o1 = offs[l + 1];
      if (o1 - o0 < min_rows) continue;       // the streaming kernel's
      const int i_in = tau - mt0 * NT;
      const int nt = i_in / mtl, mt = i_in - nt * mtl;
      next.row0 = o0 + mt * kGemmBM;
      next.rows = min(kGemmBM, o1 - next.row0);
      next.c0 = nt * kCols;
      return true;
    }
  };

  // fills: this wave's row groups g = wave*4 + i (rows g*8 + lrow) of the A and B tiles, as in
  // the bf16 and MXFP8 tiles (wave-uniform bases, 32-bit offsets); scale words: waves 0-3 fetch A
  // rows 64*wave + lane, waves 4-7 B rows 64*(wave-4) + lane.  Rows past the last re-read it.
  const uint8_t *abase, *bbase, *sp;
  uint32_t aoff[4], boff[4];
  const int64_t splane = wave < 4 ? 4 * nmax : 4 * int64_t(El) * Nout;   // weight planes hold every expert's rows
  auto column = [&](int c0, int row) -> int {
    return (MODE == 0) ? min(c0 + (row >> 6) * 32 + (row & 31), Nout - 1) : min(c0 + row, Nout - 1);
  };
  auto aim = [&](const Tile& t) {
    int lane_o = lane;                        // opaque: nothing of this is hoisted out of the tile loop,
    asm volatile("" : "+v"(lane_o));          // where it would hold registers
    const int lrow = lane_o >> 3, lpos = lane_o & 7;
    const int lch_even = lpos ^ (lrow >> 1), lch_odd = lpos ^ (4 + (lrow >> 1));
    abase = wave_uniform(A + size_t(t.row0) * rb);
    bbase = wave_uniform(((MODE == 0 && (wave & 1)) ? B1 : B0) + size_t(t.l) * Nout * rb);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int row = (wave * 4 + i) * 8 + lrow;
      const int lch = (i & 1) ? lch_odd : lch_even;
      aoff[i] = uint32_t(min(row, t.rows - 1)) * rb + lch * 16;
      boff[i] = uint32_t(column(t.c0, row)) * rb + lch * 16;
    }
    const int row = (wave & 3) * 64 + lane_o;
    if (wave < 4) sp = As + 4 * size_t(t.row0 + min(row, t.rows - 1));
    else sp = ((MODE == 0 && ((row >> 5) & 1)) ? Bs1 : Bs0) + 4 * (size_t(t.l) * Nout + column(t.c0, row));
  };
  const uint32_t lds_dst0 = __builtin_amdgcn_readfirstlane(lds_addr(smem + wave * 4 * 1024));
  const uint32_t lds_sc0 = __builtin_amdgcn_readfirstlane(lds_addr(smem + kMx4DataBytes + wave * 256));
  // part: which of a stage's ten loads (bits 0-3 A, 4-7 B, 8-9 the scales of its two K tiles)
  auto issue_part = [&](int ks, auto part) {
    constexpr int P = decltype(part)::value;
    const uint32_t stage = uint32_t((ks & 1) * kMx4StageBytes);
    const uint32_t da = lds_dst0 + stage, db = da + uint32_t(kGemmBM * kMx4RowBytes);
    const uint32_t ls = lds_sc0 + stage;
    // the K offset goes into the scalar bases: no vector address work per fill
    const uint8_t* ak = abase + size_t(ks) * kMx4RowBytes;
    const uint8_t* bk = bbase + size_t(ks) * kMx4RowBytes;
    const uint8_t* s0 = sp + (2 * ks) * splane;
    const uint8_t* s1 = s0 + ((half_tail && ks == nk - 1) ? 0 : splane);
    // chunks 4..7 of a half stage lie past the row's end: re-read chunks 0..3 (never used)
    const bool tail = half_tail && ks == nk - 1;
    const uint32_t te = uint32_t(lch_even & (tail ? 4 : 0)) * 16, to = uint32_t(~lch_even & (tail ? 4 : 0)) * 16;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint32_t t = (i & 1) ? to : te;
      uint32_t ao = aoff[i] - t, bo = boff[i] - t;           // opaque: kept as one register each, not as pairs
      asm volatile("" : "+v"(ao), "+v"(bo));
      if ((P >> i) & 1)
        __builtin_amdgcn_global_load_lds(static_cast<const void*>(ak + ao), (lds_void_ptr)(uintptr_t)(da + uint32_t(i * 1024)),
                                         16, 0, 0);
      if ((P >> (4 + i)) & 1)
        __builtin_amdgcn_global_load_lds(static_cast<const void*>(bk + bo), (lds_void_ptr)(uintptr_t)(db + uint32_t(i * 1024)),
                                         16, 0, 0);
    }
    if constexpr ((P >> 8) & 1)
      __builtin_amdgcn_global_load_lds(static_cast<const void*>(s0), (lds_void_ptr)(uintptr_t)ls, 4, 0, 0);
    if constexpr ((P >> 9) & 1)
      __builtin_amdgcn_global_load_lds(static_cast<const void*>(s1),
                                     (lds_void_ptr)(uintptr_t)(ls + uint32_t(4 * (kGemmBM + kGemmBN))), 4, 0, 0);
  };

  // waves whose 64 token rows lie wholly past the tile's valid rows do not fill their share of the rows
  bool lean = false;
  auto issue = [&](int ks) {
    if (lean) issue_part(ks, std::integral_constant<int, kSecond>{});
    else issue_part(ks, std::integral_constant<int, kFirst | kSecond>{});
  };

  f32x16 acc[2][4];
  // Software pipeline over K, four sub-steps of 64 per 256-value stage.  The fragments of the
  // next sub-step are read while this one's MFMAs run (an FP4 fragment is 4 registers, so both
  // sets fit).  The stage's barrier sits before its last sub-step, whose fragments are in
  // registers by then: the fill two stages ahead starts into the stage nobody reads any more, and
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

  // stores an epilogue certainly issues for a whole tile (waits may leave so many operations in flight)
  constexpr int kStores = (MODE == 0) ? 4 : (MODE == 3) ? 32 : 16;
  auto kloop = [&](auto mvc, int behind) {
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
            acc[m][n] = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(wide(fb[buf][n]), wide(fa[buf][m]), acc[m][n], 4,
                                                                        4, 2, sb[w][n], 2, sa[w][m]);
          else
            acc[m][n] = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(wide(fb[buf][n]), wide(fa[buf][m]), acc[m][n], 4,
                                                                        4, 0, sb[w][n], 0, sa[w][m]);
        }
    };
    // this wave's fills of the next stage and its reads of this one are done; then everyone's.  Stage 1
    // was filled before the last epilogue's stores, which may still fly; the later stages after them.
    // The accumulators pass through, so no MFMA moves across the barrier.
    auto meet = [&]() {                   // one block of code: a branch here would split the schedule
      asm volatile("s_waitcnt vmcnt(%c9)\n\ts_cmp_lg_u32 %8, 0\n\ts_cbranch_scc1 1f\n\ts_waitcnt vmcnt(0)\n1:\n\t"
                   "s_waitcnt lgkmcnt(0)\n\ts_barrier"
                   : "+v"(acc[0][0]), "+v"(acc[0][1]), "+v"(acc[0][2]), "+v"(acc[0][3]), "+v"(acc[1][0]),
                     "+v"(acc[1][1]), "+v"(acc[1][2]), "+v"(acc[1][3])
                   : "s"(behind), "n"(kStores)
                   : "memory", "scc");
      behind = 0;                         // opaque below, or the compiler peels the first iteration
      asm volatile("" : "+s"(behind));
    };
    if constexpr (MV > 0) {
      load(0, smem, 0);
      scales(smem, 0);
    }
    const int nfull = half_tail ? nk - 1 : nk;
    int ks = 0;
    // `early`: the last sub-step starts the fill of stage ks + 2, into stage ks, which nobody reads any
    // more; `late`: the first sub-step issues the rest of stage ks + 1's.
    auto stage = [&](auto early, auto late) {
      constexpr bool E = decltype(early)::value, L = decltype(late)::value;
      const char* cs = smem + (ks & 1) * kMx4StageBytes;
      const char* ns = smem + ((ks + 1) & 1) * kMx4StageBytes;   // after the last stage: stale, unused
      asm volatile("" : "+v"(offA[0]), "+v"(offA[1]), "+v"(offA[2]), "+v"(offA[3]), "+v"(offB[0]), "+v"(offB[1]),
                   "+v"(offB[2]), "+v"(offB[3]), "+v"(offSA), "+v"(offSB));
      if constexpr (MV > 0) load(1, cs, 1);
      if constexpr (L) issue_part(ks + 1, std::integral_constant<int, kSecond>{});
      if constexpr (MV > 0) {
        mfmas(0);
        load(0, cs, 2);
        scales(cs, 1);
        mfmas(1);
        load(1, cs, 3);
        mfmas(2);
      }
      if constexpr (MV == 2) {
        spread<L ? kSecond : 0>();
        spread<0>();
        spread<0>();
      }
      meet();
      if constexpr (MV > 0) {
        load(0, ns, 0);
        scales(ns, 0);
      }
      if constexpr (E && MV > 0) issue_part(ks + 2, std::integral_constant<int, kFirst>{});
      if constexpr (MV > 0) mfmas(3);
      if constexpr (MV == 2) spread<E ? kFirst : 0>();
    };
    if (nk > 2) {
      stage(std::true_type{}, std::false_type{});
      for (++ks; ks + 2 < nk; ++ks) stage(std::true_type{}, std::true_type{});
      stage(std::false_type{}, std::true_type{});
      ++ks;
    }
    for (; ks < nfull; ++ks) stage(std::false_type{}, std::false_type{});
    if (half_tail) {                      // the last stage's first half: sub-steps 0 and 1
      if constexpr (MV > 0) {
        load(1, smem + (nfull & 1) * kMx4StageBytes, 1);
        mfmas(0);
        mfmas(1);
      }
    }
  };

  if (!advance()) return;
  aim(next);
  lean = __builtin_amdgcn_readfirstlane(next.rows <= wm * 64);
  issue(0);
  if (nk > 1) issue(1);
  int stores = 0;                       // the fills in flight are followed by kStores stores at least
  for (;;) {
    const Tile t = next;
#pragma unroll
    for (int a = 0; a < 2; ++a)
#pragma unroll
      for (int b = 0; b < 4; ++b)
#pragma unroll
        for (int e = 0; e < 16; ++e) acc[a][b][e] = 0.0f;
    // stage 0 landed: behind its fills are stage 1's and the stores
    auto landed = [&](auto fills) {
      constexpr int n = decltype(fills)::value;
      if (stores) asm volatile("s_waitcnt vmcnt(%0)\n\ts_barrier" ::"n"(n + kStores) : "memory");
      else asm volatile("s_waitcnt vmcnt(%0)\n\ts_barrier" ::"n"(n) : "memory");
    };
    if (nk == 1) landed(std::integral_constant<int, 0>{});
    else if (lean) landed(std::integral_constant<int, __builtin_popcount(kSecond)>{});
    else landed(std::integral_constant<int, __builtin_popcount(kFirst | kSecond)>{});
    // Row padding: a wave whose 32-row blocks lie wholly past the tile's valid rows skips their
    // fragment reads and MFMAs; it still fills and meets every barrier.
    const int mv = __builtin_amdgcn_readfirstlane(min(2, max(0, (t.rows - wm * 64 + 31) >> 5)));
    if (mv == 2) kloop(std::integral_constant<int, 2>{}, __builtin_amdgcn_readfirstlane(stores));
    else if (mv == 1) kloop(std::integral_constant<int, 1>{}, __builtin_amdgcn_readfirstlane(stores));
    else kloop(std::integral_constant<int, 0>{}, __builtin_amdgcn_readfirstlane(stores));
    const bool more = advance();
    asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");   // every wave has read both stages
    if (more) {
      aim(next);
      lean = __builtin_amdgcn_readfirstlane(next.rows <= wm * 64);
      issue(0);
      if (nk > 1) issue(1);
    }
    stores = t.rows == kGemmBM && (MODE == 0 || t.c0 + kGemmBN <= Nout);

    // Epilogue.  The lane indices are re-derived through an opaque copy, so the compiler cannot
    // hoist its offsets above the main loop, where they would hold registers.  Value 4 c + j of an
    // accumulator is column 8 c + 4 hi + j of its block of 32, of token row r32.  No store moves up past
    // the fills (the memory clobber): the waits above count on their order.
    int lane_o = lane;
    asm volatile("" : "+v"(lane_o) : : "memory");
    const int r32o = lane_o & 31, hio = lane_o >> 5;
    if constexpr (MODE == 0) {
      // h is rounded once, from fp32 to E2M1 under its block's scale: 4-bit activations are what this
      // dtype means.  Half s stores block 2 wn + s of its row: 16 code bytes and the scale.
#pragma unroll
      for (int m = 0; m < 2; ++m) {
        const int row = wm * 64 + m * 32 + r32o;
        uint32_t lo[2], up[2], sc[2];         // codes of this half's columns c = 0, 1 and c = 2, 3
#pragma unroll
        for (int q = 0; q < 2; ++q) {
          float h[16];
          uint32_t mx = 0;
#pragma unroll
          for (int e = 0; e < 16; ++e) {
            h[e] = mx4_silu(acc[m][2 * q][e]) * acc[m][2 * q + 1][e];
            mx = max(mx, __float_as_uint(h[e]) & 0x7FFFFFFFu);
          }
          mx = max(mx, uint32_t(__shfl_xor(int(mx), 32, 64)));
          sc[q] = mx4_scale_code(mx);
          const float f = e8m0_f32(sc[q]);
          lo[q] = mx4_blank(mx) ? 0u : mx4_pack8(f32x4{h[0], h[1], h[2], h[3]}, f32x4{h[4], h[5], h[6], h[7]}, f);
          up[q] = mx4_blank(mx) ? 0u : mx4_pack8(f32x4{h[8], h[9], h[10], h[11]}, f32x4{h[12], h[13], h[14], h[15]}, f);
        }
        swap_halves(lo[0], lo[1]);            // now [0]: the lower half's codes of block s, [1]: the upper half's
        swap_halves(up[0], up[1]);
        const u32x4 code = {(lo[0] & 0xFFFFu) | (lo[1] << 16), (lo[0] >> 16) | (lo[1] & 0xFFFF0000u),
                            (up[0] & 0xFFFFu) | (up[1] << 16), (up[0] >> 16) | (up[1] & 0xFFFF0000u)};
        if (row < t.rows) {
          const int blk = wn * 2 + hio;
          *reinterpret_cast<u32x4*>(static_cast<uint8_t*>(C) + size_t(t.row0 + row) * (Nout >> 1) + (t.c0 >> 1) + blk * 16) = code;
          Cs[(t.c0 >> 7) * (4 * nmax) + 4 * size_t(t.row0 + row) + blk] = uint8_t(hio ? sc[1] : sc[0]);
        }
      }
    } else if (MODE == 3 && t.c0 + wn * 128 < Nout) {
#pragma unroll
      for (int m = 0; m < 2; ++m) {
        const int row = wm * 64 + m * 32 + r32o;
        f32x4* const dst = reinterpret_cast<f32x4*>(static_cast<float*>(C) + size_t(t.row0 + min(row, t.rows - 1)) * Nout +
                                                    t.c0 + wn * 128 + hio * 4);
#pragma unroll
        for (int n = 0; n < 4; ++n)
#pragma unroll
          for (int c = 0; c < 4; ++c)
            if (row < t.rows)
              dst[8 * n + 2 * c] = f32x4{acc[m][n][4 * c], acc[m][n][4 * c + 1], acc[m][n][4 * c + 2], acc[m][n][4 * c + 3]};
      }
    } else if (t.c0 + wn * 128 < Nout) {
      // bf16 rows, rounded once from fp32 (the row type of this library's expert outputs).  Two
      // exchanges turn a block's column quads into 16 rows x 64 bytes: lane group g = lane / 16 holds
      // columns 16 (g & 1) + 8 (g >> 1) .. + 7 of row lane % 16 (first store) and of row + 16 (second).
      const int r16 = lane_o & 15, g = lane_o >> 4;
      const int col = t.c0 + wn * 128 + (g & 1) * 16 + (g >> 1) * 8;
      typedef __attribute__((address_space(1))) u32x4* grow_t;      // global, or a row's address makes flat stores
      auto row_at = [&](int r, int c) -> grow_t {
        const int row = t.row0 + min(r, t.rows - 1);
        uintptr_t p = reinterpret_cast<uintptr_t>(C) + size_t(row) * Nout * 2;
        if constexpr (MODE == 2) p = RowDst[row];
        return (grow_t)(p + size_t(c) * 2);
      };
#pragma unroll
      for (int m = 0; m < 2; ++m) {
        const int ra = wm * 64 + m * 32 + r16;
        grow_t pa = row_at(ra, col), pb = row_at(ra + 16, col);
#pragma unroll
        for (int n = 0; n < 4; ++n) {
          uint32_t v[2][4];
#pragma unroll
          for (int p = 0; p < 2; ++p) {
#pragma unroll
            for (int w = 0; w < 4; ++w) v[p][w] = pack_bf16x2(acc[m][n][8 * p + 2 * w], acc[m][n][8 * p + 2 * w + 1]);
            swap_halves(v[p][0], v[p][2]);
            swap_halves(v[p][1], v[p][3]);
          }
#pragma unroll
          for (int w = 0; w < 4; ++w) swap_rows16(v[0][w], v[1][w]);
          if (ra < t.rows) pa[4 * n] = u32x4{v[0][0], v[0][1], v[0][2], v[0][3]};
          if (ra + 16 < t.rows) pb[4 * n] = u32x4{v[1][0], v[1][1], v[1][2], v[1][3]};
        }
      }
    }
    if (!more) break;
  }
}

hipError_t launch_thin_mx4(bool gate_up, const uint8_t* a, const uint8_t* as, const uint8_t* b0, const uint8_t* b1,
                           const uint8_t* bs0, const uint8_t* bs1, void* o, uint8_t* os, const int32_t* offsets,
                           const uint64_t* row_dst, bool rows32, int64_t nmax, int El, int64_t experts, int K, int Nout,
                           int cus, hipStream_t st);

hipError_t launch_ffn_mx4(const moe_shape_t& s, int El, const uint8_t* xe, const uint8_t* xe_scales,
                          const int32_t* offsets, const uint8_t* w1, const uint8_t* w3, const uint8_t* w2,
                          const moe_mx_scales_t& w_scales, void* ye, char* ws, const WsLayout& L, int cus,
                          hipStream_t st, const uint64_t* row_dst, bool rows32) {
  static std::atomic<uint64_t> attr_set{0};
  const hipError_t ea = once_per_device(attr_set, [] {
    hipError_t e = hipFuncSetAttribute(reinterpret_cast<const void*>(grouped_gemm_mx4_kernel<0>),
                                       hipFuncAttributeMaxDynamicSharedMemorySize, kMx4Lds);
    if (e == hipSuccess)
      e = hipFuncSetAttribute(reinterpret_cast<const void*>(grouped_gemm_mx4_kernel<1>),
                              hipFuncAttributeMaxDynamicSharedMemorySize, kMx4Lds);
    if (e == hipSuccess)
      e = hipFuncSetAttribute(reinterpret_cast<const void*>(grouped_gemm_mx4_kernel<2>),
                              hipFuncAttributeMaxDynamicSharedMemorySize, kMx4Lds);
    if (e == hipSuccess)
      e = hipFuncSetAttribute(reinterpret_cast<const void*>(grouped_gemm_mx4_kernel<3>),
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
  // streaming kernel does it all; with kThinMean rows expected of an expert or more the tile kernel
  // does; in between both run, each on its experts.  The layer on 32 of 256 experts of 2048 x 7168
  // with both and with the tile kernel alone: 4 rows an expert 130 us and 168, 16 rows 149 and 179,
  // 24 rows 193 and 187, 30 rows (of which many have more than 32) 251 and 200.  64 experts of 1408 x 2048: 4 rows
  // 70 and 78, 16 rows 80 and 86, 20 rows 83 and 86, 24 rows 105 and 89.  The rule sees no loads: where a
  // few experts have most of the rows (Zipf's popularity), both in turn cost more than the tile kernel on all
  // (64 experts of 1408 x 2048, 4 and 20 rows on average: 78 and 60, 120 and 94 us; 32 of 256 of 2048 x 7168 with
  // 10 and 16 rows: 133 and 119, but 151 and 169).
  const int64_t tokens = int64_t(s.R) * s.T;
  const bool thin = tokens <= kThinRows || tokens * s.k <= int64_t(kThinMean) * s.E;
  const bool wide = tokens > kThinRows;
  const int min_rows = thin ? kThinRows + 1 : 0;
  const int64_t nmax = L.max_pairs;
  const int64_t experts = El < nmax ? El : nmax;             // with a row, at most
  if (thin) {
    const hipError_t e = launch_thin_mx4(true, xe, xe_scales, w1, w3, w_scales.w1, w_scales.w3, hq, hs, offsets, nullptr,
                                         false, nmax, El, experts, s.d, s.F, cus, st);
    if (e != hipSuccess) return e;
  }
  if (wide)
    hipLaunchKernelGGL(grouped_gemm_mx4_kernel<0>, dim3(grid), dim3(kGemmThreads), kMx4Lds, st, xe, xe_scales, w1, w3,
                       w_scales.w1, w_scales.w3, static_cast<void*>(hq), hs, offsets, mtb, ctrl, El, s.d, s.F, nmax,
                       nullptr, min_rows);
  if (thin) {
    const hipError_t e = launch_thin_mx4(false, hq, hs, w2, w2, w_scales.w2, w_scales.w2, ye, nullptr, offsets, row_dst,
                                         rows32, nmax, El, experts, s.F, s.d, cus, st);
    if (e != hipSuccess) return e;
  }
  if (wide) {
    const auto kernel = row_dst ? grouped_gemm_mx4_kernel<2> : rows32 ? grouped_gemm_mx4_kernel<3> : grouped_gemm_mx4_kernel<1>;
    hipLaunchKernelGGL(kernel, dim3(grid), dim3(kGemmThreads), kMx4Lds, st, hq, hs, w2, nullptr, w_scales.w2, nullptr, ye,
                       nullptr, offsets, mtb, ctrl, El, s.F, s.d, nmax, row_dst, min_rows);
  }
  return hipGetLastError();
}

}  // namespace moe
