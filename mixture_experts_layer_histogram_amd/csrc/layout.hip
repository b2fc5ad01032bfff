// Routing and sort-free layout generation for gfx950.
//
// Operation (MoK article, kucoin.com/es "Cursor's MoK logra un aumento del 2.37x ...",
// section 01; qubstore.ru "Смесь котят ...", pull paragraph): every token keeps its
// k best experts; the expert side counts pairs per expert, takes an exclusive
// prefix over its local experts and gives each pair a destination row so that one
// expert's rows are contiguous, recording only (source rank, source token) -- a
// two-column pull schedule built without sorting.
//
// Three launches:
//   1. topk_hist   : one 16-lane group per token (4 tokens per wave, a block's 64
//                    tokens at once for E <= 256); k rounds of a 16-lane max over
//                    packed (logit, ~id) keys; gate = softmax over the kept logits;
//                    per-block expert histogram in LDS.
//   2. layout_scan : block 0 validates the placement, scans the local experts'
//                    block histograms (flattened exclusive scan = offsets and
//                    per-block bases at once) and the GEMM-tile / chunk tables;
//                    blocks 1.. reduce the global per-expert counts.
//   3. slot_assign : one wave per histogram block walks its pairs in (r, t, j)
//                    order; equal-expert lanes are found with ballots over the id
//                    bits, ranked with a popcount, offset by an LDS running count.
#include "common.hpp"

namespace moe {

// ---------------------------------------------------------------------------
// packed ordering key: larger key = larger logit, ties -> lower expert id
// ---------------------------------------------------------------------------
__device__ __forceinline__ unsigned long long make_key(float v, int e) {
  uint32_t u = __float_as_uint(v);
  if ((u << 1) == 0u) u = 0u;                           // -0.0 orders like +0.0
  u = (u & 0x80000000u) ? ~u : (u | 0x80000000u);       // monotone float -> uint
  return (static_cast<unsigned long long>(u) << 32) | (0xFFFFFFFFu - static_cast<uint32_t>(e));
}

__device__ __forceinline__ float key_value(unsigned long long key) {
  uint32_t u = static_cast<uint32_t>(key >> 32);
  u = (u & 0x80000000u) ? (u & 0x7FFFFFFFu) : ~u;
  return __uint_as_float(u);
}

__device__ __forceinline__ int key_expert(unsigned long long key) {
  return static_cast<int>(0xFFFFFFFFu - static_cast<uint32_t>(key));
}

// VPL = logits held per lane (E <= 16 * VPL); NT threads per block, so NT / 16 tokens in
// flight per pass over the block's kTokPerLayoutBlock tokens.  With up to 256 experts the
// block has 1024 threads (every token of the block in one pass) and the ordering keys are
// built once per token; wider rows keep 256 threads and rebuild the keys every round.
template <int VPL, int NT>
__global__ __launch_bounds__(NT) void topk_hist_kernel(RankPtrs<const float*> logits, int R, int T,
                                                       int E, int k, int32_t* __restrict__ topk_idx,
                                                       float* __restrict__ topk_w,
                                                       int32_t* __restrict__ blockhist) {
  constexpr bool kKeys = VPL <= 16;        // keys kept in registers
  constexpr int kGroups = NT / 16;         // tokens in flight per pass
  __shared__ int hist[1024];
  const int tid = threadIdx.x;
  for (int e = tid; e < E; e += NT) hist[e] = 0;
  __syncthreads();

  const int grp = tid >> 4, sl = tid & 15;
  const int64_t RT = int64_t(R) * T;
  const int64_t tok0 = int64_t(blockIdx.x) * kTokPerLayoutBlock;

#pragma unroll 1
  for (int pass = 0; pass < kTokPerLayoutBlock / kGroups; ++pass) {
    const int64_t g = tok0 + pass * kGroups + grp;
    const bool valid = g < RT;
    float v[VPL];
    if (valid) {
      const int r = int(g / T);
      const int t = int(g - int64_t(r) * T);
      const float* row = logits.p[r] + size_t(t) * E;
#pragma unroll
      for (int i = 0; i < VPL; ++i) {
        const int e = sl + 16 * i;
        v[i] = (e < E) ? row[e] : 0.0f;
      }
    } else {
#pragma unroll
      for (int i = 0; i < VPL; ++i) v[i] = 0.0f;
    }
    unsigned long long keys[kKeys ? VPL : 1];
    if constexpr (kKeys) {
#pragma unroll
      for (int i = 0; i < VPL; ++i) {
        const int e = sl + 16 * i;
        keys[i] = (e < E) ? make_key(v[i], e) : 0ull;       // 0 is below every real key
      }
    }

    unsigned long long taken = 0ull;
    int my_idx = 0;
    float my_val = 0.0f;
    for (int j = 0; j < k; ++j) {
      unsigned long long best = 0ull;
#pragma unroll
      for (int i = 0; i < VPL; ++i) {
        const int e = sl + 16 * i;
        const unsigned long long key = kKeys ? keys[i] : make_key(v[i], e);
        const bool ok = (e < E) && !((taken >> i) & 1ull);
        best = (ok && key > best) ? key : best;
      }
#pragma unroll
      for (int off = 8; off >= 1; off >>= 1) {
        const unsigned long long o = __shfl_xor(best, off, 16);
        best = o > best ? o : best;
      }
      const int ew = key_expert(best);
      if ((ew & 15) == sl) taken |= 1ull << (ew >> 4);
      if (sl == j) {
        my_idx = ew;
        my_val = key_value(best);
      }
    }
    // gate: softmax over the kept logits, max = the first kept logit
    const float m = __shfl(my_val, 0, 16);
    const float z = (sl < k) ? expf(my_val - m) : 0.0f;
    float zs = z;
#pragma unroll
    for (int off = 8; off >= 1; off >>= 1) zs += __shfl_xor(zs, off, 16);
    if (valid && sl < k) {
      topk_idx[g * k + sl] = my_idx;
      topk_w[g * k + sl] = z / zs;
      atomicAdd(&hist[my_idx], 1);
    }
  }
  __syncthreads();
  for (int e = tid; e < E; e += NT) blockhist[size_t(blockIdx.x) * E + e] = hist[e];
}

// exclusive scan over a 1024-thread block; returns the thread's exclusive prefix
__device__ int block_excl_scan_1024(int v, int* tmp16, int* total) {
  const int lane = threadIdx.x & 63, w = threadIdx.x >> 6;
  int x = v;
#pragma unroll
  for (int off = 1; off < 64; off <<= 1) {
    const int y = __shfl_up(x, off, 64);
    if (lane >= off) x += y;
  }
  if (lane == 63) tmp16[w] = x;
  __syncthreads();
  if (w == 0) {
    int s = (lane < 16) ? tmp16[lane] : 0;
#pragma unroll
    for (int off = 1; off < 16; off <<= 1) {
      const int y = __shfl_up(s, off, 64);
      if (lane >= off) s += y;
    }
    if (lane < 16) tmp16[lane] = s;
  }
  __syncthreads();
  const int excl = (w > 0 ? tmp16[w - 1] : 0) + x - v;
  *total = tmp16[15];
  __syncthreads();
  return excl;
}

__global__ __launch_bounds__(1024) void layout_scan_kernel(
    const int32_t* __restrict__ e2l, int E, int El, int nb, int bm, int mb,
    const int32_t* __restrict__ blockhist, int32_t* __restrict__ blockbase,
    int32_t* __restrict__ counts, int32_t* __restrict__ offsets, int32_t* __restrict__ l2g,
    int32_t* __restrict__ mtile_base, int32_t* __restrict__ chunk_base, int32_t* __restrict__ ctrl) {
  const int tid = threadIdx.x;
  if (blockIdx.x > 0) {
    // global per-expert counts: 16 threads per expert
    const int e = (blockIdx.x - 1) * 64 + (tid >> 4), q = tid & 15;
    int sum = 0;
    if (e < E) {
#pragma unroll 8
      for (int b = q; b < nb; b += 16) sum += blockhist[size_t(b) * E + e];
    }
#pragma unroll
    for (int off = 8; off >= 1; off >>= 1) sum += __shfl_xor(sum, off, 16);
    if (e < E && q == 0) counts[e] = sum;
    return;
  }

  __shared__ int seen[1024];
  __shared__ int l2g_s[1024];
  __shared__ int col_off[1025];
  __shared__ int tmp16[16];
  __shared__ int bad;
  for (int l = tid; l < El; l += 1024) seen[l] = 0;
  if (tid == 0) bad = 0;
  __syncthreads();
  for (int e = tid; e < E; e += 1024) {
    const int l = e2l[e];
    if (l < -1 || l >= El) {
      atomicOr(&bad, 1);
    } else if (l >= 0) {
      atomicAdd(&seen[l], 1);
      l2g_s[l] = e;
    }
  }
  __syncthreads();
  for (int l = tid; l < El; l += 1024)
    if (seen[l] != 1) atomicOr(&bad, 1);
  __syncthreads();
  if (bad) {
    for (int l = tid; l <= El; l += 1024) {
      offsets[l] = 0;
      mtile_base[l] = 0;
      chunk_base[l] = 0;
    }
    if (tid == 0) {
      ctrl[kCtrlStatus] = MOE_EINVAL;
      ctrl[kCtrlN] = 0;
      ctrl[kCtrlMTiles] = 0;
      ctrl[kCtrlChunks] = 0;
    }
    return;
  }
  for (int l = tid; l < El; l += 1024) l2g[l] = l2g_s[l];

  // flattened (column, segment) exclusive scan: column c = local expert, segment q
  // = a run of histogram blocks.  Its value at (c, q) is offsets[c] plus all earlier
  // segments of column c, i.e. the base row of the segment's first block.
  int p2 = 1;
  while (p2 < El) p2 <<= 1;
  const int tpc = 1024 / p2;                 // threads per column (>= 1; El <= 1024)
  const int c = tid / tpc, q = tid - c * tpc;
  const int seg = (nb + tpc - 1) / tpc;
  const int b0 = q * seg, b1 = min(nb, b0 + seg);
  // a thread's segment of at most kSegRegs blocks is loaded once, all loads in flight
  // together, and kept in registers for the second pass
  constexpr int kSegRegs = 16;
  int hv[kSegRegs];
  int mysum = 0;
  const int col = (c < El) ? l2g_s[c] : 0;
  if (c < El) {
    if (seg <= kSegRegs) {
#pragma unroll
      for (int i = 0; i < kSegRegs; ++i) {
        const int b = b0 + i;
        hv[i] = (b < b1) ? blockhist[size_t(b) * E + col] : 0;
      }
#pragma unroll
      for (int i = 0; i < kSegRegs; ++i) mysum += hv[i];
    } else {
      for (int b = b0; b < b1; ++b) mysum += blockhist[size_t(b) * E + col];
    }
  }
  int N = 0;
  const int ex = block_excl_scan_1024(mysum, tmp16, &N);
  if (c < El) {
    int run = ex;
    if (seg <= kSegRegs) {
#pragma unroll
      for (int i = 0; i < kSegRegs; ++i) {
        const int b = b0 + i;
        if (b < b1) blockbase[size_t(b) * El + c] = run;
        run += hv[i];
      }
    } else {
      for (int b = b0; b < b1; ++b) {
        blockbase[size_t(b) * El + c] = run;
        run += blockhist[size_t(b) * E + col];
      }
    }
    if (q == 0) col_off[c] = ex;
  }
  if (tid == 0) col_off[El] = N;
  __syncthreads();
  for (int l = tid; l <= El; l += 1024) offsets[l] = col_off[l];

  // per-expert GEMM row tiles (bm rows) and minibatch chunks (mb rows)
  int cnt = (tid < El) ? col_off[tid + 1] - col_off[tid] : 0;
  int nt_total = 0, nc_total = 0;
  const int mt_ex = block_excl_scan_1024((cnt + bm - 1) / bm, tmp16, &nt_total);
  const int ch_ex = block_excl_scan_1024((cnt + mb - 1) / mb, tmp16, &nc_total);
  if (tid < El) {
    mtile_base[tid] = mt_ex;
    chunk_base[tid] = ch_ex;
  }
  if (tid == 0) {
    mtile_base[El] = nt_total;
    chunk_base[El] = nc_total;
    ctrl[kCtrlN] = N;
    ctrl[kCtrlMTiles] = nt_total;
    ctrl[kCtrlChunks] = nc_total;
    ctrl[kCtrlStatus] = MOE_OK;
  }
}

__global__ __launch_bounds__(64) void slot_assign_kernel(
    const int32_t* __restrict__ topk_idx, const int32_t* __restrict__ e2l, int R, int T, int E, int k,
    int El, const int32_t* __restrict__ blockbase, const int32_t* __restrict__ ctrl,
    int32_t* __restrict__ slot_of, int32_t* __restrict__ pull_src) {
  __shared__ int cnt[1024];
  __shared__ int map[1024];
  const int lane = threadIdx.x;
  for (int e = lane; e < E; e += 64) map[e] = e2l[e];
  for (int l = lane; l < El; l += 64) cnt[l] = 0;
  __syncthreads();
  const bool ok = ctrl[kCtrlStatus] == MOE_OK;
  const int64_t RT = int64_t(R) * T;
  const int64_t g0 = int64_t(blockIdx.x) * kTokPerLayoutBlock;
  const int64_t g1 = min(g0 + kTokPerLayoutBlock, RT);
  const int64_t p0 = g0 * k, p1 = g1 * k;
  const int nbits = 32 - __clz(El);          // bits of (l + 1) in [0, El]
  const int32_t* base = blockbase + size_t(blockIdx.x) * El;
  const unsigned long long below = (1ull << lane) - 1ull;

  for (int64_t pb = p0; pb < p1; pb += 64) {
    const int64_t p = pb + lane;
    const bool inr = p < p1;
    int l = -1;
    if (inr && ok) l = map[topk_idx[p]];
    const int key = l + 1;
    unsigned long long m = __ballot(l >= 0);
    for (int b = 0; b < nbits; ++b) {
      const bool bit = (key >> b) & 1;
      const unsigned long long bb = __ballot(bit);
      m &= bit ? bb : ~bb;
    }
    if (inr) {
      if (l >= 0) {
        const int slot = base[l] + cnt[l] + __popcll(m & below);
        slot_of[p] = slot;
        const int64_t g = p / k;
        const int r = int(g / T);
        pull_src[2 * int64_t(slot)] = r;
        pull_src[2 * int64_t(slot) + 1] = int(g - int64_t(r) * T);
      } else {
        slot_of[p] = -1;
      }
    }
    __syncthreads();
    if (l >= 0 && (m >> lane) == 1ull) cnt[l] += __popcll(m);
    __syncthreads();
  }
}

template <int VPL>
static void launch_topk(dim3 grid, hipStream_t st, const RankPtrs<const float*>& lp, const moe_shape_t& s,
                        int32_t* topk_idx, float* topk_w, int32_t* blockhist) {
  constexpr int NT = VPL <= 16 ? 1024 : 256;
  hipLaunchKernelGGL((topk_hist_kernel<VPL, NT>), grid, dim3(NT), 0, st, lp, s.R, s.T, s.E, s.k, topk_idx,
                     topk_w, blockhist);
}

hipError_t launch_layout(const moe_shape_t& s, const int32_t* e2l, int El, int mb,
                         const float* const* logits, int32_t* topk_idx, float* topk_w, int32_t* counts,
                         int32_t* offsets, int32_t* pull_src, int32_t* slot_of, char* ws,
                         const WsLayout& L, hipStream_t st) {
  RankPtrs<const float*> lp{};
  for (int r = 0; r < s.R; ++r) lp.p[r] = logits[r];
  int32_t* blockhist = reinterpret_cast<int32_t*>(ws + L.blockhist);
  int32_t* blockbase = reinterpret_cast<int32_t*>(ws + L.blockbase);
  int32_t* ctrl = reinterpret_cast<int32_t*>(ws + L.ctrl);
  const dim3 grid(L.nb);
  const int vpl_need = (s.E + 15) / 16;
  if (vpl_need <= 1) launch_topk<1>(grid, st, lp, s, topk_idx, topk_w, blockhist);
  else if (vpl_need <= 2) launch_topk<2>(grid, st, lp, s, topk_idx, topk_w, blockhist);
  else if (vpl_need <= 4) launch_topk<4>(grid, st, lp, s, topk_idx, topk_w, blockhist);
  else if (vpl_need <= 8) launch_topk<8>(grid, st, lp, s, topk_idx, topk_w, blockhist);
  else if (vpl_need <= 16) launch_topk<16>(grid, st, lp, s, topk_idx, topk_w, blockhist);
  else if (vpl_need <= 32) launch_topk<32>(grid, st, lp, s, topk_idx, topk_w, blockhist);
  else launch_topk<64>(grid, st, lp, s, topk_idx, topk_w, blockhist);

  const int bm = (s.dtype == MOE_F32) ? kF32BM : kGemmBM;
  hipLaunchKernelGGL(layout_scan_kernel, dim3(1 + (s.E + 63) / 64), dim3(1024), 0, st, e2l, s.E, El,
                     L.nb, bm, mb, blockhist, blockbase, counts, offsets,
                     reinterpret_cast<int32_t*>(ws + L.l2g), reinterpret_cast<int32_t*>(ws + L.mtile_base),
                     reinterpret_cast<int32_t*>(ws + L.chunk_base), ctrl);
  hipLaunchKernelGGL(slot_assign_kernel, grid, dim3(64), 0, st, topk_idx, e2l, s.R, s.T, s.E, s.k, El,
                     blockbase, ctrl, slot_of, pull_src);
  return hipGetLastError();
}

// ---------------------------------------------------------------------------
// Layout of given choices (any router; -1 = no expert).  Same outputs and tables as above.
//
// The choices are [R][T][k] in (r, t, j) order, so a block of consecutive pairs needs only how
// many pairs of each expert came before it.  At most kChoiceBlocks blocks, each at least
// 4096 pairs: choices_count_kernel writes every block's histogram, and choices_slots_kernel
// sums the blocks before its own (and all of them, for the offsets) itself, so there is no scan
// kernel between them; up to 4096 pairs one workgroup does it all in one launch.  Bound by the
// latency of its dependent steps and of fetching its code, not by bytes, so a wave holds its pairs'
// choices in registers through all phases where they are four groups of 64 (HELD; 262144 pairs: 5.8 +
// 9.8 us, reading them again 7.2 + 14.4), one match by ballots serves the checks and the places, and
// few pairs and experts take a workgroup of 256 threads, whose barriers are cheaper (512 pairs: 4.5
// us against 5.3 with 1024).  4096 pairs: 8.6 us.
// ---------------------------------------------------------------------------
constexpr int kChoiceBlocks = 128, kChoiceHeld = 4;

// the sum of this and all lower lanes: within rows of 16 lanes, then a row's last lane to the next
// row, then lane 31 to the upper half
__device__ __forceinline__ int wave_incl_scan(int x) {
  x += __builtin_amdgcn_update_dpp(0, x, 0x111, 0xF, 0xF, false);
  x += __builtin_amdgcn_update_dpp(0, x, 0x112, 0xF, 0xF, false);
  x += __builtin_amdgcn_update_dpp(0, x, 0x114, 0xF, 0xF, false);
  x += __builtin_amdgcn_update_dpp(0, x, 0x118, 0xF, 0xF, false);
  x += __builtin_amdgcn_update_dpp(0, x, 0x142, 0xA, 0xF, false);
  x += __builtin_amdgcn_update_dpp(0, x, 0x143, 0xC, 0xF, false);
  return x;
}

// exclusive prefixes over the block's first `waves` waves of three values at once, and their totals
// (the other waves' values are zero)
__device__ __forceinline__ void block_excl_scan3(const int (&v)[3], int (&ex)[3], int (&total)[3], int (*tmp)[16],
                                                 int waves) {
  const int lane = threadIdx.x & 63, w = threadIdx.x >> 6;
  if (w < waves) {
#pragma unroll
    for (int i = 0; i < 3; ++i) {
      const int x = wave_incl_scan(v[i]);
      if (lane == 63) tmp[i][w] = x;
      ex[i] = x - v[i];
    }
  }
  __syncthreads();
  if (w >= waves) return;
#pragma unroll
  for (int i = 0; i < 3; ++i) total[i] = 0;
  for (int q = 0; q < waves; ++q) {
#pragma unroll
    for (int i = 0; i < 3; ++i) {
      const int x = tmp[i][q];
      ex[i] += q < w ? x : 0;
      total[i] += x;
    }
  }
}

// A wave's run of whole 64-pair groups of a block's pairs [p0, p1)
struct PairRun {
  uint32_t begin, end;
};
template <int NT>
__device__ __forceinline__ PairRun wave_pairs(uint32_t p0, uint32_t p1) {
  const uint32_t run = ((p1 - p0 + NT - 1) / NT) * 64;
  const uint32_t b = p0 + (threadIdx.x >> 6) * run;
  return {b, min(p1, b + run)};
}

template <bool HELD>
__device__ __forceinline__ void hold(const int32_t* __restrict__ idx, const PairRun r, int (&held)[kChoiceHeld]) {
#pragma unroll
  for (int i = 0; i < kChoiceHeld; ++i) {
    const uint32_t p = r.begin + i * 64 + (threadIdx.x & 63);
    held[i] = HELD && p < r.end ? idx[p] : -1;
  }
}

// G groups of 64 pairs from pair pb on, this lane's choice of each in e (-1: none).  m: the lanes of a
// group that chose what this lane chose, by ballots over the bits of e.  A choice outside [-1, E) or,
// where `check`, an expert that a token names twice (the tables hold at most one row per token and
// expert) sets *wrong; the former becomes -1.
template <int G>
__device__ __forceinline__ void match_choices(const int32_t* __restrict__ idx, uint32_t pb, uint32_t end, int (&e)[G],
                                              int E, int k, unsigned long long (&m)[G], int* wrong, bool check) {
  const int lane = threadIdx.x & 63;
  bool bad = false;
#pragma unroll
  for (int i = 0; i < G; ++i) {
    if (e[i] < -1 || e[i] >= E) {
      bad = true;
      e[i] = -1;
    }
    m[i] = __ballot(e[i] >= 0);
  }
#pragma nounroll                             // executed once: short code costs less than its fetching
  for (int b = 32 - __clz(E - 1); --b >= 0;)
#pragma unroll
    for (int i = 0; i < G; ++i) {
      const bool bit = (e[i] >> b) & 1;
      const unsigned long long bb = __ballot(bit);
      m[i] &= bit ? bb : ~bb;
    }
  if (!check) {
    if (bad) *wrong = 1;
    return;
  }
  int j = int((pb + lane) % uint32_t(k));    // this lane's place in its token
  const int step = 64 % k;
  const unsigned long long token = (1ull << k) - 1ull;
#pragma unroll
  for (int i = 0; i < G; ++i) {
    const int first = lane - j;              // the lane of the token's first choice; in an earlier group if < 0
    const unsigned long long others = (first >= 0 ? token << first : token >> -first) & ~(1ull << lane);
    if (e[i] >= 0) {
      bad |= (m[i] & others) != 0;
      const uint32_t p = pb + i * 64 + lane;
      for (int o = lane + 1; o <= j; ++o) bad |= idx[p - o] == e[i];
    }
    j += step;
    if (j >= k) j -= k;
  }
  if (bad) *wrong = 1;
}

// adds a wave's run of pairs to hist; sets *wrong as above
template <bool HELD>
__device__ __forceinline__ void count_choices(const int32_t* __restrict__ idx, const PairRun r, int (&held)[kChoiceHeld],
                                              int E, int k, int* hist, int* wrong, bool check) {
  const int lane = threadIdx.x & 63;
  const unsigned long long below = (1ull << lane) - 1ull;
  if constexpr (HELD) {
    unsigned long long m[kChoiceHeld];
    match_choices<kChoiceHeld>(idx, r.begin, r.end, held, E, k, m, wrong, check);
#pragma unroll
    for (int i = 0; i < kChoiceHeld; ++i)
      if (held[i] >= 0 && !(m[i] & below)) atomicAdd(&hist[held[i]], __popcll(m[i]));
  } else {
    for (uint32_t pb = r.begin; pb < r.end; pb += 64) {
      int e[1] = {pb + lane < r.end ? idx[pb + lane] : -1};
      unsigned long long m[1];
      match_choices<1>(idx, pb, r.end, e, E, k, m, wrong, check);
      if (e[0] >= 0 && !(m[0] & below)) atomicAdd(&hist[e[0]], __popcll(m[0]));
    }
  }
}

// table[b][E + 1]: block b's histogram over the experts, then whether its choices are invalid
template <bool HELD>
__global__ __launch_bounds__(1024) void choices_count_kernel(const int32_t* __restrict__ idx, uint32_t P, uint32_t PB,
                                                             int E, int k, int32_t* __restrict__ table) {
  __shared__ int hist[1024];
  __shared__ int wrong;
  const uint32_t p0 = blockIdx.x * PB;
  const PairRun run = wave_pairs<1024>(p0, min(P, p0 + PB));
  int held[kChoiceHeld];
  hold<HELD>(idx, run, held);
  for (int e = threadIdx.x; e < E; e += 1024) hist[e] = 0;
  if (threadIdx.x == 0) wrong = 0;
  __syncthreads();
  count_choices<HELD>(idx, run, held, E, k, hist, &wrong, true);
  __syncthreads();
  int32_t* row = table + size_t(blockIdx.x) * (E + 1);
  for (int e = threadIdx.x; e < E; e += 1024) row[e] = hist[e];
  if (threadIdx.x == 0) row[E] = wrong;
}

// E <= MAXE, El <= NT.  A pair's slot = its expert's offset + the expert's pairs in earlier blocks
// (both in `total` after the scan) + in earlier waves and groups (cnt) + in earlier lanes.
template <int NT, int MAXE, bool HELD>
__global__ __launch_bounds__(NT) void choices_slots_kernel(
    const int32_t* __restrict__ idx, uint32_t P, uint32_t PB, const int32_t* __restrict__ e2l, int T, int E, int El,
    int k, int bm, int mb, const int32_t* __restrict__ table, int32_t* __restrict__ counts,
    int32_t* __restrict__ offsets, int32_t* __restrict__ l2g, int32_t* __restrict__ mtile_base,
    int32_t* __restrict__ chunk_base, int32_t* __restrict__ ctrl, int32_t* __restrict__ slot_of,
    int32_t* __restrict__ pull_src) {
  constexpr int kWaves = NT / 64;
  extern __shared__ int cnt[];               // [kWaves][E]: pairs of (wave, expert), then of those before them
  __shared__ int total[MAXE], before[MAXE];  // pairs of an expert: of all blocks, of earlier ones
  __shared__ int map[MAXE], seen[MAXE], home[MAXE];
  __shared__ int tmp[3][16];
  __shared__ int bad;
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int nb = gridDim.x, blk = blockIdx.x;
  const uint32_t p0 = blk * PB, p1 = min(P, p0 + PB);        // P < 2^31, PB a multiple of 64 * kWaves
  const PairRun run = wave_pairs<NT>(p0, p1);
  int held[kChoiceHeld];
  hold<HELD>(idx, run, held);
  int pe = 1;
  while (pe < E) pe <<= 1;
  const int per = NT / pe, ge = tid & (pe - 1);  // threads of one expert's column of the table (nb > 1: E <= 1024 = NT)
  int sum_all = 0, sum_before = 0, wrong = 0;
  if (nb > 1) {
    if (ge < E) {
#pragma unroll 8
      for (int b = tid / pe; b < nb; b += per) {
        const int v = table[size_t(b) * (E + 1) + ge];
        sum_all += v;
        sum_before += b < blk ? v : 0;
      }
    }
    for (int b = tid; b < nb; b += NT) wrong |= table[size_t(b) * (E + 1) + E];
  }
  for (int e = tid; e < E; e += NT) {
    total[e] = 0;
    before[e] = 0;
    map[e] = e2l[e];
    seen[e] = 0;
  }
  for (int i = tid; i < kWaves * E; i += NT) cnt[i] = 0;
  if (tid == 0) bad = 0;
  __syncthreads();
  for (int e = tid; e < E; e += NT) {
    const int l = map[e];
    if (l < -1 || l >= El) {
      bad = 1;
    } else if (l >= 0) {
      atomicAdd(&seen[l], 1);
      home[l] = e;
    }
  }
  // rank: a held pair's place among the wave's pairs of its expert.  The first lane that chose an expert
  // takes the places of all in its group from the wave's counter; the groups' counters are asked
  // for one after another (the LDS keeps a wave's order) before the first answer is needed.
  int* const mine = cnt + wave * E;
  const unsigned long long below = (1ull << lane) - 1ull;
  int rank[kChoiceHeld];
  if constexpr (HELD) {
    unsigned long long m[kChoiceHeld];
    int old[kChoiceHeld];
    match_choices<kChoiceHeld>(idx, run.begin, run.end, held, E, k, m, &bad, nb == 1);   // else checked by the count
#pragma unroll
    for (int i = 0; i < kChoiceHeld; ++i) {
      old[i] = 0;
      if (held[i] >= 0 && !(m[i] & below)) old[i] = atomicAdd(&mine[held[i]], __popcll(m[i]));
      __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");   // another lane may ask for the same counter next
    }
#pragma unroll
    for (int i = 0; i < kChoiceHeld; ++i)
      rank[i] = __shfl(old[i], held[i] >= 0 ? __builtin_ctzll(m[i]) : 0, 64) + __popcll(m[i] & below);
  } else {
    count_choices<false>(idx, run, held, E, k, mine, &bad, nb == 1);
  }
  if (nb > 1) {
    if (ge < E) {
      atomicAdd(&total[ge], sum_all);
      atomicAdd(&before[ge], sum_before);
    }
    if (wrong) bad = 1;
  }
  __syncthreads();
  for (int e = tid; e < E; e += NT) {
    int sum = 0;
#pragma unroll
    for (int w = 0; w < kWaves; ++w) {
      const int c = cnt[w * E + e];
      cnt[w * E + e] = sum;
      sum += c;
    }
    if (nb == 1) total[e] = sum;
  }
  if (tid < El && seen[tid] != 1) bad = 1;
  __syncthreads();
  if (bad) {                                 // nothing is local; slots say so
    for (uint32_t p = p0 + tid; p < p1; p += NT) slot_of[p] = -1;
    if (blk == 0) {
      for (int l = tid; l <= El; l += NT) {
        offsets[l] = 0;
        mtile_base[l] = 0;
        chunk_base[l] = 0;
      }
      if (tid == 0) {
        ctrl[kCtrlStatus] = MOE_EINVAL;
        ctrl[kCtrlN] = 0;
        ctrl[kCtrlMTiles] = 0;
        ctrl[kCtrlChunks] = 0;
      }
    }
    return;
  }
  const int e_of = tid < El ? home[tid] : 0;
  const int rows = tid < El ? total[e_of] : 0;
  if (blk == 0)
    for (int e = tid; e < E; e += NT) counts[e] = total[e];
  const int v[3] = {rows, (rows + bm - 1) / bm, (rows + mb - 1) / mb};
  int ex[3], all[3];                         // offsets, row tiles, chunks
  block_excl_scan3(v, ex, all, tmp, (El + 63) >> 6);     // its barrier: everyone has read total
  if (tid < El) {
    total[e_of] = ex[0] + before[e_of];
    if (blk == 0) {
      offsets[tid] = ex[0];
      l2g[tid] = e_of;
      mtile_base[tid] = ex[1];
      chunk_base[tid] = ex[2];
    }
  }
  if (blk == 0 && tid == 0) {
    offsets[El] = all[0];
    mtile_base[El] = all[1];
    chunk_base[El] = all[2];
    ctrl[kCtrlN] = all[0];
    ctrl[kCtrlMTiles] = all[1];
    ctrl[kCtrlChunks] = all[2];
    ctrl[kCtrlStatus] = MOE_OK;
  }
  __syncthreads();
  auto put = [&](uint32_t p, uint32_t t, int e, int rank_in_wave) {
    const int slot = e >= 0 && map[e] >= 0 ? total[e] + rank_in_wave : -1;
    if (p < run.end) slot_of[p] = slot;
    if (slot >= 0) {
      const uint32_t r = t / uint32_t(T);
      reinterpret_cast<int2*>(pull_src)[slot] = make_int2(int(r), int(t - r * uint32_t(T)));
    }
  };
  const uint32_t pl = run.begin + lane, tl = pl / uint32_t(k);
  uint32_t t = tl, j = pl - tl * uint32_t(k);                // pair pl is choice j of token t
  const uint32_t tstep = 64 / k, jstep = 64 % k;
  auto further = [&]() {
    t += tstep;
    j += jstep;
    if (j >= uint32_t(k)) {
      j -= k;
      ++t;
    }
  };
  if constexpr (HELD) {
#pragma unroll
    for (int i = 0; i < kChoiceHeld; ++i) {
      put(pl + i * 64, t, held[i], held[i] >= 0 ? mine[held[i]] + rank[i] : 0);
      further();
    }
  } else {
    for (uint32_t pb = run.begin; pb < run.end; pb += 64) {
      int e[1] = {pb + lane < run.end ? idx[pb + lane] : -1};
      unsigned long long m[1];
      match_choices<1>(idx, pb, run.end, e, E, k, m, &bad, false);
      int old = 0;
      if (e[0] >= 0 && !(m[0] & below)) old = atomicAdd(&mine[e[0]], __popcll(m[0]));
      old = __shfl(old, e[0] >= 0 ? __builtin_ctzll(m[0]) : 0, 64);
      put(pb + lane, t, e[0], old + __popcll(m[0] & below));
      further();
    }
  }
}

hipError_t launch_layout_choices(const moe_shape_t& s, const int32_t* e2l, int El, int mb, const int32_t* topk_idx,
                                 int32_t* counts, int32_t* offsets, int32_t* pull_src, int32_t* slot_of, char* ws,
                                 const WsLayout& L, hipStream_t st) {
  static std::atomic<uint64_t> attr_set{0};
  const hipError_t ea = once_per_device(attr_set, [] {
    hipError_t e = hipFuncSetAttribute(reinterpret_cast<const void*>(choices_slots_kernel<1024, 1024, true>),
                                       hipFuncAttributeMaxDynamicSharedMemorySize, 16 * 1024 * 4);
    if (e == hipSuccess)
      e = hipFuncSetAttribute(reinterpret_cast<const void*>(choices_slots_kernel<1024, 1024, false>),
                              hipFuncAttributeMaxDynamicSharedMemorySize, 16 * 1024 * 4);
    return e;
  });
  if (ea != hipSuccess) return ea;
  const int64_t P = int64_t(s.R) * s.T * s.k;
  int64_t PB = (P + kChoiceBlocks - 1) / kChoiceBlocks;
  const bool held = PB <= 1024 * kChoiceHeld;
  PB = held ? 1024 * kChoiceHeld : (PB + 1023) / 1024 * 1024;
  const int nb = int((P + PB - 1) / PB);
  // the histogram region holds E words for each of ceil(R T / 64) token blocks: with k <= 16 there
  // are at most a quarter as many pair blocks (of at least 4096 pairs, so of 256 tokens), rounded up
  int32_t* table = reinterpret_cast<int32_t*>(ws + L.blockhist);
  int32_t* ctrl = reinterpret_cast<int32_t*>(ws + L.ctrl);
  const int bm = (s.dtype == MOE_F32) ? kF32BM : kGemmBM;
  const uint32_t p = uint32_t(P), pb = uint32_t(PB);
  int32_t* l2g = reinterpret_cast<int32_t*>(ws + L.l2g);
  int32_t* mtb = reinterpret_cast<int32_t*>(ws + L.mtile_base);
  int32_t* chb = reinterpret_cast<int32_t*>(ws + L.chunk_base);
  if (P <= 256 * kChoiceHeld && s.E <= 256) {
    hipLaunchKernelGGL((choices_slots_kernel<256, 256, true>), dim3(1), dim3(256), size_t(4) * s.E * 4, st, topk_idx, p, pb,
                       e2l, s.T, s.E, El, s.k, bm, mb, table, counts, offsets, l2g, mtb, chb, ctrl, slot_of, pull_src);
  } else if (held) {
    if (nb > 1)
      hipLaunchKernelGGL(choices_count_kernel<true>, dim3(nb), dim3(1024), 0, st, topk_idx, p, pb, s.E, s.k, table);
    hipLaunchKernelGGL((choices_slots_kernel<1024, 1024, true>), dim3(nb), dim3(1024), size_t(16) * s.E * 4, st, topk_idx, p,
                       pb, e2l, s.T, s.E, El, s.k, bm, mb, table, counts, offsets, l2g, mtb, chb, ctrl, slot_of, pull_src);
  } else {
    hipLaunchKernelGGL(choices_count_kernel<false>, dim3(nb), dim3(1024), 0, st, topk_idx, p, pb, s.E, s.k, table);
    hipLaunchKernelGGL((choices_slots_kernel<1024, 1024, false>), dim3(nb), dim3(1024), size_t(16) * s.E * 4, st, topk_idx, p,
                       pb, e2l, s.T, s.E, El, s.k, bm, mb, table, counts, offsets, l2g, mtb, chb, ctrl, slot_of, pull_src);
  }
  return hipGetLastError();
}

}  // namespace moe
