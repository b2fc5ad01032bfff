// Products grouped by expert with ragged row counts, for experts of any form:
//   y[s] = x[s] W_g^T (W_g stored [N][K]) or x[s] W_g (stored [K][N]) for the rows s of group g;
//   dW_g = sum over s of dy[s]^T x[s] (or its transpose), the gradient by the weights.
// The gradient by the rows is the first product in the weights' other orientation.
#include "grouped.hpp"
#include "grouped_mid.hpp"
#include "grouped_thin.hpp"
#include "grouped_tile.hpp"

namespace moe {

// fp32, on the fp32 MFMA (v_mfma_f32_32x32x2_f32): a TB x TB tile of C = A B^T, A and B each stored with K contiguous (element (r, k) at
// r * ld + k) or with the row index contiguous (at k * ld + r), by 256 threads.  TB 64: wave w owns the 32 x 32 block (w >> 1, w & 1).  TB 32:
// the four waves share the block's K and add up through LDS in wave order, for so few tiles that 64 x 64 would leave most of the card
// idle (64 MFMAs of 64 cycles a wave and step: half of what a tiny product takes).  K goes by steps of 128 through LDS, in the order it is
// stored in (rows padded so that 64 lanes' reads touch all banks), and the next step's loads are on their way in registers while one is
// at work: small products are a chain of such round trips.  us with TB 32 and 64: 8 groups of 512 x 512, 512 rows (64 tiles of 64) 8.6 and 16.2,
// 512 x 1024, 1024 rows (256 tiles, as many as CUs) 19.4 and 18.1, 16 groups of 1024 x 1024, 4096 rows 109 and 86 (100 TFLOP/s).
constexpr int kF32Step = 128, kF32PitchK = kF32Step + 4;
constexpr int f32_panel(int tb) { return kF32Step * (tb + 8) > tb * kF32PitchK ? kF32Step * (tb + 8) : tb * kF32PitchK; }   // values
constexpr int f32_lds_bytes(int tb) { return 2 * f32_panel(tb) * 4; }

struct F32Operand {
  const float* p;
  int64_t ld;
  int rows;                    // valid ones of the tile
};

template <int TB, bool MN>
struct F32Fill {
  static constexpr int kVecs = TB * kF32Step / 4 / 256, kPitchR = TB + 8, kPerRow = TB / 4;
  f32x4 v[kVecs];              // a thread's share of a step

  // from k0 on, zeros past `left` values of K and past the rows (multiples of 4 along the contiguous axis)
  __device__ __forceinline__ void load(const F32Operand& o, int k0, int left) {
#pragma unroll
    for (int i = 0; i < kVecs; ++i) {
      const int t = threadIdx.x + i * 256;
      const int r = MN ? t % kPerRow * 4 : t >> 5, k = MN ? t / kPerRow : (t & 31) * 4;
      v[i] = f32x4{0, 0, 0, 0};
      if (r < o.rows && k < left)
        v[i] = *reinterpret_cast<const f32x4*>(o.p + (MN ? int64_t(k0 + k) * o.ld + r : int64_t(r) * o.ld + k0 + k));
    }
  }
  __device__ __forceinline__ void put(float* lds) const {
#pragma unroll
    for (int i = 0; i < kVecs; ++i) {
      const int t = threadIdx.x + i * 256;
      *reinterpret_cast<f32x4*>(lds + (MN ? t / kPerRow * kPitchR + t % kPerRow * 4 : (t >> 5) * kF32PitchK + (t & 31) * 4)) = v[i];
    }
  }
  // lane's four K values of row r: k = 8 c + 4 hi + 0..3
  static __device__ __forceinline__ f32x4 frag(const float* lds, int r, int c, int hi) {
    if constexpr (!MN) return *reinterpret_cast<const f32x4*>(lds + r * kF32PitchK + c * 8 + hi * 4);
    const float* q = lds + (c * 8 + hi * 4) * kPitchR + r;
    return f32x4{q[0], q[kPitchR], q[2 * kPitchR], q[3 * kPitchR]};
  }
};

// out(row, column, value) of the tile's valid values
template <int TB, bool A_MN, bool B_MN, typename OUT>
__device__ __forceinline__ void f32_tile(const F32Operand& A, const F32Operand& B, int K, float* smem, OUT out) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int wm = TB == 64 ? wave >> 1 : 0, wn = TB == 64 ? wave & 1 : 0, r32 = lane & 31, hi = lane >> 5;
  float *sa = smem, *sb = smem + f32_panel(TB);
  f32x16 acc;
#pragma unroll
  for (int e = 0; e < 16; ++e) acc[e] = 0.0f;
  F32Fill<TB, A_MN> fa;
  F32Fill<TB, B_MN> fb;
  fa.load(A, 0, K);
  fb.load(B, 0, K);
  for (int k0 = 0; k0 < K; k0 += kF32Step) {
    fa.put(sa);
    fb.put(sb);
    __syncthreads();
    fa.load(A, k0 + kF32Step, K - k0 - kF32Step);
    fb.load(B, k0 + kF32Step, K - k0 - kF32Step);
    const int steps = min(kF32Step, K - k0 + 7) >> 3;
    for (int c = TB == 64 ? 0 : wave; c < steps; c += TB == 64 ? 1 : 4) {
      const f32x4 a = F32Fill<TB, A_MN>::frag(sa, wm * 32 + r32, c, hi);
      const f32x4 b = F32Fill<TB, B_MN>::frag(sb, wn * 32 + r32, c, hi);
#pragma unroll
      for (int s = 0; s < 4; ++s) acc = __builtin_amdgcn_mfma_f32_32x32x2f32(a[s], b[s], acc, 0, 0, 0);
    }
    __syncthreads();                         // the next step overwrites these
  }
  // lane holds column r32 and rows 8 (e / 4) + 4 hi + e % 4 of its block
  if constexpr (TB == 64) {
    const int col = wn * 32 + r32;
#pragma unroll
    for (int e = 0; e < 16; ++e) {
      const int row = wm * 32 + 8 * (e >> 2) + 4 * hi + (e & 3);
      if (row < A.rows && col < B.rows) out(row, col, acc[e]);
    }
  } else {
#pragma unroll
    for (int e = 0; e < 16; ++e) smem[(wave * 16 + e) * 64 + lane] = acc[e];
    __syncthreads();
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int e = wave * 4 + j, row = 8 * wave + 4 * hi + j;
      float t = smem[e * 64 + lane];
#pragma unroll
      for (int w = 1; w < 4; ++w) t += smem[(w * 16 + e) * 64 + lane];
      if (row < A.rows && r32 < B.rows) out(row, r32, t);
    }
    __syncthreads();
  }
}

template <int TB, bool W_KN>
__global__ __launch_bounds__(256) void grouped_f32_kernel(GroupedArgs g) {
  extern __shared__ __attribute__((aligned(16))) char smem[];
  __shared__ int32_t base[kMaxGroups + 1], part[5];
  bool bad;
  const int mtiles = group_tiles<256>(g.offsets, g.G, g.rows, TB == 64 ? 6 : 5, base, part, &bad);
  if (g.status && blockIdx.x == 0 && threadIdx.x == 0) *g.status = bad ? MOE_EINVAL : MOE_OK;
  const int NT = (g.N + TB - 1) / TB;
  const int64_t total = int64_t(mtiles) * NT;
  for (int64_t tau = blockIdx.x; tau < total; tau += gridDim.x) {
    const int mtg = int(tau / NT), nt = int(tau - int64_t(mtg) * NT);
    const int l = find_expert(base, g.G, mtg);
    const int64_t row0 = g.offsets[l] + int64_t(mtg - base[l]) * TB;
    const int rows = int(min(int64_t(TB), g.offsets[l + 1] - row0));
    const int c0 = nt * TB, cols = min(TB, g.N - c0);
    const float* w = static_cast<const float*>(g.w) + int64_t(l) * g.N * g.K;
    const F32Operand A{static_cast<const float*>(g.x) + row0 * g.ldx, g.ldx, rows};
    const F32Operand B{W_KN ? w + c0 : w + int64_t(c0) * g.K, W_KN ? g.N : g.K, cols};
    float* y = static_cast<float*>(g.y) + row0 * g.ldy + c0;
    f32_tile<TB, false, W_KN>(A, B, g.K, reinterpret_cast<float*>(smem), [&](int r, int c, float v) { y[r * g.ldy + c] = v; });
  }
}

// fp32 products of few rows and columns (a latency): tiles of 16 x 16 (v_mfma_f32_16x16x4_f32), whose K sixteen waves share, 16 values at a time straight into
// registers, four such loads in flight, and add up through LDS in wave order.
template <bool W_KN>
__global__ __launch_bounds__(1024) void grouped_f32_thin_kernel(GroupedArgs g) {
  __shared__ int32_t base[kMaxGroups + 1], part[17];
  __shared__ f32x4 sums[16][64];
  bool bad;
  const int mtiles = group_tiles<1024>(g.offsets, g.G, g.rows, 4, base, part, &bad);
  if (g.status && blockIdx.x == 0 && threadIdx.x == 0) *g.status = bad ? MOE_EINVAL : MOE_OK;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, r16 = lane & 15, q = lane >> 4;
  const int NT = (g.N + 15) >> 4;
  const int64_t total = int64_t(mtiles) * NT;
  for (int64_t tau = blockIdx.x; tau < total; tau += gridDim.x) {
    const int mtg = int(tau / NT), c0 = int(tau - int64_t(mtg) * NT) * 16;
    const int l = find_expert(base, g.G, mtg);
    const int64_t row0 = g.offsets[l] + int64_t(mtg - base[l]) * 16;
    const int rows = int(min(int64_t(16), g.offsets[l + 1] - row0));
    const float* x = static_cast<const float*>(g.x) + (row0 + min(r16, rows - 1)) * g.ldx;
    const int64_t c = min(c0 + r16, g.N - 1);
    const float* w = static_cast<const float*>(g.w) + int64_t(l) * g.N * g.K + (W_KN ? c : c * g.K);
    f32x4 acc{0, 0, 0, 0};
    for (int k0 = wave * 16 + q * 4; k0 - q * 4 < g.K; k0 += 1024) {
      f32x4 a[4], b[4];
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        const int k = min(k0 + u * 256, g.K - 4);             // past K: some values of the row, which become zeros
        b[u] = *reinterpret_cast<const f32x4*>(x + k);
        if constexpr (W_KN) {
          const float* p = w + int64_t(k) * g.N;
          a[u] = f32x4{p[0], p[g.N], p[2 * int64_t(g.N)], p[3 * int64_t(g.N)]};
        } else {
          a[u] = *reinterpret_cast<const f32x4*>(w + k);
        }
      }
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        const bool in = k0 + u * 256 < g.K;
#pragma unroll
        for (int e = 0; e < 4; ++e)                            // columns first: a lane gets four of them of one row
          acc = __builtin_amdgcn_mfma_f32_16x16x4f32(in ? a[u][e] : 0.0f, in ? b[u][e] : 0.0f, acc, 0, 0, 0);
      }
    }
    sums[wave][lane] = acc;
    __syncthreads();
    if (threadIdx.x < 64 && r16 < rows && c0 + 4 * q < g.N) {
#pragma unroll
      for (int v = 1; v < 16; ++v) acc += sums[v][lane];
      *reinterpret_cast<f32x4*>(static_cast<float*>(g.y) + (row0 + r16) * g.ldy + c0 + 4 * q) = acc;
    }
    __syncthreads();
  }
}

struct WgradArgs {
  const void* a;               // the rows whose columns become the gradient's rows
  const void* b;
  void* dw;                    // [G][M][N]
  const int32_t* offsets;
  int32_t* status;
  int64_t rows, lda, ldb;
  int G, M, N;
  const int32_t* used;         // null, or where the number of groups is (at most G)
};

template <int TB, bool ADD>
__global__ __launch_bounds__(256) void grouped_f32_wgrad_kernel(WgradArgs g) {
  extern __shared__ __attribute__((aligned(16))) char smem[];
  __shared__ int32_t base[kMaxGroups + 1], part[5];
  bool bad;
  if (g.used) g.G = *g.used;
  group_tiles<256>(g.offsets, g.G, g.rows, 6, base, part, &bad);
  if (g.status && blockIdx.x == 0 && threadIdx.x == 0) *g.status = bad ? MOE_EINVAL : MOE_OK;
  if (bad) return;
  const int MT = (g.M + TB - 1) / TB, NT = (g.N + TB - 1) / TB;
  const int64_t total = int64_t(g.G) * MT * NT;
  for (int64_t tau = blockIdx.x; tau < total; tau += gridDim.x) {
    const int l = int(tau / (int64_t(MT) * NT));
    const int rem = int(tau - int64_t(l) * MT * NT);
    const int m0 = (rem % MT) * TB, c0 = (rem / MT) * TB;
    const int64_t r0 = g.offsets[l];
    const int n = int(g.offsets[l + 1] - r0);
    const F32Operand A{static_cast<const float*>(g.a) + r0 * g.lda + m0, g.lda, min(TB, g.M - m0)};
    const F32Operand B{static_cast<const float*>(g.b) + r0 * g.ldb + c0, g.ldb, min(TB, g.N - c0)};
    float* dw = static_cast<float*>(g.dw) + (int64_t(l) * g.M + m0) * g.N + c0;
    f32_tile<TB, true, true>(A, B, n, reinterpret_cast<float*>(smem), [&](int r, int c, float v) {
      if constexpr (ADD) dw[int64_t(r) * g.N + c] += v;
      else dw[int64_t(r) * g.N + c] = v;
    });
  }
}

// 256 x 256 tiles in bf16 (grouped_tile.hpp): the list of all tiles is cut into eight contiguous ranges, one for an XCD (workgroup w
// runs on XCD w mod 8), by group, then as big_place says.  A workgroup takes every 32nd tile of its XCD's range, 64 at a
// time: lane i of each wave looks up the i-th and keeps it.
template <int T, bool W_KN, bool CUT>
struct BigProducts {
  static constexpr int kCut = CUT, kAt = T == 256 ? 18 : 17;   // rows - 1 take 8 bits or 7
  const GroupedArgs& g;
  uint32_t what;                 // this lane's tile: group | (rows - 1) << 10 | column tile << kAt
  int32_t row0;
  int n;

  __device__ __forceinline__ uint32_t w_(int i) const { return uint32_t(__builtin_amdgcn_readlane(int(what), i)); }
  __device__ __forceinline__ int count() const { return n; }
  __device__ __forceinline__ int K(int) const { return g.K; }
  __device__ __forceinline__ int rows(int i) const { return int((w_(i) >> 10) & (T - 1)) + 1; }
  __device__ __forceinline__ int cols(int i) const { return min(T, g.N - int(w_(i) >> kAt) * T); }
  __device__ __forceinline__ BigOperand a(int i) const {
    return BigOperand{static_cast<const uint16_t*>(g.x) + int64_t(__builtin_amdgcn_readlane(row0, i)) * g.ldx, g.ldx, rows(i)};
  }
  __device__ __forceinline__ BigOperand b(int i) const {
    const int c0 = int(w_(i) >> kAt) * T;
    const uint16_t* w = static_cast<const uint16_t*>(g.w) + int64_t(w_(i) & 1023) * g.N * g.K;
    return BigOperand{W_KN ? w + c0 : w + int64_t(c0) * g.K, W_KN ? g.N : g.K, cols(i)};
  }
  template <typename WALK>
  __device__ __forceinline__ void store(int i, const WALK& walk) const {
    big_store<uint16_t, false, false>(walk, static_cast<uint16_t*>(g.y) + int64_t(__builtin_amdgcn_readlane(row0, i)) * g.ldy +
                               int(w_(i) >> kAt) * T, g.ldy, rows(i), cols(i));
  }
};

template <int T, int THREADS, bool W_KN, bool CUT>
__device__ __forceinline__ void grouped_tiles(const GroupedArgs& g, char* smem) {
  const int NT = (g.N + T - 1) / T;
  const int xcd = blockIdx.x & 7, wg_per_xcd = gridDim.x >> 3, lane = threadIdx.x & 63;
  int32_t* base = reinterpret_cast<int32_t*>(smem);
  int64_t per_xcd = int64_t(1) << 40;     // known after the first look at the offsets
  for (int64_t t0 = blockIdx.x >> 3; t0 < per_xcd; t0 += 64 * int64_t(wg_per_xcd)) {
    bool bad;
    const int mtiles = group_tiles<THREADS>(g.offsets, g.G, g.rows, T == 256 ? 8 : 7, base, base + kMaxGroups + 8, &bad);
    if (g.status && blockIdx.x == 0 && threadIdx.x == 0) *g.status = bad ? MOE_EINVAL : MOE_OK;
    const int64_t total = int64_t(mtiles) * NT;
    per_xcd = (total + 7) >> 3;
    const int64_t tt = t0 + int64_t(lane) * wg_per_xcd, tau = xcd * per_xcd + tt;
    BigProducts<T, W_KN, CUT> tiles{g, 0, 0, 0};
    const bool mine = tt < per_xcd && tau < total;
    if (mine) {
      const int l = find_expert(base, g.G, int(tau / NT));
      int mt, nt;
      big_place(tau - int64_t(base[l]) * NT, base[l + 1] - base[l], NT, &mt, &nt);
      tiles.row0 = g.offsets[l] + mt * T;
      tiles.what = uint32_t(l) | uint32_t(min(T, g.offsets[l + 1] - tiles.row0) - 1) << 10 | uint32_t(nt) << tiles.kAt;
    }
    tiles.n = __popcll(__ballot(mine));
    __syncthreads();                      // the tables' LDS becomes the ring's
    if constexpr (T == 256) {
      BigWalk<false, W_KN, BigProducts<T, W_KN, CUT>> walk(tiles, smem);
      walk.run();
    } else {
      MidWalk<false, W_KN, BigProducts<T, W_KN, CUT>> walk;
      walk.run(tiles, smem);
    }
    __syncthreads();
  }
}

template <bool W_KN, bool CUT>
__global__ __launch_bounds__(kBigThreads, 2) void grouped_big_kernel(GroupedArgs g) {
  extern __shared__ __attribute__((aligned(16))) char smem[];
  grouped_tiles<256, kBigThreads, W_KN, CUT>(g, smem);
}
template <bool W_KN>
__global__ __launch_bounds__(kMidThreads, 1) void grouped_mid_kernel(GroupedArgs g) {
  extern __shared__ __attribute__((aligned(16))) char smem[];
  grouped_tiles<128, kMidThreads, W_KN, true>(g, smem);
}

// The same for the gradient by the weights: a tile of 256 x 256 of one group's gradient sums over the group's rows.
template <int T, typename O, bool ADD>
struct BigGradients {
  static constexpr int kCut = 2;
  const WgradArgs& g;
  uint32_t gm;                   // this lane's tile: group | row tile << 10
  int32_t nt, r0, k;             // its column tile, its group's first row and rows
  int n;

  __device__ __forceinline__ int group(int i) const { return __builtin_amdgcn_readlane(int(gm), i) & 1023; }
  __device__ __forceinline__ int m0(int i) const { return int(uint32_t(__builtin_amdgcn_readlane(int(gm), i)) >> 10) * T; }
  __device__ __forceinline__ int c0(int i) const { return __builtin_amdgcn_readlane(nt, i) * T; }
  __device__ __forceinline__ int count() const { return n; }
  __device__ __forceinline__ int K(int i) const { return __builtin_amdgcn_readlane(k, i); }
  __device__ __forceinline__ int64_t first(int i) const { return __builtin_amdgcn_readlane(r0, i); }
  __device__ __forceinline__ int rows(int i) const { return min(T, g.M - m0(i)); }
  __device__ __forceinline__ int cols(int i) const { return min(T, g.N - c0(i)); }
  __device__ __forceinline__ BigOperand a(int i) const {
    return BigOperand{static_cast<const uint16_t*>(g.a) + first(i) * g.lda + m0(i), g.lda, rows(i)};
  }
  __device__ __forceinline__ BigOperand b(int i) const {
    return BigOperand{static_cast<const uint16_t*>(g.b) + first(i) * g.ldb + c0(i), g.ldb, cols(i)};
  }
  template <typename WALK>
  __device__ __forceinline__ void store(int i, const WALK& walk) const {
    big_store<O, ADD, true>(walk, static_cast<O*>(g.dw) + (int64_t(group(i)) * g.M + m0(i)) * g.N + c0(i), g.N, rows(i), cols(i));
  }
};

constexpr int kTileSteps = 3;            // what a tile's stores take, in steps
template <int T, int THREADS, typename O, bool ADD>
__device__ __forceinline__ void grouped_gradients(WgradArgs& g, char* smem) {
  int32_t* base = reinterpret_cast<int32_t*>(smem);
  bool bad;
  if (g.used) g.G = *g.used;
  group_tiles<THREADS>(g.offsets, g.G, g.rows, 6, base, base + kMaxGroups + 8, &bad);
  if (g.status && blockIdx.x == 0 && threadIdx.x == 0) *g.status = bad ? MOE_EINVAL : MOE_OK;
  if (bad || g.G == 0) return;
  __syncthreads();
  const int MT = (g.M + T - 1) / T, NT = (g.N + T - 1) / T, per_group = MT * NT;
  // Every XCD gets consecutive tiles of an eighth of the work, by the K steps of 64 that its groups' rows make.
  auto ahead = [&](int l) { return int64_t(per_group) * (base[l] + kTileSteps * l); };
  auto tile_at = [&](int64_t work) -> int64_t {
    int l = 0;
    for (int hi = g.G - 1; l < hi;) {
      const int mid = (l + hi + 1) >> 1;
      if (ahead(mid) <= work) l = mid;
      else hi = mid - 1;
    }
    const int64_t one = base[l + 1] - base[l] + kTileSteps, in = (work - ahead(l) + one - 1) / one;
    return int64_t(l) * per_group + (in < per_group ? in : per_group);
  };
  const int xcd = blockIdx.x & 7, wg_per_xcd = gridDim.x >> 3, lane = threadIdx.x & 63;
  const int64_t work = ahead(g.G), first = tile_at(work * xcd / 8), past = tile_at(work * (xcd + 1) / 8);
  __syncthreads();                        // the tables' LDS becomes the ring's
  for (int64_t t0 = first + (blockIdx.x >> 3); t0 < past; t0 += 64 * int64_t(wg_per_xcd)) {
    const int64_t tau = t0 + int64_t(lane) * wg_per_xcd;
    const bool mine = tau < past;
    int l = 0, mt = 0, nt = 0, r0 = 0, rows = 0;
    if (mine) {
      l = int(tau / per_group);
      // Bands over the longer axis: 32 groups of about 512 rows, 7168 x 2048 545 us, 2048 x 7168 544, over the shorter one 649 and 677; as long: the same
      if (MT >= NT) big_place(tau - int64_t(l) * per_group, MT, NT, &mt, &nt);
      else big_place(tau - int64_t(l) * per_group, NT, MT, &nt, &mt);
      r0 = g.offsets[l];
      rows = g.offsets[l + 1] - r0;
    }
    const uint64_t full = __ballot(mine && rows > 0), empty = __ballot(mine && rows == 0);
    // tiles of groups with rows first in the lanes' order, the others behind them get zeros
    const uint64_t below = (uint64_t(1) << lane) - 1;
    const int to = rows > 0 ? __popcll(full & below) : mine ? __popcll(full) + __popcll(empty & below) : 63;
    BigGradients<T, O, ADD> tiles{g, 0, 0, 0, 0, int(__popcll(full))};
    if (full | empty) {
      tiles.gm = uint32_t(__builtin_amdgcn_ds_permute(to * 4, mine ? int(uint32_t(l) | uint32_t(mt) << 10) : 0));
      tiles.nt = __builtin_amdgcn_ds_permute(to * 4, nt);
      tiles.r0 = __builtin_amdgcn_ds_permute(to * 4, r0);
      tiles.k = __builtin_amdgcn_ds_permute(to * 4, rows);
    }
    if constexpr (!ADD) {
      for (int i = tiles.n; i < tiles.n + int(__popcll(empty)); ++i) {
        O* out = static_cast<O*>(g.dw) + (int64_t(tiles.group(i)) * g.M + tiles.m0(i)) * g.N + tiles.c0(i);
        constexpr int V = 16 / sizeof(O);
        for (int v = threadIdx.x; v < T * (T / V); v += THREADS) {
          const int row = v / (T / V), col = v % (T / V) * V;
          if (row < tiles.rows(i) && col < tiles.cols(i))
            *reinterpret_cast<u32x4*>(out + int64_t(row) * g.N + col) = u32x4{0, 0, 0, 0};
        }
      }
    }
    if constexpr (T == 256) {
      BigWalk<true, true, BigGradients<T, O, ADD>> walk(tiles, smem);
      walk.run();
    } else {
      MidWalk<true, true, BigGradients<T, O, ADD>> walk;
      walk.run(tiles, smem);
    }
    __syncthreads();
  }
}

template <typename O, bool ADD>
__global__ __launch_bounds__(kBigThreads, 2) void grouped_big_wgrad_kernel(WgradArgs g) {
  extern __shared__ __attribute__((aligned(16))) char smem[];
  grouped_gradients<256, kBigThreads, O, ADD>(g, smem);
}
template <typename O, bool ADD>
__global__ __launch_bounds__(kMidThreads, 1) void grouped_mid_wgrad_kernel(WgradArgs g) {
  extern __shared__ __attribute__((aligned(16))) char smem[];
  grouped_gradients<128, kMidThreads, O, ADD>(g, smem);
}

// the dynamic LDS that each kernel asks for, granted once per device
static hipError_t set_grouped_lds() {
  static std::atomic<uint64_t> done{0};
  return once_per_device(done, [] {
    const struct {
      const void* k;
      int bytes;
    } ks[] = {{reinterpret_cast<const void*>(grouped_big_kernel<false, false>), kBigLds},
              {reinterpret_cast<const void*>(grouped_big_kernel<false, true>), kBigLds},
              {reinterpret_cast<const void*>(grouped_big_kernel<true, false>), kBigLds},
              {reinterpret_cast<const void*>(grouped_big_kernel<true, true>), kBigLds},
              {reinterpret_cast<const void*>(grouped_big_wgrad_kernel<uint16_t, false>), kBigLds},
              {reinterpret_cast<const void*>(grouped_big_wgrad_kernel<float, false>), kBigLds},
              {reinterpret_cast<const void*>(grouped_big_wgrad_kernel<float, true>), kBigLds},
              {reinterpret_cast<const void*>(grouped_mid_kernel<false>), kMidLds},
              {reinterpret_cast<const void*>(grouped_mid_kernel<true>), kMidLds},
              {reinterpret_cast<const void*>(grouped_mid_wgrad_kernel<uint16_t, false>), kMidLds},
              {reinterpret_cast<const void*>(grouped_mid_wgrad_kernel<float, false>), kMidLds},
              {reinterpret_cast<const void*>(grouped_mid_wgrad_kernel<float, true>), kMidLds},
              {reinterpret_cast<const void*>(grouped_f32_kernel<32, false>), f32_lds_bytes(32)},
              {reinterpret_cast<const void*>(grouped_f32_kernel<32, true>), f32_lds_bytes(32)},
              {reinterpret_cast<const void*>(grouped_f32_kernel<64, false>), f32_lds_bytes(64)},
              {reinterpret_cast<const void*>(grouped_f32_kernel<64, true>), f32_lds_bytes(64)},
              {reinterpret_cast<const void*>(grouped_f32_wgrad_kernel<32, false>), f32_lds_bytes(32)},
              {reinterpret_cast<const void*>(grouped_f32_wgrad_kernel<32, true>), f32_lds_bytes(32)},
              {reinterpret_cast<const void*>(grouped_f32_wgrad_kernel<64, false>), f32_lds_bytes(64)},
              {reinterpret_cast<const void*>(grouped_f32_wgrad_kernel<64, true>), f32_lds_bytes(64)},
              {reinterpret_cast<const void*>(grouped_thin_kernel<false>), kThinLds},
              {reinterpret_cast<const void*>(grouped_thin_kernel<true>), kThinLds}};
    for (const auto& k : ks) {
      const hipError_t e = hipFuncSetAttribute(k.k, hipFuncAttributeMaxDynamicSharedMemorySize, k.bytes);
      if (e != hipSuccess) return e;
    }
    return hipSuccess;
  });
}

// How a bf16 product goes.  us streaming the weights past the rows, with tiles of 128 and of 256 (weights stored [K][N] in brackets):
// - up to 24 rows a group on the mean, streaming: 32 groups of 7168 x 2048, 16 rows a group 149, -, 169; 24 rows 181, -, 170 (163, -, 211;
//   177, -, 214); 32 rows 198, -, 171 (213, -, 216).
// - where the tiles of 256 take no more than half of the CUs, streaming up to 4096 outputs a CU: 512 x 2048 x 2048 16, 27, 44 (22, 30, 47), 8 groups,
//   256 x 2048 x 1408 13, 26, 27 (19, 26, 27), 2000 x 2048 x 1408 60, 28, 46.
// - past those, tiles of 128: 2048 x 2048 x 2048 52, 29, 47 (70, 40, 49), 8 groups, 1024 x 7168 x 2048 160, 79, 131.  Weights stored [K][N] take
//   two LDS reads for one there, and the tiles may be a third of the CUs (8 groups, 2000 x 1408 x 2048, 120 tiles: (69, 48, 38)).
// - tiles of 256 else: 8 groups, 8000 x 2048 x 1408 140, 75, 52 (204, 118, 72).
enum class Rows { kThin, kMid, kBig };
static Rows rows_way(const moe_gemm_t& s, int cus) {
  if (s.rows <= int64_t(s.groups) * 24) return Rows::kThin;
  const int64_t tiles = (s.rows / kBig + s.groups) * ((s.N + kBig - 1) / kBig);        // at most
  if (tiles * 2 > cus) return Rows::kBig;
  if (s.rows * s.N <= int64_t(cus) * 4096) return Rows::kThin;
  return s.w_layout && tiles * 3 > cus ? Rows::kBig : Rows::kMid;
}

// fp32 workgroups for at most `tiles` tiles of 64 x 64 (four times as many of 32 x 32 where they are fewer than the CUs)
static int f32_grid(int64_t tiles, int cus) {
  const int64_t n = tiles < cus ? tiles * 4 : tiles;
  return int(n < 1 ? 1 : n < cus * 2 ? n : cus * 2);
}

hipError_t launch_grouped(const moe_gemm_t& s, const void* x, const void* w, const int32_t* offsets, void* y,
                          int32_t* status, int cus, hipStream_t st) {
  const GroupedArgs g{x, w, y, offsets, status, s.rows, s.ldx ? s.ldx : s.K, s.ldy ? s.ldy : s.N, s.groups, s.K, s.N};
  const dim3 threads(256);
  const hipError_t e = set_grouped_lds();
  if (e != hipSuccess) return e;
  if (s.dtype == MOE_F32) {
    const int64_t rows = s.rows / 64 + (s.rows < s.groups ? s.rows : s.groups), tiles = rows * ((s.N + 63) / 64);     // at most
    const int64_t small = (s.rows / 16 + (s.rows < s.groups ? s.rows : s.groups)) * ((s.N + 15) / 16);                 // tiles of 16 x 16
    // us with those and with tiles of 32: 5 groups, 5 rows of 7108 x 96 (30) 16 and 58; 1 group, 80 rows of 6652 x 212 (84) 23 and 55; 35 groups, 2 rows of
    // 4244 x 848 (106) 12 and 37; 64 groups, 64 rows of 2048 x 128 (544) 17 and 23, weights stored [K][N] 25 and 23; 8 groups, 509 rows of 256 x 128
    // (312) 11 and 7
    if (small <= cus && s.K >= 512) {
      const dim3 few(int(small < 1 ? 1 : small));
      if (s.w_layout) hipLaunchKernelGGL(grouped_f32_thin_kernel<true>, few, dim3(1024), 0, st, g);
      else hipLaunchKernelGGL(grouped_f32_thin_kernel<false>, few, dim3(1024), 0, st, g);
      return hipGetLastError();
    }
    const int lds = f32_lds_bytes(tiles < cus ? 32 : 64);
    const dim3 grid(f32_grid(tiles, cus));
    if (tiles < cus && s.w_layout) hipLaunchKernelGGL((grouped_f32_kernel<32, true>), grid, threads, lds, st, g);
    else if (tiles < cus) hipLaunchKernelGGL((grouped_f32_kernel<32, false>), grid, threads, lds, st, g);
    else if (s.w_layout) hipLaunchKernelGGL((grouped_f32_kernel<64, true>), grid, threads, lds, st, g);
    else hipLaunchKernelGGL((grouped_f32_kernel<64, false>), grid, threads, lds, st, g);
    return hipGetLastError();
  }
  const Rows way = rows_way(s, cus);
  if (way == Rows::kMid) {
    const dim3 big((cus / 8) * 8);
    if (s.w_layout) hipLaunchKernelGGL(grouped_mid_kernel<true>, big, dim3(kMidThreads), kMidLds, st, g);
    else hipLaunchKernelGGL(grouped_mid_kernel<false>, big, dim3(kMidThreads), kMidLds, st, g);
    return hipGetLastError();
  }
  if (way == Rows::kBig) {
    const dim3 big((cus / 8) * 8);
    // K of whole steps: no check at the fills (a tenth of 8192^3)
    if (s.w_layout && s.K % kBigBK) hipLaunchKernelGGL((grouped_big_kernel<true, true>), big, dim3(kBigThreads), kBigLds, st, g);
    else if (s.w_layout) hipLaunchKernelGGL((grouped_big_kernel<true, false>), big, dim3(kBigThreads), kBigLds, st, g);
    else if (s.K % kBigBK) hipLaunchKernelGGL((grouped_big_kernel<false, true>), big, dim3(kBigThreads), kBigLds, st, g);
    else hipLaunchKernelGGL((grouped_big_kernel<false, false>), big, dim3(kBigThreads), kBigLds, st, g);
    return hipGetLastError();
  }
  const int64_t tiles = s.rows / kThinRows + (s.rows < s.groups ? s.rows : s.groups);      // at most
  const int64_t items = tiles * ((s.N + kThinCols - 1) / kThinCols);
  const dim3 grid(items < 1 ? 1 : int(items < cus ? items : cus));
  if (s.w_layout) hipLaunchKernelGGL(grouped_thin_kernel<true>, grid, threads, kThinLds, st, g);
  else hipLaunchKernelGGL(grouped_thin_kernel<false>, grid, threads, kThinLds, st, g);
  return hipGetLastError();
}

// ---- gradients in pieces: the rows of every group go in pieces of `piece` rows, as if they were groups of their own, into fp32 gradients of
// theirs in the workspace, which are added up in order.  For matrices of few tiles, which would leave most of the card idle or wait for the
// group with the most rows, where writing and reading the pieces' gradients takes 20 us at most, or half of what groups of equal sizes take.
// us whole and in pieces, bf16: one matrix of 256 x 512 with 100000 rows 1626 and 67, 7168 x 256 with 32768 rows 648 and 173; 12 of 440 x 368 with 26401 rows,
// uneven (softmax of normal numbers) 208 and 57, even 46 and 43; 8 of 512 x 512 with 16384 rows 133 and 39, even 34 and 39; 36 of 128 x 96, even 16 and 24.
// Left whole: 2048 x 2048 with 2048 rows 41 and 48, 8 of 1024 x 1024 with 16384 rows, even 54 and 66.  fp32: 64 x 64 with 100000 rows 875 and 37, 104 of
// 28 x 164 with 31015 rows 77 and 34, even 20 and 26.
constexpr int kPieceCUs = 256;

struct Pieces {
  int wgs;                     // workgroups that take tiles at a time
  int64_t matrix;              // tiles of a matrix
  double most_join;            // us that writing and reading the pieces' gradients may take
};
static Pieces pieces_of(const moe_gemm_t& s) {
  const bool f32 = s.dtype == MOE_F32;
  const int T = f32 ? 32 : kBig, wgs = f32 ? 2 * kPieceCUs : kPieceCUs;
  const int64_t matrix = int64_t((s.K + T - 1) / T) * ((s.N + T - 1) / T), tiles = matrix * s.groups;
  const double turns = double((tiles + wgs - 1) / wgs), rows = double(s.rows) / s.groups;
  const double even = f32 ? rows / 128 * turns : rows / 64 * (tiles * 4 <= kPieceCUs ? 0.6 : 1.5 * turns);       // us
  return {wgs, matrix, even > 40 ? even / 2 : 20};
}
static double join_us(const moe_gemm_t& s, int64_t pieces) { return double(pieces) * s.K * s.N * 8 / 5e6; }

// Rows of a piece, a power of two, by the sizes alone; 0 for whole groups
static int64_t wgrad_piece(const moe_gemm_t& s) {
  const Pieces p = pieces_of(s);
  int64_t piece = 512;
  while (piece < s.rows * p.matrix / p.wgs || s.rows / piece + s.groups > kMaxGroups) {
    if (piece > s.rows) return 0;
    piece *= 2;
  }
  return s.rows >= 4 * piece && join_us(s, s.rows / piece + s.groups) <= p.most_join ? piece : 0;
}
static int most_pieces(const moe_gemm_t& s, int64_t piece) { return int(s.rows / piece + s.groups); }

// The workspace: the pieces' bounds, the first piece of every group, their number; the pieces' gradients
static size_t piece_table(const moe_gemm_t& s, int64_t pieces) { return align256(size_t(4) * (pieces + 1 + s.groups + 1)); }
static size_t piece_bytes(const moe_gemm_t& s, int64_t pieces) { return piece_table(s, pieces) + align256(size_t(pieces) * s.K * s.N * 4); }
size_t wgrad_need(const moe_gemm_t& s) {
  const int64_t piece = wgrad_piece(s);
  return piece == 0 ? 0 : piece_bytes(s, most_pieces(s, piece));
}
// What any number of rows up to these needs, none where none of them goes in pieces.  Pieces of one length and of one number of whole ones are
// judged at the most rows that have them, since what joining may cost grows with the rows; a piece holds its share of the rows, so that
// there are at most wgs / matrix whole ones.  (One piece more than the most is asked for.)
size_t wgrad_workspace(const moe_gemm_t& s) {
  const Pieces p = pieces_of(s);
  if (s.rows < 4 * 512 || join_us(s, s.groups + 4) > p.most_join) return 0;
  int64_t most = 0;
  for (int64_t piece = 512; 4 * piece <= s.rows; piece *= 2) {
    const int64_t fit = ((piece + 1) * p.wgs - 1) / p.matrix, top = s.rows < fit ? s.rows : fit;
    const int64_t room = kMaxGroups - s.groups;
    for (int64_t whole = top / piece < room ? top / piece : room; whole > most && whole >= 4; --whole) {
      moe_gemm_t r = s;
      r.rows = top < (whole + 1) * piece - 1 ? top : (whole + 1) * piece - 1;
      if (wgrad_piece(r) == piece) most = whole;
    }
  }
  if (most == 0) return 0;
  const int64_t share = p.wgs / p.matrix + 1, bound = s.rows / 512 < share ? s.rows / 512 : share;
  const int64_t pieces = (most < bound ? most + 1 : bound) + s.groups;
  return piece_bytes(s, pieces < kMaxGroups ? pieces : kMaxGroups);
}

// By one workgroup.  first[G] is the pieces' number; where the offsets are bad, one piece with bad bounds.
__global__ __launch_bounds__(256) void wgrad_pieces_kernel(const int32_t* __restrict__ offsets, int G, int piece_log2, int64_t rows,
                                                           int32_t* __restrict__ bounds, int32_t* __restrict__ first) {
  __shared__ int32_t base[kMaxGroups + 1], part[5];
  bool bad;
  int n = group_tiles<256>(offsets, G, rows, piece_log2, base, part, &bad);
  __syncthreads();
  for (int g = threadIdx.x; g < G; g += 256) first[g] = base[g];
  for (int v = threadIdx.x; v < n; v += 256) {
    const int g = find_expert(base, G, v);
    bounds[v] = offsets[g] + ((v - base[g]) << piece_log2);
  }
  if (bad) n = 1;
  if (threadIdx.x == 0) {
    first[G] = n;
    bounds[n] = offsets[G];
    if (bad) bounds[0] = -1;
  }
}

// dw = sum over the pieces, in order
template <typename O, bool ADD>
__global__ __launch_bounds__(256) void wgrad_join_kernel(const float* __restrict__ sums, const int32_t* __restrict__ bounds,
                                                         const int32_t* __restrict__ first, int64_t size, int64_t vectors, O* __restrict__ dw) {
  if (bounds[0] < 0) return;
  for (int64_t t = int64_t(blockIdx.x) * 256 + threadIdx.x; t < vectors; t += int64_t(gridDim.x) * 256) {
    const int64_t g = t * 4 / size;
    const int b = first[g + 1];
    f32x4 v{0, 0, 0, 0};
#pragma unroll 4
    for (int i = first[g]; i < b; ++i) v += *reinterpret_cast<const f32x4*>(sums + i * size + (t * 4 - g * size));
    if constexpr (sizeof(O) == 2) {
      *reinterpret_cast<uint2*>(dw + t * 4) = make_uint2(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]));
    } else {
      if constexpr (ADD) v += *reinterpret_cast<const f32x4*>(dw + t * 4);
      *reinterpret_cast<f32x4*>(dw + t * 4) = v;
    }
  }
}

static hipError_t launch_wgrad_whole(const moe_gemm_t& s, const void* x, const void* dy, const int32_t* offsets, void* dw,
                                int dw_dtype, bool accumulate, int32_t* status, const int32_t* used, int cus, hipStream_t st) {
  const int64_t ldx = s.ldx ? s.ldx : s.K, ldy = s.ldy ? s.ldy : s.N;
  const WgradArgs g = s.w_layout ? WgradArgs{x, dy, dw, offsets, status, s.rows, ldx, ldy, s.groups, s.K, s.N, used}
                                 : WgradArgs{dy, x, dw, offsets, status, s.rows, ldy, ldx, s.groups, s.N, s.K, used};
  const hipError_t e = set_grouped_lds();
  if (e != hipSuccess) return e;
  if (s.dtype == MOE_F32) {
    const int64_t tiles = int64_t(g.G) * ((g.M + 63) / 64) * ((g.N + 63) / 64);
    const int lds = f32_lds_bytes(tiles < cus ? 32 : 64);
    const dim3 grid(f32_grid(tiles, cus)), threads(256);
    if (tiles < cus && accumulate) hipLaunchKernelGGL((grouped_f32_wgrad_kernel<32, true>), grid, threads, lds, st, g);
    else if (tiles < cus) hipLaunchKernelGGL((grouped_f32_wgrad_kernel<32, false>), grid, threads, lds, st, g);
    else if (accumulate) hipLaunchKernelGGL((grouped_f32_wgrad_kernel<64, true>), grid, threads, lds, st, g);
    else hipLaunchKernelGGL((grouped_f32_wgrad_kernel<64, false>), grid, threads, lds, st, g);
  } else {
    const dim3 big((cus / 8) * 8), many(kBigThreads);
    // 512 rows of 2048 x 2048 (64 tiles of 256) 13 us with tiles of 128, 20 with those; 2048 rows 39 and 51; 8 groups of 2048 x 1408 (384) 46 and 33
    const int64_t tiles = int64_t(s.groups) * ((s.K + kBig - 1) / kBig) * ((s.N + kBig - 1) / kBig);
    if (tiles * 4 <= cus) {
      if (dw_dtype != MOE_F32) hipLaunchKernelGGL((grouped_mid_wgrad_kernel<uint16_t, false>), big, dim3(kMidThreads), kMidLds, st, g);
      else if (accumulate) hipLaunchKernelGGL((grouped_mid_wgrad_kernel<float, true>), big, dim3(kMidThreads), kMidLds, st, g);
      else hipLaunchKernelGGL((grouped_mid_wgrad_kernel<float, false>), big, dim3(kMidThreads), kMidLds, st, g);
      return hipGetLastError();
    }
    if (dw_dtype != MOE_F32) hipLaunchKernelGGL((grouped_big_wgrad_kernel<uint16_t, false>), big, many, kBigLds, st, g);
    else if (accumulate) hipLaunchKernelGGL((grouped_big_wgrad_kernel<float, true>), big, many, kBigLds, st, g);
    else hipLaunchKernelGGL((grouped_big_wgrad_kernel<float, false>), big, many, kBigLds, st, g);
  }
  return hipGetLastError();
}

hipError_t launch_grouped_wgrad(const moe_gemm_t& s, const void* x, const void* dy, const int32_t* offsets, void* dw,
                                int dw_dtype, bool accumulate, void* ws, int32_t* status, int cus, hipStream_t st) {
  const int64_t piece = wgrad_piece(s);
  if (piece == 0) return launch_wgrad_whole(s, x, dy, offsets, dw, dw_dtype, accumulate, status, nullptr, cus, st);
  moe_gemm_t pieces = s;
  pieces.groups = most_pieces(s, piece);
  int32_t* const bounds = static_cast<int32_t*>(ws);
  int32_t* const first = bounds + pieces.groups + 1;
  float* const sums = reinterpret_cast<float*>(static_cast<char*>(ws) + piece_table(s, pieces.groups));
  hipLaunchKernelGGL(wgrad_pieces_kernel, dim3(1), dim3(256), 0, st, offsets, s.groups, __builtin_ctzll(uint64_t(piece)), s.rows, bounds, first);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  if ((e = launch_wgrad_whole(pieces, x, dy, bounds, sums, MOE_F32, false, status, first + s.groups, cus, st)) != hipSuccess) return e;
  const int64_t size = int64_t(s.K) * s.N, vectors = s.groups * size / 4, need = (vectors + 255) / 256;
  const dim3 grid(int(need < (1 << 20) ? need : 1 << 20)), threads(256);
  if (dw_dtype != MOE_F32)
    hipLaunchKernelGGL((wgrad_join_kernel<uint16_t, false>), grid, threads, 0, st, sums, bounds, first, size, vectors, static_cast<uint16_t*>(dw));
  else if (accumulate)
    hipLaunchKernelGGL((wgrad_join_kernel<float, true>), grid, threads, 0, st, sums, bounds, first, size, vectors, static_cast<float*>(dw));
  else
    hipLaunchKernelGGL((wgrad_join_kernel<float, false>), grid, threads, 0, st, sums, bounds, first, size, vectors, static_cast<float*>(dw));
  return hipGetLastError();
}

}  // namespace moe
