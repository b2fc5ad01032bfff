// One AdamW step over many tensors.
//
//   g = grad * grad_scale;  m = b1 m + (1 - b1) g;  v = b2 v + (1 - b2) g^2;
//   p = p (1 - lr wd) - lr (m / (1 - b1^t)) / (sqrt(v / (1 - b2^t)) + eps).
//
// Bound by bytes: 28 a value with bf16 weights, fp32 masters and fp32 states, 16.1 with states in 8 bits.  Workgroups walk
// chunks of all tensors of a launch in turn, so small tensors share a launch with large ones; every array passes by once
// (non-temporal).  553 M values with fp32 masters and 8-bit states 1616 us (5.5 TB/s), with fp32 states 2734 us (5.7 TB/s); 61 tensors of
// 260000 values in all 5.8 us, a launch's submission.
//
// States in 8 bits are MXFP8 matrices of rows of 128 values: m, and the root of v (which halves the powers of ten that v
// spans).  A step changes v by a thousandth, E4M3 has steps of a sixteenth: rounded to nearest, most changes would be
// lost, so the states are rounded up with the probability of what is cut off (`stochastic`), and on average nothing is
// lost.  A positive root takes at least the smallest code: with a root of zero the next step would divide by eps alone.  A
// block's scale is the smallest that keeps its largest value within E4M3's 448, since a value cut off there at every step
// would never grow.  The random bits are a mixing of (seed, step, tensor, place), so a step can be repeated.
#include <math.h>

#include "mx.hpp"

namespace moe {

constexpr int kAdamThreads = 256;
// Four values a lane, so a part of a tensor is 1024.  A workgroup takes one at a time, and with states in 8 bits two, one after the other, where
// that leaves every workgroup that the card holds a chunk: 61 tensors of 4096 values 12 us with one, 15 with two, 500000 values 102 and 94,
// 9 million 1577 and 1479 (fp32 states 136 and 147, 2824 and 2964).
constexpr int kAdamPart = kAdamThreads * 4;

struct AdamScales {
  uint8_t *m, *v;
};

template <bool EIGHT>
struct AdamTensor {
  char* param;
  const char* grad;
  float* master;
  char* m;
  char* v;
  int64_t n_kinds;                        // its values * 4 + 1 for a bf16 param + 2 for bf16 gradients
  uint32_t chunk0;                        // chunks of the tensors before it
  float keep;                             // 1 - lr wd, or wd where lr is read on the device
};

// The tensors' descriptions travel with the launch: as many as its 4 KiB of arguments take
constexpr int adam_tensors(bool eight) { return eight ? 54 : 70; }

template <bool EIGHT>
struct AdamArgs {
  AdamTensor<EIGHT> t[adam_tensors(EIGHT)];
  AdamScales s[EIGHT ? adam_tensors(true) : 1];
  const float* grad_scale;
  const float* device_lr;
  const int64_t* device_step;
  double beta1, beta2;
  int64_t step;
  uint64_t seed;
  float lr, eps, by_m, by_r;              // by_m = 1 / (1 - b1^t), by_r = (1 - b2^t)^-1/2, unless the step is on the device
  uint32_t chunks;
  int32_t count, first;                   // tensors of this launch, and those of launches before it
};
static_assert(sizeof(AdamArgs<true>) <= 4096 && sizeof(AdamArgs<false>) <= 4096, "arguments of a launch");

// 32 bits mixed: two rounds of shift, exclusive or, and a product with an odd constant (the fractions of the golden ratio
// and of the square root of 3)
__device__ __forceinline__ uint32_t mix32(uint32_t z) {
  z ^= z >> 16;
  z *= 0x9E3779B9u;
  z ^= z >> 15;
  z *= 0xBB67AE85u;
  return z ^ (z >> 16);
}

// Correctly rounded square roots of values that are zero or between 2^-100 and infinity: the instruction's (a unit off at most), once corrected
// by its residual.  Smaller ones, and an infinity, whose residual is a NaN, take the general function: a branch that hardly any wave takes.
__device__ __forceinline__ float root_of(float v) {
  float s = __builtin_amdgcn_sqrtf(v);
  const float e = __builtin_fmaf(-s, s, v);
  s = __builtin_fmaf(e, 0.5f * __builtin_amdgcn_rcpf(fmaxf(s, 0x1p-60f)), s);
  const uint32_t bits = __float_as_uint(v);
  if (bits - 1u < 0x0D800000u - 1u || bits >= 0x7F800000u) s = sqrtf(v);      // 0 < v < 2^-100, or not finite
  return s;
}

// Four consecutive values of a lane (eight lanes hold a block) in MXFP8; returns their codes, *scale the block's.  What E4M3 cuts off (20
// bits, and more below its smallest power of two) is rounded up with the random 16 bits ahead of it: v_cvt_sr_fp8_f32 adds the upper bits
// of its second operand there (compared with that rule on four million values and bits, to the last code).  ROOT: no signs, positive
// values take the smallest code at least.
template <bool ROOT, bool STOCHASTIC>
__device__ __forceinline__ uint32_t state_quant(const float* x, const uint32_t* random, uint32_t* scale) {
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < 4; ++i) m = max(m, ROOT ? __float_as_uint(x[i]) : __float_as_uint(x[i]) & 0x7FFFFFFFu);
  m = quad_max(m);
  m = max(m, uint32_t(__builtin_amdgcn_update_dpp(int(m), int(m), 0x141, 0xF, 0xF, false)));    // the half row mirrored: the other quad
  if (m == 0 || m >= 0x7F800000u) {
    *scale = m ? 255u : 0u;
    return 0;
  }
  int e = int(m >> 23) - 127 - 8 + ((m & 0x7FFFFFu) > 0x600000u ? 1 : 0);    // 448 is 1.75 * 2^8
  e = max(e, -127);
  const float inv = mx_inv_scale(e);
  *scale = uint32_t(e + 127);
  int c = 0;
  if constexpr (STOCHASTIC) {
    c = __builtin_amdgcn_cvt_sr_fp8_f32(x[0] * inv, int(ROOT ? random[0] & 0xFFFF0000u : random[0] << 16), c, 0);
    c = __builtin_amdgcn_cvt_sr_fp8_f32(x[1] * inv, int(ROOT ? random[1] & 0xFFFF0000u : random[1] << 16), c, 1);
    c = __builtin_amdgcn_cvt_sr_fp8_f32(x[2] * inv, int(ROOT ? random[2] & 0xFFFF0000u : random[2] << 16), c, 2);
    c = __builtin_amdgcn_cvt_sr_fp8_f32(x[3] * inv, int(ROOT ? random[3] & 0xFFFF0000u : random[3] << 16), c, 3);
  } else {
    c = __builtin_amdgcn_cvt_pk_fp8_f32(x[0] * inv, x[1] * inv, c, false);
    c = __builtin_amdgcn_cvt_pk_fp8_f32(x[2] * inv, x[3] * inv, c, true);
  }
  uint32_t w = uint32_t(c);
  const uint32_t some = ((w & 0x7F7F7F7Fu) + 0x7F7F7F7Fu) & 0x80808080u;          // the codes that are not zero
  if constexpr (ROOT) {
    if (some != 0x80808080u) {
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (x[i] > 0.0f && !((w >> (8 * i)) & 0x7Fu)) w |= 1u << (8 * i);
    }
  } else {
    w &= 0x7F7F7F7Fu | some;                                                       // and zeros have no sign
  }
  return w;
}

__device__ __forceinline__ float scale_of(uint32_t code) {       // 2^(code - 127), E8M0's NaN for 255
  return code == 255u ? __uint_as_float(0x7FC00000u) : code ? __uint_as_float(code << 23) : 0x1p-127f;
}

// Four consecutive values from i on of an array, zeros from n on
__device__ __forceinline__ void load_f32(const float* p, int64_t i, int64_t n, float* f) {
  if (i + 4 <= n) {
    const f32x4 v = __builtin_nontemporal_load(reinterpret_cast<const f32x4*>(p + i));
#pragma unroll
    for (int j = 0; j < 4; ++j) f[j] = v[j];
  } else {
#pragma unroll
    for (int j = 0; j < 4; ++j) f[j] = i + j < n ? p[i + j] : 0.0f;
  }
}

__device__ __forceinline__ void store_f32(float* p, int64_t i, int64_t n, const float* f) {
  if (i + 4 <= n) {
    __builtin_nontemporal_store(f32x4{f[0], f[1], f[2], f[3]}, reinterpret_cast<f32x4*>(p + i));
  } else {
#pragma unroll
    for (int j = 0; j < 4; ++j)
      if (i + j < n) p[i + j] = f[j];
  }
}

typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));

__device__ __forceinline__ void load_bf16(const uint16_t* p, int64_t i, int64_t n, float* f) {
  if (i + 4 <= n) {
    const u32x2 v = __builtin_nontemporal_load(reinterpret_cast<const u32x2*>(p + i));
    f[0] = __uint_as_float(v[0] << 16);
    f[1] = __uint_as_float(v[0] & 0xFFFF0000u);
    f[2] = __uint_as_float(v[1] << 16);
    f[3] = __uint_as_float(v[1] & 0xFFFF0000u);
  } else {
#pragma unroll
    for (int j = 0; j < 4; ++j) f[j] = i + j < n ? bf16_to_f32(p[i + j]) : 0.0f;
  }
}

// bf16 bits of f with 16 random bits added to what is cut off (NaN and infinities stay what they are)
__device__ __forceinline__ uint32_t bf16_up(float f, uint32_t r16) {
  const uint32_t u = __float_as_uint(f);
  return (u & 0x7FFFFFFFu) >= 0x7F800000u ? pack_bf16x2(f, 0.0f) & 0xFFFFu : (u + r16) >> 16;
}

__device__ __forceinline__ void store_bf16(uint16_t* p, int64_t i, int64_t n, const uint32_t* b) {
  if (i + 4 <= n) {
    __builtin_nontemporal_store(u32x2{b[0] | (b[1] << 16), b[2] | (b[3] << 16)}, reinterpret_cast<u32x2*>(p + i));
  } else {
#pragma unroll
    for (int j = 0; j < 4; ++j)
      if (i + j < n) p[i + j] = uint16_t(b[j]);
  }
}

// Four consecutive values of a lane: what a step reads of them
template <bool EIGHT>
struct AdamPart {
  float p[4], g[4], m[4], v[4];

  __device__ __forceinline__ void load(const AdamTensor<EIGHT>& t, const AdamScales& sc, int64_t i, int64_t n, bool pb, bool gb, bool mast) {
    if (gb) load_bf16(reinterpret_cast<const uint16_t*>(t.grad), i, n, g);
    else load_f32(reinterpret_cast<const float*>(t.grad), i, n, g);
    if (mast) load_f32(t.master, i, n, p);
    else if (pb) load_bf16(reinterpret_cast<const uint16_t*>(t.param), i, n, p);
    else load_f32(reinterpret_cast<const float*>(t.param), i, n, p);
    if constexpr (EIGHT) {
      uint32_t qm = 0, qv = 0, sm = 0, sv = 0;
      if (i < n) {
        qm = __builtin_nontemporal_load(reinterpret_cast<const uint32_t*>(t.m + i));
        qv = __builtin_nontemporal_load(reinterpret_cast<const uint32_t*>(t.v + i));
        sm = sc.m[i >> 5];
        sv = sc.v[i >> 5];
        if (i + 4 > n) {                                       // what lies past the end counts as zero
          const uint32_t in = (1u << (8 * uint32_t(n - i))) - 1u;
          qm &= in;
          qv &= in;
        }
      }
      const float fs = scale_of(sm), fr = scale_of(sv);
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const auto fm = h ? __builtin_amdgcn_cvt_pk_f32_fp8(int(qm), true) : __builtin_amdgcn_cvt_pk_f32_fp8(int(qm), false);
        const auto fv = h ? __builtin_amdgcn_cvt_pk_f32_fp8(int(qv), true) : __builtin_amdgcn_cvt_pk_f32_fp8(int(qv), false);
#pragma unroll
        for (int z = 0; z < 2; ++z) {
          m[2 * h + z] = fm[z] * fs;
          const float old = fv[z] * fr;
          v[2 * h + z] = old * old;
        }
      }
    } else {
      load_f32(reinterpret_cast<const float*>(t.m), i, n, m);
      load_f32(reinterpret_cast<const float*>(t.v), i, n, v);
    }
  }
};

// Four values a lane: 16 bytes of every fp32 array, so that a wave reads and writes whole lines (eight values a lane store every second 16
// bytes: 553 M values with fp32 masters and 8-bit states 1928 us where four took 1726).  Eight lanes hold a block of 32.
template <bool EIGHT, bool STOCHASTIC, int PARTS>
__global__ __launch_bounds__(kAdamThreads) void adamw_kernel(AdamArgs<EIGHT> a) {
#pragma clang fp contract(off)
  constexpr int kChunk = PARTS * kAdamPart;
  const int64_t step = a.device_step ? *a.device_step : a.step;
  const float lr = a.device_lr ? *a.device_lr : a.lr;
  const float gs = a.grad_scale ? *a.grad_scale : 1.0f;
  const float b1 = float(a.beta1), b2 = float(a.beta2), c1 = float(1.0 - a.beta1), c2 = float(1.0 - a.beta2);
  float by_m = a.by_m, by_r = a.by_r;
  if (a.device_step) {
    by_m = float(1.0 / (1.0 - pow(a.beta1, double(step))));
    by_r = float(1.0 / sqrt(1.0 - pow(a.beta2, double(step))));
  }
  uint32_t head = 0;
  if constexpr (STOCHASTIC) head = mix32(mix32(mix32(uint32_t(a.seed)) + uint32_t(a.seed >> 32)) + uint32_t(step));
  for (uint32_t c = blockIdx.x; c < a.chunks; c += gridDim.x) {
    int ti = 0;
    for (int hi = a.count - 1; ti < hi;) {
      const int mid = (ti + hi + 1) >> 1;
      if (a.t[mid].chunk0 <= c) ti = mid;
      else hi = mid - 1;
    }
    const AdamTensor<EIGHT>& t = a.t[ti];
    const AdamScales& sc = a.s[EIGHT ? ti : 0];
    const int64_t n = t.n_kinds >> 2, first = int64_t(c - t.chunk0) * kChunk;
    const float keep = a.device_lr ? 1.0f - lr * t.keep : t.keep;
    const bool pb = t.n_kinds & 1, gb = t.n_kinds & 2, mast = t.master != nullptr, up = STOCHASTIC && pb && !mast;
    uint32_t key0 = 0, key1 = 0;
    if constexpr (STOCHASTIC) {
      const uint32_t key = mix32(mix32(head + uint32_t(a.first + ti)) + uint32_t(first >> 32));
      key0 = mix32(key + 1);
      key1 = mix32(key + 2);
    }
    // the values' places count on within 2^32 (a chunk never crosses such a border)
    for (int64_t i0 = first; i0 < min(first + kChunk, n); i0 += kAdamPart) {
      const int64_t i = i0 + threadIdx.x * 4;
      AdamPart<EIGHT> w;
      w.load(t, sc, i, n, pb, gb, mast);
      float r[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const float gj = w.g[j] * gs;
        w.m[j] = b1 * w.m[j] + c1 * gj;
        w.v[j] = b2 * w.v[j] + (c2 * gj) * gj;
        r[j] = root_of(w.v[j]);
        w.p[j] = w.p[j] * keep - lr * ((w.m[j] * by_m) * __builtin_amdgcn_rcpf(r[j] * by_r + a.eps));
      }
      if (mast) store_f32(t.master, i, n, w.p);
      if (pb) {
        uint32_t b[4];
        if (up) {
#pragma unroll
          for (int j = 0; j < 4; ++j) b[j] = bf16_up(w.p[j], mix32(key1 + uint32_t(i) + j) & 0xFFFFu);
        } else {
#pragma unroll
          for (int j = 0; j < 4; j += 2) {
            const uint32_t two = pack_bf16x2(w.p[j], w.p[j + 1]);
            b[j] = two & 0xFFFFu;
            b[j + 1] = two >> 16;
          }
        }
        store_bf16(reinterpret_cast<uint16_t*>(t.param), i, n, b);
      } else {
        store_f32(reinterpret_cast<float*>(t.param), i, n, w.p);
      }
      if constexpr (EIGHT) {
        uint32_t rand[4];
        if constexpr (STOCHASTIC) {
#pragma unroll
          for (int j = 0; j < 4; ++j) rand[j] = mix32(key0 + uint32_t(i) + j);
        }
        uint32_t scm, scv;
        const uint32_t qm = state_quant<false, STOCHASTIC>(w.m, rand, &scm);    // all lanes: eight of them agree on a block
        const uint32_t qv = state_quant<true, STOCHASTIC>(r, rand, &scv);
        if (i < ((n + 127) & ~int64_t(127))) {
          __builtin_nontemporal_store(qm, reinterpret_cast<uint32_t*>(t.m + i));
          __builtin_nontemporal_store(qv, reinterpret_cast<uint32_t*>(t.v + i));
          if ((i & 31) == 0) {
            sc.m[i >> 5] = uint8_t(scm);
            sc.v[i >> 5] = uint8_t(scv);
          }
        }
      } else {
        store_f32(reinterpret_cast<float*>(t.m), i, n, w.m);
        store_f32(reinterpret_cast<float*>(t.v), i, n, w.v);
      }
    }
  }
}

// The values of MXFP8 rows of 128 (whose scale bytes lie in the order of their blocks), such as these states, 16 bytes of values a lane.
template <bool BF16>
__global__ __launch_bounds__(256) void states_values_kernel(const uint8_t* __restrict__ codes, const uint8_t* __restrict__ scales,
                                                            int64_t vectors, void* __restrict__ dst) {
  constexpr int V = BF16 ? 8 : 4;
  for (int64_t t = int64_t(blockIdx.x) * 256 + threadIdx.x; t < vectors; t += int64_t(gridDim.x) * 256) {
    uint32_t q[V / 4];
    if constexpr (BF16) {
      const u32x2 two = __builtin_nontemporal_load(reinterpret_cast<const u32x2*>(codes) + t);
      q[0] = two[0];
      q[1] = two[1];
    } else {
      q[0] = __builtin_nontemporal_load(reinterpret_cast<const uint32_t*>(codes) + t);
    }
    const float s = scale_of(scales[t * V >> 5]);
    float f[V];
#pragma unroll
    for (int w = 0; w < V / 4; ++w) {
      const auto lo = __builtin_amdgcn_cvt_pk_f32_fp8(int(q[w]), false), up = __builtin_amdgcn_cvt_pk_f32_fp8(int(q[w]), true);
      f[4 * w] = lo[0] * s;
      f[4 * w + 1] = lo[1] * s;
      f[4 * w + 2] = up[0] * s;
      f[4 * w + 3] = up[1] * s;
    }
    if constexpr (BF16)
      __builtin_nontemporal_store(u32x4{pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]), pack_bf16x2(f[4], f[5]), pack_bf16x2(f[6], f[7])},
                                  static_cast<u32x4*>(dst) + t);
    else
      __builtin_nontemporal_store(f32x4{f[0], f[1], f[2], f[3]}, static_cast<f32x4*>(dst) + t);
  }
}

hipError_t launch_states_values(const uint8_t* codes, const uint8_t* scales, int64_t rows, void* dst, int dst_dtype, hipStream_t st) {
  const int64_t vectors = rows * (dst_dtype == MOE_BF16 ? 16 : 32), need = (vectors + 255) / 256;
  const dim3 grid(int(need < (1 << 22) ? need : 1 << 22)), threads(256);
  if (dst_dtype == MOE_BF16) hipLaunchKernelGGL(states_values_kernel<true>, grid, threads, 0, st, codes, scales, vectors, dst);
  else hipLaunchKernelGGL(states_values_kernel<false>, grid, threads, 0, st, codes, scales, vectors, dst);
  return hipGetLastError();
}

template <bool EIGHT>
static hipError_t adamw_launches(const moe_adamw_t& h, const moe_adamw_tensor_t* tensors, int count, int cus, hipStream_t st) {
  int64_t values = 0;
  for (int i = 0; i < count; ++i) values += tensors[i].n;
  const bool two = EIGHT && values >= int64_t(cus) * 8 * 2 * kAdamPart;
  const int chunk = two ? 2 * kAdamPart : kAdamPart;
  for (int i = 0; i < count;) {
    AdamArgs<EIGHT> a{};
    a.first = i;
    int64_t chunks = 0;
    for (; i < count && a.count < adam_tensors(EIGHT); ++i) {
      const moe_adamw_tensor_t& t = tensors[i];
      const int64_t mine = (t.n + chunk - 1) / chunk;          // at most 2^30
      if (chunks + mine >= int64_t(1) << 31) break;
      AdamTensor<EIGHT>& d = a.t[a.count];
      d.param = static_cast<char*>(t.param);
      d.grad = static_cast<const char*>(t.grad);
      d.master = t.master;
      d.m = static_cast<char*>(t.m);
      d.v = static_cast<char*>(t.v);
      d.n_kinds = t.n * 4 + (t.param_dtype == MOE_BF16 ? 1 : 0) + (t.grad_dtype == MOE_BF16 ? 2 : 0);
      d.chunk0 = uint32_t(chunks);
      d.keep = h.device_lr ? t.weight_decay : float(1.0 - h.lr * double(t.weight_decay));
      if constexpr (EIGHT) a.s[a.count] = AdamScales{t.m_scales, t.v_scales};
      ++a.count;
      chunks += mine;
    }
    if (chunks == 0) continue;
    a.chunks = uint32_t(chunks);
    a.grad_scale = h.grad_scale;
    a.device_lr = h.device_lr;
    a.device_step = h.device_step;
    a.beta1 = h.beta1;
    a.beta2 = h.beta2;
    a.step = h.step;
    a.seed = h.seed;
    a.lr = float(h.lr);
    a.eps = float(h.eps);
    a.by_m = float(1.0 / (1.0 - pow(h.beta1, double(h.step))));
    a.by_r = float(1.0 / sqrt(1.0 - pow(h.beta2, double(h.step))));
    // a workgroup a chunk (553 M values 1726 us, with sixteen workgroups a CU that loop 1814)
    const dim3 grid(int(chunks < (1 << 22) ? chunks : 1 << 22)), threads(kAdamThreads);
    if (two && h.stochastic) hipLaunchKernelGGL((adamw_kernel<EIGHT, true, EIGHT ? 2 : 1>), grid, threads, 0, st, a);
    else if (two) hipLaunchKernelGGL((adamw_kernel<EIGHT, false, EIGHT ? 2 : 1>), grid, threads, 0, st, a);
    else if (h.stochastic) hipLaunchKernelGGL((adamw_kernel<EIGHT, true, 1>), grid, threads, 0, st, a);
    else hipLaunchKernelGGL((adamw_kernel<EIGHT, false, 1>), grid, threads, 0, st, a);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

hipError_t launch_adamw(const moe_adamw_t& h, const moe_adamw_tensor_t* tensors, int count, int cus, hipStream_t st) {
  return h.state_dtype == MOE_MXFP8 ? adamw_launches<true>(h, tensors, count, cus, st)
                                    : adamw_launches<false>(h, tensors, count, cus, st);
}

}  // namespace moe
