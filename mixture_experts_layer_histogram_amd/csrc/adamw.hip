// One AdamW step over many tensors.
//
//   g = grad * grad_scale;  m = b1 m + (1 - b1) g;  v = b2 v + (1 - b2) g^2;
//   p = p (1 - lr wd) - lr (m / (1 - b1^t)) / (sqrt(v / (1 - b2^t)) + eps).
//
// Bound by bytes: 28 a value with bf16 weights, fp32 masters and fp32 states, 16.1 with states in 8 bits.  Workgroups walk
// chunks of all tensors of a launch in turn, so small tensors share a launch with large ones; every array passes by once
// (non-temporal).
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

constexpr int kAdamTensors = 40;          // of one launch: their descriptions travel with it
constexpr int kAdamThreads = 256;

struct AdamTensor {
  char* param;
  const char* grad;
  float* master;
  char* m;
  char* v;
  uint8_t* ms;
  uint8_t* vs;
  int64_t n;
  int64_t chunk0;                         // chunks of the tensors before it
  float keep;                             // 1 - lr wd, or wd where lr is read on the device
  int32_t bf16;                           // bit 0: param, bit 1: grad
};

struct AdamArgs {
  AdamTensor t[kAdamTensors];
  int64_t chunks;
  const float* grad_scale;
  const float* device_lr;
  const int64_t* device_step;
  double beta1, beta2;
  int64_t step;
  uint64_t seed;
  float lr, eps, by_m, by_r;              // by_m = 1 / (1 - b1^t), by_r = (1 - b2^t)^-1/2, unless the step is on the device
  int32_t count, first;                   // tensors of this launch, and those of launches before it
};

// 32 bits mixed: two rounds of shift, exclusive or, and a product with an odd constant (the fractions of the golden ratio
// and of the square root of 3)
__device__ __forceinline__ uint32_t mix32(uint32_t z) {
  z ^= z >> 16;
  z *= 0x9E3779B9u;
  z ^= z >> 15;
  z *= 0xBB67AE85u;
  return z ^ (z >> 16);
}

// One value in E4M3 units of its block (bits of |v| / 2^e): what is cut off is added to by `part` (20 bits) first, or for
// rounding to nearest even by half a step less the last bit's complement
template <bool STOCHASTIC>
__device__ __forceinline__ uint32_t e4m3_up(float y, uint32_t part) {
  const uint32_t bits = __float_as_uint(y);
  uint32_t code;
  if constexpr (STOCHASTIC) {
    const uint32_t normal = ((bits + part) >> 20) - (120u << 3);
    const uint32_t small = (uint32_t(y * 0x1p29f) + part) >> 20;
    code = y >= 0x1p-6f ? normal : small;
  } else {
    const uint32_t normal = ((bits + 0x7FFFFu + ((bits >> 20) & 1u)) >> 20) - (120u << 3);
    const uint32_t small = uint32_t(__builtin_rintf(y * 512.0f));
    code = y >= 0x1p-6f ? normal : small;
  }
  return min(code, 126u);
}

// Eight consecutive values of a lane (a quad holds a block) in MXFP8; returns codes, *scale the block's.  ROOT: no signs,
// positive values take the smallest code at least.
template <bool ROOT, bool STOCHASTIC>
__device__ __forceinline__ uint2 state_quant(const float* f, const uint32_t* part, uint32_t* scale) {
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) m = max(m, __float_as_uint(f[i]) & 0x7FFFFFFFu);
  m = quad_max(m);
  if (m == 0 || m >= 0x7F800000u) {
    *scale = m ? 255u : 0u;
    return make_uint2(0, 0);
  }
  int e = int(m >> 23) - 127 - 8 + ((m & 0x7FFFFFu) > 0x600000u ? 1 : 0);    // 448 is 1.75 * 2^8
  e = max(e, -127);
  const float inv = mx_inv_scale(e);
  *scale = uint32_t(e + 127);
  uint32_t w[2];
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    w[h] = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float x = f[4 * h + i];
      uint32_t c = e4m3_up<STOCHASTIC>(fabsf(x) * inv, part[4 * h + i]);
      if (ROOT) c = x > 0.0f ? max(c, 1u) : c;
      else c |= c ? (__float_as_uint(x) >> 24) & 0x80u : 0u;
      w[h] |= c << (8 * i);
    }
  }
  return make_uint2(w[0], w[1]);
}

__device__ __forceinline__ float scale_of(uint32_t code) {       // 2^(code - 127), E8M0's NaN for 255
  return code == 255u ? __uint_as_float(0x7FC00000u) : code ? __uint_as_float(code << 23) : 0x1p-127f;
}

// U consecutive values from i on of an array, zeros from n on
template <int U>
__device__ __forceinline__ void load_f32(const float* p, int64_t i, int64_t n, float* f) {
  if (i + U <= n) {
#pragma unroll
    for (int w = 0; w < U / 4; ++w) {
      const f32x4 v = __builtin_nontemporal_load(reinterpret_cast<const f32x4*>(p + i) + w);
#pragma unroll
      for (int j = 0; j < 4; ++j) f[4 * w + j] = v[j];
    }
  } else {
#pragma unroll
    for (int j = 0; j < U; ++j) f[j] = i + j < n ? p[i + j] : 0.0f;
  }
}

template <int U>
__device__ __forceinline__ void store_f32(float* p, int64_t i, int64_t n, const float* f) {
  if (i + U <= n) {
#pragma unroll
    for (int w = 0; w < U / 4; ++w)
      __builtin_nontemporal_store(f32x4{f[4 * w], f[4 * w + 1], f[4 * w + 2], f[4 * w + 3]},
                                  reinterpret_cast<f32x4*>(p + i) + w);
  } else {
#pragma unroll
    for (int j = 0; j < U; ++j)
      if (i + j < n) p[i + j] = f[j];
  }
}

typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));

template <int U>
__device__ __forceinline__ void load_bf16(const uint16_t* p, int64_t i, int64_t n, float* f) {
  if (i + U <= n) {
#pragma unroll
    for (int w = 0; w < U / 4; ++w) {
      const u32x2 v = __builtin_nontemporal_load(reinterpret_cast<const u32x2*>(p + i) + w);
      f[4 * w] = __uint_as_float(v[0] << 16);
      f[4 * w + 1] = __uint_as_float(v[0] & 0xFFFF0000u);
      f[4 * w + 2] = __uint_as_float(v[1] << 16);
      f[4 * w + 3] = __uint_as_float(v[1] & 0xFFFF0000u);
    }
  } else {
#pragma unroll
    for (int j = 0; j < U; ++j) f[j] = i + j < n ? bf16_to_f32(p[i + j]) : 0.0f;
  }
}

// bf16 bits of f: nearest even, or with 16 random bits added to what is cut off (NaN and infinities stay what they are)
__device__ __forceinline__ uint32_t bf16_bits(float f, bool stochastic, uint32_t r16) {
  if (!stochastic) return pack_bf16x2(f, 0.0f) & 0xFFFFu;
  const uint32_t u = __float_as_uint(f);
  if ((u & 0x7FFFFFFFu) >= 0x7F800000u) return pack_bf16x2(f, 0.0f) & 0xFFFFu;
  return (u + r16) >> 16;
}

template <int U>
__device__ __forceinline__ void store_bf16(uint16_t* p, int64_t i, int64_t n, const uint32_t* b) {
  if (i + U <= n) {
#pragma unroll
    for (int w = 0; w < U / 4; ++w)
      __builtin_nontemporal_store(u32x2{b[4 * w] | (b[4 * w + 1] << 16), b[4 * w + 2] | (b[4 * w + 3] << 16)},
                                  reinterpret_cast<u32x2*>(p + i) + w);
  } else {
#pragma unroll
    for (int j = 0; j < U; ++j)
      if (i + j < n) p[i + j] = uint16_t(b[j]);
  }
}

// U values a lane: 8 with states in 8 bits, so that a quad holds a block, else 4 (16 bytes of every fp32 array)
template <bool EIGHT, bool STOCHASTIC>
__global__ __launch_bounds__(kAdamThreads) void adamw_kernel(AdamArgs a) {
#pragma clang fp contract(off)
  constexpr int U = EIGHT ? 8 : 4;
  constexpr int kChunk = kAdamThreads * U;
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
  for (int64_t c = blockIdx.x; c < a.chunks; c += gridDim.x) {
    int ti = 0;
    for (int hi = a.count - 1; ti < hi;) {
      const int mid = (ti + hi + 1) >> 1;
      if (a.t[mid].chunk0 <= c) ti = mid;
      else hi = mid - 1;
    }
    const AdamTensor& t = a.t[ti];
    const int64_t n = t.n;
    const int64_t i = (c - t.chunk0) * kChunk + threadIdx.x * U;
    const float keep = a.device_lr ? 1.0f - lr * t.keep : t.keep;
    const int64_t padded = EIGHT ? (n + 127) & ~int64_t(127) : n;
    if (!EIGHT && i >= n) continue;
    float p[U], g[U], m[U], v[U];
    if (t.bf16 & 2) load_bf16<U>(reinterpret_cast<const uint16_t*>(t.grad), i, n, g);
    else load_f32<U>(reinterpret_cast<const float*>(t.grad), i, n, g);
    if (t.master) load_f32<U>(t.master, i, n, p);
    else if (t.bf16 & 1) load_bf16<U>(reinterpret_cast<const uint16_t*>(t.param), i, n, p);
    else load_f32<U>(reinterpret_cast<const float*>(t.param), i, n, p);
    if constexpr (EIGHT) {
      u32x2 qm = {0, 0}, qv = {0, 0};
      float sm = 0.0f, sv = 0.0f;
      if (i < n) {
        qm = __builtin_nontemporal_load(reinterpret_cast<const u32x2*>(t.m + i));
        qv = __builtin_nontemporal_load(reinterpret_cast<const u32x2*>(t.v + i));
        sm = scale_of(t.ms[i >> 5]);
        sv = scale_of(t.vs[i >> 5]);
      }
#pragma unroll
      for (int w = 0; w < 4; ++w) {
        const auto fm = (w & 1) ? __builtin_amdgcn_cvt_pk_f32_fp8(int(qm[w >> 1]), true)
                                : __builtin_amdgcn_cvt_pk_f32_fp8(int(qm[w >> 1]), false);
        const auto fv = (w & 1) ? __builtin_amdgcn_cvt_pk_f32_fp8(int(qv[w >> 1]), true)
                                : __builtin_amdgcn_cvt_pk_f32_fp8(int(qv[w >> 1]), false);
#pragma unroll
        for (int z = 0; z < 2; ++z) {
          const bool in = i + 2 * w + z < n;
          m[2 * w + z] = in ? fm[z] * sm : 0.0f;
          const float r = in ? fv[z] * sv : 0.0f;
          v[2 * w + z] = r * r;
        }
      }
    } else {
      load_f32<U>(reinterpret_cast<const float*>(t.m), i, n, m);
      load_f32<U>(reinterpret_cast<const float*>(t.v), i, n, v);
    }
    uint32_t key0 = 0, key1 = 0;
    if constexpr (STOCHASTIC) {
      const uint32_t key = mix32(mix32(head + uint32_t(a.first + ti)) + uint32_t(i >> 32));
      key0 = mix32(key + 1);
      key1 = mix32(key + 2);
    }
    uint32_t pb[U], pm[U], pv[U];
    float r[U];
#pragma unroll
    for (int j = 0; j < U; ++j) {
      const float gj = g[j] * gs;
      m[j] = b1 * m[j] + c1 * gj;
      v[j] = b2 * v[j] + (c2 * gj) * gj;
      r[j] = sqrtf(v[j]);
      p[j] = p[j] * keep - lr * ((m[j] * by_m) * __builtin_amdgcn_rcpf(r[j] * by_r + a.eps));
      uint32_t r0 = 0, r1 = 0;
      if constexpr (STOCHASTIC) {
        if (EIGHT) r0 = mix32(uint32_t(i) + j + key0);
        if ((t.bf16 & 1) && !t.master) r1 = mix32(uint32_t(i) + j + key1);
      }
      if (t.bf16 & 1) pb[j] = bf16_bits(p[j], STOCHASTIC && !t.master, r1 & 0xFFFFu);
      pm[j] = (r0 & 0xFFFFu) << 4;
      pv[j] = (r0 >> 16) << 4;
    }
    if (t.master) store_f32<U>(t.master, i, n, p);
    if (t.bf16 & 1) store_bf16<U>(reinterpret_cast<uint16_t*>(t.param), i, n, pb);
    else store_f32<U>(reinterpret_cast<float*>(t.param), i, n, p);
    if constexpr (EIGHT) {
      uint32_t scm, scv;
      const uint2 qm = state_quant<false, STOCHASTIC>(m, pm, &scm);       // all lanes: quads agree on a block
      const uint2 qv = state_quant<true, STOCHASTIC>(r, pv, &scv);
      if (i < padded) {
        __builtin_nontemporal_store(u32x2{qm.x, qm.y}, reinterpret_cast<u32x2*>(t.m + i));
        __builtin_nontemporal_store(u32x2{qv.x, qv.y}, reinterpret_cast<u32x2*>(t.v + i));
        if ((i & 31) == 0) {
          t.ms[i >> 5] = uint8_t(scm);
          t.vs[i >> 5] = uint8_t(scv);
        }
      }
    } else {
      store_f32<U>(reinterpret_cast<float*>(t.m), i, n, m);
      store_f32<U>(reinterpret_cast<float*>(t.v), i, n, v);
    }
  }
}

hipError_t launch_adamw(const moe_adamw_t& h, const moe_adamw_tensor_t* tensors, int count, int cus, hipStream_t st) {
  const bool eight = h.state_dtype == MOE_MXFP8;
  const int chunk = kAdamThreads * (eight ? 8 : 4);
  for (int first = 0; first < count; first += kAdamTensors) {
    AdamArgs a{};
    a.first = first;
    for (int i = first; i < count && i < first + kAdamTensors; ++i) {
      const moe_adamw_tensor_t& t = tensors[i];
      AdamTensor& d = a.t[a.count++];
      d.param = static_cast<char*>(t.param);
      d.grad = static_cast<const char*>(t.grad);
      d.master = t.master;
      d.m = static_cast<char*>(t.m);
      d.v = static_cast<char*>(t.v);
      d.ms = t.m_scales;
      d.vs = t.v_scales;
      d.n = t.n;
      d.chunk0 = a.chunks;
      d.keep = h.device_lr ? t.weight_decay : float(1.0 - h.lr * double(t.weight_decay));
      d.bf16 = (t.param_dtype == MOE_BF16 ? 1 : 0) | (t.grad_dtype == MOE_BF16 ? 2 : 0);
      a.chunks += (t.n + chunk - 1) / chunk;
    }
    if (a.chunks == 0) continue;
    a.grad_scale = h.grad_scale;
    a.device_lr = h.device_lr;
    a.device_step = h.device_step;
    a.beta1 = h.beta1;
    a.beta2 = h.beta2;
    a.lr = float(h.lr);
    a.by_m = float(1.0 / (1.0 - pow(h.beta1, double(h.step))));
    a.by_r = float(1.0 / sqrt(1.0 - pow(h.beta2, double(h.step))));
    a.step = h.step;
    a.seed = h.seed;
    a.eps = float(h.eps);
    const dim3 grid(int(a.chunks < int64_t(cus) * 16 ? a.chunks : int64_t(cus) * 16)), threads(kAdamThreads);
    if (eight) {
      if (h.stochastic) hipLaunchKernelGGL((adamw_kernel<true, true>), grid, threads, 0, st, a);
      else hipLaunchKernelGGL((adamw_kernel<true, false>), grid, threads, 0, st, a);
    } else {
      if (h.stochastic) hipLaunchKernelGGL((adamw_kernel<false, true>), grid, threads, 0, st, a);
      else hipLaunchKernelGGL((adamw_kernel<false, false>), grid, threads, 0, st, a);
    }
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

}  // namespace moe
