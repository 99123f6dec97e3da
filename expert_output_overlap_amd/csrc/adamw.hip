// AdamW over many tensors in one launch (formulas and the 8-bit states' format in include/moe_overlap.h).
//
// Bound by HBM: every element's parameter, gradient and states are read once, the parameter, its copy and the states
// written once (30 bytes per element with an fp32 master, gradient and states and a bf16 copy; 18 with 8-bit states).
// The tensors are cut into chunks of ADAMW_CHUNK elements, one workgroup each; a table in the plan names each chunk's
// tensor, so a launch of many small tensors has no search and no empty workgroups.  A thread takes four elements side by
// side (a 16-byte access per fp32 array and wave: 1 KB), ADAMW_CHUNK / 1024 times, every load of all of them issued before
// the first is used.  An 8-bit state's block of 32 elements is then eight lanes, whose largest magnitude three DPP steps
// find.
#include <type_traits>

#include "common.h"
#include "launch.h"

namespace {

typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));

constexpr int PASSES = ADAMW_CHUNK / 1024;

struct Hyper {  // a step's numbers, before the tensor's own factors
  float lr, beta1, beta2, one1, one2, eps, inv_c1, inv_root_c2;
};

// n (1 .. 4) elements at p; any alignment of the element type
__device__ __forceinline__ f32x4 load4(const float* p, int n) {
  f32x4 v = {0, 0, 0, 0};
  if (n >= 4) __builtin_memcpy(&v, p, 16);
  else
    for (int i = 0; i < n; ++i) v[i] = p[i];
  return v;
}
__device__ __forceinline__ u32x2 load4(const bf16_t* p, int n) {
  u32x2 v = {0, 0};
  if (n >= 4) __builtin_memcpy(&v, p, 8);
  else
    for (int i = 0; i < n; ++i) v[i >> 1] |= (uint32_t)p[i] << (16 * (i & 1));
  return v;
}
__device__ __forceinline__ uint32_t load4(const uint8_t* p, int n) {
  uint32_t v = 0;
  if (n >= 4) __builtin_memcpy(&v, p, 4);
  else
    for (int i = 0; i < n; ++i) v |= (uint32_t)p[i] << (8 * i);
  return v;
}
__device__ __forceinline__ void store4(float* p, f32x4 v, int n) {
  if (n >= 4) __builtin_memcpy(p, &v, 16);
  else
    for (int i = 0; i < n; ++i) p[i] = v[i];
}
__device__ __forceinline__ void store4(bf16_t* p, f32x4 v, int n) {
  const u32x2 q = {pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3])};
  if (n >= 4) __builtin_memcpy(p, &q, 8);
  else
    for (int i = 0; i < n; ++i) p[i] = (bf16_t)(q[i >> 1] >> (16 * (i & 1)));
}
__device__ __forceinline__ void store4(uint8_t* p, uint32_t v, int n) {
  if (n >= 4) __builtin_memcpy(p, &v, 4);
  else
    for (int i = 0; i < n; ++i) p[i] = (uint8_t)(v >> (8 * i));
}
__device__ __forceinline__ f32x4 widen(u32x2 v) {
  return f32x4{__uint_as_float(v[0] << 16), __uint_as_float(v[0] & 0xffff0000u), __uint_as_float(v[1] << 16),
               __uint_as_float(v[1] & 0xffff0000u)};
}

// 2^(b - 127) for a scale byte b >= 1 (a byte 0, which no step writes, stands for the smallest scale)
__device__ __forceinline__ float scale_of(uint32_t b) { return __uint_as_float((b ? b : 1u) << 23); }

// the e4m3 codes of v (its four bytes), as values
__device__ __forceinline__ f32x4 e4m3_values(uint32_t v) {
  typedef float f32x2 __attribute__((ext_vector_type(2)));
  const f32x2 lo = __builtin_amdgcn_cvt_pk_f32_fp8((int)v, false), hi = __builtin_amdgcn_cvt_pk_f32_fp8((int)v, true);
  return f32x4{lo[0], lo[1], hi[0], hi[1]};
}
// and back: nearest, ties to even; |v| <= 448 or NaN
__device__ __forceinline__ uint32_t e4m3_codes(f32x4 v) {
  int c = __builtin_amdgcn_cvt_pk_fp8_f32(v[0], v[1], 0, false);
  return (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(v[2], v[3], c, true);
}

// root codes: exponent and mantissa fields are those of an fp32 cut to four mantissa bits, from 2^-15
__device__ __forceinline__ float root_value(uint32_t c) {
  const float v = __uint_as_float(((127u - 15u) << 23) + (c << 19));
  return c == 0 ? 0.f : c == 255 ? __uint_as_float(0x7fc00000u) : v;
}
__device__ __forceinline__ uint32_t root_code(float r) {  // r in units of the scale, at most 1.875 if finite
  const uint32_t u = __float_as_uint(r);
  const int c = (int)((u + 0x3ffffu + ((u >> 19) & 1u)) >> 19) - ((127 - 15) << 4);
  if (!(r < INFINITY)) return 255;
  return r > 0.f ? (uint32_t)max(c, 1) : 0u;
}

// the largest of v over the eight lanes of a block
__device__ __forceinline__ float max8(float v) {
  auto dpp = [&](float x, auto ctrl) {
    return __builtin_bit_cast(
        float, __builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, x), decltype(ctrl)::value, 0xf, 0xf, false));
  };
  v = fmaxf(v, dpp(v, std::integral_constant<int, 0xB1>{}));   // lane ^ 1
  v = fmaxf(v, dpp(v, std::integral_constant<int, 0x4E>{}));   // lane ^ 2
  return fmaxf(v, dpp(v, std::integral_constant<int, 0x141>{}));  // the other half of the eight, mirrored
}

// the scale byte for a largest magnitude: its biased exponent less `lead`, one more where its significand is over `over`
__device__ __forceinline__ uint32_t scale_byte(float top, uint32_t over_mantissa, int lead, int least) {
  const uint32_t u = __float_as_uint(top);
  const int b = (int)(u >> 23) - lead + ((u & 0x7fffffu) > over_mantissa ? 1 : 0);
  return (uint32_t)max(b, least);
}

template <bool BITS8>
__device__ __forceinline__ void step_chunk(const AdamwDesc& t, int64_t start, const Hyper& h, float gs) {
  const float lr = h.lr * t.lr_scale, decay = lr * t.weight_decay, rate = lr * h.inv_c1;
  const bool pb = t.param_dtype == MOE_BF16, gb = t.grad_dtype == MOE_BF16;
  f32x4 p[PASSES], g[PASSES], m[PASSES], v[PASSES];
  uint32_t mc[PASSES], vc[PASSES], ms[PASSES], vs[PASSES];
#pragma unroll
  for (int k = 0; k < PASSES; ++k) {
    const int64_t i = start + k * 1024 + threadIdx.x * 4;
    const int n = (int)min((int64_t)4, t.n - i);
    if (n <= 0) {
      p[k] = g[k] = m[k] = v[k] = f32x4{0, 0, 0, 0};
      mc[k] = vc[k] = 0;
      ms[k] = vs[k] = 1;
      continue;
    }
    if (pb) {
      const u32x2 q = load4((const bf16_t*)t.param + i, n);
      p[k][0] = __uint_as_float(q[0]);
      p[k][1] = __uint_as_float(q[1]);
    } else p[k] = load4((const float*)t.param + i, n);
    if (gb) {
      const u32x2 q = load4((const bf16_t*)t.grad + i, n);
      g[k][0] = __uint_as_float(q[0]);
      g[k][1] = __uint_as_float(q[1]);
    } else g[k] = load4((const float*)t.grad + i, n);
    if (BITS8) {
      mc[k] = load4((const uint8_t*)t.m + i, n);
      vc[k] = load4((const uint8_t*)t.v + i, n);
      ms[k] = t.m_scale[i / MOE_ADAMW_BLOCK];
      vs[k] = t.v_scale[i / MOE_ADAMW_BLOCK];
    } else {
      m[k] = load4((const float*)t.m + i, n);
      v[k] = load4((const float*)t.v + i, n);
    }
  }
#pragma unroll
  for (int k = 0; k < PASSES; ++k) {
    const int64_t i = start + k * 1024 + threadIdx.x * 4;
    const int n = (int)min((int64_t)4, t.n - i);
    if (pb) p[k] = widen(u32x2{__float_as_uint(p[k][0]), __float_as_uint(p[k][1])});
    if (gb) g[k] = widen(u32x2{__float_as_uint(g[k][0]), __float_as_uint(g[k][1])});
    if (BITS8) {
      const float a = scale_of(ms[k]), b = scale_of(vs[k]);
      m[k] = e4m3_values(mc[k]);
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        m[k][e] *= a;
        const float r = root_value((vc[k] >> (8 * e)) & 255u) * b;
        v[k][e] = r * r;
      }
    }
    f32x4 root;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const float q = g[k][e] * gs;
      m[k][e] = fmaf(h.beta1, m[k][e], h.one1 * q);
      v[k][e] = fmaf(h.beta2, v[k][e], h.one2 * q * q);
      root[e] = __builtin_amdgcn_sqrtf(v[k][e]);  // 1 ulp
      const float den = fmaf(root[e], h.inv_root_c2, h.eps);
      // both parts of the change before it meets p: 1 - lr weight_decay, rounded, would lose most of a small decay
      p[k][e] -= fmaf(rate * m[k][e], __builtin_amdgcn_rcpf(den), decay * p[k][e]);
    }
    if (BITS8) {
      // a block's largest finite magnitudes (elements past the tensor hold 0), then scales and codes
      float tm = 0.f, tr = 0.f;
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        tm = fmaxf(tm, fabsf(m[k][e]) < INFINITY ? fabsf(m[k][e]) : 0.f);
        tr = fmaxf(tr, root[e] < INFINITY ? root[e] : 0.f);
      }
      ms[k] = scale_byte(max8(tm), 0x600000u, 8, 1);    // 448 = 1.75 x 2^8
      vs[k] = scale_byte(max8(tr), 0x700000u, 0, 16);   // 1.875
      const float a = __uint_as_float((254u - ms[k]) << 23), b = __uint_as_float((254u - vs[k]) << 23);
      f32x4 q;
      uint32_t rc = 0;
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        q[e] = fabsf(m[k][e]) < INFINITY ? m[k][e] * a : __uint_as_float(0x7fc00000u);
        rc |= root_code(root[e] * b) << (8 * e);
      }
      mc[k] = e4m3_codes(q);
      vc[k] = rc;
    }
    if (n <= 0) continue;
    if (pb) store4((bf16_t*)t.param + i, p[k], n);
    else store4((float*)t.param + i, p[k], n);
    if (t.copy) store4((bf16_t*)t.copy + i, p[k], n);
    if (BITS8) {
      store4((uint8_t*)t.m + i, mc[k], n);
      store4((uint8_t*)t.v + i, vc[k], n);
      if ((threadIdx.x & 7) == 0) {
        t.m_scale[i / MOE_ADAMW_BLOCK] = (uint8_t)ms[k];
        t.v_scale[i / MOE_ADAMW_BLOCK] = (uint8_t)vs[k];
      }
    } else {
      store4((float*)t.m + i, m[k], n);
      store4((float*)t.v + i, v[k], n);
    }
  }
}

__global__ __launch_bounds__(256) void k_adamw(AdamwStep a) {
  const AdamwChunk c = a.chunks[blockIdx.x];
  const AdamwDesc& t = a.tensors[c.tensor];
  Hyper h;
  h.lr = a.lr_dev ? *a.lr_dev : a.lr;
  h.beta1 = a.beta1;
  h.beta2 = a.beta2;
  h.one1 = a.one1;
  h.one2 = a.one2;
  h.eps = a.eps;
  h.inv_c1 = a.inv_c1;
  h.inv_root_c2 = a.inv_root_c2;
  if (a.step_dev) {  // 1 - beta^t in 64 bits: near 0 for a beta near 1 and a small t
    const double s = (double)max((int64_t)1, *a.step_dev);
    h.inv_c1 = (float)(1.0 / -expm1(s * a.log_beta1));
    h.inv_root_c2 = (float)(1.0 / sqrt(-expm1(s * a.log_beta2)));
  }
  const float gs = a.grad_scale ? *a.grad_scale : 1.0f;
  const int64_t start = (int64_t)c.index * ADAMW_CHUNK;
  if (t.state_bits == 8) step_chunk<true>(t, start, h, gs);
  else step_chunk<false>(t, start, h, gs);
}

__global__ __launch_bounds__(256) void k_adamw_read(AdamwStep a) {
  const AdamwChunk c = a.chunks[blockIdx.x];
  const AdamwDesc& t = a.tensors[c.tensor];
  if (t.state_bits != 8 || (!t.m_values && !t.root_values)) return;
#pragma unroll
  for (int k = 0; k < PASSES; ++k) {
    const int64_t i = (int64_t)c.index * ADAMW_CHUNK + k * 1024 + threadIdx.x * 4;
    const int n = (int)min((int64_t)4, t.n - i);
    if (n <= 0) return;
    if (t.m_values) {
      const float s = scale_of(t.m_scale[i / MOE_ADAMW_BLOCK]);
      f32x4 v = e4m3_values(load4((const uint8_t*)t.m + i, n));
      for (int e = 0; e < 4; ++e) v[e] *= s;
      store4((bf16_t*)t.m_values + i, v, n);
    }
    if (t.root_values) {
      const float s = scale_of(t.v_scale[i / MOE_ADAMW_BLOCK]);
      const uint32_t q = load4((const uint8_t*)t.v + i, n);
      f32x4 v;
      for (int e = 0; e < 4; ++e) v[e] = root_value((q >> (8 * e)) & 255u) * s;
      store4((bf16_t*)t.root_values + i, v, n);
    }
  }
}

}  // namespace

int launch_adamw(const AdamwStep& a, int64_t n_chunks, bool read, hipStream_t st) {
  if (n_chunks == 0) return 0;
  if (read) hipLaunchKernelGGL(k_adamw_read, dim3((unsigned)n_chunks), dim3(256), 0, st, a);
  else hipLaunchKernelGGL(k_adamw, dim3((unsigned)n_chunks), dim3(256), 0, st, a);
  return hipGetLastError() == hipSuccess ? 0 : -1;
}
