// AdamW over many tensors in one launch (formulas and the 8-bit states' format in include/moe_overlap.h).
//
// Bound by HBM: every element's parameter, gradient and states are read once, the parameter, its copy and the states
// written once (30 bytes per element with an fp32 master, gradient and states and a bf16 copy; 18 with 8-bit states).
// 138.5 million elements: 774 us (5.37 TB/s) with 32-bit states, 461 (5.41) with 8-bit ones and 138 (6.0) for their values.
// Through flat instead of global accesses and with every chunk checked against its tensor's end: 849, and 1113 for both.
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
  auto two = [](float a, float b) {
    return (uint32_t)__builtin_bit_cast(uint16_t, (__bf16)a) | ((uint32_t)__builtin_bit_cast(uint16_t, (__bf16)b) << 16);
  };
  const u32x2 q = {two(v[0], v[1]), two(v[2], v[3])};
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

// Root codes: exponent and mantissa fields are those of an fp32 cut to four mantissa bits, from 2^-15.  SPECIAL: code 255 is
// told apart
template <bool SPECIAL>
__device__ __forceinline__ float root_value(uint32_t c) {
  const float v = __uint_as_float((c << 19) + ((127u - 15u) << 23));
  return c == 0 ? 0.f : SPECIAL && c == 255 ? __uint_as_float(0x7fc00000u) : v;
}
__device__ __forceinline__ uint32_t root_code(float r) {  // r in units of the scale, in [0, 1.875]
  const int u = (int)__float_as_uint(r);
  // the nearest of four mantissa bits, ties to even, less the exponent of code 0; at least 1 where r is not 0
  const int c = (u + ((u >> 19) & 1) + (0x3ffff - ((127 - 15) << 23))) >> 19;
  return (uint32_t)max(c, min(u, 1));
}
// whether a byte of v is 255
__device__ __forceinline__ bool any255(uint32_t v) { return ((~v - 0x01010101u) & v & 0x80808080u) != 0; }

// the largest of v over the eight lanes of a block
__device__ __forceinline__ float max8(float v) {
  auto dpp = [&](float x, auto ctrl) {
    return __builtin_bit_cast(
        float, __builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, x), decltype(ctrl)::value, 0xf, 0xf, true));
  };
  v = fmaxf(v, dpp(v, std::integral_constant<int, 0xB1>{}));      // lane ^ 1
  v = fmaxf(v, dpp(v, std::integral_constant<int, 0x4E>{}));      // lane ^ 2
  return fmaxf(v, dpp(v, std::integral_constant<int, 0x141>{}));  // the other half of the eight, mirrored
}

// the scale byte for a largest magnitude: its biased exponent less `lead`, one more where its significand is over `over`
__device__ __forceinline__ uint32_t scale_byte(float top, uint32_t over_mantissa, int lead, int least) {
  const int b = (int)((__float_as_uint(top) + (0x7fffffu - over_mantissa)) >> 23) - lead;
  return (uint32_t)max(b, least);
}

// Four elements' states as codes with their block's scales.  SPECIAL: values that are not finite are told apart: they do not
// count for the scale
template <bool SPECIAL>
__device__ __forceinline__ void pack(const f32x4& m, const f32x4& root, uint32_t* mc, uint32_t* vc, uint32_t* ms, uint32_t* vs) {
  float tm = 0.f, tr = 0.f;
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    tm = fmaxf(tm, !SPECIAL || fabsf(m[e]) < INFINITY ? fabsf(m[e]) : 0.f);
    tr = fmaxf(tr, !SPECIAL || root[e] < INFINITY ? root[e] : 0.f);
  }
  *ms = scale_byte(max8(tm), 0x600000u, 8, 1);   // 448 = 1.75 x 2^8
  *vs = scale_byte(max8(tr), 0x700000u, 0, 16);  // 1.875
  const float a = __uint_as_float((254u - *ms) << 23), b = __uint_as_float((254u - *vs) << 23);
  f32x4 q;
  uint32_t c[4];
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    q[e] = !SPECIAL || fabsf(m[e]) < INFINITY ? m[e] * a : __uint_as_float(0x7fc00000u);
    c[e] = !SPECIAL || root[e] < INFINITY ? root_code(root[e] * b) : 255u;
  }
  *mc = e4m3_codes(q);
  *vc = (c[0] | (c[1] << 8)) | ((c[2] | (c[3] << 8)) << 16);
}

// A pointer out of a descriptor, to global memory as all of them (else its accesses would be flat ones)
template <class E>
__device__ __forceinline__ E* global(void* p) {
  return (E*)(__attribute__((address_space(1))) E*)p;
}

// A chunk's step.  FULL: all of its elements are the tensor's
template <bool BITS8, bool FULL>
__device__ __forceinline__ void step_chunk(const AdamwDesc& t, int64_t start, const Hyper& h, float gs) {
  const float lr = h.lr * t.lr_scale, decay = lr * t.weight_decay, rate = lr * h.inv_c1;
  const bool pb = t.param_dtype == MOE_BF16, gb = t.grad_dtype == MOE_BF16;
  const int left = FULL ? ADAMW_CHUNK : (int)(t.n - start);
  float* pf = global<float>(t.param) + start;
  bf16_t* ph = global<bf16_t>(t.param) + start;
  const float* gf = global<float>((void*)t.grad) + start;
  const bf16_t* gh = global<bf16_t>((void*)t.grad) + start;
  float *mf = global<float>(t.m) + start, *vf = global<float>(t.v) + start;
  uint8_t *mb = global<uint8_t>(t.m) + start, *vb = global<uint8_t>(t.v) + start;
  uint8_t *msp = global<uint8_t>(t.m_scale) + start / MOE_ADAMW_BLOCK, *vsp = global<uint8_t>(t.v_scale) + start / MOE_ADAMW_BLOCK;
  f32x4 p[PASSES], g[PASSES], m[PASSES], v[PASSES];
  uint32_t mc[PASSES], vc[PASSES], ms[PASSES], vs[PASSES];
  auto place = [&](int k) { return (uint32_t)(k * 1024 + threadIdx.x * 4); };
  auto count = [&](uint32_t i) { return FULL ? 4 : min(4, left - (int)i); };
#pragma unroll
  for (int k = 0; k < PASSES; ++k) {
    const uint32_t i = place(k);
    const int n = count(i);
    if (n <= 0) {
      p[k] = g[k] = m[k] = v[k] = f32x4{0, 0, 0, 0};
      mc[k] = vc[k] = 0;
      ms[k] = vs[k] = 1;
      continue;
    }
    if (pb) {
      const u32x2 q = load4(ph + i, n);
      p[k][0] = __uint_as_float(q[0]);
      p[k][1] = __uint_as_float(q[1]);
    } else p[k] = load4(pf + i, n);
    if (gb) {
      const u32x2 q = load4(gh + i, n);
      g[k][0] = __uint_as_float(q[0]);
      g[k][1] = __uint_as_float(q[1]);
    } else g[k] = load4(gf + i, n);
    if (BITS8) {
      mc[k] = load4((const uint8_t*)mb + i, n);
      vc[k] = load4((const uint8_t*)vb + i, n);
      ms[k] = msp[i / MOE_ADAMW_BLOCK];
      vs[k] = vsp[i / MOE_ADAMW_BLOCK];
    } else {
      m[k] = load4((const float*)mf + i, n);
      v[k] = load4((const float*)vf + i, n);
    }
  }
#pragma unroll
  for (int k = 0; k < PASSES; ++k) {
    const uint32_t i = place(k);
    const int n = count(i);
    if (pb) p[k] = widen(u32x2{__float_as_uint(p[k][0]), __float_as_uint(p[k][1])});
    if (gb) g[k] = widen(u32x2{__float_as_uint(g[k][0]), __float_as_uint(g[k][1])});
    if (BITS8) {
      const float a = scale_of(ms[k]), b = scale_of(vs[k]);
      m[k] = e4m3_values(mc[k]);
      const bool special = __ballot(any255(vc[k])) != 0;  // hardly ever
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const uint32_t c = (vc[k] >> (8 * e)) & 255u;
        const float r = (special ? root_value<true>(c) : root_value<false>(c)) * b;
        m[k][e] *= a;
        v[k][e] = r * r;
      }
    }
    f32x4 root;
    float all = 0.f;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const float q = g[k][e] * gs;
      if (BITS8) {
        // each product and sum rounded by itself, as the root is: what decides between two codes is then the formula's
        // plain fp32 evaluation, the same in any program, not what a compiler made of it
        m[k][e] = __fadd_rn(__fmul_rn(h.beta1, m[k][e]), __fmul_rn(h.one1, q));
        v[k][e] = __fadd_rn(__fmul_rn(h.beta2, v[k][e]), __fmul_rn(h.one2, __fmul_rn(q, q)));
      } else {
        m[k][e] = fmaf(h.beta1, m[k][e], h.one1 * q);
        v[k][e] = fmaf(h.beta2, v[k][e], h.one2 * q * q);
      }
      root[e] = __fsqrt_rn(v[k][e]);  // right for subnormals too: the root of a v of 1e-42 still divides where eps is small
      const float den = fmaf(root[e], h.inv_root_c2, h.eps);
      // both parts of the change before it meets p: 1 - lr weight_decay, rounded, would lose most of a small decay
      p[k][e] -= fmaf(rate * m[k][e], __builtin_amdgcn_rcpf(den), decay * p[k][e]);
      if (BITS8) all += fabsf(m[k][e]) + root[e];
    }
    if (BITS8) {  // elements past the tensor hold 0
      if (__ballot(!(all < INFINITY)) != 0) pack<true>(m[k], root, &mc[k], &vc[k], &ms[k], &vs[k]);
      else pack<false>(m[k], root, &mc[k], &vc[k], &ms[k], &vs[k]);
    }
    if (n <= 0) continue;
    if (pb) store4(ph + i, p[k], n);
    else store4(pf + i, p[k], n);
    if (t.copy) store4(global<bf16_t>(t.copy) + start + i, p[k], n);
    if (BITS8) {
      store4(mb + i, mc[k], n);
      store4(vb + i, vc[k], n);
      if ((threadIdx.x & 7) == 0) {
        msp[i / MOE_ADAMW_BLOCK] = (uint8_t)ms[k];
        vsp[i / MOE_ADAMW_BLOCK] = (uint8_t)vs[k];
      }
    } else {
      store4(mf + i, m[k], n);
      store4(vf + i, v[k], n);
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
  const bool full = t.n - start >= ADAMW_CHUNK;
  if (t.state_bits == 8) {
    if (full) step_chunk<true, true>(t, start, h, gs);
    else step_chunk<true, false>(t, start, h, gs);
  } else {
    if (full) step_chunk<false, true>(t, start, h, gs);
    else step_chunk<false, false>(t, start, h, gs);
  }
}

template <bool FULL>
__device__ __forceinline__ void read_chunk(const AdamwDesc& t, int64_t start) {
  const int left = FULL ? ADAMW_CHUNK : (int)(t.n - start);
  // m, then the root: codes and scales of the whole chunk first, then the values
#pragma unroll
  for (int what = 0; what < 2; ++what) {
    void* to = what ? t.root_values : t.m_values;
    if (!to) continue;
    const uint8_t* code = global<uint8_t>(what ? t.v : t.m) + start;
    const uint8_t* scale = global<uint8_t>(what ? t.v_scale : t.m_scale) + start / MOE_ADAMW_BLOCK;
    bf16_t* out = global<bf16_t>(to) + start;
    uint32_t c[PASSES], s[PASSES];
#pragma unroll
    for (int k = 0; k < PASSES; ++k) {
      const uint32_t i = (uint32_t)(k * 1024 + threadIdx.x * 4);
      if (!FULL && (int)i >= left) continue;
      c[k] = load4(code + i, FULL ? 4 : left - (int)i);
      s[k] = scale[i / MOE_ADAMW_BLOCK];
    }
#pragma unroll
    for (int k = 0; k < PASSES; ++k) {
      const uint32_t i = (uint32_t)(k * 1024 + threadIdx.x * 4);
      if (!FULL && (int)i >= left) continue;
      f32x4 v;
      if (what == 0) v = e4m3_values(c[k]);
      else
#pragma unroll
        for (int e = 0; e < 4; ++e) v[e] = root_value<true>((c[k] >> (8 * e)) & 255u);
      const float f = scale_of(s[k]);
#pragma unroll
      for (int e = 0; e < 4; ++e) v[e] *= f;
      store4(out + i, v, FULL ? 4 : left - (int)i);
    }
  }
}

__global__ __launch_bounds__(256) void k_adamw_read(AdamwStep a) {
  const AdamwChunk c = a.chunks[blockIdx.x];
  const AdamwDesc& t = a.tensors[c.tensor];
  const int64_t start = (int64_t)c.index * ADAMW_CHUNK;
  if (t.state_bits != 8) return;
  if (t.n - start >= ADAMW_CHUNK) read_chunk<true>(t, start);
  else read_chunk<false>(t, start);
}

}  // namespace

int launch_adamw(const AdamwStep& a, int64_t n_chunks, bool read, hipStream_t st) {
  if (n_chunks == 0) return 0;
  if (read) hipLaunchKernelGGL(k_adamw_read, dim3((unsigned)n_chunks), dim3(256), 0, st, a);
  else hipLaunchKernelGGL(k_adamw, dim3((unsigned)n_chunks), dim3(256), 0, st, a);
  return hipGetLastError() == hipSuccess ? 0 : -1;
}
