// The norms around a block with its gate and the residual's scale, forward and backward (formulas in include/moe_overlap.h).
//
// Both are bound by HBM: forward 4 row transfers per row, backward 6.  A row is held in registers by a group of G threads, NV
// 16-byte chunks each, and is read once; a norm's variance is the mean of squared differences to the mean, and v^ = (v - mean) rstd from
// the difference too: as one product, v rstd - mean rstd, it would carry the rounding of mean rstd, in every element of a row, which
// for a row of equal elements is over sqrt(eps) and not 0.  The gate and N1's
// parameters meet the rows as two products, A = gate post_weight and B = gate post_bias: s = rho x + c (A h^ + B).  Rows stay as they
// were loaded (bf16 pairs) and are unpacked where they are used, which is what lets 1024 threads of 128 registers hold a backward row of
// 8192, its parameters, its sums and the next row's loads.
// 16384 x 7168 bf16, RMS norms and gate: forward 188 us (5.00 TB/s), backward 283 (4.98); layer norms with biases 202 and 314.
#include <algorithm>
#include <type_traits>

#include "common.h"
#include "launch.h"
#include "row_util.h"
#include "tile_util.h"

namespace {

using std::integral_constant;

// C parameters from index i on, `empty` where there are none
template <int C>
__device__ __forceinline__ void param_chunk(const void* p, bool bf16, int i, int d, float empty, float* out) {
  if (!p) {
#pragma unroll
    for (int e = 0; e < C; ++e) out[e] = empty;
  } else if (bf16) params<bf16_t, C>((const bf16_t*)p, i, d, empty, out);
  else params<float, C>((const float*)p, i, d, empty, out);
}

// A and B (0 without biases)
template <int C>
__device__ __forceinline__ void post_chunk(const ResidualLaunch& a, bool bf16, int i, float* A, float* B) {
  float g[C];
  param_chunk<C>(a.p.post_weight, bf16, i, a.d, 1.f, A);
  param_chunk<C>(a.p.post_bias, bf16, i, a.d, 0.f, B);
  if (!a.p.gate) return;
  param_chunk<C>(a.p.gate, bf16, i, a.d, 1.f, g);
#pragma unroll
  for (int e = 0; e < C; ++e) {
    A[e] *= g[e];
    B[e] *= g[e];
  }
}

// A row's statistics over the G threads that hold it; chunk(j, v): its chunk j of NV, of C elements, 0 past the row.  turn picks the one
// of red's two halves that the last sum did not use
template <int G, int NV, int C, bool TAIL, class Get>
__device__ __forceinline__ void row_stats(Get chunk, int kind, int t, int d, float eps, float (*red)[2 * (G / 64) + 1], int& turn,
                                          float* mean_out, float* rstd_out) {
  if (kind == MOE_NORM_NONE) {
    *mean_out = 0.f;
    *rstd_out = 1.f;
    return;
  }
  float mean = 0.f, off = 0.f;
  if (kind == MOE_NORM_LAYER) {
    float s[1] = {0.f};
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      float v[C];
      chunk(j, v);
#pragma unroll
      for (int i = 0; i < C; ++i) s[0] += v[i];
    }
    group_total<G>(s, red[turn]);
    turn ^= 1;
    mean = s[0] / d;
    float q[2] = {0.f, 0.f};
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      float v[C];
      chunk(j, v);
#pragma unroll
      for (int i = 0; i < C; ++i) {
        const float e = v[i] - mean;
        if ((j * G + t) * C + (TAIL ? i : 0) < d) {
          q[0] = fmaf(e, e, q[0]);
          q[1] += e;
        }
      }
    }
    group_total<G>(q, red[turn]);
    turn ^= 1;
    off = q[1] / d;  // the differences' own sum corrects the mean's rounding
    mean += off;
    *rstd_out = 1.0f / sqrtf(fmaxf(q[0] / d - off * off, 0.f) + eps);
  } else {
    float q[1] = {0.f};
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      float v[C];
      chunk(j, v);
#pragma unroll
      for (int i = 0; i < C; ++i) q[0] = fmaf(v[i], v[i], q[0]);
    }
    group_total<G>(q, red[turn]);
    turn ^= 1;
    *rstd_out = 1.0f / sqrtf(q[0] / d + eps);
  }
  *mean_out = mean;
}

// Rows by chunks: a row's address is the wave's, a chunk's 32-bit offset the lane's.  TAIL: the row's last chunk may hold fewer
// than C elements
template <typename T, bool TAIL>
struct Rows {
  using K = Chunk<T>;
  static __device__ __forceinline__ u32x4 load(const T* row, uint32_t c, int d) {
    const T* p = (const T*)((const char*)row + c * (uint32_t)sizeof(T));
    if ((int)c >= d) return u32x4{0, 0, 0, 0};
    return TAIL ? K::load(p, d - (int)c) : load16(p);
  }
  // The same without waiting for single elements' loads, for rows that are fetched ahead: a row's last chunk comes as its last 16 bytes,
  // and settle moves them to their places
  template <bool TINY>  // rows may be shorter than a chunk
  static __device__ __forceinline__ u32x4 load_ahead(const T* row, uint32_t c, int d) {
    if ((int)c >= d) return u32x4{0, 0, 0, 0};
    if (TINY && TAIL && d < K::C) return K::load(row, d);
    const uint32_t from = TAIL ? min(c, (uint32_t)(d - K::C)) : c;
    return load16((const char*)row + from * (uint32_t)sizeof(T));
  }
  // `end`: the column behind the G chunks that c's is one of
  template <bool TINY>
  static __device__ __forceinline__ void settle(u32x4& v, uint32_t c, int end, int d) {
    if (!TAIL || end <= d || (TINY && d < K::C)) return;
    const int over = (int)c < d ? max((int)c + K::C - d, 0) : 0, bits = over * (int)sizeof(T) * 8;
    if (__ballot(over > 0) == 0) return;
    const uint64_t lo = (uint64_t)v[1] << 32 | v[0], hi = (uint64_t)v[3] << 32 | v[2];
    const uint64_t a = bits >= 64 ? hi >> (bits & 63) : bits ? lo >> bits | hi << (64 - bits) : lo, b = bits >= 64 ? 0 : hi >> bits;
    v = u32x4{(uint32_t)a, (uint32_t)(a >> 32), (uint32_t)b, (uint32_t)(b >> 32)};
  }
  template <int G, int NV>
  static __device__ __forceinline__ void settle_all(int t, int d, u32x4* v) {
#pragma unroll
    for (int j = 0; j < NV; ++j) settle<G == 16>(v[j], (uint32_t)(j * G + t) * K::C, (j + 1) * G * K::C, d);
  }
  // past: past the caches (launch_residual)
  static __device__ __forceinline__ void store(T* row, uint32_t c, int d, const float* f, bool past) {
    T* p = (T*)((char*)row + c * (uint32_t)sizeof(T));
    if ((int)c >= d) return;
    typedef uint32_t anywhere __attribute__((ext_vector_type(4), aligned(2)));
    if (TAIL && d - (int)c < K::C) K::store(p, pack(f), d - (int)c);
    else if (past) __builtin_nontemporal_store((anywhere)pack(f), (anywhere*)p);
    else store16(p, pack(f));
  }
  // one conversion instruction for two bf16 (nearest, ties to even)
  static __device__ __forceinline__ u32x4 pack(const float* f) {
    u32x4 v;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if (sizeof(T) == 4) v[i] = __float_as_uint(f[i]);
      else v[i] = bf16_bits(f[2 * i]) | bf16_bits(f[2 * i + 1]) << 16;
    }
    return v;
  }
  template <int G, int NV, bool LATE = false>
  static __device__ __forceinline__ void load_all(const void* base, int64_t row, int64_t stride, int t, int d, u32x4* v) {
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const T* p = (const T*)base + row * stride;
      v[j] = LATE ? load_ahead<G == 16>(p, (uint32_t)(j * G + t) * K::C, d) : load(p, (uint32_t)(j * G + t) * K::C, d);
    }
  }
};

// Makes the compiler forget what it knows of a chunk: it then unpacks it again where it is used next, instead of keeping twice the
// registers as fp32 from its first use on
__device__ __forceinline__ void forget(u32x4& v) { asm volatile("" : "+v"(v)); }

// The wave's number in the workgroup, as a number of the wave's
__device__ __forceinline__ int wave_of() { return __builtin_amdgcn_readfirstlane(threadIdx.x >> 6); }

// Forward.  SHARED: the parameters in LDS, once for all rows of the workgroup's eight waves, which hold a row or more each (G <= 64: no
// barrier); else read for each row, as where there are few rows or wide ones.
template <typename T, int G, int NV, bool SHARED, bool TAIL>
__global__ __launch_bounds__(SHARED ? 512 : G) void k_residual(ResidualLaunch a) {
  using K = Chunk<T>;
  using R = Rows<T, TAIL>;
  constexpr int C = K::C, PER = SHARED ? 512 / G : 1, E = NV * C;
  extern __shared__ __align__(16) float shared[];  // SHARED: A, pre_weight, then B and pre_bias where there is a bias; by four columns, then lanes
  __shared__ float red[2][2 * (G / 64) + 1];
  const int t = threadIdx.x % G, d = a.d;
  const bool pb = a.param_dtype == MOE_BF16, bias = a.p.post_bias || a.p.pre_bias;
  if (SHARED) {
    for (int c = threadIdx.x; c < NV * G; c += 512) {
      float v[4][C];
      post_chunk<C>(a, pb, c * C, v[0], v[2]);
      param_chunk<C>(a.p.pre_weight, pb, c * C, d, 1.f, v[1]);
      param_chunk<C>(a.p.pre_bias, pb, c * C, d, 0.f, v[3]);
#pragma unroll
      for (int k = 0; k < 4; ++k)
        if (k < 2 || bias)
#pragma unroll
          for (int q = 0; q < C / 4; ++q)
            *(float4*)(shared + k * E * G + ((c / G * (C / 4) + q) * G + c % G) * 4) =
                float4{v[k][4 * q], v[k][4 * q + 1], v[k][4 * q + 2], v[k][4 * q + 3]};
    }
    __syncthreads();
  }
  int here = t;  // a new number to the compiler for each row: else it would keep all of LDS in registers
  constexpr bool HELD = !SHARED && E <= 8;  // the parameters in registers, read while the first row is on its way
  float held[HELD ? 4 : 1][HELD ? E : 1];    // weights, then biases
  // chunk j of weight (0: A, 1: pre_weight) and of its bias
  auto weights = [&](int which, int j, float* w, float* b) {
    if (HELD) {
#pragma unroll
      for (int i = 0; i < C; ++i) {
        w[i] = held[HELD ? which : 0][HELD ? j * C + i : 0];
        b[i] = held[HELD ? 2 + which : 0][HELD ? j * C + i : 0];
      }
    } else if (SHARED) {
#pragma unroll
      for (int q = 0; q < C / 4; ++q) {
        const int at = ((j * (C / 4) + q) * G + here) * 4;
        *(float4*)(w + 4 * q) = *(const float4*)(shared + which * E * G + at);
        if (bias) *(float4*)(b + 4 * q) = *(const float4*)(shared + (2 + which) * E * G + at);
        else *(float4*)(b + 4 * q) = float4{0, 0, 0, 0};
      }
    } else if (which == 0) post_chunk<C>(a, pb, (j * G + t) * C, w, b);
    else {
      param_chunk<C>(a.p.pre_weight, pb, (j * G + t) * C, d, 1.f, w);
      param_chunk<C>(a.p.pre_bias, pb, (j * G + t) * C, d, 0.f, b);
    }
  };
  constexpr bool AHEAD = !SHARED && NV <= 2;  // the next row's loads go out before the current row's sums
  u32x4 nh[AHEAD ? NV : 1], nx[AHEAD ? NV : 1];
  const int64_t step = (int64_t)gridDim.x * PER;
  int64_t r = (int64_t)blockIdx.x * PER + (G < 64 ? threadIdx.x / G : SHARED ? wave_of() : 0);
  auto fetch = [&](int64_t row, u32x4* h, u32x4* x) {
    R::template load_all<G, NV>(a.h, row, a.h_stride, t, d, h);
    R::template load_all<G, NV>(a.x, row, a.x_stride, t, d, x);
  };
  if (AHEAD && r < a.rows) fetch(r, nh, nx);
  int turn = 0;
  bool first = true;
  for (; r < a.rows; r += step) {
    u32x4 h[NV], x[NV];
    if (SHARED) asm volatile("" : "+v"(here));
    if (AHEAD) {
#pragma unroll
      for (int j = 0; j < NV; ++j) {
        h[j] = nh[AHEAD ? j : 0];
        x[j] = nx[AHEAD ? j : 0];
      }
      if (r + step < a.rows) fetch(r + step, nh, nx);
    } else fetch(r, h, x);
    if (HELD && first) {
#pragma unroll
      for (int j = 0; j < NV; ++j) {
        const int at = (j * G + t) * C;
        post_chunk<C>(a, pb, at, held[0] + (HELD ? j * C : 0), held[HELD ? 2 : 0] + (HELD ? j * C : 0));
        param_chunk<C>(a.p.pre_weight, pb, at, d, 1.f, held[HELD ? 1 : 0] + (HELD ? j * C : 0));
        param_chunk<C>(a.p.pre_bias, pb, at, d, 0.f, held[HELD ? 3 : 0] + (HELD ? j * C : 0));
      }
      first = false;
    }
    const float c = a.p.row_gate ? a.p.row_gate[r] : 1.f;
    float m1, r1, m2, r2, s[E];
    auto of_h = [&](int j, float* v) {
      if (sizeof(T) == 2) forget(h[j]);
      if (NV > 4) __builtin_amdgcn_sched_barrier(0);
#pragma unroll
      for (int i = 0; i < C; ++i) v[i] = K::at(h[j], i);
    };
    row_stats<G, NV, C, TAIL>(of_h, a.post, t, d, a.eps, red, turn, &m1, &r1);
    T* to = (T*)a.s + r * a.s_stride;
#pragma unroll
    for (int j = 0; j < NV; ++j) forget(h[j]);
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      float w[C], b[C];
      if (NV > 4) __builtin_amdgcn_sched_barrier(0);
      weights(0, j, w, b);
      const int at = (j * G + t) * C;
#pragma unroll
      for (int i = 0; i < C; ++i) {
        const float z = fmaf((K::at(h[j], i) - m1) * r1, w[i], b[i]);
        s[j * C + i] = at + (TAIL ? i : 0) < d ? fmaf(a.rho, K::at(x[j], i), c * z) : 0.f;
      }
      R::store(to, at, d, s + j * C, a.past);
    }
    auto of_s = [&](int j, float* v) {
#pragma unroll
      for (int i = 0; i < C; ++i) v[i] = s[j * C + i];
    };
    row_stats<G, NV, C, TAIL>(of_s, a.pre, t, d, a.eps, red, turn, &m2, &r2);
    if (a.pre != MOE_NORM_NONE) {
      to = (T*)a.n + r * a.n_stride;
#pragma unroll
      for (int j = 0; j < NV; ++j) {
        float w[C], b[C];
        if (NV > 4) __builtin_amdgcn_sched_barrier(0);
        weights(1, j, w, b);
        const int at = (j * G + t) * C;
#pragma unroll
        for (int i = 0; i < C; ++i) w[i] = fmaf((s[j * C + i] - m2) * r2, w[i], b[i]);
        R::store(to, at, d, w, a.past);
      }
    }
    if (t == 0 && a.stats) *(float4*)(a.stats + 4 * r) = float4{m1, r1, m2, r2};
  }
}

// Column c's gradients from its sums u1 of c D h^, u0 of c D (N1's, and the gate's), or of dn s^ and dn (N2's)
__device__ __forceinline__ void put_params(const ResidualLaunch& a, bool pre, int c, float u1, float u0) {
  const bool bf16 = a.param_dtype == MOE_BF16;
  auto param = [&](const void* p, float empty) {
    return !p ? empty : bf16 ? bf16_to_f32(((const bf16_t*)p)[c]) : ((const float*)p)[c];
  };
  auto put = [&](void* p, float v) {
    if (!p) return;
    if (bf16) ((bf16_t*)p)[c] = f32_to_bf16(v);
    else ((float*)p)[c] = v;
  };
  if (pre) {
    put(a.d_pre_weight, u1);
    put(a.d_pre_bias, u0);
    return;
  }
  const float gate = param(a.p.gate, 1.f);
  put(a.d_post_weight, gate * u1);
  put(a.d_post_bias, gate * u0);
  put(a.d_gate, fmaf(param(a.p.post_weight, 1.f), u1, param(a.p.post_bias, 0.f) * u0));
}

// dx and dh of a group's rows, and its sums of c D h^ and dn s^ (SUMS = 4: also of c D and dn), which stay in registers over all of its
// rows, as the parameters do, and go to the workspace at the end: partial [workgroup][SUMS][d]; a workgroup that is alone writes the
// parameters' gradients itself (where d <= 4096: in the wider rows' kernels that code costs the loop registers).  WIDE, where registers do not hold all
// that: the first two sums are in LDS, each thread's for itself, and the parameters are read (from the L2) for each row.
template <typename T, int G, int NV, int SUMS, bool WIDE, bool TAIL>
__global__ __launch_bounds__(G <= 64 ? 256 : G) void k_residual_bwd(ResidualLaunch a) {
  using K = Chunk<T>;
  using R = Rows<T, TAIL>;
  constexpr int C = K::C, PER = G <= 64 ? 256 / G : 1, E = NV * C, HELD = WIDE ? C : E, REGS = WIDE ? SUMS - 2 : SUMS;
  constexpr bool BIAS = SUMS == 4, AHEAD = !WIDE;  // AHEAD: registers hold the next row too
  // h's and x's registers take the differences to the means (4096 x 16384 fp32, two sums: 397 us, made anew in each pass 471; with four sums
  // 781, made anew 735)
  constexpr bool KEEP = WIDE && sizeof(T) == 4 && SUMS == 2;
  extern __shared__ float sums[];  // WIDE: [2][E][G]
  __shared__ float red[2][3 * (G / 64) + 1];
  __shared__ float join[PER > 1 ? (PER - 1) * SUMS * E * G : 1];
  const int t = threadIdx.x % G, d = a.d;
  const bool pb = a.param_dtype == MOE_BF16, pre = a.pre != MOE_NORM_NONE;
  float acc[REGS > 0 ? REGS : 1][E], A[HELD], B[HELD], W[HELD];
  int here = t;  // WIDE: a new number to the compiler for each pass over the row: else it would keep the parameters for the second one
  auto read_params = [&](int j, int to) {
    post_chunk<C>(a, pb, (j * G + here) * C, A + to, B + to);
    param_chunk<C>(a.p.pre_weight, pb, (j * G + here) * C, d, 1.f, W + to);
  };
#pragma unroll
  for (int k = 0; k < REGS; ++k)
#pragma unroll
    for (int e = 0; e < E; ++e) acc[k][e] = 0.f;
  if (WIDE) {
#pragma unroll
    for (int e = 0; e < 2 * E; ++e) sums[e * G + t] = 0.f;
  } else {
#pragma unroll
    for (int j = 0; j < NV; ++j) read_params(j, WIDE ? 0 : j * C);
  }
  // sum k of element e (0: c D h^, 1: dn s^, 2: c D, 3: dn) grows by u v, or by v
  auto grow = [&](int k, int e, float u, float v) {
    if (WIDE && k < 2) sums[(k * E + e) * G + t] = fmaf(u, v, sums[(k * E + e) * G + t]);
    else if (WIDE) acc[REGS > 0 ? k - 2 : 0][e] = fmaf(u, v, acc[REGS > 0 ? k - 2 : 0][e]);
    else acc[k][e] = fmaf(u, v, acc[k][e]);
  };
  const int64_t step = (int64_t)gridDim.x * PER;
  int64_t r = (int64_t)blockIdx.x * PER + (G < 64 ? threadIdx.x / G : PER > 1 ? wave_of() : 0);
  u32x4 nh[NV], nx[NV], ns[NV], nn[NV];
  float4 nst = {0, 0, 0, 0};
  float nc = 1.f;
  auto fetch = [&](int64_t row) {
    R::template load_all<G, NV, true>(a.h, row, a.h_stride, t, d, nh);
    R::template load_all<G, NV, true>(a.x, row, a.x_stride, t, d, nx);
    if (a.ds) R::template load_all<G, NV, true>(a.ds, row, a.ds_stride, t, d, ns);
    if (pre) R::template load_all<G, NV, true>(a.dn, row, a.dn_stride, t, d, nn);
    nst = *(const float4*)(a.stats + 4 * row);
    if (a.p.row_gate) nc = a.p.row_gate[row];
  };
#pragma unroll
  for (int j = 0; j < NV; ++j) ns[j] = nn[j] = u32x4{0, 0, 0, 0};
  if (AHEAD && r < a.rows) fetch(r);
  int turn = 0;
  for (; r < a.rows; r += step) {
    if (!AHEAD) fetch(r);
    u32x4 h[NV], x[NV], g[NV], q[NV];
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      h[j] = nh[j];
      x[j] = nx[j];
      g[j] = ns[j];
      q[j] = nn[j];
    }
    R::template settle_all<G, NV>(t, d, h);
    R::template settle_all<G, NV>(t, d, x);
    R::template settle_all<G, NV>(t, d, g);
    R::template settle_all<G, NV>(t, d, q);
    // a wave's row is its own from 64 threads on: its numbers go to scalar registers (8192 x 16384 bf16 with biases 1023 us, 1135 without;
    // 16384 x 7167 452 and 505)
    auto of_row = [](float v) {
      return G >= 64 ? __builtin_bit_cast(float, __builtin_amdgcn_readfirstlane(__builtin_bit_cast(int, v))) : v;
    };
    const float c = of_row(nc), m1 = of_row(nst.x), r1 = of_row(nst.y), m2 = of_row(nst.z), r2 = of_row(nst.w);
    if (AHEAD && r + step < a.rows) fetch(r + step);
    if (KEEP) {
#pragma unroll
      for (int j = 0; j < NV; ++j)
#pragma unroll
        for (int i = 0; i < C; ++i) h[j][i] = __float_as_uint(__uint_as_float(h[j][i]) - m1);
    }
    // of element i of chunk j, whose parameters are held from p on: differences to the means, v^ = e rstd
    auto e1 = [&](int j, int i) { return KEEP ? K::at(h[j], i) : K::at(h[j], i) - m1; };
    auto z = [&](int p, int i, float n) { return BIAS ? fmaf(n, A[p + i], B[p + i]) : n * A[p + i]; };
    auto e2 = [&](int j, int p, int i, float n) { return fmaf(a.rho, K::at(x[j], i), c * z(p, i, n)) - m2; };
    float ma = 0.f, mn = 0.f;
    if (pre) {
      float v[2] = {0.f, 0.f};
#pragma unroll
      for (int j = 0; j < NV; ++j) {
        const int p = WIDE ? 0 : j * C;
        if (WIDE) {
          __builtin_amdgcn_sched_barrier(0);
          read_params(j, p);
        }
#pragma unroll
        for (int i = 0; i < C; ++i) {
          const float e = e2(j, p, i, e1(j, i) * r1), n = e * r2, y = K::at(q[j], i), w = y * W[p + i];
          grow(1, j * C + i, y, n);
          if (BIAS) grow(3, j * C + i, 1.f, y);
          v[0] += w;
          v[1] = fmaf(w, n, v[1]);
          if (KEEP) x[j][i] = __float_as_uint(e);
        }
      }
      group_total<G>(v, red[turn]);
      turn ^= 1;
      if (a.pre == MOE_NORM_LAYER) ma = v[0] / d;
      mn = v[1] / d;
    }
    if (sizeof(T) == 2) {
#pragma unroll
      for (int j = 0; j < NV; ++j) {
        forget(h[j]);
        forget(x[j]);
        forget(q[j]);
      }
    }
    if (WIDE) asm volatile("" : "+v"(here));
    float D[E], v[3] = {0.f, 0.f, 0.f}, k = r2 * mn;
    T* to = (T*)a.dx + r * a.dx_stride;
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int at = (j * G + t) * C, p = WIDE ? 0 : j * C;
      if (WIDE) {
          __builtin_amdgcn_sched_barrier(0);
          read_params(j, p);
        }
      float y[C];
      if (pre) {
#pragma unroll
        for (int i = 0; i < C; ++i)
          y[i] = fmaf(r2, fmaf(-(KEEP ? K::at(x[j], i) : e2(j, p, i, e1(j, i) * r1)), k, fmaf(K::at(q[j], i), W[p + i], -ma)),
                      K::at(g[j], i));
      } else {
#pragma unroll
        for (int i = 0; i < C; ++i) y[i] = K::at(g[j], i);
      }
      float o[C];
#pragma unroll
      for (int i = 0; i < C; ++i) {
        const float n = e1(j, i) * r1;
        if (at + (TAIL ? i : 0) >= d) y[i] = 0.f;
        o[i] = a.rho * y[i];
        v[2] = fmaf(y[i], z(p, i, n), v[2]);
        y[i] *= c;
        grow(0, j * C + i, y[i], n);
        if (BIAS) grow(2, j * C + i, 1.f, y[i]);
        y[i] *= A[p + i];
        v[0] += y[i];
        v[1] = fmaf(y[i], n, v[1]);
        D[j * C + i] = y[i];
      }
      R::store(to, at, d, o, a.past);
    }
    if (a.post != MOE_NORM_NONE || a.d_row_gate) {
      group_total<G>(v, red[turn]);
      turn ^= 1;
    }
    if (a.post == MOE_NORM_NONE) {  // dh = D: h may hold infinities, which no product with 0 takes away
#pragma unroll
      for (int j = 0; j < NV; ++j) h[j] = u32x4{0, 0, 0, 0};
    }
    // in fp32 too: else both of h's registers would be held (8192 x 7168, two sums: 326 us instead of 277)
#pragma unroll
    for (int j = 0; j < NV; ++j) forget(h[j]);
    ma = a.post == MOE_NORM_LAYER ? v[0] / d : 0.f;
    k = a.post == MOE_NORM_NONE ? 0.f : r1 * (r1 * (v[1] / d));
    to = (T*)a.dh + r * a.dh_stride;
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int at = (j * G + t) * C;
      float o[C];
#pragma unroll
      for (int i = 0; i < C; ++i) o[i] = fmaf(-e1(j, i), k, r1 * (D[j * C + i] - ma));
      R::store(to, at, d, o, a.past);
    }
    if (t == 0 && a.d_row_gate) a.d_row_gate[r] = v[2];
  }
  if (!a.partial) return;
  if (PER > 1) {  // the workgroup's groups, one after another
    const int w = threadIdx.x / G;
    if (w > 0) {
      float* to = join + (w - 1) * SUMS * E * G;
#pragma unroll
      for (int k = 0; k < SUMS; ++k)
#pragma unroll
        for (int e = 0; e < E; ++e) to[(k * E + e) * G + t] = acc[k][e];
    }
    __syncthreads();
    if (w > 0) return;
#pragma unroll 1
    for (int u = 0; u < PER - 1; ++u) {
      const float* from = join + u * SUMS * E * G;
#pragma unroll
      for (int k = 0; k < SUMS; ++k)
#pragma unroll
        for (int e = 0; e < E; ++e) acc[k][e] += from[(k * E + e) * G + t];
    }
  }
  auto sum = [&](int k, int e) { return !WIDE ? acc[WIDE ? 0 : k][e] : k < 2 ? sums[(k * E + e) * G + t] : acc[REGS > 0 && WIDE ? k - 2 : 0][e]; };
  auto col = [&](int e) { return (e / C * G + t) * C + e % C; };
  if (E == 8 && G <= 512 && gridDim.x == 1) {
#pragma unroll
    for (int e = 0; e < E; ++e)
      if (col(e) < d) {
        put_params(a, false, col(e), sum(0, e), BIAS ? sum(BIAS ? 2 : 0, e) : 0.f);
        put_params(a, true, col(e), sum(1, e), BIAS ? sum(SUMS - 1, e) : 0.f);
      }
    return;
  }
  float* out = a.partial + (int64_t)blockIdx.x * SUMS * d;
#pragma unroll
  for (int k = 0; k < SUMS; ++k)
#pragma unroll
    for (int e = 0; e < E; ++e)
      if (col(e) < d) out[(int64_t)k * d + col(e)] = sum(k, e);
}

// The parameters' gradients from the workgroups' partial sums, `sums` of them in each: {c D h^, dn s^} or {c D h^, dn s^, c D, dn}.  64
// columns of N1's (y = 0) or of N2's (1) per workgroup; its 16 waves take every 16th partial row, eight in flight, and their sums are
// added in wave order.
__global__ __launch_bounds__(1024) void k_residual_params(ResidualLaunch a, int n, int sums) {
  __shared__ float red[15][2][64];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, c = blockIdx.x * 64 + lane, d = a.d, pre = blockIdx.y;
  float s[2] = {0.f, 0.f};
  if (c < d)
    for (int k = wave; k < n; k += 128) {
      const float* p = a.partial + ((int64_t)k * sums + pre) * d + c;
      float v[2][8];
#pragma unroll
      for (int u = 0; u < 8; ++u) {
        const int64_t at = (int64_t)16 * u * sums * d;
        v[0][u] = k + 16 * u < n ? p[at] : 0.f;
        v[1][u] = sums == 4 && k + 16 * u < n ? p[at + 2 * d] : 0.f;
      }
#pragma unroll
      for (int u = 0; u < 8; ++u) {
        s[0] += v[0][u];
        s[1] += v[1][u];
      }
    }
  if (wave > 0) {
    red[wave - 1][0][lane] = s[0];
    red[wave - 1][1][lane] = s[1];
  }
  __syncthreads();
  if (wave > 0 || c >= d) return;
  for (int k = 0; k < 15; ++k) {
    s[0] += red[k][0][lane];
    s[1] += red[k][1][lane];
  }
  put_params(a, pre, c, s[0], s[1]);
}

int chunks_of(int d, int dtype) { return (d * (dtype == MOE_BF16 ? 2 : 4) + 15) / 16; }

// chunks in each of G threads, rounded up to a power of two
int per_thread(int chunks, int G) {
  int nv = 1;
  while (nv * G < chunks) nv *= 2;
  return nv;
}

template <typename T, int G, int NV, bool SHARED, bool TAIL>
void forward(const ResidualLaunch& a, hipStream_t st) {
  constexpr int PER = SHARED ? 512 / G : 1;
  const int64_t groups = (a.rows + PER - 1) / PER, most = SHARED ? 512 : 256 * 2048 / G;
  constexpr int MOST = 4 * NV * Chunk<T>::C * G * 4;
  const int lds = SHARED ? (a.p.post_bias || a.p.pre_bias ? 4 : 2) * NV * Chunk<T>::C * G * 4 : 0;
  if (SHARED && MOST > 65536 - 512)
    (void)hipFuncSetAttribute((const void*)k_residual<T, G, NV, SHARED, TAIL>, hipFuncAttributeMaxDynamicSharedMemorySize, MOST);
  hipLaunchKernelGGL((k_residual<T, G, NV, SHARED, TAIL>), dim3((unsigned)std::min(groups, most)), dim3(SHARED ? 512 : G), lds, st, a);
}

template <typename T, bool TAIL>
void forward(const ResidualLaunch& a, hipStream_t st) {
  const int chunks = chunks_of(a.d, a.dtype);
  // A wave to a row (a quarter of one to rows of up to 32 chunks) where it can hold one and there are rows for all of eight waves on each CU:
  // 16384 x 7168 bf16 with layer norms and biases 201 us, by a workgroup to a row 253; with RMS norms, which read fewer parameters, 188 and
  // 179, 8192 rows 81 and 82, 65536 x 1024 92 and 121; 65536 x 96 14, by workgroups 107, by whole waves 36.  Fewer rows by a thread to a
  // chunk: 24 x 4096 bf16 6.4 us, by half as many threads 7.8; 1000 x 7168 17.5, by a wave to a row 19.3.  Rows of more than 1024 chunks
  // by 1024 threads: 8192 x 16384 bf16 246 us, by 512 373, by 256 (which spill) 714
  const int wave = a.rows < 2048 ? 0 : chunks <= 32 ? 16 : chunks <= 1024 ? 64 : 0;
  const int G = wave ? wave : chunks <= 256 ? 256 : chunks <= 512 ? 512 : 1024;
  const int nv = per_thread(chunks, G);
  auto go = [&](auto g, auto n, auto shared) {
    forward<T, decltype(g)::value, decltype(n)::value, decltype(shared)::value, TAIL>(a, st);
  };
  using yes = std::true_type;
  using no = std::false_type;
  using g16 = integral_constant<int, 16>;
  using g64 = integral_constant<int, 64>;
  using g1024 = integral_constant<int, 1024>;
  if (G == 16 && nv == 1) go(g16{}, integral_constant<int, 1>{}, yes{});
  else if (G == 16) go(g16{}, integral_constant<int, 2>{}, yes{});
  else if (G == 64 && nv == 1) go(g64{}, integral_constant<int, 1>{}, yes{});
  else if (G == 64 && nv == 2) go(g64{}, integral_constant<int, 2>{}, yes{});
  else if (G == 64 && nv == 4) go(g64{}, integral_constant<int, 4>{}, yes{});
  else if (G == 64 && nv == 8) go(g64{}, integral_constant<int, 8>{}, yes{});
  else if (G == 64) go(g64{}, integral_constant<int, 16>{}, yes{});
  else if (G == 256) go(integral_constant<int, 256>{}, integral_constant<int, 1>{}, no{});
  else if (G == 512) go(integral_constant<int, 512>{}, integral_constant<int, 1>{}, no{});
  else if (nv == 1) go(g1024{}, integral_constant<int, 1>{}, no{});
  else if (nv == 2) go(g1024{}, integral_constant<int, 2>{}, no{});
  else if constexpr (sizeof(T) == 4) go(g1024{}, integral_constant<int, 4>{}, no{});
}

// The threads of the backward's groups.  Eight elements in a thread while registers hold what
// belongs to them: up to 1024 threads with two sums in bf16.  With four, or in fp32, 512 threads of sixteen (16384 x 7168 bf16, four sums:
// 314 us, 510 by 1024 of eight, which spill; 8192 x 7168 fp32, two: 278 and 310), but WIDE in fp32 with four (366; 726 and 887 otherwise);
// WIDE with sixteen beyond 8192 (8192 x 16384 bf16, two sums: 490 us, 796 with the next row's loads ahead, 702 by 512 threads of 32)
int backward_threads(int d, int dtype, bool bias) {
  if (d > 8192) return 1024;
  if (d > 4096) return (dtype == MOE_BF16) == bias ? 512 : 1024;
  int G = 16;
  while (G * 8 < d) G *= 2;
  return G;
}
int groups_in_block(int G) { return G <= 64 ? 256 / G : 1; }

// Groups of a launch: four rows for each one's sums, while that leaves one for every CU, and no more than fill the chip (1000 x 7168 bf16:
// 34 us by 256 groups, 41 by 128, 49 by 512; 10000 x 1024: 121, 67, 50 and 39 by 128, 256, 512 and 1024)
int64_t backward_groups(int64_t rows, int d, int G) {
  if (d <= 4096 && rows <= 4 * groups_in_block(G)) return std::min<int64_t>(rows, groups_in_block(G));  // one workgroup: one launch
  return std::min<int64_t>(std::max<int64_t>(rows / 4, std::min<int64_t>(rows, 256)), 256 * 1024 / G);
}

template <typename T, bool TAIL>
void backward(const ResidualLaunch& a, bool bias, int64_t groups, hipStream_t st) {
  constexpr int V8 = 8 / Chunk<T>::C;
  constexpr bool BF16 = sizeof(T) == 2;
  using one = integral_constant<int, V8>;
  using two = integral_constant<int, 2 * V8>;
  using none = std::false_type;
  using wide = std::true_type;
  auto go = [&](auto g, auto nv, auto sums, auto w) {
    constexpr int G = decltype(g)::value, NV = decltype(nv)::value, SUMS = decltype(sums)::value;
    constexpr bool WIDE = decltype(w)::value;
    constexpr int lds = WIDE ? 2 * NV * Chunk<T>::C * G * 4 : 0;
    const int per = groups_in_block(G);
    const auto kernel = k_residual_bwd<T, G, NV, SUMS, WIDE, TAIL>;
    if (lds > 65536 - 512) (void)hipFuncSetAttribute((const void*)kernel, hipFuncAttributeMaxDynamicSharedMemorySize, lds);
    hipLaunchKernelGGL(kernel, dim3((unsigned)((groups + per - 1) / per)), dim3(G * per), lds, st, a);
  };
  auto both = [&](auto g, auto nv, auto w) {
    if (bias) go(g, nv, integral_constant<int, 4>{}, w);
    else go(g, nv, integral_constant<int, 2>{}, w);
  };
  const int G = backward_threads(a.d, a.dtype, bias);
  if (a.d > 8192) both(integral_constant<int, 1024>{}, two{}, wide{});
  else if (a.d > 4096) {  // as the plan has it
    if (bias) go(integral_constant<int, BF16 ? 512 : 1024>{}, std::conditional_t<BF16, two, one>{}, integral_constant<int, 4>{},
                 std::conditional_t<BF16, none, wide>{});
    else go(integral_constant<int, BF16 ? 1024 : 512>{}, std::conditional_t<BF16, one, two>{}, integral_constant<int, 2>{}, none{});
  } else if (G == 512) both(integral_constant<int, 512>{}, one{}, none{});
  else if (G == 256) both(integral_constant<int, 256>{}, one{}, none{});
  else if (G == 128) both(integral_constant<int, 128>{}, one{}, none{});
  else if (G == 64) both(integral_constant<int, 64>{}, one{}, none{});
  else if (G == 32) both(integral_constant<int, 32>{}, one{}, none{});
  else both(integral_constant<int, 16>{}, one{}, none{});
}

}  // namespace

int64_t residual_partial_floats(int64_t rows, int d, int dtype) {
  int64_t most = 0;
  for (const bool bias : {false, true}) {
    const int G = backward_threads(d, dtype, bias);
    const int64_t per = groups_in_block(G);
    most = std::max(most, (backward_groups(rows, d, G) + per - 1) / per * (bias ? 4 : 2) * d);
  }
  return most;
}

int launch_residual(const ResidualLaunch& of, hipStream_t st) {
  ResidualLaunch a = of;
  const bool tb = a.dtype == MOE_BF16, tail = a.d % (tb ? 8 : 4) != 0;
  // Stores past the caches where the rows that the call moves are more than the 256 MB last-level cache: its inputs, just written by the
  // calls before, are then not driven out by results that would not stay either (16384 x 7168 bf16 forward 196 -> 188 us, 8192 x 7168
  // 107 -> 80; backward 285 -> 283 and 152 both).  Below that the next call finds the results there
  a.past = (a.backward ? 6 : 4) * a.rows * a.d * (tb ? 2 : 4) > 256ll << 20;
  if (!a.backward) {
    if (a.rows == 0) return 0;
    if (tb && tail) forward<bf16_t, true>(a, st);
    else if (tb) forward<bf16_t, false>(a, st);
    else if (tail) forward<float, true>(a, st);
    else forward<float, false>(a, st);
    return hipGetLastError() == hipSuccess ? 0 : -1;
  }
  // sums of c D and dn too, for the biases' gradients and post_bias's part of the gate's
  const bool bias = a.p.post_bias || a.d_post_bias || a.d_pre_bias;
  const int G = backward_threads(a.d, a.dtype, bias);
  const int64_t groups = backward_groups(a.rows, a.d, G), per = groups_in_block(G);
  if (a.rows > 0) {
    if (tb && tail) backward<bf16_t, true>(a, bias, groups, st);
    else if (tb) backward<bf16_t, false>(a, bias, groups, st);
    else if (tail) backward<float, true>(a, bias, groups, st);
    else backward<float, false>(a, bias, groups, st);
  }
  const int n = (int)((groups + per - 1) / per);
  if ((a.d_post_weight || a.d_post_bias || a.d_gate || a.d_pre_weight || a.d_pre_bias) && !(n == 1 && a.d <= 4096))
    hipLaunchKernelGGL(k_residual_params, dim3((unsigned)((a.d + 63) / 64), 2), dim3(1024), 0, st, a, n, bias ? 4 : 2);
  return hipGetLastError() == hipSuccess ? 0 : -1;
}
