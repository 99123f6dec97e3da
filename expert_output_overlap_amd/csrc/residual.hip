// The norms around a block with its gate and the residual's scale, forward and backward (formulas in include/moe_overlap.h).
#include <algorithm>
#include <type_traits>

#include "common.h"
#include "launch.h"
#include "row_util.h"

namespace {

// A row's statistics over the G threads that hold it, NV chunks each in v (elements past the row are 0).  turn picks the one of
// red's two halves that the last sum did not use
template <int G, int NV, int C>
__device__ __forceinline__ void row_stats(const float (&v)[NV * C], int kind, int t, int d, float eps, float (*red)[2 * (G / 64)],
                                          int& turn, float* mean_out, float* rstd_out) {
  float mean = 0.f, off = 0.f;
  if (kind == MOE_NORM_NONE) {
    *mean_out = 0.f;
    *rstd_out = 1.f;
    return;
  }
  if (kind == MOE_NORM_LAYER) {
    float s[1] = {0.f};
#pragma unroll
    for (int e = 0; e < NV * C; ++e) s[0] += v[e];
    group_sum<G>(s, red[turn]);
    turn ^= 1;
    mean = s[0] / d;
  }
  float q[2] = {0.f, 0.f};
#pragma unroll
  for (int j = 0; j < NV; ++j)
#pragma unroll
    for (int i = 0; i < C; ++i) {
      const float e = v[j * C + i] - mean;
      if ((j * G + t) * C + i < d) {
        q[0] = fmaf(e, e, q[0]);
        q[1] += e;
      }
    }
  group_sum<G>(q, red[turn]);
  turn ^= 1;
  if (kind == MOE_NORM_LAYER) {  // the differences' own sum corrects the mean's rounding
    off = q[1] / d;
    mean += off;
  }
  *mean_out = mean;
  *rstd_out = 1.0f / sqrtf(fmaxf(q[0] / d - off * off, 0.f) + eps);
}

template <typename T, int G, int NV>
__device__ __forceinline__ void load_row(const void* base, int64_t row, int64_t stride, int t, int d, float* out) {
  using K = Chunk<T>;
  constexpr int C = K::C;
  const T* p = (const T*)base + row * stride;
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    const int c = (j * G + t) * C;
    const u32x4 v = c < d ? K::load(p + c, d - c) : u32x4{0, 0, 0, 0};
#pragma unroll
    for (int i = 0; i < C; ++i) out[j * C + i] = K::at(v, i);
  }
}

template <typename T, int G, int NV>
__device__ __forceinline__ void store_row(void* base, int64_t row, int64_t stride, int t, int d, const float* v) {
  using K = Chunk<T>;
  constexpr int C = K::C;
  T* p = (T*)base + row * stride;
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    const int c = (j * G + t) * C;
    if (c < d) K::store(p + c, K::pack(v + j * C), d - c);
  }
}

template <typename PT, int C, int G, int NV>
__device__ __forceinline__ void load_params(const void* p, int t, int d, float empty, float* out) {
#pragma unroll
  for (int j = 0; j < NV; ++j) params<PT, C>((const PT*)p, (j * G + t) * C, d, empty, out + j * C);
}

template <typename T, typename PT, int G, int NV>
__global__ __launch_bounds__(G < 256 ? 256 : G) void k_residual(ResidualLaunch a) {
  constexpr int C = Chunk<T>::C, PER = G < 256 ? 256 / G : 1, E = NV * C;
  __shared__ float red[2][2 * (G / 64)];
  const int t = threadIdx.x % G, d = a.d;
  int turn = 0;
  for (int64_t r = (int64_t)blockIdx.x * PER + threadIdx.x / G; r < a.rows; r += (int64_t)gridDim.x * PER) {
    float h[E], s[E], p[E], q[E];
    load_row<T, G, NV>(a.h, r, a.h_stride, t, d, h);
    load_row<T, G, NV>(a.x, r, a.x_stride, t, d, s);
    float m1, r1, m2, r2;
    row_stats<G, NV, C>(h, a.post, t, d, a.eps, red, turn, &m1, &r1);
    const float c = a.p.row_gate ? a.p.row_gate[r] : 1.f;
    load_params<PT, C, G, NV>(a.p.post_weight, t, d, 1.f, p);
    load_params<PT, C, G, NV>(a.p.post_bias, t, d, 0.f, q);
#pragma unroll
    for (int e = 0; e < E; ++e) h[e] = fmaf((h[e] - m1) * r1, p[e], q[e]);
    load_params<PT, C, G, NV>(a.p.gate, t, d, 1.f, p);
#pragma unroll
    for (int j = 0; j < NV; ++j)
#pragma unroll
      for (int i = 0; i < C; ++i) {
        const int e = j * C + i;
        s[e] = (j * G + t) * C + i < d ? fmaf(a.rho, s[e], c * (p[e] * h[e])) : 0.f;
      }
    store_row<T, G, NV>(a.s, r, a.s_stride, t, d, s);
    row_stats<G, NV, C>(s, a.pre, t, d, a.eps, red, turn, &m2, &r2);
    if (a.pre != MOE_NORM_NONE) {
      load_params<PT, C, G, NV>(a.p.pre_weight, t, d, 1.f, p);
      load_params<PT, C, G, NV>(a.p.pre_bias, t, d, 0.f, q);
#pragma unroll
      for (int e = 0; e < E; ++e) s[e] = fmaf((s[e] - m2) * r2, p[e], q[e]);
      store_row<T, G, NV>(a.n, r, a.n_stride, t, d, s);
    }
    if (t == 0 && a.stats) *(float4*)(a.stats + 4 * r) = float4{m1, r1, m2, r2};
  }
}

// dx and dh of a group's rows, and its sums of c D h^, c D, dn s^ and dn, which stay in registers over all of its rows and go to
// the workspace at the end: partial [workgroup][4][d].
template <typename T, typename PT, int G, int NV>
__global__ __launch_bounds__(G < 256 ? 256 : G) void k_residual_bwd(ResidualLaunch a) {
  constexpr int C = Chunk<T>::C, PER = G < 256 ? 256 / G : 1, E = NV * C;
  __shared__ float red[2][3 * (G / 64)];
  __shared__ float join[PER > 1 ? (PER - 1) * 4 * E * G : 1];
  const int t = threadIdx.x % G, d = a.d;
  float acc[4][E];
#pragma unroll
  for (int k = 0; k < 4; ++k)
#pragma unroll
    for (int e = 0; e < E; ++e) acc[k][e] = 0.f;
  int turn = 0;
  for (int64_t r = (int64_t)blockIdx.x * PER + threadIdx.x / G; r < a.rows; r += (int64_t)gridDim.x * PER) {
    const float4 st = *(const float4*)(a.stats + 4 * r);
    const float c = a.p.row_gate ? a.p.row_gate[r] : 1.f;
    float h[E], s[E], D[E], p[E], q[E], z[E];
    load_row<T, G, NV>(a.h, r, a.h_stride, t, d, h);
    load_row<T, G, NV>(a.x, r, a.x_stride, t, d, s);
    if (a.ds) load_row<T, G, NV>(a.ds, r, a.ds_stride, t, d, D);
    else
#pragma unroll
      for (int e = 0; e < E; ++e) D[e] = 0.f;
    load_params<PT, C, G, NV>(a.p.post_weight, t, d, 1.f, p);
    load_params<PT, C, G, NV>(a.p.post_bias, t, d, 0.f, q);
    float g[E];
    load_params<PT, C, G, NV>(a.p.gate, t, d, 1.f, g);
#pragma unroll
    for (int e = 0; e < E; ++e) {
      h[e] = (h[e] - st.x) * st.y;
      z[e] = g[e] * fmaf(h[e], p[e], q[e]);
      s[e] = fmaf(a.rho, s[e], c * z[e]);
    }
    if (a.pre != MOE_NORM_NONE) {
      float dn[E], w[E], v[2] = {0.f, 0.f};
      load_row<T, G, NV>(a.dn, r, a.dn_stride, t, d, dn);
      load_params<PT, C, G, NV>(a.p.pre_weight, t, d, 1.f, w);
#pragma unroll
      for (int e = 0; e < E; ++e) {
        s[e] = (s[e] - st.z) * st.w;
        acc[2][e] = fmaf(dn[e], s[e], acc[2][e]);
        acc[3][e] += dn[e];
        dn[e] *= w[e];
        v[0] += dn[e];
        v[1] = fmaf(dn[e], s[e], v[1]);
      }
      group_sum<G>(v, red[turn]);
      turn ^= 1;
      const float ma = a.pre == MOE_NORM_LAYER ? v[0] / d : 0.f, mn = v[1] / d;
#pragma unroll
      for (int e = 0; e < E; ++e) D[e] += st.w * (dn[e] - ma - s[e] * mn);
    }
    float o[E], v[3] = {0.f, 0.f, 0.f};
#pragma unroll
    for (int j = 0; j < NV; ++j)
#pragma unroll
      for (int i = 0; i < C; ++i) {
        const int e = j * C + i;
        if ((j * G + t) * C + i >= d) D[e] = 0.f;
        o[e] = a.rho * D[e];
        v[2] = fmaf(D[e], z[e], v[2]);
        D[e] *= c;
        acc[0][e] = fmaf(D[e], h[e], acc[0][e]);
        acc[1][e] += D[e];
        D[e] *= g[e] * p[e];
        v[0] += D[e];
        v[1] = fmaf(D[e], h[e], v[1]);
      }
    store_row<T, G, NV>(a.dx, r, a.dx_stride, t, d, o);
    group_sum<G>(v, red[turn]);
    turn ^= 1;
    const float ma = a.post == MOE_NORM_LAYER ? v[0] / d : 0.f, mn = a.post == MOE_NORM_NONE ? 0.f : v[1] / d;
#pragma unroll
    for (int e = 0; e < E; ++e) o[e] = st.y * (D[e] - ma - h[e] * mn);
    store_row<T, G, NV>(a.dh, r, a.dh_stride, t, d, o);
    if (t == 0 && a.d_row_gate) a.d_row_gate[r] = v[2];
  }
  if (!a.partial) return;
  if (PER > 1) {  // the workgroup's groups, one after another
    const int w = threadIdx.x / G;
    if (w > 0) {
      float* to = join + (w - 1) * 4 * E * G;
#pragma unroll
      for (int k = 0; k < 4; ++k)
#pragma unroll
        for (int e = 0; e < E; ++e) to[(k * E + e) * G + t] = acc[k][e];
    }
    __syncthreads();
    if (w > 0) return;
    for (int u = 0; u < PER - 1; ++u) {
      const float* from = join + u * 4 * E * G;
#pragma unroll
      for (int k = 0; k < 4; ++k)
#pragma unroll
        for (int e = 0; e < E; ++e) acc[k][e] += from[(k * E + e) * G + t];
    }
  }
  float* out = a.partial + (int64_t)blockIdx.x * 4 * d;
#pragma unroll
  for (int k = 0; k < 4; ++k)
#pragma unroll
    for (int j = 0; j < NV; ++j)
#pragma unroll
      for (int i = 0; i < C; ++i) {
        const int c = (j * G + t) * C + i;
        if (c < d) out[(int64_t)k * d + c] = acc[k][j * C + i];
      }
}

// The parameters' gradients from the workgroups' partial sums: 64 columns per workgroup, its 16 waves take every 16th partial row,
// and their sums are added in wave order.
template <typename PT>
__global__ __launch_bounds__(1024) void k_residual_params(ResidualLaunch a, int n) {
  __shared__ float red[15][4][64];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, c = blockIdx.x * 64 + lane, d = a.d;
  float s[4] = {0.f, 0.f, 0.f, 0.f};
  if (c < d)
    for (int k = wave; k < n; k += 16)
#pragma unroll
      for (int u = 0; u < 4; ++u) s[u] += a.partial[((int64_t)k * 4 + u) * d + c];
  if (wave > 0)
#pragma unroll
    for (int u = 0; u < 4; ++u) red[wave - 1][u][lane] = s[u];
  __syncthreads();
  if (wave > 0 || c >= d) return;
  for (int k = 0; k < 15; ++k)
#pragma unroll
    for (int u = 0; u < 4; ++u) s[u] += red[k][u][lane];
  auto param = [&](const void* p, float empty) {
    if (!p) return empty;
    return sizeof(PT) == 4 ? ((const float*)p)[c] : bf16_to_f32(((const bf16_t*)p)[c]);
  };
  auto put = [&](void* p, float v) {
    if (!p) return;
    if (sizeof(PT) == 4) ((float*)p)[c] = v;
    else ((bf16_t*)p)[c] = f32_to_bf16(v);
  };
  const float gate = param(a.p.gate, 1.f);
  put(a.d_post_weight, gate * s[0]);
  put(a.d_post_bias, gate * s[1]);
  put(a.d_gate, fmaf(param(a.p.post_weight, 1.f), s[0], param(a.p.post_bias, 0.f) * s[1]));
  put(a.d_pre_weight, s[2]);
  put(a.d_pre_bias, s[3]);
}

template <bool BWD, typename T, typename PT, int G, int NV>
void go(const ResidualLaunch& a, int64_t groups, hipStream_t st) {
  constexpr int PER = G < 256 ? 256 / G : 1;
  const dim3 grid((unsigned)((groups + PER - 1) / PER)), block(G < 256 ? 256 : G);
  if constexpr (!BWD) hipLaunchKernelGGL((k_residual<T, PT, G, NV>), grid, block, 0, st, a);
  else hipLaunchKernelGGL((k_residual_bwd<T, PT, G, NV>), grid, block, 0, st, a);
}

template <typename T, typename PT>
void pick(const ResidualLaunch& a, int G, int NV, int64_t groups, hipStream_t st) {
  auto both = [&](auto g, auto nv) {
    if (a.backward) go<true, T, PT, decltype(g)::value, decltype(nv)::value>(a, groups, st);
    else go<false, T, PT, decltype(g)::value, decltype(nv)::value>(a, groups, st);
  };
  using std::integral_constant;
  if (G == 64 && NV == 1) both(integral_constant<int, 64>{}, integral_constant<int, 1>{});
  else if (G == 64) both(integral_constant<int, 64>{}, integral_constant<int, 2>{});
  else if (G == 256 && NV == 1) both(integral_constant<int, 256>{}, integral_constant<int, 1>{});
  else if (G == 256 && NV == 2) both(integral_constant<int, 256>{}, integral_constant<int, 2>{});
  else if (G == 256) go<false, T, PT, 256, 4>(a, groups, st);
  else if (G == 1024) go<true, T, PT, 1024, 1>(a, groups, st);
  else if (NV == 4) both(integral_constant<int, 512>{}, integral_constant<int, 4>{});
  else if constexpr (sizeof(T) == 4) both(integral_constant<int, 512>{}, integral_constant<int, 8>{});
}

void plan(int d, int dtype, bool backward, int* G, int* NV) {
  const int chunks = (d * (dtype == MOE_BF16 ? 2 : 4) + 15) / 16;
  *G = chunks <= 128 ? 64 : chunks <= 512 ? 256 : chunks <= 1024 ? (backward ? 1024 : 256) : 512;
  const int per = (chunks + *G - 1) / *G;
  *NV = per <= 2 ? per : per <= 4 ? 4 : 8;
}

int64_t groups_of(int64_t rows, int G, int NV, bool backward) {
  const int64_t most = 256ll * 16 * 64 / G;
  return std::min(backward ? std::max(rows / 4, std::min<int64_t>(rows, 256)) : rows, most);
}

}  // namespace

int64_t residual_partial_floats(int64_t rows, int d, int dtype) {
  int G, NV;
  plan(d, dtype, true, &G, &NV);
  const int64_t per = G < 256 ? 256 / G : 1;
  return (groups_of(rows, G, NV, true) + per - 1) / per * 4 * d;
}

int launch_residual(const ResidualLaunch& a, hipStream_t st) {
  int G, NV;
  plan(a.d, a.dtype, a.backward, &G, &NV);
  const int64_t groups = groups_of(a.rows, G, NV, a.backward);
  const bool tb = a.dtype == MOE_BF16, pb = a.param_dtype == MOE_BF16;
  if (a.rows > 0) {
    if (tb && pb) pick<bf16_t, bf16_t>(a, G, NV, groups, st);
    else if (tb) pick<bf16_t, float>(a, G, NV, groups, st);
    else if (pb) pick<float, bf16_t>(a, G, NV, groups, st);
    else pick<float, float>(a, G, NV, groups, st);
  }
  if (a.backward && (a.d_post_weight || a.d_post_bias || a.d_gate || a.d_pre_weight || a.d_pre_bias)) {
    const int64_t per = G < 256 ? 256 / G : 1;
    const int n = (int)((groups + per - 1) / per);
    const dim3 grid((unsigned)((a.d + 63) / 64));
    if (pb) hipLaunchKernelGGL(k_residual_params<bf16_t>, grid, dim3(1024), 0, st, a, n);
    else hipLaunchKernelGGL(k_residual_params<float>, grid, dim3(1024), 0, st, a, n);
  }
  return hipGetLastError() == hipSuccess ? 0 : -1;
}
