// Layer norm, forward and backward (formulas in include/moe_overlap.h).
//
// Both are bound by HBM: forward 2, backward 3 (4 with a residual) row transfers per row.  A row is held in registers
// by a group of G threads, NV 16-byte chunks each (of the backward's rows of more than 8192 elements some in scratch: plan()),
// so it is read once and its variance is the mean of squared
// differences to the mean (no difference of large sums).  Groups walk the rows with a stride; the next row's loads go out
// before the current row's sums, which hides their latency behind the reductions, and the parameters stay in registers
// for all of a group's rows (as fp32 they are four times the bytes of a bf16 row: re-reading them through the L2 for every
// row would cost more than the row itself).
#include <algorithm>
#include <type_traits>

#include "common.h"
#include "launch.h"
#include "row_util.h"

namespace {

template <typename T, typename PT, int G, int NV>
__global__ __launch_bounds__(G < 256 ? 256 : G) void k_norm(NormLaunch a) {
  using K = Chunk<T>;
  constexpr int C = K::C, PER = G < 256 ? 256 / G : 1;  // PER groups in a workgroup
  __shared__ float red[2][2 * (G / 64)];
  const int t = threadIdx.x % G, d = a.d;
  float w[NV * C], b[NV * C];
  const PT *wp = (const PT*)a.weight, *bp = (const PT*)a.bias;
  const int64_t step = (int64_t)gridDim.x * PER;
  int64_t r = (int64_t)blockIdx.x * PER + threadIdx.x / G;
  u32x4 next[NV];
  auto fetch = [&](int64_t row) {
    const T* p = (const T*)a.x + row * a.x_stride;
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int c = (j * G + t) * C;
      next[j] = c < d ? K::load(p + c, d - c) : u32x4{0, 0, 0, 0};
    }
  };
  if (r < a.rows) fetch(r);  // before the parameters: a single row's sums then run while those arrive
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    params<PT, C>(wp, (j * G + t) * C, d, 1.f, w + j * C);
    params<PT, C>(bp, (j * G + t) * C, d, 0.f, b + j * C);
  }
  for (; r < a.rows; r += step) {
    u32x4 x[NV];
#pragma unroll
    for (int j = 0; j < NV; ++j) x[j] = next[j];
    if (r + step < a.rows) fetch(r + step);
    float s[1] = {0.f};
#pragma unroll
    for (int j = 0; j < NV; ++j)
#pragma unroll
      for (int i = 0; i < C; ++i) s[0] += K::at(x[j], i);  // elements past the row are 0
    group_sum<G>(s, red[0]);
    // the differences' own sum corrects the mean's rounding, which a row of equal elements would else carry, over
    // sqrt(eps), into its output
    float mean = s[0] / d;
    float q[2] = {0.f, 0.f};
#pragma unroll
    for (int j = 0; j < NV; ++j)
#pragma unroll
      for (int i = 0; i < C; ++i) {
        const float e = K::at(x[j], i) - mean;
        if ((j * G + t) * C + i < d) {
          q[0] = fmaf(e, e, q[0]);
          q[1] += e;
        }
      }
    group_sum<G>(q, red[1]);
    const float off = q[1] / d;
    mean += off;
    const float rstd = 1.0f / sqrtf(fmaxf(q[0] / d - off * off, 0.f) + a.eps);
    T* y = (T*)a.y + r * a.y_stride;
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int c = (j * G + t) * C;
      float o[C];
#pragma unroll
      for (int i = 0; i < C; ++i) o[i] = fmaf((K::at(x[j], i) - mean) * rstd, w[j * C + i], b[j * C + i]);
      if (c < d) K::store(y + c, K::pack(o), d - c);
    }
    if (t == 0 && a.mean) {
      a.mean[r] = mean;
      a.rstd[r] = rstd;
    }
  }
}

// dx of a group's rows, and its sums of dy n and dy, which stay in registers over all of its rows and go to the workspace
// at the end: partial [workgroup][2][d].
template <typename T, typename PT, int G, int NV>
__global__ __launch_bounds__(G < 256 ? 256 : G) void k_norm_bwd(NormLaunch a) {
  using K = Chunk<T>;
  constexpr int C = K::C, PER = G < 256 ? 256 / G : 1;
  __shared__ float red[2][2 * (G / 64)];
  __shared__ float join[PER > 1 ? (PER - 1) * 2 * NV * C * G : 1];
  const int t = threadIdx.x % G, d = a.d;
  const PT* wp = (const PT*)a.weight;
  float w[NV * C], dw[NV * C], db[NV * C];
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    params<PT, C>(wp, (j * G + t) * C, d, 1.f, w + j * C);
#pragma unroll
    for (int i = 0; i < C; ++i) dw[j * C + i] = db[j * C + i] = 0.f;
  }
  const int64_t step = (int64_t)gridDim.x * PER;
  int64_t r = (int64_t)blockIdx.x * PER + threadIdx.x / G;
  u32x4 nx[NV], ny[NV];
  float nmean = 0.f, nrstd = 0.f;
  auto fetch = [&](int64_t row) {
    const T* px = (const T*)a.x + row * a.x_stride;
    const T* py = (const T*)a.dy + row * a.y_stride;
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int c = (j * G + t) * C;
      nx[j] = c < d ? K::load(px + c, d - c) : u32x4{0, 0, 0, 0};
      ny[j] = c < d ? K::load(py + c, d - c) : u32x4{0, 0, 0, 0};
    }
    nmean = a.mean[row];
    nrstd = a.rstd[row];
  };
  if (r < a.rows) fetch(r);
  int turn = 0;
  for (; r < a.rows; r += step, turn ^= 1) {
    u32x4 x[NV], dy[NV], res[NV];
    const float mean = nmean, rstd = nrstd;
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      x[j] = nx[j];
      dy[j] = ny[j];
    }
    if (a.residual) {
      const T* pr = (const T*)a.residual + r * a.dx_stride;
#pragma unroll
      for (int j = 0; j < NV; ++j) {
        const int c = (j * G + t) * C;
        res[j] = c < d ? K::load(pr + c, d - c) : u32x4{0, 0, 0, 0};
      }
    }
    if (r + step < a.rows) fetch(r + step);
    float s[2] = {0.f, 0.f};  // sums of a and a n
#pragma unroll
    for (int j = 0; j < NV; ++j)
#pragma unroll
      for (int i = 0; i < C; ++i) {
        const int e = j * C + i;
        const float n = (K::at(x[j], i) - mean) * rstd, g = K::at(dy[j], i), v = g * w[e];
        dw[e] = fmaf(g, n, dw[e]);
        db[e] += g;
        s[0] += v;
        s[1] = fmaf(v, n, s[1]);
      }
    group_sum<G>(s, red[turn]);
    const float ma = s[0] / d, mn = s[1] / d;
    T* dx = (T*)a.dx + r * a.dx_stride;
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int c = (j * G + t) * C;
      float o[C];
#pragma unroll
      for (int i = 0; i < C; ++i) {
        const float n = (K::at(x[j], i) - mean) * rstd;
        o[i] = rstd * (K::at(dy[j], i) * w[j * C + i] - ma - n * mn);
        if (a.residual) o[i] += K::at(res[j], i);
      }
      if (c < d) K::store(dx + c, K::pack(o), d - c);
    }
  }
  if (!a.partial) return;
  if (PER > 1) {  // the workgroup's groups, one after another
    const int g = threadIdx.x / G;
    if (g > 0) {
      float* q = join + (g - 1) * 2 * NV * C * G;
#pragma unroll
      for (int e = 0; e < NV * C; ++e) {
        q[2 * e * G + t] = dw[e];
        q[(2 * e + 1) * G + t] = db[e];
      }
    }
    __syncthreads();
    if (g > 0) return;
    for (int k = 0; k < PER - 1; ++k) {
      const float* q = join + k * 2 * NV * C * G;
#pragma unroll
      for (int e = 0; e < NV * C; ++e) {
        dw[e] += q[2 * e * G + t];
        db[e] += q[(2 * e + 1) * G + t];
      }
    }
  }
  float* out = a.partial + (int64_t)blockIdx.x * 2 * d;
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    const int c = (j * G + t) * C;
#pragma unroll
    for (int i = 0; i < C; ++i)
      if (c + i < d) {
        out[c + i] = dw[j * C + i];
        out[d + c + i] = db[j * C + i];
      }
  }
}

// dweight | dbias from the workgroups' partial sums: 64 columns per workgroup, its 16 waves take every 16th partial row, and
// their sums are added in wave order.
template <typename PT>
__global__ __launch_bounds__(1024) void k_norm_params(const float* __restrict__ partial, int n, int d, PT* dweight,
                                                      PT* dbias) {
  __shared__ float red[15][64];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, c = blockIdx.x * 64 + lane;
  float s = 0.f;
  if (c < 2 * d) {
    const float* p = partial + c;
    for (int k = wave; k < n; k += 128) {
      float v[8];
#pragma unroll
      for (int u = 0; u < 8; ++u) v[u] = k + 16 * u < n ? p[(int64_t)(k + 16 * u) * 2 * d] : 0.f;
#pragma unroll
      for (int u = 0; u < 8; ++u) s += v[u];
    }
  }
  if (wave > 0) red[wave - 1][lane] = s;
  __syncthreads();
  if (wave > 0 || c >= 2 * d) return;
  for (int k = 0; k < 15; ++k) s += red[k][lane];
  PT* out = c < d ? dweight : dbias;
  if (!out) return;
  if (sizeof(PT) == 4) *(float*)(out + (c < d ? c : c - d)) = s;
  else *(bf16_t*)(out + (c < d ? c : c - d)) = f32_to_bf16(s);
}

template <bool BWD, typename T, typename PT, int G, int NV>
void go(const NormLaunch& a, int64_t groups, hipStream_t st) {
  constexpr int PER = G < 256 ? 256 / G : 1;
  const dim3 grid((unsigned)((groups + PER - 1) / PER)), block(G < 256 ? 256 : G);
  if constexpr (!BWD) hipLaunchKernelGGL((k_norm<T, PT, G, NV>), grid, block, 0, st, a);
  else hipLaunchKernelGGL((k_norm_bwd<T, PT, G, NV>), grid, block, 0, st, a);
}

template <typename T, typename PT>
void pick(const NormLaunch& a, int G, int NV, int64_t groups, hipStream_t st) {
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
  else if constexpr (sizeof(T) == 4) both(integral_constant<int, 512>{}, integral_constant<int, 8>{});  // bf16: 2048 chunks
}

// Group size and chunks per thread for a row.  In the backward few chunks per thread, since it keeps three fp32 values per
// element besides the row: 16384 bf16 rows of 7168 take 263 us by 256 threads of four chunks, 221 by 512 of two and 194 (4.85
// TB/s) by 1024 of one.  In the forward the fewer waves of a smaller group's sums are worth more: 103 us (4.6 TB/s) by 256
// threads of four, 110 by 512 of two, 160 by 1024 of one.
// More than 8192 elements in the backward: four chunks (bf16) or eight (fp32) in each of 512 threads, of whose values the compiler
// keeps 43-45 or 176-179 registers' worth in scratch; 8192 rows of 16384 take 385 us (2.1 TB/s) and 968 (1.7), of 8192 119 and 156.
void plan(int d, int dtype, bool backward, int* G, int* NV) {
  const int chunks = (d * (dtype == MOE_BF16 ? 2 : 4) + 15) / 16;
  *G = chunks <= 128 ? 64 : chunks <= 512 ? 256 : chunks <= 1024 ? (backward ? 1024 : 256) : 512;
  const int per = (chunks + *G - 1) / *G;
  *NV = per <= 2 ? per : per <= 4 ? 4 : 8;
}

// Groups of a launch on 256 CUs: few, so that a group's parameters are read once for many rows and its sums written once, but
// enough to keep every CU in waves to the end.  In the backward that is up to twice what registers leave room for at once (104 of them
// for a 7168-wide bf16 row: one group of 1024 threads on a CU), in the forward with four chunks too.
int64_t norm_groups(int64_t rows, int G, int NV, bool backward) {
  const int waves = backward ? (NV == 1 ? 32 : NV == 2 ? 16 : 8) : (NV <= 2 ? 64 : 24);  // of a CU
  const int64_t most = 256ll * waves * 64 / G;
  // backward: four rows for each group's sums, while that leaves a group for every CU
  return std::min(backward ? std::max(rows / 4, std::min<int64_t>(rows, 256)) : rows, most);
}

}  // namespace

int64_t norm_partial_floats(int64_t rows, int d, int dtype) {
  int G, NV;
  plan(d, dtype, true, &G, &NV);
  const int64_t per = G < 256 ? 256 / G : 1;
  return (norm_groups(rows, G, NV, true) + per - 1) / per * 2 * d;
}

int launch_norm(const NormLaunch& a, hipStream_t st) {
  int G, NV;
  plan(a.d, a.dtype, a.backward, &G, &NV);
  const int64_t groups = norm_groups(a.rows, G, NV, a.backward);
  const bool tb = a.dtype == MOE_BF16, pb = a.param_dtype == MOE_BF16;
  if (a.rows > 0) {
    if (tb && pb) pick<bf16_t, bf16_t>(a, G, NV, groups, st);
    else if (tb) pick<bf16_t, float>(a, G, NV, groups, st);
    else if (pb) pick<float, bf16_t>(a, G, NV, groups, st);
    else pick<float, float>(a, G, NV, groups, st);
  }
  if (a.backward && (a.dweight || a.dbias)) {
    const int64_t per = G < 256 ? 256 / G : 1;
    const int n = (int)((groups + per - 1) / per);
    const dim3 grid((unsigned)((2 * a.d + 63) / 64));
    if (pb)
      hipLaunchKernelGGL(k_norm_params<bf16_t>, grid, dim3(1024), 0, st, a.partial, n, a.d, (bf16_t*)a.dweight,
                         (bf16_t*)a.dbias);
    else
      hipLaunchKernelGGL(k_norm_params<float>, grid, dim3(1024), 0, st, a.partial, n, a.d, (float*)a.dweight,
                         (float*)a.dbias);
  }
  return hipGetLastError() == hipSuccess ? 0 : -1;
}
