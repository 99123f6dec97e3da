// The router's losses, per-expert counts and the gradient of the logits (formulas in include/moe_overlap.h).
#include <algorithm>

#include "common.h"
#include "launch.h"

namespace {

constexpr int MAX_PER_LANE = 16;  // G <= 1024
constexpr int MAX_BLOCKS = 1024;

// A sequence's rows [first, last), cut to [0, T)
__device__ __forceinline__ void span_of(const RouterLaunch& a, int s, int* first, int* last) {
  const int T = (int)a.tokens;
  if (!a.spans) {
    const int part = T / a.sequences;
    *first = s * part;
    *last = *first + part;
    return;
  }
  *first = min(max(a.spans[2 * (int64_t)s], 0), T);
  *last = min(max(a.spans[2 * (int64_t)s + 1], *first), T);
}

// The sequence of row t, or -1: the last one that begins at or before it, if it has not ended
__device__ __forceinline__ int sequence_of(const RouterLaunch& a, int t) {
  if (!a.spans) return t / ((int)a.tokens / a.sequences);
  int lo = 0, hi = a.sequences;
  while (lo < hi) {
    const int mid = (lo + hi) / 2;
    if (a.spans[2 * (int64_t)mid] <= t) lo = mid + 1;
    else hi = mid;
  }
  return lo > 0 && t < a.spans[2 * (int64_t)(lo - 1) + 1] ? lo - 1 : -1;
}

__device__ __forceinline__ double wave_sum_d(double v) {
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) v += __shfl_xor(v, o, 64);
  return v;
}

// counts = 0, and (the first workgroup) the sequences with rows and their rows
__global__ __launch_bounds__(256) void k_router_init(RouterLaunch a) {
  const int64_t n = (int64_t)a.sequences * a.experts;
  for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < n; i += (int64_t)gridDim.x * 256) a.counts[i] = 0;
  if (blockIdx.x > 0) return;
  __shared__ int red[2][4];
  int live = 0, rows = 0;
  for (int s = threadIdx.x; s < a.sequences; s += 256) {
    int first, last;
    span_of(a, s, &first, &last);
    live += last > first;
    rows += last - first;
  }
  live = wave_sum(live);
  rows = wave_sum(rows);
  if ((threadIdx.x & 63) == 0) {
    red[0][threadIdx.x >> 6] = live;
    red[1][threadIdx.x >> 6] = rows;
  }
  __syncthreads();
  if (threadIdx.x < 2) a.means[threadIdx.x] = red[threadIdx.x][0] + red[threadIdx.x][1] + red[threadIdx.x][2] + red[threadIdx.x][3];
}

__global__ __launch_bounds__(256) void k_router_count(RouterLaunch a) {
  const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (i >= a.tokens * a.top_k) return;
  const int s = sequence_of(a, (int)(i / a.top_k)), id = a.topk_idx[i];
  if (s >= 0 && id >= 0 && id < a.experts) atomicAdd(&a.counts[(int64_t)s * a.experts + id], 1);
}

// A row's probabilities by one wave, logits lane + 64 i in lane: e = exp(l - top), their sum (0: no expert; NaN for a NaN or +inf)
__device__ __forceinline__ void softmax_row(const RouterLaunch& a, int t, float* e, float* den, float* top) {
  const int lane = lane_id(), G = a.experts;
  const float* l = a.logits + (int64_t)t * G;
  float mx = -INFINITY;
#pragma unroll
  for (int i = 0; i < MAX_PER_LANE; ++i) {
    e[i] = lane + 64 * i < G ? l[lane + 64 * i] : -INFINITY;
    mx = fmaxf(mx, e[i]);
  }
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) mx = fmaxf(mx, __shfl_xor(mx, o, 64));
  if (mx == -INFINITY) mx = 0.f;
  float sum = 0.f;
#pragma unroll
  for (int i = 0; i < MAX_PER_LANE; ++i) {
    e[i] = expf(e[i] - mx);
    sum += e[i];
  }
  *den = wave_sum_f(sum);
  *top = mx;
}

// f of sequence s
__device__ __forceinline__ void load_f(const RouterLaunch& a, int s, float* f) {
  const int lane = lane_id(), G = a.experts;
  const int32_t* c = a.counts + (int64_t)s * G;
  float sum = 0.f;
  int n[MAX_PER_LANE], total = 0;
#pragma unroll
  for (int i = 0; i < MAX_PER_LANE; ++i) {
    n[i] = lane + 64 * i < G ? c[lane + 64 * i] : 0;
    total += n[i];
  }
  total = wave_sum(total);
  sum = total > 0 ? (float)G / (float)total : 0.f;
#pragma unroll
  for (int i = 0; i < MAX_PER_LANE; ++i) f[i] = (float)n[i] * sum;
}

__global__ __launch_bounds__(256) void k_router_loss(RouterLaunch a) {
  const int wave = threadIdx.x >> 6;
  double balance = 0, z = 0;
  for (int64_t t = (int64_t)blockIdx.x * 4 + wave; t < a.tokens; t += (int64_t)gridDim.x * 4) {
    const int s = sequence_of(a, (int)t);
    if (s < 0) continue;
    int first, last;
    span_of(a, s, &first, &last);
    float e[MAX_PER_LANE], f[MAX_PER_LANE], den, top, dot = 0.f;
    softmax_row(a, (int)t, e, &den, &top);
    if (den == 0.f) continue;
    load_f(a, s, f);
#pragma unroll
    for (int i = 0; i < MAX_PER_LANE; ++i) dot = fmaf(e[i], f[i], dot);
    dot = wave_sum_f(dot);
    const double lse = top + logf(den);
    balance += (double)(dot / den) / (double)(last - first);
    z += lse * lse;
  }
  __shared__ double red[2][4];
  if ((threadIdx.x & 63) == 0) {
    red[0][wave] = balance;
    red[1][wave] = z;
  }
  __syncthreads();
  if (threadIdx.x < 2) {
    const double* r = red[threadIdx.x];
    ((double*)a.workspace)[2 * blockIdx.x + threadIdx.x] = r[0] + r[1] + r[2] + r[3];
  }
}

__global__ __launch_bounds__(64) void k_router_finish(RouterLaunch a, int n) {
  const double* p = (const double*)a.workspace;
  double balance = 0, z = 0;
  for (int i = threadIdx.x; i < n; i += 64) {
    balance += p[2 * i];
    z += p[2 * i + 1];
  }
  balance = wave_sum_d(balance) / max(a.means[0], 1);
  z = wave_sum_d(z) / max(a.means[1], 1);
  if (threadIdx.x == 0) {
    a.losses[0] = (float)((double)a.balance * balance + (double)a.z * z);
    a.losses[1] = (float)balance;
    a.losses[2] = (float)z;
  }
}

__global__ __launch_bounds__(256) void k_router_bwd(RouterLaunch a) {
  const int lane = lane_id(), G = a.experts;
  const float dl = a.d_loss ? *a.d_loss : 1.f;
  const float cb = dl * a.balance / (float)max(a.means[0], 1), cz = 2.f * dl * a.z / (float)max(a.means[1], 1);
  for (int64_t t = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6); t < a.tokens; t += (int64_t)gridDim.x * 4) {
    const int s = sequence_of(a, (int)t);
    float o[MAX_PER_LANE];
#pragma unroll
    for (int i = 0; i < MAX_PER_LANE; ++i) o[i] = 0.f;
    if (s >= 0) {
      int first, last;
      span_of(a, s, &first, &last);
      float e[MAX_PER_LANE], den, top, dot = 0.f;
      softmax_row(a, (int)t, e, &den, &top);
      if (den != 0.f) {
        load_f(a, s, o);
        const float share = cb / (float)(last - first), inv = 1.f / den, lse = top + logf(den);
#pragma unroll
        for (int i = 0; i < MAX_PER_LANE; ++i) o[i] *= share;
        if (a.d_weights)
          for (int j = 0; j < a.top_k; ++j) {
            const int id = a.topk_idx[t * a.top_k + j];
            const float w = a.d_weights[t * a.top_k + j];
#pragma unroll
            for (int i = 0; i < MAX_PER_LANE; ++i)
              if (id == lane + 64 * i && id < G) o[i] += w;
          }
#pragma unroll
        for (int i = 0; i < MAX_PER_LANE; ++i) {
          e[i] *= inv;
          dot = fmaf(e[i], o[i], dot);
        }
        dot = wave_sum_f(dot);
#pragma unroll
        for (int i = 0; i < MAX_PER_LANE; ++i) o[i] = e[i] * (o[i] - dot + cz * lse);
      }
    }
#pragma unroll
    for (int i = 0; i < MAX_PER_LANE; ++i)
      if (lane + 64 * i < G) {
        const int64_t at = t * G + lane + 64 * i;
        if (a.dtype == MOE_F32) ((float*)a.dlogits)[at] = o[i];
        else ((bf16_t*)a.dlogits)[at] = f32_to_bf16(o[i]);
      }
  }
}

int row_blocks(int64_t tokens) { return (int)std::min<int64_t>((tokens + 3) / 4, MAX_BLOCKS); }

}  // namespace

int64_t router_workspace_bytes(int64_t tokens, int experts, int top_k, int sequences) { return 16ll * MAX_BLOCKS; }

int launch_router_loss(const RouterLaunch& a, hipStream_t st) {
  const int64_t cells = (int64_t)a.sequences * a.experts, slots = a.tokens * a.top_k;
  const int blocks = row_blocks(a.tokens);
  hipLaunchKernelGGL(k_router_init, dim3((unsigned)std::min<int64_t>((cells + 255) / 256, 1024)), dim3(256), 0, st, a);
  if (a.tokens > 0) {
    hipLaunchKernelGGL(k_router_count, dim3((unsigned)((slots + 255) / 256)), dim3(256), 0, st, a);
    hipLaunchKernelGGL(k_router_loss, dim3(blocks), dim3(256), 0, st, a);
  }
  hipLaunchKernelGGL(k_router_finish, dim3(1), dim3(64), 0, st, a, blocks);
  return hipGetLastError() == hipSuccess ? 0 : -1;
}

int launch_router_backward(const RouterLaunch& a, hipStream_t st) {
  if (a.tokens == 0) return 0;
  hipLaunchKernelGGL(k_router_bwd, dim3(row_blocks(a.tokens)), dim3(256), 0, st, a);
  return hipGetLastError() == hipSuccess ? 0 : -1;
}
