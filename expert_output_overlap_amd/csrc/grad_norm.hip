// The global norm of many gradients, and clipping (formulas in include/moe_overlap.h).
#include <algorithm>

#include "common.h"
#include "launch.h"

namespace {

constexpr int MAX_BLOCKS = 2048;

__device__ __forceinline__ float value(const void* p, bool bf16, int64_t i) {
  return bf16 ? bf16_to_f32(((const bf16_t*)p)[i]) : ((const float*)p)[i];
}

// The workgroup's sum in every thread, waves in order
__device__ __forceinline__ double block_sum(double v) {
  __shared__ double red[4];
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) v += __shfl_xor(v, o, 64);
  if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = v;
  __syncthreads();
  return red[0] + red[1] + red[2] + red[3];
}

__global__ __launch_bounds__(256) void k_grad_sum(GradLaunch a) {
  double s = 0;
  for (int64_t c = blockIdx.x; c < a.n_chunks; c += gridDim.x) {
    const GradChunk k = a.chunks[c];
    for (int i = threadIdx.x; i < k.n; i += 256) {
      const double g = value(k.grad, k.grad_bf16, i);
      s = fma(g, g, s);
    }
  }
  s = block_sum(s);
  if (threadIdx.x == 0) a.partial[blockIdx.x] = s;
}

__global__ __launch_bounds__(256) void k_grad_finish(GradLaunch a, int n) {
  double s = 0;
  for (int i = threadIdx.x; i < n; i += 256) s += a.partial[i];
  s = block_sum(s);
  if (threadIdx.x > 0) return;
  const double norm = a.factor * sqrt(s), ratio = a.max_norm / (norm + 1e-6);
  *a.norm = (float)norm;
  // not fmin: a NaN stays one
  *a.scale = (float)(a.factor * (isinf(a.max_norm) || ratio >= 1 ? 1.0 : ratio));
}

__global__ __launch_bounds__(256) void k_grad_clip(GradLaunch a) {
  const float f = *a.scale;
  const GradChunk k = a.chunks[blockIdx.x];
  if (!k.out && f == 1.f) return;
  void* out = k.out ? k.out : (void*)k.grad;
  const bool to_bf16 = k.out ? k.out_bf16 : k.grad_bf16;
  for (int i = threadIdx.x; i < k.n; i += 256) {
    const float v = value(k.grad, k.grad_bf16, i) * f;
    if (to_bf16) ((bf16_t*)out)[i] = f32_to_bf16(v);
    else ((float*)out)[i] = v;
  }
}

int sum_blocks(int64_t n_chunks) { return (int)std::min<int64_t>(n_chunks, MAX_BLOCKS); }

}  // namespace

int64_t grad_partial_doubles(int64_t n_chunks) { return sum_blocks(n_chunks); }

int launch_grad_norm(const GradLaunch& a, hipStream_t st) {
  const int n = sum_blocks(a.n_chunks);
  if (n > 0) hipLaunchKernelGGL(k_grad_sum, dim3(n), dim3(256), 0, st, a);
  hipLaunchKernelGGL(k_grad_finish, dim3(1), dim3(256), 0, st, a, n);
  return hipGetLastError() == hipSuccess ? 0 : -1;
}

int launch_grad_clip(const GradLaunch& a, hipStream_t st) {
  if (a.n_chunks > 0) hipLaunchKernelGGL(k_grad_clip, dim3((unsigned)a.n_chunks), dim3(256), 0, st, a);
  return hipGetLastError() == hipSuccess ? 0 : -1;
}
