// The global norm of many gradients, and clipping (formulas in include/moe_overlap.h).
//
// Both are bound by HBM: 138.5 million gradients' norm takes 44 us in bf16 (6.3 TB/s) and 94 in fp32 (5.9); clipped from fp32 into bf16
// another 131 (6.3 TB/s of 6 bytes read and written per element), in place in bf16 82, in fp32 193.  The tensors are cut
// into chunks of GRAD_CHUNK elements, each a record of the plan's table with its own address, so that a launch of many small tensors
// has no search; a workgroup takes every grid-th chunk.  A square and its sum are one fp64 instruction on this chip, at the fp32 rate:
// they hide behind the loads and need no care for the gradients' range.
#include <algorithm>

#include "common.h"
#include "join.h"
#include "launch.h"
#include "row_util.h"

namespace {

// Three workgroups on a CU: 138.5 million bf16 gradients 43.3 us, by two 43.6, by four 45, by eight 48, by one 68
constexpr int MAX_BLOCKS = 768;

// Sum of squares of a thread's part of a chunk
template <typename T>
__device__ __forceinline__ void squares(const GradChunk& k, double (&s)[2]) {
  using K = Chunk<T>;
  constexpr int C = K::C, STEPS = GRAD_CHUNK / C / 256;
  const T* g = (const T*)(__attribute__((address_space(1))) const T*)(uintptr_t)k.grad;
  u32x4 v[STEPS];
  if (k.n == GRAD_CHUNK) {
#pragma unroll
    for (int j = 0; j < STEPS; ++j) v[j] = load16(g + (j * 256 + threadIdx.x) * C);
  } else {
#pragma unroll
    for (int j = 0; j < STEPS; ++j) {
      const int at = (j * 256 + (int)threadIdx.x) * C;
      v[j] = at < k.n ? K::load(g + at, k.n - at) : u32x4{0, 0, 0, 0};
    }
  }
#pragma unroll
  for (int j = 0; j < STEPS; ++j)
#pragma unroll
    for (int i = 0; i < C; ++i) {
      const double d = K::at(v[j], i);
      s[i & 1] = fma(d, d, s[i & 1]);
    }
}

// The workgroup's sum in every thread, waves in order
__device__ __forceinline__ double block_sum(double v) {
  __shared__ double red[4];
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) v += __shfl_xor(v, o, 64);
  __syncthreads();
  if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = v;
  __syncthreads();
  return red[0] + red[1] + red[2] + red[3];
}

__global__ __launch_bounds__(256) void k_grad_norm(GradLaunch a) {
  __shared__ int flag;
  double s[2] = {0, 0};
  for (int64_t c = blockIdx.x; c < a.n_chunks; c += gridDim.x) {
    const GradChunk k = a.chunks[c];
    if (k.grad_bf16) squares<bf16_t>(k, s);
    else squares<float>(k, s);
  }
  double all = block_sum(s[0] + s[1]);
  if (gridDim.x > 1) {
    if (threadIdx.x == 0) hand_out(&a.partial[blockIdx.x], all);
    if (!last_of(a.counters, blockIdx.x, gridDim.x, &flag)) return;
    all = 0;
    for (unsigned i = threadIdx.x; i < gridDim.x; i += 256) all += take(&a.partial[i]);
    all = block_sum(all);
  }
  if (threadIdx.x > 0) return;
  const double norm = a.factor * sqrt(all), ratio = a.max_norm / (norm + 1e-6);
  *a.norm = (float)norm;
  // not fmin: a NaN stays one
  *a.scale = (float)(a.factor * (isinf(a.max_norm) || ratio >= 1 ? 1.0 : ratio));
}

// N bytes at any address, past the caches
template <int N>
__device__ __forceinline__ void put(void* to, const void* from) {
  typedef uint32_t V __attribute__((ext_vector_type(N / 4 < 4 ? N / 4 : 4), aligned(2)));
  V v[N / sizeof(V)];
  __builtin_memcpy(v, from, N);
#pragma unroll
  for (int i = 0; i < (int)(N / sizeof(V)); ++i) __builtin_nontemporal_store(v[i], (V*)to + i);
}

template <typename T, typename O>
__device__ __forceinline__ void scaled(const GradChunk& k, void* to, float f) {
  using K = Chunk<T>;
  constexpr int C = K::C, STEPS = GRAD_CHUNK / C / 256;
  const T* g = (const T*)(__attribute__((address_space(1))) const T*)(uintptr_t)k.grad;
  O* out = (O*)(__attribute__((address_space(1))) O*)(uintptr_t)to;
  u32x4 v[STEPS];
#pragma unroll
  for (int j = 0; j < STEPS; ++j) {
    const int at = (j * 256 + (int)threadIdx.x) * C;
    v[j] = k.n == GRAD_CHUNK ? load16(g + at) : at < k.n ? K::load(g + at, k.n - at) : u32x4{0, 0, 0, 0};
  }
#pragma unroll
  for (int j = 0; j < STEPS; ++j) {
    const int at = (j * 256 + (int)threadIdx.x) * C, n = k.n - at;
    float w[C];
#pragma unroll
    for (int i = 0; i < C; ++i) w[i] = K::at(v[j], i) * f;
    if (n <= 0) continue;
    if (n < C) {
#pragma unroll
      for (int i = 0; i < C; ++i)
        if (i < n) {
          if constexpr (sizeof(O) == 4) out[at + i] = w[i];
          else out[at + i] = f32_to_bf16(w[i]);
        }
    } else if constexpr (sizeof(O) == 4) put<4 * C>(out + at, w);
    else {
      uint32_t q[C / 2];
#pragma unroll
      for (int i = 0; i < C / 2; ++i) q[i] = bf16_bits(w[2 * i]) | bf16_bits(w[2 * i + 1]) << 16;
      put<2 * C>(out + at, q);
    }
  }
}

// The chunks backwards: what k_grad_norm read last may still be in the last-level cache, where results that go past the caches leave
// it (138.5 million fp32 gradients into bf16: norm and this 225 us, 250 with results through the caches and flat accesses)
__global__ __launch_bounds__(256) void k_grad_clip(GradLaunch a) {
  const float f = *a.scale;
  const GradChunk k = a.chunks[a.n_chunks - 1 - blockIdx.x];
  if (!k.out && f == 1.f) return;
  void* out = k.out ? k.out : (void*)k.grad;
  const bool to_bf16 = k.out ? k.out_bf16 : k.grad_bf16;
  if (k.grad_bf16) {
    if (to_bf16) scaled<bf16_t, bf16_t>(k, out, f);
    else scaled<bf16_t, float>(k, out, f);
  } else {
    if (to_bf16) scaled<float, bf16_t>(k, out, f);
    else scaled<float, float>(k, out, f);
  }
}

int sum_blocks(int64_t n_chunks) { return (int)std::max<int64_t>(1, std::min<int64_t>(n_chunks, MAX_BLOCKS)); }

}  // namespace

int64_t grad_counter_words(int64_t n_chunks) { return join_words(sum_blocks(n_chunks)); }
int64_t grad_partial_doubles(int64_t n_chunks) { return sum_blocks(n_chunks); }

int launch_grad_norm(const GradLaunch& a, hipStream_t st) {
  hipLaunchKernelGGL(k_grad_norm, dim3(sum_blocks(a.n_chunks)), dim3(256), 0, st, a);
  return hipGetLastError() == hipSuccess ? 0 : -1;
}

int launch_grad_clip(const GradLaunch& a, hipStream_t st) {
  if (a.n_chunks > 0) hipLaunchKernelGGL(k_grad_clip, dim3((unsigned)a.n_chunks), dim3(256), 0, st, a);
  return hipGetLastError() == hipSuccess ? 0 : -1;
}
