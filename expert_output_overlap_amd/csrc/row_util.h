// Rows of a matrix in 16-byte chunks, and sums over the threads that hold one, for the norms' kernels.
#pragma once

#include <type_traits>

#include "common.h"

namespace {

typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));

// 16 bytes at any address: global memory takes unaligned dwordx4 accesses, so a row may start anywhere
__device__ __forceinline__ u32x4 load16(const void* p) {
  u32x4 v;
  __builtin_memcpy(&v, p, 16);
  return v;
}
__device__ __forceinline__ void store16(void* p, u32x4 v) { __builtin_memcpy(p, &v, 16); }

template <typename T>
struct Chunk {  // elements of one 16-byte chunk
  static constexpr int C = 16 / sizeof(T);
  static __device__ __forceinline__ float at(const u32x4& v, int i) {
    if (sizeof(T) == 4) return __uint_as_float(v[i]);
    return __uint_as_float(i & 1 ? v[i / 2] & 0xffff0000u : v[i / 2] << 16);
  }
  static __device__ __forceinline__ u32x4 pack(const float* f) {
    u32x4 v;
    if (sizeof(T) == 4) {
#pragma unroll
      for (int i = 0; i < 4; ++i) v[i] = __float_as_uint(f[i]);
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i) v[i] = pack_bf16x2(f[2 * i], f[2 * i + 1]);
    }
    return v;
  }
  // n elements (1 .. C) from p, the others 0: a whole chunk in one load, the row's last piece by elements
  static __device__ __forceinline__ u32x4 load(const T* p, int n) {
    if (n >= C) return load16(p);
    u32x4 v = {0, 0, 0, 0};
#pragma unroll
    for (int i = 0; i < C; ++i)
      if (i < n) {
        if (sizeof(T) == 4) v[i] = *(const uint32_t*)(p + i);
        else v[i / 2] |= (uint32_t) * (const uint16_t*)(p + i) << (16 * (i & 1));
      }
    return v;
  }
  static __device__ __forceinline__ void store(T* p, u32x4 v, int n) {
    if (n >= C) return store16(p, v);
#pragma unroll
    for (int i = 0; i < C; ++i)
      if (i < n) {
        if (sizeof(T) == 4) *(uint32_t*)(p + i) = v[i];
        else *(uint16_t*)(p + i) = (uint16_t)(v[i / 2] >> (16 * (i & 1)));
      }
  }
};

// N parameters from index i on, `empty` where there are none (no parameters, or past d)
template <typename PT, int N>
__device__ __forceinline__ void params(const PT* p, int i, int d, float empty, float* out) {
  constexpr int C = Chunk<PT>::C;
#pragma unroll
  for (int k = 0; k < N; k += C) {
    constexpr int M = N < C ? N : C;
    u32x4 v = {0, 0, 0, 0};
    const int n = d - i - k;
    if (p && n > 0) v = Chunk<PT>::load(p + i + k, n < M ? n : M);
#pragma unroll
    for (int e = 0; e < M; ++e) out[k + e] = p && e < n ? Chunk<PT>::at(v, e) : empty;
  }
}

// The wave's sum in every lane: shifts inside rows of 16 lanes, then over the rows (DPP moves instead of trips through LDS)
__device__ __forceinline__ float lanes_sum(float v) {
  auto dpp = [](float x, auto ctrl, auto rows) {
    return __builtin_bit_cast(float, __builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, x), decltype(ctrl)::value,
                                                                 decltype(rows)::value, 0xf, false));
  };
  using all = std::integral_constant<int, 0xf>;
  v += dpp(v, std::integral_constant<int, 0x111>{}, all{});  // row_shr 1, 2, 4, 8
  v += dpp(v, std::integral_constant<int, 0x112>{}, all{});
  v += dpp(v, std::integral_constant<int, 0x114>{}, all{});
  v += dpp(v, std::integral_constant<int, 0x118>{}, all{});
  v += dpp(v, std::integral_constant<int, 0x142>{}, std::integral_constant<int, 0xa>{});  // row_bcast 15 into rows 1, 3
  v += dpp(v, std::integral_constant<int, 0x143>{}, std::integral_constant<int, 0xc>{});  // row_bcast 31 into rows 2, 3
  return __builtin_bit_cast(float, __builtin_amdgcn_readlane(__builtin_bit_cast(int, v), 63));
}

// Sums of N values over a group of G threads: over the wave, then over the group's waves through LDS.  `buf` alternates
// between calls, so a call's barrier also covers the reads of the call before it.
template <int G, int N>
__device__ __forceinline__ void group_sum(float (&v)[N], float* buf) {
#pragma unroll
  for (int n = 0; n < N; ++n) v[n] = lanes_sum(v[n]);
  if (G > 64) {
    const int wave = threadIdx.x >> 6;
    if ((threadIdx.x & 63) == 0) {
#pragma unroll
      for (int n = 0; n < N; ++n) buf[wave * N + n] = v[n];
    }
    __syncthreads();
#pragma unroll
    for (int n = 0; n < N; ++n) {
      v[n] = 0.f;
#pragma unroll
      for (int w = 0; w < G / 64; ++w) v[n] += buf[w * N + n];
    }
  }
}

// As group_sum for N <= 4, with fewer registers: the waves' sums meet in lanes of one wave, 16 to a value, instead of one register
// each (48 for the three values of 16 waves); and for G = 16 and 32, several groups in a wave.
template <int G, int N>
__device__ __forceinline__ void group_total(float (&v)[N], float* buf) {
  static_assert(N <= 4 && G <= 1024, "16 lanes to a value");
  auto dpp = [](float x, auto ctrl) {
    return __builtin_bit_cast(float, __builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, x), decltype(ctrl)::value, 0xf, 0xf, true));
  };
  if (G < 64) {  // lane ^ 1, lane ^ 2, then the halves mirrored, then lane ^ 16
#pragma unroll
    for (int n = 0; n < N; ++n) {
      v[n] += dpp(v[n], std::integral_constant<int, 0xB1>{});
      v[n] += dpp(v[n], std::integral_constant<int, 0x4E>{});
      v[n] += dpp(v[n], std::integral_constant<int, 0x141>{});
      v[n] += dpp(v[n], std::integral_constant<int, 0x140>{});
      if (G == 32) v[n] += __shfl_xor(v[n], 16, 64);
    }
    return;
  }
#pragma unroll
  for (int n = 0; n < N; ++n) v[n] = lanes_sum(v[n]);
  if (G > 64) {
    const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63, n = lane >> 4, w = lane & 15;
    if (lane == 0) {
#pragma unroll
      for (int k = 0; k < N; ++k) buf[wave * N + k] = v[k];
    }
    __syncthreads();
    float s = n < N && w < G / 64 ? buf[w * N + n] : 0.f;
    auto add = [&](auto ctrl) {
      s += __builtin_bit_cast(float, __builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, s), decltype(ctrl)::value, 0xf, 0xf, false));
    };
    add(std::integral_constant<int, 0x111>{});  // row_shr 1, 2, 4, 8
    add(std::integral_constant<int, 0x112>{});
    add(std::integral_constant<int, 0x114>{});
    add(std::integral_constant<int, 0x118>{});
#pragma unroll
    for (int k = 0; k < N; ++k)
      v[k] = __builtin_bit_cast(float, __builtin_amdgcn_readlane(__builtin_bit_cast(int, s), 16 * k + 15));
  }
}

}  // namespace
