// The shared expert: the dense gated feed-forward block, forward and backward (formulas in include/moe_overlap.h).
#include <algorithm>
#include <type_traits>

#include "common.h"
#include "launch.h"
#include "tile_util.h"

namespace {

// What a product's epilogue does with its fp32 sums
enum Epi {
  EPI_GLU,    // gate and up sums of the same columns -> h, and g | u where wanted
  EPI_DGLU,   // dh -> dg | du, with the forward's g | u
  EPI_STORE,  // C (+ residual)
};

// One product C[m, n] = sum_k A(m, k) B(n, k).  An operand is "by rows" where its k runs along memory (element (m, k) at
// m * ld + k) and "by columns" where its m or n does (k * ld + m).  a_seg, a_jump: the contiguous index of A from a_seg on
// lies a_jump elements further (the two halves of g | u, whose rows are padded).
struct Gemm {
  const void *a, *b;
  int64_t lda, ldb;
  int a_seg, a_jump;
  int M, N, K;
  // epilogue
  void* c;  // GLU: h; DGLU: dg | du; STORE: C
  int64_t ldc;
  const void* residual;  // STORE
  float* gu;             // GLU: g | u or null; DGLU: g | u
  int64_t ldgu;
  int half;  // GLU, DGLU: from a row's g to its u (and dg to du)
  int up;    // GLU: rows of B from the gate's to the up projection's
};

template <typename T>
__device__ __forceinline__ float as_float(T v);
template <>
__device__ __forceinline__ float as_float(float v) { return v; }
template <>
__device__ __forceinline__ float as_float(bf16_t v) { return bf16_to_f32(v); }
__device__ __forceinline__ void put(float* p, float v) { *p = v; }
__device__ __forceinline__ void put(bf16_t* p, float v) { *p = f32_to_bf16(v); }

__device__ __forceinline__ void dglu(float dh, float g, float u, float* dg, float* du) {
  const float s = 1.0f / (1.0f + __expf(-g));
  *dg = dh * u * s * (1.0f + g * (1.0f - s));
  *du = dh * g * s;
}

// ---- any sizes, any type: fp32 matrix instructions ------------------------------------------------------------------
// A 128 x 64 tile of C (GLU: 32 columns of the gate and the same 32 of the up projection) by four waves of 32 x 64, in
// k-tiles of 16: each operand's k-tile is loaded by elements of its own layout into registers one k-tile ahead, widened
// to fp32 and kept in LDS as [k][m], from where a lane takes one element of A and two of B for two 32x32x2 products.
constexpr int GM = 128, GN = 64, GK = 16, GSUM = 256;

template <typename T, int EPI, bool ACOL, bool BCOL>
__global__ __launch_bounds__(256) void k_gemm_any(Gemm p) {
  __shared__ float sa[2][GK][GM + 4], sb[2][GK][GN + 4];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  constexpr int BN = EPI == EPI_GLU ? GN / 2 : GN;
  const int nt = (p.N + BN - 1) / BN;
  const int m0 = (int)(blockIdx.x / nt) * GM, n0 = (int)(blockIdx.x % nt) * BN;
  const T *A = (const T*)p.a, *B = (const T*)p.b;

  // thread -> four neighbours along memory: by rows (row tid / 4, k 4 (tid % 4)), by columns (k tid / 16 or 32, m ..)
  float ra[8], rb[4];
  auto load_a = [&](int k0) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        int m, k;
        if (ACOL) {
          k = k0 + (tid >> 5) + 8 * h;
          m = m0 + (tid & 31) * 4 + i;
        } else {
          m = m0 + (tid >> 2) + 64 * h;
          k = k0 + (tid & 3) * 4 + i;
        }
        float v = 0.f;
        if (m < p.M && k < p.K) {
          const int c = ACOL ? m : k;
          v = as_float(A[(int64_t)(ACOL ? k : m) * p.lda + c + (c >= p.a_seg ? p.a_jump : 0)]);
        }
        ra[4 * h + i] = v;
      }
    }
  };
  auto load_b = [&](int k0) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      int n, k;
      if (BCOL) {
        k = k0 + (tid >> 4);
        n = (tid & 15) * 4 + i;
      } else {
        n = tid >> 2;
        k = k0 + (tid & 3) * 4 + i;
      }
      int64_t row = n0 + n;
      bool in = row < p.N;
      if (EPI == EPI_GLU) {
        const int c = n0 + (n & (BN - 1));
        in = c < p.N;
        row = n < BN ? c : (int64_t)p.up + c;
      }
      rb[i] = in && k < p.K ? as_float(B[BCOL ? (int64_t)k * p.ldb + row : row * p.ldb + k]) : 0.f;
    }
  };
  auto keep = [&](int s) {
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        if (ACOL) sa[s][(tid >> 5) + 8 * h][(tid & 31) * 4 + i] = ra[4 * h + i];
        else sa[s][(tid & 3) * 4 + i][(tid >> 2) + 64 * h] = ra[4 * h + i];
      }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if (BCOL) sb[s][tid >> 4][(tid & 15) * 4 + i] = rb[i];
      else sb[s][(tid & 3) * 4 + i][tid >> 2] = rb[i];
    }
  };

  // sums of GSUM k each, added up: one running sum over thousands of products would lose a few bits that sums of sums keep
  f32x16_t acc[2], total[2];
#pragma unroll
  for (int j = 0; j < 2; ++j)
#pragma unroll
    for (int q = 0; q < 16; ++q) acc[j][q] = total[j][q] = 0.f;
  const int nk = (p.K + GK - 1) / GK;
  if (nk > 0) {
    load_a(0);
    load_b(0);
    keep(0);
  }
  for (int kt = 0; kt < nk; ++kt) {
    __syncthreads();
    const int s = kt & 1;
    if (kt + 1 < nk) {
      load_a((kt + 1) * GK);
      load_b((kt + 1) * GK);
    }
#pragma unroll
    for (int k = 0; k < GK; k += 2) {
      const float a = sa[s][k + (lane >> 5)][wave * 32 + (lane & 31)];
#pragma unroll
      for (int j = 0; j < 2; ++j)
        acc[j] = __builtin_amdgcn_mfma_f32_32x32x2f32(a, sb[s][k + (lane >> 5)][j * 32 + (lane & 31)], acc[j], 0, 0, 0);
    }
    if (kt + 1 < nk) keep(s ^ 1);  // its last readers passed this k-tile's barrier
    if (kt % (GSUM / GK) == GSUM / GK - 1 || kt + 1 == nk) {
#pragma unroll
      for (int j = 0; j < 2; ++j)
#pragma unroll
        for (int q = 0; q < 16; ++q) {
          total[j][q] += acc[j][q];
          acc[j][q] = 0.f;
        }
    }
  }

  // element q of an accumulator: row 8 (q / 4) + 4 (lane / 32) + q % 4, column lane % 32
#pragma unroll
  for (int q = 0; q < 16; ++q) {
    const int m = m0 + wave * 32 + 8 * (q >> 2) + 4 * (lane >> 5) + (q & 3);
    if (m >= p.M) continue;
    if (EPI == EPI_GLU) {
      const int n = n0 + (lane & 31);
      if (n >= p.N) continue;
      const float g = total[0][q], u = total[1][q];
      put((T*)p.c + m * p.ldc + n, g / (1.0f + __expf(-g)) * u);
      if (p.gu) {
        float* o = p.gu + m * p.ldgu + n;
        o[0] = g;
        o[p.half] = u;
      }
      continue;
    }
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const int n = n0 + j * 32 + (lane & 31);
      if (n >= p.N) continue;
      if (EPI == EPI_DGLU) {
        const float* i = p.gu + m * p.ldgu + n;
        float dg, du;
        dglu(total[j][q], i[0], i[p.half], &dg, &du);
        T* o = (T*)p.c + m * p.ldc + n;
        put(o, dg);
        put(o + p.half, du);
      } else {
        const int64_t at = m * p.ldc + n;
        put((T*)p.c + at, total[j][q] + (p.residual ? as_float(((const T*)p.residual)[at]) : 0.f));
      }
    }
  }
}

template <typename T, int EPI, bool ACOL, bool BCOL>
int gemm_any(const Gemm& p, hipStream_t st) {
  if (p.M == 0) return 0;
  constexpr int BN = EPI == EPI_GLU ? GN / 2 : GN;
  const int64_t tiles = (int64_t)((p.M + GM - 1) / GM) * ((p.N + BN - 1) / BN);
  if (tiles > 0x7fffffff) return -1;
  hipLaunchKernelGGL((k_gemm_any<T, EPI, ACOL, BCOL>), dim3((unsigned)tiles), dim3(256), 0, st, p);
  return hipGetLastError() == hipSuccess ? 0 : -1;
}

// ---- the block --------------------------------------------------------------------------------------------------

struct Block {  // one call's products
  Gemm glu, down;                  // forward
  Gemm dglu, dx, dw_gate_up, dw_down;  // backward
};

Block block_of(const SharedLaunch& s) {
  Block b{};
  const int T = (int)s.tokens, d = s.d, f = s.f, F = s.row, none = 0x7fffffff;
  b.glu = {s.x, s.w_gate_up, d, d, none, 0, T, f, d, s.h, F, nullptr, s.gu, 2 * F, F, f};
  b.down = {s.h, s.w_down, F, f, none, 0, T, d, f, s.y, d, s.residual, nullptr, 0, 0, 0};
  b.dglu = {s.dy, s.w_down, d, f, none, 0, T, f, d, s.dgu, 2 * F, nullptr, s.gu, 2 * F, F, 0};
  b.dx = {s.dgu, s.w_gate_up, 2 * F, d, f, F - f, T, d, 2 * f, s.dx, d, s.residual, nullptr, 0, 0, 0};
  b.dw_gate_up = {s.dgu, s.x, 2 * F, d, f, F - f, 2 * f, d, T, s.dw_gate_up, d, nullptr, nullptr, 0, 0, 0};
  b.dw_down = {s.dy, s.h, d, F, none, 0, d, f, T, s.dw_down, f, nullptr, nullptr, 0, 0, 0};
  return b;
}

template <typename T>
int run_any(const SharedLaunch& s, hipStream_t st) {
  const Block b = block_of(s);
  int rc;
  if (!s.backward) {
    if ((rc = gemm_any<T, EPI_GLU, false, false>(b.glu, st))) return rc;
    return gemm_any<T, EPI_STORE, false, false>(b.down, st);
  }
  if ((rc = gemm_any<T, EPI_DGLU, false, true>(b.dglu, st))) return rc;
  if ((rc = gemm_any<T, EPI_STORE, false, true>(b.dx, st))) return rc;
  if ((rc = gemm_any<T, EPI_STORE, true, true>(b.dw_gate_up, st))) return rc;
  return gemm_any<T, EPI_STORE, true, true>(b.dw_down, st);
}

}  // namespace

int64_t shared_workspace_bytes(int64_t tokens, int d, int f, int dtype, bool backward) { return 0; }

int launch_shared(const SharedLaunch& s, hipStream_t st) {
  return s.dtype == MOE_BF16 ? run_any<bf16_t>(s, st) : run_any<float>(s, st);
}
