// The shared expert: the dense gated feed-forward block, forward and backward (formulas in include/moe_overlap.h).
#include <algorithm>
#include <type_traits>

#include "common.h"
#include "launch.h"
#include "shared_tiles.h"
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
  int n_in;  // columns of C that B has, the others become 0 (N: a whole padded row of h, or of dg and du)
  // epilogue
  void* c;  // GLU: h; DGLU: dg | du; STORE: C
  int64_t ldc;
  const void* residual;  // STORE
  float* gu;             // GLU: g | u or null; DGLU: g | u
  int64_t ldgu;
  int half;  // GLU, DGLU: from a row's g to its u (and dg to du)
  int up;    // GLU: rows of B from the gate's to the up projection's
  // STORE: rows of C from m_pad on stand m_pad - m_real earlier; those in [m_real, m_pad) and those that would then stand
  // past 2 m_real are dg's and du's padding and stand nowhere
  int m_real, m_pad;
};

// ---- epilogues ----
// 4 columns of one row, any alignment; n: how many of them are inside the matrix
__device__ __forceinline__ void store4(bf16_t* p, f32x4_t v, int n) {
  const u32x2_t q = {bf16_bits(v[0]) | (bf16_bits(v[1]) << 16), bf16_bits(v[2]) | (bf16_bits(v[3]) << 16)};
  if (n >= 4) __builtin_memcpy(p, &q, 8);
  else
    for (int i = 0; i < n; ++i) p[i] = (bf16_t)(q[i >> 1] >> (16 * (i & 1)));
}
__device__ __forceinline__ void store4(float* p, f32x4_t v, int n) {
  if (n >= 4) __builtin_memcpy(p, &v, 16);
  else
    for (int i = 0; i < n; ++i) p[i] = v[i];
}
__device__ __forceinline__ f32x4_t load4(const bf16_t* p, int n) {
  u32x2_t q = {0, 0};
  if (n >= 4) __builtin_memcpy(&q, p, 8);
  else
    for (int i = 0; i < n; ++i) q[i >> 1] |= (uint32_t)p[i] << (16 * (i & 1));
  return f32x4_t{__uint_as_float(q[0] << 16), __uint_as_float(q[0] & 0xffff0000u), __uint_as_float(q[1] << 16),
                 __uint_as_float(q[1] & 0xffff0000u)};
}
__device__ __forceinline__ f32x4_t load4(const float* p, int n) {
  f32x4_t v = {0, 0, 0, 0};
  if (n >= 4) __builtin_memcpy(&v, p, 16);
  else
    for (int i = 0; i < n; ++i) v[i] = p[i];
  return v;
}

// 1 / (1 + exp(-g)).  bf16: with the hardware's reciprocal, 1 ulp off, in front of a rounding 2^15 times coarser
template <typename T>
__device__ __forceinline__ float sigmoid(float g) {
  return sizeof(T) == 2 ? __builtin_amdgcn_rcpf(1.0f + __expf(-g)) : 1.0f / (1.0f + __expf(-g));
}

// Four neighbouring columns n .. of row m through the epilogue (sum2: GLU's up sums).  Columns past n_in become 0 in h, gu and
// dgu, whatever was summed or stands there, and are cut in C.
template <typename T, int EPI>
__device__ __forceinline__ void finish4(const Gemm& p, int64_t m, int n, f32x4_t sum, f32x4_t sum2) {
  const int in = p.n_in - n;
  if (EPI == EPI_GLU) {
    f32x4_t h;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if (i >= in) sum[i] = sum2[i] = 0.f;
      h[i] = sum[i] * sigmoid<T>(sum[i]) * sum2[i];
    }
    store4((T*)p.c + m * p.ldc + n, h, 4);
    if (p.gu) {
      float* o = p.gu + m * p.ldgu + n;
      *(f32x4_t*)o = sum;
      *(f32x4_t*)(o + p.half) = sum2;
    }
  } else if (EPI == EPI_DGLU) {
    const float* i = p.gu + m * p.ldgu + n;
    const f32x4_t g = *(const f32x4_t*)i, u = *(const f32x4_t*)(i + p.half);
    f32x4_t dg, du;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const float s = sigmoid<T>(g[k]);
      dg[k] = k < in ? sum[k] * u[k] * s * (1.0f + g[k] * (1.0f - s)) : 0.f;
      du[k] = k < in ? sum[k] * g[k] * s : 0.f;
    }
    T* o = (T*)p.c + m * p.ldc + n;
    store4(o, dg, 4);
    store4(o + p.half, du, 4);
  } else {
    if (m >= p.m_pad) m -= p.m_pad - p.m_real;
    else if (m >= p.m_real) return;
    if (m >= 2ll * p.m_real) return;
    T* o = (T*)p.c + m * p.ldc + n;
    if (p.residual) sum += load4((const T*)p.residual + m * p.ldc + n, in);
    store4(o, sum, in);
  }
}

// A product as one or several of a launch's workgroups, one per tile and k-split
struct Part {
  Gemm p;
  int splits;
  int first, blocks;  // workgroups [first, first + blocks) of the launch; first is a multiple of 8
  float* partial;     // splits > 1: [splits][M][ld] sums
  int64_t ld;
};
// fp32: k of a partial sum at most, in the tiles and with few tokens: one running sum over thousands would lose a few bits
constexpr int FSUM = 256;

// ---- few tokens --------------------------------------------------------------------------------------------------------
// The weights stream past once and bound the time.  A workgroup takes RT x 16 rows of the weights (GLU with RT = 1: 8 of the
// gate's and the same 8 of the up projection's) as one operand of 16x16 products whose other is the tokens, 16 per product;
// its eight waves share out the k in chunks of 128 bytes of each row and add their sums in wave order at the end.  Which k
// of a chunk meet in which product does not matter as long as both operands agree.
//
// Rows that do not start at 16 bytes: a lane holds 32 neighbouring bytes of its row per chunk and gives them to the products
// as they were loaded, SU chunks in flight per wave.
template <typename T>
struct Chunk32 {  // 32 bytes of a row: 16 bf16 or 8 fp32
  u32x4_t v[2];
  static constexpr int N = 32 / sizeof(T);
  __device__ __forceinline__ void load(const T* p, int n) {  // n elements are there, the rest 0
    if (n >= N) {
      __builtin_memcpy(v, p, 32);
      return;
    }
    v[0] = v[1] = u32x4_t{0u, 0u, 0u, 0u};
#pragma unroll
    for (int i = 0; i < N; ++i)
      if (i < n) {
        if (sizeof(T) == 4) v[i / 4][i % 4] = *(const uint32_t*)(p + i);
        else v[i / 8][i / 2 % 4] |= (uint32_t) * (const uint16_t*)(p + i) << (16 * (i & 1));
      }
  }
};
// A wave's sums; fp32: fold() ends a partial sum and adds it to the whole
template <typename T, int RT, int MT>
struct FewSums {
  f32x4_t acc[RT][MT], total[sizeof(T) == 4 ? RT : 1][sizeof(T) == 4 ? MT : 1];
  __device__ __forceinline__ FewSums() {
#pragma unroll
    for (int t = 0; t < RT; ++t)
#pragma unroll
      for (int m = 0; m < MT; ++m) {
        acc[t][m] = f32x4_t{0.f, 0.f, 0.f, 0.f};
        if constexpr (sizeof(T) == 4) total[t][m] = acc[t][m];
      }
  }
  __device__ __forceinline__ void fold() {
    if constexpr (sizeof(T) == 4) {
#pragma unroll
      for (int t = 0; t < RT; ++t)
#pragma unroll
        for (int m = 0; m < MT; ++m) {
          total[t][m] += acc[t][m];
          acc[t][m] = f32x4_t{0.f, 0.f, 0.f, 0.f};
        }
    }
  }
  __device__ __forceinline__ f32x4_t of(int t, int m) const {
    if constexpr (sizeof(T) == 4) return total[t][m] + acc[t][m];
    else return acc[t][m];
  }
};
template <typename T>
__device__ __forceinline__ f32x4_t products(const Chunk32<T>& a, const Chunk32<T>& b, f32x4_t c) {
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    if constexpr (sizeof(T) == 2) {
      c = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8_t, a.v[h]), __builtin_bit_cast(bf16x8_t, b.v[h]), c,
                                                  0, 0, 0);
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i)
        c = __builtin_amdgcn_mfma_f32_16x16x4f32(__uint_as_float(a.v[h][i]), __uint_as_float(b.v[h][i]), c, 0, 0, 0);
    }
  }
  return c;
}

// The eight waves' sums in wave order, and the epilogue.  A product's element: row 4 (lane / 16) .. + 3 of the weights, token
// lane % 16
template <typename T, int EPI, int RT, int MT>
__device__ __forceinline__ void few_finish(const Part& a, int n0, int tid, const f32x4_t (*part)[RT * MT][64]) {
  const Gemm& p = a.p;
  const int lane = tid & 63;
  auto out = [&](int64_t m, int n, const f32x4_t& v, const f32x4_t& w) {
    if (a.partial) {
      float* o = a.partial + ((int64_t)blockIdx.y * p.M + m) * a.ld + n;
      *(f32x4_t*)o = v;
      if (EPI == EPI_GLU) *(f32x4_t*)(o + a.ld / 2) = w;
    } else finish4<T, EPI>(p, m, n, v, w);
  };
  auto sum = [&](int i, int l) {
    f32x4_t v = part[0][i][l];
#pragma unroll
    for (int k = 1; k < 8; ++k) v += part[k][i][l];
    return v;
  };
  if (EPI == EPI_GLU) {
    constexpr int L = RT == 1 ? 32 : 64;
    if (tid >= MT * L) return;
    const int m = tid / L, l = tid % L, tok = 16 * m + (l & 15), n = n0 + 4 * (l >> 4);
    if (tok >= p.M || n >= p.N) return;
    out(tok, n, sum(m, l), RT == 1 ? sum(m, l + 32) : sum(MT + m, l));
  } else {
    if (tid >= RT * MT * 64) return;
    const int i = tid >> 6, t = i / MT, m = i % MT, tok = 16 * m + (lane & 15), n = n0 + 16 * t + 4 * (lane >> 4);
    if (tok >= p.M || n >= p.N) return;
    out(tok, n, sum(i, lane), f32x4_t{0.f, 0.f, 0.f, 0.f});
  }
}

template <typename T, int EPI, int RT, int MT, int SU>
__global__ __launch_bounds__(512) void k_gemm_few(Part a) {
  const Gemm& p = a.p;
  constexpr int CH = 128 / sizeof(T), NW = 8;
  constexpr int COLS = EPI == EPI_GLU ? 8 * RT : 16 * RT;  // columns of C
  __shared__ f32x4_t part[NW][RT * MT][64];
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int n0 = blockIdx.x * COLS, r = lane & 15, q = lane >> 4;
  const T *w[RT], *x[MT];
#pragma unroll
  for (int t = 0; t < RT; ++t) {
    int c = EPI == EPI_GLU ? n0 + (RT == 1 ? r & 7 : r) : n0 + 16 * t + r;
    int64_t row = c < p.n_in ? c : 0;
    if (EPI == EPI_GLU && (RT == 1 ? r >= 8 : t == 1)) row += p.up;
    w[t] = (const T*)p.b + row * p.ldb + q * (32 / sizeof(T));
  }
#pragma unroll
  for (int t = 0; t < MT; ++t) x[t] = (const T*)p.a + (int64_t)(16 * t + r < p.M ? 16 * t + r : 0) * p.lda + q * (32 / sizeof(T));
  FewSums<T, RT, MT> sums;
  // this split's chunks that are full, [begin, whole)
  const int all = p.K / CH, begin = (int)((int64_t)all * blockIdx.y / a.splits), whole = (int)((int64_t)all * (blockIdx.y + 1) / a.splits);
  auto chunks = [&](int c, auto count, bool cut) {  // chunks c, c + NW, ..
    constexpr int U = decltype(count)::value;
    Chunk32<T> cw[U][RT], cx[U][MT];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int k = (c + u * NW) * CH, n = cut ? p.K - k - q * (int)(32 / sizeof(T)) : CH;
#pragma unroll
      for (int t = 0; t < RT; ++t) cw[u][t].load(w[t] + k, n);
#pragma unroll
      for (int m = 0; m < MT; ++m) cx[u][m].load(x[m] + k, n);
    }
    __builtin_amdgcn_sched_barrier(0);  // every load goes out before the first product waits for one
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
      for (int t = 0; t < RT; ++t)
#pragma unroll
        for (int m = 0; m < MT; ++m) sums.acc[t][m] = products(cw[u][t], cx[u][m], sums.acc[t][m]);
    static_assert(SU * CH <= FSUM, "fp32 sums end with the call");
    sums.fold();
  };
  int c = begin + wave;
  for (; c + (SU - 1) * NW < whole; c += SU * NW) chunks(c, std::integral_constant<int, SU>{}, false);
  if (SU >= 4 && c + ((SU + 1) / 2 - 1) * NW < whole) {
    chunks(c, std::integral_constant<int, (SU + 1) / 2>{}, false);
    c += (SU + 1) / 2 * NW;
  }
  for (; c < whole; c += NW) chunks(c, std::integral_constant<int, 1>{}, false);
  if (c == all && p.K % CH) chunks(c, std::integral_constant<int, 1>{}, true);
#pragma unroll
  for (int t = 0; t < RT; ++t)
#pragma unroll
    for (int m = 0; m < MT; ++m) part[wave][t * MT + m][lane] = sums.of(t, m);
  __syncthreads();
  few_finish<T, EPI, RT, MT>(a, n0, tid, part);
}

// Rows that start at 16 bytes: both operands through LDS.  Each wave has a ring of D slots of its own, which LDS-DMA loads of
// 8 rows of 128 bytes fill D chunks ahead; no barrier before the end.  A load asks the L2 for whole 128-byte lines, where the
// lanes' own 32 bytes above ask for each line in parts: 16 tokens of 4096 x 14336 take 69 us instead of 90 (64-byte rows: 90
// too), 24 tokens 83 instead of 107; 72 us is what the weights take at 4.9 TB/s.  Few slots suffice, since more of them let
// fewer workgroups into a CU.  16-byte piece c of row r of a slot stands at piece c ^ swz(r): a read's 16 rows hit all banks.
template <typename T, int EPI, int RT, int MT, int D>
__global__ __launch_bounds__(512) void k_gemm_ring(Part a) {
  const Gemm& p = a.p;
  constexpr int ES = sizeof(T), CK = 128 / ES, NW = 8, SLOT = (RT + MT) * 2048;
  constexpr int COLS = EPI == EPI_GLU ? 8 * RT : 16 * RT;  // columns of C
  extern __shared__ __align__(1024) unsigned char smem[];
  int tid = threadIdx.x;
  asm volatile("" : "+v"(tid));
  const int lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int n0 = blockIdx.x * COLS;
  const uint32_t ldb = (uint32_t)p.ldb * ES, lda = (uint32_t)p.lda * ES;
  auto wrow = [&](int t, int r) -> uint32_t {  // row r of weight tile t, from row n0 of the weights
    const int c = EPI == EPI_GLU ? (RT == 1 ? r & 7 : r) : 16 * t + r;
    const bool up = EPI == EPI_GLU && (RT == 1 ? r >= 8 : t == 1);
    return (uint32_t)((n0 + c < p.n_in ? c : 0) + (up ? p.up : 0)) * ldb;
  };
  auto xrow = [&](int t, int r) -> uint32_t { return (uint32_t)(16 * t + r < p.M ? 16 * t + r : 0) * lda; };
  auto swz = [](int r) { return (r & 7) ^ (r >> 3); };
  // load i of a tile: rows 8 i + lane / 8, piece lane % 8
  uint32_t off[RT + MT][2];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int r = 8 * i + (lane >> 3);
    const uint32_t piece = (uint32_t)((lane & 7) ^ swz(r)) << 4;
#pragma unroll
    for (int t = 0; t < RT + MT; ++t) off[t][i] = (t < RT ? wrow(t, r) : xrow(t - RT, r)) + piece;
  }
  const unsigned char* wbase = (const unsigned char*)p.b + (int64_t)n0 * ldb;
  const unsigned char* xbase = (const unsigned char*)p.a;
  unsigned char* ring = smem + wave * D * SLOT;
  const uint32_t lds0 = (uint32_t)(uintptr_t)ring;
  // this split's whole chunks, and this wave's of them
  const int all = p.K / CK, begin = (int)((int64_t)all * blockIdx.y / a.splits);
  const int chunks = (int)((int64_t)all * (blockIdx.y + 1) / a.splits) - begin, mine = chunks > wave ? (chunks - wave + NW - 1) / NW : 0;
  auto load = [&](int j) {  // this wave's chunk j
    const int64_t at = (int64_t)(begin + wave + j * NW) * 128;
    const uint32_t slot = lds0 + j % D * SLOT;
#pragma unroll
    for (int t = 0; t < RT + MT; ++t)
#pragma unroll
      for (int i = 0; i < 2; ++i) dma16((t < RT ? wbase : xbase) + at, off[t][i], slot + t * 2048 + i * 1024);
  };
  FewSums<T, RT, MT> sums;
  auto multiply = [&](const u32x4_t (&f)[RT + MT]) {
#pragma unroll
    for (int t = 0; t < RT; ++t)
#pragma unroll
      for (int m = 0; m < MT; ++m) {
        f32x4_t& c = sums.acc[t][m];
        if constexpr (ES == 2) {
          c = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8_t, f[t]), __builtin_bit_cast(bf16x8_t, f[RT + m]), c,
                                                      0, 0, 0);
        } else {
#pragma unroll
          for (int i = 0; i < 4; ++i)
            c = __builtin_amdgcn_mfma_f32_16x16x4f32(__uint_as_float(f[t][i]), __uint_as_float(f[RT + m][i]), c, 0, 0, 0);
        }
      }
  };
  const int r = lane & 15, q = lane >> 4;
  auto use = [&](int j) {
    const unsigned char* slot = ring + j % D * SLOT + r * 128;
    u32x4_t f[2][RT + MT];
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
      for (int t = 0; t < RT + MT; ++t) f[h][t] = *(const u32x4_t*)(slot + t * 2048 + (((4 * h + q) ^ swz(r)) << 4));
    if (j + D < mine) {
      asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");  // the slot is read: its next chunk may land
      load(j + D);
    }
    multiply(f[0]);
    multiply(f[1]);
    if (j % (FSUM / CK) == FSUM / CK - 1) sums.fold();
  };
#pragma unroll
  for (int j = 0; j < D; ++j)
    if (j < mine) load(j);
  int j = 0;
  for (; j + D <= mine; ++j) {  // D - 1 chunks after this one are in flight
    asm volatile("s_waitcnt vmcnt(%0)" ::"n"((D - 1) * (RT + MT) * 2) : "memory");
    use(j);
  }
  if (j < mine) asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
  for (; j < mine; ++j) use(j);
  if (p.K % CK && blockIdx.y + 1 == gridDim.y && chunks % NW == wave) {  // the rest of the rows, under 128 bytes in whole pieces
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int c = (4 * h + q) * 16;
      u32x4_t f[RT + MT];
#pragma unroll
      for (int t = 0; t < RT + MT; ++t) {
        const unsigned char* s = t < RT ? wbase + wrow(t, r) : xbase + xrow(t - RT, r);
        f[t] = c < p.K % CK * ES ? *(const u32x4_t*)(s + (int64_t)all * 128 + c) : u32x4_t{0u, 0u, 0u, 0u};
      }
      multiply(f);
    }
  }
  __syncthreads();  // every wave is done with its ring
  f32x4_t(*part)[RT * MT][64] = (f32x4_t(*)[RT * MT][64])smem;
#pragma unroll
  for (int t = 0; t < RT; ++t)
#pragma unroll
    for (int m = 0; m < MT; ++m) part[wave][t * MT + m][lane] = sums.of(t, m);
  __syncthreads();
  few_finish<T, EPI, RT, MT>(a, n0, tid, part);
}

// ---- bf16 tiles ------------------------------------------------------------------------------------------------------
// A BM x BN tile of C by WM x WN waves, in k-tiles of 64 that LDS-DMA loads bring from global memory into two LDS stages,
// with 32x32x16 products.  An operand by rows is staged as rows of 64 k (16-byte chunk c of row r at slot c ^ swz(r), so
// that the lanes of a fragment read spread over the banks), one by columns as 64 k-rows, read with the LDS transpose read
// (lane addresses as in bwd.hip; 32-byte granule g of k-row r at granule swz_col(g, r)).  A k-tile is four k-steps; the
// fragments of step s + 1 are read during step s, and one barrier per k-tile, between steps 2 and 3, frees its stage and
// makes the next k-tile's visible: the loads of A for two k-tiles ahead go out in step 3, those of B in step 0.
// Rows and columns past the matrix read row or column 0 and are not stored; k past K reads k 0 of its k-tile, and the last
// k-tile's rest is zeroed in LDS, in both operands, before it is read.
typedef short s16x4_t __attribute__((ext_vector_type(4)));
typedef __attribute__((address_space(3))) s16x4_t lds_s16x4_t;

__device__ __forceinline__ int swz_col(int g, int r) {
  const int x = g & 7;
  return (g & 8) | ((((x & 1) << 2) | (x >> 1)) ^ (r & 3));
}
__device__ __forceinline__ int unswz_col(int p, int r) {
  const int y = (p & 7) ^ (r & 3);
  return (p & 8) | (((y & 3) << 1) | (y >> 2));
}

template <int BM, int BN, int WM, int WN, int NS, bool ACOL, bool BCOL, int EPI>
struct Tile {
  static constexpr int NW = WM * WN, THREADS = NW * 64, MI = BM / WM / 32, NI = BN / WN / 32;
  static constexpr int A_BYTES = BM * 128, STAGE = (BM + BN) * 128;
  static constexpr int LA = BM / 8 / NW, LB = BN / 8 / NW;  // 1 KB loads per wave and k-tile
  static constexpr int COLS = EPI == EPI_GLU ? BN / 2 : BN;  // columns of C
  static_assert(EPI != EPI_GLU || (NI == 2 && !BCOL), "a wave holds the gate's and the up projection's same 32 columns");

  static_assert((!ACOL || BM % 128 == 0) && (!BCOL || BN % 128 == 0), "swz_col permutes runs of 8 granules, 128 columns");

  template <int C>
  static __device__ __forceinline__ bf16x8_t frag_col(const unsigned char* st, int cb, int ks, int lane) {
    const int gi = lane >> 4, j = lane & 15;
    const int n = cb + 16 * (gi & 1) + 4 * (j & 3);
    s16x4_t v[2];
#pragma unroll
    for (int hk = 0; hk < 2; ++hk) {
      const int k = 16 * ks + 8 * (gi >> 1) + 4 * hk + (j >> 2);
      const unsigned char* p = st + k * (2 * C) + ((swz_col(n >> 4, k) << 5) | ((n & 15) << 1));
      v[hk] = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4_t*)p);
    }
    return __builtin_bit_cast(bf16x8_t, __builtin_shufflevector(v[0], v[1], 0, 1, 2, 3, 4, 5, 6, 7));
  }
  static __device__ __forceinline__ bf16x8_t frag_row(const unsigned char* st, int rb, int ks, int lane) {
    const int swz = (lane & 7) ^ ((lane >> 3) & 1);
    return __builtin_bit_cast(bf16x8_t,
                              *(const u32x4_t*)(st + (rb + (lane & 31)) * 128 + (((2 * ks + (lane >> 5)) ^ swz) << 4)));
  }

  // Rows m0 .., columns n0 .., k-tiles [t0, t0 + nk) (nk >= 1) of the product; partial: where the sums go as they are
  // ([M][ld_partial] fp32, GLU: up sums from column ld_partial / 2 on), or null: through the epilogue
  static __device__ __forceinline__ void run(const Gemm& p, unsigned char* smem, int m0, int n0, int t0, int nk,
                                             float* partial, int64_t ld_partial) {
    int tid = threadIdx.x;
    asm volatile("" : "+v"(tid));
    const int lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int wm = wave / WN, wn = wave % WN;
    const int cnt = p.K - (t0 + nk - 1) * 64;  // k in the last k-tile; under 64: its rest is zeroed

    // a lane's offset in each of its loads, from a base that moves with the k-tile; tail: what of it is its k
    uint32_t aoff[LA], boff[LB];
    const uint32_t lda = (uint32_t)p.lda * 2, ldb = (uint32_t)p.ldb * 2;
    auto row_k = [&](int q) { return (uint32_t)(((lane & 7) ^ (lane >> 3) ^ (q & 1)) << 4); };  // by rows: 16-byte chunk
    auto col_k = [&](int q, int C) { return q * (512 / C) + lane / (C / 8); };                   // by columns: k-row
    auto col_c = [&](int q, int C) {                                                            // .. and 8-column chunk
      const int cs = lane & (C / 8 - 1);
      return (unswz_col(cs >> 1, col_k(q, C)) << 1) | (cs & 1);
    };
#pragma unroll
    for (int j = 0; j < LA; ++j) {
      const int q = wave * LA + j;
      if (ACOL) {
        int c = m0 + 8 * col_c(q, BM);
        c = c < p.M ? c : 0;
        aoff[j] = (uint32_t)col_k(q, BM) * lda + (uint32_t)c * 2;
      } else {
        const int r = 8 * q + (lane >> 3);
        aoff[j] = (uint32_t)(m0 + r < p.M ? r : 0) * lda + row_k(q);
      }
    }
#pragma unroll
    for (int j = 0; j < LB; ++j) {
      const int q = wave * LB + j;
      if (BCOL) {
        const int c = n0 + 8 * col_c(q, BN);
        boff[j] = (uint32_t)col_k(q, BN) * ldb + (uint32_t)(c < p.n_in ? c : 0) * 2;
      } else {
        const int r = (8 * q + (lane >> 3)) & (COLS - 1);  // GLU: gate rows, then up rows, whose base lies further on
        boff[j] = (uint32_t)(n0 + r < p.n_in ? r : 0) * ldb + row_k(q);
      }
    }
    const unsigned char* abase = (const unsigned char*)p.a + (ACOL ? (int64_t)t0 * 64 * lda : (int64_t)m0 * lda + (int64_t)t0 * 128);
    const unsigned char* bbase = (const unsigned char*)p.b + (BCOL ? (int64_t)t0 * 64 * ldb : (int64_t)n0 * ldb + (int64_t)t0 * 128);
    const int64_t astep = ACOL ? (int64_t)64 * lda : 128, bstep = BCOL ? (int64_t)64 * ldb : 128;
    const uint32_t lds0 = (uint32_t)(uintptr_t)smem;

    auto load = [&](int kt, int u) {  // load u of k-tile kt: A's, then B's
      const bool tail = kt == nk - 1 && cnt < 64;
      const uint32_t st = lds0 + kt % NS * STAGE;
      if (u < LA) {
        const int q = wave * LA + u;
        uint32_t o = aoff[u];
        if (tail) {
          if (ACOL) o -= col_k(q, BM) < cnt ? 0 : (uint32_t)col_k(q, BM) * lda;
          else o -= (int)row_k(q) < 2 * cnt ? 0 : row_k(q);
        }
        dma16(abase + kt * astep, o, st + q * 1024);
      } else {
        const int q = wave * LB + u - LA;
        uint32_t o = boff[u - LA];
        if (tail) {
          if (BCOL) o -= col_k(q, BN) < cnt ? 0 : (uint32_t)col_k(q, BN) * ldb;
          else o -= (int)row_k(q) < 2 * cnt ? 0 : row_k(q);
        }
        const int64_t further = EPI == EPI_GLU && 8 * q >= COLS ? (int64_t)p.up * ldb : 0;
        dma16(bbase + kt * bstep + further, o, st + A_BYTES + q * 1024);
      }
    };
    auto zero_rest = [&](int kt) {  // after the barrier that made k-tile kt visible
      if (kt != nk - 1 || cnt >= 64) return;
      unsigned char* st = smem + kt % NS * STAGE;
      auto clear = [&](unsigned char* o, int R, bool col) {
        for (int i = tid; i < R * 8; i += THREADS) {  // 16-byte pieces: by rows row i / 8, chunk i % 8; by columns in order
          const int r = i >> 3, c = i & 7, k = col ? i / (R / 8) : c * 8;
          const int at = col ? i * 16 : r * 128 + ((c ^ (r & 7) ^ ((r >> 3) & 1)) << 4);
          if (k >= cnt) *(u32x4_t*)(o + at) = u32x4_t{0u, 0u, 0u, 0u};
        }
      };
      clear(st, BM, ACOL);
      clear(st + A_BYTES, BN, BCOL);
      __syncthreads();
    };

    f32x16_t acc[MI][NI];
#pragma unroll
    for (int mi = 0; mi < MI; ++mi)
#pragma unroll
      for (int ni = 0; ni < NI; ++ni)
#pragma unroll
        for (int q = 0; q < 16; ++q) acc[mi][ni][q] = 0.f;
    bf16x8_t fa[2][MI], fb[2][NI];
    auto frag = [&](int kt, int ks, int i, bf16x8_t* A_, bf16x8_t* B_) {
      const unsigned char* sa = smem + kt % NS * STAGE;
      if (i < MI) {
        const int rb = (wm * MI + i) * 32;
        A_[i] = ACOL ? frag_col<BM>(sa, rb, ks, lane) : frag_row(sa, rb, ks, lane);
      } else {
        const int ni = i - MI, rb = EPI == EPI_GLU ? ni * COLS + wn * 32 : (wn * NI + ni) * 32;
        B_[ni] = BCOL ? frag_col<BN>(sa + A_BYTES, rb, ks, lane) : frag_row(sa + A_BYTES, rb, ks, lane);
      }
    };
    // one k-step: its products, with the next step's fragment reads in the first RS slots and the loads after them.  M1: there
    // is a next k-tile; MA, MB: k-tiles kt + NS and kt + NS - 1, whose A and B loads go out in this one
    constexpr int NSLOT = MI * NI, RS = 2, RPS = (MI + NI + RS - 1) / RS;
    constexpr int DA = (LA + NSLOT - RS - 1) / (NSLOT - RS > 0 ? NSLOT - RS : 1), DB = (LB + NSLOT - RS - 1) / (NSLOT - RS > 0 ? NSLOT - RS : 1);
    auto step = [&](auto ks_tag, auto m1_tag, auto ma_tag, auto mb_tag, int kt) {
      constexpr int ks = decltype(ks_tag)::value, c = ks & 1;
      constexpr bool M1 = decltype(m1_tag)::value, MA = decltype(ma_tag)::value, MB = decltype(mb_tag)::value;
#pragma unroll
      for (int i = 0; i < NSLOT; ++i) {
        const int mi = i / NI, ni = i % NI;
        acc[mi][ni] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(fa[c][mi], fb[c][ni], acc[mi][ni], 0, 0, 0);
        if (i < RS) {
#pragma unroll
          for (int r = i * RPS; r < (i + 1) * RPS && r < MI + NI; ++r) {
            if (ks < 3) frag(kt, ks + 1, r, fa[c ^ 1], fb[c ^ 1]);
            else if (M1) frag(kt + 1, 0, r, fa[c ^ 1], fb[c ^ 1]);
          }
        }
        if (i >= RS || NSLOT <= RS) {
          const int k = NSLOT <= RS ? i : i - RS;
          if (ks == 3 && MA) {
#pragma unroll
            for (int v = k * DA; v < (k + 1) * DA && v < LA; ++v) load(kt + NS, v);
          }
          if (ks == 0 && MB) {
#pragma unroll
            for (int v = k * DB; v < (k + 1) * DB && v < LB; ++v) load(kt + NS - 1, LA + v);
          }
        }
        __builtin_amdgcn_sched_barrier(0);
      }
      if (ks == 2) {
        // the next k-tile has landed (MB: the loads of the NS - 2 after it may be in flight; else nothing waits for long)
        if (MB) asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)\n\ts_barrier" ::"n"((NS - 2) * (LA + LB)) : "memory");
        else asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)\n\ts_barrier" ::: "memory");
        __builtin_amdgcn_sched_barrier(0);
        if (M1 && !MA) zero_rest(kt + 1);
      }
    };
    auto ktile = [&](auto m1, auto ma, auto mb, int kt) {
      step(std::integral_constant<int, 0>{}, m1, ma, mb, kt);
      step(std::integral_constant<int, 1>{}, m1, ma, mb, kt);
      step(std::integral_constant<int, 2>{}, m1, ma, mb, kt);
      step(std::integral_constant<int, 3>{}, m1, ma, mb, kt);
    };
    // before the first: k-tiles 0 .. NS - 2 and the A loads of k-tile NS - 1
    const std::true_type yes;
    const std::false_type no;
#pragma unroll
    for (int t = 0; t < NS; ++t) {
      if (t >= nk) break;
#pragma unroll
      for (int u = 0; u < (t < NS - 1 ? LA + LB : LA); ++u) load(t, u);
    }
    if (NS > 2 && nk >= NS) asm volatile("s_waitcnt vmcnt(%0)\n\ts_barrier" ::"n"((NS - 2) * (LA + LB) + LA) : "memory");
    else wait_loads_barrier();
    if (nk == 1) zero_rest(0);
#pragma unroll
    for (int i = 0; i < MI + NI; ++i) frag(0, 0, i, fa[0], fb[0]);
    int kt = 0;
    for (; kt + NS < nk; ++kt) ktile(yes, yes, yes, kt);
    if (kt + NS == nk) ktile(yes, no, yes, kt++);
    for (; kt + 1 < nk; ++kt) ktile(yes, no, no, kt);
    ktile(no, no, no, kt);

    // element q of accumulator (mi, ni): row 8 (q / 4) + 4 (lane / 32) + q % 4 of its block, column lane % 32; each group of
    // four q is transposed inside its quad of lanes, after which a lane holds four neighbouring columns of one row
    auto quad = [&](const f32x16_t& v, int q4) {
      return quad_transpose(f32x4_t{v[4 * q4], v[4 * q4 + 1], v[4 * q4 + 2], v[4 * q4 + 3]}, lane);
    };
#pragma unroll
    for (int mi = 0; mi < MI; ++mi)
#pragma unroll
      for (int q4 = 0; q4 < 4; ++q4) {
        const int m = m0 + (wm * MI + mi) * 32 + 8 * q4 + 4 * (lane >> 5) + (lane & 3);
#pragma unroll
        for (int ni = 0; ni < (EPI == EPI_GLU ? 1 : NI); ++ni) {
          const int n = n0 + (EPI == EPI_GLU ? wn * 32 : (wn * NI + ni) * 32) + 4 * ((lane & 31) >> 2);
          const f32x4_t v = quad(acc[mi][ni], q4);
          const f32x4_t w = EPI == EPI_GLU ? quad(acc[mi][1], q4) : v;
          if (m >= p.M || n >= p.N) continue;
          if (partial) {
            float* o = partial + (int64_t)m * ld_partial + n;
            *(f32x4_t*)o = v;
            if (EPI == EPI_GLU) *(f32x4_t*)(o + ld_partial / 2) = w;
          } else finish4<bf16_t, EPI>(p, m, n, v, w);
        }
      }
  }
};

struct Parts {  // dx, dw_gate_up, dw_down
  Part part[3];
};

// Workgroups go round the eight XCDs, so a run of 1/8 of a product's tiles is one XCD's, whose L2 its tiles share: bands of
// BAND tile rows, walked column by column. An XCD's 32 tiles at a time read BAND row and 32 / BAND column blocks, fewest at
// five or six. Forward and backward, us (16384 x 7168 x 2048; 8192 x 4096 x 4096): 4 rows 1222 + 2329; 694 + 1373, 6 rows
// 1213 + 2343; 685 + 1313, 8 rows 1268 + 2379; 705 + 1358, 16 rows 1290 + 2440 at the first.
constexpr int BAND = 6;

template <class G>
__device__ __forceinline__ void bf16_tile(const Part& a, int bm, unsigned char* smem) {
  const Gemm& p = a.p;
  const int mt = (p.M + bm - 1) / bm, nt = (p.N + G::COLS - 1) / G::COLS, nkt = (p.K + 63) / 64;
  const int tiles = mt * nt, n = tiles * a.splits;
  int i = blockIdx.x - a.first;
  {  // position among the product's tiles: XCD x takes [x n / 8, (x + 1) n / 8), rounded so that each is taken once
    const int x = i & 7, per = n >> 3, more = n & 7;
    i = x * per + (x < more ? x : more) + (i >> 3);
  }
  const int s = i / tiles;
  i -= s * tiles;
  const int band = i / (BAND * nt), rows = min(BAND, mt - band * BAND), r = i - band * BAND * nt;
  const int t0 = (int)((int64_t)nkt * s / a.splits), t1 = (int)((int64_t)nkt * (s + 1) / a.splits);
  G::run(p, smem, (band * BAND + r % rows) * bm, (r / rows) * G::COLS, t0, t1 - t0,
         a.partial ? a.partial + (int64_t)s * p.M * a.ld : nullptr, a.ld);
}

template <int BM, int BN, int WM, int WN, int NS, bool BCOL, int EPI>
__global__ __launch_bounds__(WM * WN * 64) void k_gemm_bf16(Part a) {
  extern __shared__ __align__(1024) unsigned char smem[];
  bf16_tile<Tile<BM, BN, WM, WN, NS, false, BCOL, EPI>>(a, BM, smem);
}

// The backward's last three products in one launch: none waits for another, and together they fill the last round of
// workgroups that each of them would leave part empty.
template <int BM, int BN, int WM, int WN, int NS>
__global__ __launch_bounds__(WM * WN * 64) void k_grads_bf16(Parts a) {
  extern __shared__ __align__(1024) unsigned char smem[];
  const int i = blockIdx.x;
  auto mine = [&](const Part& q) { return i >= q.first && i < q.first + q.blocks; };
  if (mine(a.part[0])) bf16_tile<Tile<BM, BN, WM, WN, NS, false, true, EPI_STORE>>(a.part[0], BM, smem);
  else if (mine(a.part[1]) || mine(a.part[2]))
    bf16_tile<Tile<BM, BN, WM, WN, NS, true, true, EPI_STORE>>(a.part[mine(a.part[1]) ? 1 : 2], BM, smem);
}

// The k-splits' sums, in split order, through the epilogue: four columns per thread.
template <typename T, int EPI>
__device__ __forceinline__ void finish(const Part& a, int64_t i) {
  const Gemm& p = a.p;
  const int quads = (p.N + 3) / 4;
  const int64_t m = i / quads;
  if (m >= p.M) return;
  const int n = (int)(i - m * quads) * 4;
  const float* o = a.partial + m * a.ld + n;
  f32x4_t v = {0, 0, 0, 0}, w = {0, 0, 0, 0};
  for (int s = 0; s < a.splits; ++s, o += p.M * a.ld) {
    v += *(const f32x4_t*)o;
    if (EPI == EPI_GLU) w += *(const f32x4_t*)(o + a.ld / 2);
  }
  finish4<T, EPI>(p, m, n, v, w);
}
template <typename T, int EPI>
__global__ __launch_bounds__(256) void k_finish(Part a) {
  finish<T, EPI>(a, (int64_t)blockIdx.x * 256 + threadIdx.x);
}
template <typename T>
__global__ __launch_bounds__(256) void k_finish_grads(Parts a) {  // first, blocks: of this launch
  const int i = blockIdx.x;
#pragma unroll
  for (int j = 0; j < 3; ++j)
    if (i >= a.part[j].first && i < a.part[j].first + a.part[j].blocks)
      finish<T, EPI_STORE>(a.part[j], (int64_t)(i - a.part[j].first) * 256 + threadIdx.x);
}

// Columns of a partial sum's row
int64_t partial_cols(const Gemm& p, int epi) { return (int64_t)(p.N + 3) / 4 * 4 * (epi == EPI_GLU ? 2 : 1); }

int64_t finish_blocks(const Gemm& p) { return ((int64_t)p.M * ((p.N + 3) / 4) + 255) / 256; }

// A product's part of a launch; tiles of bm rows and bn columns of B
bool make_part(Part* a, const Gemm& p, int epi, int bm, int bn, int splits, float* partial, int64_t first) {
  a->p = p;
  a->splits = splits;
  a->ld = partial_cols(p, epi);
  a->partial = splits > 1 ? partial : nullptr;
  const int cols = epi == EPI_GLU ? bn / 2 : bn;
  const int64_t n = (int64_t)((p.M + bm - 1) / bm) * ((p.N + cols - 1) / cols) * splits;
  a->first = (int)first;
  a->blocks = (int)n;
  return first + n + 8 <= 0x7fffffff;
}

template <class K>
int launch_tiles(K k, int lds, int threads, int64_t blocks, const void* args, hipStream_t st) {
  if (lds > 65536 && hipFuncSetAttribute((const void*)k, hipFuncAttributeMaxDynamicSharedMemorySize, lds) != hipSuccess) return -1;
  void* params[] = {(void*)args};
  return hipLaunchKernel((const void*)k, dim3((unsigned)blocks), dim3(threads), params, lds, st) == hipSuccess ? 0 : -1;
}

template <typename T, int EPI>
int launch_finish(const Part& a, hipStream_t st) {
  if (a.splits == 1) return 0;
  hipLaunchKernelGGL((k_finish<T, EPI>), dim3((unsigned)finish_blocks(a.p)), dim3(256), 0, st, a);
  return hipGetLastError() == hipSuccess ? 0 : -1;
}
template <typename T>
int launch_finish_grads(Parts g, hipStream_t st) {
  int64_t n = 0;
  for (Part& a : g.part) {
    a.first = (int)n;
    a.blocks = a.splits > 1 ? (int)finish_blocks(a.p) : 0;
    n += a.blocks;
  }
  if (n == 0) return 0;
  hipLaunchKernelGGL(k_finish_grads<T>, dim3((unsigned)n), dim3(256), 0, st, g);
  return hipGetLastError() == hipSuccess ? 0 : -1;
}

template <int BM, int BN, int WM, int WN, int NS, bool BCOL, int EPI>
int gemm_tiles(const Gemm& p, int splits, float* partial, hipStream_t st) {
  Part a;
  if (!make_part(&a, p, EPI, BM, BN, splits, partial, 0)) return -1;
  if (launch_tiles(k_gemm_bf16<BM, BN, WM, WN, NS, BCOL, EPI>, NS * (BM + BN) * 128, WM * WN * 64, a.blocks, &a, st)) return -1;
  return launch_finish<bf16_t, EPI>(a, st);
}

// The three gradients' parts, those with the longest sums first; the partial sums one after another
bool make_grads(Parts* g, const Gemm* const (&p)[3], int bm, int bn, const int (&splits)[3], float* partial, int64_t* blocks) {
  const bool dx_first = p[0]->K >= p[1]->K;
  const int order[3] = {dx_first ? 0 : 1, dx_first ? 1 : 2, dx_first ? 2 : 0};
  *blocks = 0;
  for (const int i : order) {
    if (!make_part(&g->part[i], *p[i], EPI_STORE, bm, bn, splits[i], partial, *blocks)) return false;
    *blocks += (g->part[i].blocks + 7) / 8 * 8;
    if (splits[i] > 1) partial += (int64_t)splits[i] * p[i]->M * g->part[i].ld;
  }
  return true;
}

template <int BM, int BN, int WM, int WN, int NS>
int grads_tiles(const Gemm* const (&p)[3], const int (&splits)[3], float* partial, hipStream_t st) {
  Parts g;
  int64_t blocks;
  if (!make_grads(&g, p, BM, BN, splits, partial, &blocks)) return -1;
  if (launch_tiles(k_grads_bf16<BM, BN, WM, WN, NS>, NS * (BM + BN) * 128, WM * WN * 64, blocks, &g, st)) return -1;
  return launch_finish_grads<bf16_t>(g, st);
}

// Few tokens: k-splits up to a workgroup for each CU, of four chunks for each wave at least
template <typename T, int EPI, int COLS>
Part few_part(const Gemm& p, float* partial) {
  const int64_t groups = (p.N + COLS - 1) / COLS, ld = partial_cols(p, EPI);
  const int64_t most = std::min(std::min(256 / groups, (int64_t)MAX_SPLITS), std::min<int64_t>(p.K * (int64_t)sizeof(T) / 128 / 32, PARTIAL / (p.M * ld)));
  const int splits = (int)std::max<int64_t>(1, most);
  return {p, splits, 0, (int)groups, splits > 1 ? partial : nullptr, ld};
}

template <typename T, int EPI, int RT, int MT, int SU>
int few(const Gemm& p, float* partial, hipStream_t st) {
  const Part a = few_part<T, EPI, EPI == EPI_GLU ? 8 * RT : 16 * RT>(p, partial);
  hipLaunchKernelGGL((k_gemm_few<T, EPI, RT, MT, SU>), dim3(a.blocks, a.splits), dim3(512), 0, st, a);
  if (hipGetLastError() != hipSuccess) return -1;
  return launch_finish<T, EPI>(a, st);
}

template <typename T, int EPI, int RT, int MT, int D>
int ring(const Gemm& p, float* partial, hipStream_t st) {
  constexpr int LDS = 8 * D * (RT + MT) * 2048;
  const Part a = few_part<T, EPI, EPI == EPI_GLU ? 8 * RT : 16 * RT>(p, partial);
  const void* k = (const void*)k_gemm_ring<T, EPI, RT, MT, D>;
  if (LDS > 65536 && hipFuncSetAttribute(k, hipFuncAttributeMaxDynamicSharedMemorySize, LDS) != hipSuccess) return -1;
  void* params[] = {(void*)&a};
  if (hipLaunchKernel(k, dim3(a.blocks, a.splits), dim3(512), params, LDS, st) != hipSuccess) return -1;
  return launch_finish<T, EPI>(a, st);
}

// Whether the weights stream past (gemm_few), or the tokens are many enough for tiles.  Measured: 4096 x 14336 with 32 tokens
// 87 us against 91 for 40 in tiles, with 64 tokens 121 against 82 (each weight meets four products' worth of tokens); 7168 x
// 2048 with 40 tokens 32 and 34, with 64 both 37; 2048 x 1408 with 64 tokens 11 and 21 (tiles need k-splits there).
bool few_tokens(int64_t tokens, int d, int f, int elem) {
  const int piece = 16 / elem;
  return tokens <= 32 || (tokens <= 64 && d % piece == 0 && f % piece == 0 && (int64_t)d * f * elem <= 1 << 25);
}

template <typename T, int EPI>
int gemm_few(const Gemm& p, float* partial, hipStream_t st) {
  constexpr int PER = 16 / sizeof(T);  // elements of a 16-byte piece
  if (p.lda % PER == 0 && p.ldb % PER == 0 && p.K % PER == 0 && ((int64_t)p.up + 32) * p.ldb * (int)sizeof(T) < (1ll << 32)) {
    if (p.M <= 16) return ring<T, EPI, 1, 1, 2>(p, partial, st);
    if (p.M <= 32) return ring<T, EPI, 1, 2, 1>(p, partial, st);
    if (p.M <= 48) return ring<T, EPI, 1, 3, 1>(p, partial, st);
    return ring<T, EPI, 1, 4, 1>(p, partial, st);
  }
  if (p.M <= 16) return few<T, EPI, 1, 1, 4>(p, partial, st);
  return few<T, EPI, 1, 2, 2>(p, partial, st);
}

template <bool BCOL, int EPI>
int gemm_bf16(const Gemm& p, float* partial, hipStream_t st) {
  const Choice c = choose(p.M, partial_cols(p, EPI), (p.K + 63) / 64);
  if (c.tile == 0) return gemm_tiles<256, 256, 2, 4, 2, BCOL, EPI>(p, c.splits, partial, st);
  if (c.tile == 1) return gemm_tiles<128, 128, 2, 2, 2, BCOL, EPI>(p, c.splits, partial, st);
  if (c.tile == 2) return gemm_tiles<128, 128, 4, 2, 4, BCOL, EPI>(p, c.splits, partial, st);
  if (c.tile == 3) return gemm_tiles<64, 128, 2, 2, 3, BCOL, EPI>(p, c.splits, partial, st);
  return gemm_tiles<256, 128, 4, 2, 3, BCOL, EPI>(p, c.splits, partial, st);
}

int grads_bf16(const Gemm* const (&p)[3], float* partial, hipStream_t st) {
  Product q[3];
  for (int i = 0; i < 3; ++i) q[i] = {p[i]->M, partial_cols(*p[i], EPI_STORE), (p[i]->K + 63) / 64};
  int splits[3];
  const Choice c = choose_grads(q, splits);
  if (c.tile == 0) return grads_tiles<256, 256, 2, 4, 2>(p, splits, partial, st);
  if (c.tile == 1) return grads_tiles<128, 128, 4, 2, 2>(p, splits, partial, st);
  return grads_tiles<128, 128, 4, 2, 4>(p, splits, partial, st);
}

// ---- fp32 --------------------------------------------------------------------------------------------------------------
// A 64 x 64 tile of C (GLU: 32 columns of the gate and the same 32 of the up projection) by four waves of 32 x 32, with
// 16x16x4 fp32 products in k-tiles of 32.  A k-tile is loaded into registers two k-tiles ahead and kept in LDS as rows of k
// for either layout of an operand, from which a lane takes 16 bytes for four products at once (which k meet in which
// product does not matter as long as both operands agree).  The tile is small so that four workgroups share a CU and hide
// each other's latency.  The products take C's columns as their rows, which leaves a lane four neighbouring columns.
constexpr int FK = 32;

struct F32Stage {
  float a[2][64 * FK], b[2][64 * FK];
};
// k of a row in a stage: its 16-byte chunks permuted by the row, so that eight neighbouring rows' same chunk, a row's eight
// chunks and every fourth row's same k fall on all banks (rows 144 bytes apart instead, as they are: the gradients' LDS
// busy 51% instead of 28% of their time, 1751 us instead of 1685)
__device__ __forceinline__ int f32_at(int row, int k) {
  return row * FK + (((k >> 2) ^ (row & 7) ^ ((row >> 3) & 7)) << 2 | (k & 3));
}

template <int EPI, bool ACOL, bool BCOL>
__device__ __forceinline__ void f32_tile(const Part& part, F32Stage& sh) {
  const Gemm& p = part.p;
  auto& sa = sh.a;
  auto& sb = sh.b;
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6), wm = wave & 1, wn = wave >> 1;
  constexpr int BN = EPI == EPI_GLU ? 32 : 64;
  const int nt = (p.N + BN - 1) / BN, tiles = (p.M + 63) / 64 * nt, nkt = (p.K + FK - 1) / FK;
  const int i0 = blockIdx.x - part.first, s = i0 / tiles, tile = i0 % tiles;
  const int m0 = tile / nt * 64, n0 = tile % nt * BN;
  const int t0 = (int)((int64_t)nkt * s / part.splits), t1 = (int)((int64_t)nkt * (s + 1) / part.splits);
  const float *A = (const float*)p.a, *B = (const float*)p.b;

  // twice four elements per thread and operand: by rows, k 4 (tid % 8) .. of rows tid / 8 and tid / 8 + 32; by columns, four
  // neighbouring rows of k kc and kc + 16: either way eight lanes take a line.  Outside the matrix: 0
  const int rc = 4 * (lane & 7) + 32 * (wave & 1), kc = (lane >> 3) + 8 * (wave >> 1);
  f32x4_t rega[2][2], regb[2][2];  // of two k-tiles: a load has two k-tiles' time to arrive
  // contiguous elements c .. c + 3 at q, those from limit on 0 (in: whether any are wanted): no branch, so that all of a
  // thread's loads go out together
  auto four = [&](const float* q, int c, int limit, int seg, int jump, bool in) {
    f32x4_t v;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int e = min(c + i, limit - 1);
      v[i] = q[e + (e >= seg ? jump : 0)];
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = in && c + i < limit ? v[i] : 0.f;
    return v;
  };
  // a k-tile that ends before the last k and does not straddle a_seg: whole fours from a lane's fixed places.  Rows past the
  // matrix read its first; columns past it read the next row (the last k is not in such a k-tile); neither is stored
  const int ca = m0 + rc, cb = n0 + rc, row = tid >> 3, kr = 4 * (tid & 7);
  const float* pa = ACOL ? A + (int64_t)kc * p.lda + (ca < p.M ? ca : 0)
                         : A + (int64_t)(m0 + row < p.M ? m0 + row : 0) * p.lda + kr;
  const float* pa1 = ACOL ? pa + 16 * p.lda : A + (int64_t)(m0 + row + 32 < p.M ? m0 + row + 32 : 0) * p.lda + kr;
  // row h of B's two: GLU's second lies in the up projection
  auto brow_of = [&](int h) -> int64_t { return n0 + row + (EPI == EPI_GLU ? 0 : 32 * h); };
  auto up_of = [&](int h) -> int64_t { return EPI == EPI_GLU && h ? p.up : 0; };
  const float* pb = BCOL ? B + (int64_t)kc * p.ldb + (cb < p.n_in ? cb : 0)
                         : B + (brow_of(0) < p.n_in ? brow_of(0) : 0) * p.ldb + kr;
  const float* pb1 = BCOL ? pb + 16 * p.ldb : B + ((brow_of(1) < p.n_in ? brow_of(1) : 0) + up_of(1)) * p.ldb + kr;
  const bool wide = p.lda >= 4 && p.ldb >= 4;
  auto fetch = [&](int kt, f32x4_t* ra, f32x4_t* rb) {
    const int k0 = kt * FK;
    if (wide && k0 + FK < p.K && (ACOL || k0 >= p.a_seg || k0 + FK <= p.a_seg)) {
      const int64_t oa = ACOL ? (int64_t)k0 * p.lda : k0 + (k0 >= p.a_seg ? p.a_jump : 0), ob = BCOL ? (int64_t)k0 * p.ldb : k0;
      ra[0] = load4(pa + oa, 4);
      ra[1] = load4(pa1 + oa, 4);
      rb[0] = load4(pb + ob, 4);
      rb[1] = load4(pb1 + ob, 4);
      return;
    }
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int k = k0 + kc + 16 * h, last = p.K - 1;
      ra[h] = ACOL ? four(A + (int64_t)min(k, last) * p.lda, ca, p.M, 0x7fffffff, 0, k <= last)
                   : four(A + (int64_t)min(m0 + row + 32 * h, p.M - 1) * p.lda, k0 + kr, p.K, p.a_seg, p.a_jump, true);
      rb[h] = BCOL ? four(B + (int64_t)min(k, last) * p.ldb, cb, p.n_in, 0x7fffffff, 0, k <= last)
                   : four(B + (min(brow_of(h), (int64_t)p.n_in - 1) + up_of(h)) * p.ldb, k0 + kr, p.K, 0x7fffffff, 0, true);
    }
  };
  auto keep = [&](int st, const f32x4_t* ra, const f32x4_t* rb) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      if (ACOL) {
#pragma unroll
        for (int i = 0; i < 4; ++i) sa[st][f32_at(rc + i, kc + 16 * h)] = ra[h][i];
      } else *(f32x4_t*)&sa[st][f32_at(row + 32 * h, kr)] = ra[h];
      if (BCOL) {
#pragma unroll
        for (int i = 0; i < 4; ++i) sb[st][f32_at(rc + i, kc + 16 * h)] = rb[h][i];
      } else *(f32x4_t*)&sb[st][f32_at(row + 32 * h, kr)] = rb[h];
    }
  };

  // [16 columns of C (GLU: of the gate, of the up projection)][16 rows]
  f32x4_t acc[2][2], total[2][2];
#pragma unroll
  for (int j = 0; j < 2; ++j)
#pragma unroll
    for (int i = 0; i < 2; ++i) acc[j][i] = total[j][i] = f32x4_t{0.f, 0.f, 0.f, 0.f};
  const int r = lane & 15, q = lane >> 4;
  const int brow[2] = {EPI == EPI_GLU ? wn * 16 : wn * 32, EPI == EPI_GLU ? 32 + wn * 16 : wn * 32 + 16};
  auto ktile = [&](auto parity, int kt) {  // k-tile kt - t0 even or odd
    constexpr int st = decltype(parity)::value;
    __syncthreads();
    if (kt + 2 < t1) fetch(kt + 2, rega[st], regb[st]);
#pragma unroll
    for (int k = 0; k < FK; k += 16) {
      f32x4_t a[2], b[2];
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        a[i] = *(const f32x4_t*)&sa[st][f32_at(wm * 32 + i * 16 + r, k + 4 * q)];
        b[i] = *(const f32x4_t*)&sb[st][f32_at(brow[i] + r, k + 4 * q)];
      }
#pragma unroll
      for (int e = 0; e < 4; ++e)
#pragma unroll
        for (int j = 0; j < 2; ++j)
#pragma unroll
          for (int i = 0; i < 2; ++i) acc[j][i] = __builtin_amdgcn_mfma_f32_16x16x4f32(b[j][e], a[i][e], acc[j][i], 0, 0, 0);
    }
    if (kt + 1 < t1) keep(st ^ 1, rega[st ^ 1], regb[st ^ 1]);  // its last readers passed this k-tile's barrier
    if (kt % (FSUM / FK) == FSUM / FK - 1 || kt + 1 == t1) {
#pragma unroll
      for (int j = 0; j < 2; ++j)
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          total[j][i] += acc[j][i];
          acc[j][i] = f32x4_t{0.f, 0.f, 0.f, 0.f};
        }
    }
  };
  if (t0 < t1) {
    fetch(t0, rega[0], regb[0]);
    if (t0 + 1 < t1) fetch(t0 + 1, rega[1], regb[1]);
    keep(0, rega[0], regb[0]);
  }
  for (int kt = t0; kt < t1; kt += 2) {
    ktile(std::integral_constant<int, 0>{}, kt);
    if (kt + 1 < t1) ktile(std::integral_constant<int, 1>{}, kt + 1);
  }
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int m = m0 + wm * 32 + i * 16 + r;
#pragma unroll
    for (int j = 0; j < (EPI == EPI_GLU ? 1 : 2); ++j) {
      const int n = n0 + brow[j] + 4 * q;
      if (m >= p.M || n >= p.N) continue;
      if (part.partial) {
        float* o = part.partial + ((int64_t)s * p.M + m) * part.ld + n;
        *(f32x4_t*)o = total[j][i];
        if (EPI == EPI_GLU) *(f32x4_t*)(o + part.ld / 2) = total[1][i];
      } else finish4<float, EPI>(p, m, n, total[j][i], total[1][i]);
    }
  }
}

// Four workgroups on a CU, at 128 registers and no spill: forward and backward at 4096 x 2048 x 2048 877-926 + 1685 us (111-117
// and 122 TFLOP/s of the 153 of a large fp32 product); left to the compiler's choice of registers 5% and 10% longer.
template <int EPI, bool BCOL>
__global__ __launch_bounds__(256, 4) void k_gemm_f32(Part a) {
  __shared__ __align__(16) F32Stage sh;
  f32_tile<EPI, false, BCOL>(a, sh);
}

__global__ __launch_bounds__(256, 4) void k_grads_f32(Parts a) {
  __shared__ __align__(16) F32Stage sh;
  const int i = blockIdx.x;
  auto mine = [&](const Part& q) { return i >= q.first && i < q.first + q.blocks; };
  if (mine(a.part[0])) f32_tile<EPI_STORE, false, true>(a.part[0], sh);
  else if (mine(a.part[1]) || mine(a.part[2])) f32_tile<EPI_STORE, true, true>(a.part[mine(a.part[1]) ? 1 : 2], sh);
}

// splits of a product of so many tiles: up to four workgroups for each CU, of 256 k at least, or up to one for each CU of 128
// (500 x 500 x 500: 33 + 48 us with 256 only, 31 + 42; more workgroups than CUs of 128 k lose to the sums' way to memory and
// back: 1000 x 300 x 900 35 us forward, 46)
int f32_splits(const Gemm& p, int epi, int64_t tiles) {
  const int64_t s = std::max(std::min<int64_t>(1024 / tiles, p.K / 256), std::min<int64_t>(256 / tiles, p.K / 128));
  return (int)std::max<int64_t>(1, std::min(std::min<int64_t>(s, MAX_SPLITS), PARTIAL / (p.M * partial_cols(p, epi))));
}

template <int EPI, bool BCOL>
int gemm_f32(const Gemm& p, float* partial, hipStream_t st) {
  Part a;
  if (!make_part(&a, p, EPI, 64, 64, 1, partial, 0)) return -1;
  if (!make_part(&a, p, EPI, 64, 64, f32_splits(p, EPI, a.blocks), partial, 0)) return -1;
  hipLaunchKernelGGL((k_gemm_f32<EPI, BCOL>), dim3((unsigned)a.blocks), dim3(256), 0, st, a);
  if (hipGetLastError() != hipSuccess) return -1;
  return launch_finish<float, EPI>(a, st);
}

int grads_f32(const Gemm* const (&p)[3], float* partial, hipStream_t st) {
  Parts g;
  int64_t blocks, room = PARTIAL, work = 0;
  int splits[3] = {1, 1, 1};
  if (!make_grads(&g, p, 64, 64, splits, partial, &blocks)) return -1;
  for (int i = 0; i < 3; ++i) work += (int64_t)g.part[i].blocks * ((p[i]->K + FK - 1) / FK);
  // sums no longer than what four workgroups on each CU would take of the whole, but of 256 k at least
  const int64_t len = std::max<int64_t>(256 / FK, work / 1024);
  for (int i = 0; i < 3; ++i) {
    const int64_t floats = p[i]->M * partial_cols(*p[i], EPI_STORE);
    if (floats > 0) splits[i] = (int)std::max<int64_t>(1, std::min(std::min<int64_t>(MAX_SPLITS, p[i]->K / FK / len), room / floats));
    if (splits[i] > 1) room -= splits[i] * floats;
  }
  if (!make_grads(&g, p, 64, 64, splits, partial, &blocks)) return -1;
  hipLaunchKernelGGL(k_grads_f32, dim3((unsigned)blocks), dim3(256), 0, st, g);
  if (hipGetLastError() != hipSuccess) return -1;
  return launch_finish_grads<float>(g, st);
}

// ---- the block --------------------------------------------------------------------------------------------------

// bf16 operands whose rows do not start at 16 bytes, copied to rows that do: one launch for all of a call's.  Row r of a
// copy, in parts of `padded` rows, is row (r / padded) * real + r % padded of the operand, or 0 where r % padded >= real;
// columns past the operand's are 0.  777 tokens of 2046 x 1406 forward: 13.6 of 45 us; 2048 in training 14.1 + 17.6 of 172.
struct PackJob {
  const bf16_t* src;
  bf16_t* dst;
  int64_t first, rows;  // first: 16-byte pieces of the jobs before
  int cols, ld, real, padded;  // ld: of the copy, a multiple of 8; the operand's is cols
};
struct PackJobs {
  PackJob job[4];
  int n;
  int64_t pieces;
};

// Workgroups of 256 threads for n elements: the kernels below walk what is past them (a launch holds under 2^32 threads)
unsigned blocks_for(int64_t n) { return (unsigned)std::min<int64_t>((n + 255) / 256, 1 << 20); }

__global__ __launch_bounds__(256) void k_pack(PackJobs a) {
  for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < a.pieces; i += (int64_t)gridDim.x * 256) {
    int j = 0;
    while (j + 1 < a.n && i >= a.job[j + 1].first) ++j;
    const PackJob& b = a.job[j];
    const int per = b.ld / 8;
    const int64_t r = (i - b.first) / per;
    const int c = (int)(i - b.first - r * per) * 8, part = (int)(r / b.padded), at = (int)(r - (int64_t)part * b.padded);
    u32x4_t v = {0u, 0u, 0u, 0u};
    if (at < b.real) {
      const bf16_t* s = b.src + ((int64_t)part * b.real + at) * b.cols + c;
      if (c + 8 <= b.cols) __builtin_memcpy(&v, s, 16);
      else
#pragma unroll
        for (int k = 0; k < 8; ++k)
          if (c + k < b.cols) v[k / 2] |= (uint32_t)s[k] << (16 * (k & 1));
    }
    *(u32x4_t*)(b.dst + r * b.ld + c) = v;
  }
}

__global__ __launch_bounds__(256) void k_clear(bf16_t* p, int64_t n) {
  for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < n; i += (int64_t)gridDim.x * 256) p[i] = 0;
}

int clear(void* p, int64_t n, hipStream_t st) {
  hipLaunchKernelGGL(k_clear, dim3(blocks_for(n)), dim3(256), 0, st, (bf16_t*)p, n);
  return hipGetLastError() == hipSuccess ? 0 : -1;
}

int64_t up8(int64_t v) { return (v + 7) / 8 * 8; }
int64_t up256(int64_t v) { return (v + 255) / 256 * 256; }

// Elements of the copies a call makes of its operands (x, w_gate_up, w_down, dy)
void pack_sizes(int64_t tokens, int d, int f, bool backward, int64_t (&n)[4]) {
  const bool odd_d = d % 8 != 0, odd = odd_d || f % 8 != 0;
  const int64_t D = up8(d), F = up8(f);
  n[0] = odd_d ? up256(tokens * D) : 0;
  n[1] = odd ? up256(2 * F * D) : 0;
  n[2] = odd ? up256(D * F) : 0;
  n[3] = odd_d && backward ? up256(tokens * D) : 0;
}

// The call's products.  f32: on the operands as they are.  bf16: on rows that start at 16 bytes, widths D and F in whole
// eights; the weights' rows and columns past d and f are 0, so that sums over a whole D or F need no care.  Either way h, g,
// u, dg and du past f are written as 0.
struct Block {
  Gemm glu, down;                      // forward
  Gemm dglu, dx, dw_gate_up, dw_down;  // backward
};

Block block_f32(const SharedLaunch& s) {
  Block b{};
  const int T = (int)s.tokens, d = s.d, f = s.f, F = s.row, none = 0x7fffffff;
  b.glu = {s.x, s.w_gate_up, d, d, none, 0, T, F, d, f, s.h, F, nullptr, s.gu, 2 * F, F, f, none, none};
  b.down = {s.h, s.w_down, F, f, none, 0, T, d, f, d, s.y, d, s.residual, nullptr, 0, 0, 0, none, none};
  b.dglu = {s.dy, s.w_down, d, f, none, 0, T, F, d, f, s.dgu, 2 * F, nullptr, s.gu, 2 * F, F, 0, none, none};
  b.dx = {s.dgu, s.w_gate_up, 2 * F, d, f, F - f, T, d, 2 * f, d, s.dx, d, s.residual, nullptr, 0, 0, 0, none, none};
  b.dw_gate_up = {s.dgu, s.x, 2 * F, d, none, 0, 2 * F, d, T, d, s.dw_gate_up, d, nullptr, nullptr, 0, 0, 0, f, F};
  b.dw_down = {s.dy, s.h, d, F, none, 0, d, f, T, f, s.dw_down, f, nullptr, nullptr, 0, 0, 0, none, none};
  return b;
}

Block block_bf16(const SharedLaunch& s, const void* x, const void* wgu, const void* wd, const void* dy) {
  Block b{};
  const int T = (int)s.tokens, d = s.d, f = s.f, F = s.row, D = (int)up8(d), none = 0x7fffffff;
  b.glu = {x, wgu, D, D, none, 0, T, F, D, f, s.h, F, nullptr, s.gu, 2 * F, F, F, none, none};
  b.down = {s.h, wd, F, F, none, 0, T, d, F, d, s.y, d, s.residual, nullptr, 0, 0, 0, none, none};
  b.dglu = {dy, wd, D, F, none, 0, T, F, D, f, s.dgu, 2 * F, nullptr, s.gu, 2 * F, F, 0, none, none};
  b.dx = {s.dgu, wgu, 2 * F, D, none, 0, T, d, 2 * F, d, s.dx, d, s.residual, nullptr, 0, 0, 0, none, none};
  b.dw_gate_up = {s.dgu, x, 2 * F, D, none, 0, 2 * F, d, T, d, s.dw_gate_up, d, nullptr, nullptr, 0, 0, 0, f, F};
  b.dw_down = {dy, s.h, D, F, none, 0, d, f, T, f, s.dw_down, f, nullptr, nullptr, 0, 0, 0, none, none};
  return b;
}

int run_f32(const SharedLaunch& s, hipStream_t st) {
  const Block b = block_f32(s);
  float* partial = (float*)s.workspace;
  int rc;
  if (!s.backward) {
    if (few_tokens(s.tokens, s.d, s.f, 4)) {
      if ((rc = gemm_few<float, EPI_GLU>(b.glu, partial, st))) return rc;
      return gemm_few<float, EPI_STORE>(b.down, partial, st);
    }
    if ((rc = gemm_f32<EPI_GLU, false>(b.glu, partial, st))) return rc;
    return gemm_f32<EPI_STORE, false>(b.down, partial, st);
  }
  if (s.tokens > 0 && (rc = gemm_f32<EPI_DGLU, true>(b.dglu, partial, st))) return rc;
  return grads_f32({&b.dx, &b.dw_gate_up, &b.dw_down}, partial, st);
}

int run_bf16(const SharedLaunch& s, hipStream_t st) {
  int rc;
  if (s.tokens == 0) {
    if ((rc = clear(s.dw_gate_up, 2ll * s.f * s.d, st))) return rc;
    return clear(s.dw_down, (int64_t)s.f * s.d, st);
  }
  if (!s.backward && few_tokens(s.tokens, s.d, s.f, 2)) {
    const Block b = block_f32(s);  // the operands as they are
    if ((rc = gemm_few<bf16_t, EPI_GLU>(b.glu, (float*)s.workspace, st))) return rc;
    return gemm_few<bf16_t, EPI_STORE>(b.down, (float*)s.workspace, st);
  }
  int64_t n[4];
  pack_sizes(s.tokens, s.d, s.f, s.backward, n);
  const void* op[4] = {s.x, s.w_gate_up, s.w_down, s.dy};
  const int D = (int)up8(s.d), T = (int)s.tokens;
  const int cols[4] = {s.d, s.d, s.f, s.d}, ld[4] = {D, D, s.row, D}, real[4] = {T, s.f, s.d, T}, padded[4] = {T, s.row, D, T};
  const int64_t rows[4] = {T, 2 * s.row, D, T};
  PackJobs jobs{};
  bf16_t* to = (bf16_t*)s.workspace;
  for (int i = 0; i < 4; ++i)
    if (n[i] && (s.backward || i < 3)) {
      jobs.job[jobs.n++] = {(const bf16_t*)op[i], to, jobs.pieces, rows[i], cols[i], ld[i], real[i], padded[i]};
      jobs.pieces += rows[i] * (ld[i] / 8);
      op[i] = to;
      to += n[i];
    }
  if (jobs.n) {
    hipLaunchKernelGGL(k_pack, dim3(blocks_for(jobs.pieces)), dim3(256), 0, st, jobs);
    if (hipGetLastError() != hipSuccess) return -1;
  }
  float* partial = (float*)to;
  const Block b = block_bf16(s, op[0], op[1], op[2], op[3]);
  if (!s.backward) {
    if ((rc = gemm_bf16<false, EPI_GLU>(b.glu, partial, st))) return rc;
    return gemm_bf16<false, EPI_STORE>(b.down, partial, st);
  }
  if ((rc = gemm_bf16<true, EPI_DGLU>(b.dglu, partial, st))) return rc;
  return grads_bf16({&b.dx, &b.dw_gate_up, &b.dw_down}, partial, st);
}

}  // namespace

int64_t shared_workspace_bytes(int64_t tokens, int d, int f, int dtype, bool backward) {
  if (tokens == 0) return 0;
  int64_t n[4] = {0, 0, 0, 0};
  if (dtype == MOE_BF16) pack_sizes(tokens, d, f, backward, n);
  // the k-splits' sums: at most PARTIAL floats, and MAX_SPLITS times a launch's products (the three gradients are one launch,
  // their sums one after another)
  const int64_t D = up8(d), F = up8(f);
  const int64_t out = backward ? std::max(tokens * F, tokens * D + 2 * F * D + D * F) : std::max(tokens * D, tokens * 2 * F);
  return 2 * (n[0] + n[1] + n[2] + n[3]) + 4 * std::min<int64_t>(PARTIAL, MAX_SPLITS * out);
}

int launch_shared(const SharedLaunch& s, hipStream_t st) { return s.dtype == MOE_BF16 ? run_bf16(s, st) : run_f32(s, st); }
