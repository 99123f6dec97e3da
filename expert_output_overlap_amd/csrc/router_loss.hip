// The router's losses, per-expert counts and the gradient of the logits (formulas in include/moe_overlap.h).
//
// Bytes bound both at many tokens (logits read once in each, their gradient written), launches and latency at few.  A row is held by
// L lanes, NV float4 each (L = 16 up to 256 experts: four rows in a wave share its instructions), so its sums are four DPP steps.
// Forward: one launch.  With P[g] the sum of a sequence's p_g, its part of B is sum over g of f_g P_g, so counts and P can be taken
// in one pass, before f is known.  Each sequence is cut into parts, a workgroup to a part; the last workgroup of a sequence joins its
// parts, the last of all the sequences (join.h).  16384 x 256 logits in 8 sequences take 16 us, of which half is this joining (four
// waits for another workgroup's sums or counter, one after another), and their gradient 11 (2.3 TB/s; few rows for each wave: latency).
// The parts are cut by the mean length: one sequence of 6000 rows among 200 of 8192 x 64 logits takes 111 us, where equal ones take 9.
#include <algorithm>
#include <type_traits>

#include "common.h"
#include "join.h"
#include "launch.h"
#include "row_util.h"

namespace {

constexpr int BLOCK = 512, WAVES = BLOCK / 64;
using std::integral_constant;

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

template <int CTRL>
__device__ __forceinline__ float dpp(float v) {
  return __builtin_bit_cast(float, __builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, v), CTRL, 0xf, 0xf, true));
}

// op over the L lanes of a row, in each of them: lane ^ 1, lane ^ 2, then the halves mirrored; beyond 16 lanes by shuffles
template <int L, class Op>
__device__ __forceinline__ float over_row(float v, Op op) {
  v = op(v, dpp<0xB1>(v));
  v = op(v, dpp<0x4E>(v));
  if (L >= 16) {
    v = op(v, dpp<0x141>(v));
    v = op(v, dpp<0x140>(v));
  }
  if (L == 64) {
    v = op(v, __shfl_xor(v, 16, 64));
    v = op(v, __shfl_xor(v, 32, 64));
  }
  return v;
}
template <int L>
__device__ __forceinline__ float sum_row(float v) {
  return over_row<L>(v, [](float a, float b) { return a + b; });
}
template <int L>
__device__ __forceinline__ float max_row(float v) {
  return over_row<L>(v, [](float a, float b) { return fmaxf(a, b); });
}

// Four columns from c on of a row of G, `empty` past it
__device__ __forceinline__ void load_cols(const float* row, int c, int G, float empty, float* v) {
  const int n = G - c;
  const u32x4 q = n > 0 ? Chunk<float>::load(row + c, n) : u32x4{0, 0, 0, 0};
#pragma unroll
  for (int i = 0; i < 4; ++i) v[i] = i < n ? __uint_as_float(q[i]) : empty;
}

// exp(x), x <= 0 or NaN, within two steps wherever it is a normal number (0 below): 2^y with y the rounded x log2 e, and what that
// rounding left of x, d = x - y ln 2, as exp(d) = 1 + d (|d| < 2^-16).  Without d the error would grow with |x|, 40 steps at -80.  At
// -inf d is NaN and 2^y 0: fmaxf makes a number of d.  65536 x 1024 logits forward 70 us; 64 without d, 81 with expf
__device__ __forceinline__ float exp_of(float x) {
  constexpr double LN2 = 0.69314718055994530942;
  constexpr float HI = (float)LN2, LO = (float)(LN2 - (double)HI);
  const float y = x * 1.44269504088896340736f, d = fmaf(-y, LO, fmaf(-y, HI, x));
  const float p = __builtin_amdgcn_exp2f(y);
  return fmaf(p, fmaxf(d, -1.f), p);
}

// A row's e = exp(l - top), their sum (0: no expert, NaN: a NaN or +inf among them) and top; l in e at the call
template <int L, int E>
__device__ __forceinline__ void softmax_row(float (&e)[E], float* den, float* top) {
  float mx = e[0];
#pragma unroll
  for (int i = 1; i < E; ++i) mx = fmaxf(mx, e[i]);
  mx = max_row<L>(mx);
  if (mx == -INFINITY) mx = 0.f;
  float sum = 0.f;
#pragma unroll
  for (int i = 0; i < E; ++i) {
    e[i] = exp_of(e[i] - mx);
    sum += e[i];
  }
  *den = sum_row<L>(sum);
  *top = mx;
}

// The workgroup's sums of N values in every thread; waves in order
template <int N>
__device__ __forceinline__ void block_sums(double (&v)[N], double* red) {
#pragma unroll
  for (int o = 32; o > 0; o >>= 1)
#pragma unroll
    for (int n = 0; n < N; ++n) v[n] += __shfl_xor(v[n], o, 64);
  __syncthreads();  // red may hold the sums before
  if ((threadIdx.x & 63) == 0)
#pragma unroll
    for (int n = 0; n < N; ++n) red[(threadIdx.x >> 6) * N + n] = v[n];
  __syncthreads();
#pragma unroll
  for (int n = 0; n < N; ++n) {
    v[n] = red[n];
#pragma unroll
    for (int w = 1; w < WAVES; ++w) v[n] += red[w * N + n];
  }
}

// Orders the wave's own LDS accesses, which execute in program order, for the compiler
__device__ __forceinline__ void wave_order() {
  __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
  __builtin_amdgcn_wave_barrier();
  __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
}

// Parts of a sequence at most: a workgroup for each CU.  Up to DIRECT of them are joined by the last one; of more, each GROUP by its
// last, and the groups by theirs
constexpr int DIRECT = 32, GROUP = 16;
__host__ __device__ inline int most_parts(int sequences) { return (256 + sequences - 1) / sequences; }
__host__ __device__ inline int groups_of(int parts) { return parts > DIRECT ? (parts + GROUP - 1) / GROUP : 0; }

// The workspace: counters (zero between calls) of the sequences and of each sequence's groups and parts, each sequence's {B, Z}, then
// each part's Z, and sums of p and counts of the parts and of the groups
struct Workspace {
  uint32_t *counters, *part_counters;
  double *seq, *part_z, *part_p, *group_p;
  int32_t *part_n, *group_n;
};
__host__ __device__ inline int64_t seq_counter_words(int sequences) {
  const int most = most_parts(sequences);
  return most > 1 ? JOIN_STRIDE * (1 + groups_of(most)) : 0;
}
__host__ __device__ inline int64_t counter_words(int sequences) { return join_words(512) + sequences * seq_counter_words(sequences); }
__host__ __device__ inline Workspace ws_of(void* p, int64_t sequences, int parts, int experts) {
  Workspace w;
  const int64_t groups = groups_of(parts);
  w.counters = (uint32_t*)p;
  w.part_counters = w.counters + join_words(512);
  w.seq = (double*)(w.counters + counter_words((int)sequences));
  w.part_z = w.seq + 2 * sequences;
  w.part_p = w.part_z + sequences * parts;
  w.group_p = w.part_p + sequences * parts * experts;
  w.part_n = (int32_t*)(w.group_p + sequences * groups * experts);
  w.group_n = w.part_n + sequences * parts * experts;
  return w;
}

// One thread: the means and the losses, from the sequences with rows, their rows, and the sums of their parts of B and Z
__device__ __forceinline__ void finish(const RouterLaunch& a, double live, double rows, double B, double Z) {
  B /= fmax(live, 1.);
  Z /= fmax(rows, 1.);
  a.means[0] = (int)live;
  a.means[1] = (int)rows;
  a.losses[0] = (float)((double)a.balance * B + (double)a.z * Z);
  a.losses[1] = (float)B;
  a.losses[2] = (float)Z;
}

template <int L, int NV>
__global__ __launch_bounds__(BLOCK, 4) void k_router_loss(RouterLaunch a, int parts) {
  constexpr int E = 4 * NV, RW = 64 / L, COLS = L * E;
  constexpr int SLICES = COLS < BLOCK ? BLOCK / COLS : 1;  // of a sequence's parts, taken by threads of their own
  constexpr int HELD = COLS <= 512 ? WAVES : WAVES / 2;    // waves whose columns' sums are in LDS at once
  __shared__ double col[(HELD > SLICES ? HELD : SLICES) * COLS], red[WAVES * 4];
  __shared__ int32_t hist[COLS], many[SLICES * COLS], flag;
  const int lane = lane_id(), wave = threadIdx.x >> 6, l = lane % L, sub = lane / L, G = a.experts;
  const Workspace ws = ws_of(a.workspace, a.sequences, parts, G);
  int mine = -1;  // the last sequence that this workgroup ended
  for (int64_t u = blockIdx.x; u < (int64_t)a.sequences * parts; u += gridDim.x) {
    const int s = (int)(u / parts), part = (int)(u % parts);
    int first, end;
    span_of(a, s, &first, &end);
    const int len = end - first, r0 = first + (int)((int64_t)len * part / parts), r1 = first + (int)((int64_t)len * (part + 1) / parts);
    // the probabilities; the next rows' loads go out before the current rows' sums
    double p[E], z = 0;
    float next[E];
#pragma unroll
    for (int e = 0; e < E; ++e) p[e] = 0;
    auto fetch = [&](int base) {
      const int t = min(base + sub, r1 - 1);
#pragma unroll
      for (int j = 0; j < NV; ++j) load_cols(a.logits + (int64_t)t * G, (j * L + l) * 4, G, -INFINITY, next + 4 * j);
    };
    int base = r0 + wave * RW;
    if (base < r1) fetch(base);
    for (int c = threadIdx.x; c < COLS; c += BLOCK) hist[c] = 0;
    __syncthreads();
    // the chosen experts
    for (int64_t i = (int64_t)r0 * a.top_k + threadIdx.x; i < (int64_t)r1 * a.top_k; i += BLOCK) {
      const int id = a.topk_idx[i];
      if (id >= 0 && id < G) atomicAdd(&hist[id], 1);
    }
    for (; base < r1; base += WAVES * RW) {
      float e[E], den, top;
#pragma unroll
      for (int i = 0; i < E; ++i) e[i] = next[i];
      if (base + WAVES * RW < r1) fetch(base + WAVES * RW);
      softmax_row<L>(e, &den, &top);
      if (base + sub < r1 && den != 0.f) {
        const float inv = 1.f / den;
        const double lse = top + logf(den);
#pragma unroll
        for (int i = 0; i < E; ++i) p[i] += e[i] * inv;
        z += lse * lse;
      }
    }
#pragma unroll
    for (int o = L; o < 64; o *= 2)
#pragma unroll
      for (int e = 0; e < E; ++e) p[e] += __shfl_xor(p[e], o, 64);
    if (l != 0) z = 0;  // a row's lanes all hold it
    // column c's sum and count in thread c (of G > BLOCK also c + BLOCK), the waves in order
    constexpr int PER = COLS > BLOCK ? COLS / BLOCK : 1;
    double q[PER];
    int n[PER];
#pragma unroll
    for (int k = 0; k < PER; ++k) q[k] = 0;
    for (int w0 = 0; w0 < WAVES; w0 += HELD) {
      if (w0 > 0) __syncthreads();
      if (sub == 0 && wave >= w0 && wave < w0 + HELD)
#pragma unroll
        for (int e = 0; e < E; ++e) col[(wave - w0) * COLS + (e / 4 * L + l) * 4 + e % 4] = p[e];
      __syncthreads();
#pragma unroll
      for (int k = 0; k < PER; ++k) {
        const int c = threadIdx.x + k * BLOCK;
        if (c < COLS)
#pragma unroll
          for (int w = 0; w < HELD; ++w) q[k] += col[w * COLS + c];
      }
    }
#pragma unroll
    for (int k = 0; k < PER; ++k) n[k] = (int)(threadIdx.x + k * BLOCK) < COLS ? hist[threadIdx.x + k * BLOCK] : 0;
    if (parts > 1) {
      double v[1] = {z};
      block_sums(v, red);
      if (threadIdx.x == 0) hand_out(&ws.part_z[u], v[0]);
      z = 0;
      // to the last of the parts, or of a group of them and on to the last of the groups
      const int groups = groups_of(parts), group = part / GROUP;
      uint32_t* counters = ws.part_counters + s * seq_counter_words(a.sequences);
      double* to_p = ws.part_p + (int64_t)s * parts * G;
      int32_t* to_n = ws.part_n + (int64_t)s * parts * G;
      int place = part, from = groups > 0 ? group * GROUP : 0, count = groups > 0 ? min(GROUP, parts - from) : parts;
      uint32_t* counter = groups > 0 ? counters + (1 + group) * JOIN_STRIDE : counters;
      bool last;
#pragma unroll 1
      for (int level = groups > 0 ? 0 : 1; level < 2; ++level) {
#pragma unroll
        for (int k = 0; k < PER; ++k) {
          const int c = threadIdx.x + k * BLOCK;
          if (c < G) {
            hand_out(&to_p[(int64_t)place * G + c], q[k]);
            hand_out(&to_n[(int64_t)place * G + c], n[k]);
          }
        }
        last = last_of(counter, 0, count, &flag);
        if (!last) break;
        if (level == 1 && (int)threadIdx.x < parts) z = take(&ws.part_z[(int64_t)s * parts + threadIdx.x]);  // parts <= 256
        const int slice = SLICES > 1 ? threadIdx.x / COLS : 0;
        const int c0 = SLICES > 1 ? threadIdx.x % COLS : threadIdx.x;
        double sum[PER];
        int total[PER];
#pragma unroll
        for (int k = 0; k < PER; ++k) sum[k] = total[k] = 0;
#pragma unroll 1
        for (int i = slice; i < count; i += 8 * SLICES) {
          double pq[PER][8];
          int pn[PER][8];
#pragma unroll
          for (int k = 0; k < PER; ++k)
#pragma unroll
            for (int m = 0; m < 8; ++m) {
              const int at = i + m * SLICES, c = c0 + k * BLOCK;
              pq[k][m] = at < count && c < G ? take(&to_p[(int64_t)(from + at) * G + c]) : 0.;
              pn[k][m] = at < count && c < G ? take(&to_n[(int64_t)(from + at) * G + c]) : 0;
            }
#pragma unroll
          for (int k = 0; k < PER; ++k)
#pragma unroll
            for (int m = 0; m < 8; ++m) {
              sum[k] += pq[k][m];
              total[k] += pn[k][m];
            }
        }
#pragma unroll
        for (int k = 0; k < PER; ++k) {
          if (SLICES > 1) {
            col[slice * COLS + c0] = sum[k];
            many[slice * COLS + c0] = total[k];
          } else {
            q[k] = sum[k];
            n[k] = total[k];
          }
        }
        if (SLICES > 1) {
          __syncthreads();
          q[0] = 0;
          n[0] = 0;
          if (threadIdx.x < COLS)
#pragma unroll
            for (int w = 0; w < SLICES; ++w) {
              q[0] += col[w * COLS + threadIdx.x];
              n[0] += many[w * COLS + threadIdx.x];
            }
        }
        to_p = ws.group_p + (int64_t)s * groups * G;
        to_n = ws.group_n + (int64_t)s * groups * G;
        place = group;
        from = 0;
        count = groups;
        counter = counters;
      }
      if (!last) continue;
    }
    // the sequence: its counts, and its parts of B (f_g = G n_g / sum of n) and Z
    double v[3] = {0, 0, z};
#pragma unroll
    for (int k = 0; k < PER; ++k) {
      const int c = threadIdx.x + k * BLOCK;
      if (c < G) {
        a.counts[(int64_t)s * G + c] = n[k];
        v[0] += n[k];
        v[1] += n[k] * q[k];
      }
    }
    block_sums(v, red);
    const double b = v[0] > 0 && len > 0 ? G / v[0] * v[1] / len : 0.;
    if (a.sequences == 1) {
      if (threadIdx.x == 0) finish(a, len > 0, len, b, v[2]);
      return;
    }
    if (threadIdx.x == 0) {
      hand_out(&ws.seq[2 * (int64_t)s], b);
      hand_out(&ws.seq[2 * (int64_t)s + 1], v[2]);
    }
    mine = s;
  }
  // the batch: the last workgroup, or, where sequences have parts (and each workgroup one of them), the last to end a sequence
  if (parts > 1 && mine < 0) return;
  int f = 0, e = 0;
  if ((int)threadIdx.x < a.sequences) span_of(a, threadIdx.x, &f, &e);  // on its way during the wait
  if (!last_of(ws.counters, parts > 1 ? mine : blockIdx.x, parts > 1 ? a.sequences : gridDim.x, &flag)) return;
  double t[4] = {0, 0, 0, 0};  // sequences with rows, rows, B, Z
  for (int k = threadIdx.x; k < a.sequences; k += BLOCK) {
    if (k >= BLOCK) span_of(a, k, &f, &e);
    t[0] += e > f;
    t[1] += e - f;
    t[2] += take(&ws.seq[2 * (int64_t)k]);
    t[3] += take(&ws.seq[2 * (int64_t)k + 1]);
  }
  block_sums(t, red);
  if (threadIdx.x == 0) finish(a, t[0], t[1], t[2], t[3]);
}

// The last sequence that begins at or before row t, by the row's L lanes: each step they look at L of what is left, so that a few dozen
// sequences are one or two loads one after another
template <int L>
__device__ __forceinline__ int sequence_of(const RouterLaunch& a, int t, int l) {
  const int shift = lane_id() / L * L;
  int at = 0, left = a.sequences;  // it is one of [at, at + left), or there is none
  bool none = false;
  do {
    const int step = (left + L - 1) / L, i = l * step;
    const uint64_t m = __ballot(i < left && a.spans[2 * (int64_t)(at + i)] <= t) >> shift;
    const int n = __popcll(L == 64 ? m : m & ((1ull << (L & 63)) - 1));
    none |= n == 0;
    const int skip = max(n - 1, 0) * step;
    at += skip;
    left = min(step, left - skip);
  } while (__ballot(left > 1) != 0);
  return none ? -1 : at;
}

// The gradient.  A wave takes `rows` rows in a row, so that it meets few sequences: f of the last one stays in registers
template <int L, int NV, class O>
__global__ __launch_bounds__(256) void k_router_bwd(RouterLaunch a, int rows) {
  constexpr int E = 4 * NV, RW = 64 / L, COLS = L * E;
  constexpr bool BY_LDS = NV > 1;  // where a row's slots' gradients find their columns: in LDS, or by comparing
  __shared__ float slots[BY_LDS ? 4 * RW * COLS : 1];
  const int lane = lane_id(), wave = threadIdx.x >> 6, l = lane % L, sub = lane / L, G = a.experts, K = a.top_k;
  float* mine = slots + (BY_LDS ? (wave * RW + sub) * COLS : 0);
  if (BY_LDS) {
#pragma unroll
    for (int j = 0; j < NV; ++j) *(float4*)(mine + (j * L + l) * 4) = float4{0, 0, 0, 0};
    wave_order();
  }
  const float dl = a.d_loss ? *a.d_loss : 1.f;
  const float cb = dl * a.balance / (float)max(a.means[0], 1), cz = 2.f * dl * a.z / (float)max(a.means[1], 1);
  const int64_t begin = ((int64_t)blockIdx.x * 4 + wave) * rows, end = min(begin + rows, a.tokens);
  int first = 0, last = 0;  // of the sequence whose f is held
  bool found = false;
  float f[E];
#pragma unroll
  for (int i = 0; i < E; ++i) f[i] = 0.f;
  for (int64_t base = begin; base < end; base += RW) {
    const int t = (int)min(base + sub, end - 1);  // rows past the end: the last one again, not stored
    const bool live = base + sub < end;
    float e[E], den, top, g[E];
#pragma unroll
    for (int j = 0; j < NV; ++j) load_cols(a.logits + (int64_t)t * G, (j * L + l) * 4, G, -INFINITY, e + 4 * j);
    int id = -1;  // BY_LDS: lane l's slot; its loads too go out before the sequence is looked up
    float w = 0.f;
    if (BY_LDS && a.d_weights && l < K) {
      id = a.topk_idx[(int64_t)t * K + l];
      w = a.d_weights[(int64_t)t * K + l];
    }
    if (__ballot(!found || t < first || t >= last)) {
      // the last sequence that begins at or before t; what lies between it and the next one is padding
      int s;
      if (!a.spans) s = t / ((int)a.tokens / a.sequences);
      else {
        s = sequence_of<L>(a, t, l);
      }
      first = 0;
      last = 0;
      if (s >= 0) span_of(a, s, &first, &last);
      found = true;
      const int32_t* n = a.counts + (int64_t)max(s, 0) * G;
      float total = 0.f;
#pragma unroll
      for (int j = 0; j < NV; ++j)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int c = (j * L + l) * 4 + i;
          const int v = c < G ? n[c] : 0;
          f[4 * j + i] = (float)v;
          total += (float)v;
        }
      total = sum_row<L>(total);
      const float share = total > 0.f && last > first ? cb / (float)(last - first) * ((float)G / total) : 0.f;
#pragma unroll
      for (int i = 0; i < E; ++i) f[i] *= share;
    }
    const bool inside = t >= first && t < last;
    softmax_row<L>(e, &den, &top);
#pragma unroll
    for (int i = 0; i < E; ++i) g[i] = f[i];
    if (a.d_weights) {
      const int64_t at = (int64_t)t * K;
      if (BY_LDS) {
        const bool good = id >= 0 && id < G;
        // all slots at once where no two of a row's have one expert, which their numbers at its place show; else one after another
        if (good) mine[id] = __int_as_float(l);
        wave_order();
        const bool taken = good && __float_as_int(mine[id]) != l;
        wave_order();
        if (__ballot(taken) == 0) {
          if (good) mine[id] = w;
        } else {
          if (good) mine[id] = 0.f;
          wave_order();
          for (int j = 0; j < K; ++j) {
            if (l == j && good) mine[id] += w;
            wave_order();  // for a lane by itself the loop is one addition: the next lane's comes after it
          }
        }
        wave_order();
#pragma unroll
        for (int j = 0; j < NV; ++j) {
          const float4 q = *(const float4*)(mine + (j * L + l) * 4);
          g[4 * j] += q.x;
          g[4 * j + 1] += q.y;
          g[4 * j + 2] += q.z;
          g[4 * j + 3] += q.w;
        }
        wave_order();
        if (good) mine[id] = 0.f;
        wave_order();
      } else {
        float q[E];
#pragma unroll
        for (int i = 0; i < E; ++i) q[i] = 0.f;
        for (int j = 0; j < K; ++j) {
          const int id = a.topk_idx[at + j];
          const float w = a.d_weights[at + j];
#pragma unroll
          for (int i = 0; i < E; ++i)
            if (id == l * 4 + i && id < G) q[i] += w;
        }
#pragma unroll
        for (int i = 0; i < E; ++i) g[i] += q[i];
      }
    }
    const bool none = !inside || den == 0.f;
    const float inv = 1.f / den, lse = top + logf(den);
    float dot = 0.f;
#pragma unroll
    for (int i = 0; i < E; ++i) {
      e[i] *= inv;
      dot = fmaf(e[i], g[i], dot);
    }
    dot = sum_row<L>(dot);
    const float off = fmaf(cz, lse, -dot);
#pragma unroll
    for (int i = 0; i < E; ++i) g[i] = none ? 0.f : e[i] * (g[i] + off);
    if (!live) continue;
    O* out = (O*)a.dlogits + (int64_t)t * G;
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int c = (j * L + l) * 4, n = G - c;
      const float* v = g + 4 * j;
      if constexpr (sizeof(O) == 4) {
        if (n > 0) Chunk<float>::store((float*)out + c, Chunk<float>::pack(v), n);
      } else if (n >= 4) {
        const uint32_t q[2] = {pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3])};
        __builtin_memcpy(out + c, q, 8);
      } else
#pragma unroll
        for (int i = 0; i < 3; ++i)
          if (i < n) out[c + i] = f32_to_bf16(v[i]);
    }
  }
}

// Lanes to a row and float4 in each: the fewest lanes that hold it in four, from quads on
template <class F>
void by_width(int G, F f) {
  if (G <= 16) f(integral_constant<int, 4>{}, integral_constant<int, 1>{});
  else if (G <= 64) f(integral_constant<int, 16>{}, integral_constant<int, 1>{});
  else if (G <= 128) f(integral_constant<int, 16>{}, integral_constant<int, 2>{});
  else if (G <= 256) f(integral_constant<int, 16>{}, integral_constant<int, 4>{});
  else if (G <= 512) f(integral_constant<int, 64>{}, integral_constant<int, 2>{});
  else f(integral_constant<int, 64>{}, integral_constant<int, 4>{});
}

// Parts of a sequence, two rounds of a workgroup's rows in each at least
int parts_of(int64_t tokens, int experts, int sequences) {
  const int64_t rows = WAVES * (experts <= 16 ? 16 : experts <= 256 ? 4 : 1) * 2;
  return (int)std::max<int64_t>(1, std::min<int64_t>(most_parts(sequences), tokens / sequences / rows));
}

}  // namespace

int64_t router_workspace_bytes(int64_t tokens, int experts, int sequences) {
  const int parts = parts_of(tokens, experts, sequences);
  return 4 * counter_words(sequences) + sequences * (16 + parts * 8ll + (parts + groups_of(parts)) * 12ll * experts);
}

int launch_router_loss(const RouterLaunch& a, hipStream_t st) {
  const int parts = parts_of(a.tokens, a.experts, a.sequences);
  const dim3 grid((unsigned)std::min<int64_t>((int64_t)a.sequences * parts, 512));  // two on a CU; with parts there are fewer
  by_width(a.experts, [&](auto l, auto nv) {
    hipLaunchKernelGGL((k_router_loss<decltype(l)::value, decltype(nv)::value>), grid, dim3(BLOCK), 0, st, a, parts);
  });
  return hipGetLastError() == hipSuccess ? 0 : -1;
}

int launch_router_backward(const RouterLaunch& a, hipStream_t st) {
  if (a.tokens == 0) return 0;
  by_width(a.experts, [&](auto l, auto nv) {
    constexpr int L = decltype(l)::value, NV = decltype(nv)::value, RW = 64 / L;
    // as many rows to a wave as leave each SIMD four waves
    const int64_t most = std::max<int64_t>(8, a.tokens >> 24);  // and few enough workgroups for a launch
    const int rows = (int)std::min<int64_t>(std::max<int64_t>((a.tokens + 4096 * RW - 1) / (4096 * RW), 1), most) * RW;
    const dim3 grid((unsigned)((a.tokens + 4 * rows - 1) / (4 * rows)));
    if (a.dtype == MOE_F32) hipLaunchKernelGGL((k_router_bwd<L, NV, float>), grid, dim3(256), 0, st, a, rows);
    else hipLaunchKernelGGL((k_router_bwd<L, NV, bf16_t>), grid, dim3(256), 0, st, a, rows);
  });
  return hipGetLastError() == hipSuccess ? 0 : -1;
}
