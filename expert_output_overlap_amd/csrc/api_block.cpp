// C ABI of the operators around the routed experts: layer norm, the shared expert's block, AdamW (declarations and
// contracts in include/moe_overlap.h).  Host side only: argument checks and launches on the caller's stream.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <cfloat>
#include <cmath>
#include <exception>
#include <vector>

#include "../../include/moe_overlap.h"
#include "launch.h"

namespace {

int64_t elem(int dtype) { return dtype == MOE_BF16 ? 2 : 4; }

bool is_dtype(int t) { return t == MOE_BF16 || t == MOE_F32; }

bool off(const void* p, uintptr_t align) { return (uintptr_t)p % align != 0; }

struct Span {  // n bytes, or rows of `row` bytes every `stride` bytes in them
  const void* p;
  int64_t n, row = 0, stride = 0;
};

// Bytes of two buffers in common.  Rows of one stride may lie between each other's, as two slices of one wider tensor do
bool meet(const Span& a, const Span& b) {
  const uintptr_t p = (uintptr_t)a.p, q = (uintptr_t)b.p;
  if (!p || !q || a.n <= 0 || b.n <= 0 || p >= q + (uintptr_t)b.n || q >= p + (uintptr_t)a.n) return false;
  if (a.stride == 0 || a.stride != b.stride) return true;
  const int64_t s = a.stride, to = (int64_t)((p < q ? q - p : p - q) % (uintptr_t)s);  // from the lower one's row on
  const Span &low = p < q ? a : b, &high = p < q ? b : a;
  return to < low.row || to + high.row > s;
}

// Whether an output overlaps an input or another output; same(o, i): a pair that may be the same buffer
template <int O, int I, class F>
bool overlaps(const Span (&out)[O], const Span (&in)[I], F same) {
  for (int o = 0; o < O; ++o) {
    for (int i = 0; i < I; ++i)
      if (meet(out[o], in[i]) && !(out[o].p == in[i].p && same(o, i))) return true;
    for (int q = 0; q < o; ++q)
      if (meet(out[o], out[q])) return true;
  }
  return false;
}

const char* check_norm(const moe_norm_shape* s) {
  if (!s) return "null shape";
  if (s->rows < 0 || s->rows > (1ll << 40)) return "rows must be in [0, 2^40]";
  if (s->d < 1 || s->d > MOE_NORM_MAX_D) return "d must be in [1, MOE_NORM_MAX_D]";
  if (!is_dtype(s->dtype) || !is_dtype(s->param_dtype)) return "dtype must be MOE_BF16 or MOE_F32";
  if (!(s->eps > 0.f) || !std::isfinite(s->eps)) return "eps must be positive and finite";
  for (const int64_t stride : {s->x_stride, s->y_stride, s->dx_stride})
    if (stride != 0 && (stride < s->d || stride > (1ll << 46) / std::max<int64_t>(s->rows, 1)))
      return "a row stride must be 0 or at least d, and rows x stride at most 2^46";
  return nullptr;
}

NormLaunch norm_of(const moe_norm_shape* s) {
  NormLaunch a{};
  a.rows = s->rows;
  a.d = s->d;
  a.dtype = s->dtype;
  a.param_dtype = s->param_dtype;
  a.eps = s->eps;
  a.x_stride = s->x_stride ? s->x_stride : s->d;
  a.y_stride = s->y_stride ? s->y_stride : s->d;
  a.dx_stride = s->dx_stride ? s->dx_stride : s->d;
  return a;
}

// All rows of a matrix of the norm's, one every `stride` elements
Span norm_rows(const moe_norm_shape* s, const void* p, int64_t stride) {
  const int64_t es = elem(s->dtype);
  return {p, ((s->rows - 1) * stride + s->d) * es, s->d * es, stride * es};
}

const char* check_shared(const moe_shared_shape* s) {
  if (!s) return "null shape";
  if (s->tokens < 0 || s->tokens > (1ll << 27)) return "tokens must be in [0, 2^27]";
  if (s->d < 1 || s->d > 65536) return "d must be in [1, 65536]";
  if (s->f < 1 || s->f > 65536) return "f must be in [1, 65536]";
  if (!is_dtype(s->dtype)) return "dtype must be MOE_BF16 or MOE_F32";
  if (s->tokens * std::max(s->d, 2 * s->f) > (1ll << 34)) return "tokens x max(d, 2f) must be at most 2^34";
  return nullptr;
}

int shared_row(const moe_shared_shape* s) { return (s->f + 7) / 8 * 8; }

const char* check_adamw(const moe_adamw_tensor* t, int32_t n) {
  if (n < 0 || (n > 0 && !t)) return "null tensors";
  int64_t chunks = 0;
  for (int i = 0; i < n; ++i) {
    const moe_adamw_tensor& a = t[i];
    if (a.n < 0 || a.n > (1ll << 40)) return "elements must be in [0, 2^40]";
    if (!is_dtype(a.param_dtype) || !is_dtype(a.grad_dtype)) return "dtype must be MOE_BF16 or MOE_F32";
    if (a.state_bits != 32 && a.state_bits != 8) return "state_bits must be 32 or 8";
    if (a.reserved != 0) return "reserved must be 0";
    if (!std::isfinite(a.weight_decay) || !std::isfinite(a.lr_scale)) return "weight_decay and lr_scale must be finite";
    if (a.n == 0) continue;
    if (!a.param || !a.grad || !a.m || !a.v) return "null pointer";
    if (a.state_bits == 8 && (!a.m_scale || !a.v_scale)) return "8-bit states need their scales";
    if (a.state_bits == 32 && (a.m_scale || a.v_scale || a.m_values || a.root_values))
      return "scales and values are for 8-bit states";
    if (off(a.param, elem(a.param_dtype)) || off(a.grad, elem(a.grad_dtype)) || off(a.copy, 2) || off(a.m_values, 2) ||
        off(a.root_values, 2) || (a.state_bits == 32 && (off(a.m, 4) || off(a.v, 4))))
      return "a tensor must be aligned to its elements";
    chunks += (a.n + ADAMW_CHUNK - 1) / ADAMW_CHUNK;
  }
  // 256 threads each, under 2^32 in a launch
  return chunks >= 1 << 24 ? "too many elements for one plan" : nullptr;
}

int64_t adamw_chunks(const moe_adamw_tensor* t, int32_t n) {
  int64_t c = 0;
  for (int i = 0; i < n; ++i) c += (t[i].n + ADAMW_CHUNK - 1) / ADAMW_CHUNK;
  return c;
}

int64_t chunk_bytes(int64_t n_chunks) { return (n_chunks * (int64_t)sizeof(AdamwChunk) + 255) / 256 * 256; }

AdamwStep adamw_of(const moe_adamw_plan* p) {
  AdamwStep a{};
  a.chunks = (const AdamwChunk*)p->table;
  a.tensors = (const AdamwDesc*)((const char*)p->table + chunk_bytes(p->n_chunks));
  return a;
}

const char* check_plan(const moe_adamw_plan* p) {
  if (!p || p->n_chunks < 0 || p->n_chunks > 0x7fffffff || (p->n_chunks > 0 && !p->table)) return "plan not bound";
  return nullptr;
}

}  // namespace

extern "C" {

int moe_layer_norm(const moe_norm_shape* s, const void* x, const void* weight, const void* bias, void* y, float* mean,
                   float* rstd, void* stream) {
  if (const char* e = check_norm(s)) return moe_fail(MOE_EINVAL, e);
  if (s->rows > 0 && (!x || !y)) return moe_fail(MOE_EINVAL, "null pointer");
  if (!mean != !rstd) return moe_fail(MOE_EINVAL, "mean and rstd go together");
  if (off(x, elem(s->dtype)) || off(y, elem(s->dtype)) || off(weight, elem(s->param_dtype)) ||
      off(bias, elem(s->param_dtype)) || off(mean, 4) || off(rstd, 4))
    return moe_fail(MOE_EINVAL, "a tensor must be aligned to its elements");
  NormLaunch a = norm_of(s);
  if (s->rows > 0) {
    const int64_t np = s->d * elem(s->param_dtype);
    const Span out[] = {norm_rows(s, y, a.y_stride), {mean, 4 * s->rows}, {rstd, 4 * s->rows}},
               in[] = {norm_rows(s, x, a.x_stride), {weight, np}, {bias, np}};
    if (overlaps(out, in, [&](int o, int i) { return o == 0 && i == 0 && a.x_stride == a.y_stride; }))
      return moe_fail(MOE_EINVAL, "an output overlaps an input or another output");
  }
  a.x = x;
  a.weight = weight;
  a.bias = bias;
  a.y = y;
  a.mean = mean;
  a.rstd = rstd;
  return launch_norm(a, (hipStream_t)stream) ? moe_fail(MOE_EHIP, "layer norm launch failed") : MOE_OK;
}

int64_t moe_layer_norm_workspace_bytes(const moe_norm_shape* s) {
  return check_norm(s) ? -1 : 4 * norm_partial_floats(s->rows, s->d, s->dtype);
}

int moe_layer_norm_backward(const moe_norm_shape* s, const void* dy, const void* x, const void* weight, const float* mean,
                            const float* rstd, const void* residual, void* dx, void* dweight, void* dbias,
                            void* workspace, int64_t workspace_bytes, void* stream) {
  if (const char* e = check_norm(s)) return moe_fail(MOE_EINVAL, e);
  if (s->rows > 0 && (!dy || !x || !mean || !rstd || !dx)) return moe_fail(MOE_EINVAL, "null pointer");
  if (off(x, elem(s->dtype)) || off(dy, elem(s->dtype)) || off(residual, elem(s->dtype)) || off(dx, elem(s->dtype)) ||
      off(weight, elem(s->param_dtype)) || off(dweight, elem(s->param_dtype)) || off(dbias, elem(s->param_dtype)) ||
      off(mean, 4) || off(rstd, 4) || off(workspace, 16))
    return moe_fail(MOE_EINVAL, "a tensor must be aligned to its elements, the workspace to 16 bytes");
  NormLaunch a = norm_of(s);
  const bool params = dweight || dbias;
  if (params) {
    const int64_t need = moe_layer_norm_workspace_bytes(s);
    if (need > 0 && (!workspace || workspace_bytes < need)) return moe_fail(MOE_EINVAL, "workspace too small");
  }
  if (s->rows > 0) {
    const int64_t np = s->d * elem(s->param_dtype);
    const Span out[] = {norm_rows(s, dx, a.dx_stride), {dweight, np}, {dbias, np},
                        {params ? workspace : nullptr, moe_layer_norm_workspace_bytes(s)}},
               in[] = {norm_rows(s, dy, a.y_stride), norm_rows(s, residual, a.dx_stride), norm_rows(s, x, a.x_stride), {weight, np}, {mean, 4 * s->rows}, {rstd, 4 * s->rows}};
    if (overlaps(out, in, [&](int o, int i) { return o == 0 && (i == 1 || (i == 0 && a.y_stride == a.dx_stride)); }))
      return moe_fail(MOE_EINVAL, "an output overlaps an input or another output");
  }
  a.backward = true;
  a.dy = dy;
  a.x = x;
  a.weight = weight;
  a.mean = (float*)mean;
  a.rstd = (float*)rstd;
  a.residual = residual;
  a.dx = dx;
  a.dweight = dweight;
  a.dbias = dbias;
  a.partial = params ? (float*)workspace : nullptr;
  return launch_norm(a, (hipStream_t)stream) ? moe_fail(MOE_EHIP, "layer norm backward launch failed") : MOE_OK;
}

int64_t moe_shared_ffn_row(const moe_shared_shape* s) { return check_shared(s) ? -1 : shared_row(s); }

int64_t moe_shared_ffn_workspace_bytes(const moe_shared_shape* s, int32_t backward) {
  return check_shared(s) ? -1 : shared_workspace_bytes(s->tokens, s->d, s->f, s->dtype, backward != 0);
}

int moe_shared_ffn(const moe_shared_shape* s, const void* x, const void* w_gate_up, const void* w_down,
                   const void* residual, void* h, float* gu, void* y, void* workspace, int64_t workspace_bytes,
                   void* stream) {
  if (const char* e = check_shared(s)) return moe_fail(MOE_EINVAL, e);
  if (s->tokens == 0) return MOE_OK;
  if (!x || !w_gate_up || !w_down || !h || !y) return moe_fail(MOE_EINVAL, "null pointer");
  for (const void* p : {x, w_gate_up, w_down, residual, (const void*)h, (const void*)gu, (const void*)y,
                        (const void*)workspace})
    if (off(p, 16)) return moe_fail(MOE_EINVAL, "every tensor must be 16-byte aligned");
  const int64_t need = moe_shared_ffn_workspace_bytes(s, 0);
  if (need > 0 && (!workspace || workspace_bytes < need)) return moe_fail(MOE_EINVAL, "workspace too small");
  const int64_t es = elem(s->dtype), nx = s->tokens * s->d * es, nw = (int64_t)s->d * s->f * es,
                nh = s->tokens * shared_row(s) * es, ngu = s->tokens * 2 * shared_row(s) * 4;
  const Span out[] = {{y, nx}, {h, nh}, {gu, ngu}, {workspace, need}},
             in[] = {{residual, nx}, {x, nx}, {w_gate_up, 2 * nw}, {w_down, nw}};
  if (overlaps(out, in, [](int o, int i) { return o == 0 && i == 0; }))
    return moe_fail(MOE_EINVAL, "an output overlaps an input or another output");
  SharedLaunch a{};
  a.tokens = s->tokens;
  a.d = s->d;
  a.f = s->f;
  a.row = shared_row(s);
  a.dtype = s->dtype;
  a.x = x;
  a.w_gate_up = w_gate_up;
  a.w_down = w_down;
  a.residual = residual;
  a.h = h;
  a.gu = gu;
  a.y = y;
  a.workspace = workspace;
  return launch_shared(a, (hipStream_t)stream) ? moe_fail(MOE_EHIP, "shared expert launch failed") : MOE_OK;
}

int moe_shared_ffn_backward(const moe_shared_shape* s, const moe_shared_bwd_args* b, void* workspace,
                            int64_t workspace_bytes, void* stream) {
  if (const char* e = check_shared(s)) return moe_fail(MOE_EINVAL, e);
  if (!b || !b->dw_gate_up || !b->dw_down || !b->w_gate_up || !b->w_down ||
      (s->tokens > 0 && (!b->x || !b->h || !b->gu || !b->dy || !b->dgu_ws || !b->dx)))
    return moe_fail(MOE_EINVAL, "null pointer");
  for (const void* p : {b->x, b->w_gate_up, b->w_down, b->h, (const void*)b->gu, b->dy, b->residual, (const void*)b->dgu_ws,
                        (const void*)b->dx, (const void*)b->dw_gate_up, (const void*)b->dw_down, (const void*)workspace})
    if (off(p, 16)) return moe_fail(MOE_EINVAL, "every tensor must be 16-byte aligned");
  const int64_t need = moe_shared_ffn_workspace_bytes(s, 1);
  if (need > 0 && (!workspace || workspace_bytes < need)) return moe_fail(MOE_EINVAL, "workspace too small");
  const int64_t es = elem(s->dtype), nx = s->tokens * s->d * es, nw = (int64_t)s->d * s->f * es,
                nh = s->tokens * shared_row(s) * es, ngu = s->tokens * 2 * shared_row(s) * 4;
  const Span out[] = {{b->dx, nx}, {b->dgu_ws, 2 * nh}, {b->dw_gate_up, 2 * nw}, {b->dw_down, nw}, {workspace, need}},
             in[] = {{b->residual, nx}, {b->x, nx}, {b->w_gate_up, 2 * nw}, {b->w_down, nw}, {b->h, nh}, {b->gu, ngu}, {b->dy, nx}};
  if (overlaps(out, in, [](int o, int i) { return o == 0 && i == 0; }))
    return moe_fail(MOE_EINVAL, "an output overlaps an input or another output");
  SharedLaunch a{};
  a.backward = true;
  a.tokens = s->tokens;
  a.d = s->d;
  a.f = s->f;
  a.row = shared_row(s);
  a.dtype = s->dtype;
  a.x = b->x;
  a.w_gate_up = b->w_gate_up;
  a.w_down = b->w_down;
  a.h = (void*)b->h;
  a.gu = (float*)b->gu;
  a.dy = b->dy;
  a.residual = b->residual;
  a.dgu = b->dgu_ws;
  a.dx = b->dx;
  a.dw_gate_up = b->dw_gate_up;
  a.dw_down = b->dw_down;
  a.workspace = workspace;
  return launch_shared(a, (hipStream_t)stream) ? moe_fail(MOE_EHIP, "shared expert backward launch failed") : MOE_OK;
}

int64_t moe_adamw_workspace_bytes(const moe_adamw_tensor* t, int32_t n_tensors) {
  if (check_adamw(t, n_tensors)) return -1;
  return chunk_bytes(adamw_chunks(t, n_tensors)) + n_tensors * (int64_t)sizeof(AdamwDesc);
}

int moe_adamw_bind(const moe_adamw_tensor* t, int32_t n_tensors, void* workspace, int64_t workspace_bytes,
                   moe_adamw_plan* plan, void* stream) {
  if (const char* e = check_adamw(t, n_tensors)) return moe_fail(MOE_EINVAL, e);
  if (!plan) return moe_fail(MOE_EINVAL, "null plan");
  const int64_t n_chunks = adamw_chunks(t, n_tensors), need = moe_adamw_workspace_bytes(t, n_tensors);
  if (n_tensors > 0 && (!workspace || workspace_bytes < need)) return moe_fail(MOE_EINVAL, "workspace too small");
  if (off(workspace, 16)) return moe_fail(MOE_EINVAL, "workspace must be 16-byte aligned");
  try {
    struct Range {
      uintptr_t at, end;
      bool written;
    };
    std::vector<Range> spans{{(uintptr_t)workspace, (uintptr_t)workspace + (uintptr_t)need, true}};
    int n8 = 0;
    for (int i = 0; i < n_tensors; ++i) {
      const moe_adamw_tensor& a = t[i];
      if (a.n == 0) continue;
      const bool small = a.state_bits == 8;
      n8 += small;
      const int64_t blocks = (a.n + MOE_ADAMW_BLOCK - 1) / MOE_ADAMW_BLOCK, ss = small ? 1 : 4;
      const struct { const void* p; int64_t n; } out[] = {{a.param, a.n * elem(a.param_dtype)}, {a.copy, a.n * 2},
                                                          {a.m, a.n * ss}, {a.v, a.n * ss}, {a.m_scale, blocks},
                                                          {a.v_scale, blocks}, {a.m_values, a.n * 2},
                                                          {a.root_values, a.n * 2}};
      for (const auto& o : out)
        if (o.p) spans.push_back({(uintptr_t)o.p, (uintptr_t)o.p + (uintptr_t)o.n, true});
      spans.push_back({(uintptr_t)a.grad, (uintptr_t)a.grad + (uintptr_t)(a.n * elem(a.grad_dtype)), false});
    }
    std::sort(spans.begin(), spans.end(), [](const Range& a, const Range& b) { return a.at < b.at; });
    uintptr_t any = 0, written = 0;  // ends of what was seen so far, and of what of it the step writes
    for (const Range& s : spans) {
      if (s.at < written || (s.written && s.at < any))
        return moe_fail(MOE_EINVAL, "a buffer that the step writes overlaps another (the same tensor twice?)");
      any = std::max(any, s.end);
      if (s.written) written = std::max(written, s.end);
    }
    if (n_tensors > 0) {
      hipStreamCaptureStatus cap = hipStreamCaptureStatusNone;
      if (hipStreamIsCapturing((hipStream_t)stream, &cap) != hipSuccess) return moe_fail(MOE_EHIP, "stream query failed");
      if (cap != hipStreamCaptureStatusNone) return moe_fail(MOE_EINVAL, "a plan cannot be bound under capture");
      std::vector<char> host((size_t)need, 0);
      AdamwChunk* c = (AdamwChunk*)host.data();
      for (int i = 0; i < n_tensors; ++i)
        for (int64_t k = 0; k < (t[i].n + ADAMW_CHUNK - 1) / ADAMW_CHUNK; ++k) *c++ = {i, (int32_t)k};
      std::copy(t, t + n_tensors, (AdamwDesc*)(host.data() + chunk_bytes(n_chunks)));
      if (hipMemcpyAsync(workspace, host.data(), (size_t)need, hipMemcpyHostToDevice, (hipStream_t)stream) != hipSuccess ||
          hipStreamSynchronize((hipStream_t)stream) != hipSuccess)
        return moe_fail(MOE_EHIP, "plan copy failed");
    }
    plan->table = workspace;
    plan->n_chunks = n_chunks;
    plan->n_tensors = n_tensors;
    plan->states8 = n8;
  } catch (const std::exception&) {
    return moe_fail(MOE_EINVAL, "out of host memory");
  }
  return MOE_OK;
}

int moe_adamw_step(const moe_adamw_plan* plan, const moe_adamw_cfg* cfg, void* stream) {
  if (const char* e = check_plan(plan)) return moe_fail(MOE_EINVAL, e);
  if (!cfg) return moe_fail(MOE_EINVAL, "null cfg");
  // the kernel's reciprocal of a divisor below 2^-126 is not finite, and makes NaN of an update of 0
  const float lr = (float)cfg->lr, eps = (float)cfg->eps;
  if (!(lr >= 0) || !std::isfinite(lr) || !(cfg->eps == 0 || eps >= FLT_MIN) || !std::isfinite(eps))
    return moe_fail(MOE_EINVAL, "lr and eps must be finite in fp32 and not negative, eps 0 or at least 2^-126");
  if (!(cfg->beta1 >= 0 && cfg->beta1 < 1) || !(cfg->beta2 >= 0 && cfg->beta2 < 1))
    return moe_fail(MOE_EINVAL, "betas must be in [0, 1)");
  if (cfg->step < 1 && !cfg->step_dev) return moe_fail(MOE_EINVAL, "step must be >= 1");
  if (off(cfg->grad_scale, 4) || off(cfg->lr_dev, 4) || off(cfg->step_dev, 8))
    return moe_fail(MOE_EINVAL, "a device number must be aligned to its size");
  AdamwStep a = adamw_of(plan);
  a.lr = lr;
  a.beta1 = (float)cfg->beta1;
  a.beta2 = (float)cfg->beta2;
  a.one1 = (float)(1.0 - cfg->beta1);
  a.one2 = (float)(1.0 - cfg->beta2);
  a.eps = eps;
  a.log_beta1 = std::log(cfg->beta1);
  a.log_beta2 = std::log(cfg->beta2);
  const double t = (double)std::max<int64_t>(cfg->step, 1);
  a.inv_c1 = (float)(1.0 / -std::expm1(t * a.log_beta1));
  a.inv_root_c2 = (float)(1.0 / std::sqrt(-std::expm1(t * a.log_beta2)));
  a.grad_scale = cfg->grad_scale;
  a.lr_dev = cfg->lr_dev;
  a.step_dev = cfg->step_dev;
  return launch_adamw(a, plan->n_chunks, false, (hipStream_t)stream) ? moe_fail(MOE_EHIP, "AdamW launch failed") : MOE_OK;
}

int moe_adamw_read_states(const moe_adamw_plan* plan, void* stream) {
  if (const char* e = check_plan(plan)) return moe_fail(MOE_EINVAL, e);
  if (plan->states8 == 0) return MOE_OK;
  return launch_adamw(adamw_of(plan), plan->n_chunks, true, (hipStream_t)stream)
             ? moe_fail(MOE_EHIP, "AdamW state launch failed")
             : MOE_OK;
}

}  // extern "C"
