// C ABI of the operators that complete a block's training step: the norms around a block, the router's losses, the gradient
// norm (declarations and contracts in include/moe_overlap.h).  Host side only: argument checks and launches on the caller's stream.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <cfloat>
#include <cmath>
#include <exception>
#include <vector>

#include "../../include/moe_overlap.h"
#include "checks.h"
#include "launch.h"

namespace {

const char* check_residual(const moe_residual_norm_shape* s) {
  if (!s) return "null shape";
  if (s->rows < 0 || s->rows > (1ll << 40)) return "rows must be in [0, 2^40]";
  if (s->d < 1 || s->d > MOE_NORM_MAX_D) return "d must be in [1, MOE_NORM_MAX_D]";
  if (!is_dtype(s->dtype) || !is_dtype(s->param_dtype)) return "dtype must be MOE_BF16 or MOE_F32";
  for (const int32_t kind : {s->post, s->pre})
    if (kind != MOE_NORM_NONE && kind != MOE_NORM_LAYER && kind != MOE_NORM_RMS)
      return "post and pre must be MOE_NORM_NONE, MOE_NORM_LAYER or MOE_NORM_RMS";
  if (!(s->eps > 0.f) || !std::isfinite(s->eps)) return "eps must be positive and finite";
  if (!std::isfinite(s->residual_scale)) return "residual_scale must be finite";
  return nullptr;
}

const char* check_params(const moe_residual_norm_shape* s, const moe_residual_norm_params* p) {
  if (!p) return "null parameters";
  if (s->post == MOE_NORM_NONE && (p->post_weight || p->post_bias)) return "parameters of a norm that is none";
  if (s->pre == MOE_NORM_NONE && (p->pre_weight || p->pre_bias)) return "parameters of a norm that is none";
  for (const void* q : {p->post_weight, p->post_bias, p->gate, p->pre_weight, p->pre_bias})
    if (off(q, elem(s->param_dtype))) return "a tensor must be aligned to its elements";
  return off(p->row_gate, 4) ? "a tensor must be aligned to its elements" : nullptr;
}

const char* check_strides(const moe_residual_norm_shape* s, std::initializer_list<int64_t> strides) {
  for (const int64_t stride : strides)
    if (stride != 0 && (stride < s->d || stride > (1ll << 46) / std::max<int64_t>(s->rows, 1)))
      return "a row stride must be 0 or at least d, and rows x stride at most 2^46";
  return nullptr;
}

// All rows of a matrix, one every `stride` elements
Span rows_of(const moe_residual_norm_shape* s, const void* p, int64_t stride) {
  const int64_t es = elem(s->dtype);
  return {p, ((s->rows - 1) * stride + s->d) * es, s->d * es, stride * es};
}

ResidualLaunch residual_of(const moe_residual_norm_shape* s, const moe_residual_norm_params* p) {
  ResidualLaunch a{};
  a.rows = s->rows;
  a.d = s->d;
  a.dtype = s->dtype;
  a.param_dtype = s->param_dtype;
  a.post = s->post;
  a.pre = s->pre;
  a.eps = s->eps;
  a.rho = s->residual_scale;
  a.p = *p;
  return a;
}

const char* check_router(const moe_router_shape* s) {
  if (!s) return "null shape";
  if (s->experts < 1 || s->experts > 1024) return "experts must be in [1, 1024]";
  if (s->top_k < 1 || s->top_k > std::min(s->experts, 16)) return "top_k must be in [1, min(G, 16)]";
  if (s->tokens < 0 || s->tokens > 1 << 30 || s->tokens * s->top_k >= 1ll << 31)
    return "tokens must be in [0, 2^30], tokens x top_k below 2^31";
  if (s->sequences < 1 || s->sequences > 1 << 30 || (int64_t)s->sequences * s->experts >= (1ll << 31))
    return "sequences must be in [1, 2^30], sequences x experts below 2^31";
  if (!is_dtype(s->dtype)) return "dtype must be MOE_BF16 or MOE_F32";
  if (!std::isfinite(s->balance) || !std::isfinite(s->z)) return "balance and z must be finite";
  return nullptr;
}

RouterLaunch router_of(const moe_router_shape* s) {
  RouterLaunch a{};
  a.tokens = s->tokens;
  a.experts = s->experts;
  a.top_k = s->top_k;
  a.sequences = s->sequences;
  a.dtype = s->dtype;
  a.balance = s->balance;
  a.z = s->z;
  return a;
}

const char* check_grads(const moe_grad_tensor* t, int32_t n) {
  if (n < 0 || (n > 0 && !t)) return "null tensors";
  int64_t chunks = 0;
  for (int i = 0; i < n; ++i) {
    const moe_grad_tensor& a = t[i];
    if (a.n < 0 || a.n > (1ll << 40)) return "elements must be in [0, 2^40]";
    if (!is_dtype(a.grad_dtype) || (a.out && !is_dtype(a.out_dtype))) return "dtype must be MOE_BF16 or MOE_F32";
    if (a.n == 0) continue;
    if (!a.grad) return "null pointer";
    if (off(a.grad, elem(a.grad_dtype)) || (a.out && off(a.out, elem(a.out_dtype))))
      return "a tensor must be aligned to its elements";
    chunks += (a.n + GRAD_CHUNK - 1) / GRAD_CHUNK;
  }
  // 256 threads each, under 2^32 in a launch
  return chunks >= 1 << 24 ? "too many elements for one plan" : nullptr;
}

int64_t grad_chunks(const moe_grad_tensor* t, int32_t n) {
  int64_t c = 0;
  for (int i = 0; i < n; ++i) c += (t[i].n + GRAD_CHUNK - 1) / GRAD_CHUNK;
  return c;
}

int64_t table_bytes(int64_t n_chunks) { return n_chunks * (int64_t)sizeof(GradChunk); }

const char* check_grad_plan(const moe_grad_plan* p) {
  if (!p || p->n_chunks < 0 || p->n_chunks >= 1 << 24 || !p->table) return "plan not bound";
  return nullptr;
}

GradLaunch grad_of(const moe_grad_plan* p) {
  GradLaunch a{};
  a.chunks = (const GradChunk*)p->table;
  a.n_chunks = p->n_chunks;
  a.counters = (uint32_t*)((char*)p->table + table_bytes(p->n_chunks));
  a.partial = (double*)(a.counters + grad_counter_words(p->n_chunks));
  return a;
}

int64_t plan_bytes(int64_t n_chunks) {
  return table_bytes(n_chunks) + 4 * grad_counter_words(n_chunks) + 8 * grad_partial_doubles(n_chunks);
}

// A device number of a call inside the plan's workspace, whose records hold addresses
bool in_plan(const moe_grad_plan* p, const void* number) {
  return meet(Span{p->table, plan_bytes(p->n_chunks)}, Span{number, 4});
}

}  // namespace

extern "C" {

int moe_residual_norm(const moe_residual_norm_shape* s, const moe_residual_norm_params* p, const moe_residual_norm_args* b,
                      void* stream) {
  if (const char* e = check_residual(s)) return moe_fail(MOE_EINVAL, e);
  if (const char* e = check_params(s, p)) return moe_fail(MOE_EINVAL, e);
  if (!b) return moe_fail(MOE_EINVAL, "null arguments");
  if (const char* e = check_strides(s, {b->x_stride, b->h_stride, b->s_stride, b->n_stride})) return moe_fail(MOE_EINVAL, e);
  if (!b->n != (s->pre == MOE_NORM_NONE) && (b->n || s->rows > 0))
    return moe_fail(MOE_EINVAL, "n is given with a norm in front of the next block, and only then");
  if (s->rows == 0) return MOE_OK;
  if (!b->x || !b->h || !b->s) return moe_fail(MOE_EINVAL, "null pointer");
  for (const void* q : {b->x, b->h, (const void*)b->s, (const void*)b->n})
    if (off(q, elem(s->dtype))) return moe_fail(MOE_EINVAL, "a tensor must be aligned to its elements");
  if (off(b->stats, 16)) return moe_fail(MOE_EINVAL, "stats must be 16-byte aligned");
  ResidualLaunch a = residual_of(s, p);
  a.x_stride = b->x_stride ? b->x_stride : s->d;
  a.h_stride = b->h_stride ? b->h_stride : s->d;
  a.s_stride = b->s_stride ? b->s_stride : s->d;
  a.n_stride = b->n_stride ? b->n_stride : s->d;
  const int64_t np = s->d * elem(s->param_dtype);
  const Span out[] = {rows_of(s, b->s, a.s_stride), rows_of(s, b->n, a.n_stride), {b->stats, 16 * s->rows}},
             in[] = {rows_of(s, b->x, a.x_stride), rows_of(s, b->h, a.h_stride), {p->post_weight, np}, {p->post_bias, np},
                     {p->gate, np}, {p->pre_weight, np}, {p->pre_bias, np}, {p->row_gate, 4 * s->rows}};
  const int64_t os[] = {a.s_stride, a.n_stride, 0}, is[] = {a.x_stride, a.h_stride};
  if (overlaps(out, in, [&](int o, int i) { return o < 2 && i < 2 && os[o] == is[i] && !b->stats; }))
    return moe_fail(MOE_EINVAL, "an output overlaps an input or another output");
  a.x = b->x;
  a.h = b->h;
  a.s = b->s;
  a.n = b->n;
  a.stats = b->stats;
  return launch_residual(a, (hipStream_t)stream) ? moe_fail(MOE_EHIP, "residual norm launch failed") : MOE_OK;
}

int64_t moe_residual_norm_workspace_bytes(const moe_residual_norm_shape* s) {
  return check_residual(s) ? -1 : 4 * residual_partial_floats(s->rows, s->d, s->dtype);
}

int moe_residual_norm_backward(const moe_residual_norm_shape* s, const moe_residual_norm_params* p,
                               const moe_residual_norm_bwd_args* b, void* workspace, int64_t workspace_bytes, void* stream) {
  if (const char* e = check_residual(s)) return moe_fail(MOE_EINVAL, e);
  if (const char* e = check_params(s, p)) return moe_fail(MOE_EINVAL, e);
  if (!b) return moe_fail(MOE_EINVAL, "null arguments");
  if (const char* e = check_strides(s, {b->x_stride, b->h_stride, b->ds_stride, b->dn_stride, b->dx_stride, b->dh_stride}))
    return moe_fail(MOE_EINVAL, e);
  if (!b->dn != (s->pre == MOE_NORM_NONE) && (b->dn || s->rows > 0))
    return moe_fail(MOE_EINVAL, "dn is given with a norm in front of the next block, and only then");
  if ((s->post == MOE_NORM_NONE && (b->d_post_weight || b->d_post_bias)) ||
      (s->pre == MOE_NORM_NONE && (b->d_pre_weight || b->d_pre_bias)))
    return moe_fail(MOE_EINVAL, "gradients of a norm that is none");
  if (s->rows > 0 && (!b->x || !b->h || !b->stats || !b->dx || !b->dh || (!b->ds && !b->dn)))
    return moe_fail(MOE_EINVAL, "null pointer");
  for (const void* q : {b->ds, b->dn, b->x, b->h, (const void*)b->dx, (const void*)b->dh})
    if (off(q, elem(s->dtype))) return moe_fail(MOE_EINVAL, "a tensor must be aligned to its elements");
  for (const void* q : {b->d_post_weight, b->d_post_bias, b->d_gate, b->d_pre_weight, b->d_pre_bias})
    if (off(q, elem(s->param_dtype))) return moe_fail(MOE_EINVAL, "a tensor must be aligned to its elements");
  if (off(b->d_row_gate, 4)) return moe_fail(MOE_EINVAL, "a tensor must be aligned to its elements");
  if (off(b->stats, 16) || off(workspace, 16)) return moe_fail(MOE_EINVAL, "stats and the workspace must be 16-byte aligned");
  const bool params = b->d_post_weight || b->d_post_bias || b->d_gate || b->d_pre_weight || b->d_pre_bias;
  const int64_t need = moe_residual_norm_workspace_bytes(s);
  if (params && need > 0 && (!workspace || workspace_bytes < need)) return moe_fail(MOE_EINVAL, "workspace too small");
  ResidualLaunch a = residual_of(s, p);
  a.x_stride = b->x_stride ? b->x_stride : s->d;
  a.h_stride = b->h_stride ? b->h_stride : s->d;
  a.ds_stride = b->ds_stride ? b->ds_stride : s->d;
  a.dn_stride = b->dn_stride ? b->dn_stride : s->d;
  a.dx_stride = b->dx_stride ? b->dx_stride : s->d;
  a.dh_stride = b->dh_stride ? b->dh_stride : s->d;
  const int64_t np = s->d * elem(s->param_dtype), live = s->rows > 0;
  auto matrix = [&](const void* q, int64_t stride) { return live ? rows_of(s, q, stride) : Span{nullptr, 0}; };
  const Span out[] = {matrix(b->dx, a.dx_stride), matrix(b->dh, a.dh_stride), {b->d_post_weight, np}, {b->d_post_bias, np},
                      {b->d_gate, np}, {b->d_pre_weight, np}, {b->d_pre_bias, np}, {b->d_row_gate, 4 * s->rows},
                      {params ? workspace : nullptr, need}},
             in[] = {matrix(b->ds, a.ds_stride), matrix(b->dn, a.dn_stride), matrix(b->x, a.x_stride), matrix(b->h, a.h_stride),
                     {p->post_weight, np}, {p->post_bias, np}, {p->gate, np}, {p->pre_weight, np}, {p->pre_bias, np},
                     {p->row_gate, 4 * s->rows}, {b->stats, 16 * s->rows}};
  const int64_t os[] = {a.dx_stride, a.dh_stride}, is[] = {a.ds_stride, a.dn_stride};
  if (overlaps(out, in, [&](int o, int i) { return o < 2 && i < 2 && os[o] == is[i]; }))
    return moe_fail(MOE_EINVAL, "an output overlaps an input or another output");
  a.backward = true;
  a.ds = b->ds;
  a.dn = b->dn;
  a.x = b->x;
  a.h = b->h;
  a.stats = (float*)b->stats;
  a.dx = b->dx;
  a.dh = b->dh;
  a.d_post_weight = b->d_post_weight;
  a.d_post_bias = b->d_post_bias;
  a.d_gate = b->d_gate;
  a.d_pre_weight = b->d_pre_weight;
  a.d_pre_bias = b->d_pre_bias;
  a.d_row_gate = b->d_row_gate;
  a.partial = params ? (float*)workspace : nullptr;
  return launch_residual(a, (hipStream_t)stream) ? moe_fail(MOE_EHIP, "residual norm backward launch failed") : MOE_OK;
}

int64_t moe_router_loss_workspace_bytes(const moe_router_shape* s) {
  return check_router(s) ? -1 : router_workspace_bytes(s->tokens, s->experts, s->sequences);
}

int moe_router_loss(const moe_router_shape* s, const float* logits, const int32_t* topk_idx, const int32_t* spans,
                    int32_t* counts, int32_t* means, float* losses, void* workspace, int64_t workspace_bytes, void* stream) {
  if (const char* e = check_router(s)) return moe_fail(MOE_EINVAL, e);
  if (!counts || !means || !losses || (s->tokens > 0 && (!logits || !topk_idx))) return moe_fail(MOE_EINVAL, "null pointer");
  if (!spans && s->tokens % s->sequences != 0)
    return moe_fail(MOE_EINVAL, "without spans the tokens must be a multiple of the sequences");
  for (const void* q : {(const void*)logits, (const void*)topk_idx, (const void*)spans, (const void*)counts, (const void*)means,
                        (const void*)losses})
    if (off(q, 4)) return moe_fail(MOE_EINVAL, "a tensor must be aligned to its elements");
  const int64_t need = moe_router_loss_workspace_bytes(s);
  if (!workspace || workspace_bytes < need) return moe_fail(MOE_EINVAL, "workspace too small");
  if (off(workspace, 16)) return moe_fail(MOE_EINVAL, "workspace must be 16-byte aligned");
  const int64_t cells = (int64_t)s->sequences * s->experts;
  const Span out[] = {{counts, 4 * cells}, {means, 8}, {losses, 12}, {workspace, need}},
             in[] = {{logits, 4 * s->tokens * s->experts}, {topk_idx, 4 * s->tokens * s->top_k}, {spans, 8ll * s->sequences}};
  if (overlaps(out, in, [](int, int) { return false; }))
    return moe_fail(MOE_EINVAL, "an output overlaps an input or another output");
  RouterLaunch a = router_of(s);
  a.logits = logits;
  a.topk_idx = topk_idx;
  a.spans = spans;
  a.counts = counts;
  a.means = means;
  a.losses = losses;
  a.workspace = workspace;
  return launch_router_loss(a, (hipStream_t)stream) ? moe_fail(MOE_EHIP, "router loss launch failed") : MOE_OK;
}

int moe_router_backward(const moe_router_shape* s, const float* logits, const int32_t* topk_idx, const int32_t* spans,
                        const int32_t* counts, const int32_t* means, const float* d_loss, const float* d_weights,
                        void* dlogits, void* stream) {
  if (const char* e = check_router(s)) return moe_fail(MOE_EINVAL, e);
  if (!spans && s->tokens % s->sequences != 0)
    return moe_fail(MOE_EINVAL, "without spans the tokens must be a multiple of the sequences");
  if (s->tokens == 0) return MOE_OK;
  if (!logits || !topk_idx || !counts || !means || !dlogits) return moe_fail(MOE_EINVAL, "null pointer");
  for (const void* q : {(const void*)logits, (const void*)topk_idx, (const void*)spans, (const void*)counts, (const void*)means,
                        (const void*)d_loss, (const void*)d_weights})
    if (off(q, 4)) return moe_fail(MOE_EINVAL, "a tensor must be aligned to its elements");
  if (off(dlogits, elem(s->dtype))) return moe_fail(MOE_EINVAL, "a tensor must be aligned to its elements");
  const Span out[] = {{dlogits, s->tokens * s->experts * elem(s->dtype)}},
             in[] = {{logits, 4 * s->tokens * s->experts}, {topk_idx, 4 * s->tokens * s->top_k}, {spans, 8ll * s->sequences},
                     {counts, 4ll * s->sequences * s->experts}, {means, 8}, {d_loss, 4}, {d_weights, 4 * s->tokens * s->top_k}};
  if (overlaps(out, in, [](int, int) { return false; }))
    return moe_fail(MOE_EINVAL, "an output overlaps an input or another output");
  RouterLaunch a = router_of(s);
  a.logits = logits;
  a.topk_idx = topk_idx;
  a.spans = spans;
  a.counts = (int32_t*)counts;
  a.means = (int32_t*)means;
  a.d_loss = d_loss;
  a.d_weights = d_weights;
  a.dlogits = dlogits;
  return launch_router_backward(a, (hipStream_t)stream) ? moe_fail(MOE_EHIP, "router backward launch failed") : MOE_OK;
}

int64_t moe_grad_workspace_bytes(const moe_grad_tensor* t, int32_t n_tensors) {
  if (check_grads(t, n_tensors)) return -1;
  return plan_bytes(grad_chunks(t, n_tensors));
}

int moe_grad_bind(const moe_grad_tensor* t, int32_t n_tensors, void* workspace, int64_t workspace_bytes, moe_grad_plan* plan,
                  void* stream) {
  if (const char* e = check_grads(t, n_tensors)) return moe_fail(MOE_EINVAL, e);
  if (!plan) return moe_fail(MOE_EINVAL, "null plan");
  const int64_t n_chunks = grad_chunks(t, n_tensors), need = moe_grad_workspace_bytes(t, n_tensors);
  if (!workspace || workspace_bytes < need) return moe_fail(MOE_EINVAL, "workspace too small");
  if (off(workspace, 16)) return moe_fail(MOE_EINVAL, "workspace must be 16-byte aligned");
  try {
    struct Range {
      uintptr_t at, end;
    };
    std::vector<Range> spans;
    spans.push_back({(uintptr_t)workspace, (uintptr_t)workspace + (uintptr_t)need});
    for (int i = 0; i < n_tensors; ++i) {
      if (t[i].n == 0) continue;
      const uintptr_t g = (uintptr_t)t[i].grad, o = (uintptr_t)t[i].out;
      spans.push_back({g, g + (uintptr_t)(t[i].n * elem(t[i].grad_dtype))});
      if (o) spans.push_back({o, o + (uintptr_t)(t[i].n * elem(t[i].out_dtype))});
    }
    std::sort(spans.begin(), spans.end(), [](const Range& a, const Range& b) { return a.at < b.at; });
    for (size_t i = 1; i < spans.size(); ++i)
      if (spans[i].at < spans[i - 1].end)
        return moe_fail(MOE_EINVAL, "a gradient or an output overlaps another (the same tensor twice?)");
    hipStreamCaptureStatus cap = hipStreamCaptureStatusNone;
    if (hipStreamIsCapturing((hipStream_t)stream, &cap) != hipSuccess) return moe_fail(MOE_EHIP, "stream query failed");
    if (cap != hipStreamCaptureStatusNone) return moe_fail(MOE_EINVAL, "a plan cannot be bound under capture");
    const size_t head = (size_t)(table_bytes(n_chunks) + 4 * grad_counter_words(n_chunks));  // the records, and zeros
    std::vector<GradChunk> table;
    table.reserve(head / sizeof(GradChunk) + 1);
    for (int i = 0; i < n_tensors; ++i)
      for (int64_t at = 0; at < t[i].n; at += GRAD_CHUNK)
        table.push_back({(const char*)t[i].grad + at * elem(t[i].grad_dtype),
                         t[i].out ? (char*)t[i].out + at * elem(t[i].out_dtype) : nullptr,
                         (int32_t)std::min<int64_t>(GRAD_CHUNK, t[i].n - at), t[i].grad_dtype == MOE_BF16,
                         t[i].out && t[i].out_dtype == MOE_BF16, 0});
    table.resize(head / sizeof(GradChunk) + 1, GradChunk{});
    if (hipMemcpyAsync(workspace, table.data(), head, hipMemcpyHostToDevice, (hipStream_t)stream) !=
            hipSuccess ||
        hipStreamSynchronize((hipStream_t)stream) != hipSuccess)
      return moe_fail(MOE_EHIP, "plan copy failed");
    plan->table = workspace;
    plan->n_chunks = n_chunks;
    plan->n_tensors = n_tensors;
    plan->reserved = 0;
  } catch (const std::exception&) {
    return moe_fail(MOE_EINVAL, "out of host memory");
  }
  return MOE_OK;
}

int moe_grad_norm(const moe_grad_plan* plan, double max_norm, double factor, float* norm, float* scale, void* stream) {
  if (const char* e = check_grad_plan(plan)) return moe_fail(MOE_EINVAL, e);
  if (!(max_norm > 0) || !((float)factor > 0) || !std::isfinite((float)factor) || (!std::isinf(max_norm) && std::isinf((float)max_norm)))
    return moe_fail(MOE_EINVAL, "max_norm and factor must be positive, factor finite, both in fp32's range");
  if (!norm || !scale) return moe_fail(MOE_EINVAL, "null pointer");
  if (off(norm, 4) || off(scale, 4)) return moe_fail(MOE_EINVAL, "a device number must be aligned to its size");
  if (norm == scale) return moe_fail(MOE_EINVAL, "an output overlaps another output");
  if (in_plan(plan, norm) || in_plan(plan, scale)) return moe_fail(MOE_EINVAL, "an output overlaps the plan's workspace");
  GradLaunch a = grad_of(plan);
  a.max_norm = max_norm;
  a.factor = factor;
  a.norm = norm;
  a.scale = scale;
  return launch_grad_norm(a, (hipStream_t)stream) ? moe_fail(MOE_EHIP, "gradient norm launch failed") : MOE_OK;
}

int moe_grad_clip(const moe_grad_plan* plan, const float* scale, void* stream) {
  if (const char* e = check_grad_plan(plan)) return moe_fail(MOE_EINVAL, e);
  if (!scale) return moe_fail(MOE_EINVAL, "null pointer");
  if (off(scale, 4)) return moe_fail(MOE_EINVAL, "a device number must be aligned to its size");
  if (in_plan(plan, scale)) return moe_fail(MOE_EINVAL, "scale overlaps the plan's workspace");
  GradLaunch a = grad_of(plan);
  a.scale = (float*)scale;
  return launch_grad_clip(a, (hipStream_t)stream) ? moe_fail(MOE_EHIP, "gradient clip launch failed") : MOE_OK;
}

}  // extern "C"
