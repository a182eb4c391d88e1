// C ABI of the one-kind paged caches: argument checks and launches.
// See include/oscar.h for the contract of every entry point.

#include <algorithm>
#include <cmath>

#include "oscar_ctx.h"
#include "oscar_paged.h"

using namespace oscar;

namespace {

bool aligned(const void* p, unsigned bytes) { return (reinterpret_cast<uintptr_t>(p) & (bytes - 1)) == 0; }

bool valid_pages(const void* pool, int64_t num_pages, const int32_t* table, int32_t max_pages) {
  return pool != nullptr && aligned(pool, 16) && num_pages > 0 && num_pages <= INT32_MAX && table != nullptr &&
         aligned(table, 4) && max_pages > 0 && max_pages <= INT32_MAX / OSCAR_PAGE_TOKENS;
}

bool valid_bf16(const oscar_bf16_cache_view* v) {
  return valid_pages(v->k_pages, v->num_pages, v->page_table, v->max_pages_per_req) && v->v_pages != nullptr &&
         aligned(v->v_pages, 16);
}

bool valid_int4(const oscar_int4_cache_view* v) {
  return valid_pages(v->pages, v->num_pages, v->page_table, v->max_pages_per_req);
}

template <typename View>
PageRefs pages_of(const View* v) {
  PageRefs p;
  p.table = v->page_table;
  p.num_pages = v->num_pages;
  p.max_pages = v->max_pages_per_req;
  p.batch = v->batch;
  return p;
}

// Elements from one token to the next: 0 selects packed rows; false for a bad stride.
bool stride_of(int64_t given, int heads, int64_t* out) {
  const int64_t row = (int64_t)heads * OSCAR_HEAD_DIM;
  *out = given == 0 ? row : given;
  return *out >= row && *out % 8 == 0 && *out <= (INT64_C(1) << 40);
}

// The tokens of a call: NULL cu_seqlens means one token per request.
oscar_status tokens_of(const int32_t* pos, const int32_t* cu, int32_t n_tokens, int32_t max_tokens, int32_t batch,
                       TokenRefs* t) {
  if (pos == nullptr || n_tokens < 0) return OSCAR_ERR_INVALID_ARG;
  if (cu == nullptr) {
    if (n_tokens != batch) return OSCAR_ERR_INVALID_ARG;
  } else if (max_tokens <= 0 || max_tokens > (1 << 28)) {
    return OSCAR_ERR_INVALID_ARG;
  }
  if (batch > 65535) return OSCAR_ERR_UNSUPPORTED;
  t->pos = pos;
  t->cu = cu;
  t->n_tokens = n_tokens;
  t->max_tokens = cu == nullptr ? 1 : std::min(max_tokens, std::max(n_tokens, 1));
  return OSCAR_OK;
}

oscar_status rope_launch(const oscar_ctx* ctx, const oscar_rope_append_args* args, int32_t batch, RopeLaunch* a) {
  const oscar_status st = tokens_of(args->pos, args->cu_seqlens, args->n_tokens, args->max_tokens_per_req, batch, &a->tok);
  if (st != OSCAR_OK) return st;
  if (args->k == nullptr || args->v == nullptr || (args->q == nullptr) != (args->q_out == nullptr))
    return OSCAR_ERR_INVALID_ARG;
  for (const void* p : {args->q, static_cast<const void*>(args->q_out), args->k, args->v,
                        static_cast<const void*>(args->rope)})
    if (!aligned(p, 16)) return OSCAR_ERR_INVALID_ARG;
  if (!stride_of(args->q_stride, args->q ? ctx->cfg.num_q_heads : 0, &a->q_stride) ||
      !stride_of(args->q_out_stride, args->q ? ctx->cfg.num_q_heads : 0, &a->qo_stride) ||
      !stride_of(args->k_stride, ctx->cfg.num_kv_heads, &a->k_stride) ||
      !stride_of(args->v_stride, ctx->cfg.num_kv_heads, &a->v_stride))
    return OSCAR_ERR_INVALID_ARG;
  if (args->interleaved != 0 && args->interleaved != 1) return OSCAR_ERR_INVALID_ARG;
  if (args->rotary_dim != 0 && args->rotary_dim != 64 && args->rotary_dim != 128)
    return args->rotary_dim < 0 || args->rotary_dim > 128 ? OSCAR_ERR_INVALID_ARG : OSCAR_ERR_UNSUPPORTED;
  if (args->rotary_dim != 0 && (args->rope == nullptr || args->rope_positions <= 0)) return OSCAR_ERR_INVALID_ARG;
  a->q = static_cast<const uint16_t*>(args->q);
  a->q_out = static_cast<uint16_t*>(args->q_out);
  a->k = static_cast<const uint16_t*>(args->k);
  a->v = static_cast<const uint16_t*>(args->v);
  a->rope = args->rope;
  a->rope_positions = args->rope_positions;
  a->rotary = args->rotary_dim;
  a->interleaved = args->interleaved;
  a->Hq = args->q ? ctx->cfg.num_q_heads : 0;
  a->Hkv = ctx->cfg.num_kv_heads;
  a->num_sms = ctx->num_sms;
  a->err = ctx->d_err;
  return OSCAR_OK;
}

// Keys one query may see, at most (the length of a work item's share follows from it).
int64_t max_visible(int32_t max_ctx, int32_t window, int32_t sinks) {
  return window < 0 ? max_ctx : std::min<int64_t>(max_ctx, (int64_t)window + sinks);
}

// Chunks and prompts over BF16 pages take the tensor-core kernel, from two tokens a request on: its tiles read the
// keys once for 128 rows, the split kernel for each token.  1 request of 32:8 heads, tensor cores against split: 2
// tokens at 300 held 11.7 us, 8.3 (the most that it loses), at 4096 14.0, 15.4; 32 tokens at 4096 17.9, 68.3; 64
// requests x 2 tokens at 4096 202, 321.
bool on_tensor_cores(const WindowLaunch& a, bool int4) { return !int4 && a.tok.max_tokens > 1; }

oscar_status window_launch(const oscar_ctx* ctx, const oscar_window_args* args, int32_t batch, bool int4, void* ws,
                           size_t ws_bytes, WindowLaunch* a) {
  const oscar_status st = tokens_of(args->pos, args->cu_seqlens, args->n_tokens, args->max_tokens_per_req, batch, &a->tok);
  if (st != OSCAR_OK) return st;
  if (args->q == nullptr || args->out == nullptr || args->ctx_len == nullptr || !aligned(args->q, 16) ||
      !aligned(args->out, 16) || args->max_ctx_len < 0 || args->sinks < 0 || std::isnan(args->sm_scale) ||
      std::isinf(args->sm_scale) || !stride_of(args->q_stride, ctx->cfg.num_q_heads, &a->q_stride))
    return OSCAR_ERR_INVALID_ARG;
  a->q = static_cast<const uint16_t*>(args->q);
  a->out = static_cast<uint16_t*>(args->out);
  a->ctx_len = args->ctx_len;
  a->window = args->window < 0 ? -1 : args->window;
  a->sinks = args->sinks;
  a->sm_scale = args->sm_scale > 0.f ? args->sm_scale : 1.0f / std::sqrt(128.0f);
  a->Hq = ctx->cfg.num_q_heads;
  a->Hkv = ctx->cfg.num_kv_heads;
  a->num_sms = ctx->num_sms;
  a->err = ctx->d_err;
  const int64_t keys = max_visible(args->max_ctx_len, args->window, args->sinks);
  a->plan = on_tensor_cores(*a, int4)
                ? plan_window_tc(batch, a->tok.max_tokens, a->Hq, a->Hkv, keys, ctx->num_sms)
                : plan_window(int4, args->n_tokens, a->Hq, a->Hkv, keys, ctx->num_sms);
  if (ws == nullptr || !aligned(ws, 256) || ws_bytes < oscar_window_workspace_bytes(ctx)) return OSCAR_ERR_WORKSPACE;
  a->workspace = static_cast<uint8_t*>(ws);
  if ((int64_t)args->n_tokens * a->Hkv > INT32_MAX) return OSCAR_ERR_UNSUPPORTED;
  return OSCAR_OK;
}

oscar_status status_of(cudaError_t e) { return e == cudaSuccess ? OSCAR_OK : OSCAR_ERR_CUDA; }

}  // namespace

extern "C" {

oscar_status oscar_rope_table(oscar_ctx* ctx, float* table, int32_t n_positions, int32_t rotary_dim, double theta,
                              void* stream) {
  if (ctx == nullptr || table == nullptr || !aligned(table, 16) || n_positions < 0 || !(theta > 0.0) ||
      !std::isfinite(theta))
    return OSCAR_ERR_INVALID_ARG;
  if (rotary_dim != 64 && rotary_dim != 128)
    return rotary_dim <= 0 || rotary_dim > 128 ? OSCAR_ERR_INVALID_ARG : OSCAR_ERR_UNSUPPORTED;
  if (n_positions == 0) return OSCAR_OK;
  DeviceGuard guard(ctx->cfg.device);
  return status_of(launch_rope_table(table, n_positions, rotary_dim, theta, static_cast<cudaStream_t>(stream)));
}

oscar_status oscar_rope_append_bf16(oscar_ctx* ctx, const oscar_bf16_cache_view* view,
                                    const oscar_rope_append_args* args, void* stream) {
  if (ctx == nullptr || view == nullptr || args == nullptr || view->batch < 0) return OSCAR_ERR_INVALID_ARG;
  if (view->batch == 0) return OSCAR_OK;
  if (!valid_bf16(view)) return OSCAR_ERR_INVALID_ARG;
  RopeLaunch a;
  const oscar_status st = rope_launch(ctx, args, view->batch, &a);
  if (st != OSCAR_OK) return st;
  if (args->n_tokens == 0) return OSCAR_OK;
  a.pages = pages_of(view);
  a.k_pages = static_cast<uint16_t*>(const_cast<void*>(view->k_pages));
  a.v_pages = static_cast<uint16_t*>(const_cast<void*>(view->v_pages));
  DeviceGuard guard(ctx->cfg.device);
  return status_of(launch_rope_append_bf16(a, static_cast<cudaStream_t>(stream)));
}

oscar_status oscar_rope_append_int4(oscar_ctx* ctx, const oscar_int4_cache_view* view,
                                    const oscar_rope_append_args* args, void* stream) {
  if (ctx == nullptr || view == nullptr || args == nullptr || view->batch < 0) return OSCAR_ERR_INVALID_ARG;
  if (view->batch == 0) return OSCAR_OK;
  if (!valid_int4(view)) return OSCAR_ERR_INVALID_ARG;
  RopeLaunch a;
  const oscar_status st = rope_launch(ctx, args, view->batch, &a);
  if (st != OSCAR_OK) return st;
  if (args->n_tokens == 0) return OSCAR_OK;
  a.pages = pages_of(view);
  a.pages4 = static_cast<uint8_t*>(view->pages);
  DeviceGuard guard(ctx->cfg.device);
  return status_of(launch_rope_append_int4(a, static_cast<cudaStream_t>(stream)));
}

oscar_status oscar_int4_to_bf16(oscar_ctx* ctx, const oscar_int4_cache_view* from, const oscar_bf16_cache_view* to,
                                const int32_t* pos, const int32_t* count, int32_t max_count, void* stream) {
  if (ctx == nullptr || from == nullptr || to == nullptr || from->batch < 0 || from->batch != to->batch)
    return OSCAR_ERR_INVALID_ARG;
  if (from->batch == 0) return OSCAR_OK;
  if (!valid_int4(from) || !valid_bf16(to) || pos == nullptr || count == nullptr || max_count < 0)
    return OSCAR_ERR_INVALID_ARG;
  if (from->batch > 65535) return OSCAR_ERR_UNSUPPORTED;
  if (max_count == 0) return OSCAR_OK;
  Read4Launch a;
  a.from = pages_of(from);
  a.to = pages_of(to);
  a.pos = pos;
  a.count = count;
  a.max_count = max_count;
  a.Hkv = ctx->cfg.num_kv_heads;
  a.num_sms = ctx->num_sms;
  a.pages4 = static_cast<const uint8_t*>(from->pages);
  a.k_pages = static_cast<uint16_t*>(const_cast<void*>(to->k_pages));
  a.v_pages = static_cast<uint16_t*>(const_cast<void*>(to->v_pages));
  a.err = ctx->d_err;
  DeviceGuard guard(ctx->cfg.device);
  return status_of(launch_int4_to_bf16(a, static_cast<cudaStream_t>(stream)));
}

size_t oscar_window_workspace_bytes(const oscar_ctx* ctx) {
  if (ctx == nullptr) return 0;
  const int Hq = ctx->cfg.num_q_heads, Hkv = ctx->cfg.num_kv_heads;
  return std::max(plan_window(false, 1, Hq, Hkv, 0, ctx->num_sms).total, plan_window_tc(1, 1, Hq, Hkv, 0, ctx->num_sms).total);
}

oscar_status oscar_window_attention_bf16(oscar_ctx* ctx, const oscar_bf16_cache_view* view,
                                         const oscar_window_args* args, void* workspace, size_t workspace_bytes,
                                         void* stream) {
  if (ctx == nullptr || view == nullptr || args == nullptr || view->batch < 0) return OSCAR_ERR_INVALID_ARG;
  if (view->batch == 0) return OSCAR_OK;
  if (!valid_bf16(view)) return OSCAR_ERR_INVALID_ARG;
  WindowLaunch a;
  const oscar_status st = window_launch(ctx, args, view->batch, false, workspace, workspace_bytes, &a);
  if (st != OSCAR_OK) return st;
  if (args->n_tokens == 0) return OSCAR_OK;
  a.pages = pages_of(view);
  a.k_pages = static_cast<const uint16_t*>(view->k_pages);
  a.v_pages = static_cast<const uint16_t*>(view->v_pages);
  DeviceGuard guard(ctx->cfg.device);
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  return status_of(on_tensor_cores(a, false) ? launch_window_tc(a, s) : launch_window_split(a, s));
}

oscar_status oscar_window_attention_int4(oscar_ctx* ctx, const oscar_int4_cache_view* view,
                                         const oscar_window_args* args, void* workspace, size_t workspace_bytes,
                                         void* stream) {
  if (ctx == nullptr || view == nullptr || args == nullptr || view->batch < 0) return OSCAR_ERR_INVALID_ARG;
  if (view->batch == 0) return OSCAR_OK;
  if (!valid_int4(view)) return OSCAR_ERR_INVALID_ARG;
  WindowLaunch a;
  const oscar_status st = window_launch(ctx, args, view->batch, true, workspace, workspace_bytes, &a);
  if (st != OSCAR_OK) return st;
  if (args->n_tokens == 0) return OSCAR_OK;
  a.pages = pages_of(view);
  a.pages4 = static_cast<const uint8_t*>(view->pages);
  DeviceGuard guard(ctx->cfg.device);
  return status_of(launch_window_split(a, static_cast<cudaStream_t>(stream)));
}

}  // extern "C"
