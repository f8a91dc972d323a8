// fm_api_serve.cu — the extern "C" boundary of the norm and rotation, the
// paged cache and the attention over it: arguments are checked on the host,
// then kernels are enqueued on the caller's stream.
#include <cmath>
#include "fm_internal.h"

using namespace fm;

namespace {

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0; }
bool head_dim(int d) { return d == 64 || d == 128 || d == 256; }
fm_status from_cuda(cudaError_t e) { return e == cudaSuccess ? FM_OK : FM_ERR_CUDA; }

bool view_ok(const fm_view* v) {
  return v && v->ptr && aligned16(v->ptr) && v->sb % 8 == 0 && v->sh % 8 == 0 && v->sn % 8 == 0;
}
bool rows_ok(const fm_rows* v) { return v && v->ptr && aligned16(v->ptr) && v->st % 8 == 0 && v->sh % 8 == 0; }

fm_status check_qk(const fm_qk_problem* p, bool* empty) {
  if (!p || p->B < 0 || p->N < 0 || p->H_q <= 0 || p->H_kv <= 0) return FM_ERR_INVALID_ARG;
  if (!(p->eps >= 0.f) || !std::isfinite(p->eps) || !std::isfinite(p->rot_scale)) return FM_ERR_INVALID_ARG;
  if (!head_dim(p->d)) return FM_ERR_UNSUPPORTED;
  if (p->rot < 0 || p->rot > p->d) return FM_ERR_INVALID_ARG;
  if (p->rot % 16) return FM_ERR_UNSUPPORTED;
  // blocks of tokens are counted in 32 bits
  if ((int64_t)p->B * p->N > (1ll << 30)) return FM_ERR_UNSUPPORTED;
  *empty = p->B == 0 || p->N == 0;
  if (!*empty && p->rot > 0 && (!p->pos || !p->inv_freq)) return FM_ERR_INVALID_ARG;
  return FM_OK;
}

fm_status check_cache(const fm_kv_cache* c) {
  if (!c || c->n_pages < 0 || c->H_kv <= 0) return FM_ERR_INVALID_ARG;
  if (!head_dim(c->d)) return FM_ERR_UNSUPPORTED;
  if (c->page_size != 16 && c->page_size != 32 && c->page_size != 64 && c->page_size != 128) return FM_ERR_UNSUPPORTED;
  if ((c->k_exp == nullptr) != (c->v_exp == nullptr)) return FM_ERR_INVALID_ARG;
  if ((int64_t)c->n_pages * c->H_kv > INT32_MAX) return FM_ERR_UNSUPPORTED;
  if (c->H_kv > 65536) return FM_ERR_UNSUPPORTED;  // rows of a block, key tiles of a call are counted
  if (c->n_pages == 0) return FM_ERR_INVALID_ARG;
  if (!c->k || !c->v || !aligned16(c->k) || !aligned16(c->v) || !aligned16(c->k_exp) || !aligned16(c->v_exp))
    return FM_ERR_INVALID_ARG;
  return FM_OK;
}

fm_status check_table(const int32_t* table, int R, int width, int page) {
  if (R <= 0 || width <= 0 || !table) return FM_ERR_INVALID_ARG;
  if ((int64_t)width * page > (1 << 30)) return FM_ERR_UNSUPPORTED;
  return FM_OK;
}

fm_status check_batch(const fm_kv_cache* c, const fm_paged_batch* b, int T) {
  if (!b || T < 0 || !b->q_off || !b->kv_len) return FM_ERR_INVALID_ARG;
  if (T > (1 << 30)) return FM_ERR_UNSUPPORTED;
  return check_table(b->page_table, b->R, b->width, c->page_size);
}

}  // namespace

extern "C" {

fm_status fm_rope_freqs(int32_t rot, double base, int32_t kind, double factor, int64_t orig_len, double beta_fast,
                        double beta_slow, float* inv_freq, float* rot_scale) {
  if (rot < 2 || rot % 2 || !(base > 1.0) || !std::isfinite(base) || !(factor >= 1.0) || !std::isfinite(factor) ||
      kind < FM_ROPE_PLAIN || kind > FM_ROPE_YARN || !inv_freq || !rot_scale)
    return FM_ERR_INVALID_ARG;
  if (kind == FM_ROPE_NTK && rot == 2) return FM_ERR_INVALID_ARG;
  if (kind == FM_ROPE_NTK) base *= std::pow(factor, (double)rot / (rot - 2));
  double first = 0, last = 0, slow = 0;
  if (kind == FM_ROPE_YARN) {
    if (orig_len <= 0 || !(beta_slow > 0.0) || !(beta_fast > beta_slow) || !std::isfinite(beta_fast))
      return FM_ERR_INVALID_ARG;
    // the pair index whose angle makes `turns` turns within orig_len positions
    auto pair_of = [&](double turns) {
      return rot * std::log((double)orig_len / (turns * 2 * M_PI)) / (2 * std::log(base));
    };
    first = std::fmax(std::floor(pair_of(beta_fast)), 0.0);
    slow = pair_of(beta_slow);
    last = std::fmin(std::ceil(slow), rot - 1.0);
  }
  for (int i = 0; i < rot / 2; ++i) {
    const double f = std::pow(base, -2.0 * i / rot);
    double v = f;
    if (kind == FM_ROPE_LINEAR) v = f / factor;
    if (kind == FM_ROPE_YARN) {
      // (where even pair 0 is slow, last <= 0 = first leaves no room for the ramp)
      const double ramp = i > slow ? 1.0 : std::fmin(std::fmax((i - first) / std::fmax(last - first, 1e-3), 0.0), 1.0);
      v = f / factor * ramp + f * (1 - ramp);
    }
    inv_freq[i] = (float)v;
  }
  *rot_scale = kind == FM_ROPE_YARN ? (float)(0.1 * std::log(factor) + 1.0) : 1.f;
  return FM_OK;
}

fm_status fm_qk_norm_rope(const fm_qk_problem* p, const fm_view* q, const fm_view* k, const fm_view* v,
                          const fm_view* qo, const fm_view* ko, const fm_view* vo, void* stream) {
  bool empty = false;
  fm_status st = check_qk(p, &empty);
  if (st != FM_OK || empty) return st;
  if (!view_ok(q) || !view_ok(k) || !view_ok(qo) || !view_ok(ko) || (v == nullptr) != (vo == nullptr))
    return FM_ERR_INVALID_ARG;
  if (v && (!view_ok(v) || !view_ok(vo))) return FM_ERR_INVALID_ARG;
  return from_cuda(launch_qk_fwd(*p, q, k, v, qo, ko, vo, static_cast<cudaStream_t>(stream)));
}

size_t fm_qk_norm_rope_bwd_workspace_bytes(const fm_qk_problem* p) {
  bool empty = false;
  if (check_qk(p, &empty) != FM_OK || empty || (!p->q_weight && !p->k_weight)) return 0;
  return qk_bwd_ws_bytes(*p);
}

fm_status fm_qk_norm_rope_bwd(const fm_qk_problem* p, const fm_view* dqo, const fm_view* dko, const fm_view* dvo,
                              const fm_view* q, const fm_view* k, const fm_view* dq, const fm_view* dk,
                              const fm_view* dv, void* dq_weight, void* dk_weight, void* ws, size_t ws_bytes,
                              void* stream) {
  bool empty = false;
  fm_status st = check_qk(p, &empty);
  if (st != FM_OK) return st;
  const bool normed = p->q_weight || p->k_weight;
  if ((p->q_weight && !dq_weight) || (p->k_weight && !dk_weight)) return FM_ERR_INVALID_ARG;
  if (empty) {
    // no token: the weights' gradients are sums of nothing
    const size_t bytes = (size_t)p->d * (p->w_f32 ? 4 : 2);
    for (void* w : {p->q_weight ? dq_weight : nullptr, p->k_weight ? dk_weight : nullptr})
      if (w && cudaMemsetAsync(w, 0, bytes, static_cast<cudaStream_t>(stream)) != cudaSuccess) return FM_ERR_CUDA;
    return FM_OK;
  }
  if (!view_ok(dqo) || !view_ok(dko) || !view_ok(dq) || !view_ok(dk) || (dvo == nullptr) != (dv == nullptr))
    return FM_ERR_INVALID_ARG;
  if (dvo && (!view_ok(dvo) || !view_ok(dv))) return FM_ERR_INVALID_ARG;
  if ((p->q_weight && !view_ok(q)) || (p->k_weight && !view_ok(k))) return FM_ERR_INVALID_ARG;
  if (normed && (!ws || !aligned16(ws) || ws_bytes < qk_bwd_ws_bytes(*p))) return FM_ERR_WORKSPACE;
  return from_cuda(launch_qk_bwd(*p, dqo, dko, dvo, q, k, dq, dk, dv, dq_weight, dk_weight, ws,
                                 static_cast<cudaStream_t>(stream)));
}

fm_status fm_cache_write(const fm_kv_cache* cache, const fm_paged_batch* batch, int32_t T, const fm_rows* k,
                         const fm_rows* v, void* stream) {
  fm_status st = check_cache(cache);
  if (st == FM_OK) st = check_batch(cache, batch, T);
  if (st != FM_OK || T == 0) return st;
  if (!rows_ok(k) || !rows_ok(v)) return FM_ERR_INVALID_ARG;
  int* err = device_error_word();
  if (!err) return FM_ERR_CUDA;
  return from_cuda(launch_cache_write(*cache, *batch, T, *k, *v, static_cast<cudaStream_t>(stream), err));
}

fm_status fm_cache_read(const fm_kv_cache* cache, const int32_t* kv_off, const int32_t* page_table, int32_t R,
                        int32_t width, int32_t n_rows, void* k, void* v, void* stream) {
  fm_status st = check_cache(cache);
  if (st == FM_OK) st = check_table(page_table, R, width, cache->page_size);
  if (st != FM_OK) return st;
  if (n_rows < 0 || !kv_off) return FM_ERR_INVALID_ARG;
  if (n_rows > (1 << 30)) return FM_ERR_UNSUPPORTED;
  if (n_rows == 0) return FM_OK;
  if (!k || !v || !aligned16(k) || !aligned16(v)) return FM_ERR_INVALID_ARG;
  int* err = device_error_word();
  if (!err) return FM_ERR_CUDA;
  return from_cuda(launch_cache_read(*cache, kv_off, page_table, R, width, n_rows, k, v,
                                     static_cast<cudaStream_t>(stream), err));
}

// Shapes of an attention call over the cache; its pointers are checked apart.
static fm_status check_paged(const fm_kv_cache* c, const fm_paged_batch* b, int32_t T, int32_t H_q) {
  fm_status st = check_cache(c);
  if (st == FM_OK) st = check_batch(c, b, T);
  if (st != FM_OK) return st;
  if (H_q <= 0 || H_q % c->H_kv) return FM_ERR_INVALID_ARG;
  if ((int64_t)T * H_q + b->R > (1 << 30)) return FM_ERR_UNSUPPORTED;  // rows and units are counted in 32 bits
  return FM_OK;
}

size_t fm_attn_paged_workspace_bytes(const fm_kv_cache* cache, const fm_paged_batch* batch, int32_t T, int32_t H_q) {
  if (check_paged(cache, batch, T, H_q) != FM_OK || T == 0) return 0;
  return paged_ws_bytes(*cache, *batch, T, H_q);
}

fm_status fm_attn_paged(const fm_kv_cache* cache, const fm_paged_batch* batch, int32_t T, int32_t H_q,
                        const fm_rows* q, float scale, int32_t causal, int32_t window, int32_t sinks,
                        const fm_rows* o, float* lse, void* ws, size_t ws_bytes, void* stream) {
  fm_status st = check_paged(cache, batch, T, H_q);
  if (st != FM_OK) return st;
  // (kernels take scale in log2 units)
  if (!(scale > 0.f) || !std::isfinite(scale * 1.4426950408889634f) || window < 0 || sinks < 0 || (!causal && (window || sinks)))
    return FM_ERR_INVALID_ARG;
  if (T == 0) return FM_OK;
  if (!rows_ok(q) || !rows_ok(o) || !lse) return FM_ERR_INVALID_ARG;
  if (!ws || !aligned16(ws) || ws_bytes < paged_ws_bytes(*cache, *batch, T, H_q)) return FM_ERR_WORKSPACE;
  int* err = device_error_word();
  if (!err) return FM_ERR_CUDA;
  return from_cuda(launch_paged(*cache, *batch, T, H_q, *q, *o, lse, scale, causal ? 1 : 0, window, sinks, ws,
                                static_cast<cudaStream_t>(stream), err));
}

}  // extern "C"
