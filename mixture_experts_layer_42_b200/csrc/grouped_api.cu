// C ABI of the grouped products and of the 4-bit expert weights (declared in
// include/moe.h): argument checks, workspace and the launches of each entry
// point.
#include "api_common.cuh"
#include "w4.cuh"

#include <cstring>

namespace moe {

namespace {

// Workspace of the grouped products: the error word, then the per-expert maps.
struct GroupedLayout {
  size_t header;
  size_t maps;  // (map_region) [2, E] TMA maps
  size_t total;
};

GroupedLayout grouped_layout(int64_t E) {
  GroupedLayout L;
  L.header = 0;
  L.maps = kWsAlign;
  L.total = align_up(L.maps + (size_t)2 * E * kMapBytes + kMapSlack, kWsAlign);
  return L;
}

moe_status check_shape(const moe_grouped_shape* g) {
  if (!g) return MOE_ERR_INVALID_ARG;
  if (g->dtype != MOE_DT_F32 && g->dtype != MOE_DT_BF16) return MOE_ERR_INVALID_ARG;
  const int q = g->dtype == MOE_DT_BF16 ? 8 : 4;  // 16-byte rows
  if (g->rows < 0 || g->n_experts < 1 || g->n < 1 || g->k < 1) return MOE_ERR_INVALID_ARG;
  if (g->n % q || g->k % q) return MOE_ERR_INVALID_ARG;
  // tile counts, rows and the weights' strides in the kernels' and the maps' types
  if (g->n_experts > 1024 || g->n > (1 << 20) || g->k > (1 << 20)) return MOE_ERR_UNSUPPORTED;
  if ((int64_t)g->n_experts * g->n > ((int64_t)1 << 39) / g->k) return MOE_ERR_UNSUPPORTED;
  if (g->rows > (int64_t)1 << 30) return MOE_ERR_UNSUPPORTED;
  return MOE_OK;
}

moe_status check_grouped_ws(const moe_grouped_shape* g, void* ws, size_t ws_bytes) {
  if (!ws) return MOE_ERR_WORKSPACE;
  if (!aligned16(ws)) return MOE_ERR_INVALID_ARG;
  if (ws_bytes < grouped_layout(g->n_experts).total) return MOE_ERR_WORKSPACE;
  return MOE_OK;
}

// A row matrix may be null when it has no rows.
bool rows_ok(const void* p, int64_t rows) { return rows == 0 || aligned16(p); }

moe_status run_gmm(int mode, const moe_grouped_shape* g, const void* a, const int32_t* offsets,
                   const void* b, void* out, int out_f32, int accumulate, void* ws, size_t ws_bytes,
                   cudaStream_t s) {
  moe_status st;
  if ((st = check_grouped_ws(g, ws, ws_bytes)) != MOE_OK) return st;
  if ((st = bind_device(s, ws)) != MOE_OK) return st;
  GmmArgs p;
  memset(&p, 0, sizeof(p));
  p.a = a;
  p.b = b;
  p.out = out;
  p.offsets = offsets;
  p.rows = g->rows;
  p.E = g->n_experts;
  p.n = g->n;
  p.k = g->k;
  p.out_f32 = out_f32;
  p.accumulate = accumulate;
  p.err = at<uint32_t>(ws, 0);
  const bool bf16 = g->dtype == MOE_DT_BF16;
  if (bf16 && !simt_selected())
    return cuda_status(launch_gmm_tc(mode, p, map_region(ws, grouped_layout(g->n_experts).maps),
                                     num_sms_current(), s));
  return cuda_status(launch_gmm_simt(mode, bf16, p, num_sms_current(), s));
}

bool w4_group_ok(int group) { return group == 32 || group == 64 || group == 128; }

moe_status check_w4(const moe_grouped_shape* g, int group) {
  if (!w4_group_ok(group)) return MOE_ERR_INVALID_ARG;
  if (g->n % 8 || g->k % group) return MOE_ERR_INVALID_ARG;
  return MOE_OK;
}

bool matrix_ok(const moe_w4_matrix& m) { return aligned16(m.q) && aligned16(m.scales); }

void set_matrix(W4Args* p, int kind, const moe_w4_matrix& w1, const moe_w4_matrix* w3) {
  p->q1[kind] = static_cast<const uint8_t*>(w1.q);
  p->s1[kind] = static_cast<const __nv_bfloat16*>(w1.scales);
  if (w3) {
    p->q3[kind] = static_cast<const uint8_t*>(w3->q);
    p->s3[kind] = static_cast<const __nv_bfloat16*>(w3->scales);
  }
}

moe_status run_w4(const moe_grouped_shape* g, int group, int64_t x_rows, const void* x,
                  const int32_t* src, const int32_t* offsets, const moe_w4_matrix* w1,
                  const moe_w4_matrix* w3, bool swiglu, void* out, void* ws, size_t ws_bytes,
                  cudaStream_t s) {
  moe_status st = check_shape(g);
  if (st != MOE_OK) return st;
  if (g->dtype != MOE_DT_BF16) return MOE_ERR_UNSUPPORTED;
  if ((st = check_w4(g, group)) != MOE_OK) return st;
  if (!w1 || !matrix_ok(*w1) || (swiglu && (!w3 || !matrix_ok(*w3)))) return MOE_ERR_INVALID_ARG;
  if (x_rows < 0 || (src == nullptr && x_rows != g->rows) || (x_rows == 0 && g->rows > 0))
    return MOE_ERR_INVALID_ARG;
  if (x_rows > (int64_t)INT32_MAX) return MOE_ERR_UNSUPPORTED;
  if (!rows_ok(x, x_rows) || !rows_ok(out, g->rows) || !aligned16(offsets)) return MOE_ERR_INVALID_ARG;
  if (src && !aligned16(src)) return MOE_ERR_INVALID_ARG;
  if ((st = check_grouped_ws(g, ws, ws_bytes)) != MOE_OK) return st;
  if ((st = bind_device(s, ws)) != MOE_OK) return st;
  W4Args p;
  memset(&p, 0, sizeof(p));
  p.x[0] = static_cast<const __nv_bfloat16*>(x);
  p.src = src;
  p.x_rows = x_rows;
  set_matrix(&p, 0, *w1, swiglu ? w3 : nullptr);
  p.out[0] = static_cast<__nv_bfloat16*>(out);
  p.n[0] = g->n;
  p.k[0] = g->k;
  p.offsets = offsets;
  p.rows = g->rows;
  p.E = g->n_experts;
  p.group = group;
  p.stall = pipeline_stall() == STALL_EXPERTS_UP;
  p.err = at<uint32_t>(ws, 0);
  return cuda_status(launch_w4(swiglu, p, num_sms_current(), s));
}

moe_status check_w4_layer(const moe_config* cfg, int64_t T, int group) {
  moe_status st = check_config(cfg, T);
  if (st != MOE_OK) return st;
  if (cfg->dtype != MOE_DT_BF16) return MOE_ERR_UNSUPPORTED;
  if (!w4_group_ok(group)) return MOE_ERR_INVALID_ARG;
  if (cfg->dim % group || cfg->moe_inter % group || cfg->shared_inter % group)
    return MOE_ERR_INVALID_ARG;
  return MOE_OK;
}

}  // namespace

}  // namespace moe

using namespace moe;

extern "C" {

moe_status moe_grouped_workspace_size(const moe_grouped_shape* g, size_t* bytes) {
  moe_status st = check_shape(g);
  if (st != MOE_OK) return st;
  if (!bytes) return MOE_ERR_INVALID_ARG;
  *bytes = grouped_layout(g->n_experts).total;
  return MOE_OK;
}

moe_status moe_grouped_matmul(const moe_grouped_shape* g, const void* x, const int32_t* offsets,
                              const void* w, void* y, void* ws, size_t ws_bytes, void* stream) {
  moe_status st = check_shape(g);
  if (st != MOE_OK) return st;
  if (!rows_ok(x, g->rows) || !rows_ok(y, g->rows) || !aligned16(offsets) || !aligned16(w))
    return MOE_ERR_INVALID_ARG;
  return run_gmm(GMM_FWD, g, x, offsets, w, y, 0, 0, ws, ws_bytes, (cudaStream_t)stream);
}

moe_status moe_grouped_matmul_dx(const moe_grouped_shape* g, const void* dy, const int32_t* offsets,
                                 const void* w, void* dx, void* ws, size_t ws_bytes, void* stream) {
  moe_status st = check_shape(g);
  if (st != MOE_OK) return st;
  if (!rows_ok(dy, g->rows) || !rows_ok(dx, g->rows) || !aligned16(offsets) || !aligned16(w))
    return MOE_ERR_INVALID_ARG;
  return run_gmm(GMM_DX, g, dy, offsets, w, dx, 0, 0, ws, ws_bytes, (cudaStream_t)stream);
}

moe_status moe_grouped_matmul_dw(const moe_grouped_shape* g, const void* dy, const void* x,
                                 const int32_t* offsets, int32_t dw_dtype, int32_t accumulate,
                                 void* dw, void* ws, size_t ws_bytes, void* stream) {
  moe_status st = check_shape(g);
  if (st != MOE_OK) return st;
  if (dw_dtype != MOE_DT_F32 && dw_dtype != MOE_DT_BF16) return MOE_ERR_INVALID_ARG;
  if (accumulate != 0 && accumulate != 1) return MOE_ERR_INVALID_ARG;
  if (!rows_ok(dy, g->rows) || !rows_ok(x, g->rows) || !aligned16(offsets) || !aligned16(dw))
    return MOE_ERR_INVALID_ARG;
  if (dw_dtype == MOE_DT_BF16 && g->dtype != MOE_DT_BF16) return MOE_ERR_UNSUPPORTED;
  return run_gmm(GMM_DW, g, dy, offsets, x, dw, dw_dtype == MOE_DT_F32, accumulate, ws, ws_bytes,
                 (cudaStream_t)stream);
}

moe_status moe_quantize_w4(const moe_grouped_shape* g, int32_t group, const void* w, void* q,
                           void* scales, void* stream) {
  moe_status st = check_shape(g);
  if (st != MOE_OK) return st;
  if ((st = check_w4(g, group)) != MOE_OK) return st;
  if (!aligned16(w) || !aligned16(q) || !aligned16(scales)) return MOE_ERR_INVALID_ARG;
  if ((st = bind_device((cudaStream_t)stream, w)) != MOE_OK) return st;
  return cuda_status(launch_quantize_w4(g->dtype == MOE_DT_BF16, w, g->n_experts, g->n, g->k, group,
                                        static_cast<uint8_t*>(q),
                                        static_cast<__nv_bfloat16*>(scales), (cudaStream_t)stream));
}

moe_status moe_grouped_matvec_w4(const moe_grouped_shape* g, int32_t group, int64_t x_rows,
                                 const void* x, const int32_t* src, const int32_t* offsets,
                                 const moe_w4_matrix* w, void* y, void* ws, size_t ws_bytes,
                                 void* stream) {
  return run_w4(g, group, x_rows, x, src, offsets, w, nullptr, false, y, ws, ws_bytes,
                (cudaStream_t)stream);
}

moe_status moe_grouped_swiglu_w4(const moe_grouped_shape* g, int32_t group, int64_t x_rows,
                                 const void* x, const int32_t* src, const int32_t* offsets,
                                 const moe_w4_matrix* w1, const moe_w4_matrix* w3, void* h, void* ws,
                                 size_t ws_bytes, void* stream) {
  return run_w4(g, group, x_rows, x, src, offsets, w1, w3, true, h, ws, ws_bytes,
                (cudaStream_t)stream);
}

moe_status moe_workspace_size_w4(const moe_config* cfg, int64_t T, size_t* bytes) {
  moe_status st = check_config(cfg, T);
  if (st != MOE_OK) return st;
  if (cfg->dtype != MOE_DT_BF16) return MOE_ERR_UNSUPPORTED;
  if (!bytes) return MOE_ERR_INVALID_ARG;
  *bytes = ws_layout(*cfg, T).total;
  return MOE_OK;
}

moe_status moe_forward_w4(const moe_config* cfg, int64_t T, const void* x, const void* w_router,
                          const float* bias, const moe_w4_weights* w, void* y, float* weights_out,
                          int32_t* idx_out, void* ws, size_t ws_bytes, void* stream) {
  moe_status st = check_config(cfg, T);
  if (st != MOE_OK) return st;
  if (!w) return MOE_ERR_INVALID_ARG;
  if ((st = check_w4_layer(cfg, T, w->group)) != MOE_OK) return st;
  const moe_config& c = *cfg;
  const bool sh = c.shared_inter > 0;
  if (!aligned16(x) || !aligned16(w_router) || !aligned16(y)) return MOE_ERR_INVALID_ARG;
  if (!matrix_ok(w->w1) || !matrix_ok(w->w3) || !matrix_ok(w->w2)) return MOE_ERR_INVALID_ARG;
  if (sh && (!matrix_ok(w->ws1) || !matrix_ok(w->ws3) || !matrix_ok(w->ws2)))
    return MOE_ERR_INVALID_ARG;
  if (c.has_bias && !aligned16(bias)) return MOE_ERR_INVALID_ARG;
  if ((weights_out && !aligned16(weights_out)) || (idx_out && !aligned16(idx_out)))
    return MOE_ERR_INVALID_ARG;
  const WsLayout L = ws_layout(c, T);
  if (!ws) return MOE_ERR_WORKSPACE;
  if (!aligned16(ws)) return MOE_ERR_INVALID_ARG;
  if (ws_bytes < L.total) return MOE_ERR_WORKSPACE;
  cudaStream_t s = (cudaStream_t)stream;
  if ((st = bind_device(s, ws)) != MOE_OK) return st;
  float* weights = weights_out ? weights_out : at<float>(ws, L.weights);
  int32_t* idx = idx_out ? idx_out : at<int32_t>(ws, L.idx);
  uint32_t* err = at<uint32_t>(ws, L.header);
  if (launch_router(c, T, x, w_router, bias, weights, idx, at<float>(ws, L.router_part),
                    L.router_splits, simt_selected(), num_sms_current(), err, s) != cudaSuccess)
    return MOE_ERR_CUDA;
  int32_t* offsets = at<int32_t>(ws, L.offsets);
  int32_t* pos = at<int32_t>(ws, L.pos);
  int32_t* src = at<int32_t>(ws, L.src);
  if (launch_dispatch(c, T, idx, x, at<int32_t>(ws, L.counts), offsets, src, pos, nullptr,
                      at<int32_t>(ws, L.chunk_hist), at<int32_t>(ws, L.pos_local), L.n_chunks, err,
                      s) != cudaSuccess)
    return MOE_ERR_CUDA;
  // up: h of the routed rows (x through src) and of the shared MLP (x itself)
  W4Args p;
  memset(&p, 0, sizeof(p));
  p.x[0] = p.x[1] = static_cast<const __nv_bfloat16*>(x);
  p.src = src;
  p.x_rows = T;
  set_matrix(&p, 0, w->w1, &w->w3);
  set_matrix(&p, 1, w->ws1, &w->ws3);
  p.out[0] = at<__nv_bfloat16>(ws, L.h);
  p.out[1] = at<__nv_bfloat16>(ws, L.hs);
  p.n[0] = c.moe_inter;
  p.n[1] = c.shared_inter;
  p.k[0] = p.k[1] = c.dim;
  p.offsets = offsets;
  p.rows = T * c.topk;
  p.E = c.n_routed;
  p.group = w->group;
  p.t_shared = sh ? T : 0;
  p.stall = pipeline_stall() == STALL_EXPERTS_UP;
  p.err = err;
  if (launch_w4(true, p, num_sms_current(), s) != cudaSuccess) return MOE_ERR_CUDA;
  // down: from h in the expert order into y_perm, from the shared h into s
  p.stall = 0;
  void* sbuf = sh ? at<void>(ws, L.s) : nullptr;
  p.x[0] = at<__nv_bfloat16>(ws, L.h);
  p.x[1] = at<__nv_bfloat16>(ws, L.hs);
  p.src = nullptr;
  p.x_rows = p.rows;
  set_matrix(&p, 0, w->w2, nullptr);
  set_matrix(&p, 1, w->ws2, nullptr);
  p.out[0] = at<__nv_bfloat16>(ws, L.y_perm);
  p.out[1] = static_cast<__nv_bfloat16*>(sbuf);
  p.n[0] = p.n[1] = c.dim;
  p.k[0] = c.moe_inter;
  p.k[1] = c.shared_inter;
  if (launch_w4(false, p, num_sms_current(), s) != cudaSuccess) return MOE_ERR_CUDA;
  return cuda_status(launch_combine(c, T, at<void>(ws, L.y_perm), pos, weights, sbuf, y, s));
}

}  // extern "C"
