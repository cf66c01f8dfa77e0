// block.h — launchers of what stands around an expert layer: the router's losses, the
// combine's gradient, norms and adapters. Beside common.h, whose text the counter
// summaries of the grouped GEMMs are tied to.
#pragma once

#include "common.h"

namespace moe {

// The combine's gradient; dy_perm or dgate may be null.
moe_status launch_combine_bwd(const void* dout, const void* y_perm, moe_dtype dt, const int32_t* perm_dst,
                              const float* gate, int T, int K, int N, void* dy_perm, float* dgate, hipStream_t s);

// The router's losses and their gradient joined with the kept gates'.
size_t router_loss_ws_bytes(int T, int E);
moe_status launch_router_loss(const void* scores, moe_dtype dt, const int32_t* idx, const uint8_t* mask, int T, int E,
                              int K, int32_t* counts, int32_t* tokens, float* probs, float* loss, void* ws,
                              hipStream_t s);
moe_status launch_router_loss_bwd(const void* scores, moe_dtype dt, const int32_t* idx, const uint8_t* mask,
                                  const int32_t* counts, const int32_t* tokens, const float* dloss, const float* gate,
                                  const float* dgate, int T, int E, int K, void* out, moe_dtype out_dt,
                                  hipStream_t s);

// Norms around a block. z and h have one type, r and r_out another; norm weights
// and the gate are binary32 (w_f32) or bf16. z null: h is the norm of r alone.
struct NormCall {
  const void *z, *r, *w_post, *b_post, *gate, *w_pre, *b_pre;
  void *r_out, *h;
  int T, N, kind, post, gate_mode;
  bool w_f32;
  float alpha, beta, eps;
};
moe_status launch_norm(const NormCall& c, moe_dtype dt, moe_dtype r_dt, hipStream_t s);
// Their gradients; every output may be null, and dh (no norm after r_out), dr_out
// (no other use of r_out) and z (the norm of r_out alone).
struct NormBwdCall {
  const void *dh, *dr_out, *z, *r_out, *w_post, *b_post, *gate, *w_pre;
  void *dr, *dz, *dw_post, *db_post, *dgate, *dw_pre, *db_pre;
  float* sums;  // workspace of norm_bwd_ws_bytes()
  int T, N, kind, post, gate_mode;
  bool w_f32, dw_f32;
  float alpha, beta, eps;
  int use = 0;  // set by the launcher: the column sums that an output needs
};
size_t norm_bwd_ws_bytes(int T, int N);
moe_status launch_norm_bwd(NormBwdCall c, moe_dtype dt, moe_dtype r_dt, hipStream_t s);

// Low-rank adapters over M rows grouped by adapter; grouped row r is row rows[r]
// (or r) of tensors of T rows. scale: binary32 per adapter, or null (1).
struct LoraCall {
  const int32_t* offsets;
  const int32_t* rows;
  const float* scale;
  int e, T, M, H, N, R;
  bool fill;                  // rows of the output that `rows` does not name get base, or zeros; T <= M
  int32_t* listed = nullptr;  // set by the launcher: (T) of the workspace, which rows are named
};
size_t lora_ws_bytes(int e, int M, int H, int R);
moe_status launch_lora(const LoraCall& c, const void* x, const void* base, moe_dtype dt, const void* a, const void* b,
                       float* u_out, void* out, void* ws, hipStream_t s);
size_t lora_bwd_ws_bytes(moe_dtype dt, int e, int M, int H, int N, int R);
moe_status launch_lora_bwd(const LoraCall& c, const void* dout, const void* x, const float* u, moe_dtype dt,
                           const void* a, const void* b, const void* dx_base, void* dx, void* da, void* db,
                           moe_dtype dw_dt, void* ws, hipStream_t s);

}  // namespace moe
