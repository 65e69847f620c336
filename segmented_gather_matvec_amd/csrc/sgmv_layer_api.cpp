// sgmv_layer_api.cpp - the layer entry points: argument checks and launches.
#include <hip/hip_runtime.h>

#include <cstdint>

#include "../../include/sgmv.h"
#include "sgmv_layer.h"
#include "sgmv_layer_host.h"

namespace {

using namespace sgmv_host;

bool misaligned(const void* p, uintptr_t a) { return reinterpret_cast<uintptr_t>(p) % a != 0; }
const uint16_t* half(const void* p) { return static_cast<const uint16_t*>(p); }
const uint64_t* table(const void* p) { return static_cast<const uint64_t*>(p); }

// Everything one call works on; both projections of a gated block in order gate, up.
struct Call {
  const sgmv_problem_t& p;
  int op;
  LayerPlan plan;
  int np;
  const void* X;
  const void* W[2];
  const sgmv_projection_t* proj[2];
  sgmv::SegMeta meta;
  char* ws;
  hipStream_t stream;
  int32_t act;

  float* at(size_t off) const { return reinterpret_cast<float*>(ws + off); }
  int8_t* row_power() const { return plan.row_powers ? reinterpret_cast<int8_t*>(ws + plan.row_power_off) : nullptr; }
};

// Checks shared by the four entry points.
sgmv_status_t check_call(const void* X, const void* const* W,
                         const sgmv_projection_t* const* proj, int np, const int32_t* seg_indptr,
                         const int32_t* lora_idx, const void* ws, size_t ws_bytes, const LayerPlan& plan) {
  const bool lora = plan.lora;
  if (!X || (lora && (!seg_indptr || !lora_idx))) return SGMV_ERR_INVALID_ARG;
  for (int i = 0; i < np; ++i) {
    if (!W[i] || !proj[i]) return SGMV_ERR_INVALID_ARG;
    if (lora && (!proj[i]->A_ptrs || !proj[i]->B_ptrs)) return SGMV_ERR_INVALID_ARG;
  }
  if (misaligned(X, 16) || misaligned(seg_indptr, 4) || misaligned(lora_idx, 4)) return SGMV_ERR_UNSUPPORTED;
  for (int i = 0; i < np; ++i) {
    if (misaligned(W[i], 16) || misaligned(proj[i]->A_ptrs, 8) || misaligned(proj[i]->B_ptrs, 8) ||
        misaligned(proj[i]->ranks, 4) || misaligned(proj[i]->scales, 4) || misaligned(proj[i]->Y, 16))
      return SGMV_ERR_UNSUPPORTED;
  }
  if (plan.total > 0 && (!ws || ws_bytes < plan.total)) return SGMV_ERR_WORKSPACE;
  if (misaligned(ws, 16)) return SGMV_ERR_UNSUPPORTED;
  return SGMV_OK;
}

sgmv::SegMeta seg_meta(const sgmv_problem_t& p, bool lora, const int32_t* seg_indptr, const int32_t* lora_idx) {
  sgmv::SegMeta m{};
  m.seg_indptr = seg_indptr;
  m.lora_idx = lora_idx;
  m.num_segs = lora ? p.num_segs : 0;
  m.num_loras = p.num_loras;
  m.n_rows = p.n_rows;
  return m;
}

// V_i = s_k Z_i @ A_k (up = false) or s_k Z_i @ B_k^T (up = true) of every projection.
// What of each is wanted: fp32 (the epilogue kernel reads it), 16-bit halves (the tiles and the LoRA gradients).
void thin_params(const Call& c, bool up, const void* const* Z, bool full, bool halves, sgmv::ThinParams* t) {
  const ThinPlan& plan = up ? c.plan.up : c.plan.down;
  for (int i = 0; i < c.np; ++i) {
    t[i] = sgmv::ThinParams{};
    t[i].Z = half(Z[i]);
    t[i].ptrs = up ? table(c.proj[i]->B_ptrs) : table(c.proj[i]->A_ptrs);
    t[i].ranks = c.proj[i]->ranks;
    t[i].scales = c.proj[i]->scales;
    t[i].V = full ? c.at(c.plan.v_off[up][i]) : nullptr;
    t[i].V16 = halves ? reinterpret_cast<uint16_t*>(c.at(c.plan.half_off[up][i])) : nullptr;
    t[i].row_scale = c.at(c.plan.row_scale_off[up][i]);
    t[i].planes = c.at(c.plan.thin_off[up][i]);
    t[i].to_planes = plan.planes > 0;
    t[i].sum_planes = plan.planes;
    t[i].K = up ? c.p.h_out : c.p.h_in;
    t[i].rank = c.p.rank;
    t[i].transposed = up ? 1 : 0;
    t[i].units = plan.units;
    t[i].direct = plan.direct;
    t[i].ksplit = plan.ksplit;
    t[i].kc = plan.kc;
    t[i].z_power = up ? c.row_power() : nullptr;
    t[i].q_power = up ? nullptr : c.row_power();  // V meets dY in dB
    t[i].meta = c.meta;
  }
}

// The lo halves' part of dV, in the planes behind the hi halves' (which t holds).
void thin_lo(const Call& c, const sgmv::ThinParams* t, sgmv::ThinParams* lo) {
  for (int i = 0; i < c.np; ++i) {
    lo[i] = t[i];
    lo[i].Z += (size_t)c.p.n_rows * c.p.h_out;
    lo[i].planes += (size_t)c.plan.up.ksplit * c.p.n_rows * c.p.rank;
    lo[i].sum_planes = 0;
  }
}

sgmv_status_t thin(const Call& c, bool up, const void* const* Z, bool full, bool halves) {
  sgmv::ThinParams t[2];
  thin_params(c, up, Z, full, halves, t);
  return sgmv::launch_thin(c.p.dtype, t, c.np, c.stream) == hipSuccess ? SGMV_OK : SGMV_ERR_HIP;
}

sgmv::DenseParams dense_params(const Call& c, const DensePlan& d, int64_t M, int64_t N, int64_t K, int64_t lda,
                               int64_t ldb) {
  sgmv::DenseParams q{};
  q.M = (int32_t)M;
  q.N = (int32_t)N;
  q.K = (int32_t)K;
  q.lda = (int32_t)lda;
  q.ldb = (int32_t)ldb;
  q.pairs = 1;
  q.projections = 1;
  q.tiles_m = d.tiles_m;
  q.tiles_n = d.tiles_n;
  q.ksplit = d.ksplit;
  q.ktiles_per_split = d.ktiles_per_split;
  q.rank = c.p.rank;
  q.act = c.act;
  q.to_planes = d.to_planes;
  q.term_in_tile = d.term_in_tile;
  q.plane_stride = M * N;
  q.v_planes = 1;
  q.planes = c.at(c.plan.planes_off);
  q.row_power = c.row_power();
  q.meta = c.meta;
  return q;
}

sgmv::LowRankTerm term(const Call& c, int i, bool up) {
  sgmv::LowRankTerm t{};
  if (c.plan.out.term_in_tile) {
    t.V16 = reinterpret_cast<const uint16_t*>(c.at(c.plan.half_off[up][i]));
    t.row_scale = c.at(c.plan.row_scale_off[up][i]);
  } else {
    t.V = c.at(c.plan.v_off[up][i]);
  }
  t.ptrs = table(up ? c.proj[i]->A_ptrs : c.proj[i]->B_ptrs);
  t.pair = table(up ? c.proj[i]->B_ptrs : c.proj[i]->A_ptrs);
  t.ranks = c.proj[i]->ranks;
  return t;
}

// fold = 2: the product's second half of rows adds onto the first (a plane of 2 n rows is two planes of n).
sgmv_status_t run_dense(const Call& c, int mode, const DensePlan& d, const sgmv::DenseParams& q, int fold = 1) {
  if (sgmv::launch_dense(c.p.dtype, mode, d.cfg, q, c.stream) != hipSuccess) return SGMV_ERR_HIP;
  if (!q.to_planes) return SGMV_OK;
  sgmv::DenseParams e = q;
  e.M /= fold;
  e.ksplit *= fold;
  e.plane_stride /= fold;
  return sgmv::launch_dense_epilogue(c.p.dtype, mode, e, c.stream) == hipSuccess ? SGMV_OK : SGMV_ERR_HIP;
}

sgmv_status_t forward(const Call& c, void* const* out) {
  const void* Z[2] = {c.X, c.X};
  if (c.plan.lora && !c.plan.one_launch) {
    const sgmv_status_t st = thin(c, false, Z, !c.plan.out.term_in_tile, c.plan.out.term_in_tile);
    if (st != SGMV_OK) return st;
  }
  const bool gated = layer_gated(c.op);
  const int mode = gated ? sgmv::kDenseGated : sgmv::kDenseForward;
  sgmv::DenseParams q = dense_params(c, c.plan.out, c.p.n_rows, c.p.h_out, c.p.h_in, c.p.h_in, c.p.h_out);
  q.A[0] = half(c.X);
  for (int i = 0; i < c.np; ++i) {
    q.B[i] = half(c.W[i]);
    if (c.plan.lora) q.term[i] = term(c, i, false);
  }
  for (int i = 0; i < (gated ? 3 : 1); ++i) q.out[i] = static_cast<uint16_t*>(out[i]);
  if (!c.plan.one_launch) return run_dense(c, mode, c.plan.out, q);
  sgmv::ThinParams t[2];
  thin_params(c, false, Z, true, false, t);
  int32_t* row_k = reinterpret_cast<int32_t*>(c.at(c.plan.row_k_off));
  q.row_k = row_k;
  q.v_planes = c.plan.down.ksplit;
  for (int i = 0; i < c.np; ++i) {
    t[i].row_k = row_k + (size_t)i * c.p.n_rows;
    if (q.v_planes > 1) q.term[i].V = t[i].planes;
  }
  if (sgmv::launch_dense_thin(c.p.dtype, mode, c.plan.out.cfg, q, t, c.np, c.stream) != hipSuccess) return SGMV_ERR_HIP;
  if (sgmv::launch_dense_epilogue(c.p.dtype, mode, q, c.stream) != hipSuccess) return SGMV_ERR_HIP;
  return SGMV_OK;
}

sgmv_status_t backward(const Call& c, const void* const* dY, void* dX, const sgmv_projection_grad_t* const* grad,
                       int accumulate) {
  const bool rows = c.p.n_rows > 0;
  bool want_a = false, want_b = false;
  for (int i = 0; i < c.np; ++i) {
    want_a = want_a || grad[i]->dA_ptrs;
    want_b = want_b || grad[i]->dB_ptrs;
  }
  if (c.plan.lora) {  // V for dB, dV for dX and dA, in one launch
    sgmv::ThinParams t[sgmv::kMaxThin];
    int count = 0;
    if (want_a || dX) {
      const bool full = dX && !c.plan.out.term_in_tile;
      thin_params(c, true, dY, full, want_a || !full, t);
      count = c.np;
      if (c.plan.halves > 1) {
        thin_lo(c, t, t + count);
        count += c.np;
      }
    }
    if (want_b) {
      const void* Z[2] = {c.X, c.X};
      thin_params(c, false, Z, false, true, t + count);
      count += c.np;
    }
    if (sgmv::launch_thin(c.p.dtype, t, count, c.stream) != hipSuccess) return SGMV_ERR_HIP;
  }
  if (dX && rows) {
    sgmv::DenseParams q = dense_params(c, c.plan.out, (int64_t)c.p.n_rows * c.plan.halves, c.p.h_in, c.p.h_out,
                                       c.p.h_out, c.p.h_out);
    q.pairs = c.np;
    for (int i = 0; i < c.np; ++i) {
      q.A[i] = half(dY[i]);
      q.B[i] = half(c.W[i]);
      if (c.plan.lora) q.term[i] = term(c, i, true);
    }
    q.out[0] = static_cast<uint16_t*>(dX);
    const sgmv_status_t st = run_dense(c, sgmv::kDenseDx, c.plan.out, q, c.plan.halves);
    if (st != SGMV_OK) return st;
  }
  // dW of the projections that want it, one launch when both do.
  sgmv::DenseParams w = dense_params(c, c.plan.dw, c.p.h_in, c.p.h_out, c.p.n_rows, c.p.h_in, c.p.h_out);
  w.projections = 0;
  w.pairs = c.plan.halves;
  w.ktiles_per_split *= c.plan.halves;
  w.A[0] = half(c.X);
  w.accumulate = accumulate;
  for (int i = 0; i < c.np; ++i) {
    if (!grad[i]->dW) continue;
    w.B[w.projections] = half(dY[i]);
    w.out[w.projections++] = static_cast<uint16_t*>(grad[i]->dW);
  }
  if (w.projections > 0 && (rows || !accumulate)) {
    const sgmv_status_t st = run_dense(c, sgmv::kDenseDw, c.plan.dw, w);
    if (st != SGMV_OK) return st;
  }
  if (!c.plan.lora && accumulate) return SGMV_OK;  // no rows: nothing to add
  sgmv::LoraGradParams g[4]{};
  int count = 0;
  float* planes = c.at(c.plan.planes_off);
  for (int b = 1; b >= 0; --b) {
    const int64_t C = b ? c.p.h_out : c.p.h_in;
    const int nsplit = b ? c.plan.nsplit_b : c.plan.nsplit_a;
    for (int i = 0; i < c.np; ++i) {
      const void* out = b ? static_cast<const void*>(grad[i]->dB_ptrs) : static_cast<const void*>(grad[i]->dA_ptrs);
      if (!out) continue;
      sgmv::LoraGradParams& e = g[count++];
      e.Z = half(b ? dY[i] : c.X);
      e.passes = b ? c.plan.halves : 1;
      e.Q = reinterpret_cast<const uint16_t*>(c.at(c.plan.half_off[!b][i]));
      e.row_scale = c.at(c.plan.row_scale_off[!b][i]);
      e.out = table(out);
      e.A = table(c.proj[i]->A_ptrs);
      e.B = table(c.proj[i]->B_ptrs);
      e.ranks = c.proj[i]->ranks;
      e.planes = planes;
      if (nsplit > 1) planes += (size_t)nsplit * c.p.num_loras * C * c.p.rank;
      e.C = (int32_t)C;
      e.rank = c.p.rank;
      e.rank_major = b;
      e.nsplit = nsplit;
      e.by_segment = c.meta.num_segs < c.meta.num_loras;
      e.accumulate = accumulate;
      e.meta = c.meta;
    }
  }
  if (count > 0 && sgmv::launch_lora_grad(c.p.dtype, g, count, c.stream) != hipSuccess) return SGMV_ERR_HIP;
  return SGMV_OK;
}

sgmv_status_t check_grads(const sgmv_projection_grad_t* const* grad, int np, const void* dX) {
  if (misaligned(dX, 16)) return SGMV_ERR_UNSUPPORTED;
  for (int i = 0; i < np; ++i)
    if (misaligned(grad[i]->dW, 16) || misaligned(grad[i]->dA_ptrs, 8) || misaligned(grad[i]->dB_ptrs, 8))
      return SGMV_ERR_UNSUPPORTED;
  return SGMV_OK;
}

}  // namespace

extern "C" {

sgmv_status_t sgmv_dense_lora_apply(const sgmv_problem_t* p, const void* X, const void* W,
                                    const sgmv_projection_t* proj, const int32_t* seg_indptr,
                                    const int32_t* lora_idx, void* ws, size_t ws_bytes, void* stream) {
  sgmv_status_t st = check_layer(p);
  if (st != SGMV_OK) return st;
  if (p->n_rows == 0) return SGMV_OK;
  if (!proj || !proj->Y) return SGMV_ERR_INVALID_ARG;
  const LayerPlan plan = plan_layer(*p, SGMV_DENSE_FORWARD);
  st = check_call(X, &W, &proj, 1, seg_indptr, lora_idx, ws, ws_bytes, plan);
  if (st != SGMV_OK) return st;
  const Call c{*p, SGMV_DENSE_FORWARD, plan, 1, X, {W, nullptr}, {proj, nullptr},
               seg_meta(*p, plan.lora, seg_indptr, lora_idx), static_cast<char*>(ws),
               static_cast<hipStream_t>(stream), 0};
  void* out[1] = {proj->Y};
  return forward(c, out);
}

sgmv_status_t sgmv_gated_lora_apply(const sgmv_problem_t* p, const void* X, const void* Wg, const void* Wu,
                                    const sgmv_projection_t* gate, const sgmv_projection_t* up, int32_t act, void* H,
                                    const int32_t* seg_indptr, const int32_t* lora_idx, void* ws, size_t ws_bytes,
                                    void* stream) {
  sgmv_status_t st = check_layer(p);
  if (st != SGMV_OK) return st;
  if (act != SGMV_ACT_SILU && act != SGMV_ACT_GELU_TANH) return SGMV_ERR_INVALID_ARG;
  if (p->n_rows == 0) return SGMV_OK;
  if (!H) return SGMV_ERR_INVALID_ARG;
  const void* W[2] = {Wg, Wu};
  const sgmv_projection_t* proj[2] = {gate, up};
  const LayerPlan plan = plan_layer(*p, SGMV_GATED_FORWARD);
  st = check_call(X, W, proj, 2, seg_indptr, lora_idx, ws, ws_bytes, plan);
  if (st != SGMV_OK) return st;
  if (misaligned(H, 16)) return SGMV_ERR_UNSUPPORTED;
  const Call c{*p, SGMV_GATED_FORWARD, plan, 2, X, {Wg, Wu}, {gate, up}, seg_meta(*p, plan.lora, seg_indptr, lora_idx),
               static_cast<char*>(ws), static_cast<hipStream_t>(stream), act};
  void* out[3] = {gate->Y, up->Y, H};
  return forward(c, out);
}

sgmv_status_t sgmv_dense_lora_backward(const sgmv_problem_t* p, const void* X, const void* W,
                                       const sgmv_projection_t* proj, const void* dY, void* dX,
                                       const sgmv_projection_grad_t* grad, int32_t accumulate,
                                       const int32_t* seg_indptr, const int32_t* lora_idx, void* ws, size_t ws_bytes,
                                       void* stream) {
  sgmv_status_t st = check_layer(p);
  if (st != SGMV_OK) return st;
  if (accumulate != 0 && accumulate != 1) return SGMV_ERR_INVALID_ARG;
  const sgmv_projection_grad_t none{};
  const sgmv_projection_grad_t* g = grad ? grad : &none;
  if (p->n_rows > 0 && !dY) return SGMV_ERR_INVALID_ARG;
  const LayerPlan plan = plan_layer(*p, SGMV_DENSE_BACKWARD);
  if (p->n_rows > 0) {
    st = check_call(X, &W, &proj, 1, seg_indptr, lora_idx, ws, ws_bytes, plan);
    if (st != SGMV_OK) return st;
  }
  if (!proj) return SGMV_ERR_INVALID_ARG;
  if (misaligned(dY, 16)) return SGMV_ERR_UNSUPPORTED;
  st = check_grads(&g, 1, dX);
  if (st != SGMV_OK) return st;
  const Call c{*p, SGMV_DENSE_BACKWARD, plan, 1, X, {W, nullptr}, {proj, nullptr},
               seg_meta(*p, plan.lora, seg_indptr, lora_idx), static_cast<char*>(ws),
               static_cast<hipStream_t>(stream), 0};
  return backward(c, &dY, dX, &g, accumulate);
}

sgmv_status_t sgmv_gated_lora_backward(const sgmv_problem_t* p, const void* X, const void* Wg, const void* Wu,
                                       const sgmv_projection_t* gate, const sgmv_projection_t* up, int32_t act,
                                       const void* dH, void* dX, const sgmv_projection_grad_t* gate_grad,
                                       const sgmv_projection_grad_t* up_grad, int32_t accumulate,
                                       const int32_t* seg_indptr, const int32_t* lora_idx, void* ws, size_t ws_bytes,
                                       void* stream) {
  sgmv_status_t st = check_layer(p);
  if (st != SGMV_OK) return st;
  if (act != SGMV_ACT_SILU && act != SGMV_ACT_GELU_TANH) return SGMV_ERR_INVALID_ARG;
  if (accumulate != 0 && accumulate != 1) return SGMV_ERR_INVALID_ARG;
  const sgmv_projection_grad_t none{};
  const sgmv_projection_grad_t* g[2] = {gate_grad ? gate_grad : &none, up_grad ? up_grad : &none};
  const void* W[2] = {Wg, Wu};
  const sgmv_projection_t* proj[2] = {gate, up};
  if (!gate || !up) return SGMV_ERR_INVALID_ARG;
  const LayerPlan plan = plan_layer(*p, SGMV_GATED_BACKWARD);
  if (p->n_rows > 0) {
    if (!dH || !gate->Y || !up->Y) return SGMV_ERR_INVALID_ARG;
    st = check_call(X, W, proj, 2, seg_indptr, lora_idx, ws, ws_bytes, plan);
    if (st != SGMV_OK) return st;
  }
  if (misaligned(dH, 16)) return SGMV_ERR_UNSUPPORTED;
  st = check_grads(g, 2, dX);
  if (st != SGMV_OK) return st;
  const Call c{*p, SGMV_GATED_BACKWARD, plan, 2, X, {Wg, Wu}, {gate, up}, seg_meta(*p, plan.lora, seg_indptr, lora_idx),
               static_cast<char*>(ws), static_cast<hipStream_t>(stream), act};
  uint16_t* d[2] = {reinterpret_cast<uint16_t*>(c.at(plan.gate_off[0])),
                    reinterpret_cast<uint16_t*>(c.at(plan.gate_off[1]))};
  if (p->n_rows > 0 &&
      sgmv::launch_gate_backward(p->dtype, act, plan.halves > 1, half(gate->Y), half(up->Y), half(dH), d[0], d[1],
                                 c.row_power(), p->n_rows, p->h_out, c.stream) != hipSuccess)
    return SGMV_ERR_HIP;
  const void* dY[2] = {d[0], d[1]};
  return backward(c, dY, dX, g, accumulate);
}

}  // extern "C"
