// C entry points of the operators of a sublayer with a root-mean-square norm
// and a gated feed-forward block: argument checks on the host, then the
// launchers.
#include <cuda_runtime.h>

#include <cstdint>

#include "arx.h"
#include "arx_internal.h"
#include "ops_check.h"
#include "ops_launch.h"

namespace {

using namespace arx::ops;
using arx::report;

arx_status check_act(int act) {
  return act >= ARX_ACT_NONE && act <= ARX_ACT_SILU ? ARX_OK : report(ARX_EINVAL, "unknown activation %d", act);
}

// Copies that a call cannot do without.
arx_status check_needed_copies(const void* p, uint64_t have, uint64_t need) {
  if (need && !p) return report(ARX_EINVAL, "copies is null, %llu bytes needed", (unsigned long long)need);
  return check_copies(p, have, need);
}

// 8-bit operands come by the copy engine alone.
arx_status check_on_16(const Mat& m) {
  if (m.bytes() && (m.begin() % 16 || (m.rows > 1 && m.ld % 16)))
    return report(ARX_EINVAL, "8-bit %s not on rows of 16 bytes", m.name);
  return ARX_OK;
}

// dg and du side by side, in rows of 16 bytes: du's first column, and the
// distance of rows.
uint64_t du_column(uint64_t N) { return (N + 7) / 8 * 8; }
uint64_t dz_pitch(uint64_t N) { return 2 * du_column(N); }

bool off_16(const void* p, uint64_t ld, uint64_t rows) {
  return reinterpret_cast<uintptr_t>(p) % 16 || (rows > 1 && ld % 8);
}

// The copies of a backward pass, of rows of K rounded up to 8: both weights for
// dx, and x for the weights' gradients.
struct BackwardCopies {
  bool gate, up, x;
  uint64_t pitch, w_bytes, bytes;
};
BackwardCopies backward_copies(const arx_gated_linear_bwd_args& a) {
  BackwardCopies c{};
  if (a.M == 0 || a.N == 0 || a.K == 0) return c;
  c.pitch = (a.K + 7) / 8 * 8;
  c.w_bytes = a.N * c.pitch * 2;
  c.gate = a.dx && off_16(a.w_gate, a.ldw_gate, a.N);
  c.up = a.dx && off_16(a.w_up, a.ldw_up, a.N);
  c.x = (a.dw_gate || a.dw_up) && off_16(a.x, a.ldx, a.M);
  c.bytes = (c.gate + c.up) * c.w_bytes + (c.x ? a.M * c.pitch * 2 : 0);
  return c;
}

// A matrix to be copied onto rows of 16 bytes at dst, which moves past it; p and ld
// become the copy's.
void add_copy(arx::RealignSet& set, const void*& p, uint64_t& ld, uint64_t rows, uint64_t cols, uint64_t pitch,
              uint8_t*& dst) {
  set.m[set.n++] = {static_cast<const uint16_t*>(p), reinterpret_cast<uint16_t*>(dst), rows, ld, pitch, int64_t(cols)};
  p = dst, ld = pitch;
  dst += rows * pitch * 2;
}

}  // namespace

extern "C" {

arx_status arx_rms_norm(const arx_rms_norm_args* a, void* stream) {
  if (!a) return report(ARX_EINVAL, "null arguments");
  ARX_TRY(check_types(a->dtype, a->wdtype, true));
  ARX_TRY(check_dims(a->rows, a->cols, 0));
  ARX_TRY(check_eps(a->eps));
  if (a->rows == 0 || a->cols == 0) return ok();
  if (!a->y && !a->q) return report(ARX_EINVAL, "y and q are null");
  const Mat in[] = {mat("x", a->x, a->rows, a->cols, a->ldx, a->dtype),
                    mat("residual", a->residual, a->rows, a->cols, a->ldresidual, a->dtype),
                    vec("weight", a->weight, a->cols, a->wdtype)};
  const Mat out[] = {mat("h", a->h, a->rows, a->cols, a->ldh, a->dtype),
                     mat("y", a->y, a->rows, a->cols, a->ldy, a->dtype),
                     mat("q", a->q, a->rows, a->cols, a->ldq, ARX_E4M3),
                     vec("scale", a->q ? a->scale : nullptr, a->rows, ARX_F32), vec("rstd", a->rstd, a->rows, ARX_F32)};
  for (int i = 0; i < 3; ++i) ARX_TRY(check_mat(in[i], i == 0));
  for (int i = 0; i < 5; ++i) {
    ARX_TRY(check_mat(out[i], i == 3 && a->q));
    ARX_TRY(check_output(out[i], in, 3, i < 2 ? 3u : 0u));
    ARX_TRY(check_output(out[i], out, i, 0));
  }
  const bool v = units(in[0]) && units(in[1]) && units(out[0]) && units(out[1]) && units(out[2]) && param_units(a->weight);
  return launched(arx::launch_rms_norm(*a, v, static_cast<cudaStream_t>(stream)), "arx_rms_norm");
}

size_t arx_rms_norm_bwd_workspace_bytes(uint64_t rows, uint64_t cols) {
  if (rows > kMaxDim || cols > kMaxDim) return 0;
  return size_t(arx::rms_bwd_parts(rows) * cols * 4);
}

arx_status arx_rms_norm_bwd(const arx_rms_norm_bwd_args* a, void* stream) {
  if (!a) return report(ARX_EINVAL, "null arguments");
  ARX_TRY(check_types(a->dtype, a->wdtype, true));
  ARX_TRY(check_dims(a->rows, a->cols, 0));
  if (a->cols == 0 || (!a->dx && !a->dweight)) return ok();
  const Mat in[] = {mat("dy", a->dy, a->rows, a->cols, a->lddy, a->dtype),
                    mat("h", a->h, a->rows, a->cols, a->ldh, a->dtype),
                    mat("dresidual", a->dresidual, a->rows, a->cols, a->lddresidual, a->dtype),
                    vec("rstd", a->rstd, a->rows, ARX_F32), vec("weight", a->weight, a->cols, a->wdtype)};
  const uint64_t need = a->dweight ? arx_rms_norm_bwd_workspace_bytes(a->rows, a->cols) : 0;
  const Mat out[] = {mat("dx", a->dx, a->rows, a->cols, a->lddx, a->dtype), vec("dweight", a->dweight, a->cols, a->wdtype),
                     vec("workspace", need ? a->workspace : nullptr, need / 4, ARX_F32)};
  ARX_TRY(check_workspace(a->workspace, a->workspace_bytes, need));
  for (int i = 0; i < 5; ++i) ARX_TRY(check_mat(in[i], i != 2 && i != 4));
  for (int i = 0; i < 3; ++i) {
    ARX_TRY(check_mat(out[i], false));
    ARX_TRY(check_output(out[i], in, 5, i == 0 ? 7u : 0u));
    ARX_TRY(check_output(out[i], out, i, 0));
  }
  const bool v = units(in[0]) && units(in[1]) && units(in[2]) && units(out[0]) && param_units(a->weight);
  return launched(arx::launch_rms_norm_bwd(*a, v, static_cast<cudaStream_t>(stream)), "arx_rms_norm_bwd");
}

arx_status arx_reduce_rms_norm(const arx_reduce_rms_norm_args* a, void* stream) {
  if (!a) return report(ARX_EINVAL, "null arguments");
  if (a->W < 1 || a->W > ARX_MAX_W) return report(ARX_EINVAL, "W=%d outside 1..%d", a->W, ARX_MAX_W);
  ARX_TRY(check_dims(a->rows, a->cols, 0));
  ARX_TRY(check_eps(a->eps));
  if (a->rows == 0 || a->cols == 0) return ok();
  if (!a->slots) return report(ARX_EINVAL, "null pointer array");
  if (!a->y && !a->q) return report(ARX_EINVAL, "y and q are null");
  Mat in[ARX_MAX_W + 2];
  int n = 0;
  in[n++] = mat("residual", a->residual, a->rows, a->cols, a->cols, ARX_BF16);
  for (int r = 0; r < a->W; ++r) in[n++] = mat("a slot", a->slots[r], a->rows, a->cols, a->cols, ARX_BF16);
  const int matrices = n;
  in[n++] = vec("weight", a->weight, a->cols, ARX_BF16);
  const Mat out[] = {mat("h", a->h, a->rows, a->cols, a->cols, ARX_BF16),
                     mat("y", a->y, a->rows, a->cols, a->cols, ARX_BF16),
                     mat("q", a->q, a->rows, a->cols, a->ldq, ARX_E4M3),
                     vec("scale", a->q ? a->scale : nullptr, a->rows, ARX_F32), vec("rstd", a->rstd, a->rows, ARX_F32)};
  for (int i = 0; i < n; ++i) ARX_TRY(check_mat(in[i], i >= 1 && i < matrices));
  for (int i = 0; i < 5; ++i) {
    ARX_TRY(check_mat(out[i], i == 3 && a->q));
    ARX_TRY(check_output(out[i], in, n, i < 2 ? (1u << matrices) - 1u : 0u));
    ARX_TRY(check_output(out[i], out, i, 0));
  }
  bool v = units(out[0]) && units(out[1]) && units(out[2]) && param_units(a->weight);
  for (int i = 0; i < matrices; ++i) v = v && units(in[i]);
  return launched(arx::launch_reduce_rms_norm(*a, v, static_cast<cudaStream_t>(stream)), "arx_reduce_rms_norm");
}

size_t arx_gated_linear_copies_bytes(const arx_gated_linear_args* a) {
  if (!a || a->M > kMaxDim || a->N > kMaxDim || a->K > kMaxDim) return 0;
  return arx::gated_copies_bytes(*a);
}

arx_status arx_gated_linear(const arx_gated_linear_args* a, void* stream) {
  if (!a) return report(ARX_EINVAL, "null arguments");
  const bool eight = a->dtype == ARX_E4M3;
  if (!eight && a->out_dtype != a->dtype) return report(ARX_EINVAL, "out_dtype %d is not dtype", a->out_dtype);
  ARX_TRY(check_types(a->out_dtype, a->wdtype, false));
  if (!eight && (a->x_scale || a->gate_scale || a->up_scale)) return report(ARX_EINVAL, "scales without 8-bit operands");
  ARX_TRY(check_dims(a->M, a->N, a->K));
  ARX_TRY(check_act(a->act));
  ARX_TRY(check_wait(a->wait_us));
  if (a->M == 0 || a->N == 0) return ok();
  const size_t copies = arx::gated_copies_bytes(*a);
  const Mat in[] = {mat("x", a->x, a->M, a->K, a->ldx, a->dtype),
                    mat("w_gate", a->w_gate, a->N, a->K, a->ldw_gate, a->dtype),
                    mat("w_up", a->w_up, a->N, a->K, a->ldw_up, a->dtype),
                    vec("bias_gate", a->bias_gate, a->N, a->wdtype),
                    vec("bias_up", a->bias_up, a->N, a->wdtype),
                    vec("x_scale", a->x_scale, a->M, ARX_F32),
                    vec("gate_scale", a->gate_scale, a->N, ARX_F32),
                    vec("up_scale", a->up_scale, a->N, ARX_F32)};
  const Mat out[] = {mat("out", a->out, a->M, a->N, a->ldout, a->out_dtype),
                     mat("z_gate", a->z_gate, a->M, a->N, a->ldz_gate, a->out_dtype),
                     mat("z_up", a->z_up, a->M, a->N, a->ldz_up, a->out_dtype),
                     vec("status", a->status, 1, ARX_F32), vec("copies", copies ? a->copies : nullptr, copies / 2, ARX_BF16)};
  for (int i = 0; i < 8; ++i) ARX_TRY(check_mat(in[i], i < 3));
  for (int i = 0; i < 3 && eight; ++i) ARX_TRY(check_on_16(in[i]));
  ARX_TRY(check_needed_copies(a->copies, a->copies_bytes, copies));
  for (int i = 0; i < 5; ++i) {
    ARX_TRY(check_mat(out[i], i == 0));
    ARX_TRY(check_output(out[i], in, 8, 0));
    ARX_TRY(check_output(out[i], out, i, 0));
  }
  arx_gated_linear_args c = *a;
  c.ldx = in[0].ld, c.ldw_gate = in[1].ld, c.ldw_up = in[2].ld;
  c.ldout = out[0].ld, c.ldz_gate = out[1].ld, c.ldz_up = out[2].ld;
  if (c.wait_us == 0) c.wait_us = kMostWaitUs;
  return launched(arx::launch_gated(c, static_cast<cudaStream_t>(stream)), "arx_gated_linear");
}

// dg and du, then the partial sums of both biases' gradients.
size_t arx_gated_linear_bwd_workspace_bytes(uint64_t M, uint64_t N) {
  if (M > kMaxDim || N > kMaxDim) return 0;
  return size_t(M * dz_pitch(N) * 2 + 2 * arx::column_parts(M, N) * N * 4);
}

size_t arx_gated_linear_bwd_copies_bytes(const arx_gated_linear_bwd_args* a) {
  if (!a || a->M > kMaxDim || a->N > kMaxDim || a->K > kMaxDim) return 0;
  return size_t(backward_copies(*a).bytes);
}

arx_status arx_gated_linear_bwd(const arx_gated_linear_bwd_args* a, void* stream) {
  if (!a) return report(ARX_EINVAL, "null arguments");
  ARX_TRY(check_types(a->dtype, a->wdtype, false));
  ARX_TRY(check_dims(a->M, a->N, a->K));
  ARX_TRY(check_act(a->act));
  ARX_TRY(check_wait(a->wait_us));
  const bool weights = a->dw_gate || a->dw_up, products = a->dx || weights;
  if (!products && !a->dbias_gate && !a->dbias_up) return ok();
  const Mat in[] = {mat("dout", a->dout, a->M, a->N, a->lddout, a->dtype),
                    mat("z_gate", a->z_gate, a->M, a->N, a->ldz_gate, a->dtype),
                    mat("z_up", a->z_up, a->M, a->N, a->ldz_up, a->dtype),
                    mat("x", weights ? a->x : nullptr, a->M, a->K, a->ldx, a->dtype),
                    mat("w_gate", a->dx ? a->w_gate : nullptr, a->N, a->K, a->ldw_gate, a->dtype),
                    mat("w_up", a->dx ? a->w_up : nullptr, a->N, a->K, a->ldw_up, a->dtype)};
  const uint64_t need = arx_gated_linear_bwd_workspace_bytes(a->M, a->N);
  ARX_TRY(check_workspace(a->workspace, a->workspace_bytes, need));
  const BackwardCopies copies = backward_copies(*a);
  const Mat out[] = {mat("dx", a->dx, a->M, a->K, a->lddx, a->dtype),
                     mat("dw_gate", a->dw_gate, a->N, a->K, a->lddw_gate, a->dtype),
                     mat("dw_up", a->dw_up, a->N, a->K, a->lddw_up, a->dtype),
                     vec("dbias_gate", a->dbias_gate, a->N, a->wdtype),
                     vec("dbias_up", a->dbias_up, a->N, a->wdtype),
                     vec("workspace", need ? a->workspace : nullptr, need / 2, ARX_BF16),
                     vec("status", a->status, 1, ARX_F32),
                     vec("copies", copies.bytes ? a->copies : nullptr, copies.bytes / 2, ARX_BF16)};
  for (int i = 0; i < 6; ++i) ARX_TRY(check_mat(in[i], i < 3 || (i == 3 ? weights : a->dx != nullptr)));
  ARX_TRY(check_needed_copies(a->copies, a->copies_bytes, copies.bytes));
  for (int i = 0; i < 8; ++i) {
    ARX_TRY(check_mat(out[i], false));
    ARX_TRY(check_output(out[i], in, 6, 0));
    ARX_TRY(check_output(out[i], out, i, 0));
  }
  if (a->N == 0 && !(a->dx && a->M && a->K)) return ok();
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  uint8_t* ws = static_cast<uint8_t*>(a->workspace);
  const uint64_t lddz = dz_pitch(a->N);
  const void *dg = ws, *du = ws + du_column(a->N) * 2;

  if (a->N) {
    arx::GatedGradCall g{};
    g.dout = a->dout, g.z_gate = a->z_gate, g.z_up = a->z_up;
    g.lddout = in[0].ld, g.ldz_gate = in[1].ld, g.ldz_up = in[2].ld;
    if (products) g.dz = ws;
    g.lddz = lddz, g.du = du_column(a->N);
    g.dbias_gate = a->dbias_gate, g.dbias_up = a->dbias_up;
    g.part = reinterpret_cast<float*>(ws + a->M * lddz * 2);
    g.rows = a->M, g.cols = a->N;
    g.act = a->act, g.dtype = a->dtype, g.wdtype = a->wdtype;
    const cudaError_t e = arx::launch_gated_grad(g, units(in[0]) && units(in[1]) && units(in[2]), st);
    if (e != cudaSuccess) return launched(e, "arx_gated_linear_bwd");
  }
  const void *wg = a->w_gate, *wu = a->w_up, *x = a->x;
  uint64_t ldg = in[4].ld, ldu = in[5].ld, ldx = in[3].ld;
  if (copies.bytes) {
    uint8_t* to = static_cast<uint8_t*>(a->copies);
    arx::RealignSet set{};
    if (copies.gate) add_copy(set, wg, ldg, a->N, a->K, copies.pitch, to);
    if (copies.up) add_copy(set, wu, ldu, a->N, a->K, copies.pitch, to);
    if (copies.x) add_copy(set, x, ldx, a->M, a->K, copies.pitch, to);
    const cudaError_t e = arx::launch_realign(set, st);
    if (e != cudaSuccess) return launched(e, "arx_gated_linear_bwd");
  }
  if (a->dx && a->M && a->K) {
    arx::GemmCall c = product(dg, lddz, false, wg, ldg, true, a->M, a->K, a->N, a->dtype, a->wdtype, a->status, a->wait_us);
    if (a->N) c.p2 = du, c.ldp2 = c.ldp, c.q2 = wu, c.ldq2 = a->N <= 1 ? a->K : ldu;
    c.out = a->dx, c.ldout = out[0].ld;
    const cudaError_t e = arx::launch_gemm(c, st);
    if (e != cudaSuccess) return launched(e, "arx_gated_linear_bwd");
  }
  if (weights && a->N && a->K) {  // both in one launch, so that their tiles fill the SMs together
    const bool both = a->dw_gate && a->dw_up && a->M;
    for (int i = 0; i < 2; ++i) {
      const Mat& dw = out[1 + i];
      if (!dw.p || (both && i)) continue;
      arx::GemmCall c = product(i ? du : dg, lddz, true, x, ldx, true, a->N, a->K, a->M, a->dtype, a->wdtype, a->status,
                                a->wait_us);
      c.out = const_cast<void*>(dw.p), c.ldout = dw.ld;
      if (both) c.p2 = du, c.ldp2 = c.ldp, c.out2 = a->dw_up, c.ldout2 = out[2].ld;
      const cudaError_t e = arx::launch_gemm(c, st);
      if (e != cudaSuccess) return launched(e, "arx_gated_linear_bwd");
    }
  }
  return ok();
}

}  // extern "C"
