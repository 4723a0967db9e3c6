// Argument checks of the operators' C entry points, on the host.
#pragma once

#include <cuda_runtime.h>

#include <cmath>
#include <cstdint>

#include "arx.h"
#include "arx_internal.h"
#include "ops_launch.h"

namespace arx {
namespace ops {


constexpr int32_t kMostWaitUs = 2000000;  // of a wait in the product: the default, and the most
constexpr uint64_t kMaxDim = (uint64_t(1) << 31) - 1;

inline arx_status ok() { return succeed(); }

inline arx_status launched(cudaError_t e, const char* what) {
  if (e == cudaSuccess) return ok();
  return report(ARX_ECUDA, "%s launch: %s (%s)", what, cudaGetErrorName(e), cudaGetErrorString(e));
}

inline size_t elem_size(int dtype) { return dtype == ARX_F32 ? 4 : dtype == ARX_E4M3 ? 1 : 2; }

// A matrix of an operator: rows of `cols` elements, `ld` elements apart.
struct Mat {
  const char* name;
  const void* p;
  uint64_t rows, cols, ld;
  int dtype;
  uintptr_t begin() const { return reinterpret_cast<uintptr_t>(p); }
  uint64_t bytes() const {
    if (!p || rows == 0 || cols == 0) return 0;
    return ((rows - 1) * ld + cols) * elem_size(dtype);
  }
};

inline Mat vec(const char* name, const void* p, uint64_t n, int dtype) { return Mat{name, p, 1, n, n, dtype}; }

// The leading dimension of a matrix of one row is not used.
inline Mat mat(const char* name, const void* p, uint64_t rows, uint64_t cols, uint64_t ld, int dtype) {
  return Mat{name, p, rows, cols, rows <= 1 ? cols : ld, dtype};
}

inline arx_status check_mat(const Mat& m, bool required) {
  if (!m.p) return required && m.rows && m.cols ? report(ARX_EINVAL, "%s is null", m.name) : ARX_OK;
  if (m.begin() % elem_size(m.dtype)) return report(ARX_EINVAL, "%s not %zu-byte aligned", m.name, elem_size(m.dtype));
  if (m.ld < m.cols)
    return report(ARX_EINVAL, "leading dimension %llu of %s below its %llu columns", (unsigned long long)m.ld, m.name,
                  (unsigned long long)m.cols);
  if (m.ld > (uint64_t(1) << 40) || m.begin() + m.bytes() < m.begin())
    return report(ARX_EINVAL, "leading dimension %llu of %s too large", (unsigned long long)m.ld, m.name);
  return ARX_OK;
}

// 0: no element in common; 1: the same elements at the same places; 2: other.
inline int overlap(const Mat& a, const Mat& b) {
  if (a.bytes() == 0 || b.bytes() == 0) return 0;
  const uintptr_t a0 = a.begin(), a1 = a0 + a.bytes(), b0 = b.begin(), b1 = b0 + b.bytes();
  if (a1 <= b0 || b1 <= a0) return 0;
  const uint64_t sa = elem_size(a.dtype), sb = elem_size(b.dtype);
  if (a0 == b0 && a.rows == b.rows && a.cols == b.cols && a.ld == b.ld && sa == sb) return 1;
  // Rows that interleave: the same distance between rows in bytes, and column
  // ranges that are disjoint modulo that distance.
  const uint64_t pitch = a.ld * sa;
  if (a.rows > 1 && b.rows > 1 && pitch == b.ld * sb) {
    const uint64_t d = b0 >= a0 ? (b0 - a0) % pitch : (pitch - (a0 - b0) % pitch) % pitch;
    if (d >= a.cols * sa && d + b.cols * sb <= pitch) return 0;
  }
  return 2;
}

// `out` against the arrays it must not touch; `exact` lists those it may equal.
inline arx_status check_output(const Mat& out, const Mat* others, int n, uint32_t may_equal) {
  for (int i = 0; i < n; ++i) {
    const int k = overlap(out, others[i]);
    if (k == 0 || (k == 1 && (may_equal >> i & 1))) continue;
    return report(ARX_EOVERLAP, "%s overlaps %s", out.name, others[i].name);
  }
  return ARX_OK;
}

inline arx_status check_types(int dtype, int wdtype, bool f32_allowed) {
  if (dtype != ARX_BF16 && dtype != ARX_F16 && !(f32_allowed && dtype == ARX_F32))
    return report(ARX_EINVAL, "dtype %d not supported", dtype);
  if (wdtype != dtype && wdtype != ARX_F32)
    return report(ARX_EINVAL, "wdtype %d is neither dtype nor ARX_F32", wdtype);
  return ARX_OK;
}

inline arx_status check_dims(uint64_t a, uint64_t b, uint64_t c) {
  if (a > kMaxDim || b > kMaxDim || c > kMaxDim) return report(ARX_EINVAL, "a dimension is 2^31 or more");
  return ARX_OK;
}

inline arx_status check_workspace(const void* ws, uint64_t have, uint64_t need) {
  if (need == 0) return ARX_OK;
  if (!ws) return report(ARX_EINVAL, "workspace is null, %llu bytes needed", (unsigned long long)need);
  if (reinterpret_cast<uintptr_t>(ws) % 16) return report(ARX_EINVAL, "workspace not 16-byte aligned");
  if (have < need)
    return report(ARX_EINVAL, "workspace %llu bytes, need %llu", (unsigned long long)have, (unsigned long long)need);
  return ARX_OK;
}

inline arx_status check_dropout(double p, const uint64_t* rng) {
  if (!(p >= 0.0 && p <= 1.0)) return report(ARX_EINVAL, "p=%g outside 0..1", p);
  if (p > 0.0 && !rng) return report(ARX_EINVAL, "rng is null");
  if (reinterpret_cast<uintptr_t>(rng) % 8) return report(ARX_EINVAL, "rng not 8-byte aligned");
  return ARX_OK;
}

inline arx_status check_wait(int32_t us) {
  return us >= 0 && us <= kMostWaitUs ? ARX_OK : report(ARX_EINVAL, "wait_us=%d outside 0..%d", us, kMostWaitUs);
}

inline arx_status check_eps(float eps) {
  return eps >= 0.0f ? ARX_OK : report(ARX_EINVAL, "eps=%g is negative or NaN", double(eps));
}

// Whole aligned units of 8 elements in every row (see ops_launch.h).
inline bool units(const Mat& m) {
  if (!m.p) return true;
  const uint64_t unit = 8 * elem_size(m.dtype);
  return m.cols % 8 == 0 && m.begin() % unit == 0 && (m.rows <= 1 || m.ld % 8 == 0);
}
// Parameters are read in 16-byte accesses.
inline bool param_units(const void* p) { return reinterpret_cast<uintptr_t>(p) % 16 == 0; }

inline uint64_t round16(uint64_t x) { return (x + 15) / 16 * 16; }

#define ARX_TRY(expr)                      \
  do {                                     \
    const arx_status s_ = (expr);          \
    if (s_ != ARX_OK) return s_;           \
  } while (0)

inline arx_status check_copies(const void* p, uint64_t have, uint64_t need) {
  if (need == 0) return ARX_OK;
  if (reinterpret_cast<uintptr_t>(p) % 16) return report(ARX_EINVAL, "copies not 16-byte aligned");
  if (have < need)
    return report(ARX_EINVAL, "copies %llu bytes, need %llu", (unsigned long long)have, (unsigned long long)need);
  return ARX_OK;
}

// The products of a layer, without their outputs: sizes, operands, types.
inline GemmCall product(const void* p, uint64_t ldp, bool p_mn, const void* q, uint64_t ldq, bool q_mn, uint64_t rows,
                      uint64_t cols, uint64_t k, int dtype, int wdtype, uint32_t* status, int32_t wait_us) {
  GemmCall c{};
  c.p = p, c.ldp = (p_mn ? k : rows) <= 1 ? (p_mn ? rows : k) : ldp, c.p_mn = p_mn;
  c.q = q, c.ldq = (q_mn ? k : cols) <= 1 ? (q_mn ? cols : k) : ldq, c.q_mn = q_mn;
  c.rows = rows, c.cols = cols, c.k = k;
  c.act = ARX_ACT_NONE, c.dtype = dtype, c.wdtype = wdtype, c.status = status;
  c.wait_ns = uint32_t(wait_us ? wait_us : kMostWaitUs) * 1000u;
  return c;
}

}  // namespace ops
}  // namespace arx
