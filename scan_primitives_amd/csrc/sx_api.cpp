// sx_api.cpp: the C ABI of libsx_scan.so (declared in include/sx_scan.h).
//
// Every argument is validated here, on the host, before anything touches the
// device: a rejected call launches nothing and leaves `out` alone. The
// shapes and strides are then reduced to the compact descriptors of
// sx_common.hpp and handed to the launchers in element_scan.hip and
// matrix_scan.hip.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstring>
#include <cstdarg>
#include <cstdio>
#include <string>

#include "sx_attention.hpp"
#include "sx_common.hpp"
#include "sx_state_space.hpp"

namespace sx {

int device_cu_count() {
  static int cached[64] = {};
  int dev = 0;
  if (hipGetDevice(&dev) != hipSuccess || dev < 0) return 256;
  if (dev < 64 && cached[dev] > 0) return cached[dev];
  int cus = 0;
  if (hipDeviceGetAttribute(&cus, hipDeviceAttributeMultiprocessorCount, dev) != hipSuccess || cus <= 0) cus = 256;
  if (dev < 64) cached[dev] = cus;
  return cus;
}

}  // namespace sx

namespace {

thread_local std::string g_last_error;

sx_status fail(sx_status st, const char* fmt, ...) {
  char buf[1024];
  va_list ap;
  va_start(ap, fmt);
  vsnprintf(buf, sizeof buf, fmt, ap);
  va_end(ap);
  g_last_error = std::string("error[") + sx_status_name(st) + "]: " + buf;
  return st;
}

sx_status ok() {
  g_last_error.clear();
  return SX_OK;
}

// The integer an enum argument holds. A C caller may pass any int where the
// ABI declares an enum; reading it as the C++ enum type before it is checked
// would be undefined for values outside the enum's range, so every entry point
// checks the bits first.
template <typename E>
int enum_code(const E& e) {
  static_assert(sizeof(E) == sizeof(int), "C enums are int-sized here");
  int v;
  std::memcpy(&v, &e, sizeof v);
  return v;
}

bool body_ok(const sx_body& b) {
  const int v = enum_code(b);
  return v == SX_BODY_TANH_AFFINE || v == SX_BODY_NORM_CAP || v == SX_BODY_MAX_PLUS;
}

bool dtype_ok(const sx_dtype& d) {
  const int v = enum_code(d);
  return v == SX_F32 || v == SX_BF16;
}

std::string shape_str(int rank, const int64_t* shape) {
  std::string s = "[";
  for (int i = 0; i < rank; ++i) {
    if (i) s += ", ";
    s += std::to_string(shape[i]);
  }
  return s + "]";
}

const char* dtype_name(int dt) { return dt == SX_F32 ? "f32" : dt == SX_BF16 ? "bf16" : "?"; }

void contiguous_strides(int rank, const int64_t* shape, int64_t* st) {
  int64_t acc = 1;
  for (int i = rank - 1; i >= 0; --i) {
    st[i] = acc;
    acc *= std::max<int64_t>(shape[i], 1);
  }
}

// Checked product; returns false on overflow past 2^62.
bool checked_numel(int rank, const int64_t* shape, int64_t* numel) {
  int64_t n = 1;
  for (int i = 0; i < rank; ++i) {
    if (shape[i] < 0) return false;
    if (shape[i] != 0 && n > (int64_t(1) << 62) / shape[i]) return false;
    n *= shape[i];
  }
  *numel = n;
  return true;
}

// Byte span [lo, hi) that a strided tensor touches (only meaningful when numel > 0).
void span_bytes(const void* base, int rank, const int64_t* shape, const int64_t* st, size_t elem,
                uintptr_t* lo, uintptr_t* hi) {
  int64_t mn = 0, mx = 0;
  for (int i = 0; i < rank; ++i) {
    const int64_t e = (shape[i] - 1) * st[i];
    if (e < 0) mn += e; else mx += e;
  }
  const uintptr_t b = reinterpret_cast<uintptr_t>(base);
  *lo = b + uintptr_t(mn * int64_t(elem));
  *hi = b + uintptr_t((mx + 1) * int64_t(elem));
}

bool overlaps(uintptr_t alo, uintptr_t ahi, uintptr_t blo, uintptr_t bhi) { return alo < bhi && blo < ahi; }

// Builds an IndexMap from per-dimension sizes and strides, dropping size-1
// dims and merging neighbours whose strides nest for every tensor.
template <int NT>
sx::IndexMap<NT> make_index_map(int nd, const int64_t* dims, const int64_t (*st)[sx::kMaxRank]) {
  sx::IndexMap<NT> m{};
  int k = 0;
  for (int d = 0; d < nd; ++d) {
    if (dims[d] == 1) continue;
    bool merge = k > 0;
    for (int t = 0; t < NT && merge; ++t) merge = st[t][d] * dims[d] == m.st[t][k - 1];
    if (merge) {
      m.dim[k - 1] *= dims[d];
      for (int t = 0; t < NT; ++t) m.st[t][k - 1] = st[t][d];
    } else {
      m.dim[k] = dims[d];
      for (int t = 0; t < NT; ++t) m.st[t][k] = st[t][d];
      ++k;
    }
  }
  if (k == 0) {
    m.dim[0] = 1;
    for (int t = 0; t < NT; ++t) m.st[t][0] = 0;
    k = 1;
  }
  m.nd = k;
  return m;
}

sx_status device_status(hipError_t e, const char* what) {
  if (e == hipSuccess) return ok();
  return fail(SX_E_DEVICE, "%s: %s", what, hipGetErrorString(e));
}

// ------------------------------------------------------------ element-scan validation

struct EsPlan {
  sx::EsParams p;
  int64_t numel;
};

sx_status plan_element_scan(sx_body body, int rank, const int64_t* shape, int axis, int state_axis,
                            const int64_t* initial_strides, int64_t x_width, const int64_t* x_strides,
                            int64_t s_width, const int64_t* s_strides, EsPlan* plan) {
  if (body != SX_BODY_TANH_AFFINE && body != SX_BODY_NORM_CAP && body != SX_BODY_MAX_PLUS)
    return fail(SX_E_UNSUPPORTED, "element-scan: unknown body %d", int(body));
  if (rank > sx::kMaxRank) return fail(SX_E_UNSUPPORTED, "element-scan: rank %d exceeds %d", rank, sx::kMaxRank);
  if (rank < 1 || shape == nullptr) return fail(SX_E_DIM_001, "element-scan: sequences need at least one axis");
  int64_t numel = 0;
  if (!checked_numel(rank, shape, &numel))
    return fail(SX_E_DIM_001, "element-scan: bad sequence shape %s", shape_str(rank, shape).c_str());
  const int ax = axis < 0 ? axis + rank : axis;
  if (ax < 0 || ax >= rank)
    return fail(SX_E_DIM_001, "element-scan: axis %d out of range for sequences %s f32", axis,
                shape_str(rank, shape).c_str());
  const bool vec = state_axis != SX_STATE_SCALAR;
  if (vec && state_axis != -1 && state_axis != rank - 1)
    return fail(SX_E_DIM_001, "element-scan: :state-axis %d is not the last axis of %s", state_axis,
                shape_str(rank, shape).c_str());
  if (!vec && body == SX_BODY_NORM_CAP)
    return fail(SX_E_DIM_001, "element-scan: the norm-cap body reduces over the state, so it needs :state-axis -1");
  int64_t n = 1;
  if (vec) {
    if (rank < 2 || ax == rank - 1)
      return fail(SX_E_DIM_001, "element-scan: :axis %d is the state axis of %s", axis, shape_str(rank, shape).c_str());
    n = shape[rank - 1];
    if (n < 1 || n > SX_MAX_N)
      return fail(SX_E_DIM_001, "element-scan: state width %lld is outside 1..16", (long long)n);
    if (x_width != 1 && x_width != n)
      return fail(SX_E_DIM_001, "element-scan: sequence x has width %lld, state width is %lld", (long long)x_width, (long long)n);
    if (s_width != 1 && s_width != n)
      return fail(SX_E_DIM_001, "element-scan: second sequence has width %lld, state width is %lld", (long long)s_width, (long long)n);
  }
  const int64_t T = shape[ax];
  if (T < 1)
    return fail(SX_E_DIM_001, "element-scan: axis %d of %s has length 0; it must be at least one", axis,
                shape_str(rank, shape).c_str());

  // Per-tensor shapes and strides (elements).
  int64_t xs[sx::kMaxRank], ss[sx::kMaxRank], is[sx::kMaxRank], os[sx::kMaxRank];
  int64_t xshape[sx::kMaxRank], sshape[sx::kMaxRank], ishape[sx::kMaxRank];
  for (int i = 0; i < rank; ++i) xshape[i] = sshape[i] = shape[i];
  if (vec) { xshape[rank - 1] = x_width; sshape[rank - 1] = s_width; }
  for (int i = 0, j = 0; i < rank; ++i)
    if (i != ax) ishape[j++] = shape[i];
  if (x_strides) std::copy(x_strides, x_strides + rank, xs); else contiguous_strides(rank, xshape, xs);
  if (s_strides) std::copy(s_strides, s_strides + rank, ss); else contiguous_strides(rank, sshape, ss);
  if (initial_strides) std::copy(initial_strides, initial_strides + rank - 1, is); else contiguous_strides(rank - 1, ishape, is);
  contiguous_strides(rank, shape, os);
  if (vec) {  // a width-1 sequence broadcasts over the state vector
    if (x_width == 1) xs[rank - 1] = 0;
    if (s_width == 1) ss[rank - 1] = 0;
  }

  sx::EsParams& p = plan->p;
  p = sx::EsParams{};
  p.T = T;
  p.t_stride[sx::ES_X] = xs[ax];
  p.t_stride[sx::ES_S] = ss[ax];
  p.t_stride[sx::ES_INIT] = 0;
  p.t_stride[sx::ES_OUT] = os[ax];
  p.n = body == SX_BODY_NORM_CAP ? int(n) : 1;
  if (body == SX_BODY_NORM_CAP) {
    p.n_stride[sx::ES_X] = xs[rank - 1];
    p.n_stride[sx::ES_S] = ss[rank - 1];
    p.n_stride[sx::ES_INIT] = is[rank - 2];
    p.n_stride[sx::ES_OUT] = 1;
  }
  // Lane dims: every dim but the axis (and but the state axis for NORM_CAP).
  const int lane_end = body == SX_BODY_NORM_CAP ? rank - 1 : rank;
  int64_t dims[sx::kMaxRank];
  int64_t st[4][sx::kMaxRank];
  int nd = 0;
  for (int i = 0; i < lane_end; ++i) {
    if (i == ax) continue;
    dims[nd] = shape[i];
    st[sx::ES_X][nd] = xs[i];
    st[sx::ES_S][nd] = ss[i];
    st[sx::ES_INIT][nd] = is[i < ax ? i : i - 1];
    st[sx::ES_OUT][nd] = os[i];
    ++nd;
  }
  p.lanes = make_index_map<4>(nd, dims, st);
  p.num_lanes = numel / T / (body == SX_BODY_NORM_CAP ? n : 1);
  plan->numel = numel;

  // Spans for the alias check are computed by the caller once the pointers are known.
  (void)xshape;
  return ok();
}

}  // namespace

extern "C" {

const char* sx_status_name(sx_status status) {
  switch (enum_code(status)) {
    case SX_OK: return "OK";
    case SX_E_DIM_001: return "E-DIM-001";
    case SX_E_DIM_002: return "E-DIM-002";
    case SX_E_DIM_003: return "E-DIM-003";
    case SX_E_UNSUPPORTED: return "E-UNSUPPORTED";
    case SX_E_ALIAS: return "E-ALIAS";
    case SX_E_WORKSPACE: return "E-WORKSPACE";
    case SX_E_DEVICE: return "E-DEVICE";
  }
  return "E-UNKNOWN";
}

const char* sx_last_error(void) { return g_last_error.c_str(); }

const char* sx_version(void) { return "sx_scan 0.1 gfx950"; }

size_t sx_element_scan_workspace_bytes(sx_body body, int rank, const int64_t* shape, int axis, int state_axis) {
  if (!body_ok(body)) return 0;
  EsPlan plan;
  const int64_t w = 1;
  if (plan_element_scan(body, rank, shape, axis, state_axis, nullptr, w, nullptr, w, nullptr, &plan) != SX_OK)
    return 0;
  return sx::element_scan_workspace(body, plan.p);
}

sx_status sx_element_scan(sx_body body, int rank, const int64_t* shape, int axis, int state_axis, int reverse,
                          const float* initial, const int64_t* initial_strides, const float* x, int64_t x_width,
                          const int64_t* x_strides, const float* s, int64_t s_width, const int64_t* s_strides,
                          float* out, void* workspace, size_t workspace_bytes, void* stream) {
  if (!body_ok(body)) return fail(SX_E_UNSUPPORTED, "element-scan: unknown body %d", enum_code(body));
  EsPlan plan;
  sx_status st = plan_element_scan(body, rank, shape, axis, state_axis, initial_strides, x_width, x_strides,
                                   s_width, s_strides, &plan);
  if (st != SX_OK) return st;
  if (plan.numel == 0) return ok();
  if (!x) return fail(SX_E_DIM_003, "element-scan: sequence x is NULL; a tensor was expected");
  if (!s) return fail(SX_E_DIM_003, "element-scan: the second sequence is NULL; a tensor was expected");
  if (!initial) return fail(SX_E_DIM_003, "element-scan: initial is NULL; a tensor was expected");
  if (!out) return fail(SX_E_DIM_003, "element-scan: out is NULL; a tensor was expected");

  // Alias check: out is contiguous over the output shape.
  const bool vec = state_axis != SX_STATE_SCALAR;
  int64_t xshape[sx::kMaxRank], sshape[sx::kMaxRank], ishape[sx::kMaxRank];
  int64_t xs[sx::kMaxRank], ss[sx::kMaxRank], is[sx::kMaxRank];
  const int ax = axis < 0 ? axis + rank : axis;
  for (int i = 0; i < rank; ++i) xshape[i] = sshape[i] = shape[i];
  if (vec) { xshape[rank - 1] = x_width; sshape[rank - 1] = s_width; }
  for (int i = 0, j = 0; i < rank; ++i)
    if (i != ax) ishape[j++] = shape[i];
  if (x_strides) std::copy(x_strides, x_strides + rank, xs); else contiguous_strides(rank, xshape, xs);
  if (s_strides) std::copy(s_strides, s_strides + rank, ss); else contiguous_strides(rank, sshape, ss);
  if (initial_strides) std::copy(initial_strides, initial_strides + rank - 1, is); else contiguous_strides(rank - 1, ishape, is);
  uintptr_t olo = reinterpret_cast<uintptr_t>(out), ohi = olo + uintptr_t(plan.numel) * sizeof(float);
  uintptr_t lo, hi;
  span_bytes(x, rank, xshape, xs, sizeof(float), &lo, &hi);
  if (overlaps(olo, ohi, lo, hi)) return fail(SX_E_ALIAS, "element-scan: out overlaps sequence x");
  span_bytes(s, rank, sshape, ss, sizeof(float), &lo, &hi);
  if (overlaps(olo, ohi, lo, hi)) return fail(SX_E_ALIAS, "element-scan: out overlaps the second sequence");
  span_bytes(initial, rank - 1, ishape, is, sizeof(float), &lo, &hi);
  if (overlaps(olo, ohi, lo, hi)) return fail(SX_E_ALIAS, "element-scan: out overlaps initial");

  const size_t need = sx::element_scan_workspace(body, plan.p);
  if (need > 0 && (workspace == nullptr || workspace_bytes < need))
    return fail(SX_E_WORKSPACE, "element-scan: workspace of %zu bytes given, %zu needed", workspace_bytes, need);
  if (need > 0 && (reinterpret_cast<uintptr_t>(workspace) & 255u) != 0)
    return fail(SX_E_WORKSPACE, "element-scan: workspace must be 256-byte aligned");

  plan.p.reverse = reverse ? 1 : 0;
  plan.p.x = x;
  plan.p.s = s;
  plan.p.init = initial;
  plan.p.out = out;
  return device_status(sx::launch_element_scan(body, plan.p, static_cast<hipStream_t>(stream)),
                       "element-scan launch");
}

// ------------------------------------------------------------------ matrix-scan

static sx_status plan_matrix_scan(int a_rank, const int64_t* a_shape, const int64_t* a_strides, int b_rank,
                                  const int64_t* b_shape, const int64_t* b_strides, int axis, sx::MsParams* p,
                                  int64_t* out_shape, int* out_rank, int64_t* out_numel) {
  if (a_rank > sx::kMaxRank || b_rank > sx::kMaxRank)
    return fail(SX_E_UNSUPPORTED, "matrix-scan: rank above %d", sx::kMaxRank);
  if (!a_shape || !b_shape || a_rank < 2 || b_rank < 2)
    return fail(SX_E_DIM_001, "matrix-scan: a must be [.., n, n] and b [.., n, m]");
  int64_t tmp;
  if (!checked_numel(a_rank, a_shape, &tmp) || !checked_numel(b_rank, b_shape, &tmp))
    return fail(SX_E_DIM_001, "matrix-scan: negative or oversized dims in a %s, b %s",
                shape_str(a_rank, a_shape).c_str(), shape_str(b_rank, b_shape).c_str());
  const int64_t n = a_shape[a_rank - 1];
  if (a_shape[a_rank - 2] != n)
    return fail(SX_E_DIM_001, "matrix-scan: a %s is not square", shape_str(a_rank, a_shape).c_str());
  if (b_shape[b_rank - 2] != n)
    return fail(SX_E_DIM_001, "matrix-scan: inner dims differ: a %s, b %s", shape_str(a_rank, a_shape).c_str(),
                shape_str(b_rank, b_shape).c_str());
  if (n > SX_MAX_N)
    return fail(SX_E_DIM_001, "matrix-scan: n = %lld, at most 16 allowed (a %s)", (long long)n,
                shape_str(a_rank, a_shape).c_str());
  const int64_t m = b_shape[b_rank - 1];
  const int la = a_rank - 2, lb = b_rank - 2, L = std::max(la, lb);
  if (L < 1)
    return fail(SX_E_DIM_001, "matrix-scan: no leading dim to scan along (a %s, b %s)",
                shape_str(a_rank, a_shape).c_str(), shape_str(b_rank, b_shape).c_str());
  if (L + 2 > sx::kMaxRank) return fail(SX_E_UNSUPPORTED, "matrix-scan: result rank above %d", sx::kMaxRank);
  int64_t lead[sx::kMaxRank], sa[sx::kMaxRank], sb[sx::kMaxRank];
  int64_t ast[sx::kMaxRank], bst[sx::kMaxRank];
  if (a_strides) std::copy(a_strides, a_strides + a_rank, ast); else contiguous_strides(a_rank, a_shape, ast);
  if (b_strides) std::copy(b_strides, b_strides + b_rank, bst); else contiguous_strides(b_rank, b_shape, bst);
  for (int i = 0; i < L; ++i) {
    const int ia = i - (L - la), ib = i - (L - lb);
    const int64_t da = ia >= 0 ? a_shape[ia] : 1, db = ib >= 0 ? b_shape[ib] : 1;
    if (da != db && da != 1 && db != 1)
      return fail(SX_E_DIM_001, "matrix-scan: leading dims of a %s and b %s do not broadcast",
                  shape_str(a_rank, a_shape).c_str(), shape_str(b_rank, b_shape).c_str());
    lead[i] = da == 1 ? db : da;
    sa[i] = (ia >= 0 && da != 1) ? ast[ia] : 0;
    sb[i] = (ib >= 0 && db != 1) ? bst[ib] : 0;
  }
  const int ax = axis < 0 ? axis + L : axis;
  if (ax < 0 || ax >= L)
    return fail(SX_E_DIM_001, "matrix-scan: axis %d out of range for leading dims %s", axis,
                shape_str(L, lead).c_str());
  if ((n > 1 && (ast[a_rank - 1] != 1 || ast[a_rank - 2] != n)) ||
      (m > 1 && bst[b_rank - 1] != 1) || (n > 1 && m > 0 && bst[b_rank - 2] != m))
    return fail(SX_E_UNSUPPORTED, "matrix-scan: the matrix dims of a and b must be row-major contiguous");

  for (int i = 0; i < L; ++i) out_shape[i] = lead[i];
  out_shape[L] = n;
  out_shape[L + 1] = m;
  *out_rank = L + 2;
  int64_t numel = 0;
  if (!checked_numel(L + 2, out_shape, &numel)) return fail(SX_E_DIM_001, "matrix-scan: result too large");
  *out_numel = numel;
  if (!p) return ok();

  int64_t ost[sx::kMaxRank + 2];
  contiguous_strides(L + 2, out_shape, ost);
  *p = sx::MsParams{};
  p->T = lead[ax];
  p->t_stride[sx::MS_A] = sa[ax];
  p->t_stride[sx::MS_B] = sb[ax];
  p->t_stride[sx::MS_OUT] = ost[ax];
  p->n = int(n);
  p->m = int(m);
  int64_t dims[sx::kMaxRank];
  int64_t st[3][sx::kMaxRank];
  int nd = 0;
  for (int i = 0; i < L; ++i) {
    if (i == ax) continue;
    dims[nd] = lead[i];
    st[sx::MS_A][nd] = sa[i];
    st[sx::MS_B][nd] = sb[i];
    st[sx::MS_OUT][nd] = ost[i];
    ++nd;
  }
  p->batch = make_index_map<3>(nd, dims, st);
  p->num_batch = p->T > 0 ? numel / (p->T * std::max<int64_t>(n * m, 1)) : 0;
  if (n * m == 0) p->num_batch = 0;
  return ok();
}

int sx_matrix_scan_out_shape(int a_rank, const int64_t* a_shape, int b_rank, const int64_t* b_shape,
                             int64_t* out_shape) {
  int64_t shp[sx::kMaxRank + 2];
  int r = 0;
  int64_t numel = 0;
  if (plan_matrix_scan(a_rank, a_shape, nullptr, b_rank, b_shape, nullptr, -1, nullptr, shp, &r, &numel) != SX_OK)
    return -1;
  if (out_shape) std::copy(shp, shp + r, out_shape);
  return r;
}

size_t sx_matrix_scan_workspace_bytes(int a_rank, const int64_t* a_shape, int b_rank, const int64_t* b_shape,
                                      int axis) {
  sx::MsParams p;
  int64_t shp[sx::kMaxRank + 2];
  int r = 0;
  int64_t numel = 0;
  if (plan_matrix_scan(a_rank, a_shape, nullptr, b_rank, b_shape, nullptr, axis, &p, shp, &r, &numel) != SX_OK)
    return 0;
  if (numel == 0) return 0;
  return sx::matrix_scan_workspace(p);
}

}  // extern "C"

namespace {

// sx_matrix_scan, and with scratch = true sx_matrix_scan_noalloc: the look-back
// state then goes to the library's fixed device array instead of `workspace`.
sx_status matrix_scan_call(const sx_dtype& dtype, int a_rank, const int64_t* a_shape, const int64_t* a_strides,
                           const void* a, int b_rank, const int64_t* b_shape, const int64_t* b_strides, const void* b,
                           int axis, int reverse, int projective, const sx_dtype& out_dtype, void* out, void* workspace,
                           size_t workspace_bytes, void* stream, bool scratch) {
  if (!dtype_ok(dtype))
    return fail(SX_E_DIM_002, "matrix-scan: a and b must be f32 or bf16 (dtype code %d)", enum_code(dtype));
  if (!dtype_ok(out_dtype))
    return fail(SX_E_DIM_002, "matrix-scan: out must be f32 or bf16 (dtype code %d)", enum_code(out_dtype));
  sx::MsParams p;
  int64_t shp[sx::kMaxRank + 2];
  int r = 0;
  int64_t numel = 0;
  sx_status st = plan_matrix_scan(a_rank, a_shape, a_strides, b_rank, b_shape, b_strides, axis, &p, shp, &r, &numel);
  if (st != SX_OK) return st;
  if (numel == 0) return ok();
  if (!a) return fail(SX_E_DIM_003, "matrix-scan: a %s %s is NULL; a tensor was expected",
                      shape_str(a_rank, a_shape).c_str(), dtype_name(dtype));
  if (!b) return fail(SX_E_DIM_003, "matrix-scan: b %s %s is NULL; a tensor was expected",
                      shape_str(b_rank, b_shape).c_str(), dtype_name(dtype));
  if (!out) return fail(SX_E_DIM_003, "matrix-scan: out is NULL; a tensor was expected");

  const size_t esz = dtype == SX_BF16 ? 2 : 4, osz = out_dtype == SX_BF16 ? 2 : 4;
  int64_t ast[sx::kMaxRank], bst[sx::kMaxRank];
  if (a_strides) std::copy(a_strides, a_strides + a_rank, ast); else contiguous_strides(a_rank, a_shape, ast);
  if (b_strides) std::copy(b_strides, b_strides + b_rank, bst); else contiguous_strides(b_rank, b_shape, bst);
  uintptr_t olo = reinterpret_cast<uintptr_t>(out), ohi = olo + uintptr_t(numel) * osz, lo, hi;
  int64_t anumel = 0, bnumel = 0;
  checked_numel(a_rank, a_shape, &anumel);
  checked_numel(b_rank, b_shape, &bnumel);
  if (anumel > 0) {
    span_bytes(a, a_rank, a_shape, ast, esz, &lo, &hi);
    if (overlaps(olo, ohi, lo, hi)) return fail(SX_E_ALIAS, "matrix-scan: out overlaps a");
  }
  if (bnumel > 0) {
    span_bytes(b, b_rank, b_shape, bst, esz, &lo, &hi);
    if (overlaps(olo, ohi, lo, hi)) return fail(SX_E_ALIAS, "matrix-scan: out overlaps b");
  }
  const size_t need = sx::matrix_scan_workspace(p);
  if (scratch) {
    if (need > sx::kMatrixScanScratchBytes)
      return fail(SX_E_WORKSPACE,
                  "matrix-scan: a %s by %s scan needs %zu bytes of look-back state, more than the %zu bytes the "
                  "allocation-free entry point keeps; use sx_matrix_scan with a workspace",
                  shape_str(a_rank, a_shape).c_str(), shape_str(b_rank, b_shape).c_str(), need,
                  sx::kMatrixScanScratchBytes);
    workspace_bytes = sx::kMatrixScanScratchBytes;
    workspace = nullptr;
    if (need > 0) {
      const hipError_t e = sx::matrix_scan_scratch(&workspace);
      if (e != hipSuccess) return device_status(e, "matrix-scan: setting up the scratch array");
    }
  }
  if (need > 0 && (workspace == nullptr || workspace_bytes < need))
    return fail(SX_E_WORKSPACE, "matrix-scan: workspace of %zu bytes given, %zu needed", workspace_bytes, need);
  if (need > 0 && (reinterpret_cast<uintptr_t>(workspace) & 255u) != 0)
    return fail(SX_E_WORKSPACE, "matrix-scan: workspace must be 256-byte aligned");
  if (projective) {
    p.in_bf16 = dtype == SX_BF16;
    p.out_bf16 = out_dtype == SX_BF16;
    p.reverse = reverse ? 1 : 0;
    p.a = a;
    p.b = b;
    p.out = out;
    return device_status(
        sx::launch_matrix_scan_projective(p, workspace, workspace_bytes, static_cast<hipStream_t>(stream)),
        "matrix-scan :projective launch");
  }

  p.in_bf16 = dtype == SX_BF16;
  p.out_bf16 = out_dtype == SX_BF16;
  p.reverse = reverse ? 1 : 0;
  p.a = a;
  p.b = b;
  p.out = out;
  return device_status(sx::launch_matrix_scan(p, workspace, workspace_bytes, static_cast<hipStream_t>(stream)),
                       "matrix-scan launch");
}

}  // namespace

extern "C" {

sx_status sx_matrix_scan(sx_dtype dtype, int a_rank, const int64_t* a_shape, const int64_t* a_strides, const void* a,
                         int b_rank, const int64_t* b_shape, const int64_t* b_strides, const void* b, int axis,
                         int reverse, int projective, sx_dtype out_dtype, void* out, void* workspace,
                         size_t workspace_bytes, void* stream) {
  return matrix_scan_call(dtype, a_rank, a_shape, a_strides, a, b_rank, b_shape, b_strides, b, axis, reverse,
                          projective, out_dtype, out, workspace, workspace_bytes, stream, false);
}

sx_status sx_matrix_scan_noalloc(sx_dtype dtype, int a_rank, const int64_t* a_shape, const int64_t* a_strides,
                                 const void* a, int b_rank, const int64_t* b_shape, const int64_t* b_strides,
                                 const void* b, int axis, int reverse, int projective, sx_dtype out_dtype, void* out,
                                 void* stream) {
  return matrix_scan_call(dtype, a_rank, a_shape, a_strides, a, b_rank, b_shape, b_strides, b, axis, reverse,
                          projective, out_dtype, out, nullptr, 0, stream, true);
}

sx_status sx_matrix_scan_workspace_status(void* workspace, size_t workspace_bytes, void* stream) {
  if (workspace == nullptr)
    return fail(SX_E_DIM_003, "matrix-scan workspace status: the workspace is NULL; a buffer was expected");
  if (workspace_bytes < 256)
    return fail(SX_E_WORKSPACE, "matrix-scan workspace status: %zu bytes is smaller than a workspace header (256)",
                workspace_bytes);
  hipStream_t s = static_cast<hipStream_t>(stream);
  char* word = static_cast<char*>(workspace) + sx::kMatrixScanStatusOffset;
  uint32_t status = 0;
  hipError_t e = hipMemcpyAsync(&status, word, sizeof status, hipMemcpyDeviceToHost, s);
  if (e == hipSuccess) e = hipStreamSynchronize(s);
  if (e != hipSuccess) return device_status(e, "matrix-scan workspace status: reading the status word");
  if (status == 0) return ok();
  static const uint32_t zero = 0;
  e = hipMemcpyAsync(word, &zero, sizeof zero, hipMemcpyHostToDevice, s);
  if (e == hipSuccess) e = hipStreamSynchronize(s);
  if (e != hipSuccess) return device_status(e, "matrix-scan workspace status: clearing the status word");
  return fail(SX_E_DEVICE,
              "matrix-scan: a look-back gave up waiting for an earlier unit's published state (spin limit reached); "
              "results of the calls on this workspace since its last check are not valid");
}

void sx_set_lookback_spin_limit(uint32_t limit) { sx::set_lookback_spin_limit(limit); }

}  // extern "C"

// ------------------------------------------------------------------ matrix-scan gradient

namespace {

constexpr size_t kAlign = 256;
size_t align_up(size_t x) { return (x + kAlign - 1) / kAlign * kAlign; }

// Sum of a contiguous full-shape f32 tensor (rank R) down to a target shape
// (right-aligned, each dim equal or 1): which dims are kept, which summed.
sx::SumToParams sum_to_plan(int R, const int64_t* full, int t_rank, const int64_t* tshape) {
  sx::SumToParams q{};
  int64_t fst[sx::kMaxRank + 2];
  contiguous_strides(R, full, fst);
  q.targets = 1;
  q.reduced = 1;
  for (int d = 0; d < R; ++d) {
    const int e = d - (R - t_rank);
    const bool summed = e < 0 || (tshape[e] == 1 && full[d] != 1);
    if (summed) {
      q.red_dim[q.nd_red] = full[d];
      q.red_st[q.nd_red++] = fst[d];
      q.reduced *= full[d];
    } else {
      q.keep_dim[q.nd_keep] = full[d];
      q.keep_st[q.nd_keep++] = fst[d];
      q.targets *= full[d];
    }
  }
  // slices of the summed space: at least 32 terms each, at most 64 MiB of partial sums
  int64_t splits = std::max<int64_t>(1, std::min<int64_t>(65535, q.reduced / 32));
  if (q.targets > 0) splits = std::max<int64_t>(1, std::min<int64_t>(splits, (int64_t(64) << 20) / 4 / q.targets));
  q.splits = splits;
  q.per = (q.reduced + splits - 1) / splits;
  return q;
}

bool same_shape(int r1, const int64_t* s1, int r2, const int64_t* s2) {
  if (r1 != r2) return false;
  for (int i = 0; i < r1; ++i)
    if (s1[i] != s2[i]) return false;
  return true;
}

struct MsBackPlan {
  sx::MsParams p;                       // the adjoint scan (b = g, out = lam)
  int out_rank;
  int64_t out_shape[sx::kMaxRank + 2];  // lead + [n, m]
  int64_t out_numel, a_full_numel;
  bool lam_direct, ga_direct;           // lam is grad_b itself (f32, or rounded to a bf16 grad_b); grad_a in place
  sx::SumToParams sum_a, sum_b;
  size_t scan_ws, lam_off, ga_off, part_off, total;
};

sx_status plan_matrix_scan_backward(int a_rank, const int64_t* a_shape, const int64_t* a_strides, int b_rank,
                                    const int64_t* b_shape, const int64_t* g_strides, int axis, MsBackPlan* bp) {
  sx::MsParams fwd;
  int64_t numel = 0;
  sx_status st = plan_matrix_scan(a_rank, a_shape, nullptr, b_rank, b_shape, nullptr, axis, &fwd, bp->out_shape,
                                  &bp->out_rank, &numel);
  if (st != SX_OK) return st;
  // the adjoint scan: a as given, the gradient of the result in b's place
  int r = 0;
  int64_t shp[sx::kMaxRank + 2];
  st = plan_matrix_scan(a_rank, a_shape, a_strides, bp->out_rank, bp->out_shape, g_strides, axis, &bp->p, shp, &r,
                        &bp->out_numel);
  if (st != SX_OK) return st;
  const int L = bp->out_rank - 2;
  const int64_t n = bp->out_shape[L];
  int64_t afull[sx::kMaxRank + 2];
  std::copy(bp->out_shape, bp->out_shape + L, afull);
  afull[L] = afull[L + 1] = n;
  checked_numel(L + 2, afull, &bp->a_full_numel);
  // with b at the result's shape, the scan writes lam straight into grad_b: in f32, or rounded to
  // bf16 when the gradients are bf16 (grad_a then forms lam h^T from the rounded lam)
  bp->lam_direct = same_shape(b_rank, b_shape, bp->out_rank, bp->out_shape);
  bp->ga_direct = same_shape(a_rank, a_shape, L + 2, afull);
  bp->sum_a = sum_to_plan(L + 2, afull, a_rank, a_shape);
  bp->sum_b = sum_to_plan(bp->out_rank, bp->out_shape, b_rank, b_shape);
  bp->scan_ws = align_up(sx::matrix_scan_workspace(bp->p));
  size_t off = bp->scan_ws;
  bp->lam_off = off;
  if (!bp->lam_direct) off += align_up(size_t(bp->out_numel) * 4);
  bp->ga_off = off;
  if (!bp->ga_direct) off += align_up(size_t(bp->a_full_numel) * 4);
  bp->part_off = off;
  size_t part = 0;
  if (!bp->ga_direct) part = std::max(part, size_t(bp->sum_a.splits * bp->sum_a.targets) * 4);
  if (!same_shape(b_rank, b_shape, bp->out_rank, bp->out_shape))
    part = std::max(part, size_t(bp->sum_b.splits * bp->sum_b.targets) * 4);
  bp->total = off + align_up(part);
  return ok();
}

}  // namespace

extern "C" {

size_t sx_matrix_scan_backward_workspace_bytes(int a_rank, const int64_t* a_shape, int b_rank, const int64_t* b_shape,
                                               int axis, sx_dtype grad_dtype) {
  MsBackPlan bp;
  if (!dtype_ok(grad_dtype)) return 0;
  if (plan_matrix_scan_backward(a_rank, a_shape, nullptr, b_rank, b_shape, nullptr, axis, &bp) != SX_OK) return 0;
  return bp.total;
}

sx_status sx_matrix_scan_backward(sx_dtype dtype, int a_rank, const int64_t* a_shape, const int64_t* a_strides,
                                  const void* a, int b_rank, const int64_t* b_shape, const void* h,
                                  const int64_t* g_strides, const void* g, int axis, int reverse, sx_dtype grad_dtype,
                                  void* grad_a, void* grad_b, void* workspace, size_t workspace_bytes, void* stream) {
  if (!dtype_ok(dtype))
    return fail(SX_E_DIM_002, "matrix-scan gradient: a, h and g must be f32 or bf16 (dtype code %d)", enum_code(dtype));
  if (!dtype_ok(grad_dtype))
    return fail(SX_E_DIM_002, "matrix-scan gradient: gradients must be f32 or bf16 (dtype code %d)", enum_code(grad_dtype));
  MsBackPlan bp;
  sx_status st = plan_matrix_scan_backward(a_rank, a_shape, a_strides, b_rank, b_shape, g_strides, axis, &bp);
  if (st != SX_OK) return st;
  int64_t a_numel = 0, b_numel = 0;
  checked_numel(a_rank, a_shape, &a_numel);
  checked_numel(b_rank, b_shape, &b_numel);
  if (a_numel == 0 && b_numel == 0) return ok();
  if (bp.out_numel > 0 || bp.a_full_numel > 0) {
    if (!a) return fail(SX_E_DIM_003, "matrix-scan gradient: a %s %s is NULL; a tensor was expected",
                        shape_str(a_rank, a_shape).c_str(), dtype_name(dtype));
  }
  if (bp.out_numel > 0) {
    if (!h) return fail(SX_E_DIM_003, "matrix-scan gradient: the forward result h %s is NULL; a tensor was expected",
                        shape_str(bp.out_rank, bp.out_shape).c_str());
    if (!g) return fail(SX_E_DIM_003, "matrix-scan gradient: the result's gradient g %s is NULL; a tensor was expected",
                        shape_str(bp.out_rank, bp.out_shape).c_str());
  }
  if (a_numel > 0 && !grad_a) return fail(SX_E_DIM_003, "matrix-scan gradient: grad_a is NULL; a tensor was expected");
  if (b_numel > 0 && !grad_b) return fail(SX_E_DIM_003, "matrix-scan gradient: grad_b is NULL; a tensor was expected");

  // outputs overlap no input and not each other
  const size_t esz = dtype == SX_BF16 ? 2 : 4, gsz = grad_dtype == SX_BF16 ? 2 : 4;
  int64_t ast[sx::kMaxRank], gst[sx::kMaxRank + 2], ost[sx::kMaxRank + 2];
  if (a_strides) std::copy(a_strides, a_strides + a_rank, ast); else contiguous_strides(a_rank, a_shape, ast);
  contiguous_strides(bp.out_rank, bp.out_shape, ost);
  if (g_strides) std::copy(g_strides, g_strides + bp.out_rank, gst); else std::copy(ost, ost + bp.out_rank, gst);
  struct Span { uintptr_t lo, hi; const char* name; };
  Span ins[3];
  int nin = 0;
  uintptr_t lo, hi;
  if (a_numel > 0) { span_bytes(a, a_rank, a_shape, ast, esz, &lo, &hi); ins[nin++] = {lo, hi, "a"}; }
  if (bp.out_numel > 0) {
    span_bytes(h, bp.out_rank, bp.out_shape, ost, esz, &lo, &hi); ins[nin++] = {lo, hi, "h"};
    span_bytes(g, bp.out_rank, bp.out_shape, gst, esz, &lo, &hi); ins[nin++] = {lo, hi, "g"};
  }
  const uintptr_t galo = reinterpret_cast<uintptr_t>(grad_a), gahi = galo + uintptr_t(a_numel) * gsz;
  const uintptr_t gblo = reinterpret_cast<uintptr_t>(grad_b), gbhi = gblo + uintptr_t(b_numel) * gsz;
  for (int i = 0; i < nin; ++i) {
    if (a_numel > 0 && overlaps(galo, gahi, ins[i].lo, ins[i].hi))
      return fail(SX_E_ALIAS, "matrix-scan gradient: grad_a overlaps %s", ins[i].name);
    if (b_numel > 0 && overlaps(gblo, gbhi, ins[i].lo, ins[i].hi))
      return fail(SX_E_ALIAS, "matrix-scan gradient: grad_b overlaps %s", ins[i].name);
  }
  if (a_numel > 0 && b_numel > 0 && overlaps(galo, gahi, gblo, gbhi))
    return fail(SX_E_ALIAS, "matrix-scan gradient: grad_a overlaps grad_b");
  if (bp.total > 0 && (workspace == nullptr || workspace_bytes < bp.total))
    return fail(SX_E_WORKSPACE, "matrix-scan gradient: workspace of %zu bytes given, %zu needed", workspace_bytes,
                bp.total);
  if (bp.total > 0 && (reinterpret_cast<uintptr_t>(workspace) & 255u) != 0)
    return fail(SX_E_WORKSPACE, "matrix-scan gradient: workspace must be 256-byte aligned");

  hipStream_t s = static_cast<hipStream_t>(stream);
  char* ws = static_cast<char*>(workspace);
  void* lam = bp.lam_direct ? grad_b : static_cast<void*>(ws + bp.lam_off);
  const bool lam_bf16 = bp.lam_direct && grad_dtype == SX_BF16;
  // 1. the adjoint: the scan in the other direction over g, on a transposed and shifted a step
  bp.p.in_bf16 = dtype == SX_BF16;
  bp.p.out_bf16 = lam_bf16 ? 1 : 0;
  bp.p.reverse = reverse ? 0 : 1;
  bp.p.adjoint = 1;
  bp.p.a = a;
  bp.p.b = g;
  bp.p.out = lam;
  // f32 with grad_a at a's full shape: the pipelined adjoint scan forms grad_a in its replay
  bool folded = false;
  if (dtype == SX_F32 && grad_dtype == SX_F32 && bp.ga_direct && a_numel > 0 && bp.out_numel > 0) {
    bp.p.fold_h = h;
    bp.p.fold_grad_a = grad_a;
    folded = sx::matrix_scan_folds_grad_a(bp.p, ws, bp.scan_ws);
    if (!folded) bp.p.fold_h = bp.p.fold_grad_a = nullptr;
  }
  hipError_t e = sx::launch_matrix_scan(bp.p, ws, bp.scan_ws, s);
  if (e != hipSuccess) return device_status(e, "matrix-scan gradient: adjoint scan launch");
  // 2. grad_a = lam h[prev]^T per step (and grad_b = lam rounded, when that is all grad_b is), unless
  // the scan formed it (f32 gradients: grad_b is lam itself, at the result's shape or summed below)
  const int L = bp.out_rank - 2;
  const int ax = axis < 0 ? axis + L : axis;
  sx::GradAParams gp{};
  gp.steps = bp.out_numel > 0 ? bp.out_numel / (bp.out_shape[L] * bp.out_shape[L + 1])
                              : (bp.a_full_numel > 0 ? bp.a_full_numel / (bp.out_shape[L] * bp.out_shape[L]) : 0);
  gp.T = bp.out_shape[ax];
  gp.inner = 1;
  for (int i = ax + 1; i < L; ++i) gp.inner *= bp.out_shape[i];
  gp.n = int(bp.out_shape[L]);
  gp.m = int(bp.out_shape[L + 1]);
  gp.reverse = reverse ? 1 : 0;
  gp.lam = lam;
  gp.lam_bf16 = lam_bf16 ? 1 : 0;
  gp.h = h;
  gp.grad_a = bp.ga_direct ? grad_a : static_cast<void*>(ws + bp.ga_off);
  const bool b_full = same_shape(b_rank, b_shape, bp.out_rank, bp.out_shape);
  gp.grad_b = (b_full && !bp.lam_direct) ? grad_b : nullptr;
  if (!folded) {
    e = sx::launch_grad_a(gp, dtype == SX_BF16, grad_dtype == SX_BF16 && bp.ga_direct, s);
    if (e != hipSuccess) return device_status(e, "matrix-scan gradient: grad_a launch");
  }
  // 3. sums over broadcast dims
  if (!bp.ga_direct && a_numel > 0) {
    bp.sum_a.src = reinterpret_cast<const float*>(ws + bp.ga_off);
    bp.sum_a.partial = reinterpret_cast<float*>(ws + bp.part_off);
    e = sx::launch_sum_to(bp.sum_a, grad_a, grad_dtype == SX_BF16, s);
    if (e != hipSuccess) return device_status(e, "matrix-scan gradient: grad_a sum launch");
  }
  if (!b_full && b_numel > 0) {
    bp.sum_b.src = static_cast<const float*>(lam);
    bp.sum_b.partial = reinterpret_cast<float*>(ws + bp.part_off);
    e = sx::launch_sum_to(bp.sum_b, grad_b, grad_dtype == SX_BF16, s);
    if (e != hipSuccess) return device_status(e, "matrix-scan gradient: grad_b sum launch");
  }
  return ok();
}

// ------------------------------------------------------------------ element-scan gradient

size_t sx_element_scan_backward_workspace_bytes(sx_body body, int rank, const int64_t* shape, int axis, int state_axis,
                                                int64_t x_width, int64_t s_width) {
  if (!body_ok(body)) return 0;
  EsPlan plan;
  if (plan_element_scan(body, rank, shape, axis, state_axis, nullptr, x_width, nullptr, s_width, nullptr, &plan) !=
      SX_OK)
    return 0;
  const bool vec = state_axis != SX_STATE_SCALAR;
  const int64_t n = vec ? shape[rank - 1] : 1;
  size_t total = 0, part = 0;
  int64_t seq[sx::kMaxRank];
  std::copy(shape, shape + rank, seq);
  for (int64_t w : {x_width, s_width}) {
    if (!vec || w != 1 || n == 1 || body == SX_BODY_NORM_CAP) continue;  // norm-cap sums in its kernels
    total += align_up(size_t(plan.numel) * 4);  // the full-width gradient before its sum over the state
    seq[rank - 1] = 1;
    const sx::SumToParams q = sum_to_plan(rank, shape, rank, seq);
    part = std::max(part, size_t(q.splits * q.targets) * 4);
  }
  // per-lane bounds of the norm-cap gradient's split along the axis
  const size_t bounds = size_t(sx::element_scan_backward_bound_words(body, plan.p)) * 4;
  return total + align_up(part) + align_up(bounds);
}

sx_status sx_element_scan_backward(sx_body body, int rank, const int64_t* shape, int axis, int state_axis, int reverse,
                                   const float* initial, const float* x, int64_t x_width, const int64_t* x_strides,
                                   const float* s, int64_t s_width, const int64_t* s_strides, const float* h,
                                   const float* g, float* grad_initial, float* grad_x, float* grad_s, void* workspace,
                                   size_t workspace_bytes, void* stream) {
  if (!body_ok(body)) return fail(SX_E_UNSUPPORTED, "element-scan gradient: unknown body %d", enum_code(body));
  EsPlan plan;
  sx_status st = plan_element_scan(body, rank, shape, axis, state_axis, nullptr, x_width, x_strides, s_width,
                                   s_strides, &plan);
  if (st != SX_OK) return st;
  if (plan.numel == 0) return ok();
  const char* what[] = {"initial", "sequence x", "the second sequence", "the forward result h",
                        "the result's gradient g", "grad_initial", "grad_x", "grad_s"};
  const void* ptrs[] = {initial, x, s, h, g, grad_initial, grad_x, grad_s};
  for (int i = 0; i < 8; ++i)
    if (!ptrs[i]) return fail(SX_E_DIM_003, "element-scan gradient: %s is NULL; a tensor was expected", what[i]);
  const bool vec = state_axis != SX_STATE_SCALAR;
  const int64_t n = vec ? shape[rank - 1] : 1;
  const int ax = axis < 0 ? axis + rank : axis;

  // byte spans: inputs, then outputs (initial, h, g and every gradient are contiguous)
  int64_t xshape[sx::kMaxRank], sshape[sx::kMaxRank], ishape[sx::kMaxRank], xs[sx::kMaxRank], ss[sx::kMaxRank];
  int64_t is[sx::kMaxRank], os[sx::kMaxRank];
  for (int i = 0; i < rank; ++i) xshape[i] = sshape[i] = shape[i];
  if (vec) { xshape[rank - 1] = x_width; sshape[rank - 1] = s_width; }
  int64_t inumel = 1;
  for (int i = 0, j = 0; i < rank; ++i)
    if (i != ax) inumel *= (ishape[j++] = shape[i]);
  if (x_strides) std::copy(x_strides, x_strides + rank, xs); else contiguous_strides(rank, xshape, xs);
  if (s_strides) std::copy(s_strides, s_strides + rank, ss); else contiguous_strides(rank, sshape, ss);
  contiguous_strides(rank - 1, ishape, is);
  contiguous_strides(rank, shape, os);
  int64_t xn = 0, sn = 0;
  checked_numel(rank, xshape, &xn);
  checked_numel(rank, sshape, &sn);
  uintptr_t lo[8], hi[8];
  span_bytes(initial, rank - 1, ishape, is, 4, &lo[0], &hi[0]);
  span_bytes(x, rank, xshape, xs, 4, &lo[1], &hi[1]);
  span_bytes(s, rank, sshape, ss, 4, &lo[2], &hi[2]);
  span_bytes(h, rank, shape, os, 4, &lo[3], &hi[3]);
  span_bytes(g, rank, shape, os, 4, &lo[4], &hi[4]);
  lo[5] = reinterpret_cast<uintptr_t>(grad_initial); hi[5] = lo[5] + uintptr_t(inumel) * 4;
  lo[6] = reinterpret_cast<uintptr_t>(grad_x); hi[6] = lo[6] + uintptr_t(xn) * 4;
  lo[7] = reinterpret_cast<uintptr_t>(grad_s); hi[7] = lo[7] + uintptr_t(sn) * 4;
  for (int o = 5; o < 8; ++o)
    for (int i = 0; i < o; ++i)
      if (overlaps(lo[o], hi[o], lo[i], hi[i]))
        return fail(SX_E_ALIAS, "element-scan gradient: %s overlaps %s", what[o], what[i]);

  // width-one sequences under a vector state: norm-cap's kernels sum their gradients over the
  // state; for the other bodies a full-width gradient goes to the workspace and is summed after
  const bool fused = body == SX_BODY_NORM_CAP;
  const bool x_one = vec && x_width == 1 && n > 1, s_one = vec && s_width == 1 && n > 1;
  const bool x_sum = x_one && !fused, s_sum = s_one && !fused;
  const size_t need = sx_element_scan_backward_workspace_bytes(body, rank, shape, axis, state_axis, x_width, s_width);
  if (need > 0 && (workspace == nullptr || workspace_bytes < need))
    return fail(SX_E_WORKSPACE, "element-scan gradient: workspace of %zu bytes given, %zu needed", workspace_bytes,
                need);
  if (need > 0 && (reinterpret_cast<uintptr_t>(workspace) & 255u) != 0)
    return fail(SX_E_WORKSPACE, "element-scan gradient: workspace must be 256-byte aligned");
  char* ws = static_cast<char*>(workspace);
  const size_t full = align_up(size_t(plan.numel) * 4);
  float* gx_full = x_sum ? reinterpret_cast<float*>(ws) : grad_x;
  float* gs_full = s_sum ? reinterpret_cast<float*>(ws + (x_sum ? full : 0)) : grad_s;
  float* part = reinterpret_cast<float*>(ws + (x_sum ? full : 0) + (s_sum ? full : 0));
  const size_t bounds_bytes = size_t(sx::element_scan_backward_bound_words(body, plan.p)) * 4;
  float* bounds = bounds_bytes > 0 ? reinterpret_cast<float*>(ws + need - align_up(bounds_bytes)) : nullptr;

  hipStream_t hs = static_cast<hipStream_t>(stream);
  sx::EsVjpParams v{};
  v.p = plan.p;
  v.p.reverse = reverse ? 1 : 0;
  v.p.x = x;
  v.p.s = s;
  v.p.init = initial;
  v.p.out = nullptr;
  v.h = h;
  v.g = g;
  v.gx = gx_full;
  v.gs = gs_full;
  v.ginit = grad_initial;
  v.gx_sum = x_one && fused;
  v.gs_sum = s_one && fused;
  v.bounds = bounds;
  hipError_t e = sx::launch_element_scan_backward(body, v, hs);
  if (e != hipSuccess) return device_status(e, "element-scan gradient launch");
  int64_t seq[sx::kMaxRank];
  std::copy(shape, shape + rank, seq);
  seq[rank - 1] = 1;
  for (int which = 0; which < 2; ++which) {
    if (!(which == 0 ? x_sum : s_sum)) continue;
    sx::SumToParams q = sum_to_plan(rank, shape, rank, seq);
    q.src = which == 0 ? gx_full : gs_full;
    q.partial = part;
    e = sx::launch_sum_to(q, which == 0 ? static_cast<void*>(grad_x) : static_cast<void*>(grad_s), false, hs);
    if (e != hipSuccess) return device_status(e, "element-scan gradient: sum over the state launch");
  }
  return ok();
}

// ------------------------------------------------------------------ table-scan

sx_status sx_table_scan(int states, int nsym, const int32_t* table, int rank, const int64_t* shape,
                        const int64_t* strides, const int32_t* symbols, int axis, int32_t start, int32_t* out,
                        void* stream) {
  if (states < 1 || nsym < 1)
    return fail(SX_E_DIM_001, "table-scan: the table is [states symbols] with at least one of each, got [%d %d]",
                states, nsym);
  if (rank > sx::kMaxRank) return fail(SX_E_UNSUPPORTED, "table-scan: rank %d exceeds %d", rank, sx::kMaxRank);
  if (rank < 1 || shape == nullptr) return fail(SX_E_DIM_001, "table-scan: symbols need at least one axis");
  int64_t numel = 0;
  if (!checked_numel(rank, shape, &numel))
    return fail(SX_E_DIM_001, "table-scan: bad symbols shape %s", shape_str(rank, shape).c_str());
  const int ax = axis < 0 ? axis + rank : axis;
  if (ax < 0 || ax >= rank)
    return fail(SX_E_DIM_001, "table-scan: axis %d out of range for symbols %s :i32", axis,
                shape_str(rank, shape).c_str());
  if (start < 0 || start >= states)
    return fail(SX_E_DIM_001, "table-scan: :start %d is not a state of a [%d %d] table", int(start), states, nsym);
  if (numel == 0) return ok();
  if (!table) return fail(SX_E_DIM_003, "table-scan: table is NULL; a tensor was expected");
  if (!symbols) return fail(SX_E_DIM_003, "table-scan: symbols is NULL; a tensor was expected");
  if (!out) return fail(SX_E_DIM_003, "table-scan: out is NULL; a tensor was expected");
  int64_t xs[sx::kMaxRank], os[sx::kMaxRank];
  if (strides) std::copy(strides, strides + rank, xs); else contiguous_strides(rank, shape, xs);
  contiguous_strides(rank, shape, os);
  uintptr_t lo, hi;
  const uintptr_t olo = reinterpret_cast<uintptr_t>(out), ohi = olo + uintptr_t(numel) * 4;
  span_bytes(symbols, rank, shape, xs, 4, &lo, &hi);
  if (overlaps(olo, ohi, lo, hi)) return fail(SX_E_ALIAS, "table-scan: out overlaps symbols");
  const uintptr_t tlo = reinterpret_cast<uintptr_t>(table), thi = tlo + uintptr_t(int64_t(states) * nsym) * 4;
  if (overlaps(olo, ohi, tlo, thi)) return fail(SX_E_ALIAS, "table-scan: out overlaps the table");

  sx::TsParams p{};
  p.T = shape[ax];
  p.t_stride[0] = xs[ax];
  p.t_stride[1] = os[ax];
  int64_t dims[sx::kMaxRank];
  int64_t st[2][sx::kMaxRank];
  int nd = 0;
  for (int i = 0; i < rank; ++i) {
    if (i == ax) continue;
    dims[nd] = shape[i];
    st[0][nd] = xs[i];
    st[1][nd] = os[i];
    ++nd;
  }
  p.seqs = make_index_map<2>(nd, dims, st);
  p.num_seq = numel / p.T;
  p.states = states;
  p.nsym = nsym;
  p.start = start;
  p.table = table;
  p.symbols = symbols;
  p.out = out;
  return device_status(sx::launch_table_scan(p, static_cast<hipStream_t>(stream)), "table-scan launch");
}

// ------------------------------------------------------------------ linear-scan

// a and b broadcast (NumPy: right-aligned, each dim equal or 1; rank 0 is a
// number) to the result shape; the scan runs along `axis` of that shape.
static sx_status plan_linear_scan(int a_rank, const int64_t* a_shape, const int64_t* a_strides, int b_rank,
                                  const int64_t* b_shape, const int64_t* b_strides, int axis, sx::EsParams* p,
                                  int64_t* out_shape, int* out_rank, int64_t* out_numel) {
  if (a_rank > sx::kMaxRank || b_rank > sx::kMaxRank)
    return fail(SX_E_UNSUPPORTED, "linear-scan: rank above %d", sx::kMaxRank);
  if (a_rank < 0 || b_rank < 0 || (a_rank > 0 && !a_shape) || (b_rank > 0 && !b_shape))
    return fail(SX_E_DIM_001, "linear-scan: invalid rank or missing shape");
  int64_t tmp;
  if (!checked_numel(a_rank, a_shape, &tmp) || !checked_numel(b_rank, b_shape, &tmp))
    return fail(SX_E_DIM_001, "linear-scan: negative or oversized dims in a %s, b %s",
                shape_str(a_rank, a_shape).c_str(), shape_str(b_rank, b_shape).c_str());
  const int L = std::max(a_rank, b_rank);
  if (L < 1)
    return fail(SX_E_DIM_001, "linear-scan: a and b are both numbers; there is no axis to scan along");
  int64_t shp[sx::kMaxRank], sa[sx::kMaxRank], sb[sx::kMaxRank];
  int64_t ast[sx::kMaxRank], bst[sx::kMaxRank];
  if (a_strides) std::copy(a_strides, a_strides + a_rank, ast); else contiguous_strides(a_rank, a_shape, ast);
  if (b_strides) std::copy(b_strides, b_strides + b_rank, bst); else contiguous_strides(b_rank, b_shape, bst);
  for (int i = 0; i < L; ++i) {
    const int ia = i - (L - a_rank), ib = i - (L - b_rank);
    const int64_t da = ia >= 0 ? a_shape[ia] : 1, db = ib >= 0 ? b_shape[ib] : 1;
    if (da != db && da != 1 && db != 1)
      return fail(SX_E_DIM_001, "linear-scan: a %s and b %s do not broadcast", shape_str(a_rank, a_shape).c_str(),
                  shape_str(b_rank, b_shape).c_str());
    shp[i] = da == 1 ? db : da;
    sa[i] = (ia >= 0 && da != 1) ? ast[ia] : 0;
    sb[i] = (ib >= 0 && db != 1) ? bst[ib] : 0;
  }
  const int ax = axis < 0 ? axis + L : axis;
  if (ax < 0 || ax >= L)
    return fail(SX_E_DIM_001, "linear-scan: axis %d out of range for shape %s", axis, shape_str(L, shp).c_str());
  int64_t numel = 0;
  if (!checked_numel(L, shp, &numel)) return fail(SX_E_DIM_001, "linear-scan: result too large");
  std::copy(shp, shp + L, out_shape);
  *out_rank = L;
  *out_numel = numel;
  if (!p) return ok();

  int64_t ost[sx::kMaxRank];
  contiguous_strides(L, shp, ost);
  *p = sx::EsParams{};
  p->T = shp[ax];
  p->t_stride[sx::ES_X] = sb[ax];
  p->t_stride[sx::ES_S] = sa[ax];
  p->t_stride[sx::ES_OUT] = ost[ax];
  p->n = 1;
  int64_t dims[sx::kMaxRank];
  int64_t st[4][sx::kMaxRank];
  int nd = 0;
  for (int i = 0; i < L; ++i) {
    if (i == ax) continue;
    dims[nd] = shp[i];
    st[sx::ES_X][nd] = sb[i];
    st[sx::ES_S][nd] = sa[i];
    st[sx::ES_INIT][nd] = 0;
    st[sx::ES_OUT][nd] = ost[i];
    ++nd;
  }
  p->lanes = make_index_map<4>(nd, dims, st);
  p->num_lanes = p->T > 0 ? numel / p->T : 0;
  return ok();
}

int sx_linear_scan_out_shape(int a_rank, const int64_t* a_shape, int b_rank, const int64_t* b_shape,
                             int64_t* out_shape) {
  int64_t shp[sx::kMaxRank];
  int r = 0;
  int64_t numel = 0;
  if (plan_linear_scan(a_rank, a_shape, nullptr, b_rank, b_shape, nullptr, 0, nullptr, shp, &r, &numel) != SX_OK)
    return -1;
  if (out_shape) std::copy(shp, shp + r, out_shape);
  return r;
}

sx_status sx_linear_scan(sx_dtype dtype, int a_rank, const int64_t* a_shape, const int64_t* a_strides, const void* a,
                         int b_rank, const int64_t* b_shape, const int64_t* b_strides, const void* b, int axis,
                         int reverse, sx_dtype out_dtype, void* out, void* stream) {
  if (!dtype_ok(dtype))
    return fail(SX_E_DIM_002, "linear-scan: a and b must be f32 or bf16 (dtype code %d)", enum_code(dtype));
  if (!dtype_ok(out_dtype))
    return fail(SX_E_DIM_002, "linear-scan: out must be f32 or bf16 (dtype code %d)", enum_code(out_dtype));
  sx::EsParams p;
  int64_t shp[sx::kMaxRank];
  int r = 0;
  int64_t numel = 0;
  sx_status st = plan_linear_scan(a_rank, a_shape, a_strides, b_rank, b_shape, b_strides, axis, &p, shp, &r, &numel);
  if (st != SX_OK) return st;
  if (numel == 0) return ok();
  if (!a) return fail(SX_E_DIM_003, "linear-scan: a %s %s is NULL; a tensor was expected",
                      shape_str(a_rank, a_shape).c_str(), dtype_name(dtype));
  if (!b) return fail(SX_E_DIM_003, "linear-scan: b %s %s is NULL; a tensor was expected",
                      shape_str(b_rank, b_shape).c_str(), dtype_name(dtype));
  if (!out) return fail(SX_E_DIM_003, "linear-scan: out is NULL; a tensor was expected");

  const size_t esz = dtype == SX_BF16 ? 2 : 4, osz = out_dtype == SX_BF16 ? 2 : 4;
  int64_t ast[sx::kMaxRank], bst[sx::kMaxRank];
  if (a_strides) std::copy(a_strides, a_strides + a_rank, ast); else contiguous_strides(a_rank, a_shape, ast);
  if (b_strides) std::copy(b_strides, b_strides + b_rank, bst); else contiguous_strides(b_rank, b_shape, bst);
  uintptr_t olo = reinterpret_cast<uintptr_t>(out), ohi = olo + uintptr_t(numel) * osz, lo, hi;
  span_bytes(a, a_rank, a_shape, ast, esz, &lo, &hi);  // numel > 0: neither operand is empty
  if (overlaps(olo, ohi, lo, hi)) return fail(SX_E_ALIAS, "linear-scan: out overlaps a");
  span_bytes(b, b_rank, b_shape, bst, esz, &lo, &hi);
  if (overlaps(olo, ohi, lo, hi)) return fail(SX_E_ALIAS, "linear-scan: out overlaps b");

  p.reverse = reverse ? 1 : 0;
  p.x = static_cast<const float*>(b);  // element type chosen by launch_linear_scan
  p.s = static_cast<const float*>(a);
  p.init = nullptr;
  p.out = static_cast<float*>(out);
  return device_status(sx::launch_linear_scan(p, dtype == SX_BF16, out_dtype == SX_BF16,
                                              static_cast<hipStream_t>(stream)),
                       "linear-scan launch");
}

// ------------------------------------------------------------------ decay attention, head norm and rotation

}  // extern "C"

namespace {

constexpr int64_t kMostHeadWidth = 256;
constexpr int64_t kMostTokens = int64_t(1) << 30;
constexpr int64_t kMostGrid = (int64_t(1) << 31) - 1;

// A [B, T, heads, d] operand (a single token: T = 1).
struct HeadArg {
  const char* name;
  const int64_t* shape;    // [B, T, heads, d]
  const int64_t* strides;  // nullptr: contiguous
  const void* data;
};

sx_status missing(const char* op, const char* name) {
  return fail(SX_E_DIM_003, "%s: %s is NULL; a tensor was expected", op, name);
}

void head_strides(const HeadArg& a, int64_t* st) {
  if (a.strides) std::copy(a.strides, a.strides + 4, st); else contiguous_strides(4, a.shape, st);
}

sx::HeadView head_view(const HeadArg& a, size_t elem, int64_t heads) {
  int64_t st[4];
  head_strides(a, st);
  sx::HeadView v{};
  v.p = a.data;
  v.sb = st[0];
  v.st = st[1];
  v.sh = st[2];
  v.sd = st[3];
  v.rep = int(heads / std::max<int64_t>(a.shape[2], 1));
  v.unit = st[3] == 1 && a.shape[3] * int64_t(elem) >= 16;
  return v;
}

int64_t numel4(const int64_t* s) { return s[0] * s[1] * s[2] * s[3]; }

struct Span {
  const char* name;
  uintptr_t lo, hi;
  unsigned align = 16;  // of an output: bytes
};

Span head_span(const HeadArg& a, size_t elem) {
  Span s{a.name, 0, 0};
  if (!a.data || numel4(a.shape) == 0) return s;
  int64_t st[4];
  head_strides(a, st);
  span_bytes(a.data, 4, a.shape, st, elem, &s.lo, &s.hi);
  return s;
}

Span flat_span(const char* name, const void* p, int64_t bytes) {
  const uintptr_t b = reinterpret_cast<uintptr_t>(p);
  return p && bytes > 0 ? Span{name, b, b + uintptr_t(bytes)} : Span{name, 0, 0};
}

// Every output against every input and every other output.
sx_status no_overlap(const char* op, const Span* in, int nin, const Span* out, int nout) {
  for (int i = 0; i < nout; ++i) {
    for (int j = 0; j < nin; ++j)
      if (overlaps(out[i].lo, out[i].hi, in[j].lo, in[j].hi))
        return fail(SX_E_ALIAS, "%s: %s overlaps %s", op, out[i].name, in[j].name);
    for (int j = i + 1; j < nout; ++j)
      if (overlaps(out[i].lo, out[i].hi, out[j].lo, out[j].hi))
        return fail(SX_E_ALIAS, "%s: %s overlaps %s", op, out[i].name, out[j].name);
    if (out[i].lo % out[i].align != 0)
      return fail(SX_E_UNSUPPORTED, "%s: %s must be %u-byte aligned", op, out[i].name, out[i].align);
  }
  return ok();
}

struct DecayShapes {
  int64_t B, T, H, hq, hk, hv, dk, dv;
  int64_t gb, gt, gh;
};

// Shapes of q, k [B, T, *, dk], v [B, T, *, dv] and log_decay ([H] or [B, T, H]).
sx_status decay_shapes(const char* op, const HeadArg& q, const HeadArg& k, const HeadArg& v, int g_rank,
                       const int64_t* g_shape, const int64_t* g_strides, DecayShapes* s) {
  for (const HeadArg* a : {&q, &k, &v}) {
    int64_t n;
    if (!a->shape) return fail(SX_E_DIM_001, "%s: %s has no shape", op, a->name);
    if (!checked_numel(4, a->shape, &n))
      return fail(SX_E_DIM_001, "%s: bad shape %s of %s", op, shape_str(4, a->shape).c_str(), a->name);
  }
  if (!g_shape || (g_rank != 1 && g_rank != 3))
    return fail(SX_E_DIM_001, "%s: log_decay must be [heads] or [batch, tokens, heads]", op);
  s->B = q.shape[0];
  s->T = q.shape[1];
  s->H = g_shape[g_rank - 1];
  s->hq = q.shape[2];
  s->hk = k.shape[2];
  s->hv = v.shape[2];
  s->dk = q.shape[3];
  s->dv = v.shape[3];
  if (k.shape[0] != s->B || k.shape[1] != s->T || k.shape[3] != s->dk)
    return fail(SX_E_DIM_001, "%s: k %s does not fit q %s", op, shape_str(4, k.shape).c_str(),
                shape_str(4, q.shape).c_str());
  if (v.shape[0] != s->B || v.shape[1] != s->T)
    return fail(SX_E_DIM_001, "%s: v %s does not fit q %s", op, shape_str(4, v.shape).c_str(),
                shape_str(4, q.shape).c_str());
  if (g_rank == 3 && (g_shape[0] != s->B || g_shape[1] != s->T))
    return fail(SX_E_DIM_001, "%s: log_decay %s does not fit q %s", op, shape_str(3, g_shape).c_str(),
                shape_str(4, q.shape).c_str());
  if (s->H < 1) return fail(SX_E_DIM_001, "%s: log_decay %s has no heads", op, shape_str(g_rank, g_shape).c_str());
  for (const HeadArg* a : {&q, &k, &v})
    if (a->shape[2] < 1 || s->H % a->shape[2] != 0)
      return fail(SX_E_DIM_001, "%s: the %lld heads of %s do not divide the %lld of log_decay", op,
                  (long long)a->shape[2], a->name, (long long)s->H);
  if (s->dk < 1 || s->dv < 1) return fail(SX_E_DIM_001, "%s: heads of width 0 (q %s, v %s)", op,
                                          shape_str(4, q.shape).c_str(), shape_str(4, v.shape).c_str());
  if (s->dk > kMostHeadWidth || s->dv > kMostHeadWidth)
    return fail(SX_E_UNSUPPORTED, "%s: heads wider than %lld (q %s, v %s)", op, (long long)kMostHeadWidth,
                shape_str(4, q.shape).c_str(), shape_str(4, v.shape).c_str());
  if (s->T > kMostTokens || s->B > kMostTokens || s->H > kMostTokens || s->B * s->H > kMostGrid / 1024)
    return fail(SX_E_UNSUPPORTED, "%s: too many tokens, rows or heads (q %s)", op, shape_str(4, q.shape).c_str());
  int64_t st[3];
  if (g_strides) std::copy(g_strides, g_strides + g_rank, st); else contiguous_strides(g_rank, g_shape, st);
  s->gb = g_rank == 3 ? st[0] : 0;
  s->gt = g_rank == 3 ? st[1] : 0;
  s->gh = st[g_rank - 1];
  return ok();
}

Span decay_span(const DecayShapes& s, const float* g) {
  const int64_t shape[3] = {s.B, s.T, s.H}, st[3] = {s.gb, s.gt, s.gh};
  Span r{"log_decay", 0, 0};
  if (g && s.B * s.T * s.H > 0) span_bytes(g, 3, shape, st, sizeof(float), &r.lo, &r.hi);
  return r;
}

sx::DaParams decay_params(const DecayShapes& s, bool bf16, const float* g, const int32_t* lengths) {
  sx::DaParams p{};
  p.B = int(s.B);
  p.T = int(s.T);
  p.H = int(s.H);
  p.dk = int(s.dk);
  p.dv = int(s.dv);
  p.g = g;
  p.gb = s.gb;
  p.gt = s.gt;
  p.gh = s.gh;
  p.lengths = lengths;
  p.bf16 = bf16;
  sx::decay_attention_split(p);
  return p;
}

// Hands out 256-byte aligned pieces of a workspace; with base 0 it only adds them up.
struct Carve {
  uintptr_t base;
  size_t used = 0;
  template <typename T>
  T* take(int64_t n) {
    const size_t at = used;
    used += (size_t(n) * sizeof(T) + 255) & ~size_t(255);
    return n > 0 && base ? reinterpret_cast<T*>(base + at) : nullptr;
  }
};

void carve_segments(Carve& c, sx::DaParams& p, sx::DaMarch& m) {
  const int64_t n = int64_t(p.segments - 1) * p.B * p.H;
  m.seg = c.take<float>(n * p.dk * p.dv);
  m.seg_decay = c.take<float>(n);
}

struct GradPieces {
  float *rows, *sources, *rows_chunk, *sources_chunk, *chunk_decay;
  double *cross, *partial;
  float *share_q, *share_k, *share_v;
  int chunks, blocks;
};

GradPieces carve_gradient(Carve& c, const DecayShapes& s, sx::DaParams& p) {
  GradPieces g{};
  carve_segments(c, p, p.m[0]);
  carve_segments(c, p, p.m[1]);
  p.m[2].seg = p.m[1].seg;
  p.m[2].seg_decay = p.m[1].seg_decay;
  for (int i = 0; i < 2; ++i)
    p.m[i].marks = c.take<float>(s.B * s.H * p.segments * (p.spans - 1) * sx::mark_floats(p.dk, p.dv));
  const int chunk = sx::decay_attention_chunk(p.bf16 != 0);
  const int64_t BH = s.B * s.H;
  g.chunks = int((s.T + chunk - 1) / chunk);
  g.blocks = sx::decay_attention_column_blocks(p.dk);
  g.rows = c.take<float>(g.blocks * BH * s.T);
  g.sources = c.take<float>(g.blocks * BH * s.T);
  g.rows_chunk = c.take<float>(g.blocks * BH * g.chunks);
  g.sources_chunk = c.take<float>(g.blocks * BH * g.chunks);
  g.chunk_decay = c.take<float>(BH * g.chunks);
  g.cross = c.take<double>(g.blocks * BH * (int64_t(p.segments) * p.spans + 1));
  g.partial = c.take<double>(BH * p.segments * p.spans);
  // gradients of shared heads are summed over the heads that share them, from f32
  const int64_t n = s.B * s.T * s.H;
  g.share_q = c.take<float>(s.hq == s.H ? 0 : n * s.dk);
  g.share_k = c.take<float>(s.hk == s.H ? 0 : n * s.dk);
  g.share_v = c.take<float>(s.hv == s.H ? 0 : n * s.dv);
  return g;
}

sx_status check_workspace(const char* op, const void* workspace, size_t bytes, size_t need) {
  if (need > 0 && (workspace == nullptr || bytes < need))
    return fail(SX_E_WORKSPACE, "%s: workspace of %zu bytes given, %zu needed", op, bytes, need);
  if (need > 0 && (reinterpret_cast<uintptr_t>(workspace) & 255u) != 0)
    return fail(SX_E_WORKSPACE, "%s: workspace must be 256-byte aligned", op);
  return ok();
}

}  // namespace

extern "C" {

size_t sx_decay_attention_workspace_bytes(sx_dtype dtype, const int64_t* q_shape, const int64_t* v_shape,
                                          int64_t heads) {
  if (!dtype_ok(dtype)) return 0;
  const HeadArg q{"q", q_shape, nullptr, nullptr}, v{"v", v_shape, nullptr, nullptr};
  DecayShapes s;
  if (decay_shapes("decay-attention", q, q, v, 1, &heads, nullptr, &s) != SX_OK) return 0;
  sx::DaParams p = decay_params(s, dtype == SX_BF16, nullptr, nullptr);
  Carve c{0};
  carve_segments(c, p, p.m[0]);
  return c.used;
}

sx_status sx_decay_attention(sx_dtype dtype, const int64_t* q_shape, const int64_t* q_strides, const void* q,
                             const int64_t* k_shape, const int64_t* k_strides, const void* k, const int64_t* v_shape,
                             const int64_t* v_strides, const void* v, int g_rank, const int64_t* g_shape,
                             const int64_t* g_strides, const float* log_decay, const float* initial,
                             const int32_t* lengths, float scale, void* out, float* final_state, void* workspace,
                             size_t workspace_bytes, void* stream) {
  const char* op = "decay-attention";
  if (!dtype_ok(dtype))
    return fail(SX_E_DIM_002, "%s: q, k and v must be f32 or bf16 (dtype code %d)", op, enum_code(dtype));
  const HeadArg qa{"q", q_shape, q_strides, q}, ka{"k", k_shape, k_strides, k}, va{"v", v_shape, v_strides, v};
  DecayShapes s;
  sx_status st = decay_shapes(op, qa, ka, va, g_rank, g_shape, g_strides, &s);
  if (st != SX_OK) return st;
  const int64_t state = s.B * s.H * s.dk * s.dv, rows = s.B * s.T * s.H;
  if (s.B == 0 || (s.T == 0 && !final_state)) return ok();
  if (rows > 0) {
    for (const HeadArg* a : {&qa, &ka, &va})
      if (!a->data) return missing(op, a->name);
    if (!log_decay) return missing(op, "log_decay");
    if (!out) return missing(op, "out");
  }
  const size_t e = dtype == SX_BF16 ? 2 : 4;
  const Span in[] = {head_span(qa, e), head_span(ka, e), head_span(va, e), decay_span(s, log_decay),
                     flat_span("initial", initial, state * 4), flat_span("lengths", lengths, s.B * 4)};
  const Span to[] = {flat_span("out", out, rows * s.dv * int64_t(e)), flat_span("the final state", final_state, state * 4)};
  if ((st = no_overlap(op, in, 6, to, 2)) != SX_OK) return st;
  sx::DaParams p = decay_params(s, dtype == SX_BF16, log_decay, lengths);
  Carve c{reinterpret_cast<uintptr_t>(workspace)};
  sx::DaMarch& m = p.m[0];
  carve_segments(c, p, m);
  if ((st = check_workspace(op, workspace, workspace_bytes, c.used)) != SX_OK) return st;
  p.marches = 1;
  m.x = head_view(qa, e, s.H);
  m.y = head_view(ka, e, s.H);
  m.z = head_view(va, e, s.H);
  m.dx = p.dk;
  m.dz = p.dv;
  m.scale_out = scale;
  m.scale_src = 1.0f;
  m.out = out;
  m.sr = s.dv;
  m.sc = 1;
  m.first = initial;
  m.last = final_state;
  return device_status(sx::launch_decay_attention(p, static_cast<hipStream_t>(stream)), "decay-attention launch");
}

size_t sx_decay_attention_backward_workspace_bytes(sx_dtype dtype, const int64_t* q_shape, const int64_t* k_shape,
                                                   const int64_t* v_shape, int64_t heads) {
  if (!dtype_ok(dtype)) return 0;
  const HeadArg q{"q", q_shape, nullptr, nullptr}, k{"k", k_shape, nullptr, nullptr}, v{"v", v_shape, nullptr, nullptr};
  DecayShapes s;
  if (decay_shapes("decay-attention gradient", q, k, v, 1, &heads, nullptr, &s) != SX_OK) return 0;
  sx::DaParams p = decay_params(s, dtype == SX_BF16, nullptr, nullptr);
  Carve c{0};
  carve_gradient(c, s, p);
  return c.used;
}

sx_status sx_decay_attention_backward(sx_dtype dtype, const int64_t* q_shape, const int64_t* q_strides, const void* q,
                                      const int64_t* k_shape, const int64_t* k_strides, const void* k,
                                      const int64_t* v_shape, const int64_t* v_strides, const void* v, int g_rank,
                                      const int64_t* g_shape, const int64_t* g_strides, const float* log_decay,
                                      const int64_t* grad_out_strides, const void* grad_out, const float* grad_state,
                                      const float* initial, const int32_t* lengths, float scale, void* grad_q,
                                      void* grad_k, void* grad_v, float* grad_log_decay, float* grad_initial,
                                      void* workspace, size_t workspace_bytes, void* stream) {
  const char* op = "decay-attention gradient";
  if (!dtype_ok(dtype))
    return fail(SX_E_DIM_002, "%s: q, k, v and grad_out must be f32 or bf16 (dtype code %d)", op, enum_code(dtype));
  const HeadArg qa{"q", q_shape, q_strides, q}, ka{"k", k_shape, k_strides, k}, va{"v", v_shape, v_strides, v};
  DecayShapes s;
  sx_status st = decay_shapes(op, qa, ka, va, g_rank, g_shape, g_strides, &s);
  if (st != SX_OK) return st;
  const int64_t out_shape[4] = {s.B, s.T, s.H, s.dv};
  const HeadArg oa{"grad_out", out_shape, grad_out_strides, grad_out};
  const int64_t state = s.B * s.H * s.dk * s.dv, rows = s.B * s.T * s.H;
  if (rows > 0) {
    for (const HeadArg* a : {&qa, &ka, &va, &oa})
      if (!a->data) return missing(op, a->name);
    if (!log_decay) return missing(op, "log_decay");
    if (!grad_q) return missing(op, "grad_q");
    if (!grad_k) return missing(op, "grad_k");
    if (!grad_v) return missing(op, "grad_v");
  }
  if (!grad_log_decay && (rows > 0 || g_rank == 1)) return missing(op, "grad_log_decay");
  if (initial && !grad_initial && state > 0) return missing(op, "grad_initial");
  const size_t e = dtype == SX_BF16 ? 2 : 4;
  const Span in[] = {head_span(qa, e), head_span(ka, e), head_span(va, e), head_span(oa, e), decay_span(s, log_decay),
                     flat_span("initial", initial, state * 4), flat_span("grad_state", grad_state, state * 4),
                     flat_span("lengths", lengths, s.B * 4)};
  const Span to[] = {flat_span("grad_q", grad_q, numel4(q_shape) * int64_t(e)),
                     flat_span("grad_k", grad_k, numel4(k_shape) * int64_t(e)),
                     flat_span("grad_v", grad_v, numel4(v_shape) * int64_t(e)),
                     flat_span("grad_log_decay", grad_log_decay, (g_rank == 1 ? s.H : rows) * 4),
                     flat_span("grad_initial", grad_initial, state * 4)};
  if ((st = no_overlap(op, in, 8, to, 5)) != SX_OK) return st;
  sx::DaParams p = decay_params(s, dtype == SX_BF16, log_decay, lengths);
  Carve c{reinterpret_cast<uintptr_t>(workspace)};
  const GradPieces w = carve_gradient(c, s, p);
  if ((st = check_workspace(op, workspace, workspace_bytes, c.used)) != SX_OK) return st;

  const sx::HeadView qv = head_view(qa, e, s.H), kv = head_view(ka, e, s.H),
                     vv = head_view(va, e, s.H), ov = head_view(oa, e, s.H);
  p.marches = 3;
  sx::DaMarch &dq = p.m[0], &dk = p.m[1], &dv = p.m[2];
  dq.x = ov; dq.y = vv; dq.z = kv; dq.w = qv;
  dk.x = vv; dk.y = ov; dk.z = qv; dk.w = kv;
  dv.x = kv; dv.y = qv; dv.z = ov;
  dq.dx = dk.dx = p.dv;
  dq.dz = dk.dz = p.dk;
  dv.dx = p.dk;
  dv.dz = p.dv;
  dq.scale_out = scale;
  dq.scale_src = 1.0f;
  dk.scale_out = dv.scale_out = 1.0f;
  dk.scale_src = dv.scale_src = scale;
  dq.sr = dk.sr = 1;   // states are [dk, dv] in memory; these two hold them transposed
  dq.sc = dk.sc = s.dv;
  dv.sr = s.dv;
  dv.sc = 1;
  dq.first = initial;
  dk.first = dv.first = grad_state;
  dk.last = grad_initial;
  dq.out = w.share_q ? w.share_q : grad_q;
  dq.out_f32 = w.share_q != nullptr;
  dk.out = w.share_k ? w.share_k : grad_k;
  dk.out_f32 = w.share_k != nullptr;
  dv.out = w.share_v ? w.share_v : grad_v;
  dv.out_f32 = w.share_v != nullptr;
  dq.mass = w.rows;
  dq.mass_chunk = w.rows_chunk;
  dq.chunk_decay = w.chunk_decay;
  dq.cross = w.cross;
  dk.mass = w.sources;
  dk.mass_chunk = w.sources_chunk;
  const hipStream_t str = static_cast<hipStream_t>(stream);
  hipError_t err = hipSuccess;
  if (s.B > 0) {
    err = sx::launch_decay_attention(p, str);
    if (err != hipSuccess) return device_status(err, "decay-attention gradient launch");
    const struct { const float* src; void* to; int64_t heads, d; } shared[3] = {
        {w.share_q, grad_q, s.hq, s.dk}, {w.share_k, grad_k, s.hk, s.dk}, {w.share_v, grad_v, s.hv, s.dv}};
    sx::DaShares sums{};
    for (const auto& x : shared) {
      if (!x.src) continue;
      sx::DaShare& sh = sums.s[sums.count++];
      sh.src = x.src;
      sh.out = x.to;
      sh.rows = s.B * s.T * x.heads;
      sh.rep = int(s.H / x.heads);
      sh.d = int(x.d);
      sh.bf16 = p.bf16;
    }
    err = sx::launch_share_sums(sums, str);
    if (err != hipSuccess) return device_status(err, "decay-attention gradient launch");
  }
  sx::DaDecayGrad d{};
  d.B = p.B;
  d.T = p.T;
  d.H = p.H;
  d.dk = p.dk;
  d.dv = p.dv;
  d.chunk = sx::decay_attention_chunk(p.bf16 != 0);
  d.chunks = w.chunks;
  d.blocks = w.blocks;
  d.g = log_decay;
  d.gb = s.gb;
  d.gt = s.gt;
  d.gh = s.gh;
  d.lengths = lengths;
  d.rows = w.rows;
  d.sources = w.sources;
  d.rows_chunk = w.rows_chunk;
  d.sources_chunk = w.sources_chunk;
  d.chunk_decay = w.chunk_decay;
  d.segments = p.segments;
  d.seg_tokens = p.seg_tokens;
  d.spans = p.spans;
  d.span_chunks = p.span_chunks;
  d.states = p.m[0].marks;
  d.adjoints = p.m[1].marks;
  d.cross = w.cross;
  d.initial = initial;
  d.grad_initial = grad_initial;
  d.partial = w.partial;
  d.grad_g = grad_log_decay;
  d.per_head = g_rank == 1;
  return device_status(sx::launch_decay_grad(d, str), "decay-attention gradient launch");
}

sx_status sx_decay_attention_step(sx_dtype dtype, const int64_t* q_shape, const int64_t* q_strides, const void* q,
                                  const int64_t* k_shape, const int64_t* k_strides, const void* k,
                                  const int64_t* v_shape, const int64_t* v_strides, const void* v, int g_rank,
                                  const int64_t* g_shape, const int64_t* g_strides, const float* log_decay,
                                  int64_t pool, const int64_t* state_strides, float* state, const int32_t* slots,
                                  float scale, void* out, void* stream) {
  const char* op = "decay-attention step";
  if (!dtype_ok(dtype))
    return fail(SX_E_DIM_002, "%s: q, k and v must be f32 or bf16 (dtype code %d)", op, enum_code(dtype));
  if (!q_shape || !k_shape || !v_shape) return fail(SX_E_DIM_001, "%s: q, k and v need shapes", op);
  // [B, heads, d] as [B, 1, heads, d]
  int64_t sh[3][4], ss[3][4];
  const int64_t* shapes[3] = {q_shape, k_shape, v_shape};
  const int64_t* strides[3] = {q_strides, k_strides, v_strides};
  for (int i = 0; i < 3; ++i) {
    int64_t st[3];
    if (strides[i]) std::copy(strides[i], strides[i] + 3, st); else contiguous_strides(3, shapes[i], st);
    sh[i][0] = shapes[i][0];
    sh[i][1] = 1;
    sh[i][2] = shapes[i][1];
    sh[i][3] = shapes[i][2];
    ss[i][0] = st[0];
    ss[i][1] = 0;
    ss[i][2] = st[1];
    ss[i][3] = st[2];
  }
  const HeadArg qa{"q", sh[0], ss[0], q}, ka{"k", sh[1], ss[1], k}, va{"v", sh[2], ss[2], v};
  if (!g_shape || (g_rank != 1 && g_rank != 2))
    return fail(SX_E_DIM_001, "%s: log_decay must be [heads] or [batch, heads]", op);
  int64_t gs[3], gst[3], gn[2];
  if (g_strides) std::copy(g_strides, g_strides + g_rank, gn); else contiguous_strides(g_rank, g_shape, gn);
  gs[0] = g_rank == 2 ? g_shape[0] : sh[0][0];
  gs[1] = 1;
  gs[2] = g_shape[g_rank - 1];
  gst[0] = g_rank == 2 ? gn[0] : 0;
  gst[1] = 0;
  gst[2] = gn[g_rank - 1];
  DecayShapes s;
  sx_status st = decay_shapes(op, qa, ka, va, 3, gs, gst, &s);
  if (st != SX_OK) return st;
  if (pool < 0) return fail(SX_E_DIM_001, "%s: a pool of %lld states", op, (long long)pool);
  if (!slots && pool < s.B)
    return fail(SX_E_DIM_001, "%s: %lld states for %lld rows and no slots", op, (long long)pool, (long long)s.B);
  const int64_t pool_shape[4] = {pool, s.H, s.dk, s.dv};
  int64_t ps[4], numel = 0;
  if (!checked_numel(4, pool_shape, &numel))
    return fail(SX_E_DIM_001, "%s: bad state shape %s", op, shape_str(4, pool_shape).c_str());
  if (state_strides) std::copy(state_strides, state_strides + 4, ps); else contiguous_strides(4, pool_shape, ps);
  if ((s.dk > 1 && ps[2] != s.dv) || (s.dv > 1 && ps[3] != 1))
    return fail(SX_E_UNSUPPORTED, "%s: a head's state must be row-major contiguous", op);
  const int64_t one = s.dk * s.dv;
  auto wide = [&](int i, int64_t below) { return pool_shape[i] <= 1 || ps[i] >= below || -ps[i] >= below; };
  if (numel > 0 && (!wide(1, one) || !wide(0, one) ||
                    (pool > 1 && s.H > 1 && !wide(0, (s.H - 1) * std::abs(ps[1]) + one) &&
                     !wide(1, (pool - 1) * std::abs(ps[0]) + one))))
    return fail(SX_E_UNSUPPORTED, "%s: states overlap each other", op);
  if (s.B == 0) return ok();
  for (const HeadArg* a : {&qa, &ka, &va})
    if (!a->data) return missing(op, a->name);
  if (!log_decay) return missing(op, "log_decay");
  if (!state && numel > 0) return missing(op, "state");
  if (!out) return missing(op, "out");
  const size_t e = dtype == SX_BF16 ? 2 : 4;
  const Span in[] = {head_span(qa, e), head_span(ka, e), head_span(va, e), decay_span(s, log_decay),
                     flat_span("slots", slots, s.B * 4)};
  // the state may be a view of a wider pool: any element of it
  Span to[] = {flat_span("out", out, s.B * s.H * s.dv * int64_t(e)), {"state", 0, 0, sizeof(float)}};
  if (state && numel > 0) span_bytes(state, 4, pool_shape, ps, sizeof(float), &to[1].lo, &to[1].hi);
  if ((st = no_overlap(op, in, 5, to, 2)) != SX_OK) return st;
  sx::DaStep p{};
  p.B = int(s.B);
  p.H = int(s.H);
  p.dk = int(s.dk);
  p.dv = int(s.dv);
  p.q = head_view(qa, e, s.H);
  p.k = head_view(ka, e, s.H);
  p.v = head_view(va, e, s.H);
  p.g = log_decay;
  p.gb = s.gb;
  p.gh = s.gh;
  p.state = state;
  p.ss = ps[0];
  p.sh = ps[1];
  p.slots_in_pool = pool;
  p.slots = slots;
  p.scale = scale;
  p.bf16 = dtype == SX_BF16;
  p.out = out;
  return device_status(sx::launch_decay_step(p, static_cast<hipStream_t>(stream)), "decay-attention step launch");
}

}  // extern "C"

namespace {

struct RotateArgs {
  HeadArg q, k, gq, gk;
  const void* positions;
  int positions_i64;
  const int64_t* position_strides;
  int64_t rotated;
  const double* turns;
  const float *qw, *kw;
  float eps;
  int neighbours;
};

sx_status plan_rotate(const char* op, const sx_dtype& dtype, const RotateArgs& a, bool gradient, sx::HrParams* p) {
  if (!dtype_ok(dtype))  // a reference: a code out of range must not be read as the enum
    return fail(SX_E_DIM_002, "%s: q and k must be f32 or bf16 (dtype code %d)", op, enum_code(dtype));
  for (const HeadArg* x : {&a.q, &a.k}) {
    int64_t n;
    if (!x->shape) return fail(SX_E_DIM_001, "%s: %s has no shape", op, x->name);
    if (!checked_numel(4, x->shape, &n))
      return fail(SX_E_DIM_001, "%s: bad shape %s of %s", op, shape_str(4, x->shape).c_str(), x->name);
  }
  const int64_t* qs = a.q.shape;
  const int64_t* ks = a.k.shape;
  if (qs[0] != ks[0] || qs[1] != ks[1] || qs[3] != ks[3])
    return fail(SX_E_DIM_001, "%s: k %s does not fit q %s", op, shape_str(4, ks).c_str(), shape_str(4, qs).c_str());
  const int64_t d = qs[3];
  if (d < 1) return fail(SX_E_DIM_001, "%s: heads of width 0 (q %s)", op, shape_str(4, qs).c_str());
  if (d > kMostHeadWidth)
    return fail(SX_E_UNSUPPORTED, "%s: heads wider than %lld (q %s)", op, (long long)kMostHeadWidth,
                shape_str(4, qs).c_str());
  if (a.rotated < 0 || a.rotated % 2 != 0 || a.rotated > d)
    return fail(SX_E_DIM_001, "%s: %lld rotated components of heads of width %lld; an even number up to the width",
                op, (long long)a.rotated, (long long)d);
  if (!(a.eps >= 0.0f)) return fail(SX_E_DIM_001, "%s: eps %g is negative", op, double(a.eps));
  if (qs[0] > kMostTokens || qs[1] > kMostTokens || qs[0] * qs[1] > kMostTokens || qs[2] + ks[2] > (1 << 20))
    return fail(SX_E_UNSUPPORTED, "%s: too many tokens or heads (q %s)", op, shape_str(4, qs).c_str());
  *p = sx::HrParams{};
  p->B = int(qs[0]);
  p->T = int(qs[1]);
  p->hq = int(qs[2]);
  p->hk = int(ks[2]);
  p->d = int(d);
  p->rot = int(a.rotated);
  const size_t e = dtype == SX_BF16 ? 2 : 4;
  p->q = head_view(a.q, e, qs[2]);
  p->k = head_view(a.k, e, ks[2]);
  if (gradient) {
    p->gq = head_view(a.gq, e, qs[2]);
    p->gk = head_view(a.gk, e, ks[2]);
  }
  p->positions = a.positions;
  p->pos64 = a.positions_i64 ? 1 : 0;
  p->pb = a.position_strides ? a.position_strides[0] : qs[1];
  p->pt = a.position_strides ? a.position_strides[1] : 1;
  p->turns = a.turns;
  p->qw = a.qw;
  p->kw = a.kw;
  p->eps = a.eps;
  p->neighbours = a.neighbours ? 1 : 0;
  p->bf16 = dtype == SX_BF16;
  return ok();
}

sx_status rotate_pointers(const char* op, const RotateArgs& a, bool gradient, int64_t rows) {
  if (rows == 0) return ok();
  for (const HeadArg* x : {&a.q, &a.k, &a.gq, &a.gk})
    if (x->shape && numel4(x->shape) > 0 && !x->data && (gradient || x == &a.q || x == &a.k))
      return missing(op, x->name);
  if (a.rotated > 0 && !a.positions) return missing(op, "positions");
  if (a.rotated > 0 && !a.turns) return missing(op, "turns");
  return ok();
}

sx_status rotate_overlap(const char* op, const RotateArgs& a, const sx::HrParams& p, const Span* out, int nout) {
  const size_t e = p.bf16 ? 2 : 4;
  const int64_t ps[2] = {p.B, p.T}, st[2] = {p.pb, p.pt};
  Span pos{"positions", 0, 0};
  if (a.positions && int64_t(p.B) * p.T > 0) span_bytes(a.positions, 2, ps, st, p.pos64 ? 8 : 4, &pos.lo, &pos.hi);
  const Span in[] = {head_span(a.q, e), head_span(a.k, e), a.gq.shape ? head_span(a.gq, e) : Span{"", 0, 0},
                     a.gk.shape ? head_span(a.gk, e) : Span{"", 0, 0}, pos,
                     flat_span("turns", a.turns, a.rotated / 2 * 8), flat_span("q_weight", a.qw, int64_t(p.d) * 4),
                     flat_span("k_weight", a.kw, int64_t(p.d) * 4)};
  return no_overlap(op, in, 8, out, nout);
}

}  // namespace

extern "C" {

sx_status sx_head_norm_rotate(sx_dtype dtype, const int64_t* q_shape, const int64_t* q_strides, const void* q,
                              const int64_t* k_shape, const int64_t* k_strides, const void* k, int positions_i64,
                              const int64_t* position_strides, const void* positions, int64_t rotated,
                              const double* turns, const float* q_weight, const float* k_weight, float eps,
                              int neighbours, void* out_q, void* out_k, void* stream) {
  const char* op = "head-norm-rotate";
  const RotateArgs a{{"q", q_shape, q_strides, q}, {"k", k_shape, k_strides, k}, {}, {}, positions, positions_i64,
                     position_strides, rotated, turns, q_weight, k_weight, eps, neighbours};
  sx::HrParams p;
  sx_status st = plan_rotate(op, dtype, a, false, &p);
  if (st != SX_OK) return st;
  const int64_t nq = numel4(q_shape), nk = numel4(k_shape);
  if (nq + nk == 0) return ok();
  if ((st = rotate_pointers(op, a, false, nq + nk)) != SX_OK) return st;
  if (nq > 0 && !out_q) return missing(op, "out_q");
  if (nk > 0 && !out_k) return missing(op, "out_k");
  const int64_t e = p.bf16 ? 2 : 4;
  const Span to[] = {flat_span("out_q", out_q, nq * e), flat_span("out_k", out_k, nk * e)};
  if ((st = rotate_overlap(op, a, p, to, 2)) != SX_OK) return st;
  p.out_q = out_q;
  p.out_k = out_k;
  return device_status(sx::launch_head_rotate(p, static_cast<hipStream_t>(stream)), "head-norm-rotate launch");
}

size_t sx_head_norm_rotate_backward_workspace_bytes(const int64_t* q_shape, const int64_t* k_shape) {
  RotateArgs a{};
  a.q.name = "q";
  a.q.shape = q_shape;
  a.k.name = "k";
  a.k.shape = k_shape;
  sx::HrParams p;
  if (plan_rotate("head-norm-rotate gradient", SX_F32, a, false, &p) != SX_OK) return 0;
  return size_t(sx::head_rotate_backward_groups(p)) * 2 * size_t(q_shape[3]) * sizeof(float);
}

sx_status sx_head_norm_rotate_backward(sx_dtype dtype, const int64_t* q_shape, const int64_t* q_strides,
                                       const void* q, const int64_t* k_shape, const int64_t* k_strides, const void* k,
                                       int positions_i64, const int64_t* position_strides, const void* positions,
                                       int64_t rotated, const double* turns, const int64_t* gq_strides,
                                       const void* grad_out_q, const int64_t* gk_strides, const void* grad_out_k,
                                       const float* q_weight, const float* k_weight, float eps, int neighbours,
                                       void* grad_q, void* grad_k, float* grad_q_weight, float* grad_k_weight,
                                       void* workspace, size_t workspace_bytes, void* stream) {
  const char* op = "head-norm-rotate gradient";
  const RotateArgs a{{"q", q_shape, q_strides, q}, {"k", k_shape, k_strides, k},
                     {"grad_out_q", q_shape, gq_strides, grad_out_q}, {"grad_out_k", k_shape, gk_strides, grad_out_k},
                     positions, positions_i64, position_strides, rotated, turns, q_weight, k_weight, eps, neighbours};
  sx::HrParams p;
  sx_status st = plan_rotate(op, dtype, a, true, &p);
  if (st != SX_OK) return st;
  const int64_t nq = numel4(q_shape), nk = numel4(k_shape);
  if ((st = rotate_pointers(op, a, true, nq + nk)) != SX_OK) return st;
  if (nq > 0 && !grad_q) return missing(op, "grad_q");
  if (nk > 0 && !grad_k) return missing(op, "grad_k");
  const int64_t e = p.bf16 ? 2 : 4;
  const Span to[] = {flat_span("grad_q", grad_q, nq * e), flat_span("grad_k", grad_k, nk * e),
                     flat_span("grad_q_weight", grad_q_weight, int64_t(p.d) * 4),
                     flat_span("grad_k_weight", grad_k_weight, int64_t(p.d) * 4)};
  if ((st = rotate_overlap(op, a, p, to, 4)) != SX_OK) return st;
  if (grad_q_weight || grad_k_weight) {
    const size_t need = sx_head_norm_rotate_backward_workspace_bytes(q_shape, k_shape);
    if ((st = check_workspace(op, workspace, workspace_bytes, need)) != SX_OK) return st;
  }
  if (nq + nk == 0 && !grad_q_weight && !grad_k_weight) return ok();
  p.out_q = grad_q;
  p.out_k = grad_k;
  p.partial = static_cast<float*>(workspace);
  p.gqw = grad_q_weight;
  p.gkw = grad_k_weight;
  return device_status(sx::launch_head_rotate_backward(p, static_cast<hipStream_t>(stream)),
                       "head-norm-rotate gradient launch");
}

}  // extern "C"

// ------------------------------------------------------------------ causal convolution, selective scan, group norm

namespace {

constexpr int64_t kMostChannels = int64_t(1) << 24;
constexpr int64_t kMostElements = int64_t(1) << 48;  // of one operand: no size of a workspace overflows below it

bool activation_ok(const sx_activation& a) {
  const int v = enum_code(a);
  return v == SX_ACT_NONE || v == SX_ACT_SILU;
}

// An operand of `rank` dims, at most four.
struct Operand {
  const char* name;
  int rank;
  const int64_t* shape;
  const int64_t* strides;  // nullptr: contiguous
  const void* data;
};

int64_t numel_of(const Operand& a) {
  int64_t n = 1;
  for (int i = 0; i < a.rank; ++i) n *= a.shape[i];
  return n;
}

void strides_of(const Operand& a, int64_t* st) {
  if (a.strides) std::copy(a.strides, a.strides + a.rank, st); else contiguous_strides(a.rank, a.shape, st);
}

Span span_of(const Operand& a, size_t elem) {
  Span s{a.name, 0, 0};
  if (!a.data || numel_of(a) == 0) return s;
  int64_t st[4];
  strides_of(a, st);
  span_bytes(a.data, a.rank, a.shape, st, elem, &s.lo, &s.hi);
  return s;
}

sx_status shape_given(const char* op, const Operand& a) {
  int64_t n;
  if (!a.shape) return fail(SX_E_DIM_001, "%s: %s has no shape", op, a.name);
  if (!checked_numel(a.rank, a.shape, &n))
    return fail(SX_E_DIM_001, "%s: bad shape %s of %s", op, shape_str(a.rank, a.shape).c_str(), a.name);
  return ok();
}

sx_status float_type(const char* op, const sx_dtype& dtype) {
  if (!dtype_ok(dtype))
    return fail(SX_E_DIM_002, "%s: the operands must be f32 or bf16 (dtype code %d)", op, enum_code(dtype));
  return ok();
}

sx_status activation_given(const char* op, const sx_activation& a) {
  if (!activation_ok(a)) return fail(SX_E_UNSUPPORTED, "%s: no activation of code %d", op, enum_code(a));
  return ok();
}

// [B, T, D], or [B, D] with T = 1.
sx_status token_shape(const char* op, const Operand& x) {
  const sx_status st = shape_given(op, x);
  if (st != SX_OK) return st;
  if (x.shape[x.rank - 1] < 1)
    return fail(SX_E_DIM_001, "%s: %s %s has no channels", op, x.name, shape_str(x.rank, x.shape).c_str());
  if (x.shape[x.rank - 1] > kMostChannels || x.shape[0] > kMostTokens || numel_of(x) > kMostElements ||
      (x.rank == 3 && x.shape[1] > kMostTokens))
    return fail(SX_E_UNSUPPORTED, "%s: too many rows, tokens or channels (%s %s)", op, x.name,
                shape_str(x.rank, x.shape).c_str());
  return ok();
}

sx::TokenView token_view(const Operand& x) {
  sx::TokenView v{};
  if (!x.data) return v;
  int64_t st[4];
  strides_of(x, st);
  v.p = x.data;
  v.sb = st[0];
  v.st = x.rank == 3 ? st[1] : 0;
  v.sd = x.shape[x.rank - 1] == 1 ? 1 : st[x.rank - 1];
  return v;
}

// A pool of states of `one` elements each, contiguous: its span, and whether they overlap.
sx_status pool_span(const char* op, int64_t pool, int64_t stride, int64_t one, const void* state, int64_t rows,
                    const int32_t* slots, size_t elem, Span* s) {
  if (pool < 0) return fail(SX_E_DIM_001, "%s: a pool of %lld states", op, (long long)pool);
  if (!slots && pool < rows)
    return fail(SX_E_DIM_001, "%s: %lld states for %lld rows and no slots", op, (long long)pool, (long long)rows);
  int64_t n;
  const int64_t shape[2] = {pool, one}, st[2] = {stride, 1};
  if (!checked_numel(2, shape, &n)) return fail(SX_E_DIM_001, "%s: bad pool of %lld states", op, (long long)pool);
  if (pool > 1 && stride < one && -stride < one) return fail(SX_E_UNSUPPORTED, "%s: states overlap each other", op);
  *s = Span{"state", 0, 0, unsigned(elem)};
  if (state && n > 0) span_bytes(state, 2, shape, st, elem, &s->lo, &s->hi);
  return ok();
}

struct ConvArgs {
  Operand x;
  int64_t taps;
  const float *weight, *bias;
};

sx_status conv_shapes(const char* op, const sx_dtype& dtype, const ConvArgs& a, const sx_activation& act) {
  sx_status st = float_type(op, dtype);
  if (st == SX_OK) st = token_shape(op, a.x);
  if (st == SX_OK) st = activation_given(op, act);
  if (st != SX_OK) return st;
  if (a.taps < 1) return fail(SX_E_DIM_001, "%s: a weight of %lld taps", op, (long long)a.taps);
  if (a.taps > SX_MAX_TAPS)
    return fail(SX_E_UNSUPPORTED, "%s: %lld taps, %d at most", op, (long long)a.taps, SX_MAX_TAPS);
  return ok();
}

sx::CcParams conv_params(const sx_dtype& dtype, const ConvArgs& a, const int32_t* lengths, const sx_activation& act,
                         bool gradient) {
  sx::CcParams p{};
  p.B = int(a.x.shape[0]);
  p.T = int(a.x.shape[1]);
  p.D = int(a.x.shape[2]);
  p.K = int(a.taps);
  p.x = token_view(a.x);
  p.w = a.weight;
  p.bias = a.bias;
  p.lengths = lengths;
  p.silu = act == SX_ACT_SILU;
  p.bf16 = dtype == SX_BF16;
  sx::causal_conv_split(p, gradient);
  return p;
}

// A launch takes fewer than 2^32 threads along its grid.
sx_status grid_fits(const char* op, double groups, int threads) {
  if (groups * threads >= 4294967296.0) return fail(SX_E_UNSUPPORTED, "%s: too many elements for one launch", op);
  return ok();
}

size_t conv_partial_floats(const sx::CcParams& p) { return size_t(p.B) * p.chunks * (p.K + 1) * size_t(p.D); }

}  // namespace

extern "C" {

sx_status sx_causal_conv(sx_dtype dtype, const int64_t* x_shape, const int64_t* x_strides, const void* x, int64_t taps,
                         const float* weight, const float* bias, const void* initial, const int32_t* lengths,
                         sx_activation activation, void* out, void* final_state, void* stream) {
  const char* op = "causal-conv";
  const ConvArgs a{{"x", 3, x_shape, x_strides, x}, taps, weight, bias};
  sx_status st = conv_shapes(op, dtype, a, activation);
  if (st != SX_OK) return st;
  const int64_t B = x_shape[0], D = x_shape[2], n = numel_of(a.x), state = B * (taps - 1) * D;
  const size_t e = dtype == SX_BF16 ? 2 : 4;
  if (B == 0 || (n == 0 && !final_state)) return ok();
  if (!weight) return missing(op, "weight");  // a launch reads it, also of no tokens
  if (n > 0) {
    if (!x) return missing(op, "x");
    if (!out) return missing(op, "out");
  }
  const Span in[] = {span_of(a.x, e), flat_span("weight", weight, D * taps * 4), flat_span("bias", bias, D * 4),
                     flat_span("initial", initial, state * int64_t(e)), flat_span("lengths", lengths, B * 4)};
  const Span to[] = {flat_span("out", out, n * int64_t(e)),
                     flat_span("the final state", final_state, state * int64_t(e))};
  if ((st = no_overlap(op, in, 5, to, 2)) != SX_OK) return st;
  sx::CcParams p = conv_params(dtype, a, lengths, activation, false);
  if ((st = grid_fits(op, sx::causal_conv_workgroups(p, false), 256)) != SX_OK) return st;
  p.initial = initial;
  p.out = out;
  p.last = final_state;
  return device_status(sx::launch_causal_conv(p, static_cast<hipStream_t>(stream)), "causal-conv launch");
}

size_t sx_causal_conv_backward_workspace_bytes(sx_dtype dtype, const int64_t* x_shape, int64_t taps) {
  const ConvArgs a{{"x", 3, x_shape, nullptr, nullptr}, taps, nullptr, nullptr};
  if (conv_shapes("causal-conv gradient", dtype, a, SX_ACT_NONE) != SX_OK) return 0;
  return conv_partial_floats(conv_params(dtype, a, nullptr, SX_ACT_NONE, true)) * sizeof(float);
}

sx_status sx_causal_conv_backward(sx_dtype dtype, const int64_t* x_shape, const int64_t* x_strides, const void* x,
                                  int64_t taps, const float* weight, const float* bias, const void* initial,
                                  const int32_t* lengths, sx_activation activation, const int64_t* grad_out_strides,
                                  const void* grad_out, const void* grad_state, void* grad_x, float* grad_weight,
                                  float* grad_bias, void* grad_initial, void* workspace, size_t workspace_bytes,
                                  void* stream) {
  const char* op = "causal-conv gradient";
  const ConvArgs a{{"x", 3, x_shape, x_strides, x}, taps, weight, bias};
  sx_status st = conv_shapes(op, dtype, a, activation);
  if (st != SX_OK) return st;
  const Operand go{"grad_out", 3, x_shape, grad_out_strides, grad_out};
  const int64_t B = x_shape[0], D = x_shape[2], n = numel_of(a.x), state = B * (taps - 1) * D;
  const int64_t e = dtype == SX_BF16 ? 2 : 4;
  if (!weight) return missing(op, "weight");
  if (!grad_weight) return missing(op, "grad_weight");
  if (n > 0) {
    if (!x) return missing(op, "x");
    if (!grad_out) return missing(op, "grad_out");
    if (!grad_x) return missing(op, "grad_x");
  }
  const Span in[] = {span_of(a.x, e), span_of(go, e), flat_span("weight", weight, D * taps * 4),
                     flat_span("bias", bias, D * 4), flat_span("initial", initial, state * e),
                     flat_span("lengths", lengths, B * 4), flat_span("grad_state", grad_state, state * e)};
  const Span to[] = {flat_span("grad_x", grad_x, n * e), flat_span("grad_weight", grad_weight, D * taps * 4),
                     flat_span("grad_bias", grad_bias, D * 4), flat_span("grad_initial", grad_initial, state * e)};
  if ((st = no_overlap(op, in, 7, to, 4)) != SX_OK) return st;
  sx::CcParams p = conv_params(dtype, a, lengths, activation, true);
  p.go = token_view(go);
  if ((st = grid_fits(op, sx::causal_conv_workgroups(p, true), 256)) != SX_OK) return st;
  if ((st = check_workspace(op, workspace, workspace_bytes, conv_partial_floats(p) * sizeof(float))) != SX_OK) return st;
  p.initial = initial;
  p.grad_state = grad_state;
  p.out = grad_x;
  p.last = grad_initial;
  p.partial = static_cast<float*>(workspace);
  p.gw = grad_weight;
  p.gbias = grad_bias;
  return device_status(sx::launch_causal_conv_backward(p, static_cast<hipStream_t>(stream)),
                       "causal-conv gradient launch");
}

sx_status sx_causal_conv_step(sx_dtype dtype, const int64_t* x_shape, const int64_t* x_strides, const void* x,
                              int64_t taps, const float* weight, const float* bias, sx_activation activation,
                              int64_t pool, int64_t state_stride, void* state, const int32_t* slots, void* out,
                              void* stream) {
  const char* op = "causal-conv step";
  const ConvArgs a{{"x", 2, x_shape, x_strides, x}, taps, weight, bias};
  sx_status st = conv_shapes(op, dtype, a, activation);
  if (st != SX_OK) return st;
  const int64_t B = x_shape[0], D = x_shape[1], one = (taps - 1) * D;
  const int64_t e = dtype == SX_BF16 ? 2 : 4;
  Span to[] = {flat_span("out", out, B * D * e), {}};
  if ((st = pool_span(op, pool, state_stride, one, state, B, slots, size_t(e), &to[1])) != SX_OK) return st;
  if (B == 0) return ok();
  if (!x) return missing(op, "x");
  if (!weight) return missing(op, "weight");
  if (!state && pool * one > 0) return missing(op, "state");
  if (!out) return missing(op, "out");
  const Span in[] = {span_of(a.x, e), flat_span("weight", weight, D * taps * 4), flat_span("bias", bias, D * 4),
                     flat_span("slots", slots, B * 4)};
  if ((st = no_overlap(op, in, 4, to, 2)) != SX_OK) return st;
  const sx::TokenView v = token_view(a.x);
  sx::CcStep p{};
  p.B = int(B);
  p.D = int(D);
  p.K = int(taps);
  p.x = x;
  p.sb = v.sb;
  p.sd = v.sd;
  p.w = weight;
  p.bias = bias;
  p.state = state;
  p.ss = state_stride;
  p.pool = pool;
  p.slots = slots;
  p.silu = activation == SX_ACT_SILU;
  p.bf16 = dtype == SX_BF16;
  p.out = out;
  if ((st = grid_fits(op, sx::causal_conv_step_workgroups(p), 256)) != SX_OK) return st;
  return device_status(sx::launch_causal_conv_step(p, static_cast<hipStream_t>(stream)), "causal-conv step launch");
}

}  // extern "C"

namespace {

struct ScanArgs {
  Operand x, delta, z, b, c;
  const float *a, *skip, *delta_bias;
};

sx_status scan_shapes(const char* op, const sx_dtype& dtype, const ScanArgs& a) {
  sx_status st = float_type(op, dtype);
  if (st == SX_OK) st = token_shape(op, a.x);
  if (st == SX_OK) st = shape_given(op, a.b);
  if (st != SX_OK) return st;
  const int64_t* xs = a.x.shape;
  const int64_t* bs = a.b.shape;
  const int dims = a.x.rank - 1;  // rows and tokens
  for (int i = 0; i < dims; ++i)
    if (bs[i] != xs[i])
      return fail(SX_E_DIM_001, "%s: b %s does not fit x %s", op, shape_str(a.b.rank, bs).c_str(),
                  shape_str(a.x.rank, xs).c_str());
  const int64_t D = xs[dims], G = bs[dims], N = bs[dims + 1];
  if (G < 1 || D % G != 0)
    return fail(SX_E_DIM_001, "%s: the %lld groups of b do not divide the %lld channels of x", op, (long long)G,
                (long long)D);
  if (N < 1) return fail(SX_E_DIM_001, "%s: no states (b %s)", op, shape_str(a.b.rank, bs).c_str());
  if (N > SX_MAX_STATES)
    return fail(SX_E_UNSUPPORTED, "%s: %lld states a channel, %d at most", op, (long long)N, SX_MAX_STATES);
  return ok();
}

sx::RowView row_view(const Operand& a) {
  int64_t st[4];
  strides_of(a, st);
  const int k = a.rank == 4 ? 1 : 0;
  return {a.data, st[0], k ? st[1] : 0, st[k + 1], st[k + 2]};
}

sx::SsParams scan_params(const sx_dtype& dtype, const ScanArgs& a, bool gradient) {
  sx::SsParams p{};
  p.B = int(a.x.shape[0]);
  p.T = int(a.x.shape[1]);
  p.D = int(a.x.shape[2]);
  p.G = int(a.b.shape[2]);
  p.N = int(a.b.shape[3]);
  p.x = token_view(a.x);
  p.delta = token_view(a.delta);
  p.z = token_view(a.z);
  p.b = row_view(a.b);
  p.c = row_view(a.c);
  p.a = a.a;
  p.skip = a.skip;
  p.delta_bias = a.delta_bias;
  p.bf16 = dtype == SX_BF16;
  sx::selective_scan_split(p, gradient);
  return p;
}

sx_status scan_pointers(const char* op, const ScanArgs& a) {
  for (const Operand* o : {&a.x, &a.delta, &a.b, &a.c})
    if (!o->data) return missing(op, o->name);
  if (!a.a) return missing(op, "a");
  return ok();
}

// The operands' spans; returns how many.
int scan_spans(const ScanArgs& a, size_t e, Span* s) {
  const int64_t D = a.x.shape[a.x.rank - 1], N = a.b.shape[a.b.rank - 1];
  s[0] = span_of(a.x, e);
  s[1] = span_of(a.delta, e);
  s[2] = span_of(a.z, e);
  s[3] = span_of(a.b, e);
  s[4] = span_of(a.c, e);
  s[5] = flat_span("a", a.a, D * N * 4);
  s[6] = flat_span("skip", a.skip, D * 4);
  s[7] = flat_span("delta_bias", a.delta_bias, D * 4);
  return 8;
}

int64_t packed_floats(const sx::SsParams& p) { return int64_t(p.B) * p.waves * p.D * sx::kScanStates; }

void carve_scan(Carve& c, sx::SsParams& p) {
  const int64_t n = p.segments - 1;
  p.seg_state = c.take<float>(n * packed_floats(p));
  p.seg_steps = c.take<float>(n * p.B * p.D);
}

void carve_scan_gradient(Carve& c, sx::SsParams& p) {
  const int64_t D = p.D, rows = int64_t(p.B) * p.segments, joined = p.segments > 1 ? p.segments : 0;
  p.seg_state = c.take<float>(joined * packed_floats(p));
  p.seg_adjoint = c.take<float>(joined * packed_floats(p));
  p.seg_steps = c.take<float>(joined * p.B * D);
  p.marks = c.take<float>(packed_floats(p) * p.row_marks);
  p.mark_steps = c.take<float>(joined ? int64_t(p.B) * p.row_marks * D : 0);
  p.rows_partial = c.take<float>(int64_t(p.B) * p.G * p.T * sx::selective_scan_grad_blocks(p) * 8 * p.waves);
  p.a_partial = c.take<float>(rows * D * p.N);
  p.skip_partial = c.take<float>(rows * D);
  p.bias_partial = c.take<float>(rows * D);
}

// The largest launches: the march, and of the gradient the sums of a token's rows and of the rates.
sx_status scan_grid(const char* op, const sx::SsParams& p, bool gradient) {
  const double blocks = double(p.G) * ((p.D / p.G + 63) / 64);
  sx_status st = grid_fits(op, blocks * p.B * p.segments, 64 * p.waves);
  if (st == SX_OK && gradient) st = grid_fits(op, std::ceil(double(p.B) * p.G * p.T * 8 * p.waves / 256), 256);
  if (st == SX_OK && gradient) st = grid_fits(op, std::ceil(double(p.D) * p.N / 64), 1024);
  return st;
}

}  // namespace

extern "C" {

size_t sx_selective_scan_workspace_bytes(sx_dtype dtype, const int64_t* x_shape, const int64_t* b_shape) {
  const ScanArgs a{{"x", 3, x_shape}, {"delta", 3, x_shape}, {"z", 3, x_shape}, {"b", 4, b_shape}, {"c", 4, b_shape}};
  if (scan_shapes("selective-scan", dtype, a) != SX_OK) return 0;
  sx::SsParams p = scan_params(dtype, a, false);
  Carve c{0};
  carve_scan(c, p);
  return c.used;
}

sx_status sx_selective_scan(sx_dtype dtype, const int64_t* x_shape, const int64_t* x_strides, const void* x,
                            const int64_t* delta_strides, const void* delta, const float* a, const int64_t* b_shape,
                            const int64_t* b_strides, const void* b, const int64_t* c_strides, const void* c,
                            const float* skip, const int64_t* z_strides, const void* z, const float* delta_bias,
                            int softplus, const float* initial, const int32_t* lengths, void* out, float* final_state,
                            void* workspace, size_t workspace_bytes, void* stream) {
  const char* op = "selective-scan";
  const ScanArgs args{{"x", 3, x_shape, x_strides, x}, {"delta", 3, x_shape, delta_strides, delta},
                      {"z", 3, x_shape, z_strides, z}, {"b", 4, b_shape, b_strides, b},
                      {"c", 4, b_shape, c_strides, c}, a, skip, delta_bias};
  sx_status st = scan_shapes(op, dtype, args);
  if (st != SX_OK) return st;
  const int64_t B = x_shape[0], T = x_shape[1], D = x_shape[2], N = b_shape[3], n = B * T * D, state = B * D * N;
  if (B == 0 || (T == 0 && !final_state)) return ok();
  if (n > 0) {
    if ((st = scan_pointers(op, args)) != SX_OK) return st;
    if (!out) return missing(op, "out");
  }
  if (!a) return missing(op, "a");  // a launch reads it, also of no tokens
  const size_t e = dtype == SX_BF16 ? 2 : 4;
  Span in[10];
  int k = scan_spans(args, e, in);
  in[k++] = flat_span("initial", initial, state * 4);
  in[k++] = flat_span("lengths", lengths, B * 4);
  const Span to[] = {flat_span("out", out, n * int64_t(e)), flat_span("the final state", final_state, state * 4)};
  if ((st = no_overlap(op, in, k, to, 2)) != SX_OK) return st;
  sx::SsParams p = scan_params(dtype, args, false);
  if ((st = scan_grid(op, p, false)) != SX_OK) return st;
  Carve w{reinterpret_cast<uintptr_t>(workspace)};
  carve_scan(w, p);
  if ((st = check_workspace(op, workspace, workspace_bytes, w.used)) != SX_OK) return st;
  p.softplus = softplus != 0;
  p.initial = initial;
  p.lengths = lengths;
  p.out = out;
  p.last = final_state;
  return device_status(sx::launch_selective_scan(p, static_cast<hipStream_t>(stream)), "selective-scan launch");
}

size_t sx_selective_scan_backward_workspace_bytes(sx_dtype dtype, const int64_t* x_shape, const int64_t* b_shape) {
  const ScanArgs a{{"x", 3, x_shape}, {"delta", 3, x_shape}, {"z", 3, x_shape}, {"b", 4, b_shape}, {"c", 4, b_shape}};
  if (scan_shapes("selective-scan gradient", dtype, a) != SX_OK) return 0;
  sx::SsParams p = scan_params(dtype, a, true);
  Carve c{0};
  carve_scan_gradient(c, p);
  return c.used;
}

sx_status sx_selective_scan_backward(sx_dtype dtype, const int64_t* x_shape, const int64_t* x_strides, const void* x,
                                     const int64_t* delta_strides, const void* delta, const float* a,
                                     const int64_t* b_shape, const int64_t* b_strides, const void* b,
                                     const int64_t* c_strides, const void* c, const float* skip,
                                     const int64_t* z_strides, const void* z, const float* delta_bias, int softplus,
                                     const float* initial, const int32_t* lengths, const int64_t* grad_out_strides,
                                     const void* grad_out, const float* grad_state, void* grad_x, void* grad_delta,
                                     float* grad_a, void* grad_b, void* grad_c, float* grad_skip, void* grad_z,
                                     float* grad_delta_bias, float* grad_initial, void* workspace,
                                     size_t workspace_bytes, void* stream) {
  const char* op = "selective-scan gradient";
  const ScanArgs args{{"x", 3, x_shape, x_strides, x}, {"delta", 3, x_shape, delta_strides, delta},
                      {"z", 3, x_shape, z_strides, z}, {"b", 4, b_shape, b_strides, b},
                      {"c", 4, b_shape, c_strides, c}, a, skip, delta_bias};
  sx_status st = scan_shapes(op, dtype, args);
  if (st != SX_OK) return st;
  const Operand go{"grad_out", 3, x_shape, grad_out_strides, grad_out};
  const int64_t B = x_shape[0], T = x_shape[1], D = x_shape[2], N = b_shape[3], n = B * T * D, state = B * D * N;
  const int64_t rows = numel_of(args.b);
  if (n > 0) {
    if ((st = scan_pointers(op, args)) != SX_OK) return st;
    if (!grad_out) return missing(op, "grad_out");
    if (!grad_x) return missing(op, "grad_x");
    if (!grad_delta) return missing(op, "grad_delta");
    if (!grad_b) return missing(op, "grad_b");
    if (!grad_c) return missing(op, "grad_c");
    if (z && !grad_z) return missing(op, "grad_z");
  }
  if (B > 0 && !a) return missing(op, "a");
  if (!grad_a) return missing(op, "grad_a");
  const int64_t e = dtype == SX_BF16 ? 2 : 4;
  Span in[12];
  int k = scan_spans(args, size_t(e), in);
  in[k++] = flat_span("initial", initial, state * 4);
  in[k++] = flat_span("lengths", lengths, B * 4);
  in[k++] = span_of(go, size_t(e));
  in[k++] = flat_span("grad_state", grad_state, state * 4);
  const Span to[] = {flat_span("grad_x", grad_x, n * e),
                     flat_span("grad_delta", grad_delta, n * e),
                     flat_span("grad_a", grad_a, D * N * 4),
                     flat_span("grad_b", grad_b, rows * e),
                     flat_span("grad_c", grad_c, rows * e),
                     flat_span("grad_skip", grad_skip, D * 4),
                     flat_span("grad_z", z ? grad_z : nullptr, n * e),
                     flat_span("grad_delta_bias", grad_delta_bias, D * 4),
                     flat_span("grad_initial", grad_initial, state * 4)};
  if ((st = no_overlap(op, in, k, to, 9)) != SX_OK) return st;
  sx::SsParams p = scan_params(dtype, args, true);
  if ((st = scan_grid(op, p, true)) != SX_OK) return st;
  Carve w{reinterpret_cast<uintptr_t>(workspace)};
  carve_scan_gradient(w, p);
  if ((st = check_workspace(op, workspace, workspace_bytes, w.used)) != SX_OK) return st;
  p.softplus = softplus != 0;
  p.initial = initial;
  p.lengths = lengths;
  p.go = token_view(go);
  p.grad_state = grad_state;
  p.gx = grad_x;
  p.gdelta = grad_delta;
  p.gz = grad_z;
  p.gb = grad_b;
  p.gc = grad_c;
  p.ga = grad_a;
  p.gskip = grad_skip;
  p.gbias = grad_delta_bias;
  p.ginitial = grad_initial;
  return device_status(sx::launch_selective_scan_backward(p, static_cast<hipStream_t>(stream)),
                       "selective-scan gradient launch");
}

sx_status sx_selective_scan_step(sx_dtype dtype, const int64_t* x_shape, const int64_t* x_strides, const void* x,
                                 const int64_t* delta_strides, const void* delta, const float* a,
                                 const int64_t* b_shape, const int64_t* b_strides, const void* b,
                                 const int64_t* c_strides, const void* c, const float* skip, const int64_t* z_strides,
                                 const void* z, const float* delta_bias, int softplus, int64_t pool,
                                 int64_t state_stride, float* state, const int32_t* slots, void* out, void* stream) {
  const char* op = "selective-scan step";
  const ScanArgs args{{"x", 2, x_shape, x_strides, x}, {"delta", 2, x_shape, delta_strides, delta},
                      {"z", 2, x_shape, z_strides, z}, {"b", 3, b_shape, b_strides, b},
                      {"c", 3, b_shape, c_strides, c}, a, skip, delta_bias};
  sx_status st = scan_shapes(op, dtype, args);
  if (st != SX_OK) return st;
  const int64_t B = x_shape[0], D = x_shape[1], N = b_shape[2], e = dtype == SX_BF16 ? 2 : 4;
  Span to[] = {flat_span("out", out, B * D * e), {}};
  if ((st = pool_span(op, pool, state_stride, D * N, state, B, slots, sizeof(float), &to[1])) != SX_OK) return st;
  if (B == 0) return ok();
  if ((st = scan_pointers(op, args)) != SX_OK) return st;
  if (!state && pool > 0) return missing(op, "state");
  if (!out) return missing(op, "out");
  Span in[9];
  int k = scan_spans(args, size_t(e), in);
  in[k++] = flat_span("slots", slots, B * 4);
  if ((st = no_overlap(op, in, k, to, 2)) != SX_OK) return st;
  if ((st = grid_fits(op, std::ceil(double(B) * double(D) * sx::selective_scan_step_lanes(int(N)) / 256), 256)) != SX_OK)
    return st;
  sx::SsStep p{};
  p.B = int(B);
  p.D = int(D);
  p.G = int(b_shape[1]);
  p.N = int(N);
  p.x = token_view(args.x);
  p.delta = token_view(args.delta);
  p.z = token_view(args.z);
  p.b = row_view(args.b);
  p.c = row_view(args.c);
  p.a = a;
  p.skip = skip;
  p.delta_bias = delta_bias;
  p.softplus = softplus != 0;
  p.bf16 = dtype == SX_BF16;
  p.state = state;
  p.ss = state_stride;
  p.pool = pool;
  p.slots = slots;
  p.out = out;
  return device_status(sx::launch_selective_scan_step(p, static_cast<hipStream_t>(stream)),
                       "selective-scan step launch");
}

}  // extern "C"

namespace {

sx_status plan_norm(const char* op, const sx_dtype& dtype, const Operand& x, int64_t groups, float eps,
                    const sx_activation& act, bool gradient, sx::GnParams* p) {
  sx_status st = float_type(op, dtype);
  if (st == SX_OK) st = shape_given(op, x);
  if (st == SX_OK) st = activation_given(op, act);
  if (st != SX_OK) return st;
  const int64_t c = x.shape[2];
  if (c < 1) return fail(SX_E_DIM_001, "%s: x %s has no channels", op, shape_str(3, x.shape).c_str());
  if (groups < 1 || c % groups != 0)
    return fail(SX_E_DIM_001, "%s: %lld groups do not divide %lld channels", op, (long long)groups, (long long)c);
  if (!(eps >= 0.0f)) return fail(SX_E_DIM_001, "%s: eps %g is negative", op, double(eps));
  if (c > kMostChannels || x.shape[0] > kMostElements || x.shape[1] > kMostElements || numel_of(x) > kMostElements)
    return fail(SX_E_UNSUPPORTED, "%s: too many samples, positions or channels (x %s)", op,
                shape_str(3, x.shape).c_str());
  int64_t xs[4];
  strides_of(x, xs);
  if (c > 1 && xs[2] != 1) return fail(SX_E_UNSUPPORTED, "%s: channels of %s must lie next to each other", op, x.name);
  *p = sx::GnParams{};
  p->n = x.shape[0];
  p->s = x.shape[1];
  p->c = int(c);
  p->g = int(groups);
  p->x = x.data;
  p->xn = xs[0];
  p->xs = xs[1];
  p->eps = eps;
  p->silu = act == SX_ACT_SILU;
  p->bf16 = dtype == SX_BF16;
  sx::group_norm_split(*p, gradient);
  return grid_fits(op, sx::group_norm_workgroups(*p, gradient), 256);
}

size_t carve_norm(Carve& c, sx::GnParams& p, bool gradient) {
  p.stats = c.take<float>(sx::group_norm_stats_floats(p));
  if (gradient) p.sums = c.take<float>(sx::group_norm_sums_floats(p));
  return c.used;
}

}  // namespace

extern "C" {

size_t sx_group_norm_workspace_bytes(sx_dtype dtype, const int64_t* x_shape, int64_t groups) {
  sx::GnParams p;
  if (plan_norm("group-norm", dtype, {"x", 3, x_shape}, groups, 0.0f, SX_ACT_NONE, false, &p) != SX_OK) return 0;
  Carve c{0};
  return p.n * p.s == 0 ? 0 : carve_norm(c, p, false);
}

sx_status sx_group_norm(sx_dtype dtype, const int64_t* x_shape, const int64_t* x_strides, const void* x, int64_t groups,
                        const float* weight, const float* bias, float eps, sx_activation activation, void* out,
                        void* workspace, size_t workspace_bytes, void* stream) {
  const char* op = "group-norm";
  const Operand xa{"x", 3, x_shape, x_strides, x};
  sx::GnParams p;
  sx_status st = plan_norm(op, dtype, xa, groups, eps, activation, false, &p);
  if (st != SX_OK) return st;
  const int64_t n = numel_of(xa), e = p.bf16 ? 2 : 4;
  if (n == 0) return ok();
  if (!x) return missing(op, "x");
  if (!out) return missing(op, "out");
  const Span in[] = {span_of(xa, size_t(e)), flat_span("weight", weight, int64_t(p.c) * 4),
                     flat_span("bias", bias, int64_t(p.c) * 4)};
  const Span to[] = {flat_span("out", out, n * e)};
  if ((st = no_overlap(op, in, 3, to, 1)) != SX_OK) return st;
  Carve c{reinterpret_cast<uintptr_t>(workspace)};
  if ((st = check_workspace(op, workspace, workspace_bytes, carve_norm(c, p, false))) != SX_OK) return st;
  p.w = weight;
  p.bias = bias;
  p.out = out;
  return device_status(sx::launch_group_norm(p, static_cast<hipStream_t>(stream)), "group-norm launch");
}

size_t sx_group_norm_backward_workspace_bytes(sx_dtype dtype, const int64_t* x_shape, int64_t groups) {
  sx::GnParams p;
  if (plan_norm("group-norm gradient", dtype, {"x", 3, x_shape}, groups, 0.0f, SX_ACT_NONE, true, &p) != SX_OK) return 0;
  Carve c{0};
  return p.n * p.s == 0 ? 0 : carve_norm(c, p, true);
}

sx_status sx_group_norm_backward(sx_dtype dtype, const int64_t* x_shape, const int64_t* x_strides, const void* x,
                                 int64_t groups, const float* weight, const float* bias, float eps,
                                 sx_activation activation, const int64_t* grad_out_strides, const void* grad_out,
                                 void* grad_x, float* grad_weight, float* grad_bias, void* workspace,
                                 size_t workspace_bytes, void* stream) {
  const char* op = "group-norm gradient";
  const Operand xa{"x", 3, x_shape, x_strides, x}, go{"grad_out", 3, x_shape, grad_out_strides, grad_out};
  sx::GnParams p;
  sx_status st = plan_norm(op, dtype, xa, groups, eps, activation, true, &p);
  if (st != SX_OK) return st;
  int64_t gs[4];
  strides_of(go, gs);
  if (p.c > 1 && gs[2] != 1)
    return fail(SX_E_UNSUPPORTED, "%s: channels of grad_out must lie next to each other", op);
  const int64_t n = numel_of(xa), e = p.bf16 ? 2 : 4, c = p.c;
  if (n > 0) {
    if (!x) return missing(op, "x");
    if (!grad_out) return missing(op, "grad_out");
    if (!grad_x) return missing(op, "grad_x");
  }
  const Span in[] = {span_of(xa, size_t(e)), span_of(go, size_t(e)), flat_span("weight", weight, c * 4),
                     flat_span("bias", bias, c * 4)};
  const Span to[] = {flat_span("grad_x", grad_x, n * e), flat_span("grad_weight", grad_weight, c * 4),
                     flat_span("grad_bias", grad_bias, c * 4)};
  if ((st = no_overlap(op, in, 4, to, 3)) != SX_OK) return st;
  Carve w{reinterpret_cast<uintptr_t>(workspace)};
  if (n > 0 && (st = check_workspace(op, workspace, workspace_bytes, carve_norm(w, p, true))) != SX_OK) return st;
  p.w = weight;
  p.bias = bias;
  p.go = grad_out;
  p.gon = gs[0];
  p.gos = gs[1];
  p.out = grad_x;
  p.gw = grad_weight;
  p.gbias = grad_bias;
  return device_status(sx::launch_group_norm_backward(p, static_cast<hipStream_t>(stream)),
                       "group-norm gradient launch");
}

}  // extern "C"
