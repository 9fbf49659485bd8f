// C ABI of the operators around the mixer in a hybrid block: norms with their
// residual and gate.  Arguments are checked completely before any launch, as
// in gdn_api.cpp; no C++ exception crosses the boundary.
#include "../../include/gdn.h"

#include <hip/hip_runtime.h>

#include <cmath>
#include <cstddef>

#include "api_util.h"
#include "gdn_internal.h"

namespace {

using namespace gdn::api;

// One row tensor of a call: its rows in bytes and what to call it.
struct Tensor {
  const char* name;
  Rows rows;
};

// Outputs share no byte with an input, unless they are that input exactly
// (`same_ok`), and none with each other.
template <size_t NI, size_t NO>
const char* clash(const Tensor (&ins)[NI], const Tensor (&outs)[NO], bool same_ok) {
  for (size_t o = 0; o < NO; ++o) {
    const Rows& r = outs[o].rows;
    for (const Tensor& i : ins)
      if (rows_overlap(r, i.rows) && !(same_ok && r.p == i.rows.p && r.stride == i.rows.stride && r.width == i.rows.width))
        return outs[o].name;
    for (size_t k = 0; k < o; ++k)
      if (rows_overlap(r, outs[k].rows)) return outs[o].name;
  }
  return nullptr;
}

template <typename A>
gdn_status check_norm(const A* a, const char* f) {
  if (!a) return fail(GDN_ERR_INVALID_ARG, "%s: args is NULL", f);
  if (a->struct_size < sizeof(A)) return fail(GDN_ERR_INVALID_ARG, "%s: struct_size %u < %zu", f, a->struct_size, sizeof(A));
  if (!is_dtype(a->dtype) || !is_dtype(a->weight_dtype)) return fail(GDN_ERR_INVALID_ARG, "%s: bad dtype", f);
  if (a->order != GDN_NORM_PRE && a->order != GDN_NORM_POST) return fail(GDN_ERR_INVALID_ARG, "%s: bad order %d", f, a->order);
  if (a->gate && a->activation != GDN_ACT_SILU && a->activation != GDN_ACT_SIGMOID)
    return fail(GDN_ERR_INVALID_ARG, "%s: a gate's activation is SiLU or sigmoid (got %d)", f, a->activation);
  if (a->heads < 1 || a->tokens < 0 || a->tokens > INT32_MAX / a->heads)
    return fail(GDN_ERR_INVALID_ARG, "%s: heads >= 1 and 0 <= tokens * heads < 2^31 required", f);
  if (a->width < 1) return fail(GDN_ERR_INVALID_ARG, "%s: width %d < 1", f, a->width);
  if (a->width > 16384) return fail(GDN_ERR_UNSUPPORTED, "%s: width %d > 16384", f, a->width);
  if (!(a->eps >= 0) || !std::isfinite(a->eps)) return fail(GDN_ERR_INVALID_ARG, "%s: bad eps", f);
  if (!aligned(a->weight, esize(a->weight_dtype))) return fail(GDN_ERR_ALIGNMENT, "%s: misaligned weight", f);
  return GDN_OK;
}

// A row tensor's stride and alignment; an absent one passes.
gdn_status check_rows(const char* f, const char* name, const void* p, int64_t stride, int64_t tokens, int64_t width, size_t es) {
  if (!p || !tokens) return GDN_OK;
  if (tokens > 1 && stride < width) return fail(GDN_ERR_INVALID_ARG, "%s: token stride of %s smaller than a token's heads", f, name);
  if (!aligned(p, es)) return fail(GDN_ERR_ALIGNMENT, "%s: misaligned %s", f, name);
  return GDN_OK;
}

}  // namespace

extern "C" {

gdn_status gdn_rms_norm(const gdn_rms_norm_args* a, void* stream) {
  const char* f = "gdn_rms_norm";
  try {
    gdn_status st = check_norm(a, f);
    if (st != GDN_OK) return st;
    if (a->tokens > 0 && (!a->x || !a->y)) return fail(GDN_ERR_INVALID_ARG, "%s: x and y are required", f);
    const bool sums = a->order == GDN_NORM_PRE && a->residual;
    if (a->tokens > 0 && sums != (a->sum != nullptr))
      return fail(GDN_ERR_INVALID_ARG, "%s: sum goes with a residual in the pre order, and with nothing else", f);
    if (a->order == GDN_NORM_PRE && !a->residual && a->scale != 1.0f)
      return fail(GDN_ERR_INVALID_ARG, "%s: the pre order scales x only where it is added to a residual", f);
    const size_t es = esize(a->dtype);
    const int64_t w = (int64_t)a->heads * a->width;
    auto rows = [&](const char* name, const void* p, int64_t stride) {
      return Tensor{name, Rows{p, (size_t)a->tokens, (size_t)w * es, (size_t)stride * es}};
    };
    const Tensor ins[] = {rows("x", a->x, a->x_stride), rows("gate", a->gate, a->gate_stride),
                          rows("residual", a->residual, a->residual_stride)};
    const Tensor outs[] = {rows("y", a->y, a->y_stride), rows("sum", a->sum, a->sum_stride)};
    const int64_t strides[] = {a->x_stride, a->gate_stride, a->residual_stride, a->y_stride, a->sum_stride};
    for (int i = 0; i < 5; ++i) {
      const Tensor& t = i < 3 ? ins[i] : outs[i - 3];
      st = check_rows(f, t.name, t.rows.p, strides[i], a->tokens, w, es);
      if (st != GDN_OK) return st;
    }
    if (const char* n = clash(ins, outs, true)) return fail(GDN_ERR_INVALID_ARG, "%s: %s overlaps another tensor", f, n);
    for (const Tensor& t : outs)
      if (overlaps(t.rows.p, t.rows.span(), a->weight, a->weight ? (size_t)a->width * esize(a->weight_dtype) : 0))
        return fail(GDN_ERR_INVALID_ARG, "%s: %s overlaps the weight", f, t.name);
    gdn::NormParams p{a->x, a->weight, a->gate, a->residual, a->y, a->sum, a->x_stride, a->gate_stride,
                      a->residual_stride, a->y_stride, a->sum_stride, a->tokens * a->heads, a->heads, a->width,
                      a->order, a->activation, a->weight_dtype == GDN_BF16 ? 1 : 0, a->eps, a->scale,
                      a->weight_offset};
    hipStream_t s = static_cast<hipStream_t>(stream);
    return finish(gdn::launch_norm(p, a->dtype, s), s, f);
  } catch (...) {
    return fail(GDN_ERR_HIP, "%s: internal error", f);
  }
}

size_t gdn_rms_norm_backward_workspace_size(const gdn_rms_norm_backward_args* a) {
  if (!a || a->struct_size < sizeof(*a) || a->heads < 1 || a->tokens < 0 || a->tokens > INT32_MAX / a->heads ||
      a->width < 1 || a->width > 16384)
    return 0;
  return gdn::norm_backward_workspace_bytes(a->tokens * a->heads, a->width);
}

gdn_status gdn_rms_norm_backward(const gdn_rms_norm_backward_args* a, void* stream) {
  const char* f = "gdn_rms_norm_backward";
  try {
    gdn_status st = check_norm(a, f);
    if (st != GDN_OK) return st;
    if (a->tokens > 0 && (!a->x || !a->dy)) return fail(GDN_ERR_INVALID_ARG, "%s: x and dy are required", f);
    if (a->tokens > 0 && (a->gate != nullptr) != (a->dgate != nullptr))
      return fail(GDN_ERR_INVALID_ARG, "%s: dgate goes with a gate", f);
    if (a->order == GDN_NORM_POST && (a->d_sum || a->d_residual))
      return fail(GDN_ERR_INVALID_ARG, "%s: d_sum and d_residual belong to the pre order", f);
    if (a->dweight && !a->weight) return fail(GDN_ERR_INVALID_ARG, "%s: dweight needs weight", f);
    const size_t es = esize(a->dtype);
    const int64_t w = (int64_t)a->heads * a->width;
    auto rows = [&](const char* name, const void* p, int64_t stride) {
      return Tensor{name, Rows{p, (size_t)a->tokens, (size_t)w * es, (size_t)stride * es}};
    };
    const Tensor ins[] = {rows("x", a->x, a->x_stride), rows("gate", a->gate, a->gate_stride),
                          rows("dy", a->dy, a->dy_stride), rows("d_sum", a->d_sum, a->d_sum_stride)};
    const Tensor outs[] = {rows("dx", a->dx, a->dx_stride), rows("d_residual", a->d_residual, a->d_residual_stride),
                           rows("dgate", a->dgate, a->dgate_stride)};
    const int64_t strides[] = {a->x_stride, a->gate_stride, a->dy_stride, a->d_sum_stride, a->dx_stride,
                               a->d_residual_stride, a->dgate_stride};
    for (int i = 0; i < 7; ++i) {
      const Tensor& t = i < 4 ? ins[i] : outs[i - 4];
      st = check_rows(f, t.name, t.rows.p, strides[i], a->tokens, w, es);
      if (st != GDN_OK) return st;
    }
    if (const char* n = clash(ins, outs, true)) return fail(GDN_ERR_INVALID_ARG, "%s: %s overlaps another tensor", f, n);
    const size_t wb = a->weight ? (size_t)a->width * esize(a->weight_dtype) : 0, db = a->dweight ? (size_t)a->width * 4 : 0;
    const size_t need = a->dweight ? gdn::norm_backward_workspace_bytes(a->tokens * a->heads, a->width) : 0;
    if (!aligned(a->dweight, 4)) return fail(GDN_ERR_ALIGNMENT, "%s: misaligned dweight", f);
    if (need && (!a->workspace || a->workspace_bytes < need))
      return fail(GDN_ERR_WORKSPACE, "%s: workspace of %zu bytes required", f, need);
    if (need && !aligned(a->workspace, 256)) return fail(GDN_ERR_ALIGNMENT, "%s: workspace must be 256-byte aligned", f);
    if (overlaps(a->dweight, db, a->weight, wb)) return fail(GDN_ERR_INVALID_ARG, "%s: dweight overlaps the weight", f);
    if (overlaps(a->dweight, db, a->workspace, need) || overlaps(a->weight, wb, a->workspace, need))
      return fail(GDN_ERR_INVALID_ARG, "%s: the workspace overlaps a tensor", f);
    for (int i = 0; i < 7; ++i) {
      const Tensor& t = i < 4 ? ins[i] : outs[i - 4];
      if (overlaps(t.rows.p, t.rows.span(), a->dweight, db) || overlaps(t.rows.p, t.rows.span(), a->workspace, need) ||
          (i >= 4 && overlaps(t.rows.p, t.rows.span(), a->weight, wb)))
        return fail(GDN_ERR_INVALID_ARG, "%s: %s overlaps another tensor", f, t.name);
    }
    gdn::NormBwdParams p{a->x, a->weight, a->gate, a->dy, a->d_sum, a->dx, a->d_residual, a->dgate, a->dweight,
                         a->x_stride, a->gate_stride, a->dy_stride, a->d_sum_stride, a->dx_stride,
                         a->d_residual_stride, a->dgate_stride, a->tokens * a->heads, a->heads, a->width, a->order,
                         a->activation, a->weight_dtype == GDN_BF16 ? 1 : 0, a->eps, a->scale, a->weight_offset,
                         a->workspace};
    hipStream_t s = static_cast<hipStream_t>(stream);
    return finish(gdn::launch_norm_backward(p, a->dtype, s), s, f);
  } catch (...) {
    return fail(GDN_ERR_HIP, "%s: internal error", f);
  }
}

}  // extern "C"
