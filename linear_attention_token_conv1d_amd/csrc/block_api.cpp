// C ABI of the operators around the mixer in a hybrid block: norms with their
// residual and gate, rotary positions, the 8-bit cache and attention over it.  Arguments are checked completely before any launch, as
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

// What gdn_cache_store and gdn_cache_attention share: the pool, its table and its sequences.
template <typename A>
gdn_status check_cache(const A* a, const char* f) {
  if (!a) return fail(GDN_ERR_INVALID_ARG, "%s: args is NULL", f);
  if (a->struct_size < sizeof(A)) return fail(GDN_ERR_INVALID_ARG, "%s: struct_size %u < %zu", f, a->struct_size, sizeof(A));
  if (!is_dtype(a->io_dtype)) return fail(GDN_ERR_INVALID_ARG, "%s: bad io_dtype %d", f, a->io_dtype);
  if (a->n_seqs < 1 || a->tokens < 0) return fail(GDN_ERR_INVALID_ARG, "%s: n_seqs >= 1 and tokens >= 0 required", f);
  if (a->h_kv < 1 || a->h_kv > 65535) return fail(GDN_ERR_INVALID_ARG, "%s: h_kv %d not in 1..65535", f, a->h_kv);
  if (a->d != 64 && a->d != 128 && a->d != 256) return fail(GDN_ERR_UNSUPPORTED, "%s: d %d not in {64, 128, 256}", f, a->d);
  if (a->page_size != 16 && a->page_size != 32 && a->page_size != 64 && a->page_size != 128 && a->page_size != 256)
    return fail(GDN_ERR_UNSUPPORTED, "%s: page_size %d not in {16, 32, 64, 128, 256}", f, a->page_size);
  if (a->pages < 1 || a->max_pages < 1) return fail(GDN_ERR_INVALID_ARG, "%s: pages and max_pages >= 1 required", f);
  if (a->tokens > 0 && (!a->k_cache || !a->v_cache || !a->k_scale || !a->v_scale || !a->page_table || !a->lens))
    return fail(GDN_ERR_INVALID_ARG, "%s: k_cache, v_cache, k_scale, v_scale, page_table and lens are required", f);
  if (!a->cu_seqlens && a->tokens % a->n_seqs)
    return fail(GDN_ERR_INVALID_ARG, "%s: without cu_seqlens every sequence has tokens / n_seqs new tokens", f);
  // tile and page numbers of a pack are 32-bit
  if (a->tokens > INT32_MAX / 2 || a->n_seqs > INT32_MAX / 4)
    return fail(GDN_ERR_INVALID_ARG, "%s: too many tokens or sequences", f);
  if (!aligned(a->k_cache, 16) || !aligned(a->v_cache, 16))
    return fail(GDN_ERR_ALIGNMENT, "%s: k_cache and v_cache must be 16-byte aligned", f);
  if (!aligned(a->k_scale, 4) || !aligned(a->v_scale, 4) || !aligned(a->page_table, 4) || !aligned(a->lens, 4) ||
      !aligned(a->cu_seqlens, 4))
    return fail(GDN_ERR_ALIGNMENT, "%s: scales, page_table, lens and cu_seqlens must be 4-byte aligned", f);
  return GDN_OK;
}

// A row tensor that is read or written 16 bytes at a time.
gdn_status check_wide(const char* f, const char* name, const void* p, int64_t stride, int64_t tokens, int64_t width, size_t es) {
  gdn_status st = check_rows(f, name, p, stride, tokens, width, es);
  if (st != GDN_OK || !p || !tokens) return st;
  if (!aligned(p, 16) || (tokens > 1 && stride % 8))
    return fail(GDN_ERR_ALIGNMENT, "%s: %s must be 16-byte aligned, its token stride a multiple of 8 elements", f, name);
  return GDN_OK;
}

bool attend_shape(const gdn_cache_attention_args* a, gdn::AttendShape* s) {
  if (a->h_q < 1 || a->h_kv < 1 || a->h_q % a->h_kv || a->tokens < 0 || a->n_seqs < 1 || a->max_pages < 1 ||
      a->tokens > INT32_MAX / (a->h_q / a->h_kv) / 2)
    return false;
  *s = gdn::AttendShape{a->tokens, a->n_seqs, a->h_q, a->h_kv, a->d, a->page_size, a->max_pages, a->cu_seqlens ? 1 : 0,
                        a->io_dtype == GDN_BF16 ? 1 : 0, a->causal, a->window};
  return true;
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

gdn_status gdn_rope(const gdn_rope_args* a, void* stream) {
  const char* f = "gdn_rope";
  try {
    if (!a) return fail(GDN_ERR_INVALID_ARG, "%s: args is NULL", f);
    if (a->struct_size < sizeof(*a)) return fail(GDN_ERR_INVALID_ARG, "%s: struct_size %u < %zu", f, a->struct_size, sizeof(*a));
    if (!is_dtype(a->dtype)) return fail(GDN_ERR_INVALID_ARG, "%s: bad dtype %d", f, a->dtype);
    if (a->layout != GDN_ROPE_HALF && a->layout != GDN_ROPE_INTERLEAVED)
      return fail(GDN_ERR_INVALID_ARG, "%s: bad layout %d", f, a->layout);
    if (a->inverse != 0 && a->inverse != 1) return fail(GDN_ERR_INVALID_ARG, "%s: inverse is 0 or 1", f);
    if (a->position_bits != 32 && a->position_bits != 64) return fail(GDN_ERR_INVALID_ARG, "%s: position_bits is 32 or 64", f);
    if (a->h_q < 1 || a->h_k < 0 || a->h_q > 65535 || a->h_k > 65535)
      return fail(GDN_ERR_INVALID_ARG, "%s: h_q in 1..65535 and h_k in 0..65535 required", f);
    if (a->d < 2 || a->d > 16384) return fail(GDN_ERR_INVALID_ARG, "%s: d %d not in 2..16384", f, a->d);
    if (a->rot < 2 || a->rot % 2 || a->rot > a->d) return fail(GDN_ERR_INVALID_ARG, "%s: rot %d is not even in 2..d", f, a->rot);
    if (!std::isfinite(a->mscale)) return fail(GDN_ERR_INVALID_ARG, "%s: bad mscale", f);
    if (a->tokens < 0 || a->tokens > INT32_MAX) return fail(GDN_ERR_INVALID_ARG, "%s: tokens out of range", f);
    if (a->tokens > 0 && (!a->q || !a->q_out || !a->positions || !a->inv_freq || (a->h_k > 0 && (!a->k || !a->k_out))))
      return fail(GDN_ERR_INVALID_ARG, "%s: q, q_out, positions, inv_freq and, with h_k, k and k_out are required", f);
    if (a->h_k == 0 && (a->k || a->k_out)) return fail(GDN_ERR_INVALID_ARG, "%s: k and k_out go with h_k > 0", f);
    if (!aligned(a->positions, a->position_bits / 8) || !aligned(a->inv_freq, 8))
      return fail(GDN_ERR_ALIGNMENT, "%s: misaligned positions or inv_freq", f);
    const size_t es = esize(a->dtype);
    const int64_t wq = (int64_t)a->h_q * a->d, wk = (int64_t)a->h_k * a->d;
    auto rows = [&](const char* name, const void* p, int64_t stride, int64_t w) {
      return Tensor{name, Rows{p, (size_t)a->tokens, (size_t)w * es, (size_t)stride * es}};
    };
    const Tensor ins[] = {rows("q", a->q, a->q_stride, wq), rows("k", a->k, a->k_stride, wk)};
    const Tensor outs[] = {rows("q_out", a->q_out, a->q_out_stride, wq), rows("k_out", a->k_out, a->k_out_stride, wk)};
    const int64_t strides[] = {a->q_stride, a->k_stride, a->q_out_stride, a->k_out_stride};
    for (int i = 0; i < 4; ++i) {
      const Tensor& t = i < 2 ? ins[i] : outs[i - 2];
      const gdn_status st = check_rows(f, t.name, t.rows.p, strides[i], a->tokens, i % 2 ? wk : wq, es);
      if (st != GDN_OK) return st;
    }
    if (a->tokens > 0) {
      for (int i = 0; i < 2; ++i) {  // an output may be its own input, and shares nothing else
        const Tensor other[] = {ins[1 - i]};
        const Tensor own[] = {ins[i]};
        const Tensor out[] = {outs[i]};
        if (clash(own, out, true) || clash(other, out, false) || (i == 1 && rows_overlap(outs[0].rows, outs[1].rows)))
          return fail(GDN_ERR_INVALID_ARG, "%s: %s overlaps another tensor", f, outs[i].name);
        if (overlaps(outs[i].rows.p, outs[i].rows.span(), a->positions, (size_t)a->tokens * (a->position_bits / 8)) ||
            overlaps(outs[i].rows.p, outs[i].rows.span(), a->inv_freq, (size_t)a->rot / 2 * 8))
          return fail(GDN_ERR_INVALID_ARG, "%s: %s overlaps positions or inv_freq", f, outs[i].name);
      }
    }
    gdn::RopeParams p{a->q, a->k, a->positions, a->inv_freq, a->q_out, a->k_out, a->q_stride, a->k_stride,
                      a->q_out_stride, a->k_out_stride, a->tokens, a->position_bits == 64 ? 1 : 0, a->h_q, a->h_k, a->d,
                      a->rot, a->layout == GDN_ROPE_HALF ? 1 : 0, a->inverse, a->mscale, 0};
    hipStream_t s = static_cast<hipStream_t>(stream);
    return finish(gdn::launch_rope(p, a->dtype, s), s, f);
  } catch (...) {
    return fail(GDN_ERR_HIP, "%s: internal error", f);
  }
}

gdn_status gdn_cache_store(const gdn_cache_store_args* a, void* stream) {
  const char* f = "gdn_cache_store";
  try {
    gdn_status st = check_cache(a, f);
    if (st != GDN_OK) return st;
    if (a->tokens > 0 && (!a->k || !a->v)) return fail(GDN_ERR_INVALID_ARG, "%s: k and v are required", f);
    const size_t es = esize(a->io_dtype);
    const int64_t w = (int64_t)a->h_kv * a->d;
    st = check_wide(f, "k", a->k, a->k_stride, a->tokens, w, es);
    if (st == GDN_OK) st = check_wide(f, "v", a->v, a->v_stride, a->tokens, w, es);
    if (st != GDN_OK) return st;
    struct R { const char* name; const void* p; size_t n; };
    const size_t T = (size_t)a->tokens, pool = (size_t)a->pages * w * a->page_size, sc = (size_t)a->pages * a->h_kv * 4;
    const R ins[] = {{"k", a->k, T ? ((T - 1) * a->k_stride + w) * es : 0}, {"v", a->v, T ? ((T - 1) * a->v_stride + w) * es : 0},
                     {"page_table", a->page_table, (size_t)a->n_seqs * a->max_pages * 4}, {"lens", a->lens, (size_t)a->n_seqs * 4},
                     {"cu_seqlens", a->cu_seqlens, ((size_t)a->n_seqs + 1) * 4}};
    const R outs[] = {{"k_cache", a->k_cache, pool}, {"v_cache", a->v_cache, pool}, {"k_scale", a->k_scale, sc}, {"v_scale", a->v_scale, sc}};
    for (int o = 0; o < 4 && T; ++o) {
      for (const R& i : ins)
        if (overlaps(outs[o].p, outs[o].n, i.p, i.n)) return fail(GDN_ERR_INVALID_ARG, "%s: %s overlaps %s", f, outs[o].name, i.name);
      for (int k = 0; k < o; ++k)
        if (overlaps(outs[o].p, outs[o].n, outs[k].p, outs[k].n))
          return fail(GDN_ERR_INVALID_ARG, "%s: %s overlaps %s", f, outs[o].name, outs[k].name);
    }
    gdn::CacheStoreParams p{a->k, a->v, static_cast<uint8_t*>(a->k_cache), static_cast<uint8_t*>(a->v_cache), a->k_scale,
                            a->v_scale, a->page_table, a->lens, a->cu_seqlens, a->k_stride, a->v_stride, a->tokens, a->n_seqs,
                            a->h_kv, a->d, a->page_size, a->pages, a->max_pages, 0, 0};
    hipStream_t s = static_cast<hipStream_t>(stream);
    return finish(gdn::launch_cache_store(p, a->io_dtype, s), s, f);
  } catch (...) {
    return fail(GDN_ERR_HIP, "%s: internal error", f);
  }
}

size_t gdn_cache_attention_workspace_size(const gdn_cache_attention_args* a) {
  gdn::AttendShape s;
  if (!a || a->struct_size < sizeof(*a) || a->page_size < 1 || a->d < 1 || !attend_shape(a, &s)) return 0;
  return gdn::attend_workspace_bytes(s);
}

gdn_status gdn_cache_attention(const gdn_cache_attention_args* a, void* stream) {
  const char* f = "gdn_cache_attention";
  try {
    gdn_status st = check_cache(a, f);
    if (st != GDN_OK) return st;
    gdn::AttendShape shape;
    if (a->h_q < 1 || a->h_q % a->h_kv)
      return fail(GDN_ERR_INVALID_ARG, "%s: h_q (%d) must be a positive multiple of h_kv (%d)", f, a->h_q, a->h_kv);
    if (!attend_shape(a, &shape)) return fail(GDN_ERR_INVALID_ARG, "%s: too many rows", f);
    if (a->causal != 0 && a->causal != 1) return fail(GDN_ERR_INVALID_ARG, "%s: causal is 0 or 1", f);
    if (a->window < 0) return fail(GDN_ERR_INVALID_ARG, "%s: window %d < 0", f, a->window);
    if (!(a->scale > 0) || !std::isfinite(a->scale * 1.4426950408889634f)) return fail(GDN_ERR_INVALID_ARG, "%s: scale must be positive and finite", f);
    if (a->tokens > 0 && (!a->q || !a->o)) return fail(GDN_ERR_INVALID_ARG, "%s: q and o are required", f);
    const size_t es = esize(a->io_dtype);
    const int64_t w = (int64_t)a->h_q * a->d;
    st = check_wide(f, "q", a->q, a->q_stride, a->tokens, w, es);
    if (st == GDN_OK) st = check_wide(f, "gate", a->gate, a->gate_stride, a->tokens, w, es);
    if (st == GDN_OK) st = check_wide(f, "o", a->o, a->o_stride, a->tokens, w, es);
    if (st != GDN_OK) return st;
    if (!aligned(a->lse, 4)) return fail(GDN_ERR_ALIGNMENT, "%s: misaligned lse", f);
    const size_t need = gdn::attend_workspace_bytes(shape);
    if (need && (!a->workspace || a->workspace_bytes < need))
      return fail(GDN_ERR_WORKSPACE, "%s: workspace of %zu bytes required", f, need);
    if (need && !aligned(a->workspace, 256)) return fail(GDN_ERR_ALIGNMENT, "%s: workspace must be 256-byte aligned", f);
    const size_t T = (size_t)a->tokens, wb = (size_t)w * es;
    const Rows q{a->q, T, wb, (size_t)a->q_stride * es}, gate{a->gate, T, wb, (size_t)a->gate_stride * es},
        o{a->o, T, wb, (size_t)a->o_stride * es};
    const size_t kv = (size_t)a->h_kv * a->d, pool = (size_t)a->pages * kv * a->page_size, sc = (size_t)a->pages * a->h_kv * 4;
    const Rows lse{a->lse, a->lse ? 1u : 0u, T * a->h_q * 4, T * a->h_q * 4}, ws{a->workspace, need ? 1u : 0u, need, need};
    const Rows other[] = {{a->k_cache, 1, pool, pool}, {a->v_cache, 1, pool, pool}, {a->k_scale, 1, sc, sc}, {a->v_scale, 1, sc, sc},
                          {a->page_table, 1, (size_t)a->n_seqs * a->max_pages * 4, 4}, {a->lens, 1, (size_t)a->n_seqs * 4, 4},
                          {a->cu_seqlens, a->cu_seqlens ? 1u : 0u, ((size_t)a->n_seqs + 1) * 4, 4}};
    if (T) {
      // o may be q itself: a tile's rows are read whole by the workgroup that writes them, unless pieces of a
      // context read them while others are being joined, which happens behind all of them
      if (rows_overlap(o, q) && !(a->o == a->q && a->o_stride == a->q_stride))
        return fail(GDN_ERR_INVALID_ARG, "%s: o overlaps q", f);
      const Rows outs[] = {o, lse, ws};
      for (int i = 0; i < 3; ++i) {
        bool bad = rows_overlap(outs[i], gate) || (i > 0 && (rows_overlap(outs[i], q) || rows_overlap(outs[i], o))) ||
                   (i == 2 && rows_overlap(ws, lse));
        for (const Rows& r : other) bad = bad || rows_overlap(outs[i], r);
        if (bad) return fail(GDN_ERR_INVALID_ARG, "%s: o, lse or the workspace overlaps another tensor", f);
      }
    }
    int shift = 4;
    while ((1 << shift) < a->page_size) ++shift;
    gdn::AttendParams p{a->q, static_cast<const uint8_t*>(a->k_cache), static_cast<const uint8_t*>(a->v_cache), a->k_scale,
                        a->v_scale, a->page_table, a->lens, a->cu_seqlens, a->gate, a->o, a->lse, a->q_stride, a->gate_stride,
                        a->o_stride, a->tokens, a->n_seqs, a->h_q, a->h_kv, shift, a->pages, a->max_pages, a->causal,
                        a->window, a->scale * 1.44269504088896340736f, 0, 0, 0, 0, 0, 0, 0, 0, nullptr, nullptr, nullptr};
    hipStream_t s = static_cast<hipStream_t>(stream);
    return finish(gdn::launch_attend(p, shape, a->workspace, a->io_dtype, s), s, f);
  } catch (...) {
    return fail(GDN_ERR_HIP, "%s: internal error", f);
  }
}

}  // extern "C"
