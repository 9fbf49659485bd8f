// Python binding of the operators around the mixer: the checks of torch-level
// properties (device, dtype, shape, strides), the outputs and the C argument
// structs of block.py's functions, in C++.  A call of a single token is over
// in the time that the same checks take in Python: they would be what it
// waits for.  Nothing is computed here.
//
// Every function takes the positional arguments of its namesake in block.py
// and raises GdnError (given to init) as the rest of the package does.
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <ATen/ops/empty.h>
#include <ATen/ops/empty_like.h>

#include <cmath>
#include <string>

#include "../../include/gdn.h"

namespace {

PyObject *g_error, *g_stream_of, *g_device, *g_set_device;

struct Raised {};  // a Python exception has been set

[[noreturn]] void raise(const std::string& what) {
  PyErr_SetString(g_error, what.c_str());
  throw Raised();
}

std::string text(at::IntArrayRef v) {
  std::string s = "[";
  for (size_t i = 0; i < v.size(); ++i) s += (i ? ", " : "") + std::to_string(v[i]);
  return s + "]";
}
std::string name_of(at::ScalarType t) {
  switch (t) {
    case at::kFloat: return "torch.float32";
    case at::kBFloat16: return "torch.bfloat16";
    case at::kInt: return "torch.int32";
    case at::kLong: return "torch.int64";
    case at::kDouble: return "torch.float64";
    case at::kFloat8_e4m3fn: return "torch.float8_e4m3fn";
    case at::kByte: return "torch.uint8";
    default: return at::toString(t);
  }
}

bool is_io(at::ScalarType t) { return t == at::kFloat || t == at::kBFloat16; }
int32_t dtype_of(at::ScalarType t) { return t == at::kBFloat16 ? GDN_BF16 : GDN_F32; }

// An argument that is a tensor or None.
const at::Tensor* tensor(PyObject* o, const char* name) {
  if (o == Py_None) return nullptr;
  if (!THPVariable_Check(o)) raise(std::string(name) + " must be a tensor");
  return &THPVariable_Unpack(o);
}
// The argument whose GPU the call runs on.
const at::Tensor& first(PyObject* o, const char* name) {
  const at::Tensor* t = o != Py_None && THPVariable_Check(o) ? &THPVariable_Unpack(o) : nullptr;
  if (!t || !t->is_cuda() || t->layout() != at::kStrided) raise(std::string(name) + " must be a GPU tensor");
  return *t;
}

void check(const at::Tensor& t, const char* name, int64_t index, at::IntArrayRef shape, at::ScalarType dtype) {
  if (!t.is_cuda() || t.get_device() != index || t.layout() != at::kStrided)
    raise(std::string(name) + " must be on the same GPU as the call's other tensors");
  if (t.scalar_type() != dtype) raise(std::string(name) + " must be " + name_of(dtype) + ", got " + name_of(t.scalar_type()));
  if (t.sizes() != shape) raise(std::string(name) + " must be " + text(shape) + ", got " + text(t.sizes()));
}

// An optional contiguous tensor: its address.
void* whole(const at::Tensor* t, const char* name, int64_t index, at::IntArrayRef shape, at::ScalarType dtype) {
  if (!t) return nullptr;
  check(*t, name, index, shape, dtype);
  if (!t->is_contiguous()) raise(std::string(name) + " must be contiguous");
  return t->data_ptr();
}

// An optional [T, H, d] or [T, d] tensor, token stride free.
struct Rows {
  void* p = nullptr;
  int64_t stride = 0;
};
Rows rows(const at::Tensor* t, const char* name, int64_t index, at::IntArrayRef shape, at::ScalarType dtype) {
  if (!t) return {};
  check(*t, name, index, shape, dtype);
  const size_t n = shape.size();
  const int64_t width = n == 3 ? shape[1] * shape[2] : shape[1];
  if (t->is_contiguous()) return {t->data_ptr(), width};
  // a stride over one element says nothing about the layout
  if ((t->stride(n - 1) != 1 && shape[n - 1] > 1) || (n == 3 && t->stride(1) != shape[2] && shape[1] > 1))
    raise(std::string(name) + " must have contiguous heads inside a token");
  return {t->data_ptr(), t->stride(0)};
}

int word(PyObject* o, const char* name, const char* a, const char* b) {
  if (PyUnicode_Check(o)) {
    if (PyUnicode_CompareWithASCIIString(o, a) == 0) return 0;
    if (PyUnicode_CompareWithASCIIString(o, b) == 0) return 1;
  }
  raise(std::string(name) + " must be '" + a + "' or '" + b + "'");
}
float number(PyObject* o) {
  const double v = PyFloat_AsDouble(o);
  if (v == -1.0 && PyErr_Occurred()) throw Raised();
  return (float)v;
}
int32_t whole_number(PyObject* o, const char* name) {
  const long long v = PyLong_AsLongLong(o);
  if (v == -1 && PyErr_Occurred()) throw Raised();
  if (v < INT32_MIN || v > INT32_MAX) raise(std::string(name) + " out of range");
  return (int32_t)v;
}
bool truth(PyObject* o) {
  const int v = PyObject_IsTrue(o);
  if (v < 0) throw Raised();
  return v != 0;
}

// A GPU made the current device for one call, where it is another.
struct OnDevice {
  PyObject* before = nullptr;
  explicit OnDevice(int64_t index) {
    PyObject* now = PyObject_CallNoArgs(g_device);
    if (!now) throw Raised();
    if (PyLong_AsLongLong(now) == index) {
      Py_DECREF(now);
      return;
    }
    before = now;
    set(index);
  }
  static void set(int64_t index) {
    PyObject* i = PyLong_FromLongLong(index);
    PyObject* r = i ? PyObject_CallOneArg(g_set_device, i) : nullptr;
    Py_XDECREF(i);
    if (!r) throw Raised();
    Py_DECREF(r);
  }
  ~OnDevice() {
    if (!before) return;
    PyObject *type, *value, *trace;
    PyErr_Fetch(&type, &value, &trace);
    PyObject* r = PyObject_CallOneArg(g_set_device, before);
    Py_XDECREF(r);
    Py_DECREF(before);
    PyErr_Restore(type, value, trace);
  }
};

template <typename A>
void run(const char* name, gdn_status (*entry)(const A*, void*), const A& args, int64_t index) {
  OnDevice on(index);
  PyObject* i = PyLong_FromLongLong(index);
  PyObject* s = i ? PyObject_CallOneArg(g_stream_of, i) : nullptr;
  Py_XDECREF(i);
  if (!s) throw Raised();
  void* stream = PyLong_AsVoidPtr(s);
  Py_DECREF(s);
  if (PyErr_Occurred()) throw Raised();
  gdn_status status;
  Py_BEGIN_ALLOW_THREADS;
  status = entry(&args, stream);
  Py_END_ALLOW_THREADS;
  if (status != GDN_OK) raise(std::string(name) + ": " + gdn_status_string(status) + ": " + gdn_last_error());
}

// The caller's workspace where it is large enough, else a new one.
at::Tensor workspace(PyObject* given, size_t need, int64_t index, const at::Tensor& like) {
  if (const at::Tensor* t = tensor(given, "workspace")) {
    if (!t->is_cuda() || t->get_device() != index || t->scalar_type() != at::kByte)
      raise("workspace must be a torch.uint8 tensor on the call's GPU");
    if ((size_t)t->numel() >= need && t->is_contiguous()) return *t;
  }
  return at::empty({(int64_t)need}, like.options().dtype(at::kByte));
}

PyObject* wrap(const at::Tensor& t) { return t.defined() ? THPVariable_Wrap(t) : (Py_INCREF(Py_None), Py_None); }
PyObject* tuple(std::initializer_list<at::Tensor> ts) {
  PyObject* r = PyTuple_New((Py_ssize_t)ts.size());
  if (!r) throw Raised();
  Py_ssize_t i = 0;
  for (const at::Tensor& t : ts) {
    PyObject* o = wrap(t);
    if (!o) {
      Py_DECREF(r);
      throw Raised();
    }
    PyTuple_SET_ITEM(r, i++, o);
  }
  return r;
}
// An output: the caller's, or new, laid out like `like`.
at::Tensor output(PyObject* given, const char* name, const at::Tensor& like) {
  const at::Tensor* t = tensor(given, name);
  return t ? *t : at::empty_like(like);
}

// What both norms check of their arguments.
struct Norm {
  const at::Tensor& x;
  const at::Tensor *weight, *gate;
  int64_t index;
  at::ScalarType dt;
  int32_t order, act, heads, width;
  Norm(PyObject* px, PyObject* pw, PyObject* pg, PyObject* porder, PyObject* pact) : x(first(px, "x")) {
    dt = x.scalar_type();
    if (!is_io(dt)) raise("x must be torch.bfloat16 or torch.float32, got " + name_of(dt));
    if (x.dim() != 2 && x.dim() != 3) raise("x must be [T, D] or [T, H, D]");
    index = x.get_device();
    const int64_t h = x.dim() == 3 ? x.size(1) : 1, w = x.size(-1);
    if (h > INT32_MAX || w > INT32_MAX) raise("x is too wide");
    heads = (int32_t)h, width = (int32_t)w;
    order = word(porder, "order", "pre", "post");
    gate = tensor(pg, "gate");
    act = gate ? (word(pact, "activation", "silu", "sigmoid") ? GDN_ACT_SIGMOID : GDN_ACT_SILU) : GDN_ACT_NONE;
    weight = tensor(pw, "weight");
    if (weight && !is_io(weight->scalar_type())) raise("weight must be a torch.bfloat16 or torch.float32 tensor");
  }
  const void* weight_at() const { return weight ? whole(weight, "weight", index, {width}, weight->scalar_type()) : nullptr; }
  int32_t weight_dtype() const { return weight ? dtype_of(weight->scalar_type()) : GDN_F32; }
};

// (x, weight, gate, residual, order, activation, scale, eps, weight_offset, out, sum_out)
PyObject* rms_norm(PyObject* const* a) {
  const Norm n(a[0], a[1], a[2], a[4], a[5]);
  const at::IntArrayRef shape = n.x.sizes();
  const at::Tensor* residual = tensor(a[3], "residual");
  const bool sums = residual && n.order == GDN_NORM_PRE;
  if (!sums && a[10] != Py_None) raise("sum_out goes with a residual in the pre order");
  const at::Tensor y = output(a[9], "out", n.x), sum = sums ? output(a[10], "sum_out", *residual) : at::Tensor();
  const Rows x = rows(&n.x, "x", n.index, shape, n.dt), g = rows(n.gate, "gate", n.index, shape, n.dt),
             r = rows(residual, "residual", n.index, shape, n.dt), o = rows(&y, "out", n.index, shape, n.dt),
             s = rows(sums ? &sum : nullptr, "sum_out", n.index, shape, n.dt);
  const gdn_rms_norm_args args = {sizeof(gdn_rms_norm_args), dtype_of(n.dt), n.weight_dtype(), n.order, n.act, n.heads, n.width,
                                  number(a[7]), number(a[6]), number(a[8]), shape[0], x.p, n.weight_at(), g.p, r.p, o.p, s.p,
                                  x.stride, g.stride, r.stride, o.stride, s.stride};
  run("gdn_rms_norm", gdn_rms_norm, args, n.index);
  return sums ? tuple({y, sum}) : wrap(y);
}

// (x, dy, weight, gate, d_sum, residual, order, activation, scale, eps, weight_offset, dx, dgate, workspace)
PyObject* rms_norm_backward(PyObject* const* a) {
  const Norm n(a[0], a[2], a[3], a[6], a[7]);
  const at::IntArrayRef shape = n.x.sizes();
  const at::Tensor *dy = tensor(a[1], "dy"), *d_sum = tensor(a[4], "d_sum");
  if (!dy) raise("dy is required");
  const bool residual = truth(a[5]) || d_sum;
  const float scale = number(a[8]);
  if (residual && n.order == GDN_NORM_POST)
    raise("residual and d_sum belong to the pre order: in the post order the residual's gradient is dy");
  if (n.order == GDN_NORM_PRE && !residual && scale != 1.f) raise("the pre order scales x only where it is added to a residual");
  if (!n.gate && a[12] != Py_None) raise("dgate goes with a gate");
  const at::Tensor dx = output(a[11], "dx", n.x), dres = !residual ? at::Tensor() : scale == 1.f ? dx : at::empty_like(n.x),
                   dgate = n.gate ? output(a[12], "dgate", *n.gate) : at::Tensor();
  const bool own = residual && scale != 1.f;  // the sum's gradient is not that of x
  const Rows x = rows(&n.x, "x", n.index, shape, n.dt), g = rows(n.gate, "gate", n.index, shape, n.dt),
             d = rows(dy, "dy", n.index, shape, n.dt), u = rows(d_sum, "d_sum", n.index, shape, n.dt),
             o = rows(&dx, "dx", n.index, shape, n.dt), r = rows(own ? &dres : nullptr, "dresidual", n.index, shape, n.dt),
             z = rows(n.gate ? &dgate : nullptr, "dgate", n.index, shape, n.dt);
  const void* w = n.weight_at();
  at::Tensor dweight, ws;
  if (n.weight) dweight = at::empty({n.width}, n.x.options().dtype(at::kFloat));
  gdn_rms_norm_backward_args args = {sizeof(gdn_rms_norm_backward_args), dtype_of(n.dt), n.weight_dtype(), n.order, n.act, n.heads,
                                     n.width, number(a[9]), scale, number(a[10]), shape[0], x.p, w, g.p, d.p, u.p, o.p, r.p, z.p,
                                     n.weight ? dweight.data_ptr<float>() : nullptr, x.stride, g.stride, d.stride, u.stride, o.stride,
                                     r.stride, z.stride, nullptr, 0};
  if (n.weight || a[13] != Py_None) {
    ws = workspace(a[13], n.weight ? gdn_rms_norm_backward_workspace_size(&args) : 0, n.index, n.x);
    args.workspace = ws.data_ptr();
    args.workspace_bytes = (size_t)ws.numel();
  }
  run("gdn_rms_norm_backward", gdn_rms_norm_backward, args, n.index);
  return tuple({dx, dres, dweight, dgate});
}

// (q, positions, inv_freq, k, layout, mscale, inverse, out, k_out)
PyObject* rope(PyObject* const* a) {
  const at::Tensor& q = first(a[0], "q");
  const at::ScalarType dt = q.scalar_type();
  if (!is_io(dt)) raise("q must be torch.bfloat16 or torch.float32, got " + name_of(dt));
  if (q.dim() != 3) raise("q must be a [T, H, d] tensor");
  const int32_t layout = word(a[4], "layout", "half", "interleaved");
  const int64_t index = q.get_device(), T = q.size(0), d = q.size(2);
  const at::Tensor *positions = tensor(a[1], "positions"), *inv_freq = tensor(a[2], "inv_freq"), *k = tensor(a[3], "k");
  if (!positions || (positions->scalar_type() != at::kLong && positions->scalar_type() != at::kInt))
    raise("positions must be a torch.int32 or torch.int64 tensor");
  if (!inv_freq || inv_freq->dim() != 1) raise("inv_freq must be a [rot / 2] tensor");
  if (k && (k->dim() != 3 || k->size(0) != T || k->size(2) != d)) raise("k must be [T, H, d] with q's T and d");
  if (!k && a[8] != Py_None) raise("k_out goes with k");
  if (q.size(1) > INT32_MAX || d > INT32_MAX || (k && k->size(1) > INT32_MAX) || inv_freq->size(0) > INT32_MAX / 2) raise("q or k is too wide");
  const at::Tensor y = output(a[7], "out", q), z = k ? output(a[8], "k_out", *k) : at::Tensor();
  const Rows rq = rows(&q, "q", index, q.sizes(), dt), ry = rows(&y, "out", index, q.sizes(), dt);
  Rows rk, rz;
  if (k) rk = rows(k, "k", index, k->sizes(), dt), rz = rows(&z, "k_out", index, k->sizes(), dt);
  const gdn_rope_args args = {sizeof(gdn_rope_args), dtype_of(dt), layout, truth(a[6]) ? 1 : 0, positions->scalar_type() == at::kLong ? 64 : 32,
                              (int32_t)q.size(1), k ? (int32_t)k->size(1) : 0, (int32_t)d, 2 * (int32_t)inv_freq->size(0), number(a[5]), T,
                              rq.p, rk.p, whole(positions, "positions", index, {T}, positions->scalar_type()),
                              static_cast<const double*>(whole(inv_freq, "inv_freq", index, inv_freq->sizes(), at::kDouble)), ry.p, rz.p,
                              rq.stride, rk.stride, ry.stride, rz.stride};
  run("gdn_rope", gdn_rope, args, index);
  return k ? tuple({y, z}) : wrap(y);
}

// The pool of pages and the sequences in it.
struct Cache {
  int32_t n, pages, page, width;
  void *k, *v;
  float *k_scale, *v_scale;
  const int32_t *table, *lens, *cu;
  // heads < 0: as many as the pool has
  Cache(PyObject* cache, PyObject* ptable, PyObject* plens, PyObject* pcu, int64_t index, int64_t* heads, int64_t d, int64_t tokens) {
    PyObject* const* c = nullptr;
    if (PyTuple_Check(cache) && PyTuple_GET_SIZE(cache) == 4) c = ((PyTupleObject*)cache)->ob_item;
    else if (PyList_Check(cache) && PyList_GET_SIZE(cache) == 4) c = ((PyListObject*)cache)->ob_item;
    const at::Tensor* t[4];
    const char* const names[4] = {"cache.k", "cache.v", "cache.k_scale", "cache.v_scale"};
    for (int i = 0; i < 4; ++i) t[i] = c ? tensor(c[i], names[i]) : nullptr;
    if (!t[0] || !t[1] || !t[2] || !t[3] || t[0]->dim() != 4) raise("cache must be (k [pages, h_kv, page_size, d], v, k_scale, v_scale)");
    if (*heads < 0) *heads = t[0]->size(1);
    const int64_t np = t[0]->size(0), ps = t[0]->size(2), h = *heads;
    if (t[0]->size(1) != h || t[0]->size(3) != d)
      raise("the cache holds " + std::to_string(t[0]->size(1)) + " heads of " + std::to_string(t[0]->size(3)) + ", not " + std::to_string(h) +
            " of " + std::to_string(d));
    k = whole(t[0], names[0], index, {np, h, ps, d}, at::kFloat8_e4m3fn);
    v = whole(t[1], names[1], index, {np, h, d, ps}, at::kFloat8_e4m3fn);
    k_scale = static_cast<float*>(whole(t[2], names[2], index, {np, h}, at::kFloat));
    v_scale = static_cast<float*>(whole(t[3], names[3], index, {np, h}, at::kFloat));
    const at::Tensor *pt = tensor(ptable, "page_table"), *pl = tensor(plens, "lens"), *pc = tensor(pcu, "cu_seqlens");
    if (!pt || pt->dim() != 2) raise("page_table must be [n_seqs, max_pages]");
    if (!pl) raise("lens is required");
    const int64_t ns = pt->size(0), mp = pt->size(1);
    if (np > INT32_MAX || ps > INT32_MAX || ns > INT32_MAX || mp > INT32_MAX || h > INT32_MAX) raise("the cache or its table is too large");
    table = static_cast<const int32_t*>(whole(pt, "page_table", index, pt->sizes(), at::kInt));
    lens = static_cast<const int32_t*>(whole(pl, "lens", index, {ns}, at::kInt));
    cu = static_cast<const int32_t*>(whole(pc, "cu_seqlens", index, {ns + 1}, at::kInt));
    if (!cu && ns && tokens % ns)
      raise("without cu_seqlens every sequence has the same number of new tokens: " + std::to_string(tokens) + " over " + std::to_string(ns) + " sequences");
    n = (int32_t)ns, pages = (int32_t)np, page = (int32_t)ps, width = (int32_t)mp;
  }
};

const at::Tensor& heads_of(PyObject* o, const char* name) {
  const at::Tensor& t = first(o, name);
  if (!is_io(t.scalar_type())) raise(std::string(name) + " must be torch.bfloat16 or torch.float32, got " + name_of(t.scalar_type()));
  if (t.dim() != 3) raise(std::string(name) + " must be a [T, H, d] tensor");
  if (t.size(1) > INT32_MAX || t.size(2) > INT32_MAX) raise(std::string(name) + " is too wide");
  return t;
}

// (k, v, cache, page_table, lens, cu_seqlens)
PyObject* cache_store(PyObject* const* a) {
  const at::Tensor& k = heads_of(a[0], "k");
  const at::Tensor* v = tensor(a[1], "v");
  if (!v) raise("v is required");
  const int64_t index = k.get_device();
  int64_t h = k.size(1);
  const Cache c(a[2], a[3], a[4], a[5], index, &h, k.size(2), k.size(0));
  const Rows rk = rows(&k, "k", index, k.sizes(), k.scalar_type()), rv = rows(v, "v", index, k.sizes(), k.scalar_type());
  const gdn_cache_store_args args = {sizeof(gdn_cache_store_args), dtype_of(k.scalar_type()), c.n, (int32_t)h, (int32_t)k.size(2), c.page, c.pages,
                                     c.width, k.size(0), rk.p, rv.p, rk.stride, rv.stride, c.k, c.v, c.k_scale, c.v_scale, c.table, c.lens, c.cu};
  run("gdn_cache_store", gdn_cache_store, args, index);
  Py_RETURN_NONE;
}

// (q, cache, page_table, lens, cu_seqlens, scale, causal, window, gate, out, return_lse, workspace)
PyObject* cache_attention(PyObject* const* a) {
  const at::Tensor& q = heads_of(a[0], "q");
  const at::ScalarType dt = q.scalar_type();
  const int64_t index = q.get_device(), T = q.size(0), d = q.size(2);
  int64_t h = -1;
  const Cache c(a[1], a[2], a[3], a[4], index, &h, d, T);
  const at::Tensor* gate = tensor(a[8], "gate");
  const at::Tensor o = output(a[9], "out", q);
  const Rows rq = rows(&q, "q", index, q.sizes(), dt), rg = rows(gate, "gate", index, q.sizes(), dt), ro = rows(&o, "out", index, q.sizes(), dt);
  const float scale = a[5] == Py_None ? (float)(1.0 / std::sqrt((double)d)) : number(a[5]);
  const bool want_lse = truth(a[10]);
  at::Tensor lse, ws;
  if (want_lse) lse = at::empty({T, q.size(1)}, q.options().dtype(at::kFloat));
  gdn_cache_attention_args args = {sizeof(gdn_cache_attention_args), dtype_of(dt), c.n, (int32_t)q.size(1), (int32_t)h, (int32_t)d, c.page, c.pages,
                                   c.width, truth(a[6]) ? 1 : 0, whole_number(a[7], "window"), scale, T, rq.p, rg.p, ro.p, rq.stride, rg.stride,
                                   ro.stride, want_lse ? lse.data_ptr<float>() : nullptr, c.k, c.v, c.k_scale, c.v_scale, c.table, c.lens, c.cu,
                                   nullptr, 0};
  const size_t need = gdn_cache_attention_workspace_size(&args);
  if (need || a[11] != Py_None) {
    ws = workspace(a[11], need, index, q);
    args.workspace = ws.data_ptr();
    args.workspace_bytes = (size_t)ws.numel();
  }
  run("gdn_cache_attention", gdn_cache_attention, args, index);
  return want_lse ? tuple({o, lse}) : wrap(o);
}

// No C++ exception leaves a call: torch's (out of memory, say) become its Python ones.
template <PyObject* (*F)(PyObject* const*), Py_ssize_t N>
PyObject* guarded(PyObject*, PyObject* const* args, Py_ssize_t n) {
  if (n != N) {
    PyErr_Format(PyExc_TypeError, "%zd arguments expected, got %zd", N, n);
    return nullptr;
  }
  HANDLE_TH_ERRORS
  try {
    return F(args);
  } catch (const Raised&) {
    return nullptr;
  }
  END_HANDLE_TH_ERRORS
}

// (GdnError, stream of a device, current device, set the current device)
PyObject* init(PyObject* const* a) {
  PyObject** const kept[] = {&g_error, &g_stream_of, &g_device, &g_set_device};
  for (int i = 0; i < 4; ++i) {
    Py_INCREF(a[i]);
    Py_XDECREF(*kept[i]);
    *kept[i] = a[i];
  }
  Py_RETURN_NONE;
}

#define GDN_METHOD(name, n) {#name, (PyCFunction)(void*)guarded<name, n>, METH_FASTCALL, nullptr}
PyMethodDef methods[] = {GDN_METHOD(init, 4), GDN_METHOD(rms_norm, 11), GDN_METHOD(rms_norm_backward, 14), GDN_METHOD(rope, 9),
                         GDN_METHOD(cache_store, 6), GDN_METHOD(cache_attention, 12), {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_binding", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__binding() { return PyModule_Create(&module); }
