// Argument marshalling of the calls that serve single tokens (rotary positions, cache append,
// prefix attention): torch tensors to the C ABI's views, one call from Python each.
//
// A decoding step makes these calls once per layer with a few microseconds of GPU work.  A call
// takes 5 to 11 us on the host, its launches included (rotary and append 5 to 9, attention 7 to
// 11, by the host); marshalled with ctypes it took 17 to 19.
// Like the ctypes binding this adds no step of its own: it checks what the C side cannot see
// (shapes, devices, dtypes of index tensors), allocates outputs that were not given and passes
// pointers and strides on.  Every function returns (status, outputs...).
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/Dtype.h>
#include <torch/csrc/autograd/python_variable.h>
#include <ATen/ATen.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>

#include "nabla.h"

namespace {

struct BadArgument {
  PyObject* type;
  std::string what;
};

[[noreturn]] void refuse(const std::string& what) { throw BadArgument{PyExc_ValueError, what}; }

std::string shape_text(const at::Tensor& t) {
  std::string s = "(";
  for (int64_t i = 0; i < t.dim(); ++i) s += (i ? ", " : "") + std::to_string(t.size(i));
  return s + ")";
}

// A tensor argument; nullptr for None.
const at::Tensor* tensor(PyObject* o, const char* what) {
  if (o == Py_None) return nullptr;
  if (!THPVariable_Check(o)) throw BadArgument{PyExc_TypeError, std::string(what) + ": expected a tensor"};
  return &THPVariable_Unpack(o);
}

int64_t whole(PyObject* o) {
  const long long v = PyLong_AsLongLong(o);
  if (v == -1 && PyErr_Occurred()) throw python_error();
  return v;
}
int32_t whole32(PyObject* o) {
  const int64_t v = whole(o);
  if (v < INT32_MIN || v > INT32_MAX) refuse("an integer argument does not fit 32 bits");
  return static_cast<int32_t>(v);
}
double real(PyObject* o) {
  const double v = PyFloat_AsDouble(o);
  if (v == -1.0 && PyErr_Occurred()) throw python_error();
  return v;
}

int32_t dtype_of(const at::Tensor& t, const char* what) {
  switch (t.scalar_type()) {
    case at::kBFloat16: return NABLA_BF16;
    case at::kFloat: return NABLA_F32;
    case at::kHalf: return NABLA_F16;
    default: throw BadArgument{PyExc_TypeError, std::string(what) + ": unsupported dtype " + c10::toString(t.scalar_type())};
  }
}

// All tensors of a call on one CUDA device.
struct Device {
  c10::Device device;
  explicit Device(const at::Tensor& t) : device(t.device()) {
    if (!t.is_cuda()) refuse("expected CUDA tensors, got " + device.str());
  }
  void has(const at::Tensor* t, const char* what) const {
    if (t && t->device() != device) refuse(std::string(what) + " is on " + t->device().str() + ", the call on " + device.str());
  }
};

nabla_heads heads(const at::Tensor& t, int64_t B, int64_t S, int64_t D, const char* what) {
  if (t.dim() != 4 || t.size(0) != B || t.size(2) != S || t.size(3) != D)
    refuse(std::string(what) + ": expected [" + std::to_string(B) + ", H, " + std::to_string(S) + ", " + std::to_string(D) +
           "], got " + shape_text(t));
  if (t.stride(3) != 1) refuse(std::string(what) + ": the last dimension must be contiguous");
  if (t.size(1) > INT32_MAX) refuse(std::string(what) + ": too many heads");
  return nabla_heads{t.data_ptr(), dtype_of(t, what), static_cast<int32_t>(t.size(1)), t.stride(0), t.stride(1), t.stride(2)};
}

const int32_t* table(const at::Tensor* t, at::IntArrayRef shape, const char* what) {
  if (!t) return nullptr;
  if (t->scalar_type() != at::kInt || t->sizes() != shape || !t->is_contiguous())
    refuse(std::string(what) + ": expected a contiguous int32 tensor of another shape or dtype, got " +
           c10::toString(t->scalar_type()) + " " + shape_text(*t));
  return static_cast<const int32_t*>(t->data_ptr());
}

// positions [B, S, axes], or [B, S] with one axis
const int32_t* positions_of(const at::Tensor* t, int64_t B, int64_t S, int32_t axes) {
  if (t && t->dim() == 2 && axes == 1) return table(t, {B, S}, "positions");
  return table(t, {B, S, axes}, "positions");
}

// (inv_freq, style, axes, dim_t, dim_h, dim_w, magnitude)
nabla_rope rope_of(PyObject* o, const Device& dev) {
  if (!PyTuple_Check(o) || PyTuple_GET_SIZE(o) != 7) throw BadArgument{PyExc_TypeError, "rope: expected a Rope"};
  const at::Tensor* f = tensor(PyTuple_GET_ITEM(o, 0), "inv_freq");
  if (!f || f->scalar_type() != at::kDouble || f->dim() != 1 || !f->is_contiguous() || f->numel() > 4096)
    refuse("inv_freq: expected a contiguous fp64 vector");
  dev.has(f, "inv_freq");
  nabla_rope r;
  r.style = whole32(PyTuple_GET_ITEM(o, 1));
  r.dim = static_cast<int32_t>(2 * f->numel());
  r.axes = whole32(PyTuple_GET_ITEM(o, 2));
  for (int i = 0; i < 3; ++i) r.axis_dim[i] = whole32(PyTuple_GET_ITEM(o, 3 + i));
  r.magnitude = static_cast<float>(real(PyTuple_GET_ITEM(o, 6)));
  r.inv_freq = static_cast<const double*>(f->data_ptr());
  return r;
}

nabla_grid grid_of(PyObject* o, const char* what) {
  PyObject* t = PySequence_Fast(o, what);
  if (!t) throw python_error();
  nabla_grid g = {0, 0, 0};
  const Py_ssize_t n = PySequence_Fast_GET_SIZE(t);
  try {
    if (n != 3 && n != 2) refuse(std::string(what) + ": expected two or three integers");
    int32_t v[3] = {0, 0, 0};
    for (Py_ssize_t i = 0; i < n; ++i) v[3 - n + i] = whole32(PySequence_Fast_GET_ITEM(t, i));
    g = {v[0], v[1], v[2]};
  } catch (...) {
    Py_DECREF(t);
    throw;
  }
  Py_DECREF(t);
  return g;
}

nabla_cache cache_of(const at::Tensor& k, const at::Tensor& v) {
  if (k.dim() != 4 || k.sizes() != v.sizes() || k.scalar_type() != v.scalar_type())
    refuse("k_cache and v_cache: expected two [pages, H, page, D] pools of one shape and dtype");
  if (!k.is_contiguous() || !v.is_contiguous()) refuse("k_cache and v_cache must be contiguous");
  for (int i = 0; i < 4; ++i)
    if (k.size(i) > INT32_MAX) refuse("k_cache: a dimension does not fit 32 bits");
  return nabla_cache{k.data_ptr(), v.data_ptr(), static_cast<int32_t>(k.size(0)), static_cast<int32_t>(k.size(1)),
                     static_cast<int32_t>(k.size(2)), static_cast<int32_t>(k.size(3)), dtype_of(k, "k_cache")};
}

int32_t dim32(const at::Tensor& t, int i, const char* what) {
  if (t.size(i) > INT32_MAX) refuse(std::string(what) + ": a dimension does not fit 32 bits");
  return static_cast<int32_t>(t.size(i));
}

at::Tensor contiguous_like(const at::Tensor& t, at::ScalarType dtype) {
  return at::empty(t.sizes(), t.options().dtype(dtype));
}
at::ScalarType dtype_arg(PyObject* o, const at::Tensor& t) {
  if (o == Py_None) return t.scalar_type();
  if (!THPDtype_Check(o)) throw BadArgument{PyExc_TypeError, "expected a torch.dtype"};
  return reinterpret_cast<THPDtype*>(o)->scalar_type;
}

nabla_stream_t stream_of(const Device& dev) {
  return reinterpret_cast<nabla_stream_t>(c10::cuda::getCurrentCUDAStream(dev.device.index()).stream());
}

PyObject* object_or_none(const at::Tensor& t) {
  if (!t.defined()) Py_RETURN_NONE;
  return THPVariable_Wrap(t);
}

template <typename F>
PyObject* guarded(Py_ssize_t got, Py_ssize_t want, F body) {
  try {
    if (got != want) throw BadArgument{PyExc_TypeError, "wrong number of arguments"};
    return body();
  } catch (const BadArgument& e) {
    PyErr_SetString(e.type, e.what.c_str());
  } catch (python_error& e) {
    e.restore();
  } catch (const std::exception& e) {
    PyErr_SetString(PyExc_RuntimeError, e.what());
  }
  return nullptr;
}

// rotary(q, k, q_out, k_out, rope, grid | None, origin, positions, out_dtype | None, src_layout,
//        dst_layout, adjoint) -> (status, q_out, k_out)
PyObject* rotary(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 12, [&]() -> PyObject* {
    const at::Tensor* in[2] = {tensor(a[0], "q"), tensor(a[1], "k")};
    const at::Tensor* given[2] = {tensor(a[2], "q_out"), tensor(a[3], "k_out")};
    const char* names[2] = {"q", "k"};
    const char* out_names[2] = {"q_out", "k_out"};
    const at::Tensor* x = in[0] ? in[0] : in[1];
    if (!x) refuse("nothing to rotate: q and k are None");
    const Device dev(*x);
    if (x->dim() != 4) refuse("expected [B, H, S, D], got " + shape_text(*x));
    const int64_t B = x->size(0), S = x->size(2), D = x->size(3);
    const nabla_rope rope = rope_of(a[4], dev);
    nabla_grid grid = {0, 1, 1};
    if (a[5] == Py_None) {
      grid.T = dim32(*x, 2, "q");
    } else {
      grid = grid_of(a[5], "grid");
      if (static_cast<int64_t>(grid.T) * grid.Hg * grid.W != S) refuse("grid does not hold " + std::to_string(S) + " tokens");
    }
    const nabla_grid origin = grid_of(a[6], "origin");
    const at::Tensor* pos = tensor(a[7], "positions");
    dev.has(pos, "positions");
    const c10::cuda::CUDAGuard guard(dev.device);
    nabla_heads views[4] = {};
    at::Tensor outs[2];
    for (int i = 0; i < 2; ++i) {
      dev.has(in[i], names[i]);
      dev.has(given[i], out_names[i]);
      if (!in[i]) {
        if (given[i]) refuse(std::string(out_names[i]) + " without " + names[i]);
        continue;
      }
      views[2 * i] = heads(*in[i], B, S, D, names[i]);
      outs[i] = given[i] ? *given[i] : contiguous_like(*in[i], dtype_arg(a[8], *in[i]));
      views[2 * i + 1] = heads(outs[i], B, S, D, out_names[i]);
    }
    const nabla_status rc = nabla_rotary(views[0], views[1], views[2], views[3], dim32(*x, 0, "q"), grid, dim32(*x, 3, "q"),
                                         rope, origin, positions_of(pos, B, S, rope.axes),
                                         static_cast<nabla_layout>(whole32(a[9])), static_cast<nabla_layout>(whole32(a[10])),
                                         whole32(a[11]), stream_of(dev));
    return Py_BuildValue("iNN", static_cast<int>(rc), object_or_none(outs[0]), object_or_none(outs[1]));
  });
}

// append(k, v, k_cache, v_cache, page_table, start, rope | None, frame, pos0, positions, counts,
//        q, q_out, status) -> (status, q_out)
PyObject* append(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 14, [&]() -> PyObject* {
    const at::Tensor* k = tensor(a[0], "k");
    const at::Tensor* v = tensor(a[1], "v");
    const at::Tensor* kc = tensor(a[2], "k_cache");
    const at::Tensor* vc = tensor(a[3], "v_cache");
    const at::Tensor* pages = tensor(a[4], "page_table");
    const at::Tensor* start = tensor(a[5], "start");
    const at::Tensor* pos = tensor(a[9], "positions");
    const at::Tensor* counts = tensor(a[10], "counts");
    const at::Tensor* q = tensor(a[11], "q");
    const at::Tensor* q_out = tensor(a[12], "q_out");
    const at::Tensor* word = tensor(a[13], "status");
    if (!k || !v || !kc || !vc || !pages || !start) refuse("k, v, k_cache, v_cache, page_table and start are required");
    const Device dev(*k);
    dev.has(v, "v"); dev.has(kc, "k_cache"); dev.has(vc, "v_cache"); dev.has(pages, "page_table");
    dev.has(start, "start"); dev.has(pos, "positions"); dev.has(counts, "counts"); dev.has(q, "q");
    dev.has(q_out, "q_out"); dev.has(word, "status");
    if (k->dim() != 4) refuse("k: expected [B, H, S, D], got " + shape_text(*k));
    const int64_t B = k->size(0), S = k->size(2), D = k->size(3);
    const nabla_cache cache = cache_of(*kc, *vc);
    if (cache.D != D) refuse("k has rows of " + std::to_string(D) + ", the cache of " + std::to_string(cache.D));
    nabla_rope rope;
    const bool turn = a[6] != Py_None;
    if (turn) rope = rope_of(a[6], dev);
    if (pos && !turn) refuse("positions without rope");
    if (pages->dim() != 2) refuse("page_table: expected [B, pages]");
    if (word && word->numel() * static_cast<int64_t>(word->element_size()) < 4) refuse("status: expected at least 4 bytes");
    if (q_out && !q) refuse("q_out without q");
    const c10::cuda::CUDAGuard guard(dev.device);
    nabla_heads qs = {}, qd = {};
    at::Tensor out;
    if (q) {
      qs = heads(*q, B, S, D, "q");
      out = q_out ? *q_out : contiguous_like(*q, q->scalar_type());
      qd = heads(out, B, S, D, "q_out");
    }
    const nabla_status rc = nabla_cache_append(
        heads(*k, B, S, D, "k"), heads(*v, B, S, D, "v"), qs, qd, dim32(*k, 0, "k"), dim32(*k, 2, "k"), cache,
        table(pages, {B, pages->size(1)}, "page_table"), dim32(*pages, 1, "page_table"), table(start, {B}, "start"),
        table(counts, {B}, "counts"), turn ? &rope : nullptr, grid_of(a[7], "frame"), whole(a[8]),
        turn ? positions_of(pos, B, S, rope.axes) : nullptr, word ? static_cast<uint32_t*>(word->data_ptr()) : nullptr,
        stream_of(dev));
    return Py_BuildValue("iN", static_cast<int>(rc), object_or_none(out));
  });
}

const float* f32_rows(const at::Tensor* t, int64_t B, int64_t H, int64_t S, const char* what) {
  if (!t) return nullptr;
  if (t->scalar_type() != at::kFloat || t->sizes() != at::IntArrayRef({B, H, S}) || !t->is_contiguous())
    refuse(std::string(what) + ": expected a contiguous f32 [" + std::to_string(B) + ", " + std::to_string(H) + ", " +
           std::to_string(S) + "] tensor, got " + c10::toString(t->scalar_type()) + " " + shape_text(*t));
  return static_cast<const float*>(t->data_ptr());
}

// prefix_attn(q, k_cache, v_cache, prefix_pages, prefix_len, tail_pages, tail_len, q_len, causal,
//             scale | None, part_o, part_lse, o, o_dtype | None, lse, workspace) -> (status, o)
PyObject* prefix_attn(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 16, [&]() -> PyObject* {
    const at::Tensor* q = tensor(a[0], "q");
    const at::Tensor* kc = tensor(a[1], "k_cache");
    const at::Tensor* vc = tensor(a[2], "v_cache");
    const at::Tensor* prefix = tensor(a[3], "prefix_pages");
    const at::Tensor* tail = tensor(a[5], "tail_pages");
    const at::Tensor* tail_len = tensor(a[6], "tail_len");
    const at::Tensor* q_len = tensor(a[7], "q_len");
    const at::Tensor* part_o = tensor(a[10], "part_o");
    const at::Tensor* part_lse = tensor(a[11], "part_lse");
    const at::Tensor* o = tensor(a[12], "o");
    const at::Tensor* lse = tensor(a[14], "lse");
    const at::Tensor* ws = tensor(a[15], "workspace");
    if (!q || !kc || !vc) refuse("q, k_cache and v_cache are required");
    const Device dev(*q);
    dev.has(kc, "k_cache"); dev.has(vc, "v_cache"); dev.has(prefix, "prefix_pages"); dev.has(tail, "tail_pages");
    dev.has(tail_len, "tail_len"); dev.has(q_len, "q_len"); dev.has(part_o, "part_o"); dev.has(part_lse, "part_lse");
    dev.has(o, "o"); dev.has(lse, "lse"); dev.has(ws, "workspace");
    if (q->dim() != 4) refuse("q: expected [B, H, S, D], got " + shape_text(*q));
    const int64_t B = q->size(0), Hq = q->size(1), Sq = q->size(2), D = q->size(3);
    const nabla_cache cache = cache_of(*kc, *vc);
    if (cache.D != D) refuse("q has rows of " + std::to_string(D) + ", the cache of " + std::to_string(cache.D));
    const int32_t prefix_len = whole32(a[4]);
    if (prefix && prefix->dim() == 1 && prefix->size(0) * cache.page < prefix_len)
      refuse(std::to_string(prefix->size(0)) + " pages of " + std::to_string(cache.page) + " do not hold a prefix of " +
             std::to_string(prefix_len));
    if (tail && tail->dim() != 2) refuse("tail_pages: expected [B, pages]");
    const c10::cuda::CUDAGuard guard(dev.device);
    const nabla_heads qv = heads(*q, B, Sq, D, "q");
    const at::Tensor out = o ? *o : contiguous_like(*q, dtype_arg(a[13], *q));
    const int32_t b32 = dim32(*q, 0, "q"), s32 = dim32(*q, 2, "q");
    at::Tensor scratch;
    if (ws) {
      if (ws->scalar_type() != at::kByte || !ws->is_contiguous()) refuse("workspace: expected a contiguous uint8 tensor");
      scratch = *ws;
    } else {
      scratch = at::empty({static_cast<int64_t>(nabla_prefix_workspace_bytes(b32, qv.H, cache.H, s32, cache.D))},
                          q->options().dtype(at::kByte));
    }
    const float scale = a[9] == Py_None ? static_cast<float>(1.0 / std::sqrt(static_cast<double>(D))) : static_cast<float>(real(a[9]));
    const int causal = PyObject_IsTrue(a[8]);
    if (causal < 0) throw python_error();
    const nabla_status rc = nabla_prefix_attn(
        qv, b32, s32, cache, prefix ? table(prefix, {prefix->size(0)}, "prefix_pages") : nullptr, prefix_len,
        tail ? table(tail, {B, tail->size(1)}, "tail_pages") : nullptr, tail ? dim32(*tail, 1, "tail_pages") : 0,
        table(tail_len, {B}, "tail_len"), table(q_len, {B}, "q_len"), causal, scale,
        part_o ? heads(*part_o, B, Sq, D, "part_o") : nabla_heads{}, f32_rows(part_lse, B, Hq, Sq, "part_lse"),
        heads(out, B, Sq, D, "o"), const_cast<float*>(f32_rows(lse, B, Hq, Sq, "lse")), scratch.data_ptr(),
        static_cast<size_t>(scratch.numel()), stream_of(dev));
    return Py_BuildValue("iN", static_cast<int>(rc), object_or_none(out));
  });
}

PyMethodDef methods[] = {
    {"rotary", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(rotary)), METH_FASTCALL, nullptr},
    {"append", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(append)), METH_FASTCALL, nullptr},
    {"prefix_attn", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(prefix_attn)), METH_FASTCALL, nullptr},
    {nullptr, nullptr, 0, nullptr}};

PyModuleDef module = {PyModuleDef_HEAD_INIT, "_binding", "Argument marshalling for libnabla.so.", -1, methods,
                      nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__binding() { return PyModule_Create(&module); }
