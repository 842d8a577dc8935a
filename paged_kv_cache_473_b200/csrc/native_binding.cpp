// Python entry of the drafting step's calls: looks at the tensors (types,
// devices, shapes, strides), then calls the C ABI (include/pagedattn.h) on the
// device's current stream.  These calls run once a layer and step, and on a few
// tokens their kernels take 3 us: marshalling their 20 to 25 arguments through ctypes
// took 13 to 17 us a call, this takes about 2 besides the launch.
//
// Plain CPython functions with positional arguments (the keywords, defaults and
// documentation are in _binding.py); no exception leaves a function.
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <ATen/ATen.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include <stdexcept>
#include <string>

#include "../../include/pagedattn.h"

namespace {

PyObject* g_error_class = nullptr;  // PagedAttnError

struct PyRaised {};  // a Python exception is set

[[noreturn]] void refuse(const std::string& why) { throw std::invalid_argument(why); }

// Argument i as a tensor; None gives an undefined one where that is allowed.
const at::Tensor& tensor(PyObject* o, const char* name, bool optional = false) {
  static const at::Tensor none;
  if (o == Py_None && optional) return none;
  if (!THPVariable_Check(o)) {
    PyErr_Format(PyExc_TypeError, "%s must be a tensor", name);
    throw PyRaised();
  }
  return THPVariable_Unpack(o);
}

int64_t integer(PyObject* o) {
  const long long v = PyLong_AsLongLong(o);
  if (v == -1 && PyErr_Occurred()) throw PyRaised();
  return v;
}

int32_t integer32(PyObject* o, const char* name) {
  const int64_t v = integer(o);
  if (v < INT32_MIN || v > INT32_MAX) refuse(std::string(name) + " does not fit 32 bits");
  return (int32_t)v;
}

float number(PyObject* o) {
  const double v = PyFloat_AsDouble(o);
  if (v == -1.0 && PyErr_Occurred()) throw PyRaised();
  return (float)v;
}

bool truth(PyObject* o) {
  const int v = PyObject_IsTrue(o);
  if (v < 0) throw PyRaised();
  return v != 0;
}

pa_dtype_t dtype_code(const at::Tensor& t) {
  if (t.scalar_type() == at::kFloat) return PA_F32;
  if (t.scalar_type() == at::kBFloat16) return PA_BF16;
  PyErr_SetString(PyExc_TypeError, "paged attention takes float32 or bfloat16 tensors");
  throw PyRaised();
}

// A call in progress: its name, its device, and what every tensor of it has to be.
struct Call {
  const char* name;
  c10::Device device;

  Call(const char* n, const at::Tensor& first) : name(n), device(first.device()) {
    if (!device.is_cuda()) refuse(std::string(n) + ": tensors must be on a CUDA device");
  }
  [[noreturn]] void no(const char* why) const { refuse(std::string(name) + ": " + why); }
  void is(const at::Tensor& t, at::ScalarType type, const char* what) const {
    if (!t.defined()) return;
    if (t.scalar_type() != type)
      no((std::string(what) + " must be " + c10::toString(type) + ", not " + c10::toString(t.scalar_type())).c_str());
    if (t.device() != device) no((std::string(what) + " is on another device").c_str());
  }
  // A contiguous tensor's address (null when undefined).
  void* ptr(const at::Tensor& t, const char* what) const {
    if (!t.defined()) return nullptr;
    if (!t.is_contiguous()) no((std::string(what) + " must be contiguous").c_str());
    return t.data_ptr();
  }
  // Elements between the token rows of a [tokens, heads, d] tensor whose rows are contiguous.
  int64_t rows(const at::Tensor& t, int64_t tokens, int64_t heads, int64_t d, const char* what) const {
    if (t.dim() != 3 || t.size(0) != tokens || t.size(1) != heads || t.size(2) != d)
      no((std::string(what) + " has another shape").c_str());
    if (t.stride(2) != 1 || (t.stride(1) != d && heads > 1)) no((std::string(what) + ": a token's heads must be contiguous").c_str());
    return tokens > 1 ? t.stride(0) : heads * d;
  }
  // The stream to launch on: the caller's (an object with cuda_stream, or its handle), or the device's current one.
  pa_stream_t stream(PyObject* o) const {
    if (o == Py_None) return reinterpret_cast<pa_stream_t>(c10::cuda::getCurrentCUDAStream(device.index()).stream());
    PyObject* h = PyObject_HasAttrString(o, "cuda_stream") ? PyObject_GetAttrString(o, "cuda_stream") : Py_NewRef(o);
    if (!h) throw PyRaised();
    void* p = PyLong_AsVoidPtr(h);
    Py_DECREF(h);
    if (!p && PyErr_Occurred()) throw PyRaised();
    return static_cast<pa_stream_t>(p);
  }
  // A new tensor that the call uses on `on`: from that stream's memory, which work queued on
  // another stream no longer uses.  One that the caller gets is not given to others while
  // the current stream, where it may be used next, still does.
  at::Tensor make(c10::IntArrayRef shape, const at::TensorOptions& options, pa_stream_t on, bool returned = true) const {
    const c10::cuda::CUDAStream current = c10::cuda::getCurrentCUDAStream(device.index());
    if (current.stream() == reinterpret_cast<cudaStream_t>(on)) return at::empty(shape, options);
    const c10::cuda::CUDAStreamGuard guard(
        c10::cuda::getStreamFromExternal(reinterpret_cast<cudaStream_t>(on), device.index()));
    const at::Tensor t = at::empty(shape, options);
    if (returned) t.record_stream(current);
    return t;
  }
  void check(pa_status_t st, const char* function) const {
    if (st == PA_OK) return;
    PyObject* e = PyObject_CallFunction(g_error_class, "is", (int)st, function);
    if (e) {
      PyErr_SetObject(g_error_class, e);
      Py_DECREF(e);
    }
    throw PyRaised();
  }
};

int32_t small(int64_t v, const Call& c) {
  if (v > INT32_MAX) c.no("a size does not fit 32 bits");
  return (int32_t)v;
}

template <typename F>
PyObject* guarded(Py_ssize_t given, Py_ssize_t wanted, F f) {
  if (given != wanted) {
    PyErr_Format(PyExc_TypeError, "%zd arguments, %zd are taken", given, wanted);
    return nullptr;
  }
  try {
    return f();
  } catch (const PyRaised&) {
  } catch (const std::invalid_argument& e) {
    PyErr_SetString(PyExc_ValueError, e.what());
  } catch (const std::exception& e) {
    PyErr_SetString(PyExc_RuntimeError, e.what());
  } catch (...) {
    PyErr_SetString(PyExc_RuntimeError, "unknown error");
  }
  return nullptr;
}

// What both rotation calls take.
struct Rotation {
  const at::Tensor &q, &k, &positions, &inv_freq, &q_weight, &k_weight;
  int64_t n, hq, hkv, d;
  int32_t rotary;

  Rotation(const Call& c, const at::Tensor& q_, const at::Tensor& k_, const at::Tensor& pos, const at::Tensor& inv,
           PyObject* rotary_dim, const at::Tensor& qw, const at::Tensor& kw)
      : q(q_), k(k_), positions(pos), inv_freq(inv), q_weight(qw), k_weight(kw) {
    if (q.dim() != 3 || k.dim() != 3) c.no("q and k are [tokens, heads, head_dim]");
    n = q.size(0);
    hq = q.size(1);
    d = q.size(2);
    hkv = k.size(1);
    c.is(k, q.scalar_type(), "k");
    c.is(inv, at::kFloat, "inv_freq");
    c.is(qw, at::kFloat, "q_weight");
    c.is(kw, at::kFloat, "k_weight");
    c.is(pos, at::kInt, "positions");
    rotary = inv.defined() ? small(2 * inv.numel(), c) : 0;
    if (rotary_dim != Py_None && integer(rotary_dim) != rotary) c.no("inv_freq has rotary_dim / 2 frequencies");
    if (rotary && (!pos.defined() || pos.numel() != n)) c.no("one position per token is needed");
    if ((qw.defined() && qw.numel() != d) || (kw.defined() && kw.numel() != d)) c.no("a norm weight has head_dim elements");
  }
};

// q, k, positions, inv_freq, rotary_dim, q_weight, k_weight, eps, interleaved, q_out, k_out, stream -> (q_out, k_out)
PyObject* qk_norm_rope(PyObject*, PyObject* const* a, Py_ssize_t n_args) {
  return guarded(n_args, 12, [&]() -> PyObject* {
    const at::Tensor &q = tensor(a[0], "q"), &k = tensor(a[1], "k");
    const Call c("qk_norm_rope", q);
    const Rotation r(c, q, k, tensor(a[2], "positions", true), tensor(a[3], "inv_freq", true), a[4],
                     tensor(a[5], "q_weight", true), tensor(a[6], "k_weight", true));
    const pa_dtype_t dt = dtype_code(q);
    const c10::cuda::CUDAGuard guard(c.device);
    at::Tensor q_out = tensor(a[9], "q_out", true), k_out = tensor(a[10], "k_out", true);
    const pa_stream_t stream = c.stream(a[11]);
    if (!q_out.defined()) q_out = c.make({r.n, r.hq, r.d}, q.options(), stream);
    if (!k_out.defined()) k_out = c.make({r.n, r.hkv, r.d}, q.options(), stream);
    c.is(q_out, q.scalar_type(), "q_out");
    c.is(k_out, q.scalar_type(), "k_out");
    c.check(pa_qk_norm_rope(q.data_ptr(), c.rows(q, r.n, r.hq, r.d, "q"), k.data_ptr(), c.rows(k, r.n, r.hkv, r.d, "k"),
                            static_cast<const float*>(c.ptr(r.q_weight, "q_weight")),
                            static_cast<const float*>(c.ptr(r.k_weight, "k_weight")), number(a[7]),
                            static_cast<const float*>(c.ptr(r.inv_freq, "inv_freq")), r.rotary, truth(a[8]),
                            static_cast<const int32_t*>(c.ptr(r.positions, "positions")), small(r.n, c), small(r.hq, c),
                            small(r.hkv, c), small(r.d, c), q_out.data_ptr(), c.rows(q_out, r.n, r.hq, r.d, "q_out"),
                            k_out.data_ptr(), c.rows(k_out, r.n, r.hkv, r.d, "k_out"), dt, stream),
            "pa_qk_norm_rope");
    PyObject* out = PyTuple_New(2);
    if (!out) throw PyRaised();
    PyTuple_SET_ITEM(out, 0, a[9] != Py_None ? Py_NewRef(a[9]) : THPVariable_Wrap(q_out));
    PyTuple_SET_ITEM(out, 1, a[10] != Py_None ? Py_NewRef(a[10]) : THPVariable_Wrap(k_out));
    return out;
  });
}

// q, k, v, positions, slot_mapping, inv_freq, k_cache, v_cache, rotary_dim, q_weight, k_weight, eps, interleaved,
// q_out, stream -> q_out
PyObject* rope_append(PyObject*, PyObject* const* a, Py_ssize_t n_args) {
  return guarded(n_args, 15, [&]() -> PyObject* {
    const at::Tensor &q = tensor(a[0], "q"), &k = tensor(a[1], "k"), &v = tensor(a[2], "v");
    const at::Tensor &slots = tensor(a[4], "slot_mapping"), &kc = tensor(a[6], "k_cache"), &vc = tensor(a[7], "v_cache");
    const Call c("rope_append", q);
    const Rotation r(c, q, k, tensor(a[3], "positions", true), tensor(a[5], "inv_freq", true), a[8],
                     tensor(a[9], "q_weight", true), tensor(a[10], "k_weight", true));
    const pa_dtype_t dt = dtype_code(q);
    if (kc.dim() != 4 || kc.size(1) != r.hkv || kc.size(3) != r.d || vc.sizes() != kc.sizes())
      c.no("k, v and the caches must agree in kv heads and head_dim");
    if (slots.numel() != r.n) c.no("one slot per token is needed");
    const c10::cuda::CUDAGuard guard(c.device);
    at::Tensor q_out = tensor(a[13], "q_out", true);
    const pa_stream_t stream = c.stream(a[14]);
    if (!q_out.defined()) q_out = c.make({r.n, r.hq, r.d}, q.options(), stream);
    else if (q_out.sizes() != q.sizes()) c.no("q_out has q's shape");
    c.is(v, q.scalar_type(), "v");
    c.is(kc, q.scalar_type(), "k_cache");
    c.is(vc, q.scalar_type(), "v_cache");
    c.is(q_out, q.scalar_type(), "q_out");
    c.is(slots, at::kLong, "slot_mapping");
    c.check(pa_rope_append(q.data_ptr(), c.rows(q, r.n, r.hq, r.d, "q"), k.data_ptr(), c.rows(k, r.n, r.hkv, r.d, "k"),
                           v.data_ptr(), c.rows(v, r.n, r.hkv, r.d, "v"),
                           static_cast<const float*>(c.ptr(r.q_weight, "q_weight")),
                           static_cast<const float*>(c.ptr(r.k_weight, "k_weight")), number(a[11]),
                           static_cast<const float*>(c.ptr(r.inv_freq, "inv_freq")), r.rotary, truth(a[12]),
                           static_cast<const int32_t*>(c.ptr(r.positions, "positions")),
                           static_cast<const int64_t*>(c.ptr(slots, "slot_mapping")), small(r.n, c), small(r.hq, c),
                           small(r.hkv, c), small(r.d, c), c.ptr(q_out, "q_out"), c.ptr(kc, "k_cache"),
                           c.ptr(vc, "v_cache"), small(kc.size(0), c), small(kc.size(2), c), dt, stream),
            "pa_rope_append");
    return a[13] != Py_None ? Py_NewRef(a[13]) : THPVariable_Wrap(q_out);
  });
}

// q, k_cache, v_cache, block_tables, context_lens, tree_mask, scale, softcap, window, max_context_len, tree_lens, out,
// workspace, stream -> out
PyObject* decode_tree(PyObject*, PyObject* const* a, Py_ssize_t n_args) {
  return guarded(n_args, 14, [&]() -> PyObject* {
    const at::Tensor &q = tensor(a[0], "q"), &kc = tensor(a[1], "k_cache"), &vc = tensor(a[2], "v_cache");
    const at::Tensor &tables = tensor(a[3], "block_tables"), &lens = tensor(a[4], "context_lens");
    const at::Tensor &mask = tensor(a[5], "tree_mask"), &tree_lens = tensor(a[10], "tree_lens", true);
    const Call c("decode_tree", q);
    const pa_dtype_t dt = dtype_code(q);
    if (q.dim() != 4) c.no("q is [batch, nodes, heads, head_dim]");
    const int64_t B = q.size(0), T = q.size(1), hq = q.size(2), d = q.size(3);
    if (kc.dim() != 4 || kc.size(3) != d || vc.sizes() != kc.sizes()) c.no("q and the caches must agree in head_dim");
    if (tables.dim() != 2 || tables.size(0) != B || lens.numel() != B)
      c.no("one table row and one length per sequence are needed");
    const bool own = mask.dim() == 2 && mask.size(0) == B && mask.size(1) == T;  // a tree for each sequence
    if (!own && !(mask.dim() == 1 && mask.size(0) == T)) c.no("tree_mask is [batch, nodes] or [nodes]");
    if (tree_lens.defined() && tree_lens.numel() != B) c.no("one tree length per sequence is needed");
    const c10::cuda::CUDAGuard guard(c.device);
    at::Tensor out = tensor(a[11], "out", true), ws = tensor(a[12], "workspace", true);
    const pa_stream_t stream = c.stream(a[13]);
    if (!out.defined()) out = c.make(q.sizes(), q.options(), stream);
    else if (out.sizes() != q.sizes()) c.no("out has q's shape");
    c.is(kc, q.scalar_type(), "k_cache");
    c.is(vc, q.scalar_type(), "v_cache");
    c.is(out, q.scalar_type(), "out");
    c.is(tables, at::kInt, "block_tables");
    c.is(lens, at::kInt, "context_lens");
    c.is(tree_lens, at::kInt, "tree_lens");
    c.is(mask, at::kLong, "tree_mask");
    const int32_t most = integer32(a[9], "max_context_len");
    if (!ws.defined() && dt == PA_BF16) {
      const size_t need = pa_decode_tree_workspace_size(small(B, c), small(T, c), small(hq, c), small(d, c), most,
                                                        small(kc.size(1), c));
      if (need > 0) ws = c.make({(int64_t)need}, q.options().dtype(at::kByte), stream, false);  // 0: sizes that the call refuses
    } else if (ws.defined() && ws.device() != c.device) {
      c.no("the workspace is on another device");
    }
    c.check(pa_decode_tree(c.ptr(q, "q"), c.ptr(kc, "k_cache"), c.ptr(vc, "v_cache"),
                           static_cast<const int32_t*>(c.ptr(tables, "block_tables")),
                           static_cast<const int32_t*>(c.ptr(lens, "context_lens")),
                           static_cast<const int32_t*>(c.ptr(tree_lens, "tree_lens")),
                           static_cast<const int64_t*>(c.ptr(mask, "tree_mask")), own ? T : 0, small(B, c), small(T, c),
                           small(hq, c), small(kc.size(1), c), small(d, c), small(kc.size(2), c),
                           small(tables.size(1), c), small(kc.size(0), c), number(a[6]), number(a[7]),
                           integer32(a[8], "window"), c.ptr(out, "out"), dt, most, c.ptr(ws, "workspace"),
                           ws.defined() ? (size_t)ws.nbytes() : 0, stream),
            "pa_decode_tree");
    return a[11] != Py_None ? Py_NewRef(a[11]) : THPVariable_Wrap(out);
  });
}

// k_cache, v_cache, block_tables, context_lens, accepted, accept_lens, tree_len, tree_lens, new_lens, stream -> new_lens
PyObject* commit_tree(PyObject*, PyObject* const* a, Py_ssize_t n_args) {
  return guarded(n_args, 10, [&]() -> PyObject* {
    const at::Tensor &kc = tensor(a[0], "k_cache"), &vc = tensor(a[1], "v_cache"), &tables = tensor(a[2], "block_tables");
    const at::Tensor &lens = tensor(a[3], "context_lens"), &path = tensor(a[4], "accepted");
    const at::Tensor &take = tensor(a[5], "accept_lens"), &tree_lens = tensor(a[7], "tree_lens", true);
    const Call c("commit_tree", kc);
    const pa_dtype_t dt = dtype_code(kc);
    if ((kc.dim() != 4 && kc.dim() != 5) || vc.sizes() != kc.sizes())
      c.no("caches are [blocks, kv heads, block_size, head_dim], or have layers before that");
    const int64_t B = lens.numel(), o = kc.dim() - 4;
    if (tables.dim() != 2 || tables.size(0) != B || path.dim() != 2 || path.size(0) != B)
      c.no("one table row and one path per sequence are needed");
    if (take.numel() != B || (tree_lens.defined() && tree_lens.numel() != B)) c.no("one length per sequence is needed");
    const c10::cuda::CUDAGuard guard(c.device);
    at::Tensor new_lens = tensor(a[8], "new_lens", true);
    const pa_stream_t stream = c.stream(a[9]);
    if (!new_lens.defined()) new_lens = c.make({B}, kc.options().dtype(at::kInt), stream);
    else if (new_lens.numel() != B) c.no("one new length per sequence is needed");
    c.is(vc, kc.scalar_type(), "v_cache");
    c.is(tables, at::kInt, "block_tables");
    c.is(lens, at::kInt, "context_lens");
    c.is(path, at::kInt, "accepted");
    c.is(take, at::kInt, "accept_lens");
    c.is(tree_lens, at::kInt, "tree_lens");
    c.is(new_lens, at::kInt, "new_lens");
    auto i32 = [&](const at::Tensor& t, const char* what) { return static_cast<int32_t*>(c.ptr(t, what)); };
    c.check(pa_commit_tree(c.ptr(kc, "k_cache"), c.ptr(vc, "v_cache"), o ? small(kc.size(0), c) : 1,
                           i32(tables, "block_tables"), i32(lens, "context_lens"), i32(tree_lens, "tree_lens"),
                           integer32(a[6], "tree_len"), i32(path, "accepted"), small(path.size(1), c),
                           i32(take, "accept_lens"), small(B, c), small(kc.size(o + 1), c), small(kc.size(o + 3), c),
                           small(kc.size(o + 2), c), small(tables.size(1), c), small(kc.size(o), c),
                           i32(new_lens, "new_lens"), dt, stream),
            "pa_commit_tree");
    return a[8] != Py_None ? Py_NewRef(a[8]) : THPVariable_Wrap(new_lens);
  });
}

PyObject* set_error_class(PyObject*, PyObject* cls) {
  Py_XDECREF(g_error_class);
  g_error_class = Py_NewRef(cls);
  Py_RETURN_NONE;
}

PyCFunction fast(PyObject* (*f)(PyObject*, PyObject* const*, Py_ssize_t)) {
  return reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(f));
}

PyMethodDef methods[] = {{"qk_norm_rope", fast(qk_norm_rope), METH_FASTCALL, nullptr},
                         {"rope_append", fast(rope_append), METH_FASTCALL, nullptr},
                         {"decode_tree", fast(decode_tree), METH_FASTCALL, nullptr},
                         {"commit_tree", fast(commit_tree), METH_FASTCALL, nullptr},
                         {"set_error_class", set_error_class, METH_O, nullptr},
                         {nullptr, nullptr, 0, nullptr}};

PyModuleDef module_def = {PyModuleDef_HEAD_INIT, "_native", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__native() { return PyModule_Create(&module_def); }
