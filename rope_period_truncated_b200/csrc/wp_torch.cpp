// The rotary, cache-append, tree-attention, compaction and page calls for
// Python: checks of the tensors, allocation of the results, and the call of the
// C ABI, whose function addresses the package hands over. These calls last a
// few microseconds on the device at their smallest, so their marshalling is
// compiled. Measured, us a call among others, here / marshalled in Python: a
// rotation of 256 tokens 5.6 / 15, an append of 128 tokens 5.7 / 18, an append
// with a compaction 9.2 / 30, a page step of two calls 10.3 / 25.
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <ATen/core/Tensor.h>
#include <ATen/cuda/EmptyTensor.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <climits>
#include <string>
#include <vector>

#include "waveprune.h"

namespace {

decltype(&wp_rope_qk) f_rope_qk;
decltype(&wp_rope_append) f_rope_append;
decltype(&wp_decode_tree_workspace_bytes) f_decode_tree_workspace_bytes;
decltype(&wp_decode_tree) f_decode_tree;
decltype(&wp_kv_compact) f_kv_compact;
decltype(&wp_pages_update_workspace_bytes) f_pages_update_workspace_bytes;
decltype(&wp_pages_update) f_pages_update;
decltype(&wp_pages_copy) f_pages_copy;
PyObject *error_class;  // WavePruneError(name, code)

constexpr auto BF16 = at::kBFloat16;
constexpr auto I32 = at::kInt;

[[noreturn]] void raise(PyObject *type, const std::string &what) {
  PyErr_SetString(type, what.c_str());
  throw python_error();
}
[[noreturn]] void type_error(const std::string &what) { raise(PyExc_TypeError, what); }
[[noreturn]] void value_error(const std::string &what) { raise(PyExc_ValueError, what); }

std::string shape_of(const at::Tensor &t) {
  std::string s = "(";
  for (int64_t d : t.sizes()) s += std::to_string(d) + ", ";
  return s + ")";
}

// The tensor of a Python object, checked. device < 0: any CUDA device.
const at::Tensor &tensor(PyObject *o, const char *name, at::ScalarType type, int64_t ndim, int device, bool contiguous = true) {
  if (!THPVariable_Check(o)) type_error(std::string(name) + " must be a CUDA tensor");
  const at::Tensor &t = THPVariable_Unpack(o);
  if (!t.is_cuda()) type_error(std::string(name) + " must be a CUDA tensor");
  if (t.scalar_type() != type)
    type_error(std::string(name) + " must be " + c10::toString(type) + ", got " + c10::toString(t.scalar_type()));
  if (t.dim() != ndim) value_error(std::string(name) + " must have " + std::to_string(ndim) + " dims, got shape " + shape_of(t));
  if (contiguous && !t.is_contiguous()) value_error(std::string(name) + " must be contiguous");
  if (device >= 0 && t.get_device() != device)
    value_error(std::string(name) + " is on cuda:" + std::to_string(t.get_device()) + ", expected cuda:" + std::to_string(device));
  return t;
}

template <class T>
T *ptr(const at::Tensor &t) {
  return static_cast<T *>(t.data_ptr());
}
const int32_t *ints(const at::Tensor &t) { return ptr<int32_t>(t); }

// A size for the C ABI.
int fit(int64_t n) {
  if (n > INT_MAX) value_error("a size does not fit 32 bits: " + std::to_string(n));
  return static_cast<int>(n);
}

double number(PyObject *o) {
  const double x = PyFloat_AsDouble(o);
  if (x == -1.0 && PyErr_Occurred()) throw python_error();
  return x;
}
int integer(PyObject *o, const char *name) {
  PyObject *i = PyNumber_Index(o);
  if (i == nullptr) throw python_error();
  const long long x = PyLong_AsLongLong(i);
  Py_DECREF(i);
  if (x == -1 && PyErr_Occurred()) throw python_error();
  if (x < INT_MIN || x > INT_MAX) value_error(std::string(name) + " does not fit 32 bits");
  return static_cast<int>(x);
}

// A host table of n numbers (a list, an array, anything with tolist()); empty for None.
template <class T, class Get>
std::vector<T> table(PyObject *o, size_t n, const char *name, Get get) {
  std::vector<T> v;
  if (o == Py_None) return v;
  PyObject *list = nullptr;
  if (PyObject_HasAttrString(o, "tolist")) {
    PyObject *l = PyObject_CallMethod(o, "tolist", nullptr);
    if (l == nullptr) throw python_error();
    list = PySequence_Fast(l, "");
    Py_DECREF(l);
  } else {
    list = PySequence_Fast(o, name);
  }
  if (list == nullptr) throw python_error();
  const size_t m = static_cast<size_t>(PySequence_Fast_GET_SIZE(list));
  try {
    if (m != n) value_error(std::string(name) + " must have " + std::to_string(n) + " entries");
    v.reserve(n);
    for (size_t i = 0; i < n; ++i) v.push_back(get(PySequence_Fast_GET_ITEM(list, static_cast<Py_ssize_t>(i))));
  } catch (...) {
    Py_DECREF(list);
    throw;
  }
  Py_DECREF(list);
  return v;
}
std::vector<double> frequencies(PyObject *o, int rot) {
  return table<double>(o, static_cast<size_t>(rot > 0 ? rot / 2 : 0), "freq_scale (rot_dim/2)", number);
}
std::vector<int32_t> cutoffs(PyObject *o, int64_t d) {
  return table<int32_t>(o, static_cast<size_t>(d / 16), "group_cut (d/16)", [](PyObject *x) { return integer(x, "a cutoff"); });
}
template <class T>
const T *data(const std::vector<T> &v) {
  return v.empty() ? nullptr : v.data();
}

wp_rows rows(const at::Tensor &t) {
  const auto st = t.strides();
  const int64_t n = t.dim();
  if (st[n - 1] != 1 && t.size(n - 1) > 1) value_error("the head dims must be contiguous");
  return wp_rows{t.data_ptr(), n == 4 ? st[0] : 0, st[n - 3], st[n - 2]};
}

// Device and stream of a call: the given stream, or the current one of the
// tensors' device. What a call allocates is written on its stream, so it comes
// from that stream's memory: memory that the current stream has given back may
// still be read by what is enqueued there. Results are marked as used on the
// current stream too, where the caller goes on with them.
struct Call {
  c10::cuda::CUDAGuard guard;
  int device;
  c10::cuda::CUDAStream current, stream;
  Call(int dev, PyObject *s)
      : guard(static_cast<c10::DeviceIndex>(dev)),
        device(dev),
        current(c10::cuda::getCurrentCUDAStream(static_cast<c10::DeviceIndex>(dev))),
        stream(current) {
    if (s == Py_None) return;
    const auto attr = [&](const char *name) {
      PyObject *x = PyObject_GetAttrString(s, name);
      if (x == nullptr) throw python_error();
      const long long v = PyLong_AsLongLong(x);
      Py_DECREF(x);
      if (v == -1 && PyErr_Occurred()) throw python_error();
      return v;
    };
    const long long index = attr("device_index");
    if (index != dev)
      value_error("the stream is on cuda:" + std::to_string(index) + ", the tensors on cuda:" + std::to_string(dev));
    stream = c10::cuda::CUDAStream::unpack3(attr("stream_id"), static_cast<c10::DeviceIndex>(index),
                                            static_cast<c10::DeviceType>(attr("device_type")));
  }
  at::Tensor empty(at::IntArrayRef size, at::ScalarType type, bool result = true) {
    const c10::Device on(c10::kCUDA, static_cast<c10::DeviceIndex>(device));
    if (stream == current) return at::detail::empty_cuda(size, type, on, std::nullopt);
    const c10::cuda::CUDAStreamGuard its(stream);
    at::Tensor t = at::detail::empty_cuda(size, type, on, std::nullopt);
    if (result) t.record_stream(current);
    return t;
  }
  void *handle() const { return stream.stream(); }
};

// Runs a call of the library without the interpreter's lock.
template <class F>
void run(const char *name, F &&f) {
  int code;
  Py_BEGIN_ALLOW_THREADS;
  code = f();
  Py_END_ALLOW_THREADS;
  if (code != WP_OK) {
    PyObject *e = PyObject_CallFunction(error_class, "si", name, code);
    if (e != nullptr) {
      PyErr_SetObject(error_class, e);
      Py_DECREF(e);
    }
    throw python_error();
  }
}

PyObject *give(PyObject *given, const at::Tensor &t) {
  if (given != Py_None) return Py_NewRef(given);
  return THPVariable_Wrap(t);
}

// A K/V cache: contiguous, or pools of pages with a block table.
struct Cache {
  void *k, *v;
  const int32_t *block_table = nullptr;
  int layout, B, Lmax = 0, max_pages = 0, page_size = 0, n_pages = 0, Hkv, d;
};
Cache cache(PyObject *ko, PyObject *vo, PyObject *bt, int device, int64_t B = -1, int64_t Hkv = -1, int64_t d = -1) {
  const at::Tensor &v = tensor(vo, "vcache", BF16, 4, device);
  const bool gm = THPVariable_Check(ko) && THPVariable_Unpack(ko).dim() == 5;
  const at::Tensor &k = tensor(ko, "kcache", BF16, gm ? 5 : 4, device);
  const int64_t n = v.size(0), H = v.size(1), rows = v.size(2), dd = v.size(3);
  if (gm) {
    if (k.size(0) != n || k.size(1) != H || k.size(2) != dd / 16 || k.size(3) != rows || k.size(4) != 16)
      value_error("group-major K cache shape mismatch");
  } else if (k.sizes() != v.sizes()) {
    value_error("K cache shape mismatch");
  }
  if ((Hkv >= 0 && H != Hkv) || (d >= 0 && dd != d)) value_error("the cache's heads or head dim do not match");
  Cache c;
  c.k = k.data_ptr();
  c.v = v.data_ptr();
  c.layout = gm ? WP_KCACHE_GROUP_MAJOR : WP_KCACHE_ROWS;
  c.Hkv = fit(H);
  c.d = fit(dd);
  if (bt == Py_None) {
    if (B >= 0 && n != B) value_error("the cache holds " + std::to_string(n) + " sequences, expected " + std::to_string(B));
    c.B = fit(n);
    c.Lmax = fit(rows);
    return c;
  }
  const at::Tensor &t = tensor(bt, "block_table", I32, 2, device);
  if (B >= 0 && t.size(0) != B) value_error("the block table has " + std::to_string(t.size(0)) + " rows, expected " + std::to_string(B));
  c.block_table = ints(t);
  c.B = fit(t.size(0));
  c.max_pages = fit(t.size(1));
  c.page_size = fit(rows);
  c.n_pages = fit(n);
  return c;
}

void count(Py_ssize_t n, Py_ssize_t want) {
  if (n != want) type_error("expected " + std::to_string(want) + " arguments, got " + std::to_string(n));
}

// (q, k, theta, layout, pos, pos0, rot_dim, freq_scale, scale_all, amplitude, inverse, out_q, out_k, stream)
PyObject *rope_qk(PyObject *, PyObject *const *a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  count(n, 14);
  const bool has[2] = {a[0] != Py_None, a[1] != Py_None};
  if (!has[0] && !has[1]) value_error("q and k are both None");
  const char *names[2] = {"q", "k"}, *out_names[2] = {"out_q", "out_k"};
  const at::Tensor &x = tensor(has[0] ? a[0] : a[1], has[0] ? "q" : "k", BF16, 4, -1, false);
  const int device = x.get_device();
  const int B = fit(x.size(0)), N = fit(x.size(1)), d = fit(x.size(3));
  Call call(device, a[13]);
  wp_rows in[2] = {}, out[2] = {};
  int H[2] = {0, 0};
  at::Tensor made[2];
  for (int i = 0; i < 2; ++i) {
    PyObject *o = a[11 + i];
    if (!has[i]) {
      if (o != Py_None) value_error(std::string(out_names[i]) + " without its input");
      continue;
    }
    const at::Tensor &t = tensor(a[i], names[i], BF16, 4, device, false);
    if (t.size(0) != B || t.size(1) != N || t.size(3) != d) value_error("q/k shape mismatch");
    H[i] = fit(t.size(2));
    if (o != Py_None) {
      const at::Tensor &given = tensor(o, out_names[i], BF16, 4, device, false);
      if (given.sizes() != t.sizes()) value_error(std::string(out_names[i]) + " shape mismatch");
      out[i] = rows(given);
    } else {
      made[i] = call.empty(t.sizes(), BF16);
      out[i] = rows(made[i]);
    }
    in[i] = rows(t);
  }
  const int32_t *pos = nullptr;
  if (a[4] != Py_None) {
    const at::Tensor &t = tensor(a[4], "pos", I32, 2, device);
    if (t.size(0) != B || t.size(1) != N) value_error("pos must be [B, N]");
    pos = ints(t);
  }
  const double theta = number(a[2]), scale_all = number(a[8]), amplitude = number(a[9]);
  const int layout = integer(a[3], "layout"), pos0 = integer(a[5], "pos0");
  const int rot = a[6] == Py_None ? d : integer(a[6], "rot_dim");
  const std::vector<double> fs = frequencies(a[7], rot);
  const int inverse = PyObject_IsTrue(a[10]);
  if (inverse < 0) throw python_error();
  run("wp_rope_qk", [&] {
    return f_rope_qk(&in[0], &out[0], H[0], &in[1], &out[1], H[1], B, N, d, rot, pos, pos0, theta, data(fs), scale_all, amplitude, layout,
                     inverse, call.handle());
  });
  PyObject *r = PyTuple_New(2);
  for (int i = 0; i < 2; ++i) PyTuple_SET_ITEM(r, i, has[i] ? give(a[11 + i], made[i]) : Py_NewRef(Py_None));
  return r;
  END_HANDLE_TH_ERRORS
}

// (q, k, v, kcache, vcache, pos, seq, slot, theta, layout, block_table, rot_dim, freq_scale, scale_all, amplitude, out_q, stream)
PyObject *rope_append(PyObject *, PyObject *const *a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  count(n, 17);
  const at::Tensor &k = tensor(a[1], "k", BF16, 3, -1, false);
  const int device = k.get_device();
  const int T = fit(k.size(0)), Hkv = fit(k.size(1)), d = fit(k.size(2));
  const at::Tensor &v = tensor(a[2], "v", BF16, 3, device, false);
  if (v.sizes() != k.sizes()) value_error("k/v shape mismatch");
  const int32_t *index[3];
  const char *names[3] = {"pos", "seq", "slot"};
  for (int i = 0; i < 3; ++i) {
    const at::Tensor &t = tensor(a[5 + i], names[i], I32, 1, device);
    if (t.size(0) != T) value_error(std::string(names[i]) + " must be [T]");
    index[i] = ints(t);
  }
  const Cache c = cache(a[3], a[4], a[10], device, -1, Hkv, d);
  const double theta = number(a[8]), scale_all = number(a[13]), amplitude = number(a[14]);
  const int layout = integer(a[9], "layout");
  const int rot = a[11] == Py_None ? d : integer(a[11], "rot_dim");
  const std::vector<double> fs = frequencies(a[12], rot);
  Call call(device, a[16]);
  wp_rows q = {}, qo = {};
  int Hq = 0;
  at::Tensor made;
  if (a[0] != Py_None) {
    const at::Tensor &t = tensor(a[0], "q", BF16, 3, device, false);
    if (t.size(0) != T || t.size(2) != d) value_error("q shape mismatch");
    Hq = fit(t.size(1));
    if (a[15] != Py_None) {
      const at::Tensor &given = tensor(a[15], "out_q", BF16, 3, device, false);
      if (given.sizes() != t.sizes()) value_error("out_q shape mismatch");
      qo = rows(given);
    } else {
      made = call.empty(t.sizes(), BF16);
      qo = rows(made);
    }
    q = rows(t);
  } else if (a[15] != Py_None) {
    value_error("out_q without q");
  }
  const wp_rows kr = rows(k), vr = rows(v);
  run("wp_rope_append", [&] {
    return f_rope_append(&q, &qo, Hq, &kr, &vr, Hkv, T, d, rot, index[0], index[1], index[2], c.k, c.layout, c.v, c.B, c.Lmax, c.block_table,
                         c.max_pages, c.page_size, c.n_pages, theta, data(fs), scale_all, amplitude, layout, call.handle());
  });
  return a[0] == Py_None ? Py_NewRef(Py_None) : give(a[15], made);
  END_HANDLE_TH_ERRORS
}

// A workspace that the caller gave, or one of `need` bytes.
struct Workspace {
  at::Tensor made;
  void *data = nullptr;
  size_t bytes = 0;
  Workspace(PyObject *given, size_t need, Call &call) {
    if (given != Py_None) {
      if (!THPVariable_Check(given)) type_error("workspace must be a CUDA tensor");
      const at::Tensor &t = THPVariable_Unpack(given);
      if (!t.is_cuda() || t.get_device() != call.device || !t.is_contiguous())
        value_error("workspace must be a contiguous tensor on the same device");
      data = t.data_ptr();
      bytes = t.nbytes();
    } else if (need > 0) {
      made = call.empty({static_cast<int64_t>(need)}, at::kByte, false);
      data = made.data_ptr();
      bytes = need;
    }
  }
};

// (q, kcache, vcache, lens, parents, n_nodes, block_table, group_cut, softmax_scale, out, lse, workspace, want_lse, stream)
PyObject *decode_tree(PyObject *, PyObject *const *a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  count(n, 14);
  const at::Tensor &q = tensor(a[0], "q", BF16, 4, -1);
  const int device = q.get_device();
  const int B = fit(q.size(0)), T = fit(q.size(1)), Hq = fit(q.size(2)), d = fit(q.size(3));
  const at::Tensor &lens = tensor(a[3], "lens", I32, 1, device);
  const at::Tensor &parents = tensor(a[4], "parents", I32, 2, device);
  if (lens.size(0) != B || parents.size(0) != B || parents.size(1) != T) value_error("lens must be [B] and parents [B, T]");
  const int32_t *nodes = nullptr;
  if (a[5] != Py_None) {
    const at::Tensor &t = tensor(a[5], "n_nodes", I32, 1, device);
    if (t.size(0) != B) value_error("n_nodes must be [B]");
    nodes = ints(t);
  }
  const Cache c = cache(a[1], a[2], a[6], device, B, -1, d);
  const std::vector<int32_t> cut = cutoffs(a[7], d);
  const double scale = number(a[8]);
  Call call(device, a[13]);
  at::Tensor made, made_lse;
  void *o;
  float *lse = nullptr;
  if (a[9] != Py_None) {
    const at::Tensor &t = tensor(a[9], "out", BF16, 4, device);
    if (t.sizes() != q.sizes()) value_error("out shape mismatch");
    o = t.data_ptr();
  } else {
    made = call.empty(q.sizes(), BF16);
    o = made.data_ptr();
  }
  const int want = PyObject_IsTrue(a[12]);
  if (want < 0) throw python_error();
  if (a[10] != Py_None) {
    const at::Tensor &t = tensor(a[10], "lse", at::kFloat, 3, device);
    if (t.size(0) != B || t.size(1) != Hq || t.size(2) != T) value_error("lse must be [B, Hq, T]");
    lse = ptr<float>(t);
  } else if (want) {
    made_lse = call.empty({B, Hq, T}, at::kFloat);
    lse = ptr<float>(made_lse);
  }
  const int64_t capacity = c.block_table == nullptr ? c.Lmax : static_cast<int64_t>(c.max_pages) * c.page_size;
  const size_t need = capacity > INT_MAX ? 0 : f_decode_tree_workspace_bytes(B, T, Hq, c.Hkv, d, static_cast<int>(capacity));
  Workspace ws(a[11], need, call);
  run("wp_decode_tree", [&] {
    return f_decode_tree(q.data_ptr(), c.k, c.layout, c.v, ints(lens), ints(parents), nodes, T, c.Lmax, c.block_table, c.max_pages,
                         c.page_size, c.n_pages, B, Hq, c.Hkv, d, data(cut), static_cast<float>(scale), o, lse, ws.data, ws.bytes,
                         call.handle());
  });
  PyObject *r = PyTuple_New(2);
  PyTuple_SET_ITEM(r, 0, give(a[9], made));
  PyTuple_SET_ITEM(r, 1, lse == nullptr ? Py_NewRef(Py_None) : give(a[10], made_lse));
  return r;
  END_HANDLE_TH_ERRORS
}

// (kcache, vcache, lens, path, n_keep, block_table, out, stream)
PyObject *kv_compact(PyObject *, PyObject *const *a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  count(n, 8);
  const at::Tensor &lens = tensor(a[2], "lens", I32, 1, -1);
  const int device = lens.get_device();
  const int64_t B = lens.size(0);
  const at::Tensor &path = tensor(a[3], "path", I32, 2, device);
  const at::Tensor &keep = tensor(a[4], "n_keep", I32, 1, device);
  if (path.size(0) != B || keep.size(0) != B) value_error("path must be [B, A] and n_keep [B]");
  const Cache c = cache(a[0], a[1], a[5], device, B);
  Call call(device, a[7]);
  at::Tensor made;
  int32_t *out;
  if (a[6] != Py_None) {
    const at::Tensor &t = tensor(a[6], "out", I32, 1, device);
    if (t.size(0) != B) value_error("out must be [B]");
    out = ptr<int32_t>(t);
  } else {
    made = call.empty({B}, I32);
    out = ptr<int32_t>(made);
  }
  const int A = fit(path.size(1));
  run("wp_kv_compact", [&] {
    return f_kv_compact(c.k, c.layout, c.v, ints(lens), ints(path), A, ints(keep), out, c.Lmax, c.block_table,
                        c.max_pages, c.page_size, c.n_pages, c.B, c.Hkv, c.d, call.handle());
  });
  return give(a[6], made);
  END_HANDLE_TH_ERRORS
}

// (refs, block_table, lens, parent, keep, new_lens, page_size, workspace, stream)
PyObject *pages_update(PyObject *, PyObject *const *a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  count(n, 9);
  const at::Tensor &refs = tensor(a[0], "refs", I32, 1, -1);
  const int device = refs.get_device();
  const at::Tensor &bt = tensor(a[1], "block_table", I32, 2, device);
  const int pages = fit(refs.size(0)), B = fit(bt.size(0)), most = fit(bt.size(1));
  const char *names[4] = {"lens", "parent", "keep", "new_lens"};
  const int32_t *in[4];
  for (int i = 0; i < 4; ++i) {
    const at::Tensor &t = tensor(a[2 + i], names[i], I32, 1, device);
    if (t.size(0) != B) value_error(std::string(names[i]) + " must be [B]");
    in[i] = ints(t);
  }
  const int page = integer(a[6], "page_size");
  Call call(device, a[8]);
  const at::Tensor out[5] = {call.empty({pages}, I32), call.empty({B, most}, I32), call.empty({B}, I32), call.empty({B, 3}, I32),
                             call.empty({4}, I32)};
  Workspace ws(a[7], f_pages_update_workspace_bytes(B, pages), call);
  run("wp_pages_update", [&] {
    return f_pages_update(ints(refs), ints(bt), in[0], in[1], in[2], in[3], ptr<int32_t>(out[0]), ptr<int32_t>(out[1]), ptr<int32_t>(out[2]),
                          ptr<int32_t>(out[3]), ptr<int32_t>(out[4]), B, most, page, pages, ws.data, ws.bytes, call.handle());
  });
  PyObject *r = PyTuple_New(5);
  for (int i = 0; i < 5; ++i) PyTuple_SET_ITEM(r, i, THPVariable_Wrap(out[i]));
  return r;
  END_HANDLE_TH_ERRORS
}

// (k_pages, v_pages, copies, stream)
PyObject *pages_copy(PyObject *, PyObject *const *a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  count(n, 4);
  const at::Tensor &copies = tensor(a[2], "copies", I32, 2, -1);
  if (copies.size(1) != 3) value_error("copies must be [n, 3]");
  const int device = copies.get_device();
  const Cache c = cache(a[0], a[1], a[2], device);
  Call call(device, a[3]);
  run("wp_pages_copy", [&] {
    return f_pages_copy(c.k, c.layout, c.v, ints(copies), c.B, c.n_pages, c.page_size, c.Hkv, c.d, call.handle());
  });
  Py_RETURN_NONE;
  END_HANDLE_TH_ERRORS
}

// (addresses of the library's functions by name, the error class)
PyObject *connect(PyObject *, PyObject *const *a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  count(n, 2);
  const auto at = [&](const char *name) {
    PyObject *o = PyDict_GetItemString(a[0], name);
    if (o == nullptr) value_error(std::string("no address of ") + name);
    void *p = PyLong_AsVoidPtr(o);
    if (p == nullptr) value_error(std::string("no address of ") + name);
    return p;
  };
#define CONNECT(name) f_##name = reinterpret_cast<decltype(f_##name)>(at("wp_" #name))
  CONNECT(rope_qk);
  CONNECT(rope_append);
  CONNECT(decode_tree_workspace_bytes);
  CONNECT(decode_tree);
  CONNECT(kv_compact);
  CONNECT(pages_update_workspace_bytes);
  CONNECT(pages_update);
  CONNECT(pages_copy);
#undef CONNECT
  error_class = Py_NewRef(a[1]);
  Py_RETURN_NONE;
  END_HANDLE_TH_ERRORS
}

using Fast = PyObject *(*)(PyObject *, PyObject *const *, Py_ssize_t);
PyMethodDef method(const char *name, Fast f) {
  return {name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(f)), METH_FASTCALL, nullptr};
}
PyMethodDef methods[] = {method("connect", connect),
                         method("rope_qk", rope_qk),
                         method("rope_append", rope_append),
                         method("decode_tree", decode_tree),
                         method("kv_compact", kv_compact),
                         method("pages_update", pages_update),
                         method("pages_copy", pages_copy),
                         {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_calls", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__calls() { return PyModule_Create(&module); }
