// The Python binding of the calls a step makes several of, natively: argument checks
// and marshalling of torch tensors in C++.
//
// A step's table, tree and commit kernels take a few microseconds each, less than the
// checks of their dozen tensors (for the commit, of every layer's pools) take in
// Python: 10 us for pa_build_tables, 36 us for a 32-layer pa_commit_tree, against
// 2 us and 4 us here. Nothing is computed and nothing kept here; the module calls the
// C entry points of libpa.so, whose addresses the Python side hands over once.
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <ATen/core/TensorBody.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include <cstring>
#include <exception>
#include <vector>

#include "pa.h"

namespace {

using at::ScalarType;
using at::Tensor;

PyObject* g_error = nullptr;  // PAError(func, status, detail)
decltype(&pa_build_tables) g_build_tables = nullptr;
decltype(&pa_decode_tree) g_decode_tree = nullptr;
decltype(&pa_commit_tree_keep) g_commit_tree = nullptr;

struct Refused {
  int status;
  const char* what;
};
void need(bool cond, const char* what, int status = PA_ERR_INVALID_ARG) {
  if (!cond) throw Refused{status, what};
}

const Tensor& tensor(PyObject* o) {
  need(THPVariable_Check(o), "a tensor was expected");
  return THPVariable_Unpack(o);
}
const Tensor* optional_tensor(PyObject* o) { return o == Py_None ? nullptr : &tensor(o); }

long long integer(PyObject* o) {
  // (numpy integers and the like have __index__; a float does not)
  PyObject* i = PyNumber_Index(o);
  need(i != nullptr, "an integer was expected");
  const long long v = PyLong_AsLongLong(i);
  Py_DECREF(i);
  need(v != -1 || !PyErr_Occurred(), "an integer is out of range");
  return v;
}
int int32(PyObject* o) {
  const long long v = integer(o);
  need(v >= -0x80000000LL && v <= 0x7fffffffLL, "an integer is out of range");
  return (int)v;
}
int int32(int64_t v) {
  need(v <= 0x7fffffffLL, "a dimension is out of range", PA_ERR_UNSUPPORTED);
  return (int)v;
}

// The current device; the calls launch there, so every tensor has to lie there.
struct Device {
  int index = -1;
  void check(const Tensor& t) {
    need(t.is_cuda() && t.is_contiguous(), "tensors must be contiguous and on the current CUDA device");
    if (index < 0) index = c10::cuda::current_device();
    need(t.get_device() == index, "tensors must be contiguous and on the current CUDA device");
  }
  // `o`: None (the current stream) or a stream's address
  cudaStream_t stream(PyObject* o) const {
    if (o == Py_None) return c10::cuda::getCurrentCUDAStream((c10::DeviceIndex)index).stream();
    return reinterpret_cast<cudaStream_t>((uintptr_t)integer(o));
  }
};

int32_t* i32(Device& d, const Tensor& t) {
  d.check(t);
  need(t.scalar_type() == ScalarType::Int, "lengths, tables and starts must be int32");
  return static_cast<int32_t*>(t.data_ptr());
}
bool is_1d(const Tensor& t, int64_t n) { return t.dim() == 1 && t.size(0) == n; }

pa_dtype dtype_of(const Tensor& t) {
  switch (t.scalar_type()) {
    case ScalarType::Float: return PA_F32;
    case ScalarType::Half: return PA_F16;
    case ScalarType::BFloat16: return PA_BF16;
    case ScalarType::Byte:
    case ScalarType::Float8_e4m3fn: return PA_FP8_E4M3;
    default: throw Refused{PA_ERR_UNSUPPORTED, "element type"};
  }
}

int64_t* mask_of(Device& d, const Tensor& t, int64_t tokens, int* words) {
  d.check(t);
  need(t.scalar_type() == ScalarType::Long && t.dim() == 2 && t.size(0) == tokens,
       "tree_mask must be int64 [num_tokens, mask_words]");
  *words = int32(t.size(1));
  return static_cast<int64_t*>(t.data_ptr());
}

struct Pool {
  pa_kv_layout layout;
  int64_t blocks;
  int G, B, D;
};
Pool pool_of(const Tensor& t, PyObject* layout) {
  const char* s = PyUnicode_Check(layout) ? PyUnicode_AsUTF8(layout) : nullptr;
  const bool hnd = s && !strcmp(s, "HND"), nhd = s && !strcmp(s, "NHD");
  need(hnd || nhd, "layout must be 'HND' or 'NHD'");
  need(t.dim() == 4, "pools are 4-D");
  return {hnd ? PA_LAYOUT_HND : PA_LAYOUT_NHD, t.size(0), int32(t.size(hnd ? 1 : 2)), int32(t.size(hnd ? 2 : 1)),
          int32(t.size(3))};
}

// Run `body`, which returns the call's status; anything but PA_OK raises.
template <typename F>
PyObject* guarded(const char* func, Py_ssize_t nargs, Py_ssize_t want, F body) {
  int status;
  const char* what = "";
  try {
    need(nargs == want, "argument count");
    status = body();
  } catch (const Refused& r) {
    status = r.status;
    what = r.what;
  } catch (const std::exception& e) {
    PyErr_SetString(PyExc_RuntimeError, e.what());
    return nullptr;
  }
  if (status == PA_OK) Py_RETURN_NONE;
  PyErr_Clear();  // (a conversion's own complaint)
  PyObject* e = PyObject_CallFunction(g_error, "sis", func, status, what);
  if (e) {
    PyErr_SetObject(g_error, e);
    Py_DECREF(e);
  }
  return nullptr;
}

// Returns True for a batch of no sequences, for which the library launches nothing, else None.
PyObject* build_tables(PyObject*, PyObject* const* a, Py_ssize_t nargs) {
  bool empty = false;
  PyObject* done = guarded("pa_build_tables", nargs, 17, [&]() -> int {
    Device d;
    const Tensor& bt = tensor(a[0]);
    int32_t* bt_p = i32(d, bt);
    need(bt.dim() == 2, "block_tables must be 2-D");
    const int64_t S = bt.size(0);
    empty = S == 0;
    auto lengths = [&](PyObject* o) {
      const Tensor& t = tensor(o);
      need(is_1d(t, S), "lengths must be [num_seqs]");
      return i32(d, t);
    };
    auto one = [&](PyObject* o) {
      const Tensor& t = tensor(o);
      need(t.numel() == 1, "free_first and free_first_out are one entry");
      return i32(d, t);
    };
    int32_t *tl_out = lengths(a[1]), *cl_out = lengths(a[2]);
    const Tensor& starts = tensor(a[3]);
    need(is_1d(starts, S + 1), "query_starts must be [num_seqs + 1]");
    const Tensor& slots = tensor(a[4]);
    d.check(slots);
    need(slots.scalar_type() == ScalarType::Long && slots.dim() == 1, "slot_mapping must be int64 [max_tokens]");
    const int64_t N = slots.size(0);
    const Tensor& pos = tensor(a[5]);
    need(is_1d(pos, N), "positions must be [max_tokens]");
    int32_t* ff_out = one(a[6]);
    const int32_t *tl = lengths(a[7]), *cl = lengths(a[8]), *nl = lengths(a[9]);
    const Tensor& free_blocks = tensor(a[10]);
    need(free_blocks.dim() == 1, "free_blocks must be 1-D");
    const int32_t *fb = i32(d, free_blocks), *ff = one(a[11]);
    const Tensor *par = optional_tensor(a[14]), *mask = optional_tensor(a[15]);
    need((par == nullptr) == (mask == nullptr), "parents and tree_mask go together");
    int words = 0;
    int32_t* par_p = nullptr;
    int64_t* mask_p = nullptr;
    if (par) {
      need(is_1d(*par, N), "parents must be [max_tokens]");
      par_p = i32(d, *par);
      mask_p = mask_of(d, *mask, N, &words);
    }
    return g_build_tables(bt_p, int32(bt.size(1)), tl_out, cl_out, i32(d, starts),
                          static_cast<int64_t*>(slots.data_ptr()), i32(d, pos), ff_out, tl, cl, nl, fb,
                          int32(free_blocks.size(0)), ff, par_p, mask_p, words, int32(S), int32(N), int32(a[12]),
                          integer(a[13]), d.stream(a[16]));
  });
  if (done == nullptr || !empty) return done;
  Py_DECREF(done);
  Py_RETURN_TRUE;
}

PyObject* decode_tree(PyObject*, PyObject* const* a, Py_ssize_t nargs) {
  return guarded("pa_decode_tree", nargs, 13, [&]() -> int {
    Device d;
    const Tensor &out = tensor(a[0]), &q = tensor(a[1]), &k = tensor(a[2]), &v = tensor(a[3]), &bt = tensor(a[4]),
                 &ctx = tensor(a[5]), &starts = tensor(a[6]), &ws = tensor(a[10]);
    for (const Tensor* t : {&out, &q, &k, &v, &ws}) d.check(*t);
    need(q.scalar_type() == k.scalar_type() && q.scalar_type() == v.scalar_type(), "q / cache dtype mismatch");
    need(q.dim() == 3 && out.sizes() == q.sizes(), "q and out must be [num_tokens, num_heads, head_dim]");
    const Pool p = pool_of(k, a[12]);
    need(v.sizes() == k.sizes() && p.D == q.size(2), "shapes");
    need(bt.dim() == 2, "block_tables must be 2-D");
    const int64_t S = bt.size(0), N = q.size(0);
    need(is_1d(ctx, S) && is_1d(starts, S + 1), "table shapes");
    const Tensor* mask = optional_tensor(a[7]);
    int words = 0;
    int64_t* mask_p = mask ? mask_of(d, *mask, N, &words) : nullptr;
    const double scale = PyFloat_AsDouble(a[8]);
    need(scale != -1.0 || !PyErr_Occurred(), "scale must be a number");
    return g_decode_tree(out.data_ptr(), q.data_ptr(), k.data_ptr(), v.data_ptr(), i32(d, bt), int32(bt.size(1)),
                         i32(d, ctx), i32(d, starts), mask_p, words, int32(S), int32(N), int32(q.size(1)), p.G, p.D,
                         p.B, p.layout, p.blocks, (float)scale, dtype_of(q), dtype_of(out), int32(a[9]),
                         ws.data_ptr(), ws.nbytes(), d.stream(a[11]));
  });
}

PyObject* commit_tree(PyObject*, PyObject* const* a, Py_ssize_t nargs) {
  return guarded("pa_commit_tree", nargs, 11, [&]() -> int {
    Device d;
    const Tensor* first = nullptr;
    auto pools = [&](PyObject* o, std::vector<void*>& ptrs) {
      need(PyList_Check(o) || PyTuple_Check(o), "pools come as a list or tuple");
      const Py_ssize_t n = PySequence_Fast_GET_SIZE(o);
      PyObject** items = PySequence_Fast_ITEMS(o);
      ptrs.reserve(n);
      for (Py_ssize_t i = 0; i < n; ++i) {
        const Tensor& t = tensor(items[i]);
        d.check(t);
        if (!first) first = &t;
        need(t.scalar_type() == first->scalar_type() && t.sizes() == first->sizes(),
             "all pools must share shape and dtype");
        ptrs.push_back(t.data_ptr());
      }
    };
    std::vector<void*> k, v;
    pools(a[0], k);
    pools(a[1], v);
    need(!k.empty() && k.size() == v.size(), "one K and one V pool per layer");
    const Pool p = pool_of(*first, a[9]);
    const Tensor &bt = tensor(a[2]), &ctx = tensor(a[3]), &starts = tensor(a[4]), &acc = tensor(a[6]),
                 &out = tensor(a[7]);
    need(bt.dim() == 2, "block_tables must be 2-D");
    const int64_t S = bt.size(0);
    const Tensor* before = optional_tensor(a[10]);
    need(is_1d(ctx, S) && is_1d(acc, S) && is_1d(out, S) && is_1d(starts, S + 1) && (!before || is_1d(*before, S)),
         "table shapes");
    const Tensor* mask = optional_tensor(a[5]);
    int words = 0;
    const int64_t N = mask && mask->dim() > 0 ? mask->size(0) : 0x7fffffff;
    int64_t* mask_p = mask ? mask_of(d, *mask, N, &words) : nullptr;
    return g_commit_tree(k.data(), v.data(), int32((int64_t)k.size()), i32(d, bt), int32(bt.size(1)), i32(d, ctx),
                         before ? i32(d, *before) : nullptr, i32(d, starts), mask_p, words, i32(d, acc), i32(d, out),
                         int32(S), int32(N), p.G, p.D, p.B, p.layout, p.blocks, dtype_of(*first), d.stream(a[8]));
  });
}

// connect(PAError, address of pa_build_tables, of pa_decode_tree, of pa_commit_tree_keep)
PyObject* connect(PyObject*, PyObject* const* a, Py_ssize_t nargs) {
  if (nargs != 4) {
    PyErr_SetString(PyExc_TypeError, "connect takes the error class and three addresses");
    return nullptr;
  }
  Py_INCREF(a[0]);
  Py_XDECREF(g_error);
  g_error = a[0];
  g_build_tables = reinterpret_cast<decltype(g_build_tables)>(PyLong_AsVoidPtr(a[1]));
  g_decode_tree = reinterpret_cast<decltype(g_decode_tree)>(PyLong_AsVoidPtr(a[2]));
  g_commit_tree = reinterpret_cast<decltype(g_commit_tree)>(PyLong_AsVoidPtr(a[3]));
  if (PyErr_Occurred()) return nullptr;
  Py_RETURN_NONE;
}

#define PA_METHOD(f) {#f, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(f)), METH_FASTCALL, nullptr}
PyMethodDef g_methods[] = {PA_METHOD(connect), PA_METHOD(build_tables), PA_METHOD(decode_tree),
                           PA_METHOD(commit_tree), {nullptr, nullptr, 0, nullptr}};
PyModuleDef g_module = {PyModuleDef_HEAD_INIT, "_pa_torch", nullptr, -1, g_methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__pa_torch(void) { return PyModule_Create(&g_module); }
