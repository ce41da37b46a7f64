// Python entry points of the selected-block operators: argument checks and the
// call into libmbt.so. (CPython C API; tensors through torch's own accessors.) These
// calls are a few microseconds long on the device and take up to a dozen tensors,
// whose checks in Python took 5 to 6 us and ctypes 1.2: extending 64 sequences took
// 10.3 us a call that way and takes 3.2 from here.
//
// Every function takes its arguments by position, the error word or None and the
// stream's handle or None (torch's current one) last, and returns the status code.
// ValueError names a tensor that is not what the entry point reads.
#include <torch/csrc/autograd/python_variable.h>

#include <climits>
#include <initializer_list>

#include <ATen/ops/empty.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>

#include "../../include/mbt.h"
#include "../../include/mbt_ops.h"

namespace {

struct Refused {};                                        // the Python error is set

class Call {
 public:
  Call(const char* fn, PyObject* const* args, Py_ssize_t given, Py_ssize_t want) : fn_(fn), args_(args) {
    if (given != want) {
      PyErr_Format(PyExc_TypeError, "%s takes %zd arguments (%zd given)", fn, want, given);
      throw Refused{};
    }
  }
  bool bad = false;                                       // a number that no int holds

  // A number, checked before 32 bits are taken of it.
  int integer(int i) {
    const long long v = PyLong_AsLongLong(args_[i]);
    if (v == -1 && PyErr_Occurred()) {
      if (!PyErr_ExceptionMatches(PyExc_OverflowError)) throw Refused{};
      PyErr_Clear();
      bad = true;
      return 0;
    }
    if (v < INT_MIN || v > INT_MAX) bad = true;
    return (int)v;
  }
  float number(int i) {
    const double v = PyFloat_AsDouble(args_[i]);
    if (v == -1.0 && PyErr_Occurred()) throw Refused{};
    return (float)v;
  }
  bool none(int i) const { return args_[i] == Py_None; }

  // The tensor that says which device the call is for: the current one.
  const at::Tensor& lead(int i, const char* name, at::ScalarType type, int dims) {
    const at::Tensor& t = sized(i, name, dims);
    if (!t.is_cuda()) refuse(name, "must be a device tensor");
    dev_ = t.get_device();
    if (dev_ != c10::cuda::current_device()) refuse(name, "is on another device than the current one");
    check(t, name, type);
    return t;
  }
  // One that brings sizes of its own.
  const at::Tensor& own(int i, const char* name, at::ScalarType type, int dims) {
    const at::Tensor& t = sized(i, name, dims);
    check(t, name, type);
    return t;
  }
  // Address of a dense tensor of this type and shape.
  template <class T>
  T* dense(int i, const char* name, at::ScalarType type, std::initializer_list<int64_t> shape) {
    const at::Tensor& t = tensor(i, name);
    check(t, name, type);
    if (t.sizes() != at::IntArrayRef(shape.begin(), shape.size())) {
      PyErr_Format(PyExc_ValueError, "%s: %s has another shape than expected", fn_, name);
      throw Refused{};
    }
    return static_cast<T*>(t.data_ptr());
  }
  // A pool of at least num_blocks + 1 blocks in the cache format, of any shape and element type.
  const void* pool(int i, const char* name, int nkv, int d, int num_blocks, int kv_dtype) {
    const at::Tensor& t = tensor(i, name);
    device(t, name);
    if (!t.is_contiguous()) refuse(name, "must be contiguous");
    const size_t unit = op_kv_unit_bytes(d, kv_dtype);
    if (!unit || nkv < 1 || num_blocks < 1 || bad) {
      bad = true;
      return nullptr;
    }
    if (t.nbytes() / unit / (size_t)nkv < (size_t)num_blocks + 1) refuse(name, "is smaller than num_blocks + 1 blocks");
    return t.data_ptr();
  }
  // Bytes on the device, any number of them.
  void* bytes(int i, const char* name, size_t& count) {
    const at::Tensor& t = tensor(i, name);
    check(t, name, at::kByte);
    count = t.nbytes();
    return t.data_ptr();
  }
  const int32_t* rows(int i, int64_t n, int64_t nseq) {   // row_seq, or null: row i is sequence i
    if (!none(i)) return dense<int32_t>(i, "row_seq", at::kInt, {n});
    if (nseq < n) {
      PyErr_Format(PyExc_ValueError, "%s: bt has fewer rows than positions (give row_seq)", fn_);
      throw Refused{};
    }
    return nullptr;
  }
  uint32_t* err(int i) { return none(i) ? nullptr : dense<uint32_t>(i, "err", at::kInt, {1}); }
  void* stream(int i) {
    if (none(i)) return c10::cuda::getCurrentCUDAStream((c10::DeviceIndex)dev_).stream();
    void* s = PyLong_AsVoidPtr(args_[i]);
    if (!s && PyErr_Occurred()) throw Refused{};
    return s;
  }
  // Scratch from torch's allocator, in the stream order of the call's stream.
  at::Tensor scratch(size_t bytes, int i) {
    const auto device = c10::Device(c10::kCUDA, (c10::DeviceIndex)dev_);
    const auto make = [&] { return at::empty({(int64_t)bytes}, at::TensorOptions().dtype(at::kByte).device(device)); };
    if (none(i)) return make();
    const c10::cuda::CUDAStreamGuard guard(c10::cuda::getStreamFromExternal((cudaStream_t)stream(i), (c10::DeviceIndex)dev_));
    return make();
  }
  // The entry point's status, without the interpreter's lock.
  template <class F>
  PyObject* run(F f) {
    if (bad) return PyLong_FromLong(MBT_ERR_BAD_ARG);
    int rc;
    Py_BEGIN_ALLOW_THREADS
    rc = f();
    Py_END_ALLOW_THREADS
    return PyLong_FromLong(rc);
  }

 private:
  [[noreturn]] void refuse(const char* name, const char* what) {
    PyErr_Format(PyExc_ValueError, "%s: %s %s", fn_, name, what);
    throw Refused{};
  }
  const at::Tensor& tensor(int i, const char* name) {
    if (!THPVariable_Check(args_[i])) refuse(name, "must be a device tensor");
    return THPVariable_Unpack(args_[i]);
  }
  const at::Tensor& sized(int i, const char* name, int dims) {
    const at::Tensor& t = tensor(i, name);
    if (t.dim() != dims) {
      PyErr_Format(PyExc_ValueError, "%s: %s must be a tensor of %d dimensions", fn_, name, dims);
      throw Refused{};
    }
    for (int64_t n : t.sizes())
      if (n > INT_MAX) refuse(name, "has a dimension beyond 2^31 - 1");
    return t;
  }
  void device(const at::Tensor& t, const char* name) {
    if (!t.is_cuda()) refuse(name, "must be a device tensor");
    if (t.get_device() != dev_) refuse(name, "is on another device than the current one");
  }
  void check(const at::Tensor& t, const char* name, at::ScalarType type) {
    device(t, name);
    if (t.scalar_type() != type) {
      PyErr_Format(PyExc_ValueError, "%s: %s must be of type %s, got %s", fn_, name, c10::toString(type), c10::toString(t.scalar_type()));
      throw Refused{};
    }
    if (!t.is_contiguous()) refuse(name, "must be contiguous");
  }

  const char* fn_;
  PyObject* const* args_;
  int64_t dev_ = -1;
};

// No exception leaves an entry point.
template <class F>
PyObject* guarded(F f) {
  try {
    return f();
  } catch (const Refused&) {
    return nullptr;
  } catch (const std::exception& e) {
    PyErr_SetString(PyExc_RuntimeError, e.what());
    return nullptr;
  }
}
int size(const at::Tensor& t, int dim) { return (int)t.size(dim); }
template <class T>
T* address(const at::Tensor& t) { return static_cast<T*>(t.data_ptr()); }

// ctx_lens, new_lens, bt, num_blocks, free_blocks, free_at, held, cu_seqlens, positions, row_seq, slots, free_next, err, stream
PyObject* kv_extend(PyObject*, PyObject* const* args, Py_ssize_t given) {
  return guarded([&] {
    Call c("op_kv_extend", args, given, 14);
    const at::Tensor& bt = c.lead(2, "bt", at::kInt, 2);
    const at::Tensor& free = c.own(4, "free_blocks", at::kInt, 1);
    const at::Tensor& pos = c.own(8, "positions", at::kInt, 1);
    const int nseq = size(bt, 0), n = size(pos, 0), blocks = c.integer(3);
    auto* ctx = c.dense<int32_t>(0, "ctx_lens", at::kInt, {nseq});
    auto* add = c.dense<int32_t>(1, "new_lens", at::kInt, {nseq});
    auto* at = c.dense<int32_t>(5, "free_at", at::kInt, {1});
    auto* held = c.dense<int32_t>(6, "held", at::kInt, {nseq});
    auto* cu = c.dense<int32_t>(7, "cu_seqlens", at::kInt, {(int64_t)nseq + 1});
    auto* seq = c.dense<int32_t>(9, "row_seq", at::kInt, {n});
    auto* slots = c.dense<int64_t>(10, "slots", at::kLong, {n});
    auto* next = c.dense<int32_t>(11, "free_next", at::kInt, {1});
    uint32_t* err = c.err(12);
    void* stream = c.stream(13);
    return c.run([&] {
      return op_kv_extend(nseq, ctx, add, address<int32_t>(bt), size(bt, 1), blocks, address<int32_t>(free), size(free, 0), at, n,
                          held, cu, address<int32_t>(pos), seq, slots, next, err, stream);
    });
  });
}

// positions, bt, kpool, nkv, d, kv_dtype, num_blocks, bounds, scales, row_seq, err, stream
PyObject* key_bounds(PyObject*, PyObject* const* args, Py_ssize_t given) {
  return guarded([&] {
    Call c("op_key_bounds", args, given, 12);
    const at::Tensor& pos = c.lead(0, "positions", at::kInt, 1);
    const at::Tensor& bt = c.own(1, "bt", at::kInt, 2);
    const int n = size(pos, 0), nseq = size(bt, 0), nkv = c.integer(3), d = c.integer(4), kv = c.integer(5), blocks = c.integer(6);
    const void* k = c.pool(2, "kpool", nkv, d, blocks, kv);
    if (c.bad) return PyLong_FromLong(MBT_ERR_BAD_ARG);
    auto* codes = c.dense<int8_t>(7, "bounds", at::kChar, {(int64_t)blocks + 1, nkv, 2, d});
    auto* scales = c.dense<float>(8, "scales", at::kFloat, {(int64_t)blocks + 1, nkv});
    const int32_t* seq = c.rows(9, n, nseq);
    uint32_t* err = c.err(10);
    void* stream = c.stream(11);
    return c.run([&] {
      return op_key_bounds(n, address<int32_t>(pos), seq, nseq, address<int32_t>(bt), size(bt, 1), nkv, d, k, kv, blocks, codes,
                           scales, err, stream);
    });
  });
}

// q, nkv, bounds, scales, positions, bt, num_blocks, keep_first, keep_last, sel, row_seq, scratch, err, stream
PyObject* block_select(PyObject*, PyObject* const* args, Py_ssize_t given) {
  return guarded([&] {
    Call c("op_block_select", args, given, 14);
    const at::Tensor& q = c.lead(0, "q", at::kFloat, 3);
    const at::Tensor& bt = c.own(5, "bt", at::kInt, 2);
    const at::Tensor& sel = c.own(9, "sel", at::kInt, 3);
    const int n = size(q, 0), nq = size(q, 1), d = size(q, 2), nseq = size(bt, 0), k = size(sel, 2);
    const int nkv = c.integer(1), blocks = c.integer(6), first = c.integer(7), last = c.integer(8);
    if (c.bad) return PyLong_FromLong(MBT_ERR_BAD_ARG);
    c.dense<int32_t>(9, "sel", at::kInt, {n, nkv, k});
    auto* codes = c.dense<int8_t>(2, "bounds", at::kChar, {(int64_t)blocks + 1, nkv, 2, d});
    auto* scales = c.dense<float>(3, "scales", at::kFloat, {(int64_t)blocks + 1, nkv});
    auto* pos = c.dense<int32_t>(4, "positions", at::kInt, {n});
    const int32_t* seq = c.rows(10, n, nseq);
    void* scratch = nullptr;
    size_t bytes = 0;
    at::Tensor made;                                      // lives until the launches are in the stream
    if (!c.none(11)) {
      scratch = c.bytes(11, "scratch", bytes);
    } else if ((bytes = op_block_select_scratch(n, nkv, size(bt, 1), k)) > 0) {
      made = c.scratch(bytes, 13);
      scratch = made.data_ptr();
    }
    uint32_t* err = c.err(12);
    void* stream = c.stream(13);
    return c.run([&] {
      return op_block_select(n, address<float>(q), nq, nkv, d, codes, scales, pos, seq, nseq, address<int32_t>(bt), size(bt, 1),
                             blocks, first, last, k, address<int32_t>(sel), scratch, bytes, err, stream);
    });
  });
}

// q, nkv, kpool, vpool, kv_dtype, k_scale, v_scale, positions, bt, sel, num_blocks, out, row_seq, err, stream
PyObject* block_attention(PyObject*, PyObject* const* args, Py_ssize_t given) {
  return guarded([&] {
    Call c("op_block_attention", args, given, 15);
    const at::Tensor& q = c.lead(0, "q", at::kFloat, 3);
    const at::Tensor& bt = c.own(8, "bt", at::kInt, 2);
    const at::Tensor& sel = c.own(9, "sel", at::kInt, 3);
    const int n = size(q, 0), nq = size(q, 1), d = size(q, 2), nseq = size(bt, 0), k = size(sel, 2);
    const int nkv = c.integer(1), kv = c.integer(4), blocks = c.integer(10);
    const float ks = c.number(5), vs = c.number(6);
    const void* kp = c.pool(2, "kpool", nkv, d, blocks, kv);
    const void* vp = c.pool(3, "vpool", nkv, d, blocks, kv);
    if (c.bad) return PyLong_FromLong(MBT_ERR_BAD_ARG);
    c.dense<int32_t>(9, "sel", at::kInt, {n, nkv, k});
    auto* pos = c.dense<int32_t>(7, "positions", at::kInt, {n});
    auto* out = c.dense<float>(11, "out", at::kFloat, {n, (int64_t)nq * d});
    const int32_t* seq = c.rows(12, n, nseq);
    uint32_t* err = c.err(13);
    void* stream = c.stream(14);
    return c.run([&] {
      return op_block_attention(n, address<float>(q), nq, nkv, d, kp, vp, kv, ks, vs, pos, seq, nseq, address<int32_t>(bt),
                                size(bt, 1), address<int32_t>(sel), k, blocks, out, err, stream);
    });
  });
}

PyMethodDef kMethods[] = {
    {"op_kv_extend", (PyCFunction)(void (*)(void))kv_extend, METH_FASTCALL, nullptr},
    {"op_key_bounds", (PyCFunction)(void (*)(void))key_bounds, METH_FASTCALL, nullptr},
    {"op_block_select", (PyCFunction)(void (*)(void))block_select, METH_FASTCALL, nullptr},
    {"op_block_attention", (PyCFunction)(void (*)(void))block_attention, METH_FASTCALL, nullptr},
    {nullptr, nullptr, 0, nullptr}};
PyModuleDef kModule = {PyModuleDef_HEAD_INIT, "_binding", nullptr, -1, kMethods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__binding() { return PyModule_Create(&kModule); }
