// The binding's ordinary calls, without its Python: arguments are looked at as tensors
// and handed to the C ABI. Each function returns None where a call is not an ordinary
// one (a tensor of another type, shape, layout or device than the call takes, a stream
// given, outputs given except to a step of pages): binding.py then checks it argument by
// argument, says what is wrong or makes the call itself. A status other than INVROPE_OK comes back as a number.
//
// A decoding step's calls take the GPU 3 to 5 us each, and took the host 12 to 28 in
// Python, most of it for attributes of tensors and arguments of ctypes.
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <ATen/ops/empty.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>

#include "kv_pages.h"
#include "latent_attn.h"
#include "rope.h"

namespace {

// The C ABI of the library that binding.py has loaded.
struct {
  decltype(&kv_pages_advance) pages_advance;
  decltype(&kv_idx_local_to_slots) idx_local_to_slots;
  decltype(&rope_apply) rope;
  decltype(&kv_latent_row_bytes) row_bytes;
  decltype(&kv_latent_write) write;
  decltype(&kv_latent_read) read;
  decltype(&invrope_latent_workspace_bytes) workspace_bytes;
  decltype(&latent_attn_decode) decode;
  decltype(&latent_attn_sparse) sparse;
} abi;

PyObject* not_ordinary() {
  PyErr_Clear();
  Py_RETURN_NONE;
}

// A contiguous CUDA tensor of this type, with this many axes, on device `index` (-1: any).
const at::Tensor* tensor(PyObject* o, at::ScalarType type, int64_t ndim, int index) {
  if (!THPVariable_Check(o)) return nullptr;
  const at::Tensor& t = THPVariable_Unpack(o);
  if (!t.is_cuda() || t.scalar_type() != type || t.dim() != ndim || !t.is_contiguous()) return nullptr;
  if (index >= 0 && t.get_device() != index) return nullptr;
  return &t;
}

bool current(const at::Tensor* t) { return t->get_device() == c10::cuda::current_device(); }

CUstream_st* stream_of(int index) {
  return reinterpret_cast<CUstream_st*>(c10::cuda::getCurrentCUDAStream(static_cast<c10::DeviceIndex>(index)).stream());
}

bool number(PyObject* o, int64_t* v) {
  if (!PyLong_Check(o)) return false;
  *v = PyLong_AsLongLong(o);
  return !(*v == -1 && PyErr_Occurred());
}
bool small(PyObject* o, int* v) {
  int64_t wide;
  if (!number(o, &wide) || wide < -0x7FFFFFFF || wide > 0x7FFFFFFF) return false;
  *v = static_cast<int>(wide);
  return true;
}
bool real(PyObject* o, double* v) {
  *v = PyFloat_AsDouble(o);
  return !(*v == -1.0 && PyErr_Occurred());
}

template <typename T>
T* data(const at::Tensor& t) {
  return static_cast<T*>(t.data_ptr());
}
at::Tensor ints(const at::Tensor& like, at::IntArrayRef shape) { return at::empty(shape, like.options().dtype(at::kInt)); }

// `size` entries from `offset` on of a vector, which they keep alive.
at::Tensor part(const at::Tensor& all, int64_t offset, int64_t size) {
  at::Tensor t = at::detail::make_tensor<c10::TensorImpl>(c10::TensorImpl::VIEW, c10::Storage(all.storage()),
                                                          all.key_set(), all.dtype());
  t.unsafeGetTensorImpl()->set_storage_offset(offset);
  t.unsafeGetTensorImpl()->set_sizes_contiguous({size});
  return t;
}

// The C ABI's part of a call, without the interpreter's lock: a launch may wait for room
// in the driver's queue.
template <typename F>
int unlocked(F call) {
  PyThreadState* state = PyEval_SaveThread();
  const int status = call();
  PyEval_RestoreThread(state);
  return status;
}

// What a call gives: `result` (a new reference), or the status that it was refused with.
template <typename F>
PyObject* done(int status, F result) {
  return status == INVROPE_OK ? result() : PyLong_FromLong(status);
}

// C++ exceptions become Python's, as torch's own calls have them: an allocation that fails
// is torch.OutOfMemoryError.
template <typename F>
PyObject* guarded(F f) {
  HANDLE_TH_ERRORS
  return f();
  END_HANDLE_TH_ERRORS
}

// (state, page_table, queue, new_tokens, page_size, max_tokens, state_out or None, a tuple of outputs or None)
PyObject* pages_advance(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    int page_size;
    int64_t room;
    if (n != 8 || !small(a[4], &page_size) || !number(a[5], &room) || room < 0 || room > 0x7FFFFFFF) return not_ordinary();
    const at::Tensor* state = tensor(a[0], at::kInt, 1, -1);
    if (!state || !current(state)) return not_ordinary();
    const int index = state->get_device();
    const at::Tensor *table = tensor(a[1], at::kInt, 2, index), *queue = tensor(a[2], at::kInt, 1, index),
                     *asked = tensor(a[3], at::kInt, 1, index),
                     *out = a[6] == Py_None ? state : tensor(a[6], at::kInt, 1, index);
    if (!table || !queue || !asked || !out) return not_ordinary();
    const int64_t b = table->size(0);
    if (state->size(0) != b + 2 || out->size(0) != b + 2 || asked->size(0) != b) return not_ordinary();
    at::Tensor got[5];
    if (a[7] == Py_None) {
      // (one allocation: five took 4 us)
      const at::Tensor all = ints(*state, {3 * room + 2 * b + 1});
      int64_t offset = 0, k = 0;
      for (const int64_t size : {room, room, room, b + 1, b}) {
        got[k++] = part(all, offset, size);
        offset += size;
      }
    } else {
      if (!PyTuple_Check(a[7]) || PyTuple_GET_SIZE(a[7]) != 5) return not_ordinary();
      int64_t k = 0;
      for (const int64_t size : {room, room, room, b + 1, b}) {
        const at::Tensor* t = tensor(PyTuple_GET_ITEM(a[7], k), at::kInt, 1, index);
        if (!t || t->size(0) != size) return not_ordinary();
        got[k++] = *t;
      }
    }
    CUstream_st* stream = stream_of(index);
    const int st = unlocked([&] { return abi.pages_advance(data<int32_t>(*state), data<int32_t>(*out), data<int32_t>(*table), data<int32_t>(*queue),
                                     data<int32_t>(*asked), data<int32_t>(got[0]), data<int32_t>(got[1]),
                                     data<int32_t>(got[2]), data<int32_t>(got[3]), data<int32_t>(got[4]), b, table->size(1),
                                     queue->size(0), page_size, room, stream); });
    return done(st, [&] {
      if (a[7] != Py_None) return Py_NewRef(a[7]);
      PyObject* tuple = PyTuple_New(5);
      for (int k = 0; tuple && k < 5; ++k) PyTuple_SET_ITEM(tuple, k, THPVariable_Wrap(got[k]));
      return tuple;
    });
  });
}

// (idx, page_table, lens, page_size, num_pages, sq, seq or None)
PyObject* idx_local_to_slots(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    int page_size;
    int64_t pages, sq;
    if (n != 7 || !small(a[3], &page_size) || !number(a[4], &pages) || !number(a[5], &sq)) return not_ordinary();
    const at::Tensor* idx = tensor(a[0], at::kInt, 2, -1);
    if (!idx || !current(idx)) return not_ordinary();
    const int index = idx->get_device();
    const at::Tensor *table = tensor(a[1], at::kInt, 2, index), *lens = tensor(a[2], at::kInt, 1, index),
                     *seq = a[6] == Py_None ? nullptr : tensor(a[6], at::kInt, 1, index);
    if (!table || !lens || (a[6] != Py_None && !seq) || lens->size(0) != table->size(0) ||
        (seq && seq->size(0) != idx->size(0)))
      return not_ordinary();
    const at::Tensor out = ints(*idx, idx->sizes());
    CUstream_st* stream = stream_of(index);
    const int st = unlocked([&] { return abi.idx_local_to_slots(data<int32_t>(*idx), data<int32_t>(*table), data<int32_t>(*lens),
                                          seq ? data<int32_t>(*seq) : nullptr, data<int32_t>(out), idx->size(0), idx->size(1),
                                          sq, table->size(0), table->size(1), pages, page_size, stream); });
    return done(st, [&] { return THPVariable_Wrap(out); });
  });
}

// (x or a list of them, freqs, positions or None, pos0, offset or None, amplitude, interleaved, inverse)
PyObject* rope(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    int64_t pos0, offset = 0;
    double amplitude;
    if (n != 8 || !number(a[3], &pos0) || (a[4] != Py_None && !number(a[4], &offset)) || !real(a[5], &amplitude))
      return not_ordinary();
    const int inter = PyObject_IsTrue(a[6]), inverse = PyObject_IsTrue(a[7]);
    if (inter < 0 || inverse < 0 || !THPVariable_Check(a[1])) return not_ordinary();
    const at::Tensor& freqs = THPVariable_Unpack(a[1]);
    if (!freqs.device().is_cpu() || freqs.scalar_type() != at::kDouble || freqs.dim() != 1 || !freqs.is_contiguous())
      return not_ordinary();
    const int64_t pe = 2 * freqs.size(0);
    const bool many = PyList_Check(a[0]) || PyTuple_Check(a[0]);
    const Py_ssize_t count = many ? PySequence_Fast_GET_SIZE(a[0]) : 1;
    if (count < 1 || count > ROPE_MAX_TENSORS || pe > 0x7FFFFFFF) return not_ordinary();
    RopeTensor list[ROPE_MAX_TENSORS];
    at::Tensor outs[ROPE_MAX_TENSORS];
    int64_t rows = 0;
    int index = -1, type = -1;
    for (Py_ssize_t k = 0; k < count; ++k) {
      PyObject* o = many ? PySequence_Fast_GET_ITEM(a[0], k) : a[0];
      if (!THPVariable_Check(o)) return not_ordinary();
      const at::Tensor& x = THPVariable_Unpack(o);
      const int64_t ndim = x.dim();
      if (!x.is_cuda() || ndim < 2 || ndim > 3 || (x.size(-1) > 1 && x.stride(-1) != 1)) return not_ordinary();
      const auto scalar = x.scalar_type();
      const int is = scalar == at::kBFloat16 ? ROPE_BF16 : scalar == at::kHalf ? ROPE_FP16 : scalar == at::kFloat ? ROPE_FP32 : -1;
      if (k == 0) {
        index = x.get_device();
        type = is;
        rows = x.size(0);
        if (is < 0 || !current(&x)) return not_ordinary();
      }
      if (is != type || x.get_device() != index || x.size(0) != rows) return not_ordinary();
      outs[k] = at::empty(x.sizes(), x.options().memory_format(at::MemoryFormat::Contiguous));
      RopeTensor& t = list[k];
      t.x = x.data_ptr();
      t.out = outs[k].data_ptr();
      t.heads = ndim == 3 ? x.size(1) : 1;
      t.d = x.size(-1);
      t.offset = a[4] == Py_None ? t.d - pe : offset;
      t.x_row = x.stride(0);
      t.x_head = ndim == 3 ? x.stride(1) : 0;
      t.out_row = outs[k].stride(0);
      t.out_head = ndim == 3 ? outs[k].stride(1) : 0;
    }
    const at::Tensor* positions = a[2] == Py_None ? nullptr : tensor(a[2], at::kInt, 1, index);
    if (a[2] != Py_None && (!positions || positions->size(0) != rows)) return not_ordinary();
    CUstream_st* stream = stream_of(index);
    const int st = unlocked([&] { return abi.rope(list, static_cast<int>(count), data<double>(freqs), positions ? data<int32_t>(*positions) : nullptr,
                            pos0, rows, static_cast<int>(pe), amplitude, type, inter, inverse, stream); });
    return done(st, [&]() -> PyObject* {
      if (!many) return THPVariable_Wrap(outs[0]);
      PyObject* all = PyList_New(count);
      for (Py_ssize_t k = 0; all && k < count; ++k) PyList_SET_ITEM(all, k, THPVariable_Wrap(outs[k]));
      return all;
    });
  });
}

// A cache's format by its type and width, -1 where it has none, or another than `said` (a
// number or None) or than the tensor carries (binding.py's kv_latent_empty).
int format_of(PyObject* o, const at::Tensor& cache, int nope, int pe, PyObject* said) {
  if (!cache.is_cuda() || cache.dim() != 3 || !cache.is_contiguous()) return -1;
  const auto width = static_cast<size_t>(cache.size(2));
  if (width == 0) return -1;
  int fmt = -1;
  if (cache.scalar_type() == at::kBFloat16) {
    fmt = 2 * width == abi.row_bytes(nope, pe, KV_LATENT_BF16) ? KV_LATENT_BF16 : -1;
  } else if (cache.scalar_type() == at::kByte) {
    fmt = width == abi.row_bytes(nope, pe, KV_LATENT_E4M3)   ? KV_LATENT_E4M3
          : width == abi.row_bytes(nope, pe, KV_LATENT_E2M1) ? KV_LATENT_E2M1
                                                             : -1;
  }
  int v;
  if (fmt < 0 || (said != Py_None && !(small(said, &v) && v == fmt))) return -1;
  static PyObject* const name = PyUnicode_InternFromString("_kv_latent_fmt");
  PyObject* dict = name ? PyObject_GenericGetDict(o, nullptr) : nullptr;
  PyObject* carried = dict ? PyDict_GetItemWithError(dict, name) : nullptr;  // borrowed
  if (carried && !(small(carried, &v) && v == fmt)) fmt = -1;
  Py_XDECREF(dict);
  return PyErr_Occurred() ? -1 : fmt;
}

// (cache, x, slots, nope, pe, fmt or None)
PyObject* latent_write(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    int nope, pe;
    if (n != 6 || !small(a[3], &nope) || !small(a[4], &pe) || !THPVariable_Check(a[0])) return not_ordinary();
    const at::Tensor& cache = THPVariable_Unpack(a[0]);
    const int fmt = format_of(a[0], cache, nope, pe, a[5]);
    if (fmt < 0 || !current(&cache)) return not_ordinary();
    const int index = cache.get_device();
    const at::Tensor *x = tensor(a[1], at::kBFloat16, 2, index), *slots = tensor(a[2], at::kInt, 1, index);
    if (!x || !slots || x->size(1) != nope + pe || slots->size(0) != x->size(0)) return not_ordinary();
    CUstream_st* stream = stream_of(index);
    const int st = unlocked([&] { return abi.write(x->data_ptr(), data<int32_t>(*slots), cache.data_ptr(), x->size(0), cache.size(0) * cache.size(1),
                             nope, pe, fmt, stream); });
    return done(st, [&] { return Py_NewRef(a[0]); });
  });
}

// (cache, slots, nope, pe, fmt or None)
PyObject* latent_read(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    int nope, pe;
    if (n != 5 || !small(a[2], &nope) || !small(a[3], &pe) || !THPVariable_Check(a[0])) return not_ordinary();
    const at::Tensor& cache = THPVariable_Unpack(a[0]);
    const int fmt = format_of(a[0], cache, nope, pe, a[4]);
    if (fmt < 0 || !current(&cache)) return not_ordinary();
    const int index = cache.get_device();
    const at::Tensor* slots = tensor(a[1], at::kInt, 1, index);
    if (!slots) return not_ordinary();
    const at::Tensor out = at::empty({slots->size(0), nope + pe}, cache.options().dtype(at::kBFloat16));
    CUstream_st* stream = stream_of(index);
    const int st = unlocked([&] { return abi.read(cache.data_ptr(), data<int32_t>(*slots), out.data_ptr(), slots->size(0),
                            cache.size(0) * cache.size(1), nope, pe, fmt, stream); });
    return done(st, [&] { return THPVariable_Wrap(out); });
  });
}

// (q, cache, page_table or idx, lens or None, nope, pe, scale or None, fmt or None)
PyObject* attn(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    int nope, pe;
    double scale = 0.0;
    if (n != 8 || !small(a[4], &nope) || !small(a[5], &pe) || (a[6] != Py_None && !real(a[6], &scale)) ||
        !THPVariable_Check(a[1]))
      return not_ordinary();
    const at::Tensor& cache = THPVariable_Unpack(a[1]);
    const int fmt = format_of(a[1], cache, nope, pe, a[7]);
    if (fmt < 0 || !current(&cache)) return not_ordinary();
    const int index = cache.get_device();
    const at::Tensor *q = tensor(a[0], at::kBFloat16, 3, index), *table = tensor(a[2], at::kInt, 2, index),
                     *lens = a[3] == Py_None ? nullptr : tensor(a[3], at::kInt, 1, index);
    if (!q || !table || (a[3] != Py_None && !lens)) return not_ordinary();
    const int64_t rows = q->size(0), nh = q->size(1), d = q->size(2), pages = cache.size(0), page = cache.size(1);
    if (d != nope + pe || table->size(0) != rows || (lens && lens->size(0) != rows) || nh > 0x7FFFFFFF || page > 0x7FFFFFFF)
      return not_ordinary();
    if (a[6] == Py_None) scale = std::pow(static_cast<double>(d), -0.5);
    const int64_t most = lens ? table->size(1) * page : table->size(1);
    const at::Tensor O = at::empty(q->sizes(), q->options()), lse = at::empty({rows, nh}, q->options().dtype(at::kFloat));
    const size_t bytes = abi.workspace_bytes(rows, static_cast<int>(nh), most, nope, pe, fmt);
    at::Tensor ws;
    if (bytes > 0) ws = at::empty({static_cast<int64_t>(bytes)}, q->options().dtype(at::kByte));
    void* at_ws = bytes > 0 ? ws.data_ptr() : nullptr;
    CUstream_st* stream = stream_of(index);
    const int heads = static_cast<int>(nh), size = static_cast<int>(page);
    const int st = unlocked([&] {
      return lens ? abi.decode(q->data_ptr(), cache.data_ptr(), data<int32_t>(*table), data<int32_t>(*lens), O.data_ptr(),
                               data<float>(lse), at_ws, bytes, rows, heads, nope, pe, fmt, pages, size, table->size(1), scale,
                               stream)
                  : abi.sparse(q->data_ptr(), cache.data_ptr(), data<int32_t>(*table), O.data_ptr(), data<float>(lse), at_ws,
                               bytes, rows, heads, nope, pe, fmt, pages * page, table->size(1), scale, stream);
    });
    return done(st, [&] {
      PyObject* all = PyTuple_New(2);
      if (all) {
        PyTuple_SET_ITEM(all, 0, THPVariable_Wrap(O));
        PyTuple_SET_ITEM(all, 1, THPVariable_Wrap(lse));
      }
      return all;
    });
  });
}

// The addresses of the C ABI's functions, in the order of `abi`.
PyObject* bind(PyObject*, PyObject* const* a, Py_ssize_t n) {
  void** to = reinterpret_cast<void**>(&abi);
  if (n != static_cast<Py_ssize_t>(sizeof(abi) / sizeof(void*))) {
    PyErr_SetString(PyExc_ValueError, "bind: one address for each function");
    return nullptr;
  }
  for (Py_ssize_t k = 0; k < n; ++k) {
    to[k] = PyLong_AsVoidPtr(a[k]);
    if (PyErr_Occurred()) return nullptr;
  }
  Py_RETURN_NONE;
}

#define CALL(name) \
  { #name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(name)), METH_FASTCALL, nullptr }
PyMethodDef methods[] = {CALL(bind),         CALL(pages_advance), CALL(idx_local_to_slots), CALL(rope),
                         CALL(latent_write), CALL(latent_read),   CALL(attn),               {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_calls", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__calls() { return PyModule_Create(&module); }
