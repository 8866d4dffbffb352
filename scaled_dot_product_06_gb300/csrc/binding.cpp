// Native binding of the calls whose kernels are shorter than their checks are in
// Python: slot maps, the norm and rotation of a step's tokens, the attention of a
// decoding step. (Their kernels take 4 to 6 us; checked and marshalled in Python,
// a call took 16 to 20.) The rules and the messages are those of the other bindings: a
// ValueError for operands that a kernel must not see, the entry point's status
// otherwise, which the Python side turns into its error. Tensors that are not given
// are allocated on the current stream, on which the entry point runs.
#include <Python.h>

#include <cmath>
#include <cstdarg>
#include <optional>

#include <ATen/ATen.h>
#include <ATen/cuda/EmptyTensor.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include "../../include/sdpa.h"

namespace {

using at::IntArrayRef;
using at::ScalarType;
using at::Tensor;

[[noreturn]] void refuse(const char* format, ...) {
  va_list args;
  va_start(args, format);
  PyErr_FormatV(PyExc_ValueError, format, args);
  va_end(args);
  throw python_error();
}

const Tensor& tensor(PyObject* o, const char* name) {
  if (!THPVariable_Check(o)) {
    PyErr_Format(PyExc_TypeError, "%s must be a tensor", name);
    throw python_error();
  }
  return THPVariable_Unpack(o);
}
// The tensor, or none.
const Tensor* maybe(PyObject* o, const char* name) { return o == Py_None ? nullptr : &tensor(o, name); }

int64_t whole(PyObject* o) {
  const long long v = PyLong_AsLongLong(o);
  if (v == -1 && PyErr_Occurred()) throw python_error();
  return v;
}
double number(PyObject* o) {
  const double v = PyFloat_AsDouble(o);
  if (v == -1.0 && PyErr_Occurred()) throw python_error();
  return v;
}
bool truth(PyObject* o) {
  const int v = PyObject_IsTrue(o);
  if (v < 0) throw python_error();
  return v != 0;
}

void check_shape(const char* name, const Tensor& t, IntArrayRef shape) {
  if (t.sizes() != shape)
    refuse("%s has shape %s, expected %s", name, c10::str(t.sizes()).c_str(), c10::str(shape).c_str());
}

// Where the operands have to be: the device of the operand `of`.
struct Place {
  int index;
  const char* of;
};

// The pointer of a contiguous tensor of this type and shape.
template <typename T = void>
T* flat(const char* name, const Tensor& t, ScalarType type, const Place& at, IntArrayRef shape) {
  if (t.scalar_type() != type || !t.is_cuda() || t.get_device() != at.index || !t.is_contiguous())
    refuse("%s must be a contiguous torch.%s tensor on the device of %s", name,
           type == at::kInt     ? "int32"
           : type == at::kLong  ? "int64"
           : type == at::kFloat ? "float32"
           : type == at::kHalf  ? "float16"
                                : "bfloat16",
           at.of);
  check_shape(name, t, shape);
  return static_cast<T*>(t.data_ptr());
}

// Memory of the current stream (past the dispatcher: it takes as long as the rest).
Tensor fresh(IntArrayRef shape, ScalarType type, const Tensor& like) {
  return at::detail::empty_cuda(shape, type, like.device(), std::nullopt);
}

// A new tensor, or the given one, checked.
Tensor made(const char* name, PyObject* given, ScalarType type, const Tensor& like, const Place& at, IntArrayRef shape) {
  if (given == Py_None) return fresh(shape, type, like);
  const Tensor& t = tensor(given, name);
  flat(name, t, type, at, shape);
  return t;
}

// The small outputs of a call that are not given, in one allocation: each asks for its
// place first, and is made of the block afterwards. (The slot maps' call, whose kernel takes
// 5 us, took the host 7.4 us with an allocation for each of five, and takes 5.8.)
class Block {
 public:
  explicit Block(const Tensor& like) : like_(like) {}
  // The given tensor, checked, or (undefined so far) a place for one.
  void want(Tensor* out, const char* name, PyObject* given, ScalarType type, const Place& at, IntArrayRef shape) {
    if (given != Py_None) {
      *out = made(name, given, type, like_, at, shape);
      return;
    }
    int64_t n = 1;
    for (const int64_t x : shape) n *= x;
    parts_[count_++] = Part{out, type, bytes_, shape};
    bytes_ += (n * static_cast<int64_t>(c10::elementSize(type)) + 127) / 128 * 128;
  }
  void make() {
    if (count_ == 0) return;
    const Tensor block = fresh({bytes_}, at::kByte, like_);
    for (int i = 0; i < count_; ++i) {
      const Part& p = parts_[i];
      Tensor t = at::detail::make_tensor<c10::TensorImpl>(c10::Storage(block.storage()), block.key_set(),
                                                          c10::scalarTypeToTypeMeta(p.type));
      t.unsafeGetTensorImpl()->set_storage_offset(p.offset / static_cast<int64_t>(c10::elementSize(p.type)));
      t.unsafeGetTensorImpl()->set_sizes_contiguous(p.shape);
      *p.out = std::move(t);
    }
  }

 private:
  struct Part {
    Tensor* out;
    ScalarType type;
    int64_t offset;
    IntArrayRef shape;  // (the caller's)
  };
  const Tensor& like_;
  Part parts_[5];
  int count_ = 0;
  int64_t bytes_ = 0;
};

// Rows of a 4-D tensor with contiguous rows; dimensions 1 and 2 are (row, head), or
// (head, row).
sdpa_rows_t rows(const char* name, const Tensor& t, ScalarType type, const Place& at, IntArrayRef shape, bool head_first) {
  check_shape(name, t, shape);
  if (t.scalar_type() != type)
    refuse("%s has dtype %s, expected %s", name, at::toString(t.scalar_type()), at::toString(type));
  if (!t.is_cuda() || t.get_device() != at.index) refuse("%s must be on the device of q", name);
  if (t.stride(3) != 1 && t.numel() > 0) refuse("%s: the elements of a row must be contiguous", name);
  return sdpa_rows_t{t.data_ptr(), t.stride(0), t.stride(head_first ? 2 : 1), t.stride(head_first ? 1 : 2)};
}
void check_output(const char* name, const Tensor& t) {
  for (int64_t i = 0; i < t.dim(); ++i)
    if (t.stride(i) == 0 && t.size(i) > 1) refuse("%s must not be an expanded tensor", name);
}

sdpa_dtype_t io_type(const Tensor& q, const char* what) {
  if (q.scalar_type() == at::kBFloat16) return SDPA_BF16;
  if (q.scalar_type() == at::kHalf) return SDPA_FP16;
  refuse("%s must be bf16 or fp16", what);
}

// (width, stride) of a block table [b, width] with contiguous rows
struct Table {
  int32_t* ptr;
  int64_t width, stride;
};
Table table_of(const Tensor& t, int64_t b, const Place& at) {
  if (t.dim() != 2 || t.size(0) != b || t.scalar_type() != at::kInt || !t.is_cuda() || t.get_device() != at.index)
    refuse("block_table must be an int32 tensor of %lld rows on the device of %s", static_cast<long long>(b), at.of);
  if (t.size(1) > 1 && t.stride(1) != 1) refuse("block_table: the entries of a row must be contiguous");
  if (b > 1 && t.stride(0) < t.size(1)) refuse("block_table: its rows must not overlap");
  return Table{static_cast<int32_t*>(t.data_ptr()), t.size(1), t.stride(0)};
}

// Calls an entry point with the device current, on its current stream.
template <typename F>
sdpa_status_t call(const Place& at, F entry) {
  const c10::cuda::CUDAGuard device(static_cast<c10::DeviceIndex>(at.index));
  void* stream = c10::cuda::getCurrentCUDAStream(static_cast<c10::DeviceIndex>(at.index)).stream();
  sdpa_status_t st;
  Py_BEGIN_ALLOW_THREADS;
  st = entry(stream);
  Py_END_ALLOW_THREADS;
  return st;
}

void want(Py_ssize_t n, Py_ssize_t have) {
  if (n == have) return;
  PyErr_Format(PyExc_TypeError, "%zd arguments, expected %zd", have, n);
  throw python_error();
}

PyObject* wrap(const Tensor& t) { return THPVariable_Wrap(t); }

// The outputs as a tuple (an undefined tensor: None).
template <size_t N>
PyObject* tuple(const Tensor (&t)[N]) {
  PyObject* out = PyTuple_New(N);
  if (out == nullptr) throw python_error();
  for (size_t i = 0; i < N; ++i) {
    PyObject* o = t[i].defined() ? wrap(t[i]) : Py_NewRef(Py_None);
    if (o == nullptr) {
      Py_DECREF(out);
      throw python_error();
    }
    PyTuple_SET_ITEM(out, static_cast<Py_ssize_t>(i), o);
  }
  return out;
}

// seqlens, new_tokens, block_table, free_pages, free_range, page_size, rows, width, slots, positions, starts,
// seqlens_out, free_range_out
PyObject* page_slots(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  want(13, n);
  const Tensor& lens = tensor(a[0], "seqlens");
  if (!lens.is_cuda()) refuse("seqlens must be a CUDA tensor");
  const bool packed = a[6] != Py_None;
  if (packed == (a[7] != Py_None)) refuse("either rows (packed) or width (padded)");
  const Tensor& ring = tensor(a[3], "free_pages");
  if (lens.dim() != 1 || ring.dim() != 1) refuse("seqlens and free_pages must have one dimension");
  const Place at{lens.get_device(), "seqlens"};
  const int64_t b = lens.size(0), n_pages = ring.size(0), page = whole(a[5]);
  const int64_t row_count = packed ? whole(a[6]) : 0, width = packed ? 0 : whole(a[7]);
  auto* lens_p = flat<int32_t>("seqlens", lens, at::kInt, at, {b});
  auto* new_p = flat<int32_t>("new_tokens", tensor(a[1], "new_tokens"), at::kInt, at, {b});
  auto* ring_p = flat<int32_t>("free_pages", ring, at::kInt, at, {n_pages});
  const Tensor& range = tensor(a[4], "free_range");
  auto* range_p = flat<int64_t>("free_range", range, at::kLong, at, {2});
  const Table table = table_of(tensor(a[2], "block_table"), b, at);
  if (!packed && a[10] != Py_None) refuse("starts are of packed rows");
  if (row_count < 0 || width < 0) refuse("rows and width must not be negative");
  if (row_count > int64_t{1} << 31 || width > int64_t{1} << 31) refuse("rows and width must stay below 2^31");
  const int64_t packed_shape[1] = {row_count}, padded_shape[2] = {b, width};
  const int64_t offsets_shape[1] = {b + 1}, lens_shape[1] = {b}, range_shape[1] = {2};
  const IntArrayRef shape = packed ? IntArrayRef(packed_shape) : IntArrayRef(padded_shape);
  Tensor out[5];
  Block block(lens);
  block.want(&out[0], "slots", a[8], at::kInt, at, shape);
  block.want(&out[1], "positions", a[9], at::kInt, at, shape);
  if (packed) block.want(&out[2], "starts", a[10], at::kInt, at, offsets_shape);
  block.want(&out[3], "seqlens_out", a[11], at::kInt, at, lens_shape);
  block.want(&out[4], "free_range_out", a[12], at::kLong, at, range_shape);
  block.make();
  auto ints = [](const Tensor& t) { return static_cast<int32_t*>(t.data_ptr()); };
  const sdpa_status_t st = call(at, [&](void* stream) {
    return sdpa_page_slots(b, page, table.width, table.stride, n_pages, row_count, width, lens_p, new_p, table.ptr,
                           ring_p, range_p, ints(out[0]), ints(out[1]), packed ? ints(out[2]) : nullptr, ints(out[3]),
                           static_cast<int64_t*>(out[4].data_ptr()), stream);
  });
  return st != SDPA_OK ? PyLong_FromLong(st) : tuple(out);
  END_HANDLE_TH_ERRORS
}

// q, k_pages, v_pages, block_table, seqlens_k, scale, softcap, window_left, out, lse, workspace
PyObject* fwd_paged(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  want(11, n);
  const Tensor &q = tensor(a[0], "q"), &k = tensor(a[1], "k_pages"), &v = tensor(a[2], "v_pages");
  if (q.dim() != 4 || k.dim() != 4 || v.dim() != 4) refuse("q, k_pages and v_pages must have 4 dimensions");
  const sdpa_dtype_t type = io_type(q, "q, k_pages, v_pages");
  if (!q.is_cuda()) refuse("q must be a CUDA tensor");
  const ScalarType dt = q.scalar_type();
  const Place at{q.get_device(), "q"};
  const int64_t b = q.size(0), h = q.size(1), s_q = q.size(2), d_qk = q.size(3);
  const int64_t n_pages = k.size(0), h_kv = k.size(1), page = k.size(2), d_v = v.size(3);
  void* q_p = flat("q", q, dt, at, {b, h, s_q, d_qk});
  const sdpa_rows_t k_rows = rows("k_pages", k, dt, at, {n_pages, h_kv, page, d_qk}, true);
  const sdpa_rows_t v_rows = rows("v_pages", v, dt, at, {n_pages, h_kv, page, d_v}, true);
  auto* lens_p = flat<int32_t>("seqlens_k", tensor(a[4], "seqlens_k"), at::kInt, at, {b});
  const Table table = table_of(tensor(a[3], "block_table"), b, at);
  const double scale = a[5] != Py_None ? number(a[5]) : 1.0 / std::sqrt(static_cast<double>(d_qk));
  const double softcap = a[6] != Py_None ? number(a[6]) : 0.0;
  const int64_t left = a[7] != Py_None ? whole(a[7]) : -1;
  Tensor out[2];
  out[0] = made("out", a[8], dt, q, at, {b, h, s_q, d_v});
  out[1] = made("lse", a[9], at::kFloat, q, at, {b, h, s_q});
  Tensor scratch;
  size_t bytes;
  if (const Tensor* w = maybe(a[10], "workspace")) {
    if (!w->is_cuda() || w->get_device() != at.index || !w->is_contiguous())
      refuse("workspace must be a contiguous tensor on the device of q");
    scratch = *w;
    bytes = w->nbytes();
  } else {
    bytes = sdpa_fwd_paged_workspace_size(h, h_kv, s_q, d_qk, d_v, page, table.width);
    if (bytes > 0) scratch = fresh({static_cast<int64_t>(bytes)}, at::kByte, q);
  }
  const sdpa_status_t st = call(at, [&](void* stream) {
    return sdpa_fwd_paged(b, h, h_kv, s_q, d_qk, d_v, static_cast<float>(scale), static_cast<float>(softcap), left, type,
                          q_p, &k_rows, &v_rows, n_pages, page, table.ptr, table.width, table.stride, lens_p,
                          out[0].data_ptr(), static_cast<float*>(out[1].data_ptr()),
                          scratch.defined() ? scratch.data_ptr() : nullptr, bytes, stream);
  });
  return st != SDPA_OK ? PyLong_FromLong(st) : tuple(out);
  END_HANDLE_TH_ERRORS
}

// q, k, cos, sin, v, positions, q_weight, k_weight, eps, interleaved, kv_rows, kv_slots, q_out, k_out, v_out
PyObject* qk_norm_rope(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  want(15, n);
  const Tensor &q = tensor(a[0], "q"), &k = tensor(a[1], "k");
  const Tensor* v = maybe(a[4], "v");
  if (q.dim() != 4 || k.dim() != 4 || (v != nullptr && v->dim() != 4)) refuse("q, k and v must have 4 dimensions");
  const sdpa_dtype_t type = io_type(q, "q, k, v");
  if (!q.is_cuda()) refuse("q must be a CUDA tensor");
  const ScalarType dt = q.scalar_type();
  const Place at{q.get_device(), "q"};
  const int64_t b = q.size(0), s = q.size(1), h = q.size(2), d = q.size(3), h_kv = k.size(2);
  const int64_t d_v = v != nullptr ? v->size(3) : d;
  const sdpa_rows_t q_in = rows("q", q, dt, at, {b, s, h, d}, false), k_in = rows("k", k, dt, at, {b, s, h_kv, d}, false);
  sdpa_rows_t v_in{}, v_to{};
  if (v != nullptr) v_in = rows("v", *v, dt, at, {b, s, h_kv, d_v}, false);
  const Tensor *q_out = maybe(a[12], "q_out"), *k_out = maybe(a[13], "k_out"), *v_out = maybe(a[14], "v_out");
  if (v == nullptr && v_out != nullptr) refuse("v_out without v");
  // the table
  const Tensor *cos = maybe(a[2], "cos"), *sin = maybe(a[3], "sin"), *positions = maybe(a[5], "positions");
  int64_t rot = 0, n_pos = 0;
  const float *cos_p = nullptr, *sin_p = nullptr;
  const int32_t* pos_p = nullptr;
  if ((cos == nullptr) != (sin == nullptr)) refuse("cos and sin go together");
  if (cos != nullptr) {
    if (cos->dim() != 2) refuse("cos and sin must have shape (n_pos, rot / 2)");
    n_pos = cos->size(0);
    rot = 2 * cos->size(1);
    cos_p = flat<float>("cos", *cos, at::kFloat, at, cos->sizes());
    sin_p = flat<float>("sin", *sin, at::kFloat, at, cos->sizes());
    if (positions != nullptr) pos_p = flat<int32_t>("positions", *positions, at::kInt, at, {b, s});
  }
  // the weights: both fp32, or both of q's type
  const Tensor *qw = maybe(a[6], "q_weight"), *kw = maybe(a[7], "k_weight");
  const void *qw_p = nullptr, *kw_p = nullptr;
  bool fp32 = false;
  if (qw != nullptr || kw != nullptr) {
    const ScalarType wt = (qw != nullptr ? qw : kw)->scalar_type();
    fp32 = wt == at::kFloat;
    if (!fp32 && wt != dt) refuse("the weights must both be fp32 or both have q's dtype");
    if (qw != nullptr) qw_p = flat("q_weight", *qw, wt, at, {d});
    if (kw != nullptr) kw_p = flat("k_weight", *kw, wt, at, {d});
  }
  // where the keys and values go
  const Tensor *kv_rows = maybe(a[10], "kv_rows"), *kv_slots = maybe(a[11], "kv_slots");
  const int32_t* to_p = nullptr;
  int64_t outer = b, cache = s;
  if (kv_rows != nullptr && kv_slots != nullptr) refuse("either kv_rows or kv_slots");
  if (kv_slots != nullptr) {
    to_p = flat<int32_t>("kv_slots", *kv_slots, at::kInt, at, {b, s});
    if (k_out == nullptr || (v != nullptr && v_out == nullptr)) refuse("kv_slots needs the pages as k_out (and v_out)");
    if (k_out->dim() != 4) refuse("k_out must have 4 dimensions");
    outer = k_out->size(0);
    cache = k_out->size(2);
  } else if (kv_rows != nullptr) {
    to_p = flat<int32_t>("kv_rows", *kv_rows, at::kInt, at, {b});
    if (k_out == nullptr || (v != nullptr && v_out == nullptr)) refuse("kv_rows needs the caches as k_out (and v_out)");
    cache = k_out->dim() == 4 ? k_out->size(2) : -1;
  }
  Tensor out[3];
  auto target = [&](const char* name, const Tensor* given, IntArrayRef shape, Tensor* t) {
    if (given == nullptr) {
      *t = fresh(shape, dt, q);
    } else {
      *t = *given;
    }
    const sdpa_rows_t r = rows(name, *t, dt, at, shape, true);
    if (given != nullptr) check_output(name, *t);
    return r;
  };
  const sdpa_rows_t q_to = target("q_out", q_out, {b, h, s, d}, &out[0]);
  const sdpa_rows_t k_to = target("k_out", k_out, {outer, h_kv, cache, d}, &out[1]);
  if (v != nullptr) v_to = target("v_out", v_out, {outer, h_kv, cache, d_v}, &out[2]);
  const float eps = static_cast<float>(number(a[8]));
  const int inter = truth(a[9]) ? 1 : 0;
  const sdpa_rows_t *vi = v != nullptr ? &v_in : nullptr, *vo = v != nullptr ? &v_to : nullptr;
  const sdpa_status_t st = call(at, [&](void* stream) {
    if (kv_slots != nullptr)
      return sdpa_qk_norm_rope_paged(b, s, h, h_kv, d, d_v, type, &q_in, &k_in, vi, &q_to, &k_to, vo, rot, inter, cos_p,
                                     sin_p, n_pos, pos_p, qw_p, kw_p, fp32, eps, to_p, outer, cache, stream);
    return sdpa_qk_norm_rope(b, s, h, h_kv, d, d_v, type, &q_in, &k_in, vi, &q_to, &k_to, vo, rot, inter, cos_p, sin_p,
                             n_pos, pos_p, qw_p, kw_p, fp32, eps, to_p, cache, stream);
  });
  return st != SDPA_OK ? PyLong_FromLong(st) : tuple(out);
  END_HANDLE_TH_ERRORS
}

template <PyObject* (*F)(PyObject*, PyObject* const*, Py_ssize_t)>
PyMethodDef method(const char* name) {
  return {name, reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(F)), METH_FASTCALL, nullptr};
}
PyMethodDef methods[] = {method<page_slots>("page_slots"), method<fwd_paged>("fwd_paged"),
                         method<qk_norm_rope>("qk_norm_rope"), {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_binding", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

// torch_version: the torch that this was compiled against, which the Python side compares
// with the one that it finds.
PyMODINIT_FUNC PyInit__binding() {
  PyObject* m = PyModule_Create(&module);
  if (m != nullptr && PyModule_AddStringConstant(m, "torch_version", SDPA_TORCH_VERSION) < 0) Py_CLEAR(m);
  return m;
}
