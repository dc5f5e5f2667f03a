// The row operators' and the page pool's calls from Python: argument checks, outputs and scratch from PyTorch's
// allocator, and the C entry point on the current stream, in one native call. A call on a few tokens lasts as long as its
// host side does: for three outputs of layer norm, creating them, marshalling twelve arguments and launching took 14 us from
// Python (ctypes) and takes about half here.
//
// CPython's C API and PyTorch's tensors; nothing is computed here. The entry points are those of the library that the
// process has loaded already (bind), so the two never disagree.
#include <Python.h>
#include <dlfcn.h>

#include <climits>
#include <cmath>
#include <optional>
#include <string>

#include <ATen/core/Tensor.h>
#include <ATen/TracerMode.h>
#include <ATen/core/grad_mode.h>
#include <ATen/cuda/EmptyTensor.h>
#include <c10/core/AutogradState.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include "../../include/jattn.h"

namespace {

using at::Tensor;

struct Library {
  decltype(&::jattn_layer_norm) layer_norm;
  decltype(&::jattn_layer_norm_bwd) layer_norm_bwd;
  decltype(&::jattn_layer_norm_bwd_scratch_size) layer_norm_bwd_scratch_size;
  decltype(&::jattn_rotary) rotary;
  decltype(&::jattn_rotary_tables) rotary_tables;
  decltype(&::jattn_page_scratch_size) page_scratch_size;
  decltype(&::jattn_page_assign) page_assign;
  decltype(&::jattn_page_release) page_release;
} lib{};
PyObject* g_check = nullptr;   // check(code, where) raises the library's error
PyObject* g_status = nullptr;  // status(device index): address of the device's status word
constexpr int kDevices = 64;
void* g_status_word[kDevices] = {};

// A Python error that is set already.
struct Raised {};

const Tensor& tensor(PyObject* o, const char* name) {
  TORCH_CHECK_TYPE(THPVariable_Check(o), name, " must be a tensor");
  return THPVariable_Unpack(o);
}
// None stands for no tensor.
const Tensor* optional(PyObject* o, const char* name) { return o == Py_None ? nullptr : &tensor(o, name); }
void* address(const Tensor* t) { return t ? t->data_ptr() : nullptr; }
int64_t* longs(const Tensor* t) { return t ? static_cast<int64_t*>(t->data_ptr()) : nullptr; }

int64_t integer(PyObject* o) {
  const long long v = PyLong_AsLongLong(o);
  if (v == -1 && PyErr_Occurred()) throw Raised{};
  return v;
}
bool truth(PyObject* o) {
  const int v = PyObject_IsTrue(o);
  if (v < 0) throw Raised{};
  return v == 1;
}
double number(PyObject* o) {
  const double v = PyFloat_AsDouble(o);
  if (v == -1.0 && PyErr_Occurred()) throw Raised{};
  return v;
}

// The GIL is given back while memory is allocated and the kernels are launched, as in PyTorch's own calls.
class Unlocked {
  PyThreadState* state_ = PyEval_SaveThread();

 public:
  ~Unlocked() { PyEval_RestoreThread(state_); }
};

// Where a call runs: the tensors' device, made current, its current stream and its status word.
struct Place {
  c10::cuda::OptionalCUDAGuard guard;
  void* status;
  void* stream;

  explicit Place(int index) {
    TORCH_CHECK_VALUE(index >= 0 && index < kDevices, "device index out of range");
    if (c10::cuda::current_device() != index) guard.set_index(index);
    if (g_status_word[index] == nullptr) {
      PyObject* a = PyObject_CallFunction(g_status, "i", index);
      if (a == nullptr) throw Raised{};
      g_status_word[index] = PyLong_AsVoidPtr(a);
      Py_DECREF(a);
      if (PyErr_Occurred()) throw Raised{};
    }
    status = g_status_word[index];
    stream = c10::cuda::getCurrentCUDAStream(static_cast<c10::DeviceIndex>(index)).stream();
  }
};
constexpr size_t kStatusBytes = 256;

void finish(int rc, const char* where) {
  if (rc == 0) return;
  PyObject* r = PyObject_CallFunction(g_check, "is", rc, where);
  Py_XDECREF(r);
  throw Raised{};
}

int type_of(const Tensor& t) {
  switch (t.scalar_type()) {
    case at::kFloat: return JATTN_F32;
    case at::kBFloat16: return JATTN_BF16;
    case at::kHalf: return JATTN_F16;
    default: return -1;
  }
}

// From PyTorch's allocator without its dispatcher.
Tensor empty(at::IntArrayRef sizes, c10::Device device, at::ScalarType type) {
  return Tensor(at::detail::empty_cuda(sizes, type, device, std::nullopt));
}
Tensor empty(at::IntArrayRef sizes, const Tensor& like, at::ScalarType type) { return empty(sizes, like.device(), type); }

// Two fp32 tensors of a shape that are used together, from one allocation (each starts at 256 bytes).
struct Pair {
  Tensor first, second;
  Pair() = default;
  Pair(at::IntArrayRef sizes, c10::Device device) {
    const int64_t n = (c10::multiply_integers(sizes) + 63) / 64 * 64;
    const Tensor both = empty({2 * n}, device, at::kFloat);
    first = part(both, sizes, 0);
    second = part(both, sizes, n);
  }

 private:
  static Tensor part(const Tensor& both, at::IntArrayRef sizes, int64_t offset) {
    Tensor t = at::detail::make_tensor<c10::TensorImpl>(c10::Storage(both.storage()), both.key_set(), both.dtype());
    t.unsafeGetTensorImpl()->set_sizes_contiguous(sizes);
    t.unsafeGetTensorImpl()->set_storage_offset(offset);
    return t;
  }
};

struct Strides {
  int64_t row, head;
};
// Of x [rows, N] or [rows, heads, N]; those of dimensions of one entry as in a dense tensor.
Strides strides_of(const Tensor& x, const char* name) {
  const int64_t dims = x.dim();
  TORCH_CHECK_VALUE(x.layout() == at::kStrided && x.is_cuda() && type_of(x) >= 0 && (dims == 2 || dims == 3), name,
                    " must be a CUDA tensor [rows, N] or [rows, heads, N] of bf16, fp16 or fp32");
  const int64_t n = x.size(-1), heads = dims == 3 ? x.size(1) : 1;
  TORCH_CHECK_VALUE(n <= 1 || x.stride(-1) == 1, "the values of a row of ", name, " must be neighbours in memory");
  const int64_t head = dims == 3 && heads > 1 ? x.stride(1) : n;
  return Strides{x.size(0) > 1 ? x.stride(0) : heads * head, head};
}

void check_like(const Tensor& t, const Tensor& x, const char* name) {
  TORCH_CHECK_VALUE(t.scalar_type() == x.scalar_type() && t.sizes() == x.sizes() && t.device() == x.device(), name,
                    " must have x's shape, type and device");
}

void check_out(const Tensor& out, const Tensor& x) {
  check_like(out, x, "out");
  TORCH_CHECK_VALUE(!(out.requires_grad() && at::GradMode::is_enabled()),
                    "outputs are written without a gradient: pass tensors that need none");
}

// A tensor that a call has written: autograd refuses a backward pass that needs what it held before.
void written(const Tensor& out) {
  if (!out.is_inference()) out.unsafeGetTensorImpl()->bump_version();
}

// Whether autograd follows t: a gradient is asked for, or a tangent (forward mode, in any grad mode) comes with it.
bool followed(const Tensor& t) {
  return (at::GradMode::is_enabled() && t.requires_grad()) ||
         (c10::AutogradState::get_tls_state().get_fw_grad_mode() && t._fw_grad(0).defined());
}

void check_index(const Tensor& t, c10::Device device, const char* name) {
  TORCH_CHECK_VALUE(t.scalar_type() == at::kLong && t.dim() == 1 && t.device() == device && t.is_contiguous(), name,
                    " must be a contiguous int64 tensor of one dimension on the other tensors' device");
}

void check_weight(const Tensor& x, const Tensor& w, const char* name) {
  TORCH_CHECK_VALUE(w.dim() == 1 && w.size(0) == x.size(-1) && w.device() == x.device() && w.is_contiguous() &&
                        (w.scalar_type() == x.scalar_type() || w.scalar_type() == at::kFloat),
                    name, " must be a contiguous tensor [N] of x's type or fp32 on x's device");
}

void check_stats(const Tensor& x, const Tensor& t, const char* name) {
  TORCH_CHECK_VALUE(t.scalar_type() == at::kFloat && t.sizes() == x.sizes().slice(0, x.dim() - 1) &&
                        t.device() == x.device() && t.is_contiguous(),
                    name, " must be a contiguous fp32 tensor of x's shape without its last dimension");
}

// Address of the number of rows that are no padding.
const int64_t* live_rows(const Tensor& x, const Tensor* off) {
  if (off == nullptr) return nullptr;
  check_index(*off, x.device(), "off");
  TORCH_CHECK_VALUE(off->numel() >= 1, "off must have at least one entry");
  return longs(off) + off->numel() - 1;
}

jattn_norm_t norm_params(const Tensor& x, const Tensor* weight, const Tensor* out) {
  const Strides xs = strides_of(x, "x");
  jattn_norm_t p{};
  const int64_t heads = x.dim() == 3 ? x.size(1) : 1, n = x.size(-1);
  TORCH_CHECK_VALUE(n >= 1 && n <= 16384 && heads >= 1 && heads <= INT_MAX,
                    "rows must have 1 to 16384 values, and at least one head");
  p.rows = x.size(0);
  p.heads = static_cast<int>(heads);
  p.N = static_cast<int>(n);
  p.type = type_of(x);
  p.weight_type = weight ? type_of(*weight) : p.type;
  p.zero_behind = out == nullptr;
  const Strides ys = out ? strides_of(*out, "out") : Strides{heads * n, n};
  p.x_row_stride = xs.row;
  p.x_head_stride = xs.head;
  p.y_row_stride = ys.row;
  p.y_head_stride = ys.head;
  return p;
}

PyObject* wrap(const Tensor& t) { return THPVariable_Wrap(t); }
PyObject* none() { Py_RETURN_NONE; }
PyObject* given(PyObject* o) {
  Py_INCREF(o);
  return o;
}
PyObject* pack(PyObject* a, PyObject* b) {
  PyObject* t = a && b ? PyTuple_Pack(2, a, b) : nullptr;
  Py_XDECREF(a);
  Py_XDECREF(b);
  return t;
}
PyObject* pack(PyObject* a, PyObject* b, PyObject* c) {
  PyObject* t = a && b && c ? PyTuple_Pack(3, a, b, c) : nullptr;
  Py_XDECREF(a);
  Py_XDECREF(b);
  Py_XDECREF(c);
  return t;
}

// (x, weight, bias, eps, off, out) -> (y, mean, rstd)
PyObject* layer_norm(PyObject* const* a) {
  const Tensor& x = tensor(a[0], "x");
  const Tensor *weight = optional(a[1], "weight"), *bias = optional(a[2], "bias"), *off = optional(a[4], "off");
  const Tensor* out = optional(a[5], "out");
  const double eps = number(a[3]);
  TORCH_CHECK_VALUE(eps > 0.0 && std::isfinite(eps), "eps must be positive and finite");
  jattn_norm_t p = norm_params(x, weight, out);
  p.eps = static_cast<float>(eps);
  p.zero_stats = true;  // the statistics are always this call's own
  if (out) check_out(*out, x);
  if (weight) check_weight(x, *weight, "weight");
  if (bias) {
    TORCH_CHECK_VALUE(weight && bias->scalar_type() == weight->scalar_type(), "a bias needs a weight of its type");
    check_weight(x, *bias, "bias");
  }
  const int64_t* live = live_rows(x, off);
  Place place(x.get_device());
  Tensor y;
  Pair stats;
  int rc;
  {
    Unlocked unlocked;
    if (!out) y = empty(x.sizes(), x, x.scalar_type());
    const auto rows = x.sizes().slice(0, x.dim() - 1);
    stats = Pair(rows, x.device());
    rc = lib.layer_norm(&p, live, x.data_ptr(), address(weight), address(bias), (out ? *out : y).data_ptr(),
                        static_cast<float*>(stats.first.data_ptr()), static_cast<float*>(stats.second.data_ptr()),
                        place.status, kStatusBytes, place.stream);
  }
  finish(rc, "jattn_layer_norm");
  if (out) written(*out);
  return pack(out ? given(a[5]) : wrap(y), wrap(stats.first), wrap(stats.second));
}

// (dy, x, weight, mean, rstd, off, bias, out) -> (dx, dweight, dbias)
PyObject* layer_norm_bwd(PyObject* const* a) {
  const Tensor &dy = tensor(a[0], "dy"), &x = tensor(a[1], "x"), &mean = tensor(a[3], "mean"), &rstd = tensor(a[4], "rstd");
  const Tensor *weight = optional(a[2], "weight"), *off = optional(a[5], "off"), *out = optional(a[7], "out");
  const bool wants_bias = truth(a[6]);
  jattn_norm_t p = norm_params(x, weight, out);
  check_like(dy, x, "dy");
  const Strides ds = strides_of(dy, "dy");
  p.dy_row_stride = ds.row;
  p.dy_head_stride = ds.head;
  if (out) check_out(*out, x);
  if (weight) check_weight(x, *weight, "weight");
  check_stats(x, mean, "mean");
  check_stats(x, rstd, "rstd");
  const int64_t* live = live_rows(x, off);
  Place place(x.get_device());
  Tensor dx, dw, db, scratch;
  int rc = 0;
  {
    Unlocked unlocked;
    if (!out) dx = empty(x.sizes(), x, x.scalar_type());
    size_t bytes = 0;
    if (weight) {
      rc = lib.layer_norm_bwd_scratch_size(&p, &bytes);
      dw = empty(weight->sizes(), x, weight->scalar_type());
      if (wants_bias) db = empty(weight->sizes(), x, weight->scalar_type());
      if (bytes > 0) scratch = empty({static_cast<int64_t>(bytes)}, x, at::kByte);
    }
    if (rc == 0)
      rc = lib.layer_norm_bwd(&p, live, dy.data_ptr(), x.data_ptr(), address(weight),
                              static_cast<const float*>(mean.data_ptr()), static_cast<const float*>(rstd.data_ptr()),
                              (out ? *out : dx).data_ptr(), weight ? dw.data_ptr() : nullptr,
                              weight && wants_bias ? db.data_ptr() : nullptr, bytes > 0 ? scratch.data_ptr() : nullptr, bytes,
                              place.status, kStatusBytes, place.stream);
  }
  finish(rc, "jattn_layer_norm_bwd");
  if (out) written(*out);
  return pack(out ? given(a[7]) : wrap(dx), weight ? wrap(dw) : none(), weight && wants_bias ? wrap(db) : none());
}

// (x, cos, sin) -> whether the rotation of x has to go through its autograd function: autograd follows x, or a trace is recorded.
PyObject* rotary_followed(PyObject* const* a) {
  TORCH_CHECK_VALUE(!followed(tensor(a[1], "cos")) && !followed(tensor(a[2], "sin")),
                    "tables take no gradient: pass detached tensors");
  return PyBool_FromLong(followed(tensor(a[0], "x")) || at::tracer::impl::is_dispatch_enabled());
}

// (x, cos, sin, off, start, layout, inverse, out) -> y
PyObject* rotary(PyObject* const* a) {
  const Tensor &x = tensor(a[0], "x"), &cos = tensor(a[1], "cos"), &sin = tensor(a[2], "sin");
  const Tensor *off = optional(a[3], "off"), *start = optional(a[4], "start"), *out = optional(a[7], "out");
  TORCH_CHECK_VALUE(x.dim() == 3, "x must be [total, H, D]");
  const Strides xs = strides_of(x, "x");
  const int64_t total = x.size(0), heads = x.size(1), D = x.size(2);
  for (const Tensor* t : {&cos, &sin})
    TORCH_CHECK_VALUE(t->scalar_type() == at::kFloat && t->dim() == 2 && t->sizes() == cos.sizes() &&
                          t->device() == x.device() && t->is_contiguous(),
                      "tables must be two contiguous fp32 tensors [rows, R/2] on x's device");
  TORCH_CHECK_VALUE(cos.size(1) >= 1 && cos.size(1) <= D / 2 && D >= 2 && D <= 16384 && heads >= 1 && heads <= INT_MAX,
                    "tables must have 1 to D/2 columns, and x at least one head of 2 to 16384 columns");
  if (off) check_index(*off, x.device(), "off");
  if (start) check_index(*start, x.device(), "start");
  const int64_t B = off ? off->numel() - 1 : total;
  TORCH_CHECK_VALUE((!off || B >= 1) && (!start || start->numel() == B),
                    "start must have an entry per sequence of off, or per row without off");
  if (out) check_out(*out, x);
  jattn_rotary_t p{};
  p.B = B;
  p.total = total;
  p.heads = static_cast<int>(heads);
  p.D = static_cast<int>(D);
  p.half = static_cast<int>(cos.size(1));
  p.type = type_of(x);
  p.layout = static_cast<int>(integer(a[5]));
  p.inverse = truth(a[6]);
  p.zero_behind = out == nullptr;
  p.table_rows = cos.size(0);
  const Strides ys = out ? strides_of(*out, "out") : Strides{heads * D, D};
  p.x_row_stride = xs.row;
  p.x_head_stride = xs.head;
  p.y_row_stride = ys.row;
  p.y_head_stride = ys.head;
  Place place(x.get_device());
  Tensor y;
  int rc;
  {
    Unlocked unlocked;
    if (!out) y = empty(x.sizes(), x, x.scalar_type());
    rc = lib.rotary(&p, longs(off), longs(start), static_cast<const float*>(cos.data_ptr()),
                    static_cast<const float*>(sin.data_ptr()), x.data_ptr(), (out ? *out : y).data_ptr(), place.status,
                    kStatusBytes, place.stream);
  }
  finish(rc, "jattn_rotary");
  if (out) written(*out);
  return out ? given(a[7]) : wrap(y);
}

// (rows, dim, base, scaling, factor, original, beta_fast, beta_slow, first, device index or -1) -> (cos, sin)
PyObject* rotary_tables(PyObject* const* a) {
  const int64_t rows = integer(a[0]), dim = integer(a[1]), first = integer(a[8]);
  int64_t index = integer(a[9]);
  TORCH_CHECK_VALUE(dim >= 2 && dim % 2 == 0 && dim <= 1024, "dim must be even, from 2 to 1024");
  TORCH_CHECK_VALUE(rows >= 0 && first >= 0 && rows <= (int64_t(1) << 31) && first <= (int64_t(1) << 31) - rows,
                    "positions must lie between 0 and 2^31");
  jattn_rotary_tables_t p{};
  p.first = first;
  p.rows = rows;
  p.half = static_cast<int>(dim / 2);
  p.scaling = static_cast<int>(integer(a[3]));
  p.base = number(a[2]);
  p.factor = number(a[4]);
  p.original = number(a[5]);
  p.beta_fast = number(a[6]);
  p.beta_slow = number(a[7]);
  if (index < 0) index = c10::cuda::current_device();
  Place place(static_cast<int>(index));
  const c10::Device device(at::kCUDA, static_cast<c10::DeviceIndex>(index));
  Pair tables;
  int rc;
  {
    Unlocked unlocked;
    tables = Pair({rows, dim / 2}, device);
    rc = lib.rotary_tables(&p, static_cast<float*>(tables.first.data_ptr()), static_cast<float*>(tables.second.data_ptr()),
                           place.stream);
  }
  finish(rc, "jattn_rotary_tables");
  return pack(wrap(tables.first), wrap(tables.second));
}

// What both page calls are given first: free pages, count, page size (checked when the pool was made), page table.
struct PoolCall {
  jattn_page_pool_t pool{};
  const Tensor& free;
  const Tensor& table;
  int64_t B, max_pages;

  explicit PoolCall(PyObject* const* a) : free(tensor(a[0], "free_pages")), table(tensor(a[3], "page_table")) {
    pool.n_pages = free.numel();
    pool.page_size = static_cast<int>(integer(a[2]));
    pool.free_pages = static_cast<int32_t*>(free.data_ptr());
    pool.count = longs(&tensor(a[1], "count"));
    TORCH_CHECK_VALUE(table.scalar_type() == at::kInt && table.dim() == 2 && table.device() == free.device() &&
                          table.is_contiguous() && table.numel() > 0,
                      "page_table must be a contiguous int32 tensor [B, max_pages] on the pool's device");
    B = table.size(0);
    max_pages = table.size(1);
  }
  void check(const Tensor& t, int64_t n, const char* name) const {
    check_index(t, free.device(), name);
    TORCH_CHECK_VALUE(t.numel() == n, name, " must have ", n, " entries");
  }
  int32_t* entries() const { return static_cast<int32_t*>(table.data_ptr()); }
};

// (free, count, page size, page table, start, off, total (-1: not known), slots: tensor, True or False) -> slots or None
PyObject* page_assign(PyObject* const* a) {
  const PoolCall c(a);
  const Tensor& start = tensor(a[4], "start");
  const Tensor* off = optional(a[5], "off");
  int64_t total = integer(a[6]);
  c.check(start, c.B, "start");
  const Tensor* to = THPVariable_Check(a[7]) ? &THPVariable_Unpack(a[7]) : nullptr;
  if (to && total < 0 && to->dim() == 1) total = to->numel();
  if (off) {
    c.check(*off, c.B + 1, "off");
    TORCH_CHECK_VALUE(total >= 0, "total must not be negative");
  } else {
    TORCH_CHECK_VALUE(total < 0 || total == c.B, "without off there is one row per sequence");
    total = c.B;
  }
  if (to) c.check(*to, total, "slots");
  const bool wanted = to || truth(a[7]);
  Place place(c.free.get_device());
  Tensor slots, scratch;
  int rc;
  {
    Unlocked unlocked;
    size_t bytes = 0;
    rc = lib.page_scratch_size(c.B, total, c.max_pages, &bytes);
    if (rc == 0) {
      if (bytes > 0) scratch = empty({static_cast<int64_t>(bytes)}, c.free, at::kByte);
      if (wanted && !to) slots = empty({total}, c.free, at::kLong);
      rc = lib.page_assign(&c.pool, c.B, total, longs(off), longs(&start), c.entries(), c.max_pages,
                           wanted ? longs(to ? to : &slots) : nullptr, bytes > 0 ? scratch.data_ptr() : nullptr, bytes,
                           place.status, kStatusBytes, place.stream);
    }
  }
  finish(rc, "jattn_page_assign");
  return to ? given(a[7]) : wanted ? wrap(slots) : none();
}

// (free, count, page size, page table, lens, keep) -> None
PyObject* page_release(PyObject* const* a) {
  const PoolCall c(a);
  const Tensor& lens = tensor(a[4], "lens");
  const Tensor* keep = optional(a[5], "keep");
  c.check(lens, c.B, "lens");
  if (keep) c.check(*keep, c.B, "keep");
  Place place(c.free.get_device());
  Tensor scratch;
  int rc;
  {
    Unlocked unlocked;
    size_t bytes = 0;
    rc = lib.page_scratch_size(c.B, -1, c.max_pages, &bytes);
    if (rc == 0) {
      if (bytes > 0) scratch = empty({static_cast<int64_t>(bytes)}, c.free, at::kByte);
      rc = lib.page_release(&c.pool, c.B, longs(&lens), longs(keep), c.entries(), c.max_pages,
                            bytes > 0 ? scratch.data_ptr() : nullptr, bytes, place.status, kStatusBytes, place.stream);
    }
  }
  finish(rc, "jattn_page_release");
  return none();
}

// (handle of the loaded library, check, status)
PyObject* bind(PyObject* const* a) {
  void* handle = PyLong_AsVoidPtr(a[0]);
  if (PyErr_Occurred()) throw Raised{};
  const auto find = [&](auto& f, const char* name) {
    f = reinterpret_cast<std::remove_reference_t<decltype(f)>>(dlsym(handle, name));
    TORCH_CHECK(f != nullptr, "the library has no ", name);
  };
  Library l{};
  find(l.layer_norm, "jattn_layer_norm");
  find(l.layer_norm_bwd, "jattn_layer_norm_bwd");
  find(l.layer_norm_bwd_scratch_size, "jattn_layer_norm_bwd_scratch_size");
  find(l.rotary, "jattn_rotary");
  find(l.rotary_tables, "jattn_rotary_tables");
  find(l.page_scratch_size, "jattn_page_scratch_size");
  find(l.page_assign, "jattn_page_assign");
  find(l.page_release, "jattn_page_release");
  lib = l;
  g_check = given(a[1]);
  g_status = given(a[2]);
  return none();
}

// A method of N arguments; nothing that C++ throws passes it.
template <PyObject* (*F)(PyObject* const*), Py_ssize_t N>
PyObject* method(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  if (n != N) {
    PyErr_Format(PyExc_TypeError, "%zd arguments, not %zd", N, n);
    return nullptr;
  }
  try {
    return F(a);
  } catch (const Raised&) {
    return nullptr;
  }
  END_HANDLE_TH_ERRORS
}
template <PyObject* (*F)(PyObject* const*), Py_ssize_t N>
PyMethodDef def(const char* name) {
  return PyMethodDef{name, reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(&method<F, N>)), METH_FASTCALL, nullptr};
}

PyMethodDef methods[] = {def<bind, 3>("bind"),
                         def<layer_norm, 6>("layer_norm"),
                         def<layer_norm_bwd, 8>("layer_norm_bwd"),
                         def<rotary, 8>("rotary"),
                         def<rotary_followed, 3>("rotary_followed"),
                         def<rotary_tables, 10>("rotary_tables"),
                         def<page_assign, 8>("page_assign"),
                         def<page_release, 6>("page_release"),
                         PyMethodDef{nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_host", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__host(void) { return PyModule_Create(&module); }
