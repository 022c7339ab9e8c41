// Marshalling of the page-pool and shared-prefix entry points from torch tensors, natively:
// the calls of a serving step take a few microseconds on the GPU, and the same checks made in
// Python took longer than that (a fork of 4 rows 15 us of host time, here 8).  Nothing is
// computed here; every call goes to the C ABI of libpka.so.
//
// Functions take positional arguments, None for what is not given, and return tensors.  A
// tensor that does not fit raises ValueError; an error code of the library is handed to the
// callable given to init(), which raises.
#include <Python.h>

#include <algorithm>
#include <climits>
#include <cstdint>
#include <initializer_list>
#include <stdexcept>
#include <string>
#include <utility>
#include <vector>

#include <ATen/ops/empty.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include "pka.h"

namespace {

PyObject* g_on_error = nullptr;   // callable(code, where)

struct PythonError {};   // the interpreter holds the error
struct ValueError : std::runtime_error {
  using std::runtime_error::runtime_error;
};

[[noreturn]] void bad(const std::string& what) { throw ValueError(what); }

void check_code(int code, const char* where) {
  if (code == PKA_OK) return;
  PyObject* r = PyObject_CallFunction(g_on_error, "is", code, where);
  Py_XDECREF(r);
  if (r != nullptr) PyErr_SetString(PyExc_RuntimeError, where);
  throw PythonError{};
}

// The arguments of a call, taken in turn.
class Args {
 public:
  Args(PyObject* const* args, Py_ssize_t n, Py_ssize_t want) : args_(args) {
    if (n != want) {
      PyErr_Format(PyExc_TypeError, "%zd arguments expected, got %zd", want, n);
      throw PythonError{};
    }
  }
  // A tensor, nullptr for None.
  const at::Tensor* tensor() {
    PyObject* o = args_[i_++];
    if (o == Py_None) return nullptr;
    if (!THPVariable_Check(o)) {
      PyErr_Format(PyExc_TypeError, "a tensor was expected, got %s", Py_TYPE(o)->tp_name);
      throw PythonError{};
    }
    return &THPVariable_Unpack(o);
  }
  const at::Tensor& need(const char* name) {
    const at::Tensor* t = tensor();
    if (t == nullptr) bad(std::string(name) + " is required");
    return *t;
  }
  int64_t number() { return as_number(args_[i_++]); }
  static int64_t as_number(PyObject* o) {
    const long long x = PyLong_AsLongLong(o);
    if (x == -1 && PyErr_Occurred()) throw PythonError{};
    return x;
  }
  // A sequence of numbers, nothing for None.
  std::vector<int64_t> numbers(bool* given) {
    PyObject* o = args_[i_++];
    std::vector<int64_t> out;
    *given = o != Py_None;
    if (!*given) return out;
    PyObject* seq = PySequence_Fast(o, "a sequence of numbers was expected");
    if (seq == nullptr) throw PythonError{};
    const Py_ssize_t n = PySequence_Fast_GET_SIZE(seq);
    for (Py_ssize_t k = 0; k < n; ++k) {
      const long long x = PyLong_AsLongLong(PySequence_Fast_GET_ITEM(seq, k));
      if (x == -1 && PyErr_Occurred()) {
        Py_DECREF(seq);
        throw PythonError{};
      }
      out.push_back(x);
    }
    Py_DECREF(seq);
    return out;
  }
  int32_t number32(const char* name) { return fit32(name, number()); }
  static int32_t fit32(const char* name, int64_t x) {
    if (x < INT32_MIN || x > INT32_MAX) bad(std::string(name) + " does not fit 32 bits");
    return (int32_t)x;
  }

 private:
  PyObject* const* args_;
  Py_ssize_t i_ = 0;
};

void* ptr(const at::Tensor* t) { return t == nullptr || t->numel() == 0 ? nullptr : t->data_ptr(); }
void* ptr(const at::Tensor& t) { return t.numel() == 0 ? nullptr : t.data_ptr(); }

// The given tensor has this type and lies on device `dev`, where the library launches.
void fits(const at::Tensor* t, at::ScalarType type, int dev, const char* name) {
  if (t == nullptr) return;
  if (t->scalar_type() != type)
    bad(std::string(name) + " must be " + c10::toString(type) + ", got " + c10::toString(t->scalar_type()));
  if (!t->is_cuda() || t->get_device() != dev)
    bad(std::string(name) + " is on " + t->device().str() + ", the current device is cuda:" + std::to_string(dev));
}
void fits(const at::Tensor& t, at::ScalarType type, int dev, const char* name) { fits(&t, type, dev, name); }

int32_t count32(const at::Tensor& t, const char* name) { return Args::fit32(name, t.numel()); }

void dense(const at::Tensor& t, int64_t n, const char* name) {
  if (t.numel() != n || !t.is_contiguous()) bad(std::string(name) + " must hold " + std::to_string(n) + " contiguous entries");
}

at::Tensor new_tensor(at::IntArrayRef shape, at::ScalarType type, int dev) {
  return at::empty(shape, at::TensorOptions().dtype(type).device(c10::Device(c10::kCUDA, (c10::DeviceIndex)dev)));
}

// An int32 output of n entries: the given one, checked, or a new one.
at::Tensor out_i32(const at::Tensor* t, int64_t n, int dev, const char* name) {
  if (t == nullptr) return new_tensor({n}, at::kInt, dev);
  fits(t, at::kInt, dev, name);
  dense(*t, n, name);
  return *t;
}

int current_device() { return (int)c10::cuda::current_device(); }
void* current_stream() { return c10::cuda::getCurrentCUDAStream().stream(); }

PyObject* pack(std::initializer_list<at::Tensor> list) {
  PyObject* tuple = PyTuple_New((Py_ssize_t)list.size());
  if (tuple == nullptr) throw PythonError{};
  Py_ssize_t i = 0;
  for (const at::Tensor& t : list) {
    PyObject* o = THPVariable_Wrap(t);
    if (o == nullptr) {
      Py_DECREF(tuple);
      throw PythonError{};
    }
    PyTuple_SET_ITEM(tuple, i++, o);
  }
  return tuple;
}

// The stride of a dimension; of one of size 1, whose own says nothing, that of a dense tensor.
int64_t stride_of(const at::Tensor& t, int64_t d) {
  if (t.size(d) > 1) return t.stride(d);
  int64_t n = 1;
  for (int64_t i = d + 1; i < t.dim(); ++i) n *= std::max<int64_t>(1, t.size(i));
  return n;
}
// The same shape, and rows at the same places.
bool alike(const at::Tensor& x, const at::Tensor& y) {
  if (!x.sizes().equals(y.sizes())) return false;
  for (int64_t d = 0; d < x.dim(); ++d)
    if (x.size(d) > 1 && x.stride(d) != y.stride(d)) return false;
  return true;
}

// Rows, width and row stride of block tables.
struct Tables {
  int32_t rows, width;
  int64_t stride;
};
Tables tables_of(const at::Tensor& kv_lens, const at::Tensor& tables, const char* name) {
  if (tables.dim() != 2 || tables.size(0) != kv_lens.numel() || !kv_lens.is_contiguous())
    bad(std::string(name) + " must have one row per request, kv_lens be contiguous");
  if (tables.stride(1) != 1 && tables.size(1) > 1) bad(std::string(name) + " rows must be dense");
  Tables t{count32(kv_lens, "kv_lens"), Args::fit32(name, tables.size(1)), tables.stride(0)};
  if (t.rows <= 1 && t.stride < t.width) t.stride = t.width;   // one row's stride says nothing
  return t;
}

// Strides of a pair of HND pools.
struct Pools {
  int64_t pages, page_stride, head_stride;
  int32_t heads, page_size, dim;
};
Pools pools_of(const at::Tensor& k, const at::Tensor& v) {
  if (k.dim() != 4 || !alike(k, v))
    bad("k_pages and v_pages must be [num_pages, num_kv_heads, page_size, head_dim] with the same strides");
  Pools p{k.size(0), stride_of(k, 0), stride_of(k, 1), Args::fit32("num_kv_heads", k.size(1)),
          Args::fit32("page_size", k.size(2)), Args::fit32("head_dim", k.size(3))};
  if (k.stride(3) != 1 || stride_of(k, 2) != p.dim) bad("each page's slots must be dense rows of head_dim elements");
  return p;
}

int32_t dtype_code(at::ScalarType t, const char* what) {
  if (t == at::kBFloat16) return PKA_DTYPE_BF16;
  if (t == at::kHalf) return PKA_DTYPE_F16;
  bad(std::string(what) + " must be bfloat16 or float16, got " + c10::toString(t));
}
at::ScalarType type_of(int64_t code) {
  return code == PKA_DTYPE_BF16 ? at::kBFloat16 : code == PKA_DTYPE_F16 ? at::kHalf : at::kFloat;
}

// (k, v, slot_map, k_pages, v_pages, q, positions, inv_freq, sections, pairs, q_out, status)
PyObject* rope_append(Args a) {
  const at::Tensor &k = a.need("k"), &v = a.need("v"), &slots = a.need("slot_map"), &kp = a.need("k_pages"),
                   &vp = a.need("v_pages");
  const at::Tensor *q = a.tensor(), *pos = a.tensor(), *freq = a.tensor();
  bool sections_given = false;
  const std::vector<int64_t> sections = a.numbers(&sections_given);
  const int32_t pairs = a.number32("pairs");
  const at::Tensor *q_out = a.tensor(), *status = a.tensor();
  const at::ScalarType type = kp.scalar_type();
  const int32_t code = dtype_code(type, "the pools");
  const int dev = current_device();
  fits(kp, type, dev, "k_pages");
  fits(vp, type, dev, "v_pages");
  fits(k, type, dev, "k");
  fits(v, type, dev, "v");
  fits(q, type, dev, "q");
  fits(q_out, type, dev, "q_out");
  fits(slots, at::kLong, dev, "slot_map");
  fits(pos, at::kInt, dev, "positions");
  fits(status, at::kInt, dev, "status");
  if (status != nullptr) dense(*status, 1, "status");
  const Pools p = pools_of(kp, vp);
  if (k.dim() != 3 || k.size(1) != p.heads || k.size(2) != p.dim || !v.sizes().equals(k.sizes()))
    bad("k and v must be [T, " + std::to_string(p.heads) + ", " + std::to_string(p.dim) + "]");
  const int64_t T = k.size(0);
  if (T > 0 && (k.stride(2) != 1 || !alike(k, v)))
    bad("k and v must have the same strides and a dense last dimension");
  if (slots.numel() != T || !slots.is_contiguous()) bad("slot_map needs one contiguous entry per token");
  at::Tensor out;
  int32_t heads = 0;
  int64_t strides[4] = {0, 0, 0, 0};
  if (q != nullptr) {
    if (q->dim() != 3 || q->size(0) != T || q->size(2) != p.dim || (T > 0 && q->stride(2) != 1))
      bad("q must be [T, Hq, head_dim] with a dense last dimension");
    heads = Args::fit32("num_qo_heads", q->size(1));
    if (q_out == nullptr) {
      out = new_tensor({T, heads, p.dim}, type, dev);
    } else {
      if (!q_out->sizes().equals(q->sizes()) || (T > 0 && q_out->stride(2) != 1))
        bad("q_out must have the shape of q and a dense last dimension");
      out = *q_out;
    }
    strides[0] = stride_of(*q, 0);
    strides[1] = stride_of(*q, 1);
    strides[2] = stride_of(out, 0);
    strides[3] = stride_of(out, 1);
  } else if (q_out != nullptr) {
    bad("q_out without q");
  }
  int32_t section[4] = {0, 0, 0, 0}, axes = 0, half = 0;
  int64_t pos_stride = 0;
  if (freq != nullptr) {
    fits(freq, at::kDouble, dev, "inv_freq");
    if (!freq->is_contiguous()) bad("inv_freq must be contiguous");
    half = Args::fit32("inv_freq", freq->numel());
    if (half > 65536) bad("inv_freq is too long");
    if (pos == nullptr) bad("a rotation needs positions");
    if (pos->dim() < 1 || pos->dim() > 2 || pos->size(-1) != T || (T > 1 && pos->stride(-1) != 1))
      bad("positions must be [axes, T] or [T] with dense rows");
    axes = pos->dim() == 1 ? 1 : Args::fit32("axes", pos->size(0));
    if (axes < 1 || axes > 4 || sections.size() > (size_t)axes)
      bad("positions need 1 to 4 axes, one for each of the sections");
    pos_stride = axes > 1 ? pos->stride(0) : T;
    if (!sections_given) section[0] = half;
    for (size_t i = 0; i < sections.size(); ++i) section[i] = Args::fit32("a section", sections[i]);
  } else if (pos != nullptr || sections_given) {
    bad("positions and sections go with inv_freq");
  }
  const bool any = heads > 0 && T > 0;
  const int rc = paged_rope_append(any ? q->data_ptr() : nullptr, strides[0], strides[1], any ? out.data_ptr() : nullptr,
                                   strides[2], strides[3], any ? heads : 0, ptr(k), ptr(v), stride_of(k, 0), stride_of(k, 1),
                                   p.heads, p.dim, static_cast<const int32_t*>(pos != nullptr ? pos->data_ptr() : nullptr),
                                   pos_stride, static_cast<const double*>(ptr(freq)), 2 * half, axes, section, pairs,
                                   static_cast<const int64_t*>(ptr(slots)), T, ptr(kp), ptr(vp), p.pages, p.page_size,
                                   p.page_stride, p.head_stride, code, static_cast<int32_t*>(ptr(status)),
                                   current_stream());
  check_code(rc, "paged_rope_append");
  if (q == nullptr) Py_RETURN_NONE;
  return THPVariable_Wrap(out);
}

// (parents, children, kv_lens, free_pages, free_head, block_tables, page_size, seq_lens, src_pages,
//  dst_pages, free_head_out, status)
PyObject* kv_fork(Args a) {
  const at::Tensor &parents = a.need("parents"), &children = a.need("children"), &kv = a.need("kv_lens"),
                   &free_pages = a.need("free_pages"), &head = a.need("free_head"), &tables = a.need("block_tables");
  const int32_t page_size = a.number32("page_size");
  const at::Tensor *seq = a.tensor(), *src = a.tensor(), *dst = a.tensor(), *head_out = a.tensor(), *status = a.tensor();
  const int dev = current_device();
  fits(parents, at::kInt, dev, "parents");
  fits(children, at::kInt, dev, "children");
  fits(kv, at::kInt, dev, "kv_lens");
  fits(free_pages, at::kInt, dev, "free_pages");
  fits(head, at::kInt, dev, "free_head");
  fits(tables, at::kInt, dev, "block_tables");
  fits(status, at::kInt, dev, "status");
  if (status != nullptr) dense(*status, 1, "status");
  const Tables t = tables_of(kv, tables, "block_tables");
  if (head.numel() != 1 || !free_pages.is_contiguous()) bad("free_head must hold one entry, free_pages be contiguous");
  const int32_t n = count32(parents, "parents");
  if (children.numel() != n || !parents.is_contiguous() || !children.is_contiguous())
    bad("parents and children must be contiguous, one child per parent");
  const at::Tensor o_seq = out_i32(seq, t.rows, dev, "seq_lens"), o_src = out_i32(src, n, dev, "src_pages"),
                   o_dst = out_i32(dst, n, dev, "dst_pages"), o_head = out_i32(head_out, 1, dev, "free_head_out");
  const int rc = paged_kv_fork(
      static_cast<int32_t*>(ptr(parents)), static_cast<int32_t*>(ptr(children)), n, static_cast<int32_t*>(ptr(kv)),
      t.rows, static_cast<int32_t*>(ptr(free_pages)), count32(free_pages, "free_pages"),
      static_cast<int32_t*>(ptr(head)), page_size, static_cast<int32_t*>(ptr(tables)), t.stride, t.width,
      static_cast<int32_t*>(ptr(o_seq)), static_cast<int32_t*>(ptr(o_src)), static_cast<int32_t*>(ptr(o_dst)),
      static_cast<int32_t*>(ptr(o_head)), static_cast<int32_t*>(ptr(status)), current_stream());
  check_code(rc, "paged_kv_fork");
  return pack({o_seq, o_src, o_dst, o_head});
}

// (rows, kv_lens, free_pages, free_head, block_tables, page_size, num_pages, seq_lens, free_head_out,
//  status)
PyObject* kv_free(Args a) {
  const at::Tensor &rows = a.need("rows"), &kv = a.need("kv_lens"), &free_pages = a.need("free_pages"),
                   &head = a.need("free_head"), &tables = a.need("block_tables");
  const int32_t page_size = a.number32("page_size");
  const int64_t pages = a.number();
  const at::Tensor *seq = a.tensor(), *head_out = a.tensor(), *status = a.tensor();
  const int dev = current_device();
  fits(rows, at::kInt, dev, "rows");
  fits(kv, at::kInt, dev, "kv_lens");
  fits(free_pages, at::kInt, dev, "free_pages");
  fits(head, at::kInt, dev, "free_head");
  fits(tables, at::kInt, dev, "block_tables");
  fits(status, at::kInt, dev, "status");
  if (status != nullptr) dense(*status, 1, "status");
  const Tables t = tables_of(kv, tables, "block_tables");
  if (head.numel() != 1 || !free_pages.is_contiguous()) bad("free_head must hold one entry, free_pages be contiguous");
  if (!rows.is_contiguous()) bad("rows must be contiguous");
  const at::Tensor o_seq = out_i32(seq, t.rows, dev, "seq_lens"), o_head = out_i32(head_out, 1, dev, "free_head_out");
  const int rc = paged_kv_free(
      static_cast<int32_t*>(ptr(rows)), count32(rows, "rows"), static_cast<int32_t*>(ptr(kv)), t.rows,
      static_cast<int32_t*>(ptr(free_pages)), count32(free_pages, "free_pages"), static_cast<int32_t*>(ptr(head)),
      page_size, static_cast<int32_t*>(ptr(tables)), t.stride, t.width, pages, static_cast<int32_t*>(ptr(o_seq)),
      static_cast<int32_t*>(ptr(o_head)), static_cast<int32_t*>(ptr(status)), current_stream());
  check_code(rc, "paged_kv_free");
  return pack({o_seq, o_head});
}

// (kv_lens, free_pages, free_head, block_tables, page_size, num_pages, block_tables_out,
//  free_pages_out, src_pages, dst_pages, num_moves, status)
PyObject* kv_compact(Args a) {
  const at::Tensor &kv = a.need("kv_lens"), &free_pages = a.need("free_pages"), &head = a.need("free_head"),
                   &tables = a.need("block_tables");
  const int32_t page_size = a.number32("page_size");
  const int64_t pages = a.number();
  const at::Tensor *tables_out = a.tensor(), *free_out = a.tensor(), *src = a.tensor(), *dst = a.tensor(),
                   *moves = a.tensor(), *status = a.tensor();
  const int dev = current_device();
  fits(kv, at::kInt, dev, "kv_lens");
  fits(free_pages, at::kInt, dev, "free_pages");
  fits(head, at::kInt, dev, "free_head");
  fits(tables, at::kInt, dev, "block_tables");
  fits(tables_out, at::kInt, dev, "block_tables_out");
  fits(status, at::kInt, dev, "status");
  if (status != nullptr) dense(*status, 1, "status");
  const Tables t = tables_of(kv, tables, "block_tables");
  if (head.numel() != 1 || !free_pages.is_contiguous()) bad("free_head must hold one entry, free_pages be contiguous");
  if (tables_out != nullptr && !tables_out->sizes().equals(tables.sizes()))
    bad("block_tables_out must have the shape of block_tables");
  const at::Tensor o_tables = tables_out != nullptr ? *tables_out : new_tensor({t.rows, t.width}, at::kInt, dev);
  const Tables o = tables_of(kv, o_tables, "block_tables_out");
  const int32_t n = count32(free_pages, "free_pages");
  const int64_t most = src != nullptr ? src->numel() : std::min<int64_t>(n, pages > 0 ? pages : 0);
  const at::Tensor o_free = out_i32(free_out, n, dev, "free_pages_out"), o_src = out_i32(src, most, dev, "src_pages"),
                   o_dst = out_i32(dst, most, dev, "dst_pages"), o_moves = out_i32(moves, 1, dev, "num_moves");
  const int rc = paged_kv_compact(
      static_cast<int32_t*>(ptr(kv)), t.rows, static_cast<int32_t*>(ptr(free_pages)), n,
      static_cast<int32_t*>(ptr(head)), page_size, static_cast<int32_t*>(ptr(tables)), t.stride, t.width, pages,
      static_cast<int32_t*>(ptr(o_tables)), o.stride, static_cast<int32_t*>(ptr(o_free)),
      static_cast<int32_t*>(ptr(o_src)), static_cast<int32_t*>(ptr(o_dst)), Args::fit32("src_pages", most),
      static_cast<int32_t*>(ptr(o_moves)), static_cast<int32_t*>(ptr(status)), current_stream());
  check_code(rc, "paged_kv_compact");
  return pack({o_tables, o_free, o_src, o_dst, o_moves});
}

// (pool addresses, page strides, page bytes, pools, pages, device, src_pages, dst_pages, count, status):
// the first three are addresses of host arrays
PyObject* kv_copy(Args a) {
  void* const* pools = reinterpret_cast<void* const*>(a.number());
  const int64_t* strides = reinterpret_cast<const int64_t*>(a.number());
  const int64_t* bytes = reinterpret_cast<const int64_t*>(a.number());
  const int32_t n_pools = a.number32("pools");
  const int64_t pages = a.number();
  const int64_t device = a.number();
  const at::Tensor &src = a.need("src_pages"), &dst = a.need("dst_pages");
  const at::Tensor *count = a.tensor(), *status = a.tensor();
  const int dev = current_device();
  if (device != dev)
    bad("the pools are on cuda:" + std::to_string(device) + ", the current device is cuda:" + std::to_string(dev));
  fits(src, at::kInt, dev, "src_pages");
  fits(dst, at::kInt, dev, "dst_pages");
  fits(count, at::kInt, dev, "count");
  fits(status, at::kInt, dev, "status");
  if (status != nullptr) dense(*status, 1, "status");
  if (count != nullptr) dense(*count, 1, "count");
  if (dst.numel() != src.numel() || !src.is_contiguous() || !dst.is_contiguous())
    bad("src_pages and dst_pages must be contiguous, one of each per entry");
  const int rc = paged_kv_copy(pools, strides, bytes, n_pools, pages, static_cast<int32_t*>(ptr(src)),
                               static_cast<int32_t*>(ptr(dst)), count32(src, "src_pages"),
                               static_cast<int32_t*>(ptr(count)), static_cast<int32_t*>(ptr(status)), current_stream());
  check_code(rc, "paged_kv_copy");
  Py_RETURN_NONE;
}

// (plan: a tuple of its handle, query rows, batch size, query heads, head dimension, pages, KV
// heads, page size, table width, input type, output type, whether it returns the LSE, and
// workspace bytes; q, k_pages, v_pages, block_tables, seq_lens_kv, sinks, out, lse, workspace)
PyObject* prefix_decode_run(PyObject* plan, Args a) {
  int64_t f[13];
  if (!PyTuple_Check(plan) || PyTuple_GET_SIZE(plan) != 13) {
    PyErr_SetString(PyExc_TypeError, "a plan's facts were expected");
    throw PythonError{};
  }
  for (int i = 0; i < 13; ++i) f[i] = Args::as_number(PyTuple_GET_ITEM(plan, i));
  const int64_t need = f[1], B = f[2], Hq = f[3], D = f[4];
  const at::ScalarType type = type_of(f[9]), out_type = type_of(f[10]);
  const at::Tensor &q = a.need("q"), &kp = a.need("k_pages"), &vp = a.need("v_pages"), &tables = a.need("block_tables");
  const at::Tensor *lens = a.tensor(), *sinks = a.tensor(), *out = a.tensor(), *lse = a.tensor(), *ws = a.tensor();
  const int dev = current_device();
  fits(q, type, dev, "q");
  fits(kp, type, dev, "k_pages");
  fits(vp, type, dev, "v_pages");
  fits(tables, at::kInt, dev, "block_tables");
  fits(lens, at::kInt, dev, "seq_lens_kv");
  fits(sinks, at::kFloat, dev, "sinks");
  fits(out, out_type, dev, "out");
  fits(lse, at::kFloat, dev, "lse");
  if (q.dim() != 3 || q.size(0) < need || q.size(1) != Hq || q.size(2) != D || q.stride(2) != 1)
    bad("q must be [>= " + std::to_string(need) + ", " + std::to_string(Hq) + ", " + std::to_string(D) +
        "] with a dense last dimension");
  const Pools p = pools_of(kp, vp);
  if (p.pages != f[5] || p.heads != f[6] || p.page_size != f[7] || p.dim != D)
    bad("the pools must be [" + std::to_string(f[5]) + ", " + std::to_string(f[6]) + ", " + std::to_string(f[7]) + ", " +
        std::to_string(D) + "]");
  if (tables.dim() != 2 || tables.size(0) < B || tables.size(1) < f[8] || (tables.size(1) > 1 && tables.stride(1) != 1))
    bad("block_tables needs dense rows, one of at least max_pages_per_seq entries per request");
  int64_t row = tables.stride(0);
  if (tables.size(0) <= 1 && row < tables.size(1)) row = tables.size(1);   // one row's stride says nothing
  if (lens != nullptr && (lens->numel() < B || !lens->is_contiguous()))
    bad("seq_lens_kv needs one contiguous entry per request");
  if (sinks != nullptr) dense(*sinks, Hq, "sinks");
  const int64_t T = q.size(0);
  at::Tensor o, l, w;
  if (out != nullptr) {
    if (out->dim() != 3 || out->size(0) < need || out->size(1) != Hq || out->size(2) != D || !out->is_contiguous())
      bad("out must be a contiguous [T, num_qo_heads, head_dim]");
    o = *out;
  } else {
    o = new_tensor({T, Hq, D}, out_type, dev);
  }
  if (lse != nullptr) {
    if (lse->dim() != 2 || lse->size(0) < need || lse->size(1) != Hq || !lse->is_contiguous())
      bad("lse must be a contiguous [T, num_qo_heads]");
    l = *lse;
  } else if (f[11]) {
    l = new_tensor({T, Hq}, at::kFloat, dev);
  }
  if (ws != nullptr) {
    if (!ws->is_cuda() || ws->get_device() != dev || !ws->is_contiguous()) bad("workspace must be contiguous, on the current device");
    w = *ws;
  } else if (f[12] > 0) {
    w = new_tensor({f[12]}, at::kByte, dev);
  }
  const int rc = paged_prefix_decode_run(
      reinterpret_cast<const pka_prefix_plan*>(f[0]), ptr(q), stride_of(q, 0), stride_of(q, 1), ptr(kp), ptr(vp), p.page_stride,
      p.head_stride, static_cast<int32_t*>(ptr(tables)), row, static_cast<int32_t*>(ptr(lens)),
      static_cast<float*>(ptr(sinks)), ptr(o), l.defined() ? static_cast<float*>(ptr(l)) : nullptr,
      w.defined() ? ptr(w) : nullptr, w.defined() ? w.nbytes() : 0, current_stream());
  check_code(rc, "paged_prefix_decode_run");
  return f[11] ? pack({o, l}) : THPVariable_Wrap(o);
}

// Runs `f`, turning its exceptions into Python's.
template <typename F>
PyObject* guarded(F&& f) {
  try {
    return f();
  } catch (const PythonError&) {
  } catch (const ValueError& e) {
    PyErr_SetString(PyExc_ValueError, e.what());
  } catch (const c10::Error& e) {
    PyErr_SetString(PyExc_RuntimeError, e.what_without_backtrace());
  } catch (const std::exception& e) {
    PyErr_SetString(PyExc_RuntimeError, e.what());
  }
  return nullptr;
}

template <PyObject* (*F)(Args), int N>
PyObject* entry(PyObject*, PyObject* const* args, Py_ssize_t n) {
  return guarded([&] { return F(Args(args, n, N)); });
}

PyObject* prefix_entry(PyObject*, PyObject* const* args, Py_ssize_t n) {
  return guarded([&] {
    Args rest(args + 1, n - 1, 9);
    return prefix_decode_run(args[0], rest);
  });
}

PyObject* init(PyObject*, PyObject* on_error) {
  Py_INCREF(on_error);
  Py_XSETREF(g_on_error, on_error);
  Py_RETURN_NONE;
}

template <typename F>
PyCFunction fast(F f) {
  return reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(f));
}

PyMethodDef methods[] = {
    {"init", init, METH_O, nullptr},
    {"rope_append", fast(&entry<rope_append, 12>), METH_FASTCALL, nullptr},
    {"kv_fork", fast(&entry<kv_fork, 12>), METH_FASTCALL, nullptr},
    {"kv_free", fast(&entry<kv_free, 10>), METH_FASTCALL, nullptr},
    {"kv_compact", fast(&entry<kv_compact, 12>), METH_FASTCALL, nullptr},
    {"kv_copy", fast(&entry<kv_copy, 10>), METH_FASTCALL, nullptr},
    {"prefix_decode_run", fast(&prefix_entry), METH_FASTCALL, nullptr},
    {nullptr, nullptr, 0, nullptr}};

PyModuleDef module = {PyModuleDef_HEAD_INIT, "_pka_binding", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__pka_binding() { return PyModule_Create(&module); }
