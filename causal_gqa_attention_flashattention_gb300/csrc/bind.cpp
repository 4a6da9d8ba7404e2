// Compiled part of the binding for the calls that serve drafted trees: checks of the tensors, outputs and the
// library's entry point in one step, since such calls take less time on the device than their checks do in
// Python (one plan for 64 sequences 4.4 us on the device, 28 us of Python and ctypes, 9 us so; a tree's attention 27
// and 10). binding.py has the public functions, gives the library's entry points to init() and turns a returned
// status into its error.
#include <ATen/core/LegacyTypeDispatch.h>
#include <ATen/core/Tensor.h>
#include <ATen/ops/as_strided.h>
#include <ATen/ops/empty.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include <cxxabi.h>

#include <algorithm>
#include <exception>
#include <stdexcept>
#include <string>

#include "../../include/ne_attn.h"

namespace {

decltype(&ne_attn_paged_plan_ex) f_plan = nullptr;
decltype(&ne_attn_kv_append_slots) f_append = nullptr;
decltype(&ne_attn_decode_tree) f_tree = nullptr;
decltype(&ne_attn_decode_tree_workspace_size) f_tree_size = nullptr;
decltype(&ne_attn_kv_keep_paged) f_keep = nullptr;
PyObject* out_of_memory = nullptr;  // torch.OutOfMemoryError

using at::Tensor;
using Sizes = c10::IntArrayRef;
constexpr auto kInt = at::kInt, kFloat = at::kFloat, kBf16 = at::kBFloat16, kHalf = at::kHalf, kByte = at::kByte;

[[noreturn]] void bad(const std::string& what) { throw std::invalid_argument(what); }
void need(bool ok, const char* what) {
  if (!ok) bad(what);
}

// Other Python threads run while this lives: an allocation may wait for the device, the library's entry points for its
// mutex, for a workspace that grows or for room in a launch queue.  (A thread that is ended while it waits for its turn, as
// the interpreter shuts down, is unwound through the destructor.)
struct NoGil {
  PyThreadState* state = PyEval_SaveThread();
  NoGil() = default;
  NoGil(const NoGil&) = delete;
  ~NoGil() noexcept(false) { PyEval_RestoreThread(state); }
};

const Tensor& tensor(PyObject* o, const char* name) {
  if (!THPVariable_Check(o)) bad(std::string(name) + " must be a tensor");
  return THPVariable_Unpack(o);
}
bool given(PyObject* o) { return o != Py_None; }
long long whole(PyObject* o) {
  const long long x = PyLong_AsLongLong(o);
  if (x == -1 && PyErr_Occurred()) throw std::domain_error("");  // the Python error stands
  return x;
}
// A C int: what does not fit is refused by the library as its largest or smallest.
int number(PyObject* o) {
  const long long x = whole(o);
  return (int)std::max(-2147483647LL - 1, std::min(2147483647LL, x));
}
float real(PyObject* o) {
  const double x = PyFloat_AsDouble(o);
  if (x == -1.0 && PyErr_Occurred()) throw std::domain_error("");
  return (float)x;
}
bool truth(PyObject* o) {
  const int x = PyObject_IsTrue(o);
  if (x < 0) throw std::domain_error("");
  return x == 1;
}

int* ints(const Tensor& t, const char* name, c10::Device dev, Sizes shape) {
  if (t.scalar_type() != kInt || t.device() != dev || t.sizes() != shape || !t.is_contiguous())
    bad(std::string(name) + " must be a contiguous int32 tensor of the call's shape on its device");
  return t.data_ptr<int>();
}
int* ints(PyObject* o, const char* name, c10::Device dev, Sizes shape) { return ints(tensor(o, name), name, dev, shape); }

// Row stride of t [.., H, D]: heads contiguous, positions evenly spaced.
long long head_rows(const Tensor& t, const char* name, c10::Device dev) {
  if (t.scalar_type() != kBf16 || t.device() != dev) bad(std::string(name) + " must be bfloat16 on the call's CUDA device");
  const auto n = t.sizes(), s = t.strides();
  const size_t d = n.size();
  const int64_t H = n[d - 2], D = n[d - 1];
  bool ok = s[d - 1] == 1 && (H == 1 || s[d - 2] == D);
  long long row;
  if (d == 3) {
    row = n[0] > 1 ? s[0] : H * D;
  } else {
    row = n[1] > 1 ? s[1] : (n[0] > 1 ? s[0] : H * D);
    ok = ok && (n[0] == 1 || n[1] == 1 || s[0] == n[1] * s[1]);
  }
  if (!ok) bad(std::string(name) + ": the heads of a position must be contiguous and the positions evenly spaced");
  return row;
}
const void* weight(PyObject* o, const char* name, c10::Device dev, int64_t D) {
  if (!given(o)) return nullptr;
  const Tensor& t = tensor(o, name);
  if (t.scalar_type() != kBf16 || t.device() != dev || t.dim() != 1 || t.size(0) != D || !t.is_contiguous())
    bad(std::string(name) + " must be a contiguous bfloat16 [D] on the call's device");
  return t.data_ptr();
}

struct Pools {
  void *k, *v;
  int pages, heads, page, D;
  long long stride;
};
Pools pools(PyObject* ok, PyObject* ov, c10::Device dev) {
  const Tensor &k = tensor(ok, "k_pages"), &v = tensor(ov, "v_pages");
  need(k.dim() == 4 && v.sizes() == k.sizes(), "pools must be [num_pages, Hkv, page_size, D]");
  need(k.scalar_type() == kHalf && v.scalar_type() == kBf16 && k.device() == dev && v.device() == dev,
       "pools must be float16 keys and bfloat16 values on the call's CUDA device");
  const auto n = k.sizes();
  const long long stride = n[0] > 1 ? k.stride(0) : n[1] * n[2] * n[3];
  for (const Tensor* t : {&k, &v}) {
    const auto s = t->strides();  // strides of dimensions of one do not matter
    need((n[3] == 1 || s[3] == 1) && (n[2] == 1 || s[2] == n[3]) && (n[1] == 1 || s[1] == n[2] * n[3]) && (n[0] <= 1 || s[0] == stride),
         "pools must be contiguous inside a page and have one page stride");
  }
  for (int i = 0; i < 4; i++) need(n[i] < (1LL << 31), "pools are too large");
  return {k.data_ptr(), v.data_ptr(), (int)n[0], (int)n[1], (int)n[2], (int)n[3], stride};
}

// Tokens and row stride of parents int32 [B, Tq], or [Tq]: one tree for the batch.
const int* tree(PyObject* o, int64_t B, c10::Device dev, int* Tq, long long* stride) {
  const Tensor& t = tensor(o, "parents");
  const int64_t d = t.dim();
  need(t.scalar_type() == kInt && t.device() == dev && (d == 1 || (d == 2 && t.size(0) == B)) &&
           (t.size(d - 1) <= 1 || t.stride(d - 1) == 1) && t.size(d - 1) < (1LL << 31),
       "parents must be int32 [B, Tq] or [Tq], rows contiguous, on the call's device");
  need(t.size(d - 1) > 0, "parents must have a token");  // an empty tensor's pointer would read as none given
  *Tq = (int)t.size(d - 1);
  *stride = d == 1 || B == 1 ? 0 : t.stride(0);
  need(*stride == 0 || *stride >= *Tq, "parents: rows must not overlap");
  return t.data_ptr<int>();
}

Tensor make(Sizes shape, at::ScalarType type, c10::Device dev) {
  NoGil others;
  return at::empty(shape, at::TensorOptions().dtype(type).device(dev));
}
// The status of a library call.
template <class F>
int library(F call) {
  NoGil others;
  return call();
}
// `o` of the given shape, or a new one.
Tensor out32(PyObject* o, const char* name, c10::Device dev, Sizes shape) {
  if (!given(o)) return make(shape, kInt, dev);
  ints(o, name, dev, shape);
  return THPVariable_Unpack(o);
}
void apart(const Tensor& a, const Tensor& b, const char* what) {
  const char *pa = static_cast<const char*>(a.data_ptr()), *pb = static_cast<const char*>(b.data_ptr());
  if (pa < pb + b.nbytes() && pb < pa + a.nbytes()) bad(what);
}

// The call's device, which is the current one as long as this lives, and its stream.
struct Call {
  c10::Device dev;
  c10::cuda::CUDAGuard guard;
  void* stream;
  explicit Call(const Tensor& t, const char* name)
      : dev(t.device()), guard(cuda(t, name)), stream(c10::cuda::getCurrentCUDAStream(dev.index()).stream()) {}
  static c10::Device cuda(const Tensor& t, const char* name) {
    if (!t.is_cuda()) bad(std::string(name) + " must be a CUDA tensor");
    return t.device();
  }
};

PyObject* status(int st) { return PyLong_FromLong(st); }
PyObject* wrap(std::initializer_list<Tensor> out) {
  PyObject* t = PyTuple_New((Py_ssize_t)out.size());
  if (!t) return nullptr;
  Py_ssize_t i = 0;
  for (const Tensor& x : out) {
    PyObject* o = THPVariable_Wrap(x);
    if (!o) {
      Py_DECREF(t);
      return nullptr;
    }
    PyTuple_SET_ITEM(t, i++, o);
  }
  return t;
}

// page_table, free_pages, held, free_span, kv_len, new_len, rows, page_size, parents, kv_len_out, held_out, span_out, new_len_out
PyObject* plan(PyObject* const* a) {
  const Tensor& table = tensor(a[0], "page_table");
  Call c(table, "page_table");
  need(table.dim() == 2, "page_table must be [B, max_pages]");
  const int64_t B = table.size(0), width = table.size(1);
  int* p_table = ints(table, "page_table", c.dev, {B, width});
  const Tensor& ring = tensor(a[1], "free_pages");
  need(ring.dim() == 1, "free_pages must be [num_pages]");
  int* p_ring = ints(ring, "free_pages", c.dev, {ring.size(0)});
  const int *held = ints(a[2], "held", c.dev, {B}), *span = ints(a[3], "free_span", c.dev, {2});
  const int *len = ints(a[4], "kv_len", c.dev, {B}), *add = ints(a[5], "new_len", c.dev, {B});
  const int rows = number(a[6]), page = number(a[7]);
  need(rows >= 0 && B < (1LL << 31) && width < (1LL << 31) && ring.size(0) < (1LL << 31), "sizes must fit");
  int Tq = 0;
  long long pstride = 0;
  const int* parents = given(a[8]) ? tree(a[8], B, c.dev, &Tq, &pstride) : nullptr;
  // what is not given lies in one allocation
  at::AutoDispatchBelowADInplaceOrView plain;
  const bool own_total = !given(a[9]), own_got = !given(a[10]), own_left = !given(a[11]), own_new = !given(a[12]);
  const int64_t most = B + 1 + 2 * (int64_t)rows + (own_total ? B : 0) + (own_got ? B : 0) + (own_left ? 2 : 0) + (own_new ? B : 0);
  const Tensor all = make({most}, kInt, c.dev);
  int64_t at = 0;
  const auto part = [&](int64_t n) {
    at += n;
    return at::as_strided(all, {n}, {1}, at - n);
  };
  const Tensor slots = part(rows), pos = part(rows), cu = part(B + 1);
  const Tensor total = own_total ? part(B) : out32(a[9], "kv_len_out", c.dev, {B});
  const Tensor got = own_got ? part(B) : out32(a[10], "held_out", c.dev, {B}), left = own_left ? part(2) : out32(a[11], "span_out", c.dev, {2});
  const Tensor granted = own_new ? part(B) : out32(a[12], "new_len_out", c.dev, {B});
  if (!own_total) apart(total, THPVariable_Unpack(a[4]), "kv_len_out and kv_len must not share memory");
  const int P = (int)ring.size(0);
  const int st = library([&] {
    return f_plan(p_table, p_ring, held, span, len, add, parents, got.data_ptr<int>(), left.data_ptr<int>(), total.data_ptr<int>(),
                  granted.data_ptr<int>(), cu.data_ptr<int>(), slots.data_ptr<int>(), pos.data_ptr<int>(), rows, (int)B, Tq, page, P,
                  (int)width, pstride, c.stream);
  });
  return st == NE_OK ? wrap({total, got, left, cu, slots, pos, granted}) : status(st);
}

// k_new, v_new, k_pages, v_pages, slots, positions, capacity, k_weight, eps, rope_base, rope_half
PyObject* append(PyObject* const* a) {
  const Tensor &k = tensor(a[0], "k_new"), &v = tensor(a[1], "v_new");
  Call c(k, "k_new");
  need(k.dim() == 3 && v.sizes() == k.sizes(), "k_new and v_new must be [N, Hkv, D], of one shape");
  const long long ks = head_rows(k, "k_new", c.dev), vs = head_rows(v, "v_new", c.dev);
  const Pools p = pools(a[2], a[3], c.dev);
  need(p.heads == k.size(1) && p.D == k.size(2), "pools must be [num_pages, Hkv, page_size, D]");
  const int64_t N = k.size(0);
  need(N < (1LL << 31), "too many rows");
  const int *slots = ints(a[4], "slots", c.dev, {N}), *pos = ints(a[5], "positions", c.dev, {N});
  const void* w = weight(a[7], "k_weight", c.dev, p.D);
  if (N == 0) return status(NE_OK);
  const void *pk = k.data_ptr(), *pv = v.data_ptr();
  const int capacity = number(a[6]), flags = truth(a[10]) ? NE_ATTN_ROPE_HALF : 0;
  const float eps = real(a[8]), base = real(a[9]);
  return status(library([&] {
    return f_append(pk, pv, w, p.k, p.v, slots, pos, (int)N, p.heads, p.D, p.page, p.pages, capacity, p.stride, ks, vs, eps, base, flags,
                    c.stream);
  }));
}

// q, k_pages, v_pages, page_table, kv_len, parents, tree_len, q_weight, eps, rope_base, o, lse, fp32 of a new o, workspace,
// rope_half
PyObject* decode_tree(PyObject* const* a) {
  const Tensor& q = tensor(a[0], "q");
  Call c(q, "q");
  need(q.dim() == 4, "q must be [B, Tq, Hq, D]");
  const int64_t B = q.size(0), Tq = q.size(1), Hq = q.size(2), D = q.size(3);
  need(B < (1LL << 31) && Tq < (1LL << 31) && Hq < (1LL << 31), "q is too large");
  const long long qs = head_rows(q, "q", c.dev);
  const Pools p = pools(a[1], a[2], c.dev);
  need(p.D == D, "pools must be [num_pages, Hkv, page_size, D]");
  const Tensor& table = tensor(a[3], "page_table");
  need(table.dim() == 2 && table.size(1) < (1LL << 31), "page_table must be [B, max_pages]");
  const int *p_table = ints(table, "page_table", c.dev, {B, table.size(1)}), *len = ints(a[4], "kv_len", c.dev, {B});
  int n = 0;
  long long pstride = 0;
  const int* parents = tree(a[5], B, c.dev, &n, &pstride);
  need(n == Tq, "parents must have a token for each of q's");
  const int* nodes = given(a[6]) ? ints(a[6], "tree_len", c.dev, {B}) : nullptr;
  const void* w = weight(a[7], "q_weight", c.dev, D);
  Tensor o, lse;
  if (given(a[10])) {
    o = tensor(a[10], "o");
    need(o.device() == c.dev && o.is_contiguous() && o.sizes() == q.sizes() && (o.scalar_type() == kFloat || o.scalar_type() == kBf16),
         "o must be a contiguous bfloat16 or float32 [B, Tq, Hq, D] on the call's device");
  } else {
    o = make(q.sizes(), truth(a[12]) ? kFloat : kBf16, c.dev);
  }
  const int64_t shape[3] = {B, Hq, Tq};
  if (given(a[11])) {
    lse = tensor(a[11], "lse");
    need(lse.scalar_type() == kFloat && lse.device() == c.dev && lse.is_contiguous() && lse.sizes() == Sizes(shape, 3),
         "lse must be a contiguous float32 [B, Hq, Tq] on the call's device");
  } else {
    lse = make(Sizes(shape, 3), kFloat, c.dev);
  }
  const int flags = (o.scalar_type() == kFloat ? NE_ATTN_O_FP32 : 0) | (truth(a[14]) ? NE_ATTN_ROPE_HALF : 0);
  const float eps = real(a[8]), base = real(a[9]);
  const void* pq = q.data_ptr();
  const int width = (int)table.size(1);
  const auto call = [&](void* ws, size_t bytes) {
    return library([&] {
      return f_tree(pq, w, p.k, p.v, p_table, len, parents, nodes, o.data_ptr(), lse.data_ptr<float>(), (int)B, (int)Tq, (int)Hq, p.heads,
                    p.D, p.page, p.pages, width, p.stride, qs, pstride, eps, base, flags, ws, bytes, c.stream);
    });
  };
  int st;
  if (given(a[13])) {
    const Tensor& ws = tensor(a[13], "workspace");
    // its size is counted in numel(): an expanded tensor has more of those than bytes
    need(ws.scalar_type() == kByte && ws.device() == c.dev && ws.is_contiguous(), "workspace must be contiguous uint8 on the call's device");
    st = call(ws.data_ptr(), (size_t)ws.numel());
  } else {
    st = call(nullptr, 0);  // the library's own for the stream; a capture needs one of its own
    const size_t bytes = st == NE_ERR_WORKSPACE ? f_tree_size((int)B, (int)Tq, (int)Hq, p.heads, p.D) : 0;
    if (bytes > 0) {
      const Tensor ws = make({(int64_t)bytes}, kByte, c.dev);
      st = call(ws.data_ptr(), bytes);
    }
  }
  return st == NE_OK ? wrap({o, lse}) : status(st);
}

// k_pages, v_pages, page_table, kv_len, tree_len (a tensor or a number), path, path_len, kv_len_out
PyObject* keep(PyObject* const* a) {
  const Tensor& k = tensor(a[0], "k_pages");
  Call c(k, "k_pages");
  const Pools p = pools(a[0], a[1], c.dev);
  const Tensor &table = tensor(a[2], "page_table"), &path = tensor(a[5], "path");
  need(table.dim() == 2 && table.size(0) < (1LL << 31) && table.size(1) < (1LL << 31), "page_table must be [B, max_pages]");
  const int64_t B = table.size(0);
  need(path.dim() == 2 && path.size(1) < (1LL << 31), "path must be [B, width]");
  const int *p_table = ints(table, "page_table", c.dev, {B, table.size(1)}), *len = ints(a[3], "kv_len", c.dev, {B});
  const int *p_path = ints(path, "path", c.dev, {B, path.size(1)}), *count = ints(a[6], "path_len", c.dev, {B});
  const bool each = THPVariable_Check(a[4]);
  const int* nodes = each ? ints(a[4], "tree_len", c.dev, {B}) : nullptr;
  const Tensor out = out32(a[7], "kv_len_out", c.dev, {B});
  if (given(a[7])) apart(out, THPVariable_Unpack(a[3]), "kv_len_out and kv_len must not share memory");
  const int tokens = each ? 0 : number(a[4]), width = (int)path.size(1), max_pages = (int)table.size(1);
  const int st = library([&] {
    return f_keep(p.k, p.v, p_table, len, nodes, p_path, count, out.data_ptr<int>(), (int)B, tokens, width, p.heads, p.D, p.page, p.pages,
                  max_pages, p.stride, c.stream);
  });
  return st == NE_OK ? THPVariable_Wrap(out) : status(st);
}

// Every error leaves as a Python one: refusals as ValueError, out of memory as torch's own, the rest as RuntimeError.
template <PyObject* (*F)(PyObject* const*), int N>
PyObject* entry(PyObject*, PyObject* const* args, Py_ssize_t n) {
  if (n != N) {
    PyErr_SetString(PyExc_TypeError, "wrong number of arguments");
    return nullptr;
  }
  try {
    return F(args);
  } catch (const std::invalid_argument& e) {
    PyErr_SetString(PyExc_ValueError, e.what());
  } catch (const std::domain_error&) {  // a Python error that is set already
  } catch (const c10::OutOfMemoryError& e) {
    PyErr_SetString(out_of_memory, e.what_without_backtrace());
  } catch (const std::exception& e) {
    PyErr_SetString(PyExc_RuntimeError, e.what());
  } catch (abi::__forced_unwind&) {  // the thread ends
    throw;
  } catch (...) {
    PyErr_SetString(PyExc_RuntimeError, "unknown error");
  }
  return nullptr;
}

template <class F>
bool take(PyObject* d, const char* name, F* f) {
  PyObject* o = PyDict_GetItemString(d, name);  // borrowed
  void* p = o ? PyLong_AsVoidPtr(o) : nullptr;
  if (!p) {
    if (!PyErr_Occurred()) PyErr_Format(PyExc_KeyError, "no address of %s", name);
    return false;
  }
  *f = reinterpret_cast<F>(p);
  return true;
}
PyObject* init(PyObject*, PyObject* d) {
  if (!PyDict_Check(d)) {
    PyErr_SetString(PyExc_TypeError, "init takes a dict of addresses");
    return nullptr;
  }
  if (!take(d, "ne_attn_paged_plan_ex", &f_plan) || !take(d, "ne_attn_kv_append_slots", &f_append) ||
      !take(d, "ne_attn_decode_tree", &f_tree) || !take(d, "ne_attn_decode_tree_workspace_size", &f_tree_size) ||
      !take(d, "ne_attn_kv_keep_paged", &f_keep))
    return nullptr;
  PyObject* e = PyDict_GetItemString(d, "OutOfMemoryError");
  if (!e || !PyExceptionClass_Check(e)) {
    PyErr_SetString(PyExc_KeyError, "OutOfMemoryError");
    return nullptr;
  }
  Py_INCREF(e);
  out_of_memory = e;
  Py_RETURN_NONE;
}

#define FAST(f, n) reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(&entry<f, n>)), METH_FASTCALL, nullptr
PyMethodDef methods[] = {{"init", init, METH_O, nullptr},
                         {"plan", FAST(plan, 13)},
                         {"append", FAST(append, 11)},
                         {"decode_tree", FAST(decode_tree, 15)},
                         {"keep", FAST(keep, 8)},
                         {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_neattn_bind", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__neattn_bind(void) { return PyModule_Create(&module); }
