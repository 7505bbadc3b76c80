// binding.cpp -- the serving operators' path from torch tensors to the C entry points.
//
// A decode step calls these operators some hundred times, and each launch takes the
// host about 3 us; checking the tensors and filling the descriptors in Python took 7
// to 9 us more a call, here it takes about 1. Argument marshalling only: types, devices and
// shapes are checked here (ValueError), numbers by the C entry points (LutGemmError).
// The entry points are handed over by address (init), so this module follows the
// library that the package has loaded.
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <ATen/core/Tensor.h>
#include <ATen/ops/empty.h>
#include <c10/core/AutogradState.h>
#include <c10/hip/HIPGuard.h>
#include <c10/hip/HIPStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include <stdexcept>
#include <string>

#include "lutgemm.h"

namespace {

decltype(&lutgemm_qk_norm_rotate) g_heads;
decltype(&lutgemm_paged_attention) g_attention;
decltype(&lutgemm_paged_attention_workspace) g_attention_ws;
decltype(&lutgemm_adapters_add) g_adapters;
decltype(&lutgemm_adapters_workspace) g_adapters_ws;
PyObject* g_status_error;  // LutGemmError(status, where)

struct Refused : std::runtime_error {
  using std::runtime_error::runtime_error;
};
struct Status {
  int code;
  const char* where;
};
struct Raised {};  // a Python error is set already

[[noreturn]] void refuse(const std::string& what) { throw Refused(what); }

const at::Tensor& tensor(PyObject* o, const char* what) {
  if (!THPVariable_Check(o)) refuse(std::string(what) + " must be a tensor");
  return THPVariable_Unpack(o);
}

int64_t whole(PyObject* o) {
  const long long v = PyLong_AsLongLong(o);
  if (v == -1 && PyErr_Occurred()) throw Raised{};
  return v;
}

int32_t small(int64_t v, const char* what) {
  if (v < INT32_MIN || v > INT32_MAX) refuse(std::string(what) + " is out of range");
  return (int32_t)v;
}

double real(PyObject* o) {
  const double v = PyFloat_AsDouble(o);
  if (v == -1.0 && PyErr_Occurred()) throw Raised{};
  return v;
}

int type_of(const at::Tensor& t, const char* what) {
  if (t.scalar_type() == at::kHalf) return LUTGEMM_F16;
  if (t.scalar_type() == at::kBFloat16) return LUTGEMM_BF16;
  refuse(std::string(what) + " must be fp16 or bf16");
}

// The operators have no gradients: a graph that would silently end here is refused, and
// so is a forward-mode tangent, which torch.no_grad() does not switch off.
// Bit i of `which`: argument i is a tensor or None.
void no_gradient(PyObject* const* args, unsigned which) {
  const c10::AutogradState& state = c10::AutogradState::get_tls_state();
  const bool backward = state.get_grad_mode(), forward = state.get_fw_grad_mode();
  if (!backward && !forward) return;
  for (; which; which &= which - 1) {
    PyObject* const o = args[__builtin_ctz(which)];
    if (o == Py_None || !THPVariable_Check(o)) continue;
    const at::Tensor& t = THPVariable_Unpack(o);
    if (backward && t.requires_grad())
      refuse("the operator has no gradient: call it under torch.no_grad() or on detached tensors");
    if (forward && t._fw_grad(/*level=*/0).defined())
      refuse("the operator has no gradient: call it on the primals of dual tensors");
  }
}

void on_gpu(const at::Tensor& t, const char* what) {
  if (!t.is_cuda()) refuse(std::string(what) + " must be on a GPU");
}

// t: of ref's type, on its device, of so many dimensions, the last contiguous.
void like(const at::Tensor& t, const at::Tensor& ref, int64_t dims, const char* what) {
  if (t.scalar_type() != ref.scalar_type() || t.device() != ref.device() || t.dim() != dims)
    refuse(std::string(what) + " must be a tensor of " + std::to_string(dims) +
           " dimensions, of the first argument's type and on its device");
  if (t.stride(dims - 1) != 1 && t.size(dims - 1) > 1)
    refuse(std::string(what) + " must be contiguous in its last dimension");
}

// The stride of a dimension; of a single entry it is never walked.
int64_t step(const at::Tensor& t, int64_t d) { return t.size(d) == 1 ? 0 : t.stride(d); }

void* flat(const at::Tensor& t, at::ScalarType type, const at::Tensor& ref, at::IntArrayRef shape,
           const char* what) {
  if (t.scalar_type() != type || t.device() != ref.device() || t.sizes() != shape ||
      !t.is_contiguous()) {
    std::string want = "[";
    for (size_t i = 0; i < shape.size(); ++i)
      want += (i ? ", " : "") + std::to_string(shape[i]);
    refuse(std::string(what) + " must be contiguous " + c10::toString(type) + " " + want +
           "] on the first argument's device");
  }
  return t.data_ptr();
}

// Memory for one call, in the current stream's order; a graph being captured keeps
// its own.
at::Tensor scratch(size_t bytes, const at::Tensor& ref) {
  return at::empty({(int64_t)bytes}, ref.options().dtype(at::kByte));
}

// A tensor of the caller's has been written: autograd tells by its version that a copy
// kept for a backward pass is no longer what it was. Tensors of inference mode have none.
void written(const at::Tensor& t) {
  if (!t.is_inference()) t.unsafeGetTensorImpl()->bump_version();
}

void check(int status, const char* where) {
  if (status != LUTGEMM_OK) throw Status{status, where};
}

void* stream_of(const at::Tensor& t) {
  return (void*)c10::hip::getCurrentHIPStream(t.device().index()).stream();
}

PyObject* heads(PyObject* const* a) {
  const at::Tensor& qkv = tensor(a[0], "qkv");
  lutgemm_heads h{};
  h.type = type_of(qkv, "qkv");
  on_gpu(qkv, "qkv");
  like(qkv, qkv, 2, "qkv");
  h.heads = small(whole(a[1]), "heads");
  h.kv_heads = small(whole(a[2]), "kv_heads");
  const int64_t parts = (int64_t)h.heads + 2 * (int64_t)h.kv_heads;
  if (h.heads < 1 || h.kv_heads < 1 || qkv.size(1) % parts)
    refuse("qkv's rows do not divide into " + std::to_string(h.heads) + " + 2 x " +
           std::to_string(h.kv_heads) + " heads");
  const int64_t tokens = qkv.size(0), dim = qkv.size(1) / parts;
  h.head_dim = small(dim, "head_dim");
  h.tokens = tokens;
  h.qkv_token = step(qkv, 0);
  const c10::hip::HIPGuard guard(qkv.device().index());
  void *positions = nullptr, *table = nullptr, *qw = nullptr, *kw = nullptr;
  if (a[4] != Py_None) {
    const at::Tensor& t = tensor(a[4], "table");
    if (t.dim() != 2) refuse("table must be [positions][rotary]");
    table = flat(t, at::kFloat, qkv, t.sizes(), "table");
    if (a[3] == Py_None) refuse("a rotation needs the tokens' positions");
    positions = flat(tensor(a[3], "positions"), at::kLong, qkv, {tokens}, "positions");
    h.positions = t.size(0);
    h.rotary = small(t.size(1), "rotary");
  }
  if ((a[5] == Py_None) != (a[6] == Py_None)) refuse("q_weight and k_weight go together");
  if (a[5] != Py_None) {
    qw = flat(tensor(a[5], "q_weight"), qkv.scalar_type(), qkv, {dim}, "q_weight");
    kw = flat(tensor(a[6], "k_weight"), qkv.scalar_type(), qkv, {dim}, "k_weight");
  }
  h.eps = (float)real(a[7]);
  h.interleaved = PyObject_IsTrue(a[8]);
  if (h.interleaved < 0) throw Raised{};
  at::Tensor out;
  if (a[12] == Py_None) {
    out = at::empty({tokens, h.heads, dim}, qkv.options());
  } else {
    out = tensor(a[12], "out");
    like(out, qkv, 3, "out");
    if (out.size(0) != tokens || out.size(1) != h.heads || out.size(2) != dim ||
        (h.heads > 1 && out.stride(1) != dim))
      refuse("out must be [tokens][heads][head_dim] with its heads side by side");
  }
  h.q_token = step(out, 0);
  if ((a[9] == Py_None) != (a[11] == Py_None) || (a[10] == Py_None) != (a[11] == Py_None))
    refuse("k_pages, v_pages and slots go together");
  constexpr const char* where = "lutgemm_qk_norm_rotate";
  if (a[11] == Py_None) {
    const at::Tensor keys = at::empty({tokens, h.kv_heads, dim}, qkv.options());
    h.page_size = 1;
    h.k_page = h.kv_heads * dim;
    h.k_head = dim;
    check(g_heads(&h, qkv.data_ptr(), (const int64_t*)positions, (const float*)table, qw, kw,
                  out.data_ptr(), keys.data_ptr(), nullptr, nullptr, stream_of(qkv)),
          where);
    if (a[12] != Py_None) written(out);
    PyObject* first = THPVariable_Wrap(out);
    PyObject* second = THPVariable_Wrap(keys);
    PyObject* both = first && second ? PyTuple_Pack(2, first, second) : nullptr;
    Py_XDECREF(first);
    Py_XDECREF(second);
    return both;
  }
  const at::Tensor &k = tensor(a[9], "k_pages"), &v = tensor(a[10], "v_pages");
  like(k, qkv, 4, "k_pages");
  like(v, qkv, 4, "v_pages");
  if (k.size(2) != h.kv_heads || k.size(3) != dim || k.sizes() != v.sizes())
    refuse("k_pages and v_pages must both be [pages][page_size][" + std::to_string(h.kv_heads) +
           "][" + std::to_string(dim) + "]");
  h.pages = k.size(0);
  h.page_size = small(k.size(1), "page_size");
  h.k_page = step(k, 0);
  h.k_slot = step(k, 1);
  h.k_head = step(k, 2);
  h.v_page = step(v, 0);
  h.v_slot = step(v, 1);
  h.v_head = step(v, 2);
  const void* slots = flat(tensor(a[11], "slots"), at::kLong, qkv, {tokens}, "slots");
  if (tokens > 0)
    check(g_heads(&h, qkv.data_ptr(), (const int64_t*)positions, (const float*)table, qw, kw,
                  out.data_ptr(), k.data_ptr(), v.data_ptr(), (const int64_t*)slots,
                  stream_of(qkv)),
          where);
  written(k);
  written(v);
  if (a[12] != Py_None) written(out);
  return THPVariable_Wrap(out);
}

PyObject* attention(PyObject* const* a) {
  const at::Tensor& q = tensor(a[0], "q");
  lutgemm_attention d{};
  d.type = type_of(q, "q");
  on_gpu(q, "q");
  const at::Tensor &k = tensor(a[1], "k_pages"), &v = tensor(a[2], "v_pages");
  like(q, q, 3, "q");
  like(k, q, 4, "k_pages");
  like(v, q, 4, "v_pages");
  const int64_t tokens = q.size(0), heads = q.size(1), dim = q.size(2);
  if (k.size(3) != dim || k.sizes() != v.sizes())
    refuse("k_pages and v_pages must both be [pages][page_size][kv_heads][" + std::to_string(dim) +
           "]");
  const at::Tensor& table = tensor(a[3], "page_table");
  if (table.scalar_type() != at::kInt || table.device() != q.device() || table.dim() != 2 ||
      (table.size(1) > 1 && table.stride(1) != 1))
    refuse("page_table must be int32 [seqs][width] on q's device, contiguous in its last dimension");
  const int64_t seqs = table.size(0), width = table.size(1), page = k.size(1);
  const void* lens = flat(tensor(a[4], "kv_lens"), at::kInt, q, {seqs}, "kv_lens");
  const void* starts = nullptr;
  if (a[5] != Py_None)
    starts = flat(tensor(a[5], "q_starts"), at::kInt, q, {seqs + 1}, "q_starts");
  else if (tokens != seqs)
    refuse(std::to_string(tokens) + " tokens of " + std::to_string(seqs) +
           " sequences need q_starts");
  const c10::hip::HIPGuard guard(q.device().index());
  at::Tensor out;
  if (a[10] == Py_None) {
    out = at::empty({tokens, heads, dim}, q.options());
  } else {
    out = tensor(a[10], "out");
    like(out, q, 3, "out");
    if (out.sizes() != q.sizes()) refuse("out must have the shape of q");
  }
  d.heads = small(heads, "heads");
  d.kv_heads = small(k.size(2), "kv_heads");
  d.head_dim = small(dim, "head_dim");
  d.page_size = small(page, "page_size");
  d.seqs = small(seqs, "seqs");
  d.table_width = small(width, "the page table's width");
  d.window = small(whole(a[9]), "window");
  d.scale = a[8] == Py_None ? (float)(1.0 / std::sqrt((double)dim)) : (float)real(a[8]);
  d.tokens = tokens;
  d.pages = k.size(0);
  d.table_stride = step(table, 0);
  d.max_q = !starts ? 1 : a[6] == Py_None ? tokens : whole(a[6]);
  d.max_kv = a[7] == Py_None ? width * page : whole(a[7]);
  d.q_token = step(q, 0);
  d.q_head = step(q, 1);
  d.o_token = step(out, 0);
  d.o_head = step(out, 1);
  d.k_page = step(k, 0);
  d.k_slot = step(k, 1);
  d.k_head = step(k, 2);
  d.v_page = step(v, 0);
  d.v_slot = step(v, 1);
  d.v_head = step(v, 2);
  constexpr const char* where = "lutgemm_paged_attention";
  size_t need = 0;
  check(g_attention_ws(&d, &need), where);
  at::Tensor ws;
  if (need) ws = scratch(need, q);
  check(g_attention(&d, q.data_ptr(), k.data_ptr(), v.data_ptr(), (const int32_t*)table.data_ptr(),
                    (const int32_t*)lens, (const int32_t*)starts, out.data_ptr(),
                    need ? ws.data_ptr() : nullptr, need, stream_of(q)),
        where);
  if (a[10] != Py_None) written(out);
  return THPVariable_Wrap(out);
}

PyObject* adapters(PyObject* const* a) {
  const at::Tensor &y = tensor(a[0], "y"), &x = tensor(a[1], "x");
  lutgemm_adapters d{};
  d.type = type_of(x, "x");
  on_gpu(x, "x");
  like(x, x, 2, "x");
  like(y, x, 2, "y");
  const int64_t rows = x.size(0), K = x.size(1), N = y.size(1);
  if (y.size(0) != rows) refuse("x and y must have the same rows");
  const at::Tensor& first = tensor(a[2], "a");
  if (first.dim() != 3) refuse("a must be [adapters][rank][K]");
  const int64_t count = first.size(0), rank = first.size(1);
  const void* pa = flat(first, x.scalar_type(), x, {count, rank, K}, "a");
  const void* pb = flat(tensor(a[3], "b"), x.scalar_type(), x, {count, N, rank}, "b");
  const void* ids = flat(tensor(a[4], "ids"), at::kInt, x, {rows}, "ids");
  const void* scales = nullptr;
  if (a[5] != Py_None) scales = flat(tensor(a[5], "scales"), at::kFloat, x, {count}, "scales");
  const c10::hip::HIPGuard guard(x.device().index());
  at::Tensor out;
  if (a[6] == Py_None) {
    out = at::empty({rows, N}, x.options());
  } else {
    out = tensor(a[6], "out");
    like(out, x, 2, "out");
    if (out.sizes() != y.sizes()) refuse("out must have the shape of y");
  }
  d.rows = small(rows, "rows");
  d.K = small(K, "K");
  d.N = small(N, "N");
  d.rank = small(rank, "rank");
  d.adapters = small(count, "adapters");
  d.x_row = K ? step(x, 0) : 0;  // rows of no entries have any stride
  d.y_row = step(y, 0);
  d.out_row = step(out, 0);
  constexpr const char* where = "lutgemm_adapters_add";
  size_t need = 0;
  check(g_adapters_ws(&d, &need), where);
  at::Tensor ws;
  if (need) ws = scratch(need, x);
  check(g_adapters(&d, x.data_ptr(), y.data_ptr(), pa, pb, (const float*)scales,
                   (const int32_t*)ids, out.data_ptr(), need ? ws.data_ptr() : nullptr, need,
                   stream_of(x)),
        where);
  if (a[6] != Py_None) written(out);
  return THPVariable_Wrap(out);
}

// One call: so many arguments, those of `Tensors` tensors or None, and every C++ exception
// as a Python error.
template <PyObject* (*F)(PyObject* const*), Py_ssize_t N, unsigned Tensors>
PyObject* entry(PyObject*, PyObject* const* args, Py_ssize_t n) {
  if (n != N) {
    PyErr_Format(PyExc_TypeError, "%zd arguments expected, not %zd", N, n);
    return nullptr;
  }
  if (!g_heads) {
    PyErr_SetString(PyExc_RuntimeError, "the library is not bound");
    return nullptr;
  }
  try {
    no_gradient(args, Tensors);
    return F(args);
  } catch (const Refused& e) {
    PyErr_SetString(PyExc_ValueError, e.what());
  } catch (const Status& s) {
    PyObject* value = PyObject_CallFunction(g_status_error, "is", s.code, s.where);
    if (value) {
      PyErr_SetObject(g_status_error, value);
      Py_DECREF(value);
    }
  } catch (const Raised&) {
  } catch (const c10::OutOfMemoryError& e) {
    PyErr_SetString(PyExc_MemoryError, e.what_without_backtrace());
  } catch (const c10::Error& e) {
    PyErr_SetString(PyExc_RuntimeError, e.what_without_backtrace());
  } catch (const std::exception& e) {
    PyErr_SetString(PyExc_RuntimeError, e.what());
  }
  return nullptr;
}

// init(addresses of the five entry points, LutGemmError)
PyObject* init(PyObject*, PyObject* args) {
  unsigned long long f[5];
  PyObject* error;
  if (!PyArg_ParseTuple(args, "KKKKKO", &f[0], &f[1], &f[2], &f[3], &f[4], &error)) return nullptr;
  g_attention = (decltype(g_attention))f[1];
  g_attention_ws = (decltype(g_attention_ws))f[2];
  g_adapters = (decltype(g_adapters))f[3];
  g_adapters_ws = (decltype(g_adapters_ws))f[4];
  Py_INCREF(error);
  Py_XSETREF(g_status_error, error);
  g_heads = (decltype(g_heads))f[0];
  Py_RETURN_NONE;
}

PyMethodDef kMethods[] = {
    {"init", init, METH_VARARGS, nullptr},
    {"qk_norm_rotate", (PyCFunction)(void*)entry<heads, 13, 0x1671>, METH_FASTCALL, nullptr},
    {"paged_attention", (PyCFunction)(void*)entry<attention, 11, 0x407>, METH_FASTCALL, nullptr},
    {"adapters_add", (PyCFunction)(void*)entry<adapters, 7, 0x6F>, METH_FASTCALL, nullptr},
    {nullptr, nullptr, 0, nullptr}};

PyModuleDef kModule = {PyModuleDef_HEAD_INIT, "_binding", nullptr, -1, kMethods,
                       nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__binding(void) { return PyModule_Create(&kModule); }
