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
decltype(&lutgemm_shared_attention) g_shared;
decltype(&lutgemm_shared_attention_workspace) g_shared_ws;
decltype(&lutgemm_batch_tables) g_tables;
decltype(&lutgemm_batch_tables_workspace) g_tables_ws;
decltype(&lutgemm_sample_tokens) g_sample;
decltype(&lutgemm_sample_tokens_workspace) g_sample_ws;
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

// A vector of `n` entries at `offset` bytes (a multiple of their size) in an allocation's
// storage: small results of one call share one, an allocation each costs the host 0.8 us.
at::Tensor part_of(const at::Tensor& base, at::ScalarType type, int64_t offset, int64_t n) {
  const caffe2::TypeMeta meta = c10::scalarTypeToTypeMeta(type);
  at::Tensor t = at::detail::make_tensor<c10::TensorImpl>(c10::Storage(base.storage()),
                                                          base.key_set(), meta);
  c10::TensorImpl* const impl = t.unsafeGetTensorImpl();
  impl->set_storage_offset(offset / (int64_t)meta.itemsize());
  impl->set_sizes_contiguous({n});
  return t;
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

// A page table: int32 [rows][width], rows apart.
const at::Tensor& page_table(PyObject* o, const at::Tensor& ref, const char* what) {
  const at::Tensor& t = tensor(o, what);
  if (t.scalar_type() != at::kInt || t.device() != ref.device() || t.dim() != 2 ||
      (t.size(1) > 1 && t.stride(1) != 1))
    refuse(std::string(what) + " must be int32 [rows][width] on the first argument's device, "
                               "contiguous in its last dimension");
  return t;
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
  const at::Tensor& table = page_table(a[3], q, "page_table");
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

PyObject* shared(PyObject* const* a) {
  const at::Tensor& q = tensor(a[0], "q");
  lutgemm_shared d{};
  d.own.type = type_of(q, "q");
  on_gpu(q, "q");
  const at::Tensor &k = tensor(a[1], "k_pages"), &v = tensor(a[2], "v_pages");
  like(q, q, 3, "q");
  like(k, q, 4, "k_pages");
  like(v, q, 4, "v_pages");
  const int64_t tokens = q.size(0), heads = q.size(1), dim = q.size(2);
  if (k.size(3) != dim || k.sizes() != v.sizes())
    refuse("k_pages and v_pages must both be [pages][page_size][kv_heads][" + std::to_string(dim) +
           "]");
  const at::Tensor& prefix = page_table(a[3], q, "prefix_table");
  const int64_t groups = prefix.size(0);
  const void* prefix_lens = flat(tensor(a[4], "prefix_lens"), at::kInt, q, {groups}, "prefix_lens");
  const at::Tensor& table = page_table(a[5], q, "page_table");
  const int64_t seqs = table.size(0), width = table.size(1), page = k.size(1);
  const void* lens = flat(tensor(a[6], "kv_lens"), at::kInt, q, {seqs}, "kv_lens");
  const void *starts = nullptr, *group_starts = nullptr;
  if (a[7] != Py_None)
    starts = flat(tensor(a[7], "q_starts"), at::kInt, q, {seqs + 1}, "q_starts");
  else if (tokens != seqs)
    refuse(std::to_string(tokens) + " tokens of " + std::to_string(seqs) +
           " sequences need q_starts");
  if (a[8] != Py_None)
    group_starts = flat(tensor(a[8], "group_starts"), at::kInt, q, {groups + 1}, "group_starts");
  else if (groups > 1)
    refuse(std::to_string(groups) + " groups need group_starts");
  const c10::hip::HIPGuard guard(q.device().index());
  at::Tensor out;
  if (a[13] == Py_None) {
    out = at::empty({tokens, heads, dim}, q.options());
  } else {
    out = tensor(a[13], "out");
    like(out, q, 3, "out");
    if (out.sizes() != q.sizes()) refuse("out must have the shape of q");
  }
  d.own.heads = small(heads, "heads");
  d.own.kv_heads = small(k.size(2), "kv_heads");
  d.own.head_dim = small(dim, "head_dim");
  d.own.page_size = small(page, "page_size");
  d.own.seqs = small(seqs, "seqs");
  d.own.table_width = small(width, "the page table's width");
  d.own.scale = a[12] == Py_None ? (float)(1.0 / std::sqrt((double)dim)) : (float)real(a[12]);
  d.own.tokens = tokens;
  d.own.pages = k.size(0);
  d.own.table_stride = step(table, 0);
  d.own.max_q = !starts ? 1 : a[9] == Py_None ? tokens : whole(a[9]);
  d.own.max_kv = a[10] == Py_None ? width * page : whole(a[10]);
  d.own.q_token = step(q, 0);
  d.own.q_head = step(q, 1);
  d.own.o_token = step(out, 0);
  d.own.o_head = step(out, 1);
  d.own.k_page = step(k, 0);
  d.own.k_slot = step(k, 1);
  d.own.k_head = step(k, 2);
  d.own.v_page = step(v, 0);
  d.own.v_slot = step(v, 1);
  d.own.v_head = step(v, 2);
  d.groups = small(groups, "groups");
  d.prefix_width = small(prefix.size(1), "the prefix table's width");
  d.prefix_stride = step(prefix, 0);
  d.max_prefix = a[11] == Py_None ? prefix.size(1) * page : whole(a[11]);
  constexpr const char* where = "lutgemm_shared_attention";
  size_t need = 0;
  check(g_shared_ws(&d, &need), where);
  at::Tensor ws;
  if (need) ws = scratch(need, q);
  check(g_shared(&d, q.data_ptr(), k.data_ptr(), v.data_ptr(), (const int32_t*)prefix.data_ptr(),
                 (const int32_t*)prefix_lens, (const int32_t*)group_starts,
                 (const int32_t*)table.data_ptr(), (const int32_t*)lens, (const int32_t*)starts,
                 out.data_ptr(), need ? ws.data_ptr() : nullptr, need, stream_of(q)),
        where);
  if (a[13] != Py_None) written(out);
  return THPVariable_Wrap(out);
}

// The tensors as a tuple.
template <size_t N>
PyObject* tuple_of(const at::Tensor (&all)[N]) {
  PyObject* t = PyTuple_New(N);
  for (size_t i = 0; t && i < N; ++i) {
    PyObject* one = THPVariable_Wrap(all[i]);
    if (!one) {
      Py_DECREF(t);
      return nullptr;
    }
    PyTuple_SET_ITEM(t, i, one);
  }
  return t;
}

PyObject* tables(PyObject* const* a) {
  const at::Tensor &change = tensor(a[0], "change"), &lens = tensor(a[1], "kv_lens");
  on_gpu(change, "change");
  const int64_t seqs = change.numel();
  lutgemm_tables d{};
  d.seqs = small(seqs, "seqs");
  const void* pc = flat(change, at::kInt, change, {seqs}, "change");
  void* pl = flat(lens, at::kInt, change, {seqs}, "kv_lens");
  const at::Tensor& table = page_table(a[2], change, "page_table");
  if (table.size(0) != seqs) refuse("page_table must have a row for each sequence");
  d.page_size = small(whole(a[3]), "page_size");
  d.tokens = whole(a[4]);
  if (d.tokens < 0) refuse("tokens must not be negative");
  d.table_width = small(table.size(1), "the page table's width");
  d.table_stride = seqs > 1 ? table.stride(0) : 0;
  if ((a[5] == Py_None) != (a[6] == Py_None)) refuse("free_pages and free_range go together");
  void *ring = nullptr, *range = nullptr, *range_out = nullptr;
  const c10::hip::HIPGuard guard(change.device().index());
  at::Tensor got[5];  // positions, slots, lengths, starts, range
  if (a[5] != Py_None) {
    const at::Tensor& t = tensor(a[5], "free_pages");
    if (t.dim() != 1 || t.numel() < 1) refuse("free_pages must be [capacity]");
    d.capacity = small(t.numel(), "free_pages' length");
    ring = flat(t, at::kInt, change, t.sizes(), "free_pages");
    range = flat(tensor(a[6], "free_range"), at::kInt, change, {2}, "free_range");
  }
  const void* offsets = nullptr;
  if (a[7] != Py_None) offsets = flat(tensor(a[7], "offsets"), at::kInt, change, {seqs}, "offsets");
  const int in_place = PyObject_IsTrue(a[8]);
  if (in_place < 0) throw Raised{};
  constexpr const char* where = "lutgemm_batch_tables";
  size_t need = 0;
  check(g_tables_ws(&d, &need), where);
  const int64_t rows8 = 8 * d.tokens;
  const at::Tensor all = scratch(2 * rows8 + 4 * (seqs + (seqs + 1) + 2), change);
  got[0] = part_of(all, at::kLong, 0, d.tokens);
  got[1] = part_of(all, at::kLong, rows8, d.tokens);
  got[2] = in_place ? lens : part_of(all, at::kInt, 2 * rows8, seqs);
  got[3] = part_of(all, at::kInt, 2 * rows8 + 4 * seqs, seqs + 1);
  if (range) {
    got[4] = in_place ? tensor(a[6], "free_range")
                      : part_of(all, at::kInt, 2 * rows8 + 4 * (2 * seqs + 1), 2);
    range_out = got[4].data_ptr();
  }
  at::Tensor ws;
  if (need) ws = scratch(need, change);
  check(g_tables(&d, (const int32_t*)pc, (const int32_t*)pl, (const int32_t*)offsets,
                 (int32_t*)table.data_ptr(), (int32_t*)ring, (const int32_t*)range,
                 (int64_t*)got[0].data_ptr(), (int64_t*)got[1].data_ptr(), (int32_t*)got[2].data_ptr(),
                 (int32_t*)got[3].data_ptr(), (int32_t*)range_out, need ? ws.data_ptr() : nullptr, need,
                 stream_of(change)),
        where);
  if (ring) {
    written(table);
    written(tensor(a[5], "free_pages"));
  }
  if (in_place) {
    written(lens);
    if (range) written(got[4]);
  }
  if (range) return tuple_of(got);
  PyObject* four[4] = {};
  bool made = true;
  for (int i = 0; i < 4; ++i) made &= (four[i] = THPVariable_Wrap(got[i])) != nullptr;
  PyObject* t = made ? PyTuple_Pack(5, four[0], four[1], four[2], four[3], Py_None) : nullptr;
  for (PyObject* o : four) Py_XDECREF(o);
  return t;
}

PyObject* sample(PyObject* const* a) {
  const at::Tensor& x = tensor(a[0], "logits");
  lutgemm_sample d{};
  if (x.scalar_type() == at::kFloat)
    d.type = LUTGEMM_F32;
  else if (x.scalar_type() == at::kHalf || x.scalar_type() == at::kBFloat16)
    d.type = type_of(x, "logits");
  else
    refuse("logits must be fp16, bf16 or fp32");
  on_gpu(x, "logits");
  like(x, x, 2, "logits");
  const int64_t rows = x.size(0);
  d.rows = small(rows, "rows");
  d.vocab = small(x.size(1), "the vocabulary");
  d.row_step = step(x, 0);
  const void* u = flat(tensor(a[1], "u"), at::kFloat, x, {rows}, "u");
  auto setting = [&](int i, at::ScalarType type, const char* what) -> const void* {
    return a[i] == Py_None ? nullptr : flat(tensor(a[i], what), type, x, {rows}, what);
  };
  const void* temperature = setting(2, at::kFloat, "temperature");
  const void* top_k = setting(3, at::kInt, "top_k");
  const void* top_p = setting(4, at::kFloat, "top_p");
  const void* min_p = setting(5, at::kFloat, "min_p");
  const c10::hip::HIPGuard guard(x.device().index());
  at::Tensor got[2];
  const at::Tensor all = scratch(12 * rows, x);
  if (a[6] == Py_None) {
    got[0] = part_of(all, at::kLong, 0, rows);
  } else {
    got[0] = tensor(a[6], "out");
    flat(got[0], at::kLong, x, {rows}, "out");
  }
  got[1] = part_of(all, at::kFloat, 8 * rows, rows);
  constexpr const char* where = "lutgemm_sample_tokens";
  size_t need = 0;
  check(g_sample_ws(&d, &need), where);
  at::Tensor ws;
  if (need) ws = scratch(need, x);
  check(g_sample(&d, x.data_ptr(), (const float*)u, (const float*)temperature, (const int32_t*)top_k,
                 (const float*)top_p, (const float*)min_p, (int64_t*)got[0].data_ptr(),
                 (float*)got[1].data_ptr(), need ? ws.data_ptr() : nullptr, need, stream_of(x)),
        where);
  if (a[6] != Py_None) written(got[0]);
  return tuple_of(got);
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

// init(addresses of the entry points, in the order in which they are bound here, LutGemmError)
PyObject* init(PyObject*, PyObject* args) {
  constexpr Py_ssize_t kPoints = 11;
  if (PyTuple_GET_SIZE(args) != kPoints + 1) {
    PyErr_SetString(PyExc_TypeError, "init takes the entry points' addresses and an exception");
    return nullptr;
  }
  void* f[kPoints];
  for (Py_ssize_t i = 0; i < kPoints; ++i) {
    f[i] = PyLong_AsVoidPtr(PyTuple_GET_ITEM(args, i));
    if (!f[i] && PyErr_Occurred()) return nullptr;
  }
  g_attention = (decltype(g_attention))f[1];
  g_attention_ws = (decltype(g_attention_ws))f[2];
  g_adapters = (decltype(g_adapters))f[3];
  g_adapters_ws = (decltype(g_adapters_ws))f[4];
  g_shared = (decltype(g_shared))f[5];
  g_shared_ws = (decltype(g_shared_ws))f[6];
  g_tables = (decltype(g_tables))f[7];
  g_tables_ws = (decltype(g_tables_ws))f[8];
  g_sample = (decltype(g_sample))f[9];
  g_sample_ws = (decltype(g_sample_ws))f[10];
  PyObject* error = PyTuple_GET_ITEM(args, kPoints);
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
    {"shared_prefix_attention", (PyCFunction)(void*)entry<shared, 14, 0x2007>, METH_FASTCALL, nullptr},
    {"batch_tables", (PyCFunction)(void*)entry<tables, 9, 0x0>, METH_FASTCALL, nullptr},
    {"sample_tokens", (PyCFunction)(void*)entry<sample, 7, 0x37>, METH_FASTCALL, nullptr},
    {nullptr, nullptr, 0, nullptr}};

PyModuleDef kModule = {PyModuleDef_HEAD_INIT, "_binding", nullptr, -1, kMethods,
                       nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__binding(void) { return PyModule_Create(&kModule); }
