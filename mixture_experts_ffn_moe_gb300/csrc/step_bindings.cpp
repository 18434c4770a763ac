// Python binding of the decode-step operators: checks tensors, allocates outputs and fills the C ABI's arguments.
//
// A decode step makes many calls of a few microseconds, and marshalling them in Python (ctypes and torch calls) took
// 8 to 17 us each on GB300's host cores; here it takes the launch and little more.  Marshalling only, as in
// gbmoe.py: every step runs in the library's kernels, whose entry points init() is given.
#include <Python.h>

#include <ATen/ATen.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include <initializer_list>
#include <stdexcept>
#include <string>

#include "gbmoe.h"

namespace {

decltype(&moe_rope) g_rope;
decltype(&moe_linear_int4) g_linear;
decltype(&moe_linear_int4_workspace_size) g_linear_workspace;
decltype(&moe_tree_attention) g_tree;
decltype(&moe_tree_attention_workspace_size) g_tree_workspace;
decltype(&moe_verify_draft) g_verify;

using at::Tensor;

[[noreturn]] void bad(const std::string& what) { throw std::invalid_argument(what); }

bool given(PyObject* o) { return o != Py_None; }
const Tensor& tensor(PyObject* o, const char* name) {
  if (!THPVariable_Check(o)) bad(std::string(name) + " must be a tensor");
  return THPVariable_Unpack(o);
}
bool truth(PyObject* o) {
  const int r = PyObject_IsTrue(o);
  if (r < 0) bad("a flag has no truth value");
  return r != 0;
}
double number(PyObject* o) {
  const double v = PyFloat_AsDouble(o);
  if (v == -1.0 && PyErr_Occurred()) bad("a factor is no number");
  return v;
}
int integer(PyObject* o) {
  const long v = PyLong_AsLong(o);
  if ((v == -1 && PyErr_Occurred()) || v < INT_MIN || v > INT_MAX) bad("a size is no integer of 32 bits");
  return static_cast<int>(v);
}

std::string text(c10::IntArrayRef s) {
  std::string r = "[";
  for (size_t i = 0; i < s.size(); ++i) r += (i ? ", " : "") + std::to_string(s[i]);
  return r + "]";
}

// A CUDA tensor on `device` (of the first tensor where device is null), of this type and shape (-1: any size), whose
// last dimension is contiguous, or all of it.
enum Layout { kRows, kContiguous };
void check(const Tensor& t, const at::Device* device, at::ScalarType type, std::initializer_list<int64_t> shape, const char* name, Layout layout) {
  const std::string n(name);
  if (!t.is_cuda()) bad(n + " must be a CUDA tensor");
  if (device && t.device() != *device) bad(n + " must be on the device of the other tensors");
  if (t.scalar_type() != type) bad(n + " must be " + c10::toString(type) + ", got " + c10::toString(t.scalar_type()));
  bool same = t.dim() == static_cast<int64_t>(shape.size());
  if (same) {
    int64_t i = 0;
    for (int64_t s : shape) {
      same = same && (s < 0 || t.size(i) == s);
      ++i;
    }
  }
  if (!same) {
    std::string want = "[";
    for (int64_t s : shape) want += (want.size() > 1 ? ", " : "") + (s < 0 ? std::string("any") : std::to_string(s));
    bad(n + " has the shape " + text(t.sizes()) + ", expected " + want + "]");
  }
  if (layout == kContiguous ? !t.is_contiguous() : t.dim() > 0 && t.size(-1) > 1 && t.stride(-1) != 1)
    bad(n + (layout == kContiguous ? " must be contiguous" : " must have a contiguous last dimension"));
}

int dtype_code(const Tensor& t, const char* name, bool fp32) {
  if (!t.is_cuda()) bad(std::string(name) + " must be a CUDA tensor");
  switch (t.scalar_type()) {
    case at::kBFloat16: return MOE_DTYPE_BF16;
    case at::kHalf: return MOE_DTYPE_FP16;
    case at::kFloat:
      if (fp32) return MOE_DTYPE_FP32;
      break;
    default: break;
  }
  bad(std::string(name) + " has an unsupported type " + c10::toString(t.scalar_type()));
}

int as_int(int64_t v, const char* name) {
  if (v > INT_MAX) bad(std::string(name) + " is too large");
  return static_cast<int>(v);
}
// The row stride of a matrix: what its tensor says wherever it has rows to step between (the C ABI refuses rows that
// overlap, such as a broadcast row's stride of 0); of one row or none any stride stands, and its length is given.
int64_t row_stride(const Tensor& t) { return t.size(0) > 1 ? t.stride(0) : t.size(1); }
template <typename T> T* ptr(const Tensor& t) { return static_cast<T*>(t.data_ptr()); }
moe_stream_t stream_of(const Tensor& t) {
  return reinterpret_cast<moe_stream_t>(c10::cuda::getCurrentCUDAStream(t.device().index()).stream());
}
Tensor new_like(const Tensor& t, at::IntArrayRef shape, at::ScalarType type) { return at::empty(shape, t.options().dtype(type)); }

PyObject* status(moe_status_t s) { return PyLong_FromLong(s); }

// Runs a binding: invalid arguments become ValueError, everything else RuntimeError.
template <typename F> PyObject* bind(Py_ssize_t got, Py_ssize_t want, F&& body) {
  if (got != want) {
    PyErr_Format(PyExc_TypeError, "expected %zd arguments, got %zd", want, got);
    return nullptr;
  }
  try {
    return body();
  } catch (const std::invalid_argument& e) {
    PyErr_SetString(PyExc_ValueError, e.what());
  } catch (const c10::Error& e) {
    PyErr_SetString(PyExc_RuntimeError, e.what_without_backtrace());
  } catch (const std::exception& e) {
    PyErr_SetString(PyExc_RuntimeError, e.what());
  }
  return nullptr;
}

// The positions, frequencies, q and k of either rope call.
moe_rope_args_t rope_args(const Tensor& q, const Tensor& positions, const Tensor& inv_freq, PyObject* const* a) {
  moe_rope_args_t r{};
  r.dtype = dtype_code(q, "q", true);
  const at::Device dev = q.device();
  check(q, nullptr, q.scalar_type(), {-1, -1, -1}, "q", kRows);
  check(positions, &dev, at::kInt, {q.size(0)}, "positions", kContiguous);
  check(inv_freq, &dev, at::kDouble, {-1}, "inv_freq", kContiguous);
  r.tokens = as_int(q.size(0), "q");
  r.q_heads = as_int(q.size(1), "q");
  r.dim = as_int(q.size(2), "q");
  r.rot_dim = 2 * as_int(inv_freq.numel() < (1 << 20) ? inv_freq.numel() : 1 << 20, "inv_freq");
  r.scale = static_cast<float>(number(a[0]));
  r.interleaved = truth(a[1]);
  r.inverse = truth(a[2]);
  r.rot_offset = integer(a[3]);
  r.positions = ptr<int32_t>(positions);
  r.inv_freq = ptr<double>(inv_freq);
  r.q = q.data_ptr();
  r.q_stride_t = q.stride(0);
  r.q_stride_h = q.stride(1);
  return r;
}

// rope(q, k, positions, inv_freq, scale, interleaved, inverse, offset, q_out, k_out) -> (q_out, k_out) or a status
PyObject* rope(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return bind(n, 10, [&]() -> PyObject* {
    const Tensor& q = tensor(a[0], "q");
    moe_rope_args_t r = rope_args(q, tensor(a[2], "positions"), tensor(a[3], "inv_freq"), a + 4);
    const at::Device dev = q.device();
    Tensor q_out = given(a[8]) ? tensor(a[8], "q_out") : new_like(q, q.sizes(), q.scalar_type()), k_out;
    check(q_out, &dev, q.scalar_type(), {q.size(0), q.size(1), q.size(2)}, "q_out", kRows);
    r.q_out = q_out.data_ptr();
    r.q_out_stride_t = q_out.stride(0);
    r.q_out_stride_h = q_out.stride(1);
    if (given(a[1])) {
      const Tensor& k = tensor(a[1], "k");
      check(k, &dev, q.scalar_type(), {q.size(0), -1, q.size(2)}, "k", kRows);
      k_out = given(a[9]) ? tensor(a[9], "k_out") : new_like(k, k.sizes(), k.scalar_type());
      check(k_out, &dev, q.scalar_type(), {q.size(0), k.size(1), q.size(2)}, "k_out", kRows);
      r.k_heads = as_int(k.size(1), "k");
      r.k = k.data_ptr();
      r.k_stride_t = k.stride(0);
      r.k_stride_h = k.stride(1);
      r.k_out = k_out.data_ptr();
      r.k_out_stride_t = k_out.stride(0);
      r.k_out_stride_h = k_out.stride(1);
    }
    if (const moe_status_t s = g_rope(&r, stream_of(q))) return status(s);
    PyObject* ko = k_out.defined() ? THPVariable_Wrap(std::move(k_out)) : Py_NewRef(Py_None);
    return Py_BuildValue("(NN)", THPVariable_Wrap(std::move(q_out)), ko);
  });
}

// rope_append(q, k, v, positions, inv_freq, slots, k_cache, v_cache, scale, interleaved, inverse, offset, q_out)
PyObject* rope_append(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return bind(n, 13, [&]() -> PyObject* {
    const Tensor &q = tensor(a[0], "q"), &k = tensor(a[1], "k"), &v = tensor(a[2], "v"), &slots = tensor(a[5], "slots");
    const Tensor &kc = tensor(a[6], "k_cache"), &vc = tensor(a[7], "v_cache");
    moe_rope_args_t r = rope_args(q, tensor(a[3], "positions"), tensor(a[4], "inv_freq"), a + 8);
    const at::Device dev = q.device();
    const at::ScalarType type = q.scalar_type();
    check(k, &dev, type, {q.size(0), -1, q.size(2)}, "k", kRows);
    check(v, &dev, type, {q.size(0), k.size(1), q.size(2)}, "v", kRows);
    check(kc, &dev, type, {-1, -1, k.size(1), q.size(2)}, "k_cache", kRows);
    check(vc, &dev, type, {kc.size(0), kc.size(1), k.size(1), q.size(2)}, "v_cache", kRows);
    check(slots, &dev, at::kInt, {q.size(0)}, "slots", kContiguous);
    Tensor q_out = given(a[12]) ? tensor(a[12], "q_out") : new_like(q, q.sizes(), type);
    check(q_out, &dev, type, {q.size(0), q.size(1), q.size(2)}, "q_out", kRows);
    r.k_heads = as_int(k.size(1), "k");
    r.num_pages = as_int(kc.size(0), "k_cache");
    r.page_size = as_int(kc.size(1), "k_cache");
    r.slots = ptr<int32_t>(slots);
    r.k = k.data_ptr();
    r.v = v.data_ptr();
    r.q_out = q_out.data_ptr();
    r.k_out = kc.data_ptr();
    r.v_cache = vc.data_ptr();
    r.k_stride_t = k.stride(0);
    r.k_stride_h = k.stride(1);
    r.v_stride_t = v.stride(0);
    r.v_stride_h = v.stride(1);
    r.q_out_stride_t = q_out.stride(0);
    r.q_out_stride_h = q_out.stride(1);
    r.k_page_stride = kc.stride(0);
    r.k_out_stride_t = kc.stride(1);
    r.k_out_stride_h = kc.stride(2);
    r.v_page_stride = vc.stride(0);
    r.v_slot_stride = vc.stride(1);
    r.v_head_stride = vc.stride(2);
    if (const moe_status_t s = g_rope(&r, stream_of(q))) return status(s);
    return THPVariable_Wrap(std::move(q_out));
  });
}

// linear_int4(x, w, w_scale, gated, out, workspace)
PyObject* linear_int4(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return bind(n, 6, [&]() -> PyObject* {
    const Tensor &x = tensor(a[0], "x"), &w = tensor(a[1], "w"), &s = tensor(a[2], "w_scale");
    const bool gated = truth(a[3]);
    const int dtype = dtype_code(x, "x", false);
    const at::Device dev = x.device();
    check(x, nullptr, x.scalar_type(), {-1, -1}, "x", kRows);
    const int64_t M = x.size(0), K = x.size(1);
    check(w, &dev, at::kByte, {-1, K / 2}, "w", kContiguous);
    check(s, &dev, at::kFloat, {w.size(0), -1}, "w_scale", kContiguous);
    const int64_t rows = w.size(0), groups = s.size(1);
    if (K % 2 || groups == 0 || K % groups || (gated && rows % 2)) bad("inconsistent shapes");
    const int64_t N = gated ? rows / 2 : rows, group = K / groups;
    Tensor out = given(a[4]) ? tensor(a[4], "out") : new_like(x, {M, N}, x.scalar_type()), ws;
    check(out, &dev, x.scalar_type(), {M, N}, "out", kRows);
    if (given(a[5])) {
      ws = tensor(a[5], "workspace");
      check(ws, &dev, at::kByte, {-1}, "workspace", kContiguous);
    } else if (M > 8 || K > 8192) {
      const size_t need = g_linear_workspace(as_int(M, "x"), as_int(N, "w"), as_int(K, "x"), as_int(group, "x"), gated);
      if (need) ws = new_like(x, {static_cast<int64_t>(need)}, at::kByte);
    }
    if (const moe_status_t st = g_linear(dtype, x.data_ptr(), row_stride(x), ptr<uint8_t>(w), ptr<float>(s), as_int(M, "x"),
                                         as_int(N, "w"), as_int(K, "x"), as_int(group, "x"), gated, out.data_ptr(), row_stride(out),
                                         ws.defined() ? ws.data_ptr() : nullptr, ws.defined() ? ws.numel() : 0, stream_of(x)))
      return status(st);
    return THPVariable_Wrap(std::move(out));
  });
}

// tree_attention(q, k_cache, v_cache, block_table, context_lens, node_offsets, tree_mask, scale, out, workspace)
PyObject* tree_attention(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return bind(n, 10, [&]() -> PyObject* {
    const Tensor &q = tensor(a[0], "q"), &kc = tensor(a[1], "k_cache"), &vc = tensor(a[2], "v_cache"), &table = tensor(a[3], "block_table");
    const Tensor &lens = tensor(a[4], "context_lens"), &offs = tensor(a[5], "node_offsets");
    moe_tree_attention_args_t r{};
    r.dtype = dtype_code(q, "q", false);
    const at::Device dev = q.device();
    const at::ScalarType type = q.scalar_type();
    check(q, nullptr, type, {-1, -1, -1}, "q", kRows);
    check(kc, &dev, type, {-1, -1, -1, q.size(2)}, "k_cache", kRows);
    check(vc, &dev, type, {kc.size(0), kc.size(1), kc.size(2), q.size(2)}, "v_cache", kRows);
    check(table, &dev, at::kInt, {-1, -1}, "block_table", kRows);
    const int64_t B = table.size(0);
    check(lens, &dev, at::kInt, {B}, "context_lens", kContiguous);
    check(offs, &dev, at::kInt, {B + 1}, "node_offsets", kContiguous);
    if (given(a[6])) {
      const Tensor& mask = tensor(a[6], "tree_mask");
      check(mask, &dev, mask.scalar_type() == at::kUInt64 ? at::kUInt64 : at::kLong, {q.size(0)}, "tree_mask", kContiguous);
      r.tree_mask = ptr<uint64_t>(mask);
    }
    r.nodes = as_int(q.size(0), "q");
    r.q_heads = as_int(q.size(1), "q");
    r.dim = as_int(q.size(2), "q");
    r.batch = as_int(B, "block_table");
    r.num_pages = as_int(kc.size(0), "k_cache");
    r.page_size = as_int(kc.size(1), "k_cache");
    r.k_heads = as_int(kc.size(2), "k_cache");
    r.table_width = as_int(table.size(1), "block_table");
    r.table_stride = table.stride(0);
    r.scale = static_cast<float>(given(a[7]) ? number(a[7]) : r.dim > 0 ? 1.0 / std::sqrt(static_cast<double>(r.dim)) : 1.0);
    Tensor out = given(a[8]) ? tensor(a[8], "out") : new_like(q, q.sizes(), type), ws;
    check(out, &dev, type, {q.size(0), q.size(1), q.size(2)}, "out", kRows);
    if (given(a[9])) {
      ws = tensor(a[9], "workspace");
      check(ws, &dev, at::kByte, {-1}, "workspace", kContiguous);
    } else if (const size_t need = g_tree_workspace(r.nodes, r.batch, r.q_heads, r.k_heads, r.dim)) {
      ws = new_like(q, {static_cast<int64_t>(need)}, at::kByte);
    }
    r.q = q.data_ptr();
    r.k_cache = kc.data_ptr();
    r.v_cache = vc.data_ptr();
    r.block_table = ptr<int32_t>(table);
    r.context_lens = ptr<int32_t>(lens);
    r.node_offsets = ptr<int32_t>(offs);
    r.out = out.data_ptr();
    r.q_stride_t = q.stride(0);
    r.q_stride_h = q.stride(1);
    r.out_stride_t = out.stride(0);
    r.out_stride_h = out.stride(1);
    r.k_page_stride = kc.stride(0);
    r.k_slot_stride = kc.stride(1);
    r.k_head_stride = kc.stride(2);
    r.v_page_stride = vc.stride(0);
    r.v_slot_stride = vc.stride(1);
    r.v_head_stride = vc.stride(2);
    if (const moe_status_t st = g_tree(&r, ws.defined() ? ws.data_ptr() : nullptr, ws.defined() ? ws.numel() : 0, stream_of(q))) return status(st);
    return THPVariable_Wrap(std::move(out));
  });
}

// verify_draft(target_probs, tokens, node_offsets, coins, last_coins, max_nodes, parents, draft_probs, out_tokens, path, accepted)
PyObject* verify_draft(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return bind(n, 11, [&]() -> PyObject* {
    const Tensor &target = tensor(a[0], "target_probs"), &tokens = tensor(a[1], "tokens"), &offs = tensor(a[2], "node_offsets");
    const Tensor &coins = tensor(a[3], "coins"), &last = tensor(a[4], "last_coins");
    const int most = integer(a[5]);
    check(target, nullptr, at::kFloat, {-1, -1}, "target_probs", kRows);
    const at::Device dev = target.device();
    check(tokens, &dev, at::kInt, {-1}, "tokens", kContiguous);
    check(last, &dev, at::kFloat, {-1}, "last_coins", kContiguous);
    const int64_t N = tokens.size(0), B = last.size(0), V = target.size(1);
    check(target, nullptr, at::kFloat, {N + B, -1}, "target_probs", kRows);
    check(offs, &dev, at::kInt, {B + 1}, "node_offsets", kContiguous);
    check(coins, &dev, at::kFloat, {N + B}, "coins", kContiguous);
    const int32_t* parents = nullptr;
    if (given(a[6])) {
      const Tensor& p = tensor(a[6], "parents");
      check(p, &dev, at::kInt, {N}, "parents", kContiguous);
      parents = ptr<int32_t>(p);
    }
    const float* draft = nullptr;
    int64_t draft_stride = 0;
    if (given(a[7])) {
      const Tensor& d = tensor(a[7], "draft_probs");
      check(d, &dev, at::kFloat, {N, V}, "draft_probs", kRows);
      draft = ptr<float>(d);
      draft_stride = row_stride(d);
    }
    if (most < 0) bad("max_nodes must not be negative");
    Tensor out = given(a[8]) ? tensor(a[8], "out_tokens") : new_like(target, {B, most + 1LL}, at::kInt);
    Tensor path = given(a[9]) ? tensor(a[9], "path") : new_like(target, {B, most}, at::kInt);
    Tensor accepted = given(a[10]) ? tensor(a[10], "accepted") : new_like(target, {B}, at::kInt);
    check(out, &dev, at::kInt, {B, most + 1LL}, "out_tokens", kContiguous);
    check(path, &dev, at::kInt, {B, most}, "path", kContiguous);
    check(accepted, &dev, at::kInt, {B}, "accepted", kContiguous);
    if (const moe_status_t st = g_verify(ptr<float>(target), row_stride(target), draft, draft_stride, ptr<int32_t>(tokens),
                                         parents, ptr<int32_t>(offs), ptr<float>(coins), ptr<float>(last), as_int(B, "last_coins"),
                                         as_int(N, "tokens"), as_int(V, "target_probs"), most, ptr<int32_t>(out), ptr<int32_t>(path),
                                         ptr<int32_t>(accepted), stream_of(target)))
      return status(st);
    return Py_BuildValue("(NNN)", THPVariable_Wrap(std::move(out)), THPVariable_Wrap(std::move(path)), THPVariable_Wrap(std::move(accepted)));
  });
}

// init(addresses of moe_rope, moe_linear_int4, its workspace size, moe_tree_attention, its workspace size, moe_verify_draft)
PyObject* init(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return bind(n, 6, [&]() -> PyObject* {
    void* p[6];
    for (int i = 0; i < 6; ++i) {
      p[i] = PyLong_AsVoidPtr(a[i]);
      if (!p[i]) bad("an entry point is missing");
    }
    g_rope = reinterpret_cast<decltype(g_rope)>(p[0]);
    g_linear = reinterpret_cast<decltype(g_linear)>(p[1]);
    g_linear_workspace = reinterpret_cast<decltype(g_linear_workspace)>(p[2]);
    g_tree = reinterpret_cast<decltype(g_tree)>(p[3]);
    g_tree_workspace = reinterpret_cast<decltype(g_tree_workspace)>(p[4]);
    g_verify = reinterpret_cast<decltype(g_verify)>(p[5]);
    return Py_NewRef(Py_None);
  });
}

#define FAST(f) reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(f)), METH_FASTCALL, nullptr
PyMethodDef kMethods[] = {{"init", FAST(init)},
                          {"rope", FAST(rope)},
                          {"rope_append", FAST(rope_append)},
                          {"linear_int4", FAST(linear_int4)},
                          {"tree_attention", FAST(tree_attention)},
                          {"verify_draft", FAST(verify_draft)},
                          {nullptr, nullptr, 0, nullptr}};
PyModuleDef kModule = {PyModuleDef_HEAD_INIT, "_step_bindings", nullptr, -1, kMethods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__step_bindings() { return PyModule_Create(&kModule); }
