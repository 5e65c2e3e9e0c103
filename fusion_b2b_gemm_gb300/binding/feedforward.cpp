// The common calls of the feed-forward plans, from torch's tensors to the C ABI
// (include/b2b.h): checks, outputs and workspace, launch.  In Python these take
// longer than the kernels of a small call (one token on 1024/2816/1024: 20 us a
// call in Python, 7 here; the kernels take 8).  Whatever is not as the call
// wants it makes a function here return None, and feedforward.py, which does the
// same in Python, finds out what and says it.
#include <Python.h>

#include <torch/csrc/autograd/python_variable.h>

#include <ATen/EmptyTensor.h>
#include <ATen/core/grad_mode.h>
#include <ATen/core/Tensor.h>
#include <torch/version.h>

#include <map>
#include <utility>

#include "b2b.h"

namespace {

// Entries of libb2b.so, which is loaded by path.
struct {
  decltype(&b2b_ffn_workspace) workspace;
  decltype(&b2b_ffn_kept_bytes) kept_bytes;
  decltype(&b2b_ffn_forward) forward;
  decltype(&b2b_ffn_backward) backward;
  decltype(&b2b_scaled_ffn_run) scaled_ffn;
  decltype(&b2b_scaled_gemm_run) scaled_gemm;
} abi;

struct Bound {
  b2b_ffn_plan_t plan;
  c10::ScalarType type;
  int64_t width, hidden, out_width;  // (a product: k, -, n)
  int device;
  std::map<std::pair<int64_t, int>, size_t> workspaces;  // bytes by rows and pass
};

constexpr char kName[] = "ffn_binding.plan";
constexpr auto kE4M3 = c10::kFloat8_e4m3fn;

int64_t blocks(int64_t n) { return (n + 127) / 128; }

const at::Tensor* tensor(const Bound& p, PyObject* o, c10::ScalarType type) {
  if (!THPVariable_Check(o)) return nullptr;
  const at::Tensor& t = THPVariable_Unpack(o);
  return t.layout() == c10::kStrided && t.scalar_type() == type && t.is_cuda() && t.get_device() == p.device && t.dim() == 2 &&
                 !(t.requires_grad() && at::GradMode::is_enabled()) && !t._fw_grad(0).defined()  // (no gradient is recorded)
             ? &t
             : nullptr;
}

// [rows][cols], consecutive in a row; rows < 0: any
const at::Tensor* matrix(const Bound& p, PyObject* o, c10::ScalarType type, int64_t rows, int64_t cols, b2b_matrix_t& m) {
  const at::Tensor* t = tensor(p, o, type);
  if (!t || t->size(1) != cols || (rows >= 0 && t->size(0) != rows) || (t->stride(1) != 1 && cols != 1)) return nullptr;
  m = {t->data_ptr(), t->stride(0)};
  return t;
}

bool scales(const Bound& p, PyObject* o, int64_t rows, int64_t cols, b2b_scales_t& s) {
  const at::Tensor* t = tensor(p, o, c10::kFloat);
  if (!t || t->size(0) != rows || t->size(1) != cols) return false;
  s = {static_cast<float*>(t->data_ptr()), t->stride(0), t->stride(1)};
  return true;
}

// Memory of the current device and stream, from torch's pool.  (at::empty goes through
// the dispatcher: a small call 8.2 us, 6.5 so; backward 16.1 and 13.0.)
at::Tensor empty(c10::IntArrayRef sizes, c10::ScalarType type) {
  return at::Tensor(at::detail::empty_generic(sizes, c10::GetAllocator(c10::kCUDA), c10::DispatchKeySet(c10::DispatchKey::CUDA), type, std::nullopt));
}

at::Tensor fresh(const Bound& p, int64_t rows, int64_t cols, b2b_matrix_t& m) {
  at::Tensor t = empty({rows, cols}, p.type);
  m = {t.data_ptr(), cols};
  return t;
}

// The workspace of a run: from the pool of the current stream.
bool workspace(Bound& p, int64_t rows, int pass, c10::DataPtr& t, void*& data, size_t& bytes) {
  auto known = p.workspaces.find({rows, pass});
  if (known == p.workspaces.end()) {
    size_t need = 0;
    if (abi.workspace(p.plan, rows, pass, &need) != B2B_OK) return false;
    if (p.workspaces.size() >= 4096) p.workspaces.clear();
    known = p.workspaces.emplace(std::make_pair(rows, pass), need).first;
  }
  bytes = known->second;
  if (bytes) {
    t = c10::GetAllocator(c10::kCUDA)->allocate(bytes);
    data = t.get();
  }
  return true;
}

template <class... T>
PyObject* tuple(T&&... t) {
  PyObject* o[] = {t.defined() ? THPVariable_Wrap(std::move(t)) : Py_NewRef(Py_None)...};
  PyObject* r = PyTuple_New(sizeof...(T));
  for (size_t i = 0; i < sizeof...(T); ++i) {
    if (r && o[i])
      PyTuple_SET_ITEM(r, i, o[i]);
    else
      Py_XDECREF(o[i]);
    if (!o[i]) Py_CLEAR(r);
  }
  return r;
}

b2b_stream_t stream_of(PyObject* o) { return reinterpret_cast<b2b_stream_t>(PyLong_AsVoidPtr(o)); }

template <bool KEEP>
PyObject* forward(Bound& p, PyObject* const* arg) {
  b2b_ffn_forward_t a = {};
  const at::Tensor* x = matrix(p, arg[2], p.type, -1, p.width, a.x);
  if (!x || !matrix(p, arg[3], p.type, p.width, p.hidden, a.w_gate) || !matrix(p, arg[4], p.type, p.width, p.hidden, a.w_up) ||
      !matrix(p, arg[5], p.type, p.hidden, p.out_width, a.w_down))
    return nullptr;
  a.tokens = x->size(0);
  if (a.tokens == 0) return nullptr;
  at::Tensor out = fresh(p, a.tokens, p.out_width, a.out), kept;
  c10::DataPtr ws;
  if (KEEP) {
    if (abi.kept_bytes(p.plan, a.tokens, &a.kept_bytes) != B2B_OK) return nullptr;
    kept = empty({static_cast<int64_t>(a.kept_bytes)}, c10::kByte);
    a.kept = kept.data_ptr();
  }
  if (!workspace(p, a.tokens, KEEP ? B2B_FFN_TRAINING : B2B_FFN_INFERENCE, ws, a.workspace, a.workspace_bytes)) return nullptr;
  if (abi.forward(p.plan, &a, stream_of(arg[1])) != B2B_OK) return nullptr;
  if (!KEEP) return THPVariable_Wrap(std::move(out));
  return tuple(std::move(out), std::move(kept));
}

// Gradients in new tensors.
PyObject* backward(Bound& p, PyObject* const* arg) {
  b2b_ffn_backward_t a = {};
  const at::Tensor* x = matrix(p, arg[3], p.type, -1, p.width, a.x);
  if (!x) return nullptr;
  const int64_t t = a.tokens = x->size(0);
  if (t == 0 || !matrix(p, arg[2], p.type, t, p.out_width, a.dy) || !matrix(p, arg[4], p.type, p.width, p.hidden, a.w_gate) ||
      !matrix(p, arg[5], p.type, p.width, p.hidden, a.w_up) || !matrix(p, arg[6], p.type, p.hidden, p.out_width, a.w_down) ||
      !THPVariable_Check(arg[7]))
    return nullptr;
  const at::Tensor& kept = THPVariable_Unpack(arg[7]);
  if (kept.scalar_type() != c10::kByte || kept.dim() != 1 || !kept.is_contiguous() || !kept.is_cuda() || kept.get_device() != p.device)
    return nullptr;
  a.kept = kept.data_ptr();
  a.kept_bytes = static_cast<size_t>(kept.numel());
  at::Tensor dx;
  c10::DataPtr ws;
  const int input_grad = PyObject_IsTrue(arg[8]);
  if (input_grad < 0) return nullptr;
  if (input_grad) dx = fresh(p, t, p.width, a.dx);
  at::Tensor dg = fresh(p, p.width, p.hidden, a.dw_gate), du = fresh(p, p.width, p.hidden, a.dw_up),
             dd = fresh(p, p.hidden, p.out_width, a.dw_down);
  if (!workspace(p, t, B2B_FFN_BACKWARD, ws, a.workspace, a.workspace_bytes)) return nullptr;
  if (abi.backward(p.plan, &a, stream_of(arg[1])) != B2B_OK) return nullptr;
  return tuple(std::move(dx), std::move(dg), std::move(du), std::move(dd));
}

PyObject* scaled_ffn(Bound& p, PyObject* const* arg) {
  b2b_scaled_ffn_t a = {};
  const at::Tensor* x = matrix(p, arg[2], p.type, -1, p.width, a.x);
  const int64_t d = blocks(p.width), f = blocks(p.hidden), o = blocks(p.out_width);
  if (!x || !matrix(p, arg[3], kE4M3, p.hidden, p.width, a.w_gate) || !scales(p, arg[4], f, d, a.gate_scale) ||
      !matrix(p, arg[5], kE4M3, p.hidden, p.width, a.w_up) || !scales(p, arg[6], f, d, a.up_scale) ||
      !matrix(p, arg[7], kE4M3, p.out_width, p.hidden, a.w_down) || !scales(p, arg[8], o, f, a.down_scale))
    return nullptr;
  a.tokens = x->size(0);
  at::Tensor out = fresh(p, a.tokens, p.out_width, a.out);
  c10::DataPtr ws;
  if (!workspace(p, a.tokens, B2B_FFN_INFERENCE, ws, a.workspace, a.workspace_bytes)) return nullptr;
  if (abi.scaled_ffn(p.plan, &a, stream_of(arg[1])) != B2B_OK) return nullptr;
  return THPVariable_Wrap(std::move(out));
}

PyObject* scaled_gemm(Bound& p, PyObject* const* arg) {
  b2b_scaled_gemm_t a = {};
  const at::Tensor* m = matrix(p, arg[2], kE4M3, -1, p.width, a.a);
  if (!m || !scales(p, arg[3], m->size(0), blocks(p.width), a.a_scale) || !matrix(p, arg[4], kE4M3, p.out_width, p.width, a.b) ||
      !scales(p, arg[5], blocks(p.out_width), blocks(p.width), a.b_scale))
    return nullptr;
  a.rows = m->size(0);
  at::Tensor out = fresh(p, a.rows, p.out_width, a.out);
  c10::DataPtr ws;
  if (!workspace(p, a.rows, B2B_FFN_INFERENCE, ws, a.workspace, a.workspace_bytes)) return nullptr;
  if (abi.scaled_gemm(p.plan, &a, stream_of(arg[1])) != B2B_OK) return nullptr;
  return THPVariable_Wrap(std::move(out));
}

// An error's text is the slow path's to give.
template <PyObject* (*call)(Bound&, PyObject* const*), Py_ssize_t kArgs>
PyObject* guarded(PyObject*, PyObject* const* arg, Py_ssize_t n) {
  PyObject* r = nullptr;
  try {
    Bound* p = n == kArgs && PyCapsule_IsValid(arg[0], kName) ? static_cast<Bound*>(PyCapsule_GetPointer(arg[0], kName)) : nullptr;
    if (p) r = call(*p, arg);
  } catch (...) {
    r = nullptr;
  }
  if (r) return r;
  PyErr_Clear();
  Py_RETURN_NONE;
}

PyObject* connect(PyObject*, PyObject* args) {
  unsigned long long e[6];
  if (!PyArg_ParseTuple(args, "KKKKKK", &e[0], &e[1], &e[2], &e[3], &e[4], &e[5])) return nullptr;
  abi = {reinterpret_cast<decltype(abi.workspace)>(e[0]),  reinterpret_cast<decltype(abi.kept_bytes)>(e[1]),
         reinterpret_cast<decltype(abi.forward)>(e[2]),    reinterpret_cast<decltype(abi.backward)>(e[3]),
         reinterpret_cast<decltype(abi.scaled_ffn)>(e[4]), reinterpret_cast<decltype(abi.scaled_gemm)>(e[5])};
  Py_RETURN_NONE;
}

PyObject* bind(PyObject*, PyObject* args) {
  unsigned long long plan;
  int bf16, device;
  long long width, hidden, out_width;
  if (!PyArg_ParseTuple(args, "KpLLLi", &plan, &bf16, &width, &hidden, &out_width, &device)) return nullptr;
  Bound* p = new (std::nothrow)
      Bound{reinterpret_cast<b2b_ffn_plan_t>(plan), bf16 ? c10::kBFloat16 : c10::kHalf, width, hidden, out_width, device, {}};
  if (!p) return PyErr_NoMemory();
  PyObject* c = PyCapsule_New(p, kName, [](PyObject* o) { delete static_cast<Bound*>(PyCapsule_GetPointer(o, kName)); });
  if (!c) delete p;
  return c;
}

template <PyObject* (*call)(Bound&, PyObject* const*), Py_ssize_t kArgs>
PyMethodDef method(const char* name, const char* doc) {
  return {name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(&guarded<call, kArgs>)), METH_FASTCALL, doc};
}

PyMethodDef methods[] = {
    {"connect", connect, METH_VARARGS, "addresses of the six C functions"},
    {"bind", bind, METH_VARARGS, "(plan, bf16, width, hidden, out_width, device) -> what the calls take first"},
    method<forward<false>, 6>("run", "(bound, stream, x, w_gate, w_up, w_down)"),
    method<forward<true>, 6>("forward", "(bound, stream, x, w_gate, w_up, w_down)"),
    method<backward, 9>("backward", "(bound, stream, dy, x, w_gate, w_up, w_down, kept, input_grad)"),
    method<scaled_ffn, 9>("scaled_ffn", "(bound, stream, x, w_gate, gate_scale, w_up, up_scale, w_down, down_scale)"),
    method<scaled_gemm, 6>("scaled_gemm", "(bound, stream, a, a_scale, b, b_scale)"),
    {nullptr, nullptr, 0, nullptr}};

PyModuleDef module = {PyModuleDef_HEAD_INIT, "ffn_binding", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit_ffn_binding() {
  PyObject* m = PyModule_Create(&module);
  if (m && PyModule_AddStringConstant(m, "torch_version", TORCH_VERSION) < 0) Py_CLEAR(m);
  return m;
}
