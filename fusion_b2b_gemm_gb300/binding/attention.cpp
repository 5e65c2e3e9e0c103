// The common call of an attention plan's run(), from torch's tensors to the C
// ABI (include/b2b.h): checks, output and workspace, launch.  In Python these
// take longer than the kernels of a small call (a prompt of 19 tokens: 11.1 us
// a call in Python, 5.6 here; the kernel takes 5.1).  Whatever is not as the
// call wants it makes a function here return None, and attention.py, which does
// the same in Python, finds out what and says it.
#include <Python.h>

#include <torch/csrc/autograd/python_variable.h>

#include <ATen/core/grad_mode.h>
#include <ATen/ops/empty.h>
#include <torch/version.h>

#include <array>
#include <map>

#include "b2b.h"

namespace {

// Entries of libb2b.so, which is loaded by path.
struct {
  decltype(&b2b_prompt_attention_workspace) prompt_workspace;
  decltype(&b2b_prompt_attention_run) prompt_run;
  decltype(&b2b_shared_attention_workspace) shared_workspace;
  decltype(&b2b_shared_attention_run) shared_run;
} abi;

struct Bound {
  b2b_attn_plan_t plan;
  c10::ScalarType type;
  int64_t q_heads, kv_heads, dim;
  int device;
  std::map<std::array<int64_t, 4>, size_t> workspaces;  // bytes by sizes
};

constexpr char kName[] = "attn_binding.plan";

const at::Tensor* tensor(const Bound& p, PyObject* o, c10::ScalarType type, int64_t dims) {
  if (!THPVariable_Check(o)) return nullptr;
  const at::Tensor& t = THPVariable_Unpack(o);
  return t.layout() == c10::kStrided && t.scalar_type() == type && t.is_cuda() && t.get_device() == p.device && t.dim() == dims
             ? &t
             : nullptr;
}

// Whether a gradient would have to be recorded, or a tangent carried on, which no run does.
bool recorded(const at::Tensor& t) { return (t.requires_grad() && at::GradMode::is_enabled()) || t._fw_grad(0).defined(); }

// [rows][heads][dim], or [blocks][rows][heads][dim]
const at::Tensor* rows(const Bound& p, PyObject* o, int64_t dims, int64_t heads, b2b_attn_rows_t& r) {
  const at::Tensor* t = tensor(p, o, p.type, dims);
  if (!t || t->size(dims - 2) != heads || t->size(dims - 1) != p.dim || t->stride(dims - 1) != 1 || recorded(*t)) return nullptr;
  r = {t->data_ptr(), t->stride(dims - 3), t->stride(dims - 2), dims == 4 ? t->stride(0) : 0};
  return t;
}

// False: not a dense array of n counts (or n rows of any width).  The address of an array without entries is null.
bool counts(const Bound& p, PyObject* o, int64_t n, int64_t dims, const int32_t*& data, int64_t& width) {
  const at::Tensor* t = tensor(p, o, c10::kInt, dims);
  if (!t || (n >= 0 && t->size(0) != n) || !t->is_contiguous()) return false;
  width = t->size(dims - 1);
  data = static_cast<const int32_t*>(t->data_ptr());
  return true;
}

// The result's tensors, the workspace, and the launch.
template <class Args, class Query, class Run>
PyObject* finish(Bound& p, const at::Tensor& q, bool want_lse, Args& a, const std::array<int64_t, 4>& sizes, Query query,
                 Run run, void* stream) {
  auto known = p.workspaces.find(sizes);
  if (known == p.workspaces.end()) {
    size_t bytes = 0;
    if (query(p.plan, sizes[0], sizes[1], sizes[2], sizes[3], &bytes) != B2B_OK) return nullptr;
    if (p.workspaces.size() >= 4096) p.workspaces.clear();
    known = p.workspaces.emplace(sizes, bytes).first;
  }
  const int64_t tokens = q.size(0);
  at::Tensor out = at::empty({tokens, p.q_heads, p.dim}, q.options()), lse, workspace;
  a.out = {out.data_ptr(), p.q_heads * p.dim, p.dim, 0};
  if (want_lse) {
    lse = at::empty({tokens, p.q_heads}, q.options().dtype(c10::kFloat));
    a.lse = static_cast<float*>(lse.data_ptr());
  }
  a.workspace_bytes = known->second;
  if (known->second) {
    workspace = at::empty({static_cast<int64_t>(known->second)}, q.options().dtype(c10::kByte));
    a.workspace = workspace.data_ptr();
  }
  if (run(p.plan, &a, reinterpret_cast<b2b_stream_t>(stream)) != B2B_OK) return nullptr;
  PyObject* o = THPVariable_Wrap(std::move(out));
  if (!want_lse || !o) return o;
  PyObject* l = THPVariable_Wrap(std::move(lse));
  PyObject* both = l ? PyTuple_Pack(2, o, l) : nullptr;
  Py_DECREF(o);
  Py_XDECREF(l);
  return both;
}

PyObject* prompt(Bound& p, PyObject* const* arg) {
  b2b_prompt_attention_t a = {};
  void* stream = PyLong_AsVoidPtr(arg[1]);
  const int causal = PyObject_IsTrue(arg[7]), want_lse = PyObject_IsTrue(arg[8]);
  if (PyErr_Occurred()) return nullptr;
  const at::Tensor* q = rows(p, arg[2], 3, p.q_heads, a.q);
  const at::Tensor* k = rows(p, arg[3], 3, p.kv_heads, a.k);
  const at::Tensor* v = rows(p, arg[4], 3, p.kv_heads, a.v);
  int64_t offsets = 0, n = 0;
  if (!q || !k || !v || k->size(0) != v->size(0) || !counts(p, arg[5], -1, 1, a.cu_q, offsets) || offsets < 1) return nullptr;
  a.cu_k = a.cu_q;
  if (arg[6] != Py_None && !counts(p, arg[6], offsets, 1, a.cu_k, n)) return nullptr;
  a.batch = offsets - 1;
  a.tokens = q->size(0);
  a.key_rows = k->size(0);
  a.causal = causal;
  return finish(p, *q, want_lse, a, {a.batch, a.tokens, a.key_rows, a.causal}, abi.prompt_workspace, abi.prompt_run, stream);
}

PyObject* shared(Bound& p, PyObject* const* arg) {
  b2b_shared_attention_t a = {};
  void* stream = PyLong_AsVoidPtr(arg[1]);
  const int want_lse = PyObject_IsTrue(arg[9]);
  if (PyErr_Occurred()) return nullptr;
  const at::Tensor* q = rows(p, arg[2], 3, p.q_heads, a.q);
  const at::Tensor* pk = rows(p, arg[3], 3, p.kv_heads, a.prefix_k);
  const at::Tensor* pv = rows(p, arg[4], 3, p.kv_heads, a.prefix_v);
  const at::Tensor* ck = rows(p, arg[5], 4, p.kv_heads, a.cache_k);
  const at::Tensor* cv = rows(p, arg[6], 4, p.kv_heads, a.cache_v);
  if (!q || !pk || !pv || !ck || !cv || pk->size(0) != pv->size(0) || ck->size(0) != cv->size(0) || ck->size(1) != cv->size(1) ||
      !counts(p, arg[7], -1, 1, a.lengths, a.batch) || a.batch < 1 || q->size(0) % a.batch)
    return nullptr;
  a.fresh = q->size(0) / a.batch;
  a.prefix = pk->size(0);
  a.cache_blocks = ck->size(0);
  a.cache_rows = ck->size(1);
  int64_t room = a.cache_rows;
  if (arg[8] == Py_None) {
    if (a.cache_blocks != a.batch) return nullptr;
  } else {
    if (!counts(p, arg[8], a.batch, 2, a.page_table, a.table_width)) return nullptr;
    if (!a.page_table) a.page_table = a.lengths;  // (a table without columns, which is not read; null means none)
    room = a.cache_blocks ? a.table_width * a.cache_rows : 0;
  }
  return finish(p, *q, want_lse, a, {a.batch, a.fresh, a.prefix, room}, abi.shared_workspace, abi.shared_run, stream);
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
  unsigned long long e[4];
  if (!PyArg_ParseTuple(args, "KKKK", &e[0], &e[1], &e[2], &e[3])) return nullptr;
  abi = {reinterpret_cast<decltype(abi.prompt_workspace)>(e[0]), reinterpret_cast<decltype(abi.prompt_run)>(e[1]),
         reinterpret_cast<decltype(abi.shared_workspace)>(e[2]), reinterpret_cast<decltype(abi.shared_run)>(e[3])};
  Py_RETURN_NONE;
}

PyObject* bind(PyObject*, PyObject* args) {
  unsigned long long plan;
  int bf16, device;
  long long q_heads, kv_heads, dim;
  if (!PyArg_ParseTuple(args, "KpLLLi", &plan, &bf16, &q_heads, &kv_heads, &dim, &device)) return nullptr;
  Bound* p = new (std::nothrow) Bound{reinterpret_cast<b2b_attn_plan_t>(plan), bf16 ? c10::kBFloat16 : c10::kHalf, q_heads,
                                      kv_heads, dim, device, {}};
  if (!p) return PyErr_NoMemory();
  PyObject* c = PyCapsule_New(p, kName, [](PyObject* o) { delete static_cast<Bound*>(PyCapsule_GetPointer(o, kName)); });
  if (!c) delete p;
  return c;
}

PyMethodDef methods[] = {
    {"connect", connect, METH_VARARGS, "addresses of the four C functions"},
    {"bind", bind, METH_VARARGS, "(plan, bf16, q_heads, kv_heads, head_dim, device) -> what the calls take first"},
    {"prompt", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(&guarded<prompt, 9>)), METH_FASTCALL,
     "(bound, stream, q, k, v, cu_q, cu_k, causal, return_lse)"},
    {"shared", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(&guarded<shared, 10>)), METH_FASTCALL,
     "(bound, stream, q, prefix_k, prefix_v, cache_k, cache_v, lengths, page_table, return_lse)"},
    {nullptr, nullptr, 0, nullptr}};

PyModuleDef module = {PyModuleDef_HEAD_INIT, "attn_binding", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit_attn_binding() {
  PyObject* m = PyModule_Create(&module);
  if (m && PyModule_AddStringConstant(m, "torch_version", TORCH_VERSION) < 0) Py_CLEAR(m);
  return m;
}
