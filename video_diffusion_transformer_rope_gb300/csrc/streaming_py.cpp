// Python entry of the streaming and conditioning calls: tensors to the structures of include/vdx.h,
// their checks, outputs and scratch from torch's allocator, and the call.  Marshalling only, no
// arithmetic.  It is compiled because these calls are short: a few microseconds on the device, where
// the same marshalling in Python took 19-28 us a call and this takes 3-4 (append 27.6 -> 6.0 us with its
// launch, paged attention 23.4 -> 6.1, cross attention 19.1 -> 6.8; one plain elementwise op of torch: 7.5).
//
// Every function takes its arguments by position (streaming.py names them) and raises VdxError before
// anything is launched; C++ exceptions end here as Python ones.
#include <Python.h>

#include <ATen/core/Tensor.h>
#include <ATen/ops/empty.h>
#include <c10/core/AutogradState.h>
#include <c10/core/GradMode.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>
#include <torch/version.h>

#include <climits>
#include <cstdarg>
#include <cstdint>
#include <string>

#include "vdx.h"

namespace {

PyObject* g_error = nullptr;                       // VdxError, set by bind()
decltype(&vdx_rope3d_append) g_append = nullptr;
decltype(&vdx_paged_attn_offset) g_paged = nullptr;
decltype(&vdx_paged_attn_workspace_bytes) g_paged_size = nullptr;
decltype(&vdx_cross_attn) g_cross = nullptr;
decltype(&vdx_cross_attn_workspace_bytes) g_cross_size = nullptr;
decltype(&vdx_last_error) g_last_error = nullptr;

struct Raised {};                                  // a Python error is set

[[noreturn]] void refuse(int status, const char* fmt, ...) {
  char buf[512];
  va_list ap;
  va_start(ap, fmt);
  vsnprintf(buf, sizeof(buf), fmt, ap);
  va_end(ap);
  PyObject* e = PyObject_CallFunction(g_error, "is", status, buf);
  if (e) {
    PyErr_SetObject(g_error, e);
    Py_DECREF(e);
  }
  throw Raised{};
}
void check(vdx_status s) {
  if (s != VDX_OK) refuse(s, "%s", g_last_error());
}

std::string text(at::IntArrayRef sizes) {
  std::string s = "(";
  for (size_t i = 0; i < sizes.size(); ++i) s += (i ? ", " : "") + std::to_string(sizes[i]);
  return s + (sizes.size() == 1 ? ",)" : ")");
}
std::string dev(const at::Tensor& t) { return t.device().str(); }

const at::Tensor* cuda_tensor(PyObject* o) {
  if (!THPVariable_Check(o)) return nullptr;
  const at::Tensor& t = THPVariable_Unpack(o);
  return t.is_cuda() && t.layout() == at::kStrided ? &t : nullptr;
}

// These calls have no derivative: neither a gradient nor a forward-mode tangent may be asked of a tensor.
void forward_only(const char* name, const at::Tensor& t) {
  if (!t.has_storage())
    refuse(VDX_ERR_UNSUPPORTED, "%s is wrapped by a function transform: these calls are forward only and take plain tensors", name);
  if (c10::GradMode::is_enabled() && t.requires_grad())
    refuse(VDX_ERR_UNSUPPORTED, "%s requires a gradient: these calls are forward only (use torch.no_grad() or detach())", name);
  if (c10::AutogradState::get_tls_state().get_fw_grad_mode() && t._fw_grad(0).defined())
    refuse(VDX_ERR_UNSUPPORTED, "%s carries a forward-mode tangent: these calls are forward only", name);
}

// A CUDA tensor of `dims` dimensions on like's device with like's type and dense channels (like NULL: a
// tensor that the others have to be like).
const at::Tensor& tensor(const char* name, PyObject* o, const at::Tensor* like, int dims) {
  const at::Tensor* t = cuda_tensor(o);
  if (!t && !like) refuse(VDX_ERR_ARG, "%s must be a CUDA tensor", name);
  if (!t || (like && (t->device() != like->device() || t->scalar_type() != like->scalar_type())))
    refuse(VDX_ERR_ARG, "%s must be a CUDA tensor of dtype %s on %s", name, c10::toString(like->scalar_type()), dev(*like).c_str());
  if (t->dim() != dims) refuse(VDX_ERR_ARG, "%s must have %d dimensions, got %s", name, dims, text(t->sizes()).c_str());
  for (int64_t n : t->sizes())
    if (n > INT_MAX) refuse(VDX_ERR_ARG, "%s: %s is too large", name, text(t->sizes()).c_str());
  if (t->stride(dims - 1) != 1 && t->size(dims - 1) > 1)
    refuse(VDX_ERR_ARG, "%s: the channels of a head must be contiguous", name);
  forward_only(name, *t);
  return *t;
}
int dtype_of(const at::Tensor& t) {
  if (t.scalar_type() == at::kBFloat16) return VDX_DTYPE_BF16;
  if (t.scalar_type() == at::kHalf) return VDX_DTYPE_FP16;
  refuse(VDX_ERR_UNSUPPORTED, "dtype %s (use bfloat16 or float16)", c10::toString(t.scalar_type()));
}
const int32_t* int32s(const char* name, PyObject* o, const at::Tensor& like, int64_t length) {
  if (o == Py_None) return nullptr;
  const at::Tensor* t = cuda_tensor(o);
  if (!t || t->scalar_type() != at::kInt || t->device() != like.device() || t->dim() != 1 || t->size(0) != length || !t->is_contiguous())
    refuse(VDX_ERR_ARG, "%s must be a contiguous int32 CUDA tensor of %lld values on %s", name, static_cast<long long>(length),
           dev(like).c_str());
  return static_cast<const int32_t*>(t->const_data_ptr());
}
// An integer that fits a C int and is not negative, from whatever int() takes.
int integer(const char* name, PyObject* o) {
  PyObject* n = PyNumber_Long(o);
  if (!n) throw Raised{};
  int over = 0;
  const long long v = PyLong_AsLongLongAndOverflow(n, &over);
  Py_DECREF(n);
  if (over || v < 0 || v > INT_MAX) refuse(VDX_ERR_ARG, "%s: integers in [0, 2^31) are needed", name);
  return static_cast<int>(v);
}
int bound(const char* name, PyObject* o) { return o == Py_None ? 0 : integer(name, o); }
void three(const char* name, PyObject* o, int* a, int* b, int* c) {
  PyObject* f = PySequence_Fast(o, "three integers are needed");
  if (!f) throw Raised{};
  struct Drop {
    PyObject* f;
    ~Drop() { Py_DECREF(f); }
  } drop{f};
  if (PySequence_Fast_GET_SIZE(f) != 3) refuse(VDX_ERR_ARG, "%s: 3 integers in [0, 2^31) are needed", name);
  int* out[3] = {a, b, c};
  for (int i = 0; i < 3; ++i) {
    PyObject* item = PySequence_Fast_GET_ITEM(f, i);       // held: converting another item may run Python code
    Py_INCREF(item);
    Drop hold{item};
    *out[i] = integer(name, item);
    if (PySequence_Fast_GET_SIZE(f) != 3) refuse(VDX_ERR_ARG, "%s changed its length", name);
  }
}
double real(PyObject* o) {
  const double v = PyFloat_AsDouble(o);
  if (v == -1.0 && PyErr_Occurred()) throw Raised{};
  return v;
}
const void* address(const at::Tensor& t) { return t.const_data_ptr(); }
// A tensor of the caller's that the call has written: autograd must be able to tell that one it saved is not
// what it was.  (Inference tensors have no version.)
void written(const at::Tensor& t) {
  if (!t.is_inference()) t.unsafeGetTensorImpl()->bump_version();
}

const at::Tensor& cache_struct(PyObject* k_, PyObject* v_, PyObject* table_, vdx_paged_kv* c, bool writes) {
  const at::Tensor& k = tensor("the key cache", k_, nullptr, 4);
  const at::Tensor& v = tensor("the value cache", v_, &k, 4);
  if (k.sizes() != v.sizes())
    refuse(VDX_ERR_ARG, "the key and value caches differ in shape: %s, %s", text(k.sizes()).c_str(), text(v.sizes()).c_str());
  const at::Tensor* t = cuda_tensor(table_);
  if (!t || t->scalar_type() != at::kInt || t->device() != k.device() || t->dim() != 2 || (t->size(1) > 1 && t->stride(1) != 1) ||
      t->size(0) > INT_MAX - 1 || t->size(1) > INT_MAX)
    refuse(VDX_ERR_ARG, "page_table must be an int32 [seqs, max_pages] tensor on %s with contiguous rows", dev(k).c_str());
  c->k = writes ? k.mutable_data_ptr() : const_cast<void*>(address(k));
  c->v = writes ? v.mutable_data_ptr() : const_cast<void*>(address(v));
  c->k_page = k.stride(0); c->k_token = k.stride(1); c->k_head = k.stride(2);
  c->v_page = v.stride(0); c->v_token = v.stride(1); c->v_head = v.stride(2);
  c->page_table = static_cast<const int32_t*>(address(*t));
  c->table_stride = t->stride(0);
  c->num_pages = static_cast<int>(k.size(0));
  c->page_size = static_cast<int>(k.size(1));
  c->max_pages = static_cast<int>(t->size(1));
  c->Hkv = static_cast<int>(k.size(2));
  c->d = static_cast<int>(k.size(3));
  c->dtype = dtype_of(k);
  c->seqs = static_cast<int>(t->size(0));
  return k;
}

// 0 bytes are an answer, or a call that the library cannot take: then it has left a message.
PyObject* bytes_or_refusal(size_t bytes) {
  if (bytes == 0 && *g_last_error()) refuse(VDX_ERR_ARG, "%s", g_last_error());
  return PyLong_FromSize_t(bytes);
}

// Device of the call made current, its current stream, and the interpreter released for the call itself.
template <typename F>
void call(const at::Tensor& like, F&& f) {
  const c10::cuda::CUDAGuard guard(like.device());
  void* stream = c10::cuda::getCurrentCUDAStream(like.device().index()).stream();
  vdx_status s;
  Py_BEGIN_ALLOW_THREADS
  s = f(stream);
  Py_END_ALLOW_THREADS
  check(s);
}

at::Tensor empty(at::IntArrayRef sizes, const at::Tensor& like, at::ScalarType type) {
  return at::empty(sizes, at::TensorOptions().dtype(type).device(like.device()));
}

// Outputs and scratch (the caller's, or torch's for this call on its stream), then the call.
template <typename Args, typename Size, typename Run>
PyObject* attention(Args& a, const at::Tensor& q, at::IntArrayRef lse_shape, PyObject* out_, PyObject* lse_, PyObject* return_lse,
                    PyObject* workspace_, Size&& size, Run&& run) {
  const c10::cuda::CUDAGuard guard(q.device());
  at::Tensor out, lse, workspace;
  if (out_ == Py_None) {
    out = empty(q.sizes(), q, q.scalar_type());
  } else {
    out = tensor("out", out_, &q, static_cast<int>(q.dim()));
    if (out.sizes() != q.sizes() || !out.is_contiguous())
      refuse(VDX_ERR_ARG, "out must be contiguous and shaped like q %s", text(q.sizes()).c_str());
  }
  a.out = out.mutable_data_ptr();
  if (lse_ != Py_None) {
    const at::Tensor* t = cuda_tensor(lse_);
    if (!t || t->scalar_type() != at::kFloat || t->sizes() != lse_shape || !t->is_contiguous() || t->device() != q.device())
      refuse(VDX_ERR_ARG, "lse must be a contiguous float32 tensor of shape %s on %s", text(lse_shape).c_str(), dev(q).c_str());
    forward_only("lse", *t);
    lse = *t;
  } else {
    const int want = PyObject_IsTrue(return_lse);
    if (want < 0) throw Raised{};
    if (want) lse = empty(lse_shape, q, at::kFloat);
  }
  if (lse.defined()) a.lse = static_cast<float*>(lse.mutable_data_ptr());
  if (workspace_ != Py_None) {
    const at::Tensor* t = cuda_tensor(workspace_);
    if (!t || t->device() != q.device() || !t->is_contiguous())
      refuse(VDX_ERR_ARG, "workspace must be a contiguous CUDA tensor on %s", dev(q).c_str());
    workspace = *t;
  } else if (const size_t need = size()) {
    workspace = empty({static_cast<int64_t>(need)}, q, at::kByte);
  }
  if (workspace.defined()) {
    a.workspace = workspace.mutable_data_ptr();
    a.workspace_bytes = static_cast<size_t>(workspace.numel()) * workspace.element_size();
  }
  call(q, run);
  if (out_ != Py_None) written(out);
  if (lse_ != Py_None) written(lse);
  if (workspace_ != Py_None) written(workspace);
  PyObject* o = out_ == Py_None ? THPVariable_Wrap(out) : Py_NewRef(out_);
  PyObject* l = !lse.defined() ? Py_NewRef(Py_None) : (lse_ == Py_None ? THPVariable_Wrap(lse) : Py_NewRef(lse_));
  PyObject* r = o && l ? PyTuple_Pack(2, o, l) : nullptr;
  Py_XDECREF(o);
  Py_XDECREF(l);
  return r;
}

// ------------------------------------------------------------------------------------------ the calls
PyObject* append(PyObject* const* a) {
  PyObject *q_ = a[0], *q_out_ = a[12];
  vdx_paged_kv c{};
  vdx_append_args x{};
  const at::Tensor& like = cache_struct(a[3], a[4], a[5], &c, true);
  const at::Tensor& k = tensor("k", a[1], &like, 3);
  const at::Tensor& v = tensor("v", a[2], &like, 3);
  if (k.size(1) != c.Hkv || k.size(2) != c.d || v.sizes() != k.sizes())
    refuse(VDX_ERR_ARG, "k %s and v %s must be [rows, %d, %d], as the cache's heads", text(k.sizes()).c_str(), text(v.sizes()).c_str(),
           c.Hkv, c.d);
  auto weights = [&](const char* name, PyObject* o) -> const void* {
    if (o == Py_None) return nullptr;
    const at::Tensor& w = tensor(name, o, &like, 1);
    if (w.size(0) != c.d) refuse(VDX_ERR_ARG, "%s must hold %d weights", name, c.d);
    return address(w);
  };
  x.q_norm = weights("q_norm", a[9]);
  x.k_norm = weights("k_norm", a[10]);
  x.rows = static_cast<int>(k.size(0));
  x.k = address(k);
  x.v = address(v);
  x.k_row = k.stride(0); x.k_head = k.stride(1);
  x.v_row = v.stride(0); x.v_head = v.stride(1);
  x.cu = int32s("cu", a[6], like, static_cast<int64_t>(c.seqs) + 1);
  x.kv_len = int32s("kv_len", a[7], like, c.seqs);
  x.pos_offset = int32s("pos_offset", a[8], like, c.seqs);
  three("grid", a[13], &x.T, &x.Hgrid, &x.Wgrid);
  three("sections", a[14], &x.sec_t, &x.sec_h, &x.sec_w);
  x.theta = real(a[15]);
  x.eps = static_cast<float>(real(a[11]));
  auto run = [&] {
    call(like, [&](void* stream) { return g_append(&c, &x, stream); });
    written(THPVariable_Unpack(a[3]));
    written(THPVariable_Unpack(a[4]));
  };
  if (q_ == Py_None) {
    if (q_out_ != Py_None) refuse(VDX_ERR_ARG, "q_out without q");
    run();
    Py_RETURN_NONE;
  }
  const at::Tensor& q = tensor("q", q_, &like, 3);
  if (q.size(0) != x.rows || q.size(2) != c.d)
    refuse(VDX_ERR_ARG, "q %s does not match the %d rows of %d channels of k", text(q.sizes()).c_str(), x.rows, c.d);
  if (q.size(1) == 0) refuse(VDX_ERR_ARG, "q has no heads (q=None appends keys and values only)");
  x.Hq = static_cast<int>(q.size(1));
  x.q = address(q);
  x.q_row = q.stride(0); x.q_head = q.stride(1);
  const c10::cuda::CUDAGuard guard(like.device());
  at::Tensor out;
  if (q_out_ == Py_None) {
    out = empty(q.sizes(), q, q.scalar_type());
  } else {
    out = tensor("q_out", q_out_, &q, 3);
    if (out.sizes() != q.sizes()) refuse(VDX_ERR_ARG, "q_out must be shaped like q %s", text(q.sizes()).c_str());
  }
  if (x.rows > 0) {                                        // empty tensors have no address
    x.q_out = out.mutable_data_ptr();
    x.q_out_row = out.stride(0); x.q_out_head = out.stride(1);
    run();
    if (q_out_ != Py_None) written(out);
  }
  return q_out_ == Py_None ? THPVariable_Wrap(out) : Py_NewRef(q_out_);
}

// q, the cache's three tensors, cu, kv_len, max_q, max_kv of a paged call
const at::Tensor& paged_args(PyObject* const* a, vdx_paged_kv* c, vdx_paged_attn_args* x) {
  const at::Tensor& like = cache_struct(a[1], a[2], a[3], c, false);
  const at::Tensor& q = tensor("q", a[0], &like, 3);
  if (q.size(2) != c->d)
    refuse(VDX_ERR_ARG, "q %s does not match the cache's head dimension %d", text(q.sizes()).c_str(), c->d);
  x->q = address(q);
  x->q_row = q.stride(0); x->q_head = q.stride(1);
  x->rows = static_cast<int>(q.size(0));
  x->Hq = static_cast<int>(q.size(1));
  x->cu = int32s("cu", a[4], q, static_cast<int64_t>(c->seqs) + 1);
  x->kv_len = int32s("kv_len", a[5], q, c->seqs);
  x->max_q = bound("max_q", a[6]);
  x->max_kv = bound("max_kv", a[7]);
  return q;
}
PyObject* paged(PyObject* const* a) {
  vdx_paged_kv c{};
  vdx_paged_attn_args x{};
  const at::Tensor& q = paged_args(a, &c, &x);
  x.causal_block = integer("causal_block", a[8]);
  x.scale = static_cast<float>(real(a[9]));
  const int32_t* pos_offset = int32s("pos_offset", a[14], q, c.seqs);
  const int64_t lse_shape[2] = {x.Hq, x.rows};
  return attention(x, q, lse_shape, a[10], a[11], a[12], a[13], [&] { return g_paged_size(&c, &x); },
                   [&](void* stream) { return g_paged(&c, &x, pos_offset, stream); });
}
PyObject* paged_size(PyObject* const* a) {
  vdx_paged_kv c{};
  vdx_paged_attn_args x{};
  const c10::cuda::CUDAGuard guard(paged_args(a, &c, &x).device());
  return bytes_or_refusal(g_paged_size(&c, &x));
}

// q, k, v, kv_len of a cross-attention call
const at::Tensor& cross_args(PyObject* const* a, vdx_cross_attn_args* x) {
  const at::Tensor& q = tensor("q", a[0], nullptr, 4);
  const at::Tensor& k = tensor("k", a[1], &q, 4);
  const at::Tensor& v = tensor("v", a[2], &q, 4);
  if (k.sizes() != v.sizes() || k.size(0) != q.size(0) || k.size(3) != q.size(3))
    refuse(VDX_ERR_ARG, "q [B, N, Hq, d], k and v [B, M, Hkv, d]: got %s, %s, %s", text(q.sizes()).c_str(), text(k.sizes()).c_str(),
           text(v.sizes()).c_str());
  x->q = address(q);
  x->k = address(k);
  x->v = address(v);
  x->q_batch = q.stride(0); x->q_row = q.stride(1); x->q_head = q.stride(2);
  x->k_batch = k.stride(0); x->k_token = k.stride(1); x->k_head = k.stride(2);
  x->v_batch = v.stride(0); x->v_token = v.stride(1); x->v_head = v.stride(2);
  x->B = static_cast<int>(q.size(0));
  x->N = static_cast<int>(q.size(1));
  x->M = static_cast<int>(k.size(1));
  x->Hq = static_cast<int>(q.size(2));
  x->Hkv = static_cast<int>(k.size(2));
  x->d = static_cast<int>(q.size(3));
  x->dtype = dtype_of(q);
  x->kv_len = int32s("kv_len", a[3], q, x->B);
  return q;
}
PyObject* cross(PyObject* const* a) {
  vdx_cross_attn_args x{};
  const at::Tensor& q = cross_args(a, &x);
  x.scale = static_cast<float>(real(a[4]));
  const int64_t lse_shape[3] = {x.B, x.Hq, x.N};
  return attention(x, q, lse_shape, a[5], a[6], a[7], a[8], [&] { return g_cross_size(&x); },
                   [&](void* stream) { return g_cross(&x, stream); });
}
PyObject* cross_size(PyObject* const* a) {
  vdx_cross_attn_args x{};
  const c10::cuda::CUDAGuard guard(cross_args(a, &x).device());
  return bytes_or_refusal(g_cross_size(&x));
}

template <PyObject* (*kCall)(PyObject* const*), int kArgs>
PyObject* entry(PyObject*, PyObject* const* args, Py_ssize_t n) {
  if (n != kArgs) return PyErr_Format(PyExc_TypeError, "%d arguments are needed, got %zd", kArgs, n);
  if (!g_error) return PyErr_Format(PyExc_RuntimeError, "bind() has not been called");
  HANDLE_TH_ERRORS
  try {
    return kCall(args);
  } catch (const Raised&) {
    return nullptr;
  }
  END_HANDLE_TH_ERRORS
}

// bind(VdxError, addresses of the library's functions in the order below)
PyObject* bind(PyObject*, PyObject* args) {
  PyObject* error;
  unsigned long long f[6];
  if (!PyArg_ParseTuple(args, "OKKKKKK", &error, f, f + 1, f + 2, f + 3, f + 4, f + 5)) return nullptr;
  g_append = reinterpret_cast<decltype(g_append)>(f[0]);
  g_paged = reinterpret_cast<decltype(g_paged)>(f[1]);
  g_paged_size = reinterpret_cast<decltype(g_paged_size)>(f[2]);
  g_cross = reinterpret_cast<decltype(g_cross)>(f[3]);
  g_cross_size = reinterpret_cast<decltype(g_cross_size)>(f[4]);
  g_last_error = reinterpret_cast<decltype(g_last_error)>(f[5]);
  Py_INCREF(error);
  Py_XSETREF(g_error, error);
  Py_RETURN_NONE;
}

#define VDX_ENTRY(name, n) \
  { #name, reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(entry<name, n>)), METH_FASTCALL, nullptr }
PyMethodDef kMethods[] = {
    {"bind", bind, METH_VARARGS, nullptr},
    VDX_ENTRY(append, 16),
    VDX_ENTRY(paged, 15),
    VDX_ENTRY(paged_size, 8),
    VDX_ENTRY(cross, 9),
    VDX_ENTRY(cross_size, 4),
    {nullptr, nullptr, 0, nullptr},
};
PyModuleDef kModule = {PyModuleDef_HEAD_INIT, "_streaming_py", nullptr, -1, kMethods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

extern "C" __attribute__((visibility("default"))) PyObject* PyInit__streaming_py() {
  PyObject* m = PyModule_Create(&kModule);
  if (m && PyModule_AddStringConstant(m, "TORCH_VERSION", TORCH_VERSION) < 0) Py_CLEAR(m);
  return m;
}
