// Argument marshalling of the packed and paged entry points (include/fa.h) for torch
// tensors: checks, output allocation and the C call, without arithmetic of its own.
//
// These calls run once per layer and token. Reading shapes, strides and pointers through
// Python costs about 10 us a call, several times the C call and longer than the small
// kernels; read in C++ they cost under 1 us. The Python functions keep the signatures,
// the documentation and the stream handling.
#include <ATen/core/Tensor.h>
#include <ATen/ops/empty.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <cmath>
#include <stdexcept>
#include <string>

#include "fa.h"

namespace {

PyObject* g_error = nullptr;  // the package's FAError

using at::Tensor;

[[noreturn]] void type_error(const std::string& m) {
  PyErr_SetString(PyExc_TypeError, m.c_str());
  throw python_error();
}
[[noreturn]] void value_error(const std::string& m) {
  PyErr_SetString(PyExc_ValueError, m.c_str());
  throw python_error();
}

const Tensor& tensor(const char* name, PyObject* o) {
  if (!THPVariable_Check(o)) type_error(std::string(name) + " must be a torch.Tensor");
  return THPVariable_Unpack(o);
}

// Elements from row to row of a bf16 [rows, heads, d] CUDA tensor whose heads and columns
// are dense.
long long row_stride(const char* name, const Tensor& t) {
  if (!t.is_cuda() || t.scalar_type() != at::kBFloat16 || t.dim() != 3)
    value_error(std::string(name) + " must be a bf16 CUDA tensor [rows, heads, d]");
  const long long rows = t.size(0), heads = t.size(1), d = t.size(2);
  if ((d > 1 && t.stride(2) != 1) || (heads > 1 && t.stride(1) != d))
    value_error(std::string(name) + " must be dense in its heads and columns");
  if (rows <= 1) return heads * d;
  const long long s = t.stride(0);
  if (s < heads * d || s % 8 != 0)
    value_error(std::string(name) +
                " must have a row stride that is a multiple of 8 and at least heads * d");
  return s;
}

// A dense tensor of this type and shape on device `dev`.
void dense(const char* name, const Tensor& t, at::ScalarType type, at::IntArrayRef shape, int dev) {
  if (t.scalar_type() != type || t.sizes() != shape || !t.is_cuda() || t.get_device() != dev ||
      !t.is_contiguous()) {
    std::string s = "(";
    for (size_t i = 0; i < shape.size(); ++i) s += (i ? ", " : "") + std::to_string(shape[i]);
    value_error(std::string(name) + " must be a contiguous " + c10::toString(type) +
                " tensor of shape " + s + ") on cuda:" + std::to_string(dev));
  }
}

void same_device(int dev, const Tensor& t) {
  if (!t.is_cuda() || t.get_device() != dev)
    value_error("all tensors of a call must be on the same device");
}

// The caller's output, checked, or a new one.
Tensor output(const char* name, PyObject* o, at::ScalarType type, at::IntArrayRef shape,
              const Tensor& like, bool* made) {
  *made = o == Py_None;
  if (*made) return at::empty(shape, like.options().dtype(type));
  const Tensor& t = tensor(name, o);
  dense(name, t, type, shape, like.get_device());
  return t;
}

size_t workspace_bytes(const Tensor& t, int dev) {
  if (!t.is_contiguous() || !t.is_cuda() || t.get_device() != dev)
    value_error("workspace must be a contiguous tensor on the inputs' device");
  return t.nbytes();
}

float scale_of(PyObject* o, long long d) {
  if (o == Py_None) return (float)(1.0 / std::sqrt((double)d));
  const double s = PyFloat_AsDouble(o);
  if (s == -1.0 && PyErr_Occurred()) throw python_error();
  return (float)s;
}

long long integer(PyObject* o) {
  const long long v = PyLong_AsLongLong(o);
  if (v == -1 && PyErr_Occurred()) throw python_error();
  return v;
}

// A size as the C interface takes it; what does not fit becomes a value it refuses.
int as_int(long long v) { return v > 0x7fffffffLL || v < 0 ? -1 : (int)v; }

void* stream_of(int dev) { return c10::cuda::getCurrentCUDAStream((c10::DeviceIndex)dev).stream(); }

void check(const char* fn, int rc) {
  if (rc == FA_OK) return;
  PyObject* e = PyObject_CallFunction(g_error, "si", fn, rc);
  if (e) {
    PyErr_SetObject(g_error, e);
    Py_DECREF(e);
  }
  throw python_error();
}

void expect_args(Py_ssize_t n, Py_ssize_t want) {
  if (n != want) type_error("wrong number of arguments");
}

struct Packed {
  long long ldq, ldk, ldv;
  int total, Hq, Hkv, d, nseq, causal, dev;
  const void* plan;
};

// Q, K, V, the plan's buffer, nseq, total and causal, from a[0] on.
Packed packed_inputs(PyObject* const* a) {
  const Tensor &Q = tensor("Q", a[0]), &K = tensor("K", a[1]), &V = tensor("V", a[2]);
  Packed p;
  p.ldq = row_stride("Q", Q);
  p.ldk = row_stride("K", K);
  p.ldv = row_stride("V", V);
  if (K.sizes() != V.sizes() || K.size(0) != Q.size(0) || K.size(2) != Q.size(2))
    value_error("K and V must be [total, Hkv, d] with Q's rows and d");
  const long long hq = Q.size(1), hkv = K.size(1), total = integer(a[5]);
  if (hkv == 0 || hq % hkv != 0)
    value_error("the number of query heads must be a multiple of the key/value heads");
  if (Q.size(0) != total)
    value_error("the plan is for " + std::to_string(total) + " rows, Q has " +
                std::to_string(Q.size(0)));
  p.dev = (int)Q.get_device();
  const Tensor& plan = tensor("plan", a[3]);
  same_device(p.dev, K);
  same_device(p.dev, V);
  same_device(p.dev, plan);
  p.total = as_int(total);
  p.Hq = as_int(hq);
  p.Hkv = as_int(hkv);
  p.d = as_int(Q.size(2));
  p.nseq = as_int(integer(a[4]));
  p.causal = PyObject_IsTrue(a[6]) == 1;
  p.plan = plan.data_ptr();
  return p;
}

// (Q, K, V, plan, nseq, total, causal, scale, O, L) -> (O, L)
PyObject* packed_forward(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  expect_args(n, 10);
  const Packed p = packed_inputs(a);
  const Tensor& Q = THPVariable_Unpack(a[0]);
  c10::cuda::CUDAGuard guard((c10::DeviceIndex)p.dev);
  bool made_o, made_l;
  const Tensor O = output("O", a[8], at::kBFloat16, {p.total, p.Hq, p.d}, Q, &made_o);
  const Tensor L = output("L", a[9], at::kFloat, {p.Hq, p.total}, Q, &made_l);
  check("fa_packed_forward",
        fa_packed_forward(Q.data_ptr(), THPVariable_Unpack(a[1]).data_ptr(),
                          THPVariable_Unpack(a[2]).data_ptr(), p.ldq, p.ldk, p.ldv, p.total, p.Hq,
                          p.Hkv, p.d, p.causal, scale_of(a[7], p.d), p.plan, p.nseq, O.data_ptr(),
                          static_cast<float*>(L.data_ptr()), made_o | made_l << 1,
                          stream_of(p.dev)));
  return Py_BuildValue("(NN)", THPVariable_Wrap(O), THPVariable_Wrap(L));
  END_HANDLE_TH_ERRORS
}

// A gradient with the shape of `like`: the caller's, with any row stride, or a new one.
Tensor gradient(const char* name, PyObject* o, const Tensor& like, long long* ld, bool* made) {
  *made = o == Py_None;
  if (*made) {
    *ld = like.size(1) * like.size(2);
    return at::empty(like.sizes(), like.options());
  }
  const Tensor& t = tensor(name, o);
  *ld = row_stride(name, t);
  if (t.sizes() != like.sizes())
    value_error(std::string(name) + " must have the shape of its input");
  same_device((int)like.get_device(), t);
  return t;
}

// (Q, K, V, plan, nseq, total, causal, scale, O, L, dO, dQ, dK, dV, workspace)
// -> (dQ, dK, dV)
PyObject* packed_backward(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  expect_args(n, 15);
  const Packed p = packed_inputs(a);
  const Tensor &Q = THPVariable_Unpack(a[0]), &K = THPVariable_Unpack(a[1]),
               &V = THPVariable_Unpack(a[2]);
  const Tensor &O = tensor("O", a[8]), &L = tensor("L", a[9]), &dO = tensor("dO", a[10]);
  dense("O", O, at::kBFloat16, Q.sizes(), p.dev);
  dense("dO", dO, at::kBFloat16, Q.sizes(), p.dev);
  dense("L", L, at::kFloat, {p.Hq, p.total}, p.dev);
  c10::cuda::CUDAGuard guard((c10::DeviceIndex)p.dev);
  long long lddq, lddk, lddv;
  bool made_q, made_k, made_v;
  const Tensor dQ = gradient("dQ", a[11], Q, &lddq, &made_q);
  const Tensor dK = gradient("dK", a[12], K, &lddk, &made_k);
  const Tensor dV = gradient("dV", a[13], V, &lddv, &made_v);
  Tensor ws;
  if (a[14] == Py_None) {
    const size_t need = fa_packed_workspace_bytes(p.nseq, p.total, p.Hq);
    if (need == 0) value_error("invalid sizes for the backward workspace");
    ws = at::empty({(long long)need}, Q.options().dtype(at::kByte));
  } else {
    ws = tensor("workspace", a[14]);
  }
  const size_t bytes = workspace_bytes(ws, p.dev);
  check("fa_packed_backward",
        fa_packed_backward(Q.data_ptr(), K.data_ptr(), V.data_ptr(), p.ldq, p.ldk, p.ldv,
                           O.data_ptr(), static_cast<const float*>(L.data_ptr()), dO.data_ptr(),
                           p.total, p.Hq, p.Hkv, p.d, p.causal, scale_of(a[7], p.d), p.plan,
                           p.nseq, dQ.data_ptr(), dK.data_ptr(), dV.data_ptr(), lddq, lddk, lddv,
                           made_q | made_k << 1 | made_v << 2, ws.data_ptr(), bytes,
                           stream_of(p.dev)));
  return Py_BuildValue("(NNN)", THPVariable_Wrap(dQ), THPVariable_Wrap(dK), THPVariable_Wrap(dV));
  END_HANDLE_TH_ERRORS
}

// The caches' common shape [pages, Hkv, page, d].
at::IntArrayRef cache_shape(const Tensor& Kc, const Tensor& Vc) {
  for (const Tensor* t : {&Kc, &Vc})
    if (!t->is_cuda() || t->scalar_type() != at::kBFloat16 || t->dim() != 4 || !t->is_contiguous())
      value_error("K_cache and V_cache must be contiguous bf16 CUDA tensors [pages, Hkv, page, d]");
  if (Kc.sizes() != Vc.sizes() || Kc.get_device() != Vc.get_device())
    value_error("K_cache and V_cache must have one shape and one device");
  return Kc.sizes();
}

// An int32 [requests, max_pages] table; returns max_pages.
long long table_width(const Tensor& t, long long requests, int dev) {
  if (t.dim() != 2) value_error("block_table must be an int32 tensor [requests, max_pages]");
  dense("block_table", t, at::kInt, {requests, t.size(1)}, dev);
  return t.size(1);
}

// (K, V, cu_seqlens, starts, block_table, K_cache, V_cache)
PyObject* cache_append(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  expect_args(n, 7);
  const Tensor &K = tensor("K", a[0]), &V = tensor("V", a[1]), &cu = tensor("cu_seqlens", a[2]),
               &starts = tensor("starts", a[3]), &table = tensor("block_table", a[4]),
               &Kc = tensor("K_cache", a[5]), &Vc = tensor("V_cache", a[6]);
  const at::IntArrayRef c = cache_shape(Kc, Vc);
  const int dev = (int)Kc.get_device();
  const long long ldk = row_stride("K", K), ldv = row_stride("V", V);
  if (K.sizes() != V.sizes() || K.size(1) != c[1] || K.size(2) != c[3])
    value_error("K and V must be [total, Hkv, d] with the caches' Hkv and d");
  same_device(dev, K);
  same_device(dev, V);
  if (starts.dim() != 1) value_error("starts must be an int32 tensor [requests]");
  const long long nseq = starts.size(0);
  dense("starts", starts, at::kInt, {nseq}, dev);
  dense("cu_seqlens", cu, at::kInt, {nseq + 1}, dev);
  const long long width = table_width(table, nseq, dev);
  c10::cuda::CUDAGuard guard((c10::DeviceIndex)dev);
  check("fa_cache_append",
        fa_cache_append(K.data_ptr(), V.data_ptr(), ldk, ldv, as_int(K.size(0)),
                        static_cast<const int*>(cu.data_ptr()),
                        static_cast<const int*>(starts.data_ptr()), as_int(nseq),
                        static_cast<const int*>(table.data_ptr()), as_int(width), Kc.data_ptr(),
                        Vc.data_ptr(), as_int(c[0]), as_int(c[1]), as_int(c[2]), as_int(c[3]),
                        stream_of(dev)));
  Py_RETURN_NONE;
  END_HANDLE_TH_ERRORS
}

// (Q, K_cache, V_cache, prefix_pages, prefix_len, block_table, lens, scale, O, L,
// workspace) -> (O, L)
PyObject* prefix_decode(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  expect_args(n, 11);
  const Tensor &Q = tensor("Q", a[0]), &Kc = tensor("K_cache", a[1]), &Vc = tensor("V_cache", a[2]),
               &table = tensor("block_table", a[5]), &lens = tensor("lens", a[6]);
  const at::IntArrayRef c = cache_shape(Kc, Vc);
  const int dev = (int)Kc.get_device();
  if (Q.dim() != 3) value_error("Q must be a bf16 tensor [B, Hq, d]");
  const long long B = Q.size(0), Hq = Q.size(1), d = c[3];
  dense("Q", Q, at::kBFloat16, {B, Hq, d}, dev);
  dense("lens", lens, at::kInt, {B}, dev);
  const long long width = table_width(table, B, dev);
  long long shared = 0;
  const int *pages = nullptr, *len = nullptr;
  if (a[3] != Py_None) {
    const Tensor &pp = tensor("prefix_pages", a[3]), &pl = tensor("prefix_len", a[4]);
    if (pp.dim() != 1) value_error("prefix_pages must be an int32 tensor [n]");
    shared = pp.size(0);
    dense("prefix_pages", pp, at::kInt, {shared}, dev);
    dense("prefix_len", pl, at::kInt, {1}, dev);
    if (shared > 0) {
      pages = static_cast<const int*>(pp.data_ptr());
      len = static_cast<const int*>(pl.data_ptr());
    }
  }
  c10::cuda::CUDAGuard guard((c10::DeviceIndex)dev);
  bool made;
  const Tensor O = output("O", a[8], at::kBFloat16, {B, Hq, d}, Q, &made);
  const Tensor L = output("L", a[9], at::kFloat, {B, Hq}, Q, &made);
  Tensor ws;
  if (a[10] == Py_None) {
    const size_t need =
        fa_prefix_workspace_bytes(as_int(B), as_int(Hq), as_int(c[1]), as_int(d),
                                  as_int(shared * c[2]), as_int(width * c[2]));
    if (need == 0) value_error("invalid sizes for the decode workspace");
    ws = at::empty({(long long)need}, Q.options().dtype(at::kByte));
  } else {
    ws = tensor("workspace", a[10]);
  }
  const size_t bytes = workspace_bytes(ws, dev);
  check("fa_prefix_decode",
        fa_prefix_decode(Q.data_ptr(), Kc.data_ptr(), Vc.data_ptr(), pages, as_int(shared), len,
                         width > 0 ? static_cast<const int*>(table.data_ptr()) : nullptr,
                         as_int(width), static_cast<const int*>(lens.data_ptr()), as_int(B),
                         as_int(Hq), as_int(c[1]), as_int(d), as_int(c[0]), as_int(c[2]),
                         scale_of(a[7], d), O.data_ptr(), static_cast<float*>(L.data_ptr()),
                         ws.data_ptr(), bytes, stream_of(dev)));
  return Py_BuildValue("(NN)", THPVariable_Wrap(O), THPVariable_Wrap(L));
  END_HANDLE_TH_ERRORS
}

PyObject* set_error(PyObject*, PyObject* cls) {
  Py_INCREF(cls);
  Py_XDECREF(g_error);
  g_error = cls;
  Py_RETURN_NONE;
}

#define FA_FAST(name) {#name, (PyCFunction)(void (*)(void))name, METH_FASTCALL, nullptr}
PyMethodDef methods[] = {FA_FAST(packed_forward), FA_FAST(packed_backward), FA_FAST(cache_append),
                         FA_FAST(prefix_decode), {"set_error", set_error, METH_O, nullptr},
                         {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_fa_binding", nullptr, -1, methods};

}  // namespace

PyMODINIT_FUNC PyInit__fa_binding() { return PyModule_Create(&module); }
