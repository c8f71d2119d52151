// The torch conveniences of include/attn_norm.h and include/attn_cache.h as a
// CPython module: checks of what the C calls cannot see (types, shapes,
// strides, devices), outputs and workspaces from torch's allocator, the call.
// These operators run once per layer and step on a few tokens; marshalling
// them in Python took 22 to 39 us a call on the Grace cores (the kernels 2 to
// 11 us), which is why this part is compiled.  A refused argument raises
// TypeError or ValueError; a status other than ATTN_OK is returned as an int.
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <ATen/core/Tensor.h>
#include <ATen/ops/empty.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <c10/util/Exception.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <climits>
#include <cmath>
#include <initializer_list>

#include "../../include/attn_cache.h"
#include "../../include/attn_norm.h"

namespace {

struct Calls {
  decltype(&attn_qk_norm_rope) norm_rope;
  decltype(&attn_qk_norm_rope_bwd) norm_rope_bwd;
  decltype(&attn_qk_norm_rope_bwd_workspace) norm_rope_bwd_workspace;
  decltype(&attn_cache_write) cache_write;
  decltype(&attn_cache_read) cache_read;
  decltype(&attn_fwd_tree) fwd_tree;
  decltype(&attn_fwd_tree_workspace) fwd_tree_workspace;
} calls;

const at::Tensor& tensor(PyObject* o, const char* name) {
  TORCH_CHECK_TYPE(THPVariable_Check(o), name, " must be a tensor");
  return THPVariable_Unpack(o);
}
const at::Tensor* optional_tensor(PyObject* o, const char* name) {
  return o == Py_None ? nullptr : &tensor(o, name);
}

int to_int(PyObject* o, const char* name) {
  const long long v = PyLong_AsLongLong(o);
  if (v == -1 && PyErr_Occurred()) {
    PyErr_Clear();
    TORCH_CHECK_TYPE(false, name, " must be an integer");
  }
  TORCH_CHECK_VALUE(v >= INT_MIN && v <= INT_MAX, name, " is out of range");
  return static_cast<int>(v);
}
float to_float(PyObject* o, const char* name) {
  const double v = PyFloat_AsDouble(o);
  if (v == -1.0 && PyErr_Occurred()) {
    PyErr_Clear();
    TORCH_CHECK_TYPE(false, name, " must be a number");
  }
  return static_cast<float>(v);
}
int extent(int64_t n, const char* name) {
  TORCH_CHECK_VALUE(n <= INT_MAX, name, " is too large");
  return static_cast<int>(n);
}

// bf16 rows [T, H, d] on a GPU: the heads of a token contiguous, tokens any
// distance apart.  Extents given as -1 are free.
struct Rows {
  void* p;
  int T, H, d;
  int64_t stride;
};
Rows rows_of(const at::Tensor& t, const char* name, int64_t T, int64_t H, int64_t d) {
  TORCH_CHECK_TYPE(t.scalar_type() == at::kBFloat16, name, " must be bf16");
  TORCH_CHECK_VALUE(t.is_cuda() && t.dim() == 3, name, " must be a CUDA tensor [tokens, heads, d]");
  TORCH_CHECK_VALUE((T < 0 || t.size(0) == T) && (H < 0 || t.size(1) == H) && (d < 0 || t.size(2) == d), name,
                    " has the wrong shape: ", t.sizes());
  TORCH_CHECK_VALUE(t.stride(2) == 1 && (t.size(1) <= 1 || t.stride(1) == t.size(2)) &&
                        (t.size(0) <= 1 || t.stride(0) >= t.size(1) * t.size(2)),
                    name, ": the heads of a token must be contiguous and tokens must not overlap");
  return {t.data_ptr(), extent(t.size(0), name), extent(t.size(1), name), extent(t.size(2), name),
          t.size(0) > 1 ? t.stride(0) : t.size(1) * t.size(2)};
}

// Contiguous, on a GPU, of the given type and number of dimensions (or shape).
void plain_dims(const at::Tensor& t, const char* name, at::ScalarType type, int64_t dims) {
  TORCH_CHECK_TYPE(t.scalar_type() == type, name, " must be ", type);
  TORCH_CHECK_VALUE(t.is_cuda() && t.is_contiguous() && t.dim() == dims, name, " must be a contiguous CUDA tensor of ",
                    dims, " dimensions");
}
void plain_shape(const at::Tensor& t, const char* name, at::ScalarType type, at::IntArrayRef shape) {
  plain_dims(t, name, type, static_cast<int64_t>(shape.size()));
  TORCH_CHECK_VALUE(t.sizes() == shape, name, " must have the shape ", shape, ", not ", t.sizes());
}

void same_device(const at::Tensor& t, const char* name, const at::Device& d) {
  TORCH_CHECK_VALUE(t.device() == d, name, " must be on ", d, ", not ", t.device());
}

attn_rotary rotary_of(PyObject* cos_o, PyObject* sin_o, PyObject* pos_o, PyObject* sections, PyObject* interleaved,
                      int T, const at::Device& dev) {
  const at::Tensor &c = tensor(cos_o, "cos"), &s = tensor(sin_o, "sin"), &pos = tensor(pos_o, "positions");
  plain_dims(c, "cos", at::kFloat, 2);
  plain_shape(s, "sin", at::kFloat, c.sizes());
  const int64_t axes = pos.dim() == 1 ? 1 : pos.dim() == 2 ? pos.size(0) : 0;
  plain_dims(pos, "positions", at::kInt, pos.dim());
  TORCH_CHECK_VALUE(axes >= 1 && axes <= 3, "positions must have one to three axes");
  TORCH_CHECK_VALUE(pos.size(-1) == T, "positions must name a position for each of the ", T, " tokens");
  same_device(c, "cos", dev);
  same_device(s, "sin", dev);
  same_device(pos, "positions", dev);
  attn_rotary r{};
  r.cos = static_cast<const float*>(c.data_ptr());
  r.sin = static_cast<const float*>(s.data_ptr());
  r.positions = static_cast<const int32_t*>(pos.data_ptr());
  r.table_len = extent(c.size(0), "cos");
  TORCH_CHECK_VALUE(c.size(1) <= 1 << 20, "cos has too many columns");
  r.rot = 2 * static_cast<int>(c.size(1));
  r.axes = static_cast<int>(axes);
  const int inter = PyObject_IsTrue(interleaved);
  if (inter < 0) throw python_error();
  r.interleaved = inter;
  if (sections == Py_None) {
    TORCH_CHECK_VALUE(axes == 1, "positions with several axes need sections");
    return r;
  }
  PyObject* seq = PySequence_Fast(sections, "sections must be a sequence");
  if (!seq) throw python_error();
  const Py_ssize_t n = PySequence_Fast_GET_SIZE(seq);
  int64_t sum = 0;
  bool ok = n == axes;
  for (Py_ssize_t i = 0; ok && i < n; ++i) {
    const long v = PyLong_AsLong(PySequence_Fast_GET_ITEM(seq, i));
    if (v == -1 && PyErr_Occurred()) PyErr_Clear();
    ok = v >= 0 && v <= 1 << 20;
    r.section[i] = static_cast<int>(v);
    sum += v;
  }
  Py_DECREF(seq);
  TORCH_CHECK_VALUE(ok && sum == c.size(1), "sections must be ", axes, " counts of pairs that add up to ", c.size(1));
  return r;
}

at::Tensor make(at::IntArrayRef shape, at::ScalarType type, const at::Device& d) {
  return at::empty(shape, at::TensorOptions().dtype(type).device(d));
}

attn_stream_t stream_of(const at::Device& d) {
  return reinterpret_cast<attn_stream_t>(c10::cuda::getCurrentCUDAStream(d.index()).stream());
}

PyObject* pack(std::initializer_list<at::Tensor> ts) {
  PyObject* r = PyTuple_New(static_cast<Py_ssize_t>(ts.size()));
  if (!r) throw python_error();
  Py_ssize_t i = 0;
  for (const at::Tensor& t : ts) PyTuple_SET_ITEM(r, i++, THPVariable_Wrap(t));
  return r;
}

void want(Py_ssize_t got, Py_ssize_t n) { TORCH_CHECK_TYPE(got == n, "expected ", n, " arguments, got ", got); }

// q, k, wq, wk, cos, sin, positions, eps, sections, interleaved, q_out, k_out
PyObject* norm_rope(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  want(n, 12);
  const at::Tensor &qt = tensor(a[0], "q"), &kt = tensor(a[1], "k"), &wq = tensor(a[2], "wq"), &wk = tensor(a[3], "wk");
  const Rows q = rows_of(qt, "q", -1, -1, -1), k = rows_of(kt, "k", q.T, -1, q.d);
  const at::Device dev = qt.device();
  plain_shape(wq, "wq", at::kBFloat16, {q.d});
  plain_shape(wk, "wk", at::kBFloat16, {q.d});
  const attn_rotary rot = rotary_of(a[4], a[5], a[6], a[8], a[9], q.T, dev);
  same_device(kt, "k", dev);
  same_device(wq, "wq", dev);
  same_device(wk, "wk", dev);
  const c10::cuda::CUDAGuard guard(dev);
  const at::Tensor *qg = optional_tensor(a[10], "q_out"), *kg = optional_tensor(a[11], "k_out");
  const at::Tensor qo = qg ? *qg : make({q.T, q.H, q.d}, at::kBFloat16, dev);
  const at::Tensor ko = kg ? *kg : make({k.T, k.H, k.d}, at::kBFloat16, dev);
  const Rows qr = rows_of(qo, "q_out", q.T, q.H, q.d), kr = rows_of(ko, "k_out", k.T, k.H, k.d);
  same_device(qo, "q_out", dev);
  same_device(ko, "k_out", dev);
  const int st = calls.norm_rope(q.p, q.stride, k.p, k.stride, wq.data_ptr(), wk.data_ptr(), qr.p, qr.stride, kr.p,
                                 kr.stride, q.T, q.H, k.H, q.d, to_float(a[7], "eps"), &rot, stream_of(dev));
  return st != ATTN_OK ? PyLong_FromLong(st) : pack({qo, ko});
  END_HANDLE_TH_ERRORS
}

// q, k, wq, wk, cos, sin, positions, dq_out, dk_out, eps, sections, interleaved
PyObject* norm_rope_bwd(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  want(n, 12);
  const at::Tensor &qt = tensor(a[0], "q"), &kt = tensor(a[1], "k"), &wq = tensor(a[2], "wq"), &wk = tensor(a[3], "wk");
  const at::Tensor &gqt = tensor(a[7], "dq_out"), &gkt = tensor(a[8], "dk_out");
  const Rows q = rows_of(qt, "q", -1, -1, -1), k = rows_of(kt, "k", q.T, -1, q.d);
  const Rows gq = rows_of(gqt, "dq_out", q.T, q.H, q.d), gk = rows_of(gkt, "dk_out", k.T, k.H, k.d);
  const at::Device dev = qt.device();
  plain_shape(wq, "wq", at::kBFloat16, {q.d});
  plain_shape(wk, "wk", at::kBFloat16, {q.d});
  const attn_rotary rot = rotary_of(a[4], a[5], a[6], a[10], a[11], q.T, dev);
  same_device(kt, "k", dev);
  same_device(wq, "wq", dev);
  same_device(wk, "wk", dev);
  same_device(gqt, "dq_out", dev);
  same_device(gkt, "dk_out", dev);
  const c10::cuda::CUDAGuard guard(dev);
  const at::Tensor dq = make({q.T, q.H, q.d}, at::kBFloat16, dev), dk = make({k.T, k.H, k.d}, at::kBFloat16, dev);
  const at::Tensor dwq = make({q.d}, at::kFloat, dev), dwk = make({q.d}, at::kFloat, dev);
  const size_t bytes = calls.norm_rope_bwd_workspace(q.T, q.H, k.H, q.d);
  const at::Tensor ws = make({static_cast<int64_t>(bytes)}, at::kByte, dev);
  const int st = calls.norm_rope_bwd(q.p, q.stride, k.p, k.stride, wq.data_ptr(), wk.data_ptr(), gq.p, gq.stride, gk.p,
                                     gk.stride, dq.data_ptr(), (int64_t)q.H * q.d, dk.data_ptr(), (int64_t)k.H * k.d,
                                     static_cast<float*>(dwq.data_ptr()), static_cast<float*>(dwk.data_ptr()), q.T, q.H,
                                     k.H, q.d, to_float(a[9], "eps"), &rot, ws.data_ptr(), bytes, stream_of(dev));
  return st != ATTN_OK ? PyLong_FromLong(st) : pack({dq, dk, dwq, dwk});
  END_HANDLE_TH_ERRORS
}

// k_cache, v_cache, page_table, k_scale, v_scale
attn_paged_cache cache_of(PyObject* const* a, int64_t B) {
  const at::Tensor &k = tensor(a[0], "k_cache"), &v = tensor(a[1], "v_cache"), &table = tensor(a[2], "page_table");
  const at::Tensor *ks = optional_tensor(a[3], "k_scale"), *vs = optional_tensor(a[4], "v_scale");
  TORCH_CHECK_VALUE(!ks == !vs, "k_scale and v_scale go together");
  const at::ScalarType type = k.scalar_type();
  TORCH_CHECK_TYPE(!ks || type == at::kFloat8_e4m3fn || type == at::kByte,
                   "a cache with scales holds e4m3 codes (float8_e4m3fn or uint8)");
  TORCH_CHECK_TYPE(ks || type == at::kBFloat16, "a cache without scales must be bf16");
  plain_dims(k, "k_cache", type, 4);
  plain_shape(v, "v_cache", type, k.sizes());
  plain_shape(table, "page_table", at::kInt, {B, table.dim() == 2 ? table.size(1) : 0});
  const at::Device dev = k.device();
  same_device(v, "v_cache", dev);
  same_device(table, "page_table", dev);
  attn_paged_cache c{};
  c.k = k.data_ptr();
  c.v = v.data_ptr();
  if (ks) {
    plain_shape(*ks, "k_scale", at::kFloat, {k.size(0), k.size(2), k.size(1)});
    plain_shape(*vs, "v_scale", at::kFloat, {k.size(0), k.size(2), k.size(1)});
    same_device(*ks, "k_scale", dev);
    same_device(*vs, "v_scale", dev);
    c.k_scale = static_cast<float*>(ks->data_ptr());
    c.v_scale = static_cast<float*>(vs->data_ptr());
  }
  c.page_table = static_cast<const int32_t*>(table.data_ptr());
  c.page_table_stride = extent(table.size(1), "page_table");
  c.num_pages = extent(k.size(0), "k_cache");
  c.page_size = extent(k.size(1), "k_cache");
  c.H = extent(k.size(2), "k_cache");
  c.d = extent(k.size(3), "k_cache");
  return c;
}

// int32 lengths [B] and offsets [B + 1]
int64_t batch_of(const at::Tensor& lens) {
  plain_dims(lens, "seqlens", at::kInt, 1);
  return lens.size(0);
}

// k, v, k_cache, v_cache, page_table, k_scale, v_scale, seqlens, cu_seqlens
PyObject* cache_write(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  want(n, 9);
  const at::Tensor &kt = tensor(a[0], "k"), &vt = tensor(a[1], "v"), &lens = tensor(a[7], "seqlens"),
                   &cu = tensor(a[8], "cu_seqlens");
  const attn_paged_cache c = cache_of(a + 2, lens.dim() == 1 ? lens.size(0) : -1);
  const int64_t B = batch_of(lens);
  const Rows k = rows_of(kt, "k", -1, c.H, c.d), v = rows_of(vt, "v", k.T, c.H, c.d);
  plain_shape(cu, "cu_seqlens", at::kInt, {B + 1});
  const at::Device dev = kt.device();
  same_device(vt, "v", dev);
  same_device(tensor(a[2], "k_cache"), "k_cache", dev);
  same_device(lens, "seqlens", dev);
  same_device(cu, "cu_seqlens", dev);
  const c10::cuda::CUDAGuard guard(dev);
  return PyLong_FromLong(calls.cache_write(&c, k.p, k.stride, v.p, v.stride,
                                           static_cast<const int32_t*>(lens.data_ptr()),
                                           static_cast<const int32_t*>(cu.data_ptr()), extent(B, "seqlens"), k.T,
                                           stream_of(dev)));
  END_HANDLE_TH_ERRORS
}

// k_cache, v_cache, page_table, k_scale, v_scale, cu_seqlens, total
PyObject* cache_read(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  want(n, 7);
  const at::Tensor& cu = tensor(a[5], "cu_seqlens");
  const attn_paged_cache c = cache_of(a, cu.dim() == 1 ? cu.size(0) - 1 : -1);
  plain_dims(cu, "cu_seqlens", at::kInt, 1);
  TORCH_CHECK_VALUE(cu.size(0) >= 1, "cu_seqlens must hold at least one offset");
  const int total = to_int(a[6], "total");
  TORCH_CHECK_VALUE(total >= 0, "total must not be negative");
  const at::Device dev = cu.device();
  same_device(tensor(a[0], "k_cache"), "k_cache", dev);
  const c10::cuda::CUDAGuard guard(dev);
  const at::Tensor k = make({total, c.H, c.d}, at::kBFloat16, dev), v = make({total, c.H, c.d}, at::kBFloat16, dev);
  const int st = calls.cache_read(&c, k.data_ptr(), v.data_ptr(), static_cast<const int32_t*>(cu.data_ptr()),
                                  extent(cu.size(0) - 1, "cu_seqlens"), total, stream_of(dev));
  return st != ATTN_OK ? PyLong_FromLong(st) : pack({k, v});
  END_HANDLE_TH_ERRORS
}

// q, k_cache, v_cache, page_table, k_scale, v_scale, seqlens, cu_seqlens, max_new, max_len, mask, scale, num_splits,
// out, lse
PyObject* tree_decode(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  want(n, 15);
  const at::Tensor &qt = tensor(a[0], "q"), &lens = tensor(a[6], "seqlens"), &cu = tensor(a[7], "cu_seqlens");
  const attn_paged_cache c = cache_of(a + 1, lens.dim() == 1 ? lens.size(0) : -1);
  const int64_t B = batch_of(lens);
  const Rows q = rows_of(qt, "q", -1, -1, c.d);
  TORCH_CHECK_VALUE(q.H >= 1 && c.H >= 1 && q.H % c.H == 0,
                    "the query heads must be a multiple of the cache's heads");
  plain_shape(cu, "cu_seqlens", at::kInt, {B + 1});
  const at::Device dev = qt.device();
  same_device(tensor(a[1], "k_cache"), "k_cache", dev);
  same_device(lens, "seqlens", dev);
  same_device(cu, "cu_seqlens", dev);
  const int max_new = to_int(a[8], "max_new"), max_len = to_int(a[9], "max_len"), splits = to_int(a[12], "num_splits");
  const at::Tensor *mask = optional_tensor(a[10], "mask"), *og = optional_tensor(a[13], "out"),
                   *lg = optional_tensor(a[14], "lse");
  if (mask) {
    plain_shape(*mask, "mask", at::kLong, {q.T});
    same_device(*mask, "mask", dev);
  }
  const float scale = a[11] == Py_None ? 1.0f / std::sqrt(static_cast<float>(c.d)) : to_float(a[11], "scale");
  const c10::cuda::CUDAGuard guard(dev);
  const at::Tensor o = og ? *og : make({q.T, q.H, q.d}, at::kBFloat16, dev);
  const at::Tensor l = lg ? *lg : make({q.T, q.H}, at::kFloat, dev);
  if (og) {
    plain_shape(o, "out", at::kBFloat16, {q.T, q.H, q.d});
    same_device(o, "out", dev);
  }
  if (lg) {
    plain_shape(l, "lse", at::kFloat, {q.T, q.H});
    same_device(l, "lse", dev);
  }
  const int Bi = extent(B, "seqlens");
  const size_t bytes = calls.fwd_tree_workspace(Bi, q.T, q.H, c.H, c.d, max_new, max_len, splits);
  at::Tensor ws;
  if (bytes) ws = make({static_cast<int64_t>(bytes)}, at::kByte, dev);
  const int st = calls.fwd_tree(q.p, q.stride, &c, static_cast<const int32_t*>(lens.data_ptr()),
                                static_cast<const int32_t*>(cu.data_ptr()),
                                mask ? static_cast<const int64_t*>(mask->data_ptr()) : nullptr, o.data_ptr(),
                                static_cast<float*>(l.data_ptr()), Bi, q.T, q.H, max_new, max_len, scale, splits,
                                bytes ? ws.data_ptr() : nullptr, bytes, stream_of(dev));
  return st != ATTN_OK ? PyLong_FromLong(st) : pack({o, l});
  END_HANDLE_TH_ERRORS
}

// Addresses of the library's seven calls, in the order of Calls.
PyObject* bind(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  want(n, 7);
  void* p[7];
  for (int i = 0; i < 7; ++i) {
    p[i] = PyLong_AsVoidPtr(a[i]);
    if (!p[i]) throw python_error();
  }
  calls.norm_rope = reinterpret_cast<decltype(calls.norm_rope)>(p[0]);
  calls.norm_rope_bwd = reinterpret_cast<decltype(calls.norm_rope_bwd)>(p[1]);
  calls.norm_rope_bwd_workspace = reinterpret_cast<decltype(calls.norm_rope_bwd_workspace)>(p[2]);
  calls.cache_write = reinterpret_cast<decltype(calls.cache_write)>(p[3]);
  calls.cache_read = reinterpret_cast<decltype(calls.cache_read)>(p[4]);
  calls.fwd_tree = reinterpret_cast<decltype(calls.fwd_tree)>(p[5]);
  calls.fwd_tree_workspace = reinterpret_cast<decltype(calls.fwd_tree_workspace)>(p[6]);
  Py_RETURN_NONE;
  END_HANDLE_TH_ERRORS
}

#define FAST(name) {#name, reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(name)), METH_FASTCALL, nullptr}
PyMethodDef methods[] = {FAST(bind),       FAST(norm_rope),  FAST(norm_rope_bwd),          FAST(cache_write),
                         FAST(cache_read), FAST(tree_decode), {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_serve", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__serve(void) { return PyModule_Create(&module); }
