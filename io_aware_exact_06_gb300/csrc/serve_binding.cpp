// The torch conveniences of include/attn_norm.h, attn_cache.h and attn_verify.h as a
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
#include "../../include/attn_verify.h"

namespace {

struct Calls {
  decltype(&attn_qk_norm_rope) norm_rope;
  decltype(&attn_qk_norm_rope_bwd) norm_rope_bwd;
  decltype(&attn_qk_norm_rope_bwd_workspace) norm_rope_bwd_workspace;
  decltype(&attn_cache_write) cache_write;
  decltype(&attn_cache_read) cache_read;
  decltype(&attn_fwd_tree) fwd_tree;
  decltype(&attn_fwd_tree_workspace) fwd_tree_workspace;
  decltype(&attn_fwd_prefix) fwd_prefix;
  decltype(&attn_fwd_prefix_workspace) fwd_prefix_workspace;
  decltype(&attn_cache_fork) cache_fork;
  decltype(&attn_cache_fork_workspace) cache_fork_workspace;
  decltype(&attn_cache_copy) cache_copy;
  decltype(&attn_cache_compact) cache_compact;
  decltype(&attn_verify_drafts) verify_drafts;
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
  for (const at::Tensor& t : ts) PyTuple_SET_ITEM(r, i++, t.defined() ? THPVariable_Wrap(t) : Py_NewRef(Py_None));
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

// The cache without a page table.
attn_paged_cache pages_of(PyObject* k_cache, PyObject* v_cache, PyObject* k_scale, PyObject* v_scale) {
  const at::Tensor &k = tensor(k_cache, "k_cache"), &v = tensor(v_cache, "v_cache");
  const at::Tensor *ks = optional_tensor(k_scale, "k_scale"), *vs = optional_tensor(v_scale, "v_scale");
  TORCH_CHECK_VALUE(!ks == !vs, "k_scale and v_scale go together");
  const at::ScalarType type = k.scalar_type();
  TORCH_CHECK_TYPE(!ks || type == at::kFloat8_e4m3fn || type == at::kByte,
                   "a cache with scales holds e4m3 codes (float8_e4m3fn or uint8)");
  TORCH_CHECK_TYPE(ks || type == at::kBFloat16, "a cache without scales must be bf16");
  plain_dims(k, "k_cache", type, 4);
  plain_shape(v, "v_cache", type, k.sizes());
  const at::Device dev = k.device();
  same_device(v, "v_cache", dev);
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
  c.num_pages = extent(k.size(0), "k_cache");
  c.page_size = extent(k.size(1), "k_cache");
  c.H = extent(k.size(2), "k_cache");
  c.d = extent(k.size(3), "k_cache");
  return c;
}

// k_cache, v_cache, page_table, k_scale, v_scale
attn_paged_cache cache_of(PyObject* const* a, int64_t B) {
  const at::Tensor& table = tensor(a[2], "page_table");
  attn_paged_cache c = pages_of(a[0], a[1], a[3], a[4]);
  plain_shape(table, "page_table", at::kInt, {B, table.dim() == 2 ? table.size(1) : 0});
  same_device(table, "page_table", tensor(a[0], "k_cache").device());
  c.page_table = static_cast<const int32_t*>(table.data_ptr());
  c.page_table_stride = extent(table.size(1), "page_table");
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
// out, lse; with shared prefixes also cu_groups, prefix_lens, max_group, max_prefix
template <bool kPrefix>
PyObject* decode(PyObject* const* a, Py_ssize_t n) {
  want(n, kPrefix ? 19 : 15);
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
  const int32_t *lens_p = static_cast<const int32_t*>(lens.data_ptr()), *cu_p = static_cast<const int32_t*>(cu.data_ptr());
  const int64_t* mask_p = mask ? static_cast<const int64_t*>(mask->data_ptr()) : nullptr;
  float* l_p = static_cast<float*>(l.data_ptr());
  at::Tensor ws;
  int st;
  if constexpr (kPrefix) {
    const at::Tensor &groups = tensor(a[15], "cu_groups"), &prefix = tensor(a[16], "prefix_lens");
    plain_dims(prefix, "prefix_lens", at::kInt, 1);
    plain_shape(groups, "cu_groups", at::kInt, {prefix.size(0) + 1});
    same_device(groups, "cu_groups", dev);
    same_device(prefix, "prefix_lens", dev);
    const int n_groups = extent(prefix.size(0), "prefix_lens"), max_group = to_int(a[17], "max_group"),
              max_prefix = to_int(a[18], "max_prefix");
    const size_t bytes =
        calls.fwd_prefix_workspace(Bi, q.T, q.H, c.H, c.d, max_new, max_len, n_groups, max_group, max_prefix, splits);
    if (bytes) ws = make({static_cast<int64_t>(bytes)}, at::kByte, dev);
    st = calls.fwd_prefix(q.p, q.stride, &c, lens_p, cu_p, mask_p, static_cast<const int32_t*>(groups.data_ptr()),
                          static_cast<const int32_t*>(prefix.data_ptr()), o.data_ptr(), l_p, Bi, q.T, q.H, max_new,
                          max_len, n_groups, max_group, max_prefix, scale, splits, bytes ? ws.data_ptr() : nullptr, bytes,
                          stream_of(dev));
  } else {
    const size_t bytes = calls.fwd_tree_workspace(Bi, q.T, q.H, c.H, c.d, max_new, max_len, splits);
    if (bytes) ws = make({static_cast<int64_t>(bytes)}, at::kByte, dev);
    st = calls.fwd_tree(q.p, q.stride, &c, lens_p, cu_p, mask_p, o.data_ptr(), l_p, Bi, q.T, q.H, max_new, max_len, scale,
                        splits, bytes ? ws.data_ptr() : nullptr, bytes, stream_of(dev));
  }
  return st != ATTN_OK ? PyLong_FromLong(st) : pack({o, l});
}
PyObject* tree_decode(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  return decode<false>(a, n);
  END_HANDLE_TH_ERRORS
}
PyObject* prefix_decode(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  return decode<true>(a, n);
  END_HANDLE_TH_ERRORS
}

const int32_t* ints(const at::Tensor& t) { return static_cast<const int32_t*>(t.data_ptr()); }

// An int32 vector [length] on the device.
const at::Tensor& int_vector(PyObject* o, const char* name, int64_t length, const at::Device& dev) {
  const at::Tensor& t = tensor(o, name);
  plain_shape(t, name, at::kInt, {length});
  same_device(t, name, dev);
  return t;
}

// page_table, seqlens, parents, new_seqlens, refs, page_size, out, refs_out
PyObject* cache_fork(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  want(n, 8);
  const at::Tensor &table = tensor(a[0], "page_table"), &parents = tensor(a[2], "parents"), &refs = tensor(a[4], "refs");
  plain_dims(table, "page_table", at::kInt, 2);
  plain_dims(parents, "parents", at::kInt, 1);
  plain_dims(refs, "refs", at::kInt, 1);
  const at::Device dev = table.device();
  same_device(parents, "parents", dev);
  same_device(refs, "refs", dev);
  const int B = extent(table.size(0), "page_table"), W = extent(table.size(1), "page_table"),
            N = extent(parents.size(0), "parents"), pages = extent(refs.size(0), "refs"), page = to_int(a[5], "page_size");
  const at::Tensor &lens = int_vector(a[1], "seqlens", B, dev), &to = int_vector(a[3], "new_seqlens", N, dev);
  const at::Tensor *og = optional_tensor(a[6], "out"), *rg = optional_tensor(a[7], "refs_out");
  const c10::cuda::CUDAGuard guard(dev);
  const at::Tensor out = og ? *og : make({N, W}, at::kInt, dev), now = rg ? *rg : make({pages}, at::kInt, dev);
  plain_shape(out, "out", at::kInt, {N, W});
  plain_shape(now, "refs_out", at::kInt, {pages});
  same_device(out, "out", dev);
  same_device(now, "refs_out", dev);
  const at::Tensor src = make({N}, at::kInt, dev), dst = make({N}, at::kInt, dev);
  const size_t bytes = calls.cache_fork_workspace(B, N, W, pages, page);
  at::Tensor ws;
  if (bytes) ws = make({static_cast<int64_t>(bytes)}, at::kByte, dev);
  const int st = calls.cache_fork(ints(table), W, ints(lens), B, ints(parents), ints(to), N, ints(refs),
                                  static_cast<int32_t*>(now.data_ptr()), pages, page, static_cast<int32_t*>(out.data_ptr()),
                                  static_cast<int32_t*>(src.data_ptr()), static_cast<int32_t*>(dst.data_ptr()),
                                  bytes ? ws.data_ptr() : nullptr, bytes, stream_of(dev));
  return st != ATTN_OK ? PyLong_FromLong(st) : pack({out, now, src, dst});
  END_HANDLE_TH_ERRORS
}

// k_cache, v_cache, k_scale, v_scale, src, dst
PyObject* cache_copy(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  want(n, 6);
  const attn_paged_cache c = pages_of(a[0], a[1], a[2], a[3]);
  const at::Device dev = tensor(a[0], "k_cache").device();
  const at::Tensor& src = tensor(a[4], "src");
  plain_dims(src, "src", at::kInt, 1);
  same_device(src, "src", dev);
  const at::Tensor& dst = int_vector(a[5], "dst", src.size(0), dev);
  const c10::cuda::CUDAGuard guard(dev);
  return PyLong_FromLong(calls.cache_copy(&c, ints(src), ints(dst), extent(src.size(0), "src"), stream_of(dev)));
  END_HANDLE_TH_ERRORS
}

// k_cache, v_cache, page_table, k_scale, v_scale, seqlens, cu_seqlens, path, accepted
PyObject* cache_compact(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  want(n, 9);
  const at::Tensor &lens = tensor(a[5], "seqlens"), &path = tensor(a[7], "path");
  const attn_paged_cache c = cache_of(a, lens.dim() == 1 ? lens.size(0) : -1);
  const int64_t B = batch_of(lens);
  plain_dims(path, "path", at::kInt, 1);
  const at::Device dev = tensor(a[0], "k_cache").device();
  same_device(lens, "seqlens", dev);
  same_device(path, "path", dev);
  const at::Tensor &cu = int_vector(a[6], "cu_seqlens", B + 1, dev), &kept = int_vector(a[8], "accepted", B, dev);
  const c10::cuda::CUDAGuard guard(dev);
  return PyLong_FromLong(calls.cache_compact(&c, ints(lens), ints(cu), ints(path), ints(kept), extent(B, "seqlens"),
                                             extent(path.size(0), "path"), stream_of(dev)));
  END_HANDLE_TH_ERRORS
}

// tokens, probs, draft_probs, cu_seqlens, mask, u_accept, u_next, seqlens
PyObject* verify_drafts(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  want(n, 8);
  const at::Tensor &tokens = tensor(a[0], "tokens"), &probs = tensor(a[1], "probs"), &cu = tensor(a[3], "cu_seqlens"),
                   &u = tensor(a[5], "u_accept"), &un = tensor(a[6], "u_next");
  const at::Tensor *draft = optional_tensor(a[2], "draft_probs"), *mask = optional_tensor(a[4], "mask"),
                   *lens = optional_tensor(a[7], "seqlens");
  plain_dims(tokens, "tokens", at::kInt, 1);
  const int64_t T = tokens.size(0);
  const at::Device dev = tokens.device();
  const at::ScalarType type = probs.scalar_type();
  TORCH_CHECK_TYPE(type == at::kFloat || type == at::kBFloat16, "probs must be fp32 or bf16");
  auto rows = [&](const at::Tensor& t, const char* name) {
    TORCH_CHECK_TYPE(t.scalar_type() == type, name, " must be ", type);
    TORCH_CHECK_VALUE(t.is_cuda() && t.dim() == 2 && t.size(0) == T && t.size(1) == probs.size(1), name,
                      " must be a CUDA tensor [tokens, vocabulary]");
    TORCH_CHECK_VALUE(t.size(1) >= 1 && (t.size(1) == 1 || t.stride(1) == 1) && (T <= 1 || t.stride(0) >= t.size(1)), name,
                      ": a row must be contiguous, and rows must not overlap");
    same_device(t, name, dev);
    return T > 1 ? t.stride(0) : t.size(1);
  };
  const int64_t p_stride = rows(probs, "probs"), q_stride = draft ? rows(*draft, "draft_probs") : 0;
  plain_dims(cu, "cu_seqlens", at::kInt, 1);
  TORCH_CHECK_VALUE(cu.size(0) >= 1, "cu_seqlens must hold at least one offset");
  const int64_t B = cu.size(0) - 1;
  plain_shape(u, "u_accept", at::kFloat, {T});
  plain_shape(un, "u_next", at::kFloat, {B});
  same_device(cu, "cu_seqlens", dev);
  same_device(u, "u_accept", dev);
  same_device(un, "u_next", dev);
  if (mask) {
    plain_shape(*mask, "mask", at::kLong, {T});
    same_device(*mask, "mask", dev);
  }
  if (lens) int_vector(a[7], "seqlens", B, dev);
  const c10::cuda::CUDAGuard guard(dev);
  const at::Tensor path = make({T}, at::kInt, dev), kept = make({B}, at::kInt, dev), next = make({B}, at::kInt, dev);
  at::Tensor to;
  if (lens) to = make({B}, at::kInt, dev);
  const int st = calls.verify_drafts(
      ints(tokens), probs.data_ptr(), p_stride, draft ? draft->data_ptr() : nullptr, q_stride, type == at::kBFloat16, ints(cu),
      mask ? static_cast<const int64_t*>(mask->data_ptr()) : nullptr, static_cast<const float*>(u.data_ptr()),
      static_cast<const float*>(un.data_ptr()), lens ? ints(*lens) : nullptr, static_cast<int32_t*>(path.data_ptr()),
      static_cast<int32_t*>(kept.data_ptr()), static_cast<int32_t*>(next.data_ptr()),
      lens ? static_cast<int32_t*>(to.data_ptr()) : nullptr, extent(B, "cu_seqlens"), extent(T, "tokens"),
      extent(probs.size(1), "probs"), stream_of(dev));
  return st != ATTN_OK ? PyLong_FromLong(st) : pack({path, kept, next, to});
  END_HANDLE_TH_ERRORS
}

// Addresses of the library's calls, in the order of Calls.
PyObject* bind(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  constexpr int kCalls = 14;
  want(n, kCalls);
  void* p[kCalls];
  for (int i = 0; i < kCalls; ++i) {
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
  calls.fwd_prefix = reinterpret_cast<decltype(calls.fwd_prefix)>(p[7]);
  calls.fwd_prefix_workspace = reinterpret_cast<decltype(calls.fwd_prefix_workspace)>(p[8]);
  calls.cache_fork = reinterpret_cast<decltype(calls.cache_fork)>(p[9]);
  calls.cache_fork_workspace = reinterpret_cast<decltype(calls.cache_fork_workspace)>(p[10]);
  calls.cache_copy = reinterpret_cast<decltype(calls.cache_copy)>(p[11]);
  calls.cache_compact = reinterpret_cast<decltype(calls.cache_compact)>(p[12]);
  calls.verify_drafts = reinterpret_cast<decltype(calls.verify_drafts)>(p[13]);
  Py_RETURN_NONE;
  END_HANDLE_TH_ERRORS
}

#define FAST(name) {#name, reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(name)), METH_FASTCALL, nullptr}
PyMethodDef methods[] = {FAST(bind),          FAST(norm_rope),     FAST(norm_rope_bwd), FAST(cache_write),
                         FAST(cache_read),    FAST(tree_decode),   FAST(prefix_decode), FAST(cache_fork),
                         FAST(cache_copy),    FAST(cache_compact), FAST(verify_drafts), {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_serve", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__serve(void) { return PyModule_Create(&module); }
