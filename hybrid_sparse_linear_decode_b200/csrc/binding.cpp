// The calls of PagedKVCache and GatedDeltaState from PyTorch tensors: argument checks, output tensors, the current
// stream, and the C ABI.  A decode step makes a few of these calls a layer, each of a few microseconds on the GPU, so
// they are compiled; nothing is computed here.
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/extension.h>

#include "../../include/hyb_attn.h"

namespace py = pybind11;
using at::Tensor;
using OptTensor = std::optional<Tensor>;

namespace {

[[noreturn]] void refuse(const std::string& what) { throw py::value_error(what); }

// Raises HybAttnError(fn, code).
[[noreturn]] void fail(const char* fn, int code) {
  const py::object cls = py::module_::import("hybrid_sparse_linear_decode_b200._abi").attr("HybAttnError");
  PyErr_SetObject(cls.ptr(), cls(fn, code).ptr());
  throw py::error_already_set();
}

std::string text_of(const Tensor& t) {
  std::ostringstream s;
  s << t.scalar_type() << " " << t.sizes() << " with strides " << t.strides() << " on " << t.device();
  return s.str();
}

bool on(const Tensor& t, int64_t index) { return t.is_cuda() && t.get_device() == index; }

// Token rows [rows, heads, d] whose heads are contiguous: the elements from row to row.
int64_t rows_of(const Tensor& t, const char* name, int64_t heads, int64_t d, int64_t index, at::ScalarType type) {
  if (t.dim() != 3 || t.size(1) != heads || t.size(2) != d || !on(t, index) || t.scalar_type() != type)
    refuse(std::string(name) + " has to be " + c10::toString(type) + " [rows, " + std::to_string(heads) + ", " + std::to_string(d) +
           "] on cuda:" + std::to_string(index) + ", not " + text_of(t));
  if (t.stride(2) != 1 || (t.stride(1) != d && heads != 1))
    refuse(std::string(name) + ": the heads of a row have to be contiguous, not " + text_of(t));
  return t.size(0) > 1 ? t.stride(0) : heads * d;
}

template <class T>
const T* vector_of(const Tensor& t, const char* name, at::ScalarType type, at::IntArrayRef shape, int64_t index) {
  if (t.scalar_type() != type || t.sizes() != shape || !on(t, index) || !t.is_contiguous()) {
    std::ostringstream s;
    s << name << " has to be a contiguous " << type << " " << shape << " tensor on cuda:" << index << ", not " << text_of(t);
    refuse(s.str());
  }
  return static_cast<const T*>(t.const_data_ptr());
}

int type_of(const Tensor& t, const char* name) {
  if (t.scalar_type() == at::kBFloat16) return HYB_TYPE_BF16;
  if (t.scalar_type() == at::kHalf) return HYB_TYPE_FP16;
  refuse(std::string(name) + " has to be bfloat16 or float16, not " + text_of(t));
}

int32_t int_of(int64_t x, const char* name) {
  if (x < INT32_MIN || x > INT32_MAX) refuse(std::string(name) + " does not fit 32 bits");
  return (int32_t)x;
}

// 0 selects a default, so what 32 bits would turn into 0 is refused.
float scale_of(double x) {
  if (x != 0 && (float)x == 0.f) refuse("scale does not fit 32 bits");
  return (float)x;
}

hyb_attn_paged_batch batch_of(int64_t index, int64_t status, const Tensor& cu, const Tensor& lens, const Tensor& table,
                              int64_t rows, int64_t max_new, int64_t max_len) {
  if (table.dim() != 2) refuse("page_table has to be [B, pages], not " + text_of(table));
  if (max_new < 1 && rows > 0) refuse("max_new has to be at least 1");
  const int64_t B = table.size(0);
  hyb_attn_paged_batch b;
  b.page_table = vector_of<int32_t>(table, "page_table", at::kInt, table.sizes(), index);
  b.cu_new = vector_of<int32_t>(cu, "cu", at::kInt, {B + 1}, index);
  b.kv_lens = vector_of<int32_t>(lens, "kv_lens", at::kInt, {B}, index);
  b.batch = int_of(B, "B");
  b.table_stride = int_of(table.size(1), "pages");
  b.n_new = int_of(rows, "rows");
  b.max_new = (int32_t)std::min(max_new, rows);
  b.max_len = (int32_t)std::min<int64_t>(std::max<int64_t>(max_len, 0), INT32_MAX);
  b.status = reinterpret_cast<uint32_t*>(status);
  return b;
}

py::object paged_append(int64_t cache_at, int64_t index, int64_t status, const Tensor& k, const Tensor& v, const Tensor& cu,
                        const Tensor& lens, const Tensor& table, int64_t max_new, const OptTensor& rope, bool interleaved,
                        const OptTensor& q, const OptTensor& q_out) {
  const auto& c = *reinterpret_cast<const hyb_attn_paged_cache*>(cache_at);
  const int type = type_of(k, "k");
  const at::ScalarType st = k.scalar_type();
  const int64_t ks = rows_of(k, "k", c.n_kv_heads, c.head_dim, index, st);
  const int64_t vs = rows_of(v, "v", c.n_kv_heads, c.head_dim, index, st);
  const int64_t n = k.size(0);
  if (v.size(0) != n) refuse("k and v have to have as many rows");
  const hyb_attn_paged_batch b = batch_of(index, status, cu, lens, table, n, max_new, 0);
  const float* angles = nullptr;
  int32_t n_pos = 0, rot = 0;
  if (rope.has_value()) {
    if (rope->dim() != 2) refuse("rope has to be [positions, rot_dim], not " + text_of(*rope));
    angles = vector_of<float>(*rope, "rope", at::kFloat, rope->sizes(), index);
    n_pos = int_of(rope->size(0), "positions");
    rot = int_of(rope->size(1), "rot_dim");
  }
  const c10::cuda::OptionalCUDAGuard guard(c10::Device(c10::kCUDA, (c10::DeviceIndex)index));
  Tensor to;
  int64_t heads = 0, qs = 0, os = 0;
  if (q.has_value()) {
    if (q->dim() != 3 || q->size(0) != n) refuse("q has to be [rows, n_q_heads, head_dim] with as many rows as k, not " + text_of(*q));
    heads = q->size(1);
    qs = rows_of(*q, "q", heads, c.head_dim, index, st);
    if (q_out.has_value()) {
      to = *q_out;
      os = rows_of(to, "q_out", heads, c.head_dim, index, st);
      if (to.size(0) != n) refuse("q_out has to have as many rows as q");
    } else {
      to = at::empty({n, heads, c.head_dim}, q->options());
      os = heads * c.head_dim;
    }
  } else if (q_out.has_value()) {
    refuse("q_out without q");
  }
  const int rc = hyb_attn_paged_append(&c, &b, type, k.const_data_ptr(), ks, v.const_data_ptr(), vs, angles, n_pos, rot, interleaved,
                                       q.has_value() ? q->const_data_ptr() : nullptr, qs, q.has_value() ? to.data_ptr() : nullptr, os,
                                       int_of(heads, "n_q_heads"), c10::cuda::getCurrentCUDAStream((c10::DeviceIndex)index).stream());
  if (rc < 0) fail("hyb_attn_paged_append", rc);
  return q.has_value() ? py::cast(to) : py::none();
}

py::object paged_attend(int64_t cache_at, int64_t index, int64_t status, const Tensor& q, const Tensor& cu, const Tensor& lens,
                        const Tensor& table, int64_t max_new, int64_t max_len, int64_t window, int64_t n_sink, double scale,
                        const OptTensor& out, bool return_lse) {
  const auto& c = *reinterpret_cast<const hyb_attn_paged_cache*>(cache_at);
  const float factor = scale_of(scale);
  const int type = type_of(q, "q");
  if (q.dim() != 3) refuse("q has to be [rows, n_q_heads, head_dim], not " + text_of(q));
  const int64_t n = q.size(0), heads = q.size(1);
  const int64_t qs = rows_of(q, "q", heads, c.head_dim, index, q.scalar_type());
  const hyb_attn_paged_batch b = batch_of(index, status, cu, lens, table, n, max_new, max_len);
  const c10::cuda::OptionalCUDAGuard guard(c10::Device(c10::kCUDA, (c10::DeviceIndex)index));
  int64_t os = heads * c.head_dim;
  Tensor to;
  if (out.has_value()) {
    to = *out;
    os = rows_of(to, "out", heads, c.head_dim, index, q.scalar_type());
    if (to.size(0) != n) refuse("out has to have as many rows as q");
  } else {
    to = at::empty({n, heads, c.head_dim}, q.options());
  }
  Tensor lse, ws;
  if (return_lse) lse = at::empty({n, heads}, q.options().dtype(at::kFloat));
  const size_t size = hyb_attn_paged_workspace_size(&c, &b, int_of(heads, "n_q_heads"));
  if (size > 0) ws = at::empty({(int64_t)size}, q.options().dtype(at::kByte));
  const int rc = hyb_attn_paged_attend(&c, &b, type, q.const_data_ptr(), qs, to.data_ptr(), os,
                                       return_lse ? static_cast<float*>(lse.data_ptr()) : nullptr, (int32_t)heads,
                                       int_of(window, "window"), int_of(n_sink, "n_sink"), factor,
                                       size > 0 ? ws.data_ptr() : nullptr, size,
                                       c10::cuda::getCurrentCUDAStream((c10::DeviceIndex)index).stream());
  if (rc < 0) fail("hyb_attn_paged_attend", rc);
  if (return_lse) return py::make_tuple(to, lse);
  return py::cast(to);
}

Tensor delta_run(int64_t state_at, int64_t index, int64_t status, const Tensor& q, const Tensor& k, const Tensor& v, const Tensor& g,
                 const Tensor& beta, const Tensor& cu, int64_t max_new, const OptTensor& slots, double scale, const OptTensor& out) {
  const auto& s = *reinterpret_cast<const hyb_attn_delta_state*>(state_at);
  const float factor = scale_of(scale);
  const int64_t qs = rows_of(q, "q", s.n_k_heads, s.key_dim, index, at::kBFloat16);
  const int64_t ks = rows_of(k, "k", s.n_k_heads, s.key_dim, index, at::kBFloat16);
  const int64_t vs = rows_of(v, "v", s.n_v_heads, s.value_dim, index, at::kBFloat16);
  const int64_t n = q.size(0);
  if (k.size(0) != n || v.size(0) != n) refuse("q, k and v have to have as many rows");
  if (cu.dim() != 1 || cu.size(0) < 2) refuse("cu has to be [B + 1], not " + text_of(cu));
  if (max_new < 1 && n > 0) refuse("max_new has to be at least 1");
  const int64_t B = cu.size(0) - 1;
  const float* gp = vector_of<float>(g, "g", at::kFloat, {n, s.n_v_heads}, index);
  const float* bp = vector_of<float>(beta, "beta", at::kFloat, {n, s.n_v_heads}, index);
  const int32_t* cup = vector_of<int32_t>(cu, "cu", at::kInt, {B + 1}, index);
  const int32_t* sp = slots.has_value() ? vector_of<int32_t>(*slots, "slots", at::kInt, {B}, index) : nullptr;
  const c10::cuda::OptionalCUDAGuard guard(c10::Device(c10::kCUDA, (c10::DeviceIndex)index));
  int64_t os = (int64_t)s.n_v_heads * s.value_dim;
  Tensor to;
  if (out.has_value()) {
    to = *out;
    os = rows_of(to, "out", s.n_v_heads, s.value_dim, index, at::kBFloat16);
    if (to.size(0) != n) refuse("out has to have as many rows as q");
  } else {
    to = at::empty({n, s.n_v_heads, s.value_dim}, q.options());
  }
  const int rc = hyb_attn_delta_run(&s, q.const_data_ptr(), qs, k.const_data_ptr(), ks, v.const_data_ptr(), vs, gp, bp, to.data_ptr(), os,
                                    cup, sp, int_of(B, "B"), int_of(n, "rows"), (int32_t)std::min(max_new, n), factor,
                                    reinterpret_cast<uint32_t*>(status),
                                    c10::cuda::getCurrentCUDAStream((c10::DeviceIndex)index).stream());
  if (rc < 0) fail("hyb_attn_delta_run", rc);
  return to;
}

}  // namespace

PYBIND11_MODULE(_binding, m) {
  m.def("paged_append", &paged_append);
  m.def("paged_attend", &paged_attend);
  m.def("delta_run", &delta_run);
}
