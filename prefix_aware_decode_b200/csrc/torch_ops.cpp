// The session-cache operators on torch tensors (Python module _cache_ops):
// checks of types, shapes, strides and devices, outputs and workspaces from
// torch's allocator, and the call of the C ABI on the device's current stream.
// A call through ctypes took 10 us of host time beside the launch, most of it in
// reading tensor attributes one by one; here it is about one.
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/extension.h>

#include <optional>
#include <string>
#include <tuple>

#include "pa.h"

namespace py = pybind11;
using at::Tensor;

namespace {

[[noreturn]] void bad(const std::string& what) { throw py::value_error(what); }

// The status as the binding's own exception.
void check(pa_status st, const char* where) {
  if (st == PA_OK) return;
  const py::object error = py::module_::import("prefix_aware_decode_b200._binding").attr("PaError");
  PyErr_SetObject(error.ptr(), error(static_cast<int>(st), where).ptr());
  throw py::error_already_set();
}

const char* type_name(at::ScalarType t) {
  return t == at::kBFloat16 ? "bfloat16" : t == at::kFloat ? "float32" : t == at::kDouble ? "float64" : t == at::kInt ? "int32" : "uint8";
}

// These operators have no backward: a result that silently left the graph would be wrong.
void no_grad(const Tensor& t, const char* name) {
  if (t.requires_grad() && at::GradMode::is_enabled())
    bad(std::string(name) + " requires grad, and this operator has no backward: call it under torch.no_grad()");
}

// A tensor that a call has changed in place counts a version, as torch's own do.
void changed(const Tensor& t) {
  if (!t.is_inference()) t.unsafeGetTensorImpl()->bump_version();
}

// Address of a contiguous tensor of one type on CUDA device `index`.
void* ptr(const Tensor& t, const char* name, at::ScalarType type, c10::DeviceIndex index, uintptr_t align) {
  if (!t.defined() || t.scalar_type() != type) bad(std::string(name) + " must be a " + type_name(type) + " tensor");
  if (!t.is_cuda() || t.get_device() != index) bad(std::string(name) + " must be on the pools' device");
  if (!t.is_contiguous()) bad(std::string(name) + " must be contiguous");
  no_grad(t, name);
  void* p = t.data_ptr();
  if (reinterpret_cast<uintptr_t>(p) % align) bad(std::string(name) + " must be " + std::to_string(align) + "-byte aligned");
  return p;
}

int32_t i32(int64_t v, const char* name) {
  if (v < INT32_MIN || v > INT32_MAX) bad(std::string(name) + " does not fit 32 bits");
  return static_cast<int32_t>(v);
}

c10::DeviceIndex index_of(const Tensor& k_pool) {
  if (k_pool.dim() != 4) bad("k_pool must be a tensor [num_pages][Hkv][P][D]");
  if (!k_pool.is_cuda()) bad("k_pool must be a CUDA tensor");
  return k_pool.get_device();
}

pa_sessions sessions(const Tensor& k_pool, const Tensor& table, const Tensor& kv_lens, const Tensor* cu_rows,
                     int64_t rows, int64_t Hq, c10::DeviceIndex index) {
  pa_sessions b{};
  b.d_block_table = static_cast<const int32_t*>(ptr(table, "block_table", at::kInt, index, 4));
  if (table.dim() != 2) bad("block_table must be [S][max_pages]");
  const int64_t S = table.size(0);
  b.d_kv_lens = static_cast<const int32_t*>(ptr(kv_lens, "kv_lens", at::kInt, index, 4));
  if (kv_lens.dim() != 1 || kv_lens.size(0) != S) bad("kv_lens must be [S], S the rows of block_table");
  if (cu_rows) {
    b.d_cu_rows = static_cast<const int32_t*>(ptr(*cu_rows, "cu_rows", at::kInt, index, 4));
    if (cu_rows->dim() != 1 || cu_rows->size(0) != S + 1) bad("cu_rows must be [S + 1], S the rows of block_table");
  }
  b.n_sessions = i32(S, "S");
  b.num_rows = i32(rows, "rows");
  b.num_q_heads = i32(Hq, "Hq");
  b.num_kv_heads = i32(k_pool.size(1), "Hkv");
  b.head_dim = i32(k_pool.size(3), "D");
  b.page_size = i32(k_pool.size(2), "P");
  b.max_pages = i32(table.size(1), "max_pages");
  b.num_pages_in_pool = i32(k_pool.size(0), "num_pages");
  return b;
}

void* pool(const Tensor& t, const char* name, const Tensor& k_pool, c10::DeviceIndex index) {
  void* p = ptr(t, name, at::kBFloat16, index, 16);
  if (t.sizes() != k_pool.sizes()) bad("v_pool must have k_pool's shape");
  return p;
}

const void* q_rows(const Tensor& q, const Tensor& k_pool, c10::DeviceIndex index) {
  const void* p = ptr(q, "q", at::kBFloat16, index, 16);
  if (q.dim() != 3 || q.size(2) != k_pool.size(3)) bad("q must be [rows][Hq][D], D that of the pools");
  return p;
}

// Rows [rows][heads][D] that may be slices of wider ones.
const void* strided(const Tensor& t, const char* name, int64_t rows, int64_t heads, int64_t D, c10::DeviceIndex index,
                    int64_t* stride) {
  if (t.scalar_type() != at::kBFloat16 || t.dim() != 3 || t.size(0) != rows || t.size(1) != heads || t.size(2) != D)
    bad(std::string(name) + " must be a bf16 tensor [" + std::to_string(rows) + "][" + std::to_string(heads) + "][" +
        std::to_string(D) + "]");
  if (!t.is_cuda() || t.get_device() != index) bad(std::string(name) + " must be on the pools' device");
  no_grad(t, name);
  if ((D > 1 && t.stride(2) != 1) || (heads > 1 && t.stride(1) != D))
    bad(std::string(name) + ": the heads of a row must be contiguous");
  *stride = rows > 1 ? t.stride(0) : heads * D;
  const void* p = t.data_ptr();
  if (*stride < heads * D || *stride % 8 || reinterpret_cast<uintptr_t>(p) % 16)
    bad(std::string(name) + ": rows must not overlap and must be 16-byte aligned");
  return p;
}

Tensor make(at::IntArrayRef shape, at::ScalarType type, c10::DeviceIndex index) {
  return at::empty(shape, at::TensorOptions().dtype(type).device(at::kCUDA, index));
}

// An output: the caller's, checked, or a new one.
Tensor output(const std::optional<Tensor>& t, const char* name, at::IntArrayRef shape, at::ScalarType type,
              c10::DeviceIndex index, uintptr_t align, void** p) {
  if (!t) {
    Tensor n = make(shape, type, index);
    *p = n.data_ptr();
    return n;
  }
  *p = ptr(*t, name, type, index, align);
  if (t->sizes() != shape) bad(std::string(name) + " has another shape than it must have");
  return *t;
}

void* current(c10::DeviceIndex index) { return c10::cuda::getCurrentCUDAStream(index).stream(); }

Tensor rope_append(const Tensor& q, const Tensor& k, const Tensor& v, const Tensor& positions, const Tensor& inv_freq,
                   const Tensor& k_pool, const Tensor& v_pool, const Tensor& table, const Tensor& kv_lens,
                   const Tensor& cu_rows, const std::optional<std::string>& axes, bool interleaved,
                   const std::optional<Tensor>& q_out) {
  const auto index = index_of(k_pool);
  if (q.dim() != 3) bad("q must be [rows][Hq][D]");
  const int64_t rows = q.size(0), Hq = q.size(1), D = k_pool.size(3), Hkv = k_pool.size(1);
  const pa_sessions b = sessions(k_pool, table, kv_lens, &cu_rows, rows, Hq, index);
  int64_t qs, ks, vs;
  const void* qp = strided(q, "q", rows, Hq, D, index, &qs);
  const void* kp = strided(k, "k", rows, Hkv, D, index, &ks);
  const void* vp = strided(v, "v", rows, Hkv, D, index, &vs);
  pa_rope r{};
  r.d_positions = static_cast<const int32_t*>(ptr(positions, "positions", at::kInt, index, 4));
  if ((positions.dim() != 1 && positions.dim() != 2) || positions.size(-1) != rows)
    bad("positions must be [rows] or [n_axes][rows]");
  r.n_axes = positions.dim() == 1 ? 1 : i32(positions.size(0), "n_axes");
  r.d_inv_freq = static_cast<const double*>(ptr(inv_freq, "inv_freq", at::kDouble, index, 8));
  if (inv_freq.dim() != 1) bad("inv_freq must be [R / 2]");
  r.rotary_dim = i32(2 * inv_freq.size(0), "R");
  r.interleaved = interleaved;
  if (axes) {
    if ((int64_t)axes->size() != inv_freq.size(0)) bad("axes must name the axis of each of inv_freq's pairs");
    r.axes = reinterpret_cast<const uint8_t*>(axes->data());
  }
  void* kpool = pool(k_pool, "k_pool", k_pool, index);
  void* vpool = pool(v_pool, "v_pool", k_pool, index);
  const c10::cuda::CUDAGuard on(index);
  void* op;
  Tensor out = output(q_out, "q_out", {rows, Hq, D}, at::kBFloat16, index, 16, &op);
  check(pa_rope_append(&b, &r, qp, qs, kp, ks, vp, vs, kpool, vpool, op, current(index)), "pa_rope_append");
  changed(out);
  changed(k_pool);
  changed(v_pool);
  return out;
}

size_t workspace_bytes(const pa_sessions& b, int64_t window, int64_t sinks) {
  size_t n = 0;
  check(pa_window_workspace_size(&b, i32(window, "window"), i32(sinks, "sinks"), &n), "pa_window_workspace_size");
  return n;
}

Tensor window_workspace(const Tensor& q, const Tensor& k_pool, const Tensor& table, const Tensor& kv_lens,
                        const Tensor& cu_rows, int64_t window, int64_t sinks) {
  const auto index = index_of(k_pool);
  q_rows(q, k_pool, index);
  const pa_sessions b = sessions(k_pool, table, kv_lens, &cu_rows, q.size(0), q.size(1), index);
  const c10::cuda::CUDAGuard on(index);
  Tensor ws = make({(int64_t)workspace_bytes(b, window, sinks)}, at::kByte, index);
  ws.narrow(0, 0, 256).zero_();  // the status of no call yet
  return ws;
}

std::tuple<Tensor, Tensor> window_attend(const Tensor& q, const Tensor& k_pool, const Tensor& v_pool,
                                         const Tensor& table, const Tensor& kv_lens, const Tensor& cu_rows,
                                         int64_t window, int64_t sinks, double scale, const std::optional<Tensor>& out,
                                         const std::optional<Tensor>& lse, const std::optional<Tensor>& workspace) {
  const auto index = index_of(k_pool);
  const void* qp = q_rows(q, k_pool, index);
  const int64_t rows = q.size(0), Hq = q.size(1), D = q.size(2);
  const pa_sessions b = sessions(k_pool, table, kv_lens, &cu_rows, rows, Hq, index);
  const void* kp = pool(k_pool, "k_pool", k_pool, index);
  const void* vp = pool(v_pool, "v_pool", k_pool, index);
  const c10::cuda::CUDAGuard on(index);
  void *op, *lp, *wp;
  Tensor o = output(out, "out", {rows, Hq, D}, at::kBFloat16, index, 16, &op);
  Tensor l = output(lse, "lse", {rows, Hq}, at::kFloat, index, 4, &lp);
  Tensor ws = workspace ? *workspace : make({(int64_t)workspace_bytes(b, window, sinks)}, at::kByte, index);
  wp = ptr(ws, "workspace", at::kByte, index, 256);
  check(pa_window_attend(&b, i32(window, "window"), i32(sinks, "sinks"), (float)scale, qp, kp, vp, wp, ws.numel(), op,
                         static_cast<float*>(lp), current(index)),
        "pa_window_attend");
  changed(o);
  changed(l);
  return {o, l};
}

// Of a workspace, or of every call on a device.
int window_status(const std::optional<Tensor>& workspace, int64_t device) {
  if (workspace && !workspace->is_cuda()) bad("workspace must be a CUDA tensor");
  const auto index = workspace ? workspace->get_device() : static_cast<c10::DeviceIndex>(device);
  const void* wp = workspace ? ptr(*workspace, "workspace", at::kByte, index, 256) : nullptr;
  const c10::cuda::CUDAGuard on(index);
  pa_status st = PA_OK;
  void* stream = current(index);
  pa_status rc;
  {
    py::gil_scoped_release nogil;
    rc = pa_window_status(wp, stream, &st);
  }
  check(rc, "pa_window_status");
  return st;
}

Tensor weigh_tokens(const Tensor& q, const Tensor& k_pool, const Tensor& lse, const Tensor& table,
                    const Tensor& kv_lens, const Tensor& cu_rows, const Tensor& scores, int64_t window, int64_t sinks,
                    double scale) {
  const auto index = index_of(k_pool);
  const void* qp = q_rows(q, k_pool, index);
  const void* kp = pool(k_pool, "k_pool", k_pool, index);
  const int64_t rows = q.size(0), Hq = q.size(1);
  const pa_sessions b = sessions(k_pool, table, kv_lens, &cu_rows, rows, Hq, index);
  const void* lp = ptr(lse, "lse", at::kFloat, index, 4);
  if (lse.dim() != 2 || lse.size(0) != rows || lse.size(1) != Hq) bad("lse must be [rows][Hq]");
  void* sp = ptr(scores, "scores", at::kFloat, index, 4);
  if (scores.dim() != 3 || scores.size(0) != b.n_sessions || scores.size(1) != b.num_kv_heads)
    bad("scores must be [S][Hkv][max_tokens]");
  const c10::cuda::CUDAGuard on(index);
  check(pa_weigh_tokens(&b, i32(window, "window"), i32(sinks, "sinks"), (float)scale, qp, kp,
                        static_cast<const float*>(lp), static_cast<float*>(sp), scores.size(2), current(index)),
        "pa_weigh_tokens");
  changed(scores);
  return scores;
}

int weigh_status(int64_t device) {
  const c10::cuda::CUDAGuard on(static_cast<c10::DeviceIndex>(device));
  pa_status st = PA_OK, rc;
  void* stream = current(static_cast<c10::DeviceIndex>(device));
  {
    py::gil_scoped_release nogil;
    rc = pa_weigh_status(stream, &st);
  }
  check(rc, "pa_weigh_status");
  return st;
}

std::tuple<Tensor, Tensor, Tensor> evict_tokens(const Tensor& scores, const Tensor& k_pool, const Tensor& v_pool,
                                                const Tensor& table, const Tensor& kv_lens, const Tensor& dst_table,
                                                int64_t budget, int64_t sinks, int64_t recent,
                                                const std::optional<Tensor>& scores_out) {
  const auto index = index_of(k_pool);
  const pa_sessions b = sessions(k_pool, table, kv_lens, nullptr, 0, k_pool.size(1), index);
  void* kp = pool(k_pool, "k_pool", k_pool, index);
  void* vp = pool(v_pool, "v_pool", k_pool, index);
  const void* sp = ptr(scores, "scores", at::kFloat, index, 4);
  if (scores.dim() != 3 || scores.size(0) != b.n_sessions || scores.size(1) != b.num_kv_heads)
    bad("scores must be [S][Hkv][max_tokens]");
  const void* dp = ptr(dst_table, "dst_table", at::kInt, index, 4);
  if (dst_table.dim() != 2 || dst_table.size(0) != b.n_sessions) bad("dst_table must be [S][pages]");
  if (budget < 1) bad("budget must be positive");
  const c10::cuda::CUDAGuard on(index);
  void* xp;
  Tensor x = output(scores_out, "scores_out", scores.sizes(), at::kFloat, index, 4, &xp);
  Tensor kept = make({scores.size(0), scores.size(1), budget}, at::kInt, index);
  Tensor lens = make({scores.size(0)}, at::kInt, index);
  check(pa_evict_tokens(&b, static_cast<const float*>(sp), scores.size(2), kp, vp, static_cast<const int32_t*>(dp),
                        i32(dst_table.size(1), "pages"), i32(budget, "budget"), i32(sinks, "sinks"),
                        i32(recent, "recent"), static_cast<float*>(xp), kept.data_ptr<int32_t>(),
                        lens.data_ptr<int32_t>(), current(index)),
        "pa_evict_tokens");
  changed(x);
  changed(k_pool);
  changed(v_pool);
  return {lens, kept, x};
}

}  // namespace

PYBIND11_MODULE(_cache_ops, m) {
  m.doc() = "session-cache operators on torch tensors (see cache_ops)";
  m.def("rope_append", &rope_append);
  m.def("window_workspace", &window_workspace);
  m.def("window_attend", &window_attend);
  m.def("window_status", &window_status);
  m.def("weigh_tokens", &weigh_tokens);
  m.def("weigh_status", &weigh_status);
  m.def("evict_tokens", &evict_tokens);
}
