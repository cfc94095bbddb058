// bind.cpp -- argument marshalling of the attention operators: torch tensors to the C ABI of
// libmoe (include/moe_cache.h), as the ctypes layer does for the other entry points.  These
// calls are made once per layer and token, and the smallest take the GPU less than 10 us;
// checking and converting their dozen arguments in Python took 8 to 12 us of each call,
// here about 2.  Nothing is computed: every check that the C ABI makes itself is left to it.
#include <c10/cuda/CUDAStream.h>
#include <torch/extension.h>

#include "moe_cache.h"

namespace py = pybind11;
using at::Tensor;
using OptTensor = std::optional<Tensor>;

namespace {

struct Refused {  // becomes MoEError(status, what)
  int status;
  std::string what;
};
[[noreturn]] void refuse(const std::string& what) { throw Refused{MOE_ERR_INVALID, what}; }
void check(int status, const char* name) {
  if (status != MOE_OK) throw Refused{status, name};
}

int dtype_of(const Tensor& t, const char* what) {
  switch (t.scalar_type()) {
    case at::kBFloat16: return MOE_BF16;
    case at::kHalf: return MOE_F16;
    case at::kFloat: return MOE_F32;
    default: refuse(std::string(what) + ": dtype " + toString(t.scalar_type()));
  }
}

int32_t* ints(const Tensor& t, int dim, c10::Device dev, const char* what, int64_t n = -1) {
  if (t.scalar_type() != at::kInt || t.dim() != dim || t.device() != dev || (n >= 0 && t.size(0) != n) ||
      (t.size(-1) > 1 && t.stride(-1) != 1))
    refuse(std::string(what) + " must be an int32 tensor of " + std::to_string(dim) + " dimension(s)" +
           (n >= 0 ? " and " + std::to_string(n) + " entries" : "") + " on " + dev.str() + ", its last one contiguous");
  return t.data_ptr<int32_t>();
}

moe_kv_pool pool_of(const Tensor& p, const OptTensor& error, const char* what) {
  if (p.scalar_type() != at::kByte || p.dim() != 4 || !p.is_cuda() || !p.is_contiguous() || p.size(3) % 18 || p.size(0) > INT32_MAX)
    refuse(std::string(what) + ": pool must be a contiguous uint8 CUDA tensor [pages, KV heads, page tokens / 16, 18 * head dim]");
  moe_kv_pool c{};
  c.pool_dev = p.data_ptr<uint8_t>();
  c.n_pages = (int32_t)p.size(0);
  c.n_kv_heads = (int32_t)p.size(1);
  c.page_tokens = (int32_t)(p.size(2) * 16);
  c.head_dim = (int32_t)(p.size(3) / 18);
  c.device = p.get_device();
  if (error) c.error_dev = ints(*error, 1, p.device(), "error");
  return c;
}

moe_kv_table table_of(const Tensor& t, c10::Device dev, const char* what) {
  moe_kv_table r{};
  r.table_dev = ints(t, 2, dev, what);
  if (t.size(0) > INT32_MAX || t.size(1) > INT32_MAX) refuse(std::string(what) + ": too large");
  r.n_seqs = (int32_t)t.size(0);
  r.width = (int32_t)t.size(1);
  r.row_stride = t.size(0) > 1 ? t.stride(0) : t.size(1);
  return r;
}

moe_rows rows_of(const Tensor& t, int64_t n, int64_t heads, int64_t dim, at::ScalarType type, c10::Device dev, const char* what) {
  if (t.dim() != 3 || t.size(0) != n || t.size(1) != heads || t.size(2) != dim || t.scalar_type() != type || t.device() != dev ||
      t.stride(2) != 1)
    refuse(std::string(what) + " must be a " + toString(type) + " tensor [" + std::to_string(n) + ", " + std::to_string(heads) + ", " +
           std::to_string(dim) + "] on " + dev.str() + ", its last dimension contiguous");
  return {t.data_ptr(), t.stride(0), t.stride(1)};
}

// These calls keep nothing for a gradient: one that would be lost without a word is refused.
void no_gradient(std::initializer_list<const Tensor*> rows, const char* what) {
  if (!at::GradMode::is_enabled()) return;
  for (const Tensor* t : rows)
    if (t->requires_grad())
      throw Refused{MOE_ERR_UNSUPPORTED, std::string(what) + ": inference only, but a row tensor requires a gradient (torch.no_grad() or detach())"};
}

moe_kv_score score_of(const Tensor& t, int64_t n, int64_t heads, int64_t most, c10::Device dev, const char* what) {
  if (t.scalar_type() != at::kFloat || t.dim() != 3 || t.size(0) != n || t.size(1) != heads || t.size(2) < most || t.device() != dev ||
      (t.size(2) > 1 && t.stride(2) != 1))
    refuse(std::string(what) + " must be a float32 tensor [" + std::to_string(n) + ", " + std::to_string(heads) + ", >= " +
           std::to_string(most) + "] on " + dev.str() + ", its last dimension contiguous");
  return {t.data_ptr<float>(), t.stride(0), t.stride(1)};
}

void* stream_of(c10::Device dev) { return c10::cuda::getCurrentCUDAStream(dev.index()).stream(); }

int32_t small(int64_t v, const char* what) {
  if (v < INT32_MIN || v > INT32_MAX) refuse(std::string(what) + " " + std::to_string(v));
  return (int32_t)v;
}

using RowsCall = int (*)(const moe_kv_pool*, const moe_kv_table*, const int32_t*, const int32_t*, const moe_rows*, const moe_rows*,
                         int32_t, int32_t, void*);
void rows_call(RowsCall call, const char* name, const Tensor& pool, const Tensor& k, const Tensor& v, const Tensor& table,
               const Tensor& cu, const OptTensor& start, int64_t n, const OptTensor& error) {
  const auto dev = pool.device();
  const moe_kv_pool c = pool_of(pool, error, name);
  const moe_kv_table t = table_of(table, dev, "table");
  const int32_t* cu_p = ints(cu, 1, dev, "cu", (int64_t)t.n_seqs + 1);
  const int32_t* st_p = start ? ints(*start, 1, dev, "start", t.n_seqs) : nullptr;
  const moe_rows rk = rows_of(k, n, c.n_kv_heads, c.head_dim, k.scalar_type(), dev, "k");
  const moe_rows rv = rows_of(v, n, c.n_kv_heads, c.head_dim, k.scalar_type(), dev, "v");
  const int d = dtype_of(k, name);
  if (n && t.n_seqs) check(call(&c, &t, cu_p, st_p, &rk, &rv, small(n, "tokens"), d, stream_of(dev)), name);
}

void kv_store(const Tensor& pool, const Tensor& k, const Tensor& v, const Tensor& table, const Tensor& cu, const OptTensor& start,
              const OptTensor& error) {
  if (k.dim() != 3) refuse("kv_store: k must have three dimensions");
  no_gradient({&k, &v}, "kv_store");
  rows_call(moe_kv_store, "moe_kv_store", pool, k, v, table, cu, start, k.size(0), error);
}

std::pair<Tensor, Tensor> kv_load(const Tensor& pool, const Tensor& table, const Tensor& cu, const OptTensor& start, int64_t n,
                                  at::ScalarType type, const std::optional<std::pair<Tensor, Tensor>>& out, const OptTensor& error) {
  std::pair<Tensor, Tensor> kv;
  if (out) {
    kv = *out;
    if (kv.first.scalar_type() != type) refuse(std::string("kv_load: out must be ") + toString(type));
  } else {
    const moe_kv_pool c = pool_of(pool, error, "kv_load");
    if (n < 0) refuse("kv_load: n_tokens " + std::to_string(n));
    const auto o = at::TensorOptions().dtype(type).device(pool.device());
    kv = {at::empty({n, c.n_kv_heads, c.head_dim}, o), at::empty({n, c.n_kv_heads, c.head_dim}, o)};
  }
  rows_call(moe_kv_load, "moe_kv_load", pool, kv.first, kv.second, table, cu, start, n, error);
  return kv;
}

int64_t workspace_bytes(const moe_kv_pool& c, const moe_kv_table& t, int64_t heads, int64_t most, bool scored) {
  size_t bytes = 0;
  check(moe_kv_attend_workspace(&c, &t, small(heads, "query heads"), small(most, "max_len"), scored, &bytes), "moe_kv_attend_workspace");
  return (int64_t)bytes;
}

int64_t kv_attend_workspace(const Tensor& pool, const Tensor& table, int64_t heads, int64_t most, bool scored) {
  return workspace_bytes(pool_of(pool, {}, "kv_attend_workspace"), table_of(table, pool.device(), "table"), heads, most, scored);
}

Tensor kv_attend(const Tensor& pool, const Tensor& q, const Tensor& table, const Tensor& lens, std::optional<int64_t> max_len,
                 std::optional<double> scale, const OptTensor& score, const OptTensor& out_arg, const OptTensor& ws_arg,
                 const OptTensor& error) {
  const auto dev = pool.device();
  const moe_kv_pool c = pool_of(pool, error, "kv_attend");
  const moe_kv_table t = table_of(table, dev, "kv_attend: table");
  const int32_t* lens_p = ints(lens, 1, dev, "kv_attend: lens", t.n_seqs);
  if (q.dim() != 3) refuse("kv_attend: q must have three dimensions");
  no_gradient({&q}, "kv_attend");
  const int64_t heads = q.size(1);
  const int64_t most = max_len ? *max_len : (int64_t)t.width * c.page_tokens;
  const auto type = q.scalar_type();
  const moe_rows rq = rows_of(q, t.n_seqs, heads, c.head_dim, type, dev, "kv_attend: q");
  moe_kv_score sc{};
  if (score) sc = score_of(*score, t.n_seqs, c.n_kv_heads, most, dev, "kv_attend: score");
  const int d = dtype_of(q, "kv_attend");
  const Tensor out = out_arg ? *out_arg : at::empty_like(q);
  const moe_rows ro = rows_of(out, t.n_seqs, heads, c.head_dim, type, dev, "kv_attend: out");
  if (!t.n_seqs) return out;
  Tensor ws;
  if (ws_arg) {
    ws = *ws_arg;
    if (ws.device() != dev || !ws.is_contiguous()) refuse("kv_attend: workspace must be contiguous on " + dev.str());
  } else {
    ws = at::empty({workspace_bytes(c, t, heads, most, score.has_value())}, at::TensorOptions().dtype(at::kByte).device(dev));
  }
  const double s = scale ? *scale : 1.0 / std::sqrt((double)c.head_dim);
  check(moe_kv_attend(&c, &t, lens_p, small(most, "max_len"), &rq, small(heads, "query heads"), d, (float)s, &ro, score ? &sc : nullptr,
                      ws.data_ptr(), (size_t)ws.nbytes(), stream_of(dev)),
        "moe_kv_attend");
  return out;
}

std::tuple<Tensor, Tensor, Tensor> kv_evict(const Tensor& pool, const Tensor& table, const Tensor& lens, int64_t max_len,
                                            const Tensor& score, int64_t keep, int64_t recent, const Tensor& out_table,
                                            const OptTensor& error) {
  const auto dev = pool.device();
  const moe_kv_pool c = pool_of(pool, error, "kv_evict");
  const moe_kv_table t = table_of(table, dev, "kv_evict: table"), o = table_of(out_table, dev, "kv_evict: out_table");
  const int32_t* lens_p = ints(lens, 1, dev, "kv_evict: lens", t.n_seqs);
  const moe_kv_score sc = score_of(score, t.n_seqs, c.n_kv_heads, max_len, dev, "kv_evict: score");
  if (keep < 1) refuse("kv_evict: keep " + std::to_string(keep));
  const auto i32 = at::TensorOptions().dtype(at::kInt).device(dev), f32 = at::TensorOptions().dtype(at::kFloat).device(dev);
  const Tensor out_lens = at::empty({t.n_seqs}, i32), kept = at::empty({t.n_seqs, c.n_kv_heads, keep}, i32),
               out_score = at::empty({t.n_seqs, c.n_kv_heads, keep}, f32);
  if (t.n_seqs)
    check(moe_kv_evict(&c, &t, lens_p, small(max_len, "max_len"), &sc, small(keep, "keep"), small(recent, "recent"), &o,
                       out_lens.data_ptr<int32_t>(), kept.data_ptr<int32_t>(), out_score.data_ptr<float>(), stream_of(dev)),
          "moe_kv_evict");
  return {out_lens, kept, out_score};
}

Tensor attend_prompt(const Tensor& q, const Tensor& k, const Tensor& v, const Tensor& cu, std::optional<double> scale,
                     const OptTensor& out_arg, const OptTensor& error) {
  if (!q.is_cuda() || q.dim() != 3 || k.dim() != 3) refuse("attend_prompt: q, k and v must be CUDA tensors of three dimensions");
  no_gradient({&q, &k, &v}, "attend_prompt");
  const auto dev = q.device();
  const auto type = q.scalar_type();
  const int64_t n = q.size(0), heads = q.size(1), dim = q.size(2), kv = k.size(1);
  const moe_rows rq = rows_of(q, n, heads, dim, type, dev, "attend_prompt: q"), rk = rows_of(k, n, kv, dim, type, dev, "attend_prompt: k"),
                 rv = rows_of(v, n, kv, dim, type, dev, "attend_prompt: v");
  const int32_t* cu_p = ints(cu, 1, dev, "attend_prompt: cu");
  if (cu.size(0) < 1) refuse("attend_prompt: cu is empty");
  int32_t* err = error ? ints(*error, 1, dev, "attend_prompt: error") : nullptr;
  const int d = dtype_of(q, "attend_prompt");
  const Tensor out = out_arg ? *out_arg : at::empty_like(q);
  const moe_rows ro = rows_of(out, n, heads, dim, type, dev, "attend_prompt: out");
  if (n)
    check(moe_attend_prompt(q.get_device(), &rq, &rk, &rv, &ro, cu_p, small(cu.size(0) - 1, "sequences"), small(n, "tokens"),
                            small(heads, "heads"), small(kv, "KV heads"), small(dim, "head dim"), d,
                            (float)(scale ? *scale : 1.0 / std::sqrt((double)dim)), err, stream_of(dev)),
          "moe_attend_prompt");
  return out;
}

}  // namespace

PYBIND11_MODULE(_moe_bind, m) {
  // The package passes its exception type in.
  m.def("set_error", [](py::object type) {
    static py::object* held = new py::object(type);
    *held = type;
    py::register_exception_translator([](std::exception_ptr p) {
      try {
        if (p) std::rethrow_exception(p);
      } catch (const Refused& r) {
        py::object e = (*held)(r.status, r.what);
        PyErr_SetObject(held->ptr(), e.ptr());
      }
    });
  });
  m.def("kv_store", &kv_store);
  m.def("kv_load", &kv_load);
  m.def("kv_attend", &kv_attend);
  m.def("kv_attend_workspace", &kv_attend_workspace);
  m.def("kv_evict", &kv_evict);
  m.def("attend_prompt", &attend_prompt);
}
