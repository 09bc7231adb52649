// The operators on torch tensors: argument checks and the calls of the C ABI.
//
// A Python function that reads a dozen attributes of six tensors and marshals
// twenty arguments through ctypes takes 16 us, more than the kernels of small
// calls; through this module a call takes 4 to 5, its launch among them (0.6 where
// there is nothing to launch).
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/extension.h>

#include <optional>
#include <string>
#include <tuple>

#include "../../include/wpk.h"

namespace {

using at::Tensor;
using OptTensor = std::optional<Tensor>;

struct Failure {
  int code;
  std::string msg;
};
PyObject* g_error = nullptr;  // the package's exception class (kept for good)

[[noreturn]] void bad(const std::string& msg) { throw Failure{WPK_ERR_INVALID_ARG, msg}; }

void check(int rc) {
  if (rc != WPK_OK) throw Failure{rc, wpk_last_error(nullptr)};
}

int type_of(const Tensor& x) {
  switch (x.scalar_type()) {
    case at::kFloat: return WPK_F32;
    case at::kBFloat16: return WPK_BF16;
    case at::kHalf: return WPK_F16;
    default: return -1;
  }
}

void* stream_of(const c10::Device& d) { return c10::cuda::getCurrentCUDAStream(d.index()).stream(); }

// Address of a contiguous vector of n elements (null for none).
template <typename T>
T* vector(const OptTensor& x, const char* name, at::ScalarType type, int64_t n, const c10::Device& dev) {
  if (!x) return nullptr;
  if (x->scalar_type() != type || x->device() != dev || x->dim() != 1 || x->size(0) != n || !x->is_contiguous())
    bad(std::string(name) + " must be a contiguous " + c10::toString(type) + " tensor [" + std::to_string(n) + "] on " +
        dev.str());
  return static_cast<T*>(x->data_ptr());
}

struct Rows {  // a tensor [total][heads][head_dim] of the call
  void* p;
  int64_t token, head;
  int type;
};

class Kv4 {
 public:
  Kv4(Tensor pages, int n_kv_heads, int head_dim, int page_tokens)
      : pages_(std::move(pages)), n_kv_(n_kv_heads), hd_(head_dim), page_(page_tokens) {}

  void append(const Tensor& k, const Tensor& v, const Tensor& pos, const Tensor& table, const OptTensor& indptr,
              const OptTensor& rope) {
    const Call c = call(pos, table, indptr, rope);
    if (k.dim() != 3) bad("k must be [total][n_kv_heads][head_dim]");
    const int64_t total = k.size(0);
    const Rows kr = rows(k, "k", total, n_kv_), vr = rows(v, "v", total, n_kv_);
    if (kr.type != vr.type) bad("k and v must have one dtype");
    if (total == 0) return;
    const c10::cuda::CUDAGuard on(pages_.device());
    check(wpk_kv4_append(&c.cache, c.pos, c.indptr, (int)total, kr.p, kr.token, kr.head, vr.p, vr.token, vr.head,
                         kr.type, c.rope, c.rope_positions, stream_of(pages_.device())));
  }

  std::tuple<Tensor, Tensor> read(const Tensor& pos, const Tensor& table, int64_t total, const OptTensor& indptr,
                                  at::ScalarType type) {
    const Call c = call(pos, table, indptr, std::nullopt);
    if (total < 0 || total > INT32_MAX) bad("total must be >= 0 and below 2^31");
    if (type != at::kFloat && type != at::kBFloat16 && type != at::kHalf)
      bad("dtype must be float32, bfloat16 or float16");
    const c10::cuda::CUDAGuard on(pages_.device());
    Tensor k = at::empty({total, n_kv_, hd_}, pages_.options().dtype(type));
    Tensor v = at::empty({total, n_kv_, hd_}, pages_.options().dtype(type));
    if (total)
      check(wpk_kv4_read(&c.cache, c.pos, c.indptr, (int)total, k.data_ptr(), k.stride(0), k.stride(1), v.data_ptr(),
                         v.stride(0), v.stride(1), type_of(k), stream_of(pages_.device())));
    return {k, v};
  }

  Tensor attention(const Tensor& q, const Tensor& pos, const Tensor& table, const OptTensor& indptr,
                   std::optional<int64_t> max_new, const OptTensor& rope, double scale, const OptTensor& out_) {
    const Call c = call(pos, table, indptr, rope);
    if (q.dim() != 3) bad("q must be [total][n_heads][head_dim]");
    const int64_t total = q.size(0), heads = q.size(1);
    const Rows qr = rows(q, "q", total, heads);
    if (max_new && (*max_new < 0 || *max_new > INT32_MAX)) bad("max_new must be >= 0 and below 2^31");
    const c10::cuda::CUDAGuard on(pages_.device());
    Tensor out = out_ ? *out_ : at::empty({total, heads, hd_}, q.options());
    const Rows o = rows(out, "out", total, heads);
    if (o.type != qr.type) bad("out must have q's dtype");
    if (total)
      check(wpk_kv4_attention(&c.cache, c.pos, c.indptr, (int)total, (int)(max_new ? *max_new : total), qr.p, qr.token,
                              qr.head, (int)heads, qr.type, c.rope, c.rope_positions, (float)scale, o.p, o.token,
                              o.head, stream_of(pages_.device())));
    return out;
  }

 private:
  struct Call {
    wpk_kv4_cache cache;
    const int32_t *pos, *indptr;
    const float* rope;
    int rope_positions;
  };

  Call call(const Tensor& pos, const Tensor& table, const OptTensor& indptr, const OptTensor& rope) const {
    const c10::Device dev = pages_.device();
    if (table.scalar_type() != at::kInt || table.device() != dev || table.dim() != 2 || !table.is_contiguous() ||
        table.numel() > INT32_MAX)
      bad("block_table must be a contiguous int32 tensor [batch][max_blocks] on " + dev.str());
    Call c{};
    const int64_t batch = table.size(0);
    c.cache = wpk_kv4_cache{pages_.data_ptr(), static_cast<const int32_t*>(table.data_ptr()), pages_.size(0),
                            (int)batch,        (int)table.size(1),
                            n_kv_,             hd_,
                            page_};
    c.pos = vector<int32_t>(pos, "pos", at::kInt, batch, dev);
    c.indptr = vector<int32_t>(indptr, "indptr", at::kInt, batch + 1, dev);
    if (rope) {
      if (rope->scalar_type() != at::kFloat || rope->device() != dev || rope->dim() != 3 || !rope->is_contiguous() ||
          rope->size(1) != hd_ / 2 || rope->size(2) != 2 || rope->size(0) > INT32_MAX)
        bad("rope must be a contiguous float32 tensor [positions][" + std::to_string(hd_ / 2) + "][2] on " + dev.str());
      c.rope = static_cast<const float*>(rope->data_ptr());
      c.rope_positions = (int)rope->size(0);
    }
    return c;
  }

  Rows rows(const Tensor& x, const char* name, int64_t total, int64_t heads) const {
    const int type = type_of(x);
    if (type < 0 || x.device() != pages_.device() || x.dim() != 3 || x.size(0) != total || x.size(1) != heads ||
        x.size(2) != hd_ || total > INT32_MAX || heads > INT32_MAX)
      bad(std::string(name) + " must be a float32, bfloat16 or float16 tensor [" + std::to_string(total) + "][" +
          std::to_string(heads) + "][" + std::to_string(hd_) + "] on " + pages_.device().str());
    if (x.stride(2) != 1) bad(std::string(name) + " must be contiguous in its last dimension");
    // the stride of a dimension of one element says nothing
    return Rows{x.data_ptr(), total > 1 ? x.stride(0) : 0, heads > 1 ? x.stride(1) : 0, type};
  }

  Tensor pages_;
  int n_kv_, hd_, page_;
};

std::tuple<Tensor, OptTensor, OptTensor> sample(const Tensor& logits, const OptTensor& uniform,
                                                const OptTensor& temperature, const OptTensor& top_k,
                                                const OptTensor& top_p, const OptTensor& min_p, const OptTensor& out,
                                                bool want_logprob, bool want_kept) {
  const int type = type_of(logits);
  if (type < 0 || logits.dim() != 2 || (logits.size(1) > 1 && logits.stride(1) != 1))
    bad("logits must be a float32, bfloat16 or float16 tensor [batch][vocab], contiguous in its last dimension");
  const c10::Device dev = logits.device();
  if (!dev.is_cuda()) bad("logits must be on a CUDA device");
  const int64_t B = logits.size(0), V = logits.size(1);
  if (B > INT32_MAX || V > INT32_MAX) bad("batch and vocab must be below 2^31");
  if (!uniform) bad("uniform must be given");
  const float* u = vector<float>(uniform, "uniform", at::kFloat, B, dev);
  const float* t = vector<float>(temperature, "temperature", at::kFloat, B, dev);
  const int32_t* k = vector<int32_t>(top_k, "top_k", at::kInt, B, dev);
  const float* p = vector<float>(top_p, "top_p", at::kFloat, B, dev);
  const float* m = vector<float>(min_p, "min_p", at::kFloat, B, dev);
  vector<int32_t>(out, "out_tok", at::kInt, B, dev);
  const c10::cuda::CUDAGuard on(dev);
  const auto options = logits.options();
  Tensor tok = out ? *out : at::empty({B}, options.dtype(at::kInt));
  OptTensor logprob, kept;
  if (want_logprob) logprob = at::empty({B}, options.dtype(at::kFloat));
  if (want_kept) kept = at::empty({B}, options.dtype(at::kInt));
  if (B)
    check(wpk_sample(logits.data_ptr(), type, (int)B, (int)V, logits.stride(0), u, t, k, p, m,
                     static_cast<int32_t*>(tok.data_ptr()),
                     want_logprob ? static_cast<float*>(logprob->data_ptr()) : nullptr,
                     want_kept ? static_cast<int32_t*>(kept->data_ptr()) : nullptr, stream_of(dev)));
  return {tok, logprob, kept};
}

}  // namespace

PYBIND11_MODULE(_wpk_torch, m) {
  m.def("set_error", [](py::object cls) { g_error = cls.release().ptr(); });
  py::register_exception_translator([](std::exception_ptr e) {
    try {
      if (e) std::rethrow_exception(e);
    } catch (const Failure& f) {
      const py::tuple args = py::make_tuple(f.code, f.msg);
      PyErr_SetObject(g_error ? g_error : PyExc_RuntimeError, args.ptr());
    }
  });
  py::class_<Kv4>(m, "Kv4")
      .def(py::init<Tensor, int, int, int>())
      .def("append", &Kv4::append)
      .def("read",
           [](Kv4& c, const Tensor& pos, const Tensor& table, int64_t total, const OptTensor& indptr,
              const py::object& type) {
             return c.read(pos, table, total, indptr, torch::python::detail::py_object_to_dtype(type));
           })
      .def("attention", &Kv4::attention);
  m.def("sample", &sample);
}
