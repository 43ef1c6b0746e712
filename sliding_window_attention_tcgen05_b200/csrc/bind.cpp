// bind.cpp -- the paged-cache wrappers' argument marshalling (paged.py) in
// C++: checks of the tensors, output and scratch allocation, the call of the C
// ABI on the tensors' device and current stream.  A decode step makes these
// calls once per layer, and through ctypes each took 10 to 15 us of host time
// (3 of them the launch), more than the kernels of a small step.
#include <ATen/ATen.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/utils/pybind.h>

#include <array>
#include <map>
#include <optional>
#include <string>

#include "vx.h"

namespace py = pybind11;
using at::Tensor;
using OptTensor = std::optional<Tensor>;

namespace {

constexpr size_t kStatusBytes = 256;    // a workspace that only holds the status word
constexpr size_t kStatusBuf = 1024;     // the largest workspace without scratch

[[noreturn]] void value_error(const std::string& what) { throw py::value_error(what); }
[[noreturn]] void type_error(const std::string& what) { throw py::type_error(what); }

std::string name_of(at::ScalarType t) {
  switch (t) {
    case at::kFloat: return "torch.float32";
    case at::kBFloat16: return "torch.bfloat16";
    case at::kInt: return "torch.int32";
    case at::kLong: return "torch.int64";
    default: return c10::toString(t);
  }
}

std::string shape_of(const Tensor& t) {
  std::string s = "[";
  for (int64_t i = 0; i < t.dim(); ++i) s += (i ? ", " : "") + std::to_string(t.size(i));
  return s + "]";
}

void check(int status, const char* where) {
  if (status == VX_OK) return;
  py::object cls = py::module_::import("sliding_window_attention_tcgen05_b200._lib").attr("VxError");
  py::object e = cls(status, where);
  PyErr_SetObject(cls.ptr(), e.ptr());
  throw py::error_already_set();
}

vx_dtype dtype_of(const Tensor& t, const char* what) {
  if (t.scalar_type() == at::kFloat) return VX_F32;
  if (t.scalar_type() == at::kBFloat16) return VX_BF16;
  type_error(std::string(what) + " must be float32 or bfloat16, not " + name_of(t.scalar_type()));
}

void on_device(int dev, const Tensor& t, const char* name) {
  if (!t.is_cuda()) value_error(std::string(name) + " must be a CUDA tensor");
  if (t.get_device() != dev)
    value_error(std::string(name) + " is on " + t.device().str() + ", expected cuda:" + std::to_string(dev));
}

// Address of a contiguous index or state tensor of the given dtype (and size).
void* whole(const Tensor& t, const char* name, at::ScalarType dt, int dev, int64_t numel = -1) {
  on_device(dev, t, name);
  if (t.scalar_type() != dt)
    type_error(std::string(name) + " must be " + name_of(dt) + ", not " + name_of(t.scalar_type()));
  if (!t.is_contiguous()) value_error(std::string(name) + " must be contiguous");
  if (numel >= 0 && t.numel() != numel)
    value_error(std::string(name) + " must have " + std::to_string(numel) + " elements, not " + std::to_string(t.numel()));
  return t.data_ptr();
}
void* whole(const OptTensor& t, const char* name, at::ScalarType dt, int dev, int64_t numel = -1) {
  return t ? whole(*t, name, dt, dev, numel) : nullptr;
}

vx_rows rows_of(const Tensor& t, const char* name, int64_t n, int64_t heads, int64_t dim, at::ScalarType dt, int dev) {
  on_device(dev, t, name);
  if (t.dim() != 3 || t.size(0) != n || t.size(2) != dim || (heads >= 0 && t.size(1) != heads))
    value_error(std::string(name) + " must be [" + std::to_string(n) + ", " +
                (heads >= 0 ? std::to_string(heads) : std::string("heads")) + ", " + std::to_string(dim) + "], not " +
                shape_of(t));
  if (t.scalar_type() != dt)
    type_error(std::string(name) + " must be " + name_of(dt) + ", not " + name_of(t.scalar_type()));
  if (dim > 1 && t.stride(2) != 1) value_error(std::string(name) + ": the elements of a head must be contiguous");
  return {t.data_ptr(), t.stride(0), t.stride(1)};
}

Tensor new_rows(const Tensor& like) { return at::empty(like.sizes(), like.options()); }

// Rows of two token tensors may meet: their storage ranges do, unless both have the same distance from row to row and
// lie beside one another within it (heads of one fused row).
bool overlap(const Tensor& a, const Tensor& b) {
  if (a.numel() == 0 || b.numel() == 0 || a.storage().data() != b.storage().data()) return false;
  auto extent = [](const Tensor& t, int64_t from) {   // bytes that dims `from` on reach over
    int64_t last = 0;
    for (int64_t i = from; i < t.dim(); ++i) last += (t.size(i) - 1) * t.stride(i);
    return (last + 1) * t.element_size();
  };
  const char *p = static_cast<const char*>(a.data_ptr()), *q = static_cast<const char*>(b.data_ptr());
  if (q >= p + extent(a, 0) || p >= q + extent(b, 0)) return false;
  if (a.dim() != 3 || b.dim() != 3) return true;
  const int64_t row = a.stride(0) * a.element_size();
  if (row <= 0 || row != b.stride(0) * b.element_size()) return true;
  const int64_t d = ((q - p) % row + row) % row;   // b's rows behind a's
  return d < extent(a, 1) || d + extent(b, 1) > row;
}
// Rows of a tensor that is written, which may not share elements with one another (an expanded tensor, say): rows of
// heads, or heads of rows.
vx_rows out_rows(const Tensor& t, const char* name, int64_t n, int64_t heads, int64_t dim, at::ScalarType dt, int dev) {
  const vx_rows r = rows_of(t, name, n, heads, dim, dt, dev);
  auto nested = [&](int64_t in, int64_t in_stride, int64_t over, int64_t over_stride) {
    const int64_t row = in > 1 ? (in - 1) * in_stride + dim : dim;
    return (in <= 1 || in_stride >= dim) && (over <= 1 || over_stride >= row);
  };
  if (t.numel() > 0 && !nested(t.size(1), r.head, n, r.row) && !nested(n, r.row, t.size(1), r.head))
    value_error(std::string(name) + ": rows overlap one another");
  return r;
}
bool same_rows(const Tensor& a, const Tensor& b) { return a.data_ptr() == b.data_ptr() && a.strides() == b.strides(); }

cudaStream_t stream_of(int dev) { return c10::cuda::getCurrentCUDAStream(static_cast<c10::DeviceIndex>(dev)).stream(); }

// Scratch of a call: the caller's workspace, else a block of torch's allocator
// (one per call, so that calls on several streams and captured graphs do not
// share one), else, where only the status word is needed, a buffer of the
// device that nobody reads.
struct Scratch {
  void* p;
  size_t bytes;
  Tensor keep;
  Scratch(int64_t ws, int64_t ws_bytes, size_t need, int dev) : p(reinterpret_cast<void*>(ws)), bytes(ws_bytes) {
    if (ws != 0) return;
    const auto opt = at::TensorOptions().dtype(at::kByte).device(at::kCUDA, dev);
    if (need <= kStatusBuf) {
      static auto* status = new std::map<int, Tensor>;   // never freed: torch may be gone at exit
      Tensor& t = (*status)[dev];
      if (!t.defined()) t = at::empty({static_cast<int64_t>(kStatusBuf)}, opt);
      p = t.data_ptr();
      bytes = kStatusBuf;
    } else {
      keep = at::empty({static_cast<int64_t>(need)}, opt);
      p = keep.data_ptr();
      bytes = need;
    }
  }
};

// The tensors of a paged cache and their C description, checked when it is
// made and again when a tensor has changed in place (moved, resized, another
// view of its storage).
struct Cache {
  Tensor k, v, table, lens, pos;
  OptTensor acc;
  vx_paged_cache c{};
  int dev = 0;
  struct Seen {
    const void* p;
    std::array<int64_t, 5> size;
    int64_t dim;
    at::ScalarType dt;
    bool operator==(const Seen& o) const { return p == o.p && size == o.size && dim == o.dim && dt == o.dt; }
  };
  std::array<Seen, 6> seen{};   // the tensors as described

  static Seen look(const Tensor& t) {
    Seen s{t.data_ptr(), {}, t.is_contiguous() ? t.dim() : -1, t.scalar_type()};
    for (int64_t i = 0; i < t.dim() && i < 5; ++i) s.size[i] = t.size(i);
    return s;
  }
  std::array<Seen, 6> look() const {
    return {look(k), look(v), look(table), look(lens), look(pos), acc ? look(*acc) : Seen{}};
  }

  Cache(Tensor k_, Tensor v_, OptTensor acc_, Tensor table_, Tensor lens_, Tensor pos_)
      : k(std::move(k_)), v(std::move(v_)), table(std::move(table_)), lens(std::move(lens_)), pos(std::move(pos_)),
        acc(std::move(acc_)) {
    describe();
  }
  void describe() {
    if (k.dim() != 5 || v.sizes() != k.sizes() || v.scalar_type() != k.scalar_type())
      value_error("cache k and v must be [layers, pages, kv_heads, page_size, head_dim] of one dtype");
    if (table.dim() != 2) value_error("cache table must be [seqs, max_pages]");
    if (!k.is_cuda()) value_error("k must be a CUDA tensor");
    dev = k.get_device();
    const int64_t S = table.size(0), D = k.size(4);
    c.dt = dtype_of(k, "k");
    c.k = whole(k, "k", k.scalar_type(), dev);
    c.v = whole(v, "v", k.scalar_type(), dev);
    c.acc = static_cast<float*>(whole(acc, "acc", at::kFloat, dev, k.numel() / (D > 0 ? D : 1)));
    c.table = static_cast<const int32_t*>(whole(table, "table", at::kInt, dev));
    c.lens = static_cast<int64_t*>(whole(lens, "lens", at::kLong, dev, S));
    c.pos = static_cast<int64_t*>(whole(pos, "pos", at::kLong, dev, S));
    auto narrow = [](int64_t x) { return static_cast<int>(x < 0 ? 0 : x > INT32_MAX ? INT32_MAX : x); };
    c.n_layers = narrow(k.size(0));
    c.n_pages = narrow(k.size(1));
    c.n_kv_heads = narrow(k.size(2));
    c.page_size = narrow(k.size(3));
    c.head_dim = narrow(D);
    c.n_seqs = narrow(S);
    c.max_pages = narrow(table.size(1));
    seen = look();
  }
  const vx_paged_cache* fresh() {
    if (!(look() == seen)) describe();
    return &c;
  }
};

const int32_t* starts(const Tensor& q_start, const Cache& cache) {
  return static_cast<const int32_t*>(whole(q_start, "q_start", at::kInt, cache.dev, cache.c.n_seqs + 1ll));
}

Tensor rope_fwd(const Tensor& x, const Tensor& pos, int64_t rope, OptTensor out) {
  if (x.dim() != 3) value_error("x must be [n, heads, head_dim], not " + shape_of(x));
  const vx_dtype dt = dtype_of(x, "x");
  if (!x.is_cuda()) value_error("x must be a CUDA tensor");
  const int dev = x.get_device();
  const int64_t n = x.size(0), heads = x.size(1), dim = x.size(2);
  const vx_rows xr = rows_of(x, "x", n, heads, dim, x.scalar_type(), dev);
  const auto* p = static_cast<const int64_t*>(whole(pos, "pos", at::kLong, dev, n));
  c10::cuda::CUDAGuard guard(static_cast<c10::DeviceIndex>(dev));
  if (!out)
    out = new_rows(x);
  else if (!same_rows(*out, x) && overlap(x, *out))
    value_error("out overlaps x without being x");
  const vx_rows yr = out_rows(*out, "out", n, heads, dim, x.scalar_type(), dev);
  check(vx_rope_fwd(&xr, &yr, dt, n, static_cast<int>(std::min<int64_t>(heads, INT32_MAX)),
                    static_cast<int>(std::min<int64_t>(dim, INT32_MAX)), p, reinterpret_cast<const vx_rope_cfg*>(rope),
                    stream_of(dev)),
        "vx_rope_fwd");
  return *out;
}

OptTensor paged_append(Cache& cache, int layer, const Tensor& k, const Tensor& v, const Tensor& q_start, int max_q,
                       int64_t rope, const OptTensor& q, OptTensor q_out, int64_t ws, int64_t ws_bytes) {
  const vx_paged_cache* c = cache.fresh();
  const auto dt = cache.k.scalar_type();
  if (k.dim() != 3) value_error("k must be [n, kv_heads, head_dim], not " + shape_of(k));
  const int64_t n = k.size(0);
  const vx_rows kr = rows_of(k, "k", n, c->n_kv_heads, c->head_dim, dt, cache.dev);
  const vx_rows vr = rows_of(v, "v", n, c->n_kv_heads, c->head_dim, dt, cache.dev);
  const int32_t* qs = starts(q_start, cache);
  c10::cuda::CUDAGuard guard(static_cast<c10::DeviceIndex>(cache.dev));
  vx_rows qr{}, qo{};
  int heads = 0;
  if (q_out && !q) value_error("q_out without q");
  if (q) {
    qr = rows_of(*q, "q", n, -1, c->head_dim, dt, cache.dev);
    heads = static_cast<int>(std::min<int64_t>(q->size(1), INT32_MAX));
    if (!q_out)
      q_out = new_rows(*q);
    else if (!same_rows(*q_out, *q) && overlap(*q, *q_out))
      value_error("q_out overlaps q without being q");
    qo = out_rows(*q_out, "q_out", n, q->size(1), c->head_dim, dt, cache.dev);
  }
  Scratch s(ws, ws_bytes, kStatusBytes, cache.dev);
  check(vx_paged_append(c, layer, reinterpret_cast<const vx_rope_cfg*>(rope), q ? &qr : nullptr, q ? &qo : nullptr, heads,
                        &kr, &vr, qs, n, max_q, s.p, s.bytes, stream_of(cache.dev)),
        "vx_paged_append");
  return q_out;
}

void paged_advance(Cache& cache, const Tensor& q_start, int64_t n_tokens, int max_q, int64_t ws, int64_t ws_bytes) {
  const vx_paged_cache* c = cache.fresh();
  const int32_t* qs = starts(q_start, cache);
  c10::cuda::CUDAGuard guard(static_cast<c10::DeviceIndex>(cache.dev));
  Scratch s(ws, ws_bytes, kStatusBytes, cache.dev);
  check(vx_paged_advance(c, qs, n_tokens, max_q, s.p, s.bytes, stream_of(cache.dev)), "vx_paged_advance");
}

py::object paged_attn_fwd(Cache& cache, int layer, const Tensor& q, const Tensor& q_start, int max_q, int64_t max_kv,
                          int window, const OptTensor& prefix, double cap, const OptTensor& slopes, double scale,
                          std::optional<double> track, bool return_lse, OptTensor out, OptTensor lse, int64_t ws,
                          int64_t ws_bytes) {
  const vx_paged_cache* c = cache.fresh();
  const auto dt = cache.k.scalar_type();
  if (q.dim() != 3) value_error("q must be [n, heads, head_dim], not " + shape_of(q));
  const int64_t n = q.size(0), heads = q.size(1);
  const int hq = static_cast<int>(std::min<int64_t>(heads, INT32_MAX));
  const vx_rows qr = rows_of(q, "q", n, heads, c->head_dim, dt, cache.dev);
  const int32_t* qs = starts(q_start, cache);
  vx_attn_opts opts{};
  opts.scale = static_cast<float>(scale);
  opts.cap = static_cast<float>(cap);
  opts.window = window;
  opts.prefix = static_cast<const int32_t*>(whole(prefix, "prefix", at::kInt, cache.dev, c->n_seqs));
  opts.slopes = static_cast<const float*>(whole(slopes, "slopes", at::kFloat, cache.dev, heads));
  c10::cuda::CUDAGuard guard(static_cast<c10::DeviceIndex>(cache.dev));
  if (!out)
    out = new_rows(q);
  else if (overlap(q, *out))
    value_error("out overlaps q");
  const vx_rows orr = out_rows(*out, "out", n, heads, c->head_dim, dt, cache.dev);
  if (!lse && return_lse) lse = at::empty({n, heads}, q.options().dtype(at::kFloat));
  auto* lp = static_cast<float*>(whole(lse, "lse", at::kFloat, cache.dev, n * heads));
  const size_t need = ws != 0 ? 0 : vx_paged_attn_workspace(c, hq, n, max_q, max_kv, lp != nullptr, track.has_value());
  Scratch s(ws, ws_bytes, need, cache.dev);
  check(vx_paged_attn_fwd(c, layer, &qr, &orr, lp, hq, qs, n, max_q, max_kv, &opts, track.has_value(),
                          static_cast<float>(track.value_or(0.0)), s.p, s.bytes, stream_of(cache.dev)),
        "vx_paged_attn_fwd");
  if (return_lse) return py::make_tuple(*out, *lse);
  return py::cast(*out);
}

void paged_evict(Cache& cache, int64_t keep, int64_t recent, Cache* dst, OptTensor kept, int64_t ws, int64_t ws_bytes) {
  const vx_paged_cache* c = cache.fresh();
  const vx_paged_cache* d = c;
  if (dst != nullptr) {
    d = dst->fresh();
    on_device(cache.dev, dst->k, "dst");
  }
  const int64_t lanes = static_cast<int64_t>(c->n_layers) * c->n_seqs * c->n_kv_heads;
  int64_t slots = -1;   // a negative keep is refused below
  if (kept && keep >= 0 && __builtin_mul_overflow(lanes, keep, &slots)) value_error("kept cannot have that many slots");
  auto* kp = static_cast<int32_t*>(whole(kept, "kept", at::kInt, cache.dev, slots));   // keep 0: no address, no entries
  c10::cuda::CUDAGuard guard(static_cast<c10::DeviceIndex>(cache.dev));
  const size_t need = ws != 0 ? 0 : kp ? kStatusBytes : vx_paged_evict_workspace(c, keep);
  Scratch s(ws, ws_bytes, need, cache.dev);
  check(vx_paged_evict(c, d, keep, recent, kp, s.p, s.bytes, stream_of(cache.dev)), "vx_paged_evict");
}

}  // namespace

PYBIND11_MODULE(_bind, m) {
  m.doc() = "Argument marshalling of the paged-cache entry points of libvx";
  py::class_<Cache>(m, "Cache")
      .def(py::init<Tensor, Tensor, OptTensor, Tensor, Tensor, Tensor>())
      .def("address", [](Cache& c) { return reinterpret_cast<int64_t>(c.fresh()); })
      .def_readonly("dev", &Cache::dev);
  m.def("rope_fwd", &rope_fwd);
  m.def("paged_append", &paged_append);
  m.def("paged_advance", &paged_advance);
  m.def("paged_attn_fwd", &paged_attn_fwd);
  m.def("paged_evict", &paged_evict);
}
