// Argument checks and marshalling of the cache operators for Python: the same
// C ABI as the ctypes binding, reached without its per-call cost (20 to 35 us
// of interpreter time on a Grace core for a dozen tensors, against 3 to 10 us
// of GPU time for a small batch's step; here about 3 us).
#include <ATen/ATen.h>
#include <c10/cuda/CUDACachingAllocator.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/utils/pybind.h>

#include <limits>
#include <vector>

#include "specdec_verify.h"

namespace py = pybind11;

namespace {

using at::Tensor;
using OptTensor = std::optional<Tensor>;

void check_type(bool ok, const char* what) {
  if (!ok) throw py::type_error(what);
}
void check_value(bool ok, const char* what) {
  if (!ok) throw py::value_error(what);
}

void same_device(const Tensor& a, const Tensor& b) {
  check_value(a.device() == b.device(), "all tensors must be on one CUDA device");
}
void same_device(const Tensor& a, const OptTensor& b) {
  if (b) same_device(a, *b);
}

template <typename T>
T* ptr(const OptTensor& t) {
  return t ? static_cast<T*>(t->data_ptr()) : nullptr;
}
template <typename T>
T* ptr(const Tensor& t) {
  return static_cast<T*>(t.data_ptr());
}

// Elements between consecutive positions of t [B, n, H, D], whose sequences
// follow each other at n times that (a contiguous tensor, or a slice of a
// fused projection).
long long row_stride(const Tensor& t) {
  const int64_t B = t.size(0), n = t.size(1), H = t.size(2), D = t.size(3);
  int64_t sn = t.stride(1);
  if (n == 1) sn = B > 1 ? t.stride(0) : H * D;
  check_value(!((t.stride(3) != 1 && D > 1) || (t.stride(2) != D && H > 1) || (t.stride(0) != n * sn && B > 1) ||
                sn < H * D || sn % 8 != 0),
              "the heads of a position must be contiguous, positions a multiple of 8 elements apart and "
              "sequences n positions apart");
  return sn;
}

void check_ints(const Tensor& t, at::IntArrayRef shape, const char* type, const char* size) {
  check_type(t.scalar_type() == at::kInt && t.is_contiguous() && t.is_cuda(), type);
  check_value(t.sizes() == shape, size);
}

void check_cache(const Tensor& k, const Tensor& v, at::ScalarType type, const char* what) {
  for (const Tensor* t : {&k, &v})
    check_type(t->scalar_type() == type && t->dim() == 4 && t->is_contiguous() && t->is_cuda(), what);
  check_value(k.sizes() == v.sizes(), "k_cache and v_cache must have one shape");
}
void check_scales(const Tensor& k, const Tensor& ks, const Tensor& vs) {
  const int64_t want[3] = {k.size(0), k.size(2), (k.size(1) + SPECDEC_KV8_BLOCK - 1) / SPECDEC_KV8_BLOCK};
  for (const Tensor* t : {&ks, &vs}) {
    check_type(t->scalar_type() == at::kFloat && t->is_contiguous() && t->is_cuda(),
               "the scales must be contiguous float32 CUDA tensors");
    check_value(t->sizes() == at::IntArrayRef(want, 3), "the scales must have shape [B, Hkv, ceil(Lmax / 32)]");
  }
}
constexpr const char* kCodes = "the caches must be contiguous float8_e4m3fn CUDA tensors [B, Lmax, Hkv, D]";

// Positive numbers too small for fp32 stay positive: 0 would mean the default.
float to_float(double x) { return x > 0 && (float)x == 0.f ? std::numeric_limits<float>::denorm_min() : (float)x; }

int narrow(int64_t x) { return (int)std::min<int64_t>(x, INT32_MAX); }   // the C call refuses what it cannot hold

// The caller's workspace, or one for this call from the current stream's pool
// (straight from the allocator, without a tensor around it).
void* workspace_of(const OptTensor& given, size_t bytes, c10::DataPtr& own, size_t& have) {
  if (given) {
    check_type(given->is_contiguous() && given->is_cuda(), "workspace must be a contiguous CUDA tensor");
    have = given->nbytes();
    return given->data_ptr();
  }
  own = c10::cuda::CUDACachingAllocator::get()->allocate(bytes);
  have = bytes;
  return own.get();
}

int append_kv8(const Tensor& k_new, const Tensor& v_new, const Tensor& k_cache, const Tensor& v_cache,
               const Tensor& k_scale, const Tensor& v_scale, const Tensor& start, const OptTensor& counts,
               const OptTensor& rows, const OptTensor& workspace) {
  for (const Tensor* t : {&k_new, &v_new})
    check_type(t->scalar_type() == at::kBFloat16 && t->is_cuda() && t->dim() == 4,
               "k_new and v_new must be bfloat16 CUDA tensors [B, n, Hkv, D]");
  check_cache(k_cache, v_cache, at::kFloat8_e4m3fn, kCodes);
  check_scales(k_cache, k_scale, v_scale);
  const int64_t B = k_new.size(0), n = k_new.size(1), Hkv = k_new.size(2), D = k_new.size(3), Lmax = k_cache.size(1);
  check_value(v_new.sizes() == k_new.sizes() && k_cache.size(0) == B && k_cache.size(2) == Hkv && k_cache.size(3) == D,
              "k_new and v_new must be [B, n, Hkv, D] for a cache [B, Lmax, Hkv, D]");
  check_ints(start, {B}, "start must be a contiguous int32 CUDA tensor", "start must have shape [B]");
  if (counts) check_ints(*counts, {B}, "counts must be a contiguous int32 CUDA tensor", "counts must have shape [B]");
  if (rows) check_ints(*rows, {B, n}, "rows must be a contiguous int32 CUDA tensor", "rows must have shape [B, n]");
  for (const Tensor* t : {&v_new, &k_cache, &v_cache, &k_scale, &v_scale, &start}) same_device(k_new, *t);
  same_device(k_new, counts);
  same_device(k_new, rows);
  same_device(k_new, workspace);
  const long long ks = B ? row_stride(k_new) : Hkv * D, vs = B ? row_stride(v_new) : Hkv * D;
  const c10::cuda::CUDAGuard guard(k_new.device());
  c10::DataPtr own;
  size_t have;
  void* ws = workspace_of(workspace, specdec_kv8_append_workspace_size(), own, have);
  return specdec_kv8_append(k_new.data_ptr(), ks, v_new.data_ptr(), vs, ptr<int32_t>(start), ptr<int32_t>(counts),
                            ptr<int32_t>(rows), narrow(B), narrow(n), narrow(Hkv), narrow(D), narrow(Lmax),
                            k_cache.data_ptr(), v_cache.data_ptr(), ptr<float>(k_scale), ptr<float>(v_scale), ws,
                            have, c10::cuda::getCurrentCUDAStream(k_new.device().index()).stream());
}

std::pair<int, Tensor> cache_attention(const Tensor& q, const Tensor& k_cache, const Tensor& v_cache,
                                       const OptTensor& k_scale, const OptTensor& v_scale, const Tensor& seq_lens,
                                       double scale, double softcap, int64_t window, const OptTensor& slopes,
                                       const py::object& parent, const OptTensor& out_given,
                                       const OptTensor& workspace) {
  const bool e4m3 = k_scale.has_value();
  if (e4m3) {
    check_type(v_scale.has_value(), "the scales must be contiguous float32 CUDA tensors");
    check_cache(k_cache, v_cache, at::kFloat8_e4m3fn, kCodes);
    check_scales(k_cache, *k_scale, *v_scale);
    same_device(q, *k_scale);
    same_device(q, *v_scale);
  } else {
    check_cache(k_cache, v_cache, at::kBFloat16,
                "the caches must be contiguous bfloat16 CUDA tensors [B, Lmax, Hkv, D]");
  }
  check_type(q.scalar_type() == at::kBFloat16 && q.is_cuda() && q.dim() == 4,
             "q must be a bfloat16 CUDA tensor [B, n_new, Hq, D]");
  const int64_t B = q.size(0), n = q.size(1), Hq = q.size(2), D = q.size(3), Lmax = k_cache.size(1),
                Hkv = k_cache.size(2);
  check_value(k_cache.size(0) == B && k_cache.size(3) == D,
              "q [B, n_new, Hq, D] and the cache [B, Lmax, Hkv, D] do not fit");
  check_ints(seq_lens, {B}, "seq_lens must be a contiguous int32 CUDA tensor", "seq_lens must have shape [B]");
  if (slopes) {
    check_type(slopes->scalar_type() == at::kFloat && slopes->is_contiguous() && slopes->is_cuda(),
               "slopes must be a contiguous float32 CUDA tensor");
    check_value(slopes->sizes() == at::IntArrayRef{Hq}, "slopes must have one entry per query head");
  }
  std::vector<int32_t> par;
  if (!parent.is_none()) {
    try {
      for (const py::handle x : parent) par.push_back(x.cast<int32_t>());
    } catch (const py::cast_error&) {
      throw py::type_error("parent must hold 32-bit integers");
    }
    check_value((int64_t)par.size() == n, "parent must have one entry per new position");
  }
  for (const Tensor* t : {&k_cache, &v_cache, &seq_lens}) same_device(q, *t);
  same_device(q, slopes);
  same_device(q, out_given);
  same_device(q, workspace);
  const long long stride = B ? row_stride(q) : Hq * D;
  const c10::cuda::CUDAGuard guard(q.device());
  Tensor out;
  if (out_given) {
    check_type(out_given->scalar_type() == at::kBFloat16 && out_given->sizes() == q.sizes() &&
                   out_given->is_contiguous(),
               "out must be a contiguous bfloat16 CUDA tensor of q's shape");
    out = *out_given;
  } else {
    out = at::empty({B, n, Hq, D}, q.options());
  }
  size_t bytes = 0;
  if (!workspace) {
    bytes = (e4m3 ? specdec_verify_attention_kv8_workspace_size : specdec_verify_attention_masked_workspace_size)(
        narrow(B), narrow(n), narrow(Hq), narrow(Hkv), narrow(D), narrow(Lmax));
    if (bytes == 0) return {SPECDEC_ERR_UNSUPPORTED, out};
  }
  c10::DataPtr own;
  size_t have;
  void* ws = workspace_of(workspace, bytes, own, have);
  void* stream = c10::cuda::getCurrentCUDAStream(q.device().index()).stream();
  const int32_t* pp = par.empty() ? nullptr : par.data();
  // a window beyond any distance is none; a negative one is the C call's to refuse
  const int win = window > INT32_MAX ? 0 : window < 0 ? -1 : (int)window;
  const int rc =
      e4m3 ? specdec_verify_attention_kv8(q.data_ptr(), stride, k_cache.data_ptr(), v_cache.data_ptr(),
                                          ptr<float>(k_scale), ptr<float>(v_scale), ptr<int32_t>(seq_lens), pp,
                                          ptr<float>(slopes), narrow(B), narrow(n), narrow(Hq), narrow(Hkv),
                                          narrow(D), narrow(Lmax), to_float(scale), to_float(softcap), win,
                                          out.data_ptr(), ws, have, stream)
           : specdec_verify_attention_masked(q.data_ptr(), stride, k_cache.data_ptr(), v_cache.data_ptr(),
                                             ptr<int32_t>(seq_lens), pp, ptr<float>(slopes), narrow(B), narrow(n),
                                             narrow(Hq), narrow(Hkv), narrow(D), narrow(Lmax), to_float(scale),
                                             to_float(softcap), win, out.data_ptr(), ws, have, stream);
  return {rc, out};
}

}  // namespace

PYBIND11_MODULE(_native, m) {
  m.def("append_kv8", &append_kv8);
  m.def("cache_attention", &cache_attention);
}
