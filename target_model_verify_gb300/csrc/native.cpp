// Argument checks and marshalling of the cache and prompt operators for Python: the same
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

// The same of packed rows t [T, H, D].
long long packed_stride(const Tensor& t) {
  const int64_t T = t.size(0), H = t.size(1), D = t.size(2);
  const int64_t sn = T > 1 ? t.stride(0) : H * D;
  check_value(!((t.stride(2) != 1 && D > 1) || (t.stride(1) != D && H > 1) || sn < H * D || sn % 8 != 0),
              "the heads of a row must be contiguous, and rows a multiple of 8 elements apart");
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
constexpr const char* kPool = "the caches must be contiguous bfloat16 CUDA tensors [pages, page, Hkv, D]";
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
                                       const OptTensor& k_scale, const OptTensor& v_scale, const OptTensor& table,
                                       const Tensor& seq_lens, double scale, double softcap, int64_t window,
                                       const OptTensor& slopes, const py::object& parent, const OptTensor& out_given,
                                       const OptTensor& workspace) {
  const bool e4m3 = k_scale.has_value();
  if (table) {
    check_cache(k_cache, v_cache, at::kBFloat16, kPool);
  } else if (e4m3) {
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
  if (table) {
    check_value(k_cache.size(3) == D, "q [B, n_new, Hq, D] and the cache [pages, page, Hkv, D] do not fit");
    check_type(table->scalar_type() == at::kInt && table->is_contiguous() && table->is_cuda() && table->dim() == 2,
               "table must be a contiguous int32 CUDA tensor [B, max_pages]");
    check_value(table->size(0) == B, "table must have shape [B, max_pages]");
    same_device(q, table);
  } else {
    check_value(k_cache.size(0) == B && k_cache.size(3) == D,
                "q [B, n_new, Hq, D] and the cache [B, Lmax, Hkv, D] do not fit");
  }
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
  const int n_pages = table ? narrow(k_cache.size(0)) : 0, max_pages = table ? narrow(table->size(1)) : 0;
  if (!workspace) {
    if (table)
      bytes = specdec_verify_attention_paged_workspace_size(narrow(B), narrow(n), narrow(Hq), narrow(Hkv), narrow(D),
                                                            n_pages, narrow(Lmax), max_pages);
    else
      bytes = (e4m3 ? specdec_verify_attention_kv8_workspace_size : specdec_verify_attention_masked_workspace_size)(
          narrow(B), narrow(n), narrow(Hq), narrow(Hkv), narrow(D), narrow(Lmax));
    if (bytes == 0) return {SPECDEC_ERR_UNSUPPORTED, out};
  }
  c10::DataPtr own;
  size_t have;
  void* ws = workspace_of(workspace, bytes, own, have);
  void* cu_stream = c10::cuda::getCurrentCUDAStream(q.device().index()).stream();
  const int32_t* pp = par.empty() ? nullptr : par.data();
  // a window beyond any distance is none; a negative one is the C call's to refuse
  const int win = window > INT32_MAX ? 0 : window < 0 ? -1 : (int)window;
  const int rc =
      table ? specdec_verify_attention_paged(q.data_ptr(), stride, k_cache.data_ptr(), v_cache.data_ptr(),
                                             ptr<int32_t>(table), ptr<int32_t>(seq_lens), pp, ptr<float>(slopes),
                                             narrow(B), narrow(n), narrow(Hq), narrow(Hkv), narrow(D), n_pages,
                                             narrow(Lmax), max_pages, to_float(scale), to_float(softcap), win,
                                             out.data_ptr(), ws, have, cu_stream)
      : e4m3 ? specdec_verify_attention_kv8(q.data_ptr(), stride, k_cache.data_ptr(), v_cache.data_ptr(),
                                          ptr<float>(k_scale), ptr<float>(v_scale), ptr<int32_t>(seq_lens), pp,
                                          ptr<float>(slopes), narrow(B), narrow(n), narrow(Hq), narrow(Hkv),
                                          narrow(D), narrow(Lmax), to_float(scale), to_float(softcap), win,
                                          out.data_ptr(), ws, have, cu_stream)
           : specdec_verify_attention_masked(q.data_ptr(), stride, k_cache.data_ptr(), v_cache.data_ptr(),
                                             ptr<int32_t>(seq_lens), pp, ptr<float>(slopes), narrow(B), narrow(n),
                                             narrow(Hq), narrow(Hkv), narrow(D), narrow(Lmax), to_float(scale),
                                             to_float(softcap), win, out.data_ptr(), ws, have, cu_stream);
  return {rc, out};
}

std::pair<int, OptTensor> plan_pages(const Tensor& table, const Tensor& held, const Tensor& free_pages,
                                     const Tensor& n_free, const Tensor& start, const Tensor& counts, int64_t page,
                                     std::optional<int64_t> n, const OptTensor& slots_given,
                                     const OptTensor& cu_rows, const OptTensor& workspace) {
  check_type(table.scalar_type() == at::kInt && table.is_contiguous() && table.is_cuda() && table.dim() == 2,
             "table must be a contiguous int32 CUDA tensor [B, max_pages]");
  check_type(free_pages.scalar_type() == at::kInt && free_pages.is_contiguous() && free_pages.is_cuda() &&
                 free_pages.dim() == 1,
             "free must be a contiguous int32 CUDA tensor [pages]");
  const int64_t B = table.size(0);
  check_ints(held, {B}, "held must be a contiguous int32 CUDA tensor", "held must have shape [B]");
  check_ints(n_free, {1}, "n_free must be a contiguous int32 CUDA tensor", "n_free must have shape [1]");
  check_ints(start, {B}, "start must be a contiguous int32 CUDA tensor", "start must have shape [B]");
  check_ints(counts, {B}, "counts must be a contiguous int32 CUDA tensor", "counts must have shape [B]");
  check_value(!(n && slots_given), "give n for a new map, or slots to fill, not both");
  check_value(!n || *n >= 0, "n must not be negative");
  if (cu_rows) {
    check_ints(*cu_rows, {B + 1}, "cu_rows must be a contiguous int32 CUDA tensor", "cu_rows must have shape [B + 1]");
    check_value(n || slots_given, "cu_rows places the rows of a map: give slots or n");
  }
  if (slots_given) {
    check_type(slots_given->scalar_type() == at::kInt && slots_given->is_contiguous() && slots_given->is_cuda(),
               "slots must be a contiguous int32 CUDA tensor");
    check_value(cu_rows ? slots_given->dim() == 1 : slots_given->dim() == 2 && slots_given->size(0) == B,
                "slots must have shape [B, n], or [rows] with cu_rows");
  }
  for (const Tensor* t : {&held, &free_pages, &n_free, &start, &counts}) same_device(table, *t);
  same_device(table, cu_rows);
  same_device(table, slots_given);
  same_device(table, workspace);
  const c10::cuda::CUDAGuard guard(table.device());
  OptTensor slots = slots_given;
  if (n) slots = cu_rows ? at::empty({*n}, table.options()) : at::empty({B, *n}, table.options());
  c10::DataPtr own;
  size_t have;
  void* ws = workspace_of(workspace, specdec_plan_pages_workspace_size(), own, have);
  const int per = slots && !cu_rows ? narrow(slots->size(1)) : 0;
  // (a map without entries has no memory, and is a map all the same: it is given an address that is not used)
  int32_t* const map = !slots ? nullptr : slots->numel() ? ptr<int32_t>(slots) : ptr<int32_t>(n_free);
  const int rc = specdec_plan_pages(
      ptr<int32_t>(table), ptr<int32_t>(held), ptr<int32_t>(free_pages), ptr<int32_t>(n_free), ptr<int32_t>(start),
      ptr<int32_t>(counts), ptr<int32_t>(cu_rows), narrow(B), narrow(table.size(1)),
      narrow(free_pages.size(0)), narrow(page), per, slots ? slots->numel() : 0, map,
      ws, have,
      c10::cuda::getCurrentCUDAStream(table.device().index()).stream());
  return {rc, slots};
}

int append_paged(const Tensor& k_new, const Tensor& v_new, const Tensor& k_pages, const Tensor& v_pages,
                 const Tensor& slots, const OptTensor& rows, const OptTensor& workspace) {
  for (const Tensor* t : {&k_new, &v_new})
    check_type(t->scalar_type() == at::kBFloat16 && t->is_cuda() && (t->dim() == 4 || t->dim() == 3),
               "k_new and v_new must be bfloat16 CUDA tensors [B, n, Hkv, D] or [rows, Hkv, D]");
  check_cache(k_pages, v_pages, at::kBFloat16, kPool);
  check_value(k_new.sizes() == v_new.sizes() && k_new.size(-2) == k_pages.size(2) && k_new.size(-1) == k_pages.size(3),
              "k_new and v_new must have one shape, and the heads of the cache [pages, page, Hkv, D]");
  const bool packed = k_new.dim() == 3;
  const int64_t B = packed ? 1 : k_new.size(0), n = k_new.size(packed ? 0 : 1), Hkv = k_new.size(-2),
                D = k_new.size(-1);
  const at::IntArrayRef lead = k_new.sizes().slice(0, k_new.dim() - 2);
  check_ints(slots, lead, "slots must be a contiguous int32 CUDA tensor", "slots must have one entry per new row");
  if (rows) check_ints(*rows, lead, "rows must be a contiguous int32 CUDA tensor", "rows must have one entry per slot");
  for (const Tensor* t : {&v_new, &k_pages, &v_pages, &slots}) same_device(k_new, *t);
  same_device(k_new, rows);
  same_device(k_new, workspace);
  auto stride = [&](const Tensor& t) { return !B || !n ? Hkv * D : packed ? packed_stride(t) : row_stride(t); };
  const long long ks = stride(k_new), vs = stride(v_new);
  const c10::cuda::CUDAGuard guard(k_new.device());
  c10::DataPtr own;
  size_t have;
  void* ws = workspace_of(workspace, specdec_paged_append_workspace_size(), own, have);
  return specdec_paged_append(k_new.data_ptr(), ks, v_new.data_ptr(), vs, ptr<int32_t>(slots), ptr<int32_t>(rows),
                              narrow(B), narrow(n), narrow(Hkv), narrow(D), narrow(k_pages.size(0)),
                              narrow(k_pages.size(1)), k_pages.data_ptr(), v_pages.data_ptr(), ws, have,
                              c10::cuda::getCurrentCUDAStream(k_new.device().index()).stream());
}

std::pair<int, Tensor> prompt_attention(const Tensor& q, const Tensor& k, const Tensor& v, const Tensor& cu_seqlens,
                                        double scale, double softcap, int64_t window, const OptTensor& slopes,
                                        const OptTensor& out_given, const OptTensor& workspace) {
  for (const Tensor* t : {&q, &k, &v})
    check_type(t->scalar_type() == at::kBFloat16 && t->is_cuda() && t->dim() == 3,
               "q, k and v must be bfloat16 CUDA tensors [T, heads, D]");
  const int64_t T = q.size(0), Hq = q.size(1), D = q.size(2), Hkv = k.size(1);
  check_value(k.sizes() == v.sizes() && k.size(0) == T && k.size(2) == D,
              "q [T, Hq, D] and k, v [T, Hkv, D] do not fit");
  check_type(cu_seqlens.scalar_type() == at::kInt && cu_seqlens.is_contiguous() && cu_seqlens.is_cuda() &&
                 cu_seqlens.dim() == 1,
             "cu_seqlens must be a contiguous int32 CUDA tensor [B + 1]");
  check_value(cu_seqlens.size(0) >= 1, "cu_seqlens must have at least one entry");
  if (slopes) {
    check_type(slopes->scalar_type() == at::kFloat && slopes->is_contiguous() && slopes->is_cuda(),
               "slopes must be a contiguous float32 CUDA tensor");
    check_value(slopes->sizes() == at::IntArrayRef{Hq}, "slopes must have one entry per query head");
  }
  for (const Tensor* t : {&k, &v, &cu_seqlens}) same_device(q, *t);
  same_device(q, slopes);
  same_device(q, out_given);
  same_device(q, workspace);
  const int64_t B = cu_seqlens.size(0) - 1;
  const long long qs = T ? packed_stride(q) : Hq * D, ks = T ? packed_stride(k) : Hkv * D,
                  vs = T ? packed_stride(v) : Hkv * D;
  const c10::cuda::CUDAGuard guard(q.device());
  Tensor out;
  if (out_given) {
    check_type(out_given->scalar_type() == at::kBFloat16 && out_given->sizes() == q.sizes() &&
                   out_given->is_contiguous(),
               "out must be a contiguous bfloat16 CUDA tensor of q's shape");
    out = *out_given;
  } else {
    out = at::empty({T, Hq, D}, q.options());
  }
  size_t bytes = 0;
  if (!workspace) {
    bytes = specdec_prompt_attention_workspace_size(narrow(B), narrow(T), narrow(Hq), narrow(Hkv), narrow(D));
    if (bytes == 0) return {SPECDEC_ERR_UNSUPPORTED, out};
  }
  c10::DataPtr own;
  size_t have;
  void* ws = workspace_of(workspace, bytes, own, have);
  const int win = window > INT32_MAX ? 0 : window < 0 ? -1 : (int)window;
  const int rc = specdec_prompt_attention(
      q.data_ptr(), qs, k.data_ptr(), ks, v.data_ptr(), vs, ptr<int32_t>(cu_seqlens), ptr<float>(slopes), narrow(B),
      narrow(T), narrow(Hq), narrow(Hkv), narrow(D), to_float(scale), to_float(softcap), win, out.data_ptr(), ws, have,
      c10::cuda::getCurrentCUDAStream(q.device().index()).stream());
  return {rc, out};
}

}  // namespace

PYBIND11_MODULE(_native, m) {
  m.def("prompt_attention", &prompt_attention);
  m.def("plan_pages", &plan_pages);
  m.def("append_paged", &append_paged);
  m.def("append_kv8", &append_kv8);
  m.def("cache_attention", &cache_attention);
}
