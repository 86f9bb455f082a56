// _kvstore_torch: the tensor-level calls of include/kvstore_paged.h.
//
// Checks torch tensors, fills the C structs and calls the library on the
// tensors' device and its current stream.  The functions take their arguments
// by position (None for those left out), as fp8_kv_quantization_amd/__init__.py
// passes them, and return the library's status (attention: the output tensor,
// or a status below 0).  Written against torch's C++ API because a call's
// checks in Python cost several times what a small kernel takes (a 16-token
// append: 15 us a call against 3.5 us of kernel).
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <ATen/core/grad_mode.h>
#include <ATen/ops/empty.h>
#include <c10/hip/HIPStream.h>
#include <hip/hip_runtime_api.h>
#include <torch/csrc/autograd/python_variable.h>

#include <cmath>
#include <cstdarg>
#include <cstdint>
#include <exception>
#include <initializer_list>
#include <optional>
#include <string>

#include "kvstore_paged.h"

namespace {

// A Python exception to raise.
struct Raise {
  PyObject* type;
  std::string text;
};

[[noreturn]] void value_error(std::string text) { throw Raise{PyExc_ValueError, std::move(text)}; }
[[noreturn]] void type_error(std::string text) { throw Raise{PyExc_TypeError, std::move(text)}; }
struct AlreadySet {};   // the Python error is set

typedef const at::Tensor* Opt;   // NULL: None

Opt tensor(PyObject* o, const char* what, bool optional = false) {
  if (o == Py_None && optional) return nullptr;
  if (!THPVariable_Check(o)) type_error(std::string(what) + " must be a tensor");
  return &THPVariable_Unpack(o);
}

int64_t integer(PyObject* o, const char* what) {
  const long long v = PyLong_AsLongLong(o);
  if (v == -1 && PyErr_Occurred()) throw AlreadySet();
  if (v < 0) value_error(std::string(what) + " must not be negative");
  return v;
}

// The one GPU that holds every tensor.
struct Device {
  int index = -1;
  void add(Opt t) {
    if (t == nullptr) return;
    if (!t->is_cuda()) value_error("every tensor must be a GPU tensor");
    const int d = t->get_device();
    if (index >= 0 && d != index)
      value_error("all tensors must be on one GPU (found cuda:" + std::to_string(index) +
                  " and cuda:" + std::to_string(d) + ")");
    index = d;
  }
};

// Makes a device current while a call runs on it.
class OnDevice {
 public:
  explicit OnDevice(int index) {
    if (hipGetDevice(&before_) != hipSuccess) before_ = index;
    if (before_ != index) (void)hipSetDevice(index);
    index_ = index;
  }
  ~OnDevice() {
    if (before_ != index_) (void)hipSetDevice(before_);
  }
  hipStream_t stream() const { return c10::hip::getCurrentHIPStream((c10::DeviceIndex)index_).stream(); }

 private:
  int before_ = 0, index_ = 0;
};

int src_code(const at::Tensor& t, const char* what) {
  if (t.scalar_type() == at::kBFloat16) return KVSTORE_SRC_BF16;
  if (t.scalar_type() == at::kHalf) return KVSTORE_SRC_FP16;
  type_error(std::string(what) + " must be bfloat16 or float16, not " + c10::toString(t.scalar_type()));
}

int idx_code(const at::Tensor& t) {
  if (t.scalar_type() == at::kInt) return KVSTORE_IDX_I32;
  if (t.scalar_type() == at::kLong) return KVSTORE_IDX_I64;
  type_error(std::string("indices must be int32 or int64, got ") + c10::toString(t.scalar_type()));
}

const float* scalar(Opt t, const char* what) {
  if (t == nullptr) return nullptr;
  if (t->scalar_type() != at::kFloat || t->numel() != 1)
    type_error(std::string(what) + " must be one-element fp32 GPU tensors");
  return static_cast<const float*>(t->data_ptr());
}

// (page, offset, head) byte strides and slots of an fp32 scale cache [slots(, H)]
// or [pages, page_size(, H)].
int64_t fp32_scales(const at::Tensor& t, bool paged, bool per_head, int64_t H, int64_t page_size,
                    int64_t* page, int64_t* offset, int64_t* head) {
  if (t.scalar_type() != at::kFloat) type_error("scale caches must be float32 GPU tensors");
  const int64_t want = (paged ? 2 : 1) + (per_head ? 1 : 0);
  if (t.dim() != want) value_error("unsupported scale cache shape");
  if (per_head && t.size(want - 1) != H) value_error("per-head scale caches end in H");
  *head = per_head ? t.stride(want - 1) * 4 : 0;
  if (!paged) {
    *page = t.stride(0) * 4 * page_size;
    *offset = t.stride(0) * 4;
    return t.size(0);
  }
  if (t.size(1) != page_size) value_error("paged scale caches must be [pages, page_size(, H)]");
  *page = t.stride(0) * 4;
  *offset = t.stride(1) * 4;
  return t.size(0) * page_size;
}

// The same of an e8m0 scale cache [slots, H, D/32] or [pages, page_size, H, D/32].
int64_t block_scales(const at::Tensor& t, bool paged, int64_t H, int64_t blocks, int64_t page_size,
                     int64_t* page, int64_t* offset, int64_t* head) {
  if (t.scalar_type() != at::kByte && t.scalar_type() != at::kFloat8_e8m0fnu)
    type_error("4-bit caches take uint8 or float8_e8m0fnu GPU scale caches");
  const int64_t n = t.dim();
  if (n != (paged ? 4 : 3) || t.size(n - 2) != H || t.size(n - 1) != blocks ||
      (blocks > 1 && t.stride(n - 1) != 1) || (paged && t.size(1) != page_size))
    value_error("4-bit scale caches must be [slots, H, D/32] or [pages, page_size, H, D/32], "
                "contiguous in the last dim");
  *head = t.stride(n - 2);
  if (!paged) {
    *page = t.stride(0) * page_size;
    *offset = t.stride(0);
    return t.size(0);
  }
  *page = t.stride(0);
  *offset = t.stride(1);
  return t.size(0) * page_size;
}

// None of the calls has a backward pass: tensors that wait for one are refused.
void no_grad(std::initializer_list<Opt> tensors) {
  if (!at::GradMode::is_enabled()) return;
  for (Opt t : tensors)
    if (t && t->requires_grad())
      value_error("this call has no backward pass: detach tensors that require grad, or call it under torch.no_grad()");
}

struct Scales {
  Opt k_scale, v_scale, k_cache, v_cache;
};

// Fills the library's description of a K and a V cache.  `src`: the rows'
// type; `reads`: the call reads scales.
void fill_cache(kvstore_paged_cache* c, const at::Tensor& k, const at::Tensor& v, int64_t page_size,
                PyObject* size_limit, at::ScalarType src, const Scales& s, bool reads) {
  const at::ScalarType type = k.scalar_type();
  if (v.scalar_type() != type)
    type_error(std::string("k_cache and v_cache must share one dtype (") + c10::toString(type) +
               " != " + c10::toString(v.scalar_type()) + ")");
  if (page_size < 1) value_error("page_size must be positive");
  const int64_t n = k.dim();
  if (n != 3 && n != 4) value_error("a cache is 3-D (flat) or 4-D (paged), not " + std::to_string(n) + "-D");
  if (k.sizes() != v.sizes()) value_error("k_cache and v_cache shapes differ");
  if (k.stride(n - 1) != 1 || v.stride(n - 1) != 1) value_error("cache dim stride must be 1");
  const bool paged = n == 4;
  if (paged && k.size(1) != page_size)
    value_error("the paged cache holds " + std::to_string(k.size(1)) + " slots per page, not page_size=" +
                std::to_string(page_size));
  if (!paged && k.size(0) % page_size)
    value_error("a flat cache of " + std::to_string(k.size(0)) + " slots does not split into pages of " +
                std::to_string(page_size));
  const int64_t slots = paged ? k.size(0) * page_size : k.size(0);
  const int64_t H = k.size(n - 2), es = (int64_t)k.element_size();
  int64_t D = k.size(n - 1);
  c->k = k.data_ptr();
  c->v = v.data_ptr();
  c->k_stride_page = k.stride(0) * es * (paged ? 1 : page_size);
  c->v_stride_page = v.stride(0) * es * (paged ? 1 : page_size);
  c->k_stride_offset = k.stride(n - 3) * es;
  c->v_stride_offset = v.stride(n - 3) * es;
  c->k_stride_head = k.stride(n - 2) * es;
  c->v_stride_head = v.stride(n - 2) * es;
  c->scale_kind = KVSTORE_SCALES_TENSOR;
  c->k_scales = c->v_scales = nullptr;
  c->ks_stride_page = c->ks_stride_offset = c->ks_stride_head = 0;
  c->vs_stride_page = c->vs_stride_offset = c->vs_stride_head = 0;
  if ((s.k_cache == nullptr) != (s.v_cache == nullptr)) value_error("give both scale caches or neither");
  if (type == at::kFloat4_e2m1fn_x2) {
    c->format = KVSTORE_FMT_FP4;
    c->scale_kind = KVSTORE_SCALES_BLOCK;
    D *= 2;
    if (s.k_cache == nullptr) value_error("4-bit caches need k_scale_cache and v_scale_cache");
    if (s.k_scale || s.v_scale) value_error("4-bit caches have block scales, not tensor scales");
    if (D % 32) value_error("a 4-bit head_dim is a multiple of 32, not " + std::to_string(D));
    const int64_t ks = block_scales(*s.k_cache, paged, H, D / 32, page_size, &c->ks_stride_page,
                                    &c->ks_stride_offset, &c->ks_stride_head);
    const int64_t vs = block_scales(*s.v_cache, paged, H, D / 32, page_size, &c->vs_stride_page,
                                    &c->vs_stride_offset, &c->vs_stride_head);
    if (ks != slots || vs != slots) value_error("scale caches must cover the same slots as the caches");
    c->k_scales = s.k_cache->data_ptr();
    c->v_scales = s.v_cache->data_ptr();
  } else if (type == at::kBFloat16 || type == at::kHalf) {
    if (type != src)
      type_error(std::string(c10::toString(type)) + " caches go with rows of that type, not " +
                 c10::toString(src));
    if (s.k_scale || s.v_scale || s.k_cache) value_error("16-bit caches have no scales");
    c->format = type == at::kHalf ? KVSTORE_FMT_FP16 : KVSTORE_FMT_BF16;
  } else if (type == at::kByte || type == at::kFloat8_e4m3fn || type == at::kFloat8_e5m2) {
    c->format = type == at::kFloat8_e5m2 ? KVSTORE_FMT_E5M2 : KVSTORE_FMT_E4M3FN;
    if (s.k_cache != nullptr) {
      if (!reads) value_error("a store into FP8 caches takes inverse scales, not scale caches");
      if (s.k_scale || s.v_scale) value_error("give scale caches or tensor scales, not both");
      const bool per_head = s.k_cache->dim() == (paged ? 3 : 2);
      c->scale_kind = per_head ? KVSTORE_SCALES_TOKEN_HEAD : KVSTORE_SCALES_TOKEN;
      const int64_t ks = fp32_scales(*s.k_cache, paged, per_head, H, page_size, &c->ks_stride_page,
                                     &c->ks_stride_offset, &c->ks_stride_head);
      const int64_t vs = fp32_scales(*s.v_cache, paged, per_head, H, page_size, &c->vs_stride_page,
                                     &c->vs_stride_offset, &c->vs_stride_head);
      if (ks != slots || vs != slots) value_error("scale caches must cover the same slots as the caches");
      c->k_scales = s.k_cache->data_ptr();
      c->v_scales = s.v_cache->data_ptr();
    } else if (reads) {
      c->k_scales = const_cast<float*>(scalar(s.k_scale, "scales"));
      c->v_scales = const_cast<float*>(scalar(s.v_scale, "scales"));
    }
  } else {
    type_error(std::string("a ") + c10::toString(type) +
               " cache is none of the formats: the rows' 16-bit dtype, uint8 or float8_e4m3fn "
               "(e4m3fn codes), float8_e5m2, float4_e2m1fn_x2");
  }
  int64_t limit = slots;
  if (size_limit != Py_None) {
    limit = integer(size_limit, "size_limit");
    if (limit > slots)
      value_error("size_limit (" + std::to_string(limit) + ") exceeds the cache's " +
                  std::to_string(slots) + " slots");
  }
  if (H > INT32_MAX || D > INT32_MAX) value_error("a cache dim is out of range");
  c->num_heads = (int32_t)H;
  c->head_dim = (int32_t)D;
  c->page_size = page_size;
  c->num_slots = limit;
}

// (token, head) byte strides of [T, H, D] or [T, H*D] 16-bit rows.
void row_strides(const at::Tensor& x, int64_t H, int64_t D, int64_t* token, int64_t* head) {
  if (x.dim() == 3) {
    if (x.size(1) != H || x.size(2) != D)
      value_error("rows of " + std::to_string(x.size(1)) + "x" + std::to_string(x.size(2)) +
                  " do not match heads/dim " + std::to_string(H) + "x" + std::to_string(D));
    if (x.stride(2) != 1) value_error("row dim stride must be 1");
    *head = x.stride(1) * 2;
  } else if (x.dim() == 2) {
    if (x.size(1) != H * D)
      value_error("row width " + std::to_string(x.size(1)) + " != " + std::to_string(H * D));
    if (x.stride(1) != 1) value_error("row dim stride must be 1");
    *head = D * 2;
  } else {
    value_error("rows are 2-D [T, H*D] or 3-D [T, H, D], not " + std::to_string(x.dim()) + "-D");
  }
  *token = x.stride(0) * 2;
}

// Runs a library call without the GIL, so that threads can issue calls
// concurrently.
template <typename F>
int without_gil(F&& call) {
  int st;
  Py_BEGIN_ALLOW_THREADS
  st = call();
  Py_END_ALLOW_THREADS
  return st;
}

uint32_t batch_of(int64_t T) {
  if (T > UINT32_MAX) throw Raise{PyExc_OverflowError, "batch does not fit in 32 bits"};
  return (uint32_t)T;
}

void check_slots(const at::Tensor& loc, int64_t T) {
  if (loc.dim() != 1 || loc.size(0) != T) value_error("cache_loc must be [T], one slot for each row");
}

// store_kv_rope_paged(k, v, k_cache, v_cache, cache_loc, positions, cos_sin, q, q_out,
//                     interleaved, page_size, inv_k_scale, inv_v_scale, k_scale_cache,
//                     v_scale_cache, size_limit) -> status
PyObject* rope(PyObject* const* a) {
  const at::Tensor &k = *tensor(a[0], "k"), &v = *tensor(a[1], "v"), &kc = *tensor(a[2], "k_cache"),
                   &vc = *tensor(a[3], "v_cache"), &loc = *tensor(a[4], "cache_loc");
  const Opt pos = tensor(a[5], "positions", true), table = tensor(a[6], "cos_sin", true);
  const Opt q = tensor(a[7], "q", true), q_out = tensor(a[8], "q_out", true);
  const Opt ik = tensor(a[11], "inv_k_scale", true), iv = tensor(a[12], "inv_v_scale", true);
  const Scales scales = {nullptr, nullptr, tensor(a[13], "k_scale_cache", true),
                         tensor(a[14], "v_scale_cache", true)};
  kvstore_rope_rows r = {};
  kvstore_paged_cache c;
  r.src_dtype = src_code(k, "k and v");
  if (v.scalar_type() != k.scalar_type() || (q && q->scalar_type() != k.scalar_type()))
    type_error("q, k and v must share one dtype");
  fill_cache(&c, kc, vc, integer(a[10], "page_size"), a[15], k.scalar_type(), scales, false);
  const bool fp8 = c.format == KVSTORE_FMT_E4M3FN || c.format == KVSTORE_FMT_E5M2;
  if (!fp8 && (ik || iv)) value_error("only FP8 caches take inverse scales");
  const int64_t H = c.num_heads, D = c.head_dim;
  row_strides(k, H, D, &r.k_stride_token, &r.k_stride_head);
  row_strides(v, H, D, &r.v_stride_token, &r.v_stride_head);
  const int64_t T = k.size(0);
  if (v.size(0) != T) value_error("k and v must have the same tokens");
  check_slots(loc, T);
  if (q) {
    const at::Tensor& o = q_out ? *q_out : *q;
    const int64_t Hq = q->dim() == 3 ? q->size(1) : q->dim() == 2 && D > 0 ? q->size(1) / D : 0;
    if (o.scalar_type() != q->scalar_type() || o.sizes() != q->sizes() || q->size(0) != T)
      value_error("q and q_out must be [T, Hq, D] or [T, Hq*D] of one dtype");
    if (Hq > INT32_MAX) value_error("q has too many heads");
    row_strides(*q, Hq, D, &r.q_stride_token, &r.q_stride_head);
    row_strides(o, Hq, D, &r.qo_stride_token, &r.qo_stride_head);
    r.q = q->data_ptr();
    r.q_out = o.data_ptr();
    r.q_heads = (int32_t)Hq;
  } else if (q_out) {
    value_error("q_out without q");
  }
  r.k = k.data_ptr();
  r.v = v.data_ptr();
  if ((pos == nullptr) != (table == nullptr)) value_error("give positions and cos_sin, or neither");
  int pos_dtype = KVSTORE_IDX_I32;
  if (table) {
    if (table->scalar_type() != at::kFloat || table->dim() != 2 || (table->size(1) > 1 && table->stride(1) != 1))
      type_error("cos_sin must be fp32 [positions, rot] with contiguous rows");
    if (pos->dim() != 1 || pos->size(0) != T || (T > 1 && pos->stride(0) != 1))
      value_error("positions must be a contiguous [T]");
    if (table->size(1) > INT32_MAX) value_error("cos_sin is too wide");
    pos_dtype = idx_code(*pos);
  }
  const int loc_dtype = idx_code(loc);
  const int inter = PyObject_IsTrue(a[9]);
  if (inter < 0) throw AlreadySet();
  const float *pik = scalar(ik, "inverse scales"), *piv = scalar(iv, "inverse scales");
  no_grad({&k, &v, &kc, &vc, table, q, q_out});
  Device dev;
  for (Opt t : {&k, &v, &kc, &vc, &loc, pos, table, q, q_out, ik, iv, scales.k_cache, scales.v_cache})
    dev.add(t);
  const uint32_t batch = batch_of(T);
  OnDevice on(dev.index);
  const hipStream_t stream = on.stream();
  return PyLong_FromLong(without_gil([&] {
    return kvstore_rope_paged(
        &r, pos ? pos->data_ptr() : nullptr, pos_dtype,
        table ? static_cast<const float*>(table->data_ptr()) : nullptr,
        table ? table->stride(0) * 4 : 0, table ? table->size(0) : 0,
        table ? (int32_t)table->size(1) : 0, inter, loc.data_ptr(), loc_dtype,
        T ? loc.stride(0) : 1, &c, pik, piv, batch, stream);
  }));
}

// load_kv_paged(k_cache, v_cache, cache_loc, k_out, v_out, page_size, k_scale, v_scale,
//               k_scale_cache, v_scale_cache, size_limit) -> status
PyObject* load(PyObject* const* a) {
  const at::Tensor &kc = *tensor(a[0], "k_cache"), &vc = *tensor(a[1], "v_cache"),
                   &loc = *tensor(a[2], "cache_loc"), &ko = *tensor(a[3], "k_out"),
                   &vo = *tensor(a[4], "v_out");
  const Scales s = {tensor(a[6], "k_scale", true), tensor(a[7], "v_scale", true),
                    tensor(a[8], "k_scale_cache", true), tensor(a[9], "v_scale_cache", true)};
  kvstore_paged_cache c;
  const int dst = src_code(ko, "k_out and v_out");
  if (vo.scalar_type() != ko.scalar_type()) type_error("k_out and v_out must share one dtype");
  fill_cache(&c, kc, vc, integer(a[5], "page_size"), a[10], ko.scalar_type(), s, true);
  int64_t kt, kh, vt, vh;
  row_strides(ko, c.num_heads, c.head_dim, &kt, &kh);
  row_strides(vo, c.num_heads, c.head_dim, &vt, &vh);
  const int64_t T = ko.size(0);
  if (vo.size(0) != T) value_error("k_out and v_out must have the same rows");
  check_slots(loc, T);
  const int loc_dtype = idx_code(loc);
  no_grad({&kc, &vc, &ko, &vo});
  Device dev;
  for (Opt t : {&kc, &vc, &loc, &ko, &vo, s.k_scale, s.v_scale, s.k_cache, s.v_cache}) dev.add(t);
  const uint32_t batch = batch_of(T);
  OnDevice on(dev.index);
  const hipStream_t stream = on.stream();
  return PyLong_FromLong(without_gil([&] {
    return kvstore_load_paged(&c, loc.data_ptr(), loc_dtype, T ? loc.stride(0) : 1, ko.data_ptr(),
                              kt, kh, vo.data_ptr(), vt, vh, dst, batch, stream);
  }));
}

// attention_paged(q, k_cache, v_cache, page_table, seq_lens, cu_q, max_q, max_len, window, sinks,
//                 sm_scale, page_size, k_scale, v_scale, k_scale_cache, v_scale_cache, out,
//                 workspace, only_workspace) -> out, or a status; or the workspace's bytes
PyObject* attention(PyObject* const* a) {
  const at::Tensor &q = *tensor(a[0], "q"), &kc = *tensor(a[1], "k_cache"),
                   &vc = *tensor(a[2], "v_cache"), &table = *tensor(a[3], "page_table"),
                   &lens = *tensor(a[4], "seq_lens");
  const Opt cu = tensor(a[5], "cu_q", true), out = tensor(a[16], "out", true),
            ws = tensor(a[17], "workspace", true);
  const Scales s = {tensor(a[12], "k_scale", true), tensor(a[13], "v_scale", true),
                    tensor(a[14], "k_scale_cache", true), tensor(a[15], "v_scale_cache", true)};
  kvstore_attention_args r = {};
  kvstore_paged_cache c;
  r.src_dtype = src_code(q, "q");
  fill_cache(&c, kc, vc, integer(a[11], "page_size"), Py_None, q.scalar_type(), s, true);
  const int64_t H = c.num_heads, D = c.head_dim;
  if (q.dim() != 3 || q.size(2) != D || H == 0 || q.size(1) % H)
    value_error("q must be [T, Hq, " + std::to_string(D) + "] with Hq a multiple of " + std::to_string(H));
  const int64_t T = q.size(0), Hq = q.size(1);
  if (lens.dim() != 1 || table.dim() != 2 || table.size(0) != lens.size(0))
    value_error("seq_lens must be [B] and page_table [B, pages]");
  const int64_t B = lens.size(0);
  for (Opt t : {&table, &lens, cu})
    if (t && t->scalar_type() != at::kInt) type_error("page_table, seq_lens and cu_q must be int32");
  if ((B > 1 && lens.stride(0) != 1) || (table.size(1) > 1 && table.stride(1) != 1))
    value_error("seq_lens and the rows of page_table must be contiguous");
  if (cu == nullptr) {
    if (T != B)
      value_error("without cu_q every sequence has one token: " + std::to_string(T) + " rows, " +
                  std::to_string(B) + " sequences");
  } else if (cu->dim() != 1 || cu->size(0) != B + 1 || cu->stride(0) != 1) {
    value_error("cu_q must be a contiguous [B + 1]");
  }
  if (out && (out->sizes() != q.sizes() || out->scalar_type() != q.scalar_type()))
    value_error("out must have q's shape and dtype");
  if ((T > 0 && q.stride(2) != 1) || (out && T > 0 && out->stride(2) != 1))
    value_error("q and out must have a dim stride of 1");
  if (Hq > INT32_MAX || table.size(1) > UINT32_MAX) value_error("q or page_table is too wide");
  no_grad({&q, &kc, &vc, s.k_scale, s.v_scale, s.k_cache, s.v_cache, out});
  r.q = q.data_ptr();
  r.q_stride_token = q.stride(0) * 2;
  r.q_stride_head = q.stride(1) * 2;
  r.q_heads = (int32_t)Hq;
  r.cu_q = cu ? static_cast<const int32_t*>(cu->data_ptr()) : nullptr;
  r.tokens = batch_of(T);
  r.seqs = batch_of(B);
  const int64_t max_q = a[6] == Py_None ? 0 : integer(a[6], "max_q");
  r.max_q = (uint32_t)(max_q < T ? max_q : T);
  r.page_table = static_cast<const int32_t*>(table.data_ptr());
  r.table_stride = table.stride(0);
  r.max_pages = (uint32_t)table.size(1);
  r.seq_lens = static_cast<const int32_t*>(lens.data_ptr());
  r.max_len = a[7] == Py_None ? 0 : integer(a[7], "max_len");
  r.window = integer(a[8], "window");
  r.sinks = integer(a[9], "sinks");
  if (a[10] == Py_None) {
    r.sm_scale = D > 0 ? (float)(1.0 / std::sqrt((double)D)) : 1.0f;
  } else {
    const double x = PyFloat_AsDouble(a[10]);
    if (x == -1.0 && PyErr_Occurred()) throw AlreadySet();
    r.sm_scale = (float)x;
  }
  Device dev;
  for (Opt t : {&q, &kc, &vc, &table, &lens, cu, s.k_scale, s.v_scale, s.k_cache, s.v_cache, out, ws})
    dev.add(t);
  r.workspace_bytes = kvstore_attention_workspace(&r, &c);
  if (r.workspace_bytes < 0 || a[18] == Py_True) return PyLong_FromLongLong(r.workspace_bytes);
  OnDevice on(dev.index);
  // Allocations follow the current stream, which is the one that the call runs on.
  at::Tensor made_out, made_ws;
  if (out == nullptr) made_out = at::empty({T, Hq, D}, q.options());
  const at::Tensor& o = out ? *out : made_out;
  if (r.workspace_bytes > 0) {
    if (ws == nullptr) {
      made_ws = at::empty({r.workspace_bytes}, q.options().dtype(at::kByte));
      r.workspace = made_ws.data_ptr();
    } else {
      if (!ws->is_contiguous()) value_error("workspace must be contiguous");
      r.workspace = ws->data_ptr();
      r.workspace_bytes = ws->numel() * (int64_t)ws->element_size();
    }
  }
  r.out = o.data_ptr();
  r.o_stride_token = o.stride(0) * 2;
  r.o_stride_head = o.stride(1) * 2;
  const hipStream_t stream = on.stream();
  const int st = without_gil([&] { return kvstore_attention_paged(&r, &c, stream); });
  if (st != KVSTORE_OK) return PyLong_FromLong(st);
  if (out == nullptr) return THPVariable_Wrap(made_out);
  Py_INCREF(a[16]);
  return a[16];
}

// Runs a function on exactly n arguments; no C++ exception leaves.
template <PyObject* (*kFunction)(PyObject* const*), int kArgs>
PyObject* entry(PyObject*, PyObject* const* a, Py_ssize_t n) {
  if (n != kArgs) {
    PyErr_Format(PyExc_TypeError, "expected %d arguments, got %zd", kArgs, n);
    return nullptr;
  }
  try {
    return kFunction(a);
  } catch (const AlreadySet&) {
  } catch (const Raise& e) {
    PyErr_SetString(e.type, e.text.c_str());
  } catch (const c10::OutOfMemoryError& e) {
    PyErr_SetString(PyExc_MemoryError, e.what_without_backtrace());
  } catch (const std::exception& e) {
    PyErr_SetString(PyExc_RuntimeError, e.what());
  }
  return nullptr;
}

#define FASTCALL(f) reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)(void)>(f))

PyMethodDef methods[] = {
    {"store_kv_rope_paged", FASTCALL((entry<rope, 16>)), METH_FASTCALL, "Returns the status."},
    {"load_kv_paged", FASTCALL((entry<load, 11>)), METH_FASTCALL, "Returns the status."},
    {"attention_paged", FASTCALL((entry<attention, 19>)), METH_FASTCALL,
     "Returns out, or a status."},
    {nullptr, nullptr, 0, nullptr}};

PyModuleDef module = {PyModuleDef_HEAD_INIT, "_kvstore_torch",
                      "Tensor-level calls of libkvstore's paged operators.", -1, methods,
                      nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__kvstore_torch(void) { return PyModule_Create(&module); }
