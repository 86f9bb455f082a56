/*
 * _kvstore_py: the CPython binding of libkvstore (include/kvstore.h,
 * include/kvstore_paged.h).
 *
 * Argument marshalling only: every function takes Python ints (pointers as
 * ints, None for NULL), calls the C function of the same name and returns its
 * status.  Functions use the vectorcall convention (METH_FASTCALL), so a call
 * converts its integers directly with no argument tuple; the GIL is released
 * around each library call, so threads can issue stores concurrently.
 */
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <stdint.h>

#include "kvstore_paged.h"

/* A device or host pointer from a Python int, or NULL from None. */
static int to_ptr(PyObject* o, void** out) {
  if (o == Py_None) {
    *out = NULL;
    return 1;
  }
  void* p = PyLong_AsVoidPtr(o);
  if (p == NULL && PyErr_Occurred()) return 0;
  *out = p;
  return 1;
}

static int to_i64(PyObject* o, int64_t* out) {
  long long v = PyLong_AsLongLong(o);
  if (v == -1 && PyErr_Occurred()) return 0;
  *out = (int64_t)v;
  return 1;
}

static int to_int(PyObject* o, int* out) {
  long v = PyLong_AsLong(o);
  if (v == -1 && PyErr_Occurred()) return 0;
  if (v < INT32_MIN || v > INT32_MAX) {
    PyErr_SetString(PyExc_OverflowError, "value does not fit in a C int");
    return 0;
  }
  *out = (int)v;
  return 1;
}

static int to_u32(PyObject* o, uint32_t* out) {
  unsigned long long v = PyLong_AsUnsignedLongLong(o);
  if (v == (unsigned long long)-1 && PyErr_Occurred()) return 0;
  if (v > UINT32_MAX) {
    PyErr_SetString(PyExc_OverflowError, "batch does not fit in 32 bits");
    return 0;
  }
  *out = (uint32_t)v;
  return 1;
}

/* The stream argument: optional, None or 0 for the null stream. */
static int stream_arg(PyObject* const* args, Py_ssize_t nargs, Py_ssize_t i, hipStream_t* s) {
  void* p = NULL;
  if (nargs > i && !to_ptr(args[i], &p)) return 0;
  *s = (hipStream_t)p;
  return 1;
}

static int check_nargs(const char* name, Py_ssize_t nargs, Py_ssize_t need) {
  if (nargs == need || nargs == need + 1) return 1;
  PyErr_Format(PyExc_TypeError, "%s takes %zd arguments (+ optional stream), got %zd", name,
               need, nargs);
  return 0;
}

static PyObject* py_kvstore_copy(PyObject* self, PyObject* const* a, Py_ssize_t n) {
  (void)self;
  void *k, *v, *kc, *vc, *ix;
  int idx_dtype;
  int64_t idx_stride, row, ks, vs, cs, limit;
  uint32_t batch;
  hipStream_t s;
  if (!check_nargs("kvstore_copy", n, 13) || !to_ptr(a[0], &k) || !to_ptr(a[1], &v) ||
      !to_ptr(a[2], &kc) || !to_ptr(a[3], &vc) || !to_ptr(a[4], &ix) ||
      !to_int(a[5], &idx_dtype) || !to_i64(a[6], &idx_stride) || !to_i64(a[7], &row) ||
      !to_i64(a[8], &ks) || !to_i64(a[9], &vs) || !to_i64(a[10], &cs) ||
      !to_u32(a[11], &batch) || !to_i64(a[12], &limit) || !stream_arg(a, n, 13, &s))
    return NULL;
  int st;
  Py_BEGIN_ALLOW_THREADS
  st = kvstore_copy(k, v, kc, vc, ix, idx_dtype, idx_stride, row, ks, vs, cs, batch, limit, s);
  Py_END_ALLOW_THREADS
  return PyLong_FromLong(st);
}

/* Arguments shared by the three FP8 stores, up to and including page_size. */
typedef struct {
  void *k, *v, *kc, *vc, *ix;
  int idx_dtype, src_dtype, heads, dim;
  int64_t idx_stride, kt, kh, vt, vh, kcp, kco, kch, vcp, vco, vch, limit, page;
  uint32_t batch;
} Fp8Args;

/* a[0..19] plus batch, size_limit and page_size at b, b + 1, b + 2. */
static int fp8_args(PyObject* const* a, Py_ssize_t b, Fp8Args* f) {
  return to_ptr(a[0], &f->k) && to_ptr(a[1], &f->v) && to_ptr(a[2], &f->kc) &&
         to_ptr(a[3], &f->vc) && to_ptr(a[4], &f->ix) && to_int(a[5], &f->idx_dtype) &&
         to_i64(a[6], &f->idx_stride) && to_int(a[7], &f->src_dtype) &&
         to_int(a[8], &f->heads) && to_int(a[9], &f->dim) && to_i64(a[10], &f->kt) &&
         to_i64(a[11], &f->kh) && to_i64(a[12], &f->vt) && to_i64(a[13], &f->vh) &&
         to_i64(a[14], &f->kcp) && to_i64(a[15], &f->kco) && to_i64(a[16], &f->kch) &&
         to_i64(a[17], &f->vcp) && to_i64(a[18], &f->vco) && to_i64(a[19], &f->vch) &&
         to_u32(a[b], &f->batch) && to_i64(a[b + 1], &f->limit) && to_i64(a[b + 2], &f->page);
}

static PyObject* fp8_static(PyObject* const* a, Py_ssize_t n, int e5m2) {
  const char* name = e5m2 ? "kvstore_fp8_paged_e5m2" : "kvstore_fp8_paged";
  Fp8Args f;
  void *ik, *iv;
  hipStream_t s;
  if (!check_nargs(name, n, 25) || !fp8_args(a, 20, &f) || !to_ptr(a[23], &ik) ||
      !to_ptr(a[24], &iv) || !stream_arg(a, n, 25, &s))
    return NULL;
  int st;
  Py_BEGIN_ALLOW_THREADS
  st = (e5m2 ? kvstore_fp8_paged_e5m2 : kvstore_fp8_paged)(
      f.k, f.v, f.kc, f.vc, f.ix, f.idx_dtype, f.idx_stride, f.src_dtype, f.heads, f.dim, f.kt,
      f.kh, f.vt, f.vh, f.kcp, f.kco, f.kch, f.vcp, f.vco, f.vch, f.batch, f.limit, f.page,
      (const float*)ik, (const float*)iv, s);
  Py_END_ALLOW_THREADS
  return PyLong_FromLong(st);
}

static PyObject* py_kvstore_fp8_paged(PyObject* self, PyObject* const* a, Py_ssize_t n) {
  (void)self;
  return fp8_static(a, n, 0);
}

static PyObject* py_kvstore_fp8_paged_e5m2(PyObject* self, PyObject* const* a, Py_ssize_t n) {
  (void)self;
  return fp8_static(a, n, 1);
}

static PyObject* py_kvstore_fp8_paged_dynamic(PyObject* self, PyObject* const* a, Py_ssize_t n) {
  (void)self;
  Fp8Args f;
  void *ksc, *vsc;
  int gran;
  int64_t ksp, kso, ksh, vsp, vso, vsh;
  hipStream_t s;
  if (!check_nargs("kvstore_fp8_paged_dynamic", n, 32) || !fp8_args(a, 29, &f) ||
      !to_ptr(a[20], &ksc) || !to_ptr(a[21], &vsc) || !to_int(a[22], &gran) ||
      !to_i64(a[23], &ksp) || !to_i64(a[24], &kso) || !to_i64(a[25], &ksh) ||
      !to_i64(a[26], &vsp) || !to_i64(a[27], &vso) || !to_i64(a[28], &vsh) ||
      !stream_arg(a, n, 32, &s))
    return NULL;
  int st;
  Py_BEGIN_ALLOW_THREADS
  st = kvstore_fp8_paged_dynamic(f.k, f.v, f.kc, f.vc, f.ix, f.idx_dtype, f.idx_stride,
                                 f.src_dtype, f.heads, f.dim, f.kt, f.kh, f.vt, f.vh, f.kcp,
                                 f.kco, f.kch, f.vcp, f.vco, f.vch, (float*)ksc, (float*)vsc,
                                 gran, ksp, kso, ksh, vsp, vso, vsh, f.batch, f.limit, f.page, s);
  Py_END_ALLOW_THREADS
  return PyLong_FromLong(st);
}

static PyObject* py_kvstore_check_error(PyObject* self, PyObject* const* a, Py_ssize_t n) {
  (void)self;
  hipStream_t s;
  if (n > 1) {
    PyErr_SetString(PyExc_TypeError, "kvstore_check_error takes an optional stream");
    return NULL;
  }
  if (!stream_arg(a, n, 0, &s)) return NULL;
  int64_t first_bad = 0;
  uint64_t count = 0;
  int st;
  Py_BEGIN_ALLOW_THREADS
  st = kvstore_check_error(s, &first_bad, &count);
  Py_END_ALLOW_THREADS
  return Py_BuildValue("(iLK)", st, (long long)first_bad, (unsigned long long)count);
}

static PyObject* py_kvstore_take_error(PyObject* self, PyObject* const* a, Py_ssize_t n) {
  (void)self;
  void* out;
  hipStream_t s;
  if (!check_nargs("kvstore_take_error", n, 1) || !to_ptr(a[0], &out) ||
      !stream_arg(a, n, 1, &s))
    return NULL;
  int st;
  Py_BEGIN_ALLOW_THREADS
  st = kvstore_take_error((int64_t*)out, s);
  Py_END_ALLOW_THREADS
  return PyLong_FromLong(st);
}

/* A struct's members from a tuple of exactly n items. */
static int check_struct(PyObject* o, Py_ssize_t n, const char* name) {
  if (PyTuple_Check(o) && PyTuple_GET_SIZE(o) == n) return 1;
  PyErr_Format(PyExc_TypeError, "%s is a tuple of %zd members", name, n);
  return 0;
}

/* kvstore_paged_cache: its 22 members in the header's order. */
static int to_cache(PyObject* o, kvstore_paged_cache* c) {
  if (!check_struct(o, 22, "kvstore_paged_cache")) return 0;
  PyObject** a = &PyTuple_GET_ITEM(o, 0);
  int format, kind, heads, dim;
  int64_t* const strides[6] = {&c->k_stride_page, &c->k_stride_offset, &c->k_stride_head,
                               &c->v_stride_page, &c->v_stride_offset, &c->v_stride_head};
  int64_t* const scale_strides[6] = {&c->ks_stride_page, &c->ks_stride_offset,
                                     &c->ks_stride_head, &c->vs_stride_page,
                                     &c->vs_stride_offset, &c->vs_stride_head};
  if (!to_ptr(a[0], &c->k) || !to_ptr(a[1], &c->v) || !to_int(a[2], &format) ||
      !to_int(a[3], &kind) || !to_int(a[4], &heads) || !to_int(a[5], &dim) ||
      !to_i64(a[6], &c->page_size) || !to_i64(a[7], &c->num_slots) ||
      !to_ptr(a[14], &c->k_scales) || !to_ptr(a[15], &c->v_scales))
    return 0;
  for (int i = 0; i < 6; ++i)
    if (!to_i64(a[8 + i], strides[i]) || !to_i64(a[16 + i], scale_strides[i])) return 0;
  c->format = format;
  c->scale_kind = kind;
  c->num_heads = heads;
  c->head_dim = dim;
  return 1;
}

static PyObject* py_kvstore_rope_paged(PyObject* self, PyObject* const* a, Py_ssize_t n) {
  (void)self;
  kvstore_rope_rows r;
  kvstore_paged_cache c;
  void *q, *k, *v, *pos, *table, *ix, *ik, *iv;
  int src, q_heads, pos_dtype, rot, inter, idx_dtype;
  int64_t table_stride, num_pos, idx_stride;
  uint32_t batch;
  hipStream_t s;
  if (!check_nargs("kvstore_rope_paged", n, 15) || !check_struct(a[0], 14, "kvstore_rope_rows"))
    return NULL;
  PyObject** m = &PyTuple_GET_ITEM(a[0], 0);
  int64_t* const strides[8] = {&r.q_stride_token, &r.q_stride_head, &r.qo_stride_token,
                               &r.qo_stride_head, &r.k_stride_token, &r.k_stride_head,
                               &r.v_stride_token, &r.v_stride_head};
  for (int i = 0; i < 8; ++i)
    if (!to_i64(m[6 + i], strides[i])) return NULL;
  if (!to_ptr(m[0], &q) || !to_ptr(m[1], &r.q_out) || !to_ptr(m[2], &k) || !to_ptr(m[3], &v) ||
      !to_int(m[4], &src) || !to_int(m[5], &q_heads) || !to_ptr(a[1], &pos) ||
      !to_int(a[2], &pos_dtype) || !to_ptr(a[3], &table) || !to_i64(a[4], &table_stride) ||
      !to_i64(a[5], &num_pos) || !to_int(a[6], &rot) || !to_int(a[7], &inter) ||
      !to_ptr(a[8], &ix) || !to_int(a[9], &idx_dtype) || !to_i64(a[10], &idx_stride) ||
      !to_cache(a[11], &c) || !to_ptr(a[12], &ik) || !to_ptr(a[13], &iv) ||
      !to_u32(a[14], &batch) || !stream_arg(a, n, 15, &s))
    return NULL;
  r.q = q;
  r.k = k;
  r.v = v;
  r.src_dtype = src;
  r.q_heads = q_heads;
  int st;
  Py_BEGIN_ALLOW_THREADS
  st = kvstore_rope_paged(&r, pos, pos_dtype, (const float*)table, table_stride, num_pos, rot,
                          inter, ix, idx_dtype, idx_stride, &c, (const float*)ik,
                          (const float*)iv, batch, s);
  Py_END_ALLOW_THREADS
  return PyLong_FromLong(st);
}

static PyObject* py_kvstore_load_paged(PyObject* self, PyObject* const* a, Py_ssize_t n) {
  (void)self;
  kvstore_paged_cache c;
  void *ix, *ko, *vo;
  int idx_dtype, dst;
  int64_t idx_stride, kt, kh, vt, vh;
  uint32_t batch;
  hipStream_t s;
  if (!check_nargs("kvstore_load_paged", n, 12) || !to_cache(a[0], &c) || !to_ptr(a[1], &ix) ||
      !to_int(a[2], &idx_dtype) || !to_i64(a[3], &idx_stride) || !to_ptr(a[4], &ko) ||
      !to_i64(a[5], &kt) || !to_i64(a[6], &kh) || !to_ptr(a[7], &vo) || !to_i64(a[8], &vt) ||
      !to_i64(a[9], &vh) || !to_int(a[10], &dst) || !to_u32(a[11], &batch) ||
      !stream_arg(a, n, 12, &s))
    return NULL;
  int st;
  Py_BEGIN_ALLOW_THREADS
  st = kvstore_load_paged(&c, ix, idx_dtype, idx_stride, ko, kt, kh, vo, vt, vh, dst, batch, s);
  Py_END_ALLOW_THREADS
  return PyLong_FromLong(st);
}

/* kvstore_attention_args: its 22 members in the header's order. */
static int to_attention(PyObject* o, kvstore_attention_args* r) {
  if (!check_struct(o, 22, "kvstore_attention_args")) return 0;
  PyObject** a = &PyTuple_GET_ITEM(o, 0);
  void *q, *cu, *table, *lens;
  int src, heads;
  if (!to_ptr(a[0], &q) || !to_ptr(a[1], &r->out) || !to_i64(a[2], &r->q_stride_token) ||
      !to_i64(a[3], &r->q_stride_head) || !to_i64(a[4], &r->o_stride_token) ||
      !to_i64(a[5], &r->o_stride_head) || !to_int(a[6], &src) || !to_int(a[7], &heads) ||
      !to_ptr(a[8], &cu) || !to_u32(a[9], &r->tokens) || !to_u32(a[10], &r->seqs) ||
      !to_u32(a[11], &r->max_q) || !to_ptr(a[12], &table) || !to_i64(a[13], &r->table_stride) ||
      !to_u32(a[14], &r->max_pages) || !to_ptr(a[15], &lens) || !to_i64(a[16], &r->max_len) ||
      !to_i64(a[17], &r->window) || !to_i64(a[18], &r->sinks) || !to_ptr(a[20], &r->workspace) ||
      !to_i64(a[21], &r->workspace_bytes))
    return 0;
  const double scale = PyFloat_AsDouble(a[19]);
  if (scale == -1.0 && PyErr_Occurred()) return 0;
  r->q = q;
  r->src_dtype = src;
  r->q_heads = heads;
  r->cu_q = (const int32_t*)cu;
  r->page_table = (const int32_t*)table;
  r->seq_lens = (const int32_t*)lens;
  r->sm_scale = (float)scale;
  return 1;
}

static PyObject* py_kvstore_attention_paged(PyObject* self, PyObject* const* a, Py_ssize_t n) {
  (void)self;
  kvstore_attention_args r;
  kvstore_paged_cache c;
  hipStream_t s;
  if (!check_nargs("kvstore_attention_paged", n, 2) || !to_attention(a[0], &r) ||
      !to_cache(a[1], &c) || !stream_arg(a, n, 2, &s))
    return NULL;
  int st;
  Py_BEGIN_ALLOW_THREADS
  st = kvstore_attention_paged(&r, &c, s);
  Py_END_ALLOW_THREADS
  return PyLong_FromLong(st);
}

static PyObject* py_kvstore_attention_workspace(PyObject* self, PyObject* const* a, Py_ssize_t n) {
  (void)self;
  kvstore_attention_args r;
  kvstore_paged_cache c;
  if (n != 2) {
    PyErr_SetString(PyExc_TypeError, "kvstore_attention_workspace takes two structs");
    return NULL;
  }
  if (!to_attention(a[0], &r) || !to_cache(a[1], &c)) return NULL;
  return PyLong_FromLongLong((long long)kvstore_attention_workspace(&r, &c));
}

static PyObject* py_kvstore_strerror(PyObject* self, PyObject* const* a, Py_ssize_t n) {
  (void)self;
  int status;
  if (n != 1) {
    PyErr_SetString(PyExc_TypeError, "kvstore_strerror takes one status");
    return NULL;
  }
  if (!to_int(a[0], &status)) return NULL;
  return PyUnicode_FromString(kvstore_strerror(status));
}

#define FASTCALL(f) ((PyCFunction)(void (*)(void))(f))

static PyMethodDef methods[] = {
    {"kvstore_copy", FASTCALL(py_kvstore_copy), METH_FASTCALL, "See include/kvstore.h."},
    {"kvstore_fp8_paged", FASTCALL(py_kvstore_fp8_paged), METH_FASTCALL,
     "See include/kvstore.h."},
    {"kvstore_fp8_paged_e5m2", FASTCALL(py_kvstore_fp8_paged_e5m2), METH_FASTCALL,
     "See include/kvstore.h."},
    {"kvstore_fp8_paged_dynamic", FASTCALL(py_kvstore_fp8_paged_dynamic), METH_FASTCALL,
     "See include/kvstore.h."},
    {"kvstore_check_error", FASTCALL(py_kvstore_check_error), METH_FASTCALL,
     "Returns (status, first_bad_token, bad_count)."},
    {"kvstore_take_error", FASTCALL(py_kvstore_take_error), METH_FASTCALL,
     "See include/kvstore.h."},
    {"kvstore_rope_paged", FASTCALL(py_kvstore_rope_paged), METH_FASTCALL,
     "See include/kvstore_paged.h; structs as tuples of their members."},
    {"kvstore_load_paged", FASTCALL(py_kvstore_load_paged), METH_FASTCALL,
     "See include/kvstore_paged.h; structs as tuples of their members."},
    {"kvstore_attention_paged", FASTCALL(py_kvstore_attention_paged), METH_FASTCALL,
     "See include/kvstore_paged.h; structs as tuples of their members."},
    {"kvstore_attention_workspace", FASTCALL(py_kvstore_attention_workspace), METH_FASTCALL,
     "Bytes of workspace, or a negative status."},
    {"kvstore_strerror", FASTCALL(py_kvstore_strerror), METH_FASTCALL, "Status text."},
    {NULL, NULL, 0, NULL}};

static struct PyModuleDef module = {PyModuleDef_HEAD_INIT, "_kvstore_py",
                                    "CPython binding of libkvstore.", -1, methods,
                                    NULL, NULL, NULL, NULL};

PyMODINIT_FUNC PyInit__kvstore_py(void) { return PyModule_Create(&module); }
