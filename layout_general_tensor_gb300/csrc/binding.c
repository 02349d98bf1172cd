/*
 * The calls from Python of the serving operators (the functions of attn_rope.h,
 * attn_prompt.h and attn_cache.h on torch tensors) and of those over groups of
 * rows (row_groups.h, gemm_grouped.h, adapters.h): the tensors' checks and
 * the marshalling, in C, because a call for one token lasts a few
 * microseconds and most of it is the host's (norm and rotation of 64 tokens:
 * 7.4 us a call with the checks in Python, of which the launch is 2.4).
 *
 * Each function returns the library's status, or -1 where a tensor is not what
 * the operator takes; the caller, in Python, then says what is wrong with it.
 * (attend: -2 where everything is, but the workspace is for fewer sequences.)
 * The library's functions come as addresses (setup), so nothing is linked.
 */
#define PY_SSIZE_T_CLEAN
#include <Python.h>
#include <stdint.h>

#include "adapters.h"
#include "attn_cache.h"
#include "attn_prompt.h"
#include "attn_rope.h"
#include "gemm_grouped.h"
#include "row_groups.h"

static PyObject *n_dtype, *n_shape, *n_stride, *n_data_ptr, *n_is_contiguous, *n_get_device;
static PyObject *current_device, *raw_stream, *t_int32, *t_float16, *t_bfloat16, *t_float32;
static __typeof__(&attn_rope_run) rope_run;
static __typeof__(&attn_prompt_run) prompt_run;
static __typeof__(&attn_cache_write) cache_write;
static __typeof__(&attn_cache_read) cache_read;
static __typeof__(&attn_cache_attend) cache_attend;
static __typeof__(&gemm_row_groups) group_rows;
static __typeof__(&gemm_grouped_run) grouped_run;
static __typeof__(&gemm_adapters_run) adapters_run;

typedef struct {
  void* ptr;
  int64_t dim[3], stride[3];
  int contiguous;
} view;

static int is_true(PyObject* v) { /* takes the reference */
  const int r = v == Py_True;
  Py_XDECREF(v);
  return r;
}

static int numbers(PyObject* v, int64_t* to, int n) { /* takes the reference; a tuple of n whole numbers */
  int ok = v && PyTuple_Check(v) && PyTuple_GET_SIZE(v) == n;
  for (int i = 0; ok && i < n; ++i) {
    to[i] = PyLong_AsLongLong(PyTuple_GET_ITEM(v, i));
    ok = !(to[i] == -1 && PyErr_Occurred());
  }
  Py_XDECREF(v);
  return ok;
}

/* A CUDA tensor of `dims` dimensions and type `dtype`, on the device of the
 * call's others (*device; -1: the first of them): its place and shape. */
static int look(PyObject* t, PyObject* dtype, int dims, view* x, int64_t* device) {
  PyObject* d;
  int64_t on;
  int ok;
  d = PyObject_CallMethodNoArgs(t, n_get_device); /* (-1: not on a GPU) */
  on = d ? PyLong_AsLongLong(d) : -1;
  Py_XDECREF(d);
  if (on < 0 || (*device >= 0 && on != *device)) return 0;
  *device = on;
  d = PyObject_GetAttr(t, n_dtype);
  ok = d == dtype;
  Py_XDECREF(d);
  if (!ok || !numbers(PyObject_GetAttr(t, n_shape), x->dim, dims)) return 0;
  x->contiguous = is_true(PyObject_CallMethodNoArgs(t, n_is_contiguous));
  if (!x->contiguous && !numbers(PyObject_CallMethodNoArgs(t, n_stride), x->stride, dims)) return 0;
  d = PyObject_CallMethodNoArgs(t, n_data_ptr);
  if (!d) return 0;
  x->ptr = PyLong_AsVoidPtr(d);
  Py_DECREF(d);
  return !PyErr_Occurred();
}

/* [rows][heads][dim] with contiguous heads; its row stride in stride[0]. */
static int look_rows(PyObject* t, PyObject* dtype, int64_t rows, int64_t heads, int64_t dim, view* x, int64_t* device) {
  if (!look(t, dtype, 3, x, device) || x->dim[1] != heads || x->dim[2] != dim || (rows >= 0 && x->dim[0] != rows)) return 0;
  if (x->contiguous) {
    x->stride[0] = heads * dim;
    return 1;
  }
  return x->stride[2] == 1 && (x->stride[1] == dim || heads == 1) && x->stride[0] >= heads * dim;
}

/* A contiguous vector of `count` values (any number where count < 0). */
static int look_vector(PyObject* t, PyObject* dtype, int64_t count, view* x, int64_t* device) {
  return look(t, dtype, 1, x, device) && x->contiguous && (count < 0 || x->dim[0] == count);
}

/* [rows][cols] (rows < 0: any number of them); its pitch in stride[0], 0 where
 * it is the dense one or there is but one row. */
static int look_matrix(PyObject* t, PyObject* dtype, int64_t rows, int64_t cols, view* x, int64_t* device) {
  if (!look(t, dtype, 2, x, device) || x->dim[1] != cols || (rows >= 0 && x->dim[0] != rows)) return 0;
  if (x->contiguous || x->dim[0] <= 1) {
    if (!x->contiguous && x->stride[1] != 1) return 0;
    x->stride[0] = 0;
    return 1;
  }
  return x->stride[1] == 1 && x->stride[0] >= cols;
}

/* [count][rows][cols]: its matrices' distance in stride[0], their pitch in
 * stride[1], 0 as above. */
static int look_matrices(PyObject* t, PyObject* dtype, int64_t count, int64_t rows, int64_t cols, view* x, int64_t* device) {
  if (!look(t, dtype, 3, x, device) || x->dim[0] != count || x->dim[1] != rows || x->dim[2] != cols) return 0;
  if (x->contiguous) {
    x->stride[0] = x->stride[1] = 0;
    return 1;
  }
  if (x->stride[2] != 1 && cols > 1) return 0;
  if (rows == 1)
    x->stride[1] = 0;
  else if (x->stride[1] < cols)
    return 0;
  if (count == 1)
    x->stride[0] = 0;
  else if (x->stride[0] < (rows - 1) * x->stride[1] + cols)
    return 0;
  return 1;
}

/* The stream given, or the current one of the tensors' device, which has to be
 * the current device: the library launches there.  1, -1 where it is another,
 * or 0 with an exception set. */
static int look_stream(PyObject* stream, int64_t on, void** to) {
  PyObject *device = PyObject_CallNoArgs(current_device), *s;
  int64_t now;
  if (!device) return 0;
  now = PyLong_AsLongLong(device);
  if (now != on) {
    Py_DECREF(device);
    return now == -1 && PyErr_Occurred() ? 0 : -1;
  }
  if (stream != Py_None) {
    Py_DECREF(device);
    *to = PyLong_AsVoidPtr(stream);
    return !PyErr_Occurred();
  }
  s = PyObject_CallOneArg(raw_stream, device);
  Py_DECREF(device);
  if (!s) return 0;
  *to = PyLong_AsVoidPtr(s);
  Py_DECREF(s);
  return !PyErr_Occurred();
}

static PyObject* status(int s) { return PyLong_FromLong(s); }
static PyObject* refused(void) {
  PyErr_Clear(); /* (something that is no tensor at all: said in Python, too) */
  return status(-1);
}
static int64_t whole(PyObject* handle, int i) { return PyLong_AsLongLong(PyTuple_GET_ITEM(handle, i)); }
static void* address(PyObject* handle, int i) { return PyLong_AsVoidPtr(PyTuple_GET_ITEM(handle, i)); }

#define STREAM(arg)                                              \
  do {                                                           \
    const int found = look_stream(arg, device, &stream);         \
    if (found < 0) return refused();                             \
    if (found == 0) return NULL;                                 \
  } while (0)

#define TAKES(count)                                             \
  do {                                                           \
    if (nargs != (count) || !PyTuple_Check(args[0])) {           \
      PyErr_SetString(PyExc_TypeError, "wrong arguments");       \
      return NULL;                                               \
    }                                                            \
  } while (0)

/* (plan, dtype, q_heads, k_heads, head_dim), q, k, positions, q_out, k_out, q_weight, k_weight, stream */
static PyObject* py_rope(PyObject* self, PyObject* const* args, Py_ssize_t nargs) {
  view q, k, pos, qo, ko, wq = {0}, wk = {0};
  void* stream;
  int64_t device = -1;
  TAKES(9);
  PyObject *h = args[0], *dtype = PyTuple_GET_ITEM(h, 1);
  const int64_t hq = whole(h, 2), hk = whole(h, 3), d = whole(h, 4);
  if (!look_rows(args[1], dtype, -1, hq, d, &q, &device) || !look_rows(args[2], dtype, q.dim[0], hk, d, &k, &device) ||
      !look_vector(args[3], t_int32, q.dim[0], &pos, &device) ||
      !look_rows(args[4], dtype, q.dim[0], hq, d, &qo, &device) ||
      !look_rows(args[5], dtype, q.dim[0], hk, d, &ko, &device) ||
      (args[6] != Py_None && !look_vector(args[6], dtype, d, &wq, &device)) ||
      (args[7] != Py_None && !look_vector(args[7], dtype, d, &wk, &device)))
    return refused();
  STREAM(args[8]);
  return status(rope_run(address(h, 0), q.ptr, q.stride[0], k.ptr, k.stride[0], wq.ptr, wk.ptr, pos.ptr, q.dim[0], qo.ptr,
                         qo.stride[0], ko.ptr, ko.stride[0], stream));
}

/* (plan, dtype, q_heads, k_heads, head_dim), q, k, v, cu_q, cu_k, out, stream */
static PyObject* py_prompt(PyObject* self, PyObject* const* args, Py_ssize_t nargs) {
  view q, k, v, cq, ck, out;
  void* stream;
  int64_t device = -1;
  TAKES(8);
  PyObject *h = args[0], *dtype = PyTuple_GET_ITEM(h, 1);
  const int64_t hq = whole(h, 2), hk = whole(h, 3), d = whole(h, 4);
  if (!look_rows(args[1], dtype, -1, hq, d, &q, &device) || !look_rows(args[2], dtype, -1, hk, d, &k, &device) ||
      !look_rows(args[3], dtype, k.dim[0], hk, d, &v, &device) || !look_vector(args[4], t_int32, -1, &cq, &device) ||
      cq.dim[0] < 1 || cq.dim[0] > INT32_MAX || !look_vector(args[5], t_int32, cq.dim[0], &ck, &device) ||
      !look_rows(args[6], dtype, q.dim[0], hq, d, &out, &device))
    return refused();
  STREAM(args[7]);
  return status(prompt_run(address(h, 0), q.ptr, q.stride[0], k.ptr, k.stride[0], v.ptr, v.stride[0], cq.ptr, ck.ptr,
                           (int32_t)(cq.dim[0] - 1), q.dim[0], k.dim[0], out.ptr, out.stride[0], stream));
}

/* (cache, k_heads, head_dim, device), k, v, slots, stream */
static PyObject* cache_call(PyObject* const* args, Py_ssize_t nargs, int write) {
  view k, v, slots;
  void* stream;
  int64_t device = -1;
  TAKES(5);
  PyObject* h = args[0];
  PyObject* dtype = PyObject_GetAttr(args[1], n_dtype);
  const int64_t hk = whole(h, 1), d = whole(h, 2);
  device = whole(h, 3);
  const int ok = (dtype == t_float16 || dtype == t_bfloat16) && look_rows(args[1], dtype, -1, hk, d, &k, &device) &&
                 look_rows(args[2], dtype, k.dim[0], hk, d, &v, &device) &&
                 look_vector(args[3], t_int32, k.dim[0], &slots, &device);
  const int32_t code = dtype == t_bfloat16 ? GEMM_BF16 : GEMM_F16;
  Py_XDECREF(dtype);
  if (!ok) return refused();
  STREAM(args[4]);
  if (write)
    return status(cache_write(address(h, 0), k.ptr, k.stride[0], v.ptr, v.stride[0], slots.ptr, k.dim[0], code, stream));
  return status(cache_read(address(h, 0), slots.ptr, k.dim[0], k.ptr, k.stride[0], v.ptr, v.stride[0], code, stream));
}
static PyObject* py_cache_write(PyObject* self, PyObject* const* args, Py_ssize_t nargs) { return cache_call(args, nargs, 1); }
static PyObject* py_cache_read(PyObject* self, PyObject* const* args, Py_ssize_t nargs) { return cache_call(args, nargs, 0); }

/* (dtype, q_heads, k_heads, head_dim, page_size, type code, scale, workspace, its bytes, its sequences, its device),
 * the cache's handle, q, page_table, lengths, out, stream */
static PyObject* py_attend(PyObject* self, PyObject* const* args, Py_ssize_t nargs) {
  view q, table, lengths, out;
  void* stream;
  int64_t device = -1;
  TAKES(7);
  PyObject *h = args[0], *dtype = PyTuple_GET_ITEM(h, 0);
  if (!PyTuple_Check(args[1])) {
    PyErr_SetString(PyExc_TypeError, "wrong arguments");
    return NULL;
  }
  const attn_cache_t* cache = address(args[1], 0);
  device = whole(h, 10);
  const int64_t hq = whole(h, 1), d = whole(h, 3);
  if (!cache || cache->k_heads != whole(h, 2) || cache->head_dim != d || cache->page_size != whole(h, 4) ||
      whole(args[1], 3) != device || !look_rows(args[2], dtype, -1, hq, d, &q, &device) ||
      !look(args[3], t_int32, 2, &table, &device) || table.dim[0] != q.dim[0] || table.dim[1] > INT32_MAX ||
      !look_vector(args[4], t_int32, q.dim[0], &lengths, &device) ||
      !look_rows(args[5], dtype, q.dim[0], hq, d, &out, &device))
    return refused();
  if (table.contiguous) {
    table.stride[0] = table.dim[1];
  } else if ((table.dim[1] > 1 && table.stride[1] != 1) || table.stride[0] < table.dim[1]) {
    return refused();
  }
  STREAM(args[6]);
  if (q.dim[0] > whole(h, 9)) return status(-2);
  return status(cache_attend(cache, q.ptr, q.stride[0], (int32_t)hq, table.ptr, table.stride[0], (int32_t)table.dim[1],
                             lengths.ptr, (int32_t)q.dim[0], (float)PyFloat_AsDouble(PyTuple_GET_ITEM(h, 6)),
                             (int32_t)whole(h, 5), out.ptr, out.stride[0], address(h, 7), (size_t)whole(h, 8), stream));
}

/* ids, offsets, order, places (or None), stream */
static PyObject* py_row_groups(PyObject* self, PyObject* const* args, Py_ssize_t nargs) {
  view ids, offsets, order, places = {0};
  void* stream;
  int64_t device = -1;
  if (nargs != 5) {
    PyErr_SetString(PyExc_TypeError, "wrong arguments");
    return NULL;
  }
  if (!look_vector(args[0], t_int32, -1, &ids, &device) || !look_vector(args[1], t_int32, -1, &offsets, &device) ||
      offsets.dim[0] < 2 || offsets.dim[0] > INT32_MAX || !look_vector(args[2], t_int32, ids.dim[0], &order, &device) ||
      (args[3] != Py_None && !look_vector(args[3], t_int32, ids.dim[0], &places, &device)))
    return refused();
  STREAM(args[4]);
  return status(group_rows(ids.ptr, ids.dim[0], (int32_t)(offsets.dim[0] - 1), offsets.ptr, order.ptr, places.ptr, stream));
}

/* (plan, dtype, groups, M, N, K, whether B's K is contiguous), A, B, offsets, C, stream; M > 0: groups along K */
static PyObject* py_grouped(PyObject* self, PyObject* const* args, Py_ssize_t nargs) {
  view A, B, offsets, C;
  void* stream;
  int64_t device = -1;
  TAKES(6);
  PyObject *h = args[0], *dtype = PyTuple_GET_ITEM(h, 1);
  const int64_t groups = whole(h, 2), m = whole(h, 3), n = whole(h, 4), k = whole(h, 5), k_contig = whole(h, 6);
  int ok;
  if (m > 0)
    ok = look_matrix(args[1], dtype, -1, m, &A, &device) && look_matrix(args[2], dtype, A.dim[0], n, &B, &device) &&
         look_matrices(args[4], dtype, groups, m, n, &C, &device);
  else
    ok = look_matrix(args[1], dtype, -1, k, &A, &device) &&
         look_matrices(args[2], dtype, groups, k_contig ? n : k, k_contig ? k : n, &B, &device) &&
         look_matrix(args[4], dtype, A.dim[0], n, &C, &device);
  if (!ok || !look_vector(args[3], t_int32, groups + 1, &offsets, &device)) return refused();
  STREAM(args[5]);
  const int64_t ldb = m > 0 ? B.stride[0] : B.stride[1], ldc = m > 0 ? C.stride[1] : C.stride[0];
  return status(grouped_run(address(h, 0), A.ptr, A.stride[0], B.ptr, ldb, m > 0 ? 0 : B.stride[0], offsets.ptr, A.dim[0],
                            C.ptr, ldc, m > 0 ? C.stride[0] : 0, stream));
}

/* (plan, dtype, groups, N, K, rank), x, A, B, offsets, order (or None), base, out, scales (or None),
 * stream */
static PyObject* py_adapters(PyObject* self, PyObject* const* args, Py_ssize_t nargs) {
  view x, A, B, offsets, order = {0}, base, out, scales = {0};
  void* stream;
  int64_t device = -1;
  TAKES(10);
  PyObject *h = args[0], *dtype = PyTuple_GET_ITEM(h, 1);
  const int64_t groups = whole(h, 2), n = whole(h, 3), k = whole(h, 4), rank = whole(h, 5);
  if (!look_matrix(args[1], dtype, -1, k, &x, &device) || !look_matrices(args[2], dtype, groups, rank, k, &A, &device) ||
      !A.contiguous || !look_matrices(args[3], dtype, groups, n, rank, &B, &device) || !B.contiguous ||
      !look_vector(args[4], t_int32, groups + 1, &offsets, &device) ||
      (args[5] != Py_None && !look_vector(args[5], t_int32, x.dim[0], &order, &device)) ||
      !look_matrix(args[6], dtype, x.dim[0], n, &base, &device) || !look_matrix(args[7], dtype, x.dim[0], n, &out, &device) ||
      (args[8] != Py_None && !look_vector(args[8], t_float32, groups, &scales, &device)))
    return refused();
  STREAM(args[9]);
  return status(adapters_run(address(h, 0), x.ptr, x.stride[0], A.ptr, B.ptr, scales.ptr, offsets.ptr, order.ptr, x.dim[0],
                             base.ptr, base.stride[0], out.ptr, out.stride[0], stream));
}

/* the addresses of the functions over groups of rows, and torch's float32 */
static PyObject* py_setup_groups(PyObject* self, PyObject* args) {
  PyObject *order, *grouped, *adapters;
  if (!PyArg_ParseTuple(args, "OOOO", &order, &grouped, &adapters, &t_float32)) return NULL;
  Py_INCREF(t_float32);
  adapters_run = (__typeof__(adapters_run))PyLong_AsVoidPtr(adapters);
  group_rows = (__typeof__(group_rows))PyLong_AsVoidPtr(order);
  grouped_run = (__typeof__(grouped_run))PyLong_AsVoidPtr(grouped);
  if (PyErr_Occurred()) return NULL;
  Py_RETURN_NONE;
}

/* the addresses of the five functions, the current device, the current stream of a device, torch's int32, float16
 * and bfloat16 */
static PyObject* py_setup(PyObject* self, PyObject* args) {
  PyObject *rope, *prompt, *write, *read, *attend;
  if (!PyArg_ParseTuple(args, "OOOOOOOOOO", &rope, &prompt, &write, &read, &attend, &current_device, &raw_stream,
                        &t_int32, &t_float16, &t_bfloat16))
    return NULL;
  rope_run = (__typeof__(rope_run))PyLong_AsVoidPtr(rope);
  prompt_run = (__typeof__(prompt_run))PyLong_AsVoidPtr(prompt);
  cache_write = (__typeof__(cache_write))PyLong_AsVoidPtr(write);
  cache_read = (__typeof__(cache_read))PyLong_AsVoidPtr(read);
  cache_attend = (__typeof__(cache_attend))PyLong_AsVoidPtr(attend);
  Py_INCREF(current_device);
  Py_INCREF(raw_stream);
  Py_INCREF(t_int32);
  Py_INCREF(t_float16);
  Py_INCREF(t_bfloat16);
  if (PyErr_Occurred()) return NULL;
  Py_RETURN_NONE;
}

static PyMethodDef methods[] = {
    {"setup", py_setup, METH_VARARGS, NULL},
    {"rope", (PyCFunction)(void (*)(void))py_rope, METH_FASTCALL, NULL},
    {"prompt", (PyCFunction)(void (*)(void))py_prompt, METH_FASTCALL, NULL},
    {"cache_write", (PyCFunction)(void (*)(void))py_cache_write, METH_FASTCALL, NULL},
    {"cache_read", (PyCFunction)(void (*)(void))py_cache_read, METH_FASTCALL, NULL},
    {"attend", (PyCFunction)(void (*)(void))py_attend, METH_FASTCALL, NULL},
    {"setup_groups", py_setup_groups, METH_VARARGS, NULL},
    {"row_groups", (PyCFunction)(void (*)(void))py_row_groups, METH_FASTCALL, NULL},
    {"grouped", (PyCFunction)(void (*)(void))py_grouped, METH_FASTCALL, NULL},
    {"adapters", (PyCFunction)(void (*)(void))py_adapters, METH_FASTCALL, NULL},
    {NULL, NULL, 0, NULL}};

static struct PyModuleDef module = {PyModuleDef_HEAD_INIT, "_binding", NULL, -1, methods, NULL, NULL, NULL, NULL};

PyMODINIT_FUNC PyInit__binding(void) {
  PyObject** names[] = {&n_dtype, &n_shape, &n_stride, &n_data_ptr, &n_is_contiguous, &n_get_device};
  const char* text[] = {"dtype", "shape", "stride", "data_ptr", "is_contiguous", "get_device"};
  for (int i = 0; i < 6; ++i)
    if (!(*names[i] = PyUnicode_InternFromString(text[i]))) return NULL;
  return PyModule_Create(&module);
}
