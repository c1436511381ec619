/* CPython binding of the per-call entry points (lora_apply, lora_apply_ranked,
 * lora_apply_device and the decoder-block operators): argument marshalling
 * only.  A serving loop calls one of these once per layer and step; through
 * ctypes the conversion of their 10 to 16 arguments costs more host time than
 * the library's own plan for a small decode batch, and the host then paces the
 * GPU.  Here each argument is one conversion.
 *
 * The library is the one ctypes has loaded: every call takes the entry
 * point's address (ctypes.cast(lib.lora_apply, c_void_p).value) as its first
 * argument and calls through a pointer of the entry point's own type, so this
 * module links nothing and cannot bind a second copy of the library.  Pointer
 * arguments are Python ints (None is NULL), and for the device memory of the
 * decoder-block operators tensors too.  An int is taken as it is; a tensor has
 * to be GPU memory, contiguous and as large as the call reads or writes it, or
 * the call is refused (LoraError): read as if it were contiguous it would give
 * wrong results, and host memory or one too short would fault the GPU.  The
 * return value is the entry point's status.  The GIL is released around the
 * call, as ctypes does. */
#define PY_SSIZE_T_CLEAN
#include <Python.h>
#include <ATen/dlpack.h>
#include <stdint.h>

#include "lora_pool.h"

typedef int32_t (*apply_fn)(const lora_pool_desc*, const void*, const void*, const void*, void*,
                            int32_t, const int32_t*, const uint8_t*, int32_t, void*, int64_t,
                            void*, int64_t, void*);
typedef int32_t (*apply_ranked_fn)(const lora_pool_desc*, const void*, const void*, const void*,
                                   void*, int32_t, const int32_t*, const uint8_t*, int32_t,
                                   const int32_t*, void*, int64_t, void*, int64_t, void*);
typedef int32_t (*apply_device_fn)(const lora_pool_desc*, const void*, const void*, const void*,
                                   void*, int32_t, const int32_t*, const uint8_t*, int32_t, void*,
                                   int64_t, void*);

typedef int32_t (*norm_fn)(const lora_norm_desc*, const void*, const void*, const void*, void*,
                           void*, void*, float*, int32_t, void*);
typedef int32_t (*linear_fn)(const lora_linear_desc*, const void*, const void*, const float*,
                             const float*, const void*, const void*, const void*, void*, int32_t,
                             void*, int64_t, void*);
typedef int32_t (*gated_fn)(const lora_gated_desc*, const void*, const void*, const float*,
                            const float*, const void*, void*, void*, int32_t, void*, int64_t,
                            void*);
typedef int32_t (*gated_backward_fn)(const lora_gated_desc*, const void*, const void*, const void*,
                                     const void*, void*, void*, void*, int32_t, void*, int64_t,
                                     void*);

/* the typedefs match the header's declarations */
_Static_assert(__builtin_types_compatible_p(__typeof__(&lora_add_rms_norm), norm_fn),
               "lora_add_rms_norm");
_Static_assert(__builtin_types_compatible_p(__typeof__(&lora_linear), linear_fn), "lora_linear");
_Static_assert(__builtin_types_compatible_p(__typeof__(&lora_gated_ffn), gated_fn),
               "lora_gated_ffn");
_Static_assert(__builtin_types_compatible_p(__typeof__(&lora_gated_ffn_backward),
                                            gated_backward_fn),
               "lora_gated_ffn_backward");
_Static_assert(__builtin_types_compatible_p(__typeof__(&lora_apply), apply_fn), "lora_apply");
_Static_assert(__builtin_types_compatible_p(__typeof__(&lora_apply_ranked), apply_ranked_fn),
               "lora_apply_ranked");
_Static_assert(__builtin_types_compatible_p(__typeof__(&lora_apply_device), apply_device_fn),
               "lora_apply_device");

/* kinds of argument; D: device memory, an int or a tensor */
enum { P = 0, I32 = 1, I64 = 2, D = 3 };

typedef __int128 wide;

static PyObject* refused;             /* LoraError(status, message), once set_error gave it */
static PyObject* tensor_type;         /* torch.Tensor, once a tensor came in */
static const DLPackExchangeAPI* api;  /* its C interface, or NULL */

static int refuse(int status, const char* name, const char* arg, const char* what) {
  PyObject* message = PyUnicode_FromFormat("%s: %s %s", name, arg, what);
  PyObject* args = message ? Py_BuildValue("(iN)", status, message) : NULL;
  if (args) PyErr_SetObject(refused ? refused : PyExc_ValueError, args);
  Py_XDECREF(args);
  return -1;
}

/* torch's type and C interface, looked up with the first tensor. */
static void find_api(void) {
  PyObject* name = PyUnicode_FromString("torch");
  PyObject* torch = name ? PyImport_GetModule(name) : NULL;
  tensor_type = torch ? PyObject_GetAttrString(torch, "Tensor") : NULL;
  PyObject* c = tensor_type ? PyObject_GetAttrString(tensor_type, "__dlpack_c_exchange_api__") : NULL;
  if (c) api = (const DLPackExchangeAPI*)PyCapsule_GetPointer(c, "dlpack_exchange_api");
  if (api && (api->header.version.major != DLPACK_MAJOR_VERSION ||
              !api->dltensor_from_py_object_no_sync))
    api = NULL;
  PyErr_Clear();
  Py_XDECREF(c); /* (the type holds the capsule) */
  Py_XDECREF(torch);
  Py_XDECREF(name);
}

static int64_t int_attribute(PyObject* a, const char* attribute) {
  PyObject* n = PyObject_GetAttrString(a, attribute);
  if (n && !PyLong_Check(n)) { /* a method */
    PyObject* r = PyObject_CallNoArgs(n);
    Py_DECREF(n);
    n = r;
  }
  const uint64_t v = n ? PyLong_AsUnsignedLongLong(n) : 0;
  Py_XDECREF(n);
  return (int64_t)v;
}

/* The address and size in bytes of a tensor that may be handed to a kernel;
 * 0, or -1 with a Python exception set. */
static int tensor(PyObject* a, const char* name, const char* arg, uint64_t* v, int64_t* bytes) {
  int gpu, contiguous = 1;
  if (!tensor_type) find_api();
  DLTensor t;
  if (api && PyObject_TypeCheck(a, (PyTypeObject*)tensor_type) &&
      api->dltensor_from_py_object_no_sync(a, &t) == 0) {
    /* as fast as data_ptr() alone: a call with seven tensors takes the host 0.94 us
     * with the checks and 0.90 by data_ptr() without them */
    int64_t n = 1;
    gpu = t.device.device_type == kDLROCM || t.device.device_type == kDLCUDA;
    for (int i = t.ndim - 1; i >= 0; --i) {
      if (t.strides && t.shape[i] != 1 && t.strides[i] != n) contiguous = 0;
      n *= t.shape[i];
    }
    if (n == 0) contiguous = 1;
    *v = (uint64_t)(uintptr_t)t.data + (n ? t.byte_offset : 0);
    *bytes = n * ((t.dtype.bits * t.dtype.lanes + 7) / 8);
  } else { /* anything else that has a tensor's attributes */
    PyErr_Clear();
    gpu = (int)int_attribute(a, "is_cuda");
    if (!PyErr_Occurred()) contiguous = (int)int_attribute(a, "is_contiguous");
    if (!PyErr_Occurred()) *bytes = int_attribute(a, "nbytes");
    if (!PyErr_Occurred()) *v = (uint64_t)int_attribute(a, "data_ptr");
    if (PyErr_Occurred()) {
      if (PyErr_ExceptionMatches(PyExc_AttributeError))
        PyErr_Format(PyExc_TypeError, "%s: %s must be None, an address or a GPU tensor, not %s",
                     name, arg, Py_TYPE(a)->tp_name);
      return -1;
    }
  }
  if (!gpu) return refuse(LORA_E_ARG, name, arg, "is not GPU memory");
  if (!contiguous) return refuse(LORA_E_SHAPE, name, arg, "is not contiguous");
  return 0;
}

/* Converts args[0 .. n) by kind into out[], and the tensors' sizes into bytes[]
 * (-1: not a tensor; bytes may be NULL where no kind is D); returns 0, or -1
 * with a Python exception set. */
static int convert_args(PyObject* const* args, Py_ssize_t nargs, const char* name,
                        const int* kinds, const char* const* names, int n, uint64_t* out,
                        int64_t* bytes) {
  if (nargs != n) {
    PyErr_Format(PyExc_TypeError, "%s takes %d arguments (%zd given)", name, n, nargs);
    return -1;
  }
  for (int i = 0; i < n; ++i) {
    PyObject* a = args[i];
    if (bytes) bytes[i] = -1;
    if (kinds[i] == P || kinds[i] == D) {
      if (a == Py_None) {
        out[i] = 0;
        continue;
      }
      if (kinds[i] == D && !PyLong_Check(a)) {
        if (tensor(a, name, names[i], &out[i], &bytes[i])) return -1;
        continue;
      }
      const unsigned long long v = PyLong_AsUnsignedLongLong(a);
      if (v == (unsigned long long)-1 && PyErr_Occurred()) return -1;
      out[i] = v;
    } else {
      const long long v = PyLong_AsLongLong(a);
      if (v == -1 && PyErr_Occurred()) return -1;
      if (kinds[i] == I32 && (v < INT32_MIN || v > INT32_MAX)) {
        PyErr_Format(PyExc_OverflowError, "%s: argument %d does not fit int32", name, i);
        return -1;
      }
      out[i] = (uint64_t)v;
    }
  }
  if (out[0] == 0) {
    PyErr_Format(PyExc_ValueError, "%s: NULL entry point address", name);
    return -1;
  }
  return 0;
}
static int convert(PyObject* const* args, Py_ssize_t nargs, const char* name, const int* kinds,
                   int n, uint64_t* out) {
  return convert_args(args, nargs, name, kinds, NULL, n, out, NULL);
}

/* Whether each tensor holds what the call takes of it; 0, or -1 with a Python
 * exception set. */
static int large_enough(const char* name, const char* const* names, int n, const int64_t* bytes,
                        const wide* need, int ws) {
  for (int i = 0; i < n; ++i)
    if (bytes[i] >= 0 && bytes[i] < need[i])
      return refuse(i == ws ? LORA_E_WORKSPACE : LORA_E_SHAPE, name, names[i],
                    "is smaller than the call takes it to be");
  return 0;
}

static wide size_of(int32_t dtype) { return dtype == LORA_F32 ? 4 : dtype == LORA_BF16 ? 2 : 1; }

#define PTR(i) ((void*)(uintptr_t)a[i])
#define I32V(i) ((int32_t)(int64_t)a[i])
#define I64V(i) ((int64_t)a[i])

/* apply(fn, desc, A_pool, B_pool, x, y, T, ids_host, prefill_host,
 *       bgmv_max_rank, ws, ws_bytes, meta_host, meta_host_bytes, stream) */
static PyObject* py_apply(PyObject* self, PyObject* const* args, Py_ssize_t nargs) {
  (void)self;
  static const int kinds[15] = {P, P, P, P, P, P, I32, P, P, I32, P, I64, P, I64, P};
  uint64_t a[15];
  if (convert(args, nargs, "apply", kinds, 15, a)) return NULL;
  const apply_fn f = (apply_fn)(uintptr_t)a[0];
  int32_t st;
  Py_BEGIN_ALLOW_THREADS
  st = f((const lora_pool_desc*)PTR(1), PTR(2), PTR(3), PTR(4), PTR(5), I32V(6),
         (const int32_t*)PTR(7), (const uint8_t*)PTR(8), I32V(9), PTR(10), I64V(11), PTR(12),
         I64V(13), PTR(14));
  Py_END_ALLOW_THREADS
  return PyLong_FromLong(st);
}

/* apply_ranked(fn, desc, A_pool, B_pool, x, y, T, ids_host, prefill_host,
 *              bgmv_max_rank, slot_ranks, ws, ws_bytes, meta_host,
 *              meta_host_bytes, stream) */
static PyObject* py_apply_ranked(PyObject* self, PyObject* const* args, Py_ssize_t nargs) {
  (void)self;
  static const int kinds[16] = {P, P, P, P, P, P, I32, P, P, I32, P, P, I64, P, I64, P};
  uint64_t a[16];
  if (convert(args, nargs, "apply_ranked", kinds, 16, a)) return NULL;
  const apply_ranked_fn f = (apply_ranked_fn)(uintptr_t)a[0];
  int32_t st;
  Py_BEGIN_ALLOW_THREADS
  st = f((const lora_pool_desc*)PTR(1), PTR(2), PTR(3), PTR(4), PTR(5), I32V(6),
         (const int32_t*)PTR(7), (const uint8_t*)PTR(8), I32V(9), (const int32_t*)PTR(10),
         PTR(11), I64V(12), PTR(13), I64V(14), PTR(15));
  Py_END_ALLOW_THREADS
  return PyLong_FromLong(st);
}

/* apply_device(fn, desc, A_pool, B_pool, x, y, T, ids, prefill,
 *              bgmv_max_rank, ws, ws_bytes, stream) */
static PyObject* py_apply_device(PyObject* self, PyObject* const* args, Py_ssize_t nargs) {
  (void)self;
  static const int kinds[13] = {P, P, P, P, P, P, I32, P, P, I32, P, I64, P};
  uint64_t a[13];
  if (convert(args, nargs, "apply_device", kinds, 13, a)) return NULL;
  const apply_device_fn f = (apply_device_fn)(uintptr_t)a[0];
  int32_t st;
  Py_BEGIN_ALLOW_THREADS
  st = f((const lora_pool_desc*)PTR(1), PTR(2), PTR(3), PTR(4), PTR(5), I32V(6),
         (const int32_t*)PTR(7), (const uint8_t*)PTR(8), I32V(9), PTR(10), I64V(11), PTR(12));
  Py_END_ALLOW_THREADS
  return PyLong_FromLong(st);
}

/* add_rms_norm(fn, desc, x, residual, weight, sum, out, out8, scale, T, stream) */
static PyObject* py_norm(PyObject* self, PyObject* const* args, Py_ssize_t nargs) {
  (void)self;
  static const int kinds[11] = {P, P, D, D, D, D, D, D, D, I32, P};
  static const char* const names[11] = {"fn",  "desc", "x",     "residual", "weight", "sum",
                                        "out", "out8", "scale", "T",        "stream"};
  uint64_t a[11];
  int64_t bytes[11];
  if (convert_args(args, nargs, "add_rms_norm", kinds, names, 11, a, bytes)) return NULL;
  const lora_norm_desc* d = (const lora_norm_desc*)PTR(1);
  const int32_t T = I32V(9);
  if (d && T > 0) {
    const wide H = d->hidden, all = H * T, e = size_of(d->dtype);
    const wide need[11] = {0, 0, all * e, all * e, H * e, all * e, all * e, all, (wide)T * 4};
    if (large_enough("add_rms_norm", names, 11, bytes, need, -1)) return NULL;
  }
  const norm_fn f = (norm_fn)(uintptr_t)a[0];
  int32_t st;
  Py_BEGIN_ALLOW_THREADS
  st = f(d, PTR(2), PTR(3), PTR(4), PTR(5), PTR(6), PTR(7), (float*)PTR(8), T, PTR(10));
  Py_END_ALLOW_THREADS
  return PyLong_FromLong(st);
}

/* linear(fn, desc, x, w, x_scale, w_scale, bias, delta, residual, out, T, ws,
 *        ws_bytes, stream) */
static PyObject* py_linear(PyObject* self, PyObject* const* args, Py_ssize_t nargs) {
  (void)self;
  static const int kinds[14] = {P, P, D, D, D, D, D, D, D, D, I32, D, I64, P};
  static const char* const names[14] = {"fn",    "desc",     "x",   "w", "x_scale", "w_scale",  "bias",
                                        "delta", "residual", "out", "T", "ws",      "ws_bytes", "stream"};
  uint64_t a[14];
  int64_t bytes[14];
  if (convert_args(args, nargs, "linear", kinds, names, 14, a, bytes)) return NULL;
  const lora_linear_desc* d = (const lora_linear_desc*)PTR(1);
  const int32_t T = I32V(10);
  if (d && T > 0) {
    const wide K = d->in_features, O = d->out_features, e = size_of(d->dtype),
               o = size_of(d->out_dtype), rows = T;
    const wide need[14] = {0,     0,     rows * K * e, O * K * e,    rows * 4, O * 4,
                           O * o, rows * O * o, rows * O * o, rows * O * o, 0, I64V(12)};
    if (large_enough("linear", names, 14, bytes, need, 11)) return NULL;
  }
  const linear_fn f = (linear_fn)(uintptr_t)a[0];
  int32_t st;
  Py_BEGIN_ALLOW_THREADS
  st = f(d, PTR(2), PTR(3), (const float*)PTR(4), (const float*)PTR(5), PTR(6), PTR(7), PTR(8),
         PTR(9), T, PTR(11), I64V(12), PTR(13));
  Py_END_ALLOW_THREADS
  return PyLong_FromLong(st);
}

/* gated_ffn(fn, desc, x, w, x_scale, w_scale, delta, pre, out, T, ws, ws_bytes,
 *           stream) */
static PyObject* py_gated(PyObject* self, PyObject* const* args, Py_ssize_t nargs) {
  (void)self;
  static const int kinds[13] = {P, P, D, D, D, D, D, D, D, I32, D, I64, P};
  static const char* const names[13] = {"fn",  "desc", "x", "w",  "x_scale",  "w_scale", "delta",
                                        "pre", "out",  "T", "ws", "ws_bytes", "stream"};
  uint64_t a[13];
  int64_t bytes[13];
  if (convert_args(args, nargs, "gated_ffn", kinds, names, 13, a, bytes)) return NULL;
  const lora_gated_desc* d = (const lora_gated_desc*)PTR(1);
  const int32_t T = I32V(9);
  if (d && T > 0) {
    const wide K = d->in_features, I = d->inter_features, e = size_of(d->dtype),
               o = size_of(d->out_dtype), rows = T;
    const wide need[13] = {0,     0, rows * K * e,     2 * I * K * e, rows * 4, 2 * I * 4,
                           rows * 2 * I * o, rows * 2 * I * o, rows * I * o, 0, I64V(11)};
    if (large_enough("gated_ffn", names, 13, bytes, need, 10)) return NULL;
  }
  const gated_fn f = (gated_fn)(uintptr_t)a[0];
  int32_t st;
  Py_BEGIN_ALLOW_THREADS
  st = f(d, PTR(2), PTR(3), (const float*)PTR(4), (const float*)PTR(5), PTR(6), PTR(7), PTR(8), T,
         PTR(10), I64V(11), PTR(12));
  Py_END_ALLOW_THREADS
  return PyLong_FromLong(st);
}

/* gated_ffn_backward(fn, desc, dout, pre, x, w, dpre, dx, dw, T, ws, ws_bytes,
 *                    stream) */
static PyObject* py_gated_backward(PyObject* self, PyObject* const* args, Py_ssize_t nargs) {
  (void)self;
  static const int kinds[13] = {P, P, D, D, D, D, D, D, D, I32, D, I64, P};
  static const char* const names[13] = {"fn", "desc", "dout", "pre", "x",        "w",     "dpre",
                                        "dx", "dw",   "T",    "ws",  "ws_bytes", "stream"};
  uint64_t a[13];
  int64_t bytes[13];
  if (convert_args(args, nargs, "gated_ffn_backward", kinds, names, 13, a, bytes)) return NULL;
  const lora_gated_desc* d = (const lora_gated_desc*)PTR(1);
  const int32_t T = I32V(9);
  if (d && T >= 0) {
    const wide K = d->in_features, I = d->inter_features, e = size_of(d->dtype), rows = T;
    const wide w = 2 * I * K * e, x = rows * K * e, half = rows * I * e;
    /* (x is read for dw and w for dx; over no rows only dw is touched) */
    const wide need[13] = {0,        0,  half, 2 * half, a[8] ? x : 0, a[7] && T ? w : 0,
                           2 * half, x,  w,    0,        T ? I64V(11) : 0};
    if (large_enough("gated_ffn_backward", names, 13, bytes, need, 10)) return NULL;
  }
  const gated_backward_fn f = (gated_backward_fn)(uintptr_t)a[0];
  int32_t st;
  Py_BEGIN_ALLOW_THREADS
  st = f(d, PTR(2), PTR(3), PTR(4), PTR(5), PTR(6), PTR(7), PTR(8), T, PTR(10), I64V(11), PTR(12));
  Py_END_ALLOW_THREADS
  return PyLong_FromLong(st);
}

/* set_error(type): what a refused tensor raises, as type(status, message) */
static PyObject* py_set_error(PyObject* self, PyObject* type) {
  (void)self;
  Py_INCREF(type);
  Py_XSETREF(refused, type);
  Py_RETURN_NONE;
}

static PyMethodDef methods[] = {
    {"set_error", py_set_error, METH_O,
     "set_error(type): the exception type(status, message) of a refused tensor"},
    {"add_rms_norm", (PyCFunction)(void (*)(void))py_norm, METH_FASTCALL,
     "add_rms_norm(fn, desc, x, residual, weight, sum, out, out8, scale, T, stream) -> status of "
     "lora_add_rms_norm"},
    {"linear", (PyCFunction)(void (*)(void))py_linear, METH_FASTCALL,
     "linear(fn, desc, x, w, x_scale, w_scale, bias, delta, residual, out, T, ws, ws_bytes, "
     "stream) -> status of lora_linear"},
    {"gated_ffn", (PyCFunction)(void (*)(void))py_gated, METH_FASTCALL,
     "gated_ffn(fn, desc, x, w, x_scale, w_scale, delta, pre, out, T, ws, ws_bytes, stream) -> "
     "status of lora_gated_ffn"},
    {"gated_ffn_backward", (PyCFunction)(void (*)(void))py_gated_backward, METH_FASTCALL,
     "gated_ffn_backward(fn, desc, dout, pre, x, w, dpre, dx, dw, T, ws, ws_bytes, stream) -> "
     "status of lora_gated_ffn_backward"},
    {"apply", (PyCFunction)(void (*)(void))py_apply, METH_FASTCALL,
     "apply(fn, desc, A_pool, B_pool, x, y, T, ids_host, prefill_host, bgmv_max_rank, ws, "
     "ws_bytes, meta_host, meta_host_bytes, stream) -> status of lora_apply"},
    {"apply_ranked", (PyCFunction)(void (*)(void))py_apply_ranked, METH_FASTCALL,
     "apply_ranked(fn, desc, A_pool, B_pool, x, y, T, ids_host, prefill_host, bgmv_max_rank, "
     "slot_ranks, ws, ws_bytes, meta_host, meta_host_bytes, stream) -> status of "
     "lora_apply_ranked"},
    {"apply_device", (PyCFunction)(void (*)(void))py_apply_device, METH_FASTCALL,
     "apply_device(fn, desc, A_pool, B_pool, x, y, T, ids, prefill, bgmv_max_rank, ws, "
     "ws_bytes, stream) -> status of lora_apply_device"},
    {NULL, NULL, 0, NULL}};

static struct PyModuleDef module = {PyModuleDef_HEAD_INIT, "_lora_call",
                                    "CPython binding of the per-call entry points", -1, methods,
                                    NULL, NULL, NULL, NULL};

PyMODINIT_FUNC PyInit__lora_call(void) { return PyModule_Create(&module); }
