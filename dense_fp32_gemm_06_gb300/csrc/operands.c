/* The Python side of the adapter and loss calls: looks tensors over and calls
 * the C ABI (include/adapters_gb300.h) with their pointers and pitches.
 *
 * A Python call of these kernels' size is mostly its checks: as Python
 * functions they took 5 to 6 us of a 9 to 13 us call, beside kernels of 4.
 * Here a tensor costs five attribute look-ups.  What is wrong is reported
 * through the `refuse` function that setup() was given, which raises.
 *
 * Every function takes, positionally: the address of the C function, the
 * device index, the stream handle, then the call's tensors (None where they
 * may be missing) and numbers; it returns the C ABI's status.
 */
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <limits.h>
#include <stdint.h>

static PyObject *s_dtype, *s_shape, *s_get_device, *s_is_contiguous, *s_data_ptr, *s_stride;
static PyObject *t_f32, *t_bf16, *t_f16, *t_i32, *g_refuse;

typedef struct {
    void *ptr;
    long long dim[3], pitch;
} Operand;

/* raises through Python: refuse(what, name, tensor, dtype, dev) */
static int refuse(const char *what, const char *name, PyObject *t, PyObject *dtype, long dev) {
    PyObject *r = PyObject_CallFunction(g_refuse, "ssOOl", what, name, t ? t : Py_None, dtype ? dtype : Py_None, dev);
    Py_XDECREF(r);
    if (!PyErr_Occurred()) PyErr_SetString(PyExc_RuntimeError, what);
    return -1;
}

static int as_long(PyObject *o, long long *v) { /* steals o */
    if (o == NULL) return -1;
    *v = PyLong_AsLongLong(o);
    Py_DECREF(o);
    return *v == -1 && PyErr_Occurred() ? -1 : 0;
}

/* the tensor's axes; -1 with an exception set */
static int dims_of(PyObject *t, int n, long long *dim, const char *name) {
    if (t == Py_None) return refuse("missing", name, t, NULL, 0);
    PyObject *shape = PyObject_GetAttr(t, s_shape);
    if (shape == NULL) return -1;
    const int ok = PyTuple_Check(shape) && PyTuple_GET_SIZE(shape) == n;
    for (int i = 0; ok && i < n; ++i) dim[i] = PyLong_AsLongLong(PyTuple_GET_ITEM(shape, i));
    Py_DECREF(shape);
    if (!ok) return refuse(n == 1 ? "one axis" : n == 2 ? "two axes" : "three axes", name, t, NULL, 0);
    return PyErr_Occurred() ? -1 : 0;
}

/* type, device, and the data's address */
static int data_of(PyObject *t, const char *name, PyObject *dtype, long dev, Operand *o) {
    PyObject *d = PyObject_GetAttr(t, s_dtype);
    if (d == NULL) return -1;
    Py_DECREF(d); /* torch keeps its types */
    long long on, p;
    if (as_long(PyObject_CallMethodNoArgs(t, s_get_device), &on)) return -1;
    if (d != dtype || on != dev) return refuse("type", name, t, dtype, dev);
    if (as_long(PyObject_CallMethodNoArgs(t, s_data_ptr), &p)) return -1;
    o->ptr = (void *)(intptr_t)p;
    return 0;
}

/* a contiguous tensor of n axes with the lengths `dim` (None: a null pointer) */
static int vector(PyObject *t, const char *name, PyObject *dtype, long dev, int n, const long long *dim, Operand *o) {
    o->ptr = NULL;
    if (t == Py_None) return 0;
    if (dims_of(t, n, o->dim, name)) return -1;
    for (int i = 0; i < n; ++i)
        if (o->dim[i] != dim[i]) return refuse("shape", name, t, NULL, 0);
    if (data_of(t, name, dtype, dev, o)) return -1;
    PyObject *c = PyObject_CallMethodNoArgs(t, s_is_contiguous);
    if (c == NULL) return -1;
    Py_DECREF(c);
    return c == Py_True ? 0 : refuse("contiguous", name, t, dtype, dev);
}

static int strides_of(PyObject *t, long long *s0, long long *s1) {
    PyObject *s = PyObject_CallMethodNoArgs(t, s_stride);
    if (s == NULL) return -1;
    *s0 = PyLong_AsLongLong(PyTuple_GET_ITEM(s, 0));
    *s1 = PyLong_AsLongLong(PyTuple_GET_ITEM(s, 1));
    Py_DECREF(s);
    return PyErr_Occurred() ? -1 : 0;
}

/* a row-major matrix of two axes; rows and cols below zero are taken from it */
static int matrix(PyObject *t, const char *name, PyObject *dtype, long dev, long long rows, long long cols, Operand *o) {
    long long one;
    if (dims_of(t, 2, o->dim, name)) return -1;
    if (rows < 0) rows = o->dim[0];
    if (cols < 0) cols = o->dim[1];
    if (o->dim[0] != rows || o->dim[1] != cols) return refuse("shape", name, t, NULL, 0);
    if (data_of(t, name, dtype, dev, o) || strides_of(t, &o->pitch, &one)) return -1;
    if (one != 1 && cols > 1) return refuse("columns", name, t, dtype, dev);
    if (rows <= 1) o->pitch = cols;
    if (o->pitch < cols || o->pitch > INT_MAX || rows > INT_MAX) return refuse("rows", name, t, dtype, dev);
    if (o->pitch < 1) o->pitch = 1;
    return 0;
}

/* the same of a matrix that the call may not need (None: a null pointer, which the C ABI refuses where it does) */
static int matrix_if(PyObject *t, const char *name, PyObject *dtype, long dev, long long rows, long long cols, Operand *o) {
    if (t != Py_None) return matrix(t, name, dtype, dev, rows, cols, o);
    o->ptr = NULL;
    o->pitch = cols > 0 ? cols : 1;
    return 0;
}

/* W, k x n: row-major (op 0) or a transposed view of a row-major matrix (1); None as of matrix_if */
static int weight(PyObject *t, PyObject *dtype, long dev, long long k, long long n, Operand *o, int *op) {
    long long s0, s1, least;
    if (t == Py_None) {
        o->ptr = NULL;
        o->pitch = n > 0 ? n : 1;
        *op = 0;
        return 0;
    }
    if (dims_of(t, 2, o->dim, "W")) return -1;
    if (o->dim[0] != k || o->dim[1] != n) return refuse("shape", "W", t, NULL, 0);
    if (data_of(t, "W", dtype, dev, o) || strides_of(t, &s0, &s1)) return -1;
    if (n <= 1 || s1 == 1) {
        *op = 0;
        o->pitch = k > 1 ? s0 : n;
        least = n;
    } else if (k <= 1 || s0 == 1) {
        *op = 1;
        o->pitch = s1;
        least = k;
    } else {
        return refuse("transposed", "W", t, dtype, dev);
    }
    if (o->pitch < least || o->pitch > INT_MAX || k > INT_MAX || n > INT_MAX) return refuse("rows", "W", t, dtype, dev);
    if (o->pitch < 1) o->pitch = 1;
    return 0;
}

static PyObject *dtype_of(PyObject *t) { /* borrowed: torch keeps its types */
    PyObject *d = PyObject_GetAttr(t, s_dtype);
    Py_XDECREF(d);
    return d;
}

typedef struct {
    void *fn, *stream;
    long dev;
} Call;

static int call_of(PyObject *const *a, Py_ssize_t n, Py_ssize_t want, Call *c) {
    if (n != want) {
        PyErr_Format(PyExc_TypeError, "%zd arguments, not %zd", n, want);
        return -1;
    }
    c->fn = PyLong_AsVoidPtr(a[0]);
    c->dev = PyLong_AsLong(a[1]);
    c->stream = PyLong_AsVoidPtr(a[2]);
    return PyErr_Occurred() ? -1 : 0;
}

/* fn, dev, stream, X, W, A, B, ids, Y, scale, H */
typedef int (*Forward)(int, int, int, int, int, int, const void *, int, int, const void *, int, const void *, const void *,
                       const int *, const float *, void *, int, float *, void *);

static PyObject *lora_forward(PyObject *self, PyObject *const *a, Py_ssize_t n) {
    (void)self;
    Call c;
    Operand X, W, A, B, ids, Y, scale, H;
    long long stack[3];
    int op, st;
    if (call_of(a, n, 11, &c)) return NULL;
    if (dims_of(a[8], 2, Y.dim, "Y") || dims_of(a[3], 2, X.dim, "X") || dims_of(a[5], 3, stack, "A")) return NULL;
    PyObject *dtype = dtype_of(a[8]);
    if (dtype == NULL) return NULL;
    const long long T = X.dim[0], K = X.dim[1], N = Y.dim[1], L = stack[0], R = stack[1];
    if ((dtype != t_f32 && dtype != t_bf16) || c.dev < 0) {
        PyObject *w = a[4];
        if (dims_of(w, 2, W.dim, "W")) return NULL;
        if (W.dim[0] != K || W.dim[1] != N) refuse("shape", "W", w, NULL, 0);
        else refuse("matrices", "Y", a[8], dtype, c.dev);
        return NULL;
    }
    const long long da[3] = {L, R, K}, db[3] = {L, R, N}, dh[2] = {T, R};
    if (weight(a[4], dtype, c.dev, K, N, &W, &op) || matrix(a[3], "X", dtype, c.dev, T, K, &X) ||
        vector(a[5], "A", dtype, c.dev, 3, da, &A) || vector(a[6], "B", dtype, c.dev, 3, db, &B) ||
        vector(a[7], "ids", t_i32, c.dev, 1, &T, &ids) || matrix(a[8], "Y", dtype, c.dev, T, N, &Y) ||
        vector(a[9], "scale", t_f32, c.dev, 1, &L, &scale) || vector(a[10], "H", t_f32, c.dev, 2, dh, &H))
        return NULL;
    if (L > INT_MAX || R > INT_MAX) {
        refuse("rows", "A", a[5], dtype, c.dev);
        return NULL;
    }
    Py_BEGIN_ALLOW_THREADS
    st = ((Forward)c.fn)((int)T, (int)K, (int)N, (int)L, (int)R, dtype == t_bf16, X.ptr, (int)X.pitch, op, W.ptr, (int)W.pitch, A.ptr,
                         B.ptr, ids.ptr, scale.ptr, Y.ptr, (int)Y.pitch, H.ptr, c.stream);
    Py_END_ALLOW_THREADS
    return PyLong_FromLong(st);
}

/* axis `axis` of the first of `count` tensors of `n` axes that is not None (-1: all are) */
typedef struct {
    PyObject *t;
    const char *name;
    int n, axis;
} Axis;
static int axis_of(const Axis *of, int count, long long *v) {
    long long dim[3];
    *v = -1;
    for (int i = 0; i < count; ++i)
        if (of[i].t != Py_None) {
            if (dims_of(of[i].t, of[i].n, dim, of[i].name)) return -1;
            *v = dim[of[i].axis];
            return 0;
        }
    return 0;
}

/* fn, dev, stream, dY, X, W, A, B, ids, H, dX, dA, dB, scale */
typedef int (*Backward)(int, int, int, int, int, int, const void *, int, const void *, int, int, const void *, int, const void *,
                        const void *, const int *, const float *, const float *, void *, int, void *, void *, void *);

static PyObject *lora_backward(PyObject *self, PyObject *const *a, Py_ssize_t n) {
    (void)self;
    Call c;
    Operand dY, X, W, A, B, ids, H, dX, dA, dB, scale;
    long long K, L, R;
    int op, st;
    if (call_of(a, n, 14, &c) || dims_of(a[3], 2, dY.dim, "dY")) return NULL;
    /* X, W, A and B may be missing where the gradients asked for do not need them */
    const Axis k[] = {{a[4], "X", 2, 1}, {a[5], "W", 2, 0}, {a[6], "A", 3, 2}, {a[10], "dX", 2, 1}, {a[11], "dA", 3, 2}};
    const Axis l[] = {{a[6], "A", 3, 0}, {a[7], "B", 3, 0}, {a[11], "dA", 3, 0}, {a[12], "dB", 3, 0}};
    const Axis r[] = {{a[6], "A", 3, 1}, {a[7], "B", 3, 1}, {a[11], "dA", 3, 1}, {a[12], "dB", 3, 1}};
    PyObject *dtype = dtype_of(a[3]);
    if (dtype == NULL || axis_of(k, 5, &K) || axis_of(l, 4, &L) || axis_of(r, 4, &R)) return NULL;
    if (L < 0) {
        refuse("missing", "A", a[6], dtype, c.dev);
        return NULL;
    }
    if (K < 0) K = 0;
    const long long T = dY.dim[0], N = dY.dim[1];
    if ((dtype != t_f32 && dtype != t_bf16) || c.dev < 0) {
        refuse("matrices", "dY", a[3], dtype, c.dev);
        return NULL;
    }
    const long long da[3] = {L, R, K}, db[3] = {L, R, N}, dh[2] = {T, R};
    if (weight(a[5], dtype, c.dev, K, N, &W, &op) || matrix(a[3], "dY", dtype, c.dev, T, N, &dY) ||
        matrix_if(a[4], "X", dtype, c.dev, T, K, &X) || vector(a[6], "A", dtype, c.dev, 3, da, &A) ||
        vector(a[7], "B", dtype, c.dev, 3, db, &B) || vector(a[8], "ids", t_i32, c.dev, 1, &T, &ids) ||
        vector(a[9], "H", t_f32, c.dev, 2, dh, &H) || matrix_if(a[10], "dX", dtype, c.dev, T, K, &dX) ||
        vector(a[11], "dA", dtype, c.dev, 3, da, &dA) || vector(a[12], "dB", dtype, c.dev, 3, db, &dB) ||
        vector(a[13], "scale", t_f32, c.dev, 1, &L, &scale))
        return NULL;
    if (L > INT_MAX || R > INT_MAX) {
        refuse("rows", "A", a[6], dtype, c.dev);
        return NULL;
    }
    Py_BEGIN_ALLOW_THREADS
    st = ((Backward)c.fn)((int)T, (int)K, (int)N, (int)L, (int)R, dtype == t_bf16, dY.ptr, (int)dY.pitch, X.ptr, (int)X.pitch, op,
                          W.ptr, (int)W.pitch, A.ptr, B.ptr, ids.ptr, scale.ptr, H.ptr, dX.ptr, (int)dX.pitch, dA.ptr, dB.ptr,
                          c.stream);
    Py_END_ALLOW_THREADS
    return PyLong_FromLong(st);
}

/* the logits, the gradient (or None) and the loss of a call over rows */
static int rows_of(PyObject *logits, PyObject *grad, PyObject *loss, Call *c, int *dtype, Operand *z, Operand *g, Operand *l) {
    if (logits == Py_None) return refuse("missing", "logits", logits, NULL, c->dev);
    PyObject *d = dtype_of(logits);
    if (d == NULL) return -1;
    if ((d != t_f32 && d != t_bf16 && d != t_f16) || c->dev < 0) return refuse("logits", "logits", logits, d, c->dev);
    *dtype = d == t_f32 ? 0 : d == t_bf16 ? 1 : 2;
    if (matrix(logits, "logits", d, c->dev, -1, -1, z)) return -1;
    if (z->dim[1] > INT_MAX) return refuse("rows", "logits", logits, d, c->dev);
    if (matrix_if(grad, "grad", d, c->dev, z->dim[0], z->dim[1], g)) return -1;
    if (loss == Py_None) return refuse("type", "loss", loss, t_f32, c->dev);
    return vector(loss, "loss", t_f32, c->dev, 1, &z->dim[0], l);
}

/* fn, dev, stream, logits, teacher, index, loss, grad, weight, temperature */
typedef int (*Distill)(int, int, int, int, const void *, int, const float *, const int *, const float *, float, float *, void *, int,
                       void *);

static PyObject *distill_topk(PyObject *self, PyObject *const *a, Py_ssize_t n) {
    (void)self;
    Call c;
    Operand z, g, l, teacher, index, weight_;
    long long top[2];
    int dtype, st;
    if (call_of(a, n, 10, &c) || rows_of(a[3], a[7], a[6], &c, &dtype, &z, &g, &l)) return NULL;
    const double tau = PyFloat_AsDouble(a[9]);
    if (PyErr_Occurred() || dims_of(a[4], 2, top, "teacher")) return NULL;
    top[0] = z.dim[0];
    if (a[5] == Py_None) {
        refuse("type", "index", a[5], t_i32, c.dev);
        return NULL;
    }
    if (vector(a[4], "teacher", t_f32, c.dev, 2, top, &teacher) || vector(a[5], "index", t_i32, c.dev, 2, top, &index) ||
        vector(a[8], "weight", t_f32, c.dev, 1, &z.dim[0], &weight_))
        return NULL;
    Py_BEGIN_ALLOW_THREADS
    st = ((Distill)c.fn)((int)z.dim[0], (int)z.dim[1], top[1] > INT_MAX ? INT_MAX : (int)top[1], dtype, z.ptr, (int)z.pitch,
                         teacher.ptr, index.ptr, weight_.ptr, (float)tau, l.ptr, g.ptr, (int)g.pitch, c.stream);
    Py_END_ALLOW_THREADS
    return PyLong_FromLong(st);
}

/* fn, dev, stream, logits, labels, old_logp, advantage, loss, grad, ref, weight, clip_low, clip_high, kl_coef, logp */
typedef int (*Policy)(int, int, int, const void *, int, const int *, const float *, const float *, const float *, const float *,
                      float, float, float, float *, float *, void *, int, void *);

static PyObject *policy_loss(PyObject *self, PyObject *const *a, Py_ssize_t n) {
    (void)self;
    Call c;
    Operand z, g, l, labels, old, adv, ref, weight_, logp;
    int dtype, st;
    if (call_of(a, n, 15, &c) || rows_of(a[3], a[8], a[7], &c, &dtype, &z, &g, &l)) return NULL;
    const double lo = PyFloat_AsDouble(a[11]), hi = PyFloat_AsDouble(a[12]), kl = PyFloat_AsDouble(a[13]);
    if (PyErr_Occurred()) return NULL;
    for (int i = 4; i < 7; ++i)
        if (a[i] == Py_None) {
            refuse("type", i == 4 ? "labels" : i == 5 ? "old_logp" : "advantage", a[i], i == 4 ? t_i32 : t_f32, c.dev);
            return NULL;
        }
    if (a[9] == Py_None && kl != 0.0) {
        refuse("kl_coef", "ref", a[9], t_f32, c.dev);
        return NULL;
    }
    const long long *T = &z.dim[0];
    if (vector(a[4], "labels", t_i32, c.dev, 1, T, &labels) || vector(a[5], "old_logp", t_f32, c.dev, 1, T, &old) ||
        vector(a[6], "advantage", t_f32, c.dev, 1, T, &adv) || vector(a[9], "ref", t_f32, c.dev, 1, T, &ref) ||
        vector(a[10], "weight", t_f32, c.dev, 1, T, &weight_) || vector(a[14], "logp", t_f32, c.dev, 1, T, &logp))
        return NULL;
    Py_BEGIN_ALLOW_THREADS
    st = ((Policy)c.fn)((int)*T, (int)z.dim[1], dtype, z.ptr, (int)z.pitch, labels.ptr, old.ptr, adv.ptr, ref.ptr, weight_.ptr,
                        (float)lo, (float)hi, (float)kl, l.ptr, logp.ptr, g.ptr, (int)g.pitch, c.stream);
    Py_END_ALLOW_THREADS
    return PyLong_FromLong(st);
}

/* setup(refuse, float32, bfloat16, float16, int32) */
static PyObject *setup(PyObject *self, PyObject *args) {
    (void)self;
    PyObject *r, *f32, *bf16, *f16, *i32;
    if (!PyArg_ParseTuple(args, "OOOOO", &r, &f32, &bf16, &f16, &i32)) return NULL;
    PyObject **const to[] = {&g_refuse, &t_f32, &t_bf16, &t_f16, &t_i32};
    PyObject *const from[] = {r, f32, bf16, f16, i32};
    for (int i = 0; i < 5; ++i) {
        Py_INCREF(from[i]);
        Py_XSETREF(*to[i], from[i]);
    }
    Py_RETURN_NONE;
}

static PyMethodDef methods[] = {
    {"setup", setup, METH_VARARGS, "setup(refuse, float32, bfloat16, float16, int32)"},
    {"lora_forward", (PyCFunction)(void (*)(void))lora_forward, METH_FASTCALL, NULL},
    {"lora_backward", (PyCFunction)(void (*)(void))lora_backward, METH_FASTCALL, NULL},
    {"distill_topk", (PyCFunction)(void (*)(void))distill_topk, METH_FASTCALL, NULL},
    {"policy_loss", (PyCFunction)(void (*)(void))policy_loss, METH_FASTCALL, NULL},
    {NULL, NULL, 0, NULL}};

static struct PyModuleDef module = {PyModuleDef_HEAD_INIT, "_operands", NULL, -1, methods, NULL, NULL, NULL, NULL};

PyMODINIT_FUNC PyInit__operands(void) {
    s_dtype = PyUnicode_InternFromString("dtype");
    s_shape = PyUnicode_InternFromString("shape");
    s_get_device = PyUnicode_InternFromString("get_device");
    s_is_contiguous = PyUnicode_InternFromString("is_contiguous");
    s_data_ptr = PyUnicode_InternFromString("data_ptr");
    s_stride = PyUnicode_InternFromString("stride");
    if (!s_dtype || !s_shape || !s_get_device || !s_is_contiguous || !s_data_ptr || !s_stride) return NULL;
    return PyModule_Create(&module);
}
