/* The Python side of the adapter, loss and microscaled calls: looks tensors over and
 * calls the C ABI (include/adapters_gb300.h, include/microscale_gb300.h) with their
 * pointers and pitches.
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
static PyObject *t_f32, *t_bf16, *t_f16, *t_i32, *t_u8, *t_i8, *g_refuse;

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

static PyObject *dtype_of(PyObject *t) { /* borrowed: torch keeps its types */
    PyObject *d = PyObject_GetAttr(t, s_dtype);
    Py_XDECREF(d);
    return d;
}

/* type (NULL: it has been looked up), device, and the data's address */
static int data_of(PyObject *t, const char *name, PyObject *dtype, long dev, Operand *o) {
    PyObject *d = dtype ? dtype_of(t) : NULL;
    if (dtype && d == NULL) return -1;
    long long on, p;
    if (as_long(PyObject_CallMethodNoArgs(t, s_get_device), &on)) return -1;
    if (d != dtype || on != dev) return refuse("type", name, t, dtype ? dtype : dtype_of(t), dev);
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

/* a coded matrix: codes (uint8: 4 bits, int8: 8 bits) of whole blocks beside scales; rows below zero and cols below
 * zero are taken from them (cols as whole blocks); one row, or rows of nothing, may have any pitch */
static int coded(PyObject *codes, PyObject *scales, const char *name, const char *scales_name, long dev, long long rows, long long cols,
                 int only4, Operand *c, Operand *s, int *bits) {
    if (codes == Py_None) return refuse("missing", name, codes, NULL, 0);
    PyObject *d = dtype_of(codes);
    if (d == NULL) return -1;
    if (d != t_u8 && (d != t_i8 || only4)) return refuse(only4 ? "codes of 4 bits" : "codes", name, codes, d, dev);
    *bits = d == t_u8 ? 4 : 8;
    if (matrix(scales, scales_name, t_u8, dev, rows, cols < 0 ? -1 : cols / 32 + (cols % 32 != 0), s) ||
        matrix(codes, name, NULL, dev, s->dim[0], s->dim[1] * *bits * 4, c))
        return -1;
    if (c->dim[0] <= 1 || s->dim[1] == 0) {
        c->pitch = (c->pitch + 15) / 16 * 16;
        s->pitch = (s->pitch + 15) / 16 * 16;
    }
    if (s->dim[1] > INT_MAX / 32) return refuse("rows", name, codes, d, dev);
    if (((uintptr_t)c->ptr | (uintptr_t)c->pitch) % 16 != 0) return refuse("sixteen", name, codes, d, dev);
    if (((uintptr_t)s->ptr | (uintptr_t)s->pitch) % 16 != 0) return refuse("sixteen", scales_name, scales, t_u8, dev);
    return 0;
}

/* the type of a call's real matrices (0 FP32, 1 bfloat16), taken from one of them */
static int real_type(PyObject *t, const char *name, long dev, PyObject **dtype) {
    if (t == Py_None) return refuse("missing", name, t, NULL, dev);
    PyObject *d = dtype_of(t);
    if (d == NULL) return -1;
    if ((d != t_f32 && d != t_bf16) || dev < 0) return refuse("matrices", name, t, d, dev);
    *dtype = d;
    return d == t_bf16;
}

/* a k x n matrix (below zero: taken from it), row-major (op 0) or a transposed view of a row-major one (1) */
static int stored(PyObject *t, const char *name, PyObject *dtype, long dev, long long k, long long n, Operand *o, int *op) {
    long long s0, s1, least;
    if (dims_of(t, 2, o->dim, name)) return -1;
    if (k < 0) k = o->dim[0];
    if (n < 0) n = o->dim[1];
    if (o->dim[0] != k || o->dim[1] != n) return refuse("shape", name, t, NULL, 0);
    if (data_of(t, name, dtype, dev, o) || strides_of(t, &s0, &s1)) return -1;
    if (n <= 1 || s1 == 1) {
        *op = 0;
        o->pitch = k > 1 ? s0 : n;
        least = n;
    } else if (k <= 1 || s0 == 1) {
        *op = 1;
        o->pitch = s1;
        least = k;
    } else {
        return refuse("transposed", name, t, dtype, dev);
    }
    if (o->pitch < least || o->pitch > INT_MAX || k > INT_MAX || n > INT_MAX) return refuse("rows", name, t, dtype, dev);
    if (o->pitch < 1) o->pitch = 1;
    return 0;
}

/* W, the same; None as of matrix_if */
static int weight(PyObject *t, PyObject *dtype, long dev, long long k, long long n, Operand *o, int *op) {
    if (t != Py_None) return stored(t, "W", dtype, dev, k, n, o, op);
    o->ptr = NULL;
    o->pitch = n > 0 ? n : 1;
    *op = 0;
    return 0;
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

/* fn, dev, stream, X, codes, scales */
typedef int (*Quantize)(int, int, int, int, const void *, int, int, void *, int, void *, int, void *);

static PyObject *mx_quantize(PyObject *self, PyObject *const *a, Py_ssize_t n) {
    (void)self;
    Call c;
    Operand X, codes, scales;
    PyObject *d;
    int bits, op, st;
    if (call_of(a, n, 6, &c)) return NULL;
    const int dtype = real_type(a[3], "X", c.dev, &d);
    if (dtype < 0 || stored(a[3], "X", NULL, c.dev, -1, -1, &X, &op) ||
        coded(a[4], a[5], "codes", "scales", c.dev, X.dim[0], X.dim[1], 0, &codes, &scales, &bits))
        return NULL;
    Py_BEGIN_ALLOW_THREADS
    st = ((Quantize)c.fn)((int)X.dim[0], (int)X.dim[1], dtype, op, X.ptr, (int)X.pitch, bits, codes.ptr, (int)codes.pitch, scales.ptr, (int)scales.pitch, c.stream);
    Py_END_ALLOW_THREADS
    return PyLong_FromLong(st);
}

/* fn, dev, stream, codes, scales, Y */
typedef int (*Dequantize)(int, int, int, int, const void *, int, const void *, int, void *, int, void *);

static PyObject *mx_dequantize(PyObject *self, PyObject *const *a, Py_ssize_t n) {
    (void)self;
    Call c;
    Operand Y, codes, scales;
    PyObject *d;
    int bits, st;
    if (call_of(a, n, 6, &c)) return NULL;
    const int dtype = real_type(a[5], "Y", c.dev, &d);
    if (dtype < 0 || matrix(a[5], "Y", NULL, c.dev, -1, -1, &Y) ||
        coded(a[3], a[4], "codes", "scales", c.dev, Y.dim[0], Y.dim[1], 0, &codes, &scales, &bits))
        return NULL;
    Py_BEGIN_ALLOW_THREADS
    st = ((Dequantize)c.fn)((int)Y.dim[0], (int)Y.dim[1], dtype, bits, codes.ptr, (int)codes.pitch, scales.ptr, (int)scales.pitch, Y.ptr, (int)Y.pitch, c.stream);
    Py_END_ALLOW_THREADS
    return PyLong_FromLong(st);
}

/* fn, dev, stream, X, codes, scales, Y */
typedef int (*Linear)(int, int, int, int, const void *, int, const void *, int, const void *, int, void *, int, void *);

static PyObject *mx4_linear(PyObject *self, PyObject *const *a, Py_ssize_t n) {
    (void)self;
    Call c;
    Operand X, W, ws, Y;
    PyObject *d;
    int bits, st;
    if (call_of(a, n, 7, &c)) return NULL;
    const int dtype = real_type(a[6], "Y", c.dev, &d);
    if (dtype < 0 || matrix(a[3], "X", d, c.dev, -1, -1, &X) || matrix(a[6], "Y", NULL, c.dev, X.dim[0], -1, &Y) ||
        coded(a[4], a[5], "codes", "scales", c.dev, Y.dim[1], X.dim[1], 1, &W, &ws, &bits))
        return NULL;
    Py_BEGIN_ALLOW_THREADS
    st = ((Linear)c.fn)((int)X.dim[0], (int)X.dim[1], (int)Y.dim[1], dtype, X.ptr, (int)X.pitch, W.ptr, (int)W.pitch, ws.ptr, (int)ws.pitch, Y.ptr, (int)Y.pitch, c.stream);
    Py_END_ALLOW_THREADS
    return PyLong_FromLong(st);
}

/* fn, dev, stream, x_codes, x_scales, codes, scales, Y */
typedef int (*Matmul)(int, int, int, int, const void *, int, const void *, int, const void *, int, const void *, int, void *, int, void *);

static PyObject *mx4_matmul(PyObject *self, PyObject *const *a, Py_ssize_t n) {
    (void)self;
    Call c;
    Operand X, xs, W, ws, Y;
    PyObject *d;
    int bits, st;
    if (call_of(a, n, 8, &c)) return NULL;
    const int dtype = real_type(a[7], "Y", c.dev, &d);
    if (dtype < 0 || matrix(a[7], "Y", NULL, c.dev, -1, -1, &Y) || coded(a[3], a[4], "x_codes", "x_scales", c.dev, Y.dim[0], -1, 1, &X, &xs, &bits) ||
        coded(a[5], a[6], "codes", "scales", c.dev, Y.dim[1], xs.dim[1] * 32, 1, &W, &ws, &bits))
        return NULL;
    Py_BEGIN_ALLOW_THREADS
    st = ((Matmul)c.fn)((int)Y.dim[0], (int)(xs.dim[1] * 32), (int)Y.dim[1], dtype, X.ptr, (int)X.pitch, xs.ptr, (int)xs.pitch, W.ptr, (int)W.pitch, ws.ptr,
                        (int)ws.pitch, Y.ptr, (int)Y.pitch, c.stream);
    Py_END_ALLOW_THREADS
    return PyLong_FromLong(st);
}

/* fn, dev, stream, dY, codes, scales, dX */
typedef int (*GradInput)(int, int, int, int, const void *, int, int, const void *, int, const void *, int, void *, int, void *);

static PyObject *mx_grad_input(PyObject *self, PyObject *const *a, Py_ssize_t n) {
    (void)self;
    Call c;
    Operand dY, W, ws, dX;
    PyObject *d;
    int bits, st;
    if (call_of(a, n, 7, &c)) return NULL;
    const int dtype = real_type(a[3], "dY", c.dev, &d);
    if (dtype < 0 || matrix(a[3], "dY", NULL, c.dev, -1, -1, &dY) || matrix(a[6], "dX", d, c.dev, dY.dim[0], -1, &dX) ||
        coded(a[4], a[5], "codes", "scales", c.dev, dY.dim[1], dX.dim[1], 0, &W, &ws, &bits))
        return NULL;
    if (dY.dim[1] > INT_MAX || dX.dim[1] > INT_MAX) {
        refuse("rows", "dY", a[3], d, c.dev);
        return NULL;
    }
    Py_BEGIN_ALLOW_THREADS
    st = ((GradInput)c.fn)((int)dY.dim[0], (int)dX.dim[1], (int)dY.dim[1], dtype, dY.ptr, (int)dY.pitch, bits, W.ptr, (int)W.pitch, ws.ptr, (int)ws.pitch, dX.ptr,
                           (int)dX.pitch, c.stream);
    Py_END_ALLOW_THREADS
    return PyLong_FromLong(st);
}

/* fn, dev, stream, dY, codes, scales, dW, accumulate */
typedef int (*GradWeight)(int, int, int, int, const void *, int, int, const void *, int, const void *, int, int, void *, int, void *);

static PyObject *mx_grad_weight(PyObject *self, PyObject *const *a, Py_ssize_t n) {
    (void)self;
    Call c;
    Operand dY, X, xs, dW;
    PyObject *d;
    int bits, st;
    if (call_of(a, n, 8, &c)) return NULL;
    const int accumulate = PyObject_IsTrue(a[7]);
    if (accumulate < 0) return NULL;
    const int dtype = real_type(a[3], "dY", c.dev, &d);
    if (dtype < 0 || matrix(a[3], "dY", NULL, c.dev, -1, -1, &dY) || matrix(a[6], "dW", d, c.dev, dY.dim[1], -1, &dW) ||
        coded(a[4], a[5], "codes", "scales", c.dev, dY.dim[0], dW.dim[1], 0, &X, &xs, &bits))
        return NULL;
    Py_BEGIN_ALLOW_THREADS
    st = ((GradWeight)c.fn)((int)dY.dim[0], (int)dW.dim[1], (int)dY.dim[1], dtype, dY.ptr, (int)dY.pitch, bits, X.ptr, (int)X.pitch, xs.ptr, (int)xs.pitch,
                            accumulate, dW.ptr, (int)dW.pitch, c.stream);
    Py_END_ALLOW_THREADS
    return PyLong_FromLong(st);
}

/* setup(refuse, float32, bfloat16, float16, int32, uint8, int8) */
static PyObject *setup(PyObject *self, PyObject *args) {
    (void)self;
    PyObject *r, *f32, *bf16, *f16, *i32, *u8, *i8;
    if (!PyArg_ParseTuple(args, "OOOOOOO", &r, &f32, &bf16, &f16, &i32, &u8, &i8)) return NULL;
    PyObject **const to[] = {&g_refuse, &t_f32, &t_bf16, &t_f16, &t_i32, &t_u8, &t_i8};
    PyObject *const from[] = {r, f32, bf16, f16, i32, u8, i8};
    for (int i = 0; i < 7; ++i) {
        Py_INCREF(from[i]);
        Py_XSETREF(*to[i], from[i]);
    }
    Py_RETURN_NONE;
}

static PyMethodDef methods[] = {
    {"setup", setup, METH_VARARGS, "setup(refuse, float32, bfloat16, float16, int32, uint8, int8)"},
    {"lora_forward", (PyCFunction)(void (*)(void))lora_forward, METH_FASTCALL, NULL},
    {"lora_backward", (PyCFunction)(void (*)(void))lora_backward, METH_FASTCALL, NULL},
    {"distill_topk", (PyCFunction)(void (*)(void))distill_topk, METH_FASTCALL, NULL},
    {"mx_quantize", (PyCFunction)(void (*)(void))mx_quantize, METH_FASTCALL, NULL},
    {"mx_dequantize", (PyCFunction)(void (*)(void))mx_dequantize, METH_FASTCALL, NULL},
    {"mx4_linear", (PyCFunction)(void (*)(void))mx4_linear, METH_FASTCALL, NULL},
    {"mx4_matmul", (PyCFunction)(void (*)(void))mx4_matmul, METH_FASTCALL, NULL},
    {"mx_grad_input", (PyCFunction)(void (*)(void))mx_grad_input, METH_FASTCALL, NULL},
    {"mx_grad_weight", (PyCFunction)(void (*)(void))mx_grad_weight, METH_FASTCALL, NULL},
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
