/* binding.c -- a small C extension that calls the library's operator entries
 * (group norm, rows in 8 bits, integer products) from Python.
 *
 * These calls take a few microseconds of GPU time for small inputs, and
 * marshalling 17 to 20 arguments through ctypes took 8 to 9 microseconds of
 * the host's: more than the kernels.  Here a call's arguments are converted in
 * about one.
 *
 * Each function's first argument is the address of the C entry (so the module
 * is not linked to one build of the library), the others are the entry's, in
 * its order.  A pointer argument is None (NULL), an integer address or an
 * object with data_ptr().  The result is the entry's return code.
 */
#define PY_SSIZE_T_CLEAN
#include <Python.h>

static PyObject* data_ptr_name;

/* Every converter leaves a Python error set when it fails, and does nothing when
 * an earlier one has (Python must not be called with an error set, and the first
 * bad argument is the one to name); the callers check once, after the last
 * argument. */
static void* as_ptr(PyObject* o) {
    if (o == Py_None || PyErr_Occurred()) return NULL;
    if (PyLong_Check(o)) return PyLong_AsVoidPtr(o);
    PyObject* r = PyObject_CallMethodNoArgs(o, data_ptr_name);
    if (!r) return NULL;
    void* p = PyLong_AsVoidPtr(r);
    Py_DECREF(r);
    return p;
}

static int as_int(PyObject* o) {
    if (PyErr_Occurred()) return 0;
    const long v = PyLong_AsLong(o);
    if (v != (int)v) {
        if (!PyErr_Occurred()) PyErr_SetString(PyExc_OverflowError, "argument does not fit a C int");
        return 0;
    }
    return (int)v;
}

static size_t as_size(PyObject* o) { return PyErr_Occurred() ? 0 : PyLong_AsSize_t(o); }
static float as_float(PyObject* o) { return PyErr_Occurred() ? 0.0f : (float)PyFloat_AsDouble(o); }

static int arity(const char* name, Py_ssize_t got, Py_ssize_t want) {
    if (got == want) return 1;
    PyErr_Format(PyExc_TypeError, "%s takes %zd arguments, got %zd", name, want, got);
    return 0;
}

#define P(k) void* p##k = as_ptr(a[k])
#define I(k) const int i##k = as_int(a[k])
#define CALL(expr)                      \
    if (PyErr_Occurred()) return NULL;  \
    int rc;                             \
    Py_BEGIN_ALLOW_THREADS              \
    rc = (expr);                        \
    Py_END_ALLOW_THREADS                \
    return PyLong_FromLong(rc)

typedef int (*norm_fn)(void*, void*, void*, void*, void*, void*, void*, size_t, int, int, int, int, int, int, int,
                       float, int, int, void*);

static PyObject* group_norm(PyObject* self, PyObject* const* a, Py_ssize_t n) {
    (void)self;
    if (!arity("group_norm", n, 20)) return NULL;
    P(0); P(1); P(2); P(3); P(4); P(5); P(6); P(7);
    const size_t bytes = as_size(a[8]);
    I(9); I(10); I(11); I(12); I(13); I(14); I(15);
    const float eps = as_float(a[16]);
    I(17); I(18); P(19);
    CALL(((norm_fn)p0)(p1, p2, p3, p4, p5, p6, p7, bytes, i9, i10, i11, i12, i13, i14, i15, eps, i17, i18, p19));
}

typedef int (*quant_fn)(void*, void*, void*, void*, void*, void*, void*, void*, size_t, int, int, int, int, int, int,
                        int, float, int, int, void*);

static PyObject* group_norm_quant(PyObject* self, PyObject* const* a, Py_ssize_t n) {
    (void)self;
    if (!arity("group_norm_quant", n, 21)) return NULL;
    P(0); P(1); P(2); P(3); P(4); P(5); P(6); P(7); P(8);
    const size_t bytes = as_size(a[9]);
    I(10); I(11); I(12); I(13); I(14); I(15); I(16);
    const float eps = as_float(a[17]);
    I(18); I(19); P(20);
    CALL(((quant_fn)p0)(p1, p2, p3, p4, p5, p6, p7, p8, bytes, i10, i11, i12, i13, i14, i15, i16, eps, i18, i19, p20));
}

typedef int (*bwd_fn)(void*, void*, void*, void*, void*, void*, void*, void*, void*, void*, size_t, int, int, int, int,
                      int, int, int, int, int, int, void*);

static PyObject* group_norm_bwd(PyObject* self, PyObject* const* a, Py_ssize_t n) {
    (void)self;
    if (!arity("group_norm_bwd", n, 23)) return NULL;
    P(0); P(1); P(2); P(3); P(4); P(5); P(6); P(7); P(8); P(9); P(10);
    const size_t bytes = as_size(a[11]);
    I(12); I(13); I(14); I(15); I(16); I(17); I(18); I(19); I(20); I(21); P(22);
    CALL(((bwd_fn)p0)(p1, p2, p3, p4, p5, p6, p7, p8, p9, p10, bytes, i12, i13, i14, i15, i16, i17, i18, i19, i20, i21,
                      p22));
}

typedef int (*rows_fn)(void*, void*, void*, int, int, int, int, int, void*);

static PyObject* quantize_rows(PyObject* self, PyObject* const* a, Py_ssize_t n) {
    (void)self;
    if (!arity("quantize_rows", n, 10)) return NULL;
    P(0); P(1); P(2); P(3);
    I(4); I(5); I(6); I(7); I(8); P(9);
    CALL(((rows_fn)p0)(p1, p2, p3, i4, i5, i6, i7, i8, p9));
}

typedef int (*product_fn)(void*, void*, void*, void*, void*, void*, void*, size_t, int, int, int, int, int, int, int,
                          int, void*);

static PyObject* int8_matmul(PyObject* self, PyObject* const* a, Py_ssize_t n) {
    (void)self;
    if (!arity("int8_matmul", n, 18)) return NULL;
    P(0); P(1); P(2); P(3); P(4); P(5); P(6); P(7);
    const size_t bytes = as_size(a[8]);
    I(9); I(10); I(11); I(12); I(13); I(14); I(15); I(16); P(17);
    CALL(((product_fn)p0)(p1, p2, p3, p4, p5, p6, p7, bytes, i9, i10, i11, i12, i13, i14, i15, i16, p17));
}

#define METHOD(name) {#name, (PyCFunction)(void (*)(void))name, METH_FASTCALL, NULL}
static PyMethodDef methods[] = {METHOD(group_norm), METHOD(group_norm_quant), METHOD(group_norm_bwd),
                                METHOD(quantize_rows), METHOD(int8_matmul), {NULL, NULL, 0, NULL}};
static struct PyModuleDef module = {.m_base = PyModuleDef_HEAD_INIT, .m_name = "_binding", .m_size = -1,
                                    .m_methods = methods};

PyMODINIT_FUNC PyInit__binding(void) {
    data_ptr_name = PyUnicode_InternFromString("data_ptr");
    return data_ptr_name ? PyModule_Create(&module) : NULL;
}
