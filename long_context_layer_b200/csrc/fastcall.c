/* Calls of the C ABI from Python with little overhead: a bound function takes its arguments positionally,
 * turns each into a machine word and calls the library with the interpreter lock released.  A call with
 * three structs and five words costs about 0.5 us where ctypes with the same checks costs 2.5 us, which
 * is a third of what the smallest layers take from a Python loop.
 *
 * bind(name, address, kinds): kinds has one entry per argument:
 *   "p"    a pointer: None, an int, or an object with data_ptr() (a tensor)
 *   "i"    a 32-bit signed integer
 *   "q"    a 64-bit signed integer (size_t too)
 *   a type a ctypes structure of exactly that type, passed by address
 * The function must take integers and pointers only and return a 32-bit integer. */
#define PY_SSIZE_T_CLEAN
#include <Python.h>
#include <stddef.h>
#include <stdint.h>
#include <string.h>

#define MAX_ARGS 16

typedef struct {
    PyObject_HEAD
    vectorcallfunc vectorcall;
    PyObject* name;
    void* fn;
    Py_ssize_t n;
    char kind[MAX_ARGS];            /* 'p', 'i', 'q' or 's' */
    PyTypeObject* type[MAX_ARGS];   /* of 's' */
} Bound;

static PyObject* str_data_ptr;

static int as_word(PyObject* x, int64_t lo, int64_t hi, int64_t* out) {
    const long long v = PyLong_AsLongLong(x);
    if (v == -1 && PyErr_Occurred()) return -1;
    if (v < lo || v > hi) {
        PyErr_Format(PyExc_OverflowError, "%lld does not fit the argument", v);
        return -1;
    }
    *out = v;
    return 0;
}

static int as_pointer(PyObject* x, int64_t* out) {
    if (x == Py_None) {
        *out = 0;
        return 0;
    }
    PyObject* word = x;
    if (PyLong_Check(x)) {
        Py_INCREF(word);
    } else {
        word = PyObject_CallMethodNoArgs(x, str_data_ptr);
        if (word == NULL) return -1;
    }
    const unsigned long long v = PyLong_AsUnsignedLongLong(word);
    Py_DECREF(word);
    if (v == (unsigned long long)-1 && PyErr_Occurred()) return -1;
    *out = (int64_t)v;
    return 0;
}

static int as_struct(PyObject* x, PyTypeObject* type, int64_t* out) {
    Py_buffer view;
    if (Py_TYPE(x) != type) {
        PyErr_Format(PyExc_TypeError, "expected %s, got %s", type->tp_name, Py_TYPE(x)->tp_name);
        return -1;
    }
    if (PyObject_GetBuffer(x, &view, PyBUF_SIMPLE) != 0) return -1;
    *out = (int64_t)(intptr_t)view.buf;     /* the caller holds x, and with it its memory, during the call */
    PyBuffer_Release(&view);
    return 0;
}

static PyObject* bound_call(PyObject* self, PyObject* const* args, size_t nargsf, PyObject* kwnames) {
    Bound* b = (Bound*)self;
    int64_t a[MAX_ARGS] = {0};
    int32_t status;
    if (PyVectorcall_NARGS(nargsf) != b->n || (kwnames != NULL && PyTuple_GET_SIZE(kwnames) != 0)) {
        PyErr_Format(PyExc_TypeError, "%U takes %zd positional arguments", b->name, b->n);
        return NULL;
    }
    for (Py_ssize_t i = 0; i < b->n; ++i) {
        int bad;
        switch (b->kind[i]) {
            case 'p': bad = as_pointer(args[i], &a[i]); break;
            case 'i': bad = as_word(args[i], INT32_MIN, INT32_MAX, &a[i]); break;
            case 'q': bad = as_word(args[i], INT64_MIN, INT64_MAX, &a[i]); break;
            default: bad = as_struct(args[i], b->type[i], &a[i]); break;
        }
        if (bad) return NULL;
    }
    /* The C calling convention passes integers and pointers of up to 64 bits alike, in registers or in 8-byte
     * stack slots, and leaves words that the function does not take unread. */
    Py_BEGIN_ALLOW_THREADS
    status = ((int32_t(*)(int64_t, int64_t, int64_t, int64_t, int64_t, int64_t, int64_t, int64_t, int64_t, int64_t,
                          int64_t, int64_t, int64_t, int64_t, int64_t, int64_t))b->fn)(
        a[0], a[1], a[2], a[3], a[4], a[5], a[6], a[7], a[8], a[9], a[10], a[11], a[12], a[13], a[14], a[15]);
    Py_END_ALLOW_THREADS
    return PyLong_FromLong(status);
}

static void bound_dealloc(Bound* b) {
    for (Py_ssize_t i = 0; i < b->n; ++i) Py_XDECREF(b->type[i]);
    Py_XDECREF(b->name);
    Py_TYPE(b)->tp_free((PyObject*)b);
}

static PyTypeObject BoundType = {
    PyVarObject_HEAD_INIT(NULL, 0)
    .tp_name = "long_context_layer_b200._fastcall.Bound",
    .tp_basicsize = sizeof(Bound),
    .tp_dealloc = (destructor)bound_dealloc,
    .tp_vectorcall_offset = offsetof(Bound, vectorcall),
    .tp_call = PyVectorcall_Call,
    .tp_flags = Py_TPFLAGS_DEFAULT | Py_TPFLAGS_HAVE_VECTORCALL,
    .tp_doc = "A function of the C ABI (see bind).",
};

static PyObject* bind(PyObject* module, PyObject* args) {
    PyObject *name, *address, *kinds;
    (void)module;
    if (!PyArg_ParseTuple(args, "UOO!", &name, &address, &PyTuple_Type, &kinds)) return NULL;
    const Py_ssize_t n = PyTuple_GET_SIZE(kinds);
    if (n > MAX_ARGS) {
        PyErr_SetString(PyExc_ValueError, "too many arguments");
        return NULL;
    }
    void* fn = PyLong_AsVoidPtr(address);
    if (fn == NULL) {
        if (!PyErr_Occurred()) PyErr_SetString(PyExc_ValueError, "null address");
        return NULL;
    }
    Bound* b = PyObject_New(Bound, &BoundType);
    if (b == NULL) return NULL;
    b->vectorcall = bound_call;
    b->fn = fn;
    b->n = n;
    Py_INCREF(name);
    b->name = name;
    for (Py_ssize_t i = 0; i < MAX_ARGS; ++i) b->type[i] = NULL;
    for (Py_ssize_t i = 0; i < n; ++i) {
        PyObject* k = PyTuple_GET_ITEM(kinds, i);
        if (PyType_Check(k)) {
            b->kind[i] = 's';
            Py_INCREF(k);
            b->type[i] = (PyTypeObject*)k;
        } else if (PyUnicode_Check(k) && PyUnicode_GET_LENGTH(k) == 1 && PyUnicode_READ_CHAR(k, 0) < 128 &&
                   strchr("piq", (int)PyUnicode_READ_CHAR(k, 0)) != NULL) {
            b->kind[i] = (char)PyUnicode_READ_CHAR(k, 0);
        } else {
            Py_DECREF(b);
            PyErr_SetString(PyExc_ValueError, "a kind is 'p', 'i', 'q' or a structure type");
            return NULL;
        }
    }
    return (PyObject*)b;
}

static PyMethodDef methods[] = {
    {"bind", bind, METH_VARARGS, "bind(name, address, kinds): a callable for a function of the C ABI."},
    {NULL, NULL, 0, NULL},
};
static struct PyModuleDef def = {PyModuleDef_HEAD_INIT, "_fastcall", NULL, -1, methods, NULL, NULL, NULL, NULL};

PyMODINIT_FUNC PyInit__fastcall(void) {
    if (PyType_Ready(&BoundType) < 0) return NULL;
    str_data_ptr = PyUnicode_InternFromString("data_ptr");
    if (str_data_ptr == NULL) return NULL;
    return PyModule_Create(&def);
}
