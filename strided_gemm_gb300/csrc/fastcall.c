/* A CPython extension that forwards the product entry points of the C-ABI
 * (sbgemm, sbgemm_ex) and the 16-bit serving operators with their arguments
 * converted straight from Python objects.  Argument marshalling only: the functions it calls are the
 * library's own, whose addresses the Python binding hands over once with
 * bind(), so the library instance is the one the binding loaded.
 *
 * Why: a ctypes call converts each of the twenty arguments through its
 * argtypes, which measured about 2.5 us per call on an Arm server core,
 * more than the library's whole host side (checks, plan, launch: 2 us); a
 * latency-bound product such as a 64 x 48 x 32 one pays that on every
 * launch.  Here the conversion is one PyLong_AsLongLong / PyFloat_AsDouble
 * per argument.
 *
 * Pointers are Python ints (0 or None for NULL), strides and sizes ints (or
 * objects with __index__), alpha a float.  Each call returns the library's
 * status as an int; a bad argument type raises TypeError or OverflowError. */
#define PY_SSIZE_T_CLEAN
#include <Python.h>
#include <stdint.h>
#include <string.h>

#include "sbgemm.h"

typedef int (*ex_fn)(const float*, int64_t, int64_t, int64_t, const float*, int64_t, int64_t, int64_t,
                     float*, int64_t, int64_t, int64_t, int64_t, int64_t, int64_t, int64_t, float, int,
                     void*, const sbgemm_options*);
typedef int (*plain_fn)(const float*, int64_t, int64_t, int64_t, const float*, int64_t, int64_t, int64_t,
                        float*, int64_t, int64_t, int64_t, int64_t, int64_t, int64_t, int64_t, float, int,
                        void*);

static ex_fn g_ex = NULL;
static plain_fn g_plain = NULL;

static int as_ptr(PyObject* o, void** out) {
    if (o == Py_None) {
        *out = NULL;
        return 1;
    }
    *out = PyLong_AsVoidPtr(o);
    return !(*out == NULL && PyErr_Occurred());
}

static int as_i64(PyObject* o, int64_t* out) {
    const long long v = PyLong_AsLongLong(o);
    if (v == -1 && PyErr_Occurred()) return 0;
    *out = (int64_t)v;
    return 1;
}

/* The twelve operand arguments and the four sizes shared by both calls. */
typedef struct {
    void *A, *B, *C;
    int64_t s[9];
    int64_t M, N, K, batch;
    float alpha;
    int accumulate;
    void* stream;
} Call;

static int parse_common(PyObject* const* args, Call* c) {
    void** ptr[3] = {&c->A, &c->B, &c->C};
    for (int op = 0; op < 3; ++op) {
        if (!as_ptr(args[4 * op], ptr[op])) return 0;
        for (int k = 0; k < 3; ++k)
            if (!as_i64(args[4 * op + 1 + k], &c->s[3 * op + k])) return 0;
    }
    if (!as_i64(args[12], &c->M) || !as_i64(args[13], &c->N) || !as_i64(args[14], &c->K) ||
        !as_i64(args[15], &c->batch))
        return 0;
    const double alpha = PyFloat_AsDouble(args[16]);
    if (alpha == -1.0 && PyErr_Occurred()) return 0;
    c->alpha = (float)alpha;
    const int acc = PyObject_IsTrue(args[17]);
    if (acc < 0) return 0;
    c->accumulate = acc;
    return as_ptr(args[18], &c->stream);
}

static PyObject* fc_bind(PyObject* self, PyObject* const* args, Py_ssize_t nargs) {
    (void)self;
    if (nargs != 2) {
        PyErr_SetString(PyExc_TypeError, "bind(sbgemm_ex address, sbgemm address)");
        return NULL;
    }
    void *ex = NULL, *plain = NULL;
    if (!as_ptr(args[0], &ex) || !as_ptr(args[1], &plain)) return NULL;
    g_ex = (ex_fn)ex;
    g_plain = (plain_fn)plain;
    Py_RETURN_NONE;
}

/* sbgemm_ex(A, rsA, csA, bsA, B, rsB, csB, bsB, C, rsC, csC, bsC, M, N, K,
 *           batch, alpha, accumulate, stream, options address) -> status */
static PyObject* fc_sbgemm_ex(PyObject* self, PyObject* const* args, Py_ssize_t nargs) {
    (void)self;
    if (nargs != 20) {
        PyErr_SetString(PyExc_TypeError, "sbgemm_ex takes 20 arguments");
        return NULL;
    }
    if (!g_ex) {
        PyErr_SetString(PyExc_RuntimeError, "the library is not bound");
        return NULL;
    }
    Call c;
    void* opt = NULL;
    if (!parse_common(args, &c) || !as_ptr(args[19], &opt)) return NULL;
    int st;
    Py_BEGIN_ALLOW_THREADS
    st = g_ex((const float*)c.A, c.s[0], c.s[1], c.s[2], (const float*)c.B, c.s[3], c.s[4], c.s[5],
              (float*)c.C, c.s[6], c.s[7], c.s[8], c.M, c.N, c.K, c.batch, c.alpha, c.accumulate,
              c.stream, (const sbgemm_options*)opt);
    Py_END_ALLOW_THREADS
    return PyLong_FromLong(st);
}

/* sbgemm(A, rsA, csA, bsA, B, rsB, csB, bsB, C, rsC, csC, bsC, M, N, K,
 *        batch, alpha, accumulate, stream) -> status */
static PyObject* fc_sbgemm(PyObject* self, PyObject* const* args, Py_ssize_t nargs) {
    (void)self;
    if (nargs != 19) {
        PyErr_SetString(PyExc_TypeError, "sbgemm takes 19 arguments");
        return NULL;
    }
    if (!g_plain) {
        PyErr_SetString(PyExc_RuntimeError, "the library is not bound");
        return NULL;
    }
    Call c;
    if (!parse_common(args, &c)) return NULL;
    int st;
    Py_BEGIN_ALLOW_THREADS
    st = g_plain((const float*)c.A, c.s[0], c.s[1], c.s[2], (const float*)c.B, c.s[3], c.s[4], c.s[5],
                 (float*)c.C, c.s[6], c.s[7], c.s[8], c.M, c.N, c.K, c.batch, c.alpha, c.accumulate,
                 c.stream);
    Py_END_ALLOW_THREADS
    return PyLong_FromLong(st);
}

/* ---- the 16-bit serving operators -------------------------------------------- */

typedef union {
    int64_t i;
    float f;
    void* p;
} Slot;

/* Converts args by `spec`, one letter each: i an integer, p a pointer, f a
 * float, b a truth value. */
static int parse(PyObject* const* args, Py_ssize_t nargs, const char* spec, const char* name, Slot* out) {
    const Py_ssize_t want = (Py_ssize_t)strlen(spec);
    if (nargs != want) {
        PyErr_Format(PyExc_TypeError, "%s takes %zd arguments", name, want);
        return 0;
    }
    for (Py_ssize_t k = 0; k < want; ++k) {
        if (spec[k] == 'i') {
            if (!as_i64(args[k], &out[k].i)) return 0;
        } else if (spec[k] == 'p') {
            if (!as_ptr(args[k], &out[k].p)) return 0;
        } else if (spec[k] == 'b') {
            const int v = PyObject_IsTrue(args[k]);
            if (v < 0) return 0;
            out[k].i = v;
        } else {
            const double v = PyFloat_AsDouble(args[k]);
            if (v == -1.0 && PyErr_Occurred()) return 0;
            out[k].f = (float)v;
        }
    }
    return 1;
}

typedef int (*half_fn)(int, const void*, int64_t, int64_t, int64_t, const void*, int64_t, int64_t, int64_t, void*,
                       int64_t, int64_t, int64_t, int64_t, int64_t, int64_t, int64_t, float, int, void*);
typedef int (*paged_fn)(int, const void*, int64_t, int64_t, int64_t, const void*, int64_t, int64_t, int64_t, int64_t,
                        const int32_t*, int64_t, const int32_t*, void*, int64_t, int64_t, int64_t, int64_t, int64_t,
                        int64_t, int64_t, int64_t, int64_t, float, int, void*, const sbgemm_options*);
typedef int (*packed_fn)(int, const void*, int64_t, int64_t, int64_t, const void*, int64_t, int64_t, const void*,
                         int64_t, const void*, int64_t, int64_t, int64_t, const int32_t*, const int32_t*, int64_t,
                         int64_t, void*, int64_t, int64_t, int64_t, int64_t, int64_t, int64_t, float, int, void*);
typedef int (*copy_fn)(const sbgemm_page_pool*, const int32_t*, int64_t, void*, const sbgemm_options*);
typedef int (*fork_fn)(const sbgemm_page_pool*, const int32_t*, const int32_t*, int64_t, void*, const sbgemm_options*);
typedef int (*append_fn)(const sbgemm_page_pool*, const int32_t*, const int32_t*, int64_t, const void* const*,
                         const int64_t*, int64_t, void*, const sbgemm_options*);
typedef int (*free_fn)(const sbgemm_page_pool*, const int32_t*, int64_t, void*);
typedef int (*compact_fn)(const sbgemm_page_pool*, int32_t*, void*, const sbgemm_options*);

static half_fn g_half = NULL;
static paged_fn g_paged = NULL;
static packed_fn g_packed = NULL;
static copy_fn g_copy = NULL;
static fork_fn g_fork = NULL;
static append_fn g_append = NULL;
static free_fn g_free = NULL;
static compact_fn g_compact = NULL;

/* bind_serving(addresses of sbgemm_half, sbgemm_latent_attention_paged,
 * sbgemm_latent_attention, sbgemm_pages_copy, _fork, _append, _free, _compact) */
static PyObject* fc_bind_serving(PyObject* self, PyObject* const* args, Py_ssize_t nargs) {
    (void)self;
    Slot a[8];
    if (!parse(args, nargs, "pppppppp", "bind_serving", a)) return NULL;
    g_half = (half_fn)a[0].p;
    g_paged = (paged_fn)a[1].p;
    g_packed = (packed_fn)a[2].p;
    g_copy = (copy_fn)a[3].p;
    g_fork = (fork_fn)a[4].p;
    g_append = (append_fn)a[5].p;
    g_free = (free_fn)a[6].p;
    g_compact = (compact_fn)a[7].p;
    Py_RETURN_NONE;
}

static PyObject* not_bound(void) {
    PyErr_SetString(PyExc_RuntimeError, "the library is not bound");
    return NULL;
}

/* The C arguments of sbgemm_half in order. */
static PyObject* fc_half(PyObject* self, PyObject* const* args, Py_ssize_t nargs) {
    (void)self;
    Slot a[20];
    int st;
    if (!g_half) return not_bound();
    if (!parse(args, nargs, "ipiiipiiipiiiiiiifbp", "sbgemm_half", a)) return NULL;
    Py_BEGIN_ALLOW_THREADS
    st = g_half((int)a[0].i, a[1].p, a[2].i, a[3].i, a[4].i, a[5].p, a[6].i, a[7].i, a[8].i, a[9].p, a[10].i, a[11].i,
                a[12].i, a[13].i, a[14].i, a[15].i, a[16].i, a[17].f, (int)a[18].i, a[19].p);
    Py_END_ALLOW_THREADS
    return PyLong_FromLong(st);
}

/* The C arguments of sbgemm_latent_attention_paged in order (the options by address). */
static PyObject* fc_paged(PyObject* self, PyObject* const* args, Py_ssize_t nargs) {
    (void)self;
    Slot a[27];
    int st;
    if (!g_paged) return not_bound();
    if (!parse(args, nargs, "ipiiipiiiipippiiiiiiiiifipp", "sbgemm_latent_attention_paged", a)) return NULL;
    Py_BEGIN_ALLOW_THREADS
    st = g_paged((int)a[0].i, a[1].p, a[2].i, a[3].i, a[4].i, a[5].p, a[6].i, a[7].i, a[8].i, a[9].i,
                 (const int32_t*)a[10].p, a[11].i, (const int32_t*)a[12].p, a[13].p, a[14].i, a[15].i, a[16].i,
                 a[17].i, a[18].i, a[19].i, a[20].i, a[21].i, a[22].i, a[23].f, (int)a[24].i, a[25].p,
                 (const sbgemm_options*)a[26].p);
    Py_END_ALLOW_THREADS
    return PyLong_FromLong(st);
}

/* The C arguments of sbgemm_latent_attention in order. */
static PyObject* fc_packed(PyObject* self, PyObject* const* args, Py_ssize_t nargs) {
    (void)self;
    Slot a[28];
    int st;
    if (!g_packed) return not_bound();
    if (!parse(args, nargs, "ipiiipiipipiiippiipiiiiiifip", "sbgemm_latent_attention", a)) return NULL;
    Py_BEGIN_ALLOW_THREADS
    st = g_packed((int)a[0].i, a[1].p, a[2].i, a[3].i, a[4].i, a[5].p, a[6].i, a[7].i, a[8].p, a[9].i, a[10].p,
                  a[11].i, a[12].i, a[13].i, (const int32_t*)a[14].p, (const int32_t*)a[15].p, a[16].i, a[17].i,
                  a[18].p, a[19].i, a[20].i, a[21].i, a[22].i, a[23].i, a[24].i, a[25].f, (int)a[26].i, a[27].p);
    Py_END_ALLOW_THREADS
    return PyLong_FromLong(st);
}

/* A tuple of n pointers or integers; -1 with an error set, else n. */
static Py_ssize_t tuple_of(PyObject* t, int pointers, void** p, int64_t* v) {
    if (!PyTuple_Check(t) || PyTuple_GET_SIZE(t) > SBGEMM_MAX_CACHES) {
        PyErr_SetString(PyExc_TypeError, "a tuple of at most SBGEMM_MAX_CACHES entries is wanted");
        return -1;
    }
    const Py_ssize_t n = PyTuple_GET_SIZE(t);
    for (Py_ssize_t k = 0; k < n; ++k)
        if (pointers ? !as_ptr(PyTuple_GET_ITEM(t, k), &p[k]) : !as_i64(PyTuple_GET_ITEM(t, k), &v[k])) return -1;
    return n;
}

/* pages(op, caches, page_bytes, num_blocks, block_size, ref_counts,
 *       block_table, n_seqs, max_blocks, seq_lens, a, b, n, rows, row_strides,
 *       total, stream, options address) -> status
 * op: 0 copy (a = pairs), 1 fork (a = parents, b = children), 2 append (a =
 * sequences, b = starts, rows), 3 free (a = sequences), 4 compact (a = moved). */
static PyObject* fc_pages(PyObject* self, PyObject* const* args, Py_ssize_t nargs) {
    (void)self;
    if (!g_copy) return not_bound();
    if (nargs != 18) {
        PyErr_SetString(PyExc_TypeError, "pages takes 18 arguments");
        return NULL;
    }
    void *caches[SBGEMM_MAX_CACHES], *rows[SBGEMM_MAX_CACHES];
    int64_t bytes[SBGEMM_MAX_CACHES], strides[SBGEMM_MAX_CACHES];
    Slot op, a[10], e[3];
    sbgemm_page_pool pool;
    int st = SBGEMM_ERR_INVALID_VALUE;
    if (!as_i64(args[0], &op.i)) return NULL;
    const Py_ssize_t n = tuple_of(args[1], 1, caches, NULL);
    if (n < 0 || tuple_of(args[2], 0, NULL, bytes) != n || !parse(args + 3, 10, "iippiipppi", "pages", a) ||
        !parse(args + 15, 3, "ipp", "pages", e)) {
        if (!PyErr_Occurred()) PyErr_SetString(PyExc_TypeError, "caches and page_bytes differ in length");
        return NULL;
    }
    const Py_ssize_t r = tuple_of(args[13], 1, rows, NULL);
    if (r < 0) return NULL;
    if (tuple_of(args[14], 0, NULL, strides) != r || (op.i == 2 && r != n)) {
        if (!PyErr_Occurred()) PyErr_SetString(PyExc_TypeError, "rows and row_strides need one entry a cache");
        return NULL;
    }
    memset(&pool, 0, sizeof(pool));
    pool.caches = caches;
    pool.page_bytes = bytes;
    pool.n_caches = n;
    pool.num_blocks = a[0].i;
    pool.block_size = a[1].i;
    pool.ref_counts = (int32_t*)a[2].p;
    pool.block_table = (int32_t*)a[3].p;
    pool.n_seqs = a[4].i;
    pool.max_blocks = a[5].i;
    pool.seq_lens = (int32_t*)a[6].p;
    const sbgemm_options* opt = (const sbgemm_options*)e[2].p;
    int32_t *x = (int32_t*)a[7].p, *y = (int32_t*)a[8].p;
    Py_BEGIN_ALLOW_THREADS
    switch (op.i) {
        case 0: st = g_copy(&pool, x, a[9].i, e[1].p, opt); break;
        case 1: st = g_fork(&pool, x, y, a[9].i, e[1].p, opt); break;
        case 2:
            st = g_append(&pool, x, y, a[9].i, (const void* const*)rows, strides, e[0].i, e[1].p, opt);
            break;
        case 3: st = g_free(&pool, x, a[9].i, e[1].p); break;
        case 4: st = g_compact(&pool, x, e[1].p, opt); break;
        default: break;
    }
    Py_END_ALLOW_THREADS
    return PyLong_FromLong(st);
}

static PyMethodDef kMethods[] = {
    {"bind", (PyCFunction)(void (*)(void))fc_bind, METH_FASTCALL, "bind the library's entry points"},
    {"sbgemm_ex", (PyCFunction)(void (*)(void))fc_sbgemm_ex, METH_FASTCALL, "sbgemm_ex; returns the status"},
    {"sbgemm", (PyCFunction)(void (*)(void))fc_sbgemm, METH_FASTCALL, "sbgemm; returns the status"},
    {"bind_serving", (PyCFunction)(void (*)(void))fc_bind_serving, METH_FASTCALL, "bind the serving entry points"},
    {"half", (PyCFunction)(void (*)(void))fc_half, METH_FASTCALL, "sbgemm_half; returns the status"},
    {"paged", (PyCFunction)(void (*)(void))fc_paged, METH_FASTCALL, "sbgemm_latent_attention_paged; returns the status"},
    {"packed", (PyCFunction)(void (*)(void))fc_packed, METH_FASTCALL, "sbgemm_latent_attention; returns the status"},
    {"pages", (PyCFunction)(void (*)(void))fc_pages, METH_FASTCALL, "sbgemm_pages_*; returns the status"},
    {NULL, NULL, 0, NULL},
};

static struct PyModuleDef kModule = {PyModuleDef_HEAD_INIT, "_fastcall", NULL, -1, kMethods,
                                     NULL, NULL, NULL, NULL};

PyMODINIT_FUNC PyInit__fastcall(void) { return PyModule_Create(&kModule); }
