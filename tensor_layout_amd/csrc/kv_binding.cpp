// kv_binding.cpp -- reading of torch tensors for tensor_layout_amd/kv.py and
// linear.py.
//
// A call's tensors are looked at and its structures filled here, then the C
// entry point is called: 3.6 to 4 us a call with its launch, against 9 to 11
// through Python's own attributes and ctypes, which is more than the smallest
// calls take on the GPU.  Nothing is judged here: where anything is not as it
// should be the call returns kLook, and the Python looks for what it is and says
// so.
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <torch/csrc/autograd/python_variable.h>

#include "../../include/tpl_kv.h"
#include "../../include/tpl_linear.h"

namespace {

typedef int (*AppendFn)(const tpl_kv_cache*, const tpl_kv_batch*, const tpl_kv_new*, hipStream_t);
typedef int (*AttendFn)(const tpl_kv_cache*, const tpl_kv_batch*, const tpl_kv_query*, void*, int64_t, hipStream_t);
typedef int64_t (*WorkspaceFn)(const tpl_kv_cache*, const tpl_kv_batch*, const tpl_kv_query*);

typedef int (*SharedFn)(const tpl_kv_cache*, const tpl_kv_batch*, const tpl_kv_groups*, const tpl_kv_query*, void*, int64_t, hipStream_t);
typedef int64_t (*SharedWorkspaceFn)(const tpl_kv_cache*, const tpl_kv_batch*, const tpl_kv_groups*, const tpl_kv_query*);
typedef int (*ReadFn)(const tpl_kv_cache*, const tpl_kv_batch*, const tpl_kv_rows*, hipStream_t);

typedef int (*LinearFn)(const tpl_linear_pool*, const tpl_linear_batch*, const tpl_linear_new*, void*, int64_t, hipStream_t);
typedef int64_t (*LinearWorkspaceFn)(const tpl_linear_pool*, const tpl_linear_batch*, const tpl_linear_new*);

AppendFn g_append = nullptr;
AttendFn g_attend = nullptr;
WorkspaceFn g_workspace = nullptr;
SharedFn g_shared = nullptr;
SharedWorkspaceFn g_shared_workspace = nullptr;
ReadFn g_read = nullptr;
LinearFn g_linear = nullptr;
LinearWorkspaceFn g_linear_workspace = nullptr;

constexpr long kLook = -1;       // something is not right, or not known here
constexpr long kWorkspace = -2;  // the workspace is too small

const at::Tensor* tensor_of(PyObject* o) { return THPVariable_Check(o) ? &THPVariable_Unpack(o) : nullptr; }

bool on(const at::Tensor& t, int64_t index) { return t.is_cuda() && t.get_device() == index; }

// [tokens, heads, dim] of one type with contiguous channels.
bool rows(const at::Tensor* t, at::ScalarType type, int64_t index, int64_t tokens, int64_t heads, int64_t dim) {
    return t && t->scalar_type() == type && t->dim() == 3 && t->size(0) == tokens && t->size(1) == heads && t->size(2) == dim &&
           t->stride(2) == 1 && on(*t, index);
}

bool ints(const at::Tensor* t, int64_t dims, int64_t index) {
    return t && t->scalar_type() == at::kInt && t->dim() == dims && on(*t, index) &&
           (t->size(dims - 1) < 2 || t->stride(dims - 1) == 1);
}

bool batch_of(PyObject* table, PyObject* starts, PyObject* lengths, int64_t index, int64_t tokens, tpl_kv_batch& g) {
    const at::Tensor *t = tensor_of(table), *s = tensor_of(starts), *n = tensor_of(lengths);
    if (!ints(t, 2, index) || !ints(s, 1, index) || !ints(n, 1, index)) return false;
    if (s->size(0) != t->size(0) + 1 || n->size(0) != t->size(0)) return false;
    if (t->size(0) > INT32_MAX || t->size(1) > INT32_MAX || tokens > INT32_MAX) return false;
    g.table = (const int32_t*)t->data_ptr();
    g.starts = (const int32_t*)s->data_ptr();
    g.lengths = (const int32_t*)n->data_ptr();
    g.table_row = t->stride(0);
    g.batch = (int32_t)t->size(0);
    g.width = (int32_t)t->size(1);
    g.tokens = (int32_t)tokens;
    return true;
}

// append(cache, index, k, v, table, starts, lengths, q, q_out, inv_freq, positions, sections, interleaved, stream)
PyObject* append(PyObject*, PyObject* const* a, Py_ssize_t n) {
    if (n != 14) return PyErr_Format(PyExc_TypeError, "append takes 14 arguments"), nullptr;
    try {
        const tpl_kv_cache* c = (const tpl_kv_cache*)PyLong_AsVoidPtr(a[0]);
        const int64_t index = PyLong_AsLongLong(a[1]);
        const at::Tensor *k = tensor_of(a[2]), *v = tensor_of(a[3]);
        if (!g_append || !c || index < 0 || !k || k->dim() != 3) return PyLong_FromLong(kLook);
        const at::ScalarType type = k->scalar_type();
        const int64_t tokens = k->size(0);
        if ((type != at::kBFloat16 && type != at::kHalf) || !rows(k, type, index, tokens, c->kv_heads, c->dim) ||
            !rows(v, type, index, tokens, c->kv_heads, c->dim))
            return PyLong_FromLong(kLook);
        tpl_kv_batch g;
        if (!batch_of(a[4], a[5], a[6], index, tokens, g)) return PyLong_FromLong(kLook);
        tpl_kv_new x = {};
        x.k = k->data_ptr(), x.v = v->data_ptr();
        x.k_token = k->stride(0), x.k_head = k->stride(1), x.v_token = v->stride(0), x.v_head = v->stride(1);
        x.type = type == at::kBFloat16 ? TPL_KV_BF16 : TPL_KV_FP16;
        x.axes = 1;
        if (a[7] != Py_None) {
            const at::Tensor *q = tensor_of(a[7]), *o = tensor_of(a[8]);
            if (!q || q->dim() != 3 || q->size(1) > INT32_MAX || !rows(q, type, index, tokens, q->size(1), c->dim) ||
                !rows(o, type, index, tokens, q->size(1), c->dim))
                return PyLong_FromLong(kLook);
            x.q = q->data_ptr(), x.q_out = o->data_ptr(), x.heads = (int32_t)q->size(1);
            x.q_token = q->stride(0), x.q_head = q->stride(1), x.o_token = o->stride(0), x.o_head = o->stride(1);
        } else if (a[8] != Py_None) {
            return PyLong_FromLong(kLook);
        }
        if (a[9] != Py_None) {
            const at::Tensor* f = tensor_of(a[9]);
            if (!f || f->scalar_type() != at::kFloat || f->dim() != 1 || !on(*f, index) || f->size(0) > 65536 ||
                (f->size(0) > 1 && f->stride(0) != 1))
                return PyLong_FromLong(kLook);
            x.inv_freq = (const float*)f->data_ptr();
            x.rot = 2 * (int32_t)f->size(0);
            const int t = PyObject_IsTrue(a[12]);
            if (t < 0) return nullptr;
            x.interleaved = t;
        }
        if (a[10] != Py_None) {
            const at::Tensor* p = tensor_of(a[10]);
            if (!ints(p, 2, index) || p->size(1) != tokens || p->size(0) < 1 || p->size(0) > TPL_KV_MAX_AXES) return PyLong_FromLong(kLook);
            x.positions = (const int32_t*)p->data_ptr();
            x.positions_row = p->stride(0);
            x.axes = (int32_t)p->size(0);
        }
        if (a[11] != Py_None) {
            if (!PyTuple_Check(a[11]) || PyTuple_GET_SIZE(a[11]) != x.axes || a[9] == Py_None || a[10] == Py_None)
                return PyLong_FromLong(kLook);
            int64_t sum = 0;
            for (int i = 0; i < x.axes; ++i) {
                PyObject* s = PyTuple_GET_ITEM(a[11], i);
                const int64_t e = PyLong_Check(s) ? PyLong_AsLongLong(s) : -1;
                if (e < 0 || e > 65536) {
                    PyErr_Clear();
                    return PyLong_FromLong(kLook);
                }
                x.sections[i] = (int32_t)e;
                sum += e;
            }
            if (sum * 2 != x.rot) return PyLong_FromLong(kLook);
        } else if (x.axes != 1) {
            return PyLong_FromLong(kLook);
        }
        hipStream_t st = (hipStream_t)PyLong_AsVoidPtr(a[13]);
        if (PyErr_Occurred()) return nullptr;
        return PyLong_FromLong(g_append(c, &g, &x, st));
    } catch (const std::exception& e) {
        return PyErr_Format(PyExc_RuntimeError, "%s", e.what()), nullptr;
    }
}

// A query's tensors and numbers; whether all is as it should be.  A Python
// error may be left.
bool query_of(const tpl_kv_cache* c, int64_t index, const at::Tensor* q, PyObject* scale, PyObject* out, PyObject* lse, tpl_kv_query& x) {
    if (!c || index < 0 || !q || q->dim() != 3 || q->size(1) > INT32_MAX) return false;
    const at::Tensor* o = tensor_of(out);
    const at::ScalarType type = q->scalar_type();
    const int64_t tokens = q->size(0), heads = q->size(1);
    if ((type != at::kBFloat16 && type != at::kHalf) || !rows(q, type, index, tokens, heads, c->dim) ||
        !rows(o, type, index, tokens, heads, c->dim))
        return false;
    x.q = q->data_ptr(), x.out = o->data_ptr();
    x.q_token = q->stride(0), x.q_head = q->stride(1), x.o_token = o->stride(0), x.o_head = o->stride(1);
    x.type = type == at::kBFloat16 ? TPL_KV_BF16 : TPL_KV_FP16;
    x.heads = (int32_t)heads;
    x.scale = (float)(scale == Py_None ? 1.0 / std::sqrt((double)c->dim) : PyFloat_AsDouble(scale));
    if (lse != Py_None) {
        const at::Tensor* l = tensor_of(lse);
        if (!l || l->scalar_type() != at::kFloat || l->dim() != 2 || l->size(0) != tokens || l->size(1) != heads || !on(*l, index))
            return false;
        x.lse = (float*)l->data_ptr();
        x.l_token = l->stride(0), x.l_head = l->stride(1);
    }
    return true;
}

// attend(cache, index, q, table, starts, lengths, scale, window, sinks, out, lse, workspace, bytes, stream)
PyObject* attend(PyObject*, PyObject* const* a, Py_ssize_t n) {
    if (n != 14) return PyErr_Format(PyExc_TypeError, "attend takes 14 arguments"), nullptr;
    try {
        const tpl_kv_cache* c = (const tpl_kv_cache*)PyLong_AsVoidPtr(a[0]);
        const int64_t index = PyLong_AsLongLong(a[1]);
        const at::Tensor* q = tensor_of(a[2]);
        tpl_kv_query x = {};
        const bool ok = g_attend && query_of(c, index, q, a[6], a[9], a[10], x);
        if (PyErr_Occurred()) return nullptr;
        tpl_kv_batch g;
        if (!ok || !batch_of(a[3], a[4], a[5], index, q->size(0), g)) return PyLong_FromLong(kLook);
        const int64_t window = PyLong_AsLongLong(a[7]), sinks = PyLong_AsLongLong(a[8]);
        if (PyErr_Occurred()) return nullptr;
        if (window < INT32_MIN || window > INT32_MAX || sinks < INT32_MIN || sinks > INT32_MAX) return PyLong_FromLong(kLook);
        x.window = (int32_t)window, x.sinks = (int32_t)sinks;
        void* ws = PyLong_AsVoidPtr(a[11]);
        const int64_t bytes = PyLong_AsLongLong(a[12]);
        hipStream_t st = (hipStream_t)PyLong_AsVoidPtr(a[13]);
        if (PyErr_Occurred()) return nullptr;
        const int64_t need = g_workspace(c, &g, &x);
        if (need < 0) return PyLong_FromLong(kLook);
        if (need > bytes) return PyLong_FromLong(kWorkspace);
        return PyLong_FromLong(g_attend(c, &g, &x, ws, bytes, st));
    } catch (const std::exception& e) {
        return PyErr_Format(PyExc_RuntimeError, "%s", e.what()), nullptr;
    }
}

// attend_shared(cache, index, q, table, starts, lengths, groups, shared, scale, out, lse, workspace, bytes, stream)
PyObject* attend_shared(PyObject*, PyObject* const* a, Py_ssize_t n) {
    if (n != 14) return PyErr_Format(PyExc_TypeError, "attend_shared takes 14 arguments"), nullptr;
    try {
        const tpl_kv_cache* c = (const tpl_kv_cache*)PyLong_AsVoidPtr(a[0]);
        const int64_t index = PyLong_AsLongLong(a[1]);
        const at::Tensor *q = tensor_of(a[2]), *gs = tensor_of(a[6]), *sh = tensor_of(a[7]);
        tpl_kv_query x = {};
        const bool ok = g_shared && query_of(c, index, q, a[8], a[9], a[10], x);
        if (PyErr_Occurred()) return nullptr;
        tpl_kv_batch g;
        if (!ok || !batch_of(a[3], a[4], a[5], index, q->size(0), g) || !ints(gs, 1, index) || !ints(sh, 1, index) ||
            gs->size(0) != sh->size(0) + 1 || sh->size(0) > INT32_MAX)
            return PyLong_FromLong(kLook);
        const tpl_kv_groups s = {(const int32_t*)gs->data_ptr(), (const int32_t*)sh->data_ptr(), (int32_t)sh->size(0)};
        void* ws = PyLong_AsVoidPtr(a[11]);
        const int64_t bytes = PyLong_AsLongLong(a[12]);
        hipStream_t st = (hipStream_t)PyLong_AsVoidPtr(a[13]);
        if (PyErr_Occurred()) return nullptr;
        const int64_t need = g_shared_workspace(c, &g, &s, &x);
        if (need < 0) return PyLong_FromLong(kLook);
        if (need > bytes) return PyLong_FromLong(kWorkspace);
        return PyLong_FromLong(g_shared(c, &g, &s, &x, ws, bytes, st));
    } catch (const std::exception& e) {
        return PyErr_Format(PyExc_RuntimeError, "%s", e.what()), nullptr;
    }
}

// read(cache, index, table, starts, lengths, k, v, stream)
PyObject* read(PyObject*, PyObject* const* a, Py_ssize_t n) {
    if (n != 8) return PyErr_Format(PyExc_TypeError, "read takes 8 arguments"), nullptr;
    try {
        const tpl_kv_cache* c = (const tpl_kv_cache*)PyLong_AsVoidPtr(a[0]);
        const int64_t index = PyLong_AsLongLong(a[1]);
        const at::Tensor *k = tensor_of(a[5]), *v = tensor_of(a[6]), *some = k ? k : v;
        if (!g_read || !c || index < 0 || !some || some->dim() != 3 || (!k && a[5] != Py_None) || (!v && a[6] != Py_None))
            return PyLong_FromLong(kLook);
        const at::ScalarType type = some->scalar_type();
        const int64_t tokens = some->size(0);
        if ((type != at::kBFloat16 && type != at::kHalf) || (k && !rows(k, type, index, tokens, c->kv_heads, c->dim)) ||
            (v && !rows(v, type, index, tokens, c->kv_heads, c->dim)))
            return PyLong_FromLong(kLook);
        tpl_kv_batch g;
        if (!batch_of(a[2], a[3], a[4], index, tokens, g)) return PyLong_FromLong(kLook);
        tpl_kv_rows x = {};
        if (k) x.k = k->data_ptr(), x.k_token = k->stride(0), x.k_head = k->stride(1);
        if (v) x.v = v->data_ptr(), x.v_token = v->stride(0), x.v_head = v->stride(1);
        x.type = type == at::kBFloat16 ? TPL_KV_BF16 : TPL_KV_FP16;
        hipStream_t st = (hipStream_t)PyLong_AsVoidPtr(a[7]);
        if (PyErr_Occurred()) return nullptr;
        return PyLong_FromLong(g_read(c, &g, &x, st));
    } catch (const std::exception& e) {
        return PyErr_Format(PyExc_RuntimeError, "%s", e.what()), nullptr;
    }
}

// bind: the loaded library's entry points, in the order of kv.py's EXPORTED.
PyObject* bind(PyObject*, PyObject* const* a, Py_ssize_t n) {
    if (n != 6) return PyErr_Format(PyExc_TypeError, "bind takes 6 arguments"), nullptr;
    void* p[6];
    for (int i = 0; i < 6; ++i) p[i] = PyLong_AsVoidPtr(a[i]);
    if (PyErr_Occurred()) return nullptr;
    g_append = (AppendFn)p[0], g_attend = (AttendFn)p[1], g_workspace = (WorkspaceFn)p[2];
    g_shared = (SharedFn)p[3], g_shared_workspace = (SharedWorkspaceFn)p[4], g_read = (ReadFn)p[5];
    Py_RETURN_NONE;
}

// linear_attend(pool, index, q, k, v, slots, starts, sources, scale, out, stream)
PyObject* linear_attend(PyObject*, PyObject* const* a, Py_ssize_t n) {
    if (n != 11) return PyErr_Format(PyExc_TypeError, "linear_attend takes 11 arguments"), nullptr;
    try {
        const tpl_linear_pool* c = (const tpl_linear_pool*)PyLong_AsVoidPtr(a[0]);
        const int64_t index = PyLong_AsLongLong(a[1]);
        const at::Tensor *q = tensor_of(a[2]), *k = tensor_of(a[3]), *v = tensor_of(a[4]), *sl = tensor_of(a[5]), *st = tensor_of(a[6]),
                         *so = tensor_of(a[7]), *o = tensor_of(a[9]);
        if (!g_linear || !c || index < 0 || !q || q->dim() != 3 || q->size(1) > INT32_MAX || (!so && a[7] != Py_None))
            return PyLong_FromLong(kLook);
        const at::ScalarType type = q->scalar_type();
        const int64_t tokens = q->size(0), heads = q->size(1);
        if ((type != at::kBFloat16 && type != at::kHalf) || tokens > INT32_MAX || !rows(q, type, index, tokens, heads, c->key_dim) ||
            !rows(k, type, index, tokens, heads, c->key_dim) || !rows(v, type, index, tokens, c->heads, c->value_dim) ||
            !rows(o, type, index, tokens, c->heads, c->value_dim) || !ints(sl, 1, index) || !ints(st, 1, index) ||
            st->size(0) != sl->size(0) + 1 || sl->size(0) > INT32_MAX || (so && (!ints(so, 1, index) || so->size(0) != sl->size(0))))
            return PyLong_FromLong(kLook);
        const tpl_linear_batch g = {(const int32_t*)sl->data_ptr(), so ? (const int32_t*)so->data_ptr() : nullptr,
                                    (const int32_t*)st->data_ptr(), (int32_t)sl->size(0), (int32_t)tokens};
        tpl_linear_new x = {};
        x.q = q->data_ptr(), x.k = k->data_ptr(), x.v = v->data_ptr(), x.out = o->data_ptr();
        x.q_token = q->stride(0), x.q_head = q->stride(1), x.k_token = k->stride(0), x.k_head = k->stride(1);
        x.v_token = v->stride(0), x.v_head = v->stride(1), x.o_token = o->stride(0), x.o_head = o->stride(1);
        x.scale = (float)(a[8] == Py_None ? 1.0 / std::sqrt((double)c->key_dim) : PyFloat_AsDouble(a[8]));
        x.type = type == at::kBFloat16 ? TPL_KV_BF16 : TPL_KV_FP16;
        x.key_heads = (int32_t)heads;
        hipStream_t stream = (hipStream_t)PyLong_AsVoidPtr(a[10]);
        if (PyErr_Occurred()) return nullptr;
        const int64_t need = g_linear_workspace(c, &g, &x);
        if (need < 0) return PyLong_FromLong(kLook);
        if (need > 0) return PyLong_FromLong(kWorkspace);
        return PyLong_FromLong(g_linear(c, &g, &x, nullptr, 0, stream));
    } catch (const std::exception& e) {
        return PyErr_Format(PyExc_RuntimeError, "%s", e.what()), nullptr;
    }
}

PyObject* bind_linear(PyObject*, PyObject* const* a, Py_ssize_t n) {
    if (n != 2) return PyErr_Format(PyExc_TypeError, "bind_linear takes 2 arguments"), nullptr;
    g_linear = (LinearFn)PyLong_AsVoidPtr(a[0]);
    g_linear_workspace = (LinearWorkspaceFn)PyLong_AsVoidPtr(a[1]);
    if (PyErr_Occurred()) return nullptr;
    Py_RETURN_NONE;
}

PyMethodDef methods[] = {{"append", (PyCFunction)(void*)append, METH_FASTCALL, nullptr},
                         {"attend", (PyCFunction)(void*)attend, METH_FASTCALL, nullptr},
                         {"attend_shared", (PyCFunction)(void*)attend_shared, METH_FASTCALL, nullptr},
                         {"read", (PyCFunction)(void*)read, METH_FASTCALL, nullptr},
                         {"linear_attend", (PyCFunction)(void*)linear_attend, METH_FASTCALL, nullptr},
                         {"bind", (PyCFunction)(void*)bind, METH_FASTCALL, nullptr},
                         {"bind_linear", (PyCFunction)(void*)bind_linear, METH_FASTCALL, nullptr},
                         {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_kv_call", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__kv_call() { return PyModule_Create(&module); }
