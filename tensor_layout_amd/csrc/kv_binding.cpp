// kv_binding.cpp -- reading of torch tensors for tensor_layout_amd/kv.py.
//
// A call's tensors are looked at and its structures filled here, then the C
// entry point is called: 3.6 to 4 us a call with its launch, against 9 to 11
// through Python's own attributes and ctypes, which is more than the smallest
// calls take on the GPU.  Nothing is judged here: where anything is not as it
// should be the call returns kLook, and kv.py looks for what it is and says
// so.
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <torch/csrc/autograd/python_variable.h>

#include "../../include/tpl_kv.h"

namespace {

typedef int (*AppendFn)(const tpl_kv_cache*, const tpl_kv_batch*, const tpl_kv_new*, hipStream_t);
typedef int (*AttendFn)(const tpl_kv_cache*, const tpl_kv_batch*, const tpl_kv_query*, void*, int64_t, hipStream_t);
typedef int64_t (*WorkspaceFn)(const tpl_kv_cache*, const tpl_kv_batch*, const tpl_kv_query*);

AppendFn g_append = nullptr;
AttendFn g_attend = nullptr;
WorkspaceFn g_workspace = nullptr;

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

// attend(cache, index, q, table, starts, lengths, scale, window, sinks, out, lse, workspace, bytes, stream)
PyObject* attend(PyObject*, PyObject* const* a, Py_ssize_t n) {
    if (n != 14) return PyErr_Format(PyExc_TypeError, "attend takes 14 arguments"), nullptr;
    try {
        const tpl_kv_cache* c = (const tpl_kv_cache*)PyLong_AsVoidPtr(a[0]);
        const int64_t index = PyLong_AsLongLong(a[1]);
        const at::Tensor *q = tensor_of(a[2]), *o = tensor_of(a[9]);
        if (!g_attend || !c || index < 0 || !q || q->dim() != 3 || q->size(1) > INT32_MAX) return PyLong_FromLong(kLook);
        const at::ScalarType type = q->scalar_type();
        const int64_t tokens = q->size(0), heads = q->size(1);
        if ((type != at::kBFloat16 && type != at::kHalf) || !rows(q, type, index, tokens, heads, c->dim) ||
            !rows(o, type, index, tokens, heads, c->dim))
            return PyLong_FromLong(kLook);
        tpl_kv_batch g;
        if (!batch_of(a[3], a[4], a[5], index, tokens, g)) return PyLong_FromLong(kLook);
        tpl_kv_query x = {};
        x.q = q->data_ptr(), x.out = o->data_ptr();
        x.q_token = q->stride(0), x.q_head = q->stride(1), x.o_token = o->stride(0), x.o_head = o->stride(1);
        x.type = type == at::kBFloat16 ? TPL_KV_BF16 : TPL_KV_FP16;
        x.heads = (int32_t)heads;
        x.scale = (float)(a[6] == Py_None ? 1.0 / std::sqrt((double)c->dim) : PyFloat_AsDouble(a[6]));
        const int64_t window = PyLong_AsLongLong(a[7]), sinks = PyLong_AsLongLong(a[8]);
        if (PyErr_Occurred()) return nullptr;
        if (window < INT32_MIN || window > INT32_MAX || sinks < INT32_MIN || sinks > INT32_MAX) return PyLong_FromLong(kLook);
        x.window = (int32_t)window, x.sinks = (int32_t)sinks;
        if (a[10] != Py_None) {
            const at::Tensor* l = tensor_of(a[10]);
            if (!l || l->scalar_type() != at::kFloat || l->dim() != 2 || l->size(0) != tokens || l->size(1) != heads || !on(*l, index))
                return PyLong_FromLong(kLook);
            x.lse = (float*)l->data_ptr();
            x.l_token = l->stride(0), x.l_head = l->stride(1);
        }
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

// bind(append, attend, workspace): the loaded library's entry points.
PyObject* bind(PyObject*, PyObject* const* a, Py_ssize_t n) {
    if (n != 3) return PyErr_Format(PyExc_TypeError, "bind takes 3 arguments"), nullptr;
    g_append = (AppendFn)PyLong_AsVoidPtr(a[0]);
    g_attend = (AttendFn)PyLong_AsVoidPtr(a[1]);
    g_workspace = (WorkspaceFn)PyLong_AsVoidPtr(a[2]);
    if (PyErr_Occurred()) return nullptr;
    Py_RETURN_NONE;
}

PyMethodDef methods[] = {{"append", (PyCFunction)(void*)append, METH_FASTCALL, nullptr},
                         {"attend", (PyCFunction)(void*)attend, METH_FASTCALL, nullptr},
                         {"bind", (PyCFunction)(void*)bind, METH_FASTCALL, nullptr},
                         {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_kv_call", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__kv_call() { return PyModule_Create(&module); }
