// Marshalling of the attention and cache calls from torch tensors to the C ABI
// (include/tilefuse_attention.h), as a Python module.  These calls stand
// between two linears of a decode step and their kernels take 3 to 10 us at
// the smallest sizes, less than checking two dozen attributes and converting
// as many arguments takes in Python: a call through ctypes took the host 10 us,
// one through here takes 4.8, of which the launch is 3.3.
//
// Each function takes its C call's tensors and sizes by position, then the
// output(s) or None, the workspace or None, the stream handle.  It checks what
// the C side cannot see (types, devices, shapes that do not fit each other),
// allocates what is None on the current stream, and returns the output; or a
// number: a tf_status above zero, or minus the bytes of a workspace that is
// needed and was not given.
//
// The GIL is held throughout, as it is over the linears' calls.  Some calls
// launch two kernels that hand over a workspace, which is the stream's and which
// the linears use too: two threads that call on one stream must not get between
// them.
#include <Python.h>

#include <cmath>
#include <string>

#include <ATen/ATen.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include "tilefuse_attention.h"

namespace {

[[noreturn]] void refuse(const char *fn, const std::string &text, PyObject *type = PyExc_ValueError)
{
    PyErr_Format(type, "%s: %s", fn, text.c_str());
    throw python_error();
}

std::string text_of(const at::Tensor &t)
{
    std::string s = std::string("(got ") + c10::toString(t.scalar_type()) + " on " + t.device().str() + ", sizes";
    for (int64_t n : t.sizes())
        s += " " + std::to_string(n);
    s += ", strides";
    for (int64_t n : t.strides())
        s += " " + std::to_string(n);
    return s + ")";
}

// One call: its name, and the device that every tensor of it lies on.
struct Call {
    const char *fn;
    int index = -1;

    const at::Tensor &any(PyObject *o, const char *name) const
    {
        if (!THPVariable_Check(o))
            refuse(fn, std::string(name) + " must be a torch.Tensor", PyExc_TypeError);
        return THPVariable_Unpack(o);
    }
    // the call's first tensor names the device
    const at::Tensor &first(PyObject *o, const char *name)
    {
        const at::Tensor &t = any(o, name);
        if (!t.is_cuda())
            refuse(fn, std::string(name) + " must be a device tensor " + text_of(t));
        index = t.get_device();
        return t;
    }
    const at::Tensor &of(PyObject *o, const char *name, at::ScalarType type, bool contiguous = true) const
    {
        const at::Tensor &t = any(o, name);
        if (t.scalar_type() != type || !t.is_cuda() || t.get_device() != index || (contiguous && !t.is_contiguous()))
            refuse(fn, std::string(name) + " must be a " + (contiguous ? "contiguous " : "") + c10::toString(type) +
                           " tensor on cuda:" + std::to_string(index) + " " + text_of(t));
        return t;
    }
    const at::Tensor &ints(PyObject *o, const char *name) const { return of(o, name, at::kInt); }

    int kind(const at::Tensor &t, const char *name) const
    {
        if (t.scalar_type() == at::kBFloat16)
            return TF_TYPE_BF16;
        if (t.scalar_type() != at::kHalf)
            refuse(fn, std::string(name) + " must be bfloat16 or float16 " + text_of(t));
        return TF_TYPE_F16;
    }
    // the given output, or a new one
    at::Tensor result(PyObject *o, const char *name, at::IntArrayRef sizes, const at::Tensor &like) const
    {
        if (o == Py_None)
            return at::empty(sizes, like.options());
        const at::Tensor &t = of(o, name, like.scalar_type());
        if (t.sizes() != sizes)
            refuse(fn, std::string(name) + " has the wrong shape " + text_of(t));
        return t;
    }
};

int64_t number(PyObject *o)
{
    const Py_ssize_t n = PyNumber_AsSsize_t(o, PyExc_OverflowError);
    if (n == -1 && PyErr_Occurred())
        throw python_error();
    return n;
}

float scale_of(PyObject *o, int64_t d)
{
    if (o == Py_None)
        return (float)(1.0 / std::sqrt((double)d));
    const double s = PyFloat_AsDouble(o);
    if (s == -1.0 && PyErr_Occurred())
        throw python_error();
    return (float)s;
}

void *stream_of(PyObject *o) { return reinterpret_cast<void *>(number(o)); }

const uint16_t *halves(const at::Tensor &t) { return static_cast<const uint16_t *>(t.data_ptr()); }
uint16_t *halves_out(const at::Tensor &t) { return static_cast<uint16_t *>(t.data_ptr()); }
const int32_t *words(const at::Tensor &t) { return static_cast<const int32_t *>(t.data_ptr()); }
int32_t *words_out(const at::Tensor &t) { return static_cast<int32_t *>(t.data_ptr()); }

struct Workspace {
    void *at = nullptr;
    size_t bytes = 0;
    bool missing = false;

    Workspace(const Call &c, PyObject *o, size_t need)
    {
        if (need == 0)
            return;
        missing = o == Py_None;
        if (missing)
            return;
        const at::Tensor &t = c.any(o, "workspace");
        if (!t.is_cuda() || t.get_device() != c.index || !t.is_contiguous())
            refuse(c.fn, "workspace must be a contiguous tensor on cuda:" + std::to_string(c.index) + " " + text_of(t));
        at = t.data_ptr();
        bytes = t.nbytes();
    }
};

// Strides of [tokens][heads][D] with contiguous channels; the stride of an
// axis of one entry means nothing.
struct Strides {
    int64_t token, head;
    Strides(const Call &c, const at::Tensor &t, const char *name)
    {
        if (t.stride(2) != 1 && t.numel() && t.size(2) > 1)
            refuse(c.fn, std::string("the channels of ") + name + " must be contiguous " + text_of(t));
        head = t.size(1) > 1 ? t.stride(1) : t.size(2);
        token = t.size(0) > 1 ? t.stride(0) : t.size(1) * t.size(2);
    }
};

struct Pages {
    const at::Tensor &k, &v, &tables;
    int64_t pages, hkv, page, d, seqs, width;
    Pages(const Call &c, PyObject *k_, PyObject *v_, PyObject *tables_, at::ScalarType type)
        : k(c.of(k_, "k_pages", type)), v(c.of(v_, "v_pages", type)), tables(c.ints(tables_, "tables"))
    {
        if (k.dim() != 4 || k.sizes() != v.sizes() || tables.dim() != 2)
            refuse(c.fn, "k_pages and v_pages must be [pages][Hkv][page][D] of one shape, tables [seqs][width]");
        pages = k.size(0), hkv = k.size(1), page = k.size(2), d = k.size(3);
        seqs = tables.size(0), width = tables.size(1);
    }
};

PyObject *wrong_count(const char *fn)
{
    PyErr_Format(PyExc_TypeError, "%s: wrong number of arguments", fn);
    return nullptr;
}

PyObject *outcome(int status, const at::Tensor &out) { return status == TF_OK ? THPVariable_Wrap(out) : PyLong_FromLong(status); }

// qkv, rope, seq, pos, tables, k_pages, v_pages, hq, q, stream
PyObject *kv_append(PyObject *, PyObject *const *p, Py_ssize_t n)
{
    HANDLE_TH_ERRORS
    Call c{"tf_kv_append"};
    if (n != 10)
        return wrong_count(c.fn);
    const at::Tensor &qkv = c.first(p[0], "qkv");
    const int kind = c.kind(qkv, "qkv");
    const at::Tensor &rope = c.of(p[1], "rope", at::kFloat), &seq = c.ints(p[2], "seq"), &pos = c.ints(p[3], "pos");
    const Pages g(c, p[5], p[6], p[4], qkv.scalar_type());
    const int64_t hq = number(p[7]), tokens = seq.numel(), wide = (hq + 2 * g.hkv) * g.d;
    if (qkv.dim() != 2 || qkv.size(0) != tokens || qkv.size(1) != wide || (qkv.stride(1) != 1 && wide > 1 && tokens))
        refuse(c.fn, "qkv must be [" + std::to_string(tokens) + "][" + std::to_string(wide) + "] with contiguous channels " + text_of(qkv));
    if (pos.numel() != tokens || rope.dim() != 2 || rope.size(1) != g.d)
        refuse(c.fn, "pos must have " + std::to_string(tokens) + " entries, rope must be [positions][" + std::to_string(g.d) + "]");
    const at::Tensor q = c.result(p[8], "q", {tokens, hq, g.d}, qkv);
    void *const stream = stream_of(p[9]);
    const int status = tf_kv_append(kind, halves(qkv), tokens > 1 ? qkv.stride(0) : wide, static_cast<const float *>(rope.data_ptr()),
        rope.size(0), words(seq), words(pos), tokens, words(g.tables), g.seqs, g.width, halves_out(q),
        halves_out(g.k), halves_out(g.v), g.pages, g.page, hq, g.hkv, g.d, stream);
    return outcome(status, q);
    END_HANDLE_TH_ERRORS
}

// q, k_pages, v_pages, tables, lens, longest, scale, out, workspace, stream
PyObject *attn_decode(PyObject *, PyObject *const *p, Py_ssize_t n)
{
    HANDLE_TH_ERRORS
    Call c{"tf_attn_decode"};
    if (n != 10)
        return wrong_count(c.fn);
    const at::Tensor &q = c.first(p[0], "q");
    const int kind = c.kind(q, "q");
    const Pages g(c, p[1], p[2], p[3], q.scalar_type());
    const at::Tensor &lens = c.ints(p[4], "lens");
    if (q.dim() != 3 || q.size(2) != g.d)
        refuse(c.fn, "q must be [seqs][Hq][" + std::to_string(g.d) + "] " + text_of(q));
    const int64_t seqs = q.size(0), hq = q.size(1), longest = number(p[5]);
    if (lens.numel() != seqs || g.seqs != seqs)
        refuse(c.fn, "lens and tables must have " + std::to_string(seqs) + " rows");
    const Strides s(c, q, "q");
    const Workspace ws(c, p[8], tf_attn_decode_workspace_bytes(seqs, hq, g.hkv, g.d, longest));
    if (ws.missing)
        return PyLong_FromLongLong(-(long long)tf_attn_decode_workspace_bytes(seqs, hq, g.hkv, g.d, longest));
    const at::Tensor out = c.result(p[7], "out", {seqs, hq, g.d}, q);
    const float scale = scale_of(p[6], g.d);
    void *const stream = stream_of(p[9]);
    const int status = tf_attn_decode(kind, halves(q), s.token, s.head, halves(g.k), halves(g.v), g.pages, g.page, words(g.tables),
        g.width, words(lens), halves_out(out), seqs, hq, g.hkv, g.d, longest, scale, ws.at, ws.bytes,
        stream);
    return outcome(status, out);
    END_HANDLE_TH_ERRORS
}

// q, k, v, cu_q, cu_k, longest, scale, out, workspace, stream
PyObject *attn_prefill(PyObject *, PyObject *const *p, Py_ssize_t n)
{
    HANDLE_TH_ERRORS
    Call c{"tf_attn_prefill"};
    if (n != 10)
        return wrong_count(c.fn);
    const at::Tensor &q = c.first(p[0], "q");
    const int kind = c.kind(q, "q");
    const at::Tensor &k = c.of(p[1], "k", q.scalar_type(), false), &v = c.of(p[2], "v", q.scalar_type(), false);
    const at::Tensor &cu_q = c.ints(p[3], "cu_q"), &cu_k = c.ints(p[4], "cu_k");
    if (q.dim() != 3 || k.dim() != 3 || k.sizes() != v.sizes() || k.size(2) != q.size(2))
        refuse(c.fn, "q must be [T][Hq][D], k and v [keys][Hkv][D] of one shape");
    const int64_t seqs = cu_q.numel() - 1, tokens = q.size(0), hq = q.size(1), d = q.size(2), keys = k.size(0),
                  hkv = k.size(1), longest = number(p[5]);
    if (seqs < 0 || cu_k.numel() != seqs + 1)
        refuse(c.fn, "cu_q and cu_k must have seqs + 1 entries");
    const Strides sq(c, q, "q"), sk(c, k, "k"), sv(c, v, "v");
    const size_t need = tf_attn_prefill_workspace_bytes(seqs, tokens, hq, hkv, d, longest, keys);
    const Workspace ws(c, p[8], need);
    if (ws.missing)
        return PyLong_FromLongLong(-(long long)need);
    const at::Tensor out = c.result(p[7], "out", {tokens, hq, d}, q);
    const float scale = scale_of(p[6], d);
    void *const stream = stream_of(p[9]);
    const int status = tf_attn_prefill(kind, halves(q), sq.token, sq.head, halves(k), sk.token, sk.head, halves(v), sv.token, sv.head,
        words(cu_q), words(cu_k), halves_out(out), seqs, tokens, keys, hq, hkv, d, longest, scale,
        ws.at, ws.bytes, stream);
    return outcome(status, out);
    END_HANDLE_TH_ERRORS
}

// q, k_pages, v_pages, tables, cu_q, lens, longest, scale, out, workspace, stream
PyObject *attn_prefill_paged(PyObject *, PyObject *const *p, Py_ssize_t n)
{
    HANDLE_TH_ERRORS
    Call c{"tf_attn_prefill_paged"};
    if (n != 11)
        return wrong_count(c.fn);
    const at::Tensor &q = c.first(p[0], "q");
    const int kind = c.kind(q, "q");
    const Pages g(c, p[1], p[2], p[3], q.scalar_type());
    const at::Tensor &cu_q = c.ints(p[4], "cu_q"), &lens = c.ints(p[5], "lens");
    if (q.dim() != 3 || q.size(2) != g.d)
        refuse(c.fn, "q must be [T][Hq][" + std::to_string(g.d) + "] " + text_of(q));
    const int64_t seqs = lens.numel(), tokens = q.size(0), hq = q.size(1), longest = number(p[6]);
    if (cu_q.numel() != seqs + 1 || g.seqs != seqs)
        refuse(c.fn, "cu_q must have " + std::to_string(seqs + 1) + " entries, tables " + std::to_string(seqs) + " rows");
    const Strides s(c, q, "q");
    const size_t need = tf_attn_prefill_workspace_bytes(seqs, tokens, hq, g.hkv, g.d, longest, g.width * g.page);
    const Workspace ws(c, p[9], need);
    if (ws.missing)
        return PyLong_FromLongLong(-(long long)need);
    const at::Tensor out = c.result(p[8], "out", {tokens, hq, g.d}, q);
    const float scale = scale_of(p[7], g.d);
    void *const stream = stream_of(p[10]);
    const int status = tf_attn_prefill_paged(kind, halves(q), s.token, s.head, halves(g.k), halves(g.v), g.pages, g.page,
        words(g.tables), g.width, words(cu_q), words(lens), halves_out(out), seqs, tokens, hq,
        g.hkv, g.d, longest, scale, ws.at, ws.bytes, stream);
    return outcome(status, out);
    END_HANDLE_TH_ERRORS
}

struct Pool {
    const at::Tensor &cache, &refs, &tables;
    Pool(Call &c, PyObject *cache_, PyObject *refs_, PyObject *tables_)
        : cache(c.first(cache_, "cache")), refs(c.ints(refs_, "refs")), tables(c.ints(tables_, "tables"))
    {
        if (cache.dim() != 5 || cache.element_size() != 2 || !cache.is_contiguous())
            refuse(c.fn, "cache must be a contiguous 16-bit tensor [planes][pages][Hkv][page][D] " + text_of(cache));
        if (refs.numel() != cache.size(1) || tables.dim() != 2)
            refuse(c.fn, "refs must have " + std::to_string(cache.size(1)) + " entries, tables must be [seqs][width]");
    }
};

// the given output of an input's shape, or the input itself
const at::Tensor &or_input(const Call &c, PyObject *o, const char *name, const at::Tensor &input)
{
    if (o == Py_None)
        return input;
    const at::Tensor &t = c.ints(o, name);
    if (t.sizes() != input.sizes())
        refuse(c.fn, std::string(name) + " has the wrong shape " + text_of(t));
    return t;
}

// cache, refs, tables, lens, parents, children, refs_out, tables_out, lens_out, status, workspace, stream
PyObject *kv_fork(PyObject *, PyObject *const *p, Py_ssize_t n)
{
    HANDLE_TH_ERRORS
    Call c{"tf_kv_fork"};
    if (n != 12)
        return wrong_count(c.fn);
    const Pool g(c, p[0], p[1], p[2]);
    const at::Tensor &lens = c.ints(p[3], "lens"), &parents = c.ints(p[4], "parents"), &children = c.ints(p[5], "children");
    const int64_t seqs = g.tables.size(0), forks = parents.numel();
    if (lens.numel() != seqs || children.numel() != forks)
        refuse(c.fn, "lens must have " + std::to_string(seqs) + " entries, parents and children equally many");
    const at::Tensor &refs_out = or_input(c, p[6], "refs_out", g.refs), &tables_out = or_input(c, p[7], "tables_out", g.tables),
                     &lens_out = or_input(c, p[8], "lens_out", lens);
    const size_t need = tf_kv_fork_workspace_bytes(forks);
    const Workspace ws(c, p[10], need);
    if (ws.missing)
        return PyLong_FromLongLong(-(long long)need);
    const at::Tensor status = c.result(p[9], "status", {1}, g.refs);
    void *const stream = stream_of(p[11]);
    const int done = tf_kv_fork(halves_out(g.cache), g.cache.size(0), g.cache.size(1), g.cache.size(2), g.cache.size(3),
        g.cache.size(4), words(g.refs), words(g.tables), words(lens), seqs, g.tables.size(1), words(parents),
        words(children), forks, words_out(refs_out), words_out(tables_out), words_out(lens_out),
        words_out(status), ws.at, ws.bytes, stream);
    return outcome(done, status);
    END_HANDLE_TH_ERRORS
}

// cache, refs, tables, refs_out, tables_out, moved, workspace, stream
PyObject *kv_compact(PyObject *, PyObject *const *p, Py_ssize_t n)
{
    HANDLE_TH_ERRORS
    Call c{"tf_kv_compact"};
    if (n != 8)
        return wrong_count(c.fn);
    const Pool g(c, p[0], p[1], p[2]);
    const at::Tensor &refs_out = or_input(c, p[3], "refs_out", g.refs), &tables_out = or_input(c, p[4], "tables_out", g.tables);
    const size_t need = tf_kv_compact_workspace_bytes(g.cache.size(1));
    const Workspace ws(c, p[6], need);
    if (ws.missing)
        return PyLong_FromLongLong(-(long long)need);
    const at::Tensor moved = c.result(p[5], "moved", {g.cache.size(1)}, g.refs);
    void *const stream = stream_of(p[7]);
    const int done = tf_kv_compact(halves_out(g.cache), g.cache.size(0), g.cache.size(1), g.cache.size(2), g.cache.size(3),
        g.cache.size(4), words(g.refs), words(g.tables), g.tables.size(0), g.tables.size(1),
        words_out(refs_out), words_out(tables_out), words_out(moved), ws.at, ws.bytes, stream);
    return outcome(done, moved);
    END_HANDLE_TH_ERRORS
}

#define TF_CALL(name) {#name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)(void)>(name)), METH_FASTCALL, nullptr}
PyMethodDef methods[] = {TF_CALL(kv_append), TF_CALL(attn_decode), TF_CALL(attn_prefill), TF_CALL(attn_prefill_paged),
                         TF_CALL(kv_fork),   TF_CALL(kv_compact),  {nullptr, nullptr, 0, nullptr}};
PyModuleDef module_def = {PyModuleDef_HEAD_INIT, "_calls", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

} // namespace

PyMODINIT_FUNC PyInit__calls() { return PyModule_Create(&module_def); }
