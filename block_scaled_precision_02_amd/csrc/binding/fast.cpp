// fast.cpp -- the ordinary calls of the expert operators without the
// interpreter between their checks.
//
// Between the GEMMs of a decode step the host's time is the step's.  A call
// through Python and ctypes spends 4 to 8 us on reading attributes, allocating and
// converting beside the 2 us of the launch itself; here the same checks read the
// tensors directly (us a call on one MI355X's host: sort of 64 x 8 choices 10.3 ->
// 5.9, gather and combine of 64 tokens together 15.2 -> 8.4, SwiGLU into given
// memory 7.7 -> 4.6, norm of one token with three results 13.4 -> 7.3).
//
// Every function takes the address of its C entry point and the caller's
// arguments.  It does the whole call and returns its result, or does nothing and
// returns None: where anything about the arguments is out of the ordinary
// (another type, layout, device or shape than the common one, or wrong) or the
// entry point refuses them.  The Python function then goes its full way, which says
// what is wrong.  What is taken here is a subset of what is taken there, with the
// same result.  A device or launch error is raised here: part of the call may be
// on the stream, and it must not be made again.  The entry points are called by
// their prototypes in the library's header.
#include <Python.h>

#include <ATen/ATen.h>
#include <torch/csrc/autograd/python_variable.h>

#include <cstdint>
#include <cstring>

#include "../../../include/qgemm.h"

namespace {

// An address of what a checked tensor holds, as any pointer that a prototype names.
struct Address {
    void *p;
    Address(void *p = nullptr) : p(p) {}
    template <class T> operator T *() const { return (T *)p; }
};

PyObject *g_get_device, *g_get_stream;   // torch._C._cuda_getDevice, _cuda_getCurrentRawStream
PyObject *g_check;                       // raises what a status stands for

// Leaves the function: the full way decides.
struct Decline {};

// Leaves the function: the call failed with this status.
struct Failed {
    int status;
};

void need(bool ok)
{
    if (!ok)
        throw Decline();
}

int64_t whole(PyObject *o)
{
    const long long v = PyLong_AsLongLong(o);
    need(!(v == -1 && PyErr_Occurred()));
    return v;
}

double real(PyObject *o)
{
    const double v = PyFloat_AsDouble(o);
    need(!(v == -1.0 && PyErr_Occurred()));
    return v;
}

const at::Tensor &tensor(PyObject *o)
{
    need(THPVariable_Check(o));
    const at::Tensor &t = THPVariable_Unpack(o);
    need(t.defined() && t.is_cuda() && t.layout() == at::kStrided);
    return t;
}

// The device all of a call's tensors are on, which has to be the current one,
// and its current stream.
struct Place {
    c10::Device device;
    void *stream;

    explicit Place(const at::Tensor &t) : device(t.device()), stream(nullptr)
    {
        PyObject *d = PyObject_CallNoArgs(g_get_device);
        need(d);
        const int64_t current = whole(d);
        Py_DECREF(d);
        need(current == device.index());
        PyObject *i = PyLong_FromLong((long)device.index());
        PyObject *s = i ? PyObject_CallOneArg(g_get_stream, i) : nullptr;
        Py_XDECREF(i);
        need(s);
        stream = PyLong_AsVoidPtr(s);
        Py_DECREF(s);
        need(!PyErr_Occurred());
    }
};

// A contiguous tensor of n elements.
Address flat(PyObject *o, const Place &p, at::ScalarType dtype, int64_t n)
{
    const at::Tensor &t = tensor(o);
    need(t.scalar_type() == dtype && t.device() == p.device && t.numel() == n && t.is_contiguous());
    return t.data_ptr();
}

// A matrix with unit stride along its rows.
struct Rows {
    int64_t rows, cols, ld;
    Address data;
};

Rows rows_of(const at::Tensor &t, const Place &p)
{
    need(t.dim() == 2 && t.device() == p.device && (t.size(1) <= 1 || t.stride(1) == 1));
    return {t.size(0), t.size(1), t.size(0) > 1 ? t.stride(0) : t.size(1), t.data_ptr()};
}

Rows rows_of(PyObject *o, const Place &p, at::ScalarType dtype)
{
    const at::Tensor &t = tensor(o);
    need(t.scalar_type() == dtype);
    return rows_of(t, p);
}

Rows rows_of(PyObject *o, const Place &p, at::ScalarType dtype, int64_t rows, int64_t cols)
{
    const Rows r = rows_of(o, p, dtype);
    need(r.rows == rows && r.cols == cols);
    return r;
}

at::Tensor fresh(at::IntArrayRef shape, at::ScalarType dtype, const Place &p)
{
    return at::empty(shape, at::TensorOptions().dtype(dtype).device(p.device));
}

// The caller's output or a new one: [rows, cols], and the object to return.
struct Out {
    Rows r;
    at::Tensor made;
    PyObject *given;

    PyObject *object() const
    {
        if (!given)
            return THPVariable_Wrap(made);
        Py_INCREF(given);
        return given;
    }
};

Out out_rows(PyObject *o, const Place &p, at::ScalarType dtype, int64_t rows, int64_t cols)
{
    if (o != Py_None)
        return {rows_of(o, p, dtype, rows, cols), {}, o};
    at::Tensor t = fresh({rows, cols}, dtype, p);
    return {{rows, cols, cols, t.data_ptr()}, t, nullptr};
}

// Codes (row: bytes of a row) as the quantisers' out argument.
Out out_codes(PyObject *o, const Place &p, bool i8, int64_t rows, int64_t row)
{
    if (o == Py_None) {
        need(row % 16 == 0);
        return out_rows(o, p, i8 ? at::kChar : at::kByte, rows, row);
    }
    const at::Tensor &t = tensor(o);
    need(i8 ? t.scalar_type() == at::kChar
            : t.scalar_type() == at::kByte || t.scalar_type() == at::kFloat8_e4m3fn);
    Rows r = rows_of(t, p);
    need(r.rows == rows && r.cols == row);
    if (rows <= 1)
        r.ld = row + (16 - row % 16) % 16;
    return {r, {}, o};
}

// Scales: one a row (part 0), or one for each part elements.
Out out_scales(PyObject *o, const Place &p, at::ScalarType dtype, int64_t rows, int64_t cols, int64_t part)
{
    if (part)
        return out_rows(o, p, dtype, rows, cols / part);
    if (o != Py_None)
        return {{rows, 1, 1, flat(o, p, dtype, rows)}, {}, o};
    at::Tensor t = fresh({rows}, dtype, p);
    return {{rows, 1, 1, t.data_ptr()}, t, nullptr};
}

// The entry point at an address, by its prototype.
template <class F, class... A>
auto enter(void *entry, A... a)
{
    return ((F *)entry)(a...);
}

// ran: whether the call was made, after which there is no way back.  Refused
// arguments (status 1 to 4) leave nothing on the stream.
template <class F, class... A>
void enqueue(bool &ran, void *entry, A... a)
{
    qgemm_status status;
    Py_BEGIN_ALLOW_THREADS
    status = enter<F>(entry, a...);
    Py_END_ALLOW_THREADS
    need(status < QGEMM_ERR_NULL_POINTER || status > QGEMM_ERR_BAD_FORMAT);
    if (status != QGEMM_OK)
        throw Failed{status};
    ran = true;
}

// A prototype as a value.
template <class T> struct Type {
    using F = T;
};

void *entry_of(PyObject *o)
{
    void *f = PyLong_AsVoidPtr(o);
    need(f && !PyErr_Occurred());
    return f;
}

PyObject *pack(std::initializer_list<PyObject *> items)
{
    PyObject *t = PyTuple_New((Py_ssize_t)items.size());
    Py_ssize_t i = 0;
    for (PyObject *o : items) {
        if (t)
            PyTuple_SET_ITEM(t, i++, o);
        else
            Py_XDECREF(o);
    }
    return t;
}

// f(ran), or None where the call was not made; raises where it failed.
template <class F>
PyObject *attempt(Py_ssize_t got, Py_ssize_t want, F &&f)
{
    bool ran = false;
    if (got == want) {
        PyObject *r = nullptr;
        try {
            r = f(ran);
        } catch (const Failed &e) {
            PyObject *none = PyObject_CallFunction(g_check, "i", e.status);
            if (none)
                PyErr_Format(PyExc_RuntimeError, "the call failed with status %d", e.status);
            Py_XDECREF(none);
            return nullptr;
        } catch (...) {
        }
        if (r)
            return r;
        if (ran) {
            if (!PyErr_Occurred())
                PyErr_SetString(PyExc_MemoryError, "the result could not be returned");
            return nullptr;
        }
        PyErr_Clear();
    }
    Py_RETURN_NONE;
}

using P = Address;
using I = int64_t;

// entry, workspace's entry, ids, experts
PyObject *moe_sort(PyObject *, PyObject *const *a, Py_ssize_t n)
{
    return attempt(n, 4, [&](bool &ran) -> PyObject * {
        const at::Tensor &ids = tensor(a[2]);
        const Place p(ids);
        need(ids.scalar_type() == at::kInt && ids.dim() == 2 && ids.is_contiguous() && PyLong_CheckExact(a[3]));
        const I tokens = ids.size(0), k = ids.size(1), experts = whole(a[3]);
        need(experts >= 1 && experts <= 1024);
        const I bytes = enter<decltype(qgemm_moe_sort_workspace)>(entry_of(a[1]), tokens, k, experts);
        need(bytes >= 0);
        at::Tensor offsets = fresh({experts + 1}, at::kInt, p), order = fresh({tokens * k}, at::kInt, p),
                   position = fresh({tokens, k}, at::kInt, p), ws;
        if (bytes > 0)
            ws = fresh({bytes}, at::kByte, p);
        enqueue<decltype(qgemm_moe_sort)>(ran, entry_of(a[0]), P(ids.data_ptr()), tokens, k, experts, P(offsets.data_ptr()),
                                          P(order.data_ptr()), P(position.data_ptr()),
                                          P(bytes > 0 ? ws.data_ptr() : nullptr), bytes, p.stream);
        return pack({THPVariable_Wrap(offsets), THPVariable_Wrap(order), THPVariable_Wrap(position)});
    });
}

struct Choices {
    I tokens, k;
    P data;
    explicit Choices(const at::Tensor &t) : tokens(0), k(0), data(nullptr)
    {
        need(t.scalar_type() == at::kInt && t.dim() == 2 && t.is_contiguous());
        tokens = t.size(0);
        k = t.size(1);
        data = t.data_ptr();
    }
};

// One value for each choice: [tokens, top_k].
Address per_choice(PyObject *o, const Place &p, const Choices &c)
{
    const at::Tensor &t = tensor(o);
    need(t.dim() == 2 && t.size(0) == c.tokens && t.size(1) == c.k);
    return flat(o, p, at::kFloat, c.tokens * c.k);
}

// entry, X, position, rows, out
PyObject *moe_gather(PyObject *, PyObject *const *a, Py_ssize_t n)
{
    return attempt(n, 5, [&](bool &ran) -> PyObject * {
        const at::Tensor &position = tensor(a[2]);
        const Place p(position);
        const Choices c(position);
        const Rows x = rows_of(a[1], p, at::kBFloat16);
        need(x.rows == c.tokens);
        I rows = c.tokens * c.k;
        if (a[3] != Py_None)
            rows = whole(a[3]);
        else if (a[4] != Py_None)
            rows = rows_of(a[4], p, at::kBFloat16).rows;
        need(rows >= 0 && rows < (I)1 << 31);
        const Out y = out_rows(a[4], p, at::kBFloat16, rows, x.cols);
        enqueue<decltype(qgemm_moe_gather)>(ran, entry_of(a[0]), x.data, x.ld, c.data, y.r.data, y.r.ld, c.tokens, c.k, rows,
                                            x.cols, p.stream);
        return y.object();
    });
}

// entry, Y, position, weights, residual, out
PyObject *moe_combine(PyObject *, PyObject *const *a, Py_ssize_t n)
{
    return attempt(n, 6, [&](bool &ran) -> PyObject * {
        const at::Tensor &position = tensor(a[2]);
        const Place p(position);
        const Choices c(position);
        const Rows y = rows_of(a[1], p, at::kBFloat16);
        P w = nullptr;
        if (a[3] != Py_None)
            w = per_choice(a[3], p, c);
        Rows r = {0, 0, 0, nullptr};
        if (a[4] != Py_None)
            r = rows_of(a[4], p, at::kBFloat16, c.tokens, y.cols);
        const Out o = out_rows(a[5], p, at::kBFloat16, c.tokens, y.cols);
        enqueue<decltype(qgemm_moe_combine)>(ran, entry_of(a[0]), y.data, y.ld, c.data, w, r.data, r.ld, o.r.data, o.r.ld,
                                             c.tokens, c.k, y.rows, y.cols, p.stream);
        return o.object();
    });
}

// entry, dout, Y, position, weights, dY, dweights
PyObject *moe_combine_grad(PyObject *, PyObject *const *a, Py_ssize_t n)
{
    return attempt(n, 7, [&](bool &ran) -> PyObject * {
        const at::Tensor &position = tensor(a[3]);
        const Place p(position);
        const Choices c(position);
        const Rows y = rows_of(a[2], p, at::kBFloat16), d = rows_of(a[1], p, at::kBFloat16, c.tokens, y.cols);
        P w = per_choice(a[4], p, c);
        const Out dy = out_rows(a[5], p, at::kBFloat16, y.rows, y.cols);
        Out dw = {};
        if (a[6] == Py_None) {
            dw = out_rows(a[6], p, at::kFloat, c.tokens, c.k);
        } else {
            dw.r.data = per_choice(a[6], p, c);
            dw.given = a[6];
        }
        enqueue<decltype(qgemm_moe_combine_grad)>(ran, entry_of(a[0]), d.data, d.ld, y.data, y.ld, c.data, w, dy.r.data,
                                                  dy.r.ld, dw.r.data, c.tokens, c.k, y.rows, y.cols, p.stream);
        return pack({dy.object(), dw.object()});
    });
}

// The kind of a quantised output: MX element format or -1, codes a byte,
// elements a scale covers (0: the row), int8 codes, ue8m0 scales.
struct Quant {
    int fmt;
    I per_byte, part;
    bool i8, ue8m0;
    explicit Quant(PyObject *const *a)
        : fmt((int)whole(a[0])), per_byte(whole(a[1])), part(whole(a[2])), i8(whole(a[3]) != 0), ue8m0(whole(a[4]) != 0)
    {
    }
    at::ScalarType scale_type() const { return ue8m0 ? at::kByte : at::kFloat; }
};

// entry, the five of Quant, X, count, out, scale
PyObject *swiglu(PyObject *, PyObject *const *a, Py_ssize_t n)
{
    return attempt(n, 10, [&](bool &ran) -> PyObject * {
        const Quant q(a + 1);
        const at::Tensor &xt = tensor(a[6]);
        const Place p(xt);
        const Rows x = rows_of(a[6], p, at::kBFloat16);
        const I M = x.rows, I2 = x.cols / 2;
        need(x.cols % 2 == 0 && I2 > 0 && I2 % (q.part ? q.part : 32) == 0);
        P count = nullptr;
        if (a[7] != Py_None)
            count = flat(a[7], p, at::kInt, 1);
        const Out o = out_codes(a[8], p, q.i8, M, I2 / q.per_byte);
        const Out s = out_scales(a[9], p, q.scale_type(), M, I2, q.part);
        void *f = entry_of(a[0]);
        auto rows = [&](auto type) {                     // one scale a row
            enqueue<typename decltype(type)::F>(ran, f, x.data, x.ld, count, o.r.data, o.r.ld, s.r.data, M, I2, p.stream);
        };
        if (q.fmt >= 0)
            enqueue<decltype(qgemm_swiglu_quant_mx)>(ran, f, (qgemm_mx_fmt)q.fmt, x.data, x.ld, count, o.r.data, o.r.ld,
                                                     s.r.data, s.r.ld, M, I2, p.stream);
        else if (q.part)
            enqueue<decltype(qgemm_swiglu_quant_f8_block)>(ran, f, x.data, x.ld, count, o.r.data, o.r.ld, s.r.data, s.r.ld,
                                                           M, I2, p.stream);
        else if (q.i8)
            rows(Type<decltype(qgemm_swiglu_quant_i8_rowwise)>());
        else
            rows(Type<decltype(qgemm_swiglu_quant_f8_pertoken)>());
        return pack({o.object(), s.object()});
    });
}

// entry, the five of Quant, Y, residual, gamma_post, gamma, eps, gate, alpha,
// residual_out, out, scale
PyObject *postnorm(PyObject *, PyObject *const *a, Py_ssize_t n)
{
    return attempt(n, 16, [&](bool &ran) -> PyObject * {
        const Quant q(a + 1);
        const at::Tensor &yt = tensor(a[6]);
        const Place p(yt);
        const Rows y = rows_of(a[6], p, at::kBFloat16);
        const I M = y.rows, K = y.cols;
        need(K > 0 && K % (q.part ? q.part : 32) == 0);
        const Rows r = rows_of(a[7], p, at::kBFloat16, M, K);
        qgemm_postnorm v = {};
        v.Y = y.data;
        v.R = r.data;
        v.gamma_post = flat(a[8], p, at::kBFloat16, K);
        v.gamma = flat(a[9], p, at::kBFloat16, K);
        v.eps = (float)real(a[10]);
        if (a[11] != Py_None)
            v.gate = flat(a[11], p, at::kBFloat16, K);
        v.alpha = (float)real(a[12]);
        const Out ro = out_rows(a[13], p, at::kBFloat16, M, K);
        const Out o = out_codes(a[14], p, q.i8, M, K / q.per_byte);
        const Out s = out_scales(a[15], p, q.scale_type(), M, K, q.part);
        v.Rout = ro.r.data;
        v.ldy = y.ld;
        v.ldr = r.ld;
        v.ldo = ro.r.ld;
        void *f = entry_of(a[0]);
        auto rows = [&](auto type) {
            enqueue<typename decltype(type)::F>(ran, f, &v, o.r.data, o.r.ld, s.r.data, M, K, p.stream);
        };
        if (q.fmt >= 0)
            enqueue<decltype(qgemm_postnorm_quant_mx)>(ran, f, (qgemm_mx_fmt)q.fmt, &v, o.r.data, o.r.ld, s.r.data, s.r.ld, M,
                                                       K, p.stream);
        else if (q.part)
            enqueue<decltype(qgemm_postnorm_quant_f8_block)>(ran, f, &v, o.r.data, o.r.ld, s.r.data, s.r.ld, M, K, p.stream);
        else if (q.i8)
            rows(Type<decltype(qgemm_postnorm_quant_i8_rowwise)>());
        else
            rows(Type<decltype(qgemm_postnorm_quant_f8_pertoken)>());
        return pack({o.object(), s.object(), ro.object()});
    });
}

// entry, MX element format or -1, elements a byte, K elements a scale covers (0:
// the row), rows of B a scale covers, A, B, scale_a, scale_b, offsets, order,
// top_k, bias, out
PyObject *grouped(PyObject *, PyObject *const *a, Py_ssize_t n)
{
    return attempt(n, 14, [&](bool &ran) -> PyObject * {
        const int fmt = (int)whole(a[1]);
        const I per_byte = whole(a[2]), part = whole(a[3]), b_rows = whole(a[4]);
        const at::Tensor &at_ = tensor(a[5]), &bt = tensor(a[6]);
        const Place p(at_);
        auto is_code = [&](const at::Tensor &t) {
            const at::ScalarType s = t.scalar_type();
            // (the int8 entry is the one that covers no rows of B by a scale)
            return b_rows == 0 ? s == at::kChar : s == at::kByte || (per_byte == 1 && s == at::kFloat8_e4m3fn);
        };
        need(is_code(at_) && is_code(bt));
        const Rows A = rows_of(at_, p);
        need(bt.dim() == 3 && bt.device() == p.device);
        const I E = bt.size(0), N = bt.size(1), row = bt.size(2), K = row * per_byte;
        need(E >= 1 && N >= 1 && row > 1 && row == A.cols && bt.stride(2) == 1 && K % 128 == 0);
        const I ldb = N > 1 ? bt.stride(1) : row;
        need(E == 1 || bt.stride(0) == N * ldb);
        P offsets = flat(a[9], p, at::kInt, E + 1), order = nullptr;
        I rows = A.rows, top_k = 1;
        if (a[10] != Py_None) {
            const at::Tensor &ot = tensor(a[10]);
            need(ot.dim() == 1);
            rows = ot.size(0);
            order = flat(a[10], p, at::kInt, rows);
            if (a[11] == Py_None) {
                need(A.rows > 0 && rows % A.rows == 0);
                top_k = rows ? rows / A.rows : 1;
            } else {
                need(PyLong_CheckExact(a[11]));
                top_k = whole(a[11]);
            }
            need(top_k >= 1 && top_k <= 64);
        }
        // the scales' shapes, as the full way has them
        auto scales = [&](PyObject *o, std::initializer_list<I> shape) -> P {
            const at::Tensor &t = tensor(o);
            need(t.device() == p.device && t.is_contiguous() && t.sizes() == at::IntArrayRef(shape));
            const at::ScalarType s = t.scalar_type();
            need(fmt >= 0 ? s == at::kByte || s == at::kFloat8_e8m0fnu : s == at::kFloat);
            return t.data_ptr();
        };
        P sa, sb;
        if (!part) {
            sa = scales(a[7], {A.rows});
            sb = scales(a[8], {E, N});
        } else {
            sa = scales(a[7], {A.rows, K / part});
            sb = scales(a[8], {E, (N + b_rows - 1) / b_rows, K / part});
        }
        P bias = nullptr;
        if (a[12] != Py_None) {
            const at::Tensor &t = tensor(a[12]);
            need(t.dim() == 2 && t.size(0) == E && t.size(1) == N);
            bias = flat(a[12], p, at::kBFloat16, E * N);
        }
        need(N % 8 == 0 || a[13] != Py_None);
        Out c = out_rows(a[13], p, at::kBFloat16, rows, N);
        if (rows <= 1)
            c.r.ld = N + (8 - N % 8) % 8;
        void *f = entry_of(a[0]);
        auto call = [&](auto type, auto... format) {
            enqueue<typename decltype(type)::F>(ran, f, format..., A.data, A.ld, A.rows, P(bt.data_ptr()), ldb, sa, sb, offsets,
                                                order, top_k, bias, c.r.data, c.r.ld, rows, E, N, K, p.stream);
        };
        if (fmt >= 0)
            call(Type<decltype(qgemm_mx_grouped)>(), (qgemm_mx_fmt)fmt);
        else if (b_rows == 0)
            call(Type<decltype(qgemm_i8_rowwise_grouped)>());
        else if (part)
            call(Type<decltype(qgemm_f8_blockscale_grouped)>());
        else
            call(Type<decltype(qgemm_f8_pertoken_grouped)>());
        return c.object();
    });
}

// get_device, get_stream, check
PyObject *init(PyObject *, PyObject *const *a, Py_ssize_t n)
{
    if (n != 3 || !PyCallable_Check(a[0]) || !PyCallable_Check(a[1]) || !PyCallable_Check(a[2])) {
        PyErr_SetString(PyExc_TypeError, "init(get_device, get_stream, check)");
        return nullptr;
    }
    Py_INCREF(a[0]);
    Py_INCREF(a[1]);
    Py_INCREF(a[2]);
    Py_XSETREF(g_get_device, a[0]);
    Py_XSETREF(g_get_stream, a[1]);
    Py_XSETREF(g_check, a[2]);
    Py_RETURN_NONE;
}

#define FUNCTION(name) {#name, (PyCFunction)(void (*)(void))name, METH_FASTCALL, nullptr}
PyMethodDef methods[] = {FUNCTION(init),     FUNCTION(moe_sort),         FUNCTION(moe_gather),
                         FUNCTION(moe_combine), FUNCTION(moe_combine_grad), FUNCTION(swiglu),
                         FUNCTION(postnorm), FUNCTION(grouped),          {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_fast", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__fast(void) { return PyModule_Create(&module); }
