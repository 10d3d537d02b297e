// bind.cpp -- argument checks and marshalling of the Python binding for the
// operators around a block's allreduce: tensors in, a status out. In C++
// because these calls are also made for single tokens: rx_moe_dispatch with its
// seven tensors takes the host 4.1 us this way and took 9.6 us in Python (3.3 us
// of it the kernel's launch), rx_residual_norm over eight sources 4.1 and 14.6.
// Raises ValueError or TypeError for what the C entry points cannot see (shapes,
// devices, contiguity); computes nothing.
#include <torch/csrc/autograd/python_variable.h>
#include <torch/csrc/Exceptions.h>

#include "rx.h"

namespace {

struct Raised {};   // a Python error is set

using Sizes = std::initializer_list<int64_t>;

// The entry points of the librx that is loaded already (connect()).
struct {
    decltype(&rx_moe_dispatch) moe_dispatch;
    decltype(&rx_moe_combine) moe_combine;
    decltype(&rx_moe_combine_backward) moe_combine_backward;
    decltype(&rx_residual_norm) residual_norm;
    decltype(&rx_residual_norm_backward) residual_norm_backward;
    decltype(&rx_quant_i8) quant_i8;
    decltype(&rx_gemm_i8) gemm_i8;
} rx;

template <class... A>
[[noreturn]] void refuse(PyObject* type, const char* format, A... a)
{
    PyErr_Format(type, format, a...);
    throw Raised();
}

// Other threads run while a launch waits for room in the queue.
struct NoGil {
    PyThreadState* state = PyEval_SaveThread();
    ~NoGil() { PyEval_RestoreThread(state); }
};

bool given(PyObject* o) { return o != Py_None; }

const at::Tensor& tensor(PyObject* o, const char* name)
{
    if (!THPVariable_Check(o))
        refuse(PyExc_TypeError, "%s must be a tensor", name);
    return THPVariable_Unpack(o);
}

int64_t integer(PyObject* o)
{
    const long long v = PyLong_AsLongLong(o);
    if (v == -1 && PyErr_Occurred())
        throw Raised();
    return v;
}

int integer32(PyObject* o, const char* name)
{
    const int64_t v = integer(o);
    if (v < INT32_MIN || v > INT32_MAX)
        refuse(PyExc_ValueError, "%s must fit 32 bits", name);
    return (int)v;
}

float real(PyObject* o)
{
    const double v = PyFloat_AsDouble(o);
    if (v == -1.0 && PyErr_Occurred())
        throw Raised();
    return (float)v;
}

// A GPU tensor of the given shape and type.
void check(int dev, at::ScalarType type, Sizes shape, const char* name, const at::Tensor& t)
{
    if (!t.is_cuda())
        refuse(PyExc_ValueError, "%s must be a GPU tensor", name);
    if (t.get_device() != dev)
        refuse(PyExc_ValueError, "%s is on cuda:%d, the current device is cuda:%d", name, (int)t.get_device(), dev);
    if (t.scalar_type() != type)
        refuse(PyExc_TypeError, "%s must be %s, not %s", name, c10::toString(type), c10::toString(t.scalar_type()));
    if (t.sizes() != c10::IntArrayRef(shape)) {
        std::ostringstream want, have;
        want << c10::IntArrayRef(shape);
        have << t.sizes();
        refuse(PyExc_ValueError, "%s must have shape %s, not %s", name, want.str().c_str(), have.str().c_str());
    }
}

// ... whose rows (its last dimension) are packed, at any stride: the stride.
// The stride of a single row, or of rows without elements, may be any number
// in a tensor: it is taken as the row's length.
size_t block(int dev, at::ScalarType type, Sizes shape, const char* name, const at::Tensor& t)
{
    check(dev, type, shape, name, t);
    const int64_t n = (int64_t)shape.size(), rows = t.size(n - 2), width = t.size(n - 1), ld = t.stride(n - 2);
    if (rows > 0 && width > 1 && t.stride(n - 1) != 1)
        refuse(PyExc_ValueError, "%s's rows must be contiguous", name);
    if (rows <= 1 || width == 0)
        return (size_t)width;
    if (ld < width)
        refuse(PyExc_ValueError, "%s's rows overlap", name);
    return (size_t)ld;
}

void* packed(int dev, at::ScalarType type, Sizes shape, const char* name, const at::Tensor& t)
{
    check(dev, type, shape, name, t);
    if (!t.is_contiguous())
        refuse(PyExc_ValueError, "%s must be contiguous", name);
    return t.data_ptr();
}
void* packed(int dev, at::ScalarType type, Sizes shape, const char* name, PyObject* o)
{
    return given(o) ? packed(dev, type, shape, name, tensor(o, name)) : nullptr;
}

rx_dtype_t data_type(const at::Tensor& t)
{
    if (t.scalar_type() == at::kFloat)
        return RX_FP32;
    if (t.scalar_type() == at::kBFloat16)
        return RX_BF16;
    refuse(PyExc_TypeError, "unsupported tensor dtype %s (float32 or bfloat16)", c10::toString(t.scalar_type()));
}

void two_dims(const at::Tensor& t, const char* name)
{
    if (t.dim() != 2)
        refuse(PyExc_ValueError, "%s must have two dimensions", name);
}

// A workspace's bytes.
void* workspace(int dev, PyObject* o, size_t* bytes)
{
    *bytes = 0;
    if (!given(o))
        return nullptr;
    const at::Tensor& t = tensor(o, "workspace");
    *bytes = (size_t)t.numel();
    return packed(dev, at::kByte, {t.numel()}, "workspace", t);
}

PyObject* current_stream;   // torch's: device -> the current stream's handle

// The leading arguments of every call: the device, and the stream's handle or
// None for the current stream, looked up once the arguments are checked.
struct Where {
    int dev;
    PyObject* handle;
    hipStream_t stream() const
    {
        if (given(handle))
            return reinterpret_cast<hipStream_t>((intptr_t)integer(handle));
        PyObject* index = PyLong_FromLong(dev);
        PyObject* got = index ? PyObject_CallFunctionObjArgs(current_stream, index, nullptr) : nullptr;
        Py_XDECREF(index);
        if (!got)
            throw Raised();
        const long long h = PyLong_AsLongLong(got);
        Py_DECREF(got);
        if (h == -1 && PyErr_Occurred())
            throw Raised();
        return reinterpret_cast<hipStream_t>((intptr_t)h);
    }
};
Where where(PyObject* const* a, Py_ssize_t n, Py_ssize_t want)
{
    if (n != want)
        refuse(PyExc_TypeError, "%d arguments, not %d", (int)want, (int)n);
    return {integer32(a[0], "device"), a[1]};
}

int moe_dispatch(PyObject* const* a, Py_ssize_t n)
{
    const Where w = where(a, n, 12);
    const at::Tensor &ids = tensor(a[2], "expert_ids"), &offsets = tensor(a[4], "offsets"), &order = tensor(a[5], "order"),
                     &slots = tensor(a[6], "slots");
    two_dims(ids, "expert_ids");
    const int experts = integer32(a[3], "experts"), first = integer32(a[10], "first_expert");
    const int64_t tokens = ids.size(0), topk = ids.size(1), pairs = tokens * topk;
    if (topk > INT32_MAX)
        refuse(PyExc_ValueError, "too many choices a token");
    const int* pi = (const int*)packed(w.dev, at::kInt, {tokens, topk}, "expert_ids", ids);
    int* po = (int*)packed(w.dev, at::kInt, {(int64_t)experts + 1}, "offsets", offsets);
    int* pr = (int*)packed(w.dev, at::kInt, {pairs}, "order", order);
    int* ps = (int*)packed(w.dev, at::kInt, {tokens, topk}, "slots", slots);
    const void* x = nullptr;
    void* rows = nullptr;
    float* scales = nullptr;
    size_t ld_x = 0, ld_rows = 0, hidden = 0, bytes;
    rx_dtype_t xt = RX_FP32, rt = RX_FP32;
    if (given(a[7]) || given(a[8]) || given(a[9])) {
        if (!given(a[7]) || !given(a[8]))
            refuse(PyExc_ValueError, "x and rows come together");
        const at::Tensor &tx = tensor(a[7], "x"), &tr = tensor(a[8], "rows");
        two_dims(tx, "x");
        hidden = (size_t)tx.size(1);
        xt = data_type(tx);
        ld_x = block(w.dev, tx.scalar_type(), {tokens, (int64_t)hidden}, "x", tx);
        const bool quant = tr.scalar_type() == at::kChar;
        if (quant != given(a[9]))
            refuse(PyExc_ValueError, "scales come with int8 rows");
        rt = quant ? RX_INT8 : xt;
        ld_rows = block(w.dev, quant ? at::kChar : tx.scalar_type(), {pairs, (int64_t)hidden}, "rows", tr);
        scales = (float*)packed(w.dev, at::kFloat, {pairs}, "scales", a[9]);
        x = tx.data_ptr();
        rows = tr.data_ptr();
    }
    void* ws = workspace(w.dev, a[11], &bytes);
    const hipStream_t stream = w.stream();
    NoGil open;
    return rx.moe_dispatch(pi, tokens, (int)topk, first, experts, x, ld_x, hidden, xt, po, pr, ps, rows, ld_rows, rt, scales,
                           ws, bytes, stream);
}

int moe_combine(PyObject* const* a, Py_ssize_t n)
{
    const Where w = where(a, n, 6);
    const at::Tensor &rows = tensor(a[2], "rows"), &slots = tensor(a[3], "slots"), &out = tensor(a[5], "out");
    two_dims(rows, "rows");
    two_dims(slots, "slots");
    const int64_t nrows = rows.size(0), hidden = rows.size(1), tokens = slots.size(0), topk = slots.size(1);
    const rx_dtype_t dt = data_type(rows);
    const size_t ld = block(w.dev, rows.scalar_type(), {nrows, hidden}, "rows", rows);
    const size_t ld_out = block(w.dev, rows.scalar_type(), {tokens, hidden}, "out", out);
    const int* ps = (const int*)packed(w.dev, at::kInt, {tokens, topk}, "slots", slots);
    const float* pw = (const float*)packed(w.dev, at::kFloat, {tokens, topk}, "weights", a[4]);
    if (topk > INT32_MAX)
        refuse(PyExc_ValueError, "too many choices a token");
    const hipStream_t stream = w.stream();
    NoGil open;
    return rx.moe_combine(rows.data_ptr(), ld, nrows, ps, pw, tokens, (int)topk, hidden, dt, out.data_ptr(), ld_out, stream);
}

int moe_combine_backward(PyObject* const* a, Py_ssize_t n)
{
    const Where w = where(a, n, 9);
    const at::Tensor &g = tensor(a[2], "d_out"), &slots = tensor(a[4], "slots"), &offsets = tensor(a[6], "offsets"),
                     &dr = tensor(a[7], "d_rows");
    two_dims(slots, "slots");
    two_dims(dr, "d_rows");
    const int64_t tokens = slots.size(0), topk = slots.size(1), nrows = dr.size(0), hidden = dr.size(1);
    const rx_dtype_t dt = data_type(g);
    const size_t ld_g = block(w.dev, g.scalar_type(), {tokens, hidden}, "d_out", g);
    const size_t ld_dr = block(w.dev, g.scalar_type(), {nrows, hidden}, "d_rows", dr);
    size_t ld_r = 0;
    const void* rows = nullptr;
    if (given(a[3])) {
        const at::Tensor& r = tensor(a[3], "rows");
        ld_r = block(w.dev, g.scalar_type(), {nrows, hidden}, "rows", r);
        rows = r.data_ptr();
    } else if (given(a[8])) {
        refuse(PyExc_ValueError, "d_weights needs rows");
    }
    const int* ps = (const int*)packed(w.dev, at::kInt, {tokens, topk}, "slots", slots);
    if (offsets.dim() != 1 || offsets.numel() < 1)
        refuse(PyExc_ValueError, "offsets must hold experts + 1 values");
    const int* po = (const int*)packed(w.dev, at::kInt, {offsets.numel()}, "offsets", offsets);
    const float* pw = (const float*)packed(w.dev, at::kFloat, {tokens, topk}, "weights", a[5]);
    float* dw = (float*)packed(w.dev, at::kFloat, {tokens, topk}, "d_weights", a[8]);
    if (topk > INT32_MAX)
        refuse(PyExc_ValueError, "too many choices a token");
    const hipStream_t stream = w.stream();
    NoGil open;
    return rx.moe_combine_backward(g.data_ptr(), ld_g, rows, ld_r, nrows, ps, pw, po + offsets.numel() - 1, tokens, (int)topk,
                                   hidden, dt, dr.data_ptr(), ld_dr, dw, stream);
}

// What both directions of the residual norm read: a = srcs, residual, gate,
// gate_rows (None: all rows share one), w_post, w_pre.
struct NormInputs {
    at::Tensor held[RX_MAX_SRC];   // the sources, which a generator alone may have had, until the launch
    const void* src[RX_MAX_SRC];
    int nsrc;
    size_t ld_src = 0, ld_residual = 0, gate_rows;
    const void *residual = nullptr, *gate = nullptr, *w_post, *w_pre;
    int64_t rows = 0, hidden = 0, groups;
    at::ScalarType type;
    rx_dtype_t dtype;
};

NormInputs norm_inputs(int dev, PyObject* const* a)
{
    NormInputs in;
    PyObject* seq = PySequence_Fast(a[0], "srcs must be a sequence of tensors");
    if (!seq)
        throw Raised();
    struct Listed {
        PyObject* o;
        ~Listed() { Py_DECREF(o); }
    } listed{seq};
    const Py_ssize_t n = PySequence_Fast_GET_SIZE(seq);
    if (n < 1 || n > RX_MAX_SRC)
        refuse(PyExc_ValueError, "1 to %d sources, not %d", RX_MAX_SRC, (int)n);
    in.nsrc = (int)n;
    for (Py_ssize_t k = 0; k < n; ++k) {
        const at::Tensor& t = tensor(PySequence_Fast_GET_ITEM(seq, k), "a source");
        if (k == 0) {
            two_dims(t, "srcs[0]");
            in.rows = t.size(0);
            in.hidden = t.size(1);
            in.dtype = data_type(t);
            in.type = t.scalar_type();
        }
        const size_t ld = block(dev, in.type, {in.rows, in.hidden}, k ? "a source" : "srcs[0]", t);
        if (k == 0)
            in.ld_src = ld;
        else if (ld != in.ld_src)
            refuse(PyExc_ValueError, "srcs[%d] has another row stride than srcs[0]", (int)k);
        in.held[k] = t;
        in.src[k] = t.data_ptr();
    }
    if (given(a[1])) {
        const at::Tensor& t = tensor(a[1], "residual");
        in.ld_residual = block(dev, in.type, {in.rows, in.hidden}, "residual", t);
        in.residual = t.data_ptr();
    }
    const int64_t gate_rows = given(a[3]) ? integer(a[3]) : in.rows > 0 ? in.rows : 1;
    if (given(a[2]) && gate_rows < 1)
        refuse(PyExc_ValueError, "gate_rows must be positive");
    in.gate_rows = gate_rows < 1 ? 0 : (size_t)gate_rows;
    in.groups = gate_rows < 1 ? 0 : in.rows / gate_rows + (in.rows % gate_rows != 0);
    // one gate row for all rows, of which there are none
    if (in.rows == 0 && !given(a[3]) && given(a[2])) {
        const at::Tensor& t = tensor(a[2], "gate");
        in.groups = t.dim() > 0 && t.size(0) == 0 ? 0 : 1;
    }
    in.gate = packed(dev, in.type, {in.groups, in.hidden}, "gate", a[2]);
    in.w_post = packed(dev, in.type, {in.hidden}, "w_post", a[4]);
    in.w_pre = packed(dev, in.type, {in.hidden}, "w_pre", a[5]);
    return in;
}

void* norm_matrix(int dev, const NormInputs& in, const char* name, PyObject* o, size_t* ld)
{
    *ld = 0;
    if (!given(o))
        return nullptr;
    const at::Tensor& t = tensor(o, name);
    *ld = block(dev, in.type, {in.rows, in.hidden}, name, t);
    return t.data_ptr();
}

int residual_norm(PyObject* const* a, Py_ssize_t n)
{
    const Where w = where(a, n, 14);
    const NormInputs in = norm_inputs(w.dev, a + 2);
    size_t ld_h, ld_z;
    void *h = norm_matrix(w.dev, in, "out_h", a[8], &ld_h), *z = norm_matrix(w.dev, in, "out_z", a[9], &ld_z);
    float* p = (float*)packed(w.dev, at::kFloat, {in.rows}, "rstd_post", a[10]);
    float* q = (float*)packed(w.dev, at::kFloat, {in.rows}, "rstd_pre", a[11]);
    const float rs = real(a[12]), eps = real(a[13]);
    const hipStream_t stream = w.stream();
    NoGil open;
    return rx.residual_norm(in.src, in.nsrc, in.ld_src, in.residual, in.ld_residual, in.gate, in.gate_rows, in.w_post,
                            in.w_pre, rs, eps, in.rows, in.hidden, in.dtype, h, ld_h, z, ld_z, p, q, stream);
}

int residual_norm_backward(PyObject* const* a, Py_ssize_t n)
{
    const Where w = where(a, n, 19);
    const NormInputs in = norm_inputs(w.dev, a + 2);
    const float* p = (const float*)packed(w.dev, at::kFloat, {in.rows}, "rstd_post", a[8]);
    const float* q = (const float*)packed(w.dev, at::kFloat, {in.rows}, "rstd_pre", a[9]);
    size_t ld[4], bytes;
    const void *dh = norm_matrix(w.dev, in, "d_h", a[10], &ld[0]), *dz = norm_matrix(w.dev, in, "d_z", a[11], &ld[1]);
    void *ds = norm_matrix(w.dev, in, "d_src", a[12], &ld[2]), *dr = norm_matrix(w.dev, in, "d_residual", a[13], &ld[3]);
    float* dg = (float*)packed(w.dev, at::kFloat, {in.groups, in.hidden}, "d_gate", a[14]);
    float* dwp = (float*)packed(w.dev, at::kFloat, {in.hidden}, "d_w_post", a[15]);
    float* dwq = (float*)packed(w.dev, at::kFloat, {in.hidden}, "d_w_pre", a[16]);
    const float rs = real(a[17]);
    void* ws = workspace(w.dev, a[18], &bytes);
    const hipStream_t stream = w.stream();
    NoGil open;
    // Without rows the C call knows no gate row, but writes a weight's gradient: zeros for the gate's, too.
    if (in.rows == 0 && in.groups == 1 && dg) {
        const int status = rx.residual_norm_backward(in.src, in.nsrc, 0, nullptr, 0, nullptr, 1, nullptr, nullptr, nullptr, nullptr,
                                                     rs, 0, in.hidden, in.dtype, nullptr, 0, nullptr, 0, nullptr, in.hidden,
                                                     nullptr, 0, nullptr, dg, nullptr, nullptr, 0, stream);
        if (status != RX_OK)
            return status;
        dg = nullptr;
    }
    return rx.residual_norm_backward(in.src, in.nsrc, in.ld_src, in.residual, in.ld_residual, in.gate, in.gate_rows, in.w_post,
                                     in.w_pre, p, q, rs, in.rows, in.hidden, in.dtype, dh, ld[0], dz, ld[1], ds,
                                     ld[2], dr, ld[3], dg, dwp, dwq, ws, bytes, stream);
}

int quant_i8(PyObject* const* a, Py_ssize_t n)
{
    const Where w = where(a, n, 5);
    const at::Tensor &x = tensor(a[2], "x"), &codes = tensor(a[3], "codes"), &scales = tensor(a[4], "scales");
    two_dims(x, "x");
    const int64_t rows = x.size(0), k = x.size(1);
    const rx_dtype_t dt = data_type(x);
    const size_t ld_x = block(w.dev, x.scalar_type(), {rows, k}, "x", x);
    const size_t ld_c = block(w.dev, at::kChar, {rows, k}, "codes", codes);
    float* ps = (float*)packed(w.dev, at::kFloat, {rows}, "scales", scales);
    const hipStream_t stream = w.stream();
    NoGil open;
    return rx.quant_i8(x.data_ptr(), ld_x, rows, k, dt, codes.data_ptr(), ld_c, ps, stream);
}

// The product's row stride: of a row that has no second one, its whole chunks.
size_t chunked(size_t ld, const at::Tensor& t, int64_t k)
{
    return t.size(-2) > 1 && k > 0 ? ld : (size_t)((k + 15) / 16 * 16);
}

// The product reads whole 16-byte chunks: the last row's must lie in the
// tensor's storage too.
void check_padded(const at::Tensor& t, int64_t k, const char* name)
{
    if (k % 16 == 0 || t.numel() == 0)
        return;
    int64_t last = t.storage_offset();
    for (int64_t d = 0; d + 1 < t.dim(); ++d)
        last += (t.size(d) - 1) * t.stride(d);
    if ((size_t)(last + (k + 15) / 16 * 16) > t.storage().nbytes())
        refuse(PyExc_ValueError, "%s's last row must be padded to a multiple of 16 bytes", name);
}

int gemm_i8(PyObject* const* a, Py_ssize_t n)
{
    const Where w = where(a, n, 8);
    const at::Tensor &ta = tensor(a[2], "a"), &tb = tensor(a[4], "b"), &out = tensor(a[6], "out");
    two_dims(ta, "a");
    const bool grouped = given(a[7]);
    if (tb.dim() != (grouped ? 3 : 2))
        refuse(PyExc_ValueError, "b must have %s dimensions", grouped ? "three" : "two");
    const int64_t rows = ta.size(0), k = ta.size(1), cols = tb.size(-2), experts = grouped ? tb.size(0) : 1;
    if (experts > INT32_MAX)
        refuse(PyExc_ValueError, "too many experts");
    const size_t ld_a = chunked(block(w.dev, at::kChar, {rows, k}, "a", ta), ta, k);
    size_t ld_b, stride_b = 0;
    const int* offsets = nullptr;
    const float* sb;
    if (grouped) {
        ld_b = chunked(block(w.dev, at::kChar, {experts, cols, k}, "b", tb), tb, k);
        offsets = (const int*)packed(w.dev, at::kInt, {experts + 1}, "offsets", a[7]);
        if (tb.stride(0) < 0)
            refuse(PyExc_ValueError, "b's matrices must follow each other");
        stride_b = experts > 1 && tb.numel() > 0 ? (size_t)tb.stride(0) : 0;
        sb = (const float*)packed(w.dev, at::kFloat, {experts, cols}, "b_scales", tensor(a[5], "b_scales"));
    } else {
        ld_b = chunked(block(w.dev, at::kChar, {cols, k}, "b", tb), tb, k);
        sb = (const float*)packed(w.dev, at::kFloat, {cols}, "b_scales", tensor(a[5], "b_scales"));
    }
    const float* sa = (const float*)packed(w.dev, at::kFloat, {rows}, "a_scales", tensor(a[3], "a_scales"));
    const rx_dtype_t dt = data_type(out);
    const size_t ld_o = block(w.dev, out.scalar_type(), {rows, cols}, "out", out);
    check_padded(ta, k, "a");
    check_padded(tb, k, "b");
    const hipStream_t stream = w.stream();
    NoGil open;
    return rx.gemm_i8((const int8_t*)ta.data_ptr(), ld_a, sa, tb.data_ptr(), ld_b, stride_b, sb, offsets, (int)experts, rows,
                      cols, k, out.data_ptr(), ld_o, dt, stream);
}

// connect(torch's stream lookup, addresses of the entry points in the order
// of `rx` above)
int connect(PyObject* const* a, Py_ssize_t n)
{
    if (n != 8)
        refuse(PyExc_TypeError, "a function and 7 addresses");
    Py_INCREF(a[0]);
    current_stream = a[0];
    void** to = reinterpret_cast<void**>(&rx);
    for (int i = 0; i < 7; ++i)
        to[i] = reinterpret_cast<void*>((intptr_t)integer(a[i + 1]));
    return 0;
}

// No C++ exception leaves a call.
template <int (*F)(PyObject* const*, Py_ssize_t)>
PyObject* entry(PyObject*, PyObject* const* a, Py_ssize_t n)
{
    HANDLE_TH_ERRORS
    try {
        return PyLong_FromLong(F(a, n));
    } catch (const Raised&) {
        return nullptr;
    }
    END_HANDLE_TH_ERRORS
}

#define RX_ENTRY(NAME) {#NAME, (PyCFunction)(void*)entry<NAME>, METH_FASTCALL, nullptr}
PyMethodDef methods[] = {
    RX_ENTRY(connect), RX_ENTRY(moe_dispatch), RX_ENTRY(moe_combine), RX_ENTRY(moe_combine_backward),
    RX_ENTRY(residual_norm), RX_ENTRY(residual_norm_backward), RX_ENTRY(quant_i8), RX_ENTRY(gemm_i8),
    {nullptr, nullptr, 0, nullptr},
};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_rxbind", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__rxbind() { return PyModule_Create(&module); }
