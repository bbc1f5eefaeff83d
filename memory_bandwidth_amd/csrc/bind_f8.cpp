// bind_f8.cpp -- the Python side of q4f8.h, functions of the module that
// bind_i8.cpp makes, and like those: each checks its tensors, allocates the
// outputs where none are given, and calls the entry point on the device's
// current stream.  It returns the outputs, None where an argument is not what
// it must be, or the entry point's error status.
#include "bind.h"
#include "q4f8.h"

namespace {

using namespace q4py;

struct {
    decltype(&quant_f8) quant;
    decltype(&quant_f8_block) quant_block;
    decltype(&gemm_f8) gemm;
    decltype(&gemm_f8_swiglu) swiglu;
    decltype(&gemm_f8_swiglu_backward) backward;
} g;

constexpr at::ScalarType kCodes = at::kFloat8_e4m3fn;

int64_t blocks(int64_t n) { return n / 128 + (n % 128 != 0); }

// A tensor of float32 on a device and of two dimensions, whatever its strides.
bool is_scales(const at::Tensor *t, int dev) {
    return t && t->scalar_type() == at::kFloat && t->is_cuda() && t->get_device() == dev && t->dim() == 2 &&
           t->layout() == at::kStrided;
}

// A stride along a dimension that has several places, else 0.
int64_t stride_of(const at::Tensor &t, int d) { return t.size(d) > 1 ? t.stride(d) : 0; }

// The activations of a product, its output's type and the output.
struct Rows {
    const at::Tensor *a, *sa;
    int dev = -1, type = -1, a_block = 1;
    int64_t M = 0, K = 0;
    at::ScalarType dtype = at::kFloat;

    Rows(PyObject *pa, PyObject *psa, PyObject *pdtype) : a(tensor(pa)), sa(tensor(psa)) {
        if (!a || a->dim() != 2 || !a->is_cuda() || !THPDtype_Check(pdtype)) return;
        dtype = reinterpret_cast<THPDtype *>(pdtype)->scalar_type;
        dev = a->get_device(), M = a->size(0), K = a->size(1);
        if (!is(a, kCodes, dev, {M, K}) || !is_scales(sa, dev) || sa->size(1) != blocks(K)) return;
        if (sa->size(0) != M) {
            if (sa->size(0) != blocks(M)) return;
            a_block = 128;
        }
        type = type_code(dtype);
    }
    // Weights [N, K] and their scales.
    bool weights(const at::Tensor *w, const at::Tensor *sw, int64_t &N) const {
        if (!w || w->dim() != 2) return false;
        N = w->size(0);
        return is(w, kCodes, dev, {N, K}) && is(sw, at::kFloat, dev, {blocks(N), blocks(K)});
    }
    // y [M, N]: none given, or one that fits.
    bool takes(PyObject *given, int64_t N) const {
        return given == Py_None || is(tensor(given), dtype, dev, {M, N});
    }
    at::Tensor output(const at::Tensor *given, int64_t N) const {
        return given ? *given : at::empty({M, N}, a->options().dtype(dtype));
    }
    bool too_large(int64_t N) const { return !fits_int(M) || !fits_int(K) || !fits_int(N); }
};

const uint8_t *codes_of(const at::Tensor *t) { return static_cast<const uint8_t *>(t->data_ptr()); }

// gemm_f8(a, a_scales, w, w_scales, bias, dtype, out)
PyObject *gemm(PyObject *, PyObject *const *args, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    if (n != 7) return PyErr_Format(PyExc_TypeError, "7 arguments");
    const Rows r(args[0], args[1], args[5]);
    const at::Tensor *w = tensor(args[2]), *sw = tensor(args[3]), *bias = tensor(args[4]);
    int64_t N = 0;
    if (r.type < 0 || !r.weights(w, sw, N) || (args[4] != Py_None && !is(bias, at::kFloat, r.dev, {N})) ||
        !r.takes(args[6], N))
        Py_RETURN_NONE;
    if (r.too_large(N)) return PyLong_FromLong(Q4_EINVAL);
    const OnDevice on(*r.a);
    if (!on.fine) return nullptr;
    const at::Tensor *out = tensor(args[6]);
    at::Tensor y;
    int status;
    {
        const NoGil no_gil;
        y = r.output(out, N);
        status = g.gemm(codes_of(r.a), ptr<float>(r.sa), stride_of(*r.sa, 0), stride_of(*r.sa, 1), r.a_block,
                        codes_of(w), ptr<float>(sw), bias ? ptr<float>(bias) : nullptr, y.data_ptr(), r.type, (int)r.M,
                        (int)N, (int)r.K, on.stream);
    }
    return finish(status, args[6], y);
    END_HANDLE_TH_ERRORS
}

// Both gated calls; dh None: the forward one.
PyObject *gated(PyObject *pdh, PyObject *const *args) {
    const Rows r(args[0], args[1], args[6]);
    const at::Tensor *wg = tensor(args[2]), *sg = tensor(args[3]), *wu = tensor(args[4]), *su = tensor(args[5]);
    const bool back = pdh != nullptr;
    const at::Tensor *dh = back ? tensor(pdh) : nullptr;
    int64_t N = 0, up = 0;
    if (r.type < 0 || !r.weights(wg, sg, N) || !r.weights(wu, su, up) || up != N || !fits_int(2 * N) ||
        !r.takes(args[7], back ? 2 * N : N))
        Py_RETURN_NONE;
    if (back && (!dh || type_code(dh->scalar_type()) < 0 || !is(dh, dh->scalar_type(), r.dev, {r.M, N}))) Py_RETURN_NONE;
    if (r.too_large(N)) return PyLong_FromLong(Q4_EINVAL);
    const OnDevice on(*r.a);
    if (!on.fine) return nullptr;
    const at::Tensor *out = tensor(args[7]);
    at::Tensor y;
    int status;
    const int64_t sm = stride_of(*r.sa, 0), sk = stride_of(*r.sa, 1);
    {
        const NoGil no_gil;
        y = r.output(out, back ? 2 * N : N);
        status = back ? g.backward(dh->data_ptr(), type_code(dh->scalar_type()), codes_of(r.a), ptr<float>(r.sa), sm,
                                   sk, r.a_block, codes_of(wg), ptr<float>(sg), codes_of(wu), ptr<float>(su),
                                   y.data_ptr(), r.type, (int)r.M, (int)N, (int)r.K, on.stream)
                      : g.swiglu(codes_of(r.a), ptr<float>(r.sa), sm, sk, r.a_block, codes_of(wg), ptr<float>(sg),
                                 codes_of(wu), ptr<float>(su), y.data_ptr(), r.type, (int)r.M, (int)N, (int)r.K,
                                 on.stream);
    }
    return finish(status, args[7], y);
}

// swiglu_f8(a, a_scales, w_gate, scales_gate, w_up, scales_up, dtype, out)
PyObject *swiglu(PyObject *, PyObject *const *args, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    if (n != 8) return PyErr_Format(PyExc_TypeError, "8 arguments");
    return gated(nullptr, args);
    END_HANDLE_TH_ERRORS
}

// swiglu_backward_f8(dh, a, a_scales, w_gate, scales_gate, w_up, scales_up, dtype, out)
PyObject *swiglu_backward(PyObject *, PyObject *const *args, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    if (n != 9) return PyErr_Format(PyExc_TypeError, "9 arguments");
    return gated(args[0], args + 1);
    END_HANDLE_TH_ERRORS
}

// A tuple of new references to what wraps the tensors.
PyObject *pack(at::Tensor *const *t, int n) {
    PyObject *all = PyTuple_New(n);
    for (int i = 0; all && i < n; ++i) {
        PyObject *o = THPVariable_Wrap(*t[i]);
        if (!o) {
            Py_CLEAR(all);
            break;
        }
        PyTuple_SET_ITEM(all, i, o);
    }
    return all;
}

// The input of a quantiser.
struct Input {
    const at::Tensor *x;
    int type = -1, dev = -1;
    int64_t rows = 0, cols = 0;
    explicit Input(PyObject *o) : x(tensor(o)) {
        if (!x || x->dim() != 2 || !x->is_cuda() || !x->is_contiguous()) return;
        dev = x->get_device(), rows = x->size(0), cols = x->size(1);
        type = type_code(x->scalar_type());
    }
    at::TensorOptions codes() const { return x->options().dtype(kCodes); }
    at::TensorOptions scales() const { return x->options().dtype(at::kFloat); }
};

// quant_f8(x, codes, scales) -> (codes, scales); None for new ones, whose scales lie block by block.
PyObject *quant(PyObject *, PyObject *const *args, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    if (n != 3) return PyErr_Format(PyExc_TypeError, "3 arguments");
    const Input in(args[0]);
    if (in.type < 0) Py_RETURN_NONE;
    if (!fits_int(in.rows) || !fits_int(in.cols)) return PyLong_FromLong(Q4_EINVAL);
    const bool given = args[1] != Py_None || args[2] != Py_None;
    const at::Tensor *gc = tensor(args[1]), *gs = tensor(args[2]);
    const int64_t KB = blocks(in.cols);
    if (given && (!is(gc, kCodes, in.dev, {in.rows, in.cols}) || !is_scales(gs, in.dev) || gs->size(0) != in.rows ||
                  gs->size(1) != KB))
        Py_RETURN_NONE;
    const OnDevice on(*in.x);
    if (!on.fine) return nullptr;
    at::Tensor codes, scales;
    int status;
    {
        const NoGil no_gil;
        codes = given ? *gc : at::empty({in.rows, in.cols}, in.codes());
        scales = given ? *gs : at::empty_strided({in.rows, KB}, {1, in.rows}, in.scales());
        status = g.quant(in.x->data_ptr(), in.type, static_cast<uint8_t *>(codes.data_ptr()), ptr<float>(&scales),
                         stride_of(scales, 0), stride_of(scales, 1), (int)in.rows, (int)in.cols, on.stream);
    }
    if (status != Q4_OK) return PyLong_FromLong(status);
    if (given) return PyTuple_Pack(2, args[1], args[2]);
    at::Tensor *const both[] = {&codes, &scales};
    return pack(both, 2);
    END_HANDLE_TH_ERRORS
}

// quant_block_f8(x, as_is, turned, codes, scales, codes_t, scales_t) -> the two, or four, that
// are asked for; all of those given, or None for each.
PyObject *quant_block(PyObject *, PyObject *const *args, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    if (n != 7) return PyErr_Format(PyExc_TypeError, "7 arguments");
    const Input in(args[0]);
    const bool as_is = args[1] == Py_True, turned = args[2] == Py_True;
    if (in.type < 0 || (!as_is && !turned)) Py_RETURN_NONE;
    if (!fits_int(in.rows) || !fits_int(in.cols)) return PyLong_FromLong(Q4_EINVAL);
    bool given = false;
    for (int i = 3; i < 7; ++i) given = given || args[i] != Py_None;
    const int64_t RB = blocks(in.rows), CB = blocks(in.cols), R16 = (in.rows + 15) / 16 * 16;
    at::Tensor t[4];
    if (given) {
        const bool want[4] = {as_is, as_is, turned, turned};
        const int64_t shape[4][2] = {{in.rows, in.cols}, {RB, CB}, {in.cols, R16}, {CB, RB}};
        for (int i = 0; i < 4; ++i) {
            if (!want[i]) continue;
            const at::Tensor *o = tensor(args[3 + i]);
            if (!is(o, i & 1 ? at::kFloat : kCodes, in.dev, {shape[i][0], shape[i][1]})) Py_RETURN_NONE;
            t[i] = *o;
        }
    }
    const OnDevice on(*in.x);
    if (!on.fine) return nullptr;
    int status;
    {
        const NoGil no_gil;
        if (!given && as_is) {
            t[0] = at::empty({in.rows, in.cols}, in.codes());
            t[1] = at::empty({RB, CB}, in.scales());
        }
        if (!given && turned) {
            t[2] = at::empty({in.cols, R16}, in.codes());
            t[3] = at::empty({CB, RB}, in.scales());
        }
        status = g.quant_block(in.x->data_ptr(), in.type, as_is ? static_cast<uint8_t *>(t[0].data_ptr()) : nullptr,
                               as_is ? ptr<float>(&t[1]) : nullptr,
                               turned ? static_cast<uint8_t *>(t[2].data_ptr()) : nullptr,
                               turned ? ptr<float>(&t[3]) : nullptr, (int)in.rows, (int)in.cols, on.stream);
    }
    if (status != Q4_OK) return PyLong_FromLong(status);
    at::Tensor *const all[] = {&t[0], &t[1], &t[2], &t[3]};
    return pack(as_is ? all : all + 2, as_is && turned ? 4 : 2);
    END_HANDLE_TH_ERRORS
}

// init_f8(addresses): the entry points in the order of g.
PyObject *init(PyObject *, PyObject *args) {
    unsigned long long a[5];
    if (!PyArg_ParseTuple(args, "KKKKK", a, a + 1, a + 2, a + 3, a + 4)) return nullptr;
    g.quant = reinterpret_cast<decltype(g.quant)>(a[0]);
    g.quant_block = reinterpret_cast<decltype(g.quant_block)>(a[1]);
    g.gemm = reinterpret_cast<decltype(g.gemm)>(a[2]);
    g.swiglu = reinterpret_cast<decltype(g.swiglu)>(a[3]);
    g.backward = reinterpret_cast<decltype(g.backward)>(a[4]);
    Py_RETURN_NONE;
}

template <typename F>
PyCFunction fast(F *f) { return reinterpret_cast<PyCFunction>(reinterpret_cast<void *>(f)); }

}  // namespace

PyMethodDef q4py::kF8Methods[] = {
    {"init_f8", init, METH_VARARGS, nullptr},
    {"gemm_f8", fast(gemm), METH_FASTCALL, nullptr},
    {"swiglu_f8", fast(swiglu), METH_FASTCALL, nullptr},
    {"swiglu_backward_f8", fast(swiglu_backward), METH_FASTCALL, nullptr},
    {"quant_f8", fast(quant), METH_FASTCALL, nullptr},
    {"quant_block_f8", fast(quant_block), METH_FASTCALL, nullptr},
    {nullptr, nullptr, 0, nullptr}};
