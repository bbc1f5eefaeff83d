// bind_i8.cpp -- the Python side of q4i8.h as a CPython module.
//
// A product of one row takes 2 us on the GPU and 3.7 us in the runtime's
// launch, so what the binding adds is most of a call: 3.2 us with the checks
// in Python and ctypes, 1.4 here.  Each function checks its tensors, allocates
// the output where none is given, and calls the entry point on the device's
// current stream.  It returns the output, None where an argument is not what
// it must be (the caller then finds out which, and raises), or the entry
// point's error status.
#include "bind.h"

namespace {

using namespace q4py;

// The entry points, from the loaded library.
struct {
    decltype(&quant_i8) quant;
    decltype(&gemm_i8) gemm;
    decltype(&gemm_i8_swiglu) swiglu;
    decltype(&gemm_i8_grouped) grouped;
    decltype(&gemm_i8_grouped_swiglu) grouped_swiglu;
} g;

// What all products share: the rows, the output's type and the output.
struct Rows {
    const at::Tensor *a, *sa;
    int dev = -1;
    int64_t M = 0, K = 0;
    int type = -1;
    at::ScalarType dtype = at::kFloat;

    Rows(PyObject *pa, PyObject *psa, PyObject *pdtype) : a(tensor(pa)), sa(tensor(psa)) {
        if (!a || a->dim() != 2 || !a->is_cuda() || !THPDtype_Check(pdtype)) return;
        dtype = reinterpret_cast<THPDtype *>(pdtype)->scalar_type;
        dev = a->get_device(), M = a->size(0), K = a->size(1);
        if (!is(a, at::kChar, dev, {M, K}) || !is(sa, at::kFloat, dev, {M})) return;
        type = type_code(dtype);
    }

    // y [M, N]: none given, or one that fits.
    bool takes(PyObject *given, int64_t N) const {
        return given == Py_None || is(tensor(given), dtype, dev, {M, N});
    }
    at::Tensor output(const at::Tensor *given, int64_t N) const {
        return given ? *given : at::empty({M, N}, a->options().dtype(dtype));
    }
};

// Weights [N, K] (E < 0) or [E, N, K] and their scales.
bool weights(const Rows &r, const at::Tensor *w, const at::Tensor *sw, int64_t E, int64_t &N) {
    if (!w || w->dim() != (E >= 0 ? 3 : 2)) return false;
    N = w->size(-2);
    if (E >= 0) return is(w, at::kChar, r.dev, {E, N, r.K}) && is(sw, at::kFloat, r.dev, {E, N});
    return is(w, at::kChar, r.dev, {N, r.K}) && is(sw, at::kFloat, r.dev, {N});
}

int64_t experts(const Rows &r, const at::Tensor *offsets) {
    if (!offsets || offsets->dim() != 1) return -1;
    const int64_t E = offsets->size(0) - 1;
    return is(offsets, at::kInt, r.dev, {E + 1}) ? E : -1;
}

// gemm(a, a_scales, w, w_scales, bias, offsets, dtype, out): offsets None for
// a product without groups.
PyObject *gemm(PyObject *, PyObject *const *args, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    if (n != 8) return PyErr_Format(PyExc_TypeError, "8 arguments");
    const Rows r(args[0], args[1], args[6]);
    const at::Tensor *w = tensor(args[2]), *sw = tensor(args[3]), *bias = tensor(args[4]), *off = tensor(args[5]);
    const bool groups = args[5] != Py_None;
    int64_t E = -1, N = 0;
    if (r.type < 0 || (groups && (E = experts(r, off)) < 0) || !weights(r, w, sw, E, N) ||
        (args[4] != Py_None && !is(bias, at::kFloat, r.dev, {N})) || !r.takes(args[7], N))
        Py_RETURN_NONE;
    if (!fits_int(r.M) || !fits_int(r.K) || !fits_int(N) || !fits_int(E)) return PyLong_FromLong(Q4_EINVAL);
    const OnDevice on(*r.a);
    if (!on.fine) return nullptr;
    const at::Tensor *out = tensor(args[7]);
    at::Tensor y;
    int status;
    const int8_t *pa = ptr<int8_t>(r.a), *pw = ptr<int8_t>(w);
    const float *psa = ptr<float>(r.sa), *psw = ptr<float>(sw), *pb = bias ? ptr<float>(bias) : nullptr;
    {
        const NoGil no_gil;
        y = r.output(out, N);
        status = groups ? g.grouped(pa, psa, pw, psw, ptr<int32_t>(off), y.data_ptr(), r.type, (int)r.M, (int)E, (int)N,
                                    (int)r.K, on.stream)
                        : g.gemm(pa, psa, pw, psw, pb, y.data_ptr(), r.type, (int)r.M, (int)N, (int)r.K, on.stream);
    }
    return finish(status, args[7], y);
    END_HANDLE_TH_ERRORS
}

// swiglu(a, a_scales, w_gate, scales_gate, w_up, scales_up, offsets, dtype, out)
PyObject *swiglu(PyObject *, PyObject *const *args, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    if (n != 9) return PyErr_Format(PyExc_TypeError, "9 arguments");
    const Rows r(args[0], args[1], args[7]);
    const at::Tensor *wg = tensor(args[2]), *sg = tensor(args[3]), *wu = tensor(args[4]), *su = tensor(args[5]),
                     *off = tensor(args[6]);
    const bool groups = args[6] != Py_None;
    int64_t E = -1, N = 0, up = 0;
    if (r.type < 0 || (groups && (E = experts(r, off)) < 0) || !weights(r, wg, sg, E, N) ||
        !weights(r, wu, su, E, up) || up != N || !r.takes(args[8], N))
        Py_RETURN_NONE;
    if (!fits_int(r.M) || !fits_int(r.K) || !fits_int(N) || !fits_int(E)) return PyLong_FromLong(Q4_EINVAL);
    const OnDevice on(*r.a);
    if (!on.fine) return nullptr;
    const at::Tensor *out = tensor(args[8]);
    at::Tensor y;
    int status;
    const int8_t *pa = ptr<int8_t>(r.a), *pg = ptr<int8_t>(wg), *pu = ptr<int8_t>(wu);
    const float *psa = ptr<float>(r.sa), *psg = ptr<float>(sg), *psu = ptr<float>(su);
    {
        const NoGil no_gil;
        y = r.output(out, N);
        status = groups ? g.grouped_swiglu(pa, psa, pg, psg, pu, psu, ptr<int32_t>(off), y.data_ptr(), r.type, (int)r.M,
                                           (int)E, (int)N, (int)r.K, on.stream)
                        : g.swiglu(pa, psa, pg, psg, pu, psu, y.data_ptr(), r.type, (int)r.M, (int)N, (int)r.K,
                                   on.stream);
    }
    return finish(status, args[8], y);
    END_HANDLE_TH_ERRORS
}

// quant(x, codes, scales) -> (codes, scales); codes and scales None for new ones.
PyObject *quant(PyObject *, PyObject *const *args, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    if (n != 3) return PyErr_Format(PyExc_TypeError, "3 arguments");
    const at::Tensor *x = tensor(args[0]);
    if (!x || x->dim() != 2 || !x->is_cuda() || !x->is_contiguous()) Py_RETURN_NONE;
    const int type = type_code(x->scalar_type()), dev = x->get_device();
    const int64_t M = x->size(0), K = x->size(1);
    if (type < 0) Py_RETURN_NONE;
    if (!fits_int(M) || !fits_int(K)) return PyLong_FromLong(Q4_EINVAL);
    const bool given = args[1] != Py_None || args[2] != Py_None;
    const at::Tensor *gc = tensor(args[1]), *gs = tensor(args[2]);
    if (given && (!is(gc, at::kChar, dev, {M, K}) || !is(gs, at::kFloat, dev, {M}))) Py_RETURN_NONE;
    const OnDevice on(*x);
    if (!on.fine) return nullptr;
    at::Tensor codes, scales;
    int status;
    {
        const NoGil no_gil;
        codes = given ? *gc : at::empty({M, K}, x->options().dtype(at::kChar));
        scales = given ? *gs : at::empty({M}, x->options().dtype(at::kFloat));
        status = g.quant(x->data_ptr(), type, ptr<int8_t>(&codes), ptr<float>(&scales), (int)M, (int)K, on.stream);
    }
    if (status != Q4_OK) return PyLong_FromLong(status);
    if (given) return PyTuple_Pack(2, args[1], args[2]);
    PyObject *c = THPVariable_Wrap(codes), *s = c ? THPVariable_Wrap(scales) : nullptr;
    PyObject *both = s ? PyTuple_Pack(2, c, s) : nullptr;
    Py_XDECREF(c);
    Py_XDECREF(s);
    return both;
    END_HANDLE_TH_ERRORS
}

// init(stream_of, addresses): the entry points in the order of g.
PyObject *init(PyObject *, PyObject *args) {
    PyObject *lookup;
    unsigned long long a[5];
    if (!PyArg_ParseTuple(args, "OKKKKK", &lookup, a, a + 1, a + 2, a + 3, a + 4)) return nullptr;
    g.quant = reinterpret_cast<decltype(g.quant)>(a[0]);
    g.gemm = reinterpret_cast<decltype(g.gemm)>(a[1]);
    g.swiglu = reinterpret_cast<decltype(g.swiglu)>(a[2]);
    g.grouped = reinterpret_cast<decltype(g.grouped)>(a[3]);
    g.grouped_swiglu = reinterpret_cast<decltype(g.grouped_swiglu)>(a[4]);
    Py_INCREF(lookup);
    Py_XSETREF(stream_of, lookup);
    Py_RETURN_NONE;
}

PyMethodDef kMethods[] = {
    {"init", init, METH_VARARGS, nullptr},
    {"gemm", reinterpret_cast<PyCFunction>(reinterpret_cast<void *>(gemm)), METH_FASTCALL, nullptr},
    {"swiglu", reinterpret_cast<PyCFunction>(reinterpret_cast<void *>(swiglu)), METH_FASTCALL, nullptr},
    {"quant", reinterpret_cast<PyCFunction>(reinterpret_cast<void *>(quant)), METH_FASTCALL, nullptr},
    {nullptr, nullptr, 0, nullptr}};

PyModuleDef kModule = {PyModuleDef_HEAD_INIT, "_bind_i8", nullptr, -1, kMethods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__bind_i8() {
    PyObject *m = PyModule_Create(&kModule);
    // What the tensors' layout here is that of.
    if (m && (PyModule_AddFunctions(m, kF8Methods) < 0 || PyModule_AddStringConstant(m, "torch", BUILT_FOR_TORCH) < 0))
        Py_CLEAR(m);
    return m;
}
