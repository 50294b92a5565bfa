// binding.cpp -- argument marshalling of the serving stages for Python, in C++: a decoder calls them
// once per layer and token, and interpreted checks and calls cost more than the kernels run
// (norm of 8 x 1024 to 8 bits: 1.9 us on the GPU, 17 us of host time through ctypes).
//
// Each function checks its tensors, makes the outputs that were not given, and calls the C ABI on the
// current stream of the operands' device, with that device current. Refusals raise ValueError,
// a non-zero status what api.py's handler raises for it. Computes nothing.
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <ATen/core/Tensor.h>
#include <ATen/cuda/EmptyTensor.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Dtype.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <string>

#include "vit_block.h"

namespace {

// The C entry points, by address (set_entry), so that the one library that is loaded serves.
decltype(&vit_rmsnorm) p_rmsnorm;
decltype(&vit_quantize) p_quantize;
decltype(&vit_quantize_weight) p_quantize_weight;
decltype(&vit_linear_fp8) p_linear_fp8;
decltype(&vit_cross_attention) p_cross_attention;
decltype(&vit_rotary) p_rotary;
decltype(&vit_cache_append) p_cache_append;
decltype(&vit_paged_attention) p_paged_attention;
decltype(&vit_paged_attention_plan) p_paged_attention_plan;
PyObject* g_on_error;   // called with (status, name)

struct Refused : std::exception {
    std::string text;
    explicit Refused(std::string t) : text(std::move(t)) {}
    const char* what() const noexcept override { return text.c_str(); }
};

[[noreturn]] void refuse(const char* name, const std::string& why) { throw Refused(std::string(name) + why); }

// VIT_* code of an element type; with e4m3 allowed or not.
int code_of(at::ScalarType t, bool e4m3, const char* name) {
    switch (t) {
        case at::kFloat: return VIT_F32;
        case at::kBFloat16: return VIT_BF16;
        case at::kDouble: return VIT_F64;
        case at::kFloat8_e4m3fn:
            if (e4m3) return VIT_E4M3;
            break;
        default: break;
    }
    refuse(name, std::string(": unsupported dtype ") + c10::toString(t));
}

const at::Tensor& tensor(PyObject* o, const char* name) {
    if (!THPVariable_Check(o)) refuse(name, " must be a tensor");
    return THPVariable_Unpack(o);
}

std::string dims(at::IntArrayRef s) {
    std::string t = "(";
    for (size_t i = 0; i < s.size(); ++i) t += (i ? ", " : "") + std::to_string(s[i]);
    return t + ")";
}

void on_device(const at::Tensor& t, const char* name, int64_t device) {
    if (!t.is_cuda() || (device >= 0 && t.get_device() != device))
        refuse(name, " must be a CUDA tensor" + (device >= 0 ? " on cuda:" + std::to_string(device) : std::string()));
}

// A contiguous CUDA tensor of this type and shape.
void* fits(const at::Tensor& t, const char* name, at::ScalarType dt, at::IntArrayRef shape, int64_t device) {
    on_device(t, name, device);
    if (t.scalar_type() != dt)
        refuse(name, std::string(" has dtype ") + c10::toString(t.scalar_type()) + ", expected " + c10::toString(dt));
    if (t.sizes() != shape) refuse(name, " has shape " + dims(t.sizes()) + ", expected " + dims(shape));
    if (!t.is_contiguous()) refuse(name, " must be contiguous");
    return t.data_ptr();
}

// An output: the one given, checked, or a new one. `keep` holds what is returned for it.
void* output(PyObject* given, const char* name, at::ScalarType dt, at::IntArrayRef shape, const at::Tensor& like,
             PyObject** keep) {
    if (given != Py_None) {
        void* p = fits(tensor(given, name), name, dt, shape, like.get_device());
        Py_INCREF(given);
        *keep = given;
        return p;
    }
    at::Tensor t = at::detail::empty_cuda(shape, dt, like.device(), std::nullopt);
    void* p = t.data_ptr();
    *keep = THPVariable_Wrap(std::move(t));
    if (!*keep) throw python_error();
    return p;
}

at::ScalarType dtype_arg(PyObject* o, PyObject* out, at::ScalarType otherwise) {
    if (o != Py_None) {
        if (!THPDtype_Check(o)) refuse("out_dtype", " must be a torch.dtype");
        return reinterpret_cast<THPDtype*>(o)->scalar_type;
    }
    return out != Py_None ? tensor(out, "out").scalar_type() : otherwise;
}

double number(PyObject* o) {
    const double v = PyFloat_AsDouble(o);
    if (v == -1.0 && PyErr_Occurred()) throw python_error();
    return v;
}

int64_t integer(PyObject* o) {
    const long long v = PyLong_AsLongLong(o);
    if (v == -1 && PyErr_Occurred()) throw python_error();
    return v;
}

// call(stream) with the device current; raises on a non-zero status.
template <class F> void call(const char* what, int64_t device, F&& f) {
    c10::cuda::OptionalCUDAGuard guard;
    if (c10::cuda::current_device() != device) guard.set_index((c10::DeviceIndex)device);
    const int rc = f(static_cast<void*>(c10::cuda::getCurrentCUDAStream((c10::DeviceIndex)device).stream()));
    if (rc == 0) return;
    PyObject* r = PyObject_CallFunction(g_on_error, "is", rc, what);
    Py_XDECREF(r);
    throw python_error();
}

// References that a failed call gives back.
struct Kept {
    PyObject* o[3] = {nullptr, nullptr, nullptr};
    ~Kept() {
        for (PyObject* p : o) Py_XDECREF(p);
    }
    PyObject* take(int i) {
        PyObject* p = o[i];
        o[i] = nullptr;
        return p;
    }
    // the first n of them, alone or as a tuple
    PyObject* result(int n) {
        if (n == 1) return take(0);
        PyObject* t = PyTuple_New(n);
        if (!t) throw python_error();
        for (int i = 0; i < n; ++i) PyTuple_SET_ITEM(t, i, take(i));
        return t;
    }
};

int64_t blocks(int64_t n) { return (n + 127) / 128; }

// Rows and columns of a tensor (..., n) with elements.
void matrix_of(const at::Tensor& t, const char* name, int64_t* rows, int64_t* cols) {
    if (t.dim() < 1 || t.numel() == 0) refuse(name, " must have at least one element and a last dimension");
    *cols = t.sizes().back();
    *rows = t.numel() / *cols;
}

// ---- (x, eps, gamma, residual, out_dtype, out, scales, sum_out)
PyObject* rmsnorm(PyObject* const* a) {
    const at::Tensor& x = tensor(a[0], "x");
    int64_t rows, D;
    matrix_of(x, "x", &rows, &D);
    const int xc = code_of(x.scalar_type(), false, "x");
    on_device(x, "x", -1);
    if (!x.is_contiguous()) refuse("x", " must be contiguous");
    const int64_t dev = x.get_device();
    const double eps = number(a[1]);
    const at::ScalarType od = dtype_arg(a[4], a[5], x.scalar_type());
    const int oc = code_of(od, true, "out");
    const void *gp = nullptr, *rp = nullptr;
    void *sp = nullptr, *cp = nullptr;
    int gc = xc, rc = xc;
    if (a[2] != Py_None) {
        const at::Tensor& g = tensor(a[2], "gamma");
        gc = code_of(g.scalar_type(), false, "gamma");
        gp = fits(g, "gamma", g.scalar_type(), {D}, dev);
    }
    Kept k;
    const bool res = a[3] != Py_None, e4m3 = oc == VIT_E4M3;
    if (!e4m3 && a[6] != Py_None) refuse("scales", " belong to a float8_e4m3fn output");
    if (res) {
        const at::Tensor& r = tensor(a[3], "residual");
        rc = code_of(r.scalar_type(), false, "residual");
        rp = fits(r, "residual", r.scalar_type(), x.sizes(), dev);
        sp = output(a[7], "sum_out", r.scalar_type(), x.sizes(), x, &k.o[e4m3 ? 2 : 1]);
    } else if (a[7] != Py_None) {
        refuse("sum_out", " needs a residual");
    }
    void* op = output(a[5], "out", od, x.sizes(), x, &k.o[0]);
    if (e4m3) cp = output(a[6], "scales", at::kFloat, {rows, blocks(D)}, x, &k.o[1]);
    call("vit_rmsnorm", dev, [&](void* s) {
        return p_rmsnorm(x.data_ptr(), xc, rp, rc, rows, D, eps, gp, gc, sp, op, oc, static_cast<float*>(cp), s);
    });
    return k.result(1 + e4m3 + res);
}

// ---- (x, out, scales)
PyObject* quantize(PyObject* const* a) {
    const at::Tensor& x = tensor(a[0], "x");
    int64_t rows, K;
    matrix_of(x, "x", &rows, &K);
    const int xc = code_of(x.scalar_type(), false, "x");
    on_device(x, "x", -1);
    if (!x.is_contiguous()) refuse("x", " must be contiguous");
    Kept k;
    void* op = output(a[1], "out", at::kFloat8_e4m3fn, x.sizes(), x, &k.o[0]);
    void* cp = output(a[2], "scales", at::kFloat, {rows, blocks(K)}, x, &k.o[1]);
    call("vit_quantize", x.get_device(),
         [&](void* s) { return p_quantize(x.data_ptr(), xc, rows, K, op, static_cast<float*>(cp), s); });
    return k.result(2);
}

// ---- (w, out, scales)
PyObject* quantize_weight(PyObject* const* a) {
    const at::Tensor& w = tensor(a[0], "w");
    if (w.dim() != 2 || w.numel() == 0) refuse("w", " must be a matrix (K, N) with at least one element");
    const int wc = code_of(w.scalar_type(), false, "w");
    on_device(w, "w", -1);
    if (!w.is_contiguous()) refuse("w", " must be contiguous");
    const int64_t K = w.size(0), N = w.size(1);
    Kept k;
    void* op = output(a[1], "out", at::kFloat8_e4m3fn, {N, K}, w, &k.o[0]);
    void* cp = output(a[2], "scales", at::kFloat, {blocks(N), blocks(K)}, w, &k.o[1]);
    call("vit_quantize_weight", w.get_device(),
         [&](void* s) { return p_quantize_weight(w.data_ptr(), wc, K, N, op, static_cast<float*>(cp), s); });
    return k.result(2);
}

// ---- (a, a_scales, w, w_scales, bias, residual, epilogue, out_dtype, out, out_scales)
PyObject* linear_fp8(PyObject* const* a) {
    const at::Tensor &x = tensor(a[0], "a"), &w = tensor(a[2], "w");
    const int64_t epi = integer(a[6]);
    if (epi < VIT_EPI_STORE || epi > VIT_EPI_RESIDUAL) refuse("epilogue", " must be EPI_STORE, EPI_GELU or EPI_RESIDUAL");
    int64_t M, K;
    matrix_of(x, "a", &M, &K);
    if (w.dim() != 2 || w.numel() == 0) refuse("w", " must be a matrix (N, K) with at least one element");
    const int64_t N = w.size(0), kb = blocks(K), nb = blocks(N);
    if (w.size(1) != K) refuse("a", " has " + std::to_string(K) + " columns, w " + std::to_string(w.size(1)));
    on_device(x, "a", -1);
    const int64_t dev = x.get_device();
    const void* xp = fits(x, "a", at::kFloat8_e4m3fn, x.sizes(), dev);
    const void* wp = fits(w, "w", at::kFloat8_e4m3fn, w.sizes(), dev);
    const void* xs = fits(tensor(a[1], "a_scales"), "a_scales", at::kFloat, {M, kb}, dev);
    const void* ws = fits(tensor(a[3], "w_scales"), "w_scales", at::kFloat, {nb, kb}, dev);
    c10::SmallVector<int64_t, 6> shape(x.sizes().begin(), x.sizes().end());
    shape.back() = N;
    const void *bp = nullptr, *rp = nullptr;
    int bc = 0, rc = 0;
    if (a[4] != Py_None) {
        const at::Tensor& b = tensor(a[4], "bias");
        bc = code_of(b.scalar_type(), false, "bias");
        bp = fits(b, "bias", b.scalar_type(), {N}, dev);
    }
    if (a[5] != Py_None) {
        const at::Tensor& r = tensor(a[5], "residual");
        rc = code_of(r.scalar_type(), false, "residual");
        rp = fits(r, "residual", r.scalar_type(), shape, dev);
    }
    const at::ScalarType od = dtype_arg(a[7], a[8], at::kBFloat16);
    const int oc = code_of(od, true, "out");
    const bool e4m3 = oc == VIT_E4M3;
    if (!e4m3 && a[9] != Py_None) refuse("out_scales", " belong to a float8_e4m3fn output");
    Kept k;
    void *op = output(a[8], "out", od, shape, x, &k.o[0]), *sp = nullptr;
    if (e4m3) sp = output(a[9], "out_scales", at::kFloat, {M, nb}, x, &k.o[1]);
    call("vit_linear_fp8", dev, [&](void* s) {
        return p_linear_fp8(xp, static_cast<const float*>(xs), wp, static_cast<const float*>(ws), bp, bc, rp, rc, M, K, N,
                            (int)epi, op, oc, static_cast<float*>(sp), s);
    });
    return k.result(1 + e4m3);
}

// Pointer and (sequence, token, head) strides of t (B, T, heads, dh).
const void* strided(const at::Tensor& t, const char* name, at::ScalarType dt, int64_t dev, int64_t (&st)[3]) {
    on_device(t, name, dev);
    if (t.scalar_type() != dt)
        refuse(name, std::string(" has dtype ") + c10::toString(t.scalar_type()) + ", expected " + c10::toString(dt));
    const auto s = t.strides();
    if (s[3] != 1 && t.size(3) != 1) refuse(name, ": the elements of a head must be contiguous");
    for (int i = 0; i < 3; ++i) st[i] = s[i];
    return t.data_ptr();
}

// ---- (q, k, v, kv_lens, scale, out)
PyObject* cross_attention(PyObject* const* a) {
    const at::Tensor &q = tensor(a[0], "q"), &k = tensor(a[1], "k"), &v = tensor(a[2], "v");
    if (q.dim() != 4 || k.dim() != 4 || v.dim() != 4 || q.numel() == 0 || k.numel() == 0)
        refuse("q", " must be (B, Tq, H, dh) and k and v (B, Tk, Hkv, dh), with at least one element");
    const int64_t B = q.size(0), Tq = q.size(1), H = q.size(2), dh = q.size(3), Tk = k.size(1), Hkv = k.size(2);
    if (k.size(0) != B || k.size(3) != dh || v.sizes() != k.sizes())
        refuse("q ", dims(q.sizes()) + ", k " + dims(k.sizes()) + " and v " + dims(v.sizes()) + " do not fit");
    const at::ScalarType dt = q.scalar_type();
    const int code = code_of(dt, false, "q");
    on_device(q, "q", -1);
    const int64_t dev = q.get_device();
    int64_t qs[3], ks[3], vs[3];
    const void *qp = strided(q, "q", dt, dev, qs), *kp = strided(k, "k", dt, dev, ks), *vp = strided(v, "v", dt, dev, vs);
    const void* lp = nullptr;
    if (a[3] != Py_None) lp = fits(tensor(a[3], "kv_lens"), "kv_lens", at::kInt, {B}, dev);
    const double scale = number(a[4]);
    Kept keep;
    void* op = output(a[5], "out", dt, q.sizes(), q, &keep.o[0]);
    call("vit_cross_attention", dev, [&](void* s) {
        return p_cross_attention(qp, qs, kp, ks, vp, vs, static_cast<const int32_t*>(lp), B, Tq, Tk, H, Hkv, dh, scale, code,
                                 op, s);
    });
    return keep.result(1);
}

// A tensor (B, T, heads, dh) with elements; its first dimensions as given where those are set (>= 0).
const void* rows_of(const at::Tensor& t, const char* name, at::ScalarType dt, int64_t dev, int64_t B, int64_t T, int64_t heads,
                    int64_t dh, int64_t (&st)[3]) {
    if (t.dim() != 4 || t.numel() == 0) refuse(name, " must have four dimensions and at least one element");
    const int64_t want[4] = {B, T, heads, dh};
    for (int i = 0; i < 4; ++i)
        if (want[i] >= 0 && t.size(i) != want[i])
            refuse(name, " has shape " + dims(t.sizes()) + ", expected " + std::to_string(want[i]) + " in dimension " + std::to_string(i));
    return strided(t, name, dt, dev, st);
}

// A contiguous int32 CUDA tensor of this shape, or none.
const int32_t* ints(PyObject* o, const char* name, at::IntArrayRef shape, int64_t dev) {
    return o == Py_None ? nullptr : static_cast<const int32_t*>(fits(tensor(o, name), name, at::kInt, shape, dev));
}

// (frequencies, layout, scale); null where there are no frequencies
const vit_rope* rope_of(PyObject* f, PyObject* layout, PyObject* scale, int64_t dev, vit_rope* r) {
    const int64_t l = integer(layout);
    if (l != VIT_ROTARY_HALF && l != VIT_ROTARY_INTERLEAVED) refuse("layout", " must be ROTARY_HALF or ROTARY_INTERLEAVED");
    const double s = number(scale);
    if (f == Py_None) return nullptr;
    const at::Tensor& t = tensor(f, "frequencies");
    if (t.dim() != 1 || t.numel() == 0) refuse("frequencies", " must have one dimension and at least one element");
    r->frequencies = static_cast<const double*>(fits(t, "frequencies", at::kDouble, t.sizes(), dev));
    r->n = t.numel();
    r->layout = (int)l;
    r->scale = s;
    return r;
}

// Where x (B, T, H, dh) goes rotated: into a new tensor, a contiguous one that is given, or x itself. The C call takes an
// output at x's address for x, with x's strides, so one that steps otherwise is refused; dimensions of one are not stepped along.
void* turned_output(PyObject* given, const char* name, const at::Tensor& x, PyObject** keep) {
    if (given != Py_None) {
        const at::Tensor& o = tensor(given, name);
        if (o.is_cuda() && o.data_ptr() == x.data_ptr() && o.sizes() == x.sizes() && o.scalar_type() == x.scalar_type()) {
            for (int i = 0; i < 4; ++i)
                if (x.size(i) > 1 && o.stride(i) != x.stride(i))
                    refuse(name, " starts at the input's address with strides " + dims(o.strides()) + ", the input's are " + dims(x.strides()));
            Py_INCREF(given);
            *keep = given;
            return o.data_ptr();
        }
    }
    return output(given, name, x.scalar_type(), x.sizes(), x, keep);
}

// ---- (x, frequencies, positions, layout, scale, out)
PyObject* rotary(PyObject* const* a) {
    const at::Tensor& x = tensor(a[0], "x");
    const int code = code_of(x.scalar_type(), false, "x");
    on_device(x, "x", -1);
    const int64_t dev = x.get_device();
    int64_t st[3];
    const void* xp = rows_of(x, "x", x.scalar_type(), dev, -1, -1, -1, -1, st);
    vit_rope r;
    if (!rope_of(a[1], a[3], a[4], dev, &r)) refuse("frequencies", " must be a tensor");
    const int32_t* pos = ints(a[2], "positions", {x.size(0), x.size(1)}, dev);
    Kept keep;
    void* op = turned_output(a[5], "out", x, &keep.o[0]);
    call("vit_rotary", dev, [&](void* s) {
        return p_rotary(xp, st, pos, &r, x.size(0), x.size(1), x.size(2), x.size(3), code, op, s);
    });
    return keep.result(1);
}

// The pools k_pages and v_pages (pages, page, heads, dh).
vit_paged_cache cache_of(const at::Tensor& k, const at::Tensor& v) {
    vit_paged_cache c;
    const int code = code_of(k.scalar_type(), false, "k_pages");
    on_device(k, "k_pages", -1);
    const int64_t dev = k.get_device();
    c.k = const_cast<void*>(rows_of(k, "k_pages", k.scalar_type(), dev, -1, -1, -1, -1, c.k_strides));
    c.v = const_cast<void*>(rows_of(v, "v_pages", k.scalar_type(), dev, k.size(0), k.size(1), k.size(2), k.size(3), c.v_strides));
    c.pages = k.size(0);
    c.page = k.size(1);
    c.heads = k.size(2);
    c.dh = k.size(3);
    c.dtype = code;
    return c;
}

// A page table (rows, pages per row).
const int32_t* table_of(PyObject* o, const char* name, int64_t rows, int64_t dev, int64_t* pages) {
    const at::Tensor& t = tensor(o, name);
    if (t.dim() != 2 || t.numel() == 0 || (rows >= 0 && t.size(0) != rows))
        refuse(name, " has shape " + dims(t.sizes()) + ", expected a row of pages for each of " + std::to_string(rows));
    *pages = t.size(1);
    return static_cast<const int32_t*>(fits(t, name, at::kInt, t.sizes(), dev));
}

// ---- (k, v, k_pages, v_pages, table, starts, lens, q, frequencies, positions, layout, scale, q_out)
PyObject* cache_append(PyObject* const* a) {
    const at::Tensor &k = tensor(a[0], "k"), &v = tensor(a[1], "v"), &kp = tensor(a[2], "k_pages"), &vp = tensor(a[3], "v_pages");
    const vit_paged_cache c = cache_of(kp, vp);
    const at::ScalarType dt = kp.scalar_type();
    const int64_t dev = kp.get_device();
    int64_t ks[3], vs[3], qs[3], pages;
    const void* k_ = rows_of(k, "k", dt, dev, -1, -1, c.heads, c.dh, ks);
    const int64_t B = k.size(0), T = k.size(1);
    const void *v_ = rows_of(v, "v", dt, dev, B, T, c.heads, c.dh, vs), *q_ = nullptr;
    const int32_t* table = table_of(a[4], "page_table", B, dev, &pages);
    if (a[5] == Py_None) refuse("starts", " must be a tensor");
    const int32_t *starts = ints(a[5], "starts", {B}, dev), *lens = ints(a[6], "lens", {B}, dev);
    vit_rope r;
    const vit_rope* rope = rope_of(a[8], a[10], a[11], dev, &r);
    const int32_t* pos = ints(a[9], "positions", {B, T}, dev);
    Kept keep;
    void* op = nullptr;
    int64_t H = 0;
    if (a[7] != Py_None) {
        const at::Tensor& q = tensor(a[7], "q");
        q_ = rows_of(q, "q", dt, dev, B, T, -1, c.dh, qs);
        H = q.size(2);
        op = turned_output(a[12], "q_out", q, &keep.o[0]);
    } else if (a[12] != Py_None) {
        refuse("q_out", " needs a q");
    }
    call("vit_cache_append", dev, [&](void* s) {
        return p_cache_append(k_, ks, v_, vs, q_, qs, &c, table, pages, starts, lens, rope, pos, B, T, H, op, s);
    });
    if (!op) Py_RETURN_NONE;
    return keep.result(1);
}

// ---- (q, k_pages, v_pages, table, kv_lens, q_lens, prefix_table, prefix_lens, scale, out): the attention, or its plan
template <bool PLAN> PyObject* paged_attention(PyObject* const* a) {
    const at::Tensor &q = tensor(a[0], "q"), &kp = tensor(a[1], "k_pages"), &vp = tensor(a[2], "v_pages");
    const vit_paged_cache c = cache_of(kp, vp);
    const at::ScalarType dt = kp.scalar_type();
    const int64_t dev = kp.get_device();
    int64_t qs[3], pages, prefix_pages = 0, groups = 1;
    const void* q_ = rows_of(q, "q", dt, dev, -1, -1, -1, c.dh, qs);
    const int64_t B = q.size(0), T = q.size(1), H = q.size(2);
    const int32_t *table = table_of(a[3], "page_table", B, dev, &pages), *before = nullptr;
    if (a[4] == Py_None) refuse("kv_lens", " must be a tensor");
    const int32_t *kv = ints(a[4], "kv_lens", {B}, dev), *ql = ints(a[5], "q_lens", {B}, dev);
    if ((a[6] == Py_None) != (a[7] == Py_None)) refuse("prefix_table", " and prefix_lens go together");
    if (a[6] != Py_None) {
        before = table_of(a[6], "prefix_table", -1, dev, &prefix_pages);
        groups = tensor(a[6], "prefix_table").size(0);
        if (B % groups != 0) refuse("prefix_table", " has " + std::to_string(groups) + " rows, which do not divide " + std::to_string(B) + " sequences");
    }
    const int32_t* pl = ints(a[7], "prefix_lens", {groups}, dev);
    const double scale = number(a[8]);
    Kept keep;
    void* op = output(a[9], "out", dt, q.sizes(), q, &keep.o[0]);
    if constexpr (PLAN) {
        vit_paged_plan p;
        call("vit_paged_attention_plan", dev, [&](void*) {
            return p_paged_attention_plan(q_, qs, &c, table, pages, kv, ql, before, prefix_pages, pl, groups, B, T, H, scale, op, &p);
        });
        return Py_BuildValue("iiiiiiiL", p.kernel, p.prefix_kernel, p.own_parts, p.prefix_parts, p.own_rows, p.prefix_rows, p.launches,
                             (long long)p.scratch);
    }
    call("vit_paged_attention", dev, [&](void* s) {
        return p_paged_attention(q_, qs, &c, table, pages, kv, ql, before, prefix_pages, pl, groups, B, T, H, scale, op, s);
    });
    return keep.result(1);
}

template <PyObject* (*F)(PyObject* const*), int N> PyObject* entry(PyObject*, PyObject* const* args, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    if (n != N) {
        PyErr_Format(PyExc_TypeError, "takes %d arguments, got %zd", N, n);
        return nullptr;
    }
    try {
        return F(args);
    } catch (const Refused& e) {
        PyErr_SetString(PyExc_ValueError, e.what());
        return nullptr;
    }
    END_HANDLE_TH_ERRORS
}

// set_entry(on_error, addresses of the nine entry points)
PyObject* set_entry(PyObject*, PyObject* const* args, Py_ssize_t n) {
    if (n != 10) {
        PyErr_SetString(PyExc_TypeError, "set_entry takes a callable and nine addresses");
        return nullptr;
    }
    void* p[9];
    for (int i = 0; i < 9; ++i) {
        p[i] = PyLong_AsVoidPtr(args[i + 1]);
        if (PyErr_Occurred()) return nullptr;
    }
    Py_INCREF(args[0]);
    Py_XSETREF(g_on_error, args[0]);
    p_rmsnorm = reinterpret_cast<decltype(p_rmsnorm)>(p[0]);
    p_quantize = reinterpret_cast<decltype(p_quantize)>(p[1]);
    p_quantize_weight = reinterpret_cast<decltype(p_quantize_weight)>(p[2]);
    p_linear_fp8 = reinterpret_cast<decltype(p_linear_fp8)>(p[3]);
    p_cross_attention = reinterpret_cast<decltype(p_cross_attention)>(p[4]);
    p_rotary = reinterpret_cast<decltype(p_rotary)>(p[5]);
    p_cache_append = reinterpret_cast<decltype(p_cache_append)>(p[6]);
    p_paged_attention = reinterpret_cast<decltype(p_paged_attention)>(p[7]);
    p_paged_attention_plan = reinterpret_cast<decltype(p_paged_attention_plan)>(p[8]);
    Py_RETURN_NONE;
}

#define ENTRY(name, f, n) {name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(&entry<f, n>)), METH_FASTCALL, nullptr}
PyMethodDef methods[] = {ENTRY("rmsnorm", rmsnorm, 8),
                         ENTRY("quantize", quantize, 3),
                         ENTRY("quantize_weight", quantize_weight, 3),
                         ENTRY("linear_fp8", linear_fp8, 10),
                         ENTRY("cross_attention", cross_attention, 6),
                         ENTRY("rotary", rotary, 6),
                         ENTRY("cache_append", cache_append, 13),
                         ENTRY("paged_attention", paged_attention<false>, 10),
                         ENTRY("paged_attention_plan", paged_attention<true>, 10),
                         {"set_entry", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(&set_entry)), METH_FASTCALL, nullptr},
                         {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_serving", "Marshalling of the serving stages.", -1, methods,
                      nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__serving(void) { return PyModule_Create(&module); }
