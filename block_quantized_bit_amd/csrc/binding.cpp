// Python binding of the calls that a decode step makes over and over: e4m3
// product, key/value cache, routed MLP. It checks the tensors and passes their
// addresses and the current stream to the C entry points of f8.h, kv8.h and
// moe.h; nothing is computed here. In C++ because at these sizes the host
// decides the speed: through ctypes, checks and argument conversion took 12 to
// 28 us a call, the kernels 6 to 18.
#define PY_SSIZE_T_CLEAN
#include <ATen/ATen.h>
#include <c10/core/impl/VirtualGuardImpl.h>
#include <c10/hip/HIPStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include <cmath>
#include <stdexcept>
#include <string>

#include "f8.h"
#include "kv8.h"
#include "moe.h"

namespace {

struct TypeProblem : std::runtime_error {
    using std::runtime_error::runtime_error;
};
struct ValueProblem : std::runtime_error {
    using std::runtime_error::runtime_error;
};
struct PythonProblem {};  // the Python error is set

[[noreturn]] void bad(const std::string& what) { throw ValueProblem(what); }

PyObject* status_error = nullptr;  // called with (status, entry point), returns the exception

void check(int status, const char* entry) {
    if (status == Q4_OK) return;
    PyObject* e = PyObject_CallFunction(status_error, "is", status, entry);
    if (e) {
        PyErr_SetObject((PyObject*)Py_TYPE(e), e);
        Py_DECREF(e);
    }
    throw PythonProblem();
}

bool none(PyObject* o) { return o == nullptr || o == Py_None; }

const at::Tensor& tensor(PyObject* o, const char* what) {
    if (!THPVariable_Check(o)) throw TypeProblem(std::string(what) + ": expected a torch tensor");
    return THPVariable_Unpack(o);
}

long integer(PyObject* o, const char* what) {
    const long v = PyLong_AsLong(o);
    if (v == -1 && PyErr_Occurred()) throw PythonProblem();
    if (v > 0x7FFFFFFFL || v < -0x80000000L) bad(std::string(what) + ": out of range");
    return v;
}

bool truth(PyObject* o) {
    const int v = PyObject_IsTrue(o);
    if (v < 0) throw PythonProblem();
    return v == 1;
}

const c10::impl::VirtualGuardImpl& gpu() {
    static const c10::impl::VirtualGuardImpl impl(c10::DeviceType::CUDA);
    return impl;
}

// The GPU that holds t; it has to be the current one, on whose stream the kernels are put.
c10::Device device_of(const at::Tensor& t, const char* what) {
    if (!t.is_cuda()) bad(std::string(what) + ": tensors must live on the GPU");
    const c10::Device d = t.device(), now = gpu().getDevice();
    if (d.index() != now.index())
        bad(std::string(what) + ": the tensor is on GPU " + std::to_string(d.index()) + ", the current one is " +
            std::to_string(now.index()));
    return d;
}

// The stream of a call: the current one, or the one given (any object with a `cuda_stream` handle), which is then the
// current one while this lives. Workspaces and results that the call allocates so belong to the stream that uses them:
// the allocator may hand a workspace's memory on as soon as the call returns, but only to later work of that stream.
class OnStream {
  public:
    OnStream(PyObject* stream, c10::Device dev) : before_(c10::hip::getCurrentHIPStream(dev.index())) {
        if (none(stream)) {
            handle = before_.stream();
            return;
        }
        PyObject* h = PyObject_GetAttrString(stream, "cuda_stream");
        if (!h) throw PythonProblem();
        handle = PyLong_AsVoidPtr(h);
        Py_DECREF(h);
        if (!handle && PyErr_Occurred()) throw PythonProblem();
        if (handle == before_.stream()) return;
        c10::hip::setCurrentHIPStream(c10::hip::getStreamFromExternal((hipStream_t)handle, dev.index()));
        moved_ = true;
    }
    ~OnStream() {
        if (moved_) c10::hip::setCurrentHIPStream(before_);
    }
    OnStream(const OnStream&) = delete;
    OnStream& operator=(const OnStream&) = delete;

    void* handle;

  private:
    c10::hip::HIPStream before_;
    bool moved_ = false;
};

int dtype_of(const at::Tensor& t, const char* what) {
    if (t.scalar_type() == at::kFloat) return Q4_DT_F32;
    if (t.scalar_type() == at::kBFloat16) return Q4_DT_BF16;
    bad(std::string(what) + ": unsupported dtype " + c10::toString(t.scalar_type()) + " (float32 or bfloat16)");
}

std::string text(at::IntArrayRef v) {
    std::string s = "(";
    for (size_t i = 0; i < v.size(); ++i) s += (i ? ", " : "") + std::to_string(v[i]);
    return s + ")";
}

// Address of a contiguous tensor of this shape and dtype on the call's GPU.
void* pointer(const at::Tensor& t, c10::Device dev, at::IntArrayRef shape, at::ScalarType dtype, const char* what) {
    if (t.device() != dev) bad(std::string(what) + ": must live on GPU " + std::to_string(dev.index()));
    if (t.scalar_type() != dtype)
        bad(std::string(what) + ": expected " + c10::toString(dtype) + ", got " + c10::toString(t.scalar_type()));
    if (t.sizes() != shape) bad(std::string(what) + ": expected shape " + text(shape) + ", got " + text(t.sizes()));
    if (!t.is_contiguous()) bad(std::string(what) + ": must be contiguous");
    return t.data_ptr();
}
void* pointer(PyObject* o, c10::Device dev, at::IntArrayRef shape, at::ScalarType dtype, const char* what) {
    return pointer(tensor(o, what), dev, shape, dtype, what);
}

at::Tensor fresh(c10::Device dev, at::IntArrayRef shape, at::ScalarType dtype) {
    return at::empty(shape, at::TensorOptions().device(dev).dtype(dtype));
}

// The caller's workspace if it is large enough, or a new one.
at::Tensor workspace(PyObject* o, size_t bytes, c10::Device dev) {
    if (none(o)) return fresh(dev, {(int64_t)bytes}, at::kByte);
    const at::Tensor& t = tensor(o, "work");
    if (t.device() != dev || !t.is_contiguous())
        bad("work: must be contiguous and live on GPU " + std::to_string(dev.index()));
    if (t.nbytes() < bytes) bad("workspace needs " + std::to_string(bytes) + " bytes");
    return t;
}

at::Tensor given_or_fresh(PyObject* o, c10::Device dev, at::IntArrayRef shape, at::ScalarType dtype) {
    return none(o) ? fresh(dev, shape, dtype) : tensor(o, "out");
}

template <typename F>
PyObject* guarded(F f) {
    try {
        return f();
    } catch (const PythonProblem&) {
    } catch (const TypeProblem& e) {
        PyErr_SetString(PyExc_TypeError, e.what());
    } catch (const ValueProblem& e) {
        PyErr_SetString(PyExc_ValueError, e.what());
    } catch (const c10::OutOfMemoryError& e) {
        PyErr_SetString(PyExc_MemoryError, e.what_without_backtrace());
    } catch (const std::exception& e) {
        PyErr_SetString(PyExc_RuntimeError, e.what());
    }
    return nullptr;
}

int64_t up128(int64_t v) { return (v + 127) / 128 * 128; }

// ---- e4m3 product -------------------------------------------------------------------

struct Rows {
    int dtype;
    int64_t M, K, stride;
    const void* p;
};

// A matrix with contiguous rows, which may be a slice of a wider one.
Rows rows_of(const at::Tensor& x, c10::Device dev, const char* what) {
    Rows r;
    r.dtype = dtype_of(x, what);
    if (x.device() != dev) bad(std::string(what) + ": must live on GPU " + std::to_string(dev.index()));
    if (x.dim() != 2 || x.size(0) < 1 || x.size(1) < 1)
        bad(std::string(what) + ": expected a matrix [rows][columns], got " + text(x.sizes()));
    r.M = x.size(0);
    r.K = x.size(1);
    r.stride = r.M > 1 ? x.stride(0) : r.K;
    if ((r.K > 1 && x.stride(1) != 1) || r.stride < r.K)
        bad(std::string(what) + ": the values of a row must be contiguous and rows must not overlap");
    if (r.M > 0x7FFFFFFF || r.K > 0x7FFFFFFF) bad(std::string(what) + ": too large");
    r.p = x.data_ptr();
    return r;
}

// (x, wq, ws, out, work, stream) -> out
PyObject* linear(PyObject*, PyObject* const* a, Py_ssize_t) {
    return guarded([&]() -> PyObject* {
        const at::Tensor &x = tensor(a[0], "x"), &wq = tensor(a[1], "wq");
        const c10::Device dev = device_of(x, "x");
        const OnStream on(a[5], dev);
        const Rows r = rows_of(x, dev, "x");
        if (wq.dim() != 2) bad("wq: expected [N][K padded to 128]");
        const int64_t N = wq.size(0), Kp = up128(r.K);
        const void* pq = pointer(wq, dev, {N, Kp}, at::kFloat8_e4m3fn, "wq");
        const void* ps = pointer(a[2], dev, {up128(N) / 128, Kp / 128}, at::kFloat, "ws");
        const at::Tensor out = given_or_fresh(a[3], dev, {r.M, N}, x.scalar_type());
        void* po = pointer(out, dev, {r.M, N}, x.scalar_type(), "out");
        const at::Tensor work = workspace(a[4], f8_linear_work_bytes((int)r.M, (int)r.K), dev);
        check(f8_linear((int)r.M, (int)r.K, (int)N, r.dtype, r.p, r.stride, (const uint8_t*)pq, (const float*)ps, po,
                        work.data_ptr(), on.handle),
              "f8_linear");
        return THPVariable_Wrap(out);
    });
}

// (dy, x, wqt, wst, dx, dw, need_dx, need_dw, work, stream) -> (dx, dw)
PyObject* linear_backward(PyObject*, PyObject* const* a, Py_ssize_t) {
    return guarded([&]() -> PyObject* {
        const at::Tensor& dy = tensor(a[0], "dy");
        const c10::Device dev = device_of(dy, "dy");
        const OnStream on(a[9], dev);
        const Rows d = rows_of(dy, dev, "dy");
        const bool need_dx = truth(a[6]), need_dw = truth(a[7]);
        const auto type = dy.scalar_type();
        Rows x{d.dtype, d.M, 0, 0, nullptr};
        if (need_dw || !none(a[1])) {
            x = rows_of(tensor(a[1], "x"), dev, "x");
            if (x.dtype != d.dtype || x.M != d.M) bad("dy and x disagree on dtype or rows");
        } else {
            x.K = x.stride = tensor(a[2], "wqt").size(0);
        }
        const void *pq = nullptr, *ps = nullptr;
        void *pdx = nullptr, *pdw = nullptr;
        int dwtype = d.dtype;
        at::Tensor dx, dw;
        if (need_dx) {
            pq = pointer(a[2], dev, {x.K, up128(d.K)}, at::kFloat8_e4m3fn, "wqt");
            ps = pointer(a[3], dev, {up128(x.K) / 128, up128(d.K) / 128}, at::kFloat, "wst");
            dx = given_or_fresh(a[4], dev, {d.M, x.K}, type);
            pdx = pointer(dx, dev, {d.M, x.K}, type, "dx");
        }
        if (need_dw) {
            dw = given_or_fresh(a[5], dev, {d.K, x.K}, type);
            dwtype = dtype_of(dw, "dw");
            pdw = pointer(dw, dev, {d.K, x.K}, dw.scalar_type(), "dw");
        }
        const at::Tensor work = workspace(a[8], f8_linear_backward_work_bytes((int)d.M, (int)x.K, (int)d.K), dev);
        check(f8_linear_backward((int)d.M, (int)x.K, (int)d.K, d.dtype, d.p, d.stride, x.p, x.stride,
                                 (const uint8_t*)pq, (const float*)ps, pdx, dwtype, pdw, work.data_ptr(),
                                 on.handle),
              "f8_linear_backward");
        PyObject* first = need_dx ? THPVariable_Wrap(dx) : (Py_INCREF(Py_None), Py_None);
        PyObject* second = need_dw ? THPVariable_Wrap(dw) : (Py_INCREF(Py_None), Py_None);
        PyObject* both = PyTuple_Pack(2, first, second);
        Py_XDECREF(first);
        Py_XDECREF(second);
        return both;
    });
}

// ---- 8-bit cache ----------------------------------------------------------------------

// k_codes, v_codes, k_scale, v_scale, page_table, kv_len, cu
c10::Device cache_of(PyObject* const* a, kv8_cache& c) {
    const at::Tensor &k = tensor(a[0], "k_codes"), &table = tensor(a[4], "page_table");
    const c10::Device dev = device_of(k, "k_codes");
    const auto kind = k.scalar_type();
    if (kind == at::kChar)
        c.format = KV8_INT8;
    else if (kind == at::kFloat8_e4m3fn)
        c.format = KV8_E4M3;
    else
        bad(std::string("k_codes: unsupported dtype ") + c10::toString(kind) + " (int8 or float8_e4m3fn)");
    if (k.dim() != 4) bad("k_codes: expected [pages][kv heads][page size][head size]");
    if (table.dim() != 2) bad("page_table: expected [sequences][pages of a sequence]");
    const int64_t pages = k.size(0), H = k.size(1), P = k.size(2), D = k.size(3), B = table.size(0), most = table.size(1);
    for (int64_t v : {pages, H, P, D, B, most})
        if (v > 0x7FFFFFFF) bad("the cache is too large");
    c.pages = (int)pages;
    c.kv_heads = (int)H;
    c.page_size = (int)P;
    c.head_dim = (int)D;
    c.batch = (int)B;
    c.max_pages = (int)most;
    c.k_codes = pointer(k, dev, {pages, H, P, D}, kind, "k_codes");
    c.v_codes = pointer(a[1], dev, {pages, H, D, P}, kind, "v_codes");
    c.k_scale = (float*)pointer(a[2], dev, {pages, H}, at::kFloat, "k_scale");
    c.v_scale = (float*)pointer(a[3], dev, {pages, H}, at::kFloat, "v_scale");
    c.page_table = (const int32_t*)pointer(table, dev, {B, most}, at::kInt, "page_table");
    c.kv_len = (const int32_t*)pointer(a[5], dev, {B}, at::kInt, "kv_len");
    c.cu = (const int32_t*)pointer(a[6], dev, {B + 1}, at::kInt, "cu");
    return dev;
}

// Row stride of packed tokens [total][heads][D]; rows may be strided (a slice of a wider projection).
int64_t tokens_of(const at::Tensor& x, c10::Device dev, int64_t heads, int64_t D, const char* what) {
    if (x.device() != dev) bad(std::string(what) + ": must live on GPU " + std::to_string(dev.index()));
    if (x.dim() != 3 || x.size(1) != heads || x.size(2) != D || x.size(0) < 1 || x.size(0) > 0x7FFFFFFF)
        bad(std::string(what) + ": expected [tokens][" + std::to_string(heads) + "][" + std::to_string(D) + "], got " +
            text(x.sizes()));
    const int64_t stride = x.size(0) > 1 ? x.stride(0) : heads * D;
    if (x.stride(2) != 1 || (heads > 1 && x.stride(1) != D) || stride < heads * D)
        bad(std::string(what) + ": the heads of a token must be contiguous and tokens must not overlap");
    return stride;
}

// (k, v, cache x 7, max_new, stream)
PyObject* append(PyObject*, PyObject* const* a, Py_ssize_t) {
    return guarded([&]() -> PyObject* {
        kv8_cache c;
        const c10::Device dev = cache_of(a + 2, c);
        const OnStream on(a[10], dev);
        const at::Tensor &k = tensor(a[0], "k"), &v = tensor(a[1], "v");
        const int64_t ks = tokens_of(k, dev, c.kv_heads, c.head_dim, "k");
        const int64_t vs = tokens_of(v, dev, c.kv_heads, c.head_dim, "v");
        if (v.scalar_type() != k.scalar_type() || v.size(0) != k.size(0)) bad("k and v disagree on dtype or tokens");
        check(kv8_append(&c, (int)k.size(0), (int)integer(a[9], "max_new"), dtype_of(k, "k"), k.data_ptr(), ks,
                         v.data_ptr(), vs, on.handle),
              "kv8_append");
        Py_RETURN_NONE;
    });
}

// (cache x 7, max_new, k_out, v_out, stream)
PyObject* read(PyObject*, PyObject* const* a, Py_ssize_t) {
    return guarded([&]() -> PyObject* {
        kv8_cache c;
        const c10::Device dev = cache_of(a, c);
        const OnStream on(a[10], dev);
        const at::Tensor &k = tensor(a[8], "out[0]"), &v = tensor(a[9], "out[1]");
        const int dt = dtype_of(k, "out[0]");
        if (k.dim() != 3 || k.size(0) < 1 || k.size(0) > 0x7FFFFFFF) bad("out[0]: expected [tokens][kv heads][head size]");
        void* pk = pointer(k, dev, {k.size(0), c.kv_heads, c.head_dim}, k.scalar_type(), "out[0]");
        void* pv = pointer(v, dev, {k.size(0), c.kv_heads, c.head_dim}, k.scalar_type(), "out[1]");
        check(kv8_read(&c, (int)k.size(0), (int)integer(a[7], "max_new"), dt, pk, pv, on.handle), "kv8_read");
        Py_RETURN_NONE;
    });
}

// (q, cache x 7, max_new, max_kv, scale, window, out, lse, work, stream) -> out
PyObject* attention(PyObject*, PyObject* const* a, Py_ssize_t) {
    return guarded([&]() -> PyObject* {
        kv8_cache c;
        const c10::Device dev = cache_of(a + 1, c);
        const OnStream on(a[15], dev);
        const at::Tensor& q = tensor(a[0], "q");
        if (q.dim() != 3) bad("q: expected [tokens][heads][head size]");
        const int64_t total = q.size(0), heads = q.size(1), D = c.head_dim;
        if (heads == 0 || c.kv_heads == 0 || heads % c.kv_heads)
            bad("q: " + std::to_string(heads) + " heads are no multiple of the cache's " + std::to_string(c.kv_heads));
        const int64_t stride = tokens_of(q, dev, heads, D, "q");
        const int dt = dtype_of(q, "q");
        const int max_new = (int)integer(a[8], "max_new"), max_kv = (int)integer(a[9], "max_kv");
        double scale = 0.0;
        if (!none(a[10])) {
            scale = PyFloat_AsDouble(a[10]);
            if (scale == -1.0 && PyErr_Occurred()) throw PythonProblem();
        } else {
            scale = 1.0 / std::sqrt((double)D);
        }
        const int window = (int)integer(a[11], "window");
        const at::Tensor out = given_or_fresh(a[12], dev, {total, heads, D}, q.scalar_type());
        void* po = pointer(out, dev, {total, heads, D}, q.scalar_type(), "out");
        float* lse = none(a[13]) ? nullptr : (float*)pointer(a[13], dev, {total, heads}, at::kFloat, "lse");
        const at::Tensor work =
            workspace(a[14], kv8_attention_work_bytes(&c, (int)total, max_new, max_kv, (int)heads), dev);
        check(kv8_attention(&c, (int)total, max_new, max_kv, (int)heads, dt, q.data_ptr(), stride, (float)scale, window,
                            po, lse, work.data_ptr(), on.handle),
              "kv8_attention");
        return THPVariable_Wrap(out);
    });
}

// ---- routed MLP -----------------------------------------------------------------------

// (x, logits, w13, s13, b13, w2, s2, b2, top_k, fmt, bs, renormalize, out, work, stream) -> out
PyObject* moe(PyObject*, PyObject* const* a, Py_ssize_t) {
    return guarded([&]() -> PyObject* {
        const at::Tensor &x = tensor(a[0], "x"), &logits = tensor(a[1], "logits"), &w13 = tensor(a[2], "w13");
        const c10::Device dev = device_of(x, "x");
        const OnStream on(a[14], dev);
        const int dt = dtype_of(x, "x");
        if (x.dim() != 2 || logits.dim() != 2 || w13.dim() != 3)
            bad("expected x [T][H], logits [T][E], w13 [E][2I][H/2]");
        const int64_t T = x.size(0), H = x.size(1), E = w13.size(0), two = w13.size(1), I = two / 2;
        const int top_k = (int)integer(a[8], "top_k"), fmt = (int)integer(a[9], "fmt"), bs = (int)integer(a[10], "bs");
        if ((bs != 32 && bs != 64 && bs != 128) || H % bs || I % bs || two % 2)
            bad("H (" + std::to_string(H) + ") and I (" + std::to_string(I) + ") must be multiples of the block size (" +
                std::to_string(bs) + ": 32 for q4_0, 64 or 128 for affine)");
        if (T > 64 || H > 32768 || E > 512 || I > 32768) check(Q4_ERR_DIM, "moe_q4");
        const auto st = fmt == Q4_FMT_Q4_0 ? at::kHalf : at::kBFloat16;
        const void* px = pointer(x, dev, {T, H}, x.scalar_type(), "x");
        const void* pl = pointer(logits, dev, {T, E}, at::kFloat, "logits");
        const void* p13 = pointer(w13, dev, {E, two, H / 2}, at::kByte, "w13");
        const void* ps13 = pointer(a[3], dev, {E, two, H / bs}, st, "s13");
        const void* p2 = pointer(a[5], dev, {E, H, I / 2}, at::kByte, "w2");
        const void* ps2 = pointer(a[6], dev, {E, H, I / bs}, st, "s2");
        const void *pb13 = nullptr, *pb2 = nullptr;
        if (fmt != Q4_FMT_Q4_0) {
            pb13 = pointer(a[4], dev, {E, two, H / bs}, st, "b13");
            pb2 = pointer(a[7], dev, {E, H, I / bs}, st, "b2");
        }
        const at::Tensor out = given_or_fresh(a[12], dev, {T, H}, x.scalar_type());
        void* po = pointer(out, dev, {T, H}, x.scalar_type(), "out");
        const at::Tensor work =
            workspace(a[13], moe_q4_work_bytes((int)T, (int)H, (int)I, (int)E, top_k, bs), dev);
        check(moe_q4((int)T, (int)H, (int)I, (int)E, top_k, bs, fmt, dt, px, (const float*)pl, (const uint8_t*)p13, ps13,
                     pb13, (const uint8_t*)p2, ps2, pb2, truth(a[11]), po, work.data_ptr(),
                     on.handle),
              "moe_q4");
        return THPVariable_Wrap(out);
    });
}

// Each function is called by this package's Python wrappers alone, with all its arguments in order.
template <PyObject* (*F)(PyObject*, PyObject* const*, Py_ssize_t), int N>
PyObject* counted(PyObject* self, PyObject* const* a, Py_ssize_t n) {
    if (n != N) {
        PyErr_Format(PyExc_TypeError, "expected %d arguments, got %zd", N, n);
        return nullptr;
    }
    return F(self, a, n);
}

PyObject* set_status_error(PyObject*, PyObject* f) {
    Py_XDECREF(status_error);
    Py_INCREF(f);
    status_error = f;
    Py_RETURN_NONE;
}

#define CALL(f, n) (PyCFunction)(void (*)(void)) counted<f, n>, METH_FASTCALL, nullptr
PyMethodDef methods[] = {{"f8_linear", CALL(linear, 6)},
                         {"f8_linear_backward", CALL(linear_backward, 10)},
                         {"kv8_append", CALL(append, 11)},
                         {"kv8_read", CALL(read, 11)},
                         {"kv8_attention", CALL(attention, 16)},
                         {"moe_q4", CALL(moe, 15)},
                         {"set_status_error", set_status_error, METH_O, nullptr},
                         {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_native", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__native(void) { return PyModule_Create(&module); }
