// Python binding of the packed attention and int8 calls: the checks of their tensors, their outputs and
// workspaces, and the call itself, on the current stream.  These calls can take the GPU less time than
// Python takes to look at their arguments (six short prompts: 10 us of GPU time, 17.5 us of host time with
// the checks in Python and ctypes, 8 us here), so they are looked at here.
//
// Each function takes all its arguments by position (None: not given) and returns its outputs, or the
// library's status as an int where the call was refused or failed.  The library is the one that Python
// loaded: `bind` is given its entry points.
#include <ATen/ATen.h>
#include <ATen/cuda/EmptyTensor.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <climits>
#include <cstring>

#include "wan_attn.h"

namespace {

struct Library {
    decltype(&wan_attn_varlen_fwd_workspace_size) varlen_fwd_workspace_size;
    decltype(&wan_attn_varlen_fwd) varlen_fwd;
    decltype(&wan_attn_varlen_bwd_workspace_size) varlen_bwd_workspace_size;
    decltype(&wan_attn_varlen_bwd) varlen_bwd;
    decltype(&wan_int8_quantize_rows) quantize_rows;
    decltype(&wan_int8_dequantize_rows) dequantize_rows;
    decltype(&wan_int8_gemm) gemm;
    decltype(&wan_int8_linear) linear;
    decltype(&wan_int8_grad_weight) grad_weight;
    decltype(&wan_int8_grad_input) grad_input;
} lib;
constexpr int LIBRARY_ENTRIES = sizeof(Library) / sizeof(void*);

const char* type_name(at::ScalarType t) {
    switch (t) {
        case at::kBFloat16: return "bfloat16";
        case at::kFloat: return "float32";
        case at::kInt: return "int32";
        case at::kChar: return "int8";
        default: return c10::toString(t);
    }
}

// The one device that every tensor of a call is on: the current one, whose context and stream it uses.
// Asked for at the first tensor that is on a GPU at all.
struct Device {
    mutable c10::DeviceIndex index = -1;
    void check(const char* name, const at::Tensor& t) const {
        if (index < 0) index = c10::cuda::current_device();
        TORCH_CHECK_VALUE(t.get_device() == index, name, " is on ", t.device(), ", the current device is cuda:",
                          static_cast<int>(index));
    }
};

int as_int(const char* name, int64_t v) {
    TORCH_CHECK_VALUE(v <= INT_MAX, name, " is too large");
    return static_cast<int>(v);
}

// A CUDA tensor of the type, on the device.
const at::Tensor& cuda_tensor(const Device& dev, const char* name, PyObject* o, at::ScalarType type) {
    TORCH_CHECK_TYPE(THPVariable_Check(o) && THPVariable_Unpack(o).is_cuda(), name, " must be a CUDA tensor");
    const at::Tensor& t = THPVariable_Unpack(o);
    TORCH_CHECK_TYPE(t.scalar_type() == type, name, " must be ", type_name(type), ", got ", type_name(t.scalar_type()));
    dev.check(name, t);
    return t;
}

// ... contiguous, of `numel` elements (-1: any).
const at::Tensor& plain(const Device& dev, const char* name, PyObject* o, at::ScalarType type, int64_t numel = -1) {
    const at::Tensor& t = cuda_tensor(dev, name, o, type);
    TORCH_CHECK_TYPE(t.is_contiguous(), name, " must be contiguous");
    TORCH_CHECK_VALUE(numel < 0 || t.numel() == numel, name, " has ", t.numel(), " elements, expected ", numel);
    return t;
}

// Whether a contiguous tensor of shape `a` has the elements of one of shape `b` in their order: neighbouring axes
// joined ([T, H D] for [T, H, D]) or split, never exchanged.  Then every axis of the one ends where one of the
// other does.
bool same_order(at::IntArrayRef a, at::IntArrayRef b) {
    if (c10::multiply_integers(a) == 0) return true;                       // no elements
    const at::IntArrayRef few = a.size() < b.size() ? a : b, many = a.size() < b.size() ? b : a;
    int64_t end = 1, at = 1;
    size_t i = 0;
    for (const int64_t n : few) {
        end *= n;
        while (at < end && i < many.size()) at *= many[i++];
        if (at != end) return false;
    }
    return true;
}

// ... contiguous, of this shape or one of the same order.
const at::Tensor& plain(const Device& dev, const char* name, PyObject* o, at::ScalarType type, at::IntArrayRef sizes) {
    const at::Tensor& t = plain(dev, name, o, type, c10::multiply_integers(sizes));
    TORCH_CHECK_VALUE(same_order(t.sizes(), sizes), name, " has shape ", t.sizes(), ", expected ", sizes);
    return t;
}

// ... a matrix of `cols` columns (-1: any).
const at::Tensor& matrix(const Device& dev, const char* name, PyObject* o, at::ScalarType type, int64_t cols = -1) {
    const at::Tensor& t = plain(dev, name, o, type);
    TORCH_CHECK_VALUE(t.dim() == 2, name, " must be 2-D");
    TORCH_CHECK_VALUE(cols < 0 || t.size(1) == cols, name, " has ", t.size(1), " columns, expected ", cols);
    return t;
}

// An output: the tensor given, checked, or a new one of the sizes.
at::Tensor output(const Device& dev, const char* name, PyObject* o, at::ScalarType type, at::IntArrayRef sizes) {
    if (o != Py_None) return plain(dev, name, o, type, sizes);
    return at::detail::empty_cuda(sizes, type, at::Device(at::kCUDA, dev.index), std::nullopt);
}

// The element stride between rows of a tensor whose rows (all dimensions but the first) are contiguous and
// start a multiple of 8 elements apart; a single row's stride means nothing.
int64_t row_stride(const char* name, const at::Tensor& t, int64_t row) {
    if (t.is_contiguous()) return row;
    bool inner = true;
    for (int64_t d = t.dim() - 1, s = 1; d > 0; s *= t.size(d--)) inner = inner && (t.size(d) == 1 || t.stride(d) == s);
    const int64_t ld = t.size(0) == 1 ? row : t.stride(0);
    TORCH_CHECK_VALUE(inner && ld >= row && ld % 8 == 0, name,
                      " must hold each row contiguously, rows a multiple of 8 elements apart");
    return ld;
}

// bf16 [tokens, heads, D], tokens strided.
struct Rows {
    at::Tensor t;
    int64_t ld;
    void* ptr() const { return t.data_ptr(); }
};
Rows packed(const Device& dev, const char* name, PyObject* o) {
    const at::Tensor& t = cuda_tensor(dev, name, o, at::kBFloat16);
    TORCH_CHECK_VALUE(t.dim() == 3, name, " must be [tokens, heads, D]");
    return {t, row_stride(name, t, t.size(1) * t.size(2))};
}
Rows packed_like(const Device& dev, const char* name, PyObject* o, const Rows& like) {
    const Rows r = packed(dev, name, o);
    TORCH_CHECK_VALUE(r.t.sizes() == like.t.sizes(), name, " has shape ", r.t.sizes(), ", expected ", like.t.sizes());
    return r;
}
Rows packed_output(const Device& dev, const char* name, PyObject* o, const Rows& like) {
    if (o != Py_None) return packed_like(dev, name, o, like);
    return {at::detail::empty_cuda(like.t.sizes(), at::kBFloat16, like.t.device(), std::nullopt),
            like.t.size(1) * like.t.size(2)};
}

struct PackedCall {
    Device dev;
    Rows q, k, v;
    const at::Tensor &cu_q, &cu_k;
    int N, Tq, Tk, H, Hkv, D;
    explicit PackedCall(PyObject* const* a)
        : q(packed(dev, "q", a[0])), k(packed(dev, "k", a[1])), v(packed_like(dev, "v", a[2], k)),
          cu_q(plain(dev, "cu_q", a[3], at::kInt)), cu_k(plain(dev, "cu_k", a[4], at::kInt)) {
        Tq = as_int("q", q.t.size(0));
        H = as_int("q", q.t.size(1));
        D = as_int("q", q.t.size(2));
        Tk = as_int("k", k.t.size(0));
        Hkv = as_int("k", k.t.size(1));
        TORCH_CHECK_VALUE(k.t.size(2) == D && Hkv >= 1 && H % Hkv == 0, "k has shape ", k.t.sizes(),
                          ": its heads must divide q's ", H, ", its D be ", D);
        TORCH_CHECK_VALUE(cu_q.dim() == 1 && cu_q.size(0) >= 2, "cu_q must be [sequences + 1]");
        TORCH_CHECK_VALUE(cu_k.dim() == 1 && cu_k.size(0) == cu_q.size(0),
                          "cu_q and cu_k must name the same number of sequences");
        N = as_int("cu_q", cu_q.size(0) - 1);
    }
    const int* offsets(const at::Tensor& cu) const { return static_cast<const int*>(cu.data_ptr()); }
};

// The workspace given, or a new one if the call needs any.
struct Workspace {
    at::Tensor t;
    size_t bytes = 0;
    Workspace(const Device& dev, PyObject* o, size_t need) {
        if (o != Py_None) {
            TORCH_CHECK_TYPE(THPVariable_Check(o) && THPVariable_Unpack(o).is_cuda(), "workspace must be a CUDA tensor");
            t = THPVariable_Unpack(o);
            TORCH_CHECK_TYPE(t.is_contiguous(), "workspace must be contiguous");
            dev.check("workspace", t);
            bytes = t.nbytes();
        } else if (need) {
            t = at::detail::empty_cuda({static_cast<int64_t>(need)}, at::kByte, at::Device(at::kCUDA, dev.index), std::nullopt);
            bytes = need;
        }
    }
    void* ptr() const { return t.defined() ? t.data_ptr() : nullptr; }
};

void* current_stream() { return c10::cuda::getCurrentCUDAStream().stream(); }

// The library call without the interpreter's lock.
template <typename F>
int call(F f) {
    int status;
    Py_BEGIN_ALLOW_THREADS
    status = f();
    Py_END_ALLOW_THREADS
    return status;
}

template <typename... T>
PyObject* results(int status, const T&... t) {
    if (status != WAN_ATTN_OK) return PyLong_FromLong(status);
    if constexpr (sizeof...(T) == 1) {
        return THPVariable_Wrap(t...);
    } else {
        PyObject* tuple = PyTuple_New(sizeof...(T));
        if (!tuple) return nullptr;
        Py_ssize_t i = 0;
        bool ok = true;
        auto put = [&](const at::Tensor& x) {
            PyObject* o = ok ? THPVariable_Wrap(x) : nullptr;
            ok = o != nullptr;
            if (ok) PyTuple_SET_ITEM(tuple, i++, o);
        };
        (put(t), ...);
        if (!ok) Py_CLEAR(tuple);
        return tuple;
    }
}

void check_count(Py_ssize_t n, Py_ssize_t want) { TORCH_CHECK_TYPE(n == want, "expected ", want, " arguments, got ", n); }

float* floats(const at::Tensor& t) { return static_cast<float*>(t.data_ptr()); }

// q, k, v, cu_q, cu_k, causal, o, lse, workspace
PyObject* varlen_fwd(PyObject*, PyObject* const* a, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    check_count(n, 9);
    const PackedCall c(a);
    const int causal = PyObject_IsTrue(a[5]);
    if (causal < 0) throw python_error();
    const at::Tensor o = output(c.dev, "o", a[6], at::kBFloat16, {c.Tq, c.H, c.D});
    const at::Tensor lse = output(c.dev, "lse", a[7], at::kFloat, {c.H, c.Tq});
    const Workspace ws(c.dev, a[8], lib.varlen_fwd_workspace_size(c.N, c.Tq, c.Tk, c.H, c.Hkv, c.D));
    void* stream = current_stream();
    const int status = call([&] {
        return lib.varlen_fwd(c.q.ptr(), c.k.ptr(), c.v.ptr(), o.data_ptr(), floats(lse), c.offsets(c.cu_q),
                              c.offsets(c.cu_k), c.N, c.Tq, c.Tk, c.H, c.Hkv, c.D, c.q.ld, c.k.ld, c.v.ld, causal,
                              ws.ptr(), ws.bytes, stream);
    });
    return results(status, o, lse);
    END_HANDLE_TH_ERRORS
}

// q, k, v, cu_q, cu_k, causal, o, do, lse, dq, dk, dv, workspace
PyObject* varlen_bwd(PyObject*, PyObject* const* a, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    check_count(n, 13);
    const PackedCall c(a);
    const int causal = PyObject_IsTrue(a[5]);
    if (causal < 0) throw python_error();
    const at::Tensor& o = plain(c.dev, "o", a[6], at::kBFloat16, {c.Tq, c.H, c.D});
    const at::Tensor& dout = plain(c.dev, "do", a[7], at::kBFloat16, {c.Tq, c.H, c.D});
    const at::Tensor& lse = plain(c.dev, "lse", a[8], at::kFloat, {c.H, c.Tq});
    const Rows dq = packed_output(c.dev, "dq", a[9], c.q), dk = packed_output(c.dev, "dk", a[10], c.k),
               dv = packed_output(c.dev, "dv", a[11], c.k);
    const Workspace ws(c.dev, a[12], lib.varlen_bwd_workspace_size(c.N, c.Tq, c.Tk, c.H, c.Hkv, c.D));
    void* stream = current_stream();
    const int status = call([&] {
        return lib.varlen_bwd(c.q.ptr(), c.k.ptr(), c.v.ptr(), o.data_ptr(), dout.data_ptr(), floats(lse), dq.ptr(), dk.ptr(),
                              dv.ptr(), c.offsets(c.cu_q), c.offsets(c.cu_k), c.N, c.Tq, c.Tk, c.H, c.Hkv, c.D, c.q.ld,
                              c.k.ld, c.v.ld, dq.ld, dk.ld, dv.ld, causal, ws.ptr(), ws.bytes, stream);
    });
    return results(status, dq.t, dk.t, dv.t);
    END_HANDLE_TH_ERRORS
}

// bf16 x [M, K], rows strided.
struct Activations {
    const at::Tensor& x;
    int M, K;
    int64_t ld;
    Activations(const Device& dev, PyObject* o) : x(cuda_tensor(dev, "x", o, at::kBFloat16)) {
        TORCH_CHECK_VALUE(x.dim() == 2, "x must be [M, K]");
        M = as_int("x", x.size(0));
        K = as_int("x", x.size(1));
        ld = row_stride("x", x, K);
    }
};

// x, codes, scales
PyObject* int8_quantize_rows(PyObject*, PyObject* const* a, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    check_count(n, 3);
    const Device dev;
    const Activations x(dev, a[0]);
    const at::Tensor codes = output(dev, "codes", a[1], at::kChar, {x.M, x.K});
    const at::Tensor scales = output(dev, "scales", a[2], at::kFloat, {x.M});
    void* stream = current_stream();
    return results(call([&] {
        return lib.quantize_rows(x.x.data_ptr(), codes.data_ptr(), floats(scales), x.M, x.K, x.ld, stream);
    }), codes, scales);
    END_HANDLE_TH_ERRORS
}

// codes, scales, x
PyObject* int8_dequantize_rows(PyObject*, PyObject* const* a, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    check_count(n, 3);
    const Device dev;
    const at::Tensor& codes = matrix(dev, "codes", a[0], at::kChar);
    const int M = as_int("codes", codes.size(0)), K = as_int("codes", codes.size(1));
    const at::Tensor& scales = plain(dev, "scales", a[1], at::kFloat, M);
    const at::Tensor x = output(dev, "x", a[2], at::kBFloat16, {M, K});
    void* stream = current_stream();
    return results(call([&] {
        return lib.dequantize_rows(codes.data_ptr(), floats(scales), x.data_ptr(), M, K, stream);
    }), x);
    END_HANDLE_TH_ERRORS
}

// A quantised weight [N, K] and the layer's bias.
struct Weight {
    const at::Tensor& codes;
    int N;
    const at::Tensor& scales;
    const void* bias;
    Weight(const Device& dev, PyObject* codes_, PyObject* scales_, PyObject* bias_, int K)
        : codes(matrix(dev, "w_codes", codes_, at::kChar, K)), N(as_int("w_codes", codes.size(0))),
          scales(plain(dev, "w_scales", scales_, at::kFloat, N)),
          bias(bias_ == Py_None ? nullptr : plain(dev, "bias", bias_, at::kBFloat16, N).data_ptr()) {}
};

// a_codes, a_scales, w_codes, w_scales, bias, y
PyObject* int8_gemm(PyObject*, PyObject* const* a, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    check_count(n, 6);
    const Device dev;
    const at::Tensor& codes = matrix(dev, "a_codes", a[0], at::kChar);
    const int M = as_int("a_codes", codes.size(0)), K = as_int("a_codes", codes.size(1));
    const at::Tensor& scales = plain(dev, "a_scales", a[1], at::kFloat, M);
    const Weight w(dev, a[2], a[3], a[4], K);
    const at::Tensor y = output(dev, "y", a[5], at::kBFloat16, {M, w.N});
    void* stream = current_stream();
    return results(call([&] {
        return lib.gemm(codes.data_ptr(), floats(scales), w.codes.data_ptr(), floats(w.scales), w.bias, y.data_ptr(), M, w.N,
                        K, stream);
    }), y);
    END_HANDLE_TH_ERRORS
}

// x, w_codes, w_scales, bias, return_checkpoint
PyObject* int8_linear(PyObject*, PyObject* const* a, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    check_count(n, 5);
    const Device dev;
    const Activations x(dev, a[0]);
    const Weight w(dev, a[1], a[2], a[3], x.K);
    const int keep = PyObject_IsTrue(a[4]);
    if (keep < 0) throw python_error();
    const at::Device device(at::kCUDA, dev.index);
    const at::Tensor y = at::detail::empty_cuda({x.M, w.N}, at::kBFloat16, device, std::nullopt);
    void* stream = current_stream();
    auto layer = [&](void* codes, float* scales) {
        return call([&] {
            return lib.linear(x.x.data_ptr(), w.codes.data_ptr(), floats(w.scales), w.bias, y.data_ptr(), codes, scales, x.M,
                              w.N, x.K, x.ld, stream);
        });
    };
    if (keep) {
        const at::Tensor codes = at::detail::empty_cuda({x.M, x.K}, at::kChar, device, std::nullopt);
        const at::Tensor scales = at::detail::empty_cuda({x.M}, at::kFloat, device, std::nullopt);
        return results(layer(codes.data_ptr(), floats(scales)), y, codes, scales);
    }
    int status = x.M > 16 ? WAN_ATTN_ERR_WORKSPACE : layer(nullptr, nullptr);
    if (status == WAN_ATTN_ERR_WORKSPACE) {      // too large to keep the codes on the SMs: scratch for the codes,
        const int64_t codes = static_cast<int64_t>(x.M) * x.K;                // then (K % 16 == 0) the scales
        const at::Tensor scratch = at::detail::empty_cuda({codes + 4 * static_cast<int64_t>(x.M)}, at::kByte, device,
                                                          std::nullopt);
        char* s = static_cast<char*>(scratch.data_ptr());
        status = layer(s, reinterpret_cast<float*>(s + codes));
    }
    return results(status, y);
    END_HANDLE_TH_ERRORS
}

// dy, codes, scales, dw
PyObject* int8_grad_weight(PyObject*, PyObject* const* a, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    check_count(n, 4);
    const Device dev;
    const at::Tensor& dy = matrix(dev, "dy", a[0], at::kBFloat16);
    const at::Tensor& codes = matrix(dev, "codes", a[1], at::kChar);
    const int M = as_int("dy", dy.size(0)), N = as_int("dy", dy.size(1)), K = as_int("codes", codes.size(1));
    TORCH_CHECK_VALUE(codes.size(0) == M, "codes has ", codes.size(0), " rows, dy ", M);
    const at::Tensor& scales = plain(dev, "scales", a[2], at::kFloat, M);
    const at::Tensor dw = output(dev, "dw", a[3], at::kBFloat16, {N, K});
    void* stream = current_stream();
    return results(call([&] {
        return lib.grad_weight(dy.data_ptr(), codes.data_ptr(), floats(scales), dw.data_ptr(), M, N, K, stream);
    }), dw);
    END_HANDLE_TH_ERRORS
}

// dy, w_codes, w_scales, dx
PyObject* int8_grad_input(PyObject*, PyObject* const* a, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    check_count(n, 4);
    const Device dev;
    const at::Tensor& dy = matrix(dev, "dy", a[0], at::kBFloat16);
    const at::Tensor& codes = matrix(dev, "w_codes", a[1], at::kChar);
    const int M = as_int("dy", dy.size(0)), N = as_int("dy", dy.size(1)), K = as_int("w_codes", codes.size(1));
    TORCH_CHECK_VALUE(codes.size(0) == N, "w_codes has ", codes.size(0), " rows, dy ", N, " columns");
    const at::Tensor& scales = plain(dev, "w_scales", a[2], at::kFloat, N);
    const at::Tensor dx = output(dev, "dx", a[3], at::kBFloat16, {M, K});
    void* stream = current_stream();
    return results(call([&] {
        return lib.grad_input(dy.data_ptr(), codes.data_ptr(), floats(scales), dx.data_ptr(), M, N, K, stream);
    }), dx);
    END_HANDLE_TH_ERRORS
}

// The library's entry points, in Library's order, as integers.
PyObject* bind(PyObject*, PyObject* const* a, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    check_count(n, LIBRARY_ENTRIES);
    void* at[LIBRARY_ENTRIES];
    for (int i = 0; i < LIBRARY_ENTRIES; ++i) {
        at[i] = PyLong_AsVoidPtr(a[i]);
        if (PyErr_Occurred()) throw python_error();
    }
    std::memcpy(&lib, at, sizeof(lib));
    Py_RETURN_NONE;
    END_HANDLE_TH_ERRORS
}

template <PyObject* (*F)(PyObject*, PyObject* const*, Py_ssize_t)>
PyMethodDef method(const char* name) {
    return {name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(F)), METH_FASTCALL, nullptr};
}

}  // namespace

extern "C" __attribute__((visibility("default"))) PyObject* PyInit__bind() {
    static PyMethodDef methods[] = {method<bind>("bind"),
                                    method<varlen_fwd>("varlen_fwd"),
                                    method<varlen_bwd>("varlen_bwd"),
                                    method<int8_quantize_rows>("int8_quantize_rows"),
                                    method<int8_dequantize_rows>("int8_dequantize_rows"),
                                    method<int8_gemm>("int8_gemm"),
                                    method<int8_linear>("int8_linear"),
                                    method<int8_grad_weight>("int8_grad_weight"),
                                    method<int8_grad_input>("int8_grad_input"),
                                    {nullptr, nullptr, 0, nullptr}};
    static PyModuleDef module = {PyModuleDef_HEAD_INIT, "_bind", nullptr, -1, methods};
    return PyModule_Create(&module);
}
