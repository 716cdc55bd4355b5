// ds_torch.cpp -- the torch side of the Python binding for the operators around the top-k:
// checks of the argument tensors, outputs from torch's allocator, the current stream, and the
// call of the C ABI.  A call costs the host one pass through this file (4.2 to 4.6 us for the
// gate; the same steps in Python with ctypes took 14), which is what a decoding step's small calls wait for.
// Every function here takes its arguments by position from the documented Python function of the
// same name.  The tensors' device is current for the length of a call, whichever was before: the C ABI
// launches on the current one.
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <ATen/core/Tensor.h>
#include <ATen/cuda/EmptyTensor.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <cmath>
#include <initializer_list>
#include <optional>
#include <string>

#include "ds_topk.h"

namespace {

PyObject* g_error = nullptr;  // the package's DSError

struct Refused {  // an argument that is refused: the Python exception to raise
    PyObject* type;
    std::string what;
};
[[noreturn]] void refuse_type(std::string what) { throw Refused{PyExc_TypeError, std::move(what)}; }
[[noreturn]] void refuse(std::string what) { throw Refused{PyExc_ValueError, std::move(what)}; }
struct PythonError {};  // an error that is set already
struct Failed {         // a status of the C ABI
    int status;
    const char* what;
};

std::string shape_text(at::IntArrayRef s) {
    std::string t = "(";
    for (size_t i = 0; i < s.size(); ++i) t += (i ? ", " : "") + std::to_string(s[i]);
    return t + (s.size() == 1 ? ",)" : ")");
}

const at::Tensor& tensor(PyObject* o, const char* what) {
    if (!THPVariable_Check(o)) refuse_type(std::string(what) + " must be a tensor, not " + Py_TYPE(o)->tp_name);
    return THPVariable_Unpack(o);
}

int64_t integer(PyObject* o) {
    const int64_t v = PyLong_AsLongLong(o);
    if (v == -1 && PyErr_Occurred()) throw PythonError{};
    return v;
}
int32_t integer32(PyObject* o, const char* what) {
    const int64_t v = integer(o);
    if (v != static_cast<int32_t>(v)) refuse(std::string(what) + " does not fit 32 bits");
    return static_cast<int32_t>(v);
}
float real(PyObject* o) {
    const double v = PyFloat_AsDouble(o);
    if (v == -1.0 && PyErr_Occurred()) throw PythonError{};
    return static_cast<float>(v);
}
bool truth(PyObject* o) {
    const int v = PyObject_IsTrue(o);
    if (v < 0) throw PythonError{};
    return v != 0;
}

// The argument the others follow: a CUDA tensor of `dims` dimensions with a unit last stride.
const at::Tensor& leading(PyObject* o, const char* what, int64_t dims) {
    const at::Tensor& t = tensor(o, what);
    if (!t.is_cuda()) refuse(std::string(what) + " must be a CUDA tensor (there is no CPU path)");
    if (t.dim() != dims)
        refuse(std::string(what) + " must have " + std::to_string(dims) + " dimensions, not " + std::to_string(t.dim()));
    if (!t.is_contiguous() && t.stride(-1) != 1)
        refuse(std::string(what) + " must have unit stride in its last dimension");
    return t;
}

int32_t float_code(const at::Tensor& t, const char* what) {
    if (t.scalar_type() == at::kBFloat16) return DS_BF16;
    if (t.scalar_type() == at::kFloat) return DS_FP32;
    refuse_type(std::string(what) + ": unsupported dtype " + c10::toString(t.scalar_type()) + ": bfloat16 and float32 only");
}

// Any other argument: type, shape, device, and contiguity or (strided) a unit last stride.
const at::Tensor& want(PyObject* o, const char* what, std::initializer_list<int64_t> shape, at::ScalarType type,
                       c10::DeviceIndex index, bool strided = false) {
    const at::Tensor& t = tensor(o, what);
    const at::IntArrayRef s(shape.begin(), shape.size());
    if (t.scalar_type() != type)
        refuse_type(std::string(what) + " must have dtype " + c10::toString(type) + ", not " + c10::toString(t.scalar_type()));
    if (t.sizes() != s) refuse(std::string(what) + " must have shape " + shape_text(s) + ", not " + shape_text(t.sizes()));
    if (!t.is_cuda() || t.get_device() != index)
        refuse(std::string(what) + " must be on cuda:" + std::to_string(index) + " (there is no CPU path)");
    if (!t.is_contiguous() && !(strided && t.stride(-1) == 1))
        refuse(std::string(what) + (strided ? " must have unit stride in its last dimension" : " must be contiguous"));
    return t;
}

// Where a call runs: the tensors' device, made current, and its current stream or the caller's.  Another
// stream than the current one is torch's current stream for the length of the call, so that outputs
// come from its memory: what the current stream still has to do with memory that it has freed does
// not meet them.  Outputs count as used on the current stream as well, where the caller goes on.
class Place {
    c10::cuda::CUDAGuard device_;
    c10::cuda::CUDAStream here_;
    std::optional<c10::cuda::CUDAStreamGuard> other_;
    cudaStream_t stream_;

   public:
    Place(PyObject* o, c10::DeviceIndex index)
        : device_(index), here_(c10::cuda::getCurrentCUDAStream(index)), stream_(here_.stream()) {
        if (o == Py_None) return;
        void* p = PyLong_AsVoidPtr(o);
        if (!p && PyErr_Occurred()) throw PythonError{};
        if (p == stream_) return;
        stream_ = static_cast<cudaStream_t>(p);
        other_.emplace(c10::cuda::getStreamFromExternal(stream_, index));
    }
    cudaStream_t stream() const { return stream_; }
    at::Tensor make(std::initializer_list<int64_t> shape, at::ScalarType type) const {
        at::Tensor t = at::detail::empty_cuda(at::IntArrayRef(shape.begin(), shape.size()), type, here_.device(), std::nullopt);
        if (other_) t.record_stream(here_);
        return t;
    }
    // bytes that only the call itself uses: a graph that is being captured gets its own
    at::Tensor scratch(size_t bytes) const {
        if (bytes == 0) return {};
        return at::detail::empty_cuda(static_cast<int64_t>(bytes), at::kByte, here_.device(), std::nullopt);
    }
};

void check(int status, const char* what) {
    if (status != DS_OK) throw Failed{status, what};
}

template <typename T>
T* data(const at::Tensor& t) { return static_cast<T*>(t.data_ptr()); }

PyObject* tuple_of(std::initializer_list<at::Tensor> list) {
    PyObject* out = PyTuple_New(static_cast<Py_ssize_t>(list.size()));
    if (!out) throw PythonError{};
    Py_ssize_t i = 0;
    for (const at::Tensor& t : list) {
        PyObject* v = THPVariable_Wrap(t);
        if (!v) {
            Py_DECREF(out);
            throw PythonError{};
        }
        PyTuple_SET_ITEM(out, i++, v);
    }
    return out;
}

// Runs a call's body and turns what it throws into Python exceptions.
template <typename Body>
PyObject* guarded(Py_ssize_t given, Py_ssize_t wanted, Body body) {
    HANDLE_TH_ERRORS
    if (given != wanted) {
        PyErr_Format(PyExc_TypeError, "%zd arguments given, %zd wanted", given, wanted);
        return nullptr;
    }
    try {
        return body();
    } catch (const Refused& r) {
        PyErr_SetString(r.type, r.what.c_str());
    } catch (const PythonError&) {
    } catch (const Failed& f) {
        PyObject* e = g_error ? PyObject_CallFunction(g_error, "is", f.status, f.what) : nullptr;
        if (e) {
            PyErr_SetObject(g_error, e);
            Py_DECREF(e);
        } else if (!PyErr_Occurred()) {
            PyErr_Format(PyExc_RuntimeError, "%s failed: %s", f.what, ds_status_string(static_cast<ds_status>(f.status)));
        }
    }
    return nullptr;
    END_HANDLE_TH_ERRORS
}

using Args = PyObject* const*;

PyObject* route(PyObject*, Args a, Py_ssize_t n) {
    return guarded(n, 11, [&]() -> PyObject* {
        const at::Tensor& x = leading(a[0], "logits", 2);
        const int32_t code = float_code(x, "logits"), k = integer32(a[1], "k");
        const int64_t rows = x.size(0), E = x.size(1);
        const auto index = x.get_device();
        const Place place(a[10], index);
        const float* bias = a[3] == Py_None ? nullptr : data<float>(want(a[3], "bias", {E}, at::kFloat, index));
        int32_t* counts = a[9] == Py_None ? nullptr : data<int32_t>(want(a[9], "counts", {E}, at::kInt, index));
        if (E > 0x7FFFFFFF) refuse("logits has too many columns");
        const int64_t width = k > 0 ? k : 0;
        const at::Tensor w = place.make({rows, width}, at::kFloat), e = place.make({rows, width}, at::kInt);
        check(ds_route(x.data_ptr(), code, rows, static_cast<int32_t>(E), rows > 1 ? x.stride(0) : E, k,
                       integer32(a[2], "scoring"), bias, integer32(a[4], "groups"), integer32(a[5], "topk_groups"),
                       integer32(a[6], "group_score"), truth(a[7]), real(a[8]), data<float>(w), data<int32_t>(e), counts,
                       place.stream()), "ds_route");
        return tuple_of({w, e});
    });
}

PyObject* route_backward(PyObject*, Args a, Py_ssize_t n) {
    return guarded(n, 7, [&]() -> PyObject* {
        const at::Tensor& x = leading(a[1], "logits", 2);
        const int32_t code = float_code(x, "logits");
        const int64_t rows = x.size(0), E = x.size(1);
        const auto index = x.get_device();
        const Place place(a[6], index);
        const at::Tensor& chosen = tensor(a[2], "experts");
        const int64_t k = chosen.dim() > 0 ? chosen.size(-1) : 0;
        const at::Tensor& experts = want(a[2], "experts", {rows, k}, at::kInt, index);
        const at::Tensor& grad = want(a[0], "grad_weights", {rows, k}, at::kFloat, index);
        if (E > 0x7FFFFFFF || k > 0x7FFFFFFF) refuse("logits or experts has too many columns");
        const at::Tensor out = place.make({rows, E}, x.scalar_type());
        check(ds_route_backward(data<float>(grad), x.data_ptr(), code, rows, static_cast<int32_t>(E),
                                rows > 1 ? x.stride(0) : E, static_cast<int32_t>(k), data<int32_t>(experts),
                                integer32(a[3], "scoring"), truth(a[4]), real(a[5]), out.data_ptr(), E,
                                place.stream()), "ds_route_backward");
        return THPVariable_Wrap(out);
    });
}

PyObject* verify_drafts(PyObject*, Args a, Py_ssize_t n) {
    return guarded(n, 8, [&]() -> PyObject* {
        const at::Tensor& x = leading(a[0], "logits", 3);
        const int32_t code = float_code(x, "logits");
        const int64_t B = x.size(0), rows = x.size(1), V = x.size(2), S = rows - 1;
        if (S < 0) refuse("logits must have at least one row per sequence");
        if (S > 0x7FFFFFFE) refuse("logits has too many rows per sequence");
        const auto index = x.get_device();
        const Place place(a[7], index);
        const at::Tensor& drafts = want(a[1], "drafts", {B, S}, at::kInt, index);
        const at::Tensor& uniforms = want(a[2], "uniforms", {B, S}, at::kFloat, index);
        const at::Tensor& noise = want(a[3], "noise", {B, V}, at::kFloat, index, true);
        const float* q = nullptr;
        int64_t q_seq = 0, q_row = V;
        if (a[4] != Py_None) {
            const at::Tensor& t = want(a[4], "draft_probs", {B, S, V}, at::kFloat, index, true);
            q = data<float>(t);
            q_seq = t.stride(0);
            if (S > 1) q_row = t.stride(1);
        }
        const int32_t* lens = a[5] == Py_None ? nullptr : data<int32_t>(want(a[5], "draft_lens", {B}, at::kInt, index));
        const float* temps = nullptr;
        float temperature = 0.f;
        if (THPVariable_Check(a[6])) temps = data<float>(want(a[6], "temperature", {B}, at::kFloat, index));
        else temperature = real(a[6]);
        const at::Tensor tokens = place.make({B, rows}, at::kInt), accepted = place.make({B}, at::kInt),
                         probs = place.make({B, rows}, at::kFloat);
        check(ds_verify_drafts(x.data_ptr(), code, B, static_cast<int32_t>(S), V, x.stride(0), rows > 1 ? x.stride(1) : V,
                               data<int32_t>(drafts), lens, q, q_seq, q_row, data<float>(uniforms), data<float>(noise),
                               B > 1 ? noise.stride(0) : V, temps, temperature, data<int32_t>(tokens),
                               data<int32_t>(accepted), data<float>(probs), place.stream()), "ds_verify_drafts");
        return tuple_of({tokens, accepted, probs});
    });
}

// A 4-bit cache: codes (pages, heads, page, 2, D / 2) and scales (pages, heads, page, 4).
struct Cache {
    const at::Tensor *codes, *scales;
    int64_t pages;
    int32_t heads, page, D;
    c10::DeviceIndex index;
    Cache(PyObject* c, PyObject* s) {
        codes = &leading(c, "cache", 5);
        index = codes->get_device();
        pages = codes->size(0);
        const int64_t h = codes->size(1), p = codes->size(2), half = codes->size(4);
        if (codes->size(3) != 2) refuse("cache must have shape (pages, heads, page, 2, D / 2)");
        if (h > 0x7FFFFFFF || p > 0x7FFFFFFF || half > 0x3FFFFFFF) refuse("cache is too large");
        want(c, "cache", {pages, h, p, 2, half}, at::kByte, index);
        scales = &want(s, "scales", {pages, h, p, 4}, at::kBFloat16, index);
        heads = static_cast<int32_t>(h);
        page = static_cast<int32_t>(p);
        D = static_cast<int32_t>(2 * half);
    }
};

PyObject* cache_store(PyObject*, Args a, Py_ssize_t n) {
    return guarded(n, 6, [&]() -> PyObject* {
        const Cache c(a[2], a[3]);
        const Place place(a[5], c.index);
        const at::Tensor& k = leading(a[0], "k", 3);
        const int32_t code = float_code(k, "k");
        const int64_t T = k.size(0);
        want(a[0], "k", {T, c.heads, c.D}, k.scalar_type(), c.index, true);
        const at::Tensor& v = want(a[1], "v", {T, c.heads, c.D}, k.scalar_type(), c.index, true);
        const at::Tensor& slots = want(a[4], "slots", {T}, at::kInt, c.index);
        // the stride of an extent of 1 is never used, whatever torch calls it
        const auto stride = [](const at::Tensor& t, int d) { return t.size(d) > 1 ? t.stride(d) : 0; };
        check(ds_cache_store(k.data_ptr(), v.data_ptr(), code, T, c.heads, c.D, stride(k, 0), stride(k, 1), stride(v, 0),
                             stride(v, 1), c.codes->data_ptr(), c.scales->data_ptr(), c.pages, c.page,
                             data<int32_t>(slots), place.stream()), "ds_cache_store");
        Py_RETURN_NONE;
    });
}

PyObject* cache_load(PyObject*, Args a, Py_ssize_t n) {
    return guarded(n, 5, [&]() -> PyObject* {
        const Cache c(a[0], a[1]);
        const Place place(a[4], c.index);
        const at::Tensor& s = tensor(a[2], "slots");
        const int64_t T = s.dim() > 0 ? s.size(0) : 0;
        const at::Tensor& slots = want(a[2], "slots", {T}, at::kInt, c.index);
        const bool wide = truth(a[3]);
        const at::ScalarType type = wide ? at::kFloat : at::kBFloat16;
        const at::Tensor k = place.make({T, c.heads, c.D}, type), v = place.make({T, c.heads, c.D}, type);
        check(ds_cache_load(c.codes->data_ptr(), c.scales->data_ptr(), c.pages, c.page, data<int32_t>(slots), T, c.heads,
                            c.D, wide ? DS_FP32 : DS_BF16, k.data_ptr(), v.data_ptr(), place.stream()),
              "ds_cache_load");
        return tuple_of({k, v});
    });
}

PyObject* cache_attention(PyObject*, Args a, Py_ssize_t n) {
    return guarded(n, 8, [&]() -> PyObject* {
        const Cache c(a[1], a[2]);
        const Place place(a[7], c.index);
        const at::Tensor& q = leading(a[0], "q", 4);
        const int32_t code = float_code(q, "q");
        const int64_t B = q.size(0), Q = q.size(1), hq = q.size(2);
        want(a[0], "q", {B, Q, hq, c.D}, q.scalar_type(), c.index, true);
        if (Q > 0x7FFFFFFF || hq > 0x7FFFFFFF) refuse("q has too many tokens or heads");
        const at::Tensor& pages = tensor(a[3], "table");
        if (pages.dim() != 2) refuse("table must have 2 dimensions");
        const int64_t width = pages.size(1);
        const at::Tensor& table = want(a[3], "table", {B, width}, at::kInt, c.index, true);
        const at::Tensor& lens = want(a[4], "lens", {B}, at::kInt, c.index);
        const int32_t* indices = nullptr;
        int64_t K = 0;
        if (a[5] != Py_None) {
            const at::Tensor& t = tensor(a[5], "indices");
            K = t.dim() > 0 ? t.size(-1) : 0;
            indices = data<int32_t>(want(a[5], "indices", {B, Q, K}, at::kInt, c.index));
            if (K > 0x7FFFFFFF) refuse("indices has too many columns");
            if (K == 0) indices = data<int32_t>(lens);  // a list of nothing has no memory; none of it is read
        }
        const float scale = a[6] == Py_None ? static_cast<float>(1.0 / std::sqrt(static_cast<double>(c.D))) : real(a[6]);
        const at::Tensor out = place.make({B, Q, hq, c.D}, q.scalar_type()), lse = place.make({B, Q, hq}, at::kFloat);
        const int32_t tokens = static_cast<int32_t>(Q), heads = static_cast<int32_t>(hq), list = static_cast<int32_t>(K);
        size_t bytes = 0;
        check(ds_cache_attention_workspace_bytes(code, B, tokens, heads, c.D, c.heads, c.page, width, indices != nullptr,
                                                 list, &bytes), "ds_cache_attention");
        const at::Tensor ws = place.scratch(bytes);
        check(ds_cache_attention_ex(q.data_ptr(), code, B, tokens, heads, c.D, q.stride(0), q.stride(1), q.stride(2),
                                    c.codes->data_ptr(), c.scales->data_ptr(), c.pages, c.heads, c.page,
                                    data<int32_t>(table), width, B > 1 ? table.stride(0) : width, data<int32_t>(lens),
                                    indices, list, scale, out.data_ptr(), data<float>(lse),
                                    bytes ? ws.data_ptr() : nullptr, bytes, place.stream()), "ds_cache_attention");
        return tuple_of({out, lse});
    });
}

PyObject* token_logprobs(PyObject*, Args a, Py_ssize_t n) {
    return guarded(n, 4, [&]() -> PyObject* {
        const at::Tensor& x = leading(a[0], "logits", 2);
        const int32_t code = float_code(x, "logits"), top = integer32(a[2], "top");
        const int64_t rows = x.size(0), V = x.size(1);
        const auto index = x.get_device();
        const Place place(a[3], index);
        const at::Tensor& tokens = want(a[1], "tokens", {rows}, at::kInt, index);
        const int64_t width = top > 0 ? top : 0;
        if (width > V) refuse("top is larger than the number of logits");
        const at::Tensor logprobs = place.make({rows}, at::kFloat), lse = place.make({rows}, at::kFloat),
                         entropy = place.make({rows}, at::kFloat), top_logprobs = place.make({rows, width}, at::kFloat),
                         top_tokens = place.make({rows, width}, at::kInt);
        check(ds_token_logprobs(x.data_ptr(), code, rows, V, rows > 1 ? x.stride(0) : V, data<int32_t>(tokens), top,
                                data<float>(logprobs), data<float>(lse), data<float>(entropy), data<float>(top_logprobs),
                                data<int32_t>(top_tokens), place.stream()), "ds_token_logprobs");
        return tuple_of({logprobs, lse, entropy, top_logprobs, top_tokens});
    });
}

PyObject* token_logprobs_backward(PyObject*, Args a, Py_ssize_t n) {
    return guarded(n, 7, [&]() -> PyObject* {
        const at::Tensor& x = leading(a[1], "logits", 2);
        const int32_t code = float_code(x, "logits");
        const int64_t rows = x.size(0), V = x.size(1);
        const auto index = x.get_device();
        const Place place(a[6], index);
        const at::Tensor& grad = want(a[0], "grad_logprobs", {rows}, at::kFloat, index);
        const at::Tensor& tokens = want(a[2], "tokens", {rows}, at::kInt, index);
        const at::Tensor& lse = want(a[3], "lse", {rows}, at::kFloat, index);
        const float *grad_entropy = nullptr, *entropy = nullptr;
        if (a[4] != Py_None) {
            if (a[5] == Py_None) refuse("grad_entropy needs entropy");
            grad_entropy = data<float>(want(a[4], "grad_entropy", {rows}, at::kFloat, index));
        }
        if (a[5] != Py_None) entropy = data<float>(want(a[5], "entropy", {rows}, at::kFloat, index));
        const at::Tensor out = place.make({rows, V}, x.scalar_type());
        check(ds_token_logprobs_backward(data<float>(grad), x.data_ptr(), code, rows, V, rows > 1 ? x.stride(0) : V,
                                         data<int32_t>(tokens), data<float>(lse), grad_entropy, entropy, out.data_ptr(), V,
                                         place.stream()), "ds_token_logprobs_backward");
        return THPVariable_Wrap(out);
    });
}

// A token's choices: (tokens, k) int32.
const at::Tensor& choices(PyObject* o, const char* what) {
    const at::Tensor& t = leading(o, what, 2);
    want(o, what, {t.size(0), t.size(1)}, at::kInt, t.get_device());
    if (t.size(1) > 0x7FFFFFFF) refuse(std::string(what) + " has too many columns");
    return t;
}
// The first row of each expert, and behind the last: (experts + 1,) int32.
int32_t experts_of(PyObject* o, c10::DeviceIndex index) {
    const at::Tensor& t = tensor(o, "offsets");
    const int64_t size = t.dim() > 0 ? t.size(0) : 0;
    if (size < 2 || size > 0x7FFFFFFF) refuse("offsets must have one number more than there are experts");
    want(o, "offsets", {size}, at::kInt, index);
    return static_cast<int32_t>(size - 1);
}
int32_t width_of(const at::Tensor& t, const char* what) {
    if (t.size(-1) > 0x7FFFFFFF) refuse(std::string(what) + " has too many columns");
    return static_cast<int32_t>(t.size(-1));
}

PyObject* expert_sort(PyObject*, Args a, Py_ssize_t n) {
    return guarded(n, 3, [&]() -> PyObject* {
        const at::Tensor& experts = choices(a[0], "experts");
        const int32_t E = integer32(a[1], "E");
        const Place place(a[2], experts.get_device());
        const at::Tensor places = place.make({experts.size(0), experts.size(1)}, at::kInt),
                         offsets = place.make({(E > 0 ? static_cast<int64_t>(E) : 0) + 1}, at::kInt);
        check(ds_expert_sort(data<int32_t>(experts), experts.size(0), static_cast<int32_t>(experts.size(1)), E,
                             data<int32_t>(places), data<int32_t>(offsets), place.stream()), "ds_expert_sort");
        return tuple_of({places, offsets});
    });
}

PyObject* expert_gather(PyObject*, Args a, Py_ssize_t n) {
    return guarded(n, 5, [&]() -> PyObject* {
        const at::Tensor& x = leading(a[0], "x", 2);
        const int32_t code = float_code(x, "x"), D = width_of(x, "x");
        const int64_t T = x.size(0);
        const auto index = x.get_device();
        const Place place(a[4], index);
        const at::Tensor& places = choices(a[1], "places");
        const int64_t k = places.size(1);
        want(a[1], "places", {T, k}, at::kInt, index);
        const int32_t E = experts_of(a[2], index);
        const int32_t* offsets = data<int32_t>(tensor(a[2], "offsets"));
        const int64_t stride = T > 1 ? x.stride(0) : D;
        if (truth(a[3])) {
            const at::Tensor codes = place.make({T * k, D}, at::kFloat8_e4m3fn),
                             scales = place.make({T * k, (static_cast<int64_t>(D) + 127) / 128}, at::kFloat);
            check(ds_expert_gather_quantised(x.data_ptr(), code, T, D, stride, data<int32_t>(places), static_cast<int32_t>(k),
                                             offsets, E, codes.data_ptr(), data<float>(scales), place.stream()),
                  "ds_expert_gather_quantised");
            return tuple_of({codes, scales});
        }
        const at::Tensor out = place.make({T * k, D}, x.scalar_type());
        check(ds_expert_gather(x.data_ptr(), code, T, D, stride, data<int32_t>(places), static_cast<int32_t>(k), offsets, E,
                               out.data_ptr(), place.stream()), "ds_expert_gather");
        return THPVariable_Wrap(out);
    });
}

PyObject* expert_combine(PyObject*, Args a, Py_ssize_t n) {
    return guarded(n, 4, [&]() -> PyObject* {
        const at::Tensor& y = leading(a[0], "y", 2);
        const int32_t code = float_code(y, "y"), D = width_of(y, "y");
        const auto index = y.get_device();
        const Place place(a[3], index);
        const at::Tensor& places = choices(a[1], "places");
        const int64_t T = places.size(0), k = places.size(1);
        want(a[1], "places", {T, k}, at::kInt, index);
        const float* weights = a[2] == Py_None ? nullptr : data<float>(want(a[2], "weights", {T, k}, at::kFloat, index));
        const at::Tensor out = place.make({T, D}, y.scalar_type());
        check(ds_expert_combine(y.data_ptr(), code, y.size(0), D, y.size(0) > 1 ? y.stride(0) : D, data<int32_t>(places), T,
                                static_cast<int32_t>(k), weights, out.data_ptr(), place.stream()), "ds_expert_combine");
        return THPVariable_Wrap(out);
    });
}

PyObject* expert_combine_backward(PyObject*, Args a, Py_ssize_t n) {
    return guarded(n, 6, [&]() -> PyObject* {
        const at::Tensor& grad = leading(a[0], "grad", 2);
        const int32_t code = float_code(grad, "grad"), D = width_of(grad, "grad");
        const int64_t T = grad.size(0);
        const auto index = grad.get_device();
        const Place place(a[5], index);
        const at::Tensor& places = choices(a[2], "places");
        const int64_t k = places.size(1);
        want(a[2], "places", {T, k}, at::kInt, index);
        const at::Tensor& y = want(a[1], "y", {T * k, D}, grad.scalar_type(), index, true);
        const int32_t E = experts_of(a[3], index);
        const at::Tensor& weights = want(a[4], "weights", {T, k}, at::kFloat, index);
        const at::Tensor grad_y = place.make({T * k, D}, grad.scalar_type()), grad_weights = place.make({T, k}, at::kFloat);
        check(ds_expert_combine_backward(grad.data_ptr(), T > 1 ? grad.stride(0) : D, y.data_ptr(), code, D,
                                         T * k > 1 ? y.stride(0) : D, data<int32_t>(places), T, static_cast<int32_t>(k),
                                         data<int32_t>(tensor(a[3], "offsets")), E, data<float>(weights), grad_y.data_ptr(),
                                         data<float>(grad_weights), place.stream()), "ds_expert_combine_backward");
        return tuple_of({grad_y, grad_weights});
    });
}

PyObject* quantise_blocks(PyObject*, Args a, Py_ssize_t n) {
    return guarded(n, 3, [&]() -> PyObject* {
        const at::Tensor& t = tensor(a[0], "x");
        const bool many = t.dim() == 3;
        const at::Tensor& x = leading(a[0], "x", many ? 3 : 2);
        const int32_t code = float_code(x, "x"), K = width_of(x, "x"), block = integer32(a[1], "block_rows");
        if (block != 1 && block != 128) refuse("block_rows must be 1 or 128");
        const Place place(a[2], x.get_device());
        const int64_t E = many ? x.size(0) : 1, N = x.size(-2), n_scales = (N + block - 1) / block,
                      k_scales = (static_cast<int64_t>(K) + 127) / 128;
        const int64_t row_stride = N > 1 ? x.stride(-2) : K, matrix_stride = E > 1 ? x.stride(0) : N * row_stride;
        const at::Tensor codes = many ? place.make({E, N, K}, at::kFloat8_e4m3fn) : place.make({N, K}, at::kFloat8_e4m3fn),
                         scales = many ? place.make({E, n_scales, k_scales}, at::kFloat) : place.make({n_scales, k_scales}, at::kFloat);
        check(ds_quantise_blocks(x.data_ptr(), code, E, N, K, matrix_stride, row_stride, block, codes.data_ptr(),
                                 data<float>(scales), place.stream()), "ds_quantise_blocks");
        return tuple_of({codes, scales});
    });
}

PyObject* expert_product(PyObject*, Args a, Py_ssize_t n) {
    return guarded(n, 7, [&]() -> PyObject* {
        const at::Tensor& x = leading(a[0], "x", 2);
        const int64_t T = x.size(0), blocks = (x.size(1) + 127) / 128;
        const int32_t K = width_of(x, "x");
        const auto index = x.get_device();
        const Place place(a[6], index);
        want(a[0], "x", {T, K}, at::kFloat8_e4m3fn, index, true);
        const at::Tensor& xs = want(a[1], "x_scales", {T, blocks}, at::kFloat, index);
        const bool many = tensor(a[2], "w").dim() == 3;  // one expert's may come as a matrix
        const at::Tensor& w = leading(a[2], "w", many ? 3 : 2);
        const int64_t E = many ? w.size(0) : 1, N = w.size(-2), n_blocks = (N + 127) / 128;
        if (many) want(a[2], "w", {E, N, K}, at::kFloat8_e4m3fn, index, true);
        else want(a[2], "w", {N, K}, at::kFloat8_e4m3fn, index, true);
        const at::Tensor& ws = many ? want(a[3], "w_scales", {E, n_blocks, blocks}, at::kFloat, index)
                                    : want(a[3], "w_scales", {n_blocks, blocks}, at::kFloat, index);
        if (E > 0x7FFFFFFE || N > 0x7FFFFFFF) refuse("w has too many experts or rows");
        const int32_t* offsets = nullptr;
        if (a[4] != Py_None) offsets = data<int32_t>(want(a[4], "offsets", {E + 1}, at::kInt, index));
        else if (E != 1) refuse("w of several experts needs offsets");
        const bool wide = truth(a[5]);
        const at::Tensor out = place.make({T, N}, wide ? at::kFloat : at::kBFloat16);
        const int64_t w_row = N > 1 ? w.stride(-2) : K;
        check(ds_expert_product(x.data_ptr(), data<float>(xs), T, K, T > 1 ? x.stride(0) : K, w.data_ptr(), data<float>(ws),
                                static_cast<int32_t>(E), static_cast<int32_t>(N), w_row, E > 1 ? w.stride(0) : N * w_row,
                                offsets, wide ? DS_FP32 : DS_BF16, out.data_ptr(), place.stream()), "ds_expert_product");
        return THPVariable_Wrap(out);
    });
}

PyObject* set_error(PyObject*, PyObject* type) {
    Py_INCREF(type);
    Py_XDECREF(g_error);
    g_error = type;
    Py_RETURN_NONE;
}

#define FAST(name) {#name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(name)), METH_FASTCALL, nullptr}
PyMethodDef methods[] = {FAST(route), FAST(route_backward), FAST(verify_drafts), FAST(cache_store), FAST(cache_load),
                         FAST(cache_attention), FAST(token_logprobs), FAST(token_logprobs_backward), FAST(expert_sort),
                         FAST(expert_gather), FAST(expert_combine), FAST(expert_combine_backward), FAST(quantise_blocks),
                         FAST(expert_product), {"set_error", set_error, METH_O, nullptr}, {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_ops", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__ops() { return PyModule_Create(&module); }
