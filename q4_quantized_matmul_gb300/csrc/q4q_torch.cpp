// q4q_torch.cpp -- the Python side of the MXFP4, expert and attention calls: torch tensors in, the C ABI
// of include/q4q.h out.
//
// These calls take a few microseconds on the GPU, about as long as ctypes and Python need
// for one call's checks and allocations (measured on the host of a GB300: 14 us for a sort,
// of which the launch is 2.7).  Every function takes its arguments by position, checks what
// the C ABI cannot see (types, contiguity, sizes), allocates what was not given and calls
// the entry point of its name on the tensors' device and the given or current stream.  What
// sizes an allocation is checked before it, so a call that is refused has taken no memory.
#include <Python.h>

#include <ATen/core/Tensor.h>
#include <ATen/cuda/EmptyTensor.h>
#include <c10/cuda/CUDACachingAllocator.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Dtype.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <algorithm>
#include <cmath>
#include <exception>
#include <initializer_list>
#include <optional>
#include <string>

#include "q4q.h"

namespace {

PyObject* g_error = nullptr;       // Q4QError(fn, status)

constexpr int MAX_EXPERTS = 1024;  // q4q_moe_sort's limit

// carries a Python exception that is already set
struct Raised {};

[[noreturn]] void raise(PyObject* type, const std::string& what) {
    PyErr_SetString(type, what.c_str());
    throw Raised{};
}

const char* type_name(at::ScalarType t) {
    switch (t) {
        case at::kFloat: return "float32";
        case at::kInt: return "int32";
        case at::kHalf: return "float16";
        case at::kBFloat16: return "bfloat16";
        default: return "other";
    }
}

const at::Tensor& tensor(PyObject* o, const char* name) {
    if (!THPVariable_Check(o)) raise(PyExc_TypeError, std::string(name) + " must be a CUDA tensor");
    return THPVariable_Unpack(o);
}

int type_of(const at::Tensor& t, const char* name) {
    switch (t.scalar_type()) {
        case at::kFloat: return Q4Q_TYPE_F32;
        case at::kHalf: return Q4Q_TYPE_F16;
        case at::kBFloat16: return Q4Q_TYPE_BF16;
        default: raise(PyExc_TypeError, std::string(name) + " must be a float32, float16 or bfloat16 tensor");
    }
}

// The address of a contiguous CUDA tensor on `device` that holds `count` elements.
void* address(const at::Tensor& t, const char* name, int64_t count, c10::DeviceIndex device) {
    if (!t.is_cuda()) raise(PyExc_TypeError, std::string(name) + " must be a CUDA tensor");
    if (t.get_device() != device) raise(PyExc_ValueError, std::string(name) + " is on another device");
    if (!t.is_contiguous()) raise(PyExc_ValueError, std::string(name) + " must be contiguous");
    if (t.numel() < count)
        raise(PyExc_ValueError, std::string(name) + " holds " + std::to_string(t.numel()) + " elements, the call reads or writes " + std::to_string(count));
    return t.data_ptr();
}

void* typed(const at::Tensor& t, const char* name, at::ScalarType type, int64_t count, c10::DeviceIndex device) {
    if (t.scalar_type() != type) raise(PyExc_TypeError, std::string(name) + " must be a " + type_name(type) + " tensor");
    return address(t, name, count, device);
}

// uint8 buffers may come in any type: their bytes count
void* bytes(const at::Tensor& t, const char* name, int64_t count, c10::DeviceIndex device) {
    void* p = address(t, name, 0, device);
    if (t.numel() * t.element_size() < count)
        raise(PyExc_ValueError, std::string(name) + " holds " + std::to_string(t.numel() * t.element_size()) + " bytes, the call reads or writes " + std::to_string(count));
    return p;
}

int64_t integer(PyObject* o, const char* name) {
    const long long v = PyLong_AsLongLong(o);
    if (v == -1 && PyErr_Occurred()) {
        PyErr_Clear();
        raise(PyExc_TypeError, std::string(name) + " must be an integer");
    }
    return v;
}

int small_integer(PyObject* o, const char* name) {
    const int64_t v = integer(o, name);
    if (v < INT32_MIN || v > INT32_MAX) raise(PyExc_OverflowError, std::string(name) + " is out of range");
    return (int)v;
}

void need(PyObject* const* args, Py_ssize_t n, Py_ssize_t want) {
    (void)args;
    if (n != want) raise(PyExc_TypeError, "wrong number of arguments");
}

// The device and stream of a call: its first tensor's device, made current for the call; a
// torch.cuda.Stream, an integer, or for None the device's current stream.
class Place {
   public:
    Place(const at::Tensor& first, const char* name, PyObject* stream) {
        if (!first.is_cuda()) raise(PyExc_TypeError, std::string(name) + " must be a CUDA tensor");
        device_ = first.get_device();
        guard_.emplace(device_);
        if (stream == Py_None) {
            stream_ = c10::cuda::getCurrentCUDAStream(device_).stream();
            return;
        }
        PyObject* value = PyLong_Check(stream) ? Py_NewRef(stream) : PyObject_GetAttrString(stream, "cuda_stream");
        if (!value) throw Raised{};
        void* p = PyLong_AsVoidPtr(value);
        Py_DECREF(value);
        if (!p && PyErr_Occurred()) throw Raised{};
        stream_ = static_cast<cudaStream_t>(p);
        other_ = stream_ != c10::cuda::getCurrentCUDAStream(device_).stream();
    }
    c10::DeviceIndex device() const { return device_; }
    q4q_stream_t stream() const { return reinterpret_cast<q4q_stream_t>(stream_); }
    // A tensor of the call's own.  Where the call runs on another stream than the current, its
    // memory is that stream's (of the current stream's free memory, work in flight there may still
    // be reading), and is kept from its next user until the current stream, where the tensor may
    // be used next, is past that use.
    at::Tensor make(at::IntArrayRef shape, at::ScalarType type) const {
        if (!other_) return empty(shape, type);
        const c10::cuda::CUDAStream current = c10::cuda::getCurrentCUDAStream(device_);
        const c10::cuda::CUDAStreamGuard its(c10::cuda::getStreamFromExternal(stream_, device_));
        at::Tensor t = empty(shape, type);
        if (t.numel() > 0) t.record_stream(current.unwrap());
        return t;
    }
    // Memory of the call's stream for the length of the call: what is freed is used next by work
    // that is queued behind the call's.
    c10::DataPtr scratch(size_t n) const {
        if (!other_) return c10::cuda::CUDACachingAllocator::get()->allocate(n);
        const c10::cuda::CUDAStreamGuard its(c10::cuda::getStreamFromExternal(stream_, device_));
        return c10::cuda::CUDACachingAllocator::get()->allocate(n);
    }

   private:
    // what at::empty comes to, without its way through the dispatcher (1.2 us on the host of a GB300,
    // about as long as a launch)
    at::Tensor empty(at::IntArrayRef shape, at::ScalarType type) const {
        return at::Tensor(at::detail::empty_cuda(shape, type, at::Device(at::kCUDA, device_), std::nullopt));
    }
    c10::DeviceIndex device_ = 0;
    cudaStream_t stream_ = nullptr;
    bool other_ = false;
    std::optional<c10::cuda::CUDAGuard> guard_;
};

void check(const char* fn, q4q_status status) {
    if (status == Q4Q_OK) return;
    PyObject* e = PyObject_CallFunction(g_error, "si", fn, (int)status);
    if (e) {
        PyErr_SetObject(reinterpret_cast<PyObject*>(Py_TYPE(e)), e);
        Py_DECREF(e);
    }
    throw Raised{};
}

size_t matrix_bytes(int64_t ne00, int64_t ne01) {
    size_t n = 0;
    check("q4q_mxfp4_size", q4q_mxfp4_size(ne00, ne01, &n));
    return n;
}

at::Tensor given(PyObject* o, const char* name, const Place& at, at::IntArrayRef shape, at::ScalarType type) {
    return o == Py_None ? at.make(shape, type) : tensor(o, name);
}

PyObject* wrap(const at::Tensor& t) { return THPVariable_Wrap(t); }

template <typename F>
PyObject* guarded(F f) {
    try {
        return f();
    } catch (const Raised&) {
    } catch (const std::exception&) {
        // as torch raises them, torch.OutOfMemoryError among them
        torch::translate_exception_to_python(std::current_exception());
    }
    return nullptr;
}

// ------------------------------------------------------------------ MXFP4 --

// quantize_mxfp4(src, dst, stream)
PyObject* quantize(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return guarded([&] {
        need(a, n, 3);
        const at::Tensor& src = tensor(a[0], "src");
        const int type = type_of(src, "src");
        if (src.dim() != 2 && src.dim() != 3) raise(PyExc_ValueError, "src must be [rows, K] or [matrices, rows, K]");
        const Place at(src, "src", a[2]);
        const int64_t mats = src.dim() == 3 ? src.size(0) : 1, rows = src.size(-2), cols = src.size(-1);
        const int64_t size = (int64_t)matrix_bytes(cols, rows);
        const at::Tensor dst = src.dim() == 3 ? given(a[1], "dst", at, {mats, size}, at::kByte) : given(a[1], "dst", at, {size}, at::kByte);
        check("q4q_quantize_mxfp4", q4q_quantize_mxfp4(address(src, "src", 0, at.device()), type, bytes(dst, "dst", mats * size, at.device()),
                                                       cols, rows, mats, at.stream()));
        return wrap(dst);
    });
}

// get_rows_mxfp4(src0, ne00, ne01, ids, n_ids, dst, stream)
PyObject* get_rows(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return guarded([&] {
        need(a, n, 7);
        const at::Tensor& src0 = tensor(a[0], "src0");
        const int64_t ne00 = integer(a[1], "ne00"), ne01 = integer(a[2], "ne01");
        const Place at(src0, "src0", a[6]);
        const int32_t* ids = nullptr;
        int64_t n_ids = a[4] == Py_None ? ne01 : integer(a[4], "n_ids");
        if (a[3] != Py_None) {
            const at::Tensor& t = tensor(a[3], "ids");
            n_ids = t.numel();
            ids = static_cast<const int32_t*>(typed(t, "ids", at::kInt, 0, at.device()));
        }
        if (n_ids < 0) raise(PyExc_ValueError, "n_ids is negative");
        const void* w = n_ids > 0 ? bytes(src0, "src0", (int64_t)matrix_bytes(ne00, ne01), at.device()) : nullptr;
        if (!ids && n_ids > ne01) check("q4q_get_rows_mxfp4", Q4Q_ERR_SHAPE);
        const at::Tensor dst = given(a[5], "dst", at, {n_ids, ne00}, at::kFloat);
        if (n_ids > 0)
            check("q4q_get_rows_mxfp4", q4q_get_rows_mxfp4(w, ne00, ne01, ids, n_ids,
                                                           static_cast<float*>(typed(dst, "dst", at::kFloat, n_ids * ne00, at.device())), at.stream()));
        return wrap(dst);
    });
}

// the rows of x, which a view holds: a copy would be made on the current stream, not the call's
at::Tensor rows_2d(const at::Tensor& x) {
    if (!x.is_contiguous()) raise(PyExc_ValueError, "src1 must be contiguous");
    return x.dim() == 2 ? x : x.view({-1, x.size(-1)});
}

at::ScalarType output_type(PyObject* dtype, const at::Tensor& like) {
    if (dtype == Py_None) return like.scalar_type();
    if (!THPDtype_Check(dtype)) raise(PyExc_TypeError, "dst_dtype must be a torch.dtype");
    return reinterpret_cast<THPDtype*>(dtype)->scalar_type;
}

// a workspace of `need` bytes, or the one given: its address and size
void* workspace_of(PyObject* o, size_t need, const Place& at, c10::DataPtr& hold, size_t& size) {
    size = need;
    if (o == Py_None) {
        if (need == 0) return nullptr;
        hold = at.scratch(need);
        return hold.get();
    }
    const at::Tensor& given = tensor(o, "workspace");
    size = (size_t)(given.numel() * given.element_size());
    return bytes(given, "workspace", 0, at.device());
}

// mul_mat_mxfp4(src0, ne00, ne01, src1, acts, dst, dst_dtype, workspace, stream, flags)
PyObject* mul_mat(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return guarded([&] {
        need(a, n, 10);
        const at::Tensor& src0 = tensor(a[0], "src0");
        const int64_t ne00 = integer(a[1], "ne00"), ne01 = integer(a[2], "ne01");
        const at::Tensor& src1 = tensor(a[3], "src1");
        const int type = type_of(src1, "src1"), acts = small_integer(a[4], "acts");
        const Place at(src0, "src0", a[8]);
        const at::Tensor x = rows_2d(src1);
        const int64_t ne11 = x.size(0), ne10 = x.size(1);
        const bool empty = ne01 == 0 || ne11 == 0;
        const void* w = empty ? nullptr : bytes(src0, "src0", (int64_t)matrix_bytes(ne00, ne01), at.device());
        const at::Tensor dst = given(a[5], "dst", at, {ne11, ne01}, output_type(a[6], x));
        if (empty) return wrap(dst);
        size_t need_bytes = 0, size = 0;
        c10::DataPtr hold;
        if (a[7] == Py_None)
            check("q4q_mul_mat_mxfp4_workspace_size", q4q_mul_mat_mxfp4_workspace_size(ne00, ne01, ne11, acts, &need_bytes));
        void* ws = workspace_of(a[7], need_bytes, at, hold, size);
        check("q4q_mul_mat_mxfp4",
              q4q_mul_mat_mxfp4(w, ne00, ne01, address(x, "src1", 0, at.device()), type, ne10, ne11, acts,
                                address(dst, "dst", ne11 * ne01, at.device()), type_of(dst, "dst"), ws, size, (unsigned int)integer(a[9], "flags"), at.stream()));
        return wrap(dst);
    });
}

// ---------------------------------------------------------------- experts --

const int32_t* places(const at::Tensor& t, const char* name, int64_t count, const Place& at) {
    return static_cast<const int32_t*>(typed(t, name, at::kInt, count, at.device()));
}

// n elements of `all` from `at` on, a tensor of their own in its storage
at::Tensor piece(const at::Tensor& all, int64_t at, int64_t n) {
    at::Tensor t = at::detail::make_tensor<c10::TensorImpl>(c10::Storage(all.storage()), all.key_set(), all.dtype());
    t.unsafeGetTensorImpl()->set_storage_offset(at);
    t.unsafeGetTensorImpl()->set_sizes_contiguous({n});
    return t;
}

// moe_sort(ids, n_experts, first, slot, row, stream) -> (first, slot, row)
PyObject* moe_sort(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return guarded([&]() -> PyObject* {
        need(a, n, 6);
        const at::Tensor& ids = tensor(a[0], "ids");
        if (ids.scalar_type() != at::kInt) raise(PyExc_TypeError, "ids must be a int32 tensor");
        if (ids.dim() != 2) raise(PyExc_ValueError, "ids must be [tokens, top_k]");
        const int experts = small_integer(a[1], "n_experts");
        const Place at(ids, "ids", a[5]);
        const int64_t tokens = ids.size(0), top_k = ids.size(1), slots = tokens * top_k;
        // refused here what sizes the results, before they are allocated
        if (experts < 1 || experts > MAX_EXPERTS || top_k < 1) check("q4q_moe_sort", Q4Q_ERR_ARG);
        if (slots >= (1ll << 31)) check("q4q_moe_sort", Q4Q_ERR_SHAPE);
        at::Tensor first, slot, row;
        if (a[2] == Py_None && a[3] == Py_None && a[4] == Py_None) {
            // one allocation instead of three: 1.2 us less
            const int64_t n_first = experts + 1;
            const at::Tensor all = at.make({n_first + 2 * slots}, at::kInt);
            first = piece(all, 0, n_first);
            slot = piece(all, n_first, slots);
            row = piece(all, n_first + slots, slots);
        } else {
            first = given(a[2], "first", at, {experts + 1}, at::kInt);
            slot = given(a[3], "slot", at, {slots}, at::kInt);
            row = given(a[4], "row", at, {slots}, at::kInt);
        }
        check("q4q_moe_sort", q4q_moe_sort(places(ids, "ids", slots, at), tokens, (int)top_k, experts,
                                           const_cast<int32_t*>(places(first, "first", (int64_t)experts + 1, at)),
                                           const_cast<int32_t*>(places(slot, "slot", slots, at)),
                                           const_cast<int32_t*>(places(row, "row", slots, at)), at.stream()));
        PyObject *f = wrap(first), *s = wrap(slot), *r = wrap(row);
        PyObject* all = f && s && r ? PyTuple_Pack(3, f, s, r) : nullptr;
        Py_XDECREF(f);
        Py_XDECREF(s);
        Py_XDECREF(r);
        return all;
    });
}

int64_t columns(const at::Tensor& t, const char* name) {
    if (t.dim() != 2) raise(PyExc_ValueError, std::string(name) + " must have two dimensions");
    return t.size(1);
}

int experts_of(const at::Tensor& first) { return (int)first.numel() - 1; }

// moe_gather(src, first, row, top_k, dst, stream)
PyObject* gather(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return guarded([&] {
        need(a, n, 6);
        const at::Tensor &src = tensor(a[0], "src"), &first = tensor(a[1], "first"), &row = tensor(a[2], "row");
        const int type = type_of(src, "src"), top_k = small_integer(a[3], "top_k");
        const Place at(src, "src", a[5]);
        const int64_t ne0 = columns(src, "src"), tokens = src.size(0), slots = tokens * top_k;
        const int32_t* places_of_slots = places(row, "row", slots, at);
        const at::Tensor dst = given(a[4], "dst", at, {std::max<int64_t>(slots, 0), ne0}, src.scalar_type());
        check("q4q_moe_gather", q4q_moe_gather(address(src, "src", 0, at.device()), type, ne0, tokens, top_k, places(first, "first", 1, at),
                                               experts_of(first), places_of_slots,
                                               typed(dst, "dst", src.scalar_type(), slots * ne0, at.device()), at.stream()));
        return wrap(dst);
    });
}

// moe_gather_back(d_dst, first, row, top_k, d_src, stream)
PyObject* gather_back(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return guarded([&] {
        need(a, n, 6);
        const at::Tensor &d_dst = tensor(a[0], "d_dst"), &first = tensor(a[1], "first"), &row = tensor(a[2], "row");
        const int type = type_of(d_dst, "d_dst"), top_k = small_integer(a[3], "top_k");
        const Place at(d_dst, "d_dst", a[5]);
        const int64_t ne0 = columns(d_dst, "d_dst"), slots = d_dst.size(0);
        if (top_k < 1 || slots % top_k) raise(PyExc_ValueError, "d_dst must hold top_k rows for each token");
        const int64_t tokens = slots / top_k;
        const at::Tensor d_src = given(a[4], "d_src", at, {tokens, ne0}, d_dst.scalar_type());
        check("q4q_moe_gather_back", q4q_moe_gather_back(address(d_dst, "d_dst", 0, at.device()), type, ne0, tokens, top_k, places(first, "first", 1, at),
                                                         experts_of(first), places(row, "row", slots, at),
                                                         typed(d_src, "d_src", d_dst.scalar_type(), tokens * ne0, at.device()), at.stream()));
        return wrap(d_src);
    });
}

// the weights' [tokens, top_k]
std::pair<int64_t, int64_t> choices(const at::Tensor& weights) {
    if (weights.dim() != 2) raise(PyExc_ValueError, "weights must be [tokens, top_k]");
    return {weights.size(0), weights.size(1)};
}

// moe_combine(rows, first, row, weights, dst, stream)
PyObject* combine(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return guarded([&] {
        need(a, n, 6);
        const at::Tensor &rows = tensor(a[0], "rows"), &first = tensor(a[1], "first"), &row = tensor(a[2], "row"), &weights = tensor(a[3], "weights");
        const int type = type_of(rows, "rows");
        const Place at(rows, "rows", a[5]);
        const auto [tokens, top_k] = choices(weights);
        const int64_t ne0 = columns(rows, "rows"), slots = tokens * top_k;
        const at::Tensor dst = given(a[4], "dst", at, {tokens, ne0}, rows.scalar_type());
        check("q4q_moe_combine", q4q_moe_combine(address(rows, "rows", slots * ne0, at.device()), type, ne0, tokens, (int)top_k, places(first, "first", 1, at),
                                                 experts_of(first), places(row, "row", slots, at),
                                                 static_cast<const float*>(typed(weights, "weights", at::kFloat, slots, at.device())),
                                                 typed(dst, "dst", rows.scalar_type(), tokens * ne0, at.device()), at.stream()));
        return wrap(dst);
    });
}

// moe_combine_back(d_dst, rows, first, row, weights, d_rows, d_weights, stream) -> (d_rows, d_weights)
PyObject* combine_back(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return guarded([&]() -> PyObject* {
        need(a, n, 8);
        const at::Tensor &d_dst = tensor(a[0], "d_dst"), &rows = tensor(a[1], "rows"), &first = tensor(a[2], "first"), &row = tensor(a[3], "row"),
                         &weights = tensor(a[4], "weights");
        const int type = type_of(rows, "rows");
        const Place at(d_dst, "d_dst", a[7]);
        const auto [tokens, top_k] = choices(weights);
        const int64_t ne0 = columns(rows, "rows"), slots = tokens * top_k;
        const at::Tensor d_rows = given(a[5], "d_rows", at, {slots, ne0}, rows.scalar_type());
        const at::Tensor d_weights = given(a[6], "d_weights", at, {tokens, top_k}, at::kFloat);
        check("q4q_moe_combine_back",
              q4q_moe_combine_back(typed(d_dst, "d_dst", rows.scalar_type(), tokens * ne0, at.device()), address(rows, "rows", slots * ne0, at.device()), type,
                                   ne0, tokens, (int)top_k, places(first, "first", 1, at), experts_of(first), places(row, "row", slots, at),
                                   static_cast<const float*>(typed(weights, "weights", at::kFloat, slots, at.device())),
                                   typed(d_rows, "d_rows", rows.scalar_type(), slots * ne0, at.device()),
                                   static_cast<float*>(typed(d_weights, "d_weights", at::kFloat, slots, at.device())), at.stream()));
        PyObject *r = wrap(d_rows), *w = wrap(d_weights);
        PyObject* both = r && w ? PyTuple_Pack(2, r, w) : nullptr;
        Py_XDECREF(r);
        Py_XDECREF(w);
        return both;
    });
}

// mul_mat_id_mxfp4(src0, ne00, ne01, src1, first, slot, top_k, acts, dst, dst_dtype, workspace, stream, flags)
PyObject* mul_mat_id(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return guarded([&] {
        need(a, n, 13);
        const at::Tensor& src0 = tensor(a[0], "src0");
        const int64_t ne00 = integer(a[1], "ne00"), ne01 = integer(a[2], "ne01");
        const at::Tensor &src1 = tensor(a[3], "src1"), &first = tensor(a[4], "first");
        const int type = type_of(src1, "src1"), top_k = small_integer(a[6], "top_k"), acts = small_integer(a[7], "acts");
        const Place at(src0, "src0", a[11]);
        const at::Tensor x = rows_2d(src1);
        const int64_t n_src1 = x.size(0), ne10 = x.size(1);
        const int experts = experts_of(first);
        const int32_t* slot = nullptr;
        int64_t n_rows = n_src1;
        if (a[5] != Py_None) {
            const at::Tensor& t = tensor(a[5], "slot");
            n_rows = t.numel();
            slot = places(t, "slot", 0, at);
        }
        const bool empty = ne01 == 0 || n_rows == 0;
        if (!empty && (experts < 1 || experts > MAX_EXPERTS)) check("q4q_mul_mat_id_mxfp4", Q4Q_ERR_ARG);
        const void* w = empty ? nullptr : bytes(src0, "src0", (int64_t)matrix_bytes(ne00, ne01) * experts, at.device());
        const at::Tensor dst = given(a[8], "dst", at, {n_rows, ne01}, output_type(a[9], x));
        if (empty) return wrap(dst);
        size_t need_bytes = 0, size = 0;
        c10::DataPtr hold;
        if (a[10] == Py_None)
            check("q4q_mul_mat_id_mxfp4_workspace_size", q4q_mul_mat_id_mxfp4_workspace_size(ne00, ne01, n_src1, n_rows, experts, acts, &need_bytes));
        void* ws = workspace_of(a[10], need_bytes, at, hold, size);
        check("q4q_mul_mat_id_mxfp4",
              q4q_mul_mat_id_mxfp4(w, ne00, ne01, experts, address(x, "src1", 0, at.device()), type, ne10, n_src1,
                                   places(first, "first", (int64_t)experts + 1, at), slot, n_rows, top_k, acts, address(dst, "dst", n_rows * ne01, at.device()), type_of(dst, "dst"), ws, size,
                                   (unsigned int)integer(a[12], "flags"), at.stream()));
        return wrap(dst);
    });
}

// -------------------------------------------------------------- attention --

// [tokens, heads, dim] whose heads lie one after another: a view of a projection's rows
struct Heads {
    void* at = nullptr;
    int64_t tokens = 0, heads = 0, dim = 0, stride = 0;
};

Heads heads_of(const at::Tensor& t, const char* name, c10::DeviceIndex device) {
    if (!t.is_cuda()) raise(PyExc_TypeError, std::string(name) + " must be a CUDA tensor");
    if (t.get_device() != device) raise(PyExc_ValueError, std::string(name) + " is on another device");
    if (t.dim() != 3) raise(PyExc_ValueError, std::string(name) + " must be [tokens, heads, head_dim]");
    Heads h;
    h.tokens = t.size(0);
    h.heads = t.size(1);
    h.dim = t.size(2);
    const int64_t row = h.heads * h.dim;
    h.stride = h.tokens > 1 ? t.stride(0) : row;
    if (t.numel() == 0) h.stride = row;          // strides of an empty tensor say nothing
    else if ((h.dim > 1 && t.stride(2) != 1) || (h.heads > 1 && t.stride(1) != h.dim) || h.stride < row)
        raise(PyExc_ValueError, std::string(name) + " must have its heads' values one after another, and its tokens apart");
    h.at = t.data_ptr();
    return h;
}

bool none(PyObject* o) { return o == Py_None; }

void same_type(const at::Tensor& t, const at::Tensor& like, const char* name) {
    if (t.scalar_type() != like.scalar_type()) raise(PyExc_TypeError, std::string(name) + " must be a " + type_name(like.scalar_type()) + " tensor");
}

void* ints(PyObject* o, const char* name, int64_t count, const Place& at) { return typed(tensor(o, name), name, at::kInt, count, at.device()); }

// a head's weight, or nothing
const float* weight_of(PyObject* o, const char* name, int64_t dim, const Place& at) {
    return none(o) ? nullptr : static_cast<const float*>(typed(tensor(o, name), name, at::kFloat, dim, at.device()));
}

// the table of cosines and sines [n_pos, rot] and the tokens' positions, or nothing
struct Angles {
    const float* table = nullptr;
    const int32_t* pos = nullptr;
    int64_t n_pos = 0;
    int rot = 0;
};

Angles angles_of(PyObject* table, PyObject* pos, int64_t tokens, const Place& at) {
    Angles r;
    if (none(table)) return r;
    const at::Tensor& t = tensor(table, "table");
    if (t.dim() != 2) raise(PyExc_ValueError, "table must be [positions, rot]");
    r.table = static_cast<const float*>(typed(t, "table", at::kFloat, 0, at.device()));
    // its address is null, which would say that there is no table
    if (t.numel() == 0 && tokens > 0) raise(PyExc_ValueError, "table must hold positions");
    r.n_pos = t.size(0);
    r.rot = (int)std::min<int64_t>(t.size(1), 1 << 20);
    if (none(pos)) raise(PyExc_ValueError, "a table needs pos");
    r.pos = static_cast<const int32_t*>(ints(pos, "pos", tokens, at));
    return r;
}

float real(PyObject* o, const char* name) {
    const double v = PyFloat_AsDouble(o);
    if (v == -1.0 && PyErr_Occurred()) {
        PyErr_Clear();
        raise(PyExc_TypeError, std::string(name) + " must be a number");
    }
    return (float)v;
}

void head_dim_ok(const char* fn, int64_t dim) {
    if (dim != 64 && dim != 96 && dim != 128 && dim != 256) check(fn, Q4Q_ERR_SHAPE);
}

PyObject* pack(std::initializer_list<PyObject*> items) {
    PyObject* all = PyTuple_New((Py_ssize_t)items.size());
    Py_ssize_t i = 0;
    bool ok = all != nullptr;
    for (PyObject* o : items) {
        ok = ok && o;
        if (all) PyTuple_SET_ITEM(all, i++, o);
        else Py_XDECREF(o);
    }
    if (!ok) Py_CLEAR(all);
    return all;
}

PyObject* wrap_or_none(const at::Tensor& t) { return t.defined() ? wrap(t) : Py_NewRef(Py_None); }

// rope_table(n_pos, rot, base, dst, stream)
PyObject* rope_table(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return guarded([&] {
        need(a, n, 5);
        const int64_t n_pos = integer(a[0], "n_pos");
        const int rot = small_integer(a[1], "rot");
        const double base = PyFloat_AsDouble(a[2]);
        if (base == -1.0 && PyErr_Occurred()) throw Raised{};
        const at::Tensor& dst = tensor(a[3], "dst");
        const Place at(dst, "dst", a[4]);
        if (n_pos < 0 || rot < 0) check("q4q_rope_table", Q4Q_ERR_SHAPE);
        check("q4q_rope_table", q4q_rope_table(static_cast<float*>(typed(dst, "dst", at::kFloat, n_pos * rot, at.device())), n_pos, rot, base, at.stream()));
        return wrap(dst);
    });
}

// qk_norm_rope(q, k, q_weight, k_weight, eps, table, pos, mode, q_dst, k_dst, stream) -> (q, k)
PyObject* qk_norm_rope(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return guarded([&] {
        need(a, n, 11);
        const at::Tensor& q = tensor(a[0], "q");
        const int type = type_of(q, "q");
        const Place at(q, "q", a[10]);
        const Heads hq = heads_of(q, "q", at.device());
        Heads hk;
        if (!none(a[1])) {
            const at::Tensor& k = tensor(a[1], "k");
            same_type(k, q, "k");
            hk = heads_of(k, "k", at.device());
            if (hk.tokens != hq.tokens || hk.dim != hq.dim) raise(PyExc_ValueError, "k must have the tokens and head_dim of q");
        }
        head_dim_ok("q4q_qk_norm_rope", hq.dim);
        const float* qw = weight_of(a[2], "q_weight", hq.dim, at);
        const float* kw = weight_of(a[3], "k_weight", hq.dim, at);
        const Angles w = angles_of(a[5], a[6], hq.tokens, at);
        const int mode = small_integer(a[7], "mode");
        const at::Tensor dq = given(a[8], "q_dst", at, {hq.tokens, hq.heads, hq.dim}, q.scalar_type());
        at::Tensor dk;
        if (!none(a[1])) dk = given(a[9], "k_dst", at, {hk.tokens, hk.heads, hk.dim}, q.scalar_type());
        check("q4q_qk_norm_rope",
              q4q_qk_norm_rope(hq.at, hq.stride, (int)hq.heads, hk.at, hk.stride, (int)hk.heads, type, hq.dim, hq.tokens, qw, kw, real(a[4], "eps"), w.table,
                               w.n_pos, w.rot, mode, w.pos, typed(dq, "q_dst", q.scalar_type(), hq.tokens * hq.heads * hq.dim, at.device()),
                               dk.defined() ? typed(dk, "k_dst", q.scalar_type(), hk.tokens * hk.heads * hk.dim, at.device()) : nullptr, at.stream()));
        return pack({wrap(dq), wrap_or_none(dk)});
    });
}

// qk_norm_rope_back(d_q_dst, d_k_dst, q, k, q_weight, k_weight, eps, table, pos, mode, d_q, d_k, d_q_weight, d_k_weight, workspace, stream)
//   -> (d_q, d_k, d_q_weight, d_k_weight)
PyObject* qk_norm_rope_back(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return guarded([&] {
        need(a, n, 16);
        const at::Tensor& q = tensor(a[2], "q");
        const int type = type_of(q, "q");
        const Place at(q, "q", a[15]);
        const Heads hq = heads_of(q, "q", at.device());
        Heads hk;
        if (!none(a[3])) {
            const at::Tensor& k = tensor(a[3], "k");
            same_type(k, q, "k");
            hk = heads_of(k, "k", at.device());
            if (hk.tokens != hq.tokens || hk.dim != hq.dim) raise(PyExc_ValueError, "k must have the tokens and head_dim of q");
        }
        head_dim_ok("q4q_qk_norm_rope_back", hq.dim);
        const int64_t nq = hq.tokens * hq.heads * hq.dim, nk = hk.tokens * hk.heads * hk.dim;
        const void* gq = typed(tensor(a[0], "d_q_dst"), "d_q_dst", q.scalar_type(), nq, at.device());
        const void* gk = none(a[3]) ? nullptr : typed(tensor(a[1], "d_k_dst"), "d_k_dst", q.scalar_type(), nk, at.device());
        const float* qw = weight_of(a[4], "q_weight", hq.dim, at);
        const float* kw = none(a[3]) ? nullptr : weight_of(a[5], "k_weight", hq.dim, at);
        const Angles w = angles_of(a[7], a[8], hq.tokens, at);
        const int mode = small_integer(a[9], "mode");
        const at::Tensor dq = given(a[10], "d_q", at, {hq.tokens, hq.heads, hq.dim}, q.scalar_type());
        at::Tensor dk, dqw, dkw;
        if (!none(a[3])) dk = given(a[11], "d_k", at, {hk.tokens, hk.heads, hk.dim}, q.scalar_type());
        if (qw) dqw = given(a[12], "d_q_weight", at, {hq.dim}, at::kFloat);
        if (kw) dkw = given(a[13], "d_k_weight", at, {hq.dim}, at::kFloat);
        size_t need_bytes = 0, size = 0;
        c10::DataPtr hold;
        if (none(a[14]) && (qw || kw)) check("q4q_qk_norm_rope_back_workspace_size", q4q_qk_norm_rope_back_workspace_size(hq.dim, &need_bytes));
        void* ws = workspace_of(a[14], need_bytes, at, hold, size);
        check("q4q_qk_norm_rope_back",
              q4q_qk_norm_rope_back(gq, gk, hq.at, hq.stride, (int)hq.heads, hk.at, hk.stride, (int)hk.heads, type, hq.dim, hq.tokens, qw, kw,
                                    real(a[6], "eps"), w.table, w.n_pos, w.rot, mode, w.pos, typed(dq, "d_q", q.scalar_type(), nq, at.device()),
                                    dk.defined() ? typed(dk, "d_k", q.scalar_type(), nk, at.device()) : nullptr,
                                    qw ? static_cast<float*>(typed(dqw, "d_q_weight", at::kFloat, hq.dim, at.device())) : nullptr,
                                    kw ? static_cast<float*>(typed(dkw, "d_k_weight", at::kFloat, hq.dim, at.device())) : nullptr, ws, size, at.stream()));
        return pack({wrap(dq), wrap_or_none(dk), wrap_or_none(dqw), wrap_or_none(dkw)});
    });
}

// the whole pages that a buffer holds
int64_t pages_in(const char* fn, const at::Tensor& cache, int heads, int64_t dim, int page_tokens, const Place& at, void** address_of) {
    size_t page = 0;
    check(fn, q4q_kv_page_size(heads, dim, page_tokens, &page));
    *address_of = bytes(cache, "cache", 0, at.device());
    const int64_t size = cache.numel() * cache.element_size();
    if (size % (int64_t)page) raise(PyExc_ValueError, "cache must hold whole pages of " + std::to_string(page) + " bytes");
    return size / (int64_t)page;
}

// kv_append(cache, page_tokens, k, v, slots, k_weight, eps, table, pos, mode, stream) -> cache
PyObject* kv_append(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return guarded([&] {
        need(a, n, 11);
        const at::Tensor &cache = tensor(a[0], "cache"), &k = tensor(a[2], "k"), &v = tensor(a[3], "v");
        const int page_tokens = small_integer(a[1], "page_tokens"), type = type_of(k, "k");
        const Place at(cache, "cache", a[10]);
        same_type(v, k, "v");
        const Heads hk = heads_of(k, "k", at.device()), hv = heads_of(v, "v", at.device());
        if (hk.tokens != hv.tokens || hk.heads != hv.heads || hk.dim != hv.dim) raise(PyExc_ValueError, "k and v must have the same shape");
        if (hk.heads > 1024) check("q4q_kv_append", Q4Q_ERR_SHAPE);
        void* buffer = nullptr;
        const int64_t n_pages = pages_in("q4q_kv_append", cache, (int)hk.heads, hk.dim, page_tokens, at, &buffer);
        const Angles w = angles_of(a[7], a[8], hk.tokens, at);
        check("q4q_kv_append", q4q_kv_append(buffer, n_pages, page_tokens, hk.at, hk.stride, hv.at, hv.stride, type, (int)hk.heads, hk.dim, hk.tokens,
                                             static_cast<const int32_t*>(ints(a[4], "slots", hk.tokens, at)), weight_of(a[5], "k_weight", hk.dim, at),
                                             real(a[6], "eps"), w.table, w.n_pos, w.rot, small_integer(a[9], "mode"), w.pos, at.stream()));
        return wrap(cache);
    });
}

// kv_get_rows(cache, page_tokens, n_kv_heads, head_dim, slots, dst_dtype, k_dst, v_dst, stream) -> (k, v)
PyObject* kv_get_rows(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return guarded([&] {
        need(a, n, 9);
        const at::Tensor &cache = tensor(a[0], "cache"), &slots = tensor(a[4], "slots");
        const int page_tokens = small_integer(a[1], "page_tokens"), heads = small_integer(a[2], "n_kv_heads");
        const int64_t dim = integer(a[3], "head_dim"), count = slots.numel();
        const Place at(cache, "cache", a[8]);
        void* buffer = nullptr;
        const int64_t n_pages = pages_in("q4q_kv_get_rows", cache, heads, dim, page_tokens, at, &buffer);
        const void* ids = ints(a[4], "slots", 0, at);
        if (!THPDtype_Check(a[5])) raise(PyExc_TypeError, "dst_dtype must be a torch.dtype");
        at::ScalarType type = reinterpret_cast<THPDtype*>(a[5])->scalar_type;
        if (type != at::kFloat && type != at::kHalf && type != at::kBFloat16) raise(PyExc_TypeError, "dst_dtype must be float32, float16 or bfloat16");
        const at::Tensor k = given(a[6], "k_dst", at, {count, heads, dim}, type), v = given(a[7], "v_dst", at, {count, heads, dim}, type);
        check("q4q_kv_get_rows", q4q_kv_get_rows(buffer, n_pages, page_tokens, heads, dim, static_cast<const int32_t*>(ids), count,
                                                 typed(k, "k_dst", type, count * heads * dim, at.device()),
                                                 typed(v, "v_dst", type, count * heads * dim, at.device()), type_of(k, "k_dst"), at.stream()));
        return pack({wrap(k), wrap(v)});
    });
}

// kv_attn(q, cache, page_tokens, n_kv_heads, pages, kv_len, first, scale, causal, window, dst, lse, workspace, stream, path, limit_ns) -> dst;
// with a path the debug call
PyObject* kv_attn(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return guarded([&] {
        need(a, n, 16);
        const at::Tensor &q = tensor(a[0], "q"), &cache = tensor(a[1], "cache"), &pages = tensor(a[4], "pages"), &len = tensor(a[5], "kv_len");
        const int type = type_of(q, "q"), page_tokens = small_integer(a[2], "page_tokens"), kv_heads = small_integer(a[3], "n_kv_heads");
        const Place at(q, "q", a[13]);
        const Heads h = heads_of(q, "q", at.device());
        if (h.heads > 1024) check("q4q_kv_attn", Q4Q_ERR_SHAPE);
        head_dim_ok("q4q_kv_attn", h.dim);
        void* buffer = nullptr;
        const int64_t n_pages = pages_in("q4q_kv_attn", cache, kv_heads, h.dim, page_tokens, at, &buffer);
        if (pages.dim() != 2) raise(PyExc_ValueError, "pages must be [sequences, pages]");
        const int64_t seqs = pages.size(0), max_pages = pages.size(1);
        const void* table = ints(a[4], "pages", seqs * max_pages, at);
        const void* lengths = typed(len, "kv_len", at::kInt, seqs, at.device());
        const void* first = none(a[6]) ? nullptr : ints(a[6], "first", seqs + 1, at);
        const float scale = none(a[7]) ? (float)(1.0 / std::sqrt((double)h.dim)) : real(a[7], "scale");
        const int64_t causal = PyObject_IsTrue(a[8]), window = integer(a[9], "window");
        if (causal < 0) throw Raised{};
        const at::Tensor dst = given(a[10], "dst", at, {h.tokens, h.heads, h.dim}, q.scalar_type());
        void* out = typed(dst, "dst", q.scalar_type(), h.tokens * h.heads * h.dim, at.device());
        float* lse = none(a[11]) ? nullptr : static_cast<float*>(typed(tensor(a[11], "lse"), "lse", at::kFloat, h.tokens * h.heads, at.device()));
        if (h.tokens == 0 || seqs == 0) return wrap(dst);
        size_t need_bytes = 0, size = 0;
        c10::DataPtr hold;
        if (none(a[12])) check("q4q_kv_attn_workspace_size", q4q_kv_attn_workspace_size(h.tokens, (int)h.heads, kv_heads, h.dim, seqs, type, &need_bytes));
        void* ws = workspace_of(a[12], need_bytes, at, hold, size);
        if (none(a[14]))
            check("q4q_kv_attn", q4q_kv_attn(h.at, h.stride, type, h.tokens, (int)h.heads, kv_heads, h.dim, buffer, n_pages, page_tokens,
                                             static_cast<const int32_t*>(table), max_pages, static_cast<const int32_t*>(lengths),
                                             static_cast<const int32_t*>(first), seqs, scale, (int)causal, window, out, lse, ws, size, at.stream()));
        else
            check("q4q_debug_kv_attn_timeout",
                  q4q_debug_kv_attn_timeout(h.at, h.stride, type, h.tokens, (int)h.heads, kv_heads, h.dim, buffer, n_pages, page_tokens,
                                            static_cast<const int32_t*>(table), max_pages, static_cast<const int32_t*>(lengths),
                                            static_cast<const int32_t*>(first), seqs, scale, out, ws, size, small_integer(a[14], "path"),
                                            (uint64_t)integer(a[15], "limit_ns"), at.stream()));
        return wrap(dst);
    });
}

// set_error(Q4QError): the class of the exceptions for statuses other than Q4Q_OK
PyObject* set_error(PyObject*, PyObject* cls) {
    Py_XDECREF(g_error);
    g_error = Py_NewRef(cls);
    Py_RETURN_NONE;
}

#define Q4Q_FAST(name, fn) {name, reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(fn)), METH_FASTCALL, nullptr}
PyMethodDef methods[] = {
    Q4Q_FAST("quantize_mxfp4", quantize),
    Q4Q_FAST("get_rows_mxfp4", get_rows),
    Q4Q_FAST("mul_mat_mxfp4", mul_mat),
    Q4Q_FAST("moe_sort", moe_sort),
    Q4Q_FAST("moe_gather", gather),
    Q4Q_FAST("moe_gather_back", gather_back),
    Q4Q_FAST("moe_combine", combine),
    Q4Q_FAST("moe_combine_back", combine_back),
    Q4Q_FAST("mul_mat_id_mxfp4", mul_mat_id),
    Q4Q_FAST("rope_table", rope_table),
    Q4Q_FAST("qk_norm_rope", qk_norm_rope),
    Q4Q_FAST("qk_norm_rope_back", qk_norm_rope_back),
    Q4Q_FAST("kv_append", kv_append),
    Q4Q_FAST("kv_get_rows", kv_get_rows),
    Q4Q_FAST("kv_attn", kv_attn),
    {"set_error", set_error, METH_O, nullptr},
    {nullptr, nullptr, 0, nullptr},
};

PyModuleDef module = {PyModuleDef_HEAD_INIT, "_q4q_torch", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__q4q_torch(void) { return PyModule_Create(&module); }
