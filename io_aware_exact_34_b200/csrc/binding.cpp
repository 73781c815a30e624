// binding.cpp -- the ordinary case of the paged-cache calls of fattn.py in
// native code: check the tensors, allocate the outputs, call the C ABI.
//
// A serving step makes these calls back to back and the GPU needs a few us for
// each, which the checks and allocations of an interpreted binding exceed.  A
// function here returns None whenever anything is not as the ordinary call has
// it (a wrong type or shape, a tensor elsewhere, an optional buffer given, an
// error status): the caller then takes the Python path, which makes every
// check again and raises with a message.  A call that the library refuses has
// enqueued nothing by then; one whose launch fails is made again, over the
// same outputs, and its second failure is the one that is raised.
//
// The library's functions are handed over as addresses, so this module links
// against nothing but torch.
#include <torch/csrc/autograd/python_variable.h>

#include <ATen/ATen.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>

#include <cmath>
#include <cstdint>
#include <string>

namespace {

using PlanFn = int (*)(const int*, const int*, int, const int*, int, int*, int, int, long long*, int, int*, int*, int*, void*);
using AppendFn = int (*)(const void*, const void*, long long, long long, const long long*, int, void*, void*, float*, float*,
                         int, int, int, int, void*);
using DecodeFn = int (*)(const void*, const void*, const void*, const float*, const float*, const int*, int, int, int, void*,
                         float*, const int*, int, int, int, int, float, int, int, void*, size_t, void*);
using SplitsFn = int (*)(int, int, int, int, int);
using FwdFn = int (*)(const void*, const void*, const void*, const float*, const float*, const int*, int, int, int, void*,
                      float*, const int*, const int*, int, int, int, int, int, int, float, int, int, int, void*, size_t, void*);
using FwdBytesFn = size_t (*)(int, int, int, int, int, int, int);

PlanFn g_plan = nullptr;
AppendFn g_append = nullptr;
DecodeFn g_decode = nullptr;
SplitsFn g_splits = nullptr;
FwdFn g_fwd = nullptr;
FwdBytesFn g_fwd_bytes = nullptr;

constexpr int64_t kIntMax = 0x7fffffff;

// Thrown and caught here: the call is not the ordinary one.
struct NotOrdinary {};

void need(bool ok) {
    if (!ok) throw NotOrdinary{};
}

const at::Tensor& tensor(PyObject* o) {
    need(THPVariable_Check(o));
    const at::Tensor& t = THPVariable_Unpack(o);
    need(t.is_cuda() && t.layout() == at::kStrided);
    return t;
}

const at::Tensor& dense(PyObject* o, at::ScalarType type, int64_t dims) {
    const at::Tensor& t = tensor(o);
    need(t.scalar_type() == type && t.dim() == dims && t.is_contiguous());
    for (int64_t s : t.sizes()) need(s <= kIntMax);
    return t;
}

const at::Tensor& dense(PyObject* o, at::ScalarType type, at::IntArrayRef shape, int dev) {
    const at::Tensor& t = tensor(o);
    need(t.scalar_type() == type && t.sizes() == shape && t.get_device() == dev && t.is_contiguous());
    return t;
}

int64_t integer(PyObject* o) {
    need(PyLong_Check(o));
    const long long v = PyLong_AsLongLong(o);
    if (v == -1 && PyErr_Occurred()) {
        PyErr_Clear();
        throw NotOrdinary{};
    }
    return v;
}

int small(PyObject* o) {
    const int64_t v = integer(o);
    need(v >= -kIntMax && v <= kIntMax);
    return static_cast<int>(v);
}

float scale_of(PyObject* o, int64_t d) {
    if (o == Py_None) return static_cast<float>(std::pow(static_cast<double>(d), -0.5));
    need(PyFloat_Check(o));
    return static_cast<float>(PyFloat_AS_DOUBLE(o));
}

// The device of a call's first tensor, which has to be the current one, and its stream.
struct Place {
    int dev;
    void* stream;
    explicit Place(const at::Tensor& t) : dev(t.get_device()) {
        need(dev == c10::cuda::current_device());
        stream = c10::cuda::getCurrentCUDAStream(static_cast<c10::DeviceIndex>(dev)).stream();
    }
};

struct Cache {
    const at::Tensor &k, &v, &ks, &vs;
    int pages, page_size, heads, d;
    Cache(PyObject* const* a, int dev)
        : k(dense(a[0], at::kByte, 4)),
          v(dense(a[1], at::kByte, k.sizes(), dev)),
          ks(dense(a[2], at::kFloat, {k.size(0), k.size(2)}, dev)),
          vs(dense(a[3], at::kFloat, {k.size(0), k.size(2)}, dev)) {
        need(k.get_device() == dev);
        pages = static_cast<int>(k.size(0));
        page_size = static_cast<int>(k.size(1));
        heads = static_cast<int>(k.size(2));
        d = static_cast<int>(k.size(3));
    }
};

// Runs f, whose answer is a new reference, or None where the call is not the
// ordinary one (torch's own exceptions included: the Python path meets them too).
template <typename F>
PyObject* ordinary(F&& f) {
    try {
        return f();
    } catch (const NotOrdinary&) {
    } catch (const std::exception&) {
    }
    PyErr_Clear();
    Py_RETURN_NONE;
}

// A tuple of tensors.
template <typename... T>
PyObject* tuple(const T&... t) {
    PyObject* items[] = {THPVariable_Wrap(t)...};
    constexpr Py_ssize_t n = sizeof...(T);
    PyObject* r = PyTuple_New(n);
    for (Py_ssize_t i = 0; i < n; ++i) {
        if (r != nullptr && items[i] != nullptr) PyTuple_SET_ITEM(r, i, items[i]);
        else Py_XDECREF(items[i]);
    }
    for (PyObject* item : items) need(r != nullptr && item != nullptr);
    return r;
}

// n elements of a tensor's memory from `first` on as a tensor of their own: what
// an allocation and its way through the dispatcher would cost more is most of a
// small call's time (plan of 64 sequences, its four results in two allocations: 7.2 -> 5.7 us a call).
at::Tensor piece(const at::Tensor& base, int64_t first, int64_t n) {
    at::Tensor t = at::detail::make_tensor<c10::TensorImpl>(c10::TensorImpl::VIEW, c10::Storage(base.storage()), base.key_set(),
                                                            base.dtype());
    t.unsafeGetTensorImpl()->set_storage_offset(first);
    t.unsafeGetTensorImpl()->set_sizes_contiguous(n);
    return t;
}

// plan(seqlens_k, seqlens_new, free_pages, block_table, page_size, max_tokens)
PyObject* plan(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return ordinary([&]() -> PyObject* {
        need(n == 6 && g_plan);
        const at::Tensor& lens = dense(a[0], at::kInt, 1);
        const Place place(lens);
        const int64_t B = lens.size(0);
        const at::Tensor& add = dense(a[1], at::kInt, {B}, place.dev);
        const at::Tensor& free = dense(a[2], at::kInt, 1);
        const at::Tensor& table = dense(a[3], at::kInt, 2);
        need(free.get_device() == place.dev && table.get_device() == place.dev && table.size(0) == B);
        const int page_size = small(a[4]), room = small(a[5]);
        need(B > 0 && room > 0);
        const at::Tensor slots = at::empty({room}, lens.options().dtype(at::kLong));
        const int64_t at_out = (B + 1 + 31) / 32 * 32, at_counts = at_out + (B + 31) / 32 * 32;  // on 128 bytes
        const at::Tensor small_ones = at::empty({at_counts + 2}, lens.options());
        const at::Tensor cu = piece(small_ones, 0, B + 1), out = piece(small_ones, at_out, B), counts = piece(small_ones, at_counts, 2);
        static_assert(sizeof(long long) == sizeof(int64_t), "slots");
        need(g_plan(lens.data_ptr<int>(), add.data_ptr<int>(), static_cast<int>(B), free.data_ptr<int>(),
                    static_cast<int>(free.size(0)), table.data_ptr<int>(), static_cast<int>(table.size(1)), page_size,
                    static_cast<long long*>(slots.data_ptr()), room, cu.data_ptr<int>(), out.data_ptr<int>(),
                    counts.data_ptr<int>(), place.stream) == 0);
        return tuple(slots, cu, out, counts);
    });
}

// append(k, v, slot_map, k_pages, v_pages, k_scales, v_scales) -> True
PyObject* append(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return ordinary([&]() -> PyObject* {
        need(n == 7 && g_append);
        const at::Tensor& slots = dense(a[2], at::kLong, 1);
        const Place place(slots);
        const Cache c(a + 3, place.dev);
        const int64_t T = slots.size(0), H = c.heads, d = c.d;
        long long stride[2];
        const void* x[2];
        for (int i = 0; i < 2; ++i) {
            const at::Tensor& t = tensor(a[i]);
            need(t.scalar_type() == at::kBFloat16 && t.get_device() == place.dev && t.sizes() == at::IntArrayRef({T, H, d}) &&
                 t.stride(2) == 1 && (H == 1 || t.stride(1) == d) && (T == 1 || t.stride(0) >= H * d));
            stride[i] = T > 1 ? t.stride(0) : H * d;
            x[i] = t.data_ptr();
        }
        need(g_append(x[0], x[1], stride[0], stride[1], static_cast<const long long*>(slots.data_ptr()), static_cast<int>(T),
                      c.k.data_ptr(), c.v.data_ptr(), c.ks.data_ptr<float>(), c.vs.data_ptr<float>(), c.pages, c.page_size,
                      c.heads, c.d, place.stream) == 0);
        Py_RETURN_TRUE;
    });
}

// decode(q, k_pages, v_pages, k_scales, v_scales, block_table, seqlens_k, scale, window_left, num_splits)
PyObject* decode(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return ordinary([&]() -> PyObject* {
        need(n == 10 && g_decode && g_splits);
        const at::Tensor& q = dense(a[0], at::kBFloat16, 4);
        const Place place(q);
        const int64_t B = q.size(0), Hq = q.size(1), d = q.size(3);
        const Cache c(a + 1, place.dev);
        const at::Tensor& table = dense(a[5], at::kInt, 2);
        need(q.size(2) == 1 && c.d == d && B > 0 && table.get_device() == place.dev && table.size(0) == B);
        const at::Tensor& lens = dense(a[6], at::kInt, {B}, place.dev);
        const int left = small(a[8]);
        const int splits = small(a[9]);
        const int64_t Lk = table.size(1) * c.page_size;
        need(Lk > 0 && Lk <= kIntMax && splits >= 0);
        const int S = splits ? splits : g_splits(static_cast<int>(B), static_cast<int>(Hq), c.heads, static_cast<int>(Lk), static_cast<int>(d));
        need(S > 0);
        const at::Tensor o = at::empty(q.sizes(), q.options()), lse = at::empty({B, Hq}, c.ks.options());
        const int64_t bytes = S > 1 ? 4 * B * Hq * S * (d + 1) : 0;
        at::Tensor ws;
        if (bytes > 0) ws = at::empty({bytes}, c.k.options());
        need(g_decode(q.data_ptr(), c.k.data_ptr(), c.v.data_ptr(), c.ks.data_ptr<float>(), c.vs.data_ptr<float>(),
                      table.data_ptr<int>(), static_cast<int>(table.size(1)), c.page_size, c.pages, o.data_ptr(),
                      lse.data_ptr<float>(), lens.data_ptr<int>(), static_cast<int>(B), static_cast<int>(Hq), c.heads,
                      static_cast<int>(d), scale_of(a[7], d), left, splits, bytes > 0 ? ws.data_ptr() : nullptr,
                      static_cast<size_t>(bytes), place.stream) == 0);
        return tuple(o, lse);
    });
}

// fwd(q, k_pages, v_pages, k_scales, v_scales, block_table, seqlens_k, cu_seqlens_q, max_seqlen_q, scale, causal,
//     window_left, window_right)
PyObject* fwd(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return ordinary([&]() -> PyObject* {
        need(n == 13 && g_fwd && g_fwd_bytes);
        const at::Tensor& q = dense(a[0], at::kBFloat16, 3);
        const Place place(q);
        const int64_t T = q.size(0), Hq = q.size(1), d = q.size(2);
        const Cache c(a + 1, place.dev);
        const at::Tensor& lens = dense(a[6], at::kInt, 1);
        const int64_t B = lens.size(0);
        const at::Tensor& table = dense(a[5], at::kInt, 2);
        need(c.d == d && B > 0 && T > 0 && lens.get_device() == place.dev && table.get_device() == place.dev &&
             table.size(0) == B && c.heads > 0 && Hq % c.heads == 0);
        const at::Tensor& cu = dense(a[7], at::kInt, {B + 1}, place.dev);
        const int most = small(a[8]);
        const int64_t Lk = table.size(1) * c.page_size;
        need(most > 0 && Lk > 0 && Lk <= kIntMax);
        need(PyBool_Check(a[10]));
        const size_t bytes = g_fwd_bytes(static_cast<int>(B), static_cast<int>(T), most, static_cast<int>(Hq), c.heads,
                                         static_cast<int>(Lk), static_cast<int>(d));
        const at::Tensor o = at::empty(q.sizes(), q.options()), lse = at::empty({Hq, T}, c.ks.options());
        at::Tensor ws;
        if (bytes > 0) ws = at::empty({static_cast<int64_t>(bytes)}, c.k.options());
        need(g_fwd(q.data_ptr(), c.k.data_ptr(), c.v.data_ptr(), c.ks.data_ptr<float>(), c.vs.data_ptr<float>(),
                   table.data_ptr<int>(), static_cast<int>(table.size(1)), c.page_size, c.pages, o.data_ptr(),
                   lse.data_ptr<float>(), lens.data_ptr<int>(), cu.data_ptr<int>(), static_cast<int>(B), static_cast<int>(T),
                   most, static_cast<int>(Hq), c.heads, static_cast<int>(d), scale_of(a[9], d), a[10] == Py_True,
                   small(a[11]), small(a[12]), bytes > 0 ? ws.data_ptr() : nullptr, bytes, place.stream) == 0);
        return tuple(o, lse);
    });
}

// bind(name, address): the library's function of that name.
PyObject* bind(PyObject*, PyObject* args) {
    const char* name = nullptr;
    unsigned long long at = 0;
    if (!PyArg_ParseTuple(args, "sK", &name, &at)) return nullptr;
    const std::string s(name);
    void* p = reinterpret_cast<void*>(static_cast<uintptr_t>(at));
    if (s == "attn_paged_plan") g_plan = reinterpret_cast<PlanFn>(p);
    else if (s == "attn_append_paged_fp8") g_append = reinterpret_cast<AppendFn>(p);
    else if (s == "attn_decode_paged_fp8") g_decode = reinterpret_cast<DecodeFn>(p);
    else if (s == "attn_decode_paged_fp8_auto_splits") g_splits = reinterpret_cast<SplitsFn>(p);
    else if (s == "attn_fwd_paged_fp8") g_fwd = reinterpret_cast<FwdFn>(p);
    else if (s == "attn_fwd_paged_fp8_workspace_bytes") g_fwd_bytes = reinterpret_cast<FwdBytesFn>(p);
    else {
        PyErr_Format(PyExc_KeyError, "no function %s", name);
        return nullptr;
    }
    Py_RETURN_NONE;
}

PyMethodDef kMethods[] = {
    {"bind", bind, METH_VARARGS, "Hand over the address of a function of the library."},
    {"plan", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)(void)>(plan)), METH_FASTCALL, nullptr},
    {"append", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)(void)>(append)), METH_FASTCALL, nullptr},
    {"decode", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)(void)>(decode)), METH_FASTCALL, nullptr},
    {"fwd", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)(void)>(fwd)), METH_FASTCALL, nullptr},
    {nullptr, nullptr, 0, nullptr}};

PyModuleDef kModule = {PyModuleDef_HEAD_INIT, "_fattn_calls", "Native checks and calls of the paged-cache operators.", -1, kMethods};

}  // namespace

PyMODINIT_FUNC PyInit__fattn_calls() { return PyModule_Create(&kModule); }
