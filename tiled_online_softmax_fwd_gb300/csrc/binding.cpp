// binding.cpp -- torch tensors for the calls of a drafting or searching step and
// of cross attention: attn_fwd_tree, fattn_tree_mask, fattn_kv_append,
// fattn_kv_keep, fattn_kv_fork, attn_fwd_cross, attn_bwd_cross.
//
// Such a call is a few microseconds of GPU work, made once a layer or a step.
// Checking its tensors, making its outputs and passing some thirty arguments took
// 28 us in Python; here they take a few.  Each function takes all of its call's
// arguments by position (fattn.py gives them their names and defaults), raises
// TypeError or ValueError for what is no tensor or does not fit, and hands the
// library's status to the callable that fattn.py gives to `init`.
#include <Python.h>

#include <ATen/core/Tensor.h>
#include <ATen/cuda/EmptyTensor.h>
#include <c10/cuda/CUDACachingAllocator.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include <cmath>
#include <optional>
#include <string>

#include "fattn.h"

namespace {

using at::Tensor;

// A Python exception to raise.
struct Error {
    PyObject *type;
    std::string what;
};
// One that Python has raised already.
struct Raised {};

PyObject *g_check;  // (status, entry): raises the library's error

[[noreturn]] void bad_value(const std::string &what) { throw Error{PyExc_ValueError, what}; }

std::string shape_of(at::IntArrayRef s)
{
    std::string x = "[";
    for (size_t i = 0; i < s.size(); ++i)
        x += (i ? ", " : "") + std::to_string(s[i]);
    return x + "]";
}

const Tensor &tensor(const char *name, PyObject *o)
{
    if (!THPVariable_Check(o))
        throw Error{PyExc_TypeError, std::string(name) + " must be a torch.Tensor"};
    return THPVariable_Unpack(o);
}

// What the call's tensors have to share.
struct Kind {
    at::ScalarType dtype;
    int dev;
    int f16() const { return dtype == at::kHalf ? 1 : 0; }
};

bool last_contiguous(const Tensor &t) { return t.size(-1) <= 1 || t.stride(-1) == 1; }

// A 16-bit tensor that sets the kind, or has to fit it.
const Tensor &half(const char *name, PyObject *o, int dims, std::optional<Kind> &kind)
{
    const Tensor &t = tensor(name, o);
    if (!kind) {
        if (!t.is_cuda() || (t.scalar_type() != at::kBFloat16 && t.scalar_type() != at::kHalf))
            bad_value(std::string(name) + " must be a bf16 or fp16 CUDA tensor");
        kind = Kind{t.scalar_type(), t.get_device()};
    }
    if (t.dim() != dims || t.scalar_type() != kind->dtype || !t.is_cuda() || t.get_device() != kind->dev ||
        !last_contiguous(t))
        bad_value(std::string(name) + " must be a " + std::to_string(dims) + "-dimensional " +
                  c10::toString(kind->dtype) + " tensor on CUDA device " + std::to_string(kind->dev) +
                  " with a contiguous last dimension, got " + shape_of(t.sizes()) + " of " +
                  c10::toString(t.scalar_type()));
    return t;
}

// A list of `dims` dimensions whose last one is contiguous; dev < 0: any
// device, which it sets.
const Tensor &list(const char *name, PyObject *o, int dims, int &dev)
{
    const Tensor &t = tensor(name, o);
    if (dev < 0 && t.is_cuda())
        dev = t.get_device();
    if (t.scalar_type() != at::kInt || t.dim() != dims || !t.is_cuda() || t.get_device() != dev ||
        !last_contiguous(t))
        bad_value(std::string(name) + " must be a " + std::to_string(dims) +
                  "-dimensional int32 CUDA tensor with a contiguous last dimension, on the others' device");
    return t;
}

void expect(const char *name, const Tensor &t, at::IntArrayRef shape)
{
    if (t.sizes() != shape)
        bad_value(std::string(name) + " must be " + shape_of(shape) + ", got " + shape_of(t.sizes()));
}

int small(const char *name, int64_t x)
{
    if (x < 0 || x > 0x7fffffff)
        bad_value(std::string(name) + " is too large");
    return static_cast<int>(x);
}

int64_t number(PyObject *o)
{
    PyObject *i = PyNumber_Index(o);
    if (i == nullptr)
        throw Raised{};
    const int64_t x = PyLong_AsLongLong(i);
    Py_DECREF(i);
    if (x == -1 && PyErr_Occurred())
        throw Raised{};
    return x;
}

float scale_of(PyObject *o, int64_t d)
{
    if (o == Py_None)
        return static_cast<float>(1.0 / std::sqrt(static_cast<double>(d)));
    const double x = PyFloat_AsDouble(o);
    if (x == -1.0 && PyErr_Occurred())
        throw Raised{};
    return static_cast<float>(x);
}

// Strides of the outer dimensions.
struct Strides {
    long long at[3] = {0, 0, 0};
    explicit Strides(const Tensor &t)
    {
        for (int64_t i = 0; i + 1 < t.dim() && i < 3; ++i)
            at[i] = t.stride(i);
    }
};

// The stream of a call (None: the current one) and, while it lives, the current
// device and stream: new tensors are the stream's, so memory that is freed while
// the call still runs there is reused only behind it.
struct Place {
    c10::cuda::OptionalCUDAGuard device;
    c10::cuda::OptionalCUDAStreamGuard guard;
    CUstream_st *stream;
    Place(PyObject *o, int dev)
    {
        device.set_index(static_cast<c10::DeviceIndex>(dev));
        if (o == Py_None) {
            stream = c10::cuda::getCurrentCUDAStream(static_cast<c10::DeviceIndex>(dev)).stream();
            return;
        }
        PyObject *handle = PyObject_HasAttrString(o, "cuda_stream") ? PyObject_GetAttrString(o, "cuda_stream")
                                                                    : Py_NewRef(o);
        if (handle == nullptr)
            throw Raised{};
        const unsigned long long x = PyLong_AsUnsignedLongLong(handle);
        Py_DECREF(handle);
        if (PyErr_Occurred())
            throw Raised{};
        stream = reinterpret_cast<CUstream_st *>(x);
        guard.reset_stream(stream == nullptr
                               ? c10::cuda::getDefaultCUDAStream(static_cast<c10::DeviceIndex>(dev))
                               : c10::cuda::getStreamFromExternal(stream, static_cast<c10::DeviceIndex>(dev)));
    }
};

// Past the dispatcher, which takes as long as the allocation.
Tensor make(at::IntArrayRef shape, at::ScalarType type, int dev)
{
    return Tensor(at::detail::empty_cuda(shape, type, at::Device(at::kCUDA, static_cast<c10::DeviceIndex>(dev)),
                                         std::nullopt));
}

// An output: as given, checked, or new.
Tensor half_out(const char *name, PyObject *o, at::IntArrayRef shape, std::optional<Kind> &kind)
{
    if (o == Py_None)
        return make(shape, kind->dtype, kind->dev);
    const Tensor &t = half(name, o, static_cast<int>(shape.size()), kind);
    expect(name, t, shape);
    return t;
}
Tensor plain_out(const char *name, PyObject *o, at::IntArrayRef shape, at::ScalarType type, int dev)
{
    if (o == Py_None)
        return make(shape, type, dev);
    const Tensor &t = tensor(name, o);
    if (t.scalar_type() != type || t.sizes() != shape || !t.is_cuda() || t.get_device() != dev ||
        !t.is_contiguous())
        bad_value(std::string(name) + " must be a contiguous " + c10::toString(type) + " " + shape_of(shape) +
                  " tensor on CUDA device " + std::to_string(dev));
    return t;
}
// A call's workspace: as given, or memory of the current device and stream until
// the call has been enqueued.
struct Workspace {
    c10::DataPtr own;
    void *at;
    size_t bytes;
    Workspace(PyObject *o, size_t need, int dev)
    {
        if (o == Py_None) {
            bytes = need < 16 ? 16 : need;
            own = c10::cuda::CUDACachingAllocator::get()->allocate(bytes);
            at = own.get();
            return;
        }
        const Tensor &t = tensor("workspace", o);
        if (!t.is_cuda() || t.get_device() != dev || !t.is_contiguous())
            bad_value("workspace must be a contiguous tensor on CUDA device " + std::to_string(dev));
        at = t.data_ptr();
        bytes = t.nbytes();
    }
};

template <class T> T *ptr(const Tensor &t) { return static_cast<T *>(t.data_ptr()); }
const int *ints(const Tensor &t) { return ptr<const int>(t); }

// Runs the C call without the interpreter's lock and has its status looked at.
struct Unlocked {  // takes the lock again when an exception leaves, too
    PyThreadState *state = PyEval_SaveThread();
    ~Unlocked() { PyEval_RestoreThread(state); }
};
template <class F> void call(const char *entry, F f)
{
    fattn_status_t s;
    {
        const Unlocked unlocked;
        s = f();
    }
    if (s == FATTN_OK)
        return;
    PyObject *r = PyObject_CallFunction(g_check, "is", static_cast<int>(s), entry);
    Py_XDECREF(r);
    throw Raised{};
}

// ------------------------------------------------------------------ paged cache
struct Cache {
    const Tensor &k, &v;
    int pages, heads, page, d;
};
Cache cache_of(PyObject *ko, PyObject *vo, std::optional<Kind> &kind)
{
    const Tensor &k = half("k_cache", ko, 4, kind), &v = half("v_cache", vo, 4, kind);
    expect("v_cache", v, k.sizes());
    const int64_t page = k.size(2), d = k.size(3);
    if (page < 16 || (page & (page - 1)) != 0)
        bad_value("page size must be a power of two, 16 or more, got " + std::to_string(page));
    if (d != 64 && d != 96 && d != 128 && d != 256)
        bad_value("head dimension must be 64, 96, 128 or 256, got " + std::to_string(d));
    return Cache{k, v, small("the pool", k.size(0)), small("Hk", k.size(1)), small("the page size", k.size(2)),
                 small("d", k.size(3))};
}
long long row_stride(const Tensor &t) { return t.size(0) > 1 ? t.stride(0) : t.size(1); }

// q, k_cache, v_cache, page_table, cu_q, kv_len, mask, max_q, scale, workspace, out, lse, stream
PyObject *attn_fwd_tree(PyObject *const *a)
{
    std::optional<Kind> kind;
    const Tensor &q = half("q", a[0], 3, kind);
    const Cache c = cache_of(a[1], a[2], kind);
    int dev = kind->dev;
    const Tensor &table = list("page_table", a[3], 2, dev), &cu = list("cu_q", a[4], 1, dev),
                 &kv_len = list("kv_len", a[5], 1, dev), &mask = list("mask", a[6], 2, dev);
    const int T = small("T", q.size(0)), Hq = small("Hq", q.size(1)), d = small("d", q.size(2));
    const int B = small("B", table.size(0)), max_q = small("max_q", number(a[7]));
    expect("cu_q", cu, {B + 1});
    expect("kv_len", kv_len, {B});
    expect("mask", mask, {T, mask.size(1)});
    if (c.d != d || (d != 64 && d != 96 && d != 128))
        bad_value("head dimension must be 64, 96 or 128 and the caches', got " + std::to_string(d));
    if (c.heads == 0 || Hq % c.heads != 0)
        bad_value("Hq must be a multiple of the caches' heads");
    const float scale = scale_of(a[8], d);
    Place place(a[12], dev);
    const Tensor out = half_out("out", a[10], q.sizes(), kind);
    const Tensor lse = plain_out("lse", a[11], {T, Hq}, at::kFloat, dev);
    const Workspace ws(a[9], attn_fwd_paged_workspace_size(Hq, c.heads, d, max_q), dev);
    const Strides qs(q), ks(c.k), vs(c.v), os(out);
    call("attn_fwd_tree", [&] {
        return ::attn_fwd_tree(q.data_ptr(), c.k.data_ptr(), c.v.data_ptr(), ints(table), ints(cu),
                               ints(kv_len), ptr<const unsigned>(mask), out.data_ptr(), ptr<float>(lse), T, B,
                               Hq, c.heads, d, c.pages, c.page, small("the table", table.size(1)),
                               row_stride(table), max_q, small("the mask", mask.size(1)), row_stride(mask),
                               qs.at, ks.at, vs.at, os.at, scale, kind->f16(), ws.at, ws.bytes,
                               place.stream);
    });
    return Py_BuildValue("NN", THPVariable_Wrap(out), THPVariable_Wrap(lse));
}

// parents, cu_q, kv_len, max_q, mask, positions, stream
PyObject *tree_mask(PyObject *const *a)
{
    int dev = -1;
    const Tensor &parents = list("parents", a[0], 1, dev), &cu = list("cu_q", a[1], 1, dev),
                 &kv_len = list("kv_len", a[2], 1, dev);
    const int T = small("T", parents.size(0)), B = small("B", kv_len.size(0));
    expect("cu_q", cu, {B + 1});
    const int64_t max_q = number(a[3]);
    if (max_q < 1)
        bad_value("max_q must be at least 1, got " + std::to_string(max_q));
    const int words = small("max_q", (max_q + 31) / 32);
    Place place(a[6], dev);
    const Tensor mask = plain_out("mask", a[4], {T, words}, at::kInt, dev);
    const Tensor pos = plain_out("positions", a[5], {1, T}, at::kInt, dev);
    call("fattn_tree_mask", [&] {
        return fattn_tree_mask(ints(parents), ints(cu), ints(kv_len), ptr<unsigned>(mask), ptr<int>(pos), T, B,
                               words, place.stream);
    });
    return Py_BuildValue("NN", THPVariable_Wrap(mask), THPVariable_Wrap(pos));
}

// k, v, k_cache, v_cache, page_table, cu_q, kv_len, rope, interleaved, stream
PyObject *kv_append(PyObject *const *a)
{
    std::optional<Kind> kind;
    const Tensor &k = half("k", a[0], 3, kind), &v = half("v", a[1], 3, kind);
    expect("v", v, k.sizes());
    const Cache c = cache_of(a[2], a[3], kind);
    int dev = kind->dev;
    const Tensor &table = list("page_table", a[4], 2, dev), &cu = list("cu_q", a[5], 1, dev),
                 &kv_len = list("kv_len", a[6], 1, dev);
    const int T = small("T", k.size(0)), B = small("B", table.size(0));
    expect("k", k, {T, c.heads, c.d});
    expect("cu_q", cu, {B + 1});
    expect("kv_len", kv_len, {B});
    const float *rope = nullptr;
    int rot = 0, max_pos = 0;
    if (a[7] != Py_None) {
        const Tensor &t = tensor("rope", a[7]);
        if (t.scalar_type() != at::kFloat || t.dim() != 2 || !t.is_contiguous() || !t.is_cuda() ||
            t.get_device() != dev)
            bad_value("rope must be a contiguous fp32 [positions, rot_dim] tensor on CUDA device " +
                      std::to_string(dev));
        if (t.size(1) % 16 != 0 || t.size(1) < 1 || t.size(1) > c.d)
            bad_value("rope must have 16, 32, ... up to " + std::to_string(c.d) + " columns, got " +
                      std::to_string(t.size(1)));
        rope = ptr<const float>(t);
        rot = small("rope", t.size(1));
        max_pos = small("rope", t.size(0));
    }
    const int interleaved = PyObject_IsTrue(a[8]);
    if (interleaved < 0)
        throw Raised{};
    Place place(a[9], dev);
    const Strides ks(k), vs(v), kcs(c.k), vcs(c.v);
    call("fattn_kv_append", [&] {
        return fattn_kv_append(k.data_ptr(), v.data_ptr(), c.k.data_ptr(), c.v.data_ptr(), ints(table), ints(cu),
                               ints(kv_len), rope, T, B, c.heads, c.d, c.pages, c.page,
                               small("the table", table.size(1)), row_stride(table), rot, max_pos, ks.at, vs.at,
                               kcs.at, vcs.at, interleaved, kind->f16(), place.stream);
    });
    return Py_BuildValue("OO", a[2], a[3]);
}

// k_cache, v_cache, page_table, cu_q, kv_len, kept, kept_len, kv_len_out, stream
PyObject *kv_keep(PyObject *const *a)
{
    std::optional<Kind> kind;
    tensor("kv_len", a[4]);
    const Cache c = cache_of(a[0], a[1], kind);
    int dev = kind->dev;
    const Tensor &table = list("page_table", a[2], 2, dev), &cu = list("cu_q", a[3], 1, dev),
                 &kv_len = list("kv_len", a[4], 1, dev), &kept = list("kept", a[5], 2, dev),
                 &kept_len = list("kept_len", a[6], 1, dev);
    const int B = small("B", kv_len.size(0));
    expect("page_table", table, {B, table.size(1)});
    expect("cu_q", cu, {B + 1});
    expect("kept", kept, {B, kept.size(1)});
    expect("kept_len", kept_len, {B});
    Place place(a[8], dev);
    const Tensor out = plain_out("kv_len_out", a[7], {B}, at::kInt, dev);
    const Strides ks(c.k), vs(c.v);
    call("fattn_kv_keep", [&] {
        return fattn_kv_keep(c.k.data_ptr(), c.v.data_ptr(), ints(table), ints(cu), ints(kv_len), ints(kept),
                             ints(kept_len), ptr<int>(out), B, c.heads, c.d, c.pages, c.page,
                             small("the table", table.size(1)), row_stride(table),
                             small("kept", kept.size(1)), row_stride(kept), ks.at, vs.at, place.stream);
    });
    return a[7] == Py_None ? THPVariable_Wrap(out) : Py_NewRef(a[7]);
}

// k_cache, v_cache, page_table, kv_len, page_refs, parents, cu_q, page_table_out, kv_len_out,
// page_refs_out, workspace, stream
PyObject *kv_fork(PyObject *const *a)
{
    std::optional<Kind> kind;
    tensor("kv_len", a[3]);
    const Cache c = cache_of(a[0], a[1], kind);
    int dev = kind->dev;
    const Tensor &table = list("page_table", a[2], 2, dev), &kv_len = list("kv_len", a[3], 1, dev),
                 &refs = list("page_refs", a[4], 1, dev);
    const int B = small("B", kv_len.size(0)), cols = small("the table", table.size(1));
    expect("page_table", table, {B, cols});
    expect("page_refs", refs, {c.pages});
    const int *parents = nullptr, *cu = nullptr;
    if (a[5] != Py_None) {
        const Tensor &t = list("parents", a[5], 1, dev);
        expect("parents", t, {B});
        parents = ints(t);
    }
    if (a[6] != Py_None) {
        const Tensor &t = list("cu_q", a[6], 1, dev);
        expect("cu_q", t, {B + 1});
        cu = ints(t);
    }
    Place place(a[11], dev);
    Tensor table_out;
    if (a[7] == Py_None) {
        table_out = make({B, cols}, at::kInt, dev);
    } else {
        table_out = list("page_table_out", a[7], 2, dev);
        expect("page_table_out", table_out, {B, cols});
    }
    const Tensor len_out = plain_out("kv_len_out", a[8], {B}, at::kInt, dev);
    const Tensor refs_out = plain_out("page_refs_out", a[9], {c.pages}, at::kInt, dev);
    const Workspace ws(a[10], fattn_kv_fork_workspace_size(B, cols, c.pages), dev);
    const Strides ks(c.k), vs(c.v);
    call("fattn_kv_fork", [&] {
        return fattn_kv_fork(c.k.data_ptr(), c.v.data_ptr(), ints(table), ints(kv_len), ints(refs), parents, cu,
                             ptr<int>(table_out), ptr<int>(len_out), ptr<int>(refs_out), B, c.heads, c.d,
                             c.pages, c.page, cols, row_stride(table), row_stride(table_out), ks.at, vs.at,
                             ws.at, ws.bytes, place.stream);
    });
    auto give = [](PyObject *o, const Tensor &t) { return o == Py_None ? THPVariable_Wrap(t) : Py_NewRef(o); };
    return Py_BuildValue("NNN", give(a[7], table_out), give(a[8], len_out), give(a[9], refs_out));
}

// ------------------------------------------------------------------ cross attention
struct Cross {
    std::optional<Kind> kind;
    const Tensor &q, &k, &v;
    const int *kv_len = nullptr;
    int B, Hq, Hk, Nq, Nk, d, dev;
    Cross(PyObject *qo, PyObject *ko, PyObject *vo, PyObject *lo)
        : q(half("q", qo, 4, kind)), k(half("k", ko, 4, kind)), v(half("v", vo, 4, kind)),
          B(small("B", q.size(0))), Hq(small("Hq", q.size(1))), Hk(small("Hk", k.size(1))),
          Nq(small("Nq", q.size(2))), Nk(small("Nk", k.size(2))), d(small("d", q.size(3))), dev(kind->dev)
    {
        expect("k", k, {B, Hk, Nk, d});
        expect("v", v, k.sizes());
        if (d != 64 && d != 96 && d != 128)
            bad_value("head dimension must be 64, 96 or 128, got " + std::to_string(d));
        if (Hk == 0 || Hq % Hk != 0 || Hq / Hk > 128)
            bad_value("Hq must be 1 to 128 times Hk, got " + std::to_string(Hq) + " and " + std::to_string(Hk));
        if (lo != Py_None) {
            const Tensor &t = list("kv_len", lo, 1, dev);
            expect("kv_len", t, {B});
            kv_len = ints(t);
        }
    }
};

// q, k, v, kv_len, scale, workspace, out, lse, stream
PyObject *attn_fwd_cross(PyObject *const *a)
{
    Cross c(a[0], a[1], a[2], a[3]);
    const float scale = scale_of(a[4], c.d);
    Place place(a[8], c.dev);
    const Tensor out = half_out("out", a[6], c.q.sizes(), c.kind);
    const Tensor lse = plain_out("lse", a[7], {c.B, c.Hq, c.Nq}, at::kFloat, c.dev);
    const Workspace ws(a[5], attn_fwd_cross_workspace_size(c.Hq, c.Hk, c.Nq, c.d), c.dev);
    const Strides qs(c.q), ks(c.k), vs(c.v), os(out);
    call("attn_fwd_cross", [&] {
        return ::attn_fwd_cross(c.q.data_ptr(), c.k.data_ptr(), c.v.data_ptr(), c.kv_len, out.data_ptr(),
                                ptr<float>(lse), c.B, c.Hq, c.Hk, c.Nq, c.Nk, c.d, qs.at, ks.at, vs.at, os.at,
                                scale, c.kind->f16(), ws.at, ws.bytes, place.stream);
    });
    return Py_BuildValue("NN", THPVariable_Wrap(out), THPVariable_Wrap(lse));
}

// q, k, v, o, lse, do, kv_len, scale, dq, dk, dv, workspace, stream
PyObject *attn_bwd_cross(PyObject *const *a)
{
    Cross c(a[0], a[1], a[2], a[6]);
    const Tensor &o = half("o", a[3], 4, c.kind), &dout = half("do", a[5], 4, c.kind);
    expect("o", o, c.q.sizes());
    expect("do", dout, c.q.sizes());
    if (a[4] == Py_None)
        throw Error{PyExc_TypeError, "lse must be a torch.Tensor"};
    const Tensor lse = plain_out("lse", a[4], {c.B, c.Hq, c.Nq}, at::kFloat, c.dev);
    const float scale = scale_of(a[7], c.d);
    Place place(a[12], c.dev);
    const Tensor dq = half_out("dq", a[8], c.q.sizes(), c.kind);
    const Tensor dk = half_out("dk", a[9], c.k.sizes(), c.kind), dv = half_out("dv", a[10], c.v.sizes(), c.kind);
    const Workspace ws(a[11], attn_bwd_cross_workspace_size(c.B, c.Hq, c.Hk, c.Nq, c.Nk, c.d), c.dev);
    const Strides qs(c.q), ks(c.k), vs(c.v), os(o), gs(dout), dqs(dq), dks(dk), dvs(dv);
    call("attn_bwd_cross", [&] {
        return ::attn_bwd_cross(c.q.data_ptr(), c.k.data_ptr(), c.v.data_ptr(), o.data_ptr(),
                                ptr<const float>(lse), dout.data_ptr(), c.kv_len, dq.data_ptr(), dk.data_ptr(),
                                dv.data_ptr(), c.B, c.Hq, c.Hk, c.Nq, c.Nk, c.d, qs.at, ks.at, vs.at, os.at,
                                gs.at, dqs.at, dks.at, dvs.at, scale, c.kind->f16(), ws.at, ws.bytes,
                                place.stream);
    });
    return Py_BuildValue("NNN", THPVariable_Wrap(dq), THPVariable_Wrap(dk), THPVariable_Wrap(dv));
}

// ------------------------------------------------------------------ module
// torch's own exception, as its allocations raise it in Python.
void raise_out_of_memory(const char *what)
{
    PyObject *torch = PyImport_ImportModule("torch");
    PyObject *type = torch != nullptr ? PyObject_GetAttrString(torch, "OutOfMemoryError") : nullptr;
    if (type != nullptr)
        PyErr_SetString(type, what);
    Py_XDECREF(type);
    Py_XDECREF(torch);
}

template <PyObject *(*kF)(PyObject *const *), int kArgs>
PyObject *entry(PyObject *, PyObject *const *args, Py_ssize_t n)
{
    try {
        if (n != kArgs)
            throw Error{PyExc_TypeError, std::to_string(kArgs) + " arguments expected, got " + std::to_string(n)};
        return kF(args);
    } catch (const Error &e) {
        PyErr_SetString(e.type, e.what.c_str());
    } catch (const Raised &) {
        if (!PyErr_Occurred())
            PyErr_SetString(PyExc_RuntimeError, "the library's error was not raised");
    } catch (const c10::OutOfMemoryError &e) {
        raise_out_of_memory(e.what_without_backtrace());
    } catch (const std::exception &e) {  // a device that is not there
        PyErr_SetString(PyExc_RuntimeError, e.what());
    }
    return nullptr;
}

PyObject *init(PyObject *, PyObject *check)
{
    Py_XSETREF(g_check, Py_NewRef(check));
    Py_RETURN_NONE;
}

#define ENTRY(name, args)                                                                             \
    {                                                                                                 \
#name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)(void)>(entry<name, args>)), METH_FASTCALL, \
            nullptr                                                                                   \
    }
PyMethodDef methods[] = {ENTRY(attn_fwd_tree, 13),
                         ENTRY(tree_mask, 7),
                         ENTRY(kv_append, 10),
                         ENTRY(kv_keep, 9),
                         ENTRY(kv_fork, 12),
                         ENTRY(attn_fwd_cross, 9),
                         ENTRY(attn_bwd_cross, 13),
                         {"init", init, METH_O, nullptr},
                         {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "fattn_binding", nullptr, -1, methods};

}  // namespace

PyMODINIT_FUNC PyInit_fattn_binding(void) { return PyModule_Create(&module); }
