// kamera_binding.cpp -- Python binding of the decode-step entry points.
//
// A decode step calls these once per layer and step, for kernels of a few
// microseconds, so what a call costs on the host counts: marshalling the same
// arguments through ctypes took 15 to 28 us a call.  This module checks torch
// tensors, allocates outputs and workspaces and calls the C entry points
// (kamera.h); it holds no arithmetic and keeps nothing between calls.
//
// Memory: outputs and workspaces come from torch's allocator on the call's
// stream.  With another stream than the current one they come from that
// stream's pool -- a block of the current stream's could still be in use there
// -- and outputs are marked as used on the current one, where the caller reads
// them.  A captured graph therefore owns its workspace.
#include <Python.h>

#include <array>
#include <cmath>
#include <cstdint>
#include <cstring>
#include <optional>
#include <stdexcept>
#include <string>

#include <ATen/core/Tensor.h>
#include <ATen/cuda/EmptyTensor.h>
#include <ATen/ops/empty.h>
#include <c10/cuda/CUDACachingAllocator.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include "kamera.h"

namespace {

struct Refused : std::runtime_error {   // a ValueError (or TypeError) for the caller
    PyObject* type;
    Refused(PyObject* t, const std::string& what) : std::runtime_error(what), type(t) {}
};
struct Raised {};   // a Python exception is already set

[[noreturn]] void value_error(const std::string& what) { throw Refused(PyExc_ValueError, what); }

class Ref {   // an owned reference
public:
    explicit Ref(PyObject* o = nullptr) : o_(o) {}
    ~Ref() { Py_XDECREF(o_); }
    Ref(const Ref&) = delete;
    Ref& operator=(const Ref&) = delete;
    PyObject* get() const { return o_; }
    void set(PyObject* o)
    {
        Py_XDECREF(o_);
        o_ = o;
    }

private:
    PyObject* o_;
};

const at::Tensor* optional(PyObject* o, const char* name)
{
    if (o == Py_None)
        return nullptr;
    if (!THPVariable_Check(o))
        throw Refused(PyExc_TypeError, std::string(name) + " must be a tensor");
    return &THPVariable_Unpack(o);
}

const at::Tensor& tensor(PyObject* o, const char* name)
{
    const at::Tensor* t = optional(o, name);
    if (!t)
        throw Refused(PyExc_TypeError, std::string(name) + " must be a tensor");
    return *t;
}

int64_t integer(PyObject* o, const char* name)
{
    const long long v = PyLong_AsLongLong(o);
    if (v == -1 && PyErr_Occurred()) {
        PyErr_Clear();
        Ref i(PyNumber_Index(o));   // numpy integers and the like
        if (!i.get()) {
            PyErr_Clear();
            throw Refused(PyExc_TypeError, std::string(name) + " must be an integer");
        }
        const long long w = PyLong_AsLongLong(i.get());
        if (w == -1 && PyErr_Occurred()) {
            PyErr_Clear();
            value_error(std::string(name) + " is out of range");
        }
        return w;
    }
    return v;
}

int32_t int32(PyObject* o, const char* name)
{
    const int64_t v = integer(o, name);
    if (v > INT32_MAX || v < INT32_MIN)
        value_error(std::string(name) + " is out of range");
    return (int32_t)v;
}

int32_t size32(int64_t v, const char* name)
{
    if (v > INT32_MAX)
        value_error(std::string(name) + " is too large");
    return (int32_t)v;
}

void* addr(const at::Tensor* t) { return t ? t->data_ptr() : nullptr; }

void bf16(const at::Tensor& t, const char* name)
{
    if (t.scalar_type() != at::kBFloat16)
        throw Refused(PyExc_TypeError, std::string(name) + " must be bfloat16");
}

std::string shape_text(at::IntArrayRef s)
{
    std::string o = "[";
    for (size_t i = 0; i < s.size(); ++i)
        o += (i ? ", " : "") + std::to_string(s[i]);
    return o + "]";
}

void exact(const at::Tensor& t, const char* name, at::ScalarType type, at::IntArrayRef shape)
{
    if (t.scalar_type() != type || t.sizes() != shape || !t.is_contiguous())
        value_error(std::string(name) + " must be a contiguous " + c10::toString(type) + " tensor of shape " +
                    shape_text(shape));
}

// A dimension's stride; 0 where it has one element and none is taken.
int64_t step(const at::Tensor& t, int64_t dim) { return t.size(dim) > 1 ? t.stride(dim) : 0; }

// Rows [..., H, d] whose heads lie behind one another.
bool packed(const at::Tensor& t)
{
    const int64_t n = t.dim();
    return t.stride(n - 1) == 1 && (t.size(n - 2) <= 1 || t.stride(n - 2) == t.size(n - 1));
}

// The same shape, and every element at the same offset.
bool same_layout(const at::Tensor& a, const at::Tensor& b)
{
    if (a.sizes() != b.sizes())
        return false;
    for (int64_t i = 0; i < a.dim(); ++i)
        if (step(a, i) != step(b, i))
            return false;
    return true;
}

// Where a call runs: the device every tensor must live on, its stream.
class Place {
public:
    explicit Place(const char* where, const at::Tensor& ref) : where_(where), device_(ref.device()) {}

    void check(const at::Tensor* t, const char* name) const
    {
        if (!t)
            return;
        if (!t->is_cuda() && cuda_present())
            value_error(std::string(where_) + ": " + name + " must be a CUDA tensor");
        if (t->device() != device_)
            value_error(std::string(where_) + ": " + name + " is on " + t->device().str() + ", not on " +
                        device_.str());
    }
    void check(const at::Tensor& t, const char* name) const { check(&t, name); }

    // Makes the device current (until this object goes) and finds the call's stream.
    void enter(PyObject* stream)
    {
        if (!device_.is_cuda())
            return;
        guard_.set_device(device_);
        current_ = c10::cuda::getCurrentCUDAStream(device_.index());
        handle_ = current_->stream();
        if (stream == Py_None)
            return;
        uintptr_t h;
        if (PyLong_Check(stream)) {
            h = (uintptr_t)PyLong_AsUnsignedLongLong(stream);
        } else {
            Ref a(PyObject_GetAttrString(stream, "cuda_stream"));
            if (!a.get())
                throw Raised{};
            h = (uintptr_t)PyLong_AsUnsignedLongLong(a.get());
        }
        if (PyErr_Occurred())
            throw Raised{};
        if (h == (uintptr_t)handle_)
            return;
        handle_ = reinterpret_cast<cudaStream_t>(h);
        side_ = c10::cuda::getStreamFromExternal(handle_, device_.index());
    }

    at::Tensor empty(at::IntArrayRef shape, at::ScalarType type)
    {
        if (!device_.is_cuda())
            return at::empty(shape, at::TensorOptions().dtype(type).device(device_));
        // torch's allocation itself: on the way through its dispatcher it takes twice as long
        auto make = [&] { return at::Tensor(at::detail::empty_cuda(shape, type, device_, std::nullopt)); };
        if (!side_)
            return make();
        at::Tensor t;
        {
            c10::cuda::CUDAStreamGuard g(*side_);
            t = make();
        }
        t.record_stream(current_->unwrap());
        return t;
    }

    // Bytes of the call's stream, back in its pool when the call returns: what the
    // stream runs later comes after the kernels that use them.
    void* borrow(size_t bytes)
    {
        return device_.is_cuda() ? c10::cuda::CUDACachingAllocator::raw_alloc_with_stream(bytes, handle_) : nullptr;
    }

    struct CUstream_st* stream() const { return reinterpret_cast<struct CUstream_st*>(handle_); }

private:
    static bool cuda_present()
    {
        Ref m(PyImport_ImportModule("torch.cuda"));
        Ref r(m.get() ? PyObject_CallMethod(m.get(), "is_available", nullptr) : nullptr);
        if (!r.get())
            throw Raised{};
        return PyObject_IsTrue(r.get()) == 1;
    }

    const char* where_;
    c10::Device device_;
    c10::cuda::OptionalCUDAGuard guard_;
    std::optional<c10::cuda::CUDAStream> current_, side_;
    cudaStream_t handle_ = nullptr;
};

// A workspace for the call: the caller's tensor, or `need` bytes of the call's stream.
class Scratch {
public:
    Scratch(Place& on, const at::Tensor* given, size_t need)
    {
        if (given) {
            if (!given->is_contiguous())
                value_error("workspace must be contiguous");
            p = given->data_ptr();
            bytes = given->nbytes();
        } else if (need > 0) {
            p = own_ = on.borrow(need);
            bytes = p ? need : 0;
        }
    }
    ~Scratch()
    {
        if (own_)
            c10::cuda::CUDACachingAllocator::raw_delete(own_);
    }
    Scratch(const Scratch&) = delete;
    Scratch& operator=(const Scratch&) = delete;
    void* p = nullptr;
    size_t bytes = 0;

private:
    void* own_ = nullptr;
};

void status(int rc, const char* where)
{
    if (rc == KAMERA_OK)
        return;
    Ref m(PyImport_ImportModule("position_invariant_kv_chunk_gb300"));
    Ref type(m.get() ? PyObject_GetAttrString(m.get(), "KameraError") : nullptr);
    Ref e(type.get() ? PyObject_CallFunction(type.get(), "is", rc, where) : nullptr);
    if (e.get())
        PyErr_SetObject(type.get(), e.get());
    throw Raised{};
}

int32_t* error_word(const at::Tensor* err)
{
    if (!err)
        return nullptr;
    if (err->scalar_type() != at::kInt || err->numel() < 1)
        value_error("err must be an int32 tensor");
    return err->data_ptr<int32_t>();
}

// The Rope object: its plain fields here, tables and axes through the object's
// own marshalling (`keep` holds what that returns).
class RopeArg {
public:
    RopeArg(PyObject* o, int64_t n_tokens)
    {
        Ref inv(get(o, "inv_freq")), axes(get(o, "freq_axis"));
        axis_obj_.set(get(o, "axis_delta"));
        if (axis_obj_.get() != Py_None)
            axis = &tensor(axis_obj_.get(), "rope.axis_delta");
        if (axis && (axis->dim() != 2 || axis->size(0) != n_tokens || !axis->is_contiguous()))
            value_error("rope.axis_delta must be a contiguous [T, n_axes] tensor of positions");
        if (inv.get() == Py_None && axes.get() == Py_None && !axis) {
            std::memset(&c_, 0, sizeof(c_));
            Ref b(get(o, "base")), d(get(o, "rot_dim")), f(get(o, "rot_offset")), p(get(o, "pairing"));
            c_.base = PyFloat_AsDouble(b.get());
            if (PyErr_Occurred())
                throw Raised{};
            c_.rot_dim = int32(d.get(), "rot_dim");
            c_.rot_offset = int32(f.get(), "rot_offset");
            c_.pairing = int32(p.get(), "pairing");
            return;
        }
        keep_.set(PyObject_CallMethod(o, "_c", "L", (long long)n_tokens));
        if (!keep_.get())
            throw Raised{};
        Py_buffer b;
        if (PyObject_GetBuffer(PyTuple_GetItem(keep_.get(), 0), &b, PyBUF_SIMPLE))
            throw Raised{};
        const bool fits = b.len == (Py_ssize_t)sizeof(c_);
        if (fits)
            std::memcpy(&c_, b.buf, sizeof(c_));
        PyBuffer_Release(&b);
        if (!fits)
            value_error("rope does not marshal to a KameraRope");
    }
    const KameraRope* c() const { return &c_; }
    const at::Tensor* axis = nullptr;

private:
    static PyObject* get(PyObject* o, const char* name)
    {
        PyObject* a = PyObject_GetAttrString(o, name);
        if (!a)
            throw Raised{};
        return a;
    }
    Ref keep_, axis_obj_;
    KameraRope c_;
};

template <typename F>
PyObject* guarded(F f)
{
    try {
        return f();
    } catch (const Raised&) {
    } catch (const Refused& e) {
        PyErr_SetString(e.type, e.what());
    } catch (const std::exception& e) {   // torch's own errors, out of memory among them
        PyErr_SetString(PyExc_RuntimeError, e.what());
    }
    return nullptr;
}

void count(Py_ssize_t n, Py_ssize_t want)
{
    if (n != want)
        throw Refused(PyExc_TypeError, "wrong number of arguments");
}

// ------------------------------------------------------------------ append --


// What both append entry points share: rows k [T][...] and v, q [T][H_q][width].
template <typename Call>
PyObject* append(const char* where, Place& on, const at::Tensor& k, const at::Tensor& v, PyObject* rope_o,
                 PyObject* const* a, int64_t T, int64_t width, Call call)
{
    // a: positions, slots, layer, q, q_out, err, stream
    RopeArg rope(rope_o, T);
    const at::Tensor* positions = optional(a[0], "positions");
    const at::Tensor& slots = tensor(a[1], "slots");
    exact(slots, "slots", at::kLong, {T});
    if (rope.axis) {
        if (positions)
            value_error("with rope.axis_delta the positions are its rows; positions must be None");
    } else if (!positions) {
        value_error("positions are needed");
    } else {
        exact(*positions, "positions", at::kLong, {T});
    }
    const at::Tensor *q = optional(a[3], "q"), *q_out = optional(a[4], "q_out"), *err = optional(a[5], "err");
    if (q_out && !q)
        value_error("q_out without q");
    if (q && (q->dim() != 3 || q->size(0) != T || q->size(2) != width))
        value_error("k, v and q must hold the same tokens and head width");
    on.check(positions, "positions");
    on.check(slots, "slots");
    on.check(q, "q");
    on.check(q_out, "q_out");
    on.check(err, "err");
    on.check(rope.axis, "axis_delta");
    KameraAppendRows r;
    std::memset(&r, 0, sizeof(r));
    int32_t* e = error_word(err);
    on.enter(a[6]);
    at::Tensor made;
    if (q) {
        if (!q_out) {
            made = on.empty(q->sizes(), at::kBFloat16);
            q_out = &made;
        }
        if (q->scalar_type() != at::kBFloat16 || q_out->scalar_type() != at::kBFloat16 || q_out->sizes() != q->sizes() ||
            (width > 0 && (q->stride(2) != 1 || q_out->stride(2) != 1)))
            value_error("q and q_out must be bf16 [T, H_q, width] with packed rows");
        r.q = q->data_ptr();
        r.q_out = q_out->data_ptr();
        r.q_stride = q->stride(0);
        r.q_head_stride = q->stride(1);
        r.q_out_stride = q_out->stride(0);
        r.q_out_head_stride = q_out->stride(1);
        r.num_q_heads = size32(q->size(1), "q");
    }
    r.k = k.data_ptr();
    r.v = v.data_ptr();
    r.k_stride = k.stride(0);
    r.v_stride = v.stride(0);
    r.positions = positions ? positions->data_ptr<int64_t>() : nullptr;
    r.slots = slots.data_ptr<int64_t>();
    r.n_tokens = size32(T, "the token count");
    r.layer = int32(a[2], "layer");
    status(call(&r, rope.c(), e, on.stream()), where);
    if (made.defined())
        return THPVariable_Wrap(made);
    return Py_NewRef(q ? a[4] : Py_None);
}

// append_kv(pool_k, pool_v, k, v, rope, positions, slots, layer, q, q_out, err, stream)
PyObject* append_kv(PyObject*, PyObject* const* a, Py_ssize_t n)
{
    return guarded([&]() -> PyObject* {
        count(n, 12);
        const at::Tensor &pk = tensor(a[0], "pool_k"), &pv = tensor(a[1], "pool_v");
        const at::Tensor &k = tensor(a[2], "k"), &v = tensor(a[3], "v");
        bf16(pk, "pool_k");
        bf16(pv, "pool_v");
        bf16(k, "k");
        bf16(v, "v");
        if (pk.dim() != 4 || !packed(pk))
            value_error("pool_k must be [L, S, H, d] with packed heads");
        if (!same_layout(pk, pv))
            value_error("pool_k and pool_v must share shape and strides");
        const int64_t H = pk.size(2), d = pk.size(3), T = k.dim() == 3 ? k.size(0) : -1;
        auto rows = [&](const at::Tensor& t, const char* name) {
            if (t.dim() != 3 || t.size(0) != T || t.size(1) != H || t.size(2) != d || !packed(t))
                value_error(std::string(name) + " must be [T, H, d] with packed heads, the same T for k and v");
        };
        rows(k, "k");
        rows(v, "v");
        Place on("kamera_append_kv", k);
        on.check(k, "k");
        on.check(v, "v");
        on.check(pk, "pool_k");
        on.check(pv, "pool_v");
        KameraGqaPool pool;
        std::memset(&pool, 0, sizeof(pool));
        pool.num_layers = size32(pk.size(0), "pool_k");
        pool.num_kv_heads = size32(H, "pool_k");
        pool.head_dim = size32(d, "pool_k");
        pool.k = pk.data_ptr();
        pool.v = pv.data_ptr();
        pool.num_slots = pk.size(1);
        pool.layer_stride = step(pk, 0);
        pool.slot_stride = pk.stride(1);
        return append("kamera_append_kv", on, k, v, a[4], a + 5, T, d,
                      [&](const KameraAppendRows* r, const KameraRope* rope, int32_t* e, struct CUstream_st* s) {
                          return kamera_append_kv(&pool, r, rope, e, s);
                      });
    });
}

// mla_append_kv(pool, kv_lora, c, k_rope, rope, positions, slots, layer, q, q_out, err, stream)
PyObject* mla_append_kv(PyObject*, PyObject* const* a, Py_ssize_t n)
{
    return guarded([&]() -> PyObject* {
        count(n, 12);
        const at::Tensor &p = tensor(a[0], "pool"), &c = tensor(a[2], "c"), &kr = tensor(a[3], "k_rope");
        bf16(p, "pool");
        bf16(c, "c");
        bf16(kr, "k_rope");
        if (p.dim() != 3 || p.stride(2) != 1)
            value_error("pool must be [L, S, kv_lora + rope_dim] with packed rows");
        const int64_t lora = integer(a[1], "kv_lora"), rd = p.size(2) - lora, T = c.dim() == 2 ? c.size(0) : -1;
        auto rows = [&](const at::Tensor& t, const char* name, int64_t w) {
            if (t.dim() != 2 || t.size(0) != T || t.size(1) != w || (w > 1 && t.stride(1) != 1))
                value_error(std::string(name) + " must be [T, " + std::to_string(w) +
                            "] with packed rows, the same T for c and k_rope");
        };
        rows(c, "c", lora);
        rows(kr, "k_rope", rd);
        Place on("kamera_mla_append_kv", kr);
        on.check(kr, "k_rope");
        on.check(c, "c");
        on.check(p, "pool");
        KameraMlaPool pool;
        std::memset(&pool, 0, sizeof(pool));
        pool.num_layers = size32(p.size(0), "pool");
        pool.kv_lora_rank = size32(lora, "kv_lora");
        pool.rope_dim = size32(rd, "pool");
        pool.kv = p.data_ptr();
        pool.num_slots = p.size(1);
        pool.layer_stride = step(p, 0);
        pool.slot_stride = p.stride(1);
        return append("kamera_mla_append_kv", on, kr, c, a[4], a + 5, T, rd,
                      [&](const KameraAppendRows* r, const KameraRope* rope, int32_t* e, struct CUstream_st* s) {
                          return kamera_mla_append_kv(&pool, r, rope, e, s);
                      });
    });
}

// --------------------------------------------------------------- attention --
KameraPagedKV paged_kv(const at::Tensor& k, const at::Tensor* v, PyObject* page_size)
{
    bf16(k, "pool_k");
    if (k.dim() != 3 || !packed(k))
        value_error("pool_k must be [S, H, d] (one layer) with packed heads");
    if (v && (v->scalar_type() != at::kBFloat16 || !same_layout(k, *v)))
        value_error("pool_k and pool_v must share type, shape and strides");
    KameraPagedKV kv;
    std::memset(&kv, 0, sizeof(kv));
    kv.k = k.data_ptr();
    kv.v = addr(v);
    kv.num_slots = k.size(0);
    kv.slot_stride = k.stride(0);
    kv.num_kv_heads = size32(k.size(1), "pool_k");
    kv.head_dim = size32(k.size(2), "pool_k");
    kv.page_size = int32(page_size, "page_size");
    return kv;
}

void check_q(const at::Tensor& q, int64_t d)
{
    bf16(q, "q");
    if (q.dim() != 3 || q.size(2) != d || !q.is_contiguous())
        value_error("q must be a contiguous [S, H_q, d] tensor");
}

KameraPageTable page_table(const at::Tensor* pages, const at::Tensor* lens, int64_t n, int64_t max_len)
{
    KameraPageTable t;
    std::memset(&t, 0, sizeof(t));
    if (!pages && !lens && max_len == 0)
        return t;
    if (!pages || !lens || pages->dim() != 2)
        value_error("pages must be [S, max_pages] and lens [S]");
    exact(*pages, "pages", at::kInt, {n, pages->size(1)});
    exact(*lens, "lens", at::kInt, {n});
    t.pages = pages->data_ptr<int32_t>();
    t.lens = lens->data_ptr<int32_t>();
    t.max_pages = size32(pages->size(1), "pages");
    if (max_len > INT32_MAX || max_len < INT32_MIN)
        value_error("max_len is out of range");
    t.max_len = (int32_t)max_len;
    return t;
}

// q with its outputs: out and lse (None: allocated; lse False: not computed).
struct QueryArg {
    KameraPagedQuery c;
    const at::Tensor *out, *lse = nullptr;
    bool want_lse;
    PyObject *out_o, *lse_o;
    at::Tensor made_out, made_lse;
    std::array<int64_t, 3> shape;   // of out: q's, or another width

    QueryArg(const at::Tensor& q, PyObject* scale, PyObject* out_obj, PyObject* lse_obj, int64_t width = -1)
        : out_o(out_obj), lse_o(lse_obj), shape{q.size(0), q.size(1), width >= 0 ? width : q.size(2)}
    {
        std::memset(&c, 0, sizeof(c));
        out = optional(out_obj, "out");
        want_lse = lse_obj != Py_False;
        if (want_lse)
            lse = optional(lse_obj, "lse");
        if (out && (out->sizes() != at::IntArrayRef(shape) || out->scalar_type() != at::kBFloat16 || !out->is_contiguous()))
            value_error(width >= 0 ? "out must be a contiguous bf16 tensor of shape " + shape_text(shape)
                                   : std::string("out must be a contiguous bf16 tensor shaped like q"));
        if (lse && (lse->sizes() != q.sizes().slice(0, 2) || lse->scalar_type() != at::kFloat || !lse->is_contiguous()))
            value_error("lse must be a contiguous fp32 [S, H_q] tensor");
        c.q = q.data_ptr();
        c.n_seqs = size32(q.size(0), "q");
        c.num_q_heads = size32(q.size(1), "q");
        if (scale == Py_None) {
            c.scale = (float)(1.0 / std::sqrt((double)q.size(2)));
        } else {
            c.scale = (float)PyFloat_AsDouble(scale);
            if (PyErr_Occurred())
                throw Raised{};
        }
    }
    void allocate(Place& on, const at::Tensor& q)
    {
        if (!out) {
            made_out = on.empty(shape, at::kBFloat16);
            out = &made_out;
        }
        if (want_lse && !lse) {
            made_lse = on.empty(q.sizes().slice(0, 2), at::kFloat);
            lse = &made_lse;
        }
        c.out = out->data_ptr();
        c.lse = lse ? lse->data_ptr<float>() : nullptr;
    }
    PyObject* result()
    {
        Ref o(made_out.defined() ? THPVariable_Wrap(made_out) : Py_NewRef(out_o));
        Ref l(made_lse.defined() ? THPVariable_Wrap(made_lse) : Py_NewRef(lse ? lse_o : Py_None));
        if (!o.get() || !l.get())
            throw Raised{};
        return PyTuple_Pack(2, o.get(), l.get());
    }
};

// attend_shared(pool_k, pool_v, q, page_size, group_start, prefix_pages, prefix_len, pages, lens, max_group,
//               max_prefix, max_len, scale, out, lse, err, stream, workspace)
PyObject* attend_shared(PyObject*, PyObject* const* a, Py_ssize_t n_args)
{
    return guarded([&]() -> PyObject* {
        count(n_args, 18);
        const at::Tensor &pk = tensor(a[0], "pool_k"), &pv = tensor(a[1], "pool_v"), &q = tensor(a[2], "q");
        KameraPagedKV kv = paged_kv(pk, &pv, a[3]);
        check_q(q, kv.head_dim);
        const at::Tensor *gs = optional(a[4], "group_start"), *pp = optional(a[5], "prefix_pages"),
                         *pl = optional(a[6], "prefix_len"), *pages = optional(a[7], "pages"),
                         *lens = optional(a[8], "lens"), *err = optional(a[15], "err"),
                         *ws = optional(a[17], "workspace");
        KameraPageTable own = page_table(pages, lens, q.size(0), integer(a[11], "max_len"));
        if ((gs == nullptr) != (pp == nullptr) || (gs == nullptr) != (pl == nullptr) || (pp && pp->dim() != 2))
            value_error("group_start, prefix_pages and prefix_len go together");
        KameraPrefixGroups pre;
        std::memset(&pre, 0, sizeof(pre));
        if (gs) {
            const int64_t groups = pp->size(0);
            exact(*gs, "group_start", at::kInt, {groups + 1});
            exact(*pp, "prefix_pages", at::kInt, {groups, pp->size(1)});
            exact(*pl, "prefix_len", at::kInt, {groups});
            pre.group_start = gs->data_ptr<int32_t>();
            pre.pages = pp->data_ptr<int32_t>();
            pre.lens = pl->data_ptr<int32_t>();
            pre.n_groups = size32(groups, "prefix_pages");
            pre.max_pages = size32(pp->size(1), "prefix_pages");
            pre.max_group = int32(a[9], "max_group");
            pre.max_len = int32(a[10], "max_prefix");
        }
        QueryArg qq(q, a[12], a[13], a[14]);
        Place on("kamera_attend_shared", q);
        on.check(q, "q");
        on.check(pk, "pool_k");
        on.check(pv, "pool_v");
        on.check(gs, "group_start");
        on.check(pp, "prefix_pages");
        on.check(pl, "prefix_len");
        on.check(pages, "pages");
        on.check(lens, "lens");
        on.check(qq.out, "out");
        on.check(qq.lse, "lse");
        on.check(err, "err");
        on.check(ws, "workspace");
        int32_t* e = error_word(err);
        on.enter(a[16]);
        qq.allocate(on, q);
        const KameraPrefixGroups* p = gs ? &pre : nullptr;
        Scratch s(on, ws, ws ? 0 : kamera_attend_shared_workspace_bytes(&kv, &qq.c, p, &own));
        status(kamera_attend_shared(&kv, &qq.c, p, &own, s.p, s.bytes, e, on.stream()), "kamera_attend_shared");
        return qq.result();
    });
}

// attend_selected(pool_k, pool_v, q, page_size, pages, lens, selected, max_len, scale, out, lse, err, stream, workspace)
PyObject* attend_selected(PyObject*, PyObject* const* a, Py_ssize_t n_args)
{
    return guarded([&]() -> PyObject* {
        count(n_args, 14);
        const at::Tensor &pk = tensor(a[0], "pool_k"), &pv = tensor(a[1], "pool_v"), &q = tensor(a[2], "q");
        KameraPagedKV kv = paged_kv(pk, &pv, a[3]);
        check_q(q, kv.head_dim);
        const at::Tensor *pages = optional(a[4], "pages"), *lens = optional(a[5], "lens"), *err = optional(a[11], "err"),
                         *ws = optional(a[13], "workspace");
        const at::Tensor& sel = tensor(a[6], "selected");
        KameraPageTable t = page_table(pages, lens, q.size(0), integer(a[7], "max_len"));
        if (sel.dim() != 3)
            value_error("selected must be [S, H, k]");
        exact(sel, "selected", at::kInt, {q.size(0), (int64_t)kv.num_kv_heads, sel.size(2)});
        QueryArg qq(q, a[8], a[9], a[10]);
        Place on("kamera_attend_selected", q);
        on.check(q, "q");
        on.check(pk, "pool_k");
        on.check(pv, "pool_v");
        on.check(pages, "pages");
        on.check(lens, "lens");
        on.check(sel, "selected");
        on.check(qq.out, "out");
        on.check(qq.lse, "lse");
        on.check(err, "err");
        on.check(ws, "workspace");
        int32_t* e = error_word(err);
        on.enter(a[12]);
        qq.allocate(on, q);
        const int32_t k = size32(sel.size(2), "selected");
        Scratch s(on, ws, ws ? 0 : kamera_attend_selected_workspace_bytes(&kv, &qq.c, &t, k));
        status(kamera_attend_selected(&kv, &qq.c, &t, sel.data_ptr<int32_t>(), k, s.p, s.bytes, e, on.stream()),
               "kamera_attend_selected");
        return qq.result();
    });
}

// --------------------------------------------------------------- selection --
// summarize_pages(pool_k, page_size, page_ids, page_tokens, summary, err, stream)
PyObject* summarize_pages(PyObject*, PyObject* const* a, Py_ssize_t n_args)
{
    return guarded([&]() -> PyObject* {
        count(n_args, 7);
        const at::Tensor &pk = tensor(a[0], "pool_k"), &ids = tensor(a[2], "page_ids"),
                         &tokens = tensor(a[3], "page_tokens"), &summary = tensor(a[4], "summary");
        KameraPagedKV kv = paged_kv(pk, nullptr, a[1]);
        if (kv.page_size < 1)
            value_error("page_size must be positive");
        bf16(summary, "summary");
        exact(summary, "summary", at::kBFloat16,
              {kv.num_slots / kv.page_size, (int64_t)kv.num_kv_heads, 2, (int64_t)kv.head_dim});
        const int64_t n = ids.numel();
        exact(ids, "page_ids", at::kInt, {n});
        exact(tokens, "page_tokens", at::kInt, {n});
        const at::Tensor* err = optional(a[5], "err");
        Place on("kamera_summarize_pages", pk);
        on.check(pk, "pool_k");
        on.check(ids, "page_ids");
        on.check(tokens, "page_tokens");
        on.check(summary, "summary");
        on.check(err, "err");
        int32_t* e = error_word(err);
        on.enter(a[6]);
        status(kamera_summarize_pages(&kv, ids.data_ptr<int32_t>(), tokens.data_ptr<int32_t>(), size32(n, "page_ids"),
                                      summary.data_ptr(), e, on.stream()),
               "kamera_summarize_pages");
        return Py_NewRef(a[4]);
    });
}

// select_pages(q, summary, page_size, pages, lens, max_len, n_select, n_first, n_last, selected, err, stream, workspace)
PyObject* select_pages(PyObject*, PyObject* const* a, Py_ssize_t n_args)
{
    return guarded([&]() -> PyObject* {
        count(n_args, 13);
        const at::Tensor &q = tensor(a[0], "q"), &summary = tensor(a[1], "summary");
        bf16(summary, "summary");
        if (summary.dim() != 4 || summary.size(2) != 2 || !summary.is_contiguous())
            value_error("summary must be a contiguous [n_pages, H, 2, d] tensor");
        const int64_t H = summary.size(1), d = summary.size(3);
        check_q(q, d);
        const at::Tensor *pages = optional(a[3], "pages"), *lens = optional(a[4], "lens"),
                         *given = optional(a[9], "selected"), *err = optional(a[10], "err"),
                         *ws = optional(a[12], "workspace");
        KameraPageTable t = page_table(pages, lens, q.size(0), integer(a[5], "max_len"));
        KameraPageSelect x;
        std::memset(&x, 0, sizeof(x));
        x.n_select = int32(a[6], "n_select");
        if (x.n_select < 0)
            value_error("n_select must not be negative");
        if (given)
            exact(*given, "selected", at::kInt, {q.size(0), H, (int64_t)x.n_select});
        Place on("kamera_select_pages", q);
        on.check(q, "q");
        on.check(summary, "summary");
        on.check(pages, "pages");
        on.check(lens, "lens");
        on.check(given, "selected");
        on.check(err, "err");
        on.check(ws, "workspace");
        int32_t* e = error_word(err);
        on.enter(a[11]);
        at::Tensor made;
        if (!given)
            made = on.empty({q.size(0), H, (int64_t)x.n_select}, at::kInt);
        x.q = q.data_ptr();
        x.summary = summary.data_ptr();
        x.selected = (given ? *given : made).data_ptr<int32_t>();
        x.num_pages = summary.size(0);
        x.n_seqs = size32(q.size(0), "q");
        x.num_q_heads = size32(q.size(1), "q");
        x.num_kv_heads = size32(H, "summary");
        x.head_dim = size32(d, "summary");
        x.page_size = int32(a[2], "page_size");
        x.n_first = int32(a[7], "n_first");
        x.n_last = int32(a[8], "n_last");
        Scratch s(on, ws, ws ? 0 : kamera_select_pages_workspace_bytes(&x, &t));
        status(kamera_select_pages(&x, &t, s.p, s.bytes, e, on.stream()), "kamera_select_pages");
        return given ? Py_NewRef(a[9]) : THPVariable_Wrap(made);
    });
}

// -------------------------------------------------------- latent attention --
// One layer of the paged MLA pool; the row splits after kv_lora columns.
KameraPagedMlaKV paged_mla(const at::Tensor& p, PyObject* kv_lora, PyObject* page_size)
{
    bf16(p, "pool");
    if (p.dim() != 2 || (p.size(1) > 1 && p.stride(1) != 1))
        value_error("pool must be [S, kv_lora + rope_dim] (one layer) with packed rows");
    KameraPagedMlaKV kv;
    std::memset(&kv, 0, sizeof(kv));
    kv.kv = p.data_ptr();
    kv.num_slots = p.size(0);
    kv.slot_stride = p.size(0) > 1 ? p.stride(0) : p.size(1);
    kv.kv_lora_rank = int32(kv_lora, "kv_lora");
    kv.rope_dim = size32(p.size(1) - kv.kv_lora_rank, "pool");
    kv.page_size = page_size ? int32(page_size, "page_size") : 0;
    return kv;
}

// mla_attend_paged(pool, kv_lora, q, page_size, pages, lens, max_len, scale, out, lse, err, stream, workspace)
PyObject* mla_attend_paged(PyObject*, PyObject* const* a, Py_ssize_t n_args)
{
    return guarded([&]() -> PyObject* {
        count(n_args, 13);
        const at::Tensor &p = tensor(a[0], "pool"), &q = tensor(a[2], "q");
        KameraPagedMlaKV kv = paged_mla(p, a[1], a[3]);
        check_q(q, p.size(1));
        const at::Tensor *pages = optional(a[4], "pages"), *lens = optional(a[5], "lens"), *err = optional(a[10], "err"),
                         *ws = optional(a[12], "workspace");
        if (!pages || !lens)
            value_error("pages and lens are needed");
        KameraPageTable t = page_table(pages, lens, q.size(0), integer(a[6], "max_len"));
        QueryArg qq(q, a[7], a[8], a[9], kv.kv_lora_rank < 0 ? 0 : kv.kv_lora_rank);
        Place on("kamera_mla_attend_paged", q);
        on.check(q, "q");
        on.check(p, "pool");
        on.check(pages, "pages");
        on.check(lens, "lens");
        on.check(qq.out, "out");
        on.check(qq.lse, "lse");
        on.check(err, "err");
        on.check(ws, "workspace");
        int32_t* e = error_word(err);
        on.enter(a[11]);
        qq.allocate(on, q);
        Scratch s(on, ws, ws ? 0 : kamera_mla_attend_paged_workspace_bytes(&kv, &qq.c, &t));
        status(kamera_mla_attend_paged(&kv, &qq.c, &t, s.p, s.bytes, e, on.stream()), "kamera_mla_attend_paged");
        return qq.result();
    });
}

// mla_expand(pool, kv_lora, weight, slots, kv, k_rope, err, stream)
PyObject* mla_expand(PyObject*, PyObject* const* a, Py_ssize_t n_args)
{
    return guarded([&]() -> PyObject* {
        count(n_args, 8);
        const at::Tensor &p = tensor(a[0], "pool"), &w = tensor(a[2], "weight"), &slots = tensor(a[3], "slots");
        KameraPagedMlaKV pool = paged_mla(p, a[1], nullptr);
        bf16(w, "weight");
        if (w.dim() != 3 || w.size(2) != pool.kv_lora_rank || !w.is_contiguous())
            value_error("weight must be a contiguous [H, head_width, kv_lora] tensor");
        const int64_t T = slots.numel();
        exact(slots, "slots", at::kLong, {T});
        const at::Tensor *kv = optional(a[4], "kv"), *kr = optional(a[5], "k_rope"), *err = optional(a[6], "err");
        const std::array<int64_t, 3> wide{T, w.size(0), w.size(1)};
        const std::array<int64_t, 2> narrow{T, p.size(1) - w.size(2)};
        if (kv)
            exact(*kv, "kv", at::kBFloat16, wide);
        if (kr)
            exact(*kr, "k_rope", at::kBFloat16, narrow);
        Place on("kamera_mla_expand", p);
        on.check(p, "pool");
        on.check(w, "weight");
        on.check(slots, "slots");
        on.check(kv, "kv");
        on.check(kr, "k_rope");
        on.check(err, "err");
        int32_t* e = error_word(err);
        on.enter(a[7]);
        at::Tensor made_kv, made_kr;
        if (!kv) {
            made_kv = on.empty(wide, at::kBFloat16);
            kv = &made_kv;
        }
        if (!kr) {
            made_kr = on.empty(narrow, at::kBFloat16);
            kr = &made_kr;
        }
        KameraMlaExpand x;
        std::memset(&x, 0, sizeof(x));
        x.weight = w.data_ptr();
        x.slots = slots.data_ptr<int64_t>();
        x.kv_out = kv->data_ptr();
        x.k_rope_out = kr->data_ptr();
        x.n_tokens = size32(T, "slots");
        x.num_heads = size32(w.size(0), "weight");
        x.head_width = size32(w.size(1), "weight");
        status(kamera_mla_expand(&pool, &x, e, on.stream()), "kamera_mla_expand");
        Ref o(made_kv.defined() ? THPVariable_Wrap(made_kv) : Py_NewRef(a[4]));
        Ref r(made_kr.defined() ? THPVariable_Wrap(made_kr) : Py_NewRef(a[5]));
        if (!o.get() || !r.get())
            throw Raised{};
        return PyTuple_Pack(2, o.get(), r.get());
    });
}

// mla_prefill_attend(q, kv, k_rope, q_start, kv_start, max_q, causal, scale, out, lse, err, stream)
PyObject* mla_prefill_attend(PyObject*, PyObject* const* a, Py_ssize_t n_args)
{
    return guarded([&]() -> PyObject* {
        count(n_args, 12);
        const at::Tensor &q = tensor(a[0], "q"), &kv = tensor(a[1], "kv"), &kr = tensor(a[2], "k_rope"),
                         &qs = tensor(a[3], "q_start"), &ks = tensor(a[4], "kv_start");
        bf16(q, "q");
        bf16(kv, "kv");
        bf16(kr, "k_rope");
        if (q.dim() != 3 || (q.size(2) > 1 && q.stride(2) != 1))
            value_error("q must be [T, H, nope + rope] with packed rows");
        if (kv.dim() != 3 || kv.size(1) != q.size(1) || !packed(kv))
            value_error("kv must be [R, H, nope + v] with packed heads, the heads of q");
        if (kr.dim() != 2 || kr.size(0) != kv.size(0) || kr.size(1) > q.size(2) || (kr.size(1) > 1 && kr.stride(1) != 1))
            value_error("k_rope must be [R, rope] with packed rows, the rows of kv");
        const int64_t n = qs.numel() - 1, nope = q.size(2) - kr.size(1), v = kv.size(2) - nope;
        if (n < 0 || v < 0)
            value_error(n < 0 ? "q_start must hold n + 1 values" : "kv is narrower than the keys' no-position part");
        exact(qs, "q_start", at::kInt, {n + 1});
        exact(ks, "kv_start", at::kInt, {n + 1});
        const at::Tensor *out = optional(a[8], "out"), *lse = nullptr, *err = optional(a[10], "err");
        const bool want_lse = a[9] != Py_False;
        if (want_lse)
            lse = optional(a[9], "lse");
        const std::array<int64_t, 3> shape{q.size(0), q.size(1), v};
        const std::array<int64_t, 2> rows{q.size(0), q.size(1)};
        if (out)
            exact(*out, "out", at::kBFloat16, shape);
        if (lse)
            exact(*lse, "lse", at::kFloat, rows);
        KameraMlaPrefill x;
        std::memset(&x, 0, sizeof(x));
        x.max_q = int32(a[5], "max_q");
        const int causal = PyObject_IsTrue(a[6]);
        if (causal < 0)
            throw Raised{};
        x.causal = causal;
        if (a[7] == Py_None) {
            x.scale = (float)(1.0 / std::sqrt((double)q.size(2)));
        } else {
            x.scale = (float)PyFloat_AsDouble(a[7]);
            if (PyErr_Occurred())
                throw Raised{};
        }
        Place on("kamera_mla_prefill_attend", q);
        on.check(q, "q");
        on.check(kv, "kv");
        on.check(kr, "k_rope");
        on.check(qs, "q_start");
        on.check(ks, "kv_start");
        on.check(out, "out");
        on.check(lse, "lse");
        on.check(err, "err");
        int32_t* e = error_word(err);
        on.enter(a[11]);
        at::Tensor made_out, made_lse;
        if (!out) {
            made_out = on.empty(shape, at::kBFloat16);
            out = &made_out;
        }
        if (want_lse && !lse) {
            made_lse = on.empty(rows, at::kFloat);
            lse = &made_lse;
        }
        x.q = q.data_ptr();
        x.kv = kv.data_ptr();
        x.k_rope = kr.data_ptr();
        x.out = out->data_ptr();
        x.lse = lse ? lse->data_ptr<float>() : nullptr;
        x.q_start = qs.data_ptr<int32_t>();
        x.kv_start = ks.data_ptr<int32_t>();
        x.q_stride = step(q, 0);
        x.q_head_stride = step(q, 1);
        x.kv_stride = step(kv, 0);
        x.k_rope_stride = step(kr, 0);
        x.n_q = size32(q.size(0), "q");
        x.n_kv = size32(kv.size(0), "kv");
        x.n_seqs = size32(n, "q_start");
        x.num_heads = size32(q.size(1), "q");
        x.nope_dim = size32(nope, "q");
        x.rope_dim = size32(kr.size(1), "k_rope");
        x.v_dim = size32(v, "kv");
        status(kamera_mla_prefill_attend(&x, e, on.stream()), "kamera_mla_prefill_attend");
        Ref o(made_out.defined() ? THPVariable_Wrap(made_out) : Py_NewRef(a[8]));
        Ref l(made_lse.defined() ? THPVariable_Wrap(made_lse) : Py_NewRef(lse ? a[9] : Py_None));
        if (!o.get() || !l.get())
            throw Raised{};
        return PyTuple_Pack(2, o.get(), l.get());
    });
}

// ------------------------------------------------------------ pages in 4 bits --
KameraPackedPool packed_pool(const at::Tensor& t, int64_t d, PyObject* page_size, PyObject* k_unit, PyObject* v_unit)
{
    KameraPackedPool p;
    std::memset(&p, 0, sizeof(p));
    p.page_size = int32(page_size, "page_size");
    p.head_dim = size32(d, "head_dim");
    if (t.scalar_type() != at::kByte || t.dim() != 3 || !t.is_contiguous() || p.page_size < 1 ||
        t.size(2) != (int64_t)p.page_size * (d + d / 8))
        value_error("packed must be a contiguous uint8 [n_pages, H, page_size * (d + d / 8)] tensor");
    p.data = t.data_ptr();
    p.num_pages = t.size(0);
    p.num_kv_heads = size32(t.size(1), "packed");
    p.k_unit = (float)PyFloat_AsDouble(k_unit);
    p.v_unit = (float)PyFloat_AsDouble(v_unit);
    if (PyErr_Occurred())
        throw Raised{};
    return p;
}

// pages(pool_k, pool_v, page_size, kv_pages, tokens, packed, packed_pages, k_unit, v_unit, err, stream): what packing and
// unpacking share
PyObject* convert_pages(PyObject* const* a, Py_ssize_t n_args, bool pack)
{
    return guarded([&]() -> PyObject* {
        count(n_args, 11);
        const char* where = pack ? "kamera_pack_pages" : "kamera_unpack_pages";
        const at::Tensor &pk = tensor(a[0], "pool_k"), &pv = tensor(a[1], "pool_v"), &kp = tensor(a[3], "kv_pages"),
                         &tokens = tensor(a[4], "page_tokens"), &packed = tensor(a[5], "packed"),
                         &pp = tensor(a[6], "packed_pages");
        const at::Tensor* err = optional(a[9], "err");
        const KameraPagedKV kv = paged_kv(pk, &pv, a[2]);
        const KameraPackedPool pool = packed_pool(packed, kv.head_dim, a[2], a[7], a[8]);
        const int64_t n = kp.numel();
        exact(kp, "the bf16 pages", at::kInt, {n});
        exact(pp, "the packed pages", at::kInt, {n});
        exact(tokens, "page_tokens", at::kInt, {n});
        Place on(where, pk);
        on.check(pk, "pool_k");
        on.check(pv, "pool_v");
        on.check(kp, "the bf16 pages");
        on.check(pp, "the packed pages");
        on.check(tokens, "page_tokens");
        on.check(packed, "packed");
        on.check(err, "err");
        KameraGqaPool g;
        std::memset(&g, 0, sizeof(g));
        g.num_layers = 1;
        g.num_kv_heads = kv.num_kv_heads;
        g.head_dim = kv.head_dim;
        g.k = pk.data_ptr();
        g.v = pv.data_ptr();
        g.num_slots = kv.num_slots;
        g.slot_stride = kv.num_slots > 1 ? kv.slot_stride : (int64_t)kv.num_kv_heads * kv.head_dim;
        int32_t* e = error_word(err);
        on.enter(a[10]);
        status((pack ? kamera_pack_pages : kamera_unpack_pages)(&g, 0, &pool, kp.data_ptr<int32_t>(), pp.data_ptr<int32_t>(),
                                                                tokens.data_ptr<int32_t>(), size32(n, "the pages"), e,
                                                                on.stream()),
               where);
        return Py_NewRef(Py_None);
    });
}
PyObject* pack_pages(PyObject*, PyObject* const* a, Py_ssize_t n) { return convert_pages(a, n, true); }
PyObject* unpack_pages(PyObject*, PyObject* const* a, Py_ssize_t n) { return convert_pages(a, n, false); }

// attend_packed(packed, q, page_size, pages, lens, max_len, pool_k, pool_v, tail_pages, tail_lens, max_tail, tail_page_size,
//               k_unit, v_unit, scale, out, lse, err, stream, workspace)
PyObject* attend_packed(PyObject*, PyObject* const* a, Py_ssize_t n_args)
{
    return guarded([&]() -> PyObject* {
        count(n_args, 20);
        const at::Tensor &packed = tensor(a[0], "packed"), &q = tensor(a[1], "q");
        if (q.dim() != 3)
            value_error("q must be a contiguous [S, H_q, d] tensor");
        const KameraPackedPool pool = packed_pool(packed, q.size(2), a[2], a[12], a[13]);
        check_q(q, pool.head_dim);
        const at::Tensor *pages = optional(a[3], "pages"), *lens = optional(a[4], "lens"), *pk = optional(a[6], "pool_k"),
                         *pv = optional(a[7], "pool_v"), *tp = optional(a[8], "tail_pages"),
                         *tl = optional(a[9], "tail_lens"), *err = optional(a[17], "err"), *ws = optional(a[19], "workspace");
        KameraPageTable t = page_table(pages, lens, q.size(0), integer(a[5], "max_len"));
        KameraPagedKV kv;
        KameraPageTable tail;
        const bool some = pk || pv || tp || tl;
        if (some) {
            if (!pk || !pv || !tp || !tl)
                value_error("pool_k, pool_v, tail_pages and tail_lens go together");
            kv = paged_kv(*pk, pv, a[11] == Py_None ? a[2] : a[11]);
            if (kv.num_kv_heads != pool.num_kv_heads || kv.head_dim != pool.head_dim)
                value_error("pool_k must have the packed pool's heads and width");
            tail = page_table(tp, tl, q.size(0), integer(a[10], "max_tail"));
        }
        QueryArg qq(q, a[14], a[15], a[16]);
        Place on("kamera_attend_packed", q);
        on.check(q, "q");
        on.check(packed, "packed");
        on.check(pages, "pages");
        on.check(lens, "lens");
        on.check(pk, "pool_k");
        on.check(pv, "pool_v");
        on.check(tp, "tail_pages");
        on.check(tl, "tail_lens");
        on.check(qq.out, "out");
        on.check(qq.lse, "lse");
        on.check(err, "err");
        on.check(ws, "workspace");
        int32_t* e = error_word(err);
        on.enter(a[18]);
        qq.allocate(on, q);
        const KameraPagedKV* k = some ? &kv : nullptr;
        const KameraPageTable* tt = some ? &tail : nullptr;
        Scratch s(on, ws, ws ? 0 : kamera_attend_packed_workspace_bytes(&pool, &qq.c, &t, k, tt));
        status(kamera_attend_packed(&pool, &qq.c, &t, k, tt, s.p, s.bytes, e, on.stream()), "kamera_attend_packed");
        return qq.result();
    });
}

// A version check for the loader.
PyObject* abi_version(PyObject*, PyObject*) { return PyLong_FromLong(kamera_abi_version()); }

#define FAST(name) {#name, (PyCFunction)(void (*)(void))name, METH_FASTCALL, nullptr}
PyMethodDef methods[] = {FAST(append_kv),       FAST(mla_append_kv), FAST(attend_shared),
                         FAST(attend_selected), FAST(summarize_pages), FAST(select_pages),
                         FAST(mla_attend_paged), FAST(mla_expand), FAST(mla_prefill_attend), FAST(pack_pages),
                         FAST(unpack_pages), FAST(attend_packed),
                         {"abi_version", abi_version, METH_NOARGS, nullptr}, {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_kamera_binding", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__kamera_binding(void) { return PyModule_Create(&module); }
