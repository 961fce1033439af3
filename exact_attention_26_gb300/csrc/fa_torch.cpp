// The tensor front end of the paged-cache calls as a CPython extension.
//
// A decode step makes these calls once per layer, on kernels that take a few microseconds; the
// checks, allocations and argument marshalling of the Python wrappers take longer than that
// (27 us for a decode, 20 us for a store of one token per sequence, 75 us for a fork on a
// Grace core).  Here they are a few hundred nanoseconds.  Each function takes what the wrapper
// of the same name takes, checks it, allocates the outputs and makes the C call.  It returns
// the outputs, an int for a status other than FA_OK, or None when some argument is not as
// expected; the Python wrapper then says what is wrong with it.
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <ATen/core/Tensor.h>
#include <ATen/cuda/EmptyTensor.h>
#include <c10/cuda/CUDACachingAllocator.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <cmath>
#include <optional>

#include "fa.h"

namespace {

using at::Tensor;

// Exact torch.Tensor on a CUDA device, contiguous, of this type; null otherwise.
const Tensor *tensor(PyObject *o, at::ScalarType type, int dim) {
    if (!THPVariable_CheckExact(o)) return nullptr;
    const Tensor &t = THPVariable_Unpack(o);
    if (!t.is_cuda() || t.scalar_type() != type || t.dim() != dim || !t.is_contiguous()) return nullptr;
    return &t;
}

bool on(const Tensor *t, int device) { return t && t->get_device() == device; }

bool shaped(const Tensor &t, std::initializer_list<int64_t> sizes) {
    return t.sizes().equals(at::IntArrayRef(sizes));
}

bool is_int(int64_t v) { return v >= 0 && v <= INT32_MAX; }

Tensor make(std::initializer_list<int64_t> sizes, at::ScalarType type, int device) {
    return Tensor(at::detail::empty_cuda(at::IntArrayRef(sizes), type,
                                         c10::Device(c10::kCUDA, (c10::DeviceIndex)device), std::nullopt));
}

// int32 outputs of one call as parts of one allocation (each allocation is most of a
// microsecond): a buffer, and tensors over its elements in turn.
struct Parts {
    Tensor buffer;
    int64_t used = 0;
    Parts(int64_t elements, int device) : buffer(make({elements}, at::kInt, device)) {}
    Tensor take(std::initializer_list<int64_t> sizes) {
        Tensor t = at::detail::make_tensor<c10::TensorImpl>(c10::Storage(buffer.storage()), buffer.key_set(),
                                                            buffer.dtype());
        t.unsafeGetTensorImpl()->set_sizes_contiguous(at::IntArrayRef(sizes));
        t.unsafeGetTensorImpl()->set_storage_offset(used);
        used += t.numel();
        return t;
    }
};

PyObject *declined() { Py_RETURN_NONE; }

// The stream of a call on `device`: argument `o`, None for the device's current stream or the
// handle of another, which is current while this lives.  So what the call allocates belongs to
// the stream that its kernels run on, and scratch that is released on return is handed out
// again only behind them.
class CallStream {
   public:
    void *raw = nullptr;

    bool read(PyObject *o, int device) {
        const c10::cuda::CUDAStream current = c10::cuda::getCurrentCUDAStream((c10::DeviceIndex)device);
        raw = current.stream();
        if (o == Py_None) return true;
        raw = PyLong_AsVoidPtr(o);
        if (PyErr_Occurred()) return false;
        if (raw != current.stream()) {
            caller_ = current;
            guard_.emplace(c10::cuda::getStreamFromExternal(static_cast<cudaStream_t>(raw),
                                                            (c10::DeviceIndex)device));
        }
        return true;
    }

    // `t`, allocated by the call, goes to a caller who works on another stream: its memory is
    // kept, once released, until what that stream holds by then is done too.
    void hand_out(const Tensor &t) const {
        if (caller_) c10::cuda::CUDACachingAllocator::recordStream(t.storage().data_ptr(), *caller_);
    }

   private:
    std::optional<c10::cuda::CUDAStream> caller_;
    std::optional<c10::cuda::CUDAStreamGuard> guard_;
};

template <typename T>
T *ptr(const Tensor &t) {
    return static_cast<T *>(t.data_ptr());
}

// A paged e4m3 cache and its table.
struct Cache {
    const Tensor *kc, *vc, *ks, *vs, *bt, *lens;
    int B, num_pages, Hkv, page_size, d, max_pages, group;

    bool read(PyObject *const *a, int device) {
        kc = tensor(a[0], at::kByte, 4);
        vc = tensor(a[1], at::kByte, 4);
        ks = tensor(a[2], at::kFloat, 3);
        vs = tensor(a[3], at::kFloat, 3);
        bt = tensor(a[4], at::kInt, 2);
        lens = tensor(a[5], at::kInt, 1);
        if (!on(kc, device) || !on(vc, device) || !on(ks, device) || !on(vs, device) || !on(bt, device) ||
            !on(lens, device))
            return false;
        for (int64_t s : kc->sizes())
            if (s < 1 || !is_int(s)) return false;
        const int64_t groups = ks->size(2);
        if (!vc->sizes().equals(kc->sizes()) || !vs->sizes().equals(ks->sizes()) || groups < 1 ||
            ks->size(0) != kc->size(0) || ks->size(1) != kc->size(1) || kc->size(2) % groups)
            return false;
        if (!is_int(bt->size(0)) || !is_int(bt->size(1)) || bt->size(1) < 1 || lens->size(0) != bt->size(0))
            return false;
        num_pages = (int)kc->size(0);
        Hkv = (int)kc->size(1);
        page_size = (int)kc->size(2);
        d = (int)kc->size(3);
        B = (int)bt->size(0);
        max_pages = (int)bt->size(1);
        group = (int)(kc->size(2) / groups);
        return true;
    }
};

// q, k_cache, v_cache, k_scale, v_scale, block_table, seq_lens, causal, scale, out, lse,
// workspace, stream
PyObject *decode_paged_fp8(PyObject *, PyObject *const *a, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    if (n != 13) return declined();
    const Tensor *q = tensor(a[0], at::kBFloat16, 4);
    if (!q) return declined();
    const int device = q->get_device();
    Cache c;
    if (!c.read(a + 1, device)) return declined();
    const int64_t B = q->size(0), H = q->size(1), Nq = q->size(2);
    if (B != c.B || q->size(3) != c.d || H % c.Hkv || !is_int(H) || !is_int(Nq)) return declined();
    const int causal = PyObject_IsTrue(a[7]);
    if (causal < 0) return nullptr;
    double scale = 1.0 / std::sqrt((double)c.d);
    if (a[8] != Py_None) {
        scale = PyFloat_AsDouble(a[8]);
        if (PyErr_Occurred()) return nullptr;
    }
    const c10::cuda::CUDAGuard guard((c10::DeviceIndex)device);
    CallStream stream;
    if (!stream.read(a[12], device)) return nullptr;
    Tensor out, lse, ws;
    if (a[9] == Py_None) {
        out = make({B, H, Nq, c.d}, at::kBFloat16, device);
        stream.hand_out(out);
    } else {
        const Tensor *t = tensor(a[9], at::kBFloat16, 4);
        if (!on(t, device) || !t->sizes().equals(q->sizes())) return declined();
        out = *t;
    }
    if (a[10] == Py_None) {
        lse = make({B, H, Nq}, at::kFloat, device);
        stream.hand_out(lse);
    } else {
        const Tensor *t = tensor(a[10], at::kFloat, 3);
        if (!on(t, device) || !shaped(*t, {B, H, Nq})) return declined();
        lse = *t;
    }
    if (a[11] == Py_None) {
        const size_t need = fa_decode_paged_fp8_workspace_bytes((int)B, (int)H, c.Hkv, (int)Nq, c.d,
                                                                c.page_size, c.max_pages);
        ws = make({(int64_t)need}, at::kByte, device);
    } else {
        const Tensor *t = THPVariable_CheckExact(a[11]) ? &THPVariable_Unpack(a[11]) : nullptr;
        if (!t || !t->is_cuda() || t->scalar_type() != at::kByte || !t->is_contiguous() || !on(t, device))
            return declined();
        ws = *t;
    }
    const int rc = fa_decode_paged_fp8(
        q->data_ptr(), c.kc->data_ptr(), c.vc->data_ptr(), ptr<float>(*c.ks), ptr<float>(*c.vs),
        ptr<int>(*c.bt), ptr<int>(*c.lens), out.data_ptr(), ptr<float>(lse), (int)B, (int)H, c.Hkv, (int)Nq,
        c.d, c.page_size, c.max_pages, c.num_pages, c.group, causal, (float)scale, ws.data_ptr(),
        (size_t)ws.numel(), stream.raw);
    if (rc != FA_OK) return PyLong_FromLong(rc);
    PyObject *po = a[9] == Py_None ? THPVariable_Wrap(out) : Py_NewRef(a[9]);
    PyObject *pl = a[10] == Py_None ? THPVariable_Wrap(lse) : Py_NewRef(a[10]);
    PyObject *r = po && pl ? PyTuple_Pack(2, po, pl) : nullptr;
    Py_XDECREF(po);
    Py_XDECREF(pl);
    return r;
    END_HANDLE_TH_ERRORS
}

// New rows [T, Hkv, d] at any row stride; -1 if they are not that.
long long row_stride(const Tensor &t, const Cache &c) {
    if (!t.is_cuda() || t.scalar_type() != at::kBFloat16 || t.dim() != 3 || t.size(0) < 1 || !is_int(t.size(0)) ||
        t.size(1) != c.Hkv || t.size(2) != c.d || t.stride(2) != 1 || (c.Hkv > 1 && t.stride(1) != c.d))
        return -1;
    const long long row = (long long)c.Hkv * c.d;
    return t.size(0) > 1 ? t.stride(0) : (t.stride(0) > row ? t.stride(0) : row);
}

// k, v, k_cache, v_cache, k_scale, v_scale, block_table, seq_lens, cu_seqlens, stream.  Returns
// the status.
PyObject *append_paged_fp8(PyObject *, PyObject *const *a, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    if (n != 10 || !THPVariable_CheckExact(a[0]) || !THPVariable_CheckExact(a[1])) return declined();
    const Tensor &k = THPVariable_Unpack(a[0]), &v = THPVariable_Unpack(a[1]);
    if (!k.is_cuda() || !v.is_cuda() || v.get_device() != k.get_device()) return declined();
    const int device = k.get_device();
    Cache c;
    if (!c.read(a + 2, device)) return declined();
    const long long ks = row_stride(k, c), vs = row_stride(v, c);
    if (ks < 0 || vs < 0 || v.size(0) != k.size(0)) return declined();
    const int *cu = nullptr;
    if (a[8] != Py_None) {
        const Tensor *t = tensor(a[8], at::kInt, 1);
        if (!on(t, device) || t->size(0) != (int64_t)c.B + 1) return declined();
        cu = ptr<int>(*t);
    } else if (k.size(0) != c.B) {
        return declined();
    }
    const c10::cuda::CUDAGuard guard((c10::DeviceIndex)device);
    CallStream stream;
    if (!stream.read(a[9], device)) return nullptr;
    return PyLong_FromLong(fa_append_paged_fp8(
        k.data_ptr(), v.data_ptr(), c.kc->data_ptr(), c.vc->data_ptr(), ptr<float>(*c.ks), ptr<float>(*c.vs),
        ptr<int>(*c.bt), ptr<int>(*c.lens), cu, c.B, (int)k.size(0), c.Hkv, c.d, c.page_size, c.max_pages,
        c.num_pages, c.group, ks, vs, stream.raw));
    END_HANDLE_TH_ERRORS
}

// A block table and its lengths, and two host integers.
struct Table {
    const Tensor *bt, *lens;
    int device, B, max_pages, page_size, num_pages;

    bool read(PyObject *table, PyObject *lengths, PyObject *page, PyObject *num) {
        bt = tensor(table, at::kInt, 2);
        lens = tensor(lengths, at::kInt, 1);
        if (!bt || !on(lens, device = bt->get_device()) || lens->size(0) != bt->size(0)) return false;
        if (!is_int(bt->size(0)) || !is_int(bt->size(1)) || !PyLong_Check(page) || !PyLong_Check(num)) return false;
        int over = 0, over2 = 0;
        const long p = PyLong_AsLongAndOverflow(page, &over), m = PyLong_AsLongAndOverflow(num, &over2);
        if (over || over2 || !is_int(p) || !is_int(m)) return false;
        B = (int)bt->size(0);
        max_pages = (int)bt->size(1);
        page_size = (int)p;
        num_pages = (int)m;
        return true;
    }
};

PyObject *results(std::initializer_list<Tensor> ts) {
    PyObject *r = PyTuple_New((Py_ssize_t)ts.size());
    if (!r) return nullptr;
    Py_ssize_t i = 0;
    for (const Tensor &t : ts) {
        PyObject *o = THPVariable_Wrap(t);
        if (!o) {
            Py_DECREF(r);
            return nullptr;
        }
        PyTuple_SET_ITEM(r, i++, o);
    }
    return r;
}

// block_table, seq_lens, page_size, num_pages, stream
PyObject *free_pages(PyObject *, PyObject *const *a, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    Table t;
    if (n != 5 || !t.read(a[0], a[1], a[2], a[3])) return declined();
    const c10::cuda::CUDAGuard guard((c10::DeviceIndex)t.device);
    CallStream stream;
    if (!stream.read(a[4], t.device)) return nullptr;
    Parts parts((int64_t)t.num_pages + 1, t.device);
    stream.hand_out(parts.buffer);
    const Tensor pages = parts.take({t.num_pages}), count = parts.take({1});
    const int rc = fa_free_pages(ptr<int>(*t.bt), ptr<int>(*t.lens), ptr<int>(pages), ptr<int>(count), t.B,
                                 t.max_pages, t.page_size, t.num_pages, stream.raw);
    return rc != FA_OK ? PyLong_FromLong(rc) : results({pages, count});
    END_HANDLE_TH_ERRORS
}

// block_table, seq_lens, parents, fresh, page_size, num_pages, stream
PyObject *fork_pages(PyObject *, PyObject *const *a, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    Table t;
    if (n != 7 || !t.read(a[0], a[1], a[4], a[5])) return declined();
    const Tensor *parents = tensor(a[2], at::kInt, 1), *fresh = tensor(a[3], at::kInt, 1);
    if (!on(parents, t.device) || !on(fresh, t.device) || fresh->size(0) != parents->size(0) ||
        !is_int(parents->size(0)))
        return declined();
    const c10::cuda::CUDAGuard guard((c10::DeviceIndex)t.device);
    CallStream stream;
    if (!stream.read(a[6], t.device)) return nullptr;
    const int64_t m = parents->size(0);
    Parts parts(m * t.max_pages + 3 * m, t.device);
    stream.hand_out(parts.buffer);
    const Tensor rows = parts.take({m, t.max_pages}), lens = parts.take({m});
    const Tensor src = parts.take({m}), dst = parts.take({m});
    const int rc = fa_fork_pages(ptr<int>(*t.bt), ptr<int>(*t.lens), ptr<int>(*parents), ptr<int>(*fresh),
                                 ptr<int>(rows), ptr<int>(lens), ptr<int>(src), ptr<int>(dst), t.B, (int)m,
                                 t.max_pages, t.page_size, t.num_pages, stream.raw);
    return rc != FA_OK ? PyLong_FromLong(rc) : results({rows, lens, src, dst});
    END_HANDLE_TH_ERRORS
}

// block_table, seq_lens, page_size, num_pages, stream
PyObject *compact_pages(PyObject *, PyObject *const *a, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    Table t;
    if (n != 5 || !t.read(a[0], a[1], a[2], a[3])) return declined();
    const c10::cuda::CUDAGuard guard((c10::DeviceIndex)t.device);
    CallStream stream;
    if (!stream.read(a[4], t.device)) return nullptr;
    const int64_t cap = t.num_pages / 2 > 1 ? t.num_pages / 2 : 1;
    Parts parts((int64_t)t.B * t.max_pages + 2 * cap + 2, t.device);
    stream.hand_out(parts.buffer);
    const Tensor table = parts.take({t.B, t.max_pages}), src = parts.take({cap});
    const Tensor dst = parts.take({cap}), counts = parts.take({2});
    const int rc = fa_compact_pages(ptr<int>(*t.bt), ptr<int>(*t.lens), ptr<int>(table), ptr<int>(src),
                                    ptr<int>(dst), ptr<int>(counts), t.B, t.max_pages, t.page_size,
                                    t.num_pages, stream.raw);
    return rc != FA_OK ? PyLong_FromLong(rc) : results({table, src, dst, counts});
    END_HANDLE_TH_ERRORS
}

// caches (a list), src, dst, count, stream.  Returns the status.
PyObject *copy_pages(PyObject *, PyObject *const *a, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    if (n != 5 || !PyList_Check(a[0])) return declined();
    const Py_ssize_t m = PyList_GET_SIZE(a[0]);
    const Tensor *src = tensor(a[1], at::kInt, 1), *dst = tensor(a[2], at::kInt, 1);
    if (m < 1 || m > FA_MAX_COPY_CACHES || !src) return declined();
    const int device = src->get_device();
    if (!on(dst, device) || dst->size(0) != src->size(0) || !is_int(src->size(0))) return declined();
    const int *count = nullptr;
    if (a[3] != Py_None) {
        const Tensor *t = tensor(a[3], at::kInt, 1);
        if (!on(t, device) || t->size(0) != 1) return declined();
        count = ptr<int>(*t);
    }
    void *caches[FA_MAX_COPY_CACHES];
    size_t bytes[FA_MAX_COPY_CACHES];
    int64_t num_pages = 0;
    for (Py_ssize_t i = 0; i < m; ++i) {
        PyObject *o = PyList_GET_ITEM(a[0], i);
        if (!THPVariable_CheckExact(o)) return declined();
        const Tensor &t = THPVariable_Unpack(o);
        if (!t.is_cuda() || t.get_device() != device || !t.is_contiguous() || t.dim() < 2 || t.numel() == 0)
            return declined();
        if (i == 0) num_pages = t.size(0);
        if (t.size(0) != num_pages || !is_int(num_pages)) return declined();
        caches[i] = t.data_ptr();
        bytes[i] = t.nbytes() / (size_t)num_pages;
    }
    const c10::cuda::CUDAGuard guard((c10::DeviceIndex)device);
    CallStream stream;
    if (!stream.read(a[4], device)) return nullptr;
    return PyLong_FromLong(fa_copy_pages(caches, bytes, (int)m, (int)num_pages, ptr<int>(*src), ptr<int>(*dst),
                                         (int)src->size(0), count, stream.raw));
    END_HANDLE_TH_ERRORS
}

#define FN(name) {#name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(name)), METH_FASTCALL, nullptr}
PyMethodDef kMethods[] = {FN(decode_paged_fp8), FN(append_paged_fp8), FN(free_pages), FN(fork_pages),
                          FN(compact_pages), FN(copy_pages), {nullptr, nullptr, 0, nullptr}};
PyModuleDef kModule = {PyModuleDef_HEAD_INIT, "_fa_torch", nullptr, -1, kMethods, nullptr, nullptr, nullptr,
                       nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__fa_torch() { return PyModule_Create(&kModule); }
