// Native half of the Python binding of the paged-cache calls.
//
// These calls run in serving loops, a few per layer and step, and their kernels
// take a few microseconds, so what checks the tensors, finds the stream, takes
// result and scratch from torch's allocator and calls the C ABI of
// include/spec.h is compiled: a page step costs 6 us of host time through
// ctypes, an attention call 12 to 17.
//
// Every function returns what the C ABI returned, or -1 for arguments that the
// kernels could not read; the Python side then says which and why.
#include <ATen/ops/empty.h>
#include <c10/cuda/CUDACachingAllocator.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <climits>
#include <cmath>

#include "spec.h"

namespace {

constexpr long kBadArgs = -1;

// A tensor argument; null when the object is none.
const at::Tensor* tensor(PyObject* o) { return THPVariable_Check(o) ? &THPVariable_Unpack(o) : nullptr; }

bool on(const at::Tensor& t, int dev, at::ScalarType type) {
    return t.is_cuda() && t.get_device() == dev && t.scalar_type() == type;
}

// A contiguous int32 tensor of at least `need` entries.
bool int32(const at::Tensor* t, int dev, int64_t need) {
    return t && on(*t, dev, at::kInt) && t->is_contiguous() && t->numel() >= need && t->numel() <= INT_MAX;
}

// A pool [pages][kv heads][SPEC_PAGE][head_dim].
bool pool(const at::Tensor* t, int dev) {
    return t && on(*t, dev, at::kBFloat16) && t->dim() == 4 && t->size(2) == SPEC_PAGE && t->is_contiguous() &&
           t->size(0) <= INT_MAX && t->size(1) <= INT_MAX;
}

// Rows [rows][heads][head_dim], each contiguous, any distance apart (a stride
// over a dimension of size one is not looked at).
bool rows(const at::Tensor* t, int dev, int64_t n, int64_t heads, int64_t hd, int64_t* stride) {
    if (!t || !on(*t, dev, at::kBFloat16) || t->dim() != 3 || t->size(0) != n || t->size(1) != heads || t->size(2) != hd ||
        n > INT_MAX)
        return false;
    if ((t->stride(2) != 1 && hd > 1) || (t->stride(1) != hd && heads > 1)) return false;
    *stride = n > 1 ? t->stride(0) : heads * hd;
    return true;
}

// Device of a tensor when it is the current one, else -1.
int current(const at::Tensor* t) {
    if (!t || !t->is_cuda()) return -1;
    const int dev = t->get_device();
    return dev == c10::cuda::current_device() ? dev : -1;
}

int32_t* i32(const at::Tensor* t) { return static_cast<int32_t*>(t->data_ptr()); }

PyObject* status(long s) { return PyLong_FromLong(s); }

// pages_step(pool, tables, len, keep, add, row_start, slots)
PyObject* pages_step(PyObject*, PyObject* const* a, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    const at::Tensor* t[7];
    if (n != 7) return status(kBadArgs);
    for (int i = 0; i < 7; ++i) t[i] = tensor(a[i]);
    const int dev = current(t[0]);
    if (dev < 0 || !int32(t[0], dev, SPEC_POOL_HEADER + 1) || !int32(t[1], dev, 0) || t[1]->dim() != 2) return status(kBadArgs);
    const int64_t nseq = t[1]->size(0);
    if (!int32(t[2], dev, nseq) || !int32(t[3], dev, nseq) || !int32(t[4], dev, nseq) || !int32(t[5], dev, nseq + 1) ||
        !int32(t[6], dev, 0))
        return status(kBadArgs);
    return status(spec_pages_step(i32(t[0]), (int32_t)(t[0]->numel() - SPEC_POOL_HEADER), i32(t[1]), (int32_t)t[1]->size(1),
                                  i32(t[2]), i32(t[3]), i32(t[4]), (int32_t)nseq, i32(t[5]), i32(t[6]),
                                  (int32_t)t[6]->numel(), c10::cuda::getCurrentCUDAStream(dev).stream()));
    END_HANDLE_TH_ERRORS
}

// paged_append(k, v, slots, row_count or None, kpool, vpool, error or None)
PyObject* paged_append(PyObject*, PyObject* const* a, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    if (n != 7) return status(kBadArgs);
    const at::Tensor *k = tensor(a[0]), *v = tensor(a[1]), *slots = tensor(a[2]), *kp = tensor(a[4]), *vp = tensor(a[5]);
    const at::Tensor *count = a[3] == Py_None ? nullptr : tensor(a[3]), *err = a[6] == Py_None ? nullptr : tensor(a[6]);
    const int dev = current(k);
    if (dev < 0 || !pool(kp, dev) || !pool(vp, dev) || kp->sizes() != vp->sizes() || k->dim() != 3) return status(kBadArgs);
    int64_t ks, vs;
    if (!rows(k, dev, k->size(0), kp->size(1), kp->size(3), &ks) || !rows(v, dev, k->size(0), kp->size(1), kp->size(3), &vs) ||
        !int32(slots, dev, k->size(0)) || (a[3] != Py_None && !int32(count, dev, 1)) || (a[6] != Py_None && !int32(err, dev, 1)))
        return status(kBadArgs);
    return status(spec_paged_append(k->data_ptr(), ks, v->data_ptr(), vs, i32(slots), count ? i32(count) : nullptr,
                                    (int32_t)k->size(0), (int32_t)kp->size(1), (int32_t)kp->size(3), kp->data_ptr(),
                                    vp->data_ptr(), (int32_t)kp->size(0), err ? i32(err) : nullptr,
                                    c10::cuda::getCurrentCUDAStream(dev).stream()));
    END_HANDLE_TH_ERRORS
}

// Scratch from torch's allocator, given back in the stream's order as a tensor would be.
struct Scratch {
    void* p = nullptr;
    Scratch(size_t bytes, cudaStream_t s) {
        if (bytes) p = c10::cuda::CUDACachingAllocator::raw_alloc_with_stream(bytes, s);
    }
    ~Scratch() {
        if (p) c10::cuda::CUDACachingAllocator::raw_delete(p);
    }
};

// paged_attention(q, row_start, len, tables, kpool, vpool, max_new, scale or
// None, out or None, error or None, work or None): the output tensor, or a status
PyObject* paged_attention(PyObject*, PyObject* const* a, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    if (n != 11) return status(kBadArgs);
    const at::Tensor *q = tensor(a[0]), *start = tensor(a[1]), *len = tensor(a[2]), *tables = tensor(a[3]), *kp = tensor(a[4]),
                     *vp = tensor(a[5]);
    const at::Tensor *out = a[8] == Py_None ? nullptr : tensor(a[8]), *err = a[9] == Py_None ? nullptr : tensor(a[9]),
                     *work = a[10] == Py_None ? nullptr : tensor(a[10]);
    const int dev = current(q);
    if (dev < 0 || !pool(kp, dev) || !pool(vp, dev) || kp->sizes() != vp->sizes() || q->dim() != 3 || !int32(tables, dev, 0) ||
        tables->dim() != 2 || q->size(1) > INT_MAX)
        return status(kBadArgs);
    const int64_t nrows = q->size(0), hq = q->size(1), hkv = kp->size(1), hd = kp->size(3), nseq = tables->size(0);
    int64_t qs, os = hq * hd;
    if (!rows(q, dev, nrows, hq, hd, &qs) || !int32(start, dev, nseq + 1) || !int32(len, dev, nseq) ||
        (a[8] != Py_None && !rows(out, dev, nrows, hq, hd, &os)) || (a[9] != Py_None && !int32(err, dev, 1)) ||
        (a[10] != Py_None && !(work && on(*work, dev, at::kByte) && work->is_contiguous())))
        return status(kBadArgs);
    int overflow = 0;
    const long long asked = PyLong_AsLongLongAndOverflow(a[6], &overflow);
    if (asked == -1 && PyErr_Occurred()) return nullptr;
    const int32_t max_new = overflow > 0 || asked > INT_MAX ? INT_MAX : overflow < 0 || asked < 0 ? 0 : (int32_t)asked;
    const double scale = a[7] == Py_None ? 1.0 / std::sqrt((double)hd) : PyFloat_AsDouble(a[7]);
    if (scale == -1.0 && PyErr_Occurred()) return nullptr;
    cudaStream_t s = c10::cuda::getCurrentCUDAStream(dev).stream();
    size_t bytes = 0;
    if (work) {
        bytes = work->nbytes();
    } else {
        const spec_status st = spec_paged_attention_workspace((int32_t)hq, (int32_t)hkv, (int32_t)hd, max_new,
                                                              (int32_t)tables->size(1), &bytes);
        if (st != SPEC_OK) return status(st);
    }
    const Scratch scratch(work ? 0 : bytes, s);
    at::Tensor result;
    if (!out) result = at::empty({nrows, hq, hd}, q->options());
    const spec_status st = spec_paged_attention(
        q->data_ptr(), qs, i32(start), i32(len), i32(tables), (int32_t)tables->size(1), (int32_t)nseq, (int32_t)nrows, max_new,
        (int32_t)hq, (int32_t)hkv, (int32_t)hd, (float)scale, kp->data_ptr(), vp->data_ptr(), (int32_t)kp->size(0),
        out ? out->data_ptr() : result.data_ptr(), os, err ? i32(err) : nullptr, work ? work->data_ptr() : scratch.p, bytes, s);
    if (st != SPEC_OK) return status(st);
    if (out) {
        Py_INCREF(a[8]);
        return a[8];
    }
    return THPVariable_Wrap(std::move(result));
    END_HANDLE_TH_ERRORS
}

PyMethodDef methods[] = {
    {"pages_step", reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(pages_step)), METH_FASTCALL, nullptr},
    {"paged_append", reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(paged_append)), METH_FASTCALL, nullptr},
    {"paged_attention", reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(paged_attention)), METH_FASTCALL, nullptr},
    {nullptr, nullptr, 0, nullptr}};

PyModuleDef module = {PyModuleDef_HEAD_INIT, "_paged", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__paged() { return PyModule_Create(&module); }
