// The host side of the tree-speculation calls, compiled: argument checks, output
// allocation and the call into libpa for arguments that are all in order.
//
// These kernels run for 2 to 20 microseconds, and the same steps take 10 to 20 in
// Python.  Each function here takes its Python namesake's arguments in order and
// answers NotImplemented, having done nothing, as soon as anything is not plainly
// right (a wrong type, device, shape or layout, another current device, a workspace
// that has yet to be allocated, arguments that the library refuses); the Python
// function then goes through its own checks and says what is wrong.  PA_ERR_CUDA may
// come after a launch, and moving rows or rotating queries twice is not the same as
// once: it is raised from here.
#include <Python.h>

#include <ATen/core/TensorBody.h>
#include <ATen/ops/empty.h>
#include <ATen/ops/empty_like.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAGraphsC10Utils.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include <exception>

#include "../../include/pa.h"

namespace {

PyObject* declined() {
    PyErr_Clear();                       // an int too large for a long
    Py_RETURN_NOTIMPLEMENTED;
}

PyObject* check_status = nullptr;        // Python's check(status, call), which raises the package's error

// A call that the library did not take.
PyObject* refused(pa_status st, const char* call) {
    if (st != PA_ERR_CUDA) return declined();                    // before any launch
    if (check_status) Py_XDECREF(PyObject_CallFunction(check_status, "is", (int)st, call));
    if (!PyErr_Occurred()) PyErr_Format(PyExc_RuntimeError, "%s: %s", call, pa_status_string(st));
    return nullptr;
}

PyObject* on_failure(PyObject*, PyObject* const* a, Py_ssize_t n) {
    if (n != 1) return declined();
    Py_XSETREF(check_status, Py_NewRef(a[0]));
    Py_RETURN_NONE;
}

// The tensor behind `o` if it is contiguous, of type `t` and on device `dev`; else null.
const at::Tensor* tensor(PyObject* o, at::ScalarType t, int dev) {
    if (!THPVariable_Check(o)) return nullptr;
    const at::Tensor& x = THPVariable_Unpack(o);
    return x.is_cuda() && x.get_device() == dev && x.scalar_type() == t && x.is_contiguous() ? &x : nullptr;
}

// An optional argument: false if it is there and not as tensor() wants it.
bool optional(PyObject* o, at::ScalarType t, int dev, const at::Tensor*& out) {
    out = nullptr;
    return o == Py_None || (out = tensor(o, t, dev)) != nullptr;
}

// The device of the argument that the others have to share, if it is the current one; else -1.
int device_of(PyObject* o) {
    if (!THPVariable_Check(o)) return -1;
    const at::Tensor& x = THPVariable_Unpack(o);
    return x.is_cuda() && x.get_device() == c10::cuda::current_device() ? (int)x.get_device() : -1;
}

bool is_shape(const at::Tensor& t, at::IntArrayRef want) { return t.sizes() == want; }

bool fits_int(int64_t v) { return v >= 0 && v <= 0x7fffffff; }

void* stream_of(int dev) { return c10::cuda::getCurrentCUDAStream((c10::DeviceIndex)dev).stream(); }

template <class T>
T* data(const at::Tensor* t) { return t ? static_cast<T*>(t->data_ptr()) : nullptr; }

// fp16 / bf16 pools [NB, Hkv, B, d] of one type, as a shape; false if they are not that.
bool pool_shape(PyObject* k, PyObject* v, int dev, const at::Tensor*& kt, const at::Tensor*& vt, pa_shape& s) {
    if (!THPVariable_Check(k)) return false;
    const at::ScalarType t = THPVariable_Unpack(k).scalar_type();
    if (t != at::kHalf && t != at::kBFloat16) return false;
    kt = tensor(k, t, dev);
    vt = tensor(v, t, dev);
    if (!kt || !vt || kt->dim() != 4 || kt->sizes() != vt->sizes()) return false;
    const auto z = kt->sizes();
    for (int64_t n : z)
        if (!fits_int(n)) return false;
    s = pa_shape{0, 1, (int32_t)z[1], (int32_t)z[3], (int32_t)z[2], (int32_t)z[0], 1,
                 t == at::kBFloat16 ? PA_BF16 : PA_FP16};
    return true;
}

// A contiguous tensor over part of another's memory, `at` elements of type `t` in.
at::Tensor part(const at::Tensor& whole, at::ScalarType t, at::IntArrayRef sizes, int64_t at) {
    auto impl = c10::make_intrusive<c10::TensorImpl>(c10::Storage(whole.storage()), whole.key_set(),
                                                     c10::scalarTypeToTypeMeta(t));
    impl->set_storage_offset(at);
    impl->set_sizes_contiguous(sizes);
    return at::Tensor(std::move(impl));
}

// Runs `f` and turns a C++ exception (an allocation that failed) into NotImplemented.
template <class F>
PyObject* guarded(F f) {
    try {
        return f();
    } catch (const std::exception&) {
        return declined();
    }
}

// (path, q_start, context_lens, block_tables, k_pool, v_pool, err)
PyObject* keep_kv(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return guarded([&]() -> PyObject* {
        if (n != 7) return declined();
        const int dev = device_of(a[4]);
        const at::Tensor *k, *v, *err;
        pa_shape s;
        if (dev < 0 || !pool_shape(a[4], a[5], dev, k, v, s)) return declined();
        const at::Tensor *path = tensor(a[0], at::kInt, dev), *start = tensor(a[1], at::kInt, dev),
                         *ctx = tensor(a[2], at::kInt, dev), *table = tensor(a[3], at::kInt, dev);
        if (!path || !start || !ctx || !table || !optional(a[6], at::kInt, dev, err)) return declined();
        if (path->dim() != 2 || table->dim() != 2) return declined();
        const int64_t N = path->size(0), P = path->size(1);
        if (!fits_int(N) || P < 1 || P > 64 || !is_shape(*start, {N + 1}) || !is_shape(*ctx, {N}) ||
            table->size(0) != N || !fits_int(table->size(1)))
            return declined();
        s.num_seqs = (int32_t)N;
        s.max_blocks_per_seq = (int32_t)table->size(1);
        const pa_status st =
            pa_keep_kv(&s, (int32_t)P, data<int32_t>(path), data<int32_t>(start), data<int32_t>(table), data<int32_t>(ctx),
                       data<void>(k), data<void>(v), data<uint32_t>(err), stream_of(dev));
        if (st != PA_OK) return refused(st, "pa_keep_kv");
        Py_RETURN_NONE;
    });
}

// (tree_masks, draft_tokens, target_tokens, q_start, context_lens, max_nodes, path, err)
PyObject* tree_verify(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return guarded([&]() -> PyObject* {
        if (n != 8 || !PyLong_Check(a[5])) return declined();
        const int dev = device_of(a[0]);
        if (dev < 0) return declined();
        const at::Tensor *masks = tensor(a[0], at::kLong, dev), *draft = tensor(a[1], at::kLong, dev),
                         *target = tensor(a[2], at::kLong, dev), *start = tensor(a[3], at::kInt, dev),
                         *ctx = tensor(a[4], at::kInt, dev), *given, *err;
        if (!masks || !draft || !target || !start || !ctx || !optional(a[6], at::kInt, dev, given) ||
            !optional(a[7], at::kInt, dev, err))
            return declined();
        const long P = PyLong_AsLong(a[5]);
        if (P < 1 || P > 64 || masks->dim() != 1 || ctx->dim() != 1) return declined();
        const int64_t T = masks->size(0), N = ctx->size(0);
        if (!fits_int(T) || !fits_int(N) || !is_shape(*draft, {T}) || !is_shape(*target, {T}) ||
            !is_shape(*start, {N + 1}) || (given && !is_shape(*given, {N, (int64_t)P})))
            return declined();
        // one allocation for the four answers: next [N] of 8 bytes, then [N], [N], [N, P] of 4
        const at::Tensor room = at::empty({N + (N * (2 + (given ? 0 : P)) + 1) / 2}, masks->options());
        const at::Tensor next = part(room, at::kLong, {N}, 0), accepted = part(room, at::kInt, {N}, 2 * N),
                         lens = part(room, at::kInt, {N}, 3 * N),
                         path = given ? *given : part(room, at::kInt, {N, (int64_t)P}, 4 * N);
        const pa_status st =
            pa_tree_verify((int32_t)N, (int32_t)P, (int32_t)T, data<int32_t>(start), data<uint64_t>(masks),
                           data<int64_t>(draft), data<int64_t>(target), data<int32_t>(ctx), data<int32_t>(&path),
                           data<int32_t>(&accepted), data<int64_t>(&next), data<int32_t>(&lens), data<uint32_t>(err),
                           stream_of(dev));
        if (st != PA_OK) return refused(st, "pa_tree_verify");
        PyObject* r = PyTuple_New(4);
        if (!r) return nullptr;
        PyTuple_SET_ITEM(r, 0, given ? Py_NewRef(a[6]) : THPVariable_Wrap(path));
        PyTuple_SET_ITEM(r, 1, THPVariable_Wrap(accepted));
        PyTuple_SET_ITEM(r, 2, THPVariable_Wrap(next));
        PyTuple_SET_ITEM(r, 3, THPVariable_Wrap(lens));
        for (int i = 0; i < 4; ++i)
            if (!PyTuple_GET_ITEM(r, i)) {
                Py_DECREF(r);
                return (PyObject*)nullptr;
            }
        return r;
    });
}

// (workspaces, q, k_pool, v_pool, block_tables, context_lens, q_start, tree_masks, scale, max_nodes, out, workspace,
// err); workspaces: the dict of kept workspaces by (device, stream)
PyObject* decode_tree(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return guarded([&]() -> PyObject* {
        if (n != 13 || !PyFloat_Check(a[8]) || !PyLong_Check(a[9])) return declined();
        const int dev = device_of(a[1]);
        const at::Tensor *k, *v, *given, *err;
        pa_shape s;
        if (dev < 0 || !pool_shape(a[2], a[3], dev, k, v, s)) return declined();
        const at::Tensor *q = tensor(a[1], k->scalar_type(), dev), *table = tensor(a[4], at::kInt, dev),
                         *ctx = tensor(a[5], at::kInt, dev), *start = tensor(a[6], at::kInt, dev),
                         *masks = tensor(a[7], at::kLong, dev);
        if (!q || !table || !ctx || !start || !masks || !optional(a[10], k->scalar_type(), dev, given) ||
            !optional(a[12], at::kInt, dev, err))
            return declined();
        const long P = PyLong_AsLong(a[9]);
        if (P < 1 || P > 64 || q->dim() != 3 || table->dim() != 2 || q->size(2) != s.head_dim) return declined();
        const int64_t T = q->size(0), N = table->size(0);
        if (!fits_int(T) || !fits_int(N) || !fits_int(q->size(1)) || !fits_int(table->size(1)) ||
            !is_shape(*start, {N + 1}) || !is_shape(*ctx, {N}) || !is_shape(*masks, {T}) ||
            (given && given->sizes() != q->sizes()))
            return declined();
        s.num_seqs = (int32_t)N;
        s.num_q_heads = (int32_t)q->size(1);
        s.max_blocks_per_seq = (int32_t)table->size(1);
        void* stream = stream_of(dev);
        const at::Tensor out = given ? *given : at::empty_like(*q);
        // From here to the end of the call the interpreter lock stays held, so no other thread
        // takes the stream's workspace or queues a call that uses it; while one that runs
        // without the lock uses it, it is not in the dict.
        const at::Tensor* ws = nullptr;
        if (a[11] != Py_None) {
            if (!THPVariable_Check(a[11])) return declined();
            ws = tensor(a[11], THPVariable_Unpack(a[11]).scalar_type(), dev);
        } else if (c10::cuda::currentStreamCaptureStatusMayInitCtx() == c10::cuda::CaptureStatus::None) {
            PyObject* key = Py_BuildValue("(iK)", dev, (unsigned long long)(uintptr_t)stream);
            PyObject* kept = key ? PyDict_GetItem(a[0], key) : nullptr;      // borrowed
            Py_XDECREF(key);
            if (kept) ws = tensor(kept, at::kByte, dev);
            if (ws && ws->nbytes() < pa_decode_tree_workspace_bytes(&s, (int32_t)P)) ws = nullptr;
        }
        if (!ws) return declined();
        const pa_status st =
            pa_decode_tree(&s, (int32_t)P, (int32_t)T, data<void>(q), data<int32_t>(start), data<uint64_t>(masks),
                           data<void>(k), data<void>(v), data<int32_t>(table), data<int32_t>(ctx),
                           (float)PyFloat_AS_DOUBLE(a[8]), data<void>(&out), data<void>(ws), ws->nbytes(),
                           data<uint32_t>(err), stream);
        if (st != PA_OK) return refused(st, "pa_decode_tree");
        return given ? Py_NewRef(a[10]) : THPVariable_Wrap(out);
    });
}

// Elements between the tokens of [T, H, d] with contiguous heads; -1 if it is not that.
int64_t token_stride(PyObject* o, at::ScalarType t, int dev, int64_t T, int64_t H, int64_t d, const at::Tensor*& out) {
    if (!THPVariable_Check(o)) return -1;
    const at::Tensor& x = THPVariable_Unpack(o);
    if (!x.is_cuda() || x.get_device() != dev || x.scalar_type() != t || !is_shape(x, {T, H, d})) return -1;
    out = &x;
    if (T == 0) return H * d;                          // nothing is read
    if (x.stride(2) != 1 || (x.stride(1) != d && H > 1)) return -1;
    if (T == 1) return H * d;                          // a single token's own stride is never used
    return x.stride(0) >= H * d ? x.stride(0) : -1;
}

// (q, k_new, v_new, positions, slot_mapping, k_pool, v_pool, inv_freq, interleaved, rope_scale, q_weight, k_weight,
// eps, out, err)
PyObject* rope_append_kv(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return guarded([&]() -> PyObject* {
        if (n != 15 || !PyBool_Check(a[8]) || !PyFloat_Check(a[9]) || !PyFloat_Check(a[12])) return declined();
        const int dev = device_of(a[5]);
        const at::Tensor *kp, *vp, *q, *k, *v, *freq, *qw, *kw, *given, *err;
        pa_shape s;
        if (dev < 0 || !pool_shape(a[5], a[6], dev, kp, vp, s) || !THPVariable_Check(a[0])) return declined();
        const at::ScalarType t = kp->scalar_type();
        const at::Tensor& q_any = THPVariable_Unpack(a[0]);
        if (q_any.dim() != 3) return declined();
        const int64_t T = q_any.size(0), Hq = q_any.size(1), d = s.head_dim;
        if (!fits_int(T) || !fits_int(Hq)) return declined();
        const int64_t qs = token_stride(a[0], t, dev, T, Hq, d, q),
                      ks = token_stride(a[1], t, dev, T, s.num_kv_heads, d, k),
                      vs = token_stride(a[2], t, dev, T, s.num_kv_heads, d, v);
        const at::Tensor *pos = tensor(a[3], at::kInt, dev), *slots = tensor(a[4], at::kLong, dev);
        if (qs < 0 || ks < 0 || vs < 0 || !pos || !slots || !is_shape(*pos, {T}) || !is_shape(*slots, {T}))
            return declined();
        if (!optional(a[7], at::kFloat, dev, freq) || !optional(a[10], t, dev, qw) || !optional(a[11], t, dev, kw) ||
            !optional(a[13], t, dev, given) || !optional(a[14], at::kInt, dev, err))
            return declined();
        if ((freq && (freq->dim() != 1 || 2 * freq->size(0) > d)) || (qw && !is_shape(*qw, {d})) ||
            (kw && !is_shape(*kw, {d})) || (given && given->sizes() != q->sizes()))
            return declined();
        s.num_q_heads = (int32_t)Hq;
        const int32_t rotary = freq ? (int32_t)(2 * freq->size(0)) : 0;
        const pa_rope rope{rotary ? data<float>(freq) : nullptr, rotary, a[8] == Py_True, (float)PyFloat_AS_DOUBLE(a[9]),
                           (float)PyFloat_AS_DOUBLE(a[12]), data<void>(qw), data<void>(kw)};
        const at::Tensor out = given ? *given : at::empty({T, Hq, d}, q->options());
        const pa_status st =
            pa_rope_append_kv(&s, &rope, (int32_t)T, data<void>(q), qs, data<void>(k), ks, data<void>(v), vs,
                              data<int32_t>(pos), data<int64_t>(slots), data<void>(&out), data<void>(kp),
                              data<void>(vp), data<uint32_t>(err), stream_of(dev));
        if (st != PA_OK) return refused(st, "pa_rope_append_kv");
        return given ? Py_NewRef(a[13]) : THPVariable_Wrap(out);
    });
}

#define METHOD(name) {#name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(&name)), METH_FASTCALL, nullptr}
PyMethodDef methods[] = {METHOD(keep_kv), METHOD(tree_verify), METHOD(decode_tree), METHOD(rope_append_kv),
                         METHOD(on_failure), {nullptr, nullptr, 0, nullptr}};

PyModuleDef module = {PyModuleDef_HEAD_INIT, "_pa_fast", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__pa_fast() { return PyModule_Create(&module); }
