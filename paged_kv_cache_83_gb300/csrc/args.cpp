// args.cpp: argument checks and marshalling of the calls that a step or a sampled token repeats
// (pa_rope_store_kv, pa_chunk_attn, pa_sample), as an extension module of the binding.
//
// The kernel of a decode step's rotation takes 2 us. Its eleven tensors checked in Python and 27 arguments passed
// through ctypes made the call 10.4 us (4 tokens) and 11.1 us (256 tokens), back to back; checked here it is 4.1 us for
// both. A draft's attention of two launches went from 12.5 to 8.9 us, where its kernels
// bound it.
// Each function takes the tensors and settings of the binding's function of the same name, all of them and
// in that order, raises TypeError or ValueError for what does not fit, and returns the entry point's status.
// The entry points are those of the loaded library: bind() takes their addresses. No C++ exception leaves
// a function.
#include <torch/csrc/autograd/python_variable.h>

#include <c10/core/DeviceGuard.h>

#include <cstdint>
#include <exception>

#include "../../include/pa.h"

namespace {

decltype(&::pa_rope_store_kv) call_rope_store_kv = nullptr;
decltype(&::pa_chunk_attn) call_chunk_attn = nullptr;
decltype(&::pa_sample) call_sample = nullptr;

struct Refused {  // a Python exception has been set
};

[[noreturn]] void refuse(PyObject *type, const char *what) {
    PyErr_SetString(type, what);
    throw Refused{};
}

template <class F>
void bound(F entry) {
    if (!entry) refuse(PyExc_RuntimeError, "the library is not loaded");
}

const at::Tensor &tensor(PyObject *o, const char *what) {
    if (!THPVariable_Check(o)) refuse(PyExc_TypeError, what);
    return THPVariable_Unpack(o);
}

// The call's device: every tensor that is given has to be on one CUDA device.
struct Device {
    int index = -1;
    bool first = true;
    void add(const at::Tensor &t) {
        const int i = t.is_cuda() ? static_cast<int>(t.get_device()) : -1;
        if (first)
            index = i, first = false;
        else if (i != index)
            refuse(PyExc_ValueError, "tensors must be on one CUDA device");
    }
    void check() const {
        if (index < 0) refuse(PyExc_ValueError, "tensors must be on a CUDA device");
    }
};

const void *contiguous(const at::Tensor &t) {
    if (!t.is_contiguous()) refuse(PyExc_ValueError, "tensors must be contiguous");
    return t.data_ptr();
}

void int32(const at::Tensor &t, const char *what) {
    if (t.scalar_type() != at::kInt) refuse(PyExc_TypeError, what);
}

pa_dtype dtype_of(const at::Tensor &t) {
    if (t.scalar_type() == at::kHalf) return PA_F16;
    if (t.scalar_type() == at::kBFloat16) return PA_BF16;
    refuse(PyExc_TypeError, "unsupported dtype (of 16 bits: float16 or bfloat16)");
}

// an optional tensor of `dev`, int32
int32_t *error_word(PyObject *o, Device &dev) {
    if (o == Py_None) return nullptr;
    const at::Tensor &t = tensor(o, "err must be a tensor");
    int32(t, "err must be int32");
    dev.add(t);
    return const_cast<int32_t *>(static_cast<const int32_t *>(contiguous(t)));
}

// the elements between tokens of a [T, H, D] tensor whose tokens may lie apart
int64_t token_stride(const at::Tensor &t, int64_t T, int64_t H, int64_t D, const char *what) {
    const auto s = t.strides();
    if (s[2] != 1 || (s[1] != D && H > 1)) refuse(PyExc_ValueError, what);
    return T > 1 ? s[0] : H * D;
}

int small(int64_t v) {  // a size as the C interface takes it
    if (v > INT32_MAX) refuse(PyExc_ValueError, "a size is beyond 2^31 - 1");
    return static_cast<int>(v);
}

int number(PyObject *o, const char *what) {
    const long long v = PyLong_AsLongLong(o);
    if (v == -1 && PyErr_Occurred()) throw Refused{};
    if (v < 0 || v > INT32_MAX) refuse(PyExc_ValueError, what);
    return static_cast<int>(v);
}

PyObject *current_raw_stream = nullptr;  // torch._C._cuda_getCurrentRawStream

// the given stream (an object with cuda_stream, or a number), or the current one of `dev`
cudaStream_t stream_of(PyObject *o, int dev) {
    PyObject *v;
    if (o == Py_None) {
        if (!current_raw_stream) {
            PyObject *m = PyImport_ImportModule("torch._C");
            if (!m) throw Refused{};
            current_raw_stream = PyObject_GetAttrString(m, "_cuda_getCurrentRawStream");
            Py_DECREF(m);
            if (!current_raw_stream) throw Refused{};
        }
        PyObject *d = PyLong_FromLong(dev);
        v = d ? PyObject_CallOneArg(current_raw_stream, d) : nullptr;
        Py_XDECREF(d);
    } else if (PyIndex_Check(o)) {
        v = PyNumber_Index(o);
    } else {
        v = PyObject_GetAttrString(o, "cuda_stream");
    }
    if (!v) throw Refused{};
    const unsigned long long raw = PyLong_AsUnsignedLongLong(v);
    Py_DECREF(v);
    if (PyErr_Occurred()) throw Refused{};
    return reinterpret_cast<cudaStream_t>(raw);
}

// the status of call(), made with `dev` current and without the interpreter's lock
template <class F>
PyObject *run(int dev, F call) {
    const c10::DeviceGuard guard(c10::Device(c10::kCUDA, static_cast<c10::DeviceIndex>(dev)));
    pa_status status;
    Py_BEGIN_ALLOW_THREADS;
    status = call();
    Py_END_ALLOW_THREADS;
    return PyLong_FromLong(status);
}

template <class F>
PyObject *guarded(Py_ssize_t given, Py_ssize_t wanted, F body) {
    try {
        if (given != wanted) refuse(PyExc_TypeError, "wrong number of arguments");
        return body();
    } catch (const Refused &) {
    } catch (const std::exception &e) {
        PyErr_SetString(PyExc_RuntimeError, e.what());
    }
    return nullptr;
}

// q_out, q, k, v, k_cache, v_cache, slot_mapping, positions, cos_sin, pair_axis, interleaved, err, stream
PyObject *rope_store_kv(PyObject *, PyObject *const *a, Py_ssize_t n) {
    return guarded(n, 13, [&] {
        bound(call_rope_store_kv);
        const at::Tensor &q_out = tensor(a[0], "q_out must be a tensor"), &q = tensor(a[1], "q must be a tensor"),
                         &k = tensor(a[2], "k must be a tensor"), &v = tensor(a[3], "v must be a tensor"),
                         &kc = tensor(a[4], "k_cache must be a tensor"), &vc = tensor(a[5], "v_cache must be a tensor"),
                         &slots = tensor(a[6], "slot_mapping must be a tensor"),
                         &pos = tensor(a[7], "positions must be a tensor"), &tab = tensor(a[8], "cos_sin must be a tensor");
        if (kc.dim() != 4 || q.dim() != 3 || k.dim() != 3) refuse(PyExc_ValueError, "shape mismatch");
        const int64_t NB = kc.size(0), bs = kc.size(1), Hkv = kc.size(2), D = kc.size(3), T = q.size(0), Hq = q.size(1);
        if (q.size(2) != D || q_out.sizes() != q.sizes() || k.size(0) != T || k.size(1) != Hkv || k.size(2) != D ||
            v.sizes() != k.sizes() || vc.sizes() != kc.sizes())
            refuse(PyExc_ValueError, "shape mismatch");
        if (slots.dim() != 1 || slots.size(0) != T) refuse(PyExc_ValueError, "slot_mapping must be [T]");
        if (pos.dim() < 1 || pos.dim() > 2 || pos.size(-1) != T)
            refuse(PyExc_ValueError, "positions must be [T] or [axes, T]");
        if (tab.scalar_type() != at::kFloat || tab.dim() != 2)
            refuse(PyExc_TypeError, "cos_sin must be a float32 [max_pos, rot_dim] table");
        const int64_t rot = tab.size(1);
        const uint8_t *pairs = nullptr;
        if (a[9] != Py_None) {
            if (!PyBytes_CheckExact(a[9]) || PyBytes_GET_SIZE(a[9]) != rot / 2)
                refuse(PyExc_ValueError, "pair_axis must be rot_dim / 2 bytes");
            pairs = reinterpret_cast<const uint8_t *>(PyBytes_AS_STRING(a[9]));
        }
        const int interleaved = PyObject_IsTrue(a[10]);
        if (interleaved < 0) throw Refused{};
        const pa_dtype dt = dtype_of(kc);
        const auto type = kc.scalar_type();
        if (q.scalar_type() != type || q_out.scalar_type() != type || k.scalar_type() != type || v.scalar_type() != type ||
            vc.scalar_type() != type)
            refuse(PyExc_TypeError, "q, q_out, k, v and the pools must share a dtype");
        int32(slots, "slot_mapping must be int32");
        int32(pos, "positions must be int32");
        Device dev;
        for (const at::Tensor *t : {&q, &q_out, &k, &v, &kc, &vc, &slots, &pos, &tab}) dev.add(*t);
        int32_t *err = error_word(a[11], dev);
        dev.check();
        const int64_t sqo = token_stride(q_out, T, Hq, D, "q_out: the heads of a token must be contiguous"), sq = token_stride(q, T, Hq, D, "q: the heads of a token must be contiguous"),
                      sk = token_stride(k, T, Hkv, D, "k: the heads of a token must be contiguous"), sv = token_stride(v, T, Hkv, D, "v: the heads of a token must be contiguous");
        const void *kcp = contiguous(kc), *vcp = contiguous(vc), *sp = contiguous(slots), *pp = contiguous(pos),
                   *tp = contiguous(tab);
        const cudaStream_t stream = stream_of(a[12], dev.index);
        const int axes = pos.dim() == 1 ? 1 : small(pos.size(0)), max_pos = small(tab.size(0)), Ti = small(T), NBi = small(NB),
                  bsi = small(bs), Hqi = small(Hq), Hkvi = small(Hkv), Di = small(D), roti = small(rot);
        return run(dev.index, [&] {
            return call_rope_store_kv(q_out.data_ptr(), sqo, q.data_ptr(), sq, k.data_ptr(), sk, v.data_ptr(), sv,
                                    const_cast<void *>(kcp), const_cast<void *>(vcp), static_cast<const int32_t *>(sp),
                                    static_cast<const int32_t *>(pp), axes, pairs, static_cast<const float *>(tp), max_pos,
                                    roti, interleaved, Ti, NBi, bsi, Hqi, Hkvi, Di, dt, err, stream);
        });
    });
}

// out, q, k_cache, v_cache, block_tables, cu_seqlens_q, context_lens, max_seqlen_q, scale, window, workspace, err, stream
PyObject *chunk_attn(PyObject *, PyObject *const *a, Py_ssize_t n) {
    return guarded(n, 13, [&] {
        bound(call_chunk_attn);
        const at::Tensor &out = tensor(a[0], "out must be a tensor"), &q = tensor(a[1], "q must be a tensor"),
                         &kc = tensor(a[2], "k_cache must be a tensor"), &vc = tensor(a[3], "v_cache must be a tensor"),
                         &bt = tensor(a[4], "block_tables must be a tensor"), &cu = tensor(a[5], "cu_seqlens_q must be a tensor"),
                         &ctx = tensor(a[6], "context_lens must be a tensor");
        if (kc.dim() != 4 || q.dim() != 3 || bt.dim() != 2 || ctx.dim() != 1 || cu.dim() != 1)
            refuse(PyExc_ValueError, "shape mismatch");
        const int64_t NB = kc.size(0), bs = kc.size(1), Hkv = kc.size(2), D = kc.size(3), Tq = q.size(0), Hq = q.size(1),
                      S = ctx.size(0);
        if (q.size(2) != D || out.sizes() != q.sizes() || vc.sizes() != kc.sizes() || bt.size(0) != S || cu.size(0) != S + 1)
            refuse(PyExc_ValueError, "shape mismatch");
        const pa_dtype dt = dtype_of(q);
        const auto type = q.scalar_type();
        if (out.scalar_type() != type || kc.scalar_type() != type || vc.scalar_type() != type)
            refuse(PyExc_TypeError, "q, out and the pools must share a dtype");
        int32(bt, "block_tables must be int32");
        int32(cu, "cu_seqlens_q must be int32");
        int32(ctx, "context_lens must be int32");
        const int max_q = number(a[7], "max_seqlen_q must be from 0 to 2^31 - 1");
        const double scale = PyFloat_AsDouble(a[8]);
        if (scale == -1.0 && PyErr_Occurred()) throw Refused{};
        const int window = number(a[9], "window must be from 0 to 2^31 - 1");
        Device dev;
        for (const at::Tensor *t : {&q, &out, &kc, &vc, &bt, &cu, &ctx}) dev.add(*t);
        void *ws = nullptr;
        size_t ws_bytes = 0;
        if (a[10] != Py_None) {
            const at::Tensor &w = tensor(a[10], "workspace must be a tensor");
            dev.add(w);
            ws = const_cast<void *>(contiguous(w));
            ws_bytes = static_cast<size_t>(w.numel()) * w.element_size();
        }
        int32_t *err = error_word(a[11], dev);
        dev.check();
        const void *op = contiguous(out), *qp = contiguous(q), *kcp = contiguous(kc), *vcp = contiguous(vc),
                   *btp = contiguous(bt), *cup = contiguous(cu), *cxp = contiguous(ctx);
        const cudaStream_t stream = stream_of(a[12], dev.index);
        const int maxb = small(bt.size(1)), Si = small(S), Tqi = small(Tq), Hqi = small(Hq), Hkvi = small(Hkv), Di = small(D),
                  bsi = small(bs), NBi = small(NB);
        return run(dev.index, [&] {
            return call_chunk_attn(const_cast<void *>(op), qp, kcp, vcp, static_cast<const int32_t *>(btp), maxb,
                                 static_cast<const int32_t *>(cup), static_cast<const int32_t *>(cxp), Si, Tqi, max_q, window,
                                 Hqi, Hkvi, Di, bsi, NBi, static_cast<float>(scale), dt, ws, ws_bytes, err, stream);
        });
    });
}

// tokens, logits, u, temperature, top_k, top_p, min_p, err, stream
PyObject *sample(PyObject *, PyObject *const *a, Py_ssize_t n) {
    return guarded(n, 9, [&] {
        bound(call_sample);
        const at::Tensor &tokens = tensor(a[0], "tokens must be a tensor"), &logits = tensor(a[1], "logits must be a tensor");
        if (logits.dim() != 2) refuse(PyExc_ValueError, "logits must be [B, V]");
        const int64_t B = logits.size(0), V = logits.size(1);
        if (tokens.dim() != 1 || tokens.size(0) != B) refuse(PyExc_ValueError, "tokens must be [B]");
        const pa_dtype dt = logits.scalar_type() == at::kFloat ? PA_F32 : dtype_of(logits);
        int32(tokens, "tokens must be int32");
        Device dev;
        dev.add(logits);
        dev.add(tokens);
        const void *rows[5];
        static const char *const names[5] = {"u must be float32 [B]", "temperature must be float32 [B]", "top_k must be int32 [B]",
                                             "top_p must be float32 [B]", "min_p must be float32 [B]"};
        for (int i = 0; i < 5; ++i) {
            rows[i] = nullptr;
            if (a[2 + i] == Py_None) continue;
            const at::Tensor &t = tensor(a[2 + i], names[i]);
            if (t.scalar_type() != (i == 2 ? at::kInt : at::kFloat) || t.dim() != 1 || t.size(0) != B)
                refuse(PyExc_TypeError, names[i]);
            dev.add(t);
            rows[i] = contiguous(t);
        }
        int32_t *err = error_word(a[7], dev);
        dev.check();
        if (logits.stride(1) != 1 && V > 1) refuse(PyExc_ValueError, "a row of logits must be contiguous");
        const int64_t stride = B > 1 ? logits.stride(0) : V;
        const void *tp = contiguous(tokens);
        const cudaStream_t stream = stream_of(a[8], dev.index);
        const int Bi = small(B), Vi = small(V);
        return run(dev.index, [&] {
            return call_sample(static_cast<int32_t *>(const_cast<void *>(tp)), logits.data_ptr(), stride, Bi, Vi, dt,
                             static_cast<const float *>(rows[0]), static_cast<const float *>(rows[1]),
                             static_cast<const int32_t *>(rows[2]), static_cast<const float *>(rows[3]),
                             static_cast<const float *>(rows[4]), err, stream);
        });
    });
}

// bind(addresses of pa_rope_store_kv, pa_chunk_attn, pa_sample)
PyObject *bind(PyObject *, PyObject *const *a, Py_ssize_t n) {
    return guarded(n, 3, [&]() -> PyObject * {
        uintptr_t at[3];
        for (int i = 0; i < 3; ++i) {
            at[i] = static_cast<uintptr_t>(PyLong_AsUnsignedLongLong(a[i]));
            if (PyErr_Occurred()) throw Refused{};
            if (!at[i]) refuse(PyExc_ValueError, "an entry point has no address");
        }
        call_rope_store_kv = reinterpret_cast<decltype(call_rope_store_kv)>(at[0]);
        call_chunk_attn = reinterpret_cast<decltype(call_chunk_attn)>(at[1]);
        call_sample = reinterpret_cast<decltype(call_sample)>(at[2]);
        Py_RETURN_NONE;
    });
}

template <class F>
PyCFunction fast(F *f) {
    return reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(f));
}

PyMethodDef methods[] = {{"bind", fast(bind), METH_FASTCALL, nullptr},
                         {"pa_rope_store_kv", fast(rope_store_kv), METH_FASTCALL, nullptr},
                         {"pa_chunk_attn", fast(chunk_attn), METH_FASTCALL, nullptr},
                         {"pa_sample", fast(sample), METH_FASTCALL, nullptr},
                         {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "pa_args", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit_pa_args() { return PyModule_Create(&module); }
