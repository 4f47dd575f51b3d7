// Python binding of the calls that a decode step makes: the paged appends with
// the rotary embedding and the attentions over 8-bit pages. At decode sizes
// their kernels take 4 to 8 us, less than ctypes and checks tensor by tensor
// in Python need (15 us a call; here 4, launch included): a call's tensors are
// checked and read here, and the C entry runs on the tensors' device and its
// current stream with the interpreter lock released. What is refused here is
// refused as the package does elsewhere, with TypeError and ValueError; the C
// entry's own status goes back to the package, which raises on it.
#include <ATen/ATen.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Dtype.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>
#include <torch/version.h>

#include <cstdarg>
#include <cstdio>
#include <initializer_list>
#include <map>
#include <string>
#include <vector>

#include "loki.h"

namespace {

struct Refusal {
    PyObject* type;
    std::string text;
};

[[noreturn]] void refuse(PyObject* type, const char* fmt, ...) {
    char text[512];
    va_list va;
    va_start(va, fmt);
    vsnprintf(text, sizeof text, fmt, va);
    va_end(va);
    throw Refusal{type, text};
}

// a Python exception is set already
struct Raised {};

using Args = PyObject* const*;
using Ten = const at::Tensor*;

// argument i: a tensor, or nullptr for None where that is allowed
Ten tensor(PyObject* o, const char* name, bool optional = false) {
    if (optional && o == Py_None) return nullptr;
    if (!THPVariable_Check(o)) refuse(PyExc_TypeError, "%s must be a tensor", name);
    return &THPVariable_Unpack(o);
}

int64_t integer(PyObject* o) {
    const long long v = PyLong_AsLongLong(o);
    if (v == -1 && PyErr_Occurred()) throw Raised();
    return v;
}

int small(int64_t v) {
    if (v < INT32_MIN || v > INT32_MAX) refuse(PyExc_OverflowError, "%lld does not fit a C int", (long long)v);
    return (int)v;
}

double real(PyObject* o) {
    const double v = PyFloat_AsDouble(o);
    if (v == -1 && PyErr_Occurred()) throw Raised();
    return v;
}

bool truth(PyObject* o) {
    const int v = PyObject_IsTrue(o);
    if (v < 0) throw Raised();
    return v;
}

void* ptr(Ten t) { return t != nullptr ? t->data_ptr() : nullptr; }

// the device that contiguous CUDA tensors share
int place(std::initializer_list<Ten> ts) {
    int device = -1;
    for (Ten t : ts) {
        if (t == nullptr) continue;
        if (!t->is_cuda()) refuse(PyExc_ValueError, "all tensors must be CUDA tensors");
        if (device >= 0 && t->get_device() != device) refuse(PyExc_ValueError, "all tensors must be on the same device");
        if (!t->is_contiguous()) refuse(PyExc_ValueError, "all tensors must be contiguous");
        device = t->get_device();
    }
    return device;
}

bool fits(Ten t, at::ScalarType type, at::IntArrayRef shape) { return t->scalar_type() == type && t->sizes() == shape; }

std::string type_name(at::ScalarType t) {
    switch (t) {
        case at::kFloat: return "torch.float32";
        case at::kBFloat16: return "torch.bfloat16";
        case at::kInt: return "torch.int32";
        case at::kFloat8_e4m3fn: return "torch.float8_e4m3fn";
        default: return c10::toString(t);
    }
}

std::string list_of(at::IntArrayRef s) {
    std::string r = "[";
    for (size_t i = 0; i < s.size(); ++i) r += (i ? ", " : "") + std::to_string(s[i]);
    return r + "]";
}

void expect(Ten t, const char* name, at::ScalarType type, at::IntArrayRef shape) {
    if (t != nullptr && !fits(t, type, shape))
        refuse(PyExc_ValueError, "%s must be %s %s (got %s %s)", name, type_name(type).c_str(), list_of(shape).c_str(),
               type_name(t->scalar_type()).c_str(), list_of(t->sizes()).c_str());
}

loki_dtype dtype_of(at::ScalarType t) {
    if (t == at::kFloat) return LOKI_DTYPE_F32;
    if (t == at::kBFloat16) return LOKI_DTYPE_BF16;
    refuse(PyExc_TypeError, "unsupported dtype %s: use torch.float32 or torch.bfloat16", type_name(t).c_str());
}

// the interpreter lock, released for a scope (reading a tensor's address may throw)
struct Unlocked {
    PyThreadState* const state = PyEval_SaveThread();
    ~Unlocked() { PyEval_RestoreThread(state); }
};

// `call` on the device's current stream, the device being the current one
template <class F>
loki_status launch(int device, F call) {
    const c10::cuda::CUDAGuard guard(device);
    void* stream = c10::cuda::getCurrentCUDAStream(device).stream();
    const Unlocked unlocked;
    return call(stream);
}

// a new reference to the tensor argument that was given, or to the fresh tensor in its place
PyObject* object(PyObject* o, Ten given, const at::Tensor& fresh) {
    if (given == nullptr) return THPVariable_Wrap(fresh);
    Py_INCREF(o);
    return o;
}

// 8-bit pages and their scales: the tokens of a scale block
int check_q8(Ten K8, Ten V8, Ten ks, Ten vs) {
    if (K8->scalar_type() != at::kFloat8_e4m3fn || V8->scalar_type() != at::kFloat8_e4m3fn)
        refuse(PyExc_TypeError, "8-bit pages must be torch.float8_e4m3fn");
    if (K8->dim() != 4 || V8->sizes() != K8->sizes() || ks->dim() != 3)
        refuse(PyExc_ValueError, "pages [n_pages, H_kv, page_size, D] and scales [n_pages, H_kv, page_size / block] expected");
    const int64_t page_size = K8->size(2), nb = ks->size(2);
    if (nb < 1 || page_size % nb)
        refuse(PyExc_ValueError, "page_size must be a multiple of the scales' blocks per page");
    expect(ks, "k_scales", at::kFloat, {K8->size(0), K8->size(1), nb});
    expect(vs, "v_scales", at::kFloat, {K8->size(0), K8->size(1), nb});
    return small(page_size / nb);
}

// append(K_new, V_new, P, K_pages, V_pages, k_scales, v_scales, block_table, positions, rope_table,
// interleaved, plane, new_lens, q, q_out): (status, q_out); k_scales None: pages of K_new's type
PyObject* append(Args o, PyObject** out_obj) {
    Ten K = tensor(o[0], "K_new"), V = tensor(o[1], "V_new"), P = tensor(o[2], "P", true);
    Ten Kp = tensor(o[3], "K_pages"), Vp = tensor(o[4], "V_pages");
    const bool q8 = o[5] != Py_None;
    Ten ks = q8 ? tensor(o[5], "k_scales") : nullptr, vs = q8 ? tensor(o[6], "v_scales") : nullptr;
    Ten bt = tensor(o[7], "block_table"), pos = tensor(o[8], "positions"), rope = tensor(o[9], "rope_table", true);
    Ten lo = tensor(o[11], "Kt_lo_pages", true), new_lens = tensor(o[12], "new_lens", true);
    Ten q = tensor(o[13], "q", true), q_out = tensor(o[14], "q_out", true);
    const int block = q8 ? check_q8(Kp, Vp, ks, vs) : 0;
    const int device = place({K, V, P, Kp, Vp, ks, vs, bt, pos, rope, lo, new_lens, q, q_out});
    for (Ten t : {P, rope, lo, new_lens, q, q_out})  // (a null address would mean: not given)
        if (t != nullptr && ptr(t) == nullptr) refuse(PyExc_ValueError, "an optional tensor is given, but has no elements (or no memory)");
    if (K->dim() != 4 || Kp->dim() != 4 || bt->dim() != 2)
        refuse(PyExc_ValueError,
               "K_new [B, H_kv, T, D], pages [n_pages, H_kv, page_size, D] and block_table [B, max_pages] expected");
    const int64_t B = K->size(0), H_kv = K->size(1), T = K->size(2), D = K->size(3);
    const int64_t n_pages = Kp->size(0), page_size = Kp->size(2), max_pages = bt->size(1);
    if (V->sizes() != K->sizes() || Vp->sizes() != Kp->sizes() || Kp->size(1) != H_kv || Kp->size(3) != D ||
        bt->size(0) != B || pos->dim() != 1 || pos->size(0) != B)
        refuse(PyExc_ValueError,
               "K_new, V_new [B, H_kv, T, D], the pages, block_table [B, max_pages] and positions [B] disagree");
    if (bt->scalar_type() != at::kInt || pos->scalar_type() != at::kInt)
        refuse(PyExc_TypeError, "block_table and positions must be int32");
    const at::ScalarType type = K->scalar_type();
    const loki_dtype dt = dtype_of(type);
    if (V->scalar_type() != type || Vp->scalar_type() != Kp->scalar_type())
        refuse(PyExc_TypeError, "K_new and V_new, and the two page pools, must share a dtype");
    if (!q8 && Kp->scalar_type() != type) refuse(PyExc_TypeError, "K_new and the pages must share a dtype");
    expect(P, "P", at::kFloat, {H_kv, D, D});
    if (rope != nullptr && (rope->dim() != 2 || rope->scalar_type() != at::kFloat))
        refuse(PyExc_ValueError, "rope_table must be float32 [n_pos, rot_dim]");
    if (lo != nullptr && lo->dim() != 4) refuse(PyExc_ValueError, "Kt_lo_pages must be [n_pages, H_kv, page_size, d_lo]");
    const int64_t d_lo = lo != nullptr ? lo->size(3) : 0;
    expect(lo, "Kt_lo_pages", type, {n_pages, H_kv, page_size, d_lo});
    expect(new_lens, "new_lens", at::kInt, {B});
    int64_t H_q = H_kv;
    at::Tensor fresh;
    if (q != nullptr) {
        if (q->dim() != 4) refuse(PyExc_ValueError, "q must be [B, H_q, T, D]");
        H_q = q->size(1);
        expect(q, "q", type, {B, H_q, T, D});
        expect(q_out, "q_out", type, {B, H_q, T, D});
        if (q_out == nullptr) {
            fresh = at::empty(q->sizes(), q->options());
            q_out = &fresh;
        }
    } else if (q_out != nullptr) {
        refuse(PyExc_ValueError, "q_out needs q");
    }
    const int inter = truth(o[10]), rot = rope != nullptr ? small(rope->size(1)) : 0;
    const int64_t n_pos = rope != nullptr ? rope->size(0) : 0;
    const auto f32 = [](Ten t) { return static_cast<float*>(ptr(t)); };
    const auto i32 = [](Ten t) { return static_cast<const int32_t*>(ptr(t)); };
    const int iB = small(B), iH = small(H_kv), iT = small(T), ip = small(page_size), im = small(max_pages), iD = small(D),
              iq = small(H_q), il = small(d_lo);
    const loki_status st = launch(device, [&](void* stream) {
        return q8 ? loki_append_keys_paged_q8(ptr(K), ptr(V), f32(P), f32(rope), n_pos, rot, inter, ptr(q), ptr(q_out), iq,
                                              ptr(Kp), ptr(Vp), f32(ks), f32(vs), block, ptr(lo), il, i32(bt), i32(pos),
                                              i32(new_lens), iB, iH, iT, ip, im, n_pages, iD, dt, stream)
                  : loki_append_keys_paged_rope(ptr(K), ptr(V), f32(P), f32(rope), n_pos, rot, inter, ptr(q), ptr(q_out),
                                                iq, ptr(Kp), ptr(Vp), ptr(lo), il, i32(bt), i32(pos), i32(new_lens), iB,
                                                iH, iT, ip, im, n_pages, iD, dt, stream);
    });
    *out_obj = object(o[14], fresh.defined() ? nullptr : K, fresh);  // (o[14] is None without q)
    return PyLong_FromLong(st);
}

// what the attentions over 8-bit pages share
struct Attend {
    Ten q, K8, V8, ks, vs, bt, sl;
    int device, block, B, H_q, H_kv, page_size, max_pages, D;
    int64_t n_pages;
    Attend(Args o, std::initializer_list<Ten> more)
        : q(tensor(o[0], "q")), K8(tensor(o[1], "K8_pages")), V8(tensor(o[2], "V8_pages")), ks(tensor(o[3], "k_scales")),
          vs(tensor(o[4], "v_scales")), bt(tensor(o[5], "block_table")), sl(tensor(o[6], "seq_lens")) {
        block = check_q8(K8, V8, ks, vs);
        device = place({q, K8, V8, ks, vs, bt, sl});
        for (Ten t : more)
            if (t != nullptr) place({q, t});
        if (q->dim() != 3 || bt->dim() != 2) refuse(PyExc_ValueError, "q [B, H_q, D] and block_table [B, max_pages] expected");
        if (q->size(2) != K8->size(3) || bt->size(0) != q->size(0) || sl->dim() != 1 || sl->size(0) != q->size(0))
            refuse(PyExc_ValueError, "q [B, H_q, D], block_table [B, max_pages], seq_lens [B] disagree");
        if (bt->scalar_type() != at::kInt || sl->scalar_type() != at::kInt)
            refuse(PyExc_TypeError, "block_table and seq_lens must be int32");
        B = small(q->size(0));
        H_q = small(q->size(1));
        D = small(q->size(2));
        n_pages = K8->size(0);
        H_kv = small(K8->size(1));
        page_size = small(K8->size(2));
        max_pages = small(bt->size(1));
    }
    const float* scales(Ten t) const { return static_cast<const float*>(t->data_ptr()); }
    const int32_t* ints(Ten t) const { return static_cast<const int32_t*>(t->data_ptr()); }
};

// The caller's workspace, or one of the size the call needs. Calls that need none (the least size a
// query gives) share one per device, which they leave alone.
at::Tensor workspace(Ten given, size_t need, const at::Tensor& like) {
    if (given != nullptr) return *given;
    const auto bytes = like.options().dtype(at::kByte);
    if (need > 256) return at::empty({(int64_t)need}, bytes);
    static auto* spare = new std::map<int, at::Tensor>();  // (under the interpreter lock)
    at::Tensor& t = (*spare)[like.get_device()];
    if (!t.defined()) t = at::empty({256}, bytes);
    return t;
}

// dense(q, K8, V8, k_scales, v_scales, block_table, seq_lens, scale, out, workspace): (status, out)
PyObject* dense(Args o, PyObject** out_obj) {
    Ten out = tensor(o[8], "out", true), ws = tensor(o[9], "workspace", true);
    const Attend a(o, {out, ws});
    const loki_dtype dt = dtype_of(a.q->scalar_type());
    const float scale = (float)real(o[7]);
    expect(out, "out", a.q->scalar_type(), a.q->sizes());
    const at::Tensor w = workspace(
        ws, dense_decode_paged_q8_workspace_size(a.B, a.H_q, a.H_kv, a.page_size, a.max_pages, a.D), *a.q);
    const at::Tensor r = out != nullptr ? *out : at::empty(a.q->sizes(), a.q->options());
    const loki_status st = launch(a.device, [&](void* stream) {
        return dense_decode_attention_paged_q8(a.q->data_ptr(), a.K8->data_ptr(), a.V8->data_ptr(), a.scales(a.ks),
                                               a.scales(a.vs), a.block, a.ints(a.bt), a.ints(a.sl), a.B, a.H_q, a.H_kv,
                                               a.page_size, a.max_pages, a.n_pages, a.D, scale, dt, r.data_ptr(),
                                               w.data_ptr(), w.nbytes(), stream);
    });
    *out_obj = object(o[8], out, r);
    return PyLong_FromLong(st);
}

// sparse(q_rot, K8, V8, k_scales, v_scales, block_table, seq_lens, selected_idx, scale, dtype, out, workspace)
PyObject* sparse(Args o, PyObject** out_obj) {
    Ten idx = tensor(o[7], "selected_idx"), out = tensor(o[10], "out", true), ws = tensor(o[11], "workspace", true);
    const Attend a(o, {idx, out, ws});
    if (a.q->scalar_type() != at::kFloat) refuse(PyExc_TypeError, "q_rot must be float32");
    if (idx->dim() != 3) refuse(PyExc_ValueError, "selected_idx must be [B, H_q, k]");
    const int64_t k = idx->size(2);
    expect(idx, "selected_idx", at::kInt, {a.B, a.H_q, k});
    if (!THPDtype_Check(o[9])) refuse(PyExc_TypeError, "dtype must be a torch.dtype");
    const at::ScalarType type = out != nullptr ? out->scalar_type() : reinterpret_cast<THPDtype*>(o[9])->scalar_type;
    const loki_dtype dt = dtype_of(type);
    expect(out, "out", type, a.q->sizes());
    const float scale = (float)real(o[8]);
    const at::Tensor w = workspace(ws, loki_sparse_attention_paged_q8_workspace_size(a.B, a.H_q, a.H_kv, k, a.D), *a.q);
    const at::Tensor r = out != nullptr ? *out : at::empty(a.q->sizes(), a.q->options().dtype(type));
    const loki_status st = launch(a.device, [&](void* stream) {
        return loki_sparse_attention_paged_q8(static_cast<const float*>(a.q->data_ptr()), a.K8->data_ptr(), a.V8->data_ptr(),
                                              a.scales(a.ks), a.scales(a.vs), a.block, a.ints(a.bt), a.ints(a.sl),
                                              a.ints(idx), a.B, a.H_q, a.H_kv, a.page_size, a.max_pages, a.n_pages, a.D, k,
                                              scale, dt, r.data_ptr(), w.data_ptr(), w.nbytes(), stream);
    });
    *out_obj = object(o[10], out, r);
    return PyLong_FromLong(st);
}

// decode(q, K8, V8, k_scales, v_scales, block_table, seq_lens, plane, P, d, k, scale, out, selected_idx, workspace):
// (status, (out, selected_idx))
PyObject* decode(Args o, PyObject** out_obj) {
    Ten lo = tensor(o[7], "Kt_lo_pages"), P = tensor(o[8], "P"), out = tensor(o[12], "out", true);
    Ten idx = tensor(o[13], "selected_idx", true), ws = tensor(o[14], "workspace", true);
    const Attend a(o, {lo, P, out, idx, ws});
    const at::ScalarType type = a.q->scalar_type();
    const loki_dtype dt = dtype_of(type);
    if (lo->dim() != 4) refuse(PyExc_ValueError, "Kt_lo_pages must be [n_pages, H_kv, page_size, d_lo]");
    const int64_t d_lo = lo->size(3), k = integer(o[10]);
    const int d = small(integer(o[9])), il = small(d_lo);
    expect(lo, "Kt_lo_pages", type, {a.n_pages, a.H_kv, a.page_size, d_lo});
    expect(P, "P", at::kFloat, {a.H_kv, a.D, a.D});
    if (k < 0) refuse(PyExc_ValueError, "k must not be negative");
    expect(out, "out", type, a.q->sizes());
    expect(idx, "selected_idx", at::kInt, {a.B, a.H_q, k});
    const float scale = (float)real(o[11]);
    const at::Tensor w = workspace(
        ws, loki_paged_q8_decode_workspace_size(a.B, a.H_q, a.H_kv, a.page_size, a.max_pages, a.D, d, k), *a.q);
    const at::Tensor r = out != nullptr ? *out : at::empty(a.q->sizes(), a.q->options());
    const at::Tensor si = idx != nullptr ? *idx : at::empty({a.B, a.H_q, k}, a.q->options().dtype(at::kInt));
    const loki_status st = launch(a.device, [&](void* stream) {
        return loki_decode_attention_paged_q8(a.q->data_ptr(), a.K8->data_ptr(), a.V8->data_ptr(), a.scales(a.ks),
                                              a.scales(a.vs), a.block, lo->data_ptr(), il, a.scales(P), a.ints(a.bt),
                                              a.ints(a.sl), a.B, a.H_q, a.H_kv, a.page_size, a.max_pages, a.n_pages,
                                              a.D, d, k, scale, dt, r.data_ptr(), static_cast<int32_t*>(si.data_ptr()),
                                              w.data_ptr(), w.nbytes(), stream);
    });
    // ("N" takes the new references)
    *out_obj = Py_BuildValue("(NN)", object(o[12], out, r), object(o[13], idx, si));
    return PyLong_FromLong(st);
}

// rope_table(table, base, pos_scale): (status, None)
PyObject* rope_table(Args o, PyObject** out_obj) {
    Ten t = tensor(o[0], "table");
    const int device = place({t});
    if (t->dim() != 2 || t->scalar_type() != at::kFloat) refuse(PyExc_ValueError, "table must be torch.float32 [n_pos, rot_dim]");
    const double base = real(o[1]), pos_scale = real(o[2]);
    const int rot = small(t->size(1));
    Py_INCREF(Py_None);
    *out_obj = Py_None;
    return PyLong_FromLong(launch(device, [&](void* stream) {
        return loki_rope_table(static_cast<float*>(t->data_ptr()), t->size(0), rot, base, pos_scale, stream);
    }));
}

template <PyObject* (*F)(Args, PyObject**), int N>
PyObject* entry(PyObject*, PyObject* const* args, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    if (n != N) return PyErr_Format(PyExc_TypeError, "%d arguments expected (got %zd)", N, n);
    PyObject *out = nullptr, *status = nullptr;
    try {
        status = F(args, &out);
    } catch (const Refusal& r) {
        PyErr_SetString(r.type, r.text.c_str());
    } catch (const Raised&) {
    } catch (...) {
        Py_XDECREF(out);
        throw;
    }
    if (status == nullptr || out == nullptr) {
        Py_XDECREF(status);
        Py_XDECREF(out);
        return nullptr;
    }
    PyObject* pair = PyTuple_Pack(2, status, out);
    Py_DECREF(status);
    Py_DECREF(out);
    return pair;
    END_HANDLE_TH_ERRORS
}

#define LOKI_ENTRY(f, n) {#f, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(&entry<&f, n>)), METH_FASTCALL, nullptr}
PyMethodDef methods[] = {LOKI_ENTRY(append, 15), LOKI_ENTRY(dense, 10),     LOKI_ENTRY(sparse, 12),
                         LOKI_ENTRY(decode, 15), LOKI_ENTRY(rope_table, 3), {nullptr, nullptr, 0, nullptr}};

PyModuleDef module = {PyModuleDef_HEAD_INIT, "_binding", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__binding() {
    PyObject* m = PyModule_Create(&module);
    if (m != nullptr && PyModule_AddStringConstant(m, "torch_version", TORCH_VERSION) < 0) {
        Py_DECREF(m);
        return nullptr;
    }
    return m;
}
