// Python binding of the speculative-step calls: argument checks, output allocation and the call of the C entry
// point of the same name on the current stream.
//
// These calls run once per layer and decoding step on small inputs, where checking the tensors in Python takes
// longer than the kernels; here a call's host side is a few microseconds.  The functions take their arguments by
// position (None for absent ones); spec.py has the signatures and their documentation.
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <ATen/core/Tensor.h>
#include <ATen/ops/empty.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <cmath>
#include <initializer_list>
#include <string>

#include "../../include/kda.h"

namespace {

// A refused argument: becomes the Python exception of the given type.
struct Refused {
    PyObject *type;
    std::string text;
};
[[noreturn]] void type_error(const std::string &text) { throw Refused{PyExc_TypeError, text}; }
[[noreturn]] void value_error(const std::string &text) { throw Refused{PyExc_ValueError, text}; }
std::string str(int64_t x) { return std::to_string(x); }

const at::Tensor &tensor(PyObject *o, const char *name) {
    if (!THPVariable_Check(o)) type_error(std::string(name) + " must be a torch.Tensor");
    const at::Tensor &t = THPVariable_Unpack(o);
    if (!t.is_cuda()) value_error(std::string(name) + " must be a CUDA tensor");
    return t;
}
bool absent(PyObject *o) { return o == Py_None; }

kda_dtype code(const at::Tensor &t, const char *name) {
    if (t.scalar_type() == at::kBFloat16) return KDA_BF16;
    if (t.scalar_type() == at::kFloat) return KDA_F32;
    type_error(std::string(name) + " must be bf16 or fp32");
}
void same_dtype(const at::Tensor &t, at::ScalarType want, const char *name) {
    if (t.scalar_type() != want) type_error(std::string(name) + " has dtype " + c10::toString(t.scalar_type()) + ", expected " + c10::toString(want));
}

// A [T, H, d] tensor whose tokens may be strided (a slice of a fused projection); T < 0: any.  Its token stride, 0
// for packed.
int64_t token_stride(const at::Tensor &t, const char *name, at::ScalarType dtype, int64_t T, int64_t H, int64_t d) {
    same_dtype(t, dtype, name);
    if (t.dim() != 3 || t.size(1) != H || t.size(2) != d || (T >= 0 && t.size(0) != T))
        value_error(std::string(name) + " has the wrong shape: expected (" + (T < 0 ? "T" : str(T)) + ", " + str(H) + ", " + str(d) + ")");
    if ((t.stride(2) != 1 && d > 1) || (H > 1 && t.stride(1) != d))
        value_error(std::string(name) + " must have contiguous tokens (only its first dimension may be strided)");
    if (t.size(0) <= 1) return 0;
    if (t.stride(0) < H * d) value_error(std::string(name) + " must not have overlapping tokens");
    return t.stride(0);
}

// A contiguous vector of n elements (n < 0: any).
const at::Tensor &vec(PyObject *o, const char *name, at::ScalarType dtype, int64_t n) {
    const at::Tensor &t = tensor(o, name);
    if (t.scalar_type() != dtype || t.dim() != 1 || !t.is_contiguous())
        value_error(std::string(name) + " must be a contiguous " + c10::toString(dtype) + " CUDA vector");
    if (n >= 0 && t.size(0) != n) value_error(std::string(name) + " has " + str(t.size(0)) + " entries, expected " + str(n));
    return t;
}
int32_t *ints(PyObject *o, const char *name, int64_t n) {
    return absent(o) ? nullptr : vec(o, name, at::kInt, n).data_ptr<int32_t>();
}

// A contiguous tensor that the caller passed for an output.
const at::Tensor &given(PyObject *o, const char *name, at::ScalarType dtype, at::IntArrayRef shape) {
    const at::Tensor &t = tensor(o, name);
    same_dtype(t, dtype, name);
    if (t.sizes() != shape || !t.is_contiguous()) value_error(std::string(name) + " must be contiguous and have the output's shape");
    return t;
}
at::Tensor fresh(at::IntArrayRef shape, at::ScalarType dtype, const at::Tensor &like) {
    return at::empty(shape, at::TensorOptions().dtype(dtype).device(like.device()));
}

// The workspace passed, or one of this call's own.
struct Workspace {
    at::Tensor t;
    size_t bytes;
    Workspace(PyObject *o, size_t need, const at::Tensor &like) {
        if (absent(o)) {
            bytes = need < KDA_WS_HEADER_BYTES ? KDA_WS_HEADER_BYTES : need;
            t = fresh({static_cast<int64_t>(bytes)}, at::kByte, like);
        } else {
            t = tensor(o, "workspace");
            if (!t.is_contiguous()) value_error("workspace must be contiguous");
            bytes = static_cast<size_t>(t.numel()) * t.element_size();
        }
    }
};

struct Cache {
    kda_paged_kv c;
    int64_t N, max_ctx;
};
Cache cache(PyObject *k_pages, PyObject *v_pages, PyObject *table, PyObject *ctx_len, at::ScalarType dtype, int64_t Hkv, int64_t dk,
            int64_t dv) {
    const at::Tensor &k = tensor(k_pages, "k_pages"), &v = tensor(v_pages, "v_pages"), &b = tensor(table, "block_table");
    for (int i = 0; i < 2; ++i) {
        const at::Tensor &t = i ? v : k;
        const char *name = i ? "v_pages" : "k_pages";
        same_dtype(t, dtype, name);
        if (t.dim() != 4 || t.stride(3) != 1 || t.size(2) != Hkv || t.size(3) != (i ? dv : dk))
            value_error(std::string(name) + " must be [pages, page_size, " + str(Hkv) + ", " + str(i ? dv : dk) + "] with contiguous channels");
    }
    if (k.size(0) != v.size(0) || k.size(1) != v.size(1)) value_error("k_pages and v_pages must have the same pages and page size");
    if (b.scalar_type() != at::kInt || b.dim() != 2 || (b.size(1) > 1 && b.stride(1) != 1))
        value_error("block_table must be an int32 CUDA matrix [N, max_pages] with contiguous rows");
    if (k.size(1) > 0x7fffffffLL || b.size(1) > 0x7fffffffLL || b.size(0) > 0x7fffffffLL) value_error("the cache is too large");
    const int64_t N = b.size(0);
    Cache out;
    out.N = N;
    out.max_ctx = b.size(1) * k.size(1);
    out.c = kda_paged_kv{k.data_ptr(), v.data_ptr(), k.stride(0), k.stride(1), k.stride(2), v.stride(0), v.stride(1), v.stride(2),
                         k.size(0), N > 1 ? b.stride(0) : b.size(1), b.data_ptr<int32_t>(), ints(ctx_len, "ctx_len", N),
                         static_cast<int>(k.size(1)), static_cast<int>(b.size(1))};
    return out;
}

int small(int64_t x, const char *name) {
    if (x < -0x7fffffffLL || x > 0x7fffffffLL) value_error(std::string(name) + " is out of range");
    return static_cast<int>(x);
}
int64_t integer(PyObject *o) {
    const long long x = PyLong_AsLongLong(o);
    if (x == -1 && PyErr_Occurred()) throw python_error();
    return x;
}
double number(PyObject *o) {
    const double x = PyFloat_AsDouble(o);
    if (x == -1.0 && PyErr_Occurred()) throw python_error();
    return x;
}
bool truth(PyObject *o) {
    const int x = PyObject_IsTrue(o);
    if (x < 0) throw python_error();
    return x != 0;
}

// A status other than KDA_OK becomes the package's KdaError.
void check(kda_status rc, const char *where) {
    if (rc == KDA_OK) return;
    PyObject *mod = PyImport_ImportModule("gated_linear_attention_chunk_gb300.kda");
    PyObject *type = mod ? PyObject_GetAttrString(mod, "KdaError") : nullptr;
    PyObject *err = type ? PyObject_CallFunction(type, "is", static_cast<int>(rc), where) : nullptr;
    if (err) PyErr_SetObject(type, err);
    Py_XDECREF(err);
    Py_XDECREF(type);
    Py_XDECREF(mod);
    throw python_error();
}

void *stream_of(const at::Tensor &t) { return c10::cuda::getCurrentCUDAStream(t.device().index()).stream(); }

PyObject *wrap(const at::Tensor &t) { return t.defined() ? THPVariable_Wrap(t) : Py_NewRef(Py_None); }
PyObject *tuple(std::initializer_list<at::Tensor> ts) {
    PyObject *out = PyTuple_New(static_cast<Py_ssize_t>(ts.size()));
    if (!out) throw python_error();
    Py_ssize_t i = 0;
    for (const at::Tensor &t : ts) {
        PyObject *o = wrap(t);
        if (!o) {
            Py_DECREF(out);
            throw python_error();
        }
        PyTuple_SET_ITEM(out, i++, o);
    }
    return out;
}

// (backward, q, k, positions, inv_freq, interleaved, mscale, q_out, k_out) -> (q_out, k_out)
PyObject *rope(PyObject *const *a) {
    const bool backward = truth(a[0]);
    const at::Tensor &q = tensor(a[1], "q");
    const kda_dtype dt = code(q, "q");
    const at::ScalarType st = q.scalar_type();
    if (q.dim() != 3) value_error("q must be [T, Hq, d]");
    const int64_t T = q.size(0), Hq = q.size(1), d = q.size(2);
    const int64_t qs = token_stride(q, "q", st, T, Hq, d);
    int64_t Hk = 0, ks = 0, qos = 0, kos = 0;
    const bool has_k = !absent(a[2]);
    if (has_k) {
        const at::Tensor &k = tensor(a[2], "k");
        if (k.dim() != 3) value_error("k must be [T, Hk, d]");
        Hk = k.size(1);
        ks = token_stride(k, "k", st, T, Hk, d);
    }
    const int32_t *pos = vec(a[3], "positions", at::kInt, T).data_ptr<int32_t>();
    const at::Tensor &w = vec(a[4], "inv_freq", at::kDouble, -1);
    const c10::cuda::CUDAGuard guard(q.device());
    at::Tensor qo, ko;
    if (absent(a[7])) {
        qo = fresh({T, Hq, d}, st, q);
    } else {
        qo = tensor(a[7], "q_out");
        qos = token_stride(qo, "q_out", st, T, Hq, d);
    }
    if (has_k) {
        if (absent(a[8])) {
            ko = fresh({T, Hk, d}, st, q);
        } else {
            ko = tensor(a[8], "k_out");
            kos = token_stride(ko, "k_out", st, T, Hk, d);
        }
    }
    auto call = backward ? kda_rope_bwd : kda_rope;
    check(call(q.data_ptr(), has_k ? THPVariable_Unpack(a[2]).data_ptr() : nullptr, dt, pos, w.data_ptr<double>(), T, small(Hq, "Hq"),
               small(Hk, "Hk"), small(d, "d"), small(2 * w.size(0), "rot"), qs, ks, truth(a[5]) ? 1 : 0, static_cast<float>(number(a[6])),
               qo.data_ptr(), has_k ? ko.data_ptr() : nullptr, qos, kos, stream_of(q)),
          backward ? "kda_rope_bwd" : "kda_rope");
    return tuple({qo, ko});
}

// (q, k, v, k_pages, v_pages, block_table, ctx_len, cu_nodes, parent, scale, max_nodes, o, lse, return_lse, workspace)
// -> (o, lse)
PyObject *tree_attn(PyObject *const *a) {
    const at::Tensor &q = tensor(a[0], "q"), &k = tensor(a[1], "k"), &v = tensor(a[2], "v");
    const kda_dtype dt = code(q, "q");
    const at::ScalarType st = q.scalar_type();
    if (q.dim() != 3 || v.dim() != 3) value_error("q must be [T, Hq, dk] and v [T, Hkv, dv]");
    const int64_t T = q.size(0), Hq = q.size(1), dk = q.size(2), Hkv = v.size(1), dv = v.size(2);
    const int64_t qs = token_stride(q, "q", st, T, Hq, dk), ks = token_stride(k, "k", st, T, Hkv, dk), vs = token_stride(v, "v", st, T, Hkv, dv);
    const Cache c = cache(a[3], a[4], a[5], a[6], st, Hkv, dk, dv);
    const int32_t *cu = absent(a[7]) ? nullptr : ints(a[7], "cu_nodes", c.N + 1), *parent = ints(a[8], "parent", T);
    const int max_nodes = small(integer(a[10]), "max_nodes");
    const float scale = absent(a[9]) ? 1.f / std::sqrt(static_cast<float>(dk)) : static_cast<float>(number(a[9]));
    const c10::cuda::CUDAGuard guard(q.device());
    const at::Tensor o = absent(a[11]) ? fresh({T, Hq, dv}, st, q) : given(a[11], "o", st, {T, Hq, dv});
    at::Tensor lse;
    if (!absent(a[12])) lse = given(a[12], "lse", at::kFloat, {T, Hq});
    else if (truth(a[13])) lse = fresh({T, Hq}, at::kFloat, q);
    const size_t need = absent(a[14]) ? kda_tree_attn_workspace_size_for(dt, small(c.N, "N"), T, small(Hq, "Hq"), small(Hkv, "Hkv"), small(dv, "dv"),
                                                                     max_nodes, c.max_ctx) : 0;
    const Workspace ws(a[14], need, q);
    check(kda_tree_attn(q.data_ptr(), k.data_ptr(), v.data_ptr(), dt, &c.c, cu, parent, small(c.N, "N"), T, small(Hq, "Hq"),
                        small(Hkv, "Hkv"), small(dk, "dk"), small(dv, "dv"), qs, ks, vs, max_nodes, scale, o.data_ptr(),
                        lse.defined() ? lse.data_ptr<float>() : nullptr, ws.t.data_ptr(), ws.bytes, stream_of(q)),
          "kda_tree_attn");
    return tuple({o, lse});
}

// (k, v, k_pages, v_pages, block_table, ctx_len, cu, rows, new_len, workspace) -> new_len
PyObject *cache_append(PyObject *const *a) {
    const at::Tensor &k = tensor(a[0], "k"), &v = tensor(a[1], "v");
    const kda_dtype dt = code(k, "k");
    const at::ScalarType st = k.scalar_type();
    if (k.dim() != 3 || v.dim() != 3) value_error("k must be [T, Hkv, dk] and v [T, Hkv, dv]");
    const int64_t T = k.size(0), Hkv = k.size(1), dk = k.size(2), dv = v.size(2);
    const int64_t ks = token_stride(k, "k", st, T, Hkv, dk), vs = token_stride(v, "v", st, T, Hkv, dv);
    const Cache c = cache(a[2], a[3], a[4], a[5], st, Hkv, dk, dv);
    const int32_t *cu = vec(a[6], "cu", at::kInt, c.N + 1).data_ptr<int32_t>();
    const int32_t *rows = ints(a[7], "rows", -1);
    const int64_t total = rows || !absent(a[7]) ? THPVariable_Unpack(a[7]).size(0) : T;
    const c10::cuda::CUDAGuard guard(k.device());
    const at::Tensor new_len = absent(a[8]) ? fresh({c.N}, at::kInt, k) : vec(a[8], "new_len", at::kInt, c.N);
    const Workspace ws(a[9], KDA_WS_HEADER_BYTES, k);
    check(kda_cache_append(k.data_ptr(), v.data_ptr(), dt, &c.c, cu, rows, small(c.N, "N"), total, T, small(Hkv, "Hkv"), small(dk, "dk"),
                           small(dv, "dv"), ks, vs, new_len.data_ptr<int32_t>(), ws.t.data_ptr(), ws.bytes, stream_of(k)),
          "kda_cache_append");
    return wrap(new_len);
}

// (tokens, cu_nodes, target_probs, u_accept, u_sample, parent, draft_probs, cu_accept, rows, next_token, workspace)
// -> (cu_accept, rows, next_token)
PyObject *draft_verify(PyObject *const *a) {
    const at::Tensor &p = tensor(a[2], "target_probs");
    const kda_dtype dt = code(p, "target_probs");
    auto matrix = [&](const at::Tensor &t, const char *name) -> int64_t {  // its row stride
        same_dtype(t, p.scalar_type(), name);
        if (t.dim() != 2 || t.sizes() != p.sizes() || (t.size(1) > 1 && t.stride(1) != 1))
            value_error(std::string(name) + " must be a CUDA matrix [T, V] with contiguous rows");
        return t.size(0) > 1 ? t.stride(0) : 0;
    };
    const int64_t ps = matrix(p, "target_probs"), T = p.size(0), V = p.size(1);
    const bool draft = !absent(a[6]);
    const int64_t ds = draft ? matrix(tensor(a[6], "draft_probs"), "draft_probs") : 0;
    const at::Tensor &cu = vec(a[1], "cu_nodes", at::kInt, -1);
    const int64_t N = cu.size(0) - 1;
    if (N < 0) value_error("cu_nodes must have at least one entry");
    const int32_t *tokens = vec(a[0], "tokens", at::kInt, T).data_ptr<int32_t>(), *parent = ints(a[5], "parent", T);
    const float *ua = vec(a[3], "u_accept", at::kFloat, T).data_ptr<float>(), *us = vec(a[4], "u_sample", at::kFloat, N).data_ptr<float>();
    const c10::cuda::CUDAGuard guard(p.device());
    const at::Tensor counts = absent(a[7]) ? fresh({N + 1}, at::kInt, p) : vec(a[7], "cu_accept", at::kInt, N + 1);
    const at::Tensor rows = absent(a[8]) ? fresh({T}, at::kInt, p) : vec(a[8], "rows", at::kInt, T);
    const at::Tensor next = absent(a[9]) ? fresh({N}, at::kInt, p) : vec(a[9], "next_token", at::kInt, N);
    const Workspace ws(a[10], kda_draft_verify_workspace_size(small(N, "N")), p);
    check(kda_draft_verify(tokens, cu.data_ptr<int32_t>(), parent, p.data_ptr(), draft ? THPVariable_Unpack(a[6]).data_ptr() : nullptr,
                           dt, ua, us, small(N, "N"), T, small(V, "V"), ps, ds, counts.data_ptr<int32_t>(), rows.data_ptr<int32_t>(),
                           next.data_ptr<int32_t>(), ws.t.data_ptr(), ws.bytes, stream_of(p)),
          "kda_draft_verify");
    return tuple({counts, rows, next});
}

// The arguments of a call lie on one device.
void on_device(const at::Tensor &t, const char *name, const at::Tensor &first) {
    if (t.device() != first.device()) value_error(std::string(name) + " is on another device");
}

// A [T, H, d] argument of a norm: its tensor and token stride.
struct Rows {
    at::Tensor t;
    int64_t stride = 0;
    const void *ptr() const { return t.defined() ? t.data_ptr() : nullptr; }
    void *out() const { return t.defined() ? t.data_ptr() : nullptr; }
};
Rows rows_of(PyObject *o, const char *name, const at::Tensor &q, int64_t T, int64_t H, int64_t d) {
    Rows r;
    r.t = tensor(o, name);
    on_device(r.t, name, q);
    r.stride = token_stride(r.t, name, q.scalar_type(), T, H, d);
    return r;
}
Rows rows_out(PyObject *o, const char *name, const at::Tensor &q, int64_t T, int64_t H, int64_t d) {
    if (!absent(o)) return rows_of(o, name, q, T, H, d);
    Rows r;
    r.t = fresh({T, H, d}, q.scalar_type(), q);
    return r;
}

// (q, k, d_q_out, d_k_out, positions, inv_freq, q_weight, k_weight, eps, interleaved, mscale, q_out, k_out, d_q_weight, d_k_weight,
// workspace) -> (q_out, k_out), or with d_q_out (the gradient) (d_q, d_k, d_q_weight, d_k_weight)
PyObject *norm_rope(PyObject *const *a) {
    const at::Tensor &q = tensor(a[0], "q");
    const kda_dtype dt = code(q, "q");
    if (q.dim() != 3) value_error("q must be [T, Hq, d]");
    const int64_t T = q.size(0), Hq = q.size(1), d = q.size(2);
    const int64_t qs = token_stride(q, "q", q.scalar_type(), T, Hq, d);
    const bool backward = !absent(a[2]), has_k = !absent(a[1]);
    if (has_k != !absent(a[3]) && backward) value_error("k and d_k_out go together");
    if (!has_k && (!absent(a[12]) || !absent(a[14]))) value_error("an output for k without k");
    const c10::cuda::CUDAGuard guard(q.device());
    Rows k, gq, gk, yq, yk;
    int64_t Hk = 0;
    if (has_k) {
        const at::Tensor &t = tensor(a[1], "k");
        if (t.dim() != 3) value_error("k must be [T, Hk, d]");
        Hk = t.size(1);
        k = rows_of(a[1], "k", q, T, Hk, d);
    }
    if (backward) {
        gq = rows_of(a[2], "d_q_out", q, T, Hq, d);
        if (has_k) gk = rows_of(a[3], "d_k_out", q, T, Hk, d);
    }
    const at::Tensor &pos = vec(a[4], "positions", at::kInt, T), &freq = vec(a[5], "inv_freq", at::kDouble, -1);
    on_device(pos, "positions", q);
    on_device(freq, "inv_freq", q);
    kda_dtype wdt = KDA_F32;
    const void *w[2] = {nullptr, nullptr};
    for (int i = 0; i < 2; ++i) {
        const char *name = i ? "k_weight" : "q_weight";
        if (absent(a[6 + i])) continue;
        const at::Tensor &t = tensor(a[6 + i], name);
        const kda_dtype c = code(t, name);
        if (i && w[0] && c != wdt) type_error("q_weight and k_weight must have one dtype");
        wdt = c;
        vec(a[6 + i], name, t.scalar_type(), d);
        on_device(t, name, q);
        w[i] = t.data_ptr();
    }
    const float eps = static_cast<float>(number(a[8])), mscale = static_cast<float>(number(a[10]));
    const int inter = truth(a[9]) ? 1 : 0, rot = small(2 * freq.size(0), "rot");
    yq = rows_out(a[11], backward ? "d_q" : "q_out", q, T, Hq, d);
    if (has_k) yk = rows_out(a[12], backward ? "d_k" : "k_out", q, T, Hk, d);
    if (!backward) {
        check(kda_norm_rope(q.data_ptr(), k.ptr(), dt, w[0], w[1], wdt, pos.data_ptr<int32_t>(), freq.data_ptr<double>(), T, small(Hq, "Hq"),
                            small(Hk, "Hk"), small(d, "d"), rot, qs, k.stride, inter, mscale, eps, yq.out(), yk.out(), yq.stride, yk.stride,
                            stream_of(q)),
              "kda_norm_rope");
        return tuple({yq.t, yk.t});
    }
    at::Tensor dw[2];
    for (int i = 0; i < (has_k ? 2 : 1); ++i) {
        const char *name = i ? "d_k_weight" : "d_q_weight";
        if (!absent(a[13 + i])) {
            dw[i] = vec(a[13 + i], name, at::kFloat, d);
            on_device(dw[i], name, q);
        } else if (w[i]) {
            dw[i] = fresh({d}, at::kFloat, q);
        }
    }
    const Workspace ws(a[15], kda_norm_rope_bwd_workspace_size(small(d, "d")), q);
    on_device(ws.t, "workspace", q);
    check(kda_norm_rope_bwd(q.data_ptr(), k.ptr(), gq.ptr(), gk.ptr(), dt, w[0], w[1], wdt, pos.data_ptr<int32_t>(), freq.data_ptr<double>(), T,
                            small(Hq, "Hq"), small(Hk, "Hk"), small(d, "d"), rot, qs, k.stride, gq.stride, gk.stride, inter, mscale, eps,
                            yq.out(), yk.out(), yq.stride, yk.stride, dw[0].defined() ? dw[0].data_ptr<float>() : nullptr,
                            dw[1].defined() ? dw[1].data_ptr<float>() : nullptr, ws.t.data_ptr(), ws.bytes, stream_of(q)),
          "kda_norm_rope_bwd");
    return tuple({yq.t, yk.t, dw[0], dw[1]});
}

// (q, k_pages, v_pages, block_table, prefix_len, cu_tokens, scale, o_tail, lse_tail, o, lse, return_lse, workspace) -> (o, lse)
PyObject *prefix_attn(PyObject *const *a) {
    const at::Tensor &q = tensor(a[0], "q"), &kp = tensor(a[1], "k_pages"), &vp = tensor(a[2], "v_pages");
    const kda_dtype dt = code(q, "q");
    const at::ScalarType st = q.scalar_type();
    if (q.dim() != 3) value_error("q must be [T, Hq, dk]");
    if (kp.dim() != 4 || vp.dim() != 4) value_error("k_pages and v_pages must be [pages, page_size, Hkv, dk] and [.., dv]");
    const int64_t T = q.size(0), Hq = q.size(1), dk = q.size(2), Hkv = kp.size(2), dv = vp.size(3);
    const int64_t qs = token_stride(q, "q", st, T, Hq, dk);
    const Cache c = cache(a[1], a[2], a[3], a[4], st, Hkv, dk, dv);
    const at::Tensor &cu = vec(a[5], "cu_tokens", at::kInt, c.N + 1);
    if (absent(a[4])) type_error("prefix_len must be a torch.Tensor");
    for (int i = 1; i < 6; ++i) on_device(THPVariable_Unpack(a[i]), "an argument", q);
    const float scale = absent(a[6]) ? 1.f / std::sqrt(static_cast<float>(dk)) : static_cast<float>(number(a[6]));
    if (absent(a[7]) != absent(a[8])) value_error("o_tail and lse_tail go together");
    const c10::cuda::CUDAGuard guard(q.device());
    const bool tail = !absent(a[7]);
    if (tail) {
        on_device(given(a[7], "o_tail", st, {T, Hq, dv}), "o_tail", q);
        on_device(given(a[8], "lse_tail", at::kFloat, {T, Hq}), "lse_tail", q);
    }
    const at::Tensor o = absent(a[9]) ? fresh({T, Hq, dv}, st, q) : given(a[9], "o", st, {T, Hq, dv});
    at::Tensor lse;
    if (!absent(a[10])) lse = given(a[10], "lse", at::kFloat, {T, Hq});
    else if (truth(a[11])) lse = fresh({T, Hq}, at::kFloat, q);
    on_device(o, "o", q);
    if (lse.defined()) on_device(lse, "lse", q);
    const size_t need = absent(a[12]) ? kda_prefix_attn_workspace_size(small(c.N, "N"), T, small(Hq, "Hq"), small(Hkv, "Hkv"), small(dv, "dv")) : 0;
    const Workspace ws(a[12], need, q);
    on_device(ws.t, "workspace", q);
    check(kda_prefix_attn(q.data_ptr(), dt, &c.c, cu.data_ptr<int32_t>(), small(c.N, "N"), T, small(Hq, "Hq"), small(Hkv, "Hkv"), small(dk, "dk"),
                          small(dv, "dv"), qs, scale, tail ? THPVariable_Unpack(a[7]).data_ptr() : nullptr,
                          tail ? THPVariable_Unpack(a[8]).data_ptr<float>() : nullptr, o.data_ptr(),
                          lse.defined() ? lse.data_ptr<float>() : nullptr, ws.t.data_ptr(), ws.bytes, stream_of(q)),
          "kda_prefix_attn");
    return tuple({o, lse});
}

// (logits, u, temperature, top_k, top_p, min_p, return_probs, token, probs) -> token or (token, probs)
PyObject *sample(PyObject *const *a) {
    const at::Tensor &l = tensor(a[0], "logits");
    const kda_dtype dt = code(l, "logits");
    auto rows = [&](const at::Tensor &t, const char *name) -> int64_t {  // its row stride
        if (t.dim() != 2 || t.sizes() != l.sizes() || (t.size(1) > 1 && t.stride(1) != 1))
            value_error(std::string(name) + " must be a CUDA matrix [N, V] with contiguous rows");
        if (t.size(0) > 1 && t.stride(0) < t.size(1)) value_error(std::string(name) + " must not have overlapping rows");
        return t.size(0) > 1 ? t.stride(0) : 0;
    };
    const int64_t ls = rows(l, "logits"), N = l.size(0), V = l.size(1);
    auto floats = [&](PyObject *o, const char *name) -> const float * {
        if (absent(o)) return nullptr;
        const at::Tensor &t = vec(o, name, at::kFloat, N);
        on_device(t, name, l);
        return t.data_ptr<float>();
    };
    if (absent(a[1])) type_error("u must be a torch.Tensor");
    const float *u = floats(a[1], "u"), *t = floats(a[2], "temperature"), *top_p = floats(a[4], "top_p"), *min_p = floats(a[5], "min_p");
    const int32_t *top_k = ints(a[3], "top_k", N);
    if (top_k) on_device(THPVariable_Unpack(a[3]), "top_k", l);
    const bool want = truth(a[6]) || !absent(a[8]);
    const c10::cuda::CUDAGuard guard(l.device());
    const at::Tensor token = absent(a[7]) ? fresh({N}, at::kInt, l) : vec(a[7], "token", at::kInt, N);
    on_device(token, "token", l);
    at::Tensor probs;
    kda_dtype pdt = KDA_F32;
    int64_t ps = 0;
    if (!absent(a[8])) {
        probs = tensor(a[8], "probs");
        on_device(probs, "probs", l);
        pdt = code(probs, "probs");
        ps = rows(probs, "probs");
    } else if (want) {
        probs = fresh({N, V}, at::kFloat, l);
    }
    check(kda_sample(l.data_ptr(), dt, u, t, top_k, top_p, min_p, small(N, "N"), small(V, "V"), ls, token.data_ptr<int32_t>(),
                     probs.defined() ? probs.data_ptr() : nullptr, pdt, ps, stream_of(l)),
          "kda_sample");
    return want ? tuple({token, probs}) : wrap(token);
}

// Runs a function with the given number of arguments; nothing but a Python exception leaves it.
template <PyObject *(*kFunction)(PyObject *const *), int kArgs>
PyObject *guarded(PyObject *, PyObject *const *args, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    if (n != kArgs) {
        PyErr_Format(PyExc_TypeError, "expected %d arguments, got %zd", kArgs, n);
        return nullptr;
    }
    try {
        return kFunction(args);
    } catch (const Refused &r) {
        PyErr_SetString(r.type, r.text.c_str());
        return nullptr;
    }
    END_HANDLE_TH_ERRORS
}

template <PyObject *(*kFunction)(PyObject *const *), int kArgs>
PyMethodDef method(const char *name) {
    return {name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(&guarded<kFunction, kArgs>)), METH_FASTCALL, nullptr};
}

PyMethodDef methods[] = {method<rope, 9>("rope"), method<tree_attn, 15>("tree_attn"), method<cache_append, 10>("cache_append"),
                         method<draft_verify, 11>("draft_verify"), method<norm_rope, 16>("norm_rope"), method<sample, 9>("sample"),
                         method<prefix_attn, 13>("prefix_attn"),
                         {nullptr, nullptr, 0, nullptr}};
PyModuleDef module_def = {PyModuleDef_HEAD_INIT, "_spec", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__spec(void) { return PyModule_Create(&module_def); }
