// binding.cpp -- the rotary, append, quantised-cache and eviction calls on torch tensors.
//
// Argument checks and marshalling only: every tensor's type, shape, placement and
// strides are checked against what the call reads and writes, outputs are
// allocated by torch, and raw pointers go to the C ABI (include/attn.h) on the
// current CUDA stream.  Native, because these calls run a few microseconds on the
// GPU and a step makes several: checked from Python through ctypes a call took
// 15 us of host time for its two output tensors, three times the launch.
// The Python functions of attn.py, which name and document the arguments, are the
// only callers.
#include <Python.h>

#include <ATen/core/Tensor.h>
#include <ATen/cuda/EmptyTensor.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <cmath>
#include <cstring>
#include <optional>
#include <sstream>
#include <string>

#include "../../include/attn.h"

namespace {

using at::Tensor;

PyObject* g_error = nullptr;  // the binding's exception class: (status, message)

struct Refusal {  // a ValueError
    std::string what;
};
struct PythonError {};  // already set

template <typename... Parts>
[[noreturn]] void refuse(const Parts&... parts) {
    std::ostringstream s;
    (s << ... << parts);
    throw Refusal{s.str()};
}

// f(), its C++ exceptions as Python's.
template <typename F>
PyObject* guarded(F f) {
    HANDLE_TH_ERRORS
    try {
        return f();
    } catch (const Refusal& r) {
        PyErr_SetString(PyExc_ValueError, r.what.c_str());
        return nullptr;
    } catch (const PythonError&) {
        return nullptr;
    }
    END_HANDLE_TH_ERRORS
}

const Tensor& tensor(PyObject* o, const char* name) {
    if (!THPVariable_Check(o)) refuse(name, " must be a tensor");
    return THPVariable_Unpack(o);
}
// A tensor or None.
const Tensor* maybe(PyObject* o, const char* name) { return o == Py_None ? nullptr : &tensor(o, name); }

attn_dtype type_of(const Tensor& t) {
    switch (t.scalar_type()) {
        case at::kFloat: return ATTN_F32;
        case at::kBFloat16: return ATTN_BF16;
        case at::kHalf: return ATTN_F16;
        default: refuse("unsupported dtype ", t.scalar_type());
    }
}

int device_of(const Tensor& t, const char* name) {
    if (!t.is_cuda()) refuse(name, " must be a CUDA tensor");
    return t.get_device();
}

void on_device(const Tensor& t, const char* name, int device) {
    if (!t.is_cuda() || t.get_device() != device) refuse(name, " must be a CUDA tensor on the device of the others");
}

// The library launches on the current device.
void current(int device) {
    const int now = c10::cuda::current_device();
    if (now != device)
        refuse("tensors are on cuda:", device, " but the current device is cuda:", now,
               "; call under torch.cuda.device(", device, ")");
}

// The stream a call runs on: the given handle, or torch's current one.  While this
// lives it is torch's current stream, so that new outputs come out of its own memory:
// torch's allocator orders the reuse of a block by the stream it was asked for on, and
// one freed by the caller's current stream may still be in use there.
struct OnStream {
    cudaStream_t stream;
    std::optional<c10::cuda::CUDAStreamGuard> guard;
    OnStream(PyObject* o, int device) {
        const auto index = static_cast<c10::DeviceIndex>(device);
        if (o == Py_None) {
            stream = c10::cuda::getCurrentCUDAStream(index).stream();
            return;
        }
        void* p = PyLong_AsVoidPtr(o);
        if (PyErr_Occurred()) throw PythonError{};
        stream = static_cast<cudaStream_t>(p);
        guard.emplace(p ? c10::cuda::getStreamFromExternal(stream, index) : c10::cuda::getDefaultCUDAStream(index));
    }
};

// A contiguous tensor of this type and shape on the device.
void exact(const Tensor& t, const char* name, at::ScalarType type, at::IntArrayRef shape, int device) {
    if (t.scalar_type() != type || t.sizes() != shape || !t.is_contiguous())
        refuse(name, " must be a contiguous ", type, " tensor ", shape, " (got ", t.scalar_type(), " ", t.sizes(), ")");
    on_device(t, name, device);
}
const int* ints(const Tensor& t, const char* name, at::IntArrayRef shape, int device) {
    exact(t, name, at::kInt, shape, device);
    return t.data_ptr<int>();
}

void last_dim(const Tensor& t, const char* name) {
    if (t.stride(-1) != 1 && t.size(-1) > 1) refuse(name, "'s last dimension must be contiguous");
}

int as_int(int64_t n, const char* what) {
    if (n > 0x7fffffff) refuse(what, " must fit in 31 bits (got ", n, ")");
    return static_cast<int>(n);
}

// x, [T, H, D] or [B, H, T, D], with the tokens, head dim and type of `like`.
attn_rows rows_in(const char* name, const Tensor& x, const Tensor& like, int device) {
    on_device(x, name, device);
    if (x.scalar_type() != like.scalar_type()) refuse(name, " must be ", like.scalar_type(), " (got ", x.scalar_type(), ")");
    const auto n = x.dim();
    if (n != like.dim() || x.size(0) != like.size(0) || x.size(-1) != like.size(-1) ||
        (n == 4 && x.size(2) != like.size(2)))
        refuse(name, " must have the tokens and head dim of the others (got ", x.sizes(), ")");
    last_dim(x, name);
    attn_rows r{};
    r.x = x.data_ptr();
    r.heads = as_int(x.size(1), "heads");
    r.x_head = x.stride(1);
    r.x_token = x.stride(n == 3 ? 0 : 2);
    r.x_batch = n == 3 ? 0 : x.stride(0);
    return r;
}

// A new contiguous tensor from torch's CUDA allocator (at::empty without the
// dispatcher: these calls are not traced).
Tensor fresh(at::IntArrayRef shape, at::ScalarType type, const Tensor& like) {
    return Tensor(at::detail::empty_cuda(shape, type, like.device(), std::nullopt));
}

// The output of x: the caller's, or a new tensor.
Tensor rows_out(const char* name, const Tensor& x, const Tensor* given, attn_rows& r) {
    Tensor out;
    if (given) {
        out = *given;
        if (out.sizes() != x.sizes() || out.scalar_type() != x.scalar_type() || out.device() != x.device())
            refuse("out_", name, " must be ", x.sizes(), " ", x.scalar_type(), " on ", x.device());
        last_dim(out, name);
    } else {
        out = fresh(x.sizes(), x.scalar_type(), x);
    }
    const auto n = out.dim();
    r.y = out.data_ptr();
    r.y_head = out.stride(1);
    r.y_token = out.stride(n == 3 ? 0 : 2);
    r.y_batch = n == 3 ? 0 : out.stride(0);
    return out;
}

// What rotation() makes, as a bytes object; the caller keeps the table alive.
struct Rotation {
    attn_rotation r;
    int device;
};

// The call's rotation, or null for None.
struct RotationArg {
    Rotation held;
    const attn_rotation* r = nullptr;
    RotationArg(PyObject* o, int device) {
        if (o == Py_None) return;
        if (!PyBytes_Check(o) || PyBytes_GET_SIZE(o) != static_cast<Py_ssize_t>(sizeof(Rotation)))
            refuse("rotation must be a Rotation");
        std::memcpy(&held, PyBytes_AS_STRING(o), sizeof(held));
        if (held.device != device) refuse("the rotation's table must be on the device of the tensors");
        r = &held.r;
    }
};

PyObject* failed(attn_status st) {
    PyObject* e = PyObject_CallFunction(g_error, "is", static_cast<int>(st), attn_last_error());
    if (e) {
        PyErr_SetObject(g_error, e);
        Py_DECREF(e);
    }
    return nullptr;
}

PyObject* wrapped(const std::optional<Tensor>& t) {
    if (t) return THPVariable_Wrap(*t);
    Py_RETURN_NONE;
}
PyObject* two(const std::optional<Tensor>& a, const std::optional<Tensor>& b) {
    PyObject* x = wrapped(a);
    PyObject* y = x ? wrapped(b) : nullptr;
    PyObject* r = y ? PyTuple_Pack(2, x, y) : nullptr;
    Py_XDECREF(x);
    Py_XDECREF(y);
    return r;
}

void arguments(Py_ssize_t n, Py_ssize_t want) {
    if (n != want) refuse(want, " arguments wanted, ", n, " given");
}

// rotation(turns, interleaved, magnitude) -> bytes
PyObject* rotation(PyObject* const* a, Py_ssize_t n) {
    arguments(n, 3);
    const Tensor& turns = tensor(a[0], "turns");
    if (turns.scalar_type() != at::kLong || turns.dim() != 1 || !turns.is_contiguous())
        refuse("turns must be a contiguous int64 tensor [rot_dim / 2]");
    Rotation o;
    std::memset(&o, 0, sizeof(o));
    o.device = device_of(turns, "turns");
    o.r.turns = static_cast<const unsigned long long*>(turns.data_ptr());
    o.r.rot_dim = as_int(2 * turns.size(0), "rot_dim");
    o.r.interleaved = a[1] == Py_True ? 1 : 0;
    const double m = PyFloat_AsDouble(a[2]);
    if (PyErr_Occurred()) throw PythonError{};
    o.r.magnitude = static_cast<float>(m);
    return PyBytes_FromStringAndSize(reinterpret_cast<const char*>(&o), sizeof(o));
}

// rope(q, k, positions, rotation, out_q, out_k, stream, norm, q_weight, k_weight, eps)
//   -> (out_q, out_k)
PyObject* rope(PyObject* const* a, Py_ssize_t n) {
    arguments(n, 11);
    const Tensor& q = tensor(a[0], "q");
    const Tensor* k = maybe(a[1], "k");
    const Tensor& positions = tensor(a[2], "positions");
    const Tensor *given_q = maybe(a[4], "out_q"), *given_k = maybe(a[5], "out_k");
    const bool norm = a[7] == Py_True;
    const attn_dtype type = type_of(q);
    const int device = device_of(q, "q");
    if (q.dim() != 3 && q.dim() != 4) refuse("q must be [T, H, D] or [B, H, T, D] (got ", q.sizes(), ")");
    const int64_t B = q.dim() == 3 ? 1 : q.size(0), T = q.size(q.dim() == 3 ? 0 : 2), D = q.size(-1);
    if (!k && given_k) refuse("out_k without k");
    attn_rows rq = rows_in("q", q, q, device), rk{};
    if (k) rk = rows_in("k", *k, q, device);
    const int* pos = q.dim() == 3 ? ints(positions, "positions", {T}, device) : ints(positions, "positions", {B, T}, device);
    const RotationArg rotation(a[3], device);
    const void* weight[2] = {nullptr, nullptr};
    double eps = 0.0;
    if (norm) {
        for (int i = 0; i < 2; ++i) {
            const char* name = i ? "k_weight" : "q_weight";
            if (const Tensor* w = maybe(a[8 + i], name)) {
                exact(*w, name, q.scalar_type(), {D}, device);
                weight[i] = w->data_ptr();
            }
        }
        eps = PyFloat_AsDouble(a[10]);
        if (PyErr_Occurred()) throw PythonError{};
    }
    current(device);
    const OnStream on(a[6], device);
    const Tensor yq = rows_out("q", q, given_q, rq);
    std::optional<Tensor> yk;
    if (k) yk = rows_out("k", *k, given_k, rk);
    const int b = as_int(B, "B"), t = as_int(T, "T"), d = as_int(D, "D");
    attn_status st;
    Py_BEGIN_ALLOW_THREADS
    st = norm ? attn_qk_norm_rope(&rq, k ? &rk : nullptr, weight[0], weight[1], static_cast<float>(eps), pos, b, t, d,
                                  rotation.r, type, on.stream)
              : attn_rope(&rq, k ? &rk : nullptr, pos, b, t, d, rotation.r, type, on.stream);
    Py_END_ALLOW_THREADS
    return st == ATTN_OK ? two(yq, yk) : failed(st);
}

// A paged cache's pool: 16-bit rows of `type`, e4m3 codes (scales: float32 for each block, K
// or V, and head), or e2m1 codes in pairs (scales: e4m3 for each 16 elements of a row; factors:
// float32 [2, Hkv] or none).
enum class Held { k16, kE4m3, kE2m1 };
struct Pool {
    int64_t blocks, Hkv, page, D;
    void* cache;
    void* scales = nullptr;
    const float* factors = nullptr;
    // heads: the KV heads there have to be, 0: any.  D: the head dim, 0: the cache's.
    Pool(Held held, const Tensor& t, const Tensor* s, const Tensor* f, at::ScalarType type, int64_t heads, int64_t dim,
         int device) {
        const at::ScalarType kind = held == Held::k16 ? type : held == Held::kE4m3 ? at::kFloat8_e4m3fn : at::kByte;
        const int64_t per = held == Held::kE2m1 ? 2 : 1;
        if (t.dim() != 5 || t.scalar_type() != kind || t.size(1) != 2 || (heads && t.size(2) != heads) ||
            (dim && t.size(4) * per != dim) || !t.is_contiguous()) {
            std::ostringstream shape;
            shape << "[num_blocks, 2, ";
            if (heads) shape << heads; else shape << "Hkv";
            shape << ", page_size, ";
            if (dim) shape << dim / per; else shape << (per == 2 ? "D / 2" : "D");
            refuse("kv_cache must be a contiguous ", kind, " tensor ", shape.str(), "] (got ", t.scalar_type(), " ", t.sizes(), ")");
        }
        on_device(t, "kv_cache", device);
        blocks = t.size(0);
        Hkv = t.size(2);
        page = t.size(3);
        D = t.size(4) * per;
        cache = t.data_ptr();
        if (held == Held::kE4m3) {
            exact(*s, "scales", at::kFloat, {blocks, 2, Hkv}, device);
            scales = s->data_ptr();
        }
        if (held == Held::kE2m1) {
            exact(*s, "scales", at::kFloat8_e4m3fn, {blocks, 2, Hkv, page, D / 16}, device);
            scales = s->data_ptr();
            if (f) {
                exact(*f, "factors", at::kFloat, {2, Hkv}, device);
                factors = f->data_ptr<float>();
            }
        }
    }
};

// The weights of a pool's slots.
float* weights_of(const Tensor& w, const Pool& pool, int device) {
    exact(w, "weights", at::kFloat, {pool.blocks, pool.Hkv, pool.page}, device);
    return w.data_ptr<float>();
}

// append(k, v, kv_cache, scales, block_table, cu_seqlens, seq_lens, rotation, positions, q, out_q,
//        out_k, stream, factors, four) -> (out_q, out_k)
PyObject* append(PyObject* const* a, Py_ssize_t n) {
    arguments(n, 15);
    const Tensor &k = tensor(a[0], "k"), &v = tensor(a[1], "v"), &cache = tensor(a[2], "kv_cache");
    const Tensor* scales = maybe(a[3], "scales");
    const Tensor &table = tensor(a[4], "block_table"), &cu = tensor(a[5], "cu_seqlens"), &lens = tensor(a[6], "seq_lens");
    const Tensor *positions = maybe(a[8], "positions"), *q = maybe(a[9], "q");
    const Tensor *given_q = maybe(a[10], "out_q"), *given_k = maybe(a[11], "out_k");
    if (k.scalar_type() != at::kBFloat16 && k.scalar_type() != at::kHalf)
        refuse("the paged append takes bf16 or fp16 tensors");
    const int device = device_of(k, "k");
    if (k.dim() != 3) refuse("k must be [total, Hkv, D] (got ", k.sizes(), ")");
    const int64_t total = k.size(0), Hkv = k.size(1), D = k.size(2);
    attn_rows rk = rows_in("k", k, k, device), rv = rows_in("v", v, k, device), rq{};
    if (v.size(1) != Hkv) refuse("k and v must have the same heads");
    if (q) rq = rows_in("q", *q, k, device);
    else if (given_q) refuse("out_q without q");
    const Tensor* factors = maybe(a[13], "factors");
    const Held held = !scales ? Held::k16 : a[14] == Py_True ? Held::kE2m1 : Held::kE4m3;
    const Pool pool(held, cache, scales, factors, k.scalar_type(), Hkv, D, device);
    if (table.dim() != 2) refuse("block_table must be [B, max_pages]");
    const int64_t B = table.size(0), pages = table.size(1);
    const int* table_p = ints(table, "block_table", {B, pages}, device);
    const int* lens_p = ints(lens, "seq_lens", {B}, device);
    const int* cu_p = ints(cu, "cu_seqlens", {B + 1}, device);
    const int* pos_p = positions ? ints(*positions, "positions", {total}, device) : nullptr;
    const RotationArg rotation(a[7], device);
    current(device);
    const OnStream on(a[12], device);
    std::optional<Tensor> yq, yk;
    if (q) yq = rows_out("q", *q, given_q, rq);
    if (given_k) yk = rows_out("k", k, given_k, rk);
    const int b = as_int(B, "B"), t = as_int(total, "total"), d = as_int(D, "D"), p = as_int(pool.page, "page_size");
    const int w = as_int(pages, "max_pages"), nb = as_int(pool.blocks, "num_blocks");
    const attn_dtype type = type_of(k);
    attn_status st;
    Py_BEGIN_ALLOW_THREADS
    if (held == Held::kE2m1)
        st = attn_append_paged_e2m1(q ? &rq : nullptr, &rk, &rv, cu_p, lens_p, pos_p, table_p, pool.cache, pool.scales,
                                    pool.factors, b, t, d, p, w, nb, rotation.r, type, on.stream);
    else if (held == Held::kE4m3)
        st = attn_append_paged_e4m3(q ? &rq : nullptr, &rk, &rv, cu_p, lens_p, pos_p, table_p, pool.cache,
                                    static_cast<float*>(pool.scales), b, t, d, p, w, nb, rotation.r, type, on.stream);
    else
        st = attn_append_paged(q ? &rq : nullptr, &rk, &rv, cu_p, lens_p, pos_p, table_p, pool.cache, b, t, d, p, w, nb,
                               rotation.r, type, on.stream);
    Py_END_ALLOW_THREADS
    return st == ATTN_OK ? two(yq, yk) : failed(st);
}

// decode(q, kv_cache, scales, block_table, seq_lens, scale, out, lse, want_lse, stream, factors, weights, four)
//   -> (out, lse); scale None: 1 / sqrt(D)
PyObject* decode(PyObject* const* a, Py_ssize_t n) {
    arguments(n, 13);
    const Tensor &q = tensor(a[0], "q"), &cache = tensor(a[1], "kv_cache"), &scales = tensor(a[2], "scales");
    const Tensor &table = tensor(a[3], "block_table"), &lens = tensor(a[4], "seq_lens");
    const Tensor *given = maybe(a[6], "out"), *given_lse = maybe(a[7], "lse");
    const Tensor *factors = maybe(a[10], "factors"), *weights = maybe(a[11], "weights");
    const bool four = a[12] == Py_True;
    if (!q.is_cuda() || q.dim() != 4 || q.size(2) != 1 || !q.is_contiguous() ||
        (q.scalar_type() != at::kBFloat16 && q.scalar_type() != at::kHalf))
        refuse("q must be a contiguous bf16 or fp16 CUDA tensor [B, Hq, 1, D]");
    const int device = q.get_device();
    const int64_t B = q.size(0), Hq = q.size(1), D = q.size(3);
    const Pool pool(four ? Held::kE2m1 : Held::kE4m3, cache, &scales, factors, q.scalar_type(), 0, D, device);
    float* weights_p = weights ? weights_of(*weights, pool, device) : nullptr;
    if (table.dim() != 2) refuse("block_table must be [B, max_pages]");
    const int64_t pages = table.size(1);
    const int* table_p = ints(table, "block_table", {B, pages}, device);
    const int* lens_p = ints(lens, "seq_lens", {B}, device);
    double scale = 1.0 / std::sqrt(static_cast<double>(D));
    if (a[5] != Py_None) {
        scale = PyFloat_AsDouble(a[5]);
        if (PyErr_Occurred()) throw PythonError{};
    }
    current(device);
    const OnStream on(a[9], device);
    // The caller's buffers hold exactly what is written: [B, Hq, 1] serves [B, Hq].
    if (given) {
        if (given->scalar_type() != q.scalar_type() || given->numel() != q.numel() || !given->is_contiguous())
            refuse("out must hold ", q.sizes(), " = ", q.numel(), " contiguous elements of ", q.scalar_type());
        on_device(*given, "out", device);
    }
    if (given_lse) {
        if (given_lse->scalar_type() != at::kFloat || given_lse->numel() != B * Hq || !given_lse->is_contiguous())
            refuse("lse must hold [", B, ", ", Hq, "] = ", B * Hq, " contiguous float32 elements");
        on_device(*given_lse, "lse", device);
    }
    const Tensor out = given ? *given : fresh(q.sizes(), q.scalar_type(), q);
    std::optional<Tensor> lse;
    if (given_lse) lse = *given_lse;
    else if (a[8] == Py_True) lse = fresh({B, Hq}, at::kFloat, q);
    const int b = as_int(B, "B"), hq = as_int(Hq, "Hq"), hkv = as_int(pool.Hkv, "Hkv"), d = as_int(D, "D");
    const int p = as_int(pool.page, "page_size"), w = as_int(pages, "max_pages"), nb = as_int(pool.blocks, "num_blocks");
    const attn_dtype type = type_of(q);
    const void* q_p = q.data_ptr();
    void* out_p = out.data_ptr();
    float* lse_p = lse ? lse->data_ptr<float>() : nullptr;
    attn_status st;
    Py_BEGIN_ALLOW_THREADS
    if (four)
        st = attn_fwd_decode_paged_e2m1(q_p, pool.cache, pool.scales, pool.factors, table_p, lens_p, out_p, lse_p,
                                        weights_p, b, hq, hkv, d, p, w, nb, static_cast<float>(scale), type, on.stream);
    else
        st = attn_fwd_decode_paged_e4m3(q_p, pool.cache, static_cast<const float*>(pool.scales), table_p, lens_p, out_p,
                                        lse_p, b, hq, hkv, d, p, w, nb, static_cast<float>(scale), type, on.stream);
    Py_END_ALLOW_THREADS
    return st == ATTN_OK ? two(out, lse) : failed(st);
}

// add_weights(q, lse, kv_cache, scales, block_table, cu_seqlens, seq_lens, weights, scale, factors, stream) -> weights
PyObject* add_weights(PyObject* const* a, Py_ssize_t n) {
    arguments(n, 11);
    const Tensor &q = tensor(a[0], "q"), &lse = tensor(a[1], "lse"), &cache = tensor(a[2], "kv_cache");
    const Tensor* scales = maybe(a[3], "scales");
    const Tensor &table = tensor(a[4], "block_table"), &cu = tensor(a[5], "cu_seqlens"), &lens = tensor(a[6], "seq_lens");
    const Tensor& weights = tensor(a[7], "weights");
    const Tensor* factors = maybe(a[9], "factors");
    if (q.scalar_type() != at::kBFloat16 && q.scalar_type() != at::kHalf)
        refuse("the weights of a paged cache take bf16 or fp16 queries");
    const int device = device_of(q, "q");
    if (q.dim() != 3) refuse("q must be [total, Hq, D] (got ", q.sizes(), ")");
    const int64_t total = q.size(0), Hq = q.size(1), D = q.size(2);
    attn_rows rq = rows_in("q", q, q, device);
    const Pool pool(scales ? Held::kE2m1 : Held::k16, cache, scales, factors, q.scalar_type(), 0, D, device);
    float* weights_p = weights_of(weights, pool, device);
    on_device(lse, "lse", device);
    if (lse.scalar_type() != at::kFloat || lse.dim() != 2 || lse.size(0) != Hq || lse.size(1) != total)
        refuse("lse must be a float32 tensor [", Hq, ", ", total, "] (got ", lse.scalar_type(), " ", lse.sizes(), ")");
    if (table.dim() != 2) refuse("block_table must be [B, max_pages]");
    const int64_t B = table.size(0), pages = table.size(1);
    const int* table_p = ints(table, "block_table", {B, pages}, device);
    const int* lens_p = ints(lens, "seq_lens", {B}, device);
    const int* cu_p = ints(cu, "cu_seqlens", {B + 1}, device);
    double scale = 1.0 / std::sqrt(static_cast<double>(D));
    if (a[8] != Py_None) {
        scale = PyFloat_AsDouble(a[8]);
        if (PyErr_Occurred()) throw PythonError{};
    }
    current(device);
    const OnStream on(a[10], device);
    const int b = as_int(B, "B"), t = as_int(total, "total"), hkv = as_int(pool.Hkv, "Hkv"), d = as_int(D, "D");
    const int p = as_int(pool.page, "page_size"), w = as_int(pages, "max_pages"), nb = as_int(pool.blocks, "num_blocks");
    const attn_dtype type = type_of(q);
    const float* lse_p = lse.data_ptr<float>();
    const long long head = lse.stride(0), token = lse.stride(1);
    attn_status st;
    Py_BEGIN_ALLOW_THREADS
    st = scales ? attn_weights_paged_e2m1(&rq, lse_p, head, token, pool.cache, pool.scales, pool.factors, table_p, cu_p,
                                          lens_p, weights_p, b, t, hkv, d, p, w, nb, static_cast<float>(scale), type,
                                          on.stream)
                : attn_weights_paged(&rq, lse_p, head, token, pool.cache, table_p, cu_p, lens_p, weights_p, b, t, hkv, d,
                                     p, w, nb, static_cast<float>(scale), type, on.stream);
    Py_END_ALLOW_THREADS
    if (st != ATTN_OK) return failed(st);
    Py_INCREF(a[7]);
    return a[7];
}

// evict(kv_cache, scales, weights, block_table, seq_lens, keep, recent, new_lens, kept, want_kept, stream)
//   -> (new_lens, kept)
PyObject* evict(PyObject* const* a, Py_ssize_t n) {
    arguments(n, 11);
    const Tensor& cache = tensor(a[0], "kv_cache");
    const Tensor* scales = maybe(a[1], "scales");
    const Tensor &weights = tensor(a[2], "weights"), &table = tensor(a[3], "block_table"), &lens = tensor(a[4], "seq_lens");
    const Tensor *given_lens = maybe(a[7], "new_lens"), *given_kept = maybe(a[8], "kept");
    const int device = device_of(cache, "kv_cache");
    if (!scales && cache.scalar_type() != at::kBFloat16 && cache.scalar_type() != at::kHalf)
        refuse("the eviction takes bf16 or fp16 caches (got ", cache.scalar_type(), ")");
    const Pool pool(scales ? Held::kE2m1 : Held::k16, cache, scales, nullptr, cache.scalar_type(), 0, 0, device);
    float* weights_p = weights_of(weights, pool, device);
    if (table.dim() != 2) refuse("block_table must be [B, max_pages]");
    const int64_t B = table.size(0), pages = table.size(1);
    const int* table_p = ints(table, "block_table", {B, pages}, device);
    const int* lens_p = ints(lens, "seq_lens", {B}, device);
    const int64_t keep = PyLong_AsLongLong(a[5]), recent = PyLong_AsLongLong(a[6]);
    if (PyErr_Occurred()) throw PythonError{};
    if (keep < 1 || recent < 0 || recent > keep)
        refuse("keep must be >= 1 and recent in 0..keep (got ", keep, ", ", recent, ")");
    const int k = as_int(keep, "keep"), r = as_int(recent, "recent");
    current(device);
    const OnStream on(a[10], device);
    if (given_lens) exact(*given_lens, "new_lens", at::kInt, {B}, device);
    if (given_kept) exact(*given_kept, "kept", at::kInt, {B, pool.Hkv, keep}, device);
    const Tensor new_lens = given_lens ? *given_lens : fresh({B}, at::kInt, cache);
    std::optional<Tensor> kept;
    if (given_kept) kept = *given_kept;
    else if (a[9] == Py_True) kept = fresh({B, pool.Hkv, keep}, at::kInt, cache);
    const int b = as_int(B, "B"), hkv = as_int(pool.Hkv, "Hkv"), d = as_int(pool.D, "D");
    const int p = as_int(pool.page, "page_size"), w = as_int(pages, "max_pages"), nb = as_int(pool.blocks, "num_blocks");
    int* new_p = new_lens.data_ptr<int>();
    int* kept_p = kept ? kept->data_ptr<int>() : nullptr;
    const attn_dtype type = scales ? ATTN_BF16 : type_of(cache);
    attn_status st;
    Py_BEGIN_ALLOW_THREADS
    st = scales ? attn_evict_paged_e2m1(pool.cache, pool.scales, weights_p, table_p, lens_p, new_p, kept_p, b, hkv, d, p,
                                        w, nb, k, r, on.stream)
                : attn_evict_paged(pool.cache, weights_p, table_p, lens_p, new_p, kept_p, b, hkv, d, p, w, nb, k, r, type,
                                   on.stream);
    Py_END_ALLOW_THREADS
    return st == ATTN_OK ? two(new_lens, kept) : failed(st);
}

// set_error(cls): the exception class of a status other than ATTN_OK.
PyObject* set_error(PyObject*, PyObject* cls) {
    Py_INCREF(cls);
    Py_XDECREF(g_error);
    g_error = cls;
    Py_RETURN_NONE;
}

using Call = PyObject* (*)(PyObject* const*, Py_ssize_t);
template <Call kCall>
PyObject* entry(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return guarded([&] { return kCall(a, n); });
}
template <Call kCall>
PyCFunction fast() {
    return reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(&entry<kCall>));
}

PyMethodDef g_methods[] = {
    {"rotation", fast<rotation>(), METH_FASTCALL, nullptr},
    {"rope", fast<rope>(), METH_FASTCALL, nullptr},
    {"append", fast<append>(), METH_FASTCALL, nullptr},
    {"decode", fast<decode>(), METH_FASTCALL, nullptr},
    {"add_weights", fast<add_weights>(), METH_FASTCALL, nullptr},
    {"evict", fast<evict>(), METH_FASTCALL, nullptr},
    {"set_error", set_error, METH_O, nullptr},
    {nullptr, nullptr, 0, nullptr},
};
PyModuleDef g_module = {PyModuleDef_HEAD_INIT, "_attn_binding", nullptr, -1, g_methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__attn_binding() { return PyModule_Create(&g_module); }
