// attention_binding.cpp -- argument marshalling of the attention layer's calls
// (ops.qk_norm_rope, ops.fp8_kv_append, ops.fp8_kv_attention).
//
// A decode step makes these calls for every attention layer and a small one
// takes the GPU a few microseconds, less than reading some sixty tensor
// properties from Python takes the host.  So the checks and the host structs
// of include/nvfp4.h are made here, from the tensors themselves; ops.py fills
// in defaults and allocates outputs.  Every tensor is checked for type, shape,
// strides and device before its address is passed on; the library checks the
// rest (alignment, sizes, null pointers) and its status is returned.
//
// The library's functions are bound by address (bind()), so that this module
// is linked to torch and Python alone.
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <algorithm>
#include <cstdint>
#include <cmath>
#include <exception>
#include <stdexcept>
#include <string>

#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include "nvfp4.h"

namespace {

using NormFn = decltype(&nvfp4_qk_norm_rope);
using AppendFn = decltype(&nvfp4_fp8_kv_append);
using AttendFn = decltype(&nvfp4_fp8_kv_attention);
using BytesFn = decltype(&nvfp4_fp8_kv_attention_workspace_bytes);

struct {
    NormFn norm = nullptr;
    AppendFn append = nullptr;
    AttendFn attend = nullptr;
    BytesFn attend_bytes = nullptr;
    bool any_device = false;  // tests: CPU tensors stand in for device ones
} g;

// A message for ValueError; what a check throws.
struct Refused : std::runtime_error {
    using std::runtime_error::runtime_error;
};

std::string describe(const at::Tensor &t)
{
    std::string s = std::string("got ") + c10::toString(t.scalar_type()) + ", shape [";
    for (int64_t i = 0; i < t.dim(); ++i)
        s += (i ? ", " : "") + std::to_string(t.size(i));
    s += "], strides [";
    for (int64_t i = 0; i < t.dim(); ++i)
        s += (i ? ", " : "") + std::to_string(t.stride(i));
    return s + "], " + t.device().str();
}

[[noreturn]] void refuse(const char *name, const char *what, const at::Tensor &t)
{
    throw Refused(std::string(name) + ' ' + what + " (" + describe(t) + ")");
}

// The tensor of a Python argument; null for None where that is allowed.
const at::Tensor *tensor(PyObject *o, const char *name, bool optional = false)
{
    if (optional && o == Py_None)
        return nullptr;
    if (!THPVariable_Check(o))
        throw Refused(std::string(name) + " must be a tensor");
    return &THPVariable_Unpack(o);
}

// The device of a call: that of its first tensor, which has to be the current one.
struct Call {
    int64_t device = -1;

    void on(const at::Tensor &t, const char *name)
    {
        if (g.any_device)
            return;
        if (!t.is_cuda())
            throw Refused("nvfp4 ops take CUDA tensors only (there is no CPU path)");
        const int64_t d = t.get_device();
        if (device < 0) {
            device = d;
            if (d != c10::cuda::current_device())
                throw Refused(std::string("tensors on ") + t.device().str() + ", but the current device is cuda:" +
                              std::to_string(c10::cuda::current_device()));
        } else if (d != device) {
            refuse(name, "is on another device than the other tensors", t);
        }
    }

    void *stream(PyObject *o) const
    {
        if (o != Py_None) {
            PyObject *v = PyObject_GetAttrString(o, "cuda_stream");
            if (v == nullptr) {
                PyErr_Clear();
                throw Refused("stream must be a torch.cuda.Stream");
            }
            void *p = PyLong_Check(v) ? PyLong_AsVoidPtr(v) : nullptr;
            const bool bad = !PyLong_Check(v) || PyErr_Occurred() != nullptr;
            Py_DECREF(v);
            if (bad) {
                PyErr_Clear();
                throw Refused("stream must be a torch.cuda.Stream");
            }
            return p;
        }
        return g.any_device ? nullptr : c10::cuda::getCurrentCUDAStream(static_cast<c10::DeviceIndex>(device)).stream();
    }

    // Head rows of a bf16 [tokens, heads, head_dim] tensor or view; `written`: no two rows may overlap.
    nvfp4_heads heads(const at::Tensor &t, const char *name, const at::Tensor *like = nullptr, bool written = false)
    {
        if (t.scalar_type() != at::kBFloat16 || t.dim() != 3 || t.stride(2) != 1)
            refuse(name, "must be a bf16 [tokens, heads, head_dim] tensor with unit stride along head_dim", t);
        if (like != nullptr && t.sizes() != like->sizes())
            refuse(name, "has another shape than the tensor it goes with", t);
        on(t, name);
        const int64_t T = t.size(0), H = t.size(1), D = t.size(2);
        const int64_t s0 = T > 1 ? t.stride(0) : 0, s1 = H > 1 ? t.stride(1) : 0;
        const bool by_token = (H <= 1 || s1 >= D) && (T <= 1 || s0 >= (H - 1) * s1 + D);
        const bool by_head = (T <= 1 || s0 >= D) && (H <= 1 || s1 >= (T - 1) * s0 + D);
        if (written && !by_token && !by_head)
            refuse(name, "has rows that overlap", t);
        return nvfp4_heads{t.data_ptr(), s0, s1, H};
    }

    // Address of a contiguous vector of n elements or more (exactly n: `exact`); null for None.
    const void *vector(const at::Tensor *t, const char *name, at::ScalarType type, int64_t n, bool exact = false)
    {
        if (t == nullptr)
            return nullptr;
        if (t->scalar_type() != type || t->dim() != 1 || t->size(0) < n || (exact && t->size(0) != n) ||
            (t->size(0) > 1 && t->stride(0) != 1))
            refuse(name, (std::string("must be a contiguous ") + c10::toString(type) + " vector of " +
                          (exact ? "" : "at least ") + std::to_string(n)).c_str(), *t);
        on(*t, name);
        return t->data_ptr();
    }

    const float *scalar(const at::Tensor &t, const char *name)
    {
        if (t.scalar_type() != at::kFloat || t.numel() != 1)
            refuse(name, "must hold one fp32 value", t);
        on(t, name);
        return static_cast<const float *>(t.data_ptr());
    }

    nvfp4_norm_rope norm_rope(int64_t head_dim, const at::Tensor *inv_freq, const at::Tensor *q_weight,
                              const at::Tensor *k_weight, double eps, bool plus_one)
    {
        nvfp4_norm_rope n;
        n.q_weight = vector(q_weight, "q_weight", at::kBFloat16, head_dim, true);
        n.k_weight = vector(k_weight, "k_weight", at::kBFloat16, head_dim, true);
        n.inv_freq = static_cast<const float *>(vector(inv_freq, "inv_freq", at::kFloat, 0));
        n.rotary_dim = 0;
        if (inv_freq != nullptr) {
            if (inv_freq->size(0) > 1024)
                refuse("inv_freq", "has too many frequencies", *inv_freq);
            n.rotary_dim = static_cast<int32_t>(2 * inv_freq->size(0));
        }
        n.eps = static_cast<float>(eps);
        n.flags = plus_one ? NVFP4_NORM_PLUS_ONE : 0;
        return n;
    }

    // Byte strides of pages, rows and heads; a dimension of one element gets a stride that nests with the others
    // (torch leaves it arbitrary).
    static void page_strides(const at::Tensor &t, int64_t &page, int64_t &row, int64_t &head)
    {
        row = t.stride(1);
        head = t.size(2) > 1 ? t.stride(2) : row;
        page = t.size(0) > 1 ? t.stride(0) : std::max(row * t.size(1), head * t.size(2));
    }

    nvfp4_kv_pages pages(const at::Tensor &k, const at::Tensor &v, const at::Tensor &k_scale, const at::Tensor &v_scale)
    {
        for (const at::Tensor *t : {&k, &v})
            if (t->scalar_type() != at::kByte || t->dim() != 4 || t->stride(3) != 1 || t->sizes() != k.sizes())
                refuse(t == &k ? "k_pages" : "v_pages",
                       "must be a uint8 [pages, page_size, kv_heads, head_dim] tensor with unit stride along head_dim, of "
                       "the other's shape", *t);
        on(k, "k_pages");
        on(v, "v_pages");
        for (int i = 1; i < 4; ++i)
            if (k.size(i) > (1 << 20))
                refuse("k_pages", "is too large", k);
        nvfp4_kv_pages p;
        p.k_pages = k.data_ptr();
        p.v_pages = v.data_ptr();
        p.k_scale = scalar(k_scale, "k_scale");
        p.v_scale = scalar(v_scale, "v_scale");
        page_strides(k, p.k_page_stride, p.k_token_stride, p.k_head_stride);
        page_strides(v, p.v_page_stride, p.v_token_stride, p.v_head_stride);
        p.num_pages = k.size(0);
        p.page_size = static_cast<int32_t>(k.size(1));
        p.kv_heads = static_cast<int32_t>(k.size(2));
        p.head_dim = static_cast<int32_t>(k.size(3));
        return p;
    }

    nvfp4_kv_batch batch(const at::Tensor &table, const at::Tensor &cu, const at::Tensor &lens)
    {
        if (table.scalar_type() != at::kInt || table.dim() != 2 || (table.size(1) > 1 && table.stride(1) != 1) ||
            table.size(0) >= INT32_MAX || table.size(1) > INT32_MAX)
            refuse("page_table", "must be an int32 [sequences, pages] tensor with unit stride along pages", table);
        on(table, "page_table");
        nvfp4_kv_batch b;
        b.page_table = static_cast<const int32_t *>(table.data_ptr());
        b.cu_tokens = static_cast<const int32_t *>(vector(&cu, "cu_tokens", at::kInt, table.size(0) + 1));
        b.seq_lens = static_cast<const int32_t *>(vector(&lens, "seq_lens", at::kInt, table.size(0)));
        b.table_stride = table.size(0) > 1 ? table.stride(0) : table.size(1);
        b.num_seqs = static_cast<int32_t>(table.size(0));
        b.max_pages = static_cast<int32_t>(table.size(1));
        return b;
    }
};

double number(PyObject *o, const char *name)
{
    const double v = PyFloat_AsDouble(o);
    if (v == -1.0 && PyErr_Occurred()) {
        PyErr_Clear();
        throw Refused(std::string(name) + " must be a number");
    }
    return v;
}

bool truth(PyObject *o, const char *name)
{
    const int v = PyObject_IsTrue(o);
    if (v < 0) {
        PyErr_Clear();
        throw Refused(std::string(name) + " must be true or false");
    }
    return v != 0;
}

// Runs a call with C++ exceptions turned into Python's.
template <typename F>
PyObject *guarded(const char *name, Py_ssize_t got, Py_ssize_t want, F f)
{
    if (got != want) {
        PyErr_Format(PyExc_TypeError, "%s takes %zd arguments (got %zd)", name, want, got);
        return nullptr;
    }
    try {
        return PyLong_FromLong(f());
    } catch (const Refused &e) {
        PyErr_SetString(PyExc_ValueError, e.what());
    } catch (const std::exception &e) {
        PyErr_SetString(PyExc_RuntimeError, e.what());
    }
    return nullptr;
}

template <typename F>
int without_gil(F f)
{
    int rc;
    Py_BEGIN_ALLOW_THREADS
    rc = f();
    Py_END_ALLOW_THREADS
    return rc;
}

// q, k, positions, inv_freq, q_weight, k_weight, eps, plus_one, q_out, k_out, stream
PyObject *norm_rope(PyObject *, PyObject *const *a, Py_ssize_t n)
{
    return guarded("qk_norm_rope", n, 11, [&] {
        Call c;
        const at::Tensor &q = *tensor(a[0], "q"), &q_out = *tensor(a[8], "q_out");
        const at::Tensor *k = tensor(a[1], "k", true), *k_out = tensor(a[9], "k_out", true);
        const at::Tensor *positions = tensor(a[2], "positions", true), *inv_freq = tensor(a[3], "inv_freq", true);
        const nvfp4_heads hq = c.heads(q, "q"), hqo = c.heads(q_out, "q_out", &q, true);
        nvfp4_heads hk{}, hko{};
        if ((k == nullptr) != (k_out == nullptr))
            throw Refused("k and k_out go together");
        if (k != nullptr) {
            hk = c.heads(*k, "k");
            if (k->size(0) != q.size(0) || k->size(2) != q.size(2))
                refuse("k", "has other tokens or another head_dim than q", *k);
            hko = c.heads(*k_out, "k_out", k, true);
        }
        if (inv_freq != nullptr && positions == nullptr)
            throw Refused("a rotation needs positions");
        const nvfp4_norm_rope nr = c.norm_rope(q.size(2), inv_freq, tensor(a[4], "q_weight", true),
                                               tensor(a[5], "k_weight", true), number(a[6], "eps"), truth(a[7], "plus_one"));
        const auto *pos = static_cast<const int32_t *>(c.vector(positions, "positions", at::kInt, q.size(0)));
        void *stream = c.stream(a[10]);
        return without_gil([&] {
            return g.norm(&hq, k != nullptr ? &hk : nullptr, &hqo, k != nullptr ? &hko : nullptr, q.size(0), q.size(2), pos, &nr,
                          stream);
        });
    });
}

// k, v, k_pages, v_pages, k_scale, v_scale, page_table, cu_tokens, seq_lens, inv_freq, k_weight, eps, plus_one, positions, stream
PyObject *append(PyObject *, PyObject *const *a, Py_ssize_t n)
{
    return guarded("fp8_kv_append", n, 15, [&] {
        Call c;
        const at::Tensor &k = *tensor(a[0], "k"), &v = *tensor(a[1], "v");
        const nvfp4_heads hk = c.heads(k, "k"), hv = c.heads(v, "v", &k);
        const at::Tensor &kp = *tensor(a[2], "k_pages");
        const nvfp4_kv_pages pages = c.pages(kp, *tensor(a[3], "v_pages"), *tensor(a[4], "k_scale"), *tensor(a[5], "v_scale"));
        if (k.size(1) != kp.size(2) || k.size(2) != kp.size(3))
            refuse("k", "has other heads or another head_dim than the pages", k);
        const nvfp4_kv_batch batch = c.batch(*tensor(a[6], "page_table"), *tensor(a[7], "cu_tokens"), *tensor(a[8], "seq_lens"));
        const nvfp4_norm_rope nr = c.norm_rope(k.size(2), tensor(a[9], "inv_freq", true), nullptr,
                                               tensor(a[10], "k_weight", true), number(a[11], "eps"), truth(a[12], "plus_one"));
        const auto *pos =
            static_cast<const int32_t *>(c.vector(tensor(a[13], "positions", true), "positions", at::kInt, k.size(0)));
        void *stream = c.stream(a[14]);
        return without_gil([&] { return g.append(&hk, &hv, k.size(0), &pages, &batch, pos, &nr, stream); });
    });
}

// q, k_pages, v_pages, k_scale, v_scale, page_table, cu_tokens, seq_lens, softmax_scale, gate, out, out_amax, ws, single_tokens, stream
PyObject *attend(PyObject *, PyObject *const *a, Py_ssize_t n)
{
    return guarded("fp8_kv_attention", n, 15, [&] {
        Call c;
        const at::Tensor &q = *tensor(a[0], "q"), &out = *tensor(a[10], "out"), &ws = *tensor(a[12], "ws");
        const at::Tensor *gate = tensor(a[9], "gate", true), *amax = tensor(a[11], "out_amax", true);
        const nvfp4_heads hq = c.heads(q, "q");
        const at::Tensor &kp = *tensor(a[1], "k_pages");
        const nvfp4_kv_pages pages = c.pages(kp, *tensor(a[2], "v_pages"), *tensor(a[3], "k_scale"), *tensor(a[4], "v_scale"));
        if (q.size(2) != kp.size(3) || kp.size(2) == 0 || q.size(1) % kp.size(2) != 0)
            refuse("q", "has heads that the pages' do not divide, or another head_dim", q);
        const nvfp4_kv_batch batch = c.batch(*tensor(a[5], "page_table"), *tensor(a[6], "cu_tokens"), *tensor(a[7], "seq_lens"));
        nvfp4_heads hg{};
        if (gate != nullptr)
            hg = c.heads(*gate, "gate", &q);
        const nvfp4_heads ho = c.heads(out, "out", &q, true);
        // CTAs read an item's queries while others write its results
        if (out.numel() > 0 && (ho.data == hq.data || ho.data == hg.data))
            refuse("out", "must not be q or the gate", out);
        if (!ws.is_contiguous())
            refuse("ws", "must be contiguous", ws);
        if (ws.nbytes() < g.attend_bytes(q.size(0), hq.heads, pages.kv_heads, q.size(2)))
            refuse("ws", "is smaller than fp8_kv_attention_workspace_bytes()", ws);
        c.on(ws, "ws");
        if (amax != nullptr) {
            if (!amax->is_contiguous() || amax->nbytes() < 4)
                refuse("out_amax", "must be contiguous and hold 4 bytes", *amax);
            c.on(*amax, "out_amax");
        }
        const nvfp4_attention_opts opts{
            static_cast<float>(a[8] == Py_None ? 1.0 / std::sqrt(static_cast<double>(q.size(2))) : number(a[8], "softmax_scale")),
            truth(a[13], "single_tokens") ? NVFP4_SINGLE_TOKENS : 0u};
        void *stream = c.stream(a[14]);
        return without_gil([&] {
            return g.attend(&hq, gate != nullptr ? &hg : nullptr, &ho, q.size(0), &pages, &batch, &opts,
                            amax != nullptr ? static_cast<uint32_t *>(amax->data_ptr()) : nullptr, ws.data_ptr(), ws.nbytes(), stream);
        });
    });
}

// Addresses of the library's functions; any_device (tests): no device checks, the null stream.
PyObject *bind(PyObject *, PyObject *args)
{
    unsigned long long norm_, append_, attend_, bytes_;
    int any;
    if (!PyArg_ParseTuple(args, "KKKKp", &norm_, &append_, &attend_, &bytes_, &any))
        return nullptr;
    g.norm = reinterpret_cast<NormFn>(static_cast<uintptr_t>(norm_));
    g.append = reinterpret_cast<AppendFn>(static_cast<uintptr_t>(append_));
    g.attend = reinterpret_cast<AttendFn>(static_cast<uintptr_t>(attend_));
    g.attend_bytes = reinterpret_cast<BytesFn>(static_cast<uintptr_t>(bytes_));
    g.any_device = any != 0;
    Py_RETURN_NONE;
}

PyMethodDef methods[] = {
    {"bind", bind, METH_VARARGS, "bind(norm, append, attend, attend_workspace_bytes, any_device)"},
    {"qk_norm_rope", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(norm_rope)), METH_FASTCALL, nullptr},
    {"fp8_kv_append", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(append)), METH_FASTCALL, nullptr},
    {"fp8_kv_attention", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(attend)), METH_FASTCALL, nullptr},
    {nullptr, nullptr, 0, nullptr}};

PyModuleDef module = {PyModuleDef_HEAD_INIT, "_attention", "Argument marshalling of the attention layer's calls.", -1,
                      methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__attention() { return PyModule_Create(&module); }
