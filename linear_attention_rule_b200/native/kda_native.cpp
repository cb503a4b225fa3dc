// Argument marshalling of the calls of a decode step, whose kernels take a few microseconds: through
// ctypes a call took 16 to 20 us of host time, here 3.6 (an append) to 7.2 (a pool's step), launch included.
// The functions check torch tensors, take their pointers and call libkda's C entry points, whose
// addresses init() is given; they return the status.  No computation, no fallback.
#include <torch/csrc/autograd/python_variable.h>

#include <ATen/core/Tensor.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>

#include <cmath>
#include <string>

#include "libkda.h"

namespace {

struct PyError {};   // a Python exception is set

decltype(&kda_decode_pool) g_pool = nullptr;
decltype(&kda_kv_append) g_append = nullptr;
decltype(&kda_kv_decode) g_decode = nullptr;

std::string text(c10::IntArrayRef s) {
    std::string r = "(";
    for (size_t i = 0; i < s.size(); ++i) r += (i ? ", " : "") + std::to_string(s[i]);
    return r + (s.size() == 1 ? ",)" : ")");
}
[[noreturn]] void fail(PyObject* type, const std::string& what) {
    PyErr_SetString(type, what.c_str());
    throw PyError();
}

const at::Tensor& tensor(PyObject* o, const char* name) {
    if (!THPVariable_Check(o)) fail(PyExc_TypeError, std::string(name) + " must be a torch.Tensor");
    return THPVariable_Unpack(o);
}
void check_type(const at::Tensor& t, const char* name, at::ScalarType type) {
    if (t.scalar_type() != type)
        fail(PyExc_TypeError, std::string(name) + " must be " + c10::toString(type) + ", got " + c10::toString(t.scalar_type()));
}
void check_shape(const at::Tensor& t, const char* name, c10::IntArrayRef shape) {
    if (t.sizes() != shape) fail(PyExc_ValueError, std::string(name) + " must have shape " + text(shape) + ", got " + text(t.sizes()));
}
// The tensors of a call.  Types and shapes are looked at first, then that all are on one device.
struct Call {
    c10::Device dev;
    int count = 0;
    const at::Tensor* tensors[20];
    const char* names[20];

    explicit Call(const c10::Device& d) : dev(d) {}
    void add(const at::Tensor& t, const char* name) {
        tensors[count] = &t;
        names[count++] = name;
    }
    void check() const {
        for (int i = 0; i < count; ++i)
            if (tensors[i]->device() != dev || !dev.is_cuda())
                fail(PyExc_ValueError, std::string(names[i]) + " must be on " + (dev.is_cuda() ? dev.str() : "a GPU") +
                                           " (libkda takes device pointers), got " + tensors[i]->device().str());
    }
};
void* data(const at::Tensor& t) { return t.mutable_data_ptr(); }

// A dense argument (None: null).
void* dense(Call& call, const char* name, PyObject* o, c10::IntArrayRef shape, at::ScalarType type) {
    if (o == Py_None) return nullptr;
    const at::Tensor& t = tensor(o, name);
    check_type(t, name, type);
    check_shape(t, name, shape);
    if (!t.is_contiguous()) fail(PyExc_ValueError, std::string(name) + " must be contiguous");
    call.add(t, name);
    return data(t);
}
void* needed(Call& call, const char* name, PyObject* o, c10::IntArrayRef shape, at::ScalarType type) {
    if (o == Py_None) fail(PyExc_TypeError, std::string(name) + " must be a torch.Tensor");
    return dense(call, name, o, shape, type);
}
// q, k or v [tokens, heads, D]: heads and channels dense, tokens apart as they are (a slice of a
// fused projection).
void* rows(Call& call, const char* name, PyObject* o, c10::IntArrayRef shape, at::ScalarType type, int64_t* stride) {
    const at::Tensor& t = tensor(o, name);
    check_type(t, name, type);
    check_shape(t, name, shape);
    const int64_t T = shape[0], H = shape[1], D = shape[2];
    if (T * H && ((t.stride(1) != D && H > 1) || t.stride(2) != 1)) fail(PyExc_ValueError, std::string(name) + " must be dense in its last two axes");
    call.add(t, name);
    *stride = T > 1 ? t.stride(0) : H * D;
    return data(t);
}
// The type of q, k, v; the C code of it.
kda_dtype type_code(const at::Tensor& t) {
    if (t.scalar_type() == at::kFloat) return KDA_F32;
    if (t.scalar_type() == at::kBFloat16) return KDA_BF16;
    fail(PyExc_TypeError, std::string("q/k/v/out must be float32 or bfloat16, got ") + c10::toString(t.scalar_type()));
}
const at::Tensor& axes(PyObject* o, const char* name, int64_t dim, const char* what) {
    const at::Tensor& t = tensor(o, name);
    if (t.dim() != dim) fail(PyExc_ValueError, what);
    return t;
}
int32_t i32(int64_t x, const char* name) {
    if (x != (int32_t)x) fail(PyExc_ValueError, std::string(name) + " does not fit 32 bits");
    return (int32_t)x;
}
int64_t integer(PyObject* o) {
    const int64_t x = PyLong_AsLongLong(o);
    if (x == -1 && PyErr_Occurred()) throw PyError();
    return x;
}
float real(PyObject* o) {
    const double x = PyFloat_AsDouble(o);
    if (x == -1.0 && PyErr_Occurred()) throw PyError();
    return (float)x;
}
// cu_seqlens (None: one token per sequence) and the number of sequences.
const int32_t* sequences(Call& call, PyObject* o, int64_t T, int64_t* N) {
    *N = T;
    if (o == Py_None) return nullptr;
    if (!THPVariable_Check(o) || THPVariable_Unpack(o).dim() != 1 || THPVariable_Unpack(o).size(0) < 1)
        fail(PyExc_ValueError, "cu_seqlens must be an int32 tensor [N+1]");
    *N = THPVariable_Unpack(o).size(0) - 1;
    return static_cast<const int32_t*>(dense(call, "cu_seqlens", o, {*N + 1}, at::kInt));
}

// The device of a call made current, the raw stream (a torch stream, or the device's current one), and
// the interpreter free during the call.
class Launch {
  public:
    Launch(const c10::Device& dev, PyObject* stream) : guard_(dev) {
        if (stream == Py_None) {
            raw_ = reinterpret_cast<kda_stream_t>(c10::cuda::getCurrentCUDAStream(dev.index()).stream());
        } else {
            PyObject* d = PyObject_GetAttrString(stream, "device_index");
            if (!d) throw PyError();
            const int64_t index = PyLong_AsLongLong(d);
            Py_DECREF(d);
            if (PyErr_Occurred()) throw PyError();
            if (index != dev.index())
                fail(PyExc_ValueError, "the stream must be on " + dev.str() + ", got cuda:" + std::to_string(index));
            PyObject* r = PyObject_GetAttrString(stream, "cuda_stream");
            if (!r) throw PyError();
            raw_ = reinterpret_cast<kda_stream_t>(PyLong_AsVoidPtr(r));
            Py_DECREF(r);
            if (PyErr_Occurred()) throw PyError();
        }
        state_ = PyEval_SaveThread();
    }
    ~Launch() {
        if (state_) PyEval_RestoreThread(state_);
    }
    kda_stream_t stream() const { return raw_; }

  private:
    c10::cuda::CUDAGuard guard_;
    kda_stream_t raw_ = nullptr;
    PyThreadState* state_ = nullptr;
};

// The paged cache of k_cache, v_cache [pages, Hkv, page_size, D], any strides, alike.
kda_kv_cache cache_of(Call& call, PyObject* ko, PyObject* vo, PyObject* to, PyObject* lo, PyObject* kso, PyObject* vso, int64_t N) {
    const at::Tensor &k = tensor(ko, "k_cache"), &v = tensor(vo, "v_cache");
    const at::ScalarType ty = k.scalar_type();
    if (k.dim() != 4 || (ty != at::kFloat && ty != at::kBFloat16 && ty != at::kFloat8_e4m3fn))
        fail(PyExc_ValueError, "k_cache must be [pages, Hkv, page_size, D] in float32, bfloat16 or float8_e4m3fn");
    bool alike = v.sizes() == k.sizes() && v.scalar_type() == ty;
    for (int i = 0; alike && i < 4; ++i) alike = v.stride(i) == k.stride(i) || k.size(i) <= 1;   // one of an axis: any stride
    if (!alike)
        fail(PyExc_ValueError, "v_cache must have the shape, type and strides of k_cache");
    if (k.stride(3) != 1 || v.stride(3) != 1) fail(PyExc_ValueError, "the caches must be dense in their last axis");
    call.add(k, "k_cache");
    call.add(v, "v_cache");
    if (!THPVariable_Check(to)) fail(PyExc_TypeError, "block_table must be a torch.Tensor");
    const at::Tensor& table = THPVariable_Unpack(to);
    if (table.dim() != 2 || table.scalar_type() != at::kInt || table.size(0) != N || (table.size(1) > 1 && table.stride(1) != 1))
        fail(PyExc_ValueError, "block_table must be int32 [" + std::to_string(N) + ", pages of a sequence], dense in its last axis");
    call.add(table, "block_table");
    const int64_t pages = k.size(0), H = k.size(1), ps = k.size(2), D = k.size(3), width = table.size(1);
    kda_kv_cache c = {};
    c.k = data(k);
    c.v = data(v);
    c.k_scale = static_cast<const float*>(dense(call, "k_scale", kso, {H}, at::kFloat));
    c.v_scale = static_cast<const float*>(dense(call, "v_scale", vso, {H}, at::kFloat));
    c.block_table = static_cast<const int32_t*>(data(table));
    c.seq_lens = static_cast<const int32_t*>(needed(call, "seq_lens", lo, {N}, at::kInt));
    c.page_stride = pages > 1 ? k.stride(0) : D;
    c.head_stride = H > 1 ? k.stride(1) : D;
    c.row_stride = ps > 1 ? k.stride(2) : D;
    c.table_stride = N > 1 ? table.stride(0) : width;
    c.num_pages = i32(pages, "pages");
    c.page_size = i32(ps, "page_size");
    c.max_pages = i32(width, "pages of a sequence");
    c.Hkv = i32(H, "Hkv");
    c.D = i32(D, "D");
    c.dt = ty == at::kFloat ? KDA_F32 : ty == at::kBFloat16 ? KDA_BF16 : KDA_E4M3;
    return c;
}

PyObject* init(PyObject*, PyObject* const* a, Py_ssize_t n) {
    if (n != 3) return PyErr_SetString(PyExc_TypeError, "init takes three addresses"), nullptr;
    void* p[3];
    for (int i = 0; i < 3; ++i) {
        p[i] = PyLong_AsVoidPtr(a[i]);
        if (PyErr_Occurred()) return nullptr;
    }
    g_pool = reinterpret_cast<decltype(g_pool)>(p[0]);
    g_append = reinterpret_cast<decltype(g_append)>(p[1]);
    g_decode = reinterpret_cast<decltype(g_decode)>(p[2]);
    Py_RETURN_NONE;
}

// q, k, v, g, beta, state_pool, slots_in, slots_out, out, cu_seqlens, in_flags, stream
PyObject* decode_pool(PyObject* const* a) {
    const char* shapes = "q and v must be [T, H, D] and state_pool [slots, Hv, D, D]";
    const at::Tensor &q = axes(a[0], "q", 3, shapes), &v = axes(a[2], "v", 3, shapes), &pool = axes(a[5], "state_pool", 4, shapes);
    const kda_dtype dt = type_code(q);
    const at::ScalarType ty = q.scalar_type();
    Call call(q.device());
    const int64_t T = q.size(0), Hk = q.size(1), D = q.size(2), Hv = v.size(1), slots = pool.size(0), flags = integer(a[10]);
    if (flags < 0 || flags > UINT32_MAX) fail(PyExc_ValueError, "in_flags must be KDA_IN_* flags");
    int64_t N, sq, sk, sv;
    const int32_t* cu = sequences(call, a[9], T, &N);
    const void* pq = rows(call, "q", a[0], {T, Hk, D}, ty, &sq);
    const void* pk = rows(call, "k", a[1], {T, Hk, D}, ty, &sk);
    const void* pv = rows(call, "v", a[2], {T, Hv, D}, ty, &sv);
    const auto* g = static_cast<const float*>(flags & KDA_IN_G_SCALAR ? needed(call, "g", a[3], {T, Hv}, at::kFloat)
                                                                      : needed(call, "g", a[3], {T, Hv, D}, at::kFloat));
    const auto* beta = static_cast<const float*>(needed(call, "beta", a[4], {T, Hv}, at::kFloat));
    auto* state = static_cast<float*>(needed(call, "state_pool", a[5], {slots, Hv, D, D}, at::kFloat));
    const auto* in = static_cast<const int32_t*>(needed(call, "slots_in", a[6], {N}, at::kInt));
    const auto* out_slots = static_cast<const int32_t*>(needed(call, "slots_out", a[7], {T}, at::kInt));
    void* out = needed(call, "out", a[8], {T, Hv, D}, ty);
    const int32_t n_slots = i32(slots, "slots"), n = i32(N, "N"), hk = i32(Hk, "Hk"), hv = i32(Hv, "Hv"), d = i32(D, "D");
    call.check();
    kda_status st;
    {
        Launch on(call.dev, a[11]);
        st = g_pool(pq, pk, pv, g, beta, sq, sk, sv, state, n_slots, in, out_slots, cu, n, T, hk, hv, d, d, dt, out, (uint32_t)flags, on.stream());
    }
    return PyLong_FromLong(st);
}

// k, v, k_cache, v_cache, block_table, seq_lens, cu_seqlens, q, q_out, inv_freq, positions, axis_pairs,
// adjacent, k_scale, v_scale, stream
PyObject* kv_append(PyObject* const* a) {
    const at::Tensor& k = axes(a[0], "k", 3, "k must be [T, Hkv, D]");
    const kda_dtype dt = type_code(k);
    const at::ScalarType ty = k.scalar_type();
    Call call(k.device());
    const int64_t T = k.size(0), H = k.size(1), D = k.size(2);
    int64_t N, sk, sv, sq = 0, Hq = 0;
    const int32_t* cu = sequences(call, a[6], T, &N);
    const void* pk = rows(call, "k", a[0], {T, H, D}, ty, &sk);
    const void* pv = rows(call, "v", a[1], {T, H, D}, ty, &sv);
    const kda_kv_cache c = cache_of(call, a[2], a[3], a[4], a[5], a[13], a[14], N);
    if (c.Hkv != H || c.D != D)
        fail(PyExc_ValueError, "the caches must hold " + std::to_string(H) + " heads of " + std::to_string(D) + " channels, got " +
                                   std::to_string(c.Hkv) + " of " + std::to_string(c.D));
    kda_rope rope = {};
    const bool turns = a[9] != Py_None;
    if (turns) {
        const at::Tensor& f = axes(a[9], "inv_freq", 1, "inv_freq must be fp32 [pairs]");
        const int64_t pairs = f.size(0);
        int64_t n_axes = 1, per[4] = {pairs, 0, 0, 0}, given = 1;
        bool flat = true;
        if (a[10] != Py_None) {
            const at::Tensor& p = tensor(a[10], "positions");
            flat = p.dim() == 1;
            if (!flat && p.dim() != 2) fail(PyExc_ValueError, "positions must be int32 [T] or [axes, T]");
            n_axes = flat ? 1 : p.size(0);
        }
        if (a[11] != Py_None || n_axes != 1) {
            given = 0;
            PyObject* seq = a[11] == Py_None ? PyTuple_New(0) : PySequence_Fast(a[11], "axis_pairs must be a sequence of numbers of pairs");
            if (!seq) throw PyError();
            given = PySequence_Fast_GET_SIZE(seq);
            for (int64_t i = 0; i < given && i < 4; ++i) {
                per[i] = PyLong_AsLongLong(PySequence_Fast_GET_ITEM(seq, i));
                if (per[i] == -1 && PyErr_Occurred()) break;
            }
            Py_DECREF(seq);
            if (PyErr_Occurred()) throw PyError();
        }
        if (given != n_axes || n_axes < 1 || n_axes > 4)
            fail(PyExc_ValueError, "axis_pairs must name the pairs of each of the " + std::to_string(n_axes) + " position axes (1 to 4)");
        rope.inv_freq = static_cast<const float*>(needed(call, "inv_freq", a[9], {pairs}, at::kFloat));
        rope.positions = static_cast<const int32_t*>(flat ? dense(call, "positions", a[10], {T}, at::kInt)
                                                          : dense(call, "positions", a[10], {n_axes, T}, at::kInt));
        rope.rot_dim = i32(2 * pairs, "pairs");
        rope.num_axes = (int32_t)n_axes;
        for (int i = 0; i < 4; ++i) rope.axis_pairs[i] = i32(i < n_axes ? per[i] : 0, "axis_pairs");
        rope.adjacent = PyObject_IsTrue(a[12]);
        if (rope.adjacent < 0) throw PyError();
    } else if (a[10] != Py_None || a[11] != Py_None) {
        fail(PyExc_ValueError, "positions and axis_pairs go with inv_freq");
    }
    const void* pq = nullptr;
    void* q_out = nullptr;
    if (a[7] != Py_None) {
        Hq = axes(a[7], "q", 3, "q must be [T, Hq, D]").size(1);
        pq = rows(call, "q", a[7], {T, Hq, D}, ty, &sq);
        q_out = needed(call, "q_out", a[8], {T, Hq, D}, ty);
    } else if (a[8] != Py_None) {
        fail(PyExc_ValueError, "q_out goes with q");
    }
    const int32_t n = i32(N, "N"), hq = i32(Hq, "Hq");
    call.check();
    kda_status st;
    {
        Launch on(call.dev, a[15]);
        st = g_append(pk, pv, pq, sk, sv, sq, dt, &c, cu, n, T, hq, turns ? &rope : nullptr, q_out, on.stream());
    }
    return PyLong_FromLong(st);
}

// q, k_cache, v_cache, block_table, seq_lens, out, cu_seqlens, max_q, scale, softcap, window, alibi_slopes,
// kv_start, lse, k_scale, v_scale, workspace, stream
PyObject* kv_decode(PyObject* const* a) {
    const at::Tensor& q = axes(a[0], "q", 3, "q must be [T, Hq, D]");
    const kda_dtype dt = type_code(q);
    const at::ScalarType ty = q.scalar_type();
    Call call(q.device());
    const int64_t T = q.size(0), Hq = q.size(1), D = q.size(2);
    int64_t N, sq;
    const int32_t* cu = sequences(call, a[6], T, &N);
    const void* pq = rows(call, "q", a[0], {T, Hq, D}, ty, &sq);
    const kda_kv_cache c = cache_of(call, a[1], a[2], a[3], a[4], a[14], a[15], N);
    if (c.D != D || c.Hkv < 1 || Hq % c.Hkv)
        fail(PyExc_ValueError, "the caches must hold heads of " + std::to_string(D) + " channels that divide " + std::to_string(Hq) + ", got " +
                                   std::to_string(c.Hkv) + " of " + std::to_string(c.D));
    void* out = needed(call, "out", a[5], {T, Hq, D}, ty);
    const int32_t max_q = i32(integer(a[7]), "max_q"), window = i32(integer(a[10]), "window");
    const float scale = a[8] == Py_None ? (float)(1.0 / std::sqrt((double)D)) : real(a[8]), softcap = real(a[9]);
    const auto* slopes = static_cast<const float*>(dense(call, "alibi_slopes", a[11], {Hq}, at::kFloat));
    const auto* start = static_cast<const int32_t*>(dense(call, "kv_start", a[12], {N}, at::kInt));
    auto* lse = static_cast<float*>(dense(call, "lse", a[13], {T, Hq}, at::kFloat));
    const at::Tensor& ws = tensor(a[16], "workspace");
    void* pw = needed(call, "workspace", a[16], {ws.numel()}, at::kByte);
    const size_t bytes = (size_t)ws.numel();
    const int32_t n = i32(N, "N"), hq = i32(Hq, "Hq");
    call.check();
    kda_status st;
    {
        Launch on(call.dev, a[17]);
        st = g_decode(pq, sq, dt, &c, cu, n, T, max_q, hq, scale, softcap, window, slopes, start, out, lse, pw, bytes, on.stream());
    }
    return PyLong_FromLong(st);
}

template <PyObject* (*F)(PyObject* const*), int ARGS>
PyObject* entry(PyObject*, PyObject* const* a, Py_ssize_t n) {
    if (n != ARGS) return PyErr_Format(PyExc_TypeError, "expected %d arguments, got %d", ARGS, (int)n);
    if (!g_pool) return PyErr_SetString(PyExc_RuntimeError, "libkda is not loaded"), nullptr;
    try {
        return F(a);
    } catch (const PyError&) {
        return nullptr;
    } catch (const std::exception& e) {
        PyErr_SetString(PyExc_RuntimeError, e.what());
        return nullptr;
    }
}

#define KDA_ENTRY(f, n) {#f, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(&entry<f, n>)), METH_FASTCALL, nullptr}
PyMethodDef g_methods[] = {
    {"init", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(&init)), METH_FASTCALL, nullptr},
    KDA_ENTRY(decode_pool, 12), KDA_ENTRY(kv_append, 16), KDA_ENTRY(kv_decode, 18), {nullptr, nullptr, 0, nullptr}};
PyModuleDef g_module = {PyModuleDef_HEAD_INIT, "kda_native", nullptr, -1, g_methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

// Read from the file by the build, which makes it anew for another torch, and checked when it is loaded.
constexpr char kBuiltFor[] = "kda_native for torch " KDA_TORCH_VERSION;

PyMODINIT_FUNC PyInit_kda_native() {
    PyObject* m = PyModule_Create(&g_module);
    if (m && PyModule_AddStringConstant(m, "built_for", kBuiltFor) < 0) Py_CLEAR(m);
    return m;
}
