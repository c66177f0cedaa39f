// Python binding of the single-token operators (include/kda_serve.h).
//
// One token's kernels take a few microseconds, less than a call through ctypes does (20 to 37 us measured on the
// GPU's Arm host for the checks, three allocations and the conversion of two dozen arguments). This module reads the
// tensors' metadata in C++: it checks shapes, types and strides, allocates outputs and the workspace with PyTorch's
// caching allocator, and calls the C ABI on the current stream. Nothing is computed here.
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <ATen/core/Tensor.h>
#include <ATen/cuda/EmptyTensor.h>
#include <c10/cuda/CUDACachingAllocator.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>
#include <torch/csrc/utils/object_ptr.h>

#include <cmath>
#include <mutex>
#include <sstream>
#include <string>

#include "../../include/kda_serve.h"

namespace {

using at::Tensor;

[[noreturn]] void refuse(const char* name, const std::string& want, const Tensor* t) {
    std::ostringstream s;
    s << name << " must be " << want;
    if (t)
        s << ", got " << t->dtype().name() << " " << t->sizes() << " on " << t->device().str() << ", strides "
          << t->strides();
    TORCH_CHECK_VALUE(false, s.str());
}

const Tensor& tensor(PyObject* o, const char* name) {
    TORCH_CHECK_TYPE(THPVariable_Check(o), name, " must be a tensor");
    return THPVariable_Unpack(o);
}

const Tensor& cuda_tensor(PyObject* o, const char* name, int64_t dims) {
    const Tensor& t = tensor(o, name);
    if (!t.is_cuda() || t.dim() != dims) refuse(name, "a CUDA tensor of " + std::to_string(dims) + " dimensions", &t);
    return t;
}

// A contiguous tensor of this shape and type (None stays null).
void* like(PyObject* o, const char* name, at::IntArrayRef shape, at::ScalarType type, at::Device dev,
           bool optional = false) {
    if (optional && o == Py_None) return nullptr;
    const Tensor& t = tensor(o, name);
    if (t.sizes() != shape || t.scalar_type() != type || t.device() != dev || !t.is_contiguous()) {
        std::ostringstream s;
        s << "contiguous " << c10::toString(type) << " of shape " << shape << " on " << dev.str();
        refuse(name, s.str(), &t);
    }
    return t.data_ptr();
}

int32_t dtype_of(const Tensor& t, const char* name) {
    if (t.scalar_type() == at::kBFloat16) return KDA_DTYPE_BF16;
    if (t.scalar_type() == at::kFloat) return KDA_DTYPE_F32;
    TORCH_CHECK_TYPE(false, "unsupported dtype ", t.dtype().name(), " of ", name);
}

int32_t int32_of(int64_t x, const char* name) {
    TORCH_CHECK_VALUE(x >= INT32_MIN && x <= INT32_MAX, name, " is beyond 32 bits");
    return (int32_t)x;
}

float scale_of(PyObject* o, int32_t K) {
    if (o == Py_None) return (float)(1.0 / std::sqrt((double)K));
    const double x = PyFloat_AsDouble(o);
    if (x == -1.0 && PyErr_Occurred()) throw python_error();
    return (float)x;
}

int64_t whole_of(PyObject* o) {
    const long long x = PyLong_AsLongLong(o);
    if (x == -1 && PyErr_Occurred()) throw python_error();
    return x;
}

// The result of a call: the outputs, or the status code as a number for the caller to raise.
PyObject* finish(kda_status s, PyObject* out) {
    if (s == KDA_OK) return out;
    Py_XDECREF(out);
    return PyLong_FromLong(s);
}

void expect(Py_ssize_t n, Py_ssize_t want) {
    TORCH_CHECK_TYPE(n == want, want, " arguments wanted, got ", n);
}

void* stream_of(at::Device dev) { return c10::cuda::getCurrentCUDAStream(dev.index()).stream(); }

// A new tensor, straight from the caching allocator: half the time of at::empty with its dispatch.
Tensor make(at::IntArrayRef shape, at::ScalarType type, at::Device dev) {
    return at::detail::empty_cuda(shape, type, dev, std::nullopt);
}

// Other Python threads run while this lives: allocations and launches may wait (for memory, for room in the queue of
// launches), and what they wait for may need the interpreter.
struct WithoutGil {
    PyThreadState* state = PyEval_SaveThread();
    WithoutGil() = default;
    WithoutGil(const WithoutGil&) = delete;
    ~WithoutGil() { PyEval_RestoreThread(state); }
};

// ------------------------------------------------------------------ kda_step

// step(q, k, v, g, beta, state, scale, slots, out, status)
PyObject* step(PyObject*, PyObject* const* a, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    expect(n, 10);
    const Tensor &q = cuda_tensor(a[0], "q", 4), &v = cuda_tensor(a[2], "v", 4), &state = cuda_tensor(a[5], "state", 4);
    const auto type = q.scalar_type();
    const auto dev = q.device();
    const int64_t N = q.size(0), T = q.size(1), H = q.size(2), K = q.size(3), HV = v.size(2), V = v.size(3);
    kda_step_dims d{int32_of(N, "N"), int32_of(T, "T"), int32_of(H, "H"), int32_of(HV, "HV"), int32_of(K, "K"),
                    int32_of(V, "V"), int32_of(state.size(0), "the number of states"), dtype_of(q, "q"), 0.f};
    d.scale = scale_of(a[6], d.K);
    const int64_t sv[4] = {N, T, HV, V}, sg[4] = {N, T, HV, K}, ss[4] = {state.size(0), HV, K, V};
    void* qp = like(a[0], "q", q.sizes(), type, dev);
    void* kp = like(a[1], "k", q.sizes(), type, dev);
    void* vp = like(a[2], "v", sv, type, dev);
    void* gp = like(a[3], "g", sg, at::kFloat, dev);
    void* bp = like(a[4], "beta", {sv, 3}, type, dev);
    void* sp = like(a[5], "state", ss, at::kFloat, dev);
    void* slots = like(a[7], "slots", {sv, 1}, at::kInt, dev, true);
    void* status = like(a[9], "status", {1}, at::kInt, dev, true);
    const c10::cuda::CUDAGuard guard(dev);
    const bool given = a[8] != Py_None;
    void* op = given ? like(a[8], "out", sv, type, dev) : nullptr;
    Tensor made;
    kda_status s;
    {
        const WithoutGil others;
        if (!given) {
            made = make({sv, 4}, type, dev);
            op = made.data_ptr();
        }
        s = kda_step(&d, qp, kp, vp, (const float*)gp, bp, (float*)sp, (const int32_t*)slots, op, (int32_t*)status,
                     stream_of(dev));
    }
    return finish(s, given ? Py_NewRef(a[8]) : THPVariable_Wrap(std::move(made)));
    END_HANDLE_TH_ERRORS
}

// ------------------------------------------------------------------ the paged cache

struct CacheArgs : kda_cache8 {  // (of a cache in 16 or 32 bits: its `cache` alone)
    at::ScalarType type;         // of rows, queries and outputs
    at::Device dev;
    const int32_t *table, *lens;
    int64_t table_stride;
    int32_t width, N;
    bool eight() const { return cache.dtype == KDA_DTYPE_E4M3; }
};

// The scales of a cache in 8 bits, [pages, blocks of a page, heads] in fp32; returns the blocks.
int64_t scales_of(PyObject* o, const char* name, const kda_cache& c, at::Device dev, float*& p, int64_t& page, int64_t& block,
                  int64_t& head) {
    const Tensor& t = cuda_tensor(o, name, 3);
    if (t.scalar_type() != at::kFloat || t.device() != dev || t.size(0) != c.num_pages || t.size(2) != c.HKV ||
        t.size(1) < 1 || c.page_size % t.size(1) != 0)
        refuse(name, "fp32 [pages, blocks, heads] on the cache's device, of blocks that divide its pages", &t);
    p = t.data_ptr<float>();
    page = t.size(0) > 1 ? t.stride(0) : 0;
    block = t.size(1) > 1 ? t.stride(1) : 0;
    head = t.size(2) > 1 ? t.stride(2) : 0;
    return t.size(1);
}

// k_cache, v_cache [pages, page_size, heads, channels]; page_table [N, width]; kv_lens [N]; with a cache in 8 bits the
// scales, and the rows or queries, which say what type goes in and out.
CacheArgs cache_of(PyObject* ko, PyObject* vo, PyObject* table, PyObject* lens, PyObject* ks, PyObject* vs, const Tensor& rows) {
    const Tensor &k = cuda_tensor(ko, "k_cache", 4), &v = cuda_tensor(vo, "v_cache", 4);
    if (v.sizes().slice(0, 3) != k.sizes().slice(0, 3) || v.scalar_type() != k.scalar_type() || v.device() != k.device())
        refuse("v_cache", "of k_cache's pages, rows, heads, type and device", &v);
    if (k.stride(3) != 1) refuse("k_cache", "of contiguous channels", &k);
    if (v.stride(3) != 1) refuse("v_cache", "of contiguous channels", &v);
    const Tensor& t = cuda_tensor(table, "page_table", 2);
    if (t.scalar_type() != at::kInt || t.device() != k.device() || (t.size(1) > 1 && t.stride(1) != 1))
        refuse("page_table", "int32 [N, max_pages] of contiguous rows, on the cache's device", &t);
    // (the stride of a dimension of one says nothing)
    const auto stride = [](const Tensor& c, int i) { return c.size(i) > 1 ? c.stride(i) : 0; };
    CacheArgs x{{{k.data_ptr(), v.data_ptr(), stride(k, 0), stride(k, 1), stride(k, 2), stride(v, 0), stride(v, 1),
                  stride(v, 2), int32_of(k.size(0), "the number of pages"), int32_of(k.size(1), "the page size"),
                  int32_of(k.size(2), "the number of heads"), int32_of(k.size(3), "K"), int32_of(v.size(3), "V"),
                  k.scalar_type() == at::kFloat8_e4m3fn ? KDA_DTYPE_E4M3 : dtype_of(k, "k_cache")}},
                k.scalar_type(), k.device(), t.data_ptr<int32_t>(), nullptr, t.stride(0),
                int32_of(t.size(1), "max_pages"), int32_of(t.size(0), "N")};
    if (x.eight()) {
        TORCH_CHECK_VALUE(x.cache.num_pages > 0 && x.cache.page_size > 0, "k_cache must have pages and rows");
        x.type = rows.scalar_type();
        x.dtype = dtype_of(rows, "the rows");
        kda_cache8& c = x;
        const int64_t blocks = scales_of(ks, "k_scale", x.cache, x.dev, c.k_scale, c.k_scale_page, c.k_scale_block, c.k_scale_head);
        if (scales_of(vs, "v_scale", x.cache, x.dev, c.v_scale, c.v_scale_page, c.v_scale_block, c.v_scale_head) != blocks)
            refuse("v_scale", "of k_scale's blocks", &tensor(vs, "v_scale"));
        c.block = (int32_t)(x.cache.page_size / blocks);
    } else {
        TORCH_CHECK_VALUE(ks == Py_None && vs == Py_None, "k_scale and v_scale are for a cache in float8_e4m3fn");
    }
    x.lens = (const int32_t*)like(lens, "kv_lens", {t.size(0)}, at::kInt, x.dev);
    return x;
}

// A [rows, heads, channels] tensor whose rows may lie apart, the heads of a row contiguous.
struct Rows {
    void* p;
    int64_t stride;
};
Rows rows_of(PyObject* o, const char* name, int64_t rows, int64_t heads, int64_t channels, const CacheArgs& x) {
    const Tensor& t = tensor(o, name);
    // (the stride of a dimension of one says nothing)
    if (t.dim() != 3 || t.size(0) != rows || t.size(1) != heads || t.size(2) != channels || t.scalar_type() != x.type ||
        t.device() != x.dev || t.stride(2) != 1 || (heads > 1 && t.stride(1) != channels)) {
        std::ostringstream s;
        s << c10::toString(x.type) << " [" << rows << ", " << heads << ", " << channels << "] of contiguous rows on "
          << x.dev.str();
        refuse(name, s.str(), &t);
    }
    return {t.data_ptr(), rows > 1 ? t.stride(0) : heads * channels};
}

// append(k, v, k_cache, v_cache, page_table, kv_lens, q, rope, interleaved, cu_seqlens, q_out, status, k_scale, v_scale,
//        granted)
PyObject* append(PyObject*, PyObject* const* a, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    expect(n, 15);
    const Tensor& kt = cuda_tensor(a[0], "k", 3);
    const CacheArgs x = cache_of(a[2], a[3], a[4], a[5], a[12], a[13], kt);
    const int64_t R = kt.size(0);
    const Rows k = rows_of(a[0], "k", R, x.cache.HKV, x.cache.K, x), v = rows_of(a[1], "v", R, x.cache.HKV, x.cache.V, x);
    void* cu = like(a[9], "cu_seqlens", {x.N + (int64_t)1}, at::kLong, x.dev, true);
    void* status = like(a[11], "status", {1}, at::kInt, x.dev, true);
    void* granted = like(a[14], "granted", {x.N}, at::kInt, x.dev, true);
    const float* rope = nullptr;
    int32_t positions = 0, turned = 0;
    if (a[7] != Py_None) {
        const Tensor& t = cuda_tensor(a[7], "rope", 2);
        rope = (const float*)like(a[7], "rope", t.sizes(), at::kFloat, x.dev);
        positions = int32_of(t.size(0), "the rotation's length");
        turned = int32_of(t.size(1), "the rotation's width");
    }
    const int inter = PyObject_IsTrue(a[8]);
    if (inter < 0) throw python_error();
    const c10::cuda::CUDAGuard guard(x.dev);
    Rows q{nullptr, 0};
    int32_t HQ = 0;
    void* op = nullptr;
    const bool given = a[10] != Py_None;
    int64_t shape[3] = {R, 0, x.cache.K};
    if (a[6] != Py_None) {
        const Tensor& t = cuda_tensor(a[6], "q", 3);
        HQ = int32_of(t.size(1), "the number of query heads");
        q = rows_of(a[6], "q", R, HQ, x.cache.K, x);
        shape[1] = HQ;
        if (given) op = like(a[10], "q_out", shape, x.type, x.dev);
    } else if (given) {
        refuse("q_out", "None where q is", nullptr);
    }
    Tensor made;
    kda_status s;
    {
        const WithoutGil others;
        if (a[6] != Py_None && !given) {
            made = make(shape, x.type, x.dev);
            op = made.data_ptr();
        }
        s = x.eight() ? kda_cache8_append_granted(&x, k.p, k.stride, v.p, v.stride, q.p, q.stride, op, HQ, x.N, R,
                                                  (const int64_t*)cu, rope, positions, turned, inter, x.table,
                                                  x.table_stride, x.width, x.lens, (const int32_t*)granted,
                                                  (int32_t*)status, stream_of(x.dev))
                      : kda_cache_append_granted(&x.cache, k.p, k.stride, v.p, v.stride, q.p, q.stride, op, HQ, x.N, R,
                                                 (const int64_t*)cu, rope, positions, turned, inter, x.table,
                                                 x.table_stride, x.width, x.lens, (const int32_t*)granted,
                                                 (int32_t*)status, stream_of(x.dev));
    }
    return finish(s, made.defined() ? THPVariable_Wrap(std::move(made)) : Py_NewRef(a[10]));  // (None without q)
    END_HANDLE_TH_ERRORS
}

// A workspace of the least size on the present device. No kernel touches one of that size, so one serves all calls (an
// allocation takes half a microsecond of a call's five).
void* untouched(int device) {
    constexpr int kDevices = 32;
    static std::mutex lock;
    static void* known[kDevices];
    TORCH_CHECK(device < kDevices, "device ", device, " is beyond ", kDevices);
    const std::lock_guard<std::mutex> held(lock);
    if (!known[device]) known[device] = c10::cuda::CUDACachingAllocator::raw_alloc(KDA_ATTEND_WORKSPACE_MIN);
    return known[device];
}

// attend(q, k_cache, v_cache, page_table, kv_lens, scale, window, ws, out, status, sinks, k_scale, v_scale)
PyObject* attend(PyObject*, PyObject* const* a, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    expect(n, 13);
    const Tensor& qt = cuda_tensor(a[0], "q", 3);
    const CacheArgs x = cache_of(a[1], a[2], a[3], a[4], a[11], a[12], qt);
    const int32_t HQ = int32_of(qt.size(1), "the number of query heads"), window = int32_of(whole_of(a[6]), "window"),
                  sinks = int32_of(whole_of(a[10]), "sinks");
    const Rows q = rows_of(a[0], "q", x.N, HQ, x.cache.K, x);
    const float scale = scale_of(a[5], x.cache.K);
    void* status = like(a[9], "status", {1}, at::kInt, x.dev, true);
    const c10::cuda::CUDAGuard guard(x.dev);
    const size_t need = x.eight() ? kda_cache8_attend_workspace_bytes(&x, HQ, x.N, x.width, window, sinks)
                                  : kda_cache_attend_sinks_workspace_bytes(&x.cache, HQ, x.N, x.width, window, sinks);
    void* wp = nullptr;
    size_t room = 0;
    if (a[7] != Py_None) {
        const Tensor& t = tensor(a[7], "ws");
        if (t.scalar_type() != at::kByte || t.device() != x.dev || !t.is_contiguous())
            refuse("ws", "a contiguous uint8 tensor on the cache's device", &t);
        if ((size_t)t.numel() >= need) {
            wp = t.data_ptr();
            room = t.numel();
        }
    }
    const int64_t shape[3] = {x.N, HQ, x.cache.V};
    const bool given = a[8] != Py_None;
    void* op = given ? like(a[8], "out", shape, x.type, x.dev) : nullptr;
    Tensor made, lse;
    kda_status s;
    {
        const WithoutGil others;
        if (!given) {
            made = make(shape, x.type, x.dev);
            op = made.data_ptr();
        }
        lse = make({shape, 2}, at::kFloat, x.dev);
        c10::DataPtr scratch;  // (its memory is free again for what follows on this stream)
        if (!wp && need == KDA_ATTEND_WORKSPACE_MIN) {
            wp = untouched(x.dev.index());
            room = need;
        } else if (!wp) {
            scratch = c10::cuda::CUDACachingAllocator::get()->allocate(need);
            wp = scratch.get();
            room = need;
        }
        float* lp = (float*)lse.data_ptr();
        s = x.eight() ? kda_cache8_attend(&x, q.p, q.stride, HQ, x.N, x.table, x.table_stride, x.width, x.lens, window,
                                          sinks, scale, op, lp, (int32_t*)status, wp, room, stream_of(x.dev))
                      : kda_cache_attend_sinks(&x.cache, q.p, q.stride, HQ, x.N, x.table, x.table_stride, x.width, x.lens,
                                               window, sinks, scale, op, lp, (int32_t*)status, wp, room,
                                               stream_of(x.dev));
    }
    THPObjectPtr first(given ? Py_NewRef(a[8]) : THPVariable_Wrap(std::move(made))), second(THPVariable_Wrap(std::move(lse)));
    if (!first || !second) throw python_error();
    return finish(s, PyTuple_Pack(2, first.get(), second.get()));
    END_HANDLE_TH_ERRORS
}

// ------------------------------------------------------------------ kda_cache_resize

// resize(page_table, kv_lens, new_lens, free_pages, free_count, page_size, rows, status)
PyObject* resize(PyObject*, PyObject* const* a, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    expect(n, 8);
    const Tensor& t = cuda_tensor(a[0], "page_table", 2);
    if (t.scalar_type() != at::kInt || (t.size(1) > 1 && t.stride(1) != 1))
        refuse("page_table", "int32 [N, max_pages] of contiguous rows", &t);
    const auto dev = t.device();
    const int64_t N = t.size(0), rows = whole_of(a[6]);
    TORCH_CHECK_VALUE(rows >= 0, "rows must not be negative");
    void* lens = like(a[1], "kv_lens", {N}, at::kInt, dev);
    void* wanted = like(a[2], "new_lens", {N}, at::kInt, dev);
    const Tensor& list = cuda_tensor(a[3], "free_pages", 1);
    void* free = like(a[3], "free_pages", list.sizes(), at::kInt, dev);
    void* count = like(a[4], "free_count", {1}, at::kInt, dev);
    void* status = like(a[7], "status", {1}, at::kInt, dev, true);
    const int32_t width = int32_of(t.size(1), "max_pages"), size = int32_of(whole_of(a[5]), "page_size"),
                  pages = int32_of(list.numel(), "the number of pages"), seqs = int32_of(N, "N");
    // (the stride of a dimension of one says nothing)
    const int64_t stride = N > 1 ? t.stride(0) : t.size(1);
    const c10::cuda::CUDAGuard guard(dev);
    const size_t need = kda_cache_resize_workspace_bytes(seqs, width, rows);
    Tensor cu, slots, granted;
    kda_status s;
    {
        const WithoutGil others;
        cu = make({N + 1}, at::kLong, dev);
        slots = make({rows}, at::kLong, dev);
        granted = make({N}, at::kInt, dev);
        c10::DataPtr scratch;  // (its memory is free again for what follows on this stream)
        if (need > 0) scratch = c10::cuda::CUDACachingAllocator::get()->allocate(need);
        s = kda_cache_resize(t.data_ptr<int32_t>(), stride, width, seqs, size, (const int32_t*)lens, (const int32_t*)wanted,
                             (int32_t*)free, pages, (int32_t*)count, cu.data_ptr<int64_t>(),
                             rows > 0 ? slots.data_ptr<int64_t>() : nullptr, rows, (int32_t*)granted.data_ptr(),
                             (int32_t*)status, scratch.get(), need, stream_of(dev));
    }
    THPObjectPtr x(THPVariable_Wrap(std::move(cu))), y(THPVariable_Wrap(std::move(slots))), z(THPVariable_Wrap(std::move(granted)));
    if (!x || !y || !z) throw python_error();
    return finish(s, PyTuple_Pack(3, x.get(), y.get(), z.get()));
    END_HANDLE_TH_ERRORS
}

PyMethodDef methods[] = {
    {"step", (PyCFunction)(void*)step, METH_FASTCALL, "kda_step"},
    {"append", (PyCFunction)(void*)append, METH_FASTCALL, "kda_cache_append_granted, kda_cache8_append_granted"},
    {"attend", (PyCFunction)(void*)attend, METH_FASTCALL, "kda_cache_attend_sinks, kda_cache8_attend"},
    {"resize", (PyCFunction)(void*)resize, METH_FASTCALL, "kda_cache_resize"},
    {nullptr, nullptr, 0, nullptr},
};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_kda_serve", nullptr, -1, methods};

}  // namespace

PyMODINIT_FUNC PyInit__kda_serve() { return PyModule_Create(&module); }
