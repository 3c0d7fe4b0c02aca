// calls.cpp -- the Python side of a decoding and verifying step's calls: reads the
// tensors, checks them, allocates results and workspaces with torch and calls the C entry
// points of w4moe.h.  A module of its own (w4_calls), so that libw4moe.so stays free of
// torch and Python.  _lib.py has the calls' documentation, hands over the library's
// functions (bind) and is called for what belongs to a stream other than the current one.
//
// What bounds it: nothing but the number of steps.  Through ctypes a call's checks,
// conversions and allocations took 7 to 14 us of the host's time, where most small calls
// take 3 to 5 on the GPU; here 1 to 2, beside the launches (2 each).
#include <torch/csrc/autograd/python_variable.h>

#include <torch/csrc/Exceptions.h>

#include <ATen/cuda/EmptyTensor.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>

#include <climits>
#include <cmath>
#include <initializer_list>
#include <optional>

#include "../../include/w4moe.h"
#include "strides.h"

namespace {

using at::Tensor;

// The library's functions and _lib.py's: (status, name) -> raises; (tensor, shape, stream) ->
// a result of the stream's; (tensor, bytes, stream) -> a workspace of the stream's.
struct Library {
    decltype(&w4_w4a16_linear_few) linear_few;
    decltype(&w4_qk_norm_rope) qk_norm_rope;
    decltype(&w4_kv_append_rope) kv_append_rope;
    decltype(&w4_kv_keep) kv_keep;
    decltype(&w4_attn_shared_prefix) attn_shared_prefix;
    decltype(&w4_attn_tree) attn_tree;
    decltype(&w4_attn_shared_prefix_workspace_size) attn_workspace_size;
    PyObject *check, *result, *workspace;
} lib;

// A test's stand-in for the calling thread's current device, or -1.
thread_local int pretended_device = -1;

struct Refused {                           // becomes a ValueError
    const char *why;
};
struct Raised {};                          // a Python error is set

constexpr const char *kNotOnGpu = "tensors passed to the CUDA library must live on the GPU";
constexpr const char *kOtherDevice =
    "tensors passed to the CUDA library must live on the current device";
constexpr const char *kNotContiguous = "tensors passed to the CUDA library must be contiguous";

// Other Python threads run meanwhile.
struct WithoutGil {
    PyThreadState *state = PyEval_SaveThread();
    ~WithoutGil() { PyEval_RestoreThread(state); }
};

const Tensor *optional(PyObject *o)
{
    if (o == Py_None)
        return nullptr;
    if (!THPVariable_Check(o)) {
        PyErr_Format(PyExc_TypeError, "expected a tensor, not %s", Py_TYPE(o)->tp_name);
        throw Raised{};
    }
    return &THPVariable_Unpack(o);
}

const Tensor &tensor(PyObject *o)
{
    const Tensor *t = optional(o);
    if (!t) {
        PyErr_SetString(PyExc_TypeError, "expected a tensor, not None");
        throw Raised{};
    }
    return *t;
}

int integer(PyObject *o)
{
    const long long v = PyLong_AsLongLong(o);
    if (v == -1 && PyErr_Occurred())
        throw Raised{};
    if (v < INT_MIN || v > INT_MAX)
        throw Refused{"an integer argument is out of range"};
    return static_cast<int>(v);
}

int size(int64_t v)
{
    if (v > INT_MAX)
        throw Refused{"a tensor has more than 2^31 - 1 of something"};
    return static_cast<int>(v);
}

float number(PyObject *o)
{
    const double v = PyFloat_AsDouble(o);
    if (v == -1.0 && PyErr_Occurred())
        throw Raised{};
    return static_cast<float>(v);
}

bool truth(PyObject *o)
{
    const int v = PyObject_IsTrue(o);
    if (v < 0)
        throw Raised{};
    return v != 0;
}

int current_device()
{
    return pretended_device >= 0 ? pretended_device : c10::cuda::current_device();
}

// A call's stream: a Stream's handle, or the current device's current one.
w4_stream_t stream_of(PyObject *stream)
{
    if (stream == Py_None)
        return c10::cuda::getCurrentCUDAStream().stream();
    PyObject *handle = PyObject_GetAttrString(stream, "cuda_stream");
    if (!handle)
        throw Raised{};
    void *s = PyLong_AsVoidPtr(handle);
    Py_DECREF(handle);
    if (!s && PyErr_Occurred())
        throw Raised{};
    return static_cast<w4_stream_t>(s);
}

// Refuses tensors that are not on the current device.
void on_device(std::initializer_list<const Tensor *> ts)
{
    for (const Tensor *t : ts)
        if (t && !t->is_cuda())
            throw Refused{kNotOnGpu};
    const int device = current_device();
    for (const Tensor *t : ts)
        if (t && t->get_device() != device)
            throw Refused{kOtherDevice};
}

// Contiguous int32 CUDA tensors (or none).
void int32s(std::initializer_list<const Tensor *> ts)
{
    for (const Tensor *t : ts) {
        if (!t)
            continue;
        if (!t->is_cuda())
            throw Refused{kNotOnGpu};
        if (!t->is_contiguous())
            throw Refused{kNotContiguous};
        if (t->scalar_type() != at::kInt)
            throw Refused{"tables, lengths, slots, page lists and status must be int32"};
    }
}

template <class T> T *ptr(const Tensor &t) { return static_cast<T *>(t.data_ptr()); }
template <class T> T *ptr(const Tensor *t) { return t ? static_cast<T *>(t->data_ptr()) : nullptr; }
const int32_t *ints(const Tensor &t) { return ptr<const int32_t>(t); }
const int32_t *ints(const Tensor *t) { return ptr<const int32_t>(t); }

// A result or workspace that _lib.py's function makes for another stream.
Tensor from_python(PyObject *made)
{
    if (!made)
        throw Raised{};
    const Tensor t = THPVariable_Unpack(made);
    Py_DECREF(made);
    return t;
}

Tensor new_result(PyObject *like, at::IntArrayRef shape, at::ScalarType type, PyObject *stream)
{
    if (stream == Py_None) {
        const at::Device device = THPVariable_Unpack(like).device();
        WithoutGil no_gil;
        return at::detail::empty_cuda(shape, type, device, std::nullopt);
    }
    PyObject *sizes = PyTuple_New(static_cast<Py_ssize_t>(shape.size()));
    if (!sizes)
        throw Raised{};
    for (size_t i = 0; i < shape.size(); i++)
        PyTuple_SET_ITEM(sizes, i, PyLong_FromLongLong(shape[i]));
    PyObject *made = PyObject_CallFunctionObjArgs(lib.result, like, sizes, stream, nullptr);
    Py_DECREF(sizes);
    return from_python(made);
}

Tensor new_workspace(PyObject *like, size_t bytes, PyObject *stream)
{
    if (stream == Py_None) {
        const at::Device device = THPVariable_Unpack(like).device();
        WithoutGil no_gil;
        return at::detail::empty_cuda({static_cast<int64_t>(bytes)}, at::kByte, device,
                                      std::nullopt);
    }
    PyObject *n = PyLong_FromSize_t(bytes);
    if (!n)
        throw Raised{};
    PyObject *made = PyObject_CallFunctionObjArgs(lib.workspace, like, n, stream, nullptr);
    Py_DECREF(n);
    return from_python(made);
}

// Calls an entry point and raises what its status says.
template <class F> void run(const char *name, F &&call)
{
    int rc;
    {
        WithoutGil no_gil;
        rc = call();
    }
    if (rc == W4_OK)
        return;
    PyObject *none = PyObject_CallFunction(lib.check, "is", rc, name);
    Py_XDECREF(none);
    if (none)
        PyErr_SetString(PyExc_RuntimeError, name);
    throw Raised{};
}

// x as Python's: the caller's own object, or a new one's.
PyObject *give(PyObject *own, const Tensor &made)
{
    if (own == Py_None)
        return THPVariable_Wrap(made);
    Py_INCREF(own);
    return own;
}

// ------------------------------------------------------------------- the few-token linear
// (x, q, s, z, group, out, dev_status, stream)
PyObject *linear_few(PyObject *const *a)
{
    const Tensor &x = tensor(a[0]), &q = tensor(a[1]), &s = tensor(a[2]), &z = tensor(a[3]);
    const int group = integer(a[4]);
    const Tensor *own = optional(a[5]), *status = optional(a[6]);
    if (x.dim() != 2 || q.dim() != 2 || group <= 0)
        throw Refused{"x must be [M, K] and the packed weight [N, K / 2]"};
    const int64_t M = x.size(0), K = x.size(1), N = q.size(0);
    const auto of_groups = [&](const Tensor &t) {
        return t.scalar_type() == at::kHalf && t.dim() == 2 && t.size(0) == N &&
               t.size(1) == K / group;
    };
    if (x.scalar_type() != at::kBFloat16 || q.scalar_type() != at::kByte || q.size(1) != K / 2 ||
        !of_groups(s) || !of_groups(z))
        throw Refused{"x must be [M, K] bf16, q [N, K / 2] uint8, s and z [N, K / group] fp16"};
    if (!x.is_contiguous() || !q.is_contiguous() || !s.is_contiguous() || !z.is_contiguous())
        throw Refused{kNotContiguous};
    int32s({status});
    on_device({&x, &q, &s, &z, status});
    if (own && (own->scalar_type() != at::kBFloat16 || own->dim() != 2 || own->size(0) != M ||
                own->size(1) != N || !own->is_contiguous() || !own->is_cuda() ||
                own->get_device() != current_device()))
        throw Refused{"out must be [M, N] bf16, contiguous, on the current device"};
    const w4_stream_t stream = stream_of(a[7]);
    const int m = size(M), k = size(K), n = size(N);
    const Tensor out = own ? *own : new_result(a[0], {M, N}, at::kBFloat16, a[7]);
    run("w4_w4a16_linear_few", [&] {
        return lib.linear_few(ptr<const uint16_t>(x), m, k, n, ptr<const uint8_t>(q),
                              ptr<const uint16_t>(s), ptr<const uint16_t>(z), group,
                              ptr<uint16_t>(out), ptr<int32_t>(status), stream);
    });
    return give(a[5], out);
}

// ------------------------------------------------------------------- norms and rotation
struct RopeInputs {
    const Tensor &q, &k, &steps;
    const Tensor *positions, *q_weight, *k_weight;
    int T, Hq, Hkv, D, code;
};

bool is_weight(const Tensor *w, const Tensor &q)
{
    return !w || (w->scalar_type() == q.scalar_type() && w->dim() == 1 && w->size(0) == q.size(2) &&
                  w->is_contiguous());
}

RopeInputs rope_inputs(PyObject *q_, PyObject *k_, PyObject *steps_, PyObject *positions_,
                       PyObject *q_weight_, PyObject *k_weight_)
{
    const Tensor &q = tensor(q_), &k = tensor(k_), &steps = tensor(steps_);
    const Tensor *positions = optional(positions_), *qw = optional(q_weight_),
                 *kw = optional(k_weight_);
    const bool bf16 = q.scalar_type() == at::kBFloat16;
    if ((!bf16 && q.scalar_type() != at::kHalf) || k.scalar_type() != q.scalar_type())
        throw Refused{"q and k must be of one type, bf16 or fp16"};
    if (q.dim() != 3 || k.dim() != 3 || q.stride(2) != 1 || k.stride(2) != 1)
        throw Refused{"q must be [T, Hq, D] and k [T, Hkv, D], contiguous along the last axis"};
    if (k.size(0) != q.size(0) || k.size(2) != q.size(2))
        throw Refused{"q must be [T, Hq, D] and k [T, Hkv, D]"};
    if (steps.scalar_type() != at::kLong || steps.dim() != 1 || !steps.is_contiguous())
        throw Refused{"steps must be a table of w4_rope_steps"};
    if (positions && (positions->scalar_type() != at::kInt || positions->dim() != 1 ||
                      positions->size(0) != q.size(0) || !positions->is_contiguous()))
        throw Refused{"positions must be [T] int32, contiguous"};
    if (!is_weight(qw, q))
        throw Refused{"q_weight must be [D] of q's type, contiguous"};
    if (!is_weight(kw, q))
        throw Refused{"k_weight must be [D] of q's type, contiguous"};
    on_device({&q, &k, &steps, positions, qw, kw});
    return {q, k, steps, positions, qw, kw, size(q.size(0)), size(q.size(1)), size(k.size(1)),
            size(q.size(2)), bf16 ? 0 : 1};
}

// A new result like `like`, or the caller's, checked.
Tensor rope_out(PyObject *own_, PyObject *like_, PyObject *stream)
{
    const Tensor &like = THPVariable_Unpack(like_);
    const Tensor *own = optional(own_);
    if (!own)
        return new_result(like_, like.sizes(), like.scalar_type(), stream);
    if (!own->is_cuda())
        throw Refused{kNotOnGpu};
    if (own->get_device() != like.get_device())
        throw Refused{kOtherDevice};
    if (own->sizes() != like.sizes() || own->scalar_type() != like.scalar_type() ||
        own->stride(2) != 1)
        throw Refused{"q_out and k_out must be like q and k, contiguous along the last axis"};
    if (w4::rows_overlap(own->size(0), own->size(1), own->size(2), own->stride(0), own->stride(1)))
        throw Refused{"tokens or heads of q_out or k_out overlap"};
    return *own;
}

// (q, k, positions, steps, q_weight, k_weight, eps, interleaved, amplitude, q_out, k_out, stream)
PyObject *qk_norm_rope(PyObject *const *a)
{
    if (a[2] == Py_None)
        throw Refused{"positions must be [T] int32, contiguous"};
    const RopeInputs r = rope_inputs(a[0], a[1], a[3], a[2], a[4], a[5]);
    const float eps = number(a[6]), amplitude = number(a[8]);
    const bool interleaved = truth(a[7]);
    const w4_stream_t stream = stream_of(a[11]);
    const int rot = size(2 * r.steps.size(0));
    const Tensor q_out = rope_out(a[9], a[0], a[11]), k_out = rope_out(a[10], a[1], a[11]);
    run("w4_qk_norm_rope", [&] {
        return lib.qk_norm_rope(
            ptr<const uint16_t>(r.q), r.q.stride(0), r.q.stride(1), ptr<const uint16_t>(r.k),
            r.k.stride(0), r.k.stride(1), ints(r.positions), ptr<const int64_t>(r.steps),
            ptr<const uint16_t>(r.q_weight), ptr<const uint16_t>(r.k_weight), r.T, r.Hq, r.Hkv, r.D,
            rot, interleaved, r.code, eps, amplitude, ptr<uint16_t>(q_out), q_out.stride(0),
            q_out.stride(1), ptr<uint16_t>(k_out), k_out.stride(0), k_out.stride(1), stream);
    });
    PyObject *first = give(a[9], q_out), *second = give(a[10], k_out);
    PyObject *both = first && second ? PyTuple_Pack(2, first, second) : nullptr;
    Py_XDECREF(first);
    Py_XDECREF(second);
    return both;
}

// B of q_offsets [B + 1], with a table and lengths for as many.
int batch(const Tensor &table, const Tensor &lens, const Tensor &q_offsets)
{
    if (q_offsets.dim() != 1 || q_offsets.size(0) < 1 || table.dim() != 2 || lens.dim() != 1 ||
        table.size(0) < q_offsets.size(0) - 1 || lens.size(0) < q_offsets.size(0) - 1)
        throw Refused{"q_offsets must be [B + 1] for a table [B, W] and lens [B]"};
    return size(q_offsets.size(0) - 1);
}

// (k_pages, v_pages, table, lens, q, k, v, q_offsets, steps, positions, q_weight, k_weight, eps,
//  interleaved, amplitude, q_out, dev_status, stream)
PyObject *kv_append_rope(PyObject *const *a)
{
    const Tensor &kp = tensor(a[0]), &vp = tensor(a[1]), &table = tensor(a[2]), &lens = tensor(a[3]);
    const Tensor &v = tensor(a[6]), &q_offsets = tensor(a[7]);
    const Tensor *status = optional(a[16]);
    const RopeInputs r = rope_inputs(a[4], a[5], a[8], a[9], a[10], a[11]);
    const float eps = number(a[12]), amplitude = number(a[14]);
    const bool interleaved = truth(a[13]);
    if (kp.scalar_type() != r.q.scalar_type() || vp.scalar_type() != r.q.scalar_type() ||
        kp.dim() != 4 || kp.stride(3) != 1 || vp.sizes() != kp.sizes() ||
        vp.strides() != kp.strides())
        throw Refused{"k_pages and v_pages must be alike, [P, page_size, Hkv, D] of q's type, "
                      "contiguous along the last axis"};
    if (kp.size(2) != r.Hkv || kp.size(3) != r.D || v.scalar_type() != r.q.scalar_type() ||
        v.sizes() != r.k.sizes() || v.stride(2) != 1)
        throw Refused{"k and v must be [T, Hkv, D] of the pages' type"};
    int32s({&table, &lens, &q_offsets, status});
    const int B = batch(table, lens, q_offsets), W = size(table.size(1));
    on_device({&kp, &vp, &v, &table, &lens, &q_offsets, status});
    const w4_stream_t stream = stream_of(a[17]);
    const int P = size(kp.size(0)), page = size(kp.size(1)), rot = size(2 * r.steps.size(0));
    const Tensor q_out = rope_out(a[15], a[4], a[17]);
    if (B > 0)
        run("w4_kv_append_rope", [&] {
            return lib.kv_append_rope(
                ptr<uint16_t>(kp), ptr<uint16_t>(vp), kp.stride(0), kp.stride(1), kp.stride(2), P,
                page, ints(table), B, W, ints(lens), ptr<const uint16_t>(r.q), r.q.stride(0),
                r.q.stride(1), ptr<const uint16_t>(r.k), r.k.stride(0), r.k.stride(1),
                ptr<const uint16_t>(v), v.stride(0), v.stride(1), ints(q_offsets),
                ints(r.positions), ptr<const int64_t>(r.steps), ptr<const uint16_t>(r.q_weight),
                ptr<const uint16_t>(r.k_weight), r.T, r.Hq, r.Hkv, r.D, rot, interleaved, r.code,
                eps, amplitude, ptr<uint16_t>(q_out), q_out.stride(0), q_out.stride(1),
                ptr<int32_t>(status), stream);
        });
    return give(a[15], q_out);
}

// ------------------------------------------------------------------- kept tokens
// (pool, table, lens, refs, q_offsets, kept, kept_offsets, lens_out, dev_status, stream)
PyObject *kv_keep(PyObject *const *a)
{
    const Tensor &pool = tensor(a[0]), &table = tensor(a[1]), &lens = tensor(a[2]),
                 &refs = tensor(a[3]), &q_offsets = tensor(a[4]), &kept = tensor(a[5]),
                 &kept_offsets = tensor(a[6]), &lens_out = tensor(a[7]);
    const Tensor *status = optional(a[8]);
    int32s({&table, &lens, &refs, status});
    if (table.dim() != 2 || refs.dim() != 1 || lens.dim() != 1 || lens.size(0) != table.size(0))
        throw Refused{"lens must be [B] and refs [P] for a table [B, W]"};
    const int B = size(table.size(0)), W = size(table.size(1)), P = size(refs.size(0));
    if (!pool.is_cuda())
        throw Refused{kNotOnGpu};
    if (!pool.is_contiguous())
        throw Refused{kNotContiguous};
    if (pool.dim() < 4 || pool.size(-4) != P || pool.element_size() != 2)
        throw Refused{"the pool must be [..., P, page_size, Hkv, D] of 16-bit values"};
    const int64_t page_bytes = pool.size(-3) * pool.size(-2) * pool.size(-1) * 2;
    const int planes = size(pool.numel() * 2 / std::max<int64_t>(P * page_bytes, 1));
    const int page = size(pool.size(-3));
    int32s({&q_offsets, &kept, &kept_offsets, &lens_out});
    if (q_offsets.dim() != 1 || q_offsets.size(0) != B + 1ll || kept_offsets.dim() != 1 ||
        kept_offsets.size(0) != B + 1ll || kept.dim() != 1 || lens_out.sizes() != lens.sizes())
        throw Refused{"q_offsets and kept_offsets must be [B + 1], kept a list, lens_out [B]"};
    on_device({&pool, &table, &lens, &refs, &q_offsets, &kept, &kept_offsets, &lens_out, status});
    const w4_stream_t stream = stream_of(a[9]);
    const int n_kept = size(kept.size(0));
    run("w4_kv_keep", [&] {
        return lib.kv_keep(pool.data_ptr(), planes, page_bytes, ints(table), B, W, ints(lens),
                           ints(refs), P, ints(q_offsets), ints(kept), ints(kept_offsets), n_kept,
                           page, ptr<int32_t>(lens_out), ptr<int32_t>(status), stream);
    });
    Py_INCREF(a[7]);
    return a[7];
}

// ------------------------------------------------------------------- attention
// (q, k_pages, v_pages, table, lens, q_offsets, tree, causal, group_offsets, shared_lens, max_q,
//  scale, workspace, out, dev_status, stream); tree None: causal counts
PyObject *attn(PyObject *const *a)
{
    const Tensor &q = tensor(a[0]), &kp = tensor(a[1]), &vp = tensor(a[2]), &table = tensor(a[3]),
                 &lens = tensor(a[4]), &q_offsets = tensor(a[5]);
    const Tensor *tree = optional(a[6]), *group_offsets = optional(a[8]), *shared = optional(a[9]),
                 *ws = optional(a[12]), *own = optional(a[13]), *status = optional(a[14]);
    const bool causal = truth(a[7]);
    const int max_q = integer(a[10]);
    if (!q.is_cuda() || !kp.is_cuda() || !vp.is_cuda())
        throw Refused{kNotOnGpu};
    if (kp.dim() != 4 || kp.element_size() != 2 || kp.stride(3) != 1 ||
        vp.scalar_type() != kp.scalar_type() || vp.sizes() != kp.sizes() ||
        vp.strides() != kp.strides())
        throw Refused{"k_pages and v_pages must be alike, [P, page_size, Hkv, D] of 16 bits, "
                      "contiguous along the last axis"};
    int32s({&table, &lens, &q_offsets, group_offsets, shared, status});
    const bool bf16 = kp.scalar_type() == at::kBFloat16;
    if (q.dim() != 3 || (!bf16 && kp.scalar_type() != at::kHalf) ||
        q.scalar_type() != kp.scalar_type() || q.stride(2) != 1 || q.size(2) != kp.size(3))
        throw Refused{"q must be [T, Hq, D] of the pages' type, bf16 or fp16, contiguous along "
                      "the last axis"};
    const int T = size(q.size(0)), Hq = size(q.size(1)), D = size(q.size(2));
    const int P = size(kp.size(0)), page = size(kp.size(1)), Hkv = size(kp.size(2));
    const int B = batch(table, lens, q_offsets), W = size(table.size(1));
    const int64_t G = group_offsets ? group_offsets->numel() - 1 : 0;
    if (G < 0 || (G > 0 && (!shared || shared->numel() != G)))
        throw Refused{"group_offsets must be [G + 1] and shared_lens [G]"};
    const int g = size(G);
    int words = 0;
    if (tree) {
        int32s({tree});
        if (tree->dim() != 2 || tree->size(0) != T)
            throw Refused{"tree must be [T, words], a bit for each of max_q tokens in a row"};
        words = size(tree->size(1));
    }
    on_device({&q, &kp, &vp, &table, &lens, &q_offsets, tree, group_offsets, shared, ws, own, status});
    if (own) {
        if (!own->is_cuda())
            throw Refused{kNotOnGpu};
        if (!own->is_contiguous())
            throw Refused{kNotContiguous};
        if (own->scalar_type() != q.scalar_type() || own->sizes() != q.sizes())
            throw Refused{"out must be [T, Hq, D] of q's type"};
    }
    if (ws && !ws->is_cuda())
        throw Refused{kNotOnGpu};
    if (ws && !ws->is_contiguous())
        throw Refused{kNotContiguous};
    const float scale = a[11] == Py_None ? static_cast<float>(1.0 / std::sqrt(static_cast<double>(D)))
                                         : number(a[11]);
    const w4_stream_t stream = stream_of(a[15]);
    const Tensor out = own ? *own : new_result(a[0], q.sizes(), q.scalar_type(), a[15]);
    const Tensor workspace =
        ws ? *ws
           : new_workspace(a[0],
                           std::max<size_t>(Hkv > 0 && Hq % Hkv == 0
                                                ? lib.attn_workspace_size(T, B, g, max_q, Hq, Hkv, D)
                                                : 0,
                                            256),
                           a[15]);
    const size_t bytes = workspace.nbytes();
    if (tree)
        run("w4_attn_tree", [&] {
            return lib.attn_tree(ptr<const uint16_t>(q), q.stride(0), q.stride(1),
                                 ptr<const uint16_t>(kp), ptr<const uint16_t>(vp), kp.stride(0),
                                 kp.stride(1), kp.stride(2), P, page, ints(table), W, ints(lens),
                                 ints(q_offsets), T, B, max_q, ptr<const uint32_t>(*tree), words,
                                 ints(group_offsets), ints(shared), g, Hq, Hkv, D, bf16 ? 0 : 1,
                                 scale, workspace.data_ptr(), bytes, ptr<uint16_t>(out),
                                 ptr<int32_t>(status), stream);
        });
    else
        run("w4_attn_shared_prefix", [&] {
            return lib.attn_shared_prefix(
                ptr<const uint16_t>(q), q.stride(0), q.stride(1), ptr<const uint16_t>(kp),
                ptr<const uint16_t>(vp), kp.stride(0), kp.stride(1), kp.stride(2), P, page,
                ints(table), W, ints(lens), ints(q_offsets), T, B, max_q, ints(group_offsets),
                ints(shared), g, Hq, Hkv, D, bf16 ? 0 : 1, causal, scale, workspace.data_ptr(),
                bytes, ptr<uint16_t>(out), ptr<int32_t>(status), stream);
        });
    return give(a[13], out);
}

// ------------------------------------------------------------------- the module
template <PyObject *(*F)(PyObject *const *), Py_ssize_t N>
PyObject *method(PyObject *, PyObject *const *args, Py_ssize_t n)
{
    HANDLE_TH_ERRORS
    if (n != N) {
        PyErr_Format(PyExc_TypeError, "expected %zd arguments, not %zd", N, n);
        return nullptr;
    }
    try {
        return F(args);
    } catch (const Refused &r) {
        PyErr_SetString(PyExc_ValueError, r.why);
    } catch (const Raised &) {
    }
    return nullptr;
    END_HANDLE_TH_ERRORS
}

// (addresses of the seven functions in Library's order, check, result, workspace)
PyObject *bind(PyObject *const *a)
{
    void **to[7] = {reinterpret_cast<void **>(&lib.linear_few),
                    reinterpret_cast<void **>(&lib.qk_norm_rope),
                    reinterpret_cast<void **>(&lib.kv_append_rope),
                    reinterpret_cast<void **>(&lib.kv_keep),
                    reinterpret_cast<void **>(&lib.attn_shared_prefix),
                    reinterpret_cast<void **>(&lib.attn_tree),
                    reinterpret_cast<void **>(&lib.attn_workspace_size)};
    for (int i = 0; i < 7; i++) {
        *to[i] = PyLong_AsVoidPtr(a[i]);
        if (!*to[i])
            throw Refused{"an entry point is missing"};
    }
    PyObject **own[3] = {&lib.check, &lib.result, &lib.workspace};
    for (int i = 0; i < 3; i++) {
        Py_INCREF(a[7 + i]);
        Py_XDECREF(*own[i]);
        *own[i] = a[7 + i];
    }
    Py_RETURN_NONE;
}

// (device): stands for the calling thread's current one until it is -1 (for tests: tensors
// of another device than the current one, where there is only one)
PyObject *pretend_device(PyObject *const *a)
{
    pretended_device = integer(a[0]);
    Py_RETURN_NONE;
}

template <PyObject *(*F)(PyObject *const *), Py_ssize_t N> PyMethodDef entry(const char *name)
{
    return {name, reinterpret_cast<PyCFunction>(reinterpret_cast<void *>(&method<F, N>)),
            METH_FASTCALL, nullptr};
}

PyMethodDef methods[] = {entry<bind, 10>("bind"),
                         entry<pretend_device, 1>("pretend_device"),
                         entry<linear_few, 8>("linear_few"),
                         entry<qk_norm_rope, 12>("qk_norm_rope"),
                         entry<kv_append_rope, 18>("kv_append_rope"),
                         entry<kv_keep, 10>("kv_keep"),
                         entry<attn, 16>("attn"),
                         {nullptr, nullptr, 0, nullptr}};

PyModuleDef module_def = {PyModuleDef_HEAD_INIT, "w4_calls", nullptr, -1, methods,
                          nullptr,               nullptr,    nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit_w4_calls()
{
    return PyModule_Create(&module_def);
}
