// Python entry of the operators around the attention: checks torch tensors,
// allocates outputs and workspaces and calls the C ABI (attn_fwd.h), which
// does the rest.  The same in Python took more host time than the kernels of
// a small batch take: a decoding step's norm issued in 24 us, and in 4.3 from
// here; its append in 14 and 3.2; its attention in 26 and 7.6 (the host's time
// of a call among a hundred).
//
// Every function takes its arguments by position (binding.py has the
// signatures and documents them); None stands for what is left out, and the
// stream is a number or None.  A failed check raises binding.AttnError.
#include <Python.h>

#include <cmath>
#include <cstring>
#include <string>
#include <utility>

#include <ATen/cuda/EmptyTensor.h>
#include <ATen/core/Tensor.h>
#include <c10/cuda/CUDACachingAllocator.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include "attn_fwd.h"

namespace {

PyObject *g_error = nullptr;  // binding.AttnError

// The entry points of the library that binding.py has loaded.
struct Library {
    decltype(&attn_last_error) last_error;
    decltype(&attn_qk_norm_rope) qk_norm_rope;
    decltype(&attn_qk_norm_rope_bwd) qk_norm_rope_bwd;
    decltype(&attn_qk_norm_rope_bwd_workspace_bytes) qk_norm_rope_bwd_workspace_bytes;
    decltype(&attn_kvcache_append_paged) kvcache_append_paged;
    decltype(&attn_fwd_kvcache_paged_fp8) fwd_kvcache_paged_fp8;
    decltype(&attn_fwd_kvcache_paged_fp8_workspace_bytes) fwd_kvcache_paged_fp8_workspace_bytes;
    decltype(&attn_latent_append_paged) latent_append_paged;
    decltype(&attn_fwd_latent_paged) fwd_latent_paged;
    decltype(&attn_fwd_latent_paged_workspace_bytes) fwd_latent_paged_workspace_bytes;
    decltype(&attn_fwd_latent) fwd_latent;
    decltype(&attn_bwd_latent) bwd_latent;
    decltype(&attn_bwd_latent_workspace_bytes) bwd_latent_workspace_bytes;
} g_lib;

struct Err {
    int code;
    std::string msg;
};

[[noreturn]] void fail(int code, std::string msg) { throw Err{code, std::move(msg)}; }

void check(int rc)
{
    if (rc < 0) fail(rc, g_lib.last_error());
}

// The tensor of an argument that must be one / may be None.
const at::Tensor &tensor(PyObject *o, const char *name)
{
    if (!THPVariable_Check(o)) fail(ATTN_ERR_NULL, std::string(name) + " must be a tensor");
    return THPVariable_Unpack(o);
}

const at::Tensor *maybe(PyObject *o, const char *name) { return o == Py_None ? nullptr : &tensor(o, name); }

void *ptr(const at::Tensor &t) { return t.data_ptr(); }
void *ptr(const at::Tensor *t) { return t ? t->data_ptr() : nullptr; }

std::string shape_of(const at::Tensor &t)
{
    std::string s = "(";
    for (int64_t n : t.sizes()) s += (s.size() > 1 ? ", " : "") + std::to_string(n);
    return s + ")";
}

double number(PyObject *o, const char *name)
{
    const double v = PyFloat_AsDouble(o);
    if (v == -1.0 && PyErr_Occurred()) {
        PyErr_Clear();
        fail(ATTN_ERR_SCALE, std::string(name) + " must be a number");
    }
    return v;
}

int truth(PyObject *o)
{
    const int v = PyObject_IsTrue(o);
    if (v < 0) {
        PyErr_Clear();
        fail(ATTN_ERR_SHAPE, "a truth value is expected");
    }
    return v;
}

int dtype_code(const at::Tensor &t)
{
    if (t.scalar_type() == at::kHalf) return ATTN_FP16;
    if (t.scalar_type() == at::kBFloat16) return ATTN_BF16;
    fail(ATTN_ERR_DTYPE, std::string("unsupported dtype ") + c10::toString(t.scalar_type()));
}

// The stream of a call and the memory allocated for it.  On a stream that was
// given, the memory comes from that stream's pool: what the current stream
// has let go of may still be in use there, and the given one does not wait
// for that.
class Call {
public:
    Call(const at::Tensor &t, PyObject *stream)
        : device_(t.device()), guard_(t.device()), current_(c10::cuda::getCurrentCUDAStream(device_.index()))
    {
        raw_ = current_.stream();
        if (stream == Py_None) return;
        raw_ = reinterpret_cast<cudaStream_t>(PyLong_AsVoidPtr(stream));
        if (PyErr_Occurred()) {
            PyErr_Clear();
            fail(ATTN_ERR_NULL, "stream must be a stream");
        }
        if (raw_ != current_.stream()) on_.reset_stream(c10::cuda::getStreamFromExternal(raw_, device_.index()));
    }
    void *stream() const { return raw_; }
    // An output: the caller goes on with it on the current stream, so it is not handed out again before that is done.
    at::Tensor empty(at::IntArrayRef sizes, at::ScalarType type) const
    {
        at::Tensor t(at::detail::empty_cuda(sizes, type, device_, std::nullopt));
        if (raw_ != current_.stream() && t.numel() > 0)
            c10::cuda::CUDACachingAllocator::recordStream(t.storage().data_ptr(), current_);
        return t;
    }
    // Memory that nobody sees: from the same allocator, without a tensor.
    c10::DataPtr scratch(int64_t bytes) const
    {
        return c10::cuda::CUDACachingAllocator::get()->allocate(static_cast<size_t>(bytes));
    }

private:
    c10::Device device_;
    c10::cuda::CUDAGuard guard_;
    c10::cuda::CUDAStream current_;
    c10::cuda::OptionalCUDAStreamGuard on_;
    cudaStream_t raw_ = nullptr;
};

// A [b, h, s, d] tensor, or a packed [total, h, d] one as b = 1: shape, and
// the strides of b, of the head and of s (an axis of one has none).
struct Dense {
    int64_t b, h, s, d;
    int64_t st[3];
};

Dense as_dense(const char *name, const at::Tensor &t)
{
    const auto n = t.sizes(), st = t.strides();
    Dense r;
    int64_t last;
    if (n.size() == 4) {
        r = {n[0], n[1], n[2], n[3], {st[0], st[1], st[2]}};
        last = st[3];
    } else if (n.size() == 3) {
        r = {1, n[1], n[0], n[2], {0, st[1], st[0]}};
        last = st[2];
    } else {
        fail(ATTN_ERR_SHAPE, std::string(name) + " must be [b, h, s, d] or [total, h, d]");
    }
    if (last != 1 && r.d > 1 && t.numel() > 0)
        fail(ATTN_ERR_SHAPE, std::string("the values of a head of ") + name + " must be contiguous");
    if (r.b <= 1) r.st[0] = 0;
    if (r.h <= 1) r.st[1] = 0;
    if (r.s <= 1) r.st[2] = 0;
    return r;
}

// A workspace: allocated with the bytes that a call needs, or the given
// tensor.
struct Workspace {
    c10::DataPtr own;
    void *p = nullptr;
    int64_t bytes = 0;
};

Workspace workspace(const Call &call, const at::Tensor *given, int64_t need, c10::Device device)
{
    Workspace w;
    if (!given) {
        check(need < 0 ? static_cast<int>(need) : 0);
        w.own = call.scratch(need);
        w.p = w.own.get();
        w.bytes = need;
    } else {
        if (given->device() != device || !given->is_contiguous())
            fail(ATTN_ERR_SHAPE, "workspace must be a contiguous tensor on the inputs' device");
        w.p = ptr(*given);
        w.bytes = static_cast<int64_t>(given->nbytes());
    }
    return w;
}

// An output shaped and typed like its input: allocated (contiguous) or checked.
struct Output {
    at::Tensor t;
    Dense dense;
};

Output output(const Call &call, const char *name, const at::Tensor *given, const at::Tensor &like)
{
    Output r;
    if (!given) {
        r.t = call.empty(like.sizes(), like.scalar_type());
    } else {
        r.t = *given;
        if (r.t.sizes() != like.sizes() || r.t.scalar_type() != like.scalar_type() || r.t.device() != like.device())
            fail(ATTN_ERR_SHAPE, std::string(name) + " must be shaped and typed like its input, on its device");
    }
    r.dense = as_dense(name, r.t);
    return r;
}

// What is returned for a tensor: the caller's own object where it gave one, None where there is none.
PyObject *object(PyObject *given, const at::Tensor &t)
{
    if (given == Py_None && t.defined()) return THPVariable_Wrap(t);
    Py_INCREF(given);
    return given;
}

// The interpreter's lock, let go while a call allocates and launches, as the
// other entry points do: both can wait for the device, and the device for a
// host function that needs the lock.  No Python object is touched meanwhile.
class WithoutLock {
public:
    WithoutLock() : state_(PyEval_SaveThread()) {}
    ~WithoutLock() { PyEval_RestoreThread(state_); }
    WithoutLock(const WithoutLock &) = delete;
    WithoutLock &operator=(const WithoutLock &) = delete;

private:
    PyThreadState *state_;
};

struct Rotation {
    const float *cos = nullptr, *sin = nullptr;
    int64_t rot = 0, length = 0;
};

Rotation rotation(PyObject *co, PyObject *so, c10::Device dev)
{
    if ((co == Py_None) != (so == Py_None)) fail(ATTN_ERR_NULL, "cos and sin must both be given or both be None");
    if (co == Py_None) return {};
    const at::Tensor &c = tensor(co, "cos"), &s = tensor(so, "sin");
    if (c.dim() != 2 || c.sizes() != s.sizes()) fail(ATTN_ERR_SHAPE, "cos and sin must be [table_len, rot / 2]");
    if (c.scalar_type() != at::kFloat || s.scalar_type() != at::kFloat || c.device() != dev || s.device() != dev ||
        !c.is_contiguous() || !s.is_contiguous())
        fail(ATTN_ERR_DTYPE, "cos and sin must be contiguous fp32 tensors on the inputs' device");
    return {static_cast<const float *>(ptr(c)), static_cast<const float *>(ptr(s)), 2 * c.size(1), c.size(0)};
}

// Queries, keys and their weights.
struct NormInputs {
    const at::Tensor &q, &k;
    const at::Tensor *wq, *wk;
    Dense dq, dk;
    int dtype;
};

NormInputs norm_inputs(PyObject *qo, PyObject *ko, PyObject *wqo, PyObject *wko)
{
    NormInputs r{tensor(qo, "q"), tensor(ko, "k"), maybe(wqo, "q_weight"), maybe(wko, "k_weight"), {}, {}, 0};
    r.dq = as_dense("q", r.q);
    r.dk = as_dense("k", r.k);
    if (r.dk.b != r.dq.b || r.dk.s != r.dq.s || r.dk.d != r.dq.d || r.q.dim() != r.k.dim())
        fail(ATTN_ERR_SHAPE, "shape mismatch q" + shape_of(r.q) + " k" + shape_of(r.k));
    if (!r.q.is_cuda() || r.k.scalar_type() != r.q.scalar_type() || r.k.device() != r.q.device())
        fail(ATTN_ERR_DTYPE, "q and k must be CUDA tensors of one dtype on one device");
    r.dtype = dtype_code(r.q);
    for (const at::Tensor *w : {r.wq, r.wk})
        if (w && (w->dim() != 1 || w->size(0) != r.dq.d || w->scalar_type() != r.q.scalar_type() ||
                  w->device() != r.q.device() || !w->is_contiguous()))
            fail(ATTN_ERR_SHAPE, "norm weights must be contiguous [d] tensors typed like q, on its device");
    return r;
}

struct Positions {
    const int32_t *p = nullptr;
    int64_t stride = 0;
};

Positions positions(PyObject *o, const NormInputs &in, bool turns)
{
    const bool packed = in.q.dim() == 3;
    if (o == Py_None) {
        if (packed && turns) fail(ATTN_ERR_NULL, "a packed batch needs positions: they start again in every sequence");
        return {};
    }
    const at::Tensor &t = tensor(o, "positions");
    const bool one = t.dim() == 1 && t.size(0) == in.dq.s;
    const bool each = !packed && t.dim() == 2 && t.size(0) == in.dq.b && t.size(1) == in.dq.s;
    if (t.scalar_type() != at::kInt || t.device() != in.q.device() || !(one || each))
        fail(ATTN_ERR_DTYPE, "positions must be int32 [s], [b, s] or (packed) [total] on the inputs' device");
    if (in.dq.s > 1 && t.stride(-1) != 1) fail(ATTN_ERR_SHAPE, "the positions of a sequence must be contiguous");
    return {static_cast<const int32_t *>(ptr(t)), each && in.dq.b > 1 ? t.stride(0) : 0};
}

PyObject *qk_norm_rope(PyObject *const *a)
{
    // q, k, q_weight, k_weight, cos, sin, positions, eps, interleaved, q_out, k_out, stream
    const NormInputs in = norm_inputs(a[0], a[1], a[2], a[3]);
    const Rotation r = rotation(a[4], a[5], in.q.device());
    const Positions pos = positions(a[6], in, r.cos != nullptr);
    const float eps = static_cast<float>(number(a[7], "eps"));
    const int interleaved = truth(a[8]);
    const at::Tensor *gq = maybe(a[9], "q_out"), *gk = maybe(a[10], "k_out");
    const Call call(in.q, a[11]);
    Output qo, ko;
    {
        const WithoutLock unlocked;
        qo = output(call, "q_out", gq, in.q), ko = output(call, "k_out", gk, in.k);
        check(g_lib.qk_norm_rope(ptr(in.q), ptr(in.k), ptr(in.wq), ptr(in.wk), r.cos, r.sin, pos.p, ptr(qo.t), ptr(ko.t),
                                 in.dq.st, in.dk.st, qo.dense.st, ko.dense.st, in.dq.b, in.dq.h, in.dk.h, in.dq.s, in.dq.d,
                                 r.rot, r.length, pos.stride, interleaved, eps, in.dtype, call.stream()));
    }
    return Py_BuildValue("(NN)", object(a[9], qo.t), object(a[10], ko.t));
}

PyObject *qk_norm_rope_bwd(PyObject *const *a)
{
    // dq_out, dk_out, q, k, q_weight, k_weight, cos, sin, positions, eps, interleaved, dq, dk, workspace, stream
    const NormInputs in = norm_inputs(a[2], a[3], a[4], a[5]);
    const Rotation r = rotation(a[6], a[7], in.q.device());
    const Positions pos = positions(a[8], in, r.cos != nullptr);
    const float eps = static_cast<float>(number(a[9], "eps"));
    const int interleaved = truth(a[10]);
    const at::Tensor &dqo = tensor(a[0], "dq_out"), &dko = tensor(a[1], "dk_out");
    const at::Tensor *gdq = maybe(a[11], "dq"), *gdk = maybe(a[12], "dk"), *gws = maybe(a[13], "workspace");
    const Call call(in.q, a[14]);
    Output dq, dk;
    at::Tensor dwq, dwk;
    {
        const WithoutLock unlocked;
        const Output gq = output(call, "dq_out", &dqo, in.q), gk = output(call, "dk_out", &dko, in.k);
        dq = output(call, "dq", gdq, in.q), dk = output(call, "dk", gdk, in.k);
        if (in.wq) dwq = call.empty({in.dq.d}, at::kFloat);
        if (in.wk) dwk = call.empty({in.dq.d}, at::kFloat);
        Workspace ws;
        if (in.wq || in.wk || gws)
            ws = workspace(call, gws, g_lib.qk_norm_rope_bwd_workspace_bytes(in.dq.d), in.q.device());
        check(g_lib.qk_norm_rope_bwd(ptr(gq.t), ptr(gk.t), ptr(in.q), ptr(in.k), ptr(in.wq), ptr(in.wk), r.cos, r.sin, pos.p,
                                     ptr(dq.t), ptr(dk.t), in.wq ? dwq.data_ptr<float>() : nullptr,
                                     in.wk ? dwk.data_ptr<float>() : nullptr, gq.dense.st, gk.dense.st, in.dq.st, in.dk.st,
                                     dq.dense.st, dk.dense.st, in.dq.b, in.dq.h, in.dk.h, in.dq.s, in.dq.d, r.rot, r.length,
                                     pos.stride, interleaved, eps, in.dtype, ws.p, ws.bytes, call.stream()));
    }
    return Py_BuildValue("(NNNN)", object(a[11], dq.t), object(a[12], dk.t), object(Py_None, dwq), object(Py_None, dwk));
}

// A paged cache.
struct Cache {
    const at::Tensor &k, &v;
    const at::Tensor *ks, *vs;
    const at::Tensor &lens, &table;
    int64_t num_pages, page_size, pages_per_seq, block;
};

Cache cache(PyObject *ko, PyObject *vo, PyObject *kso, PyObject *vso, PyObject *lo, PyObject *to, int64_t b, int64_t hkv,
            int64_t d)
{
    Cache c{tensor(ko, "k_pool"), tensor(vo, "v_pool"), maybe(kso, "k_scale"), maybe(vso, "v_scale"),
            tensor(lo, "cache_seqlens"), tensor(to, "block_table"), 0, 0, 0, 0};
    const c10::Device dev = c.k.device();
    if (c.k.dim() != 4 || c.k.size(2) != hkv || c.k.size(3) != d || c.v.sizes() != c.k.sizes() ||
        c.v.scalar_type() != c.k.scalar_type())
        fail(ATTN_ERR_SHAPE, "pools " + shape_of(c.k) + " / " + shape_of(c.v) + " must be [num_pages, page_size, h_kv, d]");
    c.num_pages = c.k.size(0);
    c.page_size = c.k.size(1);
    if (c.table.dim() != 2 || c.table.size(0) != b || c.table.scalar_type() != at::kInt)
        fail(ATTN_ERR_SHAPE, "block_table must be int32 [b, pages_per_seq]");
    c.pages_per_seq = c.table.size(1);
    if (c.lens.dim() != 1 || c.lens.size(0) != b || c.lens.scalar_type() != at::kInt)
        fail(ATTN_ERR_DTYPE, "cache_seqlens must be an int32 tensor of b elements");
    if (!c.k.is_cuda()) fail(ATTN_ERR_SHAPE, "the pools must be CUDA tensors");
    for (const at::Tensor *t : {&c.k, &c.v, &c.lens, &c.table})
        if (t->device() != dev || !t->is_contiguous())
            fail(ATTN_ERR_SHAPE, "pools, block_table and cache_seqlens must be contiguous, on one device");
    if (!c.ks != !c.vs) fail(ATTN_ERR_NULL, "k_scale and v_scale must both be given or both be None");
    if (!c.ks) return c;
    if (c.k.scalar_type() != at::kFloat8_e4m3fn) fail(ATTN_ERR_DTYPE, "a cache with scales must be float8_e4m3fn");
    if (c.ks->dim() != 3 || c.ks->size(0) != c.num_pages || c.ks->size(1) != hkv || c.ks->size(2) < 1 ||
        c.page_size % c.ks->size(2) != 0 || c.vs->sizes() != c.ks->sizes())
        fail(ATTN_ERR_SHAPE, "scales must be [num_pages, h_kv, page_size / scale_block]");
    for (const at::Tensor *t : {c.ks, c.vs})
        if (t->scalar_type() != at::kFloat || t->device() != dev || !t->is_contiguous())
            fail(ATTN_ERR_DTYPE, "scales must be contiguous fp32 tensors on the pools' device");
    c.block = c.page_size / c.ks->size(2);
    return c;
}

PyObject *kvcache_append_paged(PyObject *const *a)
{
    // k_new, v_new, k_pool, v_pool, cache_seqlens, block_table, cos, sin, interleaved, k_scale, v_scale, new_seqlens, stream
    const at::Tensor &k = tensor(a[0], "k_new"), &v = tensor(a[1], "v_new");
    if (k.dim() != 4 || k.sizes() != v.sizes())
        fail(ATTN_ERR_SHAPE, "k_new" + shape_of(k) + " and v_new" + shape_of(v) + " must be [b, h_kv, s_new, d]");
    const Dense kd = as_dense("k_new", k), vd = as_dense("v_new", v);
    const int dtype = dtype_code(k);
    const Cache c = cache(a[2], a[3], a[9], a[10], a[4], a[5], kd.b, kd.h, kd.d);
    if (v.scalar_type() != k.scalar_type() || (c.block == 0 && c.k.scalar_type() != k.scalar_type()))
        fail(ATTN_ERR_DTYPE, "k_new, v_new and a cache without scales must have one dtype");
    if (k.device() != c.k.device() || v.device() != c.k.device())
        fail(ATTN_ERR_SHAPE, "k_new, v_new and the pools must be on one device");
    const at::Tensor *news = maybe(a[11], "new_seqlens");
    if (news && (news->dim() != 1 || news->size(0) != kd.b || news->scalar_type() != at::kInt ||
                 news->device() != c.k.device() || !news->is_contiguous()))
        fail(ATTN_ERR_DTYPE, "new_seqlens must be an int32 tensor of b elements on the pools' device");
    const Rotation r = rotation(a[6], a[7], c.k.device());
    const int interleaved = truth(a[8]);
    const Call call(c.k, a[12]);
    {
        const WithoutLock unlocked;
        check(g_lib.kvcache_append_paged(ptr(k), ptr(v), ptr(c.k), ptr(c.v), static_cast<float *>(ptr(c.ks)),
                                         static_cast<float *>(ptr(c.vs)), static_cast<const int32_t *>(ptr(c.lens)),
                                         static_cast<const int32_t *>(ptr(news)), static_cast<const int32_t *>(ptr(c.table)),
                                         r.cos, r.sin, kd.st, vd.st, kd.b, kd.h, kd.s, c.num_pages, c.page_size,
                                         c.pages_per_seq, c.block, kd.d, r.rot, r.length, interleaved, dtype, call.stream()));
    }
    Py_RETURN_NONE;
}

PyObject *fwd_kvcache_paged_fp8(PyObject *const *a)
{
    // q, k_pool, v_pool, k_scale, v_scale, cache_seqlens, block_table, causal, scale, o, lse, workspace, stream
    const at::Tensor &q = tensor(a[0], "q"), &pool = tensor(a[1], "k_pool");
    if (q.dim() != 4 || pool.dim() != 4)
        fail(ATTN_ERR_SHAPE, "q must be [b, h, sq, d] and the pools [num_pages, page_size, h_kv, d]");
    const int64_t b = q.size(0), h = q.size(1), sq = q.size(2), d = q.size(3), hkv = pool.size(2);
    const int dtype = dtype_code(q);
    if (a[3] == Py_None || a[4] == Py_None) fail(ATTN_ERR_NULL, "k_scale and v_scale must be given");
    const Cache c = cache(a[1], a[2], a[3], a[4], a[5], a[6], b, hkv, d);
    if (!q.is_contiguous() || q.device() != c.k.device()) fail(ATTN_ERR_SHAPE, "q must be contiguous, on the pools' device");
    const double scale = a[8] == Py_None ? 1.0 / std::sqrt(static_cast<double>(d)) : number(a[8], "scale");
    const int causal = truth(a[7]);
    const at::Tensor *go = maybe(a[9], "o"), *glse = maybe(a[10], "lse"), *gws = maybe(a[11], "workspace");
    const Call call(q, a[12]);
    Output o;
    at::Tensor lse;
    {
        const WithoutLock unlocked;
        o = output(call, "o", go, q);
        if (!o.t.is_contiguous()) fail(ATTN_ERR_SHAPE, "o must be contiguous");
        if (!glse) {
            lse = call.empty({b, h, sq}, at::kFloat);
        } else {
            lse = *glse;
            if (lse.sizes() != at::IntArrayRef({b, h, sq}) || lse.scalar_type() != at::kFloat || !lse.is_contiguous() ||
                lse.device() != q.device())
                fail(ATTN_ERR_SHAPE, "lse must be contiguous fp32 [b, h, sq] on q's device");
        }
        const Workspace ws = workspace(call, gws, g_lib.fwd_kvcache_paged_fp8_workspace_bytes(b, h, hkv, sq, d), q.device());
        check(g_lib.fwd_kvcache_paged_fp8(ptr(q), ptr(c.k), ptr(c.v), static_cast<const float *>(ptr(c.ks)),
                                          static_cast<const float *>(ptr(c.vs)), static_cast<const int32_t *>(ptr(c.lens)),
                                          static_cast<const int32_t *>(ptr(c.table)), ptr(o.t), lse.data_ptr<float>(), b, h,
                                          hkv, sq, c.num_pages, c.page_size, c.pages_per_seq, c.block, d, causal,
                                          static_cast<float>(scale), dtype, ws.p, ws.bytes, call.stream()));
    }
    return Py_BuildValue("(NN)", object(a[9], o.t), object(a[10], lse));
}

// The paged cache of latent attention: a pool of tokens, not of keys and values.
struct LatentCache {
    const at::Tensor &pool, &lens, &table;
    int64_t num_pages, page_size, pages_per_seq;
};

constexpr int64_t kLatent = 512, kToken = 576;

LatentCache latent_cache(PyObject *po, PyObject *lo, PyObject *to, const at::Tensor &like, int64_t b)
{
    LatentCache c{tensor(po, "pool"), tensor(lo, "cache_seqlens"), tensor(to, "block_table"), 0, 0, 0};
    if (c.pool.dim() != 3 || c.pool.size(2) != kToken)
        fail(ATTN_ERR_SHAPE, "pool " + shape_of(c.pool) + " must be [num_pages, page_size, 576]");
    c.num_pages = c.pool.size(0);
    c.page_size = c.pool.size(1);
    if (!c.pool.is_cuda() || c.pool.scalar_type() != like.scalar_type())
        fail(ATTN_ERR_DTYPE, "the pool must be a CUDA tensor of the new tokens' or queries' dtype");
    if (c.table.dim() != 2 || c.table.size(0) != b || c.table.scalar_type() != at::kInt)
        fail(ATTN_ERR_SHAPE, "block_table must be int32 [b, pages_per_seq]");
    c.pages_per_seq = c.table.size(1);
    if (c.lens.dim() != 1 || c.lens.size(0) != b || c.lens.scalar_type() != at::kInt)
        fail(ATTN_ERR_DTYPE, "cache_seqlens must be an int32 tensor of b elements");
    for (const at::Tensor *t : {&c.pool, &c.lens, &c.table})
        if (t->device() != like.device() || !t->is_contiguous())
            fail(ATTN_ERR_SHAPE, "pool, block_table and cache_seqlens must be contiguous, on the inputs' device");
    return c;
}

PyObject *latent_append_paged(PyObject *const *a)
{
    // kv_new, pool, cache_seqlens, block_table, norm_weight, cos, sin, eps, interleaved, new_seqlens, stream
    const at::Tensor &x = tensor(a[0], "kv_new");
    if (x.dim() != 3 || x.size(2) != kToken) fail(ATTN_ERR_SHAPE, "kv_new " + shape_of(x) + " must be [b, s_new, 576]");
    const int dtype = dtype_code(x);
    if (x.stride(2) != 1 && x.numel() > 0) fail(ATTN_ERR_SHAPE, "the values of a token of kv_new must be contiguous");
    const int64_t b = x.size(0), s = x.size(1);
    const int64_t st[3] = {b > 1 ? x.stride(0) : 0, 0, s > 1 ? x.stride(1) : 0};
    const LatentCache c = latent_cache(a[1], a[2], a[3], x, b);
    const at::Tensor *w = maybe(a[4], "norm_weight"), *news = maybe(a[9], "new_seqlens");
    if (w && (w->dim() != 1 || w->size(0) != kLatent || w->scalar_type() != x.scalar_type() || w->device() != x.device() ||
              !w->is_contiguous()))
        fail(ATTN_ERR_SHAPE, "norm_weight must be a contiguous [512] tensor typed like kv_new, on its device");
    if (news && (news->dim() != 1 || news->size(0) != b || news->scalar_type() != at::kInt || news->device() != x.device() ||
                 !news->is_contiguous()))
        fail(ATTN_ERR_DTYPE, "new_seqlens must be an int32 tensor of b elements on the pool's device");
    const Rotation r = rotation(a[5], a[6], x.device());
    if (r.cos && r.rot != kToken - kLatent) fail(ATTN_ERR_SHAPE, "cos and sin must be [table_len, 32]");
    const float eps = static_cast<float>(number(a[7], "eps"));
    const int interleaved = truth(a[8]);
    const Call call(x, a[10]);
    {
        const WithoutLock unlocked;
        check(g_lib.latent_append_paged(ptr(x), ptr(c.pool), ptr(w), static_cast<const int32_t *>(ptr(c.lens)),
                                        static_cast<const int32_t *>(ptr(news)), static_cast<const int32_t *>(ptr(c.table)), r.cos,
                                        r.sin, st, b, s, c.num_pages, c.page_size, c.pages_per_seq, r.length, interleaved, eps,
                                        dtype, call.stream()));
    }
    Py_RETURN_NONE;
}

PyObject *fwd_latent_paged(PyObject *const *a)
{
    // q, pool, cache_seqlens, block_table, scale, causal, tree, o, lse, workspace, stream
    const at::Tensor &q = tensor(a[0], "q");
    if (q.dim() != 4 || q.size(3) != kToken) fail(ATTN_ERR_SHAPE, "q " + shape_of(q) + " must be [b, h, sq, 576]");
    const int dtype = dtype_code(q);
    if (!q.is_cuda()) fail(ATTN_ERR_SHAPE, "q must be a CUDA tensor");
    const Dense qd = as_dense("q", q);
    const LatentCache c = latent_cache(a[1], a[2], a[3], q, qd.b);
    const float scale = static_cast<float>(number(a[4], "scale"));
    const int causal = truth(a[5]);
    const at::Tensor *tree = maybe(a[6], "tree"), *go = maybe(a[7], "o"), *glse = maybe(a[8], "lse"), *gws = maybe(a[9], "workspace");
    if (tree && (tree->sizes() != at::IntArrayRef({qd.b, qd.s, (qd.s + 31) / 32}) || tree->scalar_type() != at::kInt ||
                 tree->device() != q.device() || !tree->is_contiguous()))
        fail(ATTN_ERR_SHAPE, "tree must be contiguous int32 [b, sq, ceil(sq / 32)] on q's device");
    const Call call(q, a[10]);
    at::Tensor o, lse;
    {
        const WithoutLock unlocked;
        if (!go) {
            o = call.empty({qd.b, qd.h, qd.s, kLatent}, q.scalar_type());
        } else {
            o = *go;
            if (o.sizes() != at::IntArrayRef({qd.b, qd.h, qd.s, kLatent}) || o.scalar_type() != q.scalar_type() || o.device() != q.device())
                fail(ATTN_ERR_SHAPE, "o must be [b, h, sq, 512], typed like q, on its device");
        }
        if (!glse) {
            lse = call.empty({qd.b, qd.h, qd.s}, at::kFloat);
        } else {
            lse = *glse;
            if (lse.sizes() != at::IntArrayRef({qd.b, qd.h, qd.s}) || lse.scalar_type() != at::kFloat || !lse.is_contiguous() ||
                lse.device() != q.device())
                fail(ATTN_ERR_SHAPE, "lse must be contiguous fp32 [b, h, sq] on q's device");
        }
        const Dense od = as_dense("o", o);
        const Workspace ws = workspace(call, gws, g_lib.fwd_latent_paged_workspace_bytes(qd.b, qd.h, qd.s), q.device());
        check(g_lib.fwd_latent_paged(ptr(q), ptr(c.pool), static_cast<const int32_t *>(ptr(c.lens)),
                                     static_cast<const int32_t *>(ptr(c.table)), static_cast<const int32_t *>(ptr(tree)), ptr(o),
                                     lse.data_ptr<float>(), qd.st, od.st, qd.b, qd.h, qd.s, c.num_pages, c.page_size,
                                     c.pages_per_seq, causal, scale, dtype, ws.p, ws.bytes, call.stream()));
    }
    return Py_BuildValue("(NN)", object(a[7], o), object(a[8], lse));
}

// A packed tensor of the expanded form, [tokens, heads, d], or [tokens, d] of
// one that all heads share: strides of a token and of a head.
struct PackedRows {
    int64_t tokens, heads;
    int64_t st[2];
};

PackedRows packed_rows(const char *name, const at::Tensor &t, int64_t tokens, int64_t heads, int64_t d, const at::Tensor &like)
{
    const bool one = heads == 0;  // no axis of heads
    if (t.dim() != (one ? 2 : 3) || t.size(0) != tokens || (!one && t.size(1) != heads) || t.size(-1) != d)
        fail(ATTN_ERR_SHAPE, std::string(name) + " " + shape_of(t) + " must be [" + std::to_string(tokens) + ", " +
                                 (one ? "" : std::to_string(heads) + ", ") + std::to_string(d) + "]");
    if (t.scalar_type() != like.scalar_type() || t.device() != like.device())
        fail(ATTN_ERR_DTYPE, std::string(name) + " must be of q's dtype, on its device");
    if (t.numel() > 0 && t.stride(-1) != 1) fail(ATTN_ERR_SHAPE, std::string("the values of a row of ") + name + " must be contiguous");
    return {tokens, one ? 1 : heads, {t.stride(0), one ? 0 : t.stride(1)}};
}

struct LatentInputs {
    const at::Tensor &q, &kn, &kr, &v, &cq, &ck;
    int64_t tq, tk, h, batch, max_q, max_k;
    PackedRows rq, rkn, rkr, rv;
    int dtype, causal;
    float scale;
};

int64_t whole(PyObject *o, const char *name)
{
    const long long v = PyLong_AsLongLong(o);
    if (v == -1 && PyErr_Occurred()) {
        PyErr_Clear();
        fail(ATTN_ERR_SHAPE, std::string(name) + " must be a whole number");
    }
    return v;
}

// q, k_nope, k_rope, v at a[0..3]; cu_seqlens_q, cu_seqlens_k, max_seqlen_q, max_seqlen_k, causal, scale at b[0..5]
LatentInputs latent_inputs(PyObject *const *a, PyObject *const *b)
{
    LatentInputs r{tensor(a[0], "q"), tensor(a[1], "k_nope"), tensor(a[2], "k_rope"), tensor(a[3], "v"),
                   tensor(b[0], "cu_seqlens_q"), tensor(b[1], "cu_seqlens_k"), 0, 0, 0, 0, 0, 0, {}, {}, {}, {}, 0, 0, 0.f};
    r.dtype = dtype_code(r.q);
    if (r.q.dim() != 3 || r.kn.dim() != 3) fail(ATTN_ERR_SHAPE, "q must be [total_q, h, 192] and k_nope [total_k, h, 128]");
    if (!r.q.is_cuda()) fail(ATTN_ERR_SHAPE, "q must be a CUDA tensor");
    r.tq = r.q.size(0), r.tk = r.kn.size(0), r.h = r.q.size(1);
    if (r.h == 0) fail(ATTN_ERR_SHAPE, "q has no heads");
    r.rq = packed_rows("q", r.q, r.tq, r.h, 192, r.q);
    r.rkn = packed_rows("k_nope", r.kn, r.tk, r.h, 128, r.q);
    r.rkr = packed_rows("k_rope", r.kr, r.tk, 0, 64, r.q);
    r.rv = packed_rows("v", r.v, r.tk, r.h, 128, r.q);
    for (const at::Tensor *t : {&r.cq, &r.ck})
        if (t->dim() != 1 || t->size(0) < 1 || t->size(0) != r.cq.size(0) || t->scalar_type() != at::kInt || t->device() != r.q.device() ||
            !t->is_contiguous())
            fail(ATTN_ERR_DTYPE, "cu_seqlens must be contiguous int32 tensors of batch + 1 elements on q's device");
    r.batch = r.cq.size(0) - 1;
    r.max_q = whole(b[2], "max_seqlen_q");
    r.max_k = whole(b[3], "max_seqlen_k");
    r.causal = truth(b[4]);
    r.scale = static_cast<float>(b[5] == Py_None ? 1.0 / std::sqrt(192.0) : number(b[5], "scale"));
    return r;
}

PyObject *fwd_latent(PyObject *const *a)
{
    // q, k_nope, k_rope, v, cu_seqlens_q, cu_seqlens_k, max_seqlen_q, max_seqlen_k, causal, scale, o, lse, stream
    const LatentInputs in = latent_inputs(a, a + 4);
    const at::Tensor *go = maybe(a[10], "o"), *glse = maybe(a[11], "lse");
    const Call call(in.q, a[12]);
    at::Tensor o, lse;
    {
        const WithoutLock unlocked;
        o = go ? *go : call.empty({in.tq, in.h, 128}, in.q.scalar_type());
        const PackedRows ro = packed_rows("o", o, in.tq, in.h, 128, in.q);
        lse = glse ? *glse : call.empty({in.h, in.tq}, at::kFloat);
        if (lse.sizes() != at::IntArrayRef({in.h, in.tq}) || lse.scalar_type() != at::kFloat || !lse.is_contiguous() ||
            lse.device() != in.q.device())
            fail(ATTN_ERR_SHAPE, "lse must be contiguous fp32 [h, total_q] on q's device");
        check(g_lib.fwd_latent(ptr(in.q), ptr(in.kn), ptr(in.kr), ptr(in.v), ptr(o), lse.data_ptr<float>(),
                               static_cast<const int32_t *>(ptr(in.cq)), static_cast<const int32_t *>(ptr(in.ck)), in.rq.st, in.rkn.st,
                               in.rkr.st[0], in.rv.st, ro.st, in.batch, in.h, in.tq, in.tk, in.max_q, in.max_k, in.causal, in.scale,
                               in.dtype, call.stream()));
    }
    return Py_BuildValue("(NN)", object(a[10], o), object(a[11], lse));
}

PyObject *bwd_latent(PyObject *const *a)
{
    // q, k_nope, k_rope, v, o, dout, lse, cu_seqlens_q, cu_seqlens_k, max_seqlen_q, max_seqlen_k, causal, scale, dq, dk_nope,
    // dk_rope, dv, workspace, stream
    const LatentInputs in = latent_inputs(a, a + 7);
    const at::Tensor &o = tensor(a[4], "o"), &dout = tensor(a[5], "dout"), &lse = tensor(a[6], "lse");
    const PackedRows ro = packed_rows("o", o, in.tq, in.h, 128, in.q), rg = packed_rows("dout", dout, in.tq, in.h, 128, in.q);
    if (lse.sizes() != at::IntArrayRef({in.h, in.tq}) || lse.scalar_type() != at::kFloat || !lse.is_contiguous() ||
        lse.device() != in.q.device())
        fail(ATTN_ERR_SHAPE, "lse must be contiguous fp32 [h, total_q] on q's device");
    const at::Tensor *given[4] = {maybe(a[13], "dq"), maybe(a[14], "dk_nope"), maybe(a[15], "dk_rope"), maybe(a[16], "dv")};
    const at::Tensor *gws = maybe(a[17], "workspace");
    const Call call(in.q, a[18]);
    at::Tensor out[4];
    {
        const WithoutLock unlocked;
        const char *names[4] = {"dq", "dk_nope", "dk_rope", "dv"};
        const at::Tensor *like[4] = {&in.q, &in.kn, &in.kr, &in.v};
        PackedRows r[4];
        for (int i = 0; i < 4; ++i) {
            out[i] = given[i] ? *given[i] : call.empty(like[i]->sizes(), in.q.scalar_type());
            r[i] = packed_rows(names[i], out[i], like[i]->size(0), i == 2 ? 0 : in.h, like[i]->size(-1), in.q);
        }
        const PackedRows *all[10] = {&in.rq, &in.rkn, &in.rkr, &in.rv, &ro, &rg, &r[0], &r[1], &r[2], &r[3]};
        int64_t st[20];
        for (int i = 0; i < 10; ++i) st[2 * i] = all[i]->st[0], st[2 * i + 1] = all[i]->st[1];
        const Workspace ws = workspace(call, gws, g_lib.bwd_latent_workspace_bytes(in.h, in.tq, in.tk), in.q.device());
        check(g_lib.bwd_latent(ptr(in.q), ptr(in.kn), ptr(in.kr), ptr(in.v), ptr(o), ptr(dout), lse.data_ptr<float>(), ptr(out[0]),
                               ptr(out[1]), ptr(out[2]), ptr(out[3]), static_cast<const int32_t *>(ptr(in.cq)),
                               static_cast<const int32_t *>(ptr(in.ck)), st, in.batch, in.h, in.tq, in.tk, in.max_q, in.max_k, in.causal,
                               in.scale, in.dtype, ws.p, ws.bytes, call.stream()));
    }
    return Py_BuildValue("(NNNN)", object(a[13], out[0]), object(a[14], out[1]), object(a[15], out[2]), object(a[16], out[3]));
}

// Runs a function on its positional arguments; what it throws becomes a
// Python exception.
template <PyObject *(*F)(PyObject *const *), int N>
PyObject *entry(PyObject *, PyObject *const *args, Py_ssize_t n)
{
    if (n != N) {
        PyErr_Format(PyExc_TypeError, "%d arguments are expected, got %zd", N, n);
        return nullptr;
    }
    try {
        return F(args);
    } catch (const Err &e) {
        PyObject *v = Py_BuildValue("(is)", e.code, e.msg.c_str());
        if (v) PyErr_SetObject(g_error ? g_error : PyExc_RuntimeError, v);
        Py_XDECREF(v);
    } catch (...) {  // as torch's own functions raise it (out of memory, a wrong index, ..)
        torch::translate_exception_to_python(std::current_exception());
    }
    return nullptr;
}

// bind(error class, address of each function of Library in its order)
PyObject *bind(PyObject *const *a)
{
    constexpr int kFunctions = sizeof(Library) / sizeof(void *);
    void *at[kFunctions];
    for (int i = 0; i < kFunctions; ++i) {
        at[i] = PyLong_AsVoidPtr(a[1 + i]);
        if (PyErr_Occurred()) return nullptr;
    }
    std::memcpy(&g_lib, at, sizeof(g_lib));
    Py_INCREF(a[0]);
    Py_XDECREF(g_error);
    g_error = a[0];
    Py_RETURN_NONE;
}

template <PyObject *(*F)(PyObject *const *), int N>
PyMethodDef method(const char *name)
{
    return {name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(&entry<F, N>)), METH_FASTCALL, nullptr};
}

PyMethodDef g_methods[] = {
    method<qk_norm_rope, 12>("qk_norm_rope"),
    method<qk_norm_rope_bwd, 15>("qk_norm_rope_bwd"),
    method<kvcache_append_paged, 13>("kvcache_append_paged"),
    method<fwd_kvcache_paged_fp8, 13>("fwd_kvcache_paged_fp8"),
    method<latent_append_paged, 11>("latent_append_paged"),
    method<fwd_latent_paged, 11>("fwd_latent_paged"),
    method<fwd_latent, 13>("fwd_latent"),
    method<bwd_latent, 19>("bwd_latent"),
    method<bind, 14>("bind"),
    {nullptr, nullptr, 0, nullptr},
};

PyModuleDef g_module = {PyModuleDef_HEAD_INIT, "_marshal_ext", nullptr, -1, g_methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__marshal_ext() { return PyModule_Create(&g_module); }
