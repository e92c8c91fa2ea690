// Python entry points of the gradient, adapter and vocabulary calls: tensors in, checks,
// allocation of the results from torch's caching allocator, and one call of the
// C ABI on the current stream.  They are here and not in Python because a
// decode step calls them hundreds of times: what ctypes and Python take for one
// call (about 15 us) is more than twice the kernel's time.
//
// Everything the GPU does runs in liblct.so.
#include <Python.h>

#include <cstdint>
#include <optional>
#include <vector>

#include <ATen/core/Tensor.h>
#include <ATen/core/grad_mode.h>
#include <ATen/ops/empty.h>
#include <c10/core/AutogradState.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/custom_function.h>
#include <torch/csrc/autograd/functions/basic_ops.h>
#include <torch/csrc/autograd/python_variable.h>

#include "../../include/lct.h"

namespace {

PyObject *g_error = nullptr;  // binding.LctError

// A Python error is set and has to be handed up.
struct Raised {};

[[noreturn]] void refuse(const char *what)
{
    PyErr_SetString(PyExc_ValueError, what);
    throw Raised{};
}
void need(bool ok, const char *what)
{
    if (!ok) refuse(what);
}
void check(lct_status rc, const char *what)
{
    if (rc == LCT_OK) return;
    PyObject *e = PyObject_CallFunction(g_error, "is", static_cast<int>(rc), what);
    if (e) {
        PyErr_SetObject(g_error, e);
        Py_DECREF(e);
    }
    throw Raised{};
}

const at::Tensor &tensor(PyObject *o, const char *what)
{
    if (!THPVariable_Check(o)) refuse(what);
    return THPVariable_Unpack(o);
}

at::Tensor make(at::IntArrayRef shape, at::ScalarType type, int device)
{
    return at::empty(shape, at::TensorOptions().dtype(type).device(at::kCUDA, device));
}

// A call wrote into a caller's tensor: autograd's check of tensors that it saved has to notice.  (Tensors made in
// inference mode have no version.)
void wrote(const at::Tensor &t)
{
    if (!t.is_inference()) t.unsafeGetTensorImpl()->bump_version();
}

void *stream_of(int device) { return c10::cuda::getCurrentCUDAStream(static_cast<c10::DeviceIndex>(device)).stream(); }

// Forward-mode tangents are gradients that none of the calls gives.
void no_tangent(std::initializer_list<const at::Tensor *> operands, const char *what)
{
    if (!c10::AutogradState::get_tls_state().get_fw_grad_mode()) return;
    for (const at::Tensor *t : operands)
        if (t->_fw_grad(0).defined()) {
            PyErr_Format(PyExc_RuntimeError, "%s has no forward-mode derivative, but an operand carries a tangent", what);
            throw Raised{};
        }
}
// Autograd does not see what a call does with these.
void no_gradient(std::initializer_list<const at::Tensor *> operands, const char *what)
{
    if (at::GradMode::is_enabled())
        for (const at::Tensor *t : operands)
            if (t->requires_grad()) {
                PyErr_Format(PyExc_RuntimeError,
                             "%s gives no gradients, but an operand requires one: call it under torch.no_grad()", what);
                throw Raised{};
            }
    no_tangent(operands, what);
}

// ---------------------------------------------------------------- gradients

// A reference.
struct Held {
    PyObject *o;
    explicit Held(PyObject *p) : o(p) {}
    Held(const Held &) = delete;
    Held &operator=(const Held &) = delete;
    ~Held() { Py_XDECREF(o); }
};

// A list's tensors.  They are held until the call has been enqueued: an iterable
// may make its tensors as it goes, and nobody else holds those; let go of
// earlier, their memory could become the call's own scratch.
struct Grads {
    Held seq;
    std::vector<const void *> ptr;
    std::vector<uint64_t> n;
    std::vector<int32_t> dtype;
    int device = -1;

    explicit Grads(PyObject *list);
};

Grads::Grads(PyObject *list) : seq(PySequence_Fast(list, "expected a sequence of tensors"))
{
    if (!seq.o) throw Raised{};
    const Py_ssize_t count = PySequence_Fast_GET_SIZE(seq.o);
    ptr.reserve(count);
    n.reserve(count);
    dtype.reserve(count);
    for (Py_ssize_t i = 0; i < count; ++i) {
        const at::Tensor &t = tensor(PySequence_Fast_GET_ITEM(seq.o, i), "expected tensors");
        need(t.is_cuda() && t.is_contiguous(), "expected contiguous CUDA tensors");
        need(device < 0 || t.get_device() == device, "expected tensors on one device");
        device = t.get_device();
        if (t.scalar_type() != at::kBFloat16 && t.scalar_type() != at::kFloat)
            check(LCT_ERR_UNSUPPORTED, "gradients other than BF16 and float32");
        dtype.push_back(t.scalar_type() == at::kFloat ? LCT_DTYPE_F32 : LCT_DTYPE_BF16);
        ptr.push_back(t.data_ptr());
        n.push_back(static_cast<uint64_t>(t.numel()));
    }
}

// (grads) -> norm
PyObject *grad_norm(PyObject *const *a)
{
    Grads g(a[0]);
    if (g.device < 0) g.device = c10::cuda::current_device();
    const c10::cuda::CUDAGuard guard(static_cast<c10::DeviceIndex>(g.device));
    at::Tensor norm = make({}, at::kFloat, g.device), work = make({LCT_GRAD_WORK_BYTES}, at::kByte, g.device);
    check(lct_grad_norm(g.ptr.data(), g.n.data(), g.dtype.data(), g.ptr.size(), static_cast<float *>(norm.data_ptr()),
                        work.data_ptr(), stream_of(g.device)),
          "lct_grad_norm");
    return THPVariable_Wrap(norm);
}

// (grads, max_norm, out or None) -> norm
PyObject *clip_grads(PyObject *const *a)
{
    Grads g(a[0]);
    const double max_norm = PyFloat_AsDouble(a[1]);
    if (PyErr_Occurred()) throw Raised{};
    std::optional<Grads> other;
    if (a[2] != Py_None) {
        other.emplace(a[2]);
        need(other->n == g.n && other->dtype == g.dtype && other->device == g.device,
             "out must match the gradients' sizes, types and device");
    }
    const Grads &out = other ? *other : g;
    if (g.device < 0) g.device = c10::cuda::current_device();
    const c10::cuda::CUDAGuard guard(static_cast<c10::DeviceIndex>(g.device));
    at::Tensor norm = make({}, at::kFloat, g.device), work = make({LCT_GRAD_WORK_BYTES}, at::kByte, g.device);
    check(lct_grad_clip(g.ptr.data(), const_cast<void *const *>(reinterpret_cast<const void *const *>(out.ptr.data())),
                        g.n.data(), g.dtype.data(), g.ptr.size(), static_cast<float>(max_norm),
                        static_cast<float *>(norm.data_ptr()), work.data_ptr(), stream_of(g.device)),
          "lct_grad_clip");
    for (Py_ssize_t i = 0; i < PySequence_Fast_GET_SIZE(out.seq.o); ++i)
        wrote(tensor(PySequence_Fast_GET_ITEM(out.seq.o, i), "expected tensors"));
    return THPVariable_Wrap(norm);
}

// ----------------------------------------------------------------- adapters

// a, b, scale, ranks or None
lct_adapters bank_of(PyObject *const *o, int *device)
{
    const at::Tensor &a = tensor(o[0], "a must be a tensor"), &b = tensor(o[1], "b must be a tensor");
    const at::Tensor &scale = tensor(o[2], "scale must be a tensor");
    need(a.dim() == 3 && b.dim() == 3 && b.size(0) == a.size(0) && b.size(2) == a.size(1),
         "expected a [adapters, R, k] and b [adapters, n, R]");
    need(a.scalar_type() == at::kBFloat16 && b.scalar_type() == at::kBFloat16, "a and b must be BF16");
    need(scale.scalar_type() == at::kFloat && scale.dim() == 1 && scale.size(0) == a.size(0),
         "scale must be float32 [adapters]");
    *device = a.get_device();
    need(a.is_cuda() && b.is_cuda() && scale.is_cuda() && b.get_device() == *device && scale.get_device() == *device &&
             a.is_contiguous() && b.is_contiguous() && scale.is_contiguous(),
         "the bank's tensors must be contiguous, on one CUDA device");
    lct_adapters k{};
    k.d_a = static_cast<const uint16_t *>(a.data_ptr());
    k.d_b = static_cast<const uint16_t *>(b.data_ptr());
    k.d_scale = static_cast<const float *>(scale.data_ptr());
    if (o[3] != Py_None) {
        const at::Tensor &ranks = tensor(o[3], "ranks must be a tensor or None");
        need(ranks.scalar_type() == at::kInt && ranks.dim() == 1 && ranks.size(0) == a.size(0) && ranks.is_cuda() &&
                 ranks.get_device() == *device && ranks.is_contiguous(),
             "ranks must be contiguous int32 [adapters] on the bank's device");
        k.d_ranks = static_cast<const int32_t *>(ranks.data_ptr());
    }
    k.adapters = static_cast<uint64_t>(a.size(0));
    k.rank = static_cast<uint64_t>(a.size(1));
    k.k = static_cast<uint64_t>(a.size(2));
    k.n = static_cast<uint64_t>(b.size(1));
    return k;
}

// order, starts, tiles
lct_token_plan plan_of(PyObject *const *o, int *device)
{
    const at::Tensor &order = tensor(o[0], "order must be a tensor"), &starts = tensor(o[1], "starts must be a tensor");
    const at::Tensor &tiles = tensor(o[2], "tiles must be a tensor");
    *device = tiles.get_device();
    for (const at::Tensor *t : {&order, &starts, &tiles})
        need(t->is_cuda() && t->scalar_type() == at::kInt && t->is_contiguous() && t->get_device() == *device,
             "the plan's tables must be contiguous int32, on one CUDA device");
    lct_token_plan p{};
    p.tokens = static_cast<uint64_t>(order.numel());
    need(starts.numel() > 2, "the tables do not belong to one plan");
    p.adapters = static_cast<uint64_t>(starts.numel() - 2);
    need(tiles.dim() == 2 && tiles.size(1) == 4 &&
             static_cast<uint64_t>(tiles.size(0)) == LCT_ADAPTER_TILE_ROWS(p.tokens, p.adapters),
         "the tables do not belong to one plan");
    p.d_order = static_cast<const int32_t *>(order.data_ptr());
    p.d_starts = static_cast<const int32_t *>(starts.data_ptr());
    p.d_tiles = static_cast<int32_t *>(tiles.data_ptr());
    return p;
}

struct Rows {
    uint16_t *p = nullptr;
    uint64_t ld = 0;
};

// t [..., cols] as a matrix of `tokens` rows
Rows rows_of(const at::Tensor &t, uint64_t cols, uint64_t tokens, int device, const char *what,
             at::ScalarType type = at::kBFloat16)
{
    const auto sizes = t.sizes(), strides = t.strides();
    const int64_t d = t.dim();
    if (t.scalar_type() != type || !t.is_cuda() || t.get_device() != device || d < 1 ||
        static_cast<uint64_t>(sizes[d - 1]) != cols || static_cast<uint64_t>(t.numel()) != tokens * cols) {
        PyErr_Format(PyExc_ValueError, "%s: expected a %s tensor of %llu rows of %llu on CUDA device %d", what,
                     type == at::kFloat ? "float32" : "BF16", static_cast<unsigned long long>(tokens),
                     static_cast<unsigned long long>(cols), device);
        throw Raised{};
    }
    // leading dimensions that make one row index: each one's stride is the next one's times its size
    bool ok = strides[d - 1] == 1 || cols == 1;
    int64_t ld = static_cast<int64_t>(cols), at = -1;
    for (int64_t i = d - 2; i >= 0; --i) {
        if (sizes[i] == 1) continue;
        if (at < 0)
            ld = strides[i];
        else
            ok = ok && strides[i] == strides[at] * sizes[at];
        at = i;
    }
    if (tokens <= 1) ld = static_cast<int64_t>(cols);
    if (tokens && (!ok || ld < static_cast<int64_t>(cols))) {
        PyErr_Format(PyExc_ValueError, "%s: values of a row must lie side by side, rows at one stride, and not overlap",
                     what);
        throw Raised{};
    }
    return {static_cast<uint16_t *>(t.data_ptr()), static_cast<uint64_t>(ld)};
}

PyObject *tuple_of(std::initializer_list<PyObject *> items)
{
    PyObject *t = PyTuple_New(static_cast<Py_ssize_t>(items.size()));
    Py_ssize_t i = 0;
    for (PyObject *o : items) {
        if (!o || !t) {
            Py_XDECREF(o);
            continue;
        }
        PyTuple_SET_ITEM(t, i++, o);
    }
    return t;
}

// (a, b, scale, ranks) -> (adapters, rank, k, n, device)
PyObject *check_bank(PyObject *const *a)
{
    int device;
    const lct_adapters k = bank_of(a, &device);
    return Py_BuildValue("KKKKi", k.adapters, k.rank, k.k, k.n, device);
}

// (order, starts, tiles) -> (tokens, adapters, device)
PyObject *check_plan(PyObject *const *a)
{
    int device;
    const lct_token_plan p = plan_of(a, &device);
    return Py_BuildValue("KKi", p.tokens, p.adapters, device);
}

// (index, adapters) -> (order, starts, tiles)
PyObject *adapter_plan(PyObject *const *a)
{
    const at::Tensor &index = tensor(a[0], "index must be a tensor");
    need(index.is_cuda() && index.scalar_type() == at::kInt && index.is_contiguous(),
         "index must be a contiguous int32 CUDA tensor");
    const long long adapters = PyLong_AsLongLong(a[1]);
    if (PyErr_Occurred()) throw Raised{};
    if (adapters <= 0) check(LCT_ERR_INVALID_ARG, "lct_adapter_plan");
    if (adapters > LCT_ADAPTER_MAX) check(LCT_ERR_UNSUPPORTED, "lct_adapter_plan");
    const int64_t tokens = index.numel();
    const int device = index.get_device();
    const c10::cuda::CUDAGuard guard(static_cast<c10::DeviceIndex>(device));
    at::Tensor order = make({tokens}, at::kInt, device), starts = make({adapters + 2}, at::kInt, device);
    at::Tensor tiles = make({static_cast<int64_t>(LCT_ADAPTER_TILE_ROWS(tokens, adapters)), 4}, at::kInt, device);
    check(lct_adapter_plan(static_cast<const int32_t *>(index.data_ptr()), static_cast<uint64_t>(tokens),
                           static_cast<uint64_t>(adapters), static_cast<int32_t *>(order.data_ptr()),
                           static_cast<int32_t *>(starts.data_ptr()), static_cast<int32_t *>(tiles.data_ptr()),
                           stream_of(device)),
          "lct_adapter_plan");
    return tuple_of({THPVariable_Wrap(order), THPVariable_Wrap(starts), THPVariable_Wrap(tiles)});
}

// Bank and plan of one call (seven objects), which must belong together.
void bank_and_plan(PyObject *const *o, lct_adapters *bank, lct_token_plan *plan, int *device)
{
    int other;
    *bank = bank_of(o, device);
    *plan = plan_of(o + 4, &other);
    need(plan->adapters == bank->adapters && other == *device,
         "the plan must be for the bank's adapters, on its device");
}

// (a, b, scale, ranks, order, starts, tiles, x, y, out or None, keep) -> out, or (out, xa)
PyObject *adapter_apply(PyObject *const *a)
{
    lct_adapters bank;
    lct_token_plan plan;
    int device;
    bank_and_plan(a, &bank, &plan, &device);
    const at::Tensor &x = tensor(a[7], "x must be a tensor"), &y = tensor(a[8], "y must be a tensor");
    const Rows xr = rows_of(x, bank.k, plan.tokens, device, "x"), yr = rows_of(y, bank.n, plan.tokens, device, "y");
    const bool keep = a[10] == Py_True;
    const c10::cuda::CUDAGuard guard(static_cast<c10::DeviceIndex>(device));
    at::Tensor fresh;
    if (a[9] == Py_None) fresh = make(y.sizes(), at::kBFloat16, device);
    const at::Tensor &out = a[9] == Py_None ? fresh : tensor(a[9], "out must be a tensor or None");
    const Rows outr = rows_of(out, bank.n, plan.tokens, device, "out");
    if (at::GradMode::is_enabled())
        for (const at::Tensor *t : {&x, &y, &out, &tensor(a[0], "a"), &tensor(a[1], "b"), &tensor(a[2], "scale")})
            if (t->requires_grad()) {
                PyErr_SetString(PyExc_RuntimeError, "adapter_apply gives no gradients, but an operand requires one: use "
                                                    "adapter_linear, or call it under torch.no_grad()");
                throw Raised{};
            }
    no_tangent({&x, &y, &out, &tensor(a[0], "a"), &tensor(a[1], "b"), &tensor(a[2], "scale")}, "adapter_apply");
    at::Tensor xa;
    if (keep) xa = make({static_cast<int64_t>(plan.tokens), static_cast<int64_t>(bank.rank)}, at::kFloat, device);
    check(lct_adapter_forward(&bank, &plan, xr.p, xr.ld, yr.p, yr.ld, outr.p, outr.ld,
                              keep ? static_cast<float *>(xa.data_ptr()) : nullptr, stream_of(device)),
          "lct_adapter_forward");
    if (a[9] != Py_None) wrote(out);
    PyObject *res = a[9] == Py_None ? THPVariable_Wrap(fresh) : Py_NewRef(a[9]);
    return keep ? tuple_of({res, THPVariable_Wrap(xa)}) : res;
}

// (a, b, scale, ranks, order, starts, tiles, dy, x, xa, dx or None, out or None) -> (dx' or None, da, db)
PyObject *adapter_grads(PyObject *const *a)
{
    lct_adapters bank;
    lct_token_plan plan;
    int device;
    bank_and_plan(a, &bank, &plan, &device);
    const Rows dy = rows_of(tensor(a[7], "dy must be a tensor"), bank.n, plan.tokens, device, "dy");
    const Rows x = rows_of(tensor(a[8], "x must be a tensor"), bank.k, plan.tokens, device, "x");
    const at::Tensor &xa = tensor(a[9], "xa must be a tensor");
    need(xa.scalar_type() == at::kFloat && xa.dim() == 2 && static_cast<uint64_t>(xa.size(0)) == plan.tokens &&
             static_cast<uint64_t>(xa.size(1)) == bank.rank && xa.is_contiguous() && xa.is_cuda() &&
             xa.get_device() == device,
         "xa: expected contiguous float32 [tokens, R] on the bank's device");
    const c10::cuda::CUDAGuard guard(static_cast<c10::DeviceIndex>(device));
    Rows dx, out;
    at::Tensor fresh;
    const bool wants = a[10] != Py_None, makes = wants && a[11] == Py_None;
    if (wants) {
        const at::Tensor &d = tensor(a[10], "dx must be a tensor or None");
        dx = rows_of(d, bank.k, plan.tokens, device, "dx");
        if (makes) fresh = make(d.sizes(), at::kBFloat16, device);
        out = rows_of(makes ? fresh : tensor(a[11], "out must be a tensor or None"), bank.k, plan.tokens, device, "out");
    }
    const int64_t adapters = static_cast<int64_t>(bank.adapters), rank = static_cast<int64_t>(bank.rank);
    at::Tensor da = make({adapters, rank, static_cast<int64_t>(bank.k)}, at::kBFloat16, device);
    at::Tensor db = make({adapters, static_cast<int64_t>(bank.n), rank}, at::kBFloat16, device);
    at::Tensor work =
        make({static_cast<int64_t>(LCT_ADAPTER_WORK_BYTES(plan.tokens, bank.rank))}, at::kByte, device);
    check(lct_adapter_backward(&bank, &plan, dy.p, dy.ld, x.p, x.ld, static_cast<const float *>(xa.data_ptr()), dx.p,
                               dx.ld, out.p, out.ld, static_cast<uint16_t *>(da.data_ptr()),
                               static_cast<uint16_t *>(db.data_ptr()), work.data_ptr(), stream_of(device)),
          "lct_adapter_backward");
    if (wants && !makes) wrote(tensor(a[11], "out must be a tensor or None"));
    PyObject *first = !wants ? Py_NewRef(Py_None) : makes ? THPVariable_Wrap(fresh) : Py_NewRef(a[11]);
    return tuple_of({first, THPVariable_Wrap(da), THPVariable_Wrap(db)});
}

// ------------------------------------------------------ the vocabulary's ends

// ids of any shape, flattened
lct_ids ids_of(const at::Tensor &t, uint64_t vocab, const char *what)
{
    if (!t.is_cuda() || !t.is_contiguous() || (t.scalar_type() != at::kInt && t.scalar_type() != at::kLong)) {
        PyErr_Format(PyExc_ValueError, "%s: expected a contiguous int32 or int64 CUDA tensor", what);
        throw Raised{};
    }
    lct_ids i{};
    i.d_ids = t.data_ptr();
    i.wide = t.scalar_type() == at::kLong;
    i.tokens = static_cast<uint64_t>(t.numel());
    i.vocab = vocab;
    return i;
}
lct_dtype dtype_of(const at::Tensor &t, const char *what)
{
    if (t.scalar_type() != at::kFloat && t.scalar_type() != at::kBFloat16) check(LCT_ERR_UNSUPPORTED, what);
    return t.scalar_type() == at::kFloat ? LCT_DTYPE_F32 : LCT_DTYPE_BF16;
}
uint64_t number(PyObject *o)
{
    const long long v = PyLong_AsLongLong(o);
    if (PyErr_Occurred()) throw Raised{};
    need(v >= 0, "expected a number that is not negative");
    return static_cast<uint64_t>(v);
}
double real(PyObject *o)
{
    const double v = PyFloat_AsDouble(o);
    if (PyErr_Occurred()) throw Raised{};
    return v;
}
// (ids, table, first, vocab, scale, out or None) -> out; the table's rows are `first` .. of vocab (0: all of them)
PyObject *embedding(PyObject *const *a)
{
    const at::Tensor &idt = tensor(a[0], "tokens must be a tensor"), &table = tensor(a[1], "table must be a tensor");
    need(table.dim() == 2 && table.is_cuda(), "table must be a CUDA tensor [rows, columns]");
    const lct_dtype dtype = dtype_of(table, "tables other than BF16 and float32");
    const uint64_t rows = static_cast<uint64_t>(table.size(0)), cols = static_cast<uint64_t>(table.size(1));
    const uint64_t first = number(a[2]), vocab = number(a[3]);
    const lct_ids ids = ids_of(idt, vocab ? vocab : rows, "tokens");
    const int device = table.get_device();
    need(idt.get_device() == device, "tokens and table must be on one device");
    const Rows tr = rows_of(table, cols, rows, device, "table", table.scalar_type());
    const float scale = static_cast<float>(real(a[4]));
    const c10::cuda::CUDAGuard guard(static_cast<c10::DeviceIndex>(device));
    at::Tensor fresh;
    if (a[5] == Py_None) {
        std::vector<int64_t> shape(idt.sizes().begin(), idt.sizes().end());
        shape.push_back(static_cast<int64_t>(cols));
        fresh = make(shape, table.scalar_type(), device);
    }
    const at::Tensor &out = a[5] == Py_None ? fresh : tensor(a[5], "out must be a tensor or None");
    no_gradient({&table, &out}, a[5] == Py_None ? "embedding" : "embedding into out");
    const Rows outr = rows_of(out, cols, ids.tokens, device, "out", table.scalar_type());
    check(lct_embedding(&ids, tr.p, tr.ld, dtype, first, rows, cols, scale, outr.p, outr.ld, stream_of(device)),
          "lct_embedding");
    if (a[5] == Py_None) return THPVariable_Wrap(fresh);
    wrote(out);
    return Py_NewRef(a[5]);
}

// (dy, ids, rows, scale, base or None, out or None) -> out
PyObject *embedding_grad(PyObject *const *a)
{
    const at::Tensor &dy = tensor(a[0], "dy must be a tensor"), &idt = tensor(a[1], "tokens must be a tensor");
    const uint64_t vocab = number(a[2]);
    const lct_ids ids = ids_of(idt, vocab, "tokens");
    need(dy.is_cuda() && dy.dim() >= 1 && idt.get_device() == dy.get_device(), "dy and tokens must be on one CUDA device");
    const lct_dtype dtype = dtype_of(dy, "gradients other than BF16 and float32");
    const int device = dy.get_device();
    const uint64_t cols = static_cast<uint64_t>(dy.size(dy.dim() - 1));
    const Rows dyr = rows_of(dy, cols, ids.tokens, device, "dy", dy.scalar_type());
    const float scale = static_cast<float>(real(a[3]));
    const c10::cuda::CUDAGuard guard(static_cast<c10::DeviceIndex>(device));
    Rows base;
    if (a[4] != Py_None) {
        const at::Tensor &b = tensor(a[4], "base must be a tensor or None");
        no_gradient({&b}, "embedding_grad");
        base = rows_of(b, cols, vocab, device, "base", dy.scalar_type());
    }
    at::Tensor fresh;
    if (a[5] == Py_None) fresh = make({static_cast<int64_t>(vocab), static_cast<int64_t>(cols)}, dy.scalar_type(), device);
    const at::Tensor &out = a[5] == Py_None ? fresh : tensor(a[5], "out must be a tensor or None");
    no_gradient({&dy, &out}, "embedding_grad");
    const Rows outr = rows_of(out, cols, vocab, device, "out", dy.scalar_type());
    at::Tensor work = make({static_cast<int64_t>(LCT_EMBEDDING_WORK_BYTES(ids.tokens, cols))}, at::kByte, device);
    check(lct_embedding_grad(&ids, dyr.p, dyr.ld, dtype, cols, scale, base.p, base.ld, outr.p, outr.ld, work.data_ptr(),
                             stream_of(device)),
          "lct_embedding_grad");
    if (a[5] == Py_None) return THPVariable_Wrap(fresh);
    wrote(out);
    return Py_NewRef(a[5]);
}

// What a call of the loss works on: x [..., cols], a piece of the weight [rows, cols] that begins at `first` of `vocab`
// rows (0: it is all of it), targets.
struct LossOperands {
    lct_ids ids;
    Rows x, w;
    uint64_t cols, first, rows;
    int device;
    bool unaligned;
};
LossOperands loss_operands(const at::Tensor &x, const at::Tensor &w, const at::Tensor &targets, PyObject *first,
                           PyObject *vocab)
{
    LossOperands o{};
    need(w.dim() == 2 && w.is_cuda(), "weight must be a CUDA tensor [vocabulary, columns]");
    if (w.scalar_type() != at::kBFloat16 || x.scalar_type() != at::kBFloat16)
        check(LCT_ERR_UNSUPPORTED, "x and weights other than BF16");
    o.rows = static_cast<uint64_t>(w.size(0));
    o.cols = static_cast<uint64_t>(w.size(1));
    o.first = number(first);
    const uint64_t all = number(vocab);
    o.device = w.get_device();
    o.ids = ids_of(targets, all ? all : o.rows, "targets");
    need(targets.get_device() == o.device, "targets and weight must be on one device");
    o.w = rows_of(w, o.cols, o.rows, o.device, "weight");
    o.x = rows_of(x, o.cols, o.ids.tokens, o.device, "x");
    const auto odd = [](const Rows &r, uint64_t n) {
        return n && (reinterpret_cast<uintptr_t>(r.p) % 16 || (r.ld % 8 && n > 1));
    };
    o.unaligned = odd(o.x, o.ids.tokens) || odd(o.w, o.rows);
    return o;
}
const at::Tensor &floats(const at::Tensor &t, uint64_t n, int device, const char *what)
{
    if (t.scalar_type() != at::kFloat || !t.is_cuda() || t.get_device() != device || !t.is_contiguous() ||
        static_cast<uint64_t>(t.numel()) != n) {
        PyErr_Format(PyExc_ValueError, "%s: expected contiguous float32, %llu values on CUDA device %d", what,
                     static_cast<unsigned long long>(n), device);
        throw Raised{};
    }
    return t;
}

// x [..., cols], or a weight, as a matrix whose rows the kernels can read: a copy where its leading dimensions make no single
// row index, or a row's values do not lie side by side.
at::Tensor as_rows(const at::Tensor &x, int64_t cols)
{
    at::Tensor r = x.dim() == 2 ? x : x.reshape({-1, cols});
    return r.stride(1) == 1 && r.stride(0) >= cols ? r : r.contiguous();
}

enum { MEAN = 0, SUM = 1, NONE = 2 };

struct Forward {
    at::Tensor loss, lse, total;
};
Forward loss_forward(const at::Tensor &x, const at::Tensor &w, const at::Tensor &targets, bool totals)
{
    const Held zero(PyLong_FromLong(0));
    const LossOperands o = loss_operands(x, w, targets, zero.o, zero.o);
    const c10::cuda::CUDAGuard guard(static_cast<c10::DeviceIndex>(o.device));
    Forward f{make(targets.sizes(), at::kFloat, o.device), make(targets.sizes(), at::kFloat, o.device), {}};
    if (totals) f.total = make({3}, at::kFloat, o.device);
    const uint64_t bytes =
        lct_loss_work_bytes(o.ids.tokens, o.ids.vocab, o.cols, o.rows, o.unaligned ? LCT_LOSS_UNALIGNED : 0);
    at::Tensor work = make({static_cast<int64_t>(bytes)}, at::kByte, o.device);
    check(lct_loss_forward(&o.ids, o.x.p, o.x.ld, o.cols, o.w.p, o.w.ld, 0, o.rows, static_cast<float *>(f.loss.data_ptr()),
                           static_cast<float *>(f.lse.data_ptr()),
                           totals ? static_cast<float *>(f.total.data_ptr()) : nullptr, work.data_ptr(), bytes,
                           stream_of(o.device)),
          "lct_loss_forward");
    return f;
}

// (x, weight, targets) -> (loss, lse)
PyObject *cross_entropy(PyObject *const *a)
{
    const at::Tensor &x = tensor(a[0], "x must be a tensor"), &w = tensor(a[1], "weight must be a tensor");
    no_gradient({&x, &w}, "cross_entropy");
    const Forward f = loss_forward(x, w, tensor(a[2], "targets must be a tensor"), false);
    return tuple_of({THPVariable_Wrap(f.loss), THPVariable_Wrap(f.lse)});
}

// (x, piece, first, vocab, targets, loss, lse, total or None, work) -> None
PyObject *cross_entropy_piece(PyObject *const *a)
{
    const at::Tensor &x = tensor(a[0], "x must be a tensor"), &w = tensor(a[1], "weight must be a tensor");
    no_tangent({&x}, "compressed_cross_entropy");
    const LossOperands o = loss_operands(x, w, tensor(a[4], "targets must be a tensor"), a[2], a[3]);
    const at::Tensor &loss = floats(tensor(a[5], "loss must be a tensor"), o.ids.tokens, o.device, "loss");
    const at::Tensor &lse = floats(tensor(a[6], "lse must be a tensor"), o.ids.tokens, o.device, "lse");
    float *total = a[7] == Py_None ? nullptr : static_cast<float *>(floats(tensor(a[7], "total must be a tensor or None"), 3, o.device, "total").data_ptr());
    const at::Tensor &work = tensor(a[8], "work must be a tensor");
    const c10::cuda::CUDAGuard guard(static_cast<c10::DeviceIndex>(o.device));
    check(lct_loss_forward(&o.ids, o.x.p, o.x.ld, o.cols, o.w.p, o.w.ld, o.first, o.rows,
                           static_cast<float *>(loss.data_ptr()), static_cast<float *>(lse.data_ptr()), total,
                           work.data_ptr(), static_cast<uint64_t>(work.numel()), stream_of(o.device)),
          "lct_loss_forward");
    Py_RETURN_NONE;
}

struct Upstream {
    const float *dloss, *scale;
    uint64_t stride;
};
// dloss: a value a token, or one for all; scale: a value that all are multiplied by, or undefined
Upstream upstream_of(const at::Tensor &dloss, const at::Tensor &scale, uint64_t tokens, int device)
{
    Upstream u{};
    u.stride = dloss.numel() == 1 && tokens != 1 ? 0 : 1;
    u.dloss = static_cast<const float *>(floats(dloss, u.stride ? tokens : 1, device, "dloss").data_ptr());
    if (scale.defined()) u.scale = static_cast<const float *>(floats(scale, 1, device, "scale").data_ptr());
    return u;
}
at::Tensor maybe(PyObject *o, const char *what) { return o == Py_None ? at::Tensor() : tensor(o, what); }

struct Backward {
    at::Tensor dx, dw;
};
Backward loss_backward(const at::Tensor &x, const at::Tensor &w, const at::Tensor &targets, const at::Tensor &loss,
                       const at::Tensor &lse, const at::Tensor &dloss, const at::Tensor &scale, bool weight)
{
    const Held zero(PyLong_FromLong(0));
    const LossOperands o = loss_operands(x, w, targets, zero.o, zero.o);
    floats(loss, o.ids.tokens, o.device, "loss");
    floats(lse, o.ids.tokens, o.device, "lse");
    const Upstream u = upstream_of(dloss, scale, o.ids.tokens, o.device);
    const c10::cuda::CUDAGuard guard(static_cast<c10::DeviceIndex>(o.device));
    Backward b{make(x.sizes(), at::kBFloat16, o.device), {}};
    if (weight) b.dw = make(w.sizes(), at::kBFloat16, o.device);
    const uint64_t bytes = lct_loss_work_bytes(
        o.ids.tokens, o.ids.vocab, o.cols, o.rows,
        LCT_LOSS_BACKWARD | (weight ? LCT_LOSS_WEIGHT : 0) | (o.unaligned ? LCT_LOSS_UNALIGNED : 0));
    at::Tensor work = make({static_cast<int64_t>(bytes)}, at::kByte, o.device);
    check(lct_loss_backward(&o.ids, o.x.p, o.x.ld, o.cols, o.w.p, o.w.ld, 0, o.rows,
                            static_cast<const float *>(loss.data_ptr()), static_cast<const float *>(lse.data_ptr()), u.dloss,
                            u.stride, u.scale, static_cast<uint16_t *>(b.dx.data_ptr()), o.cols,
                            weight ? static_cast<uint16_t *>(b.dw.data_ptr()) : nullptr, o.cols, work.data_ptr(), bytes,
                            stream_of(o.device)),
          "lct_loss_backward");
    return b;
}

// (x, weight, targets, loss, lse, dloss, weight_grad) -> (dx, dw or None)
PyObject *cross_entropy_grads(PyObject *const *a)
{
    const at::Tensor &x = tensor(a[0], "x must be a tensor"), &w = tensor(a[1], "weight must be a tensor");
    const at::Tensor &loss = tensor(a[3], "loss must be a tensor"), &lse = tensor(a[4], "lse must be a tensor");
    const at::Tensor &dloss = tensor(a[5], "dloss must be a tensor");
    no_gradient({&x, &w, &loss, &lse, &dloss}, "cross_entropy_grads");
    const Backward b =
        loss_backward(x, w, tensor(a[2], "targets must be a tensor"), loss, lse, dloss, at::Tensor(), a[6] == Py_True);
    return tuple_of({THPVariable_Wrap(b.dx), b.dw.defined() ? THPVariable_Wrap(b.dw) : Py_NewRef(Py_None)});
}

// The mean or sum in a tensor of its own, which shares its memory with the three totals.
at::Tensor reduced(const Forward &f, int reduction)
{
    if (reduction == NONE) return f.loss;
    at::Tensor r = at::empty({0}, f.total.options());
    r.set_(f.total.storage(), reduction == MEAN ? 1 : 0, {}, {});
    return r;
}

// Under autograd by torch's C++ side: its Python side takes longer than the kernels of a small step.  A Python error that
// the checks set is handed on as torch's.
[[noreturn]] void as_torch_error()
{
    PyGILState_STATE gil = PyGILState_Ensure();
    PyObject *type, *value, *trace;
    PyErr_Fetch(&type, &value, &trace);
    PyObject *text = value ? PyObject_Str(value) : nullptr;
    const char *c = text ? PyUnicode_AsUTF8(text) : nullptr;
    const std::string what = c ? c : "linear_cross_entropy failed";
    Py_XDECREF(text);
    Py_XDECREF(type);
    Py_XDECREF(value);
    Py_XDECREF(trace);
    PyErr_Clear();
    PyGILState_Release(gil);
    TORCH_CHECK(false, what);
}

struct LinearCrossEntropy : torch::autograd::Function<LinearCrossEntropy> {
    static at::Tensor forward(torch::autograd::AutogradContext *ctx, const at::Tensor &x, const at::Tensor &w,
                              const at::Tensor &targets, int64_t reduction)
    {
        const at::Tensor rows = as_rows(x, w.size(1)), weight = as_rows(w, w.size(1));
        const Forward f = loss_forward(rows, weight, targets, true);
        ctx->save_for_backward({rows, weight, targets, f.loss, f.lse, f.total});
        ctx->saved_data["reduction"] = reduction;
        ctx->saved_data["shape"] = x.sizes().vec();
        // (a token's losses are also saved: autograd has to be able to give the caller a tensor of its own)
        return reduction == NONE ? f.loss.clone() : reduced(f, static_cast<int>(reduction));
    }
    static torch::autograd::variable_list backward(torch::autograd::AutogradContext *ctx, torch::autograd::variable_list dy)
    {
        const auto saved = ctx->get_saved_variables();
        const int64_t reduction = ctx->saved_data["reduction"].toInt();
        torch::autograd::variable_list grads(4);
        {
            const at::AutoGradMode off(false);
            at::Tensor dloss = dy[0].to(at::kFloat).contiguous();
            const at::Tensor scale = reduction == MEAN ? saved[5].slice(0, 2, 3) : at::Tensor();
            Backward b;
            try {
                const PyGILState_STATE gil = PyGILState_Ensure();
                struct Release {
                    PyGILState_STATE gil;
                    ~Release() { PyGILState_Release(gil); }
                } release{gil};
                b = loss_backward(saved[0], saved[1], saved[2], saved[3], saved[4], dloss, scale, ctx->needs_input_grad(1));
            } catch (const Raised &) {
                as_torch_error();
            }
            if (ctx->needs_input_grad(0)) grads[0] = b.dx.view(ctx->saved_data["shape"].toIntVector());
            if (ctx->needs_input_grad(1)) grads[1] = b.dw;
        }
        // The gradients' own gradients are not there: asking for them raises.  They depend on the operands whatever the
        // saved ones (which may be copies that autograd has not seen) and the upstream say.
        if (at::GradMode::is_enabled()) {
            torch::autograd::variable_list some;
            for (const at::Tensor &g : grads)
                if (g.defined()) some.push_back(g.set_requires_grad(true));
            const auto error = std::make_shared<torch::autograd::DelayedError>(
                "linear_cross_entropy is differentiable once", static_cast<int64_t>(some.size()));
            some = (*error)(std::move(some));
            size_t i = 0;
            for (at::Tensor &g : grads)
                if (g.defined()) g = some[i++];
        }
        return grads;
    }
};

// (x, weight, targets, reduction) -> loss
PyObject *linear_cross_entropy(PyObject *const *a)
{
    const at::Tensor &x = tensor(a[0], "x must be a tensor"), &w = tensor(a[1], "weight must be a tensor");
    const at::Tensor &targets = tensor(a[2], "targets must be a tensor");
    const int reduction = static_cast<int>(number(a[3]));
    no_tangent({&x, &w}, "linear_cross_entropy");
    need(w.dim() == 2 && x.dim() >= 1 && x.size(x.dim() - 1) == w.size(1), "expected x [..., columns] and weight [vocabulary, columns]");
    if (at::GradMode::is_enabled() && (x.requires_grad() || w.requires_grad()))
        return THPVariable_Wrap(LinearCrossEntropy::apply(x, w, targets, static_cast<int64_t>(reduction)));
    return THPVariable_Wrap(reduced(loss_forward(as_rows(x, w.size(1)), as_rows(w, w.size(1)), targets, true), reduction));
}

// (x, piece, first, vocab, targets, loss, lse, dloss, scale or None, dx, dw's piece or None, work) -> None
PyObject *cross_entropy_grads_piece(PyObject *const *a)
{
    const at::Tensor &x = tensor(a[0], "x must be a tensor"), &w = tensor(a[1], "weight must be a tensor");
    const LossOperands o = loss_operands(x, w, tensor(a[4], "targets must be a tensor"), a[2], a[3]);
    const at::Tensor &loss = floats(tensor(a[5], "loss must be a tensor"), o.ids.tokens, o.device, "loss");
    const at::Tensor &lse = floats(tensor(a[6], "lse must be a tensor"), o.ids.tokens, o.device, "lse");
    const at::Tensor scale = maybe(a[8], "scale must be a tensor or None");
    const Upstream u = upstream_of(tensor(a[7], "dloss must be a tensor"), scale, o.ids.tokens, o.device);
    const Rows dx = rows_of(tensor(a[9], "dx must be a tensor"), o.cols, o.ids.tokens, o.device, "dx");
    Rows dw;
    if (a[10] != Py_None) dw = rows_of(tensor(a[10], "dw must be a tensor or None"), o.cols, o.rows, o.device, "dw");
    const at::Tensor &work = tensor(a[11], "work must be a tensor");
    const c10::cuda::CUDAGuard guard(static_cast<c10::DeviceIndex>(o.device));
    check(lct_loss_backward(&o.ids, o.x.p, o.x.ld, o.cols, o.w.p, o.w.ld, o.first, o.rows,
                            static_cast<const float *>(loss.data_ptr()), static_cast<const float *>(lse.data_ptr()), u.dloss,
                            u.stride, u.scale, dx.p, dx.ld, dw.p, dw.ld, work.data_ptr(),
                            static_cast<uint64_t>(work.numel()), stream_of(o.device)),
          "lct_loss_backward");
    Py_RETURN_NONE;
}

// (tokens, vocab, cols, rows, flags) -> bytes
PyObject *loss_work_bytes(PyObject *const *a)
{
    return PyLong_FromUnsignedLongLong(lct_loss_work_bytes(number(a[0]), number(a[1]), number(a[2]), number(a[3]),
                                                           static_cast<int32_t>(number(a[4]))));
}

// (LctError)
PyObject *set_error(PyObject *const *a)
{
    g_error = Py_NewRef(a[0]);
    Py_RETURN_NONE;
}

// No C++ exception leaves a call: errors of torch (out of memory) become Python's.
template <PyObject *(*F)(PyObject *const *), Py_ssize_t COUNT>
PyObject *entry(PyObject *, PyObject *const *args, Py_ssize_t n)
{
    if (n != COUNT) {
        PyErr_Format(PyExc_TypeError, "expected %zd arguments", COUNT);
        return nullptr;
    }
    try {
        return F(args);
    } catch (const Raised &) {
    } catch (const std::exception &e) {
        PyErr_SetString(PyExc_RuntimeError, e.what());
    }
    return nullptr;
}

template <PyObject *(*F)(PyObject *const *), Py_ssize_t COUNT>
constexpr PyMethodDef method(const char *name)
{
    return {name, reinterpret_cast<PyCFunction>(reinterpret_cast<void *>(entry<F, COUNT>)), METH_FASTCALL, nullptr};
}

PyMethodDef methods[] = {method<grad_norm, 1>("grad_norm"),
                         method<clip_grads, 3>("clip_grads"),
                         method<check_bank, 4>("check_bank"),
                         method<check_plan, 3>("check_plan"),
                         method<adapter_plan, 2>("adapter_plan"),
                         method<adapter_apply, 11>("adapter_apply"),
                         method<adapter_grads, 12>("adapter_grads"),
                         method<embedding, 6>("embedding"),
                         method<embedding_grad, 6>("embedding_grad"),
                         method<cross_entropy, 3>("cross_entropy"),
                         method<cross_entropy_piece, 9>("cross_entropy_piece"),
                         method<cross_entropy_grads, 7>("cross_entropy_grads"),
                         method<linear_cross_entropy, 4>("linear_cross_entropy"),
                         method<cross_entropy_grads_piece, 12>("cross_entropy_grads_piece"),
                         method<loss_work_bytes, 5>("loss_work_bytes"),
                         method<set_error, 1>("set_error"),
                         {nullptr, nullptr, 0, nullptr}};

PyModuleDef definition = {PyModuleDef_HEAD_INIT, "_calls", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__calls() { return PyModule_Create(&definition); }
