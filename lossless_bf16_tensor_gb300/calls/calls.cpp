// Python entry points of the gradient and adapter calls: tensors in, checks,
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
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
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
Rows rows_of(const at::Tensor &t, uint64_t cols, uint64_t tokens, int device, const char *what)
{
    const auto sizes = t.sizes(), strides = t.strides();
    const int64_t d = t.dim();
    if (t.scalar_type() != at::kBFloat16 || !t.is_cuda() || t.get_device() != device || d < 1 ||
        static_cast<uint64_t>(sizes[d - 1]) != cols || static_cast<uint64_t>(t.numel()) != tokens * cols) {
        PyErr_Format(PyExc_ValueError, "%s: expected a BF16 tensor of %llu rows of %llu on CUDA device %d", what,
                     static_cast<unsigned long long>(tokens), static_cast<unsigned long long>(cols), device);
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
                         method<set_error, 1>("set_error"),
                         {nullptr, nullptr, 0, nullptr}};

PyModuleDef definition = {PyModuleDef_HEAD_INIT, "_calls", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__calls() { return PyModule_Create(&definition); }
