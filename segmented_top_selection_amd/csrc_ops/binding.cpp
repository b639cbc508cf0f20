// binding.cpp -- the operators around the selection for torch tensors: checks of
// the arguments, outputs and workspaces from torch's allocator, and the call of
// the C library on the current stream.
//
// A decode step calls these for microseconds of work each, so the host's share
// counts: marshalled here a call costs about half of what it does in Python.
// The Python functions in model_ops carry the documentation and the stream; the
// library's functions are looked up in the file that the package has loaded.
#include <dlfcn.h>

#include <string>

#include <ATen/core/Tensor.h>
#include <ATen/ops/empty.h>
#include <c10/core/DeviceGuard.h>
#include <c10/hip/HIPStream.h>
#include <torch/csrc/DynamicTypes.h>
#include <torch/csrc/Dtype.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include "segtopk.h"

namespace {

using at::ScalarType;
using at::Tensor;

struct Library {
    decltype(&segtopk_sort_ids_workspace) sort_ids_workspace;
    decltype(&segtopk_sort_ids) sort_ids;
    decltype(&segtopk_dispatch_rows) dispatch_rows;
    decltype(&segtopk_combine_rows) combine_rows;
    decltype(&segtopk_combine_rows_backward) combine_rows_backward;
    decltype(&segtopk_embedding_rows) embedding_rows;
    decltype(&segtopk_embedding_backward_workspace) embedding_backward_workspace;
    decltype(&segtopk_embedding_backward) embedding_backward;
    decltype(&segtopk_policy_loss_workspace) policy_loss_workspace;
    decltype(&segtopk_policy_loss) policy_loss;
    decltype(&segtopk_route) route;
    decltype(&segtopk_route_backward) route_backward;
    decltype(&segtopk_quantize_rows) quantize_rows;
    decltype(&segtopk_quantize_blocks) quantize_blocks;
    decltype(&segtopk_expert_matmul) expert_matmul;
    decltype(&segtopk_expert_dweights_workspace) expert_dweights_workspace;
    decltype(&segtopk_expert_dweights) expert_dweights;
    decltype(&segtopk_verify_workspace) verify_workspace;
    decltype(&segtopk_verify_drafts) verify_drafts;
} lib;
PyObject *call_error;  // (status, name of the call) -> the exception

// ---- arguments ----------------------------------------------------------
int float_code(ScalarType t) {
    switch (t) {
    case ScalarType::Float: return SEGTOPK_KEY_F32;
    case ScalarType::BFloat16: return SEGTOPK_KEY_BF16;
    case ScalarType::Half: return SEGTOPK_KEY_F16;
    default: return -1;
    }
}

std::string type_name(ScalarType t) {
    PyObject *s = PyObject_Str(reinterpret_cast<PyObject *>(torch::getTHPDtype(t)));
    if (!s) throw python_error();
    const char *c = PyUnicode_AsUTF8(s);
    std::string r = c ? c : "";
    Py_DECREF(s);
    return r;
}

std::string shape_name(at::IntArrayRef s) {
    std::string r = "(";
    for (size_t i = 0; i < s.size(); ++i) r += (i ? ", " : "") + std::to_string(s[i]);
    return r + (s.size() == 1 ? ",)" : ")");
}

const Tensor &tensor(const char *name, PyObject *o) {
    TORCH_CHECK_TYPE(THPVariable_Check(o), name, " must be a torch tensor");
    return THPVariable_Unpack(o);
}

// The call's first tensor, which says what device it runs on.
const Tensor &device_tensor(const char *name, PyObject *o) {
    const Tensor &t = tensor(name, o);
    TORCH_CHECK_VALUE(t.is_cuda(), name, " must be a device tensor (got ", t.device().str(), ")");
    return t;
}

const Tensor &there(const char *name, PyObject *o, at::Device dev) {
    const Tensor &t = tensor(name, o);
    TORCH_CHECK_VALUE(t.device() == dev, name, " must be a device tensor on ", dev.str(), " (got ",
                      t.device().str(), ")");
    return t;
}

bool given(PyObject *o) { return o != Py_None; }

int64_t integer(PyObject *o) {
    // Integers of any kind; no text, and nothing that would lose its fraction.
    PyObject *i = PyNumber_Index(o);
    if (!i) throw python_error();
    const int64_t v = PyLong_AsLongLong(i);
    Py_DECREF(i);
    if (v == -1 && PyErr_Occurred()) throw python_error();
    return v;
}

// Before outputs of that many entries are allocated.
void check_count(const char *name, int64_t v) {
    TORCH_CHECK_VALUE(v >= 0 && v < INT32_MAX, name, " must be >= 0 and below 2^31 - 1 (got ", v, ")");
}

double real(PyObject *o) {
    const double v = PyFloat_AsDouble(o);
    if (v == -1.0 && PyErr_Occurred()) throw python_error();
    return v;
}

// Rows with a unit inner stride that do not overlap.
bool plain_rows(const Tensor &t) {
    const auto s = t.sizes(), d = t.strides();
    return (d[1] == 1 || s[1] <= 1) && (d[0] >= s[1] || s[0] <= 1);
}

// The stride of a single row is never used, and torch may say anything.
segtopk_rows view(const Tensor &t) {
    const int64_t width = t.size(1), stride = t.stride(0);
    return {t.data_ptr(), stride > width ? stride : width, float_code(t.scalar_type())};
}

struct Matrix {
    Tensor t;
    int64_t rows, width;
    segtopk_rows v;
};

// A matrix that the call reads; other layouts are copied.
Matrix matrix(const char *name, const Tensor &t) {
    TORCH_CHECK_TYPE(float_code(t.scalar_type()) >= 0, name,
                     " must be float32, bfloat16 or float16 (got ", type_name(t.scalar_type()), ")");
    TORCH_CHECK_VALUE(t.dim() == 2, name, " must have shape (rows, width) (got ",
                      shape_name(t.sizes()), ")");
    TORCH_CHECK_VALUE(t.size(1) >= 1, name, " must be at least one element wide");
    Matrix m{plain_rows(t) ? t : t.contiguous(), t.size(0), t.size(1), {}};
    m.v = view(m.t);
    return m;
}

Tensor fresh(at::IntArrayRef shape, ScalarType type, at::Device dev) {
    return at::empty(shape, at::TensorOptions().dtype(type).device(dev));
}

// An output matrix that the caller gave, checked, or a new one.
Matrix result(const char *name, PyObject *o, at::Device dev, int64_t rows, int64_t width,
              ScalarType type) {
    if (!given(o)) {
        Matrix m{fresh({rows, width}, type, dev), rows, width, {}};
        m.v = {m.t.data_ptr(), width, float_code(type)};
        return m;
    }
    const Tensor &t = there(name, o, dev);
    TORCH_CHECK_TYPE(t.scalar_type() == type, name, " must be ", type_name(type), " (got ",
                     type_name(t.scalar_type()), ")");
    TORCH_CHECK_VALUE(t.dim() == 2 && t.size(0) == rows && t.size(1) == width, name,
                      " must have shape ", shape_name({rows, width}), " (got ",
                      shape_name(t.sizes()), ")");
    TORCH_CHECK_VALUE(plain_rows(t), name,
                      " must have a unit inner stride and rows that do not overlap");
    return {t, rows, width, view(t)};
}

struct Ids {
    Tensor t;
    int code;
};

Ids ids_of(const char *name, const Tensor &t) {
    const ScalarType type = t.scalar_type();
    TORCH_CHECK_TYPE(type == ScalarType::Int || type == ScalarType::Long, name,
                     " must be int32 or int64 (got ", type_name(type), ")");
    return {t.contiguous(), type == ScalarType::Long ? SEGTOPK_KEY_I64 : SEGTOPK_KEY_I32};
}

Tensor vector(const char *name, PyObject *o, at::Device dev, int64_t n) {
    const Tensor &t = there(name, o, dev);
    TORCH_CHECK_TYPE(t.scalar_type() == ScalarType::Float, name, " must be torch.float32 (got ",
                     type_name(t.scalar_type()), ")");
    TORCH_CHECK_VALUE(t.dim() == 1 && t.size(0) == n, name, " must have shape ", shape_name({n}),
                      " (got ", shape_name(t.sizes()), ")");
    return t.contiguous();
}

Tensor offsets_of(const char *name, PyObject *o, at::Device dev) {
    const Tensor &t = there(name, o, dev);
    TORCH_CHECK_TYPE(t.scalar_type() == ScalarType::Long, name, " must be int64 (got ",
                     type_name(t.scalar_type()), ")");
    TORCH_CHECK_VALUE(t.dim() == 1 && t.size(0) >= 1, name,
                      " must be 1-D with num_segments + 1 entries");
    return t.contiguous();
}

struct Slots {
    Tensor position, offsets;
    int64_t tokens, k;
    const int32_t *at;
    const int64_t *kept;  // the number of slots kept, or nullptr: all
};

Slots slots(PyObject *position, PyObject *offsets, at::Device dev) {
    const Tensor &p = there("position", position, dev);
    TORCH_CHECK_TYPE(p.scalar_type() == ScalarType::Int, "position must be int32 (got ",
                     type_name(p.scalar_type()), ")");
    TORCH_CHECK_VALUE(p.dim() == 1 || p.dim() == 2,
                      "position must have shape (tokens, k) or (tokens,)");
    Slots s{p.contiguous(), {}, p.size(0), p.dim() == 2 ? p.size(1) : 1, nullptr, nullptr};
    TORCH_CHECK_VALUE(s.k >= 1, "position needs at least one slot a token");
    s.at = static_cast<const int32_t *>(s.position.data_ptr());
    if (given(offsets)) {
        s.offsets = offsets_of("offsets", offsets, dev);
        s.kept = static_cast<const int64_t *>(s.offsets.data_ptr()) + s.offsets.size(0) - 1;
    }
    return s;
}

struct Weights {
    Tensor t;
    void *data;
    int code;
};

Weights weights_of(PyObject *o, at::Device dev, const Tensor &position, ScalarType type) {
    if (!given(o)) return {{}, nullptr, SEGTOPK_KEY_F32};
    const Tensor &t = there("weights", o, dev);
    TORCH_CHECK_TYPE(t.scalar_type() == ScalarType::Float || t.scalar_type() == type,
                     "weights must be float32 or ", type_name(type), " (got ",
                     type_name(t.scalar_type()), ")");
    TORCH_CHECK_VALUE(t.sizes() == position.sizes(), "weights must have position's shape ",
                      shape_name(position.sizes()), " (got ", shape_name(t.sizes()), ")");
    Weights w{t.contiguous(), nullptr, float_code(t.scalar_type())};
    w.data = w.t.data_ptr();
    return w;
}

struct Workspace {
    Tensor t;
    void *data;
    int64_t bytes;
};

// torch's blocks are aligned to 512 bytes.
Workspace workspace(int64_t bytes, at::Device dev) {
    Workspace w{{}, nullptr, bytes};
    if (bytes) {
        w.t = fresh({bytes}, ScalarType::Byte, dev);
        w.data = w.t.data_ptr();
    }
    return w;
}

// Runs f, which returns a status, without the interpreter's lock: a launch waits
// where the device's queue is full.
template <class F> void call(const char *name, at::Device dev, F f) {
    const hipStream_t stream = c10::hip::getCurrentHIPStream(dev.index()).stream();
    PyThreadState *const state = PyEval_SaveThread();
    const int status = f(stream);  // throws nothing
    PyEval_RestoreThread(state);
    if (status == SEGTOPK_OK) return;
    PyObject *e = PyObject_CallFunction(call_error, "is", status, name);
    if (e) {
        PyErr_SetObject(reinterpret_cast<PyObject *>(Py_TYPE(e)), e);
        Py_DECREF(e);
    }
    throw python_error();
}

// A tuple of what the pointers own; None stays.
template <class... Objects> PyObject *tuple(Objects... objects) {
    PyObject *const all[] = {objects...};
    PyObject *t = PyTuple_New(sizeof...(objects));
    bool whole = t;
    for (PyObject *o : all) whole = whole && o;
    if (!whole) {
        Py_XDECREF(t);
        for (PyObject *o : all) Py_XDECREF(o);
        return nullptr;
    }
    Py_ssize_t i = 0;
    for (PyObject *o : all) PyTuple_SET_ITEM(t, i++, o);
    return t;
}

PyObject *same(PyObject *o) {
    Py_INCREF(o);
    return o;
}

// The tensor that the caller gave, or the new one.  Autograd is told that the
// caller's was written, so that a graph that keeps it refuses to go on.
PyObject *output(PyObject *o, const Tensor &t) {
    if (!given(o)) return THPVariable_Wrap(t);
    if (!t.is_inference()) t.unsafeGetTensorImpl()->bump_version();
    return same(o);
}

// ---- the calls ----------------------------------------------------------
// Arguments come by position from model_ops, None for those not given.
PyObject *sort_ids(PyObject *const *a) {
    const Tensor &given_ids = device_tensor("ids", a[0]);
    const at::Device dev = given_ids.device();
    const c10::DeviceGuard guard(dev);
    const Ids ids = ids_of("ids", given_ids);
    const int64_t n = ids.t.numel(), segments = integer(a[1]);
    check_count("num_segments", segments);
    const Tensor order = fresh({n}, ScalarType::Int, dev);
    const Tensor position = fresh(ids.t.sizes(), ScalarType::Int, dev);
    const Tensor offsets = fresh({segments + 1}, ScalarType::Long, dev);
    const Workspace ws = workspace(lib.sort_ids_workspace(n, segments), dev);
    const void *const in = ids.t.data_ptr();
    int32_t *const o = static_cast<int32_t *>(order.data_ptr());
    int32_t *const p = static_cast<int32_t *>(position.data_ptr());
    int64_t *const f = static_cast<int64_t *>(offsets.data_ptr());
    call("segtopk_sort_ids", dev, [&](hipStream_t stream) {
        return lib.sort_ids(in, ids.code, n, segments, o, p, f, ws.data, ws.bytes, stream);
    });
    return tuple(THPVariable_Wrap(order), THPVariable_Wrap(position), THPVariable_Wrap(offsets));
}

PyObject *dispatch(PyObject *const *a) {
    const Tensor &given_x = device_tensor("x", a[0]);
    const at::Device dev = given_x.device();
    const c10::DeviceGuard guard(dev);
    const Matrix x = matrix("x", given_x);
    const Slots s = slots(a[1], a[2], dev);
    TORCH_CHECK_VALUE(x.rows == s.tokens, "position is for ", s.tokens, " tokens, x has ", x.rows,
                      " rows");
    const Matrix out = result("out", a[3], dev, s.tokens * s.k, x.width, x.t.scalar_type());
    call("segtopk_dispatch_rows", dev, [&](hipStream_t stream) {
        return lib.dispatch_rows(&x.v, &out.v, s.tokens, s.k, x.width, s.at, s.kept, stream);
    });
    return output(a[3], out.t);
}

PyObject *combine(PyObject *const *a) {
    const Tensor &given_rows = device_tensor("rows", a[0]);
    const at::Device dev = given_rows.device();
    const c10::DeviceGuard guard(dev);
    const Slots s = slots(a[1], a[2], dev);
    const Matrix rows = matrix("rows", given_rows);
    TORCH_CHECK_VALUE(rows.rows == s.tokens * s.k, "rows must have tokens * k = ", s.tokens * s.k,
                      " rows (got ", rows.rows, ")");
    const ScalarType type = rows.t.scalar_type();
    const Weights w = weights_of(a[3], dev, s.position, type);
    const Matrix out = result("out", a[4], dev, s.tokens, rows.width, type);
    call("segtopk_combine_rows", dev, [&](hipStream_t stream) {
        return lib.combine_rows(&rows.v, &out.v, w.data, w.code, s.tokens, s.k, rows.width, s.at,
                                s.kept, stream);
    });
    return output(a[4], out.t);
}

PyObject *combine_backward(PyObject *const *a) {
    const Tensor &given_dout = device_tensor("dout", a[0]);
    const at::Device dev = given_dout.device();
    const c10::DeviceGuard guard(dev);
    const Slots s = slots(a[2], a[3], dev);
    const Matrix dout = matrix("dout", given_dout);
    TORCH_CHECK_VALUE(dout.rows == s.tokens, "position is for ", s.tokens, " tokens, dout has ",
                      dout.rows, " rows");
    const ScalarType type = dout.t.scalar_type();
    const Weights w = weights_of(a[4], dev, s.position, type);
    Matrix rows{};
    Tensor dweights;
    const bool both = given(a[1]);
    if (both) {
        rows = matrix("rows", there("rows", a[1], dev));
        TORCH_CHECK_TYPE(rows.t.scalar_type() == type, "rows must be ", type_name(type), " (got ",
                         type_name(rows.t.scalar_type()), ")");
        TORCH_CHECK_VALUE(rows.rows == s.tokens * s.k && rows.width == dout.width,
                          "rows must have shape ", shape_name({s.tokens * s.k, dout.width}),
                          " (got ", shape_name({rows.rows, rows.width}), ")");
        dweights = fresh(s.position.sizes(), w.data ? w.t.scalar_type() : ScalarType::Float, dev);
    }
    const Matrix out = result("out", a[5], dev, s.tokens * s.k, dout.width, type);
    void *const dw = both ? dweights.data_ptr() : nullptr;
    call("segtopk_combine_rows_backward", dev, [&](hipStream_t stream) {
        return lib.combine_rows_backward(&dout.v, both ? &rows.v : nullptr, &out.v, w.data, dw,
                                         w.code, s.tokens, s.k, dout.width, s.at, s.kept, stream);
    });
    return tuple(output(a[5], out.t), both ? THPVariable_Wrap(dweights) : same(Py_None));
}

PyObject *embedding(PyObject *const *a) {
    const Tensor &given_table = device_tensor("table", a[0]);
    const at::Device dev = given_table.device();
    const c10::DeviceGuard guard(dev);
    const Matrix table = matrix("table", given_table);
    const Ids ids = ids_of("ids", there("ids", a[1], dev));
    const float scale = static_cast<float>(real(a[2]));
    const int64_t n = ids.t.numel();
    const Matrix out = result("out", a[3], dev, n, table.width, table.t.scalar_type());
    const void *const in = ids.t.data_ptr();
    call("segtopk_embedding_rows", dev, [&](hipStream_t stream) {
        return lib.embedding_rows(&table.v, &out.v, in, ids.code, n, table.rows, table.width, scale,
                                  stream);
    });
    if (given(a[3]) || ids.t.dim() == 1) return output(a[3], out.t);
    auto shape = ids.t.sizes().vec();
    shape.push_back(table.width);
    return THPVariable_Wrap(out.t.view(shape));
}

PyObject *embedding_backward(PyObject *const *a) {
    const Tensor &given_dout = device_tensor("dout", a[0]);
    const at::Device dev = given_dout.device();
    const c10::DeviceGuard guard(dev);
    const Ids ids = ids_of("ids", there("ids", a[1], dev));
    const int64_t n = ids.t.numel(), num_rows = integer(a[2]);
    check_count("num_rows", num_rows);
    const bool deep = given_dout.dim() != 2 && given_dout.dim() >= 1 &&
                      given_dout.sizes().slice(0, given_dout.dim() - 1) == ids.t.sizes();
    const Matrix dout = matrix("dout", deep ? given_dout.reshape({n, given_dout.size(-1)}) : given_dout);
    TORCH_CHECK_VALUE(dout.rows == n, "dout must have one row an id (", n, "; got ", dout.rows, ")");
    const float scale = static_cast<float>(real(a[3]));
    const int64_t padding = given(a[4]) ? integer(a[4]) : -1;
    const int accumulate = PyObject_IsTrue(a[7]);
    if (accumulate < 0) throw python_error();
    TORCH_CHECK_VALUE(!accumulate || given(a[6]), "accumulate needs out");
    ScalarType type = dout.t.scalar_type();
    if (given(a[5])) {
        TORCH_CHECK_TYPE(THPDtype_Check(a[5]), "dtype must be a torch.dtype");
        type = reinterpret_cast<THPDtype *>(a[5])->scalar_type;
    } else if (given(a[6])) {
        type = tensor("out", a[6]).scalar_type();
    }
    TORCH_CHECK_TYPE(type == dout.t.scalar_type() || type == ScalarType::Float,
                     "the gradient must be float32 or ", type_name(dout.t.scalar_type()), " (got ",
                     type_name(type), ")");
    const Matrix out = result("out", a[6], dev, num_rows, dout.width, type);
    const Workspace ws = workspace(lib.embedding_backward_workspace(n, num_rows, dout.width), dev);
    const void *const in = ids.t.data_ptr();
    call("segtopk_embedding_backward", dev, [&](hipStream_t stream) {
        return lib.embedding_backward(&dout.v, &out.v, in, ids.code, n, num_rows, dout.width, scale,
                                      padding, accumulate, ws.data, ws.bytes, stream);
    });
    return output(a[6], out.t);
}

// logits, token_ids, old_logp, advantages, segment_offsets, ref_logp, kl_coef,
// clip_low, clip_high, temperature, grad_scale, dlogits, whether to give them
PyObject *policy_loss(PyObject *const *a) {
    const Tensor &given_logits = device_tensor("logits", a[0]);
    const at::Device dev = given_logits.device();
    const c10::DeviceGuard guard(dev);
    const Matrix logits = matrix("logits", given_logits);
    const Ids ids = ids_of("token_ids", there("token_ids", a[1], dev));
    TORCH_CHECK_VALUE(ids.t.dim() == 1 && ids.t.size(0) == logits.rows,
                      "token_ids must have shape ", shape_name({logits.rows}), " (got ",
                      shape_name(ids.t.sizes()), ")");
    const Tensor old = vector("old_logp", a[2], dev, logits.rows);
    const Tensor advantages = vector("advantages", a[3], dev, logits.rows);
    const Tensor offsets = offsets_of("segment_offsets", a[4], dev);
    Tensor ref;
    segtopk_policy_loss_args q{};
    q.kl_coef = real(a[6]);
    if (given(a[5])) ref = vector("ref_logp", a[5], dev, logits.rows);
    else TORCH_CHECK_VALUE(q.kl_coef == 0.0, "kl_coef needs ref_logp");
    q.clip_low = real(a[7]);
    q.clip_high = real(a[8]);
    q.temperature = real(a[9]);
    q.grad_scale = real(a[10]);
    const Tensor loss = fresh({}, ScalarType::Float, dev);
    const Tensor logp = fresh({logits.rows}, ScalarType::Float, dev);
    const bool gradient = a[12] == Py_True;
    Matrix dlogits{};
    if (gradient && a[11] == a[0]) {
        TORCH_CHECK_VALUE(logits.t.is_same(given_logits),
                          "dlogits may be the logits only where these have a unit inner stride and "
                          "rows that do not overlap");
        dlogits = logits;
    } else if (gradient) {
        dlogits = result("dlogits", a[11], dev, logits.rows, logits.width, logits.t.scalar_type());
    }
    q.logits = logits.v;
    q.dlogits = dlogits.v;
    q.token_ids = ids.t.data_ptr();
    q.id_type = ids.code;
    q.tokens = logits.rows;
    q.vocab = logits.width;
    q.num_segments = offsets.size(0) - 1;
    q.segment_offsets = static_cast<const int64_t *>(offsets.data_ptr());
    q.old_logp = static_cast<const float *>(old.data_ptr());
    q.ref_logp = ref.defined() ? static_cast<const float *>(ref.data_ptr()) : nullptr;
    q.advantages = static_cast<const float *>(advantages.data_ptr());
    q.loss = static_cast<float *>(loss.data_ptr());
    q.logp = static_cast<float *>(logp.data_ptr());
    const Workspace ws = workspace(lib.policy_loss_workspace(q.tokens, q.vocab, q.num_segments), dev);
    call("segtopk_policy_loss", dev,
         [&](hipStream_t stream) { return lib.policy_loss(&q, ws.data, ws.bytes, stream); });
    if (!gradient) return tuple(THPVariable_Wrap(loss), THPVariable_Wrap(logp));
    return tuple(THPVariable_Wrap(loss), THPVariable_Wrap(logp), output(a[11], dlogits.t));
}

// logits, k, scoring, bias, groups, kept_groups, group_best, whether to
// renormalize, scale
PyObject *route(PyObject *const *a) {
    const Tensor &given_logits = device_tensor("logits", a[0]);
    const at::Device dev = given_logits.device();
    const c10::DeviceGuard guard(dev);
    const Matrix logits = matrix("logits", given_logits);
    segtopk_route_args q{};
    q.logits = logits.v;
    q.tokens = logits.rows;
    q.num_experts = logits.width;
    q.k = integer(a[1]);
    q.scoring = (int32_t)integer(a[2]);
    Tensor bias;
    if (given(a[3])) {
        bias = vector("bias", a[3], dev, logits.width);
        q.bias = static_cast<const float *>(bias.data_ptr());
    }
    q.groups = integer(a[4]);
    q.kept_groups = given(a[5]) ? integer(a[5]) : q.groups;
    const int64_t best = integer(a[6]);
    const int renormalize = PyObject_IsTrue(a[7]);
    if (renormalize < 0) throw python_error();
    q.renormalize = renormalize;
    q.scale = real(a[8]);
    TORCH_CHECK_VALUE(q.num_experts <= 1024, "at most 1024 experts (got ", q.num_experts, ")");
    TORCH_CHECK_VALUE(q.groups >= 1 && q.groups <= 64 && q.num_experts % q.groups == 0,
                      "groups must be 1 to 64 and divide the number of experts (got ", q.groups, ")");
    TORCH_CHECK_VALUE(q.kept_groups >= 1 && q.kept_groups <= q.groups,
                      "kept_groups must be 1 to groups (got ", q.kept_groups, ")");
    TORCH_CHECK_VALUE(best == 1 || best == 2, "group_best must be 1 or 2 (got ", best, ")");
    TORCH_CHECK_VALUE(q.k >= 1 && q.k <= 64 && q.k <= q.kept_groups * (q.num_experts / q.groups),
                      "k must be 1 to 64 and at most the number of experts in the groups kept (got ",
                      q.k, ")");
    q.group_best = (int32_t)best;
    const Tensor weights = fresh({q.tokens, q.k}, ScalarType::Float, dev);
    const Tensor experts = fresh({q.tokens, q.k}, ScalarType::Int, dev);
    q.weights = static_cast<float *>(weights.data_ptr());
    q.experts = static_cast<int32_t *>(experts.data_ptr());
    call("segtopk_route", dev, [&](hipStream_t stream) { return lib.route(&q, stream); });
    return tuple(THPVariable_Wrap(weights), THPVariable_Wrap(experts));
}

// dweights, logits, experts, scoring, whether to renormalize, scale, out
PyObject *route_backward(PyObject *const *a) {
    const Tensor &given_dweights = device_tensor("dweights", a[0]);
    const at::Device dev = given_dweights.device();
    const c10::DeviceGuard guard(dev);
    const Matrix logits = matrix("logits", there("logits", a[1], dev));
    TORCH_CHECK_VALUE(logits.width <= 1024, "at most 1024 experts (got ", logits.width, ")");
    const Tensor &e = there("experts", a[2], dev);
    TORCH_CHECK_TYPE(e.scalar_type() == ScalarType::Int, "experts must be int32 (got ",
                     type_name(e.scalar_type()), ")");
    TORCH_CHECK_VALUE(e.dim() == 2 && e.size(0) == logits.rows && e.size(1) >= 1 &&
                          e.size(1) <= 64 && e.size(1) <= logits.width,
                      "experts must have shape (tokens, k), k 1 to 64 and at most the number of "
                      "experts (got ", shape_name(e.sizes()), ")");
    TORCH_CHECK_TYPE(given_dweights.scalar_type() == ScalarType::Float,
                     "dweights must be torch.float32 (got ", type_name(given_dweights.scalar_type()),
                     ")");
    TORCH_CHECK_VALUE(given_dweights.sizes() == e.sizes(), "dweights must have experts' shape ",
                      shape_name(e.sizes()), " (got ", shape_name(given_dweights.sizes()), ")");
    const Tensor experts = e.contiguous(), dweights = given_dweights.contiguous();
    const int32_t scoring = (int32_t)integer(a[3]);
    const int renormalize = PyObject_IsTrue(a[4]);
    if (renormalize < 0) throw python_error();
    const double scale = real(a[5]);
    const Matrix out = result("out", a[6], dev, logits.rows, logits.width, logits.t.scalar_type());
    const int64_t k = e.size(1);
    const int32_t *const chosen = static_cast<const int32_t *>(experts.data_ptr());
    const float *const grads = static_cast<const float *>(dweights.data_ptr());
    call("segtopk_route_backward", dev, [&](hipStream_t stream) {
        return lib.route_backward(&logits.v, &out.v, chosen, grads, logits.rows, logits.width, k,
                                  scoring, renormalize, scale, stream);
    });
    return output(a[6], out.t);
}

// ---- 8 bits ---------------------------------------------------------------
constexpr ScalarType kBits8 = ScalarType::Float8_e4m3fn;
int64_t round_up(int64_t n, int64_t to) { return (n + to - 1) / to * to; }

// Rows in 8 bits begin at multiples of 128 bytes.
Tensor fresh8(std::vector<int64_t> shape, at::Device dev) {
    const int64_t width = shape.back();
    shape.back() = round_up(width, 128);
    const Tensor t = fresh(shape, kBits8, dev);
    return shape.back() == width ? t : t.narrow(-1, 0, width);
}

// x, position, offsets
PyObject *quantize_rows(PyObject *const *a) {
    const Tensor &given_x = device_tensor("x", a[0]);
    const at::Device dev = given_x.device();
    const c10::DeviceGuard guard(dev);
    const Matrix x = matrix("x", given_x);
    Slots s{{}, {}, x.rows, 1, nullptr, nullptr};
    if (given(a[1])) s = slots(a[1], a[2], dev);
    TORCH_CHECK_VALUE(x.rows == s.tokens, "position is for ", s.tokens, " tokens, x has ", x.rows,
                      " rows");
    const int64_t rows = s.tokens * s.k;
    check_count("rows", rows);
    const Tensor q = fresh8({rows, x.width}, dev);
    const Tensor scales = fresh({rows, round_up(x.width, 128) / 128}, ScalarType::Float, dev);
    const segtopk_rows v{q.data_ptr(), round_up(x.width, 128), SEGTOPK_E4M3};
    float *const f = static_cast<float *>(scales.data_ptr());
    call("segtopk_quantize_rows", dev, [&](hipStream_t stream) {
        return lib.quantize_rows(&x.v, &v, f, s.tokens, s.k, x.width, s.at, s.kept, stream);
    });
    return tuple(THPVariable_Wrap(q), THPVariable_Wrap(scales));
}

// Matrices with a unit inner stride whose rows do not overlap, nor the matrices.
bool plain_matrices(const Tensor &t) {
    const auto s = t.sizes(), d = t.strides();
    return (d[2] == 1 || s[2] <= 1) && (d[1] >= s[2] || s[1] <= 1) &&
           (d[0] >= (s[1] - 1) * (s[1] > 1 ? d[1] : 0) + s[2] || s[0] <= 1);
}
segtopk_matrices view3(const Tensor &t, int code, int64_t least) {
    // The stride of a single row or matrix is never used.
    const int64_t stride = t.size(1) > 1 ? t.stride(1) : least;
    return {t.data_ptr(), t.size(0) > 1 ? t.stride(0) : 0, stride, code};
}

PyObject *quantize_blocks(PyObject *const *a) {
    const Tensor &given_x = device_tensor("x", a[0]);
    const at::Device dev = given_x.device();
    const c10::DeviceGuard guard(dev);
    const ScalarType type = given_x.scalar_type();
    TORCH_CHECK_TYPE(float_code(type) >= 0, "x must be float32, bfloat16 or float16 (got ",
                     type_name(type), ")");
    TORCH_CHECK_VALUE((given_x.dim() == 2 || given_x.dim() == 3) && given_x.size(-1) >= 1,
                      "x must have shape (rows, width) or (matrices, rows, width) (got ",
                      shape_name(given_x.sizes()), ")");
    const bool one = given_x.dim() == 2;
    Tensor x = one ? given_x.unsqueeze(0) : given_x;
    if (!plain_matrices(x)) x = x.contiguous();
    const int64_t m = x.size(0), rows = x.size(1), width = x.size(2);
    check_count("matrices", m);
    check_count("rows", rows);
    const Tensor q = fresh8({m, rows, width}, dev);
    const Tensor scales = fresh({m, round_up(rows, 128) / 128, round_up(width, 128) / 128},
                                ScalarType::Float, dev);
    const segtopk_matrices in = view3(x, float_code(type), width);
    const int64_t stride = round_up(width, 128);
    const segtopk_matrices to{q.data_ptr(), rows * stride, stride, SEGTOPK_E4M3};
    float *const f = static_cast<float *>(scales.data_ptr());
    call("segtopk_quantize_blocks", dev, [&](hipStream_t stream) {
        return lib.quantize_blocks(&in, &to, f, m, rows, width, stream);
    });
    return tuple(THPVariable_Wrap(one ? q.squeeze(0) : q), THPVariable_Wrap(one ? scales.squeeze(0) : scales));
}

// The operand in 8 bits, copied where its rows do not begin at multiples of 16 bytes.
Tensor bits8(const char *name, const Tensor &t, int64_t dim) {
    TORCH_CHECK_TYPE(t.scalar_type() == kBits8, name, " must be torch.float8_e4m3fn (got ",
                     type_name(t.scalar_type()), ")");
    TORCH_CHECK_VALUE(t.dim() == dim && t.size(-1) >= 1, name, " must be ", dim,
                      "-D and at least one element wide (got ", shape_name(t.sizes()), ")");
    bool good = (t.stride(-1) == 1 || t.size(-1) == 1) &&
                reinterpret_cast<uintptr_t>(t.data_ptr()) % 16 == 0;
    for (int64_t d = 0; good && d + 1 < dim; ++d)
        good = t.size(d) <= 1 || (t.stride(d) % 16 == 0 && t.stride(d) >= (d + 2 == dim ? t.size(-1) : 0));
    if (good) return t;
    Tensor c = fresh8(t.sizes().vec(), t.device());
    c.copy_(t);
    return c;
}

Tensor scales_of(const char *name, PyObject *o, at::Device dev, at::IntArrayRef shape) {
    const Tensor &t = there(name, o, dev);
    TORCH_CHECK_TYPE(t.scalar_type() == ScalarType::Float, name, " must be torch.float32 (got ",
                     type_name(t.scalar_type()), ")");
    TORCH_CHECK_VALUE(t.sizes() == shape, name, " must have shape ", shape_name(shape), " (got ",
                      shape_name(t.sizes()), ")");
    return t.contiguous();
}

ScalarType type_of(PyObject *dtype, PyObject *out, ScalarType otherwise) {
    if (given(dtype)) {
        TORCH_CHECK_TYPE(THPDtype_Check(dtype), "dtype must be a torch.dtype");
        return reinterpret_cast<THPDtype *>(dtype)->scalar_type;
    }
    return given(out) ? tensor("out", out).scalar_type() : otherwise;
}

// rows, row_scales, weights, weight_scales, offsets, dtype, out
PyObject *expert_matmul(PyObject *const *a) {
    const Tensor &given_rows = device_tensor("rows", a[0]);
    const at::Device dev = given_rows.device();
    const c10::DeviceGuard guard(dev);
    const Tensor rows = bits8("rows", given_rows, 2);
    const Tensor weights = bits8("weights", there("weights", a[2], dev), 3);
    const int64_t n = rows.size(0), depth = rows.size(1), experts = weights.size(0),
                  width = weights.size(1);
    TORCH_CHECK_VALUE(weights.size(2) == depth, "weights must be as deep as rows are wide (", depth,
                      "; got ", shape_name(weights.sizes()), ")");
    TORCH_CHECK_VALUE(experts >= 1 && experts <= 65535 && width >= 1,
                      "weights must have shape (experts, width, depth), 1 to 65535 experts (got ",
                      shape_name(weights.sizes()), ")");
    const int64_t blocks = round_up(depth, 128) / 128;
    const Tensor row_scales = scales_of("row_scales", a[1], dev, {n, blocks});
    const Tensor weight_scales =
        scales_of("weight_scales", a[3], dev, {experts, round_up(width, 128) / 128, blocks});
    const Tensor offsets = offsets_of("offsets", a[4], dev);
    TORCH_CHECK_VALUE(offsets.size(0) == experts + 1, "offsets must have ", experts + 1,
                      " entries (got ", offsets.size(0), ")");
    const ScalarType type = type_of(a[5], a[6], ScalarType::BFloat16);
    TORCH_CHECK_TYPE(float_code(type) >= 0, "the result must be float32, bfloat16 or float16 (got ",
                     type_name(type), ")");
    const Matrix out = result("out", a[6], dev, n, width, type);
    segtopk_expert_matmul_args q{};
    q.rows = {rows.data_ptr(), n > 1 ? rows.stride(0) : round_up(depth, 16), SEGTOPK_E4M3};
    q.out = out.v;
    q.weights = view3(weights, SEGTOPK_E4M3, round_up(depth, 16));
    q.row_scales = static_cast<const float *>(row_scales.data_ptr());
    q.weight_scales = static_cast<const float *>(weight_scales.data_ptr());
    q.offsets = static_cast<const int64_t *>(offsets.data_ptr());
    q.num_rows = n;
    q.num_experts = experts;
    q.width = width;
    q.depth = depth;
    call("segtopk_expert_matmul", dev,
         [&](hipStream_t stream) { return lib.expert_matmul(&q, stream); });
    return output(a[6], out.t);
}

// dout, rows, offsets, dtype, out, accumulate
PyObject *expert_dweights(PyObject *const *a) {
    const Tensor &given_dout = device_tensor("dout", a[0]);
    const at::Device dev = given_dout.device();
    const c10::DeviceGuard guard(dev);
    const Matrix dout = matrix("dout", given_dout);
    const Matrix rows = matrix("rows", there("rows", a[1], dev));
    const ScalarType in = dout.t.scalar_type();
    TORCH_CHECK_TYPE(rows.t.scalar_type() == in, "rows must be ", type_name(in), " (got ",
                     type_name(rows.t.scalar_type()), ")");
    TORCH_CHECK_VALUE(rows.rows == dout.rows, "rows must have dout's ", dout.rows, " rows (got ",
                      rows.rows, ")");
    const Tensor offsets = offsets_of("offsets", a[2], dev);
    const int64_t experts = offsets.size(0) - 1;
    TORCH_CHECK_VALUE(experts >= 1 && experts <= 65535, "offsets must be for 1 to 65535 experts (got ",
                      experts, ")");
    const int accumulate = PyObject_IsTrue(a[5]);
    if (accumulate < 0) throw python_error();
    TORCH_CHECK_VALUE(!accumulate || given(a[4]), "accumulate needs out");
    const ScalarType type = type_of(a[3], a[4], in);
    TORCH_CHECK_TYPE(type == in || type == ScalarType::Float, "the gradient must be float32 or ",
                     type_name(in), " (got ", type_name(type), ")");
    Tensor out;
    if (given(a[4])) {
        out = there("out", a[4], dev);
        TORCH_CHECK_TYPE(out.scalar_type() == type, "out must be ", type_name(type), " (got ",
                         type_name(out.scalar_type()), ")");
        TORCH_CHECK_VALUE(out.sizes() == at::IntArrayRef({experts, dout.width, rows.width}),
                          "out must have shape ", shape_name({experts, dout.width, rows.width}),
                          " (got ", shape_name(out.sizes()), ")");
        TORCH_CHECK_VALUE(plain_matrices(out),
                          "out must have a unit inner stride and rows that do not overlap");
    } else {
        out = fresh({experts, dout.width, rows.width}, type, dev);
    }
    segtopk_expert_dweights_args q{};
    q.dout = dout.v;
    q.rows = rows.v;
    q.dweights = view3(out, float_code(type), rows.width);
    q.offsets = static_cast<const int64_t *>(offsets.data_ptr());
    q.num_rows = dout.rows;
    q.num_experts = experts;
    q.width = dout.width;
    q.depth = rows.width;
    q.accumulate = accumulate;
    const Workspace ws =
        workspace(lib.expert_dweights_workspace(q.num_rows, experts, q.width, q.depth), dev);
    call("segtopk_expert_dweights", dev,
         [&](hipStream_t stream) { return lib.expert_dweights(&q, ws.data, ws.bytes, stream); });
    return output(a[4], out);
}

// target_logits, draft_tokens, draft_offsets, accept, sample, draft_logits, temperature
PyObject *verify_drafts(PyObject *const *a) {
    const Tensor &given_target = device_tensor("target_logits", a[0]);
    const at::Device dev = given_target.device();
    const c10::DeviceGuard guard(dev);
    const Matrix target = matrix("target_logits", given_target);
    const Ids ids = ids_of("draft_tokens", there("draft_tokens", a[1], dev));
    TORCH_CHECK_VALUE(ids.t.dim() == 1, "draft_tokens must be 1-D (got ", shape_name(ids.t.sizes()),
                      ")");
    const Tensor offsets = offsets_of("draft_offsets", a[2], dev);
    const int64_t drafts = ids.t.size(0), requests = offsets.size(0) - 1;
    TORCH_CHECK_VALUE(target.rows == drafts + requests, "target_logits must have one row a draft and "
                      "one a request (", drafts + requests, "; got ", target.rows, ")");
    TORCH_CHECK_VALUE(drafts == 0 || requests > 0, "drafted tokens need a request");
    const Tensor accept = vector("accept", a[3], dev, drafts);
    const Tensor sample = vector("sample", a[4], dev, requests);
    segtopk_verify_args q{};
    Matrix draft{};
    if (given(a[5])) {
        draft = matrix("draft_logits", there("draft_logits", a[5], dev));
        TORCH_CHECK_TYPE(draft.t.scalar_type() == target.t.scalar_type(), "draft_logits must be ",
                         type_name(target.t.scalar_type()), " (got ",
                         type_name(draft.t.scalar_type()), ")");
        TORCH_CHECK_VALUE(draft.rows == drafts && draft.width == target.width,
                          "draft_logits must have shape ", shape_name({drafts, target.width}),
                          " (got ", shape_name({draft.rows, draft.width}), ")");
        q.draft = draft.v;
    }
    Tensor temperatures;
    if (THPVariable_Check(a[6])) {
        temperatures = vector("temperature", a[6], dev, requests);
        q.temperatures = static_cast<const float *>(temperatures.data_ptr());
    } else {
        q.temperature = real(a[6]);
        TORCH_CHECK_VALUE(q.temperature >= 0.0 && q.temperature <= 1e300,
                          "temperature must be finite and >= 0 (got ", q.temperature, ")");
    }
    const Tensor tokens = fresh({drafts + requests}, ids.t.scalar_type(), dev);
    const Tensor counts = fresh({requests}, ScalarType::Int, dev);
    q.target = target.v;
    q.draft_tokens = ids.t.data_ptr();
    q.id_type = ids.code;
    q.draft_offsets = static_cast<const int64_t *>(offsets.data_ptr());
    q.num_drafts = drafts;
    q.num_requests = requests;
    q.vocab = target.width;
    q.accept = static_cast<const float *>(accept.data_ptr());
    q.sample = static_cast<const float *>(sample.data_ptr());
    q.tokens = tokens.data_ptr();
    q.counts = static_cast<int32_t *>(counts.data_ptr());
    const Workspace ws = workspace(lib.verify_workspace(drafts, requests, q.vocab), dev);
    call("segtopk_verify_drafts", dev,
         [&](hipStream_t stream) { return lib.verify_drafts(&q, ws.data, ws.bytes, stream); });
    return tuple(THPVariable_Wrap(tokens), THPVariable_Wrap(counts));
}

// ---- the module ---------------------------------------------------------
template <PyObject *(*CALL)(PyObject *const *), Py_ssize_t COUNT>
PyObject *method(PyObject *, PyObject *const *args, Py_ssize_t count) {
    HANDLE_TH_ERRORS
    TORCH_CHECK_TYPE(count == COUNT, "expected ", COUNT, " arguments, got ", count);
    return CALL(args);
    END_HANDLE_TH_ERRORS
}

template <class F> void find(void *file, const char *name, F &f) {
    f = reinterpret_cast<F>(dlsym(file, name));
    TORCH_CHECK(f, "the library has no ", name);
}

// load(path of the library, exception class)
PyObject *load(PyObject *const *a) {
    const char *path = PyUnicode_AsUTF8(a[0]);
    if (!path) throw python_error();
    void *const file = dlopen(path, RTLD_NOW | RTLD_LOCAL);
    TORCH_CHECK(file, "cannot load ", path, ": ", dlerror());
    find(file, "segtopk_sort_ids_workspace", lib.sort_ids_workspace);
    find(file, "segtopk_sort_ids", lib.sort_ids);
    find(file, "segtopk_dispatch_rows", lib.dispatch_rows);
    find(file, "segtopk_combine_rows", lib.combine_rows);
    find(file, "segtopk_combine_rows_backward", lib.combine_rows_backward);
    find(file, "segtopk_embedding_rows", lib.embedding_rows);
    find(file, "segtopk_embedding_backward_workspace", lib.embedding_backward_workspace);
    find(file, "segtopk_embedding_backward", lib.embedding_backward);
    find(file, "segtopk_policy_loss_workspace", lib.policy_loss_workspace);
    find(file, "segtopk_policy_loss", lib.policy_loss);
    find(file, "segtopk_route", lib.route);
    find(file, "segtopk_route_backward", lib.route_backward);
    find(file, "segtopk_quantize_rows", lib.quantize_rows);
    find(file, "segtopk_quantize_blocks", lib.quantize_blocks);
    find(file, "segtopk_expert_matmul", lib.expert_matmul);
    find(file, "segtopk_expert_dweights_workspace", lib.expert_dweights_workspace);
    find(file, "segtopk_expert_dweights", lib.expert_dweights);
    find(file, "segtopk_verify_workspace", lib.verify_workspace);
    find(file, "segtopk_verify_drafts", lib.verify_drafts);
    Py_INCREF(a[1]);
    Py_XDECREF(call_error);
    call_error = a[1];
    return same(Py_None);
}

template <PyObject *(*CALL)(PyObject *const *), Py_ssize_t COUNT>
PyMethodDef entry(const char *name) {
    return {name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(&method<CALL, COUNT>)),
            METH_FASTCALL, nullptr};
}

PyMethodDef methods[] = {
    entry<load, 2>("load"),
    entry<sort_ids, 2>("sort_ids"),
    entry<dispatch, 4>("dispatch"),
    entry<combine, 5>("combine"),
    entry<combine_backward, 6>("combine_backward"),
    entry<embedding, 4>("embedding"),
    entry<embedding_backward, 8>("embedding_backward"),
    entry<policy_loss, 13>("policy_loss"),
    entry<route, 9>("route"),
    entry<route_backward, 7>("route_backward"),
    entry<quantize_rows, 3>("quantize_rows"),
    entry<quantize_blocks, 1>("quantize_blocks"),
    entry<expert_matmul, 7>("expert_matmul"),
    entry<expert_dweights, 6>("expert_dweights"),
    entry<verify_drafts, 7>("verify_drafts"),
    {nullptr, nullptr, 0, nullptr},
};

PyModuleDef module = {PyModuleDef_HEAD_INIT, "_binding", nullptr, -1, methods,
                      nullptr, nullptr, nullptr, nullptr};

}  // namespace

extern "C" __attribute__((visibility("default"))) PyObject *PyInit__binding() {
    return PyModule_Create(&module);
}
