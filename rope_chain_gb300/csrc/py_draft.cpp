// Python side of the drafted tokens' calls (rc_rope_table, rc_rope_apply,
// rc_tree_attention, rc_logits_adjust) and of those around them
// (rc_window_attention, rc_kv4_attention, rc_head_norm_rope,
// rc_head_norm_rope_grad, rc_kv4_store, rc_kv4_load, rc_kv_compact): checks torch tensors, makes the
// output and calls the C ABI.  The other calls of the package go through ctypes, whose
// 6 to 12 us a call these cannot afford: their kernels take 2 to 20 us.
// Arguments come by position (rope_chain_gb300/__init__.py has the signatures
// and their documentation).
#include "rope_chain.h"

#include <ATen/core/Tensor.h>
#include <ATen/core/grad_mode.h>
#include <ATen/ops/empty.h>
#include <c10/core/AutogradState.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Device.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>
#include <torch/csrc/utils/object_ptr.h>

#include <optional>

namespace {

using at::Tensor;

PyObject *g_error = nullptr;                 // RopeChainError(status, message)

// Raised through Python: an error status of the library.
PyObject *raise_status(rc_status s) {
    PyObject *e = PyObject_CallFunction(g_error, "is", (int)s, rc_last_error());
    if (e != nullptr) {
        PyErr_SetObject(g_error, e);
        Py_DECREF(e);
    }
    return nullptr;
}

const Tensor &tensor(PyObject *o, const char *name) {
    TORCH_CHECK_TYPE(THPVariable_Check(o), name, " must be a tensor");
    return THPVariable_Unpack(o);
}

int64_t integer(PyObject *o) {
    const int64_t v = PyLong_AsLongLong(o);
    if (v == -1 && PyErr_Occurred())
        throw python_error();
    return v;
}

double number(PyObject *o) {
    const double v = PyFloat_AsDouble(o);
    if (v == -1.0 && PyErr_Occurred())
        throw python_error();
    return v;
}

bool truth(PyObject *o) {
    const int v = PyObject_IsTrue(o);
    if (v < 0)
        throw python_error();
    return v != 0;
}

template <typename T> T narrow(int64_t v, const char *name) {
    TORCH_CHECK_VALUE(v >= std::numeric_limits<T>::min() && v <= std::numeric_limits<T>::max(), name, " = ", v,
                      " is out of range");
    return static_cast<T>(v);
}

int32_t dtype_of(const Tensor &t, const char *name) {
    if (t.scalar_type() == at::kBFloat16)
        return RC_BF16;
    TORCH_CHECK_TYPE(t.scalar_type() == at::kFloat, name, " must be bfloat16 or float32");
    return RC_F32;
}

// Every operand lies on one device, that of the call's first tensor: a kernel of
// one GPU must not get another's addresses.
void beside(const Tensor &t, at::Device device, const char *name) {
    TORCH_CHECK_VALUE(t.device() == device, name, " is on device ", t.device(), ", other operands on ", device);
}

// A tangent of forward mode (torch.autograd.forward_ad) is carried on by no call; it is
// there under torch.no_grad() too, not in inference mode.
void no_tangent(const Tensor &t, const char *name) {
    TORCH_CHECK_VALUE(!t._fw_grad(0).defined() || !c10::AutogradState::get_tls_state().get_fw_grad_mode(), name,
                      " has a tangent (forward-mode differentiation), which this call does not carry on");
}

// The calls record nothing for autograd (rope_apply and head_norm_rope do so in Python).
void no_gradient(const Tensor &t, const char *name) {
    no_tangent(t, name);
    TORCH_CHECK_VALUE(!t.requires_grad() || !at::GradMode::is_enabled(), name, " requires a gradient, which this call "
                      "does not give: detach it or call under torch.no_grad()");
}

// The data of a contiguous CUDA array of at least `numel` elements on `device`
// (NULL for None).
template <typename T>
const T *array(PyObject *o, at::Device device, at::ScalarType type, int64_t numel, const char *name) {
    if (o == Py_None)
        return nullptr;
    const Tensor &t = tensor(o, name);
    TORCH_CHECK_TYPE(t.scalar_type() == type && t.is_cuda() && t.is_contiguous(), name,
                     " must be a contiguous CUDA ", at::toString(type), " tensor");
    beside(t, device, name);
    no_gradient(t, name);
    TORCH_CHECK_VALUE(t.numel() >= numel, name, " needs ", numel, " elements, it has ", t.numel());
    return static_cast<const T *>(t.const_data_ptr());
}

int32_t *counter(PyObject *o, at::Device device) {
    return const_cast<int32_t *>(array<int32_t>(o, device, at::kInt, 1, "err"));
}

// The device and stream of a call, current while it lasts: the operands' device
// and `stream`, a stream's handle or None (the device's current stream).  What is
// allocated meanwhile comes from that stream's memory: on the caller's it could
// still be in use by work queued there, which the call's stream does not wait for.
// (Guards where something changes only: they would cost a small call 0.3 us.)
class On {
public:
    On(std::optional<at::Device> device, PyObject *stream) {
        c10::DeviceIndex index = c10::cuda::current_device();
        if (device && device->has_index() && device->index() != index) {
            index = device->index();
            device_.set_index(index);
        }
        if (stream != Py_None) {
            handle_ = reinterpret_cast<cudaStream_t>(static_cast<uintptr_t>(integer(stream)));
            stream_.reset_stream(c10::cuda::getStreamFromExternal(handle_, index));
        } else {
            handle_ = c10::cuda::getCurrentCUDAStream(index).stream();
        }
    }
    cudaStream_t stream() const { return handle_; }

private:
    c10::cuda::OptionalCUDAGuard device_;
    c10::cuda::OptionalCUDAStreamGuard stream_;
    cudaStream_t handle_;
};

void need(Py_ssize_t n, Py_ssize_t want) { TORCH_CHECK_TYPE(n == want, "expected ", want, " arguments, got ", n); }

// The output: `o`, checked to be like `t`, or (undefined) one to be made by made().
Tensor output(PyObject *o, const Tensor &t, const char *what) {
    if (o == Py_None)
        return Tensor();
    const Tensor &out = tensor(o, "out");
    TORCH_CHECK_VALUE(out.sizes() == t.sizes() && out.scalar_type() == t.scalar_type() && out.is_cuda(),
                      "out must be a CUDA tensor of the shape and dtype of ", what);
    beside(out, t.device(), "out");
    no_gradient(out, "out");
    return out;
}

// What a call wrote into tensors that were there before it shows as torch's own in-place
// operations show it: a backward pass that has saved one of them finds it changed, and
// raises, instead of taking other values.  (Counters and workspaces hold none.)
void written(std::initializer_list<PyObject *> list) {
    for (PyObject *o : list)
        if (o != Py_None && !THPVariable_Unpack(o).is_inference())
            THPVariable_Unpack(o).unsafeGetTensorImpl()->bump_version();
}

// The result of a call: `out`, once what was `given` to be written is marked; or an error.
PyObject *result(rc_status s, const Tensor &out, std::initializer_list<PyObject *> given) {
    if (s != RC_OK)
        return raise_status(s);
    written(given);
    return THPVariable_Wrap(out);
}

// A new contiguous output like `t` where there is none yet (within an On).
void made(Tensor &out, const Tensor &t) {
    if (!out.defined())
        out = at::empty(t.sizes(), t.options(), at::MemoryFormat::Contiguous);
}

PyObject *rope_table(PyObject *, PyObject *const *args, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    // positions, rot_dim, theta, kind, factor, original, beta_fast, beta_slow,
    // attention_factor, float32, device, out, stream
    need(n, 13);
    const int64_t positions = integer(args[0]), rot_dim = integer(args[1]);
    const rc_rope_scaling sc = {narrow<int32_t>(integer(args[3]), "scaling"), number(args[4]), number(args[5]),
                                number(args[6]), number(args[7]), number(args[8])};
    Tensor out;
    std::optional<at::Device> device;
    if (args[10] != Py_None) {
        TORCH_CHECK_TYPE(THPDevice_Check(args[10]), "device must be a torch.device");
        device = reinterpret_cast<THPDevice *>(args[10])->device;
        TORCH_CHECK_VALUE(device->is_cuda(), "the table is made on a CUDA device");
    }
    if (args[11] != Py_None) {
        out = tensor(args[11], "out");
        TORCH_CHECK_VALUE(out.dim() == 2 && out.size(0) == positions && out.size(1) == rot_dim && out.is_cuda() &&
                              out.is_contiguous(), "out must be a contiguous CUDA tensor [max_position, rot_dim]");
        no_gradient(out, "out");
        if (device && device->has_index())
            beside(out, *device, "out");
        device = out.device();
    } else {
        TORCH_CHECK_VALUE(positions >= 0 && rot_dim > 0, "max_position must not be negative, rot_dim positive");
    }
    const On on(device, args[12]);
    if (!out.defined())
        out = at::empty({positions, rot_dim},
                        at::TensorOptions(integer(args[9]) ? at::kFloat : at::kBFloat16).device(at::kCUDA));
    const rc_status s = rc_rope_table(out.data_ptr(), dtype_of(out, "out"), positions,
                                      narrow<int32_t>(rot_dim, "rot_dim"), number(args[2]), &sc, on.stream());
    return result(s, out, {args[11]});
    END_HANDLE_TH_ERRORS
}

PyObject *rope_apply(PyObject *, PyObject *const *args, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    // x, positions, cos_sin, layout, inverse, out, err, stream
    need(n, 8);
    const Tensor &x = tensor(args[0], "x"), &table = tensor(args[2], "cos_sin");
    TORCH_CHECK_TYPE(x.is_cuda(), "x must be a CUDA tensor");
    TORCH_CHECK_VALUE(x.dim() == 3 && x.stride(2) == 1, "x must be [T, heads, head_dim] with a contiguous last axis");
    TORCH_CHECK_VALUE(table.dim() == 2 && table.is_cuda() && table.is_contiguous(),
                      "cos_sin must be a contiguous CUDA tensor [max_position, rot_dim]");
    beside(table, x.device(), "cos_sin");
    no_gradient(table, "cos_sin");
    no_tangent(x, "x");
    if (args[5] == Py_None && x.requires_grad() && at::GradMode::is_enabled())
        Py_RETURN_NONE;                  // to be recorded: the caller does
    no_gradient(x, "x");
    const int32_t type = dtype_of(x, "x");
    TORCH_CHECK_TYPE(args[1] != Py_None, "positions must be a tensor");
    const bool inverse = truth(args[4]);
    const int64_t *positions = array<int64_t>(args[1], x.device(), at::kLong, x.size(0), "positions");
    int32_t *err = counter(args[6], x.device());
    Tensor out = output(args[5], x, "x");
    TORCH_CHECK_VALUE(!out.defined() || out.stride(2) == 1, "the last axis of out must be contiguous");
    const On on(x.device(), args[7]);
    made(out, x);
    const rc_status s = rc_rope_apply(
        x.const_data_ptr(), type, x.stride(0), x.stride(1), x.size(0), narrow<int32_t>(x.size(1), "heads"),
        narrow<int32_t>(x.size(2), "head_dim"), positions, table.const_data_ptr(), dtype_of(table, "cos_sin"),
        table.size(0), narrow<int32_t>(table.size(1), "rot_dim"), narrow<int32_t>(integer(args[3]), "layout"),
        inverse, out.data_ptr(), out.stride(0), out.stride(1), err, on.stream());
    return result(s, out, {args[5]});
    END_HANDLE_TH_ERRORS
}

// What the attention calls have in common: q, row_start, context_len, block_table
// and, beside the cache, tree_mask, scale, out, lse, err, workspace, stream (as
// args[0] to args[3] and rest[0] to rest[6]).
struct AttentionOperands {
    const Tensor &q, &table;
    const at::Device device;
    const int64_t rows, heads, seqs;
    int64_t words = 0;
    const int32_t *row_start, *context_len;
    const uint64_t *tree_mask;
    float scale, *lse = nullptr;
    int32_t *err;
    void *workspace = nullptr;
    size_t workspace_bytes = 0;
    Tensor out;

    // `cache_checked`: looks at the cache, once q and the table have been looked at.
    template <typename Check>
    AttentionOperands(PyObject *const *args, PyObject *const *rest, const Check &cache_checked)
        : q(tensor(args[0], "q")), table(tensor(args[3], "block_table")), device(q.device()), rows(q.dim() == 3 ? q.size(0) : 0),
          heads(q.dim() == 3 ? q.size(1) : 0), seqs(table.dim() == 2 ? table.size(0) : 0) {
        TORCH_CHECK_VALUE(q.dim() == 3 && q.size(2) == 64 && q.scalar_type() == at::kBFloat16 && q.is_cuda(),
                          "q must be a CUDA bfloat16 view [rows, num_heads, 64]");
        TORCH_CHECK_VALUE(q.stride(2) == 1 && (heads == 1 || q.stride(1) == 64), "q needs strides (*, 64, 1)");
        cache_checked(device);
        TORCH_CHECK_VALUE(table.dim() == 2 && table.scalar_type() == at::kInt && table.is_cuda() &&
                              (table.size(1) <= 1 || table.stride(1) == 1),
                          "block_table must be CUDA int32 [seqs, width] with a contiguous last axis");
        beside(table, device, "block_table");
        no_gradient(q, "q");
        if (rest[0] != Py_None) {
            const Tensor &mask = tensor(rest[0], "tree_mask");
            TORCH_CHECK_VALUE(mask.dim() == 2 && mask.size(0) == rows, "tree_mask must be [rows, words]");
            words = mask.size(1);
            TORCH_CHECK_VALUE(words > 0 || rows == 0, "tree_mask needs a word per row at least");
        }
        if (rest[3] != Py_None) {
            const Tensor &t = tensor(rest[3], "lse");
            TORCH_CHECK_VALUE(t.dim() == 2 && t.size(0) == rows && t.size(1) == heads, "lse must be [rows, num_heads]");
            lse = const_cast<float *>(array<float>(rest[3], device, at::kFloat, 0, "lse"));
        }
        if (rest[5] != Py_None) {
            const Tensor &t = tensor(rest[5], "workspace");
            TORCH_CHECK_VALUE(t.is_cuda() && t.is_contiguous(), "workspace must be a contiguous CUDA tensor");
            beside(t, device, "workspace");
            workspace = t.data_ptr();
            workspace_bytes = t.nbytes();
        }
        TORCH_CHECK_TYPE(args[1] != Py_None && args[2] != Py_None, "row_start and context_len must be tensors");
        row_start = array<int32_t>(args[1], device, at::kInt, seqs + 1, "row_start");
        context_len = array<int32_t>(args[2], device, at::kInt, seqs, "context_len");
        tree_mask = reinterpret_cast<const uint64_t *>(array<int64_t>(rest[0], device, at::kLong, 0, "tree_mask"));
        err = counter(rest[4], device);
        out = output(rest[2], q, "q");
        TORCH_CHECK_VALUE(!out.defined() || (out.stride(2) == 1 && (heads == 1 || out.stride(1) == 64)),
                          "out needs strides (*, 64, 1)");
        scale = (float)number(rest[1]);
    }
    const int32_t *blocks() const { return static_cast<const int32_t *>(table.const_data_ptr()); }
    int32_t table_width() const { return narrow<int32_t>(table.size(1), "width of block_table"); }
    const uint16_t *queries() const { return static_cast<const uint16_t *>(q.const_data_ptr()); }
    uint16_t *outputs() const { return static_cast<uint16_t *>(out.data_ptr()); }
};

// A bf16 cache.
struct Cache {
    const uint16_t *data;
    int32_t blocks, heads, block_size;
    void check(PyObject *o, at::Device device) {
        const Tensor &cache = tensor(o, "cache");
        TORCH_CHECK_VALUE(cache.dim() == 4 && cache.size(3) == 128 && cache.scalar_type() == at::kBFloat16 &&
                              cache.is_cuda() && cache.is_contiguous(),
                          "cache must be contiguous CUDA bfloat16 [num_blocks, num_kv_heads, block_size, 128]");
        beside(cache, device, "cache");
        no_gradient(cache, "cache");
        data = static_cast<const uint16_t *>(cache.const_data_ptr());
        blocks = narrow<int32_t>(cache.size(0), "num_blocks");
        heads = narrow<int32_t>(cache.size(1), "num_kv_heads");
        block_size = narrow<int32_t>(cache.size(2), "block_size");
    }
};

PyObject *tree_attention(PyObject *, PyObject *const *args, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    // q, row_start, context_len, block_table, cache, tree_mask, scale, out, lse,
    // err, workspace, stream
    need(n, 12);
    Cache c;
    AttentionOperands o(args, args + 5, [&](at::Device device) { c.check(args[4], device); });
    const On on(o.device, args[11]);
    made(o.out, o.q);
    const rc_status s = rc_tree_attention(
        o.queries(), o.q.stride(0), o.rows, narrow<int32_t>(o.heads, "num_heads"), c.heads, o.row_start,
        narrow<int32_t>(o.seqs, "seqs"), o.context_len, o.blocks(), o.table.stride(0), o.table_width(), o.tree_mask,
        narrow<int32_t>(o.words, "words of tree_mask"), c.data, c.blocks, c.block_size, o.scale, o.outputs(),
        o.out.stride(0), o.lse, o.err, o.workspace, o.workspace_bytes, on.stream());
    return result(s, o.out, {args[7], args[8]});
    END_HANDLE_TH_ERRORS
}

PyObject *window_attention(PyObject *, PyObject *const *args, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    // q, row_start, context_len, block_table, cache, tree_mask, scale, out, lse,
    // err, workspace, stream, window, sinks
    need(n, 14);
    Cache c;
    AttentionOperands o(args, args + 5, [&](at::Device device) { c.check(args[4], device); });
    const int32_t window = narrow<int32_t>(integer(args[12]), "window"), sinks = narrow<int32_t>(integer(args[13]), "sinks");
    TORCH_CHECK_VALUE(window > 0 && sinks >= 0, "window must be positive, sinks not negative");
    const On on(o.device, args[11]);
    made(o.out, o.q);
    const rc_status s = rc_window_attention(
        o.queries(), o.q.stride(0), o.rows, narrow<int32_t>(o.heads, "num_heads"), c.heads, o.row_start,
        narrow<int32_t>(o.seqs, "seqs"), o.context_len, o.blocks(), o.table.stride(0), o.table_width(), o.tree_mask,
        narrow<int32_t>(o.words, "words of tree_mask"), c.data, c.blocks, c.block_size, window, sinks, o.scale,
        o.outputs(), o.out.stride(0), o.lse, o.err, o.workspace, o.workspace_bytes, on.stream());
    return result(s, o.out, {args[7], args[8]});
    END_HANDLE_TH_ERRORS
}

PyObject *logits_adjust(PyObject *, PyObject *const *args, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    // logits, row_start, history, history_start, prompt_len, draft_tokens,
    // tree_mask, repetition, frequency, presence, bias_start, bias_tokens,
    // bias_values, allowed, out, err, stream
    need(n, 17);
    const Tensor &logits = tensor(args[0], "logits"), &start = tensor(args[1], "row_start");
    TORCH_CHECK_TYPE(logits.is_cuda(), "logits must be a CUDA tensor");
    TORCH_CHECK_VALUE(logits.dim() == 2, "logits must be [rows, vocab]");
    const int64_t rows = logits.size(0), vocab = logits.size(1), seqs = start.numel() - 1;
    TORCH_CHECK_VALUE(vocab <= 1 || logits.stride(1) == 1, "rows of logits must be contiguous");
    const int32_t type = dtype_of(logits, "logits");
    const at::Device device = logits.device();
    no_gradient(logits, "logits");
    rc_logits_params p = {};
    TORCH_CHECK_VALUE((args[2] == Py_None) == (args[3] == Py_None), "history and history_start go together");
    if (args[2] != Py_None) {
        p.history = array<int32_t>(args[2], device, at::kInt, 0, "history");
        p.history_size = tensor(args[2], "history").numel();
        p.history_start = array<int64_t>(args[3], device, at::kLong, seqs + 1, "history_start");
        p.prompt_len = array<int32_t>(args[4], device, at::kInt, seqs, "prompt_len");
    }
    p.draft_tokens = array<int32_t>(args[5], device, at::kInt, rows, "draft_tokens");
    if (args[6] != Py_None) {
        const Tensor &mask = tensor(args[6], "tree_mask");
        TORCH_CHECK_VALUE(mask.dim() == 2 && mask.size(0) == rows, "tree_mask must be [rows, words]");
        p.tree_mask = reinterpret_cast<const uint64_t *>(array<int64_t>(args[6], device, at::kLong, 0, "tree_mask"));
        p.mask_words = narrow<int32_t>(mask.size(1), "words of tree_mask");
        TORCH_CHECK_VALUE(p.mask_words > 0 || rows == 0, "tree_mask needs a word per row at least");
    }
    p.repetition = array<float>(args[7], device, at::kFloat, seqs, "repetition");
    p.frequency = array<float>(args[8], device, at::kFloat, seqs, "frequency");
    p.presence = array<float>(args[9], device, at::kFloat, seqs, "presence");
    TORCH_CHECK_VALUE((args[10] == Py_None) == (args[11] == Py_None) && (args[10] == Py_None) == (args[12] == Py_None),
                      "bias_start, bias_tokens and bias_values go together");
    if (args[10] != Py_None) {
        p.bias_size = tensor(args[11], "bias_tokens").numel();
        p.bias_start = array<int32_t>(args[10], device, at::kInt, seqs + 1, "bias_start");
        p.bias_tokens = array<int32_t>(args[11], device, at::kInt, 0, "bias_tokens");
        p.bias_values = array<float>(args[12], device, at::kFloat, p.bias_size, "bias_values");
        if (p.bias_size == 0)                // none for any sequence: an empty tensor has no address
            p.bias_start = p.bias_tokens = nullptr, p.bias_values = nullptr;
    }
    if (args[13] != Py_None) {
        const Tensor &allowed = tensor(args[13], "allowed");
        TORCH_CHECK_VALUE(allowed.dim() == 2 && allowed.scalar_type() == at::kInt && allowed.is_cuda() &&
                              allowed.size(0) == rows && allowed.size(1) >= (vocab + 31) / 32 &&
                              (allowed.size(1) <= 1 || allowed.stride(1) == 1),
                          "allowed must be CUDA int32 [rows, >= ceil(vocab / 32)], rows contiguous");
        beside(allowed, device, "allowed");
        p.allowed = static_cast<const uint32_t *>(allowed.const_data_ptr());
        p.allowed_stride = allowed.stride(0);
    }
    const int32_t *row_start = array<int32_t>(args[1], device, at::kInt, 0, "row_start");
    int32_t *err = counter(args[15], device);
    Tensor out = output(args[14], logits, "logits");
    TORCH_CHECK_VALUE(!out.defined() || vocab <= 1 || out.stride(1) == 1, "rows of out must be contiguous");
    const On on(device, args[16]);
    made(out, logits);
    const rc_status s = rc_logits_adjust(logits.const_data_ptr(), type, logits.stride(0), rows,
                                         narrow<int32_t>(vocab, "vocab"), row_start,
                                         narrow<int32_t>(seqs, "seqs"), &p, out.data_ptr(), out.stride(0), err,
                                         on.stream());
    return result(s, out, {args[14]});
    END_HANDLE_TH_ERRORS
}

// What both directions of the head norm take beside x: positions, cos_sin, eps,
// q_weight, k_weight, q_heads, layout (as args[0] to args[6]).
struct NormOperands {
    rc_head_norm_params params = {};
    const int64_t *positions;
    const Tensor *table;
    int32_t layout;

    NormOperands(const Tensor &x, PyObject *const *args) {
        TORCH_CHECK_TYPE(args[0] != Py_None, "positions must be a tensor");
        positions = array<int64_t>(args[0], x.device(), at::kLong, x.size(0), "positions");
        table = &tensor(args[1], "cos_sin");
        TORCH_CHECK_VALUE(table->dim() == 2 && table->is_cuda() && table->is_contiguous(),
                          "cos_sin must be a contiguous CUDA tensor [max_position, rot_dim]");
        beside(*table, x.device(), "cos_sin");
        no_gradient(*table, "cos_sin");
        params.eps = (float)number(args[2]);
        params.q_heads = narrow<int32_t>(args[5] == Py_None ? x.size(1) : integer(args[5]), "q_heads");
        params.weight_dtype = RC_BF16;
        TORCH_CHECK_VALUE(args[5] != Py_None || args[4] == Py_None, "k_weight needs q_heads, the number of the query heads");
        params.q_weight = weight(args[3], x, "q_weight");
        params.k_weight = weight(args[4], x, "k_weight");
        if (args[3] != Py_None && args[4] != Py_None)
            TORCH_CHECK_TYPE(tensor(args[3], "q_weight").scalar_type() == tensor(args[4], "k_weight").scalar_type(),
                             "q_weight and k_weight must have one dtype");
        layout = narrow<int32_t>(integer(args[6]), "layout");
    }

private:
    const void *weight(PyObject *o, const Tensor &x, const char *name) {
        if (o == Py_None)
            return nullptr;
        const Tensor &w = tensor(o, name);
        TORCH_CHECK_VALUE(w.dim() == 1 && w.size(0) == x.size(2) && w.is_cuda() && w.is_contiguous(), name,
                          " must be a contiguous CUDA tensor [head_dim]");
        params.weight_dtype = dtype_of(w, name);
        beside(w, x.device(), name);
        no_tangent(w, name);
        return w.const_data_ptr();
    }
};

void heads_view(const Tensor &t, const char *name) {
    TORCH_CHECK_TYPE(t.is_cuda(), name, " must be a CUDA tensor");
    TORCH_CHECK_VALUE(t.dim() == 3 && (t.size(2) <= 1 || t.stride(2) == 1), name,
                      " must be [T, heads, head_dim] with a contiguous last axis");
}

bool wants_gradient(PyObject *o) { return o != Py_None && THPVariable_Check(o) && THPVariable_Unpack(o).requires_grad(); }

PyObject *head_norm_rope(PyObject *, PyObject *const *args, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    // x, positions, cos_sin, eps, q_weight, k_weight, q_heads, layout, out, err, stream
    need(n, 11);
    const Tensor &x = tensor(args[0], "x");
    heads_view(x, "x");
    const int32_t type = dtype_of(x, "x");
    const NormOperands o(x, args + 1);
    no_tangent(x, "x");
    if (at::GradMode::is_enabled() && (x.requires_grad() || wants_gradient(args[4]) || wants_gradient(args[5]))) {
        if (args[8] == Py_None)
            Py_RETURN_NONE;              // to be recorded: the caller does
        no_gradient(x, "x");
        for (const int i : {4, 5})
            if (args[i] != Py_None)
                no_gradient(tensor(args[i], "weight"), i == 4 ? "q_weight" : "k_weight");
    }
    int32_t *err = counter(args[9], x.device());
    Tensor out = output(args[8], x, "x");
    TORCH_CHECK_VALUE(!out.defined() || out.size(2) <= 1 || out.stride(2) == 1, "the last axis of out must be contiguous");
    const On on(x.device(), args[10]);
    made(out, x);
    const rc_status s = rc_head_norm_rope(
        x.const_data_ptr(), type, x.stride(0), x.stride(1), x.size(0), narrow<int32_t>(x.size(1), "heads"),
        narrow<int32_t>(x.size(2), "head_dim"), &o.params, o.positions, o.table->const_data_ptr(),
        dtype_of(*o.table, "cos_sin"), o.table->size(0), narrow<int32_t>(o.table->size(1), "rot_dim"), o.layout,
        out.data_ptr(), out.stride(0), out.stride(1), err, on.stream());
    return result(s, out, {args[8]});
    END_HANDLE_TH_ERRORS
}

PyObject *head_norm_rope_grad(PyObject *, PyObject *const *args, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    // grad, x, positions, cos_sin, eps, q_weight, k_weight, q_heads, layout,
    // weight_grads, out, err, workspace, stream
    need(n, 14);
    const Tensor &dy = tensor(args[0], "grad"), &x = tensor(args[1], "x");
    heads_view(x, "x");
    heads_view(dy, "grad");
    TORCH_CHECK_VALUE(dy.sizes() == x.sizes() && dy.scalar_type() == x.scalar_type(),
                      "grad must have the shape and dtype of x");
    beside(dy, x.device(), "grad");
    no_gradient(dy, "grad");
    no_gradient(x, "x");
    const int32_t type = dtype_of(x, "x");
    const NormOperands o(x, args + 2);
    for (const int i : {5, 6})
        if (args[i] != Py_None)
            no_gradient(tensor(args[i], "weight"), i == 5 ? "q_weight" : "k_weight");
    int32_t *err = counter(args[11], x.device());
    Tensor dx = output(args[10], x, "x");
    TORCH_CHECK_VALUE(!dx.defined() || dx.size(2) <= 1 || dx.stride(2) == 1, "the last axis of out must be contiguous");
    const int32_t dim = narrow<int32_t>(x.size(2), "head_dim");
    const bool weights = truth(args[9]);
    const bool q = weights && args[5] != Py_None, k = weights && args[6] != Py_None;
    Tensor workspace;
    if (args[12] != Py_None) {
        workspace = tensor(args[12], "workspace");
        TORCH_CHECK_VALUE(workspace.is_cuda() && workspace.is_contiguous(), "workspace must be a contiguous CUDA tensor");
        beside(workspace, x.device(), "workspace");
    }
    const On on(x.device(), args[13]);
    made(dx, x);
    const auto floats = x.options().dtype(at::kFloat);
    Tensor dq, dk;
    if (q)
        dq = at::empty({dim}, floats);
    if (k)
        dk = at::empty({dim}, floats);
    if ((q || k) && !workspace.defined())
        workspace = at::empty({(int64_t)rc_head_norm_rope_grad_workspace_size(dim)}, x.options().dtype(at::kByte));
    const rc_status s = rc_head_norm_rope_grad(
        dy.const_data_ptr(), dy.stride(0), dy.stride(1), x.const_data_ptr(), type, x.stride(0), x.stride(1), x.size(0),
        narrow<int32_t>(x.size(1), "heads"), dim, &o.params, o.positions, o.table->const_data_ptr(),
        dtype_of(*o.table, "cos_sin"), o.table->size(0), narrow<int32_t>(o.table->size(1), "rot_dim"), o.layout,
        dx.data_ptr(), dx.stride(0), dx.stride(1), q ? dq.data_ptr<float>() : nullptr, k ? dk.data_ptr<float>() : nullptr,
        workspace.defined() ? workspace.data_ptr() : nullptr, workspace.defined() ? workspace.nbytes() : 0, err, on.stream());
    if (s != RC_OK)
        return raise_status(s);
    written({args[10]});
    auto wrapped = [](bool is, Tensor &t) {
        if (is)
            return THPVariable_Wrap(t);
        Py_INCREF(Py_None);
        return Py_None;
    };
    return Py_BuildValue("NNN", THPVariable_Wrap(dx), wrapped(q, dq), wrapped(k, dk));
    END_HANDLE_TH_ERRORS
}

// A cache in 4 bits and its scales.
struct Kv4 {
    uint8_t *cache4;
    uint16_t *scales;
    int32_t blocks, heads, block_size;

    Kv4(PyObject *c, PyObject *s, at::Device device) {
        const Tensor &cache = tensor(c, "cache"), &scale = tensor(s, "scales");
        TORCH_CHECK_VALUE(cache.dim() == 4 && cache.size(3) == 64 && cache.scalar_type() == at::kByte && cache.is_cuda() &&
                              cache.is_contiguous(), "cache must be contiguous CUDA uint8 [num_blocks, num_kv_heads, block_size, 64]");
        TORCH_CHECK_VALUE(scale.dim() == 4 && scale.size(0) == cache.size(0) && scale.size(1) == cache.size(1) &&
                              scale.size(2) == cache.size(2) && scale.size(3) == 4 && scale.scalar_type() == at::kBFloat16 &&
                              scale.is_cuda() && scale.is_contiguous(),
                          "scales must be contiguous CUDA bfloat16 [num_blocks, num_kv_heads, block_size, 4]");
        beside(cache, device, "cache");
        beside(scale, device, "scales");
        no_gradient(scale, "scales");
        cache4 = static_cast<uint8_t *>(cache.data_ptr());
        scales = static_cast<uint16_t *>(scale.data_ptr());
        blocks = narrow<int32_t>(cache.size(0), "num_blocks");
        heads = narrow<int32_t>(cache.size(1), "num_kv_heads");
        block_size = narrow<int32_t>(cache.size(2), "block_size");
    }
};

PyObject *kv4_attention(PyObject *, PyObject *const *args, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    // q, row_start, context_len, block_table, cache, scales, tree_mask, scale, out,
    // lse, err, workspace, stream, window, sinks
    need(n, 15);
    std::optional<Kv4> c;
    AttentionOperands o(args, args + 6, [&](at::Device device) { c.emplace(args[4], args[5], device); });
    const int32_t window = args[13] == Py_None ? 0 : narrow<int32_t>(integer(args[13]), "window");
    const int32_t sinks = narrow<int32_t>(integer(args[14]), "sinks");
    TORCH_CHECK_VALUE((args[13] == Py_None || window > 0) && sinks >= 0 && (window > 0 || sinks == 0),
                      "window must be positive, or None without sinks; sinks not negative");
    const On on(o.device, args[12]);
    made(o.out, o.q);
    const rc_status s = rc_kv4_attention(
        o.queries(), o.q.stride(0), o.rows, narrow<int32_t>(o.heads, "num_heads"), c->heads, o.row_start,
        narrow<int32_t>(o.seqs, "seqs"), o.context_len, o.blocks(), o.table.stride(0), o.table_width(), o.tree_mask,
        narrow<int32_t>(o.words, "words of tree_mask"), c->cache4, c->scales, c->blocks, c->block_size, window, sinks,
        o.scale, o.outputs(), o.out.stride(0), o.lse, o.err, o.workspace, o.workspace_bytes, on.stream());
    return result(s, o.out, {args[8], args[9]});
    END_HANDLE_TH_ERRORS
}

PyObject *kv4_store(PyObject *, PyObject *const *args, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    // k, v, slots, cache, scales, err, stream
    need(n, 7);
    const Tensor &k = tensor(args[0], "k"), &v = tensor(args[1], "v");
    for (const Tensor *t : {&k, &v}) {
        const char *name = t == &k ? "k" : "v";
        heads_view(*t, name);
        TORCH_CHECK_TYPE(t->scalar_type() == at::kBFloat16, name, " must be bfloat16");
        no_gradient(*t, name);
    }
    TORCH_CHECK_VALUE(k.sizes() == v.sizes() && k.size(2) == 64, "k and v must be [T, num_kv_heads, 64]");
    beside(v, k.device(), "v");
    const Kv4 c(args[3], args[4], k.device());
    TORCH_CHECK_VALUE(c.heads == k.size(1), "k has ", k.size(1), " heads, the cache ", c.heads);
    TORCH_CHECK_TYPE(args[2] != Py_None, "slots must be a tensor");
    const int64_t *slots = array<int64_t>(args[2], k.device(), at::kLong, k.size(0), "slots");
    int32_t *err = counter(args[5], k.device());
    const On on(k.device(), args[6]);
    const rc_status s = rc_kv4_store(static_cast<const uint16_t *>(k.const_data_ptr()), k.stride(0), k.stride(1),
                                     static_cast<const uint16_t *>(v.const_data_ptr()), v.stride(0), v.stride(1), k.size(0),
                                     c.heads, slots, c.cache4, c.scales, c.blocks, c.block_size, err, on.stream());
    if (s != RC_OK)
        return raise_status(s);
    written({args[3], args[4]});
    Py_RETURN_NONE;
    END_HANDLE_TH_ERRORS
}

PyObject *kv4_load(PyObject *, PyObject *const *args, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    // slots, cache, scales, out, err, stream
    need(n, 6);
    const Tensor &slot = tensor(args[0], "slots");
    TORCH_CHECK_VALUE(slot.dim() == 1, "slots must be [T]");
    const at::Device device = slot.device();
    const int64_t *slots = array<int64_t>(args[0], device, at::kLong, 0, "slots");
    const Kv4 c(args[1], args[2], device);
    Tensor out;
    if (args[3] != Py_None) {
        out = tensor(args[3], "out");
        TORCH_CHECK_VALUE(out.dim() == 3 && out.size(0) == slot.size(0) && out.size(1) == c.heads && out.size(2) == 128 &&
                              out.scalar_type() == at::kBFloat16 && out.is_cuda() && out.is_contiguous(),
                          "out must be contiguous CUDA bfloat16 [T, num_kv_heads, 128]");
        beside(out, device, "out");
        no_gradient(out, "out");
    }
    int32_t *err = counter(args[4], device);
    const On on(device, args[5]);
    if (!out.defined())
        out = at::empty({slot.size(0), c.heads, 128}, slot.options().dtype(at::kBFloat16));
    const rc_status s = rc_kv4_load(slots, slot.size(0), c.heads, c.cache4, c.scales, c.blocks, c.block_size,
                                    static_cast<uint16_t *>(out.data_ptr()), err, on.stream());
    return result(s, out, {args[3]});
    END_HANDLE_TH_ERRORS
}

PyObject *kv_compact(PyObject *, PyObject *const *args, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    // caches, block_table, context_len, row_start, path, path_len, new_len, err, stream
    need(n, 9);
    constexpr Py_ssize_t kMost = 64;
    const THPObjectPtr list(PySequence_Fast(args[0], "caches must be a sequence of tensors"));
    if (!list)
        throw python_error();
    const Py_ssize_t count = PySequence_Fast_GET_SIZE(list.get());
    TORCH_CHECK_VALUE(count >= 1 && count <= kMost, "need 1 to ", kMost, " caches, not ", count);
    const Tensor &table = tensor(args[1], "block_table"), &path = tensor(args[4], "path");
    TORCH_CHECK_VALUE(table.dim() == 2 && table.scalar_type() == at::kInt && table.is_cuda() &&
                          (table.size(1) <= 1 || table.stride(1) == 1),
                      "block_table must be CUDA int32 [seqs, width] with a contiguous last axis");
    const at::Device device = table.device();
    const int64_t seqs = table.size(0);
    TORCH_CHECK_VALUE(path.dim() == 2 && path.size(0) == seqs && path.scalar_type() == at::kInt && path.is_cuda() &&
                          (path.size(1) <= 1 || path.stride(1) == 1),
                      "path must be CUDA int32 [seqs, most] with a contiguous last axis");
    beside(path, device, "path");
    void *caches[kMost];
    int32_t row_bytes[kMost];
    const Tensor &first = tensor(PySequence_Fast_GET_ITEM(list.get(), 0), "caches");
    for (Py_ssize_t i = 0; i < count; ++i) {
        const Tensor &c = tensor(PySequence_Fast_GET_ITEM(list.get(), i), "caches");
        TORCH_CHECK_VALUE(c.dim() == 4 && c.is_cuda() && c.is_contiguous(),
                          "caches must be contiguous CUDA tensors [num_blocks, num_kv_heads, block_size, width]");
        TORCH_CHECK_VALUE(c.size(0) == first.size(0) && c.size(1) == first.size(1) && c.size(2) == first.size(2),
                          "caches must agree in num_blocks, num_kv_heads and block_size");
        beside(c, device, "a cache");
        no_gradient(c, "a cache");
        caches[i] = c.data_ptr();
        row_bytes[i] = narrow<int32_t>(c.size(3) * c.element_size(), "bytes of a cache's row");
    }
    TORCH_CHECK_TYPE(args[2] != Py_None && args[3] != Py_None && args[5] != Py_None,
                     "context_len, row_start and path_len must be tensors");
    const int32_t *context_len = array<int32_t>(args[2], device, at::kInt, seqs, "context_len");
    const int32_t *row_start = array<int32_t>(args[3], device, at::kInt, seqs + 1, "row_start");
    const int32_t *path_len = array<int32_t>(args[5], device, at::kInt, seqs, "path_len");
    Tensor new_len;
    if (args[6] != Py_None) {
        array<int32_t>(args[6], device, at::kInt, seqs, "new_len");
        new_len = tensor(args[6], "new_len");
    }
    int32_t *err = counter(args[7], device);
    const On on(device, args[8]);
    if (!new_len.defined())
        new_len = at::empty({seqs}, table.options());
    // (the nodes of all sequences are not known here: row_start's own numbers count)
    const rc_status s = rc_kv_compact(
        caches, row_bytes, (int32_t)count, narrow<int32_t>(first.size(0), "num_blocks"),
        narrow<int32_t>(first.size(1), "num_kv_heads"), narrow<int32_t>(first.size(2), "block_size"),
        static_cast<const int32_t *>(table.const_data_ptr()), table.stride(0), narrow<int32_t>(table.size(1), "width of block_table"),
        context_len, row_start, narrow<int32_t>(seqs, "seqs"), 0x7FFFFFFF, static_cast<const int32_t *>(path.const_data_ptr()),
        path.stride(0), narrow<int32_t>(path.size(1), "width of path"), path_len, new_len.data_ptr<int32_t>(), err, on.stream());
    for (Py_ssize_t i = 0; s == RC_OK && i < count; ++i)
        written({PySequence_Fast_GET_ITEM(list.get(), i)});
    return result(s, new_len, {args[6]});
    END_HANDLE_TH_ERRORS
}

// The exception class that an error status raises.
PyObject *set_error(PyObject *, PyObject *cls) {
    Py_INCREF(cls);
    Py_XSETREF(g_error, cls);
    Py_RETURN_NONE;
}

PyMethodDef g_methods[] = {
    {"rope_table", reinterpret_cast<PyCFunction>(reinterpret_cast<void *>(rope_table)), METH_FASTCALL, nullptr},
    {"rope_apply", reinterpret_cast<PyCFunction>(reinterpret_cast<void *>(rope_apply)), METH_FASTCALL, nullptr},
    {"tree_attention", reinterpret_cast<PyCFunction>(reinterpret_cast<void *>(tree_attention)), METH_FASTCALL, nullptr},
    {"logits_adjust", reinterpret_cast<PyCFunction>(reinterpret_cast<void *>(logits_adjust)), METH_FASTCALL, nullptr},
    {"head_norm_rope", reinterpret_cast<PyCFunction>(reinterpret_cast<void *>(head_norm_rope)), METH_FASTCALL, nullptr},
    {"head_norm_rope_grad", reinterpret_cast<PyCFunction>(reinterpret_cast<void *>(head_norm_rope_grad)), METH_FASTCALL,
     nullptr},
    {"window_attention", reinterpret_cast<PyCFunction>(reinterpret_cast<void *>(window_attention)), METH_FASTCALL, nullptr},
    {"kv4_attention", reinterpret_cast<PyCFunction>(reinterpret_cast<void *>(kv4_attention)), METH_FASTCALL, nullptr},
    {"kv4_store", reinterpret_cast<PyCFunction>(reinterpret_cast<void *>(kv4_store)), METH_FASTCALL, nullptr},
    {"kv4_load", reinterpret_cast<PyCFunction>(reinterpret_cast<void *>(kv4_load)), METH_FASTCALL, nullptr},
    {"kv_compact", reinterpret_cast<PyCFunction>(reinterpret_cast<void *>(kv_compact)), METH_FASTCALL, nullptr},
    {"set_error", set_error, METH_O, nullptr},
    {nullptr, nullptr, 0, nullptr}};

PyModuleDef g_module = {PyModuleDef_HEAD_INIT, "_draft", nullptr, -1, g_methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__draft(void) { return PyModule_Create(&g_module); }
