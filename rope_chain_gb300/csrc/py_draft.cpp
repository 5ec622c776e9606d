// Python side of the drafted tokens' calls (rc_rope_table, rc_rope_apply,
// rc_tree_attention, rc_logits_adjust): checks torch tensors, makes the output
// and calls the C ABI.  The other calls of the package go through ctypes, whose
// 6 to 12 us a call these cannot afford: their kernels take 2 to 20 us.
// Arguments come by position (rope_chain_gb300/__init__.py has the signatures
// and their documentation).
#include "rope_chain.h"

#include <ATen/core/Tensor.h>
#include <ATen/core/grad_mode.h>
#include <ATen/ops/empty.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Device.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

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

// The calls record nothing for autograd (rope_apply does so in Python).
void no_gradient(const Tensor &t, const char *name) {
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
    return s == RC_OK ? THPVariable_Wrap(out) : raise_status(s);
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
    return s == RC_OK ? THPVariable_Wrap(out) : raise_status(s);
    END_HANDLE_TH_ERRORS
}

PyObject *tree_attention(PyObject *, PyObject *const *args, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    // q, row_start, context_len, block_table, cache, tree_mask, scale, out, lse,
    // err, workspace, stream
    need(n, 12);
    const Tensor &q = tensor(args[0], "q"), &table = tensor(args[3], "block_table"), &cache = tensor(args[4], "cache");
    TORCH_CHECK_VALUE(q.dim() == 3 && q.size(2) == 64 && q.scalar_type() == at::kBFloat16 && q.is_cuda(),
                      "q must be a CUDA bfloat16 view [rows, num_heads, 64]");
    const int64_t rows = q.size(0), heads = q.size(1);
    TORCH_CHECK_VALUE(q.stride(2) == 1 && (heads == 1 || q.stride(1) == 64), "q needs strides (*, 64, 1)");
    TORCH_CHECK_VALUE(cache.dim() == 4 && cache.size(3) == 128 && cache.scalar_type() == at::kBFloat16 &&
                          cache.is_cuda() && cache.is_contiguous(),
                      "cache must be contiguous CUDA bfloat16 [num_blocks, num_kv_heads, block_size, 128]");
    TORCH_CHECK_VALUE(table.dim() == 2 && table.scalar_type() == at::kInt && table.is_cuda() &&
                          (table.size(1) <= 1 || table.stride(1) == 1),
                      "block_table must be CUDA int32 [seqs, width] with a contiguous last axis");
    const int64_t seqs = table.size(0);
    const at::Device device = q.device();
    beside(cache, device, "cache");
    beside(table, device, "block_table");
    no_gradient(q, "q");
    no_gradient(cache, "cache");
    int64_t words = 0;
    if (args[5] != Py_None) {
        const Tensor &mask = tensor(args[5], "tree_mask");
        TORCH_CHECK_VALUE(mask.dim() == 2 && mask.size(0) == rows, "tree_mask must be [rows, words]");
        words = mask.size(1);
        TORCH_CHECK_VALUE(words > 0 || rows == 0, "tree_mask needs a word per row at least");
    }
    float *lse = nullptr;
    if (args[8] != Py_None) {
        const Tensor &t = tensor(args[8], "lse");
        TORCH_CHECK_VALUE(t.dim() == 2 && t.size(0) == rows && t.size(1) == heads, "lse must be [rows, num_heads]");
        lse = const_cast<float *>(array<float>(args[8], device, at::kFloat, 0, "lse"));
    }
    void *workspace = nullptr;
    size_t workspace_bytes = 0;
    if (args[10] != Py_None) {
        const Tensor &t = tensor(args[10], "workspace");
        TORCH_CHECK_VALUE(t.is_cuda() && t.is_contiguous(), "workspace must be a contiguous CUDA tensor");
        beside(t, device, "workspace");
        workspace = t.data_ptr();
        workspace_bytes = t.nbytes();
    }
    TORCH_CHECK_TYPE(args[1] != Py_None && args[2] != Py_None, "row_start and context_len must be tensors");
    const int32_t *row_start = array<int32_t>(args[1], device, at::kInt, seqs + 1, "row_start");
    const int32_t *context_len = array<int32_t>(args[2], device, at::kInt, seqs, "context_len");
    const int64_t *tree_mask = array<int64_t>(args[5], device, at::kLong, 0, "tree_mask");
    int32_t *err = counter(args[9], device);
    Tensor out = output(args[7], q, "q");
    TORCH_CHECK_VALUE(!out.defined() || (out.stride(2) == 1 && (heads == 1 || out.stride(1) == 64)),
                      "out needs strides (*, 64, 1)");
    const On on(device, args[11]);
    made(out, q);
    const rc_status s = rc_tree_attention(
        static_cast<const uint16_t *>(q.const_data_ptr()), q.stride(0), rows, narrow<int32_t>(heads, "num_heads"),
        narrow<int32_t>(cache.size(1), "num_kv_heads"), row_start, narrow<int32_t>(seqs, "seqs"), context_len,
        static_cast<const int32_t *>(table.const_data_ptr()), table.stride(0),
        narrow<int32_t>(table.size(1), "width of block_table"), reinterpret_cast<const uint64_t *>(tree_mask),
        narrow<int32_t>(words, "words of tree_mask"), static_cast<const uint16_t *>(cache.const_data_ptr()),
        narrow<int32_t>(cache.size(0), "num_blocks"), narrow<int32_t>(cache.size(2), "block_size"),
        (float)number(args[6]), static_cast<uint16_t *>(out.data_ptr()), out.stride(0), lse, err,
        workspace, workspace_bytes, on.stream());
    return s == RC_OK ? THPVariable_Wrap(out) : raise_status(s);
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
    return s == RC_OK ? THPVariable_Wrap(out) : raise_status(s);
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
    {"set_error", set_error, METH_O, nullptr},
    {nullptr, nullptr, 0, nullptr}};

PyModuleDef g_module = {PyModuleDef_HEAD_INIT, "_draft", nullptr, -1, g_methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__draft(void) { return PyModule_Create(&g_module); }
