// Python module _tensor_calls: the drafted-token step's calls on torch tensors.
//
// It checks the tensors, fills the descriptors of include/rank_adapter_apply.h,
// allocates outputs and workspace with torch's allocator and calls the C entry
// points, whose addresses operators.py hands over (so that one copy of the
// library is loaded). Native because a small call's time is the host's: the same
// checks and descriptor in Python and ctypes took 14-21 us a call on the GPU
// box's host cores, beside 2-3 us for the launch itself.
//
// What does not fit raises ValueError; a status of the library goes to the
// Python function given to bind(), which raises.
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <ATen/core/TensorBody.h>
#include <ATen/cuda/EmptyTensor.h>
#include <c10/core/AutogradState.h>
#include <c10/core/GradMode.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <climits>

#include "rank_adapter_apply.h"

namespace {

decltype(&lora_base_linear) g_base_linear;
decltype(&lora_rope) g_rope;
decltype(&lora_tree_attention) g_tree;
decltype(&lora_tree_attention_workspace_bytes) g_tree_bytes;
decltype(&lora_verify_drafts) g_verify;
PyObject *g_raise;          // called with a status that is not LORA_OK

using at::Tensor;

// The tensor at `o`, or nullptr for None where that is allowed.
const Tensor *tensor(PyObject *o, const char *name, bool optional = false) {
    if (optional && o == Py_None) return nullptr;
    TORCH_CHECK_VALUE(THPVariable_Check(o), name, " is not a tensor");
    return &THPVariable_Unpack(o);
}

struct Where {
    c10::Device device;
    int dtype;
    void *stream;
};

Where start(const Tensor &first, const char *name) {
    TORCH_CHECK_VALUE(first.scalar_type() == at::kBFloat16 || first.scalar_type() == at::kFloat, name, " has dtype ",
                      first.scalar_type(), ": bfloat16 or float32 is needed");
    TORCH_CHECK_VALUE(first.is_cuda(), name, " is on ", first.device(), ": a CUDA device is needed");
    TORCH_CHECK_VALUE(first.device().index() == c10::cuda::current_device(), name, " is on ", first.device(),
                      ", which is not the current device");
    return {first.device(), first.scalar_type() == at::kFloat ? LORA_DTYPE_F32 : LORA_DTYPE_BF16,
            c10::cuda::getCurrentCUDAStream(first.device().index()).stream()};
}

void same(const Tensor &t, const Where &w, at::ScalarType type, const char *name) {
    TORCH_CHECK_VALUE(t.device() == w.device, name, " is on ", t.device(), ", not on ", w.device);
    TORCH_CHECK_VALUE(t.scalar_type() == type, name, " has dtype ", t.scalar_type(), ": ", type, " is needed");
    TORCH_CHECK_VALUE(!t.requires_grad() || !c10::GradMode::is_enabled(), name,
                      " requires a gradient, which these calls do not record: detach it or use torch.no_grad()");
    TORCH_CHECK_VALUE(!c10::AutogradState::get_tls_state().get_fw_grad_mode() || !t._fw_grad(0).defined(), name,
                      " has a forward-mode tangent, which these calls do not carry on: take its primal");
}

// A call wrote `t` in place: autograd sees by its version that what it saved of it is gone. (Inference tensors have none.)
void written(const Tensor &t) {
    if (!t.is_inference()) t.unsafeGetTensorImpl()->bump_version();
}

// Last dimension contiguous (as far as it has more than one element).
void unit(const Tensor &t, int64_t dims, const char *name) {
    TORCH_CHECK_VALUE(t.dim() == dims, name, " has ", t.dim(), " dimensions: ", dims, " are needed");
    TORCH_CHECK_VALUE(t.stride(dims - 1) == 1 || t.size(dims - 1) <= 1 || t.numel() == 0, name,
                      " needs unit stride in its last dimension");
}

void whole(const Tensor &t, int64_t dims, const char *name) {
    TORCH_CHECK_VALUE(t.dim() == dims, name, " has ", t.dim(), " dimensions: ", dims, " are needed");
    TORCH_CHECK_VALUE(t.is_contiguous(), name, " has to be contiguous");
}

int count(int64_t n, const char *name) {
    TORCH_CHECK_VALUE(n <= INT_MAX, name, " (", n, ") is too large");
    return (int)n;
}

Tensor fresh(at::IntArrayRef size, at::ScalarType type, const Where &w) {
    return at::detail::empty_cuda(size, type, w.device, std::nullopt);
}

// `out` checked against `like`'s shape, or a new tensor of it.
Tensor output(const Tensor *out, at::IntArrayRef size, at::ScalarType type, const Where &w) {
    if (!out) return fresh(size, type, w);
    same(*out, w, type, "out");
    unit(*out, (int64_t)size.size(), "out");
    TORCH_CHECK_VALUE(out->sizes() == size, "out has shape ", out->sizes(), ": ", size, " is needed");
    return *out;
}

bool done(int rc) {
    if (rc == LORA_OK) return true;
    PyObject *r = PyObject_CallFunction(g_raise, "i", rc);
    Py_XDECREF(r);
    if (!PyErr_Occurred()) PyErr_SetString(PyExc_RuntimeError, "the library refused the call");
    return false;
}

// The truth of `o`; false where asking for it raised.
bool flag(PyObject *o, int &value) {
    value = PyObject_IsTrue(o);
    return value >= 0;
}

bool arguments(Py_ssize_t n, Py_ssize_t want) {
    if (n == want) return true;
    PyErr_Format(PyExc_TypeError, "%zd arguments: %zd are needed", n, want);
    return false;
}

// base_linear(x, qweight, scales, zeros, out)
PyObject *base_linear(PyObject *, PyObject *const *v, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    if (!arguments(n, 5)) return nullptr;
    const Tensor &x = *tensor(v[0], "x"), &qw = *tensor(v[1], "qweight"), &sc = *tensor(v[2], "scales");
    const Tensor *zeros = tensor(v[3], "zeros", true), *out = tensor(v[4], "out", true);
    const Where w = start(x, "x");
    const auto type = x.scalar_type();
    same(x, w, type, "x");
    same(qw, w, at::kByte, "qweight");
    same(sc, w, type, "scales");
    unit(x, 2, "x");
    whole(qw, 2, "qweight");
    whole(sc, 2, "scales");
    const int64_t tokens = x.size(0), d_in = x.size(1), d_out = sc.size(0), groups = sc.size(1);
    TORCH_CHECK_VALUE(groups > 0 && d_in % groups == 0 && qw.size(0) == d_out && 2 * qw.size(1) == d_in, "x ", x.sizes(),
                      ", qweight ", qw.sizes(), ", scales ", sc.sizes(), " do not fit");
    if (zeros) {
        same(*zeros, w, at::kByte, "zeros");
        whole(*zeros, 2, "zeros");
        TORCH_CHECK_VALUE(zeros->sizes() == sc.sizes(), "zeros ", zeros->sizes(), ": the shape of scales ", sc.sizes(),
                          " is needed");
    }
    const int64_t size[] = {tokens, d_out};
    Tensor y = output(out, size, type, w);
    lora_base_linear_desc d{};
    d.x = x.const_data_ptr();
    d.x_stride = x.stride(0);
    d.qweight = static_cast<const uint8_t *>(qw.const_data_ptr());
    d.scales = sc.const_data_ptr();
    d.zeros = zeros ? static_cast<const uint8_t *>(zeros->const_data_ptr()) : nullptr;
    d.y = y.mutable_data_ptr();
    d.y_stride = y.stride(0);
    d.n_tokens = count(tokens, "tokens");
    d.d_in = count(d_in, "d_in");
    d.d_out = count(d_out, "d_out");
    d.group = (int)(d_in / groups);
    d.dtype = w.dtype;
    if (!done(g_base_linear(&d, w.stream))) return nullptr;
    if (out) written(y);
    return THPVariable_Wrap(std::move(y));
    END_HANDLE_TH_ERRORS
}

// What rope and rope_append share: q, its output, positions and table.
Tensor rotated(const Tensor &q, const Tensor &positions, const Tensor &table, const Tensor *out, const Where &w,
               lora_rope_desc &d) {
    same(q, w, q.scalar_type(), "q");
    unit(q, 3, "q");
    same(positions, w, at::kInt, "positions");
    whole(positions, 1, "positions");
    same(table, w, at::kFloat, "table");
    whole(table, 2, "table");
    TORCH_CHECK_VALUE(positions.size(0) == q.size(0), "positions holds ", positions.size(0), " entries: one for each of ",
                      q.size(0), " tokens is needed");
    Tensor y = output(out, q.sizes(), q.scalar_type(), w);
    d.q = q.const_data_ptr();
    d.q_token = q.stride(0);
    d.q_head = q.stride(1);
    d.q_out = y.mutable_data_ptr();
    d.q_out_token = y.stride(0);
    d.q_out_head = y.stride(1);
    d.positions = static_cast<const int32_t *>(positions.const_data_ptr());
    d.table = static_cast<const float *>(table.const_data_ptr());
    d.n_positions = count(table.size(0), "table rows");
    d.rot_dim = count(table.size(1), "rot_dim");
    d.n_tokens = count(q.size(0), "tokens");
    d.n_heads = count(q.size(1), "heads");
    d.head_dim = count(q.size(2), "head_dim");
    d.page_size = 1;
    d.dtype = w.dtype;
    return y;
}

// rope(x, positions, table, interleaved, inverse, out)
PyObject *rope(PyObject *, PyObject *const *v, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    if (!arguments(n, 6)) return nullptr;
    const Tensor &x = *tensor(v[0], "x");
    const Tensor &positions = *tensor(v[1], "positions"), &table = *tensor(v[2], "table");
    const Where w = start(x, "x");
    lora_rope_desc d{};
    const Tensor *out = tensor(v[5], "out", true);
    Tensor y = rotated(x, positions, table, out, w, d);
    if (!flag(v[3], d.interleaved) || !flag(v[4], d.inverse)) return nullptr;
    if (!done(g_rope(&d, w.stream))) return nullptr;
    if (out) written(y);
    return THPVariable_Wrap(std::move(y));
    END_HANDLE_TH_ERRORS
}

void check_cache(const Tensor &k, const Tensor &v, const Where &w, at::ScalarType type, int64_t kv_heads, int64_t dim) {
    same(k, w, type, "k_cache");
    same(v, w, type, "v_cache");
    unit(k, 4, "k_cache");
    TORCH_CHECK_VALUE(k.size(2) == kv_heads && k.size(3) == dim, "k_cache ", k.sizes(), ": [pages, page_size, ", kv_heads,
                      ", ", dim, "] is needed");
    TORCH_CHECK_VALUE(v.sizes() == k.sizes() && v.strides() == k.strides(),
                      "k_cache and v_cache need one shape and one set of strides");
}

// rope_append(q, k, v, positions, table, k_cache, v_cache, slots, interleaved, out)
PyObject *rope_append(PyObject *, PyObject *const *v, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    if (!arguments(n, 10)) return nullptr;
    const Tensor &q = *tensor(v[0], "q"), &k = *tensor(v[1], "k"), &val = *tensor(v[2], "v");
    const Tensor &positions = *tensor(v[3], "positions"), &table = *tensor(v[4], "table");
    const Tensor &kc = *tensor(v[5], "k_cache"), &vc = *tensor(v[6], "v_cache"), &slots = *tensor(v[7], "slots");
    const Where w = start(q, "q");
    const auto type = q.scalar_type();
    lora_rope_desc d{};
    same(k, w, type, "k");
    same(val, w, type, "v");
    unit(k, 3, "k");
    unit(val, 3, "v");
    same(slots, w, at::kLong, "slots");
    whole(slots, 1, "slots");
    TORCH_CHECK_VALUE(q.dim() == 3 && k.size(0) == q.size(0) && k.size(2) == q.size(2) && val.sizes() == k.sizes(), "q ",
                      q.sizes(), ", k ", k.sizes(), ", v ", val.sizes(), " do not fit");
    TORCH_CHECK_VALUE(slots.size(0) == q.size(0), "slots holds ", slots.size(0), " entries: one for each of ", q.size(0),
                      " tokens is needed");
    check_cache(kc, vc, w, type, k.size(1), k.size(2));
    const Tensor *out = tensor(v[9], "out", true);
    Tensor y = rotated(q, positions, table, out, w, d);
    if (!flag(v[8], d.interleaved)) return nullptr;
    d.k = k.const_data_ptr();
    d.k_token = k.stride(0);
    d.k_head = k.stride(1);
    d.v = val.const_data_ptr();
    d.v_token = val.stride(0);
    d.v_head = val.stride(1);
    d.k_cache = kc.mutable_data_ptr();
    d.v_cache = vc.mutable_data_ptr();
    d.cache_page = kc.stride(0);
    d.cache_slot = kc.stride(1);
    d.cache_head = kc.stride(2);
    d.slots = static_cast<const int64_t *>(slots.const_data_ptr());
    d.n_pages = kc.size(0);
    d.page_size = count(kc.size(1), "page_size");
    d.n_kv_heads = count(k.size(1), "kv_heads");
    if (!done(g_rope(&d, w.stream))) return nullptr;
    if (out) written(y);
    written(kc);
    written(vc);
    return THPVariable_Wrap(std::move(y));
    END_HANDLE_TH_ERRORS
}

// tree_attention(q, k_cache, v_cache, page_table, ctx_lens, node_starts, tree_mask, scale, out)
PyObject *tree_attention(PyObject *, PyObject *const *v, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    if (!arguments(n, 9)) return nullptr;
    const Tensor &q = *tensor(v[0], "q"), &kc = *tensor(v[1], "k_cache"), &vc = *tensor(v[2], "v_cache");
    const Tensor &table = *tensor(v[3], "page_table"), &ctx = *tensor(v[4], "ctx_lens");
    const Tensor &starts = *tensor(v[5], "node_starts");
    const Tensor *mask = tensor(v[6], "tree_mask", true), *out = tensor(v[8], "out", true);
    const Where w = start(q, "q");
    const auto type = q.scalar_type();
    same(q, w, type, "q");
    unit(q, 3, "q");
    TORCH_CHECK_VALUE(kc.dim() == 4, "k_cache ", kc.sizes(), ": [pages, page_size, kv_heads, head_dim] is needed");
    check_cache(kc, vc, w, type, kc.size(2), q.size(2));
    same(table, w, at::kInt, "page_table");
    same(ctx, w, at::kInt, "ctx_lens");
    same(starts, w, at::kInt, "node_starts");
    unit(table, 2, "page_table");
    whole(ctx, 1, "ctx_lens");
    whole(starts, 1, "node_starts");
    const int64_t requests = ctx.size(0), tokens = q.size(0);
    TORCH_CHECK_VALUE(table.size(0) == requests && starts.size(0) == requests + 1, "page_table ", table.sizes(),
                      ", ctx_lens ", ctx.sizes(), ", node_starts ", starts.sizes(), " do not fit");
    lora_tree_attention_desc d{};
    if (mask) {
        same(*mask, w, at::kLong, "tree_mask");
        whole(*mask, 2, "tree_mask");
        TORCH_CHECK_VALUE(mask->size(0) == tokens, "tree_mask ", mask->sizes(), ": a row for each of ", tokens,
                          " tokens is needed");
        d.tree_mask = static_cast<const uint64_t *>(mask->const_data_ptr());
        d.mask_words = count(mask->size(1), "mask words");
    }
    if (v[7] == Py_None) {
        d.scale = q.size(2) > 0 ? 1.0f / std::sqrt((float)q.size(2)) : 1.0f;
    } else {
        d.scale = (float)PyFloat_AsDouble(v[7]);
        if (PyErr_Occurred()) return nullptr;
    }
    d.n_requests = count(requests, "requests");
    d.n_tokens = count(tokens, "tokens");
    d.n_heads = count(q.size(1), "heads");
    d.n_kv_heads = count(kc.size(2), "kv_heads");
    d.head_dim = count(q.size(2), "head_dim");
    d.dtype = w.dtype;
    Tensor y = output(out, q.sizes(), type, w);
    const int64_t lse_size[] = {tokens, q.size(1)};
    Tensor lse = fresh(lse_size, at::kFloat, w);
    const size_t bytes = g_tree_bytes(d.n_requests, d.n_tokens, d.n_heads, d.n_kv_heads, d.head_dim, d.dtype);
    const int64_t ws_size[] = {(int64_t)bytes};
    Tensor ws = fresh(ws_size, at::kByte, w);
    d.q = q.const_data_ptr();
    d.q_token = q.stride(0);
    d.q_head = q.stride(1);
    d.k_cache = kc.const_data_ptr();
    d.v_cache = vc.const_data_ptr();
    d.cache_page = kc.stride(0);
    d.cache_slot = kc.stride(1);
    d.cache_head = kc.stride(2);
    d.n_pages = kc.size(0);
    d.page_size = count(kc.size(1), "page_size");
    d.page_table = static_cast<const int32_t *>(table.const_data_ptr());
    d.table_stride = table.stride(0);
    d.table_pages = count(table.size(1), "page_table columns");
    d.ctx_lens = static_cast<const int32_t *>(ctx.const_data_ptr());
    d.node_starts = static_cast<const int32_t *>(starts.const_data_ptr());
    d.out = y.mutable_data_ptr();
    d.out_token = y.stride(0);
    d.out_head = y.stride(1);
    d.lse = static_cast<float *>(lse.mutable_data_ptr());
    d.workspace = ws.mutable_data_ptr();
    d.workspace_bytes = bytes;
    if (!done(g_tree(&d, w.stream))) return nullptr;
    if (out) written(y);
    PyObject *a = THPVariable_Wrap(std::move(y)), *b = THPVariable_Wrap(std::move(lse));
    return a && b ? Py_BuildValue("(NN)", a, b) : nullptr;
    END_HANDLE_TH_ERRORS
}

// verify_drafts(target, draft, tokens, parents, node_starts, uniforms, noise, max_path)
PyObject *verify_drafts(PyObject *, PyObject *const *v, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    if (!arguments(n, 8)) return nullptr;
    const Tensor &target = *tensor(v[0], "target"), *draft = tensor(v[1], "draft", true);
    const Tensor &tokens = *tensor(v[2], "tokens"), &parents = *tensor(v[3], "parents");
    const Tensor &starts = *tensor(v[4], "node_starts"), &uniforms = *tensor(v[5], "uniforms");
    const Tensor &noise = *tensor(v[6], "noise");
    const long most = PyLong_AsLong(v[7]);
    if (most == -1 && PyErr_Occurred()) return nullptr;
    TORCH_CHECK_VALUE(most >= 0 && most <= INT_MAX, "max_path is ", most);
    const Where w = start(target, "target");
    const auto type = target.scalar_type();
    same(target, w, type, "target");
    unit(target, 2, "target");
    if (draft) {
        same(*draft, w, type, "draft");
        unit(*draft, 2, "draft");
        TORCH_CHECK_VALUE(draft->sizes() == target.sizes(), "draft ", draft->sizes(), ": target's shape ", target.sizes(),
                          " is needed");
    }
    same(tokens, w, at::kInt, "tokens");
    same(parents, w, at::kInt, "parents");
    same(starts, w, at::kInt, "node_starts");
    same(uniforms, w, at::kFloat, "uniforms");
    same(noise, w, at::kFloat, "noise");
    whole(tokens, 1, "tokens");
    whole(parents, 1, "parents");
    whole(starts, 1, "node_starts");
    whole(uniforms, 1, "uniforms");
    unit(noise, 2, "noise");
    const int64_t nodes = target.size(0), vocab = target.size(1), requests = starts.size(0) - 1;
    TORCH_CHECK_VALUE(requests >= 0 && tokens.size(0) == nodes && parents.size(0) == nodes && uniforms.size(0) == nodes,
                      "tokens, parents and uniforms hold one entry for each of ", nodes,
                      " nodes, node_starts requests + 1");
    TORCH_CHECK_VALUE(noise.size(0) == requests && noise.size(1) == vocab, "noise ", noise.sizes(), ": [", requests, ", ",
                      vocab, "] is needed");
    const int64_t path_size[] = {requests, most}, each[] = {requests};
    Tensor path = fresh(path_size, at::kInt, w), accepted = fresh(each, at::kInt, w), next = fresh(each, at::kInt, w);
    lora_verify_desc d{};
    d.target = target.const_data_ptr();
    d.target_row = target.stride(0);
    d.draft = draft ? draft->const_data_ptr() : nullptr;
    d.draft_row = draft ? draft->stride(0) : 0;
    d.tokens = static_cast<const int32_t *>(tokens.const_data_ptr());
    d.parents = static_cast<const int32_t *>(parents.const_data_ptr());
    d.node_starts = static_cast<const int32_t *>(starts.const_data_ptr());
    d.uniforms = static_cast<const float *>(uniforms.const_data_ptr());
    d.noise = static_cast<const float *>(noise.const_data_ptr());
    d.noise_row = noise.stride(0);
    d.path = static_cast<int32_t *>(path.mutable_data_ptr());
    d.n_accepted = static_cast<int32_t *>(accepted.mutable_data_ptr());
    d.next_token = static_cast<int32_t *>(next.mutable_data_ptr());
    d.max_path = (int)most;
    d.n_requests = count(requests, "requests");
    d.n_nodes = count(nodes, "nodes");
    d.vocab = count(vocab, "vocab");
    d.dtype = w.dtype;
    if (!done(g_verify(&d, w.stream))) return nullptr;
    PyObject *a = THPVariable_Wrap(std::move(path)), *b = THPVariable_Wrap(std::move(accepted)),
             *c = THPVariable_Wrap(std::move(next));
    return a && b && c ? Py_BuildValue("(NNN)", a, b, c) : nullptr;
    END_HANDLE_TH_ERRORS
}

// bind(base_linear, rope, tree_attention, tree_attention_workspace_bytes, verify_drafts addresses, raise)
PyObject *bind(PyObject *, PyObject *const *v, Py_ssize_t n) {
    if (!arguments(n, 6)) return nullptr;
    void *p[5];
    for (int i = 0; i < 5; ++i) {
        p[i] = PyLong_AsVoidPtr(v[i]);
        if (!p[i]) return PyErr_Occurred() ? nullptr : PyErr_Format(PyExc_ValueError, "address %d is NULL", i);
    }
    g_base_linear = reinterpret_cast<decltype(g_base_linear)>(p[0]);
    g_rope = reinterpret_cast<decltype(g_rope)>(p[1]);
    g_tree = reinterpret_cast<decltype(g_tree)>(p[2]);
    g_tree_bytes = reinterpret_cast<decltype(g_tree_bytes)>(p[3]);
    g_verify = reinterpret_cast<decltype(g_verify)>(p[4]);
    Py_INCREF(v[5]);
    Py_XDECREF(g_raise);
    g_raise = v[5];
    Py_RETURN_NONE;
}

#define CALL(name) {#name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(name)), METH_FASTCALL, nullptr}
PyMethodDef methods[] = {CALL(bind),           CALL(base_linear),    CALL(rope), CALL(rope_append),
                         CALL(tree_attention), CALL(verify_drafts), {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_tensor_calls", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__tensor_calls() { return PyModule_Create(&module); }
