// The marshalling of blocks.py's calls, compiled: where a kernel takes 4 us, checks
// and allocations made in Python are what a call costs.  On the host, us in Python and
// here: one row of 4096 quantized 9.4 / 4.8 (2.9 of them the launch), a small expert
// layer 18.1 / 8.9, a small layer's gradients 16.9 / 8.3.
//
// Only the ordinary call is taken: tensors of the right types and shapes on the current
// device and stream, outputs to be allocated, the cached workspace there and large
// enough, no capture.  For anything else, errors among it, the result is None, and
// blocks.py's own route does the call or says what is wrong with it.
#include <Python.h>

#include <ATen/core/grad_mode.h>
#include <ATen/ops/empty.h>
#include <ATen/ops/narrow.h>
#include <c10/hip/HIPFunctions.h>
#include <c10/hip/HIPGraphsC10Utils.h>
#include <c10/hip/HIPStream.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include "../../include/gemm_relu_blocks.h"

namespace {

decltype(&gemm_relu_quantize_blocks) quantize_blocks;
decltype(&gemm_relu_blocks) product;
decltype(&gemm_relu_blocks_backward) backward_of;
decltype(&gemm_relu_blocks_backward_workspace) backward_space;
decltype(&gemm_relu_experts) expert_layer;
decltype(&gemm_relu_experts_workspace) experts_space;

constexpr int64_t kBlock = 128;
int64_t blocks_of(int64_t n) { return (n + kBlock - 1) / kBlock; }

const at::Tensor* tensor_of(PyObject* o) { return THPVariable_Check(o) ? &THPVariable_Unpack(o) : nullptr; }

// A contiguous tensor of this type on this device.
bool plain(const at::Tensor* t, int64_t dim, at::ScalarType type, int device)
{
    return t && t->is_cuda() && t->layout() == at::kStrided && t->scalar_type() == type && t->dim() == dim && t->is_contiguous() &&
           t->get_device() == device;
}

int dtype_code(at::ScalarType t) { return t == at::kHalf ? GEMM_RELU_F16 : t == at::kBFloat16 ? GEMM_RELU_BF16 : -1; }

at::ScalarType format_type(int64_t format) { return format == GEMM_RELU_E4M3 ? at::kFloat8_e4m3fn : at::kFloat8_e5m2; }

// Pitch of an 8-bit matrix or stack with elements, 0 where Python has to look at it.
int64_t pitch_of(const at::Tensor* t, int64_t dim, int device, int& format)
{
    if (!t || !t->is_cuda() || t->layout() != at::kStrided || t->dim() != dim || t->get_device() != device || t->requires_grad() || t->numel() == 0)
        return 0;
    format = t->scalar_type() == at::kFloat8_e4m3fn ? GEMM_RELU_E4M3 : t->scalar_type() == at::kFloat8_e5m2 ? GEMM_RELU_E5M2 : -1;
    if (format < 0 || reinterpret_cast<uintptr_t>(t->data_ptr()) % 16 != 0) return 0;
    const int64_t rows = t->size(dim - 2), row = t->size(dim - 1), whole = (row + 15) / 16 * 16;
    if (row == whole && t->is_contiguous()) return row;
    const int64_t pitch = t->stride(dim - 2), count = rows * (dim == 3 ? t->size(0) : 1);
    if (rows < 2 || t->stride(dim - 1) != 1 || pitch < row || pitch % 16 != 0 || (dim == 3 && t->stride(0) != rows * pitch)) return 0;
    return t->storage_offset() + (count - 1) * pitch + whole <= (int64_t)t->storage().nbytes() ? pitch : 0;
}

// Whether autograd asks for a derivative with respect to one of these.
bool wanted(std::initializer_list<const at::Tensor*> tensors)
{
    for (const at::Tensor* t : tensors)
        if (t && ((at::GradMode::is_enabled() && t->requires_grad()) || t->_fw_grad(0).defined())) return true;
    return false;
}

bool sizes_are(const at::Tensor* t, at::IntArrayRef want) { return t->sizes() == want; }

// An argument of another kind than the ordinary call's.
PyObject* not_here()
{
    PyErr_Clear();
    Py_RETURN_NONE;
}

// A call of the library without the interpreter's lock: a full queue makes a launch wait.
template <typename F>
int unlocked(F&& call)
{
    int rc = 0;
    Py_BEGIN_ALLOW_THREADS
    rc = call();
    Py_END_ALLOW_THREADS
    return rc;
}

// quantize(x, format, tiles, mask, rows, transposed, power_of_two)
PyObject* quantize(PyObject*, PyObject* const* args, Py_ssize_t n)
{
    HANDLE_TH_ERRORS
    if (n != 7 || !quantize_blocks) Py_RETURN_NONE;
    const at::Tensor *x = tensor_of(args[0]), *mask = args[3] == Py_None ? nullptr : tensor_of(args[3]);
    const long format = PyLong_AsLong(args[1]);
    const int tiles = PyObject_IsTrue(args[2]), rows = PyObject_IsTrue(args[4]), transposed = PyObject_IsTrue(args[5]),
              power = PyObject_IsTrue(args[6]);
    if (PyErr_Occurred()) return not_here();
    if (!x || !x->is_cuda()) Py_RETURN_NONE;           // (without a GPU there is no current device)
    const int device = c10::hip::current_device(), code = dtype_code(x->scalar_type());
    const int64_t dim = x->dim();
    if (code < 0 || (dim != 2 && dim != 3) || (format != 0 && format != 1) || (!rows && !transposed)) Py_RETURN_NONE;
    if (!plain(x, dim, x->scalar_type(), device) || x->numel() == 0) Py_RETURN_NONE;
    if (args[3] != Py_None && !(plain(mask, dim, x->scalar_type(), device) && sizes_are(mask, x->sizes()))) Py_RETURN_NONE;
    const int64_t R = x->size(dim - 2), C = x->size(dim - 1), count = dim == 3 ? x->size(0) : 1, br = blocks_of(R), bc = blocks_of(C);
    // (long rows start at whole cache lines, as blocks.py's do)
    const auto pitch = [](int64_t row) { return row <= 1024 ? (row + 15) / 16 * 16 : (row + 127) / 128 * 128; };
    const int64_t ldq = pitch(C), ldqt = pitch(R);
    const auto bytes = x->options().dtype(format_type(format)).requires_grad(false), words = bytes.dtype(at::kFloat);
    const auto make = [&](int64_t r, int64_t c, const at::TensorOptions& o) { return dim == 3 ? at::empty({count, r, c}, o) : at::empty({r, c}, o); };
    const auto pitched = [&](int64_t r, int64_t c, int64_t ld) { return ld == c ? make(r, c, bytes) : make(r, ld, bytes).narrow(-1, 0, c); };
    at::Tensor q, s, qt, st;
    if (rows) {
        q = pitched(R, C, ldq);
        s = tiles ? make(br, bc, words) : make(bc, R, words);
    }
    if (transposed) {
        qt = pitched(C, R, ldqt);
        st = tiles ? make(bc, br, words) : make(br, C, words);
    }
    void* const stream = c10::hip::getCurrentHIPStream(device).stream();
    const int rc = unlocked([&] {
        return quantize_blocks(x->data_ptr(), mask ? mask->data_ptr() : nullptr, rows ? q.data_ptr() : nullptr,
                               rows ? static_cast<float*>(s.data_ptr()) : nullptr, transposed ? qt.data_ptr() : nullptr,
                               transposed ? static_cast<float*>(st.data_ptr()) : nullptr, count, R, C, ldq, ldqt, code, (int)format, tiles,
                               power, stream);
    });
    if (rc != GEMM_RELU_OK) Py_RETURN_NONE;
    PyObject* const out = PyTuple_New(2 * (rows + transposed));
    if (!out) return nullptr;
    Py_ssize_t at = 0;
    for (at::Tensor* t : {&q, &s, &qt, &st})
        if (t->defined()) PyTuple_SET_ITEM(out, at++, THPVariable_Wrap(std::move(*t)));
    return out;
    END_HANDLE_TH_ERRORS
}

// multiply(a, a_scales, b, b_scales, ends, bf16, relu, b_rows, config)
PyObject* multiply(PyObject*, PyObject* const* args, Py_ssize_t n)
{
    HANDLE_TH_ERRORS
    if (n != 9 || !product) Py_RETURN_NONE;
    const at::Tensor *a = tensor_of(args[0]), *sa = tensor_of(args[1]), *b = tensor_of(args[2]), *sb = tensor_of(args[3]);
    const bool grouped = args[4] != Py_None;
    const at::Tensor* ends = grouped ? tensor_of(args[4]) : nullptr;
    const int bf16 = PyObject_IsTrue(args[5]), relu = PyObject_IsTrue(args[6]), b_rows = PyObject_IsTrue(args[7]);
    const long config = PyLong_AsLong(args[8]);
    if (PyErr_Occurred()) return not_here();
    if (!a || !a->is_cuda()) Py_RETURN_NONE;
    const int device = c10::hip::current_device();
    int fa = 0, fb = 0;
    const int64_t lda = pitch_of(a, 2, device, fa), ldb = pitch_of(b, grouped ? 3 : 2, device, fb);
    if (!lda || !ldb) Py_RETURN_NONE;
    const int64_t M = a->size(0), K = a->size(1), N = b->size(-2), groups = grouped ? b->size(0) : 1, kb = blocks_of(K);
    if (b->size(-1) != K || config != (int)config) Py_RETURN_NONE;
    if (!plain(sa, 2, at::kFloat, device) || !sizes_are(sa, {kb, M}) || !plain(sb, grouped ? 3 : 2, at::kFloat, device)) Py_RETURN_NONE;
    const int64_t s0 = b_rows ? kb : blocks_of(N), s1 = b_rows ? N : kb;
    if (grouped ? !sizes_are(sb, {groups, s0, s1}) : !sizes_are(sb, {s0, s1})) Py_RETURN_NONE;
    if (wanted({sa, sb})) Py_RETURN_NONE;
    if (grouped && !(plain(ends, 1, at::kInt, device) && ends->size(0) == groups)) Py_RETURN_NONE;
    at::Tensor c = at::empty({M, N}, sa->options().dtype(bf16 ? at::kBFloat16 : at::kHalf).requires_grad(false));
    void* const stream = c10::hip::getCurrentHIPStream(device).stream();
    const int rc = unlocked([&] {
        return product(a->data_ptr(), static_cast<const float*>(sa->data_ptr()), b->data_ptr(), static_cast<const float*>(sb->data_ptr()),
                       grouped ? static_cast<const int32_t*>(ends->data_ptr()) : nullptr, c.data_ptr(), M, N, K, groups, lda, ldb, fa, fb,
                       b_rows ? GEMM_RELU_SCALES_ROWS : GEMM_RELU_SCALES_TILES, bf16 ? GEMM_RELU_BF16 : GEMM_RELU_F16, relu, (int)config,
                       stream);
    });
    if (rc != GEMM_RELU_OK) Py_RETURN_NONE;
    return THPVariable_Wrap(std::move(c));
    END_HANDLE_TH_ERRORS
}

// The stream's cached workspace (groups.py's dict of (device, stream): (address, bytes,
// tensor)), held while this lives; none in a capture, or where it is too small.
struct Space {
    PyObject* entry = nullptr;
    void* at = nullptr;
    int64_t bytes = 0;
    Space(PyObject* spaces, int device, void* stream, int64_t need)
    {
        if (need <= 0 || !PyDict_Check(spaces) ||
            c10::hip::currentStreamCaptureStatusMayInitCtx() != c10::hip::CaptureStatus::None)
            return;
        PyObject* const key = Py_BuildValue("(iK)", device, (unsigned long long)reinterpret_cast<uintptr_t>(stream));
        if (!key) throw python_error();
        entry = PyDict_GetItem(spaces, key);
        Py_DECREF(key);
        if (!entry) return;
        Py_INCREF(entry);
        unsigned long long address = 0;
        long long size = 0;
        PyObject* tensor = nullptr;
        if (!PyArg_ParseTuple(entry, "KLO", &address, &size, &tensor)) throw python_error();
        if (size < need) return;
        at = reinterpret_cast<void*>((uintptr_t)address);
        bytes = size;
    }
    Space(const Space&) = delete;
    ~Space() { Py_XDECREF(entry); }
};

// backward(dc, c, xt, xt_scales, wt, wt_scales, relu, format, spaces): both gradients
PyObject* backward(PyObject*, PyObject* const* args, Py_ssize_t n)
{
    HANDLE_TH_ERRORS
    if (n != 9 || !backward_of) Py_RETURN_NONE;
    const at::Tensor *dc = tensor_of(args[0]), *c = tensor_of(args[1]), *xt = tensor_of(args[2]), *sx = tensor_of(args[3]),
                     *wt = tensor_of(args[4]), *sw = tensor_of(args[5]);
    const int relu = PyObject_IsTrue(args[6]);
    const long format = PyLong_AsLong(args[7]);
    if (PyErr_Occurred()) return not_here();
    if (!dc || !dc->is_cuda() || (format != 0 && format != 1)) Py_RETURN_NONE;
    const int device = c10::hip::current_device(), code = dtype_code(dc->scalar_type());
    if (code < 0 || !plain(dc, 2, dc->scalar_type(), device) || dc->numel() == 0) Py_RETURN_NONE;
    const int64_t M = dc->size(0), N = dc->size(1);
    if (relu && !(plain(c, 2, dc->scalar_type(), device) && sizes_are(c, {M, N}))) Py_RETURN_NONE;
    int fx = 0, fw = 0;
    const int64_t ldx = pitch_of(xt, 2, device, fx), ldw = pitch_of(wt, 2, device, fw);
    if (!ldx || !ldw) Py_RETURN_NONE;
    const int64_t K = xt->size(0);
    if (xt->size(1) != M || !sizes_are(wt, {K, N}) || !plain(sx, 2, at::kFloat, device) || !sizes_are(sx, {blocks_of(M), K}) ||
        !plain(sw, 2, at::kFloat, device) || !sizes_are(sw, {blocks_of(K), blocks_of(N)}) || wanted({sx, sw}))
        Py_RETURN_NONE;
    void* const stream = c10::hip::getCurrentHIPStream(device).stream();
    const Space space(args[8], device, stream, backward_space(M, N, K));
    if (!space.at) Py_RETURN_NONE;
    const auto like = dc->options().requires_grad(false);
    at::Tensor dx = at::empty({M, K}, like), dw = at::empty({N, K}, like);
    const int rc = unlocked([&] {
        return backward_of(dc->data_ptr(), relu ? c->data_ptr() : nullptr, xt->data_ptr(), static_cast<const float*>(sx->data_ptr()),
                           wt->data_ptr(), static_cast<const float*>(sw->data_ptr()), dx.data_ptr(), dw.data_ptr(), M, N, K, ldx, ldw,
                           (int)format, fx, fw, code, relu, space.at, space.bytes, stream);
    });
    if (rc != GEMM_RELU_OK) Py_RETURN_NONE;
    return Py_BuildValue("(NN)", THPVariable_Wrap(std::move(dx)), THPVariable_Wrap(std::move(dw)));
    END_HANDLE_TH_ERRORS
}

// experts(x, w1, w2, logits, top, w1_scales, w2_scales, b_layout, renormalize, spaces)
PyObject* experts(PyObject*, PyObject* const* args, Py_ssize_t n)
{
    HANDLE_TH_ERRORS
    if (n != 10 || !expert_layer) Py_RETURN_NONE;
    const at::Tensor *x = tensor_of(args[0]), *w1 = tensor_of(args[1]), *w2 = tensor_of(args[2]), *logits = tensor_of(args[3]),
                     *s1 = tensor_of(args[5]), *s2 = tensor_of(args[6]);
    const long top = PyLong_AsLong(args[4]), layout = PyLong_AsLong(args[7]);
    const int renormalize = PyObject_IsTrue(args[8]);
    if (PyErr_Occurred()) return not_here();
    if (!x || !w1 || !w2 || !logits || !x->is_cuda() || (layout != GEMM_RELU_B_KN && layout != GEMM_RELU_B_NK)) Py_RETURN_NONE;
    const int device = c10::hip::current_device(), code = dtype_code(x->scalar_type());
    if (code < 0 || !plain(x, 2, x->scalar_type(), device) || !plain(logits, 2, at::kFloat, device) || x->numel() == 0) Py_RETURN_NONE;
    if (wanted({x, w1, w2, logits, s1, s2})) Py_RETURN_NONE;
    const bool eight = w1->scalar_type() == at::kFloat8_e4m3fn || w1->scalar_type() == at::kFloat8_e5m2, nk = layout == GEMM_RELU_B_NK;
    int f1 = -1, f2 = -1;
    int64_t ld1 = 0, ld2 = 0;
    if (eight) {
        ld1 = pitch_of(w1, 3, device, f1);
        ld2 = pitch_of(w2, 3, device, f2);
        if (!nk || !ld1 || !ld2 || f1 != f2) Py_RETURN_NONE;
    } else if (!plain(w1, 3, x->scalar_type(), device) || !plain(w2, 3, x->scalar_type(), device)) {
        Py_RETURN_NONE;
    }
    const int64_t tokens = x->size(0), K = x->size(1), E = w1->size(0), H = w1->size(nk ? 1 : 2), N = w2->size(nk ? 1 : 2);
    if (nk ? !sizes_are(w1, {E, H, K}) || !sizes_are(w2, {E, N, H}) : !sizes_are(w1, {E, K, H}) || !sizes_are(w2, {E, H, N})) Py_RETURN_NONE;
    if (!sizes_are(logits, {tokens, E})) Py_RETURN_NONE;
    if (eight) {
        if (!plain(s1, 3, at::kFloat, device) || !sizes_are(s1, {E, blocks_of(H), blocks_of(K)}) || !plain(s2, 3, at::kFloat, device) ||
            !sizes_are(s2, {E, blocks_of(N), blocks_of(H)}))
            Py_RETURN_NONE;
    } else if (args[5] != Py_None || args[6] != Py_None) {
        Py_RETURN_NONE;
    }
    void* const stream = c10::hip::getCurrentHIPStream(device).stream();
    const Space space(args[9], device, stream, experts_space(tokens, N, H, E, top, (int)layout));
    if (!space.at) Py_RETURN_NONE;
    const auto like = logits->options().requires_grad(false);
    at::Tensor ids = at::empty({tokens, top}, like.dtype(at::kInt)), weights = at::empty({tokens, top}, like),
               y = at::empty({tokens, N}, like.dtype(x->scalar_type()));
    const int rc = unlocked([&] {
        return expert_layer(x->data_ptr(), w1->data_ptr(), eight ? static_cast<const float*>(s1->data_ptr()) : nullptr, w2->data_ptr(),
                            eight ? static_cast<const float*>(s2->data_ptr()) : nullptr, static_cast<const float*>(logits->data_ptr()),
                            static_cast<int32_t*>(ids.data_ptr()), static_cast<float*>(weights.data_ptr()), y.data_ptr(), tokens, N, K, H, E,
                            top, ld1, ld2, renormalize, code, f1, (int)layout, space.at, space.bytes, stream);
    });
    if (rc != GEMM_RELU_OK) Py_RETURN_NONE;
    return Py_BuildValue("(NNN)", THPVariable_Wrap(std::move(y)), THPVariable_Wrap(std::move(ids)), THPVariable_Wrap(std::move(weights)));
    END_HANDLE_TH_ERRORS
}

// use(..): addresses of the library's entry points
PyObject* use(PyObject*, PyObject* args)
{
    unsigned long long f[6];
    if (!PyArg_ParseTuple(args, "KKKKKK", f, f + 1, f + 2, f + 3, f + 4, f + 5)) return nullptr;
    quantize_blocks = reinterpret_cast<decltype(quantize_blocks)>(f[0]);
    product = reinterpret_cast<decltype(product)>(f[1]);
    backward_of = reinterpret_cast<decltype(backward_of)>(f[2]);
    backward_space = reinterpret_cast<decltype(backward_space)>(f[3]);
    expert_layer = reinterpret_cast<decltype(expert_layer)>(f[4]);
    experts_space = reinterpret_cast<decltype(experts_space)>(f[5]);
    Py_RETURN_NONE;
}

using Fast = PyObject* (*)(PyObject*, PyObject* const*, Py_ssize_t);
PyCFunction fast(Fast f) { return reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(f)); }

PyMethodDef methods[] = {{"quantize", fast(quantize), METH_FASTCALL, nullptr},
                         {"multiply", fast(multiply), METH_FASTCALL, nullptr},
                         {"backward", fast(backward), METH_FASTCALL, nullptr},
                         {"experts", fast(experts), METH_FASTCALL, nullptr},
                         {"use", use, METH_VARARGS, nullptr},
                         {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_blocks_calls", nullptr, -1, methods};

}  // namespace

PyMODINIT_FUNC PyInit__blocks_calls()
{
    PyObject* const m = PyModule_Create(&module);
    if (m && PyModule_AddStringConstant(m, "torch_version", GEMM_RELU_TORCH_VERSION) != 0) {
        Py_DECREF(m);
        return nullptr;
    }
    return m;
}
