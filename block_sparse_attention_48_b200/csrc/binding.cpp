// Python binding of the serving calls (fa_rope_apply, fa_paged_append, fa_decode_paged,
// fa_decode_shared).  One step's call takes a few microseconds on the GPU, so the way
// there counts: through ctypes and Python's view of the tensors it took 15 to 21 us a
// call, here 5 to 8.  The C ABI's functions come in as addresses (bind), so that this
// file needs no link against the CUDA library.
//
// It is compiled against one torch (FA_TORCH_VERSION, the build's), which the package checks
// when it is imported.
//
// Every function takes positional arguments and returns its outputs, or the fa_status of
// a call that the library refused.
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <algorithm>
#include <map>
#include <utility>

#include <ATen/ATen.h>
#include <c10/cuda/CUDAGraphsC10Utils.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include "flexattn.h"

namespace {

struct Calls {
    decltype(&fa_rope_apply) rope_apply;
    decltype(&fa_paged_append) paged_append;
    decltype(&fa_decode_paged) decode_paged;
    decltype(&fa_decode_shared) decode_shared;
    decltype(&fa_decode_paged_workspace_size) decode_paged_size;
    decltype(&fa_decode_shared_workspace_size) decode_shared_size;
    decltype(&fa_workspace_size) workspace_size;
} calls;

// ------------------------------------------------------------------ arguments

const at::Tensor& tensor(PyObject* o, const char* what)
{
    TORCH_CHECK_TYPE(THPVariable_Check(o), what, ": expected a tensor, got ", Py_TYPE(o)->tp_name);
    return THPVariable_Unpack(o);
}

long long integer(PyObject* o)
{
    const long long x = PyLong_AsLongLong(o);
    if (x == -1 && PyErr_Occurred()) throw python_error();
    return x;
}

double number(PyObject* o)
{
    const double x = PyFloat_AsDouble(o);
    if (x == -1.0 && PyErr_Occurred()) throw python_error();
    return x;
}

bool truth(PyObject* o)
{
    const int x = PyObject_IsTrue(o);
    if (x < 0) throw python_error();
    return x != 0;
}

int device_of(const at::Tensor& t, const char* what)
{
    TORCH_CHECK_TYPE(t.is_cuda(), what, ": expected CUDA tensors");
    return t.get_device();
}

fa_tensor describe(const at::Tensor& t, int device, const char* what)
{
    TORCH_CHECK_TYPE(t.scalar_type() == at::kBFloat16 && t.dim() == 4 && t.is_cuda() && t.get_device() == device, what,
                     ": expected a 4-D bf16 tensor on cuda:", device, ", got ", t.scalar_type(), " ", t.sizes(), " on ",
                     t.device());
    fa_tensor d;
    d.data = t.data_ptr();
    for (int i = 0; i < 4; ++i) {
        d.dims[i] = t.size(i);
        d.strides[i] = t.stride(i);
    }
    return d;
}

// t itself, or a contiguous copy where its strides or alignment are not ones the kernels
// read (16-byte vectors along D, no expanded dimension).
at::Tensor readable(const at::Tensor& t)
{
    if (t.dim() != 4 || t.numel() == 0) return t;
    bool ok = t.stride(3) == 1 && (reinterpret_cast<uintptr_t>(t.data_ptr()) & 15) == 0;
    for (int i = 0; i < 3; ++i) ok = ok && t.stride(i) % 8 == 0 && (t.stride(i) != 0 || t.size(i) == 1);
    return ok ? t : t.is_contiguous() ? t.clone() : t.contiguous();
}

// A tensor of the caller's has been written: autograd's count of its changes in place goes up,
// as after torch's own in-place operators (a tensor made in inference mode has none).
void written(const at::Tensor& t)
{
    if (!t.is_inference()) t.unsafeGetTensorImpl()->bump_version();
}

// Data of an int32 tensor of one or two dimensions (a size of -1: any), the last contiguous.
const int32_t* ints(const at::Tensor& t, int dims, int64_t n0, int64_t n1, int device, const char* what)
{
    bool ok = t.scalar_type() == at::kInt && t.is_cuda() && t.get_device() == device && t.dim() == dims &&
              t.size(0) == n0 && (dims == 1 || n1 < 0 || t.size(1) == n1);
    ok = ok && (t.stride(dims - 1) == 1 || t.size(dims - 1) <= 1);
    TORCH_CHECK_TYPE(ok, what, ": expected int32 [", n0, dims == 2 ? ", " : "", dims == 2 && n1 >= 0 ? std::to_string(n1) : "",
                     "] on cuda:", device, " with a contiguous last dimension, got ", t.scalar_type(), " ", t.sizes(),
                     " on ", t.device());
    return t.data_ptr<int32_t>();
}

fa_rope rope_of(const at::Tensor& f, bool interleaved, double amplitude, int device)
{
    TORCH_CHECK_TYPE(f.scalar_type() == at::kDouble && f.dim() == 1 && f.is_cuda() && f.get_device() == device &&
                         (f.size(0) <= 1 || f.stride(0) == 1),
                     "inv_freq: expected a contiguous fp64 tensor [rotary_dim / 2] on cuda:", device);
    // in fp32, where 0 would mean 1 to the C ABI
    TORCH_CHECK_VALUE((float)amplitude > 0.f, "amplitude must be positive (in fp32)");
    return {f.data_ptr<double>(), (int32_t)(2 * f.size(0)), interleaved ? 1 : 0, (float)amplitude};
}

void* stream_of(int device) { return c10::cuda::getCurrentCUDAStream(device).stream(); }

// ------------------------------------------------------------------ workspaces

constexpr int64_t kZeroed = 1 << 14;   // more than the status word and the counters
constexpr int64_t kLeast = 1 << 22;

// `size` bytes whose start, all that must have a value before a call, is zero.
at::Tensor fresh_workspace(int device, int64_t size)
{
    at::Tensor ws = at::empty({size}, at::TensorOptions().dtype(at::kByte).device(at::kCUDA, device));
    ws.narrow(0, 0, kZeroed).zero_();
    return ws;
}

// The workspace of the device's current stream, of at least `need` bytes.  A larger one takes
// over its predecessor's status word and replaces it: the allocator reuses the memory in
// the order of the stream, so calls under way keep theirs.  It is twice as large at least,
// so that a batch that grows by and by allocates a few times only.  While a graph is
// captured: one of the graph's own, whose start every replay zeroes.
at::Tensor workspace(int device, int64_t need)
{
    if (c10::cuda::currentStreamCaptureStatusMayInitCtx() != c10::cuda::CaptureStatus::None)
        return fresh_workspace(device, std::max(need, kZeroed));
    // not destroyed at exit: the CUDA context may be gone by then
    static auto* kept = new std::map<std::pair<int, void*>, at::Tensor>();
    at::Tensor& mine = (*kept)[{device, stream_of(device)}];
    if (!mine.defined() || mine.numel() < need) {
        at::Tensor ws = fresh_workspace(device, std::max({need, kLeast, mine.defined() ? 2 * mine.numel() : 0}));
        const int64_t status = (int64_t)calls.workspace_size();
        if (mine.defined()) ws.narrow(0, 0, status).copy_(mine.narrow(0, 0, status));
        mine = ws;
    }
    return mine;
}

at::Tensor workspace_arg(PyObject* o, int device, int64_t need)
{
    if (o == Py_None) return workspace(device, need);
    const at::Tensor& ws = tensor(o, "ws");
    TORCH_CHECK_TYPE(ws.scalar_type() == at::kByte && ws.is_cuda() && ws.get_device() == device && ws.is_contiguous(),
                     "ws must be a contiguous uint8 tensor on cuda:", device);
    return ws;
}

PyObject* none()
{
    Py_RETURN_NONE;
}

PyObject* pair(PyObject* a, PyObject* b)
{
    PyObject* t = PyTuple_New(2);
    if (!t) throw python_error();
    PyTuple_SET_ITEM(t, 0, a);
    PyTuple_SET_ITEM(t, 1, b);
    return t;
}

void want(Py_ssize_t got, Py_ssize_t n)
{
    TORCH_CHECK_TYPE(got == n, "expected ", n, " arguments, got ", got);
}

// ------------------------------------------------------------------ functions

// bind(addresses of Calls' members, in order)
PyObject* py_bind(PyObject*, PyObject* const* a, Py_ssize_t n)
{
    HANDLE_TH_ERRORS
    want(n, 7);
    void** to = reinterpret_cast<void**>(&calls);
    for (int i = 0; i < 7; ++i) to[i] = reinterpret_cast<void*>((uintptr_t)PyLong_AsUnsignedLongLong(a[i]));
    return none();
    END_HANDLE_TH_ERRORS
}

// workspace(device index, need)
PyObject* py_workspace(PyObject*, PyObject* const* a, Py_ssize_t n)
{
    HANDLE_TH_ERRORS
    want(n, 2);
    const int device = (int)integer(a[0]);
    c10::cuda::CUDAGuard guard((c10::DeviceIndex)device);
    return THPVariable_Wrap(workspace(device, integer(a[1])));
    END_HANDLE_TH_ERRORS
}

// rope_apply(q, k, inv_freq, positions, interleaved, amplitude, inverse, offset, q_out, k_out)
PyObject* py_rope_apply(PyObject*, PyObject* const* a, Py_ssize_t n)
{
    HANDLE_TH_ERRORS
    want(n, 10);
    const bool has_k = a[1] != Py_None;
    TORCH_CHECK_VALUE(a[8] == Py_None ? a[9] == Py_None : has_k == (a[9] != Py_None),
                      "rope_apply: out holds an output for each of q and k");
    const at::Tensor& q0 = tensor(a[0], "q");
    const int device = device_of(q0, "rope_apply");
    c10::cuda::CUDAGuard guard((c10::DeviceIndex)device);
    const fa_rope rope = rope_of(tensor(a[2], "inv_freq"), truth(a[4]), number(a[5]), device);
    fa_tensor qd, kd, qo, ko;
    const at::Tensor q = readable(q0);
    qd = describe(q, device, "q");
    const at::Tensor q_out = a[8] != Py_None ? tensor(a[8], "out[0]") : at::empty_like(q);
    qo = describe(q_out, device, "out[0]");
    at::Tensor k, k_out;
    if (has_k) {
        k = readable(tensor(a[1], "k"));
        kd = describe(k, device, "k");
        k_out = a[9] != Py_None ? tensor(a[9], "out[1]") : at::empty_like(k);
        ko = describe(k_out, device, "out[1]");
    }
    const int32_t* pos = nullptr;
    int64_t stride = 0;
    if (a[3] != Py_None) {
        const at::Tensor& p = tensor(a[3], "positions");
        const bool rows = p.dim() != 1;
        pos = ints(p, rows ? 2 : 1, rows ? q.size(0) : q.size(2), q.size(2), device, "positions");
        stride = rows && q.size(0) > 1 ? p.stride(0) : 0;
    }
    const int rc = calls.rope_apply(&qd, has_k ? &kd : nullptr, &rope, pos, stride, integer(a[7]), truth(a[6]) ? 1 : 0, &qo,
                                    has_k ? &ko : nullptr, stream_of(device));
    if (rc) return PyLong_FromLong(rc);
    if (a[8] != Py_None) written(q_out);
    if (a[9] != Py_None) written(k_out);
    return pair(THPVariable_Wrap(q_out), has_k ? THPVariable_Wrap(k_out) : none());
    END_HANDLE_TH_ERRORS
}

// paged_append(k, v, k_pages, v_pages, page_table, cache_lens, new_lens, q, q_out, inv_freq,
//              interleaved, amplitude, ws)
PyObject* py_paged_append(PyObject*, PyObject* const* a, Py_ssize_t n)
{
    HANDLE_TH_ERRORS
    want(n, 13);
    const at::Tensor& k0 = tensor(a[0], "k");
    const int device = device_of(k0, "paged_append");
    c10::cuda::CUDAGuard guard((c10::DeviceIndex)device);
    const at::Tensor k = readable(k0), v = readable(tensor(a[1], "v"));
    const fa_tensor kd = describe(k, device, "k"), vd = describe(v, device, "v");
    const at::Tensor &k_pages = tensor(a[2], "k_pages"), &v_pages = tensor(a[3], "v_pages");
    const fa_tensor kp = describe(k_pages, device, "k_pages"), vp = describe(v_pages, device, "v_pages");
    const int64_t B = k.size(0);
    const at::Tensor& table = tensor(a[4], "page_table");
    const int32_t* pages = ints(table, 2, B, -1, device, "page_table");
    const int32_t* have = ints(tensor(a[5], "cache_lens"), 1, B, 0, device, "cache_lens");
    const int32_t* fresh = a[6] != Py_None ? ints(tensor(a[6], "new_lens"), 1, B, 0, device, "new_lens") : nullptr;
    const bool has_q = a[7] != Py_None, turned = a[9] != Py_None;
    TORCH_CHECK_VALUE(has_q || a[8] == Py_None, "paged_append: q_out without q");
    fa_rope rope{};
    if (turned) rope = rope_of(tensor(a[9], "inv_freq"), truth(a[10]), number(a[11]), device);
    at::Tensor q, q_out;
    fa_tensor qd, qo;
    if (has_q) {
        q = readable(tensor(a[7], "q"));
        qd = describe(q, device, "q");
        q_out = a[8] != Py_None ? tensor(a[8], "q_out") : fresh ? at::zeros_like(q) : at::empty_like(q);
        qo = describe(q_out, device, "q_out");
    }
    const at::Tensor ws = workspace_arg(a[12], device, (int64_t)calls.workspace_size());
    const int rc = calls.paged_append(&kd, &vd, has_q ? &qd : nullptr, turned ? &rope : nullptr, have, fresh, pages,
                                      table.stride(0), table.size(1), &kp, &vp, has_q ? &qo : nullptr, ws.data_ptr(),
                                      (size_t)ws.numel(), stream_of(device));
    if (rc) return PyLong_FromLong(rc);
    written(k_pages);
    written(v_pages);
    if (a[8] != Py_None) written(q_out);
    return has_q ? THPVariable_Wrap(q_out) : none();
    END_HANDLE_TH_ERRORS
}

// decode(shared, q, k_pages, v_pages, page_table, seq_lens, window or prefix_len, score kind,
//        slopes, softcap, scale, out, lse, ws)
PyObject* py_decode(PyObject*, PyObject* const* a, Py_ssize_t n)
{
    HANDLE_TH_ERRORS
    want(n, 14);
    const bool shared = truth(a[0]);
    const at::Tensor& q0 = tensor(a[1], "q");
    const int device = device_of(q0, shared ? "flex_decode_shared" : "flex_decode_paged");
    c10::cuda::CUDAGuard guard((c10::DeviceIndex)device);
    const at::Tensor q = readable(q0);
    const fa_tensor qd = describe(q, device, "q");
    const int64_t B = q.size(0), Hq = q.size(1), len = q.size(2), D = q.size(3), extra = integer(a[6]);
    const fa_tensor kp = describe(tensor(a[2], "k_pages"), device, "k_pages");
    const fa_tensor vp = describe(tensor(a[3], "v_pages"), device, "v_pages");
    const at::Tensor& table = tensor(a[4], "page_table");
    const int32_t* pages = ints(table, 2, B, -1, device, "page_table");
    const int32_t* lens = ints(tensor(a[5], "seq_lens"), 1, B, 0, device, "seq_lens");
    fa_score_mod sm{};
    sm.kind = (int)integer(a[7]);
    sm.softcap = (float)number(a[9]);
    if (a[8] != Py_None) {
        const at::Tensor& slopes = tensor(a[8], "ALiBi slopes");
        TORCH_CHECK_TYPE(slopes.scalar_type() == at::kFloat && slopes.is_cuda() && slopes.get_device() == device &&
                             slopes.dim() == 1 && slopes.size(0) == Hq && slopes.is_contiguous(),
                         "ALiBi slopes: contiguous fp32 [Hq] on cuda:", device);
        sm.alibi_slopes = slopes.data_ptr<float>();
    }
    const at::Tensor out = a[11] != Py_None ? tensor(a[11], "out") : at::empty({B, Hq, len, D}, q.options());
    const fa_tensor od = describe(out, device, "out");
    at::Tensor lse;
    if (a[12] != Py_None) {
        lse = tensor(a[12], "lse");
        TORCH_CHECK_TYPE(lse.scalar_type() == at::kFloat && lse.is_cuda() && lse.get_device() == device && lse.dim() == 3 &&
                             lse.size(0) == B && lse.size(1) == Hq && lse.size(2) == len && lse.is_contiguous(),
                         "lse: expected a contiguous fp32 tensor [B, Hq, q_len] on cuda:", device);
    } else {
        lse = at::empty({B, Hq, len}, q.options().dtype(at::kFloat));
    }
    const int64_t Hkv = kp.dims[1];
    const size_t need = shared ? calls.decode_shared_size(B, Hq, Hkv, len, D, extra)
                               : calls.decode_paged_size(B, Hq, Hkv, len, D);
    const at::Tensor ws = workspace_arg(a[13], device, (int64_t)need);
    const int rc = (shared ? calls.decode_shared : calls.decode_paged)(
        &qd, &kp, &vp, pages, table.stride(0), table.size(1), lens, extra, &sm, (float)number(a[10]), &od,
        lse.data_ptr<float>(), ws.data_ptr(), (size_t)ws.numel(), stream_of(device));
    if (rc) return PyLong_FromLong(rc);
    if (a[11] != Py_None) written(out);
    if (a[12] != Py_None) written(lse);
    return pair(THPVariable_Wrap(out), THPVariable_Wrap(lse));
    END_HANDLE_TH_ERRORS
}

template <PyObject* (*F)(PyObject*, PyObject* const*, Py_ssize_t)>
PyMethodDef method(const char* name)
{
    return {name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(F)), METH_FASTCALL, nullptr};
}

PyMethodDef methods[] = {method<py_bind>("bind"),
                         method<py_workspace>("workspace"),
                         method<py_rope_apply>("rope_apply"),
                         method<py_paged_append>("paged_append"),
                         method<py_decode>("decode"),
                         {nullptr, nullptr, 0, nullptr}};

PyModuleDef module = {PyModuleDef_HEAD_INIT, "_binding", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

} // namespace

PyMODINIT_FUNC PyInit__binding()
{
    PyObject* m = PyModule_Create(&module);
    if (m && PyModule_AddStringConstant(m, "torch_version", FA_TORCH_VERSION) < 0) {
        Py_DECREF(m);
        return nullptr;
    }
    return m;
}
