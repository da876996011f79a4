// Native torch binding of the operators around the GEMM: a CPython module that
// checks tensors, allocates outputs and workspaces and calls the C ABI of
// libhq.so on the current stream of the tensors' device.
//
// Small calls are bound by the host. The same marshalling through ctypes took
// 14.2 us for the norm of one token (four torch.empty 6.7, the current stream
// 1.9, the call and its launch 3.5, attribute checks 2.1); a launch by itself
// takes 2.7 us.
//
// Arguments are positional and complete (api.py has the keywords and defaults);
// None stands for a tensor that is not given. Refusals raise ValueError, and
// errors of the library go through _lib.check.
//
// Each function reads its Python arguments first and then gives up the interpreter
// lock for the checks, copies, allocations and the call: a copy, an allocation or a
// launch that waits for the device (a full queue, say) stops no other Python thread.
#include <ATen/core/Tensor.h>
#include <ATen/hip/EmptyTensor.h>
#include <c10/core/DeviceGuard.h>
#include <c10/hip/HIPStream.h>
#include <torch/csrc/Device.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>
#include <torch/csrc/utils/object_ptr.h>

#include "hq.h"

namespace {

using at::ScalarType;
using at::Tensor;

PyObject* g_check = nullptr;           // _lib.check
PyObject* g_gemm_workspace = nullptr;  // api.gemm_workspace

Tensor tensor(PyObject* o, const char* name) {
  TORCH_CHECK_VALUE(THPVariable_Check(o), name, " must be a tensor");
  return THPVariable_Unpack(o);
}
Tensor maybe(PyObject* o, const char* name) { return o == Py_None ? Tensor() : tensor(o, name); }
int64_t integer(PyObject* o) {
  const long long v = PyLong_AsLongLong(o);
  if (v == -1 && PyErr_Occurred()) throw python_error();
  return v;
}
// One of the ABI's enumerations: a number that would not survive the cast to int is
// refused here, the others' range by the library.
int choice(PyObject* o, const char* name) {
  const int64_t v = integer(o);
  TORCH_CHECK_VALUE(v == (int64_t)(int)v, name, " must fit in 32 bits, got ", v);
  return (int)v;
}
double real(PyObject* o) {
  const double v = PyFloat_AsDouble(o);
  if (v == -1.0 && PyErr_Occurred()) throw python_error();
  return v;
}

// The element type of a [rows, cols] tensor as an hq_dtype.
int real_type(const Tensor& t, const char* name) {
  TORCH_CHECK_VALUE(t.scalar_type() == ScalarType::Float || t.scalar_type() == ScalarType::BFloat16, name,
                    " must be float32 or bfloat16, got ", t.scalar_type());
  TORCH_CHECK_VALUE(t.dim() == 2, name, " must be 2-D [rows, cols]");
  return t.scalar_type() == ScalarType::Float ? HQ_F32 : HQ_BF16;
}

// A given input, contiguous, of this type and shape and on this device; undefined
// stays undefined.
Tensor input(Tensor t, at::IntArrayRef shape, ScalarType dt, const Tensor& like, const char* name) {
  if (!t.defined()) return t;
  TORCH_CHECK_VALUE(t.scalar_type() == dt && t.sizes() == shape, name, " must be ", dt, " ", shape, ", got ",
                    t.scalar_type(), " ", t.sizes());
  TORCH_CHECK_VALUE(t.device() == like.device(), name, " must be on ", like.device(), ", got ", t.device());
  return t.contiguous();
}

// A new tensor on `like`'s GPU, from the caching allocator (torch.empty without
// its dispatch).
Tensor fresh(at::IntArrayRef shape, ScalarType dt, const Tensor& like, const char* name) {
  TORCH_CHECK_VALUE(like.is_cuda(), "tensors must be on the GPU, got ", like.device(), " for ", name);
  return at::detail::empty_cuda(shape, dt, like.device(), std::nullopt);
}

// The caller's output buffer, checked, or a new one.
Tensor output(Tensor t, at::IntArrayRef shape, ScalarType dt, const Tensor& like, const char* name) {
  if (!t.defined()) return fresh(shape, dt, like, name);
  TORCH_CHECK_VALUE(t.scalar_type() == dt && t.sizes() == shape && t.is_contiguous() && t.device() == like.device(), name,
                    " must be contiguous ", dt, " ", shape, " on ", like.device(), ", got ", t.scalar_type(), " ", t.sizes(),
                    " on ", t.device());
  return t;
}

void on_gpu(const Tensor& t, const char* name) {
  TORCH_CHECK_VALUE(t.is_cuda(), name, " must be on the GPU, got ", t.device());
}

void* ptr(const Tensor& t) { return t.defined() ? t.data_ptr() : nullptr; }
template <class T>
T* ptr(const Tensor& t) {
  return static_cast<T*>(ptr(t));
}

hipStream_t stream_of(const Tensor& t) { return c10::hip::getCurrentHIPStream(t.device().index()).stream(); }

// The caller's workspace, checked like an output's buffer: its bytes go to the kernels.
void check_workspace(const Tensor& t, const Tensor& like) {
  if (!t.defined()) return;
  TORCH_CHECK_VALUE(t.device() == like.device(), "workspace must be on ", like.device(), ", got ", t.device());
  TORCH_CHECK_VALUE(t.is_contiguous(), "workspace must be contiguous");
}

// Scratch without an initial value, from the caching allocator: its reuse is
// ordered on the current stream, and under graph capture it belongs to the graph.
Tensor scratch(const Tensor& given, bool allocate, size_t bytes, const Tensor& like) {
  if (given.defined() || !allocate || bytes == 0) return given;
  return fresh({(int64_t)bytes}, ScalarType::Byte, like, "workspace");
}
size_t bytes_of(const Tensor& t) { return t.defined() ? t.nbytes() : 0; }

void raise_unless_ok(hq_status st) {
  if (st == HQ_OK) return;
  PyObject* r = PyObject_CallFunction(g_check, "i", (int)st);
  Py_XDECREF(r);
  throw python_error();
}

int64_t blocks(int64_t cols, int64_t bs) {
  TORCH_CHECK_VALUE(bs == 32 || bs == 64 || bs == 128, "the checkpoint's block_size must be 32, 64 or 128, got ", bs);
  return (cols + bs - 1) / bs;
}

// A checkpoint of [rows, cols]: its tensors and the ABI's struct. Block size 0: none.
struct Ckpt {
  Tensor q, scales;
  hq_checkpoint c{};
  const hq_checkpoint* p() const { return c.block_size ? &c : nullptr; }
};
Ckpt checkpoint_in(const Tensor& q, const Tensor& s, int64_t bs, int64_t rows, int64_t cols, const Tensor& like) {
  Ckpt k;
  if (bs == 0) return k;
  const int64_t nb = blocks(cols, bs);
  TORCH_CHECK_VALUE(q.defined() && s.defined(), "a checkpoint's q and scales must be tensors");
  k.q = input(q, {rows, cols}, ScalarType::Byte, like, "checkpoint.q");
  k.scales = input(s, {rows, nb}, ScalarType::Float, like, "checkpoint.scales");
  k.c = {ptr<uint8_t>(k.q), ptr<float>(k.scales), (int32_t)bs};
  return k;
}
Ckpt checkpoint_out(const Tensor& q, const Tensor& s, int64_t bs, int64_t rows, int64_t cols, const Tensor& like) {
  Ckpt k;
  if (bs == 0) return k;
  const int64_t nb = blocks(cols, bs);
  k.q = output(q, {rows, cols}, ScalarType::Byte, like, "checkpoint.q");
  k.scales = output(s, {rows, nb}, ScalarType::Float, like, "checkpoint.scales");
  k.c = {ptr<uint8_t>(k.q), ptr<float>(k.scales), (int32_t)bs};
  return k;
}

PyObject* wrap(const Tensor& t) {
  if (!t.defined()) Py_RETURN_NONE;
  return THPVariable_Wrap(t);
}
template <class... Ts>
PyObject* wrap_all(const Ts&... ts) {
  PyObject* r = PyTuple_New(sizeof...(ts));
  if (!r) throw python_error();
  Py_ssize_t i = 0;
  (PyTuple_SET_ITEM(r, i++, wrap(ts)), ...);
  return r;
}

// Without the interpreter lock while it lives (exceptions take it back on their way).
class NoGil {
 public:
  NoGil() : state_(PyEval_SaveThread()) {}
  ~NoGil() { PyEval_RestoreThread(state_); }
  NoGil(const NoGil&) = delete;

 private:
  PyThreadState* state_;
};

void want(Py_ssize_t got, Py_ssize_t n) { TORCH_CHECK_VALUE(got == n, "expected ", n, " arguments, got ", got); }

// x, weight, eps, fmt, residual, h, write_h, ckpt q, ckpt scales, block_size, q, scale, rstd
//   -> q, scale, h, rstd, ckpt q, ckpt scales
PyObject* rmsnorm_quantize(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  want(n, 13);
  const Tensor x0 = tensor(a[0], "x"), w0 = maybe(a[1], "weight"), res0 = maybe(a[4], "residual");
  const float eps = (float)real(a[2]);
  const int fmt = choice(a[3], "fmt");
  const bool write_h = a[6] == Py_True;
  const int64_t block = integer(a[9]);
  const Tensor cq = maybe(a[7], "checkpoint.q"), cs = maybe(a[8], "checkpoint.scales");
  Tensor h = maybe(a[5], "h"), q = maybe(a[10], "q"), s = maybe(a[11], "scale_out"), r = maybe(a[12], "rstd_out");
  Ckpt k;
  hq_status st;
  {
    const NoGil nogil;
    const int xt = real_type(x0, "x");
    const Tensor x = x0.contiguous();
    const ScalarType dt = x.scalar_type();
    const int64_t rows = x.size(0), cols = x.size(1);
    const Tensor w = input(w0, {cols}, dt, x, "weight");
    const Tensor res = input(res0, {rows, cols}, dt, x, "residual");
    const c10::OptionalDeviceGuard guard(x.device());
    h = write_h ? output(h, {rows, cols}, dt, x, "h") : Tensor();
    k = checkpoint_out(cq, cs, block, rows, cols, x);
    q = output(q, {rows, cols}, ScalarType::Byte, x, "q");
    s = output(s, {rows}, ScalarType::Float, x, "scale_out");
    r = output(r, {rows}, ScalarType::Float, x, "rstd_out");
    on_gpu(x, "x");
    st = hq_rmsnorm_quantize_fp8(ptr(x), ptr(res), ptr(w), xt, rows, cols, eps, fmt, ptr<uint8_t>(q), ptr<float>(s), ptr(h),
                                 ptr<float>(r), k.p(), stream_of(x));
  }
  raise_unless_ok(st);
  return wrap_all(q, s, h, r, k.q, k.scales);
  END_HANDLE_TH_ERRORS
}

// dy, h, ckpt q, ckpt scales, block_size, weight, rstd, dresidual, dx, dweight, want_dweight, workspace
//   -> dx, dweight
PyObject* rmsnorm_backward(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  want(n, 12);
  const Tensor dy0 = tensor(a[0], "dy"), h0 = maybe(a[1], "h"), w0 = maybe(a[5], "weight"), rstd0 = tensor(a[6], "rstd");
  const Tensor dr0 = maybe(a[7], "dresidual"), given = maybe(a[11], "workspace");
  const int64_t block = integer(a[4]);
  const Tensor cq = maybe(a[2], "checkpoint.q"), cs = maybe(a[3], "checkpoint.scales");
  const bool sum = a[10] == Py_True;
  Tensor dx = maybe(a[8], "dx"), dw = maybe(a[9], "dweight");
  hq_status st;
  {
    const NoGil nogil;
    const int xt = real_type(dy0, "dy");
    const Tensor dy = dy0.contiguous();
    const ScalarType dt = dy.scalar_type();
    const int64_t rows = dy.size(0), cols = dy.size(1);
    const Tensor h = input(h0, {rows, cols}, dt, dy, "h");
    const Ckpt k = checkpoint_in(cq, cs, block, rows, cols, dy);
    const Tensor w = input(w0, {cols}, dt, dy, "weight");
    const Tensor rstd = input(rstd0, {rows}, ScalarType::Float, dy, "rstd");
    const Tensor dr = input(dr0, {rows, cols}, dt, dy, "dresidual");
    check_workspace(given, dy);
    const c10::OptionalDeviceGuard guard(dy.device());
    dx = output(dx, {rows, cols}, dt, dy, "dx");
    dw = sum ? output(dw, {cols}, ScalarType::Float, dy, "dweight") : Tensor();
    on_gpu(dy, "dy");
    const Tensor ws = scratch(given, sum, hq_rmsnorm_backward_workspace_bytes(xt, rows, cols), dy);
    st = hq_rmsnorm_backward(ptr(dy), ptr(h), k.p(), ptr(w), ptr<float>(rstd), ptr(dr), xt, rows, cols, ptr(dx), ptr<float>(dw),
                             ptr(ws), bytes_of(ws), stream_of(dy));
  }
  raise_unless_ok(st);
  return wrap_all(dx, dw);
  END_HANDLE_TH_ERRORS
}

// x, weight, bias, eps, fmt, residual, h, write_h, ckpt q, ckpt scales, block_size, q, scale, mean, rstd
//   -> q, scale, h, mean, rstd, ckpt q, ckpt scales
PyObject* layernorm_quantize(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  want(n, 15);
  const Tensor x0 = tensor(a[0], "x"), w0 = maybe(a[1], "weight"), b0 = maybe(a[2], "bias"), res0 = maybe(a[5], "residual");
  const float eps = (float)real(a[3]);
  const int fmt = choice(a[4], "fmt");
  const bool write_h = a[7] == Py_True;
  const int64_t block = integer(a[10]);
  const Tensor cq = maybe(a[8], "checkpoint.q"), cs = maybe(a[9], "checkpoint.scales");
  Tensor h = maybe(a[6], "h"), q = maybe(a[11], "q"), s = maybe(a[12], "scale_out"), m = maybe(a[13], "mean_out");
  Tensor r = maybe(a[14], "rstd_out");
  Ckpt k;
  hq_status st;
  {
    const NoGil nogil;
    const int xt = real_type(x0, "x");
    const Tensor x = x0.contiguous();
    const ScalarType dt = x.scalar_type();
    const int64_t rows = x.size(0), cols = x.size(1);
    const Tensor w = input(w0, {cols}, dt, x, "weight");
    const Tensor b = input(b0, {cols}, dt, x, "bias");
    const Tensor res = input(res0, {rows, cols}, dt, x, "residual");
    const c10::OptionalDeviceGuard guard(x.device());
    h = write_h ? output(h, {rows, cols}, dt, x, "h") : Tensor();
    k = checkpoint_out(cq, cs, block, rows, cols, x);
    q = output(q, {rows, cols}, ScalarType::Byte, x, "q");
    s = output(s, {rows}, ScalarType::Float, x, "scale_out");
    m = output(m, {rows}, ScalarType::Float, x, "mean_out");
    r = output(r, {rows}, ScalarType::Float, x, "rstd_out");
    on_gpu(x, "x");
    st = hq_layernorm_quantize_fp8(ptr(x), ptr(res), ptr(w), ptr(b), xt, rows, cols, eps, fmt, ptr<uint8_t>(q), ptr<float>(s),
                                   ptr(h), ptr<float>(m), ptr<float>(r), k.p(), stream_of(x));
  }
  raise_unless_ok(st);
  return wrap_all(q, s, h, m, r, k.q, k.scales);
  END_HANDLE_TH_ERRORS
}

// dy, h, ckpt q, ckpt scales, block_size, weight, mean, rstd, dresidual, dx, dweight, want_dweight, dbias, want_dbias,
// workspace -> dx, dweight, dbias
PyObject* layernorm_backward(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  want(n, 15);
  const Tensor dy0 = tensor(a[0], "dy"), h0 = maybe(a[1], "h"), w0 = maybe(a[5], "weight"), mean0 = tensor(a[6], "mean");
  const Tensor rstd0 = tensor(a[7], "rstd"), dr0 = maybe(a[8], "dresidual"), given = maybe(a[14], "workspace");
  const int64_t block = integer(a[4]);
  const Tensor cq = maybe(a[2], "checkpoint.q"), cs = maybe(a[3], "checkpoint.scales");
  const bool want_w = a[11] == Py_True, want_b = a[13] == Py_True;
  Tensor dx = maybe(a[9], "dx"), dw = maybe(a[10], "dweight"), db = maybe(a[12], "dbias");
  hq_status st;
  {
    const NoGil nogil;
    const int xt = real_type(dy0, "dy");
    const Tensor dy = dy0.contiguous();
    const ScalarType dt = dy.scalar_type();
    const int64_t rows = dy.size(0), cols = dy.size(1);
    const Tensor h = input(h0, {rows, cols}, dt, dy, "h");
    const Ckpt k = checkpoint_in(cq, cs, block, rows, cols, dy);
    const Tensor w = input(w0, {cols}, dt, dy, "weight");
    const Tensor mean = input(mean0, {rows}, ScalarType::Float, dy, "mean");
    const Tensor rstd = input(rstd0, {rows}, ScalarType::Float, dy, "rstd");
    const Tensor dr = input(dr0, {rows, cols}, dt, dy, "dresidual");
    check_workspace(given, dy);
    const c10::OptionalDeviceGuard guard(dy.device());
    dx = output(dx, {rows, cols}, dt, dy, "dx");
    dw = want_w ? output(dw, {cols}, ScalarType::Float, dy, "dweight") : Tensor();
    db = want_b ? output(db, {cols}, ScalarType::Float, dy, "dbias") : Tensor();
    on_gpu(dy, "dy");
    const Tensor ws = scratch(given, want_w || want_b, hq_layernorm_backward_workspace_bytes(xt, rows, cols), dy);
    st = hq_layernorm_backward(ptr(dy), ptr(h), k.p(), ptr(w), ptr<float>(mean), ptr<float>(rstd), ptr(dr), xt, rows, cols,
                               ptr(dx), ptr<float>(dw), ptr<float>(db), ptr(ws), bytes_of(ws), stream_of(dy));
  }
  raise_unless_ok(st);
  return wrap_all(dx, dw, db);
  END_HANDLE_TH_ERRORS
}

// xq, xf, wq_pre, wf, x_scale, w_scale, n, bias, bias_type, bias_scale, act, residual, out_scale, out_fmt, out,
// workspace (None: the shared one, False: none) -> out
PyObject* gemm_fused(PyObject*, PyObject* const* a, Py_ssize_t nargs) {
  HANDLE_TH_ERRORS
  want(nargs, 16);
  const Tensor xq0 = tensor(a[0], "xq"), wp = tensor(a[2], "wq_pre"), xs0 = tensor(a[4], "x_scale"), ws0 = tensor(a[5], "w_scale");
  const int xf = choice(a[1], "xf"), wf = choice(a[3], "wf"), act = choice(a[10], "act"), out_fmt = choice(a[13], "out_fmt");
  const int64_t n = integer(a[6]);
  const int bias_type = choice(a[8], "bias_type");
  const Tensor bias0 = maybe(a[7], "bias"), bs0 = maybe(a[9], "bias_scale"), res0 = maybe(a[11], "residual");
  const Tensor os0 = maybe(a[12], "out_scale");
  const bool shared = a[15] == Py_None;
  Tensor work = a[15] == Py_False ? Tensor() : maybe(a[15], "workspace");
  Tensor out = maybe(a[14], "out"), xq, xs, ws, bias, bs, res, os;
  int64_t m, k, need = 0;
  {
    const NoGil nogil;
    TORCH_CHECK_VALUE(xq0.dim() == 2 && xq0.scalar_type() == ScalarType::Byte, "xq must be uint8 codes [m, k]");
    xq = xq0.contiguous();
    m = xq.size(0);
    k = xq.size(1);
    TORCH_CHECK_VALUE(wp.scalar_type() == ScalarType::Byte && wp.is_contiguous() && wp.numel() >= hq_preshuffled_bytes(n, k),
                      "wq_pre must hold the pre-shuffled codes of a [", n, ", ", k, "] weight");
    TORCH_CHECK_VALUE(wp.device() == xq.device(), "wq_pre must be on ", xq.device(), ", got ", wp.device());
    xs = input(xs0, xs0.sizes(), ScalarType::Float, xq, "x_scale");
    ws = input(ws0, ws0.sizes(), ScalarType::Float, xq, "w_scale");
    if (bias0.defined()) {
      TORCH_CHECK_VALUE(bias0.numel() == n &&
                            bias0.scalar_type() == (bias_type == HQ_BIAS_BF16 ? ScalarType::BFloat16 : ScalarType::Byte),
                        "bias must have n elements, bf16 or (as bias_type says) uint8 FP8 codes");
      bias = input(bias0, bias0.sizes(), bias0.scalar_type(), xq, "bias");
    }
    bs = input(bs0, {1}, ScalarType::Float, xq, "bias_scale");
    res = input(res0, {m, n}, ScalarType::BFloat16, xq, "residual");
    os = input(os0, {1}, ScalarType::Float, xq, "out_scale");
    check_workspace(work, xq);
    const c10::OptionalDeviceGuard guard(xq.device());
    out = output(out, {m, n}, os.defined() ? ScalarType::Byte : ScalarType::BFloat16, xq, "out");
    on_gpu(xq, "xq");
    if (shared && m <= 16) need = hq_gemm_workspace_bytes(m, n, k);  // more rows use none
  }
  const c10::OptionalDeviceGuard guard(xq.device());
  if (need > 0) {
    THPObjectPtr dev(THPDevice_New(xq.device()));
    THPObjectPtr r(PyObject_CallFunction(g_gemm_workspace, "OL", dev.get(), (long long)need));
    if (!r) throw python_error();
    work = tensor(r.get(), "workspace");
  }
  hq_status st;
  {
    const NoGil nogil;
    const hq_fused_epilogue ep = {ptr(bias), bias_type, ptr<float>(bs), ptr<float>(os), out_fmt, act, ptr<uint16_t>(res)};
    st = hq_gemm_a8w8_fused(ptr<uint8_t>(xq), xf, ptr<uint8_t>(wp), wf, ptr<float>(xs), xs.numel(), ptr<float>(ws), ws.numel(), m,
                            n, k, &ep, ptr(out), ptr(work), bytes_of(work), stream_of(xq));
  }
  raise_unless_ok(st);
  return wrap(out);
  END_HANDLE_TH_ERRORS
}

// z, act, fmt, gated, ckpt q, ckpt scales, block_size, q, scale -> q, scale, ckpt q, ckpt scales
PyObject* act_quantize(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  want(n, 9);
  const Tensor z0 = tensor(a[0], "z");
  const int act = choice(a[1], "act"), fmt = choice(a[2], "fmt");
  const bool gated = a[3] == Py_True;
  const int64_t block = integer(a[6]);
  const Tensor cq = maybe(a[4], "checkpoint.q"), cs = maybe(a[5], "checkpoint.scales");
  Tensor q = maybe(a[7], "q"), s = maybe(a[8], "scale_out");
  Ckpt k;
  hq_status st;
  {
    const NoGil nogil;
    const int xt = real_type(z0, "z");
    const Tensor z = z0.contiguous();
    const int64_t rows = z.size(0), wide = z.size(1);
    TORCH_CHECK_VALUE(!gated || wide % 2 == 0, "a gated z has an even number of columns");
    const int64_t cols = gated ? wide / 2 : wide;
    const c10::OptionalDeviceGuard guard(z.device());
    k = checkpoint_out(cq, cs, block, rows, wide, z);
    q = output(q, {rows, cols}, ScalarType::Byte, z, "q");
    s = output(s, {rows}, ScalarType::Float, z, "scale_out");
    on_gpu(z, "z");
    st = hq_act_quantize_fp8(ptr(z), xt, rows, cols, act, gated, fmt, ptr<uint8_t>(q), ptr<float>(s), k.p(), stream_of(z));
  }
  raise_unless_ok(st);
  return wrap_all(q, s, k.q, k.scales);
  END_HANDLE_TH_ERRORS
}

// da, ckpt q, ckpt scales, block_size, act, gated, dz, dbias, want_dbias, workspace -> dz, dbias
PyObject* act_backward(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  want(n, 10);
  const Tensor da0 = tensor(a[0], "da"), given = maybe(a[9], "workspace");
  const int64_t block = integer(a[3]);
  TORCH_CHECK_VALUE(block != 0, "z must be a checkpoint");
  const Tensor cq = maybe(a[1], "checkpoint.q"), cs = maybe(a[2], "checkpoint.scales");
  const int act = choice(a[4], "act");
  const bool gated = a[5] == Py_True, sum = a[8] == Py_True;
  Tensor dz = maybe(a[6], "dz"), db = maybe(a[7], "dbias");
  hq_status st;
  {
    const NoGil nogil;
    const int xt = real_type(da0, "da");
    const Tensor da = da0.contiguous();
    const int64_t rows = da.size(0), cols = da.size(1), wide = gated ? 2 * cols : cols;
    const Ckpt k = checkpoint_in(cq, cs, block, rows, wide, da);
    check_workspace(given, da);
    const c10::OptionalDeviceGuard guard(da.device());
    dz = output(dz, {rows, wide}, da.scalar_type(), da, "dz");
    db = sum ? output(db, {wide}, ScalarType::Float, da, "dbias") : Tensor();
    on_gpu(da, "da");
    const Tensor ws = scratch(given, sum, hq_act_backward_workspace_bytes(xt, rows, cols, gated), da);
    st = hq_act_backward(ptr(da), k.p(), xt, rows, cols, act, gated, ptr(dz), ptr<float>(db), ptr(ws), bytes_of(ws),
                         stream_of(da));
  }
  raise_unless_ok(st);
  return wrap_all(dz, db);
  END_HANDLE_TH_ERRORS
}

// g, xq, xf, x_scale, dwt, base, dw, workspace (None: allocate, False: none), strict -> dw
PyObject* wgrad(PyObject*, PyObject* const* a, Py_ssize_t nargs) {
  HANDLE_TH_ERRORS
  want(nargs, 9);
  const Tensor g0 = tensor(a[0], "g"), xq0 = tensor(a[1], "xq"), xs0 = tensor(a[3], "x_scale"), base0 = maybe(a[5], "base");
  const int xf = choice(a[2], "xf"), dwt = choice(a[4], "dwt");
  const bool allocate = a[7] == Py_None, strict = a[8] == Py_True;
  const Tensor given = a[7] == Py_False ? Tensor() : maybe(a[7], "workspace");
  Tensor dw = maybe(a[6], "dw");
  hq_status st;
  {
    const NoGil nogil;
    TORCH_CHECK_VALUE(g0.dim() == 2 && g0.scalar_type() == ScalarType::BFloat16, "g must be a 2-D bfloat16 tensor [m, n]");
    const Tensor g = g0.contiguous();
    const int64_t m = g.size(0), n = g.size(1);
    TORCH_CHECK_VALUE(xq0.dim() == 2 && xq0.size(0) == m, "xq must be uint8 codes [m, k]");
    const Tensor xq = input(xq0, xq0.sizes(), ScalarType::Byte, g, "xq");
    const Tensor xs = input(xs0, xs0.sizes(), ScalarType::Float, g, "x_scale");
    const int64_t k = xq.size(1);
    const Tensor base = input(base0, {n, k}, ScalarType::Float, g, "base");
    check_workspace(given, g);
    const c10::OptionalDeviceGuard guard(g.device());
    dw = output(dw, {n, k}, dwt == HQ_F32 ? ScalarType::Float : ScalarType::BFloat16, g, "dw");
    on_gpu(g, "g");
    const int64_t need = allocate ? hq_wgrad_workspace_bytes(m, n, k, strict ? (int)HQ_F32 : dwt) : 0;
    const Tensor ws = scratch(given, allocate, need > 0 ? (size_t)need : 0, g);
    st = (strict ? hq_wgrad_a8_strict : hq_wgrad_a8)(ptr<uint16_t>(g), ptr<uint8_t>(xq), xf, ptr<float>(xs), xs.numel(), m, n, k,
                                                     ptr<float>(base), ptr(dw), dwt, ptr(ws), bytes_of(ws), stream_of(g));
  }
  raise_unless_ok(st);
  return wrap(dw);
  END_HANDLE_TH_ERRORS
}

// Router logits: [tokens, experts].
Tensor logits_of(const Tensor& t, int* xt) {
  *xt = real_type(t, "logits");
  return t.contiguous();
}

// logits, topk, score, renormalize, ids, weights -> ids, weights
PyObject* moe_route(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  want(n, 6);
  const Tensor l0 = tensor(a[0], "logits");
  const int64_t topk = integer(a[1]);
  const int score = choice(a[2], "score");
  const bool renorm = a[3] == Py_True;
  Tensor ids = maybe(a[4], "ids"), w = maybe(a[5], "weights");
  hq_status st;
  {
    const NoGil nogil;
    int xt;
    const Tensor l = logits_of(l0, &xt);
    const int64_t tokens = l.size(0), experts = l.size(1);
    TORCH_CHECK_VALUE(topk >= 1 && topk <= 16, "topk must be in [1, 16], got ", topk);
    const c10::OptionalDeviceGuard guard(l.device());
    ids = output(ids, {tokens, topk}, ScalarType::Int, l, "ids");
    w = output(w, {tokens, topk}, ScalarType::Float, l, "weights");
    on_gpu(l, "logits");
    st = hq_moe_route(ptr(l), xt, tokens, experts, (int)topk, score, renorm, ptr<int32_t>(ids), ptr<float>(w), stream_of(l));
  }
  raise_unless_ok(st);
  return wrap_all(ids, w);
  END_HANDLE_TH_ERRORS
}

// logits, ids, dweights, score, renormalize, dlogits -> dlogits
PyObject* moe_route_backward(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  want(n, 6);
  const Tensor l0 = tensor(a[0], "logits"), ids0 = tensor(a[1], "ids"), dw0 = tensor(a[2], "dweights");
  const int score = choice(a[3], "score");
  const bool renorm = a[4] == Py_True;
  Tensor dl = maybe(a[5], "dlogits");
  hq_status st;
  {
    const NoGil nogil;
    int xt;
    const Tensor l = logits_of(l0, &xt);
    const int64_t tokens = l.size(0), experts = l.size(1);
    TORCH_CHECK_VALUE(ids0.dim() == 2, "ids must be 2-D [tokens, topk]");
    const int64_t topk = ids0.size(1);
    TORCH_CHECK_VALUE(topk >= 1 && topk <= 16, "topk must be in [1, 16], got ", topk);
    const Tensor ids = input(ids0, {tokens, topk}, ScalarType::Int, l, "ids");
    const Tensor dw = input(dw0, {tokens, topk}, ScalarType::Float, l, "dweights");
    const c10::OptionalDeviceGuard guard(l.device());
    dl = output(dl, {tokens, experts}, l.scalar_type(), l, "dlogits");
    on_gpu(l, "logits");
    st = hq_moe_route_backward(ptr(l), ptr<int32_t>(ids), ptr<float>(dw), xt, tokens, experts, (int)topk, score, renorm, ptr(dl),
                               stream_of(l));
  }
  raise_unless_ok(st);
  return wrap(dl);
  END_HANDLE_TH_ERRORS
}

// The codes of an expert layer's weights, and a scale per expert [E] or per expert and row [E, rows].
void check_expert_weight(const Tensor& codes, int64_t experts, int64_t rows, int64_t k, const Tensor& like, const char* name) {
  TORCH_CHECK_VALUE(codes.scalar_type() == ScalarType::Byte && codes.is_contiguous() &&
                        codes.numel() >= experts * hq_preshuffled_bytes(rows, k),
                    name, " must hold the pre-shuffled codes of ", experts, " weights [", rows, ", ", k, "]");
  TORCH_CHECK_VALUE(codes.device() == like.device(), name, " must be on ", like.device(), ", got ", codes.device());
}
Tensor expert_scale(const Tensor& t, int64_t experts, int64_t rows, const Tensor& like, const char* name) {
  if (t.dim() == 1) return input(t, {experts}, ScalarType::Float, like, name);
  return input(t, {experts, rows}, ScalarType::Float, like, name);
}

// xq, xf, x_scale, ids, weights, w1_pre, w1_scale, w2_pre, w2_scale, wf, inner, act, gated, bias1, bias2, residual, out,
// workspace (None: the shared one) -> out
PyObject* moe(PyObject*, PyObject* const* a, Py_ssize_t nargs) {
  HANDLE_TH_ERRORS
  want(nargs, 18);
  const Tensor xq0 = tensor(a[0], "xq"), xs0 = tensor(a[2], "x_scale"), ids0 = tensor(a[3], "ids"), wt0 = tensor(a[4], "weights");
  const Tensor w1 = tensor(a[5], "w1_pre"), s10 = tensor(a[6], "w1_scale"), w2 = tensor(a[7], "w2_pre"), s20 = tensor(a[8], "w2_scale");
  const int xf = choice(a[1], "xf"), wf = choice(a[9], "wf"), act = choice(a[11], "act");
  const int64_t inner = integer(a[10]);
  const bool gated = a[12] == Py_True;
  const Tensor b10 = maybe(a[13], "bias1"), b20 = maybe(a[14], "bias2"), res0 = maybe(a[15], "residual");
  Tensor out = maybe(a[16], "out"), work = maybe(a[17], "workspace"), xq, xs, ids, wt, s1, s2, b1, b2, res;
  int64_t tokens, hidden, topk, experts, need;
  {
    const NoGil nogil;
    TORCH_CHECK_VALUE(xq0.dim() == 2 && xq0.scalar_type() == ScalarType::Byte, "xq must be uint8 codes [tokens, hidden]");
    TORCH_CHECK_VALUE(ids0.dim() == 2, "ids must be 2-D [tokens, topk]");
    TORCH_CHECK_VALUE(s10.dim() == 1 || s10.dim() == 2, "w1_scale must be [experts] or [experts, rows]");
    xq = xq0.contiguous();
    tokens = xq.size(0);
    hidden = xq.size(1);
    topk = ids0.size(1);
    experts = s10.size(0);
    TORCH_CHECK_VALUE(topk >= 1 && topk <= 16, "topk must be in [1, 16], got ", topk);
    need = hq_moe_workspace_bytes(tokens, (int)topk, experts, hidden, inner);
    TORCH_CHECK_VALUE(need >= 0 && (!gated || inner % 32 == 0), "tokens must be at most 64 (", tokens, "), experts in [1, 1024] (",
                      experts, "), hidden and inner multiples of 16 (gated: inner of 32) up to 65536 (", hidden, ", ", inner, ")");
    const int64_t n1 = gated ? 2 * inner : inner;
    ids = input(ids0, {tokens, topk}, ScalarType::Int, xq, "ids");
    wt = input(wt0, {tokens, topk}, ScalarType::Float, xq, "weights");
    xs = input(xs0, xs0.sizes(), ScalarType::Float, xq, "x_scale");
    check_expert_weight(w1, experts, n1, hidden, xq, "w1_pre");
    check_expert_weight(w2, experts, hidden, inner, xq, "w2_pre");
    s1 = expert_scale(s10, experts, n1, xq, "w1_scale");
    s2 = expert_scale(s20, experts, hidden, xq, "w2_scale");
    b1 = input(b10, {experts, n1}, ScalarType::BFloat16, xq, "bias1");
    b2 = input(b20, {experts, hidden}, ScalarType::BFloat16, xq, "bias2");
    res = input(res0, {tokens, hidden}, ScalarType::BFloat16, xq, "residual");
    check_workspace(work, xq);
    const c10::OptionalDeviceGuard guard(xq.device());
    out = output(out, {tokens, hidden}, ScalarType::BFloat16, xq, "out");
    on_gpu(xq, "xq");
  }
  const c10::OptionalDeviceGuard guard(xq.device());
  if (!work.defined() && need > 0) {
    THPObjectPtr dev(THPDevice_New(xq.device()));
    THPObjectPtr r(PyObject_CallFunction(g_gemm_workspace, "OL", dev.get(), (long long)need));
    if (!r) throw python_error();
    work = tensor(r.get(), "workspace");
  }
  hq_status st;
  {
    const NoGil nogil;
    const hq_moe_layer l = {ptr<uint8_t>(w1), ptr<float>(s1), s1.numel(), ptr<uint16_t>(b1), ptr<uint8_t>(w2), ptr<float>(s2),
                            s2.numel(), ptr<uint16_t>(b2), hidden, inner, (int32_t)experts, wf, act, gated};
    st = hq_moe_a8w8(ptr<uint8_t>(xq), xf, ptr<float>(xs), xs.numel(), ptr<int32_t>(ids), ptr<float>(wt), tokens, (int)topk, &l,
                     ptr<uint16_t>(res), ptr<uint16_t>(out), ptr(work), bytes_of(work), stream_of(xq));
  }
  raise_unless_ok(st);
  return wrap(out);
  END_HANDLE_TH_ERRORS
}

// stream handle -> the number of the capture that it is part of, 0 for none
PyObject* capture_id(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  want(n, 1);
  const hipStream_t st = reinterpret_cast<hipStream_t>(integer(a[0]));
  hipStreamCaptureStatus status = hipStreamCaptureStatusNone;
  unsigned long long id = 0;
  const hipError_t e = hipStreamGetCaptureInfo(st, &status, &id);
  if (e != hipSuccess) (void)hipGetLastError();
  TORCH_CHECK(e == hipSuccess, "hipStreamGetCaptureInfo: ", hipGetErrorString(e));
  return PyLong_FromUnsignedLongLong(status == hipStreamCaptureStatusNone ? 0 : id);
  END_HANDLE_TH_ERRORS
}

PyObject* setup(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  want(n, 2);
  Py_INCREF(a[0]);
  Py_INCREF(a[1]);
  g_check = a[0];
  g_gemm_workspace = a[1];
  Py_RETURN_NONE;
  END_HANDLE_TH_ERRORS
}

#define HQ_METHOD(F) {#F, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)(void)>(F)), METH_FASTCALL, nullptr}
PyMethodDef methods[] = {HQ_METHOD(setup),        HQ_METHOD(rmsnorm_quantize), HQ_METHOD(rmsnorm_backward), HQ_METHOD(gemm_fused),
                         HQ_METHOD(layernorm_quantize), HQ_METHOD(layernorm_backward), HQ_METHOD(moe_route),
                         HQ_METHOD(moe_route_backward), HQ_METHOD(moe),
                         HQ_METHOD(act_quantize), HQ_METHOD(act_backward),     HQ_METHOD(wgrad),            HQ_METHOD(capture_id),
                         {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_hqtorch", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__hqtorch(void) { return PyModule_Create(&module); }
