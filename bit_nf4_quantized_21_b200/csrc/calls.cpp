// calls.cpp -- the Python side of the FP8 layer, the layer norm and the
// distillation loss (module _calls): torch tensors in, device pointers to
// libqlora, torch tensors out.
//
// These calls serve single tokens, where the kernels take 3 to 8 us.  The
// same marshalling in Python took 14 us for a layer norm and 18 to 22 us for
// an FP8 product, most of it reading tensor properties one by one and
// allocating outputs through the interpreter.  Nothing is computed here: the
// arguments' shapes, types and devices are checked, outputs that the caller
// did not bring are allocated, and the C entry is called on the current
// stream of the tensors' device.  A function returns its outputs, or the
// library's status as an int where that is not QLORA_OK.
#include <torch/csrc/autograd/python_variable.h>
#include <torch/csrc/Dtype.h>
#include <torch/csrc/Exceptions.h>
#include <ATen/ATen.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <dlfcn.h>

#include "qlora.h"

namespace {

struct Api {
  decltype(&qlora_fp8_quantize) fp8_quantize;
  decltype(&qlora_fp8_linear_fwd) fp8_linear_fwd;
  decltype(&qlora_fp8_linear_bwd) fp8_linear_bwd;
  decltype(&qlora_layernorm_workspace_bytes) layernorm_workspace_bytes;
  decltype(&qlora_layernorm_fwd) layernorm_fwd;
  decltype(&qlora_layernorm_bwd) layernorm_bwd;
  decltype(&qlora_distill_topk_fwd) distill_topk_fwd;
  decltype(&qlora_distill_topk_bwd) distill_topk_bwd;
} api{};

typedef const at::Tensor* Opt;   // null where Python passed None

Opt tensor_or_none(PyObject* o, const char* name) {
  if (o == Py_None) return nullptr;
  TORCH_CHECK_TYPE(THPVariable_Check(o), name, " must be a tensor");
  return &THPVariable_Unpack(o);
}
const at::Tensor& tensor(PyObject* o, const char* name) {
  TORCH_CHECK_TYPE(THPVariable_Check(o), name, " must be a tensor");
  return THPVariable_Unpack(o);
}

// The one device of a call's tensors.
struct Device {
  c10::Device dev;
  explicit Device(const at::Tensor& t) : dev(t.device()) {
    TORCH_CHECK_VALUE(dev.is_cuda(), "libqlora takes CUDA tensors only");
  }
  void same(Opt t) const {
    TORCH_CHECK_VALUE(!t || t->device() == dev, "all tensors of a call must be on one CUDA device");
  }
  void* stream() const { return c10::cuda::getCurrentCUDAStream(dev.index()).stream(); }
};

qlora_dtype dtype_of(const at::Tensor& t, const char* name) {
  const auto s = t.scalar_type();
  TORCH_CHECK_VALUE(s == at::kFloat || s == at::kBFloat16, name, " must be fp32 or bf16");
  return s == at::kFloat ? QLORA_F32 : QLORA_BF16;
}

// A 2-D tensor whose rows are contiguous: its pointer and the elements
// between rows.  -1: any size.
struct Matrix {
  void* p = nullptr;
  int64_t rows = 0, cols = 0, ld = 0;
};
Matrix matrix(const at::Tensor& t, const char* name, int64_t rows = -1, int64_t cols = -1) {
  TORCH_CHECK_VALUE(t.dim() == 2 && (rows < 0 || t.size(0) == rows) && (cols < 0 || t.size(1) == cols), name,
                    " must be 2-D [", rows < 0 ? std::string("rows") : std::to_string(rows), ", ",
                    cols < 0 ? std::string("cols") : std::to_string(cols), "], got ", t.sizes());
  Matrix m;
  m.rows = t.size(0);
  m.cols = t.size(1);
  TORCH_CHECK_VALUE(m.cols <= 1 || t.stride(1) == 1, name, ": the elements of a row must be contiguous");
  m.ld = m.rows > 1 ? t.stride(0) : m.cols;
  TORCH_CHECK_VALUE(m.ld >= m.cols, name, ": rows overlap");
  m.p = t.data_ptr();
  return m;
}
void* vec(Opt t, const char* name, int64_t n) {
  if (!t) return nullptr;
  TORCH_CHECK_VALUE(t->numel() == n && t->is_contiguous(), name, " must have ", n, " contiguous elements");
  return t->data_ptr();
}
float* vec_f32(Opt t, const char* name, int64_t n) {
  TORCH_CHECK_VALUE(!t || t->scalar_type() == at::kFloat, name, " must be fp32");
  return static_cast<float*>(vec(t, name, n));
}
int* status_word(Opt t) {
  if (!t) return nullptr;
  TORCH_CHECK_VALUE(t->scalar_type() == at::kInt && t->numel() >= 1 && t->is_contiguous(), "d_status must be int32");
  return t->data_ptr<int>();
}
at::Tensor empty(at::IntArrayRef size, const at::Tensor& like, at::ScalarType type) {
  return at::empty(size, like.options().dtype(type).requires_grad(false));
}
int64_t as_int(PyObject* o) {
  const int64_t v = PyLong_AsLongLong(o);
  if (v == -1 && PyErr_Occurred()) throw python_error();
  return v;
}
bool as_bool(PyObject* o) {
  const int v = PyObject_IsTrue(o);
  if (v < 0) throw python_error();
  return v != 0;
}
double as_double(PyObject* o) {
  const double v = PyFloat_AsDouble(o);
  if (v == -1.0 && PyErr_Occurred()) throw python_error();
  return v;
}
PyObject* tuple_of(std::initializer_list<Opt> ts) {
  PyObject* r = PyTuple_New(static_cast<Py_ssize_t>(ts.size()));
  if (!r) throw python_error();
  Py_ssize_t i = 0;
  for (Opt t : ts) {
    PyObject* o = t ? THPVariable_Wrap(*t) : Py_NewRef(Py_None);
    if (!o) {
      Py_DECREF(r);
      throw python_error();
    }
    PyTuple_SET_ITEM(r, i++, o);
  }
  return r;
}
void arguments(Py_ssize_t n, Py_ssize_t want) { TORCH_CHECK_TYPE(n == want, want, " arguments expected, got ", n); }
// the library's call, without the interpreter's lock: a full launch queue blocks in it
template <typename F>
qlora_status unlocked(F&& f) {
  qlora_status st;
  Py_BEGIN_ALLOW_THREADS
  st = f();
  Py_END_ALLOW_THREADS
  return st;
}

// ------------------------------------------------------------------ layer norm
// (X, weight, bias, eps, Y, mean, rstd, d_status) -> (Y, mean, rstd)
PyObject* layernorm_fwd(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  arguments(n, 8);
  const at::Tensor& X = tensor(a[0], "X");
  Opt w = tensor_or_none(a[1], "weight"), b = tensor_or_none(a[2], "bias"), Y = tensor_or_none(a[4], "Y"),
      mean = tensor_or_none(a[5], "mean"), rstd = tensor_or_none(a[6], "rstd"), st = tensor_or_none(a[7], "d_status");
  const float eps = static_cast<float>(as_double(a[3]));
  const Device d(X);
  for (Opt t : {w, b, Y, mean, rstd, st}) d.same(t);
  const c10::cuda::CUDAGuard guard(d.dev);
  const Matrix x = matrix(X, "X");
  const qlora_dtype dt = dtype_of(X, "X");
  TORCH_CHECK_VALUE(!w || !b || w->scalar_type() == b->scalar_type(), "weight and bias must have one type");
  const qlora_dtype wdt = w ? dtype_of(*w, "weight and bias") : b ? dtype_of(*b, "weight and bias") : QLORA_F32;
  void* wp = vec(w, "weight", x.cols);
  void* bp = vec(b, "bias", x.cols);
  TORCH_CHECK_VALUE(!Y || Y->scalar_type() == X.scalar_type(), "Y has X's type");
  at::Tensor own_y, own_mean, own_rstd;
  if (!Y) { own_y = empty({x.rows, x.cols}, X, X.scalar_type()); Y = &own_y; }
  if (!mean) { own_mean = empty({x.rows}, X, at::kFloat); mean = &own_mean; }
  if (!rstd) { own_rstd = empty({x.rows}, X, at::kFloat); rstd = &own_rstd; }
  const Matrix y = matrix(*Y, "Y", x.rows, x.cols);
  float* mp = vec_f32(mean, "mean", x.rows);
  float* rp = vec_f32(rstd, "rstd", x.rows);
  int* sp = status_word(st);
  void* cs = d.stream();
  const qlora_status rc = unlocked(
      [&] { return api.layernorm_fwd(x.p, x.ld, x.rows, x.cols, dt, wp, bp, wdt, eps, y.p, y.ld, mp, rp, sp, cs); });
  if (rc != QLORA_OK) return PyLong_FromLong(rc);
  return tuple_of({Y, mean, rstd});
  END_HANDLE_TH_ERRORS
}

// (dY, X, weight, mean, rstd, dX, dweight, dbias, grad_dtype, want_params, workspace, d_status) -> (dX, dweight, dbias)
PyObject* layernorm_bwd(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  arguments(n, 12);
  const at::Tensor &dY = tensor(a[0], "dY"), &X = tensor(a[1], "X"), &mean = tensor(a[3], "mean"),
                   &rstd = tensor(a[4], "rstd");
  Opt w = tensor_or_none(a[2], "weight"), dX = tensor_or_none(a[5], "dX"), dw = tensor_or_none(a[6], "dweight"),
      db = tensor_or_none(a[7], "dbias"), ws = tensor_or_none(a[10], "workspace"), st = tensor_or_none(a[11], "d_status");
  const bool want_params = as_bool(a[9]);
  const Device d(dY);
  for (Opt t : {&X, &mean, &rstd, w, dX, dw, db, ws, st}) d.same(t);
  const c10::cuda::CUDAGuard guard(d.dev);
  const Matrix x = matrix(X, "X"), dy = matrix(dY, "dY", x.rows, x.cols);
  const qlora_dtype dt = dtype_of(X, "X");
  const qlora_dtype wdt = w ? dtype_of(*w, "weight") : QLORA_F32;
  void* wp = vec(w, "weight", x.cols);
  TORCH_CHECK_VALUE(dY.scalar_type() == X.scalar_type() && (!dX || dX->scalar_type() == X.scalar_type()),
                    "dY and dX have X's type");
  at::Tensor own_dx, own_dw, own_db, own_ws;
  if (!dX) { own_dx = empty({x.rows, x.cols}, X, X.scalar_type()); dX = &own_dx; }
  if (want_params) {
    TORCH_CHECK_TYPE(THPDtype_Check(a[8]), "grad_dtype must be a dtype");
    const at::ScalarType gt = dw   ? dw->scalar_type()
                              : db ? db->scalar_type()
                                   : reinterpret_cast<THPDtype*>(a[8])->scalar_type;
    if (!dw) { own_dw = empty({x.cols}, X, gt); dw = &own_dw; }
    if (!db) { own_db = empty({x.cols}, X, gt); db = &own_db; }
  }
  TORCH_CHECK_VALUE(!dw || !db || dw->scalar_type() == db->scalar_type(), "dweight and dbias must have one type");
  const qlora_dtype gdt = dw ? dtype_of(*dw, "dweight and dbias") : db ? dtype_of(*db, "dweight and dbias") : QLORA_F32;
  const Matrix dx = matrix(*dX, "dX", x.rows, x.cols);
  float* mp = vec_f32(&mean, "mean", x.rows);
  float* rp = vec_f32(&rstd, "rstd", x.rows);
  void* dwp = vec(dw, "dweight", x.cols);
  void* dbp = vec(db, "dbias", x.cols);
  if ((dw || db) && !ws) {
    own_ws = empty({std::max<int64_t>(16, static_cast<int64_t>(api.layernorm_workspace_bytes(x.rows, x.cols)))}, X, at::kByte);
    ws = &own_ws;
  }
  TORCH_CHECK_VALUE(!ws || ws->is_contiguous(), "workspace must be contiguous");
  int* sp = status_word(st);
  void* cs = d.stream();
  const qlora_status rc = unlocked([&] {
    return api.layernorm_bwd(dy.p, dy.ld, x.p, x.ld, x.rows, x.cols, dt, wp, wdt, mp, rp, dx.p, dx.ld, dwp, dbp, gdt,
                             ws ? ws->data_ptr() : nullptr, ws ? ws->nbytes() : 0, sp, cs);
  });
  if (rc != QLORA_OK) return PyLong_FromLong(rc);
  return tuple_of({dX, dw, db});
  END_HANDLE_TH_ERRORS
}

// ------------------------------------------------------------------- FP8 layer
// The codes of an FP8Matrix: E4M3, or plain bytes.  Every other one-byte type
// (E5M2, the fnuz forms, int8) means something else by its bits.
const at::Tensor& fp8_codes(PyObject* o) {
  const at::Tensor& codes = tensor(o, "codes");
  const auto s = codes.scalar_type();
  TORCH_CHECK_VALUE(s == at::kByte || s == at::kFloat8_e4m3fn, "codes must be uint8 or float8_e4m3fn, got ", s);
  return codes;
}
// an FP8Matrix as (rows, cols, block_rows, codes, scale)
qlora_fp8_matrix fp8_matrix(PyObject* const* a, const Device& d) {
  qlora_fp8_matrix m{};
  m.rows = as_int(a[0]);
  m.cols = as_int(a[1]);
  m.block_rows = static_cast<int32_t>(as_int(a[2]));
  const at::Tensor &codes = fp8_codes(a[3]), &scale = tensor(a[4], "scale");
  d.same(&codes);
  d.same(&scale);
  TORCH_CHECK_VALUE(m.rows >= 0 && m.cols >= 1 && (m.block_rows == 1 || m.block_rows == 128), "not an FP8 matrix");
  const Matrix c = matrix(codes, "codes", m.rows);
  TORCH_CHECK_VALUE(c.cols >= (m.cols + 15) / 16 * 16, "codes: a row holds cols rounded up to 16 bytes");
  m.ld = c.ld;
  m.codes = static_cast<uint8_t*>(c.p);
  m.scale = vec_f32(&scale, "scale", (m.rows + m.block_rows - 1) / m.block_rows * ((m.cols + 127) / 128));
  return m;
}

// (X, rows, cols, block_rows, codes, scale, d_status) -> status
PyObject* fp8_quantize(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  arguments(n, 7);
  const at::Tensor& X = tensor(a[0], "X");
  Opt st = tensor_or_none(a[6], "d_status");
  fp8_codes(a[4]);
  const Device d(X);
  d.same(st);
  const c10::cuda::CUDAGuard guard(d.dev);
  const qlora_fp8_matrix out = fp8_matrix(a + 1, d);
  const Matrix x = matrix(X, "X", out.rows, out.cols);
  const qlora_dtype dt = dtype_of(X, "X");
  int* sp = status_word(st);
  void* cs = d.stream();
  return PyLong_FromLong(unlocked([&] { return api.fp8_quantize(x.p, dt, x.ld, &out, sp, cs); }));
  END_HANDLE_TH_ERRORS
}

// (backward, X, xq rows .. scale, W rows .. scale, out, out_dtype, d_status) -> out.  X None: xq holds the
// activations; xq's rows None: the call brings its own scratch.
PyObject* fp8_linear(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  arguments(n, 15);
  const bool bwd = as_bool(a[0]);
  Opt X = tensor_or_none(a[1], "activations"), out = tensor_or_none(a[12], "output"), st = tensor_or_none(a[14], "d_status");
  if (a[2] != Py_None) fp8_codes(a[5]);
  const Device d(fp8_codes(a[10]));
  for (Opt t : {X, out, st}) d.same(t);
  const c10::cuda::CUDAGuard guard(d.dev);
  const qlora_fp8_matrix W = fp8_matrix(a + 7, d);
  const int64_t in_cols = bwd ? W.rows : W.cols, out_cols = bwd ? W.cols : W.rows;
  Matrix x;
  qlora_dtype dt = QLORA_F32;
  if (X) {
    x = matrix(*X, "activations", -1, in_cols);
    dt = dtype_of(*X, "activations");
  }
  qlora_fp8_matrix q{};
  at::Tensor scratch;
  if (a[2] == Py_None) {
    TORCH_CHECK_VALUE(X, "activations, or quantised activations, are needed");
    const int64_t kb = (in_cols + 127) / 128, codes = x.rows * kb * 128;
    scratch = empty({codes + 4 * kb * x.rows}, *X, at::kByte);
    q.rows = x.rows;
    q.cols = in_cols;
    q.ld = kb * 128;
    q.block_rows = 1;
    q.codes = static_cast<uint8_t*>(scratch.data_ptr());
    q.scale = reinterpret_cast<float*>(q.codes + codes);
  } else {
    q = fp8_matrix(a + 2, d);
    TORCH_CHECK_VALUE(!X || q.rows == x.rows, "the scratch must have the activations' rows");
  }
  at::Tensor own;
  if (!out) {
    TORCH_CHECK_TYPE(THPDtype_Check(a[13]), "out_dtype must be a dtype");
    own = empty({q.rows, out_cols}, THPVariable_Unpack(a[10]), reinterpret_cast<THPDtype*>(a[13])->scalar_type);
    out = &own;
  }
  const Matrix y = matrix(*out, "output", q.rows, out_cols);
  const qlora_dtype ydt = dtype_of(*out, "output");
  int* sp = status_word(st);
  void* cs = d.stream();
  const qlora_status rc = unlocked([&] {
    return (bwd ? api.fp8_linear_bwd : api.fp8_linear_fwd)(X ? x.p : nullptr, dt, x.ld, &W, &q, y.p, ydt, y.ld, sp, cs);
  });
  if (rc != QLORA_OK) return PyLong_FromLong(rc);
  return THPVariable_Wrap(*out);
  END_HANDLE_TH_ERRORS
}

// ---------------------------------------------------------------- distillation
struct Distill {
  Matrix z, dz;
  qlora_dtype dt, tdt;
  const void *ids, *t;
  int id_bits, top;
  float* weight;
};
Distill distill_args(const at::Tensor& Z, const at::Tensor& ids, const at::Tensor& t, Opt weight, Opt dZ) {
  Distill r;
  r.z = matrix(Z, "Z");
  r.dt = dtype_of(Z, "Z");
  const auto it = ids.scalar_type();
  TORCH_CHECK_VALUE(it == at::kInt || it == at::kLong, "ids are int32 or int64");
  TORCH_CHECK_VALUE(ids.dim() == 2 && ids.size(0) == r.z.rows && t.sizes() == ids.sizes(), "ids and t must be [rows, top]");
  TORCH_CHECK_VALUE(ids.is_contiguous() && t.is_contiguous(), "ids and t must be contiguous");
  TORCH_CHECK_VALUE(ids.size(1) <= 1 << 20, "ids: too many entries");
  r.ids = ids.data_ptr();
  r.id_bits = it == at::kInt ? 32 : 64;
  r.top = static_cast<int>(ids.size(1));
  r.t = t.data_ptr();
  r.tdt = dtype_of(t, "t");
  r.weight = vec_f32(weight, "row_weight", r.z.rows);
  if (dZ) {
    TORCH_CHECK_VALUE(dZ->scalar_type() == Z.scalar_type(), "dZ has Z's type");
    r.dz = matrix(*dZ, "dZ", r.z.rows, r.z.cols);
  }
  return r;
}

// (Z, ids, t, tau, row_weight, loss, lse, dZ, d_status) -> (loss, lse)
PyObject* distill_fwd(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  arguments(n, 9);
  const at::Tensor &Z = tensor(a[0], "Z"), &ids = tensor(a[1], "ids"), &t = tensor(a[2], "t");
  Opt w = tensor_or_none(a[4], "row_weight"), loss = tensor_or_none(a[5], "loss"), lse = tensor_or_none(a[6], "lse"),
      dZ = tensor_or_none(a[7], "dZ"), st = tensor_or_none(a[8], "d_status");
  const float tau = static_cast<float>(as_double(a[3]));
  const Device d(Z);
  for (Opt x : {&ids, &t, w, loss, lse, dZ, st}) d.same(x);
  const c10::cuda::CUDAGuard guard(d.dev);
  const Distill r = distill_args(Z, ids, t, w, dZ);
  at::Tensor own_loss, own_lse;
  if (!loss) { own_loss = empty({r.z.rows}, Z, at::kFloat); loss = &own_loss; }
  if (!lse) { own_lse = empty({r.z.rows}, Z, at::kFloat); lse = &own_lse; }
  float* lp = vec_f32(loss, "loss", r.z.rows);
  float* sp = vec_f32(lse, "lse", r.z.rows);
  int* status = status_word(st);
  void* cs = d.stream();
  const qlora_status rc = unlocked([&] {
    return api.distill_topk_fwd(r.z.p, r.z.ld, r.z.rows, r.z.cols, r.dt, r.ids, r.id_bits, r.t, r.tdt, r.top, tau, r.weight,
                                lp, sp, r.dz.p, r.dz.ld, status, cs);
  });
  if (rc != QLORA_OK) return PyLong_FromLong(rc);
  return tuple_of({loss, lse});
  END_HANDLE_TH_ERRORS
}

// (Z, ids, t, tau, lse, row_weight, grad_loss, dZ, d_status) -> dZ
PyObject* distill_bwd(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  arguments(n, 9);
  const at::Tensor &Z = tensor(a[0], "Z"), &ids = tensor(a[1], "ids"), &t = tensor(a[2], "t"), &lse = tensor(a[4], "lse");
  Opt w = tensor_or_none(a[5], "row_weight"), g = tensor_or_none(a[6], "grad_loss"), dZ = tensor_or_none(a[7], "dZ"),
      st = tensor_or_none(a[8], "d_status");
  const float tau = static_cast<float>(as_double(a[3]));
  const Device d(Z);
  for (Opt x : {&ids, &t, &lse, w, g, dZ, st}) d.same(x);
  const c10::cuda::CUDAGuard guard(d.dev);
  at::Tensor own;
  if (!dZ) {
    TORCH_CHECK_VALUE(Z.dim() == 2, "Z must be 2-D");
    own = empty(Z.sizes(), Z, Z.scalar_type());
    dZ = &own;
  }
  const Distill r = distill_args(Z, ids, t, w, dZ);
  float* lp = vec_f32(&lse, "lse", r.z.rows);
  float* gp = vec_f32(g, "grad_loss", r.z.rows);
  int* status = status_word(st);
  void* cs = d.stream();
  const qlora_status rc = unlocked([&] {
    return api.distill_topk_bwd(r.z.p, r.z.ld, r.z.rows, r.z.cols, r.dt, r.ids, r.id_bits, r.t, r.tdt, r.top, tau, r.weight,
                                lp, gp, r.dz.p, r.dz.ld, status, cs);
  });
  if (rc != QLORA_OK) return PyLong_FromLong(rc);
  return THPVariable_Wrap(*dZ);
  END_HANDLE_TH_ERRORS
}

// (path of the libqlora build to call)
PyObject* init(PyObject*, PyObject* path) {
  HANDLE_TH_ERRORS
  const char* p = PyUnicode_AsUTF8(path);
  if (!p) throw python_error();
  void* h = dlopen(p, RTLD_NOW | RTLD_LOCAL);
  TORCH_CHECK(h, dlerror());
  auto find = [&](const char* name, auto& f) {
    f = reinterpret_cast<std::decay_t<decltype(f)>>(dlsym(h, name));
    TORCH_CHECK(f, name, " is missing in ", p);
  };
  find("qlora_fp8_quantize", api.fp8_quantize);
  find("qlora_fp8_linear_fwd", api.fp8_linear_fwd);
  find("qlora_fp8_linear_bwd", api.fp8_linear_bwd);
  find("qlora_layernorm_workspace_bytes", api.layernorm_workspace_bytes);
  find("qlora_layernorm_fwd", api.layernorm_fwd);
  find("qlora_layernorm_bwd", api.layernorm_bwd);
  find("qlora_distill_topk_fwd", api.distill_topk_fwd);
  find("qlora_distill_topk_bwd", api.distill_topk_bwd);
  Py_RETURN_NONE;
  END_HANDLE_TH_ERRORS
}

PyCFunction fast(PyObject* (*f)(PyObject*, PyObject* const*, Py_ssize_t)) {
  return reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(f));
}
PyMethodDef methods[] = {
    {"init", init, METH_O, nullptr},
    {"layernorm_fwd", fast(layernorm_fwd), METH_FASTCALL, nullptr},
    {"layernorm_bwd", fast(layernorm_bwd), METH_FASTCALL, nullptr},
    {"fp8_quantize", fast(fp8_quantize), METH_FASTCALL, nullptr},
    {"fp8_linear", fast(fp8_linear), METH_FASTCALL, nullptr},
    {"distill_fwd", fast(distill_fwd), METH_FASTCALL, nullptr},
    {"distill_bwd", fast(distill_bwd), METH_FASTCALL, nullptr},
    {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_calls", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__calls(void) { return PyModule_Create(&module); }
