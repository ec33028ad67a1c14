// host_binding.cpp -- the Python module _host: argument checks, output
// allocation and the C call of the operators around the quantized linear layers
// in one step.  A decode step's norm and product take a few microseconds each on
// the GPU; their checks in Python took longer than that (a norm of one token
// 19 us a call, an AdamW step over 448 tensors 345 us).  Every function raises
// before the C call on a bad argument, and returns the library's status (an
// int) if the call refuses.
#include <Python.h>

#include <ATen/core/Tensor.h>
#include <ATen/ops/empty_cuda_dispatch.h>
#include <c10/core/Storage.h>
#include <c10/core/DeviceGuard.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>
#include <torch/csrc/utils/object_ptr.h>

#include "nf4.h"

namespace {

using at::Tensor;

struct BadValue {
  std::string what;
};
struct BadType {
  std::string what;
};

const Tensor &tensor(PyObject *o, const char *name) {
  if (!THPVariable_Check(o)) throw BadType{std::string(name) + " must be a tensor"};
  return THPVariable_Unpack(o);
}

std::string shape_of(const Tensor &t) {
  std::string s = "(";
  for (int64_t i = 0; i < t.dim(); ++i) s += (i ? ", " : "") + std::to_string(t.size(i));
  return s + ")";
}

int dtype_enum(const Tensor &t, const char *name) {
  if (t.scalar_type() == at::kFloat) return NF4_F32;
  if (t.scalar_type() == at::kBFloat16) return NF4_BF16;
  throw BadType{std::string("unsupported dtype of ") + name + "; use torch.float32 or torch.bfloat16"};
}

void on_device(const Tensor &t, const char *name) {
  if (!t.is_cuda()) throw BadValue{std::string(name) + " must be a device (HIP) tensor"};
}

// Leading dimension of a 2-D device matrix whose rows are contiguous.
int64_t matrix(const Tensor &t, const char *name) {
  on_device(t, name);
  dtype_enum(t, name);
  if (t.dim() != 2) throw BadValue{std::string(name) + " must be 2-D"};
  if (t.size(1) > 1 && t.stride(1) != 1)
    throw BadValue{std::string(name) + " must have contiguous rows (stride 1 along its last dimension)"};
  if (t.size(0) <= 1) return std::max<int64_t>(t.size(1), 1);
  if (t.stride(0) < t.size(1)) throw BadValue{std::string(name) + " has overlapping rows"};
  return t.stride(0);
}

void same_place(const Tensor &t, const Tensor &with, const char *name) {
  if (t.device() != with.device())
    throw BadValue{std::string(name) + " is on " + t.device().str() + ", the other operands on " + with.device().str()};
}

void contiguous(const Tensor &t, const char *name) {
  if (!t.is_contiguous()) throw BadValue{std::string(name) + " must be contiguous"};
}

void vector_of(const Tensor &t, int64_t n, const Tensor &with, const char *name) {
  if (t.dim() != 1 || t.size(0) != n)
    throw BadValue{std::string(name) + " must be (" + std::to_string(n) + ",) (got " + shape_of(t) + ")"};
  same_place(t, with, name);
  contiguous(t, name);
}

void like(const Tensor &t, const Tensor &with, const char *name) {
  if (t.sizes() != with.sizes())
    throw BadValue{std::string(name) + " must be " + shape_of(with) + " (got " + shape_of(t) + ")"};
  same_place(t, with, name);
}

int64_t up(int64_t n, int64_t m) { return (n + m - 1) / m * m; }

// Uninitialised memory on the device of `on` (whose guard the callers hold), without the dispatcher's way there.
Tensor fresh(const Tensor &on, at::IntArrayRef size, at::ScalarType t) {
  return at::cuda::empty(size, t, c10::kStrided, on.device(), false, std::nullopt);
}

// The outputs of one call.  Small ones share an allocation, which takes as long as
// such a call's kernel does (a token's norm, four outputs: 7.8 us a call with an
// allocation each, 5.6 with one); large ones do not, so that each is freed by
// itself.
class Outputs {
 public:
  explicit Outputs(const Tensor &on) : on_(on) {}
  // Adds one of `dims` (1 or 2) sizes.
  void add(int64_t rows, int64_t cols, int dims, at::ScalarType t) {
    List &o = list_[count_++];
    o = {{rows, cols}, dims, t, bytes_};
    bytes_ += up(rows * (dims == 2 ? cols : 1) * (int64_t)c10::elementSize(t), kAlign);
  }
  // Allocates what was added (under the callers' device guard).
  void allocate() {
    const bool together = count_ > 1 && bytes_ <= kTogether && bytes_ > 0;
    Tensor all;
    if (together) all = fresh(on_, {bytes_}, at::kByte);
    for (int i = 0; i < count_; ++i) {
      const List &o = list_[i];
      const at::IntArrayRef size(o.size, (size_t)o.dims);
      if (!together) {
        out_[i] = fresh(on_, size, o.type);
        continue;
      }
      out_[i] = at::detail::make_tensor<c10::TensorImpl>(c10::Storage(all.storage()), all.key_set(),
                                                         caffe2::TypeMeta::fromScalarType(o.type));
      out_[i].unsafeGetTensorImpl()->set_storage_offset(o.offset / (int64_t)c10::elementSize(o.type));
      out_[i].unsafeGetTensorImpl()->set_sizes_contiguous(size);
    }
  }
  const Tensor &operator[](int i) const { return out_[i]; }

 private:
  static constexpr int64_t kAlign = 256, kTogether = 64 << 10;
  struct List {
    int64_t size[2];
    int dims;
    at::ScalarType type;
    int64_t offset;
  };
  const Tensor &on_;
  List list_[4];
  Tensor out_[4];
  int count_ = 0;
  int64_t bytes_ = 0;
};

// Adds the two buffers of an 8-bit tensor.
void add_fp8(Outputs &out, int64_t rows, int64_t cols, int64_t block_rows, int format) {
  const int64_t pitch = up(cols, NF4_FP8_BLOCK);
  out.add(rows, pitch, 2, format == NF4_E5M2 ? at::kFloat8_e5m2 : at::kFloat8_e4m3fn);
  out.add((rows + block_rows - 1) / block_rows, up(pitch / NF4_FP8_BLOCK, 4), 2, at::kFloat);
}

// The description of existing buffers, checked.
nf4_fp8_tensor fp8_of(int64_t rows, int64_t cols, int64_t block_rows, const Tensor &data, const Tensor &scale,
                      const char *name) {
  const std::string n = std::string(name) + " (FP8Tensor)";
  if (block_rows != 1 && block_rows != NF4_FP8_BLOCK) throw BadValue{n + ".block_rows must be 1 or 128"};
  if (rows < 0 || cols < 1) throw BadValue{n + " needs rows >= 0 and cols >= 1"};
  const bool e4 = data.scalar_type() == at::kFloat8_e4m3fn;
  if (!e4 && data.scalar_type() != at::kFloat8_e5m2)
    throw BadValue{n + ".data must be float8_e4m3fn or float8_e5m2"};
  const int64_t pitch = up(cols, NF4_FP8_BLOCK), srows = (rows + block_rows - 1) / block_rows;
  const int64_t spitch = up(pitch / NF4_FP8_BLOCK, 4);
  if (data.dim() != 2 || data.size(0) != rows || data.size(1) != pitch)
    throw BadValue{n + ".data must be (" + std::to_string(rows) + ", " + std::to_string(pitch) + ") (got " + shape_of(data) + ")"};
  if (scale.scalar_type() != at::kFloat || scale.dim() != 2 || scale.size(0) != srows || scale.size(1) != spitch)
    throw BadValue{n + ".scale must be fp32 (" + std::to_string(srows) + ", " + std::to_string(spitch) + ") (got " + shape_of(scale) + ")"};
  on_device(data, (n + ".data").c_str());
  contiguous(data, (n + ".data").c_str());
  contiguous(scale, (n + ".scale").c_str());
  same_place(scale, data, (n + ".scale").c_str());
  return nf4_fp8_tensor{rows, cols, (int32_t)block_rows, e4 ? NF4_E4M3 : NF4_E5M2, (uint8_t *)data.data_ptr(),
                        (float *)scale.data_ptr()};
}

// Tells autograd that a caller's tensor was written: a backward pass that saved it then raises.
void written(const Tensor &t) {
  if (!t.is_inference()) t.unsafeGetTensorImpl()->bump_version();   // (an inference tensor counts none)
}

int64_t integer(PyObject *o) {
  const long long v = PyLong_AsLongLong(o);
  if (v == -1 && PyErr_Occurred()) throw python_error();
  return v;
}

double real(PyObject *o) {
  const double v = PyFloat_AsDouble(o);
  if (v == -1.0 && PyErr_Occurred()) throw python_error();
  return v;
}

void *pointer(PyObject *o) {
  void *p = PyLong_AsVoidPtr(o);
  if (!p && PyErr_Occurred()) throw python_error();
  return p;
}

void count_args(Py_ssize_t got, Py_ssize_t want) {
  if (got != want) throw BadType{"takes " + std::to_string(want) + " arguments (got " + std::to_string(got) + ")"};
}

PyObject *tuple_of(std::initializer_list<Tensor> ts) {
  PyObject *out = PyTuple_New((Py_ssize_t)ts.size());
  if (!out) throw python_error();
  Py_ssize_t i = 0;
  for (const Tensor &t : ts) PyTuple_SET_ITEM(out, i++, t.defined() ? THPVariable_Wrap(t) : Py_NewRef(Py_None));
  return out;
}

// rmsnorm_fwd(x, weight, residual | None, eps, out, stream): out 0 fp32, 1 bf16, 2 e4m3, -1 x's type.
// -> (y, h, rstd) or (data, scale, h, rstd); h is None without a residual
PyObject *do_rmsnorm_fwd(PyObject *const *a, Py_ssize_t n) {
  count_args(n, 6);
  const Tensor &x = tensor(a[0], "x"), &w = tensor(a[1], "weight");
  const int64_t ldx = matrix(x, "x"), T = x.size(0), H = x.size(1);
  const int xt = dtype_enum(x, "x"), wt = dtype_enum(w, "weight");
  vector_of(w, H, x, "weight");
  const c10::DeviceGuard guard(x.device());
  int64_t ldr = 0;
  const void *res = nullptr;
  if (a[2] != Py_None) {
    const Tensor &r = tensor(a[2], "residual");
    like(r, x, "residual");
    if (r.scalar_type() != x.scalar_type()) throw BadType{"residual must have x's dtype"};
    ldr = matrix(r, "residual");
    res = r.data_ptr();
  }
  const float eps = (float)real(a[3]);
  const int64_t out = integer(a[4]) < 0 ? xt : integer(a[4]);
  void *stream = pointer(a[5]);
  Outputs o(x);
  o.add(T, 0, 1, at::kFloat);
  if (out == 2) add_fp8(o, T, H, 1, NF4_E4M3);
  else o.add(T, H, 2, out == NF4_BF16 ? at::kBFloat16 : at::kFloat);
  const int hi = out == 2 ? 3 : 2;
  if (res) o.add(T, H, 2, x.scalar_type());
  o.allocate();
  const Tensor &rstd = o[0], &h = o[hi];
  void *hp = res ? h.data_ptr() : nullptr;
  if (out == 2) {
    const nf4_fp8_tensor q = {T, H, 1, NF4_E4M3, (uint8_t *)o[1].data_ptr(), (float *)o[2].data_ptr()};
    const int st = nf4_rmsnorm_fwd(x.data_ptr(), xt, ldx, res, ldr, w.data_ptr(), wt, T, H, eps, hp, nullptr, 0, &q,
                                   (float *)rstd.data_ptr(), stream);
    return st ? PyLong_FromLong(st) : tuple_of({o[1], o[2], h, rstd});
  }
  const int st = nf4_rmsnorm_fwd(x.data_ptr(), xt, ldx, res, ldr, w.data_ptr(), wt, T, H, eps, hp, o[1].data_ptr(),
                                 (int)out, nullptr, (float *)rstd.data_ptr(), stream);
  return st ? PyLong_FromLong(st) : tuple_of({o[1], h, rstd});
}

// rmsnorm_bwd(dy, h, weight, rstd, dh | None, stream) -> (dx, dweight)
PyObject *do_rmsnorm_bwd(PyObject *const *a, Py_ssize_t n) {
  count_args(n, 6);
  const Tensor &dy = tensor(a[0], "dy"), &h = tensor(a[1], "h"), &w = tensor(a[2], "weight"), &rs = tensor(a[3], "rstd");
  const int64_t ldy = matrix(dy, "dy"), ldh = matrix(h, "h"), T = h.size(0), H = h.size(1);
  like(dy, h, "dy");
  vector_of(w, H, h, "weight");
  vector_of(rs, T, h, "rstd");
  if (rs.scalar_type() != at::kFloat) throw BadType{"rstd must be torch.float32"};
  const int dt = dtype_enum(dy, "dy"), ht = dtype_enum(h, "h"), wt = dtype_enum(w, "weight");
  int64_t ldd = 0;
  const void *dh = nullptr;
  if (a[4] != Py_None) {
    const Tensor &d = tensor(a[4], "dh");
    like(d, h, "dh");
    if (d.scalar_type() != h.scalar_type()) throw BadType{"dh must have h's dtype"};
    ldd = matrix(d, "dh");
    dh = d.data_ptr();
  }
  const c10::DeviceGuard guard(h.device());
  size_t need = 0;
  int st = nf4_rmsnorm_bwd_workspace(T, H, &need);
  if (st) return PyLong_FromLong(st);
  Tensor ws = fresh(h, {(int64_t)need}, at::kByte);
  Outputs o(h);
  o.add(T, H, 2, h.scalar_type());
  o.add(H, 0, 1, w.scalar_type());
  o.allocate();
  const Tensor &dx = o[0], &dw = o[1];
  st = nf4_rmsnorm_bwd(dy.data_ptr(), dt, ldy, h.data_ptr(), ht, ldh, w.data_ptr(), wt, (const float *)rs.data_ptr(),
                       dh, ldd, T, H, dx.data_ptr(), dw.data_ptr(), ws.data_ptr(), need, pointer(a[5]));
  return st ? PyLong_FromLong(st) : tuple_of({dx, dw});
}

// fp8_quantize(x, block_rows, format, stream, data | None, scale | None) -> (data, scale); given, they are filled
PyObject *do_fp8_quantize(PyObject *const *a, Py_ssize_t n) {
  count_args(n, 6);
  const Tensor &x = tensor(a[0], "x");
  const int64_t ld = matrix(x, "x"), block_rows = integer(a[1]), format = integer(a[2]);
  if (block_rows != 1 && block_rows != NF4_FP8_BLOCK) throw BadValue{"block_rows must be 1 or 128"};
  const c10::DeviceGuard guard(x.device());
  if (x.size(1) < 1) throw BadValue{"an 8-bit tensor needs at least one column"};
  if (a[4] != Py_None) {
    const Tensor &data = tensor(a[4], "out.data"), &scale = tensor(a[5], "out.scale");
    const nf4_fp8_tensor q = fp8_of(x.size(0), x.size(1), block_rows, data, scale, "out");
    same_place(data, x, "out");
    const int st = nf4_fp8_quantize(x.data_ptr(), dtype_enum(x, "x"), ld, &q, pointer(a[3]));
    if (st) return PyLong_FromLong(st);
    written(data);
    written(scale);
    return tuple_of({data, scale});
  }
  Outputs o(x);
  add_fp8(o, x.size(0), x.size(1), block_rows, (int)format);
  o.allocate();
  const nf4_fp8_tensor q = {x.size(0), x.size(1), (int32_t)block_rows, (int32_t)format, (uint8_t *)o[0].data_ptr(),
                            (float *)o[1].data_ptr()};
  const int st = nf4_fp8_quantize(x.data_ptr(), dtype_enum(x, "x"), ld, &q, pointer(a[3]));
  return st ? PyLong_FromLong(st) : tuple_of({o[0], o[1]});
}

// fp8_matmul(x rows, x cols, x block_rows, x data, x scale, the same of w, out | None, out type, stream) -> y
PyObject *do_fp8_matmul(PyObject *const *a, Py_ssize_t n) {
  count_args(n, 13);
  const Tensor &xd = tensor(a[3], "x.data"), &xs = tensor(a[4], "x.scale"), &wd = tensor(a[8], "w.data"),
               &ws = tensor(a[9], "w.scale");
  const nf4_fp8_tensor x = fp8_of(integer(a[0]), integer(a[1]), integer(a[2]), xd, xs, "x");
  const nf4_fp8_tensor w = fp8_of(integer(a[5]), integer(a[6]), integer(a[7]), wd, ws, "w");
  if (x.cols != w.cols)
    throw BadValue{"x has " + std::to_string(x.cols) + " columns, w " + std::to_string(w.cols)};
  same_place(wd, xd, "w");
  const c10::DeviceGuard guard(xd.device());
  Tensor y;
  if (a[10] != Py_None) {
    y = tensor(a[10], "out");
    if (y.dim() != 2 || y.size(0) != x.rows || y.size(1) != w.rows)
      throw BadValue{"out must be (" + std::to_string(x.rows) + ", " + std::to_string(w.rows) + ") (got " + shape_of(y) + ")"};
    same_place(y, xd, "out");
    contiguous(y, "out");
  } else {
    y = fresh(xd, {x.rows, w.rows}, integer(a[11]) == NF4_BF16 ? at::kBFloat16 : at::kFloat);
  }
  const int st = nf4_fp8_matmul(&x, &w, y.data_ptr(), dtype_enum(y, "out"), pointer(a[12]));
  if (st) return PyLong_FromLong(st);
  if (a[10] != Py_None) written(y);
  return THPVariable_Wrap(y);
}

// adamw_step(params, grads, descriptors, count, device index, lr, beta1, beta2, eps, weight_decay, step,
// grad_scale | None, seed, state_bits, layout | None, stream): checks every tensor against its descriptor's n, writes its
// address there, and steps
PyObject *do_adamw_step(PyObject *const *a, Py_ssize_t n) {
  count_args(n, 16);
  THPObjectPtr ps(PySequence_Fast(a[0], "params must be a sequence")), gs(PySequence_Fast(a[1], "grads must be a sequence"));
  if (!ps || !gs) throw python_error();
  auto *d = reinterpret_cast<nf4_adamw_tensor *>(pointer(a[2]));
  const int64_t count = integer(a[3]), dev = integer(a[4]);
  if (PySequence_Fast_GET_SIZE(ps.get()) != count || PySequence_Fast_GET_SIZE(gs.get()) != count)
    throw BadValue{std::to_string(PySequence_Fast_GET_SIZE(ps.get())) + " params, " +
                   std::to_string(PySequence_Fast_GET_SIZE(gs.get())) + " grads, a state of " + std::to_string(count) + " tensors"};
  int types[2] = {-1, -1};
  for (int64_t i = 0; i < count; ++i)
    for (int which = 0; which < 2; ++which) {
      const char *name = which ? "grads" : "params";
      const Tensor &t = tensor(PySequence_Fast_GET_ITEM((which ? gs : ps).get(), i), name);
      const int type = dtype_enum(t, name);
      if (types[which] < 0) types[which] = type;
      if (type != types[which] || !t.is_cuda() || t.get_device() != dev || !t.is_contiguous() || t.numel() != d[i].n)
        throw BadValue{std::string(name) + "[" + std::to_string(i) + "] must be contiguous, on device " + std::to_string(dev) +
                       ", of one dtype with the others and of " + std::to_string(d[i].n) + " elements (got " + shape_of(t) +
                       " on " + t.device().str() + ")"};
      if (which) d[i].grad = t.data_ptr();
      else d[i].param = t.data_ptr();
    }
  if (!count) return PyLong_FromLong(NF4_OK);
  nf4_adamw_config c = {};
  c.lr = real(a[5]);
  c.beta1 = real(a[6]);
  c.beta2 = real(a[7]);
  c.eps = real(a[8]);
  c.weight_decay = real(a[9]);
  c.step = integer(a[10]);
  if (a[11] != Py_None) {
    const Tensor &s = tensor(a[11], "grad_scale");
    if (s.numel() != 1 || s.scalar_type() != at::kFloat || !s.is_cuda() || s.get_device() != dev)
      throw BadValue{"grad_scale must be one fp32 value on device " + std::to_string(dev)};
    c.grad_scale = (const float *)s.data_ptr();
  }
  c.seed = (uint32_t)integer(a[12]);
  c.state_bits = (int32_t)integer(a[13]);
  if (a[14] != Py_None) {
    const Tensor &l = tensor(a[14], "layout");
    if (!l.is_cuda() || l.get_device() != dev) throw BadValue{"layout must be on device " + std::to_string(dev)};
    c.layout = l.data_ptr();
  }
  c.param_dtype = types[0];
  c.grad_dtype = types[1];
  const c10::DeviceGuard guard(c10::Device(c10::kCUDA, (c10::DeviceIndex)dev));
  const int st = nf4_adamw_step(d, count, &c, pointer(a[15]));
  if (!st)
    for (int64_t i = 0; i < count; ++i) written(THPVariable_Unpack(PySequence_Fast_GET_ITEM(ps.get(), i)));
  return PyLong_FromLong(st);
}

template <PyObject *(*F)(PyObject *const *, Py_ssize_t)>
PyObject *entry(PyObject *, PyObject *const *a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  try {
    return F(a, n);
  } catch (const BadValue &e) {
    PyErr_SetString(PyExc_ValueError, e.what.c_str());
  } catch (const BadType &e) {
    PyErr_SetString(PyExc_TypeError, e.what.c_str());
  }
  return nullptr;
  END_HANDLE_TH_ERRORS
}

#define NF4_METHOD(name) {#name, (PyCFunction)(void (*)(void))entry<do_##name>, METH_FASTCALL, nullptr}
PyMethodDef methods[] = {NF4_METHOD(rmsnorm_fwd), NF4_METHOD(rmsnorm_bwd), NF4_METHOD(fp8_quantize),
                         NF4_METHOD(fp8_matmul), NF4_METHOD(adamw_step), {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_host", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__host() { return PyModule_Create(&module); }
