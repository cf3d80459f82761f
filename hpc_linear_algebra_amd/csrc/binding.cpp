// Python's way to the calls that a decode step makes often: checks, allocation
// and stream look-up in C++ (in a loop of its own a quantizer call with one result
// takes 4.7 us and a product 4.6 - 5.0, host bound; through ctypes and torch's
// Python 8.9 and 7.1).  The C entries are handed over by address at start-up; a status other than
// TLR_OK is returned as an int for the caller to raise.
#include <ATen/ATen.h>
#include <ATen/TracerMode.h>
#include <c10/core/DeviceGuard.h>
#include <c10/core/GradMode.h>
#include <c10/hip/HIPStream.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/custom_function.h>
#include <torch/csrc/autograd/functions/basic_ops.h>
#include <torch/csrc/autograd/python_variable.h>

#include <initializer_list>
#include <stdexcept>
#include <string>
#include <vector>

#include "tlrgemm.h"

namespace {

decltype(&tlr_block_quantize) quantize_entry = nullptr;
decltype(&tlr_block_gemm) gemm_entry = nullptr;
decltype(&tlr_moe) moe_entry = nullptr;
decltype(&tlr_row_quantize) row_quantize_entry = nullptr;
decltype(&tlr_row_gemm_workspace_bytes) row_gemm_bytes_entry = nullptr;
decltype(&tlr_row_gemm) row_gemm_entry = nullptr;
decltype(&tlr_row_linear_workspace_bytes) row_linear_bytes_entry = nullptr;
decltype(&tlr_row_linear) row_linear_entry = nullptr;
decltype(&tlr_expert_sort_workspace_bytes) sort_bytes_entry = nullptr;
decltype(&tlr_expert_sort) sort_entry = nullptr;
decltype(&tlr_expert_gather) gather_entry = nullptr;
decltype(&tlr_expert_combine) combine_entry = nullptr;
decltype(&tlr_expert_combine_grad) combine_grad_entry = nullptr;
decltype(&tlr_gated) gated_entry = nullptr;
decltype(&tlr_gated_grad) gated_grad_entry = nullptr;

// TLR_* of a tensor's type, -1 for types that are not X's or C's.
int code_of(const at::Tensor &t) {
  switch (t.scalar_type()) {
    case at::kFloat: return TLR_F32;
    case at::kHalf: return TLR_F16;
    case at::kBFloat16: return TLR_BF16;
    default: return -1;
  }
}

void *stream_of(const at::Device &d) { return c10::hip::getCurrentHIPStream(d.index()).stream(); }

PyObject *value_error(const char *text) {
  PyErr_SetString(PyExc_ValueError, text);
  return nullptr;
}

// Whether none of the tensors carries a tangent of forward mode, which no operator here computes: its result would come
// back without one.  Otherwise the error is set.  Tangents travel where gradients are off as well.
bool no_tangent(const char *name, std::initializer_list<const at::Tensor *> tensors) {
  for (const at::Tensor *t : tensors)
    if (t->defined() && t->_fw_grad(0).defined()) {
      PyErr_Format(PyExc_RuntimeError, "%s has no forward-mode derivative: call it on tensors without a tangent", name);
      return false;
    }
  return true;
}

// Whether torch.jit.trace is not at work, which would record a call as the allocation of its result alone.  Otherwise the
// error is set.
bool no_trace(const char *name) {
  if (!at::tracer::impl::is_dispatch_enabled()) return true;
  PyErr_Format(PyExc_RuntimeError, "%s cannot be traced: torch.jit.trace would record an empty result", name);
  return false;
}

template <typename F> void take(F &entry, PyObject *address) { entry = reinterpret_cast<F>(PyLong_AsVoidPtr(address)); }

// connect(addresses of the entries above, in their order)
PyObject *connect(PyObject *, PyObject *const *args, Py_ssize_t n) {
  if (n != 15) return value_error("connect: 15 addresses");
  take(quantize_entry, args[0]);
  take(gemm_entry, args[1]);
  take(moe_entry, args[2]);
  take(row_quantize_entry, args[3]);
  take(row_gemm_bytes_entry, args[4]);
  take(row_gemm_entry, args[5]);
  take(row_linear_bytes_entry, args[6]);
  take(row_linear_entry, args[7]);
  take(sort_bytes_entry, args[8]);
  take(sort_entry, args[9]);
  take(gather_entry, args[10]);
  take(combine_entry, args[11]);
  take(combine_grad_entry, args[12]);
  take(gated_entry, args[13]);
  take(gated_grad_entry, args[14]);
  if (PyErr_Occurred()) return nullptr;
  Py_RETURN_NONE;
}

// A rows x cols tensor of another 4-byte type in t's allocation, from byte `at` on.
at::Tensor beside(const at::Tensor &t, at::ScalarType type, int64_t at, int64_t rows, int64_t cols) {
  at::Tensor x = at::detail::make_tensor<c10::TensorImpl>(c10::Storage(t.storage()), t.key_set(), c10::scalarTypeToTypeMeta(type));
  x.unsafeGetTensorImpl()->set_storage_offset(at / 4);
  x.unsafeGetTensorImpl()->set_sizes_contiguous({rows, cols});
  return x;
}

// Codes and scales share one allocation, the scales behind the codes (a call with
// one result 4.7 us; with an allocation each 5.8).
struct Result {
  at::Tensor codes, scales;
  Result(bool wanted, int64_t rows, int64_t k, int64_t block, at::ScalarType f8, const at::Device &d) {
    if (!wanted) return;
    const int64_t ld = (k + 15) / 16 * 16, nq = (k + 127) / 128, nr = block == 1 ? rows : (rows + 127) / 128;
    const int64_t scales_at = (rows * ld + 255) / 256 * 256;
    codes = at::empty({scales_at + 4 * nq * nr}, at::TensorOptions().dtype(f8).device(d));
    scales = beside(codes, at::kFloat, scales_at, nq, nr);
    codes.unsafeGetTensorImpl()->set_sizes_contiguous({rows, ld});
  }
  int64_t ld() const { return codes.defined() ? codes.size(1) : 0; }
  int64_t lds() const { return scales.defined() ? scales.size(1) : 0; }
  void *code_ptr() const { return codes.defined() ? codes.data_ptr() : nullptr; }
  float *scale_ptr() const { return scales.defined() ? static_cast<float *>(scales.data_ptr()) : nullptr; }
};

PyObject *wrap(const at::Tensor &t) {
  if (!t.defined()) Py_RETURN_NONE;
  return THPVariable_Wrap(t);
}

// quantize(x, fmt, block, straight, transposed) -> (codes, scales, codes_t, scales_t) or a status
PyObject *quantize(PyObject *, PyObject *const *args, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  if (n != 5 || !THPVariable_Check(args[0])) return value_error("quantize: a tensor and four numbers");
  at::Tensor x = THPVariable_Unpack(args[0]);
  const int dt = code_of(x);
  if (dt < 0 || x.dim() != 2 || !x.is_cuda())
    return value_error("quantize: a 2-d float32, float16 or bfloat16 tensor on a GPU is needed");
  const long fmt = PyLong_AsLong(args[1]), block = PyLong_AsLong(args[2]);
  const int straight = PyObject_IsTrue(args[3]), transposed = PyObject_IsTrue(args[4]);
  if (PyErr_Occurred()) return nullptr;
  const int64_t rows = x.size(0), k = x.size(1);
  if (k > 1 && x.stride(1) != 1) return value_error("quantize: the rows of x have to be contiguous");
  const c10::DeviceGuard guard(x.device());
  if (rows > 1 && x.stride(0) < k) x = x.clone(at::MemoryFormat::Contiguous);     // an expanded row
  const int64_t ldx = rows > 1 ? x.stride(0) : std::max<int64_t>({x.stride(0), k, 1});
  const at::ScalarType f8 = fmt == TLR_E5M2 ? at::kFloat8_e5m2 : at::kFloat8_e4m3fn;
  const Result a(straight, rows, k, block, f8, x.device()), b(transposed, k, rows, block, f8, x.device());
  const tlr_status st = quantize_entry((tlr_dtype)dt, (tlr_dtype)fmt, (int32_t)block, rows, k, x.data_ptr(), ldx, a.code_ptr(),
                                       a.ld(), a.scale_ptr(), a.lds(), b.code_ptr(), b.ld(), b.scale_ptr(), b.lds(),
                                       stream_of(x.device()));
  if (st != TLR_OK) return PyLong_FromLong(st);
  PyObject *out = PyTuple_New(4);
  if (!out) return nullptr;
  const at::Tensor *t[4] = {&a.codes, &a.scales, &b.codes, &b.scales};
  for (int i = 0; i < 4; ++i) PyTuple_SET_ITEM(out, i, wrap(*t[i]));
  return out;
  END_HANDLE_TH_ERRORS
}

// An operand of a product from its tensors as they are now (they may have been replaced or changed since their matrix
// was made); null, or what is wrong with them.
const char *operand(const at::Tensor &codes, const at::Tensor &scales, int64_t rows, int64_t k, long block, tlr_block_matrix *x) {
  const bool e5 = codes.scalar_type() == at::kFloat8_e5m2;
  if (codes.dim() != 2 || !(e5 || codes.scalar_type() == at::kFloat8_e4m3fn)) return "codes: a 2-d float8_e4m3fn or float8_e5m2 tensor is needed";
  if (block != 1 && block != 128) return "blocks are 1 or 128 rows high";
  if (scales.dim() != 2 || scales.scalar_type() != at::kFloat || scales.device() != codes.device())
    return "scales: a 2-d float32 tensor on the codes' device is needed";
  if (codes.size(0) != rows || codes.size(1) < k || (codes.size(1) > 1 && codes.stride(1) != 1))
    return "codes: a contiguous row of the matrix's entries for each of its rows is needed";
  const int64_t nq = (k + 127) / 128, nr = block == 1 ? rows : (rows + 127) / 128;
  if (scales.size(0) != nq || scales.size(1) != nr || (nr > 1 && scales.stride(1) != 1))
    return "scales: (column blocks, row blocks), rows contiguous, are needed";
  x->ld = rows > 1 ? codes.stride(0) : std::max(codes.stride(0), codes.size(1));
  x->lds = nq > 1 ? scales.stride(0) : std::max(scales.stride(0), nr);
  if (rows > 0 && k > 0 && codes.storage_offset() + (rows - 1) * x->ld + (k + 15) / 16 * 16 > (int64_t)codes.storage().nbytes())
    return "codes: every row has to be readable up to a multiple of 16 entries";
  x->codes = codes.data_ptr();
  x->scales = static_cast<const float *>(scales.data_ptr());
  x->block = (int32_t)block;
  x->fmt = e5 ? TLR_E5M2 : TLR_E4M3;
  return nullptr;
}

// gemm(A's codes, scales, block, B's codes, scales, block, m, n, k, alpha, beta, out or None, type of a new one, flags,
// workspace bytes) -> out or a status
PyObject *gemm(PyObject *, PyObject *const *args, Py_ssize_t n_args) {
  HANDLE_TH_ERRORS
  if (n_args != 15 || !(args[11] == Py_None || THPVariable_Check(args[11]))) return value_error("gemm: 15 arguments");
  for (const int i : {0, 1, 3, 4})
    if (!THPVariable_Check(args[i])) return value_error("gemm: codes and scales are tensors");
  const int64_t m = PyLong_AsLongLong(args[6]), n = PyLong_AsLongLong(args[7]), k = PyLong_AsLongLong(args[8]);
  const double alpha = PyFloat_AsDouble(args[9]), beta = PyFloat_AsDouble(args[10]);
  const long a_block = PyLong_AsLong(args[2]), b_block = PyLong_AsLong(args[5]), type = PyLong_AsLong(args[12]);
  const unsigned long flags = PyLong_AsUnsignedLong(args[13]);
  const size_t bytes = PyLong_AsSize_t(args[14]);
  if (PyErr_Occurred()) return nullptr;
  const at::Tensor &a_codes = THPVariable_Unpack(args[0]), &b_codes = THPVariable_Unpack(args[3]);
  tlr_block_matrix A{}, B{};
  if (const char *wrong = operand(a_codes, THPVariable_Unpack(args[1]), m, k, a_block, &A)) return value_error(wrong);
  if (const char *wrong = operand(b_codes, THPVariable_Unpack(args[4]), n, k, b_block, &B)) return value_error(wrong);
  const at::Device device = b_codes.device();
  if (a_codes.device() != device) return value_error("gemm: operands on different devices");
  if (!device.is_cuda()) return value_error("gemm: operands on a GPU are needed");
  const c10::DeviceGuard guard(device);
  const bool grad = c10::GradMode::is_enabled();
  if (grad && (THPVariable_Unpack(args[1]).requires_grad() || THPVariable_Unpack(args[4]).requires_grad()))
    return value_error("gemm: scales that require a gradient would get none");
  at::Tensor c, ws;
  if (args[11] == Py_None)
    c = at::empty({n, m}, at::TensorOptions().device(device).dtype(type == TLR_F32 ? at::kFloat : type == TLR_F16 ? at::kHalf : at::kBFloat16));
  else
    c = THPVariable_Unpack(args[11]);
  if (grad && c.requires_grad()) return value_error("gemm: an out that requires a gradient would get none");
  if (!c.is_inference()) c.unsafeGetTensorImpl()->bump_version();      // written in place, as autograd sees it
  const int64_t ldc = n > 1 ? c.stride(0) : std::max<int64_t>({c.stride(0), m, 1});
  if (bytes > 0) ws = at::empty({(int64_t)bytes}, at::TensorOptions().dtype(at::kByte).device(device));
  const tlr_status st = gemm_entry((tlr_dtype)code_of(c), m, n, k, alpha, &A, &B, beta, c.data_ptr(), ldc, (uint32_t)flags,
                                   bytes > 0 ? ws.data_ptr() : nullptr, bytes, stream_of(device));
  return st == TLR_OK ? wrap(c) : PyLong_FromLong(st);
  END_HANDLE_TH_ERRORS
}

// moe(address of a tlr_moe_layer, x of its type and width, max tokens, address and bytes of its workspace) ->
// (y, ids, weights) or a status
PyObject *moe(PyObject *, PyObject *const *args, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  if (n != 5 || !THPVariable_Check(args[1])) return value_error("moe: a tensor and four numbers");
  const auto *layer = static_cast<const tlr_moe_layer *>(PyLong_AsVoidPtr(args[0]));
  at::Tensor x = THPVariable_Unpack(args[1]);
  const long most = PyLong_AsLong(args[2]);
  void *ws = PyLong_AsVoidPtr(args[3]);
  const size_t bytes = PyLong_AsSize_t(args[4]);
  if (PyErr_Occurred() || !no_trace("MoELayer") || !no_tangent("MoELayer", {&x})) return nullptr;
  if (x.dim() != 2 || x.size(1) != layer->hidden || code_of(x) != layer->dt || !x.is_cuda())
    return value_error("MoELayer: x is (tokens, hidden), of the layer's type and on its GPU");
  const int64_t tokens = x.size(0);
  if (tokens > most) return value_error("MoELayer: more tokens than the layer was made for");
  const c10::DeviceGuard guard(x.device());
  if (x.stride(1) != 1 || reinterpret_cast<uintptr_t>(x.data_ptr()) % 16 != 0 ||
      (tokens > 1 && (x.stride(0) % 8 != 0 || x.stride(0) < layer->hidden)))
    x = x.clone(at::MemoryFormat::Contiguous);      // 16-byte aligned rows; a fresh allocation starts aligned
  const at::TensorOptions on = at::TensorOptions().device(x.device());
  const at::Tensor y = at::empty({tokens, layer->hidden}, on.dtype(x.scalar_type()));
  const at::Tensor ids = at::empty({2 * tokens, layer->topk}, on.dtype(at::kInt));
  const at::Tensor weights = beside(ids, at::kFloat, 4 * tokens * layer->topk, tokens, layer->topk);
  ids.unsafeGetTensorImpl()->set_sizes_contiguous({tokens, layer->topk});
  const tlr_status st = moe_entry(layer, (int32_t)tokens, x.data_ptr(), tokens > 1 ? x.stride(0) : layer->hidden, y.data_ptr(),
                                  layer->hidden, static_cast<int32_t *>(ids.data_ptr()), static_cast<float *>(weights.data_ptr()),
                                  ws, bytes, stream_of(x.device()));
  if (st != TLR_OK) return PyLong_FromLong(st);
  PyObject *out = PyTuple_New(3);
  if (!out) return nullptr;
  const at::Tensor *t[3] = {&y, &ids, &weights};
  for (int i = 0; i < 3; ++i) PyTuple_SET_ITEM(out, i, wrap(*t[i]));
  return out;
  END_HANDLE_TH_ERRORS
}

// ---- 8-bit integers with a scale for each row ----------------------------------------------------------

// Stride between the rows of a matrix whose rows are contiguous.
int64_t row_stride(const at::Tensor &x) {
  return x.size(0) > 1 ? x.stride(0) : std::max<int64_t>({x.stride(0), x.size(1), 1});
}

// x, or a copy of it where its rows overlap or are not contiguous.
at::Tensor with_rows(const at::Tensor &x) {
  const bool fine = (x.size(1) <= 1 || x.stride(1) == 1) && (x.size(0) <= 1 || x.stride(0) >= x.size(1));
  return fine ? x : x.clone(at::MemoryFormat::Contiguous);
}

at::ScalarType type_of(long code) { return code == TLR_F32 ? at::kFloat : code == TLR_F16 ? at::kHalf : at::kBFloat16; }

PyObject *tuple_of(std::initializer_list<at::Tensor> t) {
  PyObject *out = PyTuple_New((Py_ssize_t)t.size());
  if (!out) return nullptr;
  Py_ssize_t i = 0;
  for (const at::Tensor &x : t) PyTuple_SET_ITEM(out, i++, wrap(x));
  return out;
}

// Codes (rows, ld) and scales (rows) in one allocation, the scales behind the codes.
struct RowResult {
  at::Tensor codes, scales;
  RowResult(int64_t rows, int64_t k, const at::Device &d) {
    const int64_t ld = (k + 15) / 16 * 16, scales_at = (rows * ld + 255) / 256 * 256;
    codes = at::empty({scales_at + 4 * rows}, at::TensorOptions().dtype(at::kChar).device(d));
    scales = beside(codes, at::kFloat, scales_at, rows, 1);
    scales.unsafeGetTensorImpl()->set_sizes_contiguous({rows});
    codes.unsafeGetTensorImpl()->set_sizes_contiguous({rows, ld});
  }
};

const char *quantizable(const at::Tensor &x) {
  return code_of(x) < 0 || x.dim() != 2 || !x.is_cuda() ? "quantize: a 2-d float32, float16 or bfloat16 tensor on a GPU is needed" : nullptr;
}

tlr_status quantize_rows(const at::Tensor &x, const int32_t *index, int64_t rows, const RowResult &r) {
  return row_quantize_entry((tlr_dtype)code_of(x), rows, x.size(1), x.data_ptr(), x.size(0), row_stride(x), index,
                            r.codes.data_ptr(), r.codes.size(1), static_cast<float *>(r.scales.data_ptr()), stream_of(x.device()));
}

// row_quantize(x, rows or None) -> (codes, scales) or a status
PyObject *row_quantize(PyObject *, PyObject *const *args, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  if (n != 2 || !THPVariable_Check(args[0])) return value_error("quantize: a tensor and rows");
  if (!no_trace("int8.quantize")) return nullptr;
  at::Tensor x = THPVariable_Unpack(args[0]), index;
  if (const char *wrong = quantizable(x)) return value_error(wrong);
  if (args[1] != Py_None) {
    if (!THPVariable_Check(args[1])) return value_error("quantize: rows is a tensor");
    index = THPVariable_Unpack(args[1]);
    if (index.scalar_type() != at::kInt || index.dim() != 1 || index.device() != x.device())
      return value_error("quantize: rows is a 1-d int32 tensor on x's device");
  }
  const c10::DeviceGuard guard(x.device());
  x = with_rows(x);
  if (index.defined()) index = index.contiguous();
  const int64_t rows = index.defined() ? index.size(0) : x.size(0);
  const RowResult r(rows, x.size(1), x.device());
  const tlr_status st = quantize_rows(x, index.defined() ? static_cast<const int32_t *>(index.data_ptr()) : nullptr, rows, r);
  return st == TLR_OK ? tuple_of({r.codes, r.scales}) : PyLong_FromLong(st);
  END_HANDLE_TH_ERRORS
}

// An operand of a product: the last two dimensions of codes, the last one of scales; null, or what is wrong.
const char *row_operand(const at::Tensor &codes, const at::Tensor &scales, int64_t k, tlr_row_matrix *x) {
  const int64_t d = codes.dim();
  if ((d != 2 && d != 3) || codes.scalar_type() != at::kChar) return "codes: an int8 tensor of 2 or 3 dimensions is needed";
  if (scales.dim() != d - 1 || scales.scalar_type() != at::kFloat || scales.device() != codes.device())
    return "scales: a float32 tensor on the codes' device, a scale for each row, is needed";
  for (int64_t i = 0; i < d - 1; ++i)
    if (scales.size(i) != codes.size(i)) return "scales: one for each row of codes is needed";
  const int64_t rows = codes.size(d - 2), wide = codes.size(d - 1);
  if (k < 0 || wide < k || (wide > 1 && codes.stride(d - 1) != 1)) return "codes: contiguous rows of k entries are needed";
  if (rows > 1 && scales.stride(d - 2) != 1) return "scales: contiguous rows are needed";
  x->ld = k == 0 ? 0 : rows > 1 ? codes.stride(d - 2) : (wide + 15) / 16 * 16;
  if (codes.numel() > 0 && k > 0) {
    const int64_t last = codes.storage_offset() + (d == 3 ? (codes.size(0) - 1) * codes.stride(0) : 0) + (rows - 1) * x->ld;
    if (last + (k + 15) / 16 * 16 > (int64_t)codes.storage().nbytes()) return "codes: every row has to be readable up to a multiple of 16 entries";
  }
  x->codes = codes.data_ptr();
  x->scales = static_cast<const float *>(scales.data_ptr());
  return nullptr;
}

// The product into c, with what it needs of workspace.
tlr_status multiply(const at::Tensor &c, int64_t m, int64_t n, int64_t k, const tlr_row_matrix &A, const tlr_row_matrix &B,
                    const tlr_row_groups *groups) {
  size_t bytes = 0;
  tlr_status st = row_gemm_bytes_entry(m, n, k, groups ? groups->count : 0, &bytes);
  if (st != TLR_OK) return st;
  at::Tensor ws;
  if (bytes > 0) ws = at::empty({(int64_t)bytes}, at::TensorOptions().dtype(at::kByte).device(c.device()));
  return row_gemm_entry((tlr_dtype)code_of(c), m, n, k, &A, &B, groups, c.data_ptr(), row_stride(c),
                        bytes > 0 ? ws.data_ptr() : nullptr, bytes, stream_of(c.device()));
}

// row_gemm(A's codes, scales, B's codes, scales, k, offsets or None, out or None, type of a new one) -> out or a status
PyObject *row_gemm(PyObject *, PyObject *const *args, Py_ssize_t n_args) {
  HANDLE_TH_ERRORS
  if (n_args != 8) return value_error("gemm: 8 arguments");
  for (const int i : {0, 1, 2, 3})
    if (!THPVariable_Check(args[i])) return value_error("gemm: codes and scales are tensors");
  for (const int i : {5, 6})
    if (args[i] != Py_None && !THPVariable_Check(args[i])) return value_error("gemm: offsets and out are tensors");
  const int64_t k = PyLong_AsLongLong(args[4]);
  const long type = PyLong_AsLong(args[7]);
  if (PyErr_Occurred()) return nullptr;
  const at::Tensor &a_codes = THPVariable_Unpack(args[0]), &b_codes = THPVariable_Unpack(args[2]);
  if (!no_trace("int8.gemm") || !no_tangent("int8.gemm", {&THPVariable_Unpack(args[1]), &THPVariable_Unpack(args[3])}) ||
      (args[6] != Py_None && !no_tangent("int8.gemm", {&THPVariable_Unpack(args[6])})))
    return nullptr;
  tlr_row_matrix A{}, B{};
  if (const char *wrong = row_operand(a_codes, THPVariable_Unpack(args[1]), k, &A)) return value_error(wrong);
  if (const char *wrong = row_operand(b_codes, THPVariable_Unpack(args[3]), k, &B)) return value_error(wrong);
  const at::Device device = b_codes.device();
  if (a_codes.device() != device || !device.is_cuda()) return value_error("gemm: operands on one GPU are needed");
  if (b_codes.dim() != 2) return value_error("gemm: B's codes have 2 dimensions");
  const c10::DeviceGuard guard(device);
  const bool grouped = args[5] != Py_None;
  if ((a_codes.dim() == 3) != grouped) return value_error("gemm: offsets belong to an A with a matrix for each group");
  tlr_row_groups groups{};
  at::Tensor offsets;
  if (grouped) {
    offsets = THPVariable_Unpack(args[5]);
    if (offsets.scalar_type() != at::kInt || offsets.dim() != 1 || offsets.device() != device || offsets.size(0) != a_codes.size(0) + 1)
      return value_error("gemm: offsets is a 1-d int32 tensor on the operands' device, one entry more than groups");
    offsets = offsets.contiguous();
    const bool one = a_codes.size(0) == 1;        // steps that no group takes, and strides of no codes, say nothing
    groups = tlr_row_groups{static_cast<const int32_t *>(offsets.data_ptr()), one || k == 0 ? 0 : a_codes.stride(0),
                            one ? 0 : THPVariable_Unpack(args[1]).stride(0), (int32_t)std::min<int64_t>(a_codes.size(0), 0x7fffffff),
                            args[6] == Py_None};
  }
  const int64_t m = a_codes.size(-2), n = b_codes.size(0);
  const bool grad = c10::GradMode::is_enabled();
  if (grad && (THPVariable_Unpack(args[1]).requires_grad() || THPVariable_Unpack(args[3]).requires_grad()))
    return value_error("gemm: scales that require a gradient would get none");
  at::Tensor c;
  if (args[6] == Py_None) {
    c = at::empty({n, m}, at::TensorOptions().device(device).dtype(type_of(type)));
  } else {
    c = THPVariable_Unpack(args[6]);
    if (c.dim() != 2 || c.size(0) != n || c.size(1) != m || code_of(c) < 0 || c.device() != device || (m > 1 && c.stride(1) != 1))
      return value_error("gemm: out has to be a (B's rows, A's rows) float32, float16 or bfloat16 tensor with contiguous rows");
    if (grad && c.requires_grad()) return value_error("gemm: an out that requires a gradient would get none");
    if (!c.is_inference()) c.unsafeGetTensorImpl()->bump_version();      // written in place, as autograd sees it
  }
  const tlr_status st = multiply(c, m, n, k, A, B, grouped ? &groups : nullptr);
  return st == TLR_OK ? wrap(c) : PyLong_FromLong(st);
  END_HANDLE_TH_ERRORS
}

// x (..., cols) as a matrix with contiguous rows.
at::Tensor as_matrix(const at::Tensor &x) {
  if (x.dim() == 2) return with_rows(x);
  int64_t rows = 1;
  for (int64_t i = 0; i + 1 < x.dim(); ++i) rows *= x.size(i);
  return with_rows(x.reshape({rows, x.size(-1)}));
}

// Sizes of x with another last one.
std::vector<int64_t> sizes_with(const at::Tensor &x, int64_t last) {
  std::vector<int64_t> s = x.sizes().vec();
  s.back() = last;
  return s;
}

// row_linear(x, W's codes, scales, k) -> (..., rows of W) or a status: x (..., k) quantized and multiplied in one call
PyObject *row_linear(PyObject *, PyObject *const *args, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  if (n != 4) return value_error("linear: 4 arguments");
  for (const int i : {0, 1, 2})
    if (!THPVariable_Check(args[i])) return value_error("linear: x, codes and scales are tensors");
  at::Tensor x = THPVariable_Unpack(args[0]), ws;
  const at::Tensor &codes = THPVariable_Unpack(args[1]);
  const int64_t k = PyLong_AsLongLong(args[3]);
  if (PyErr_Occurred() || !no_trace("int8.linear") || !no_tangent("int8.linear", {&x, &THPVariable_Unpack(args[2])})) return nullptr;
  const bool grad = c10::GradMode::is_enabled();
  if (grad && x.requires_grad()) {
    PyErr_SetString(PyExc_RuntimeError, "int8.linear has no backward pass: call it under torch.no_grad() or on detached tensors");
    return nullptr;
  }
  if (code_of(x) < 0 || x.dim() < 1 || !x.is_cuda()) return value_error("linear: a float32, float16 or bfloat16 x on a GPU is needed");
  tlr_row_matrix A{};
  if (const char *wrong = row_operand(codes, THPVariable_Unpack(args[2]), k, &A)) return value_error(wrong);
  if (codes.dim() != 2 || codes.device() != x.device() || x.size(-1) != k) return value_error("linear: x is (..., k) on the device of a weight of 2 dimensions");
  if (grad && THPVariable_Unpack(args[2]).requires_grad()) return value_error("linear: scales that require a gradient would get none");
  const c10::DeviceGuard guard(x.device());
  const int64_t m = codes.size(0);
  // no view of another tensor: one made without gradients cannot be changed in place with them
  const at::Tensor c = at::empty(sizes_with(x, m), at::TensorOptions().device(x.device()).dtype(x.scalar_type()));
  x = as_matrix(x);
  const int64_t tokens = x.size(0);
  size_t bytes = 0;
  tlr_status st = row_linear_bytes_entry(m, tokens, k, &bytes);
  if (st != TLR_OK) return PyLong_FromLong(st);
  if (bytes > 0) ws = at::empty({(int64_t)bytes}, at::TensorOptions().dtype(at::kByte).device(x.device()));
  st = row_linear_entry((tlr_dtype)code_of(x), m, tokens, k, &A, x.data_ptr(), row_stride(x), c.data_ptr(), std::max<int64_t>(m, 1),
                        bytes > 0 ? ws.data_ptr() : nullptr, bytes, stream_of(x.device()));
  if (st != TLR_OK) return PyLong_FromLong(st);
  return wrap(c);
  END_HANDLE_TH_ERRORS
}

// ---- tokens sorted by expert ---------------------------------------------------------------------------

// sort(ids, experts) -> (offsets, place, rows), views of one allocation, or a status
PyObject *sort(PyObject *, PyObject *const *args, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  if (n != 2 || !THPVariable_Check(args[0])) return value_error("sort: a tensor and a number");
  at::Tensor ids = THPVariable_Unpack(args[0]);
  const long experts = PyLong_AsLong(args[1]);
  if (PyErr_Occurred() || !no_trace("sort")) return nullptr;
  if (ids.dim() != 2 || !ids.is_cuda() || (ids.scalar_type() != at::kInt && ids.scalar_type() != at::kLong))
    return value_error("sort: ids is a (tokens, topk) int32 or int64 tensor on a GPU");
  if (experts < 1 || experts > 1024 || ids.size(1) < 1 || ids.size(1) > 64) return value_error("sort: experts are 1 .. 1024, topk 1 .. 64");
  const c10::DeviceGuard guard(ids.device());
  ids = ids.contiguous();
  const int64_t tokens = ids.size(0), topk = ids.size(1), all = tokens * topk;
  size_t bytes = 0;
  tlr_status st = sort_bytes_entry(tokens, (int32_t)topk, (int32_t)experts, &bytes);
  if (st != TLR_OK) return PyLong_FromLong(st);
  const at::TensorOptions on = at::TensorOptions().device(ids.device()).dtype(at::kInt);
  const at::Tensor offsets = at::empty({experts + 1 + 2 * all + (int64_t)bytes / 4}, on);
  const at::Tensor place = beside(offsets, at::kInt, 4 * (experts + 1), tokens, topk), rows = beside(offsets, at::kInt, 4 * (experts + 1 + all), all, 1);
  rows.unsafeGetTensorImpl()->set_sizes_contiguous({all});
  auto *p = static_cast<int32_t *>(offsets.data_ptr());
  offsets.unsafeGetTensorImpl()->set_sizes_contiguous({experts + 1});
  st = sort_entry(ids.scalar_type() == at::kInt ? 4 : 8, tokens, (int32_t)topk, (int32_t)experts, ids.data_ptr(), p, p + experts + 1,
                  p + experts + 1 + all, bytes ? p + experts + 1 + 2 * all : nullptr, bytes, stream_of(ids.device()));
  return st == TLR_OK ? tuple_of({offsets, place, rows}) : PyLong_FromLong(st);
  END_HANDLE_TH_ERRORS
}

// A call of the library that failed within an operator of autograd.  The Python call returns its status; from a backward
// pass it arrives as a RuntimeError.
struct Failed : std::runtime_error {
  tlr_status status;
  explicit Failed(tlr_status st) : std::runtime_error("a tlr_* call failed with status " + std::to_string(st)), status(st) {}
};
void must(tlr_status st) {
  if (st != TLR_OK) throw Failed(st);
}

// Gradients that have none themselves: where a graph of the backward pass is made, differentiating it is an error.
torch::autograd::variable_list once(const char *name, torch::autograd::variable_list grads) {
  bool any = false;
  for (const at::Tensor &g : grads) any = any || g.defined();
  if (!c10::GradMode::is_enabled() || !any) return grads;
  torch::autograd::variable_list leaves;
  for (const at::Tensor &g : grads) leaves.push_back(g.defined() ? g.detach().requires_grad_() : g);
  auto end = std::make_shared<torch::autograd::DelayedError>(std::string(name) + " has no second derivative", (int)grads.size());
  return (*end)(std::move(leaves));
}

// What the operators on sorted rows take of a sort: place (tokens, topk) and the first row of no expert.
struct Order {
  at::Tensor place, offsets;
  Order(const at::Tensor &p, const at::Tensor &o) : place(p), offsets(o) {}
  int64_t tokens() const { return place.size(0); }
  int64_t topk() const { return place.size(1); }
  const int32_t *at() const { return static_cast<const int32_t *>(place.data_ptr()); }
  const int32_t *end() const { return static_cast<const int32_t *>(offsets.data_ptr()) + offsets.size(0) - 1; }
};

const char *not_an_order(PyObject *p, PyObject *o, const at::Device &d) {
  const char *wrong = "an order as moe.sort gives it, on the operands' device, is needed";
  if (!THPVariable_Check(p) || !THPVariable_Check(o)) return wrong;
  const at::Tensor &place = THPVariable_Unpack(p), &offsets = THPVariable_Unpack(o);
  if (place.scalar_type() != at::kInt || place.dim() != 2 || place.device() != d || !place.is_contiguous()) return wrong;
  if (offsets.scalar_type() != at::kInt || offsets.dim() != 1 || offsets.size(0) < 2 || offsets.device() != d || !offsets.is_contiguous()) return wrong;
  return nullptr;
}

at::Tensor like(const at::Tensor &x, int64_t rows, int64_t cols) {
  return at::empty({rows, cols}, at::TensorOptions().device(x.device()).dtype(x.scalar_type()));
}

at::Tensor gather_rows(at::Tensor x, const Order &o) {
  const c10::DeviceGuard guard(x.device());
  x = with_rows(x);
  const at::Tensor y = like(x, o.tokens() * o.topk(), x.size(1));
  must(gather_entry((tlr_dtype)code_of(x), o.tokens(), (int32_t)o.topk(), x.size(1), x.data_ptr(), row_stride(x), o.at(), o.end(),
                    y.data_ptr(), row_stride(y), stream_of(x.device())));
  return y;
}

// weights undefined: 1
at::Tensor combine_rows(at::Tensor y, at::Tensor w, const Order &o) {
  const c10::DeviceGuard guard(y.device());
  y = with_rows(y);
  if (w.defined()) w = w.contiguous();
  const at::Tensor out = like(y, o.tokens(), y.size(1));
  must(combine_entry((tlr_dtype)code_of(y), o.tokens(), (int32_t)o.topk(), y.size(1), y.data_ptr(), row_stride(y), o.at(), o.end(),
                     w.defined() ? static_cast<const float *>(w.data_ptr()) : nullptr, out.data_ptr(), row_stride(out), stream_of(y.device())));
  return out;
}

struct Gather : torch::autograd::Function<Gather> {
  static at::Tensor forward(torch::autograd::AutogradContext *ctx, const at::Tensor &x, const at::Tensor &place, const at::Tensor &offsets) {
    ctx->save_for_backward({place, offsets});
    return gather_rows(x, Order(place, offsets));
  }
  static torch::autograd::variable_list backward(torch::autograd::AutogradContext *ctx, const torch::autograd::variable_list &grads) {
    const auto saved = ctx->get_saved_variables();
    return once("gather", {combine_rows(grads[0], at::Tensor(), Order(saved[0], saved[1])), at::Tensor(), at::Tensor()});
  }
};

// y's count of changes without its memory: saved in its place, a change of y is noticed all the same.
at::Tensor changes_of(const at::Tensor &y) {
  at::Tensor t = at::empty({0}, y.options());
  t.unsafeGetTensorImpl()->set_version_counter(y.unsafeGetTensorImpl()->version_counter());
  return t;
}

// The rows are kept for the gradient of the weights alone (8192 x 8 x 4096 in bf16: 512 MB).
struct Combine : torch::autograd::Function<Combine> {
  static at::Tensor forward(torch::autograd::AutogradContext *ctx, const at::Tensor &y, const at::Tensor &w, const at::Tensor &place,
                            const at::Tensor &offsets) {
    ctx->save_for_backward({w.requires_grad() ? y : changes_of(y), w, place, offsets});
    return combine_rows(y, w, Order(place, offsets));
  }
  static torch::autograd::variable_list backward(torch::autograd::AutogradContext *ctx, const torch::autograd::variable_list &grads) {
    const auto saved = ctx->get_saved_variables();
    const Order o(saved[2], saved[3]);
    const c10::DeviceGuard guard(grads[0].device());
    const at::Tensor dout = with_rows(grads[0]), w = saved[1].contiguous();
    const int64_t hidden = dout.size(1);
    at::Tensor y, dy, dw;
    if (ctx->needs_input_grad(0)) dy = like(dout, o.tokens() * o.topk(), hidden);
    if (ctx->needs_input_grad(1)) {
      y = with_rows(saved[0]);
      dw = like(w, o.tokens(), o.topk());
    }
    must(combine_grad_entry((tlr_dtype)code_of(dout), o.tokens(), (int32_t)o.topk(), hidden, dout.data_ptr(), row_stride(dout),
                            y.defined() ? y.data_ptr() : nullptr, y.defined() ? row_stride(y) : hidden, o.at(), o.end(),
                            static_cast<const float *>(w.data_ptr()), dy.defined() ? dy.data_ptr() : nullptr, dy.defined() ? row_stride(dy) : hidden,
                            dw.defined() ? static_cast<float *>(dw.data_ptr()) : nullptr, stream_of(dout.device())));
    return once("combine", {dy, dw, at::Tensor(), at::Tensor()});
  }
};

const char *rows_of(const at::Tensor &x, int64_t rows) {
  return code_of(x) < 0 || x.dim() != 2 || !x.is_cuda() || x.size(0) != rows ? "2-d float32, float16 or bfloat16 tensors on a GPU, of the order's rows, are needed" : nullptr;
}

// gather(x, place, offsets) -> sorted rows or a status; with their gradient where x has one
PyObject *gather(PyObject *, PyObject *const *args, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  if (n != 3 || !THPVariable_Check(args[0])) return value_error("gather: 3 tensors");
  const at::Tensor &x = THPVariable_Unpack(args[0]);
  if (!no_trace("gather") || !no_tangent("gather", {&x})) return nullptr;
  if (const char *wrong = not_an_order(args[1], args[2], x.device())) return value_error(wrong);
  const Order o(THPVariable_Unpack(args[1]), THPVariable_Unpack(args[2]));
  if (const char *wrong = rows_of(x, o.tokens())) return value_error(wrong);
  try {
    if (c10::GradMode::is_enabled() && x.requires_grad()) return wrap(Gather::apply(x, o.place, o.offsets));
    return wrap(gather_rows(x, o));
  } catch (const Failed &f) {
    return PyLong_FromLong(f.status);
  }
  END_HANDLE_TH_ERRORS
}

// combine(y, weights or None, place, offsets) -> a row for each token or a status; with gradients where y or weights have one
PyObject *combine(PyObject *, PyObject *const *args, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  if (n != 4 || !THPVariable_Check(args[0]) || !(args[1] == Py_None || THPVariable_Check(args[1]))) return value_error("combine: 4 tensors");
  const at::Tensor &y = THPVariable_Unpack(args[0]);
  at::Tensor w;
  if (args[1] != Py_None) w = THPVariable_Unpack(args[1]);
  if (!no_trace("combine") || !no_tangent("combine", {&y, &w})) return nullptr;
  if (const char *wrong = not_an_order(args[2], args[3], y.device())) return value_error(wrong);
  const Order o(THPVariable_Unpack(args[2]), THPVariable_Unpack(args[3]));
  if (const char *wrong = rows_of(y, o.tokens() * o.topk())) return value_error(wrong);
  if (w.defined() && (w.scalar_type() != at::kFloat || w.dim() != 2 || w.size(0) != o.tokens() || w.size(1) != o.topk() || w.device() != y.device()))
    return value_error("weights: a float32 (tokens, topk) tensor on the operands' device is needed");
  try {
    if (c10::GradMode::is_enabled() && (y.requires_grad() || (w.defined() && w.requires_grad()))) {
      if (!w.defined()) {
        const c10::DeviceGuard guard(y.device());
        w = at::ones({o.tokens(), o.topk()}, at::TensorOptions().device(y.device()).dtype(at::kFloat));
      }
      return wrap(Combine::apply(y, w, o.place, o.offsets));
    }
    return wrap(combine_rows(y, w, o));
  } catch (const Failed &f) {
    return PyLong_FromLong(f.status);
  }
  END_HANDLE_TH_ERRORS
}

// ---- gated activation -----------------------------------------------------------------------------------

// y (..., inter) of x (..., 2 inter), no view of another tensor: a result of autograd that is one cannot be changed in place.
// With codes (rows, 2, ld) and scales (rows, 2, blocks), in one allocation, if kept.
struct GatedResult {
  at::Tensor y, codes, scales;
  GatedResult(const at::Tensor &given, bool keep) {
    const c10::DeviceGuard guard(given.device());
    const at::Tensor x = as_matrix(given);
    const int64_t rows = x.size(0), inter = x.size(1) / 2, ld = (inter + 15) / 16 * 16, nq = (inter + 127) / 128;
    y = at::empty(sizes_with(given, inter), at::TensorOptions().device(x.device()).dtype(x.scalar_type()));
    if (keep) {
      const int64_t scales_at = (2 * rows * ld + 255) / 256 * 256;
      codes = at::empty({scales_at + 8 * rows * nq}, at::TensorOptions().dtype(at::kChar).device(x.device()));
      scales = beside(codes, at::kFloat, scales_at, 2 * rows, nq);
      scales.unsafeGetTensorImpl()->set_sizes_contiguous({rows, 2, nq});
      codes.unsafeGetTensorImpl()->set_sizes_contiguous({rows, 2, ld});
    }
    must(gated_entry((tlr_dtype)code_of(x), rows, inter, x.data_ptr(), row_stride(x), y.data_ptr(), std::max<int64_t>(inter, 1),
                     keep ? codes.data_ptr() : nullptr, ld, keep ? static_cast<float *>(scales.data_ptr()) : nullptr, nq, stream_of(x.device())));
  }
};

at::Tensor gated_rows_grad(const at::Tensor &dy, const at::Tensor &codes, const at::Tensor &scales) {
  const c10::DeviceGuard guard(dy.device());
  const int64_t rows = dy.size(0), inter = dy.size(1);
  const at::Tensor dx = like(dy, rows, 2 * inter);
  must(gated_grad_entry((tlr_dtype)code_of(dy), rows, inter, dy.data_ptr(), row_stride(dy), codes.data_ptr(), codes.size(2),
                        static_cast<const float *>(scales.data_ptr()), scales.size(2), dx.data_ptr(), row_stride(dx), stream_of(dy.device())));
  return dx;
}

struct Gated : torch::autograd::Function<Gated> {
  static at::Tensor forward(torch::autograd::AutogradContext *ctx, const at::Tensor &x) {
    const GatedResult r(x, true);
    ctx->save_for_backward({r.codes, r.scales});
    return r.y;
  }
  static torch::autograd::variable_list backward(torch::autograd::AutogradContext *ctx, const torch::autograd::variable_list &grads) {
    const auto saved = ctx->get_saved_variables();
    const c10::DeviceGuard guard(grads[0].device());
    const at::Tensor dx = gated_rows_grad(as_matrix(grads[0]), saved[0], saved[1]);
    return once("gated", {grads[0].dim() == 2 ? dx : dx.view(sizes_with(grads[0], dx.size(1)))});
  }
};

bool gateable(const at::Tensor &x) { return code_of(x) >= 0 && x.is_cuda() && x.dim() >= 1 && x.size(-1) % 2 == 0; }
const char *const NOT_GATEABLE = "gated: a float32, float16 or bfloat16 tensor (..., 2*inter) on a GPU is needed";

// gated(x) -> y or a status; with its gradient where x has one
PyObject *gated(PyObject *, PyObject *x_) {
  HANDLE_TH_ERRORS
  if (!no_trace("gated") || (THPVariable_Check(x_) && !no_tangent("gated", {&THPVariable_Unpack(x_)}))) return nullptr;
  if (!THPVariable_Check(x_) || !gateable(THPVariable_Unpack(x_))) return value_error(NOT_GATEABLE);
  const at::Tensor &x = THPVariable_Unpack(x_);
  const c10::DeviceGuard guard(x.device());
  try {
    if (c10::GradMode::is_enabled() && x.requires_grad()) return wrap(Gated::apply(x));
    return wrap(GatedResult(x, false).y);
  } catch (const Failed &f) {
    return PyLong_FromLong(f.status);
  }
  END_HANDLE_TH_ERRORS
}

// gated_forward(x of 2 dimensions) -> (y, codes, scales) or a status
PyObject *gated_forward(PyObject *, PyObject *x_) {
  HANDLE_TH_ERRORS
  if (!no_trace("gated_forward") || (THPVariable_Check(x_) && !no_tangent("gated_forward", {&THPVariable_Unpack(x_)}))) return nullptr;
  if (!THPVariable_Check(x_) || !gateable(THPVariable_Unpack(x_)) || THPVariable_Unpack(x_).dim() != 2) return value_error(NOT_GATEABLE);
  const at::Tensor &x = THPVariable_Unpack(x_);
  const c10::DeviceGuard guard(x.device());
  try {
    const GatedResult r(x, true);
    return tuple_of({r.y, r.codes, r.scales});
  } catch (const Failed &f) {
    return PyLong_FromLong(f.status);
  }
  END_HANDLE_TH_ERRORS
}

// gated_backward(dy, codes, scales) -> dx or a status
PyObject *gated_backward(PyObject *, PyObject *const *args, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  if (n != 3) return value_error("gated_backward: 3 tensors");
  for (const int i : {0, 1, 2})
    if (!THPVariable_Check(args[i])) return value_error("gated_backward: 3 tensors");
  const at::Tensor &dy = THPVariable_Unpack(args[0]), &codes = THPVariable_Unpack(args[1]), &scales = THPVariable_Unpack(args[2]);
  if (!no_trace("gated_backward") || !no_tangent("gated_backward", {&dy, &scales})) return nullptr;
  if (code_of(dy) < 0 || dy.dim() != 2 || !dy.is_cuda()) return value_error("gated_backward: dy is a 2-d float32, float16 or bfloat16 tensor on a GPU");
  const int64_t rows = dy.size(0), inter = dy.size(1), ld = (inter + 15) / 16 * 16, nq = (inter + 127) / 128;
  if (codes.scalar_type() != at::kChar || codes.sizes() != at::IntArrayRef({rows, 2, ld}) || !codes.is_contiguous() || codes.device() != dy.device() ||
      scales.scalar_type() != at::kFloat || scales.sizes() != at::IntArrayRef({rows, 2, nq}) || !scales.is_contiguous() || scales.device() != dy.device())
    return value_error("gated_backward: codes and scales as gated_forward gives them, of dy's rows, are needed");
  const c10::DeviceGuard guard(dy.device());
  try {
    return wrap(gated_rows_grad(with_rows(dy), codes, scales));
  } catch (const Failed &f) {
    return PyLong_FromLong(f.status);
  }
  END_HANDLE_TH_ERRORS
}

// no_tangent(name, x): None, or the error
PyObject *no_tangent(PyObject *, PyObject *const *args, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  const char *name = n == 2 && PyUnicode_Check(args[0]) ? PyUnicode_AsUTF8(args[0]) : nullptr;
  if (!name || !THPVariable_Check(args[1])) return value_error("no_tangent: a name and a tensor");
  if (!no_tangent(name, {&THPVariable_Unpack(args[1])})) return nullptr;
  Py_RETURN_NONE;
  END_HANDLE_TH_ERRORS
}

#define METHOD(f) {#f, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(static_cast<PyObject *(*)(PyObject *, PyObject *const *, Py_ssize_t)>(f))), METH_FASTCALL, nullptr}
PyMethodDef methods[] = {METHOD(connect), METHOD(quantize), METHOD(gemm), METHOD(moe), METHOD(row_quantize), METHOD(row_gemm),
                         METHOD(row_linear), METHOD(sort), METHOD(gather), METHOD(combine), {"gated", gated, METH_O, nullptr},
                         {"gated_forward", gated_forward, METH_O, nullptr}, METHOD(gated_backward), METHOD(no_tangent), {nullptr, nullptr, 0, nullptr}};
#undef METHOD
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_binding", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__binding() { return PyModule_Create(&module); }
