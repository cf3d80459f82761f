// Python's way to the calls that a decode step makes often: checks, allocation
// and stream look-up in C++ (in a loop of its own a quantizer call with one result
// takes 4.7 us and a product 4.6 - 5.0, host bound; through ctypes and torch's
// Python 8.9 and 7.1).  The C entries are handed over by address at start-up; a status other than
// TLR_OK is returned as an int for the caller to raise.
#include <ATen/ATen.h>
#include <c10/core/DeviceGuard.h>
#include <c10/core/GradMode.h>
#include <c10/hip/HIPStream.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include "tlrgemm.h"

namespace {

decltype(&tlr_block_quantize) quantize_entry = nullptr;
decltype(&tlr_block_gemm) gemm_entry = nullptr;
decltype(&tlr_moe) moe_entry = nullptr;

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

// connect(addresses of tlr_block_quantize, tlr_block_gemm, tlr_moe)
PyObject *connect(PyObject *, PyObject *const *args, Py_ssize_t n) {
  if (n != 3) return value_error("connect: 3 addresses");
  quantize_entry = reinterpret_cast<decltype(quantize_entry)>(PyLong_AsVoidPtr(args[0]));
  gemm_entry = reinterpret_cast<decltype(gemm_entry)>(PyLong_AsVoidPtr(args[1]));
  moe_entry = reinterpret_cast<decltype(moe_entry)>(PyLong_AsVoidPtr(args[2]));
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
  if (PyErr_Occurred()) return nullptr;
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

PyMethodDef methods[] = {
    {"connect", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(connect)), METH_FASTCALL, nullptr},
    {"quantize", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(quantize)), METH_FASTCALL, nullptr},
    {"gemm", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(gemm)), METH_FASTCALL, nullptr},
    {"moe", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(moe)), METH_FASTCALL, nullptr},
    {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_binding", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__binding() { return PyModule_Create(&module); }
