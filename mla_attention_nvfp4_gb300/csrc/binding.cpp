// Python binding of the 8-bit calls: checks, outputs, device and stream in
// one native call each.  The smallest of these calls take 2 to 6 us on the
// GPU; the same steps in Python take 10 to 20 us of the host.  Arguments are
// those of the functions of the package's __init__.py, by position, None
// where one is left out.  A failed check raises ValueError; a library status
// other than MLA_OK is returned as an int.
#include <Python.h>

#include <ATen/core/TensorBody.h>
#include <ATen/ops/empty.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <string>

#include "../../include/mla_nvfp4.h"

namespace {

using at::Tensor;
constexpr auto kBF16 = at::kBFloat16;
constexpr auto kF32 = at::kFloat;
constexpr auto kI32 = at::kInt;
constexpr auto kF8 = at::kFloat8_e4m3fn;

// Reads the arguments of one call in order.
struct Args {
  PyObject* const* a;
  Py_ssize_t n, at = 0;
  int device = -1;  // of the first tensor

  static void fail(const std::string& what) { TORCH_CHECK_VALUE(false, what); }

  PyObject* next() {
    TORCH_CHECK_TYPE(at < n, "too few arguments");
    return a[at++];
  }
  bool skip_none() {
    if (at < n && a[at] == Py_None) {
      ++at;
      return true;
    }
    return false;
  }
  const Tensor& tensor(const char* name, at::ScalarType dtype) {
    PyObject* o = next();
    TORCH_CHECK_TYPE(THPVariable_Check(o), name, " must be a tensor");
    const Tensor& t = THPVariable_Unpack(o);
    if (!t.is_cuda()) fail(std::string(name) + " must be a CUDA tensor");
    if (t.scalar_type() != dtype)
      fail(std::string(name) + " must be " + c10::toString(dtype) + ", got " + c10::toString(t.scalar_type()));
    if (device < 0) device = t.get_device();
    if (t.get_device() != device)
      fail(std::string(name) + " is on cuda:" + std::to_string(t.get_device()) + ", expected cuda:" + std::to_string(device));
    return t;
  }
  int64_t integer() {
    const long long v = PyLong_AsLongLong(next());
    if (v == -1 && PyErr_Occurred()) throw python_error();
    return v;
  }
  double number() {
    const double v = PyFloat_AsDouble(next());
    if (v == -1.0 && PyErr_Occurred()) throw python_error();
    return v;
  }
  bool flag() {
    const int v = PyObject_IsTrue(next());
    if (v < 0) throw python_error();
    return v != 0;
  }
  uint32_t* error_word() {
    if (skip_none()) return nullptr;
    const Tensor& t = tensor("error_word", kI32);
    if (t.numel() < 1 || !t.is_contiguous()) fail("error_word must be contiguous");
    return static_cast<uint32_t*>(t.data_ptr());
  }
  // A given output, checked, or a new one.
  Tensor output(const char* name, at::ScalarType dtype, at::IntArrayRef shape) {
    if (skip_none()) return at::empty(shape, at::TensorOptions(dtype).device(at::Device(at::kCUDA, static_cast<c10::DeviceIndex>(device))));
    const Tensor& t = tensor(name, dtype);
    if (t.sizes() != shape || !t.is_contiguous()) fail(std::string(name) + " must be contiguous with the output's shape");
    return t;
  }
};

// Last dimension contiguous (a tensor without elements, or a last dimension
// of one, may have any stride).
bool rows_contiguous(const Tensor& t) { return t.stride(-1) == 1 || t.size(-1) == 1 || t.numel() == 0; }

void need(bool ok, const char* what) {
  TORCH_CHECK_VALUE(ok, what);
}

// Launches on the tensors' device and its current stream.
struct Launch {
  c10::cuda::CUDAGuard guard;
  void* stream;
  explicit Launch(int device)
      : guard(static_cast<c10::DeviceIndex>(device)),
        stream(c10::cuda::getCurrentCUDAStream(static_cast<c10::DeviceIndex>(device)).stream()) {}
};

const uint8_t* bytes(const Tensor& t) { return static_cast<const uint8_t*>(t.data_ptr()); }
template <class T>
T* data(const Tensor& t) {
  return static_cast<T*>(t.data_ptr());
}

// cache and scales; returns num_slots.
int64_t check_cache(const Tensor& cache, const Tensor& scales) {
  need(cache.dim() == 2 && cache.size(1) == MLA_D_QK_DECODE && cache.is_contiguous(), "cache must be contiguous [num_slots, 576]");
  const int64_t slots = cache.size(0);
  need(slots % MLA_FP8_BLOCK == 0, "num_slots must be a multiple of 64");
  need(scales.dim() == 1 && scales.size(0) == slots / MLA_FP8_BLOCK && scales.is_contiguous(),
       "scales must be contiguous [num_slots / 64]");
  return slots;
}

// The page table's row stride.
int64_t check_pages(const Tensor& t, int64_t batch, int64_t page_size) {
  need(t.dim() == 2 && t.size(0) == batch && t.size(1) >= 1, "page_table must be [batch, max_pages]");
  need(rows_contiguous(t), "page_table rows must be contiguous");
  need(page_size >= MLA_FP8_BLOCK && page_size % MLA_FP8_BLOCK == 0 && page_size <= INT32_MAX,
       "page_size must be a multiple of 64");
  return batch > 1 ? t.stride(0) : t.size(1);  // one row: any stride
}

PyObject* status(int st) { return PyLong_FromLong(st); }
PyObject* pair(const Tensor& a, const Tensor& b) {
  PyObject* x = THPVariable_Wrap(a);
  PyObject* y = THPVariable_Wrap(b);
  return Py_BuildValue("(NN)", x, y);
}
int int32_of(int64_t v, const char* what) {
  need(v >= INT32_MIN && v <= INT32_MAX, what);
  return static_cast<int>(v);
}

PyObject* append(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  Args args{a, n};
  const Tensor &kv = args.tensor("kv_c", kBF16), &pe = args.tensor("k_pe", kBF16), &cs = args.tensor("cos_sin", kF32);
  const Tensor &cu = args.tensor("cu_seqlens", kI32), &ctx = args.tensor("context_lens", kI32);
  const Tensor &pt = args.tensor("page_table", kI32), &cache = args.tensor("cache", kF8);
  const Tensor& scales = args.tensor("scales", kF32);
  const int64_t page_size = args.integer();
  const bool interleaved = args.flag();
  const int64_t slots = check_cache(cache, scales);
  need(kv.dim() == 2 && kv.size(1) == MLA_D_LATENT && rows_contiguous(kv),
       "kv_c must be [T, 512] with a contiguous last dimension");
  const int64_t T = kv.size(0);
  need(pe.dim() == 2 && pe.size(0) == T && pe.size(1) == MLA_D_ROPE && rows_contiguous(pe),
       "k_pe must be [T, 64] with a contiguous last dimension");
  need(cs.dim() == 2 && cs.size(1) == 64 && cs.is_contiguous(), "cos_sin must be contiguous [max_position, 64]");
  need(cu.dim() == 1 && ctx.dim() == 1 && cu.is_contiguous() && ctx.is_contiguous(),
       "cu_seqlens and context_lens must be contiguous and one-dimensional");
  const int64_t B = ctx.size(0);
  need(cu.size(0) == B + 1, "cu_seqlens must have one entry more than context_lens");
  const int64_t pt_stride = check_pages(pt, B, page_size);
  int64_t H = 0, q_st = 0, q_sh = 0, o_st = 0, o_sh = 0;
  Tensor q, o;
  if (args.skip_none()) {
    need(args.skip_none(), "q_out goes with q_pe");
  } else {
    q = args.tensor("q_pe", kBF16);
    need(q.dim() == 3 && q.size(0) == T && q.size(2) == MLA_D_ROPE && q.size(1) >= 1 && rows_contiguous(q),
         "q_pe must be [T, H, 64] with a contiguous last dimension");
    if (args.skip_none()) {
      o = at::empty(q.sizes(), q.options());
    } else {
      o = args.tensor("q_out", kBF16);
      need(o.sizes() == q.sizes() && rows_contiguous(o), "q_out must have q_pe's shape and a contiguous last dimension");
    }
    H = q.size(1);
    // a dimension of one element may have any stride
    q_sh = H > 1 ? q.stride(1) : MLA_D_ROPE;
    o_sh = H > 1 ? o.stride(1) : MLA_D_ROPE;
    q_st = T > 1 ? q.stride(0) : std::max<int64_t>(MLA_D_ROPE, q_sh) * H;
    o_st = T > 1 ? o.stride(0) : std::max<int64_t>(MLA_D_ROPE, o_sh) * H;
  }
  const int64_t max_new = args.skip_none() ? T : args.integer();
  uint32_t* err = args.error_word();
  const Launch at(args.device);
  const int st = mla_nvfp4_fp8_cache_append(
      kv.data_ptr(), T > 1 ? kv.stride(0) : MLA_D_LATENT, pe.data_ptr(), T > 1 ? pe.stride(0) : MLA_D_ROPE, T,
      data<float>(cs), cs.size(0), interleaved ? 1 : 0, data<int32_t>(cu), data<int32_t>(ctx),
      int32_of(B, "too many sequences"), int32_of(max_new, "max_new_tokens out of range"), data<int32_t>(pt), pt_stride,
      pt.size(1), static_cast<int>(page_size), data<uint8_t>(cache), slots, data<float>(scales),
      H > 0 ? q.data_ptr() : nullptr, q_st, q_sh, H > 0 ? o.data_ptr() : nullptr, o_st, o_sh, int32_of(H, "too many heads"), err, at.stream);
  if (st != MLA_OK) return status(st);
  if (H > 0) return THPVariable_Wrap(o);
  Py_RETURN_NONE;
  END_HANDLE_TH_ERRORS
}

PyObject* decode(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  Args args{a, n};
  const Tensor &q = args.tensor("q", kBF16), &cache = args.tensor("cache", kF8), &scales = args.tensor("scales", kF32);
  const float softmax_scale = static_cast<float>(args.number());
  const Tensor &pt = args.tensor("page_table", kI32), &lens = args.tensor("seq_lens", kI32);
  const int64_t page_size = args.integer();
  const int64_t slots = check_cache(cache, scales);
  need(q.dim() == 3 && q.size(2) == MLA_D_QK_DECODE && q.is_contiguous(), "q must be contiguous [B, H, 576]");
  const int64_t B = q.size(0), H = q.size(1);
  const int64_t pt_stride = check_pages(pt, B, page_size);
  need(lens.dim() == 1 && lens.size(0) == B && lens.is_contiguous(), "seq_lens must be contiguous [B]");
  const int b = int32_of(B, "batch too large"), h = int32_of(H, "too many heads");
  const Tensor out = args.output("out", kBF16, {B, H, MLA_D_LATENT});
  PyObject* lse_given = args.next();
  PyObject* ws_given = args.next();
  const bool split = args.flag();
  uint32_t* err = args.error_word();
  const bool return_lse = args.flag();
  Tensor lse, ws;
  if (return_lse || lse_given != Py_None) {
    Args one{&lse_given, 1, 0, args.device};
    lse = one.output("lse", kF32, {B, H});
  }
  const Launch at(args.device);
  if (ws_given != Py_None) {
    need(split, "split=False takes no workspace");
    Args one{&ws_given, 1, 0, args.device};
    ws = one.tensor("workspace", at::kByte);
    need(ws.is_contiguous(), "workspace must be contiguous");
  } else if (split && B > 0 && H > 0) {
    ws = at::empty({static_cast<int64_t>(mla_nvfp4_fp8_decode_workspace_size(b, h))}, q.options().dtype(at::kByte));
  }
  const int st = mla_nvfp4_fp8_decode(q.data_ptr(), b, h, bytes(cache), slots, data<float>(scales), data<int32_t>(pt),
                                      pt_stride, pt.size(1), static_cast<int>(page_size), data<int32_t>(lens),
                                      softmax_scale, out.data_ptr(), lse.defined() ? data<float>(lse) : nullptr,
                                      ws.defined() ? ws.data_ptr() : nullptr, ws.defined() ? ws.numel() : 0, err,
                                      at.stream);
  if (st != MLA_OK) return status(st);
  return return_lse ? pair(out, lse) : THPVariable_Wrap(out);
  END_HANDLE_TH_ERRORS
}

PyObject* quantize(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  Args args{a, n};
  const Tensor& x = args.tensor("x", kBF16);
  need(x.dim() == 2 && rows_contiguous(x), "x must be [M, K] with a contiguous last dimension");
  const int64_t M = x.size(0), K = x.size(1);
  const Tensor codes = args.output("codes", kF8, {M, K});
  const Tensor scales = args.output("scales", kF32, {M, (K + MLA_FP8_GROUP - 1) / MLA_FP8_GROUP});
  const Launch at(args.device);
  const int st = mla_nvfp4_fp8_quantize(x.data_ptr(), M > 1 ? x.stride(0) : K, M, K, data<uint8_t>(codes),
                                        data<float>(scales), at.stream);
  return st != MLA_OK ? status(st) : pair(codes, scales);
  END_HANDLE_TH_ERRORS
}

PyObject* gemm(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  Args args{a, n};
  const Tensor &x = args.tensor("a", kF8), &xs = args.tensor("a_scales", kF32);
  const Tensor &w = args.tensor("w", kF8), &ws = args.tensor("w_scales", kF32);
  need(x.dim() == 2 && w.dim() == 2 && x.size(1) == w.size(1) && rows_contiguous(x) && rows_contiguous(w),
       "a [M, K] and w [N, K] must share K, with a contiguous last dimension");
  const int64_t M = x.size(0), K = x.size(1), N = w.size(0), kb = (K + MLA_FP8_GROUP - 1) / MLA_FP8_GROUP;
  need(xs.dim() == 2 && xs.size(0) == M && xs.size(1) == kb && xs.is_contiguous(),
       "a_scales must be contiguous [M, ceil(K / 128)]");
  need(ws.dim() == 2 && ws.size(0) == (N + MLA_FP8_GROUP - 1) / MLA_FP8_GROUP && ws.size(1) == kb && ws.is_contiguous(),
       "w_scales must be contiguous [ceil(N / 128), ceil(K / 128)]");
  Tensor out;
  if (args.skip_none()) {
    out = at::empty({M, N}, x.options().dtype(kBF16));
  } else {
    out = args.tensor("out", kBF16);
    need(out.dim() == 2 && out.size(0) == M && out.size(1) == N && rows_contiguous(out),
         "out must be [M, N] with a contiguous last dimension");
  }
  uint32_t* err = args.error_word();
  const Launch at(args.device);
  // one row: any stride
  const int st = mla_nvfp4_fp8_gemm(bytes(x), M > 1 ? x.stride(0) : K, data<float>(xs), M, bytes(w),
                                    N > 1 ? w.stride(0) : K, data<float>(ws), N, K, out.data_ptr(),
                                    M > 1 ? out.stride(0) : N, err, at.stream);
  return st != MLA_OK ? status(st) : THPVariable_Wrap(out);
  END_HANDLE_TH_ERRORS
}

#define METHOD(f) {#f, reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(f)), METH_FASTCALL, nullptr}
PyMethodDef methods[] = {METHOD(append), METHOD(decode), METHOD(quantize), METHOD(gemm), {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_mla_fp8", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__mla_fp8() { return PyModule_Create(&module); }
