// binding.cpp -- the usual call of an expert operator in one native step.
//
// A product or a dispatch of a few tokens runs for 2 to 7 us on the GPU; the
// checks, the allocation and the ctypes call of ops.py take 8 to 11 us of the
// host.  The functions here do the same for the call that most programs make:
// contiguous CUDA tensors of the right types and shapes on the current device,
// the current stream, outputs to be allocated.
// For any other call, and for one that the library refuses, they return None
// and ops.py goes its own way, which also says what is wrong.
//
// The library's entry points come from ops.py as addresses, so that this module
// and the rest of the package use one copy of it.
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/custom_function.h>
#include <torch/csrc/autograd/functions/basic_ops.h>
#include <torch/csrc/autograd/functions/utils.h>
#include <torch/csrc/autograd/python_variable.h>
#include <ATen/cuda/EmptyTensor.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <c10/core/GradMode.h>

#include "trace_fp4.h"

namespace {

struct {
  decltype(&trace_moe_sort) sort;
  decltype(&trace_moe_sort_workspace_bytes) sort_bytes;
  decltype(&trace_moe_dispatch) dispatch;
  decltype(&trace_moe_combine) combine;
  decltype(&trace_moe_combine_bwd) combine_bwd;
  decltype(&trace_fp4_matmul) nv;
  decltype(&trace_mx_matmul) mx;
  decltype(&trace_fp4_matmul_workspace_bytes) nv_bytes;
  decltype(&trace_mx_matmul_workspace_bytes) mx_bytes;
} lib;

// A contiguous tensor of `type` on device `index`, or null.
const at::Tensor* usual(PyObject* o, at::ScalarType type, int index) {
  if (index < 0 || !THPVariable_Check(o)) return nullptr;
  const at::Tensor& t = THPVariable_Unpack(o);
  return t.scalar_type() == type && t.layout() == at::kStrided && t.is_cuda() &&
                 t.get_device() == index && t.is_contiguous()
             ? &t
             : nullptr;
}

// Whether a call has to go through the autograd function: to record it, or, with
// a tangent of forward-mode differentiation (which no_grad leaves on), for that
// function to refuse it.
bool needs_grad(const at::Tensor& t) {
  return (c10::GradMode::is_enabled() && t.requires_grad()) || t._fw_grad(/*level=*/0).defined();
}

void* at_of(const at::Tensor& t) { return t.data_ptr(); }

// A library call without the interpreter's lock (a launch may wait for room in
// the stream's queue).
template <typename F>
auto unlocked(F&& f) {
  const pybind11::gil_scoped_release no_lock;
  return f();
}

bool starts(const at::Tensor& t) { return (uintptr_t)at_of(t) % 32 == 0; }

at::Tensor empty(at::IntArrayRef size, at::ScalarType type, int index) {
  return at::detail::empty_cuda(size, type, at::Device(at::kCUDA, (c10::DeviceIndex)index),
                                std::nullopt);
}

// A part of a tensor's memory as a tensor of its own.
at::Tensor part(const at::Tensor& of, int64_t offset, at::IntArrayRef size) {
  at::Tensor t = at::detail::make_tensor<c10::TensorImpl>(c10::Storage(of.storage()), of.key_set(),
                                                          of.dtype());
  t.unsafeGetTensorImpl()->set_storage_offset(offset);
  t.unsafeGetTensorImpl()->set_sizes_contiguous(size);
  return t;
}

void* stream_of(int index) {
  return c10::cuda::getCurrentCUDAStream((c10::DeviceIndex)index).stream();
}

// The current device, if the tensor is on it; else -1 (nothing is asked of CUDA
// for tensors of the host).
int device_of(PyObject* o) {
  if (!THPVariable_Check(o) || !THPVariable_Unpack(o).is_cuda()) return -1;
  const int index = THPVariable_Unpack(o).get_device();
  return index == (int)c10::cuda::current_device() ? index : -1;
}

PyObject* wrap(const at::Tensor& t) {
  if (!t.defined()) Py_RETURN_NONE;
  return THPVariable_Wrap(t);
}

// setup(address, ...) in the order of `lib`
PyObject* setup(PyObject*, PyObject* const* args, Py_ssize_t n) {
  constexpr Py_ssize_t entries = sizeof(lib) / sizeof(void*);
  if (n != entries) {
    PyErr_SetString(PyExc_TypeError, "setup: one address for each entry point");
    return nullptr;
  }
  for (Py_ssize_t i = 0; i < entries; ++i) {
    void* p = PyLong_AsVoidPtr(args[i]);
    if (p == nullptr) {
      if (!PyErr_Occurred()) PyErr_SetString(PyExc_ValueError, "setup: a null address");
      return nullptr;
    }
    memcpy((char*)&lib + i * sizeof(void*), &p, sizeof(void*));
  }
  Py_RETURN_NONE;
}

// Rows of an operand's codes and its scales' layout; false if they do not fit:
// [rows, cols / block] row-major, or flat in the tiled layout.
bool operand(const at::Tensor& codes, const at::Tensor& scales, int64_t cols, int64_t block,
             int64_t* rows, int* layout) {
  *rows = codes.numel() * 2 / cols;
  if (*rows * cols != codes.numel() * 2) return false;
  const int64_t c = cols / block;
  if (scales.dim() == 2) {
    *layout = TRACE_SCALES_ROW_MAJOR;
    return scales.size(0) == *rows && scales.size(1) == c;
  }
  *layout = TRACE_SCALES_TILED_128x4;
  return scales.dim() == 1 && scales.numel() == (*rows + 127) / 128 * ((c + 3) / 4) * 512;
}

// matmul(block, cols, matrices, offsets, a_codes, a_scales, a_gscale, w_codes, w_scales, w_gscale)
PyObject* matmul(PyObject*, PyObject* const* args, Py_ssize_t n_args) {
  HANDLE_TH_ERRORS
  if (n_args != 10) Py_RETURN_NONE;
  const long block = PyLong_AsLong(args[0]);
  const long long cols = PyLong_AsLongLong(args[1]), matrices = PyLong_AsLongLong(args[2]);
  if (PyErr_Occurred()) {
    PyErr_Clear();
    Py_RETURN_NONE;
  }
  const bool mx = block == 32;
  if ((block != 16 && block != 32) || cols <= 0 || cols % 32 != 0 || cols >= (1ll << 31) ||
      matrices < 1 || matrices > TRACE_MATMUL_MAX_GROUPS)
    Py_RETURN_NONE;
  const int index = device_of(args[4]);
  const at::Tensor* ac = usual(args[4], at::kByte, index);
  const at::Tensor* as = usual(args[5], at::kByte, index);
  const at::Tensor* wc = usual(args[7], at::kByte, index);
  const at::Tensor* ws = usual(args[8], at::kByte, index);
  const bool grouped = args[3] != Py_None;
  const at::Tensor* offs = grouped ? usual(args[3], at::kLong, index) : nullptr;
  if (!ac || !as || !wc || !ws || (grouped && !offs)) Py_RETURN_NONE;
  int64_t rows, wrows, groups = grouped ? offs->numel() - 1 : 1;
  int la, lw;
  if (!operand(*ac, *as, cols, block, &rows, &la) || !operand(*wc, *ws, cols, block, &wrows, &lw) ||
      wrows == 0 || wrows % matrices != 0 || groups < 1 || groups > TRACE_MATMUL_MAX_GROUPS)
    Py_RETURN_NONE;
  const at::Tensor *ga = nullptr, *gw = nullptr;
  if (!mx) {
    ga = usual(args[6], at::kFloat, index);
    gw = usual(args[9], at::kFloat, index);
    if (!ga || !gw || ga->dim() != 1 || gw->dim() != 1 || ga->numel() != groups ||
        gw->numel() != matrices)
      Py_RETURN_NONE;
  }
  const int64_t n = wrows / matrices;
  const int32_t g = (int32_t)groups, m = (int32_t)matrices;
  if ((mx ? lib.mx_bytes : lib.nv_bytes)(rows, cols, g, la, n, m, lw) != 0) Py_RETURN_NONE;
  const at::Tensor out = empty({rows, n}, at::kBFloat16, index);
  const int64_t* fp = grouped ? (const int64_t*)at_of(*offs) : nullptr;
  const uint8_t *pac = (const uint8_t*)at_of(*ac), *pas = (const uint8_t*)at_of(*as);
  const uint8_t *pwc = (const uint8_t*)at_of(*wc), *pws = (const uint8_t*)at_of(*ws);
  const float *pga = mx ? nullptr : (const float*)at_of(*ga);
  const float *pgw = mx ? nullptr : (const float*)at_of(*gw);
  uint16_t* po = (uint16_t*)at_of(out);
  void* stream = stream_of(index);
  const int st = unlocked([&] {
    return mx ? lib.mx(pac, pas, rows, cols, g, fp, la, pwc, pws, n, m, lw, po, stream)
              : lib.nv(pac, pas, pga, rows, cols, g, fp, la, pwc, pws, pgw, n, m, lw, po, stream);
  });
  return wrap(st == TRACE_OK ? out : at::Tensor());
  END_HANDLE_TH_ERRORS
}

// A route's row numbers [tokens, k] and its slots.
bool route(PyObject* rows, PyObject* slots, int index, const at::Tensor** r, const at::Tensor** s) {
  *r = usual(rows, at::kInt, index);
  if (!*r || (*r)->dim() != 2 || (*r)->size(1) < 1) return false;
  *s = usual(slots, at::kInt, index);
  return *s && (*s)->dim() == 1 && (*s)->numel() == (*r)->numel();
}

// What the token kernels take: bf16 [tokens, cols] that they can read 32 bytes at a time.
bool tokens_of(const at::Tensor* x) {
  return x && x->dim() == 2 && x->size(1) > 0 && x->size(1) % 32 == 0 && starts(*x);
}

// Undefined where the library refuses.
at::Tensor dispatch_fwd(const at::Tensor& x, const at::Tensor& rows, const at::Tensor& slots) {
  const int index = x.get_device();
  const int64_t tokens = rows.size(0), k = rows.size(1), cols = x.size(1);
  at::Tensor y = empty({tokens * k, cols}, at::kBFloat16, index);
  const int st = lib.dispatch((const uint16_t*)at_of(x), tokens, k, cols, (const int32_t*)at_of(rows),
                              (const int32_t*)at_of(slots), (uint16_t*)at_of(y), stream_of(index));
  return st == TRACE_OK ? y : at::Tensor();
}

at::Tensor combine_fwd(const at::Tensor& y, const at::Tensor& rows, const at::Tensor* weights) {
  const int index = y.get_device();
  const int64_t tokens = rows.size(0), k = rows.size(1), cols = y.size(1);
  at::Tensor out = empty({tokens, cols}, at::kBFloat16, index);
  const int st = lib.combine((const uint16_t*)at_of(y), tokens, k, cols, (const int32_t*)at_of(rows),
                             weights ? (const float*)at_of(*weights) : nullptr,
                             (uint16_t*)at_of(out), stream_of(index));
  return st == TRACE_OK ? out : at::Tensor();
}

using torch::autograd::AutogradContext;
using torch::autograd::variable_list;

// A gradient as the kernels read it: parts of a larger one may start anywhere.
at::Tensor upstream(const at::Tensor& grad) {
  at::NoGradGuard no_grad;
  const at::Tensor g = grad.contiguous();
  return starts(g) ? g : g.clone();
}

// The kernels are not differentiated again: a second derivative is an error.
template <typename... T>
void once(variable_list outputs, const T&... inputs) {
  if (!torch::autograd::compute_requires_grad(inputs...)) return;
  torch::autograd::set_history(
      outputs, std::make_shared<torch::autograd::Error>(
                   "the gradients of moe_dispatch and moe_combine cannot be differentiated",
                   torch::autograd::collect_next_edges(inputs...)));
}

struct Dispatch : torch::autograd::Function<Dispatch> {
  static at::Tensor forward(AutogradContext* ctx, const at::Tensor& x, const at::Tensor& rows,
                            const at::Tensor& slots) {
    at::Tensor y = dispatch_fwd(x, rows, slots);
    TORCH_CHECK(y.defined(), "trace_moe_dispatch");
    ctx->save_for_backward({rows});
    return y;
  }
  static variable_list backward(AutogradContext* ctx, const variable_list& grads) {
    const at::Tensor rows = ctx->get_saved_variables()[0], g = upstream(grads[0]);
    const c10::cuda::CUDAGuard on(g.device());
    at::Tensor dx = combine_fwd(g, rows, nullptr);
    TORCH_CHECK(dx.defined(), "trace_moe_combine failed in a backward pass");
    once({dx}, grads[0]);
    return {dx, at::Tensor(), at::Tensor()};
  }
};

struct Combine : torch::autograd::Function<Combine> {
  static at::Tensor forward(AutogradContext* ctx, const at::Tensor& y, const at::Tensor& rows,
                            const at::Tensor& slots, const at::Tensor& weights) {
    at::Tensor out = combine_fwd(y, rows, &weights);
    TORCH_CHECK(out.defined(), "trace_moe_combine");
    ctx->save_for_backward({y, rows, slots, weights});
    return out;
  }
  static variable_list backward(AutogradContext* ctx, const variable_list& grads) {
    const variable_list saved = ctx->get_saved_variables();
    const at::Tensor &y = saved[0], &rows = saved[1], &slots = saved[2], &w = saved[3];
    const at::Tensor g = upstream(grads[0]);
    const c10::cuda::CUDAGuard on(g.device());
    const int index = g.get_device();
    const int64_t tokens = rows.size(0), k = rows.size(1), cols = y.size(1);
    at::Tensor dy = empty({tokens * k, cols}, at::kBFloat16, index);
    at::Tensor dw = empty({tokens, k}, at::kFloat, index);
    const int st = lib.combine_bwd(
        (const uint16_t*)at_of(g), (const uint16_t*)at_of(y), tokens, k, cols,
        (const int32_t*)at_of(rows), (const int32_t*)at_of(slots), (const float*)at_of(w),
        (uint16_t*)at_of(dy), (float*)at_of(dw), stream_of(index));
    TORCH_CHECK(st == TRACE_OK, "trace_moe_combine_bwd failed in a backward pass");
    once({dy, dw}, grads[0], y, w);
    return {dy, at::Tensor(), at::Tensor(), dw};
  }
};

// dispatch(x, rows, slots)
PyObject* dispatch(PyObject*, PyObject* const* args, Py_ssize_t n_args) {
  HANDLE_TH_ERRORS
  if (n_args != 3) Py_RETURN_NONE;
  const int index = device_of(args[0]);
  const at::Tensor *x = usual(args[0], at::kBFloat16, index), *rows, *slots;
  if (!tokens_of(x) || !route(args[1], args[2], index, &rows, &slots) ||
      rows->size(0) != x->size(0))
    Py_RETURN_NONE;
  return wrap(unlocked([&] {
    return needs_grad(*x) ? Dispatch::apply(*x, *rows, *slots) : dispatch_fwd(*x, *rows, *slots);
  }));
  END_HANDLE_TH_ERRORS
}

// combine(y, rows, slots, weights)
PyObject* combine(PyObject*, PyObject* const* args, Py_ssize_t n_args) {
  HANDLE_TH_ERRORS
  if (n_args != 4) Py_RETURN_NONE;
  const int index = device_of(args[0]);
  const at::Tensor *y = usual(args[0], at::kBFloat16, index), *rows, *slots;
  const at::Tensor* w = usual(args[3], at::kFloat, index);
  if (!tokens_of(y) || !w || !route(args[1], args[2], index, &rows, &slots) ||
      rows->numel() != y->size(0) || w->sizes() != rows->sizes())
    Py_RETURN_NONE;
  return wrap(unlocked([&] {
    return needs_grad(*y) || needs_grad(*w) ? Combine::apply(*y, *rows, *slots, *w)
                                            : combine_fwd(*y, *rows, w);
  }));
  END_HANDLE_TH_ERRORS
}

// sort(ids, num_experts) -> (offsets, rows, slots)
PyObject* sort(PyObject*, PyObject* const* args, Py_ssize_t n_args) {
  HANDLE_TH_ERRORS
  if (n_args != 2) Py_RETURN_NONE;
  const long experts = PyLong_AsLong(args[1]);
  if (PyErr_Occurred()) {
    PyErr_Clear();
    Py_RETURN_NONE;
  }
  const int index = device_of(args[0]);
  const at::Tensor* ids = usual(args[0], at::kLong, index);
  if (!ids) ids = usual(args[0], at::kInt, index);
  if (!ids || ids->dim() != 2 || experts < 1 || experts > TRACE_MOE_MAX_EXPERTS) Py_RETURN_NONE;
  const int64_t tokens = ids->size(0), k = ids->size(1);
  const size_t bytes = lib.sort_bytes(tokens, k, (int32_t)experts);
  if (bytes == 0) Py_RETURN_NONE;
  // rows and slots share an allocation, with a small workspace in front of them
  // (an allocation is 0.5 of the 5.5 us that this call takes)
  const int64_t n = tokens * k, head = bytes <= 256 ? (int64_t)bytes / 4 : 0;
  const at::Tensor offsets = empty({experts + 2}, at::kLong, index);
  const at::Tensor words = empty({head + 2 * n}, at::kInt, index);
  const at::Tensor rows = part(words, head, {tokens, k}), slots = part(words, head + n, {n});
  const at::Tensor ws = head ? words : empty({(int64_t)bytes}, at::kByte, index);
  const void* pi = at_of(*ids);
  const int32_t width = (int32_t)ids->element_size();
  int64_t* po = (int64_t*)at_of(offsets);
  int32_t *pr = (int32_t*)at_of(rows), *ps = (int32_t*)at_of(slots);
  void *pw = at_of(ws), *stream = stream_of(index);
  const int st = unlocked([&] {
    return lib.sort(pi, width, tokens, k, (int32_t)experts, po, pr, ps, pw, bytes, stream);
  });
  if (st != TRACE_OK) Py_RETURN_NONE;
  PyObject* got = PyTuple_New(3);
  if (got == nullptr) return nullptr;
  PyTuple_SET_ITEM(got, 0, THPVariable_Wrap(offsets));
  PyTuple_SET_ITEM(got, 1, THPVariable_Wrap(rows));
  PyTuple_SET_ITEM(got, 2, THPVariable_Wrap(slots));
  return got;
  END_HANDLE_TH_ERRORS
}

PyMethodDef methods[] = {
    {"setup", (PyCFunction)(void*)setup, METH_FASTCALL, "Addresses of the library's entry points."},
    {"matmul", (PyCFunction)(void*)matmul, METH_FASTCALL, "Product of two captured operands."},
    {"dispatch", (PyCFunction)(void*)dispatch, METH_FASTCALL, "Tokens into expert order."},
    {"combine", (PyCFunction)(void*)combine, METH_FASTCALL, "Back to token order."},
    {"sort", (PyCFunction)(void*)sort, METH_FASTCALL, "Slots sorted by expert."},
    {nullptr, nullptr, 0, nullptr}};

PyModuleDef module = {PyModuleDef_HEAD_INIT, "_binding", nullptr, -1, methods};

}  // namespace

PyMODINIT_FUNC PyInit__binding() { return PyModule_Create(&module); }
