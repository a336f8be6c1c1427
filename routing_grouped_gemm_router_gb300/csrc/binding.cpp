// binding.cpp — the training operators on torch tensors, as a CPython extension (host code only).
//
// The operators' kernels take a few microseconds on small batches, where a call's cost is its
// host side: checks, output allocation, marshalling. Through ctypes a residual join of one token
// took 18.8 us a call, from here 7; every function checks its tensors (ValueError, by argument
// name), allocates its outputs from PyTorch's caching allocator on the current stream of their
// device, and calls the C entry point of libmoe_gb300.so, whose non-OK status raises MoeError.
// What the operators compute is said in include/moe_train.h; the Python functions with their
// documentation are in training.py.
#include <Python.h>

#include <ATen/core/Tensor.h>
#include <ATen/cuda/EmptyTensor.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Dtype.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <initializer_list>
#include <string>

#include "moe_train.h"

namespace {

using at::ScalarType;
using at::Tensor;

PyObject* g_moe_error = nullptr;  // _lib.MoeError

struct Refused {  // an argument that does not fit: becomes a ValueError
  std::string what;
};
struct Failed {  // a status of the C entry point: becomes a MoeError
  const char* fn;
  moe_status_t status;
};

constexpr ScalarType kAnyFloat = ScalarType::Undefined;  // bf16 or fp32
constexpr ScalarType kF32 = ScalarType::Float, kI32 = ScalarType::Int;

std::string name_of(ScalarType t) {
  switch (t) {
    case ScalarType::BFloat16: return "torch.bfloat16";
    case ScalarType::Float: return "torch.float32";
    case ScalarType::Int: return "torch.int32";
    case ScalarType::Long: return "torch.int64";
    case ScalarType::Half: return "torch.float16";
    case ScalarType::Double: return "torch.float64";
    default: return std::string("torch.") + c10::toString(t);
  }
}
template <typename R>
std::string list_of(const R& v) {
  std::string s = "(";
  for (int64_t d : v) s += (s.size() > 1 ? ", " : "") + (d < 0 ? std::string("any") : std::to_string(d));
  return s + ")";
}
bool is_float(ScalarType t) { return t == ScalarType::BFloat16 || t == ScalarType::Float; }

// The calling thread's device, where the library launches: another device's tensors are not this call's.
int current_device() {
  c10::DeviceIndex d = -1;
  return c10::cuda::GetDevice(&d) == cudaSuccess ? d : -1;
}

// A contiguous CUDA tensor of these extents (-1: any), type and device (-1: the current one, for an
// operator's first tensor). The fast way through is a handful of comparisons; only a tensor that does
// not fit is described.
const Tensor& check(const char* name, PyObject* o, std::initializer_list<int64_t> shape,
                    ScalarType type, int dev) {
  if (!THPVariable_Check(o))
    throw Refused{std::string(name) + ": a tensor is needed, got " + Py_TYPE(o)->tp_name};
  const Tensor& t = THPVariable_Unpack(o);
  const ScalarType st = t.scalar_type();
  if (type == kAnyFloat ? !is_float(st) : st != type)
    throw Refused{std::string(name) + ": dtype " + name_of(st) + ", expected " +
                  (type == kAnyFloat ? "bfloat16 or float32" : name_of(type))};
  bool fits = t.dim() == (int64_t)shape.size();
  if (fits) {
    int64_t i = 0;
    for (int64_t d : shape) {
      fits &= d < 0 || d == t.size(i);
      ++i;
    }
  }
  if (!fits)
    throw Refused{std::string(name) + ": shape " + list_of(t.sizes()) + ", expected " + list_of(shape)};
  if (!t.is_contiguous())
    throw Refused{std::string(name) + ": has to be contiguous (strides " + list_of(t.strides()) + ")"};
  if (!t.is_cuda()) throw Refused{std::string(name) + ": has to be on a CUDA device"};
  if (dev >= 0 && t.get_device() != dev)
    throw Refused{std::string(name) + ": is on another device than the other tensors"};
  if (dev < 0 && t.get_device() != current_device())
    throw Refused{std::string(name) + ": is on cuda:" + std::to_string(t.get_device()) +
                  ", which is not the current device"};
  return t;
}

Tensor empty(at::IntArrayRef shape, ScalarType type, const Tensor& like) {
  return Tensor(at::detail::empty_cuda(shape, type, like.device(), std::nullopt));
}
Tensor empty_as(const Tensor& like) { return empty(like.sizes(), like.scalar_type(), like); }

cudaStream_t stream_of(const Tensor& t) {
  return c10::cuda::getCurrentCUDAStream(t.get_device()).stream();
}
moe_dtype_t dtype_of(const Tensor& t) {
  return t.scalar_type() == ScalarType::BFloat16 ? MOE_BF16 : MOE_F32;
}
int narrow(const char* name, int64_t v) {  // extents beyond 32 bits are no sizes of these operators
  if (v > INT32_MAX || v < 0) throw Refused{std::string(name) + ": an extent of " + std::to_string(v)};
  return (int)v;
}
void done(const char* fn, moe_status_t st) {
  if (st != MOE_OK) throw Failed{fn, st};
}

int64_t integer(PyObject* o) {
  const long long v = PyLong_AsLongLong(o);
  if (v == -1 && PyErr_Occurred()) throw python_error();
  return v;
}
float number(PyObject* o) {
  const double v = PyFloat_AsDouble(o);
  if (v == -1.0 && PyErr_Occurred()) throw python_error();
  return (float)v;
}
bool given(PyObject* o) { return o != Py_None; }
void* ptr(const Tensor& t) { return t.data_ptr(); }
float* fptr(const Tensor& t) { return (float*)t.data_ptr(); }
int32_t* iptr(const Tensor& t) { return (int32_t*)t.data_ptr(); }

PyObject* wrap(const Tensor& t) { return THPVariable_Wrap(t); }
// A new tuple of tensors; undefined ones become None.
PyObject* tuple(std::initializer_list<Tensor> ts) {
  PyObject* r = PyTuple_New((Py_ssize_t)ts.size());
  if (!r) throw python_error();
  Py_ssize_t i = 0;
  for (const Tensor& t : ts) {
    PyObject* o = t.defined() ? wrap(t) : Py_NewRef(Py_None);
    PyTuple_SET_ITEM(r, i++, o);
  }
  return r;
}

// Runs an operator's body; C++ exceptions become Python's.
template <typename F>
PyObject* guarded(Py_ssize_t n, Py_ssize_t want, F body) {
  HANDLE_TH_ERRORS
  if (n != want) {
    PyErr_Format(PyExc_TypeError, "expected %zd arguments, got %zd", want, n);
    return nullptr;
  }
  try {
    return body();
  } catch (const Refused& r) {
    PyErr_SetString(PyExc_ValueError, r.what.c_str());
  } catch (const Failed& f) {
    PyObject* e = g_moe_error ? PyObject_CallFunction(g_moe_error, "si", f.fn, (int)f.status) : nullptr;
    if (e) {
      PyErr_SetObject(g_moe_error, e);
      Py_DECREF(e);
    } else if (!PyErr_Occurred()) {
      PyErr_Format(PyExc_RuntimeError, "%s failed: %d", f.fn, (int)f.status);
    }
  }
  return nullptr;
  END_HANDLE_TH_ERRORS
}

#define OPERATOR(name) PyObject* name(PyObject*, PyObject* const* a, Py_ssize_t n)

// ------------------------------------------------------------------------------ dispatch
OPERATOR(sort_tokens) {  // topk_ids, E -> sorted_ids, expert_ids, num_post_padded, counts
  return guarded(n, 2, [&]() -> PyObject* {
    const Tensor& ids = check("topk_ids", a[0], {-1, -1}, kI32, -1);
    const int T = narrow("topk_ids", ids.size(0)), k = narrow("topk_ids", ids.size(1));
    const int E = narrow("E", integer(a[1]));
    const int64_t P = moe_max_padded_rows(T, k, E, MOE_TRAIN_BLOCK);
    if (P <= 0 || E < k)
      throw Refused{"topk_ids: " + std::to_string(T) + " tokens, " + std::to_string(k) + " of " +
                    std::to_string(E) + " experts"};
    size_t ws = 0;
    done("moe_align_workspace_size", moe_align_workspace_size(T, k, E, MOE_TRAIN_BLOCK, &ws));
    const Tensor sid = empty({P}, kI32, ids), eid = empty({P / MOE_TRAIN_BLOCK}, kI32, ids);
    const Tensor npp = empty({1}, kI32, ids), counts = empty({E}, kI32, ids);
    Tensor scratch;
    if (ws) scratch = empty({(int64_t)((ws + 3) / 4)}, kI32, ids);
    done("moe_align", moe_align(iptr(ids), T, k, E, MOE_TRAIN_BLOCK, iptr(sid), iptr(eid), iptr(npp),
                                iptr(counts), ws ? ptr(scratch) : nullptr, ws, stream_of(ids)));
    return tuple({sid, eid, npp, counts});
  });
}

OPERATOR(permute) {  // x, topk_ids, sorted_ids, E -> xs, row_pos
  return guarded(n, 4, [&]() -> PyObject* {
    const Tensor& x = check("x", a[0], {-1, -1}, kAnyFloat, -1);
    const int dev = x.get_device();
    const Tensor& ids = check("topk_ids", a[1], {x.size(0), -1}, kI32, dev);
    const Tensor& sid = check("sorted_ids", a[2], {-1}, kI32, dev);
    const Tensor xs = empty({sid.size(0), x.size(1)}, x.scalar_type(), x), pos = empty_as(ids);
    done("moe_permute", moe_permute(ptr(x), iptr(ids), iptr(sid), narrow("x", x.size(0)),
                                    narrow("topk_ids", ids.size(1)), narrow("E", integer(a[3])),
                                    narrow("x", x.size(1)), dtype_of(x), narrow("sorted_ids", sid.size(0)),
                                    ptr(xs), iptr(pos), stream_of(x)));
    return tuple({xs, pos});
  });
}

OPERATOR(permute_backward) {  // dxs, row_pos -> dx
  return guarded(n, 2, [&]() -> PyObject* {
    const Tensor& dxs = check("dxs", a[0], {-1, -1}, kAnyFloat, -1);
    const Tensor& pos = check("row_pos", a[1], {-1, -1}, kI32, dxs.get_device());
    const Tensor dx = empty({pos.size(0), dxs.size(1)}, dxs.scalar_type(), dxs);
    done("moe_permute_backward",
         moe_permute_backward(ptr(dxs), iptr(pos), narrow("row_pos", pos.size(0)),
                              narrow("row_pos", pos.size(1)), narrow("dxs", dxs.size(1)), dtype_of(dxs),
                              narrow("dxs", dxs.size(0)), ptr(dx), stream_of(dxs)));
    return wrap(dx);
  });
}

OPERATOR(unpermute) {  // ys, row_pos, topk_w -> out
  return guarded(n, 3, [&]() -> PyObject* {
    const Tensor& ys = check("ys", a[0], {-1, -1}, kAnyFloat, -1);
    const int dev = ys.get_device();
    const Tensor& pos = check("row_pos", a[1], {-1, -1}, kI32, dev);
    const Tensor& w = check("topk_w", a[2], {pos.size(0), pos.size(1)}, kF32, dev);
    const Tensor out = empty({pos.size(0), ys.size(1)}, ys.scalar_type(), ys);
    done("moe_unpermute", moe_unpermute(ptr(ys), iptr(pos), fptr(w), narrow("row_pos", pos.size(0)),
                                        narrow("row_pos", pos.size(1)), narrow("ys", ys.size(1)),
                                        dtype_of(ys), narrow("ys", ys.size(0)), ptr(out), stream_of(ys)));
    return wrap(out);
  });
}

OPERATOR(unpermute_backward) {  // dout, ys, sorted_ids, row_pos, topk_w -> dys, dtopk_w
  return guarded(n, 5, [&]() -> PyObject* {
    const Tensor& ys = check("ys", a[1], {-1, -1}, kAnyFloat, -1);
    const int dev = ys.get_device();
    const Tensor& pos = check("row_pos", a[3], {-1, -1}, kI32, dev);
    const Tensor& dout = check("dout", a[0], {pos.size(0), ys.size(1)}, ys.scalar_type(), dev);
    const Tensor& sid = check("sorted_ids", a[2], {ys.size(0)}, kI32, dev);
    const Tensor& w = check("topk_w", a[4], {pos.size(0), pos.size(1)}, kF32, dev);
    const Tensor dys = empty_as(ys), dw = empty_as(w);
    done("moe_unpermute_backward",
         moe_unpermute_backward(ptr(dout), ptr(ys), iptr(sid), iptr(pos), fptr(w),
                                narrow("row_pos", pos.size(0)), narrow("row_pos", pos.size(1)),
                                narrow("ys", ys.size(1)), dtype_of(ys), narrow("ys", ys.size(0)), ptr(dys),
                                fptr(dw), stream_of(ys)));
    return tuple({dys, dw});
  });
}

// ------------------------------------------------------------------------------- experts
moe_experts_t experts(int64_t rows, int64_t E, int64_t H, int64_t I, const Tensor& t) {
  return {narrow("rows", rows), narrow("E", E), narrow("H", H), narrow("I", I), dtype_of(t)};
}
int64_t half(const char* name, int64_t two) {
  if (two % 2) throw Refused{std::string(name) + ": " + std::to_string(two) + " are no gate and up halves"};
  return two / 2;
}

OPERATOR(expert_up) {  // xs, W13, counts -> h13, act
  return guarded(n, 3, [&]() -> PyObject* {
    const Tensor& xs = check("xs", a[0], {-1, -1}, kAnyFloat, -1);
    const int dev = xs.get_device();
    const Tensor& W = check("W13", a[1], {-1, -1, xs.size(1)}, xs.scalar_type(), dev);
    const Tensor& cnt = check("counts", a[2], {W.size(0)}, kI32, dev);
    const int64_t I = half("W13", W.size(1));
    const moe_experts_t c = experts(xs.size(0), W.size(0), xs.size(1), I, xs);
    const Tensor h13 = empty({xs.size(0), 2 * I}, kF32, xs), act = empty({xs.size(0), I}, xs.scalar_type(), xs);
    done("moe_expert_up",
         moe_expert_up(&c, ptr(xs), ptr(W), iptr(cnt), fptr(h13), ptr(act), stream_of(xs)));
    return tuple({h13, act});
  });
}

OPERATOR(expert_down) {  // act, W2, counts -> ys
  return guarded(n, 3, [&]() -> PyObject* {
    const Tensor& act = check("act", a[0], {-1, -1}, kAnyFloat, -1);
    const int dev = act.get_device();
    const Tensor& W = check("W2", a[1], {-1, -1, act.size(1)}, act.scalar_type(), dev);
    const Tensor& cnt = check("counts", a[2], {W.size(0)}, kI32, dev);
    const moe_experts_t c = experts(act.size(0), W.size(0), W.size(1), act.size(1), act);
    const Tensor ys = empty({act.size(0), W.size(1)}, act.scalar_type(), act);
    done("moe_expert_down", moe_expert_down(&c, ptr(act), ptr(W), iptr(cnt), ptr(ys), stream_of(act)));
    return wrap(ys);
  });
}

OPERATOR(expert_down_backward) {  // dys, W2, h13, counts -> dh13, act
  return guarded(n, 4, [&]() -> PyObject* {
    const Tensor& dys = check("dys", a[0], {-1, -1}, kAnyFloat, -1);
    const int dev = dys.get_device();
    const Tensor& W = check("W2", a[1], {-1, dys.size(1), -1}, dys.scalar_type(), dev);
    const int64_t I = W.size(2);
    const Tensor& h13 = check("h13", a[2], {dys.size(0), 2 * I}, kF32, dev);
    const Tensor& cnt = check("counts", a[3], {W.size(0)}, kI32, dev);
    const moe_experts_t c = experts(dys.size(0), W.size(0), dys.size(1), I, dys);
    const Tensor dh = empty({dys.size(0), 2 * I}, dys.scalar_type(), dys);
    const Tensor act = empty({dys.size(0), I}, dys.scalar_type(), dys);
    done("moe_expert_down_backward",
         moe_expert_down_backward(&c, ptr(dys), ptr(W), fptr(h13), iptr(cnt), ptr(dh), ptr(act),
                                  stream_of(dys)));
    return tuple({dh, act});
  });
}

OPERATOR(expert_up_backward) {  // dh13, W13, counts -> dxs
  return guarded(n, 3, [&]() -> PyObject* {
    const Tensor& dh = check("dh13", a[0], {-1, -1}, kAnyFloat, -1);
    const int dev = dh.get_device();
    const Tensor& W = check("W13", a[1], {-1, dh.size(1), -1}, dh.scalar_type(), dev);
    const Tensor& cnt = check("counts", a[2], {W.size(0)}, kI32, dev);
    const moe_experts_t c = experts(dh.size(0), W.size(0), W.size(2), half("dh13", dh.size(1)), dh);
    const Tensor dxs = empty({dh.size(0), W.size(2)}, dh.scalar_type(), dh);
    done("moe_expert_up_backward",
         moe_expert_up_backward(&c, ptr(dh), ptr(W), iptr(cnt), ptr(dxs), stream_of(dh)));
    return wrap(dxs);
  });
}

OPERATOR(expert_weight_grad) {  // dy, a, counts, out or None, out_dtype or None, accumulate -> dW
  return guarded(n, 6, [&]() -> PyObject* {
    const Tensor& dy = check("dy", a[0], {-1, -1}, kAnyFloat, -1);
    const int dev = dy.get_device();
    const Tensor& x = check("a", a[1], {dy.size(0), -1}, dy.scalar_type(), dev);
    const Tensor& cnt = check("counts", a[2], {-1}, kI32, dev);
    const int accumulate = PyObject_IsTrue(a[5]);
    if (accumulate < 0) throw python_error();
    ScalarType type = given(a[3]) ? kAnyFloat : dy.scalar_type();
    if (given(a[4])) {
      if (!THPDtype_Check(a[4])) throw Refused{"out_dtype: a torch.dtype is needed"};
      type = reinterpret_cast<THPDtype*>(a[4])->scalar_type;
      if (!is_float(type)) throw Refused{"out_dtype: " + name_of(type) + ", expected bfloat16 or float32"};
    }
    const int64_t E = cnt.size(0), M = dy.size(1), N = x.size(1);
    if (accumulate && !given(a[3])) throw Refused{"accumulate: needs the tensor to add to (out)"};
    const Tensor dW = given(a[3]) ? check("out", a[3], {E, M, N}, type, dev) : empty({E, M, N}, type, dy);
    done("moe_expert_weight_grad",
         moe_expert_weight_grad(narrow("dy", dy.size(0)), narrow("counts", E), narrow("dy", M),
                                narrow("a", N), dtype_of(dy), dtype_of(dW), accumulate, ptr(dy), ptr(x),
                                iptr(cnt), ptr(dW), stream_of(dy)));
    if (given(a[3])) return Py_NewRef(a[3]);
    return wrap(dW);
  });
}

// ------------------------------------------------------------------- norms around the block
moe_block_t block(const Tensor& x, float scale, float offset, float eps) {
  moe_block_t c{};
  c.T = narrow("rows", x.size(0));
  c.H = narrow("H", x.size(1));
  c.dtype = dtype_of(x);
  c.gate_kind = MOE_GATE_NONE;
  c.scale = scale;
  c.offset = offset;
  c.eps = eps;
  return c;
}
// The gate, undefined for None, and its kind into c: fp32 [H], fp32 [T, 1] or [T, H] like x.
Tensor gate_of(PyObject* o, const Tensor& x, moe_block_t& c) {
  if (!given(o)) return Tensor();
  const int dev = x.get_device();
  if (THPVariable_Check(o)) {
    const Tensor& g = THPVariable_Unpack(o);
    if (g.dim() == 1) {
      c.gate_kind = MOE_GATE_CHANNEL;
      return check("gate", o, {x.size(1)}, kF32, dev);
    }
    if (g.dim() == 2 && g.size(1) == 1) {
      c.gate_kind = MOE_GATE_TOKEN;
      return check("gate", o, {x.size(0), 1}, kF32, dev);
    }
  }
  c.gate_kind = MOE_GATE_FULL;
  return check("gate", o, {x.size(0), x.size(1)}, x.scalar_type(), dev);
}
Tensor workspace(const moe_block_t& c, const Tensor& x, size_t& bytes) {
  done("moe_block_workspace_size", moe_block_workspace_size(&c, &bytes));
  return empty({(int64_t)bytes}, ScalarType::Byte, x);
}
void* maybe(const Tensor& t) { return t.defined() ? t.data_ptr() : nullptr; }
float* fmaybe(const Tensor& t) { return (float*)maybe(t); }

OPERATOR(block_norm) {  // x, gamma, eps, offset -> h, rstd
  return guarded(n, 4, [&]() -> PyObject* {
    const Tensor& x = check("x", a[0], {-1, -1}, kAnyFloat, -1);
    const Tensor& gamma = check("gamma", a[1], {x.size(1)}, kF32, x.get_device());
    const moe_block_t c = block(x, 1.f, number(a[3]), number(a[2]));
    const Tensor h = empty_as(x), r = empty({x.size(0)}, kF32, x);
    done("moe_block_norm", moe_block_norm(&c, ptr(x), fptr(gamma), ptr(h), fptr(r), stream_of(x)));
    return tuple({h, r});
  });
}

OPERATOR(block_norm_backward) {  // dh, x, gamma, rstd, dres or None, offset -> dx, dgamma
  return guarded(n, 6, [&]() -> PyObject* {
    const Tensor& x = check("x", a[1], {-1, -1}, kAnyFloat, -1);
    const int dev = x.get_device();
    const int64_t T = x.size(0), H = x.size(1);
    const Tensor& dh = check("dh", a[0], {T, H}, x.scalar_type(), dev);
    const Tensor& gamma = check("gamma", a[2], {H}, kF32, dev);
    const Tensor& r = check("rstd", a[3], {T}, kF32, dev);
    const Tensor dres = given(a[4]) ? check("dres", a[4], {T, H}, x.scalar_type(), dev) : Tensor();
    const moe_block_t c = block(x, 1.f, number(a[5]), 0.f);
    size_t bytes = 0;
    const Tensor ws = workspace(c, x, bytes), dx = empty_as(x), dg = empty_as(gamma);
    done("moe_block_norm_backward",
         moe_block_norm_backward(&c, ptr(dh), ptr(x), fptr(gamma), fptr(r), maybe(dres), ptr(dx), fptr(dg),
                                 ptr(ws), bytes, stream_of(x)));
    return tuple({dx, dg});
  });
}

OPERATOR(block_join) {  // x, y, gamma, gate, scale, gamma_next, eps, offset -> out, rstd_y, h, rstd_out
  return guarded(n, 8, [&]() -> PyObject* {
    const Tensor& x = check("x", a[0], {-1, -1}, kAnyFloat, -1);
    const int dev = x.get_device();
    const int64_t T = x.size(0), H = x.size(1);
    const Tensor& y = check("y", a[1], {T, H}, x.scalar_type(), dev);
    const Tensor& gamma = check("gamma", a[2], {H}, kF32, dev);
    moe_block_t c = block(x, number(a[4]), number(a[7]), number(a[6]));
    const Tensor gate = gate_of(a[3], x, c);
    Tensor gn, h, ro;
    const Tensor out = empty_as(x), ry = empty({T}, kF32, x);
    if (given(a[5])) {
      gn = check("gamma_next", a[5], {H}, kF32, dev);
      h = empty_as(x);
      ro = empty({T}, kF32, x);
    }
    done("moe_block_join", moe_block_join(&c, ptr(x), ptr(y), fptr(gamma), maybe(gate), fmaybe(gn), ptr(out),
                                          fptr(ry), maybe(h), fmaybe(ro), stream_of(x)));
    return tuple({out, ry, h, ro});
  });
}

// dres, y, gamma, rstd_y, gate, scale, dh, out, gamma_next, rstd_out, offset
//   -> dx, dy, dgamma, dgamma_next, dgate
OPERATOR(block_join_backward) {
  return guarded(n, 11, [&]() -> PyObject* {
    const Tensor& y = check("y", a[1], {-1, -1}, kAnyFloat, -1);
    const int dev = y.get_device();
    const int64_t T = y.size(0), H = y.size(1);
    const ScalarType type = y.scalar_type();
    const Tensor& gamma = check("gamma", a[2], {H}, kF32, dev);
    const Tensor& ry = check("rstd_y", a[3], {T}, kF32, dev);
    Tensor dres, dh, out, gn, ro, dgn, dgate;
    if (given(a[0])) dres = check("dres", a[0], {T, H}, type, dev);
    const bool next = given(a[6]);
    if (given(a[7]) != next || given(a[8]) != next || given(a[9]) != next)
      throw Refused{"dh, out, gamma_next and rstd_out are given together"};
    if (!next && !dres.defined()) throw Refused{"dres or dh: a gradient is needed"};
    if (next) {
      dh = check("dh", a[6], {T, H}, type, dev);
      out = check("out", a[7], {T, H}, type, dev);
      gn = check("gamma_next", a[8], {H}, kF32, dev);
      ro = check("rstd_out", a[9], {T}, kF32, dev);
      dgn = empty_as(gn);
    }
    moe_block_t c = block(y, number(a[5]), number(a[10]), 0.f);
    const Tensor gate = gate_of(a[4], y, c);
    if (gate.defined()) dgate = empty_as(gate);
    size_t bytes = 0;
    const Tensor ws = workspace(c, y, bytes), dx = empty_as(y), dy = empty_as(y), dg = empty_as(gamma);
    done("moe_block_join_backward",
         moe_block_join_backward(&c, maybe(dres), maybe(dh), maybe(out), ptr(y), fptr(gamma), maybe(gate),
                                 fmaybe(gn), fptr(ry), fmaybe(ro), ptr(dx), ptr(dy), fptr(dg), fmaybe(dgn),
                                 maybe(dgate), ptr(ws), bytes, stream_of(y)));
    return tuple({dx, dy, dg, dgn, dgate});
  });
}

// -------------------------------------------------------------------------------- router
// logits, topk_ids, dtopk_w, mode, renormalize, scale, logit_bias, n_shared -> dlogits
OPERATOR(route_backward) {
  return guarded(n, 8, [&]() -> PyObject* {
    const Tensor& logits = check("logits", a[0], {-1, -1}, kF32, -1);
    const int dev = logits.get_device();
    const int64_t T = logits.size(0), E = logits.size(1);
    const Tensor& ids = check("topk_ids", a[1], {T, -1}, kI32, dev);
    const Tensor& dw = check("dtopk_w", a[2], {T, ids.size(1)}, kF32, dev);
    const Tensor bias = given(a[6]) ? check("logit_bias", a[6], {E}, kF32, dev) : Tensor();
    const int renorm = PyObject_IsTrue(a[4]);
    if (renorm < 0) throw python_error();
    moe_config_t c{};
    c.T = narrow("logits", T);
    c.E = narrow("logits", E);
    const int64_t shared = integer(a[7]);
    if (shared < 0 || shared >= ids.size(1))
      throw Refused{"n_shared: " + std::to_string(shared) + " of " + std::to_string(ids.size(1)) + " slots"};
    c.n_shared = (int)shared;
    c.k = narrow("topk_ids", ids.size(1)) - c.n_shared;
    c.mode = (moe_route_mode_t)integer(a[3]);
    c.renormalize = renorm;
    c.scale = number(a[5]);
    c.logit_bias = fmaybe(bias);
    const Tensor dl = empty_as(logits);
    done("moe_route_backward",
         moe_route_backward(&c, fptr(logits), iptr(ids), fptr(dw), fptr(dl), stream_of(logits)));
    return wrap(dl);
  });
}

PyObject* set_error(PyObject*, PyObject* e) {  // the class that statuses raise
  Py_XSETREF(g_moe_error, Py_NewRef(e));
  Py_RETURN_NONE;
}

#define FAST(name) {#name, (PyCFunction)(void (*)(void))name, METH_FASTCALL, nullptr}
PyMethodDef methods[] = {FAST(sort_tokens),
                         FAST(permute),
                         FAST(permute_backward),
                         FAST(unpermute),
                         FAST(unpermute_backward),
                         FAST(expert_up),
                         FAST(expert_down),
                         FAST(expert_down_backward),
                         FAST(expert_up_backward),
                         FAST(expert_weight_grad),
                         FAST(block_norm),
                         FAST(block_norm_backward),
                         FAST(block_join),
                         FAST(block_join_backward),
                         FAST(route_backward),
                         {"set_error", set_error, METH_O, nullptr},
                         {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_native", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__native() { return PyModule_Create(&module); }
