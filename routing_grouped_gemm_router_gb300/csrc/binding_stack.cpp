// binding_stack.cpp — the operators around a stack's blocks (include/moe_stack.h) on torch tensors, as a
// CPython extension (host code only), in the manner of binding.cpp. The Python functions with their
// documentation are in training.py.
#include "binding.h"
#include "moe_stack.h"

namespace {

// ------------------------------------------------------------------------------ embedding
// Token ids, int32 or int64 [T] (-1: any).
const Tensor& token_ids(PyObject* o, int64_t T, int dev) {
  const bool wide = THPVariable_Check(o) && THPVariable_Unpack(o).scalar_type() == ScalarType::Long;
  return check("tokens", o, {T}, wide ? ScalarType::Long : kI32, dev);
}
int id_bytes(const Tensor& t) { return t.scalar_type() == ScalarType::Long ? 8 : 4; }

OPERATOR(embed) {  // tokens, table, scale -> x
  return guarded(n, 3, [&]() -> PyObject* {
    const Tensor& table = check("table", a[1], {-1, -1}, kAnyFloat, -1);
    const Tensor& tokens = token_ids(a[0], -1, table.get_device());
    const Tensor x = empty({tokens.size(0), table.size(1)}, table.scalar_type(), table);
    done("moe_embed", moe_embed(ptr(tokens), id_bytes(tokens), narrow("tokens", tokens.size(0)), ptr(table),
                                narrow("table", table.size(0)), narrow("table", table.size(1)), dtype_of(table),
                                number(a[2]), ptr(x), stream_of(table)));
    return wrap(x);
  });
}

OPERATOR(embed_backward) {  // dx, tokens, V, scale, out or None, out_dtype or None, accumulate -> dtable
  return guarded(n, 7, [&]() -> PyObject* {
    const Tensor& dx = check("dx", a[0], {-1, -1}, kAnyFloat, -1);
    const int dev = dx.get_device();
    const Tensor& tokens = token_ids(a[1], dx.size(0), dev);
    const bool accumulate = truth(a[6]);
    const ScalarType type = out_type(a[4], a[5], accumulate, dx);
    const int T = narrow("dx", dx.size(0)), V = narrow("V", integer(a[2])), H = narrow("dx", dx.size(1));
    size_t bytes = 0;
    done("moe_embed_workspace_size", moe_embed_workspace_size(T, V, H, &bytes));
    const Tensor out = given(a[4]) ? check("out", a[4], {V, H}, type, dev) : empty({V, H}, type, dx);
    const Tensor ws = empty({(int64_t)bytes}, ScalarType::Byte, dx);
    done("moe_embed_backward",
         moe_embed_backward(ptr(dx), ptr(tokens), id_bytes(tokens), T, V, H, dtype_of(dx), dtype_of(out),
                            number(a[3]), accumulate, ptr(out), ptr(ws), bytes, stream_of(dx)));
    if (given(a[4])) return Py_NewRef(a[4]);
    return wrap(out);
  });
}

// -------------------------------------------------------------- layer norm, dropout, the join
moe_layer_t layer(const Tensor& x, float scale, float eps) {
  moe_layer_t c{};
  c.T = narrow("rows", x.size(0));
  c.H = narrow("H", x.size(1));
  c.dtype = dtype_of(x);
  c.eps = eps;
  c.scale = scale;
  return c;
}
// p, rng or None (where p is 0), site
moe_drop_t drop_of(PyObject* p, PyObject* rng, PyObject* site, int dev) {
  moe_drop_t d{};
  d.p = real(p);
  if (!(d.p >= 0.0 && d.p < 1.0)) throw Refused{"p: " + std::to_string(d.p) + ", expected 0 <= p < 1"};
  if (given(rng)) d.rng = (const int64_t*)ptr(check("rng", rng, {2}, ScalarType::Long, dev));
  else if (d.p > 0.0) throw Refused{"rng: (seed, stream) is needed where p is not 0"};
  const int64_t s = integer(site);
  if (s < 0 || s > UINT32_MAX) throw Refused{"site: " + std::to_string(s) + ", expected 0 <= site < 2^32"};
  d.site = (uint32_t)s;
  return d;
}
Tensor workspace(const moe_layer_t& c, const Tensor& x, size_t& bytes) {
  done("moe_layer_workspace_size", moe_layer_workspace_size(&c, &bytes));
  return empty({(int64_t)bytes}, ScalarType::Byte, x);
}

// The gradients of a norm's weight and, if it has one, its bias.
std::array<Tensor, 2> weight_grads(const Tensor& gamma, bool beta) {
  if (!beta) return {empty_as(gamma), Tensor()};
  return empties({{{gamma.size(0)}, kF32}, {{gamma.size(0)}, kF32}}, gamma);
}

OPERATOR(layer_norm) {  // x, gamma, beta or None, eps -> h, mean, rstd
  return guarded(n, 4, [&]() -> PyObject* {
    const Tensor& x = check("x", a[0], {-1, -1}, kAnyFloat, -1);
    const int dev = x.get_device();
    const Tensor& gamma = check("gamma", a[1], {x.size(1)}, kF32, dev);
    const Tensor beta = given(a[2]) ? check("beta", a[2], {x.size(1)}, kF32, dev) : Tensor();
    const moe_layer_t c = layer(x, 1.f, number(a[3]));
    const Tensor h = empty_as(x);
    const auto [mean, r] = empties({{{x.size(0)}, kF32}, {{x.size(0)}, kF32}}, x);
    done("moe_layer_norm", moe_layer_norm(&c, ptr(x), fptr(gamma), fmaybe(beta), ptr(h), fptr(mean), fptr(r),
                                          stream_of(x)));
    return tuple({h, mean, r});
  });
}

OPERATOR(layer_norm_backward) {  // dh, x, gamma, mean, rstd, dres or None, beta -> dx, dgamma, dbeta
  return guarded(n, 7, [&]() -> PyObject* {
    const Tensor& x = check("x", a[1], {-1, -1}, kAnyFloat, -1);
    const int dev = x.get_device();
    const int64_t T = x.size(0), H = x.size(1);
    const Tensor& dh = check("dh", a[0], {T, H}, x.scalar_type(), dev);
    const Tensor& gamma = check("gamma", a[2], {H}, kF32, dev);
    const Tensor& mean = check("mean", a[3], {T}, kF32, dev);
    const Tensor& r = check("rstd", a[4], {T}, kF32, dev);
    const Tensor dres = given(a[5]) ? check("dres", a[5], {T, H}, x.scalar_type(), dev) : Tensor();
    const moe_layer_t c = layer(x, 1.f, 0.f);
    size_t bytes = 0;
    const Tensor ws = workspace(c, x, bytes), dx = empty_as(x);
    const auto [dg, db] = weight_grads(gamma, truth(a[6]));
    done("moe_layer_norm_backward",
         moe_layer_norm_backward(&c, ptr(dh), ptr(x), fptr(gamma), fptr(mean), fptr(r), maybe(dres), ptr(dx),
                                 fptr(dg), fmaybe(db), ptr(ws), bytes, stream_of(x)));
    return tuple({dx, dg, db});
  });
}

OPERATOR(dropout) {  // x, p, rng or None, site, scale -> out
  return guarded(n, 5, [&]() -> PyObject* {
    const Tensor& x = check("x", a[0], {-1, -1}, kAnyFloat, -1);
    const moe_drop_t d = drop_of(a[1], a[2], a[3], x.get_device());
    const moe_layer_t c = layer(x, number(a[4]), 0.f);
    const Tensor out = empty_as(x);
    done("moe_dropout", moe_dropout(&c, &d, ptr(x), ptr(out), stream_of(x)));
    return wrap(out);
  });
}

// x, y, p, rng or None, site, scale, gamma_next or None, beta_next or None, eps -> out, h, mean, rstd
OPERATOR(dropout_join) {
  return guarded(n, 9, [&]() -> PyObject* {
    const Tensor& x = check("x", a[0], {-1, -1}, kAnyFloat, -1);
    const int dev = x.get_device();
    const int64_t T = x.size(0), H = x.size(1);
    const Tensor& y = check("y", a[1], {T, H}, x.scalar_type(), dev);
    const moe_drop_t d = drop_of(a[2], a[3], a[4], dev);
    const moe_layer_t c = layer(x, number(a[5]), number(a[8]));
    Tensor gn, bn, h, mean, r;
    if (given(a[6])) {
      gn = check("gamma_next", a[6], {H}, kF32, dev);
      if (given(a[7])) bn = check("beta_next", a[7], {H}, kF32, dev);
      h = empty_as(x);
      auto stats = empties({{{T}, kF32}, {{T}, kF32}}, x);
      mean = std::move(stats[0]);
      r = std::move(stats[1]);
    } else if (given(a[7])) {
      throw Refused{"beta_next: needs gamma_next"};
    }
    const Tensor out = empty_as(x);
    done("moe_dropout_join", moe_dropout_join(&c, &d, ptr(x), ptr(y), fmaybe(gn), fmaybe(bn), ptr(out), maybe(h),
                                              fmaybe(mean), fmaybe(r), stream_of(x)));
    return tuple({out, h, mean, r});
  });
}

// dres, p, rng, site, scale, dh, out, gamma_next, mean, rstd, beta -> dx, dy, dgamma_next, dbeta_next
OPERATOR(dropout_join_backward) {
  return guarded(n, 11, [&]() -> PyObject* {
    const bool next = given(a[5]);
    for (int i = 6; i < 10; ++i)
      if (given(a[i]) != next) throw Refused{"dh, out, gamma_next, mean and rstd are given together"};
    if (!next) {
      if (!given(a[0])) throw Refused{"dres or dh: a gradient is needed"};
      const Tensor& dres = check("dres", a[0], {-1, -1}, kAnyFloat, -1);
      const moe_drop_t d = drop_of(a[1], a[2], a[3], dres.get_device());
      const moe_layer_t c = layer(dres, number(a[4]), 0.f);
      const Tensor dy = empty_as(dres);
      done("moe_dropout", moe_dropout(&c, &d, ptr(dres), ptr(dy), stream_of(dres)));
      return tuple({dres, dy, Tensor(), Tensor()});
    }
    const Tensor& out = check("out", a[6], {-1, -1}, kAnyFloat, -1);
    const int dev = out.get_device();
    const int64_t T = out.size(0), H = out.size(1);
    const ScalarType type = out.scalar_type();
    const Tensor dres = given(a[0]) ? check("dres", a[0], {T, H}, type, dev) : Tensor();
    const Tensor& dh = check("dh", a[5], {T, H}, type, dev);
    const Tensor& gn = check("gamma_next", a[7], {H}, kF32, dev);
    const Tensor& mean = check("mean", a[8], {T}, kF32, dev);
    const Tensor& r = check("rstd", a[9], {T}, kF32, dev);
    const moe_drop_t d = drop_of(a[1], a[2], a[3], dev);
    const moe_layer_t c = layer(out, number(a[4]), 0.f);
    size_t bytes = 0;
    const Tensor ws = workspace(c, out, bytes), dx = empty_as(out), dy = empty_as(out);
    const auto [dg, db] = weight_grads(gn, truth(a[10]));
    done("moe_dropout_join_backward",
         moe_dropout_join_backward(&c, &d, maybe(dres), ptr(dh), ptr(out), fptr(gn), fptr(mean), fptr(r), ptr(dx),
                                   ptr(dy), fptr(dg), fmaybe(db), ptr(ws), bytes, stream_of(out)));
    return tuple({dx, dy, dg, db});
  });
}

// ------------------------------------------------------------------------- the router's losses
// The parts that both directions share; the tensors stay the caller's.
moe_balance_t balance(const Tensor& logits, int64_t k, int64_t shared, PyObject* mode, PyObject* bias,
                      PyObject* offsets, PyObject* mask, int64_t S) {
  const int dev = logits.get_device();
  moe_balance_t c{};
  c.T = narrow("logits", logits.size(0));
  c.E = narrow("logits", logits.size(1));
  c.k = narrow("k", k);
  c.n_shared = (int)shared;
  c.mode = (moe_route_mode_t)integer(mode);
  if (given(bias)) c.logit_bias = fptr(check("logit_bias", bias, {logits.size(1)}, kF32, dev));
  c.S = 1;
  if (given(offsets)) {
    const Tensor& o = check("offsets", offsets, {S < 0 ? -1 : S + 1}, kI32, dev);
    if (o.size(0) < 2) throw Refused{"offsets: " + std::to_string(o.size(0)) + " of them bound no sequence"};
    c.S = narrow("offsets", o.size(0) - 1);
    c.offsets = iptr(o);
  }
  if (given(mask)) c.mask = (const uint8_t*)ptr(check("mask", mask, {logits.size(0)}, ScalarType::Bool, dev));
  return c;
}

// logits, topk_ids, mode, logit_bias, n_shared, offsets, mask -> losses, counts, tokens, prob, totals
OPERATOR(balance_loss) {
  return guarded(n, 7, [&]() -> PyObject* {
    const Tensor& logits = check("logits", a[0], {-1, -1}, kF32, -1);
    const Tensor& ids = check("topk_ids", a[1], {logits.size(0), -1}, kI32, logits.get_device());
    const int64_t shared = integer(a[4]);
    if (shared < 0 || shared >= ids.size(1))
      throw Refused{"n_shared: " + std::to_string(shared) + " of " + std::to_string(ids.size(1)) + " slots"};
    const moe_balance_t c = balance(logits, ids.size(1) - shared, shared, a[2], a[3], a[5], a[6], -1);
    size_t bytes = 0;
    done("moe_balance_workspace_size", moe_balance_workspace_size(&c, &bytes));
    const Tensor ws = empty({(int64_t)bytes}, ScalarType::Byte, logits);
    const auto [losses, counts, tokens, prob, totals] =
        empties({{{2}, kF32}, {{c.S, c.E}, kI32}, {{c.S}, kI32}, {{c.S, c.E}, kF32}, {{2}, kI32}}, logits);
    done("moe_balance_loss",
         moe_balance_loss(&c, fptr(logits), iptr(ids), fptr(losses), iptr(counts), iptr(tokens), fptr(prob),
                          iptr(totals), ptr(ws), bytes, stream_of(logits)));
    return tuple({losses, counts, tokens, prob, totals});
  });
}

// dlosses, logits, counts, tokens, totals, k, mode, logit_bias, offsets, mask, dlogits or None -> dlogits
OPERATOR(balance_loss_backward) {
  return guarded(n, 11, [&]() -> PyObject* {
    const Tensor& logits = check("logits", a[1], {-1, -1}, kF32, -1);
    const int dev = logits.get_device();
    const Tensor& dlosses = check("dlosses", a[0], {2}, kF32, dev);
    const Tensor& counts = check("counts", a[2], {-1, logits.size(1)}, kI32, dev);
    const Tensor& tokens = check("tokens", a[3], {counts.size(0)}, kI32, dev);
    const Tensor& totals = check("totals", a[4], {2}, kI32, dev);
    const moe_balance_t c = balance(logits, integer(a[5]), 0, a[6], a[7], a[8], a[9], counts.size(0));
    if (c.S != counts.size(0))
      throw Refused{"counts: of " + std::to_string(counts.size(0)) + " sequences, without their offsets"};
    const bool add = given(a[10]);
    const Tensor dl = add ? check("dlogits", a[10], {logits.size(0), logits.size(1)}, kF32, dev) : empty_as(logits);
    done("moe_balance_loss_backward",
         moe_balance_loss_backward(&c, fptr(dlosses), fptr(logits), iptr(counts), iptr(tokens), iptr(totals), add,
                                   fptr(dl), stream_of(logits)));
    if (add) return Py_NewRef(a[10]);
    return wrap(dl);
  });
}

PyMethodDef methods[] = {FAST(embed),
                         FAST(embed_backward),
                         FAST(layer_norm),
                         FAST(layer_norm_backward),
                         FAST(dropout),
                         FAST(dropout_join),
                         FAST(dropout_join_backward),
                         FAST(balance_loss),
                         FAST(balance_loss_backward),
                         {"set_error", set_error, METH_O, nullptr},
                         {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_native_stack", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__native_stack() { return PyModule_Create(&module); }
