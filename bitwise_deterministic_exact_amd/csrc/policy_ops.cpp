// The torch side of the policy and preference losses: argument checks, outputs,
// workspaces, the current stream, and the autograd functions, over the C entry
// points of libdetgemm.so (include/detgemm.h).
#include "ops_common.h"

#include <cmath>

void bind_policy(py::module_& m);

namespace {

// [.., T] float32 as rows of T with adjacent tokens
void check_logprob(const Tensor& t, at::IntArrayRef shape, const Tensor& like, const char* name, const char* what) {
  if (t.scalar_type() != at::kFloat || t.sizes() != shape || t.device() != like.device())
    refuse(what, ": ", name, " must be float32 of shape ", shape, " on the log probabilities' device (got ",
           t.scalar_type(), " ", t.sizes(), ")");
}
void check_mask(const OptTensor& t, at::IntArrayRef shape, const Tensor& like, const char* name, const char* what) {
  if (t && (t->scalar_type() != at::kBool || t->sizes() != shape || t->device() != like.device()))
    refuse(what, ": ", name, " must be bool of shape ", shape, " on the log probabilities' device");
}
// like rows(), also for no tokens
Tensor token_rows(const Tensor& t) {
  if (t.size(-1) == 0) return t.reshape({c10::multiply_integers(lead_of(t)), 0});
  return rows(t);
}
Tensor token_rows(const OptTensor& t) { return t ? token_rows(*t) : Tensor(); }
int64_t stride_of(const Tensor& t) { return t.defined() ? t.stride(0) : 0; }
template <class T>
const T* ptr(const Tensor& t) { return t.defined() ? static_cast<const T*>(t.const_data_ptr()) : nullptr; }

// an input without a gradient
Tensor constant(const Tensor& t) { return t.requires_grad() ? t.detach() : t; }
OptTensor constant(const OptTensor& t) { return wants_grad(t) ? OptTensor(t->detach()) : t; }

// ---------------------------------------------------------------- policy loss

struct PolicyOptions {
  double low, high, kl_weight;
  det_reduction reduction;
};

det_reduction reduction_of(const std::string& name, const char* what) {
  if (name == "none") return DET_REDUCE_NONE;
  if (name == "tokens") return DET_REDUCE_TOKENS;
  if (name == "sequences") return DET_REDUCE_SEQUENCES;
  refuse(what, ": reduction must be \"tokens\", \"sequences\" or \"none\" (got \"", name, "\")");
}

// the inputs as rows, checked
struct PolicyRows {
  Tensor lp, old, adv, mask, ref;
  int64_t B, T;
  int adv_t;
};
PolicyRows policy_rows(const Tensor& lp, const Tensor& old, const Tensor& adv, const OptTensor& mask,
                       const OptTensor& ref, const PolicyOptions& o, const char* what) {
  if (lp.scalar_type() != at::kFloat || lp.dim() < 1)
    refuse(what, ": logprob must be float32 [..., T] (got ", lp.scalar_type(), " ", lp.sizes(), ")");
  check_logprob(old, lp.sizes(), lp, "old_logprob", what);
  if (adv.sizes() != lp.sizes())
    check_logprob(adv, lead_of(lp), lp, "advantage (one to a row, or one to a token)", what);
  else check_logprob(adv, lp.sizes(), lp, "advantage", what);
  if (ref) check_logprob(*ref, lp.sizes(), lp, "ref_logprob", what);
  else if (o.kl_weight != 0.0) refuse(what, ": a KL term needs ref_logprob");
  check_mask(mask, lp.sizes(), lp, "mask", what);
  if (!(o.low >= 0.0) || !(o.low <= 1.0)) refuse(what, ": clip_low must lie in [0, 1] (got ", o.low, ")");
  if (!(o.high >= 0.0) || !(o.high < 1e6)) refuse(what, ": clip_high must lie in [0, 1e6) (got ", o.high, ")");
  if (!(o.kl_weight >= 0.0) || !(o.kl_weight < 1e6))
    refuse(what, ": kl_weight must lie in [0, 1e6) (got ", o.kl_weight, ")");
  on_gpu(lp, what, "logprob");
  PolicyRows r;
  r.lp = token_rows(lp);
  r.old = token_rows(old);
  r.adv_t = adv.sizes() == lp.sizes();
  r.adv = r.adv_t ? token_rows(adv) : adv.reshape({-1});
  r.mask = token_rows(mask);
  r.ref = token_rows(ref);
  r.B = r.lp.size(0);
  r.T = r.lp.size(1);
  return r;
}

struct Policy {
  Tensor loss, kl, clipped, count;
};

Policy policy_forward(const Tensor& lp, const Tensor& old, const Tensor& adv, const OptTensor& mask,
                      const OptTensor& ref, const PolicyOptions& o) {
  const char* const what = "policy_loss";
  not_traced(what);
  const PolicyRows r = policy_rows(lp, old, adv, mask, ref, o, what);
  const c10::DeviceGuard guard(lp.device());
  const bool none = o.reduction == DET_REDUCE_NONE;
  const at::IntArrayRef shape = none ? lp.sizes() : at::IntArrayRef();
  Policy p{at::empty(shape, lp.options()), at::empty(shape, lp.options()), at::empty(shape, lp.options()), Tensor()};
  if (!none) p.count = at::empty({r.B + 1}, lp.options().dtype(at::kLong));
  const int64_t bytes = det_policy_loss_workspace_bytes(r.B, r.T, o.reduction);
  const Tensor ws = bytes > 0 ? at::empty({bytes}, lp.options().dtype(at::kByte)) : Tensor();
  ok(det_policy_loss(ptr<float>(r.lp), r.lp.stride(0), ptr<float>(r.old), r.old.stride(0), ptr<float>(r.adv),
                     r.adv.stride(0), r.adv_t, ptr<uint8_t>(r.mask), stride_of(r.mask), ptr<float>(r.ref),
                     stride_of(r.ref), r.B, r.T, o.low, o.high, o.kl_weight, o.reduction, out<float>(p.loss), out<float>(p.kl), out<float>(p.clipped),
                     out<int64_t>(p.count), out<void>(ws), static_cast<size_t>(bytes), stream_of(lp)));
  return p;
}

Tensor policy_backward(const Tensor& g, const Tensor& lp, const Tensor& old, const Tensor& adv, const OptTensor& mask,
                       const OptTensor& ref, const OptTensor& count, const PolicyOptions& o) {
  const char* const what = "policy_loss_backward";
  not_traced(what);
  const PolicyRows r = policy_rows(lp, old, adv, mask, ref, o, what);
  const bool none = o.reduction == DET_REDUCE_NONE;
  const at::IntArrayRef shape = none ? lp.sizes() : at::IntArrayRef();
  check_logprob(g, shape, lp, "the incoming gradient", what);
  if (!none && (!count || count->scalar_type() != at::kLong || count->dim() != 1 || count->size(0) != r.B + 1 ||
                count->device() != lp.device()))
    refuse(what, ": count must be as policy_loss_forward gives it");
  const c10::DeviceGuard guard(lp.device());
  Tensor g2 = g, d = at::empty(lp.sizes(), lp.options());
  if (none) g2 = g.dim() == 2 ? g : g.reshape({r.B, r.T});
  const Tensor c = none ? Tensor() : count->contiguous();
  ok(det_policy_loss_grad(ptr<float>(r.lp), r.lp.stride(0), ptr<float>(r.old), r.old.stride(0), ptr<float>(r.adv),
                          r.adv.stride(0), r.adv_t, ptr<uint8_t>(r.mask), stride_of(r.mask), ptr<float>(r.ref),
                          stride_of(r.ref), r.B, r.T, o.low, o.high, o.kl_weight, o.reduction, ptr<int64_t>(c),
                          ptr<float>(g2), none ? g2.stride(0) : 0, none ? g2.stride(1) : 0, out<float>(d), stream_of(lp)));
  return d;
}

struct PolicyFn : torch::autograd::Function<PolicyFn> {
  static variable_list forward(AutogradContext* ctx, const Tensor& lp, const Tensor& old, const Tensor& adv,
                               const OptTensor& mask, const OptTensor& ref, double low, double high, double kl_weight,
                               int64_t reduction) {
    const PolicyOptions o{low, high, kl_weight, static_cast<det_reduction>(reduction)};
    const Policy p = policy_forward(lp, old, adv, mask, ref, o);
    ctx->save_for_backward({lp, old, adv, mask.value_or(Tensor()), ref.value_or(Tensor()), p.count});
    ctx->saved_data["low"] = low;
    ctx->saved_data["high"] = high;
    ctx->saved_data["kl_weight"] = kl_weight;
    ctx->saved_data["reduction"] = reduction;
    ctx->set_materialize_grads(false);
    ctx->mark_non_differentiable({p.kl, p.clipped});
    return {p.loss, p.kl, p.clipped};
  }
  static variable_list backward(AutogradContext* ctx, variable_list grads) {
    for (const Tensor& g : grads) no_tangent(g, "policy_loss");
    const auto s = ctx->get_saved_variables();
    Tensor d;
    if (grads[0].defined()) {
      const at::NoGradGuard no_grad;
      d = policy_backward(grads[0], s[0], s[1], s[2], opt(s[3]), opt(s[4]), opt(s[5]),
                          {ctx->saved_data["low"].toDouble(), ctx->saved_data["high"].toDouble(),
                           ctx->saved_data["kl_weight"].toDouble(),
                           static_cast<det_reduction>(ctx->saved_data["reduction"].toInt())});
    }
    variable_list r = once({d}, {s[0], grads[0]}, "policy_loss");
    r.resize(9);
    return r;
  }
};

std::tuple<Tensor, Tensor, Tensor> policy_loss(const Tensor& lp, const Tensor& old, const Tensor& adv,
                                               const OptTensor& mask, const OptTensor& ref, double low, double high,
                                               double kl_weight, const std::string& reduction) {
  for (const OptTensor& t : {OptTensor(lp), OptTensor(old), OptTensor(adv), ref}) no_tangent(t, "policy_loss");
  const det_reduction red = reduction_of(reduction, "policy_loss");
  if (at::GradMode::is_enabled() && wants_grad(lp)) {
    const variable_list v = PolicyFn::apply(lp, constant(old), constant(adv), mask, constant(ref), low, high, kl_weight,
                                            static_cast<int64_t>(red));
    return {v[0], v[1], v[2]};
  }
  const Policy p = policy_forward(lp, old, adv, mask, ref, {low, high, kl_weight, red});
  return {p.loss, p.kl, p.clipped};
}

// ---------------------------------------------------------------- preference loss

struct PreferenceOptions {
  det_preference kind;
  double beta, margin, smooth;
  bool by_length;
};

det_preference kind_of(const std::string& name, const char* what) {
  if (name == "sigmoid") return DET_PREFER_SIGMOID;
  if (name == "hinge") return DET_PREFER_HINGE;
  if (name == "ipo") return DET_PREFER_IPO;
  refuse(what, ": kind must be \"sigmoid\", \"hinge\" or \"ipo\" (got \"", name, "\")");
}

struct Preference {
  Tensor loss, chosen, rejected, slope;
};

Preference preference_forward(const Tensor& chosen, const Tensor& rejected, const OptTensor& ref_chosen,
                              const OptTensor& ref_rejected, const OptTensor& mask_chosen,
                              const OptTensor& mask_rejected, const PreferenceOptions& o) {
  const char* const what = "preference_loss";
  not_traced(what);
  for (const auto& [t, name] : {std::pair{&chosen, "chosen_logprob"}, std::pair{&rejected, "rejected_logprob"}})
    if (t->scalar_type() != at::kFloat || t->dim() < 1)
      refuse(what, ": ", name, " must be float32 [..., T] (got ", t->scalar_type(), " ", t->sizes(), ")");
  if (lead_of(chosen) != lead_of(rejected) || chosen.device() != rejected.device())
    refuse(what, ": both sides must have one leading shape, on one device (got ", chosen.sizes(), " and ",
           rejected.sizes(), ")");
  if (ref_chosen.has_value() != ref_rejected.has_value())
    refuse(what, ": reference log probabilities are given for both sides or for none");
  if (ref_chosen) {
    check_logprob(*ref_chosen, chosen.sizes(), chosen, "ref_chosen_logprob", what);
    check_logprob(*ref_rejected, rejected.sizes(), chosen, "ref_rejected_logprob", what);
  }
  check_mask(mask_chosen, chosen.sizes(), chosen, "chosen_mask", what);
  check_mask(mask_rejected, rejected.sizes(), chosen, "rejected_mask", what);
  if (!(o.beta > 0.0) || !(o.beta < 1e6)) refuse(what, ": beta must lie in (0, 1e6) (got ", o.beta, ")");
  if (!std::isfinite(o.margin)) refuse(what, ": margin must be finite (got ", o.margin, ")");
  if (o.margin != 0.0 && o.kind == DET_PREFER_IPO) refuse(what, ": ipo takes no margin");
  if (!(o.smooth >= 0.0) || !(o.smooth <= 0.5))
    refuse(what, ": label_smoothing must lie in [0, 0.5] (got ", o.smooth, ")");
  if (o.smooth != 0.0 && o.kind != DET_PREFER_SIGMOID) refuse(what, ": label_smoothing is the sigmoid loss's");
  on_gpu(chosen, what, "chosen_logprob");
  const c10::DeviceGuard guard(chosen.device());
  const Tensor c = token_rows(chosen), r = token_rows(rejected), rc = token_rows(ref_chosen), rr = token_rows(ref_rejected);
  const Tensor mc = token_rows(mask_chosen), mr = token_rows(mask_rejected);
  const int64_t P = c.size(0);
  const at::IntArrayRef lead = lead_of(chosen);
  Preference p{at::empty(lead, chosen.options()), at::empty(lead, chosen.options()), at::empty(lead, chosen.options()),
               at::empty({P, 2}, chosen.options())};
  ok(det_preference_loss(ptr<float>(c), c.stride(0), ptr<float>(rc), stride_of(rc), ptr<uint8_t>(mc), stride_of(mc),
                         c.size(1), ptr<float>(r), r.stride(0), ptr<float>(rr), stride_of(rr), ptr<uint8_t>(mr),
                         stride_of(mr), r.size(1), P, o.kind, o.beta, o.margin, o.smooth, o.by_length, out<float>(p.loss), out<float>(p.chosen),
                         out<float>(p.rejected), out<float>(p.slope), stream_of(chosen)));
  return p;
}

std::tuple<Tensor, Tensor> preference_backward(const Tensor& g, const Tensor& slope, at::IntArrayRef chosen,
                                               at::IntArrayRef rejected, const OptTensor& mask_chosen,
                                               const OptTensor& mask_rejected, bool need_chosen, bool need_rejected) {
  const char* const what = "preference_loss_backward";
  not_traced(what);
  if (chosen.empty() || rejected.empty() ||
      chosen.slice(0, chosen.size() - 1) != rejected.slice(0, rejected.size() - 1))
    refuse(what, ": both sides must have one leading shape");
  const at::IntArrayRef lead = chosen.slice(0, chosen.size() - 1);
  const int64_t P = c10::multiply_integers(lead);
  if (slope.scalar_type() != at::kFloat || slope.dim() != 2 || slope.size(0) != P || slope.size(1) != 2)
    refuse(what, ": slope must be as preference_loss_forward gives it");
  check_logprob(g, lead, slope, "the incoming gradient", what);
  check_mask(mask_chosen, chosen, slope, "chosen_mask", what);
  check_mask(mask_rejected, rejected, slope, "rejected_mask", what);
  on_gpu(slope, what, "slope");
  const c10::DeviceGuard guard(slope.device());
  Tensor dc, dr;
  if (need_chosen) dc = at::empty(chosen, slope.options());
  if (need_rejected) dr = at::empty(rejected, slope.options());
  const Tensor s = slope.contiguous(), mc = token_rows(mask_chosen), mr = token_rows(mask_rejected);
  const Tensor g1 = g.reshape({P});
  ok(det_preference_loss_grad(ptr<uint8_t>(mc), stride_of(mc), chosen.back(), ptr<uint8_t>(mr), stride_of(mr),
                              rejected.back(), P, ptr<float>(s), ptr<float>(g1), g1.stride(0), out<float>(dc),
                              out<float>(dr), stream_of(slope)));
  return {dc, dr};
}

struct PreferenceFn : torch::autograd::Function<PreferenceFn> {
  static variable_list forward(AutogradContext* ctx, const Tensor& chosen, const Tensor& rejected,
                               const OptTensor& ref_chosen, const OptTensor& ref_rejected, const OptTensor& mask_chosen,
                               const OptTensor& mask_rejected, int64_t kind, double beta, double margin, double smooth,
                               bool by_length) {
    const Preference p = preference_forward(chosen, rejected, ref_chosen, ref_rejected, mask_chosen, mask_rejected,
                                            {static_cast<det_preference>(kind), beta, margin, smooth, by_length});
    // the slopes and the shapes are what the gradient needs: the log probabilities are not kept
    ctx->save_for_backward({p.slope, mask_chosen.value_or(Tensor()), mask_rejected.value_or(Tensor())});
    ctx->saved_data["chosen"] = chosen.sizes().vec();
    ctx->saved_data["rejected"] = rejected.sizes().vec();
    ctx->set_materialize_grads(false);
    ctx->mark_non_differentiable({p.chosen, p.rejected});
    return {p.loss, p.chosen, p.rejected};
  }
  static variable_list backward(AutogradContext* ctx, variable_list grads) {
    for (const Tensor& g : grads) no_tangent(g, "preference_loss");
    const auto s = ctx->get_saved_variables();
    Tensor dc, dr;
    if (grads[0].defined()) {
      const at::NoGradGuard no_grad;
      std::tie(dc, dr) = preference_backward(grads[0], s[0], ctx->saved_data["chosen"].toIntVector(),
                                             ctx->saved_data["rejected"].toIntVector(), opt(s[1]), opt(s[2]),
                                             ctx->needs_input_grad(0), ctx->needs_input_grad(1));
    }
    variable_list r = once_at_node({dc, dr}, grads, "preference_loss");
    r.resize(11);
    return r;
  }
};

std::tuple<Tensor, Tensor, Tensor> preference_loss(const Tensor& chosen, const Tensor& rejected,
                                                   const OptTensor& ref_chosen, const OptTensor& ref_rejected,
                                                   const OptTensor& mask_chosen, const OptTensor& mask_rejected,
                                                   const std::string& kind, double beta, double margin, double smooth,
                                                   bool by_length) {
  for (const OptTensor& t : {OptTensor(chosen), OptTensor(rejected), ref_chosen, ref_rejected})
    no_tangent(t, "preference_loss");
  const det_preference k = kind_of(kind, "preference_loss");
  if (at::GradMode::is_enabled() && (wants_grad(chosen) || wants_grad(rejected))) {
    const variable_list v = PreferenceFn::apply(chosen, rejected, constant(ref_chosen), constant(ref_rejected),
                                                mask_chosen, mask_rejected, static_cast<int64_t>(k), beta, margin, smooth,
                                                by_length);
    return {v[0], v[1], v[2]};
  }
  const Preference p = preference_forward(chosen, rejected, ref_chosen, ref_rejected, mask_chosen, mask_rejected,
                                          {k, beta, margin, smooth, by_length});
  return {p.loss, p.chosen, p.rejected};
}

}  // namespace

void bind_policy(py::module_& m) {
  using release = py::call_guard<py::gil_scoped_release>;
  m.def("policy_loss", &policy_loss, release());
  m.def("policy_loss_forward", [](const Tensor& lp, const Tensor& old, const Tensor& adv, const OptTensor& mask,
                                  const OptTensor& ref, double low, double high, double kl_weight, const std::string& red) {
    const Policy p = policy_forward(lp, old, adv, mask, ref, {low, high, kl_weight, reduction_of(red, "policy_loss")});
    return std::make_tuple(p.loss, p.kl, p.clipped, opt(p.count));
  }, release());
  m.def("policy_loss_backward", [](const Tensor& g, const Tensor& lp, const Tensor& old, const Tensor& adv,
                                   const OptTensor& mask, const OptTensor& ref, const OptTensor& count, double low,
                                   double high, double kl_weight, const std::string& red) {
    return policy_backward(g, lp, old, adv, mask, ref, count,
                           {low, high, kl_weight, reduction_of(red, "policy_loss_backward")});
  }, release());
  m.def("preference_loss", &preference_loss, release());
  m.def("preference_loss_forward", [](const Tensor& c, const Tensor& r, const OptTensor& rc, const OptTensor& rr,
                                      const OptTensor& mc, const OptTensor& mr, const std::string& kind, double beta,
                                      double margin, double smooth, bool by_length) {
    const Preference p = preference_forward(c, r, rc, rr, mc, mr,
                                            {kind_of(kind, "preference_loss"), beta, margin, smooth, by_length});
    return std::make_tuple(p.loss, p.chosen, p.rejected, p.slope);
  }, release());
  m.def("preference_loss_backward", [](const Tensor& g, const Tensor& slope, const std::vector<int64_t>& chosen,
                                       const std::vector<int64_t>& rejected, const OptTensor& mc, const OptTensor& mr) {
    const auto [dc, dr] = preference_backward(g, slope, chosen, rejected, mc, mr, true, true);
    return std::make_tuple(dc, dr);
  }, release());
}
