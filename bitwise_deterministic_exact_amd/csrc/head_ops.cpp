// The torch side of layer norm, token log probabilities and distillation:
// argument checks, outputs, workspaces, the current stream, and the autograd
// functions, over the C entry points of libdetgemm.so (include/detgemm.h).
//
// It is compiled code because these operators are called once or twice per
// step on small inputs too, where the time of a call is the host's: marshalled
// from Python (ctypes, torch.autograd.Function) a forward and backward pass
// took 150 us of host time on [512, 1000] logits.
#include <ATen/ATen.h>
#include <c10/core/AutogradState.h>
#include <c10/core/DeviceGuard.h>
#include <c10/core/impl/LocalDispatchKeySet.h>
#include <c10/core/impl/TorchDispatchModeTLS.h>
#include <c10/hip/HIPStream.h>
#include <torch/csrc/autograd/custom_function.h>
#include <torch/csrc/autograd/functions/basic_ops.h>
#include <torch/csrc/autograd/functions/utils.h>
#include <torch/csrc/jit/frontend/tracer.h>
#include <torch/csrc/utils/pybind.h>

#include <optional>
#include <sstream>
#include <string>
#include <tuple>

#include "detgemm.h"

namespace py = pybind11;
using at::Tensor;
using c10::ScalarType;
using torch::autograd::AutogradContext;
using torch::autograd::variable_list;
using OptTensor = std::optional<Tensor>;

namespace {

// ---------------------------------------------------------------- checks

template <class... A>
[[noreturn]] void refuse(const A&... parts) {
  std::ostringstream s;
  (s << ... << parts);
  throw py::value_error(s.str());
}

bool known(ScalarType t) { return t == at::kFloat || t == at::kBFloat16; }
det_dtype dt_of(ScalarType t) { return t == at::kFloat ? DET_F32 : DET_BF16; }

void on_gpu(const Tensor& t, const char* what, const char* name) {
  if (!t.is_cuda()) refuse(what, ": ", name, " must be on a GPU");
}

void* stream_of(const Tensor& t) {
  return static_cast<void*>(c10::hip::getCurrentHIPStream(t.get_device()).stream());
}

// the library's status as the exceptions the rest of the package raises: bad
// arguments are ValueError, a HIP failure is DetGemmError
struct HipFailure : std::runtime_error {
  using std::runtime_error::runtime_error;
};
PyObject* g_hip_error = nullptr;               // the package's DetGemmError, held by the module

void ok(det_status st) {
  if (st == DET_OK) return;
  if (st == DET_EHIP) throw HipFailure(det_last_error());
  throw py::value_error(det_last_error());
}

const void* in(const Tensor& t) { return t.const_data_ptr(); }
const void* in(const OptTensor& t) { return t ? t->const_data_ptr() : nullptr; }
template <class T>
T* out(const Tensor& t) { return t.defined() ? static_cast<T*>(t.mutable_data_ptr()) : nullptr; }

// [..., C] as [N, C] rows with adjacent elements: a copy only when one stride
// cannot describe the rows, or a row's elements are apart
Tensor rows(const Tensor& t) {
  Tensor r = t.dim() == 2 ? t : t.reshape({t.numel() / t.size(-1), t.size(-1)});
  return r.size(1) <= 1 || r.stride(1) == 1 ? r : r.contiguous();
}

// an incoming gradient over the flattened rows and its stride; one broadcast
// value stays one value
std::pair<Tensor, int64_t> grad_rows(const Tensor& g, at::IntArrayRef lead, const Tensor& like, const char* what) {
  if (!g.defined()) return {g, 0};
  if (g.sizes() != lead || g.scalar_type() != at::kFloat || g.device() != like.device())
    refuse(what, ": incoming gradients must be float32 of shape ", lead, " on the logits' device");
  if (g.dim() == 1) return {g, g.stride(0)};
  bool one = true;
  for (int64_t d = 0; d < g.dim(); ++d) one = one && (g.size(d) == 1 || g.stride(d) == 0);
  if (one) return {g, 0};
  return {g.contiguous(), 1};
}

// Gradients of gradients are not formed.  A backward pass that is itself
// recorded (create_graph) gives gradients whose node refuses to run; it has
// edges to everything they depend on, the saved inputs and the incoming
// gradients, so that a derivative through any of these reaches it, also where
// it is asked for one input alone.  Torch's own DelayedError hangs on the
// results only: grad(loss + g.pow(2).sum(), x) would leave it out and return
// the first-order terms.
variable_list once(variable_list grads, const variable_list& sources, const char* name) {
  if (!at::GradMode::is_enabled()) return grads;
  const auto refusal = std::make_shared<torch::autograd::Error>(
      std::string(name) + " is differentiable once",
      torch::autograd::collect_next_edges(at::ArrayRef<Tensor>(sources)));
  for (auto& g : grads)
    if (g.defined()) torch::autograd::set_history(g, refusal);
  return grads;
}

// A trace (torch.jit.trace, make_fx) sees the allocations of the results but
// not what fills them: the traced function would return whatever lies there.
// So a call that is being traced is refused.
void not_traced(const char* what) {
  using c10::impl::TorchDispatchModeKey;
  if (torch::jit::tracer::isTracing() || c10::impl::TorchDispatchModeTLS::get_mode(TorchDispatchModeKey::PROXY) ||
      c10::impl::tls_is_dispatch_key_included(c10::DispatchKey::PreDispatch))
    throw std::runtime_error(std::string(what) + " cannot be traced: its kernels are not torch operators");
}

// Forward-mode derivatives are not formed: a result without its tangent would pass
// for a constant, so inputs and incoming gradients that carry one are refused.
void no_tangent(const OptTensor& t, const char* what) {
  if (t && t->defined() && t->_fw_grad(0).defined() && c10::AutogradState::get_tls_state().get_fw_grad_mode())
    throw std::runtime_error(std::string(what) + " forms no forward-mode derivatives");
}

bool wants_grad(const Tensor& t) { return t.defined() && t.requires_grad(); }
bool wants_grad(const OptTensor& t) { return t && t->requires_grad(); }

// ---------------------------------------------------------------- layer norm

void check_norm(const Tensor& x, const OptTensor& w, const OptTensor& b, const char* what) {
  if (!known(x.scalar_type())) refuse(what, ": x must be float32 or bfloat16 (got ", x.scalar_type(), ")");
  if (x.dim() < 1 || x.size(-1) < 1)
    refuse(what, ": x needs a last dimension of at least 1 (got shape ", x.sizes(), ")");
  const int64_t C = x.size(-1);
  if (C > DET_NORM_C_MAX) refuse(what, ": rows of ", C, " exceed the limit ", DET_NORM_C_MAX);
  if (x.numel() / C > DET_ROWS_MAX) refuse(what, ": more than 2^22 rows in one call");
  for (const auto& [p, name] : {std::pair{&w, "weight"}, std::pair{&b, "bias"}}) {
    if (!*p) continue;
    const Tensor& t = **p;
    if (!known(t.scalar_type()) || t.dim() != 1 || t.size(0) != C || t.device() != x.device())
      refuse(what, ": ", name, " must be float32 or bfloat16 of shape [", C, "] on x's device");
  }
  if (w && b && w->scalar_type() != b->scalar_type()) refuse(what, ": weight and bias must share a dtype");
  on_gpu(x, what, "x");
}

std::tuple<Tensor, Tensor, Tensor> norm_forward(const Tensor& x, const OptTensor& w, const OptTensor& b, double eps,
                                                std::optional<ScalarType> out_dtype, bool stats) {
  const char* const what = "layer_norm";
  not_traced(what);
  check_norm(x, w, b, what);
  const ScalarType yt = out_dtype.value_or(x.scalar_type());
  if (!known(yt)) refuse(what, ": out_dtype must be float32 or bfloat16 (got ", yt, ")");
  if (!(eps >= 0.0) || !(eps < 1e30)) refuse(what, ": eps must be >= 0 and finite");
  const c10::DeviceGuard guard(x.device());
  const Tensor x2 = rows(x);
  const int64_t N = x2.size(0), C = x2.size(1);
  Tensor y = at::empty(x.sizes(), x.options().dtype(yt)), mean, rstd;
  if (stats) {
    mean = at::empty(x.sizes().slice(0, x.dim() - 1), x.options().dtype(at::kFloat));
    rstd = at::empty_like(mean);
  }
  const OptTensor wc = w ? OptTensor(w->contiguous()) : w, bc = b ? OptTensor(b->contiguous()) : b;
  const ScalarType wt = w ? w->scalar_type() : b ? b->scalar_type() : at::kFloat;
  ok(det_layer_norm(dt_of(x.scalar_type()), in(x2), x2.stride(0), dt_of(wt), in(wc), in(bc), N, C, eps, dt_of(yt),
                    out<void>(y), out<float>(mean), out<float>(rstd), stream_of(x)));
  return {y, mean, rstd};
}

struct NormGrads {
  Tensor dx, dw, db, digits;
};

NormGrads norm_backward(const Tensor& dy, const Tensor& x, const OptTensor& w, const Tensor& mean,
                        const Tensor& rstd, bool need_dx, bool need_dw, bool need_db,
                        std::optional<ScalarType> grad_dtype, bool digits) {
  const char* const what = "layer_norm_backward";
  not_traced(what);
  check_norm(x, w, std::nullopt, what);
  if (dy.sizes() != x.sizes() || !known(dy.scalar_type()) || dy.device() != x.device())
    refuse(what, ": dy must be float32 or bfloat16 of x's shape on x's device");
  const int64_t C = x.size(-1), N = x.numel() / C;
  for (const Tensor* s : {&mean, &rstd})
    if (s->scalar_type() != at::kFloat || s->numel() != N || s->device() != x.device())
      refuse(what, ": mean and rstd must be float32, one per row, on x's device");
  const ScalarType gt = grad_dtype.value_or(w ? w->scalar_type() : at::kFloat);
  if (!known(gt)) refuse(what, ": grad_dtype must be float32 or bfloat16");
  if (w && w->scalar_type() == at::kFloat && gt != at::kFloat)
    refuse(what, ": a float32 weight takes float32 gradients");
  const c10::DeviceGuard guard(x.device());
  const Tensor x2 = rows(x), dy2 = rows(dy), m = mean.contiguous(), r = rstd.contiguous();
  const OptTensor wc = w ? OptTensor(w->to(gt).contiguous()) : w;
  NormGrads g;
  if (need_dx) g.dx = at::empty(x.sizes(), x.options());
  if (need_dw) g.dw = at::empty({C}, x.options().dtype(gt));
  if (need_db) g.db = at::empty({C}, x.options().dtype(gt));
  if (digits) g.digits = at::empty({2, C, DET_NUM_DIGITS}, x.options().dtype(at::kLong));
  Tensor ws;
  int64_t bytes = 0;
  if (need_dw || need_db || digits) {
    bytes = det_layer_norm_grad_workspace_bytes(N, C);
    if (bytes > 0) ws = at::empty({bytes}, x.options().dtype(at::kByte));
  }
  ok(det_layer_norm_grad(dt_of(x.scalar_type()), in(x2), x2.stride(0), dt_of(dy.scalar_type()), in(dy2),
                         dy2.stride(0), dt_of(gt), in(wc), static_cast<const float*>(in(m)),
                         static_cast<const float*>(in(r)), N, C, out<void>(g.dx), out<void>(g.dw), out<void>(g.db),
                         out<int64_t>(g.digits), out<void>(ws), static_cast<size_t>(bytes), stream_of(x)));
  return g;
}

struct NormFn : torch::autograd::Function<NormFn> {
  static Tensor forward(AutogradContext* ctx, const Tensor& x, const OptTensor& w, const OptTensor& b, double eps,
                        std::optional<ScalarType> out_dtype) {
    auto [y, mean, rstd] = norm_forward(x, w, b, eps, out_dtype, true);
    ctx->save_for_backward({x, w.value_or(Tensor()), mean, rstd});
    const ScalarType gt = w ? w->scalar_type() : b ? b->scalar_type() : at::kFloat;
    ctx->saved_data["grad_dtype"] = static_cast<int64_t>(gt);
    ctx->saved_data["has_weight"] = w.has_value();
    ctx->saved_data["has_bias"] = b.has_value();
    return y;
  }
  static variable_list backward(AutogradContext* ctx, variable_list grads) {
    no_tangent(grads[0], "layer_norm");
    const auto saved = ctx->get_saved_variables();
    const OptTensor w = saved[1].defined() ? OptTensor(saved[1]) : std::nullopt;
    const auto gt = static_cast<ScalarType>(ctx->saved_data["grad_dtype"].toInt());
    // the inputs' edges are numbered without the absent ones
    const bool has_w = ctx->saved_data["has_weight"].toBool(), has_b = ctx->saved_data["has_bias"].toBool();
    const bool need_w = has_w && ctx->needs_input_grad(1);
    const bool need_b = has_b && ctx->needs_input_grad(has_w ? 2 : 1);
    NormGrads g;
    {
      const at::NoGradGuard no_grad;
      g = norm_backward(grads[0], saved[0], w, saved[2], saved[3], ctx->needs_input_grad(0), need_w, need_b, gt,
                        false);
    }
    variable_list r = once({g.dx, g.dw, g.db}, {saved[0], saved[1], grads[0]}, "layer_norm");
    r.resize(5);
    return r;
  }
};

Tensor layer_norm(const Tensor& x, const OptTensor& w, const OptTensor& b, double eps,
                  std::optional<ScalarType> out_dtype) {
  for (const OptTensor& t : {OptTensor(x), w, b}) no_tangent(t, "layer_norm");
  if (at::GradMode::is_enabled() && (wants_grad(x) || wants_grad(w) || wants_grad(b)))
    return NormFn::apply(x, w, b, eps, out_dtype);
  return std::get<0>(norm_forward(x, w, b, eps, out_dtype, false));
}

// ---------------------------------------------------------------- logits

void check_logits(const Tensor& z, const char* what) {
  if (!known(z.scalar_type())) refuse(what, ": logits must be float32 or bfloat16 (got ", z.scalar_type(), ")");
  if (z.dim() < 1 || z.size(-1) < 1 || z.size(-1) > DET_HEAD_V_MAX)
    refuse(what, ": logits must be [..., V] with 1 <= V <= 2^24 (got shape ", z.sizes(), ")");
  if (z.numel() / z.size(-1) > DET_ROWS_MAX) refuse(what, ": more than 2^22 rows in one call");
}

void check_scale(double scale, const char* what) {
  if (!(scale >= 1e-6) || !(scale < 1e6))
    refuse(what, ": the scale (1 / temperature) must lie in [1e-6, 1e6) (got ", scale, ")");
}

void check_temperature(double T, const char* what) {
  if (!(T > 0.0)) refuse(what, ": the temperature must be positive (got ", T, ")");
  check_scale(1.0 / T, what);
}

void check_index(const Tensor& t, at::IntArrayRef shape, const Tensor& like, const char* name, const char* what) {
  if (t.scalar_type() != at::kLong || t.sizes() != shape || t.device() != like.device())
    refuse(what, ": ", name, " must be int64 of shape ", shape, " on the logits' device");
}

void check_stat(const Tensor& stat, int64_t N, const Tensor& like, const char* what) {
  if (stat.dim() != 2 || stat.size(0) != N || stat.size(1) != 4 || stat.scalar_type() != at::kFloat ||
      stat.device() != like.device())
    refuse(what, ": stat must be float32 [", N, ", 4] on the logits' device");
}

at::IntArrayRef lead_of(const Tensor& t) { return t.sizes().slice(0, t.dim() - 1); }
std::vector<int64_t> with_last(at::IntArrayRef lead, int64_t n) {
  std::vector<int64_t> s(lead.begin(), lead.end());
  s.push_back(n);
  return s;
}

struct Scores {
  Tensor logprob, entropy, top_logprob, top_index, stat;
};

Scores score_forward(const Tensor& logits, const OptTensor& targets, double scale, int64_t top, int64_t ignore) {
  const char* const what = "token_logprobs";
  not_traced(what);
  check_logits(logits, what);
  check_scale(scale, what);
  const at::IntArrayRef lead = lead_of(logits);
  const int64_t V = logits.size(-1), N = logits.numel() / V;
  if (top < 0 || top > DET_HEAD_TOP_MAX || top > V)
    refuse(what, ": top must lie in 0..min(", DET_HEAD_TOP_MAX, ", V) (got ", top, ")");
  if (targets) check_index(*targets, lead, logits, "targets", what);
  on_gpu(logits, what, "logits");
  const c10::DeviceGuard guard(logits.device());
  const Tensor z = rows(logits);
  const Tensor t = targets ? targets->reshape({N}) : Tensor();
  const auto f32 = logits.options().dtype(at::kFloat);
  Scores r;
  if (targets) r.logprob = at::empty(lead, f32);
  r.entropy = at::empty(lead, f32);
  r.stat = at::empty({N, 4}, f32);
  r.top_logprob = at::empty(with_last(lead, top), f32);
  r.top_index = at::empty(with_last(lead, top), logits.options().dtype(at::kLong));
  const int64_t bytes = det_head_workspace_bytes(N, V, static_cast<int>(top));
  const Tensor ws = bytes > 0 ? at::empty({bytes}, logits.options().dtype(at::kByte)) : Tensor();
  ok(det_token_logprobs(dt_of(z.scalar_type()), in(z), z.stride(0), N, V, scale, out<int64_t>(t),
                        targets ? t.stride(0) : 0, ignore, static_cast<int>(top), out<float>(r.logprob),
                        out<float>(r.entropy), out<float>(r.stat), out<int64_t>(r.top_index),
                        out<float>(r.top_logprob), out<void>(ws), static_cast<size_t>(bytes), stream_of(logits)));
  return r;
}

Tensor score_backward(const Tensor& logits, const OptTensor& targets, const Tensor& stat, double scale,
                      int64_t ignore, const OptTensor& top_index, const OptTensor& g_logprob,
                      const OptTensor& g_entropy, const OptTensor& g_top) {
  const char* const what = "token_logprobs_backward";
  not_traced(what);
  check_logits(logits, what);
  check_scale(scale, what);
  const at::IntArrayRef lead = lead_of(logits);
  const int64_t V = logits.size(-1), N = logits.numel() / V;
  if (targets) check_index(*targets, lead, logits, "targets", what);
  else if (g_logprob) refuse(what, ": a gradient of the log probability needs the targets");
  check_stat(stat, N, logits, what);
  int64_t top = 0;
  if (g_top) {
    if (!top_index) refuse(what, ": a gradient of the alternatives needs top_index");
    top = top_index->dim() > 0 ? top_index->size(-1) : 0;
    check_index(*top_index, with_last(lead, top), logits, "top_index", what);
    if (g_top->sizes() != top_index->sizes() || g_top->scalar_type() != at::kFloat ||
        g_top->device() != logits.device())
      refuse(what, ": g_top must be float32 of top_index's shape on the logits' device");
  }
  on_gpu(logits, what, "logits");
  const c10::DeviceGuard guard(logits.device());
  const auto [glp, s_glp] = grad_rows(g_logprob.value_or(Tensor()), lead, logits, what);
  const auto [gent, s_gent] = grad_rows(g_entropy.value_or(Tensor()), lead, logits, what);
  const Tensor z = rows(logits), st = stat.contiguous();
  const Tensor t = targets ? targets->reshape({N}) : Tensor();
  Tensor gt, ti;
  if (top > 0) {
    gt = g_top->reshape({N, top});
    ti = top_index->reshape({N, top}).contiguous();
  }
  Tensor dz = at::empty(logits.sizes(), logits.options());
  ok(det_token_logprobs_grad(dt_of(z.scalar_type()), in(z), z.stride(0), N, V, scale, out<int64_t>(t),
                             targets ? t.stride(0) : 0, ignore, static_cast<int>(top), out<int64_t>(ti),
                             out<float>(st), out<float>(glp), s_glp, out<float>(gent), s_gent, out<float>(gt),
                             top > 0 ? gt.stride(0) : 0, top > 0 ? gt.stride(1) : 0, out<void>(dz), V,
                             stream_of(logits)));
  return dz;
}

struct ScoreFn : torch::autograd::Function<ScoreFn> {
  static variable_list forward(AutogradContext* ctx, const Tensor& logits, const OptTensor& targets, double scale,
                               int64_t top, int64_t ignore) {
    Scores r = score_forward(logits, targets, scale, top, ignore);
    ctx->save_for_backward({logits, targets.value_or(Tensor()), r.stat, top > 0 ? r.top_index : Tensor()});
    ctx->saved_data["scale"] = scale;
    ctx->saved_data["ignore"] = ignore;
    ctx->set_materialize_grads(false);
    ctx->mark_non_differentiable({r.top_index});
    variable_list outs = {r.entropy, r.top_logprob, r.top_index};
    if (targets) outs.push_back(r.logprob);
    return outs;
  }
  static variable_list backward(AutogradContext* ctx, variable_list grads) {
    for (const Tensor& g : grads) no_tangent(g, "token_logprobs");
    const auto saved = ctx->get_saved_variables();
    auto opt = [](const Tensor& t) { return t.defined() ? OptTensor(t) : std::nullopt; };
    Tensor dz;
    const OptTensor ti = opt(saved[3]), gtop = ti ? opt(grads[1]) : std::nullopt;
    const OptTensor gent = opt(grads[0]), glp = grads.size() > 3 ? opt(grads[3]) : std::nullopt;
    if (glp || gent || gtop) {
      const at::NoGradGuard no_grad;
      dz = score_backward(saved[0], opt(saved[1]), saved[2], ctx->saved_data["scale"].toDouble(),
                          ctx->saved_data["ignore"].toInt(), ti, glp, gent, gtop);
    }
    variable_list sources = grads;
    sources.push_back(saved[0]);
    variable_list r = once({dz}, sources, "token_logprobs");
    r.resize(5);
    return r;
  }
};

using ScoreTuple = std::tuple<OptTensor, Tensor, Tensor, Tensor>;

ScoreTuple token_logprobs(const Tensor& logits, const OptTensor& targets, double scale, int64_t top, int64_t ignore) {
  no_tangent(logits, "token_logprobs");
  auto opt = [](const Tensor& t) { return t.defined() ? OptTensor(t) : std::nullopt; };
  if (at::GradMode::is_enabled() && wants_grad(logits)) {
    const variable_list r = ScoreFn::apply(logits, targets, scale, top, ignore);
    return {r.size() > 3 ? opt(r[3]) : std::nullopt, r[0], r[1], r[2]};
  }
  const Scores r = score_forward(logits, targets, scale, top, ignore);
  return {opt(r.logprob), r.entropy, r.top_logprob, r.top_index};
}

// ---------------------------------------------------------------- distillation

void check_teacher(const Tensor& z, const Tensor& teacher, const Tensor& index, const char* what) {
  if (!known(teacher.scalar_type()) || teacher.device() != z.device())
    refuse(what, ": teacher logits must be float32 or bfloat16 on the logits' device");
  if (teacher.dim() != z.dim() || lead_of(teacher) != lead_of(z) || teacher.size(-1) < 1 ||
      teacher.size(-1) > DET_HEAD_ENTRIES_MAX)
    refuse(what, ": teacher logits must be [..., K] with the logits' leading shape and 1 <= K <= ", DET_HEAD_ENTRIES_MAX,
           " (got ", teacher.sizes(), ")");
  check_index(index, teacher.sizes(), z, "the teacher's indices", what);
}

struct Distilled {
  Tensor loss, stat, q;
};

Distilled distill_forward(const Tensor& logits, const Tensor& teacher, const Tensor& index, double T) {
  const char* const what = "distill_loss";
  not_traced(what);
  check_logits(logits, what);
  check_temperature(T, what);
  check_teacher(logits, teacher, index, what);
  on_gpu(logits, what, "logits");
  const c10::DeviceGuard guard(logits.device());
  const Tensor z = rows(logits), t = rows(teacher), i = rows(index);
  const int64_t N = z.size(0), V = z.size(1), K = t.size(1);
  const auto f32 = logits.options().dtype(at::kFloat);
  Distilled r{at::empty(lead_of(logits), f32), at::empty({N, 4}, f32), at::empty({N, K}, f32)};
  const int64_t bytes = det_head_workspace_bytes(N, V, 0);
  const Tensor ws = bytes > 0 ? at::empty({bytes}, logits.options().dtype(at::kByte)) : Tensor();
  ok(det_distill(dt_of(z.scalar_type()), in(z), z.stride(0), N, V, T, dt_of(t.scalar_type()), in(t), t.stride(0),
                 static_cast<const int64_t*>(in(i)), i.stride(0), K, out<float>(r.loss), out<float>(r.stat),
                 out<float>(r.q), out<void>(ws), static_cast<size_t>(bytes), stream_of(logits)));
  return r;
}

Tensor distill_backward(const Tensor& logits, const Tensor& index, const Tensor& stat, const Tensor& q,
                        const Tensor& g, double T) {
  const char* const what = "distill_backward";
  not_traced(what);
  check_logits(logits, what);
  check_temperature(T, what);
  const int64_t V = logits.size(-1), N = logits.numel() / V;
  check_stat(stat, N, logits, what);
  if (q.dim() != 2 || q.size(0) != N || q.size(1) < 1 || q.size(1) > DET_HEAD_ENTRIES_MAX || q.scalar_type() != at::kFloat ||
      q.device() != logits.device())
    refuse(what, ": q must be float32 [", N, ", K] with 1 <= K <= ", DET_HEAD_ENTRIES_MAX, " on the logits' device");
  const int64_t K = q.size(1);
  check_index(index, with_last(lead_of(logits), K), logits, "the teacher's indices", what);
  on_gpu(logits, what, "logits");
  const c10::DeviceGuard guard(logits.device());
  const auto [gv, s_g] = grad_rows(g, lead_of(logits), logits, what);
  const Tensor z = rows(logits), i = rows(index), st = stat.contiguous(), qc = q.contiguous();
  Tensor dz = at::empty(logits.sizes(), logits.options());
  ok(det_distill_grad(dt_of(z.scalar_type()), in(z), z.stride(0), N, V, T, static_cast<const int64_t*>(in(i)),
                      i.stride(0), K, static_cast<const float*>(in(st)), static_cast<const float*>(in(qc)),
                      static_cast<const float*>(in(gv)), s_g, out<void>(dz), V, stream_of(logits)));
  return dz;
}

struct DistillFn : torch::autograd::Function<DistillFn> {
  static Tensor forward(AutogradContext* ctx, const Tensor& logits, const Tensor& teacher, const Tensor& index,
                        double T) {
    Distilled r = distill_forward(logits, teacher, index, T);
    ctx->save_for_backward({logits, index, r.stat, r.q});
    ctx->saved_data["T"] = T;
    return r.loss;
  }
  static variable_list backward(AutogradContext* ctx, variable_list grads) {
    no_tangent(grads[0], "distill_loss");
    const auto saved = ctx->get_saved_variables();
    Tensor dz;
    {
      const at::NoGradGuard no_grad;
      dz = distill_backward(saved[0], saved[1], saved[2], saved[3], grads[0], ctx->saved_data["T"].toDouble());
    }
    variable_list r = once({dz}, {saved[0], grads[0]}, "distill_loss");
    r.resize(4);
    return r;
  }
};

Tensor distill_loss(const Tensor& logits, const Tensor& teacher, const Tensor& index, double T) {
  no_tangent(logits, "distill_loss");
  if (at::GradMode::is_enabled() && wants_grad(logits)) return DistillFn::apply(logits, teacher.detach(), index, T);
  return distill_forward(logits, teacher, index, T).loss;
}

OptTensor opt(const Tensor& t) { return t.defined() ? OptTensor(t) : std::nullopt; }

}  // namespace

PYBIND11_MODULE(_ops, m) {
  g_hip_error = py::object(py::module_::import("bitwise_deterministic_exact_amd._lib").attr("DetGemmError")).release().ptr();
  py::register_exception_translator([](std::exception_ptr p) {
    try {
      if (p) std::rethrow_exception(p);
    } catch (const HipFailure& e) {
      PyErr_SetString(g_hip_error, e.what());
    }
  });
  using release = py::call_guard<py::gil_scoped_release>;
  m.def("not_traced", &not_traced);
  m.def("layer_norm", &layer_norm, release());
  m.def("layer_norm_forward", [](const Tensor& x, const OptTensor& w, const OptTensor& b, double eps,
                                 std::optional<ScalarType> dt) { return norm_forward(x, w, b, eps, dt, true); },
        release());
  m.def("layer_norm_backward",
        [](const Tensor& dy, const Tensor& x, const OptTensor& w, const Tensor& mean, const Tensor& rstd, bool need_dx,
           bool need_dw, bool need_db, std::optional<ScalarType> gt, bool digits) {
          const NormGrads g = norm_backward(dy, x, w, mean, rstd, need_dx, need_dw, need_db, gt, digits);
          return std::make_tuple(opt(g.dx), opt(g.dw), opt(g.db), opt(g.digits));
        }, release());
  m.def("token_logprobs", &token_logprobs, release());
  m.def("token_logprobs_forward", [](const Tensor& z, const OptTensor& t, double scale, int64_t top, int64_t ignore) {
    const Scores r = score_forward(z, t, scale, top, ignore);
    return std::make_tuple(opt(r.logprob), r.entropy, r.top_logprob, r.top_index, r.stat);
  }, release());
  m.def("token_logprobs_backward", &score_backward, release());
  m.def("distill_loss", &distill_loss, release());
  m.def("distill_forward", [](const Tensor& z, const Tensor& t, const Tensor& i, double T) {
    const Distilled r = distill_forward(z, t, i, T);
    return std::make_tuple(r.loss, r.stat, r.q);
  }, release());
  m.def("distill_backward", &distill_backward, release());
}
