// The torch side of the gated projection and the 8-bit checkpoints: argument
// checks, outputs, workspaces, the current stream, and the autograd function,
// over the C entry points of libdetgemm.so (include/detgemm.h).
#include "ops_common.h"

void bind_block(py::module_& m);

namespace {

// ---------------------------------------------------------------- gated projection

det_activation act_of(const std::string& name, const char* what) {
  if (name == "silu") return DET_ACT_SILU;
  if (name == "gelu") return DET_ACT_GELU;
  if (name == "gelu_tanh") return DET_ACT_GELU_TANH;
  refuse(what, ": activation must be \"silu\", \"gelu\" or \"gelu_tanh\" (got \"", name, "\")");
}

det_save save_of(const std::optional<std::string>& name, const char* what) {
  if (!name) return DET_SAVE_HALF;
  if (*name == "int8") return DET_SAVE_INT8;
  refuse(what, ": checkpoint must be None or \"int8\" (got \"", *name, "\")");
}

void check_gated(at::IntArrayRef x, ScalarType xt, const Tensor& like, const Tensor& wg, const Tensor& wu,
                 const char* what) {
  if (xt != at::kBFloat16) refuse(what, ": x must be bfloat16 (got ", xt, ")");
  if (x.empty() || x.back() < 1) refuse(what, ": x needs a last dimension of at least 1 (got shape ", x, ")");
  const int64_t C = x.back();
  for (const auto& [w, name] : {std::pair{&wg, "w_gate"}, std::pair{&wu, "w_up"}})
    if (w->scalar_type() != at::kBFloat16 || w->dim() != 2 || w->size(0) < 1 || w->size(1) != C ||
        w->device() != like.device())
      refuse(what, ": ", name, " must be bfloat16 of shape [F, ", C, "] on x's device (got ", w->scalar_type(), " ",
             w->sizes(), ")");
  if (wg.size(0) != wu.size(0)) refuse(what, ": w_gate and w_up must have one shape");
  if (C > DET_GATED_MAX || wg.size(0) > DET_GATED_MAX)
    refuse(what, ": widths of ", C, " and ", wg.size(0), " exceed the limit ", DET_GATED_MAX);
  if (c10::multiply_integers(x) / C > DET_ROWS_MAX) refuse(what, ": more than 2^22 rows in one call");
}

// whether the matrix product can copy rows 16 bytes at a time as they lie
bool wide(const Tensor& r) {
  return reinterpret_cast<uintptr_t>(r.const_data_ptr()) % 16 == 0 && r.stride(0) % 8 == 0 &&
         r.stride(0) >= r.size(1) && r.stride(0) <= (int64_t{1} << 21);
}
// other layouts of a width that is a multiple of 64 (narrow slices, odd offsets)
// are copied here, other widths padded by the library
Tensor wide_rows(const Tensor& t) {
  const Tensor r = rows(t);
  return r.size(1) % 64 != 0 || r.size(0) == 0 || wide(r) ? r : r.clone(at::MemoryFormat::Contiguous);
}

// what a forward call keeps of both projections: fp16 elements or int8 codes
// [.., F], and the exponents of their blocks
struct Saved {
  Tensor gate, up, gate_exp, up_exp;
};

Tensor gated_forward(const Tensor& x, const Tensor& wg, const Tensor& wu, det_activation act,
                     std::optional<ScalarType> out_dtype, det_save save, Saved& kept) {
  const char* const what = "gated_linear";
  not_traced(what);
  check_gated(x.sizes(), x.scalar_type(), x, wg, wu, what);
  const ScalarType ht = out_dtype.value_or(x.scalar_type());
  if (!known(ht)) refuse(what, ": out_dtype must be float32 or bfloat16 (got ", ht, ")");
  on_gpu(x, what, "x");
  const c10::DeviceGuard guard(x.device());
  Tensor x2 = rows(x), g2 = rows(wg), u2 = rows(wu);
  const int64_t N = x2.size(0), C = x2.size(1), F = wg.size(0);
  // few tokens of which nothing is kept read the weights at any alignment, and
  // copying these would move their bytes three times; x alone is little
  if (!(save == DET_SAVE_NONE && (N <= 16 || (N <= 64 && !(wide(g2) && wide(u2)))))) {
    x2 = wide_rows(x2);
    g2 = wide_rows(g2);
    u2 = wide_rows(u2);
  }
  const std::vector<int64_t> shape = with_last(lead_of(x), F), blocks = with_last(lead_of(x), (F + 31) / 32);
  Tensor h = at::empty(shape, x.options().dtype(ht));
  if (save != DET_SAVE_NONE) {
    const auto o = x.options().dtype(save == DET_SAVE_INT8 ? at::kChar : at::kHalf), e = x.options().dtype(at::kChar);
    // rows of a multiple of 32, so that every row is written and read in aligned words
    const int64_t Fs = (F + 31) / 32 * 32;
    kept.gate = at::empty(with_last(lead_of(x), Fs), o);
    kept.up = at::empty(with_last(lead_of(x), Fs), o);
    if (Fs != F) {
      kept.gate = kept.gate.narrow(-1, 0, F);
      kept.up = kept.up.narrow(-1, 0, F);
    }
    kept.gate_exp = at::empty(blocks, e);
    kept.up_exp = at::empty(blocks, e);
  }
  const int64_t bytes = det_gated_linear_workspace_bytes(N, C, F, save, C % 64 == 0);
  const Tensor ws = bytes > 0 ? at::empty({bytes}, x.options().dtype(at::kByte)) : Tensor();
  ok(det_gated_linear(in(x2), x2.stride(0), in(g2), g2.stride(0), in(u2), u2.stride(0), N, C, F, act,
                      dt_of(ht), out<void>(h), save, out<void>(kept.gate), out<void>(kept.up), (F + 31) / 32 * 32,
                      out<int8_t>(kept.gate_exp), out<int8_t>(kept.up_exp), out<void>(ws),
                      static_cast<size_t>(bytes), stream_of(x)));
  return h;
}

struct GatedGrads {
  Tensor dx, dwg, dwu;
};

// x: bfloat16 with no exponents, or its codes with them; undefined where the
// weights' gradients are not needed
GatedGrads gated_backward(const Tensor& dh, const Tensor& x, const OptTensor& x_exp, const Tensor& wg,
                          const Tensor& wu, const Saved& kept, det_activation act, bool need_dx, bool need_dw) {
  const char* const what = "gated_linear_backward";
  not_traced(what);
  if (kept.gate.dim() < 1 || wg.dim() != 2) refuse(what, ": gate must be [..., F], w_gate [F, C]");
  const at::IntArrayRef lead = lead_of(kept.gate);
  const int64_t C = wg.size(1), F = wg.size(0);
  const std::vector<int64_t> xs = with_last(lead, C), hs = with_last(lead, F), blocks = with_last(lead, (F + 31) / 32);
  check_gated(xs, x.defined() && !x_exp ? x.scalar_type() : at::kBFloat16, wg, wg, wu, what);
  auto has = [&](const Tensor& t, ScalarType type, const std::vector<int64_t>& shape) {
    return t.scalar_type() == type && t.sizes() == at::IntArrayRef(shape) && t.device() == wg.device();
  };
  if (!has(dh, dh.scalar_type(), hs) || !known(dh.scalar_type()))
    refuse(what, ": dh must be float32 or bfloat16 of shape ", hs, " on the weights' device");
  const bool int8 = kept.gate.scalar_type() == at::kChar;
  for (const Tensor* t : {&kept.gate, &kept.up})
    if (!has(*t, int8 ? at::kChar : at::kHalf, hs))
      refuse(what, ": gate and up must be as gated_linear_forward gives them");
  for (const Tensor* t : {&kept.gate_exp, &kept.up_exp})
    if (!has(*t, at::kChar, blocks)) refuse(what, ": gate and up must be as gated_linear_forward gives them");
  if (x_exp && (!has(x, at::kChar, xs) || !has(*x_exp, at::kChar, with_last(lead, (C + 31) / 32))))
    refuse(what, ": a packed x needs int8 codes of shape ", xs, " and one int8 exponent for each 32 of them");
  if (!x_exp && x.defined() && !has(x, at::kBFloat16, xs))
    refuse(what, ": x must be of shape ", xs, " on the weights' device");
  if (need_dw && !x.defined()) refuse(what, ": the weights' gradients need x");
  on_gpu(wg, what, "w_gate");
  const c10::DeviceGuard guard(wg.device());
  GatedGrads g;
  const auto bf16 = wg.options().dtype(at::kBFloat16);
  if (need_dx) g.dx = at::empty(xs, bf16);
  if (need_dw) {
    g.dwg = at::empty(wg.sizes(), bf16);
    g.dwu = at::empty(wu.sizes(), bf16);
  }
  const Tensor dh2 = rows(dh), x2 = !need_dw ? Tensor() : x_exp ? x.contiguous() : wide_rows(x);
  const Tensor xe = need_dw && x_exp ? x_exp->contiguous() : Tensor();
  const Tensor ge = kept.gate_exp.contiguous(), ue = kept.up_exp.contiguous();
  Tensor g2 = wg, u2 = wu, kg = rows(kept.gate), ku = rows(kept.up);
  if (need_dx) {                          // nothing else reads the weights
    g2 = wide_rows(wg);
    u2 = wide_rows(wu);
    if (g2.stride(0) != u2.stride(0)) {   // dx runs over both with one stride
      g2 = g2.clone(at::MemoryFormat::Contiguous);            // contiguous() would keep a single row's stride
      u2 = u2.clone(at::MemoryFormat::Contiguous);
    }
  }
  if (kg.stride(0) != ku.stride(0)) {
    kg = kg.contiguous();
    ku = ku.contiguous();
  }
  auto bytes_of = [](const Tensor& t) { return t.defined() ? static_cast<const int8_t*>(t.const_data_ptr()) : nullptr; };
  const int64_t N = kg.size(0);
  const int64_t bytes = det_gated_linear_grad_workspace_bytes(N, C, F, need_dx, need_dw, C % 64 == 0, xe.defined());
  const Tensor ws = bytes > 0 ? at::empty({bytes}, wg.options().dtype(at::kByte)) : Tensor();
  ok(det_gated_linear_grad(dt_of(dh.scalar_type()), in(dh2), dh2.stride(0), bytes_of(x2),
                           xe.defined() || !x2.defined() ? C : x2.stride(0), bytes_of(xe), in(g2), g2.stride(0), in(u2),
                           u2.stride(0), int8 ? DET_SAVE_INT8 : DET_SAVE_HALF, in(kg), in(ku), kg.stride(0), bytes_of(ge),
                           bytes_of(ue), N, C, F, act, out<void>(g.dx), out<void>(g.dwg), out<void>(g.dwu), out<void>(ws),
                           static_cast<size_t>(bytes), stream_of(wg)));
  return g;
}

// ---------------------------------------------------------------- 8-bit checkpoints

std::tuple<Tensor, Tensor> pack_int8(const Tensor& x) {
  const char* const what = "pack_int8";
  not_traced(what);
  if (!known(x.scalar_type())) refuse(what, ": x must be float32 or bfloat16 (got ", x.scalar_type(), ")");
  if (x.dim() < 1 || x.size(-1) < 1 || x.size(-1) > (int64_t{1} << 24))
    refuse(what, ": x must be [..., C] with 1 <= C <= 2^24 (got shape ", x.sizes(), ")");
  on_gpu(x, what, "x");
  const c10::DeviceGuard guard(x.device());
  const Tensor x2 = rows(x);
  const int64_t N = x2.size(0), C = x2.size(1);
  const auto o = x.options().dtype(at::kChar);
  Tensor codes = at::empty(x.sizes(), o), exps = at::empty(with_last(lead_of(x), (C + 31) / 32), o);
  ok(det_int8_pack(dt_of(x.scalar_type()), in(x2), x2.stride(0), N, C, out<int8_t>(codes), out<int8_t>(exps),
                   stream_of(x)));
  return {codes, exps};
}

Tensor unpack_int8(const Tensor& codes, const Tensor& exps, ScalarType dtype) {
  const char* const what = "unpack_int8";
  not_traced(what);
  if (!known(dtype)) refuse(what, ": dtype must be float32 or bfloat16 (got ", dtype, ")");
  if (codes.scalar_type() != at::kChar || exps.scalar_type() != at::kChar || codes.device() != exps.device())
    refuse(what, ": codes and exponents must be int8 on one device");
  if (codes.dim() < 1 || codes.size(-1) < 1 || codes.size(-1) > (int64_t{1} << 24))
    refuse(what, ": codes must be [..., C] with 1 <= C <= 2^24 (got shape ", codes.sizes(), ")");
  if (exps.sizes() != at::IntArrayRef(with_last(lead_of(codes), (codes.size(-1) + 31) / 32)))
    refuse(what, ": one exponent for each 32 codes of a row is needed (got shapes ", codes.sizes(), " and ",
           exps.sizes(), ")");
  on_gpu(codes, what, "codes");
  const c10::DeviceGuard guard(codes.device());
  const Tensor c2 = rows(codes), e = exps.contiguous();
  Tensor y = at::empty(codes.sizes(), codes.options().dtype(dtype));
  ok(det_int8_unpack(static_cast<const int8_t*>(in(c2)), c2.stride(0), static_cast<const int8_t*>(in(e)), c2.size(0),
                     c2.size(1), dt_of(dtype), out<void>(y), stream_of(codes)));
  return y;
}

// ---------------------------------------------------------------- autograd

struct GatedFn : torch::autograd::Function<GatedFn> {
  static Tensor forward(AutogradContext* ctx, const Tensor& x, const Tensor& wg, const Tensor& wu, int64_t act,
                        std::optional<ScalarType> out_dtype, int64_t save) {
    Saved kept;
    Tensor h = gated_forward(x, wg, wu, static_cast<det_activation>(act), out_dtype, static_cast<det_save>(save), kept);
    // x enters the weights' gradients only
    Tensor kx, xe;
    if (wants_grad(wg) || wants_grad(wu)) {
      if (save == DET_SAVE_INT8) std::tie(kx, xe) = pack_int8(x);
      else kx = x;
    }
    ctx->save_for_backward({kx, xe, wg, wu, kept.gate, kept.up, kept.gate_exp, kept.up_exp});
    ctx->saved_data["act"] = act;
    return h;
  }
  static variable_list backward(AutogradContext* ctx, variable_list grads) {
    no_tangent(grads[0], "gated_linear");
    const auto s = ctx->get_saved_variables();
    GatedGrads g;
    {
      const at::NoGradGuard no_grad;
      g = gated_backward(grads[0], s[0], opt(s[1]), s[2], s[3], {s[4], s[5], s[6], s[7]},
                         static_cast<det_activation>(ctx->saved_data["act"].toInt()), ctx->needs_input_grad(0),
                         ctx->needs_input_grad(1) || ctx->needs_input_grad(2));
    }
    variable_list r = once_at_node({g.dx, ctx->needs_input_grad(1) ? g.dwg : Tensor(),
                                    ctx->needs_input_grad(2) ? g.dwu : Tensor()},
                                   grads, "gated_linear");
    r.resize(6);
    return r;
  }
};

Tensor gated_linear(const Tensor& x, const Tensor& wg, const Tensor& wu, const std::string& activation,
                    std::optional<ScalarType> out_dtype, const std::optional<std::string>& checkpoint) {
  for (const Tensor* t : {&x, &wg, &wu}) no_tangent(*t, "gated_linear");
  const det_activation act = act_of(activation, "gated_linear");
  const det_save save = save_of(checkpoint, "gated_linear");
  if (at::GradMode::is_enabled() && (wants_grad(x) || wants_grad(wg) || wants_grad(wu)))
    return GatedFn::apply(x, wg, wu, static_cast<int64_t>(act), out_dtype, static_cast<int64_t>(save));
  Saved none;
  return gated_forward(x, wg, wu, act, out_dtype, DET_SAVE_NONE, none);
}

}  // namespace

void bind_block(py::module_& m) {
  using release = py::call_guard<py::gil_scoped_release>;
  m.def("gated_linear", &gated_linear, release());
  m.def("gated_linear_forward",
        [](const Tensor& x, const Tensor& wg, const Tensor& wu, const std::string& activation,
           std::optional<ScalarType> dt, const std::optional<std::string>& checkpoint) {
          Saved k;
          const Tensor h = gated_forward(x, wg, wu, act_of(activation, "gated_linear"), dt,
                                         save_of(checkpoint, "gated_linear"), k);
          return std::make_tuple(h, k.gate, k.up, k.gate_exp, k.up_exp);
        }, release());
  m.def("gated_linear_backward",
        [](const Tensor& dh, const OptTensor& x, const OptTensor& x_exp, const Tensor& wg, const Tensor& wu,
           const Tensor& gate, const Tensor& up, const Tensor& gate_exp, const Tensor& up_exp,
           const std::string& activation, bool need_dx, bool need_dw) {
          const GatedGrads g = gated_backward(dh, x.value_or(Tensor()), x_exp, wg, wu, {gate, up, gate_exp, up_exp},
                                              act_of(activation, "gated_linear_backward"), need_dx, need_dw);
          return std::make_tuple(opt(g.dx), opt(g.dwg), opt(g.dwu));
        }, release());
  m.def("pack_int8", &pack_int8, release());
  m.def("unpack_int8", &unpack_int8, release());
}
