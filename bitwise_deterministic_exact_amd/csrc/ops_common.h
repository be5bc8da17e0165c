// What the torch sides of the operators share: argument checks, errors, the
// current stream, and the refusals of what autograd might ask beyond a first
// derivative.
#ifndef DETGEMM_OPS_COMMON_H
#define DETGEMM_OPS_COMMON_H

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

// a HIP failure inside the library; one type for all sources of the module
namespace detops {
struct HipFailure : std::runtime_error {
  using std::runtime_error::runtime_error;
};
}  // namespace detops

namespace {

// ---------------------------------------------------------------- checks

template <class... A>
[[noreturn]] void refuse(const A&... parts) {
  std::ostringstream s;
  (s << ... << parts);
  throw py::value_error(s.str());
}

inline bool known(ScalarType t) { return t == at::kFloat || t == at::kBFloat16; }
inline det_dtype dt_of(ScalarType t) { return t == at::kFloat ? DET_F32 : DET_BF16; }

inline void on_gpu(const Tensor& t, const char* what, const char* name) {
  if (!t.is_cuda()) refuse(what, ": ", name, " must be on a GPU");
}

inline void* stream_of(const Tensor& t) {
  return static_cast<void*>(c10::hip::getCurrentHIPStream(t.get_device()).stream());
}

// the library's status as the exceptions the rest of the package raises: bad
// arguments are ValueError, a HIP failure is DetGemmError
inline void ok(det_status st) {
  if (st == DET_OK) return;
  if (st == DET_EHIP) throw detops::HipFailure(det_last_error());
  throw py::value_error(det_last_error());
}

inline const void* in(const Tensor& t) { return t.const_data_ptr(); }
inline const void* in(const OptTensor& t) { return t ? t->const_data_ptr() : nullptr; }
template <class T>
T* out(const Tensor& t) { return t.defined() ? static_cast<T*>(t.mutable_data_ptr()) : nullptr; }

// [..., C] as [N, C] rows with adjacent elements: a copy only when one stride
// cannot describe the rows, or a row's elements are apart
inline Tensor rows(const Tensor& t) {
  Tensor r = t.dim() == 2 ? t : t.reshape({t.numel() / t.size(-1), t.size(-1)});
  return r.size(1) <= 1 || r.stride(1) == 1 ? r : r.contiguous();
}

// Gradients of gradients are not formed.  A backward pass that is itself
// recorded (create_graph) gives gradients whose node refuses to run; it has
// edges to everything they depend on, the saved inputs and the incoming
// gradients, so that a derivative through any of these reaches it, also where
// it is asked for one input alone.  Torch's own DelayedError hangs on the
// results only: grad(loss + g.pow(2).sum(), x) would leave it out and return
// the first-order terms.
inline variable_list refuse_more(variable_list grads, torch::autograd::edge_list&& edges, const char* name) {
  const auto refusal = std::make_shared<torch::autograd::Error>(std::string(name) + " is differentiable once",
                                                                std::move(edges));
  for (auto& g : grads)
    if (g.defined()) torch::autograd::set_history(g, refusal);
  return grads;
}
inline variable_list once(variable_list grads, const variable_list& sources, const char* name) {
  if (!at::GradMode::is_enabled()) return grads;
  return refuse_more(std::move(grads), torch::autograd::collect_next_edges(at::ArrayRef<Tensor>(sources)), name);
}
// the same for a backward pass that does not keep its inputs: their edges are
// those of the node that is running
inline variable_list once_at_node(variable_list grads, const variable_list& incoming, const char* name) {
  if (!at::GradMode::is_enabled()) return grads;
  torch::autograd::edge_list edges = torch::autograd::collect_next_edges(at::ArrayRef<Tensor>(incoming));
  if (const auto node = torch::autograd::get_current_node())
    for (const auto& e : node->next_edges())
      if (e.is_valid()) edges.push_back(e);
  return refuse_more(std::move(grads), std::move(edges), name);
}

// A trace (torch.jit.trace, make_fx) sees the allocations of the results but
// not what fills them: the traced function would return whatever lies there.
// So a call that is being traced is refused.
inline void not_traced(const char* what) {
  using c10::impl::TorchDispatchModeKey;
  if (torch::jit::tracer::isTracing() || c10::impl::TorchDispatchModeTLS::get_mode(TorchDispatchModeKey::PROXY) ||
      c10::impl::tls_is_dispatch_key_included(c10::DispatchKey::PreDispatch))
    throw std::runtime_error(std::string(what) + " cannot be traced: its kernels are not torch operators");
}

// Forward-mode derivatives are not formed: a result without its tangent would pass
// for a constant, so inputs and incoming gradients that carry one are refused.
inline void no_tangent(const OptTensor& t, const char* what) {
  if (t && t->defined() && t->_fw_grad(0).defined() && c10::AutogradState::get_tls_state().get_fw_grad_mode())
    throw std::runtime_error(std::string(what) + " forms no forward-mode derivatives");
}

inline bool wants_grad(const Tensor& t) { return t.defined() && t.requires_grad(); }
inline bool wants_grad(const OptTensor& t) { return t && t->requires_grad(); }

inline OptTensor opt(const Tensor& t) { return t.defined() ? OptTensor(t) : std::nullopt; }
inline at::IntArrayRef lead_of(const Tensor& t) { return t.sizes().slice(0, t.dim() - 1); }
inline std::vector<int64_t> with_last(at::IntArrayRef lead, int64_t n) {
  std::vector<int64_t> s(lead.begin(), lead.end());
  s.push_back(n);
  return s;
}

}  // namespace

#endif  // DETGEMM_OPS_COMMON_H
